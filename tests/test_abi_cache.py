"""The 8-bit paged cache's entry points without a GPU: invalid arguments are
refused on the host, before any launch."""
import ctypes

import pytest

from sliding_window_learned_b200 import abi

E4, E8, I32, F32 = abi.ATTN_DTYPE_E4M3, abi.ATTN_DTYPE_E8M0, abi.ATTN_DTYPE_I32, abi.ATTN_DTYPE_F32


@pytest.fixture(scope="module")
def lib():
    from sliding_window_learned_b200 import build
    build.build()
    return abi.load()


def _t(shape, dtype=abi.ATTN_DTYPE_BF16, ptr=0x10000, strides=None):
    d = abi.AttnTensor()
    d.data, d.dtype, d.ndim = ptr, dtype, len(shape)
    acc = 1
    for i in reversed(range(len(shape))):
        d.shape[i] = shape[i]
        d.stride[i] = acc if strides is None else strides[i]
        acc *= shape[i]
    return d


def _good(NB=40, P=64, Hkv=2, D=128, B=3, MP=8, T=20, G=4):
    return dict(q=_t([B, Hkv * G, D]), out=_t([B, Hkv * G, D]), sinks=_t([Hkv * G], F32),
                k=_t([T, Hkv, D]), v=_t([T, Hkv, D]), cu=_t([B + 1], I32), table=_t([B, MP], I32),
                sl=_t([B], I32), kp=_t([NB, P, Hkv, D], E4), vp=_t([NB, P, Hkv, D], E4),
                ks=_t([NB, Hkv, P], E8), vs=_t([NB, Hkv, P], E8), W=100, scale=0.1)


ORDER = {"append": ("k", "v", "table", "sl", "cu", "kp", "vp", "ks", "vs"),
         "read": ("kp", "vp", "ks", "vs", "table", "sl", "cu", "k", "v"),
         "decode": ("q", "kp", "vp", "ks", "vs", "table", "sl", "sinks", "W", "scale", "out")}
NAMES = {"append": "attn_sink_cache_append_fp8", "read": "attn_sink_cache_read_fp8",
         "decode": "attn_sink_decode_paged_fp8"}


def _call(lib, op, a):
    args = [ctypes.byref(a[n]) if isinstance(a[n], abi.AttnTensor) else a[n] for n in ORDER[op]]
    return getattr(lib, NAMES[op])(*args, None)


POOL_FAULTS = {
    "kpages dtype": ("kp", _t([40, 64, 2, 128])),
    "vpages shape": ("vp", _t([41, 64, 2, 128], E4)),
    "kscales dtype": ("ks", _t([40, 2, 64], E4)),
    "kscales per position first": ("ks", _t([40, 64, 2], E8)),
    "vscales shape": ("vs", _t([40, 2, 32], E8)),
    "scale strides": ("ks", _t([40, 2, 64], E8, strides=[136, 68, 1])),
    "page strides": ("kp", _t([40, 64, 2, 128], E4, strides=[64 * 264, 264, 132, 1])),
    "inner stride": ("vp", _t([40, 64, 2, 128], E4, strides=[64 * 512, 512, 256, 2])),
    "misaligned pool": ("vp", _t([40, 64, 2, 128], E4, ptr=0x10008)),
    "null pool": ("kp", _t([40, 64, 2, 128], E4, ptr=0)),
    "table dtype": ("table", _t([3, 8], F32)),
    "table rows": ("table", _t([4, 8], I32)),
    "lengths dtype": ("sl", _t([3], F32)),
    "lengths stride": ("sl", _t([3], I32, strides=[2])),
}
ROW_FAULTS = {
    "k dtype": ("k", _t([20, 2, 128], F32)), "k heads": ("k", _t([20, 1, 128])), "v rows": ("v", _t([21, 2, 128])),
    "k row stride": ("k", _t([20, 2, 128], strides=[260, 128, 1])), "cu entries": ("cu", _t([3], I32)),
    "cu dtype": ("cu", _t([4], F32)), "cu stride": ("cu", _t([4], I32, strides=[3])),
}
DECODE_FAULTS = {
    "q dtype": ("q", _t([3, 8, 128], F32)), "q head dim": ("q", _t([3, 8, 64])), "q rows": ("q", _t([4, 8, 128])),
    "out shape": ("out", _t([3, 8, 64])), "sinks entries": ("sinks", _t([7], F32)), "window": ("W", 0),
    "scale": ("scale", float("nan")), "q stride": ("q", _t([3, 8, 128], strides=[8 * 129, 129, 1])),
}


@pytest.mark.parametrize("op", ["append", "read", "decode"])
@pytest.mark.parametrize("fault", POOL_FAULTS)
def test_pools_are_checked(lib, op, fault):
    a = _good()
    a[POOL_FAULTS[fault][0]] = POOL_FAULTS[fault][1]
    assert _call(lib, op, a) == abi.ATTN_EINVAL, abi.attn_sink_last_error()
    assert abi.attn_sink_last_error() != ""


@pytest.mark.parametrize("op", ["append", "read"])
@pytest.mark.parametrize("fault", ROW_FAULTS)
def test_rows_are_checked(lib, op, fault):
    a = _good()
    a[ROW_FAULTS[fault][0]] = ROW_FAULTS[fault][1]
    assert _call(lib, op, a) == abi.ATTN_EINVAL, abi.attn_sink_last_error()


@pytest.mark.parametrize("fault", DECODE_FAULTS)
def test_decode_arguments_are_checked(lib, fault):
    a = _good()
    a[DECODE_FAULTS[fault][0]] = DECODE_FAULTS[fault][1]
    assert _call(lib, "decode", a) == abi.ATTN_EINVAL, abi.attn_sink_last_error()


def test_heads_that_do_not_divide(lib):
    a = _good(Hkv=3, G=1)
    a["q"] = a["out"] = _t([3, 4, 128])
    a["sinks"] = _t([4], F32)
    assert _call(lib, "decode", a) == abi.ATTN_EINVAL


@pytest.mark.parametrize("sizes", [dict(D=96), dict(D=512), dict(P=8), dict(P=48), dict(P=1 << 17),
                                   dict(MP=1 << 25), dict(B=(1 << 20) + 1)])
@pytest.mark.parametrize("op", ["append", "read", "decode"])
def test_sizes_that_are_not_supported(lib, op, sizes):
    assert _call(lib, op, _good(**sizes)) == abi.ATTN_EUNSUPPORTED, abi.attn_sink_last_error()


@pytest.mark.parametrize("D,G", [(64, 17), (128, 17), (256, 9)])
def test_groups_that_are_not_supported(lib, D, G):
    assert _call(lib, "decode", _good(D=D, G=G)) == abi.ATTN_EUNSUPPORTED


@pytest.mark.parametrize("op", ["append", "read", "decode"])
def test_no_page_is_refused_and_no_work_is_not(lib, op):
    a = _good(NB=0)
    assert _call(lib, op, a) == abi.ATTN_EINVAL
    a = _good(B=0, T=0)
    assert _call(lib, op, a) == abi.ATTN_OK
    if op != "decode":
        assert _call(lib, op, _good(T=0)) == abi.ATTN_OK


def _extend(lib, **over):
    a = dict(q=_t([50, 8, 128]), k=_t([90, 2, 128]), v=_t([90, 2, 128]), cq=_t([4], I32), ck=_t([4], I32), mq=50,
             s=_t([8], F32), W=100, scale=0.1, out=_t([50, 8, 128]), lse=_t([8, 50], F32))
    a.update(over)
    r = lambda n: ctypes.byref(a[n]) if a[n] is not None else None  # noqa: E731
    return lib.attn_sink_fwd_extend(r("q"), r("k"), r("v"), r("cq"), r("ck"), a["mq"], r("s"), a["W"], a["scale"],
                                    r("out"), r("lse"), None)


@pytest.mark.parametrize("over", [
    dict(q=_t([50, 8, 128], F32)), dict(k=_t([90, 2, 64])), dict(v=_t([91, 2, 128])), dict(cq=_t([5], I32)),
    dict(ck=_t([4], F32)), dict(ck=_t([4], I32, strides=[2])), dict(cq=_t([0], I32), ck=_t([0], I32)), dict(mq=-1),
    dict(s=_t([7], F32)), dict(W=0), dict(scale=0.0), dict(out=_t([49, 8, 128])), dict(lse=_t([50, 8], F32)),
    dict(k=_t([90, 3, 128]), v=_t([90, 3, 128])), dict(k=_t([90, 2, 128], strides=[260, 128, 1])),
    dict(q=None), dict(out=_t([50, 8, 128], ptr=0x10008))])
def test_extend_arguments_are_checked(lib, over):
    assert _extend(lib, **over) == abi.ATTN_EINVAL, abi.attn_sink_last_error()


def test_extend_sizes(lib):
    bad = dict(q=_t([50, 8, 96]), k=_t([90, 2, 96]), v=_t([90, 2, 96]), out=_t([50, 8, 96]))
    assert _extend(lib, **bad) == abi.ATTN_EUNSUPPORTED
    long = dict(q=_t([1 << 30, 8, 128]), out=_t([1 << 30, 8, 128]), lse=None, mq=1 << 30, cq=_t([60001], I32),
                ck=_t([60001], I32))
    assert _extend(lib, **long) == abi.ATTN_EUNSUPPORTED
    assert _extend(lib, mq=0) == abi.ATTN_OK
    assert _extend(lib, cq=_t([1], I32), ck=_t([1], I32)) == abi.ATTN_OK
