"""The 8-bit paged cache on the GPU: append and read back bit for bit, decode
against the double-precision definition.

Decode's tolerance, for every output: half a bf16 step of the result, 2^-8 |o|,
and an error relative to A = sum_j p_j |v_j| / den from the terms themselves:
P in f16 (2^-11, and 2^-25 * 2^-7 of the largest term for each key below its
normal range), the fp32 scores of D products of magnitude at most S in all
(D * 2^-24 * S each in numerator and denominator), fp32 sums over n keys and
the exponentials' few 2^-22."""
import numpy as np
import pytest
import torch

import sliding_window_learned_b200 as swl
from oracle import cache8
from sliding_window_learned_b200 import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN_CODE, INF = 0x7F, float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sliding_window_learned_b200 import build
    build.build()


def _tol(o, mag, top, n, D):
    c = 2.0 ** -11 + 2 * D * 2.0 ** -24 * top + 2 * n * 2.0 ** -24 + n * 2.0 ** -32 + 2.0 ** -19
    return 2.0 ** -8 * np.abs(o) + c[..., None] * mag * 1.01 + 1e-37


def _dev(codes, kind):
    # (a fresh copy: numpy leaves odd strides on dimensions of size 1)
    return torch.empty(codes.shape, dtype=torch.uint8).copy_(torch.from_numpy(codes)).to(DEV).view(kind)


def _pools(kp, vp, ks, vs):
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    return _dev(kp, e4), _dev(vp, e4), _dev(ks, e8), _dev(vs, e8)


def _u8(t):
    return t.view(torch.uint8).cpu().numpy()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _rows(rng, T, H, D, spread=4):
    x = rng.standard_normal((T, H, D)) * 2.0 ** rng.integers(-spread, spread + 1, (T, H, 1))
    return torch.from_numpy(x).bfloat16()


def _random_pools(rng, NB, P, Hkv, D, spread=2):
    """Pools with every row quantised from normals; unused rows are overwritten by the caller."""
    outs = []
    for _ in range(2):
        c, s = cache8.quantise(inputs.bits(_rows(rng, NB * P, Hkv, D, spread)))
        outs += [c.reshape(NB, P, Hkv, D), np.ascontiguousarray(s.reshape(NB, P, Hkv).transpose(0, 2, 1))]
    return outs[0], outs[2], outs[1], outs[3]


# ----------------------------------------------------------- append and read
APPEND = [  # new rows, total positions, Hkv, D, P, MP
    ([1], [1], 1, 64, 16, 1),
    ([1, 1, 1], [5, 64, 65], 4, 128, 64, 2),
    ([0, 3, 0, 0, 200, 17], [4, 3, 0, 9, 777, 17], 3, 128, 16, 49),
    ([130, 1], [131, 1000], 5, 256, 32, 32),
    ([70, 65], [70, 300], 8, 64, 256, 2),
    ([1] * 300, [2] * 300, 1, 128, 16, 1),
    ([2] * 1100, [3] * 1100, 1, 64, 16, 1),           # more sequences than shared memory keeps
    ([33], [20], 2, 64, 16, 2),                       # more rows than positions: the first 13 have no place
]


def _append_case(seed, new, total, Hkv, D, P, MP, tail=3):
    rng = np.random.default_rng(seed)
    B = len(new)
    NB = B * MP + 2
    table = rng.permutation(NB)[: B * MP].reshape(B, MP).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + tail                            # rows behind the last sequence
    k, v = _rows(rng, T, Hkv, D, 40), _rows(rng, T, Hkv, D)
    return rng, table, np.array(total), cu, k, v, _random_pools(rng, NB, P, Hkv, D)


@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_and_read_are_exact(case):
    new, total, Hkv, D, P, MP = APPEND[case]
    rng, table, sl, cu, k, v, ref = _append_case(case, new, total, Hkv, D, P, MP)
    if table.size > 20:
        table[rng.integers(0, len(new)), rng.integers(0, MP)] = -1       # no page: dropped, reads zeros
        table[rng.integers(0, len(new)), rng.integers(0, MP)] = ref[0].shape[0]
        table[rng.integers(0, len(new)), rng.integers(0, MP)] = -2
    k[0, 0, :4] = torch.tensor([INF, -INF, float("nan"), 0.0])
    v[-1] = 0.0
    pools = _pools(*ref)
    args = (_i32(table), _i32(sl), _i32(cu))
    swl.attn_sink_cache_append_fp8(k.to(DEV), v.to(DEV), *args, *pools)
    cache8.append(inputs.bits(k), inputs.bits(v), table, sl, cu, *ref)
    for got, want, name in zip(pools, ref, ("kpages", "vpages", "kscales", "vscales")):
        np.testing.assert_array_equal(_u8(got), want, err_msg=name)
    # read back into rows that hold something else
    ko, vo = (torch.full_like(x, 7.0, device=DEV) for x in (k, v))
    swl.attn_sink_cache_read_fp8(*pools, *args, ko, vo)
    rk, rv = cache8.read(*ref, table, sl, cu, k.shape[0])
    for got, want in ((ko, rk), (vo, rv)):
        own = cache8.places(sl, cu, k.shape[0], table, ref[0].shape[0], P)[:, 0] != -2
        np.testing.assert_array_equal(got.double().cpu().numpy()[own], want[own])
        assert (got.double().cpu().numpy()[~own] == 7.0).all(), "rows of no sequence were written"


def test_append_strided_rows_and_pools():
    """k and v as slices of one projection, pools as slices of larger ones."""
    rng, table, sl, cu, k, v, ref = _append_case(3, [9, 20], [30, 20], 2, 64, 16, 3, tail=0)
    T = k.shape[0]
    kv = torch.zeros(T, 5, 2, 64, dtype=torch.bfloat16, device=DEV)
    kv[:, 1], kv[:, 3] = k.to(DEV), v.to(DEV)
    flat = _pools(*ref)
    big = [torch.zeros((2 * t.shape[0], t.shape[1], 3 * t.shape[2]) + tuple(t.shape[3:]), dtype=torch.uint8,
                       device=DEV).view(t.dtype) for t in flat]
    pools = [b[::2, :, : t.shape[2]] for b, t in zip(big, flat)]
    for p, t in zip(pools, flat):
        p.view(torch.uint8).copy_(t.view(torch.uint8))
    swl.attn_sink_cache_append_fp8(kv[:, 1], kv[:, 3], _i32(table), _i32(sl), _i32(cu), *pools)
    cache8.append(inputs.bits(k), inputs.bits(v), table, sl, cu, *ref)
    for got, want, b in zip(pools, ref, big):
        np.testing.assert_array_equal(_u8(got.contiguous()), want)
        assert not _u8(b)[1::2].any(), "a skipped page was written"
    out = torch.zeros_like(kv)
    swl.attn_sink_cache_read_fp8(*pools, _i32(table), _i32(sl), _i32(cu), out[:, 0], out[:, 4])
    rk, rv = cache8.read(*ref, table, sl, cu, T)
    np.testing.assert_array_equal(out[:, 0].double().cpu().numpy(), rk)
    np.testing.assert_array_equal(out[:, 4].double().cpu().numpy(), rv)
    assert not out[:, 1:4].any()


def test_malformed_tables_stay_inside():
    """Offsets that decrease or pass T, negative and huge lengths: rows may go
    astray inside the pools, the bytes around them stay."""
    rng, table, sl, cu, k, v, ref = _append_case(4, [9, 20, 5], [30, 20, 5], 2, 64, 16, 3)
    for bad_cu, bad_sl in (([0, 50, 10, 900], sl), ([5, 3, 2, 30], sl), (cu, [-4, 1 << 30, 5])):
        NB = ref[0].shape[0]
        guard = [torch.full((NB + 2,) + t.shape[1:], 0x55, dtype=torch.uint8, device=DEV) for t in ref]
        pools = [g[1:-1].view(d) for g, d in zip(guard, (torch.float8_e4m3fn,) * 2 + (torch.float8_e8m0fnu,) * 2)]
        swl.attn_sink_cache_append_fp8(k.to(DEV), v.to(DEV), _i32(table), _i32(bad_sl), _i32(bad_cu), *pools)
        for g in guard:
            assert (g[0] == 0x55).all() and (g[-1] == 0x55).all()
        out = [torch.full((k.shape[0] + 2,) + k.shape[1:], 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        swl.attn_sink_cache_read_fp8(*pools, _i32(table), _i32(bad_sl), _i32(bad_cu), *[o[1:-1] for o in out])
        for o in out:
            assert (o[0] == 3.0).all() and (o[-1] == 3.0).all()


@pytest.mark.parametrize("bad", [-1, -2, -(1 << 31), 6, (1 << 31) - 1])
def test_entries_outside_the_pool(bad):
    """Every row of a page outside the pool is dropped by the append and read back as zeros."""
    rng, table, sl, cu, k, v, ref = _append_case(5, [20, 9], [20, 9], 2, 64, 16, 2)
    table[0, 0] = bad
    pools = _pools(*ref)
    args = (_i32(table), _i32(sl), _i32(cu))
    swl.attn_sink_cache_append_fp8(k.to(DEV), v.to(DEV), *args, *pools)
    cache8.append(inputs.bits(k), inputs.bits(v), table, sl, cu, *ref)
    for got, want in zip(pools, ref):
        np.testing.assert_array_equal(_u8(got), want)
    out = [torch.full_like(x, 7.0, device=DEV) for x in (k, v)]
    swl.attn_sink_cache_read_fp8(*pools, *args, *out)
    for o, x in zip(out, cache8.read(*ref, table, sl, cu, k.shape[0])):
        np.testing.assert_array_equal(o.double().cpu().numpy()[:29], x[:29])
        assert (o[:16] == 0).all() and (o[29:] == 7.0).all()


def test_a_pool_beyond_32_bits():
    """Pages whose byte offsets pass 2^32 in the codes (4.6 GB a pool): written, read
    back and attended to like the same rows in a small pool."""
    rng = np.random.default_rng(6)
    NB, P, Hkv, D, G, n = 70000, 64, 8, 128, 2, 200
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    empty = lambda *s: torch.empty(*s, dtype=torch.uint8, device=DEV)  # noqa: E731
    big = (empty(NB, P, Hkv, D).view(e4), empty(NB, P, Hkv, D).view(e4), empty(NB, Hkv, P).view(e8), empty(NB, Hkv, P).view(e8))
    small = (empty(4, P, Hkv, D).view(e4), empty(4, P, Hkv, D).view(e4), empty(4, Hkv, P).view(e8), empty(4, Hkv, P).view(e8))
    k, v = _rows(rng, n, Hkv, D).to(DEV), _rows(rng, n, Hkv, D).to(DEV)
    q = _rows(rng, 1, Hkv * G, D, 1).to(DEV)
    sl, cu, sinks = _i32([n]), _i32([0, n]), torch.zeros(Hkv * G, device=DEV)
    outs = []
    for pools, table in ((big, [[NB - 1, 65999, NB - 3, 69000]]), (small, [[3, 2, 0, 1]])):
        t = _i32(table)
        swl.attn_sink_cache_append_fp8(k, v, t, sl, cu, *pools)
        ko, vo, out = torch.empty_like(k), torch.empty_like(v), torch.empty_like(q)
        swl.attn_sink_cache_read_fp8(*pools, t, sl, cu, ko, vo)
        swl.attn_sink_decode_paged_fp8(q, *pools, t, sl, sinks, 1 << 30, 0.1, out)
        outs.append((ko, vo, out))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert swl.attn_sink_get_status() == 0


# --------------------------------------------------------------------- decode
DECODE = [  # seqlens, MP, P, Hkv, G, D, W
    ([1], 1, 16, 1, 1, 64, 1 << 30),
    ([17, 0, 64, 320], 20, 16, 2, 4, 128, 1 << 30),
    ([320, 1, 171, 0], 10, 32, 1, 8, 128, 100),
    ([640, 100, 513, 300], 10, 64, 4, 8, 128, 513),
    ([777, 512, 37], 7, 128, 2, 3, 64, 1),
    ([768, 600], 3, 256, 1, 16, 128, 513),
    ([384, 100, 0, 383], 6, 64, 2, 4, 256, 1 << 30),
    ([700, 65], 48, 16, 2, 3, 256, 200),
    ([2048, 1500], 2, 1024, 2, 4, 64, 1000),
    ([900, 380, 45], 60, 16, 2, 12, 64, 600),
    ([250, 64, 1], 16, 16, 2, 16, 128, 200),
    ([5000], 79, 64, 1, 2, 128, 1 << 30),             # one sequence over many SMs
    ([300] * 40, 5, 64, 5, 1, 64, 1 << 30),           # a head count that does not divide the SMs
    ([130] * 3, 3, 64, 200, 1, 64, 150),              # more heads than SMs
    ([3] * 500, 1, 16, 1, 2, 128, 2),                 # more sequences than threads of a block
]


def _decode_case(seed, seqlens, MP, P, Hkv, G, D, W, spread=2):
    rng = np.random.default_rng(seed)
    B = len(seqlens)
    NB = B * MP + 3
    perm = rng.permutation(NB)
    table = perm[: B * MP].reshape(B, MP).astype(np.int32)
    kp, vp, ks, vs = _random_pools(rng, NB, P, Hkv, D, spread)
    used = np.zeros((NB, P), bool)
    for b, n in enumerate(seqlens):
        for t in range(max(0, n - W), n):
            used[table[b, t // P], t % P] = True
    # whatever no query sees is NaN: codes, scales, whole pages
    kp[~used], vp[~used] = NAN_CODE, NAN_CODE
    for s in (ks, vs):
        s.transpose(0, 2, 1)[~used] = 255
    for b, n in enumerate(seqlens):
        for pg in range(MP):
            if (pg + 1) * P <= max(0, n - W) or pg * P >= n:
                table[b, pg] = [perm[-1], -1, NB + 7][(b + pg) % 3]
    q = torch.from_numpy(rng.standard_normal((B, Hkv * G, D)) * 2.0 ** rng.integers(-3, 3, (1, Hkv * G, 1))).bfloat16()
    sinks = rng.uniform(-4, 8, Hkv * G).astype(np.float32)
    return q, kp, vp, ks, vs, table, np.array(seqlens), sinks


def _decode(q, kp, vp, ks, vs, table, sl, sinks, W, scale):
    out = torch.full((q.shape[0] + 2,) + tuple(q.shape[1:]), float("nan"), dtype=torch.bfloat16, device=DEV)
    swl.attn_sink_decode_paged_fp8(q.to(DEV), *_pools(kp, vp, ks, vs), _i32(table), _i32(sl),
                                   torch.from_numpy(sinks).to(DEV), W, scale, out[1:-1])
    torch.cuda.synchronize()
    assert swl.attn_sink_get_status() == 0
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isnan(out[-1]).all()), "guard written"
    return out[1:-1].double().cpu().numpy()


@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode_against_the_definition(case):
    seqlens, MP, P, Hkv, G, D, W = DECODE[case]
    c = _decode_case(case, seqlens, MP, P, Hkv, G, D, W)
    scale = D ** -0.5
    ref, mag, top = cache8.decode(inputs.bits(c[0]), *c[1:], W, scale)
    got = _decode(*c, W, scale)
    bad = ~(np.abs(got - ref) <= _tol(ref, mag, top, min(W, max(seqlens)), D))
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])
    assert (got[c[6] == 0] == 0).all()


@pytest.mark.parametrize("kind", ["no sink", "huge sink", "value scales over many binades", "one key dominates",
                                  "zero values", "key scales over many binades"])
def test_decode_extremes(kind):
    seqlens, MP, P, Hkv, G, D, W = [500, 70, 193], 8, 64, 2, 4, 128, 1 << 30
    c = list(_decode_case(21, seqlens, MP, P, Hkv, G, D, W))
    rng = np.random.default_rng(22)
    scale = D ** -0.5
    if kind == "no sink":
        c[7][:] = -np.inf
    elif kind == "huge sink":
        c[7][:] = [60.0, -60.0] * 4
    elif kind == "value scales over many binades":
        c[4] = np.where(c[4] == 255, 255, rng.integers(60, 200, c[4].shape)).astype(np.uint8)
    elif kind == "one key dominates":
        page, pos = c[5][0, 3], 40
        c[1][page, pos] = c[1][page, pos] & 0x80 | 0x7E
        c[4][page, :, pos] = 12                        # and its values are tiny
        c[0] = c[0] * 4
    elif kind == "zero values":
        c[2][:] = np.where(c[2] == NAN_CODE, NAN_CODE, 0)
        c[4] = np.where(c[4] == 255, 255, 10).astype(np.uint8)
    else:
        c[3] = np.where(c[3] == 255, 255, rng.integers(100, 127, c[3].shape)).astype(np.uint8)
    ref, mag, top = cache8.decode(inputs.bits(c[0]), *c[1:], W, scale)
    got = _decode(*c, W, scale)
    assert (np.abs(got - ref) <= _tol(ref, mag, top, 500, D)).all(), np.abs(got - ref).max()


@pytest.mark.parametrize("scale", [1e-9, 0.0883, 1e-38])
def test_decode_queries_of_zeros_and_tiny_ones(scale):
    """A head of zeros weighs every visible key alike, whatever the scale, beside masked keys too."""
    seqlens, MP, P, Hkv, G, D, W = [500, 70, 1], 8, 64, 2, 4, 128, 333
    c = list(_decode_case(25, seqlens, MP, P, Hkv, G, D, W))
    c[0][:, 0::4] = 0
    c[0][:, 1::4] = c[0][:, 1::4] * 2.0 ** -118
    ref, mag, top = cache8.decode(inputs.bits(c[0]), *c[1:], W, scale)
    got = _decode(*c, W, scale)
    assert (np.abs(got - ref) <= _tol(ref, mag, top, 500, D)).all(), np.abs(got - ref).max()


def test_decode_nan_of_a_visible_row_reaches_its_heads_only():
    seqlens, MP, P, Hkv, G, D, W = [300, 90], 5, 64, 2, 4, 64, 1 << 30
    c = _decode_case(23, seqlens, MP, P, Hkv, G, D, W)
    c[1][c[5][0, 2], 10, 1, 5] = NAN_CODE
    got = _decode(*c, W, 0.125)
    assert np.isnan(got[0, 4:]).all() and np.isfinite(got[0, :4]).all() and np.isfinite(got[1]).all()


def test_decode_pages_out_of_the_pool_are_zero_rows():
    seqlens, MP, P, Hkv, G, D, W = [300, 90], 20, 16, 2, 4, 64, 1 << 30
    c = _decode_case(24, seqlens, MP, P, Hkv, G, D, W)
    c[5][0, 3], c[5][0, 18], c[5][1, 0] = -1, c[1].shape[0], 1 << 30
    ref, mag, top = cache8.decode(inputs.bits(c[0]), *c[1:], W, 0.125)
    got = _decode(*c, W, 0.125)
    assert (np.abs(got - ref) <= _tol(ref, mag, top, 300, D)).all()


def test_decode_strided_tensors_and_shared_pages():
    """q and out as slices, pools as slices, a prefix shared by two sequences; on a side stream."""
    seqlens, MP, P, Hkv, G, D, W = [200, 150], 4, 64, 2, 3, 128, 1 << 30
    c = list(_decode_case(25, seqlens, MP, P, Hkv, G, D, W))
    c[5][1, :2] = c[5][0, :2]
    ref, mag, top = cache8.decode(inputs.bits(c[0]), *c[1:], W, 0.09)
    flat = _pools(*c[1:5])
    pools = []
    for t in flat:
        b = torch.full((2 * t.shape[0], t.shape[1], 2 * t.shape[2]) + tuple(t.shape[3:]), 0x7F, dtype=torch.uint8,
                       device=DEV).view(t.dtype)
        p = b[::2, :, t.shape[2]:]
        p.view(torch.uint8).copy_(t.view(torch.uint8))
        pools.append(p)
    qo = torch.zeros(2, 3 * Hkv * G, D + 2, dtype=torch.bfloat16, device=DEV)
    q, out = qo[:, : Hkv * G, :D], qo[:, 2 * Hkv * G:, :D]
    q.copy_(c[0].to(DEV))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    swl.attn_sink_decode_paged_fp8(q, *pools, _i32(c[5]), _i32(c[6]), torch.from_numpy(c[7]).to(DEV), W, 0.09, out,
                                   stream=s)
    s.synchronize()
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref) <= _tol(ref, mag, top, 200, D)).all()
    assert not qo[..., D:].any() and not qo[:, Hkv * G: 2 * Hkv * G].any()


def test_decode_is_the_same_every_time():
    c = _decode_case(26, [3000, 100, 900], 47, 64, 2, 8, 128, 1 << 30)
    a, b = (_decode(*c, 1 << 30, 0.1) for _ in range(2))
    np.testing.assert_array_equal(a, b)


def test_calls_on_two_streams_and_threads_at_once():
    """Each with its own workspace: overlapping decodes give what they give alone."""
    import threading
    cases = [_decode_case(40 + i, [6000 + 500 * i, 300, 2000], 110, 64, 2, 8, 128, 1 << 30) for i in range(2)]
    args = [(c[0].to(DEV), *_pools(*c[1:5]), _i32(c[5]), _i32(c[6]), torch.from_numpy(c[7]).to(DEV), 1 << 30, 0.1)
            for c in cases]
    want = []
    for a in args:
        want.append(torch.empty_like(a[0]))
        swl.attn_sink_decode_paged_fp8(*a, want[-1])
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            outs = [torch.empty_like(want[i]) for _ in range(40)]
            s.wait_stream(torch.cuda.default_stream())
            for o in outs:
                swl.attn_sink_decode_paged_fp8(*args[i], o, stream=s)
            s.synchronize()
            assert all(torch.equal(o, want[i]) for o in outs)
        except BaseException as e:
            errors.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors
    assert swl.attn_sink_get_status() == 0


@pytest.mark.parametrize("W", [100, 1 << 30])
@pytest.mark.parametrize("captured", [False, True])
def test_calls_follow_the_kernels_before_them(W, captured):
    """Kernels that come up while the one before them ends read and write only behind it: every
    step's inputs are written by a kernel just before its calls, its outputs read just behind
    them, twenty steps in a row without a wait (W = 100: one launch a decode; else two)."""
    B, Hkv, G, D, P, MP, steps = 3, 2, 4, 128, 64, 30, 20
    g = torch.Generator().manual_seed(91)
    rnd = lambda *s: torch.randn(*s, generator=g).bfloat16().to(DEV)  # noqa: E731
    table = torch.randperm(B * MP, generator=g).reshape(B, MP).int().to(DEV)
    sinks = torch.zeros(Hkv * G, device=DEV)
    new = 5                                            # rows of every sequence in a step
    cu = _i32(np.arange(B + 1) * new)
    qs, ks, vs = rnd(steps, B, Hkv * G, D), rnd(steps, B * new, Hkv, D), rnd(steps, B * new, Hkv, D)
    lens = torch.tensor([[1800 + 5 * t, 70 + 5 * t, 5 + 5 * t] for t in range(steps)], dtype=torch.int32, device=DEV)
    first = _pools(*_random_pools(np.random.default_rng(92), B * MP, P, Hkv, D))
    q, k, v, sl = qs[0].clone(), ks[0].clone(), vs[0].clone(), lens[0].clone()
    out, kb, vb, ext = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), rnd(B * new, Hkv * G, D)
    q2 = rnd(B * new, Hkv * G, D)

    def serve(pools, wait):
        """All steps' outputs."""
        res = []
        for t in range(steps):
            for x, y in ((q, qs), (k, ks), (v, vs), (sl, lens)):
                x.copy_(y[t])
            for call in (lambda: swl.attn_sink_cache_append_fp8(k, v, table, sl, cu, *pools),
                         lambda: swl.attn_sink_decode_paged_fp8(q, *pools, table, sl, sinks, W, 0.09, out),
                         lambda: swl.attn_sink_cache_read_fp8(*pools, table, sl, cu, kb, vb),
                         lambda: swl.attn_sink_fwd_extend(q2, kb, vb, cu, cu, new, sinks, W, 0.09, ext)):
                if wait:
                    torch.cuda.synchronize()
                call()
            if wait:
                torch.cuda.synchronize()
            res.append([x.clone() for x in (out, kb, vb, ext)])
            for x in (out, kb, vb, ext):
                x.fill_(7)
        return res

    clone = lambda: [x.view(torch.uint8).clone().view(x.dtype) for x in first]  # noqa: E731
    want = serve(clone(), True)
    pools = clone()
    if captured:
        serve(clone(), False)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = serve(pools, False)
        graph.replay()
    else:
        got = serve(pools, False)
    torch.cuda.synchronize()
    assert swl.attn_sink_get_status() == 0
    for t in range(steps):
        for a, b in zip(got[t], want[t]):
            assert torch.equal(a, b), t


@pytest.mark.parametrize("captured", [False, True])
def test_calls_behind_two_streams(captured):
    """The kernels before a call are on two streams that join just before it."""
    B, Hkv, G, D, P, MP = 2, 2, 4, 128, 64, 20
    c = _decode_case(93, [1200, 600], MP, P, Hkv, G, D, 1 << 30)
    first, table, sinks = _pools(*c[1:5]), _i32(c[5]), torch.from_numpy(c[7]).to(DEV)
    sl, q0 = _i32(c[6]), c[0].to(DEV)
    k0, v0 = (torch.randn(B, Hkv, D, device=DEV).bfloat16() for _ in range(2))
    cu = _i32([0, 1, 2])
    junk, big = torch.randn(2500, 2500, device=DEV), torch.empty(2500, 2500, device=DEV)
    q, k, v, out = (torch.zeros_like(x) for x in (q0, k0, v0, q0))
    kb, vb, ext = torch.zeros_like(k), torch.zeros_like(v), torch.zeros(B, Hkv * G, D, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()

    def step(pools, wait=lambda: None):
        main = torch.cuda.current_stream()
        for call, slow, fast in (
                (lambda: swl.attn_sink_cache_append_fp8(k, v, table, sl, cu, *pools), (k, k0), (v, v0)),
                (lambda: swl.attn_sink_decode_paged_fp8(q, *pools, table, sl, sinks, 1 << 30, 0.09, out), (q, q0), (k, k0)),
                (lambda: swl.attn_sink_decode_paged_fp8(q, *pools, table, sl, sinks, 30, 0.09, ext), (q, 0.5 * q0), (k, k0)),
                (lambda: swl.attn_sink_cache_read_fp8(*pools, table, sl, cu, kb, vb), (kb, 2 * k0), (vb, v0)),
                (lambda: swl.attn_sink_fwd_extend(q, kb, vb, cu, cu, 1, sinks, 9, 0.09, ext), (q, q0), (vb, 3 * v0))):
            side.wait_stream(main)
            with torch.cuda.stream(side):              # the slower stream writes an input last
                torch.mm(junk, junk, out=big)
                torch.add(slow[1], big[0, 0] * 0, out=slow[0])
            torch.mul(fast[1], 1, out=fast[0])
            main.wait_stream(side)
            wait()
            call()
            wait()

    clone = lambda: [x.view(torch.uint8).clone().view(x.dtype) for x in first]  # noqa: E731
    res = (out, kb, vb, ext)
    pools = clone()
    step(pools, torch.cuda.synchronize)
    want = [x.clone() for x in res] + [x.view(torch.uint8).clone() for x in pools]
    pools = clone()
    for x in (q, k, v, *res):
        x.zero_()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(pools)
        graph.replay()
    else:
        step(pools)
    torch.cuda.synchronize()
    assert swl.attn_sink_get_status() == 0
    for a, b in zip(list(res) + [x.view(torch.uint8) for x in pools], want):
        assert torch.equal(a, b)


def test_decode_empty_table_and_batch():
    c = _decode_case(27, [0, 0], 1, 16, 1, 2, 64, 5)
    out = torch.full((2, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    pools = _pools(*c[1:5])
    sinks = torch.from_numpy(c[7]).to(DEV)
    table = torch.empty(2, 0, dtype=torch.int32, device=DEV)
    swl.attn_sink_decode_paged_fp8(c[0].to(DEV), *pools, table, _i32([9, 9]), sinks, 5, 0.1, out)
    assert (out == 0).all()
    swl.attn_sink_decode_paged_fp8(c[0].to(DEV)[:0], *pools, table[:0], _i32([]), sinks, 5, 0.1, out[:0])


def _under_short_limit(c):
    """The status of a decode whose waits give up at once, L2 flushed before it, and its output."""
    args = (c[0].to(DEV), *_pools(*c[1:5]), _i32(c[5]), _i32(c[6]), torch.from_numpy(c[7]).to(DEV))
    out = torch.empty(c[0].shape, dtype=torch.bfloat16, device=DEV)
    torch.empty(64 << 20, device=DEV).fill_(1.0)
    swl.attn_sink_set_wait_limit_ns(1)
    try:
        swl.attn_sink_decode_paged_fp8(*args, 1 << 30, 0.1, out)
        torch.cuda.synchronize()
        return swl.attn_sink_get_status(), out.double().cpu().numpy()
    finally:
        swl.attn_sink_set_wait_limit_ns(0)


def test_decode_short_waits_are_served_or_reported():
    """One tile for each SM: its wait may end within a step of the clock that the limit is held to."""
    c = _decode_case(28, [3000] * 4, 47, 64, 2, 8, 128, 1 << 30)
    ref, mag, top = cache8.decode(inputs.bits(c[0]), *c[1:], 1 << 30, 0.1)
    tol = _tol(ref, mag, top, 3000, 128)
    rc, got = _under_short_limit(c)
    assert rc == -5 or (rc == 0 and (np.abs(got - ref) <= tol).all())
    assert (np.abs(_decode(*c, 1 << 30, 0.1) - ref) <= tol).all()


def test_decode_wait_runs_out_then_recovers():
    c = _decode_case(31, [40000, 50000, 30000], 782, 64, 2, 1, 128, 1 << 30)
    assert _under_short_limit(c)[0] == -5
    assert swl.attn_sink_get_status() == 0
    ref, mag, top = cache8.decode(inputs.bits(c[0]), *c[1:], 1 << 30, 0.1)
    assert (np.abs(_decode(*c, 1 << 30, 0.1) - ref) <= _tol(ref, mag, top, 50000, 128)).all()


def test_decode_workspace_failure_launches_nothing():
    c = _decode_case(29, [1900], 30, 64, 1, 1, 64, 1 << 30)
    out = torch.full((1, 1, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    args = (c[0].to(DEV), *_pools(*c[1:5]), _i32(c[5]), _i32(c[6]), torch.from_numpy(c[7]).to(DEV))
    swl.attn_sink_fail_workspace_allocs(1)
    try:
        with pytest.raises(swl.AttnSinkError) as e:
            swl.attn_sink_decode_paged_fp8(*args, 1 << 30, 0.1, out)
        assert e.value.code == -4
        assert (out == 5.0).all()
        # sequences that are never cut need no workspace
        swl.attn_sink_fail_workspace_allocs(1)
        swl.attn_sink_decode_paged_fp8(*args, 5, 0.1, out)
        assert (out != 5.0).any()
    finally:
        swl.attn_sink_fail_workspace_allocs(0)


def test_tensors_on_the_host_are_refused():
    c = _decode_case(30, [100], 2, 64, 1, 1, 64, 1 << 30)
    pools = _pools(*c[1:5])
    with pytest.raises(ValueError):
        swl.attn_sink_decode_paged_fp8(c[0].to(DEV), *pools, torch.from_numpy(c[5]), _i32(c[6]),
                                       torch.from_numpy(c[7]).to(DEV), 5, 0.1, c[0].to(DEV))
