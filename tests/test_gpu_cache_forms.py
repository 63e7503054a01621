"""The forms that the 8-bit cache's calls take at larger sizes, against the oracle:
decodes whose sequences are cut over the SMs (plan, partials, combine) beside ones
finished whole, appends and reads of several iterations a warp.

Which form a decode takes is seen, not restated: only the cut one needs workspace,
so only it fails when the next workspace allocation is made to fail.  Tolerances
as in test_gpu_cache_fp8."""
import numpy as np
import pytest
import torch

import sliding_window_learned_b200 as swl
from oracle import cache8
from sliding_window_learned_b200 import inputs
from test_gpu_cache_fp8 import DEV, INF, _decode, _decode_case, _i32, _pools, _rows, _tol, _u8

pytestmark = pytest.mark.gpu
FULL = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sliding_window_learned_b200 import build
    build.build()


def _is_cut(c, W):
    """Whether this decode takes the cut form."""
    out = torch.empty(c[0].shape, dtype=torch.bfloat16, device=DEV)
    swl.attn_sink_fail_workspace_allocs(1)
    try:
        swl.attn_sink_decode_paged_fp8(c[0].to(DEV), *_pools(*c[1:5]), _i32(c[5]), _i32(c[6]),
                                       torch.from_numpy(c[7]).to(DEV), W, 0.1, out)
        return False
    except swl.AttnSinkError as e:
        assert e.code == -4
        return True
    finally:
        swl.attn_sink_fail_workspace_allocs(0)


CUT = [  # seqlens, MP, P, Hkv, G, D, W
    ([2000, 0, 37, 1700, 0, 5], 32, 64, 2, 4, 64, FULL),
    ([1900, 300, 0, 1601], 125, 16, 1, 12, 64, 1600),          # two head tiles
    ([1300, 0, 900, 64], 24, 64, 2, 16, 128, FULL),
    ([700, 1300, 0, 1], 82, 16, 2, 9, 128, 1000),
    ([3000, 0, 1200, 200, 2999], 48, 64, 2, 8, 128, 1300),     # a window over several tiles
    ([2500, 2177, 830], 40, 64, 4, 3, 128, 769),
    ([1000, 0, 600, 17, 530], 64, 16, 2, 5, 256, FULL),
    ([1000, 513, 0, 999], 8, 128, 1, 8, 256, 700),
    ([800, 0, 1023, 769, 5, 64], 16, 64, 5, 1, 128, FULL),     # heads that do not divide the SMs
    ([1600, 1, 0, 1700], 27, 64, 64, 1, 64, FULL),             # several rounds of items
    ([520, 0, 576], 9, 64, 200, 1, 256, FULL),                 # more heads than SMs
    ([900] + [3] * 70 + [0] * 5 + [800, 0, 1], 16, 64, 1, 2, 128, FULL),   # several sequences a lane
    ([0, 0, 1000], 1, 1024, 2, 2, 128, FULL),                  # one page a sequence
    ([0, 0, 0], 16, 64, 2, 2, 128, FULL),                      # nothing at all
    ([30000, 1], 469, 64, 1, 4, 128, FULL),                    # more than 32 parts
]


@pytest.mark.parametrize("case", range(len(CUT)))
def test_cut_sequences_against_the_definition(case):
    seqlens, MP, P, Hkv, G, D, W = CUT[case]
    c = _decode_case(100 + case, seqlens, MP, P, Hkv, G, D, W)
    assert _is_cut(c, W)
    ref, mag, top = cache8.decode(inputs.bits(c[0]), *c[1:], W, D ** -0.5)
    got = _decode(*c, W, D ** -0.5)
    bad = ~(np.abs(got - ref) <= _tol(ref, mag, top, min(W, max(seqlens)), D))
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])
    assert (got[c[6] == 0] == 0).all()
    np.testing.assert_array_equal(got, _decode(*c, W, D ** -0.5))      # the same every time


@pytest.mark.parametrize("kind", ["no sink", "huge sink", "values over many binades", "one key dominates", "zero values",
                                  "keys over many binades", "pages outside the pool", "zero queries"])
@pytest.mark.parametrize("D,G,P", [(64, 4, 64), (64, 12, 16), (128, 4, 64), (128, 16, 16), (256, 5, 16)])
def test_cut_sequences_at_the_extremes(kind, D, G, P):
    seqlens, Hkv = [1700, 70, 0, 1900], 2
    MP = 2048 // P
    c = list(_decode_case(200, seqlens, MP, P, Hkv, G, D, FULL))
    rng = np.random.default_rng(201)
    if kind == "no sink":
        c[7][:] = -np.inf
    elif kind == "huge sink":
        c[7][:] = np.where(np.arange(Hkv * G) % 2, -60.0, 60.0)
    elif kind == "values over many binades":
        c[4] = np.where(c[4] == 255, 255, rng.integers(60, 200, c[4].shape)).astype(np.uint8)
    elif kind == "one key dominates":
        page, pos = c[5][0, 1000 // P], 1000 % P
        c[1][page, pos] = c[1][page, pos] & 0x80 | 0x7E
        c[4][page, :, pos] = 12
        c[0] = c[0] * 4
    elif kind == "zero values":
        c[2][:] = np.where(c[2] == 0x7F, 0x7F, 0)
    elif kind == "keys over many binades":
        c[3] = np.where(c[3] == 255, 255, rng.integers(100, 127, c[3].shape)).astype(np.uint8)
    elif kind == "pages outside the pool":
        c[5][0, :: 5], c[5][3, 3], c[5][1, 0] = -1, c[1].shape[0], -(1 << 31)
    else:
        c[0][:, ::3] = 0
    assert _is_cut(c, FULL)
    ref, mag, top = cache8.decode(inputs.bits(c[0]), *c[1:], FULL, D ** -0.5)
    got = _decode(*c, FULL, D ** -0.5)
    bad = ~(np.abs(got - ref) <= _tol(ref, mag, top, max(seqlens), D))
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])


@pytest.mark.parametrize("D,G", [(64, 4), (128, 16), (256, 3)])
def test_a_nan_in_a_cut_sequence_reaches_its_heads_only(D, G):
    c = _decode_case(210, [1700, 1800], 32, 64, 2, G, D, FULL)
    assert _is_cut(c, FULL)
    c[1][c[5][0, 20], 10, 1, 5] = 0x7F
    got = _decode(*c, FULL, 0.1)
    assert np.isnan(got[0, G:]).all() and np.isfinite(got[0, :G]).all() and np.isfinite(got[1]).all()


def test_the_longest_uncut_and_the_shortest_cut():
    """A key more in the table's reach turns one form into the other; both give the same answer."""
    for D, most in ((64, 1536), (128, 768), (256, 512)):
        for W, cut in ((most - 63, False), (most - 62, True)):
            c = _decode_case(220, [1999, W, 3], 32, 64, 2, 2, D, W)
            assert _is_cut(c, W) == cut, (D, W)
            ref, mag, top = cache8.decode(inputs.bits(c[0]), *c[1:], W, 0.1)
            assert (np.abs(_decode(*c, W, 0.1) - ref) <= _tol(ref, mag, top, W, D)).all()


# ----------------------------------------------- appends and reads of many rows
LONG = [  # D, Hkv, P, sequences, rows
    (128, 5, 16, 40, 33000),
    (128, 3, 64, 7, 54000),
    (256, 5, 16, 30, 17000),
    (64, 7, 32, 1100, 46000),              # more sequences than shared memory keeps
]


@pytest.mark.parametrize("case", range(len(LONG)))
def test_rows_of_many_iterations_are_exact(case):
    """Every warp comes back at least twice, by a stride that the heads do not divide, and the
    last iteration is cut short; the read is past the size up to which it takes more blocks."""
    D, Hkv, P, B, T = LONG[case]
    per_pass, sms = 512 // D, torch.cuda.get_device_properties(0).multi_processor_count
    assert T * Hkv > 2 * sms * 32 * 2 * per_pass                # append: 32 warps an SM, two passes an iteration
    assert T * Hkv > 4 * sms * 32 * 2 * per_pass                # read: beyond four iterations 16 warps an SM
    assert (sms * 32 * 2 * per_pass) % Hkv and ((T + 5) * Hkv) % (2 * per_pass)
    rng = np.random.default_rng(300 + case)
    cut = np.sort(rng.integers(0, T + 1, B - 1))
    cu = np.concatenate([[0], cut, [T]])
    new = np.diff(cu)
    past = rng.integers(0, 3 * P, B)
    total = new + past
    MP = int(-(-total.max() // P))
    pages = -(-total // P)
    NB = int(pages.sum()) + 2
    order, table, at = rng.permutation(NB), np.full((B, MP), -1, np.int32), 0
    for b, m in enumerate(pages):
        table[b, :m] = order[at: at + m]
        at += m
    table[B // 2, pages[B // 2] // 2] = NB                      # no such page: dropped, reads zeros
    tail = 5
    k, v = _rows(rng, T + tail, Hkv, D, 30), _rows(rng, T + tail, Hkv, D)
    k[::1001, 0, 3] = INF
    v[5::997, Hkv - 1, 0] = float("nan")
    ref = [np.full((NB, P, Hkv, D), 0x33, np.uint8), np.full((NB, P, Hkv, D), 0x44, np.uint8),
           np.full((NB, Hkv, P), 0x55, np.uint8), np.full((NB, Hkv, P), 0x66, np.uint8)]
    pools = _pools(*ref)
    args = (_i32(table), _i32(total), _i32(cu))
    swl.attn_sink_cache_append_fp8(k.to(DEV), v.to(DEV), *args, *pools)
    cache8.append(inputs.bits(k), inputs.bits(v), table, total, cu, *ref)
    for got, want, name in zip(pools, ref, ("kpages", "vpages", "kscales", "vscales")):
        np.testing.assert_array_equal(_u8(got), want, err_msg=name)
    out = [torch.full((T + tail, Hkv, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    swl.attn_sink_cache_read_fp8(*pools, *args, *out)
    for o, want in zip(out, cache8.read(*ref, table, total, cu, T + tail)):
        np.testing.assert_array_equal(o[:T].float().cpu().numpy(), want[:T].astype(np.float32))
        assert (o[T:] == 7.0).all(), "rows of no sequence were written"


def test_a_read_of_a_few_iterations_is_exact():
    """Between one iteration and the size from which the read takes fewer blocks."""
    D, Hkv, P, T = 64, 3, 16, 60000
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert sms * 32 * 8 < T * Hkv <= 4 * sms * 32 * 16
    rng = np.random.default_rng(310)
    NB = T // P + 3
    table = rng.permutation(NB)[None, : T // P].astype(np.int32)
    ref = [rng.integers(0, 256, (NB, P, Hkv, D)).astype(np.uint8) for _ in range(2)]
    ref += [rng.integers(10, 247, (NB, Hkv, P)).astype(np.uint8) for _ in range(2)]
    out = [torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    swl.attn_sink_cache_read_fp8(*_pools(*ref), _i32(table), _i32([T]), _i32([0, T]), *out)
    for o, want in zip(out, cache8.read(*ref, table, np.array([T]), np.array([0, T]), T)):
        np.testing.assert_array_equal(o.float().cpu().numpy(), want.astype(np.float32))
