"""Calls that the header allows and no other test makes: empty tensors, tables that are
slices, the widest window, the largest pages, graphs of two streams at once."""
import numpy as np
import pytest
import torch

import sliding_window_learned_b200 as swl
from oracle import cache8
from sliding_window_learned_b200 import inputs
from test_gpu_cache_fp8 import DEV, _decode, _decode_case, _i32, _pools, _rows, _tol, _u8
from test_gpu_extend import _case, _tol_lse
from test_gpu_extend import _tol as _tol_extend

pytestmark = pytest.mark.gpu
FULL, WIDEST = 1 << 30, (1 << 31) - 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sliding_window_learned_b200 import build
    build.build()


@pytest.mark.parametrize("rows", [3, 700])
def test_no_key_tensor_at_all(rows):
    """k and v of no row: every query sees nothing."""
    q, _, _, cu_q, cu_k, sinks = _case(90, [rows, 2], [0, 0], 2, 4, 64, tail=(0, 0))
    k = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = torch.full_like(q, 9.0, device=DEV), torch.full((8, rows + 2), 9.0, device=DEV)
    swl.attn_sink_fwd_extend(q.to(DEV), k, k, _i32(cu_q), _i32(cu_k), rows, torch.from_numpy(sinks).to(DEV), FULL, 0.1,
                             out, lse)
    assert (out == 0).all()
    want = torch.from_numpy(sinks)[:, None]
    assert ((lse.cpu() - want).abs() <= 2.0 ** -22 * want.abs() + 2.0 ** -22).all()
    assert swl.attn_sink_get_status() == 0


def test_no_row_and_no_page():
    c = _decode_case(91, [5, 9], 1, 16, 2, 2, 64, FULL)
    pools, ref = _pools(*c[1:5]), [x.copy() for x in c[1:5]]
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    table, sl = _i32(c[5]), _i32(c[6])
    swl.attn_sink_cache_append_fp8(none, none, table, sl, _i32([0, 0, 0]), *pools)
    swl.attn_sink_cache_read_fp8(*pools, table, sl, _i32([0, 0, 0]), none, none)
    rows = torch.ones(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    wide = torch.empty(2, 0, dtype=torch.int32, device=DEV)             # a table of no page: no row has a place
    swl.attn_sink_cache_append_fp8(rows, rows, wide, sl, _i32([0, 3, 4]), *pools)
    for got, want in zip(pools, ref):
        np.testing.assert_array_equal(_u8(got), want)
    back = [torch.full_like(rows, 7.0) for _ in range(2)]
    swl.attn_sink_cache_read_fp8(*pools, wide, sl, _i32([0, 3, 4]), *back)
    assert all((x == 0).all() for x in back)
    assert swl.attn_sink_get_status() == 0


@pytest.mark.parametrize("seqlens,MP,P,D,W", [([300, 70], 5, 64, 128, FULL), ([1700, 0, 900], 120, 16, 64, WIDEST),
                                              ([600, 40], 12, 64, 256, 513)])
def test_a_table_that_is_a_slice(seqlens, MP, P, D, W):
    """Rows further apart than they are long, entries behind them anything."""
    c = _decode_case(92, seqlens, MP, P, 2, 3, D, W)
    B = len(seqlens)
    big = torch.full((B, MP + 7), 1 << 30, dtype=torch.int32, device=DEV)
    big[:, :MP] = _i32(c[5])
    table, pools, sinks = big[:, :MP], _pools(*c[1:5]), torch.from_numpy(c[7]).to(DEV)
    out = torch.empty(c[0].shape, dtype=torch.bfloat16, device=DEV)
    swl.attn_sink_decode_paged_fp8(c[0].to(DEV), *pools, table, _i32(c[6]), sinks, W, 0.1, out)
    ref, mag, top = cache8.decode(inputs.bits(c[0]), *c[1:], W, 0.1)
    assert (np.abs(out.double().cpu().numpy() - ref) <= _tol(ref, mag, top, max(seqlens), D)).all()
    new = [min(n, 20) for n in seqlens]
    cu = np.concatenate([[0], np.cumsum(new)])
    rng = np.random.default_rng(93)
    k, v = _rows(rng, int(cu[-1]), 2, D), _rows(rng, int(cu[-1]), 2, D)
    swl.attn_sink_cache_append_fp8(k.to(DEV), v.to(DEV), table, _i32(c[6]), _i32(cu), *pools)
    ref = [x.copy() for x in c[1:5]]
    cache8.append(inputs.bits(k), inputs.bits(v), c[5], c[6], cu, *ref)
    for got, want in zip(pools, ref):
        np.testing.assert_array_equal(_u8(got), want)
    assert swl.attn_sink_get_status() == 0


@pytest.mark.parametrize("lq,lk", [([3], [200]), ([40], [4000]), ([90, 20], [100, 300])])
def test_the_widest_window(lq, lk):
    """W = 2^31 - 1 is full causal attention."""
    q, k, v, cu_q, cu_k, sinks = _case(94, lq, lk, 1, 8, 128, tail=(0, 0))
    args = (q.to(DEV), k.to(DEV), v.to(DEV), _i32(cu_q), _i32(cu_k), max(lq), torch.from_numpy(sinks).to(DEV))
    outs = []
    for W in (WIDEST, FULL):
        out, lse = torch.empty_like(q, device=DEV), torch.empty(8, q.shape[0], device=DEV)
        swl.attn_sink_fwd_extend(*args, W, 0.1, out, lse)
        outs.append((out, lse))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    ro, rl, mag, top = cache8.extend(inputs.bits(q), inputs.bits(k), inputs.bits(v), cu_q, cu_k, sinks, WIDEST, 0.1)
    assert (np.abs(outs[0][0].double().cpu().numpy() - ro) <= _tol_extend(ro, mag, top, max(lk), 128)).all()
    assert (np.abs(outs[0][1].double().cpu().numpy() - rl) <= _tol_lse(rl, top, max(lk), 128)).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_largest_pages(D):
    """Pages of 65536 positions, written up to their last one."""
    P, n, Hkv, G = 65536, 65536 + 700, 1, 2
    rng = np.random.default_rng(95)
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    z = lambda *s: torch.full(s, 0x7F, dtype=torch.uint8, device=DEV)  # noqa: E731
    pools = (z(2, P, Hkv, D).view(e4), z(2, P, Hkv, D).view(e4), z(2, Hkv, P).view(e8), z(2, Hkv, P).view(e8))
    k, v = torch.zeros(n, Hkv, D, dtype=torch.bfloat16), _rows(rng, n, Hkv, D, 1)
    k[-900:] = _rows(rng, 900, Hkv, D, 1)
    k[: n - 900, :, 0] = -64.0                                     # (the far keys weigh next to nothing)
    table, sl, cu = _i32([[1, 0]]), _i32([n]), _i32([0, n])
    swl.attn_sink_cache_append_fp8(k.to(DEV), v.to(DEV), table, sl, cu, *pools)
    kb, vb = (torch.empty(n, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    swl.attn_sink_cache_read_fp8(*pools, table, sl, cu, kb, vb)
    ks, bytes_ = cache8.quantise(inputs.bits(k[-900:]))
    np.testing.assert_array_equal(kb[-900:].double().cpu().numpy(), cache8.E4M3[ks] * cache8.scales(bytes_)[..., None])
    q = torch.from_numpy(rng.standard_normal((1, Hkv * G, D))).bfloat16()
    q[..., 0] = 4.0                                                # (-256 of the far keys' logits)
    sinks = torch.zeros(Hkv * G)
    for W in (FULL, 800):
        out = torch.empty(1, Hkv * G, D, dtype=torch.bfloat16, device=DEV)
        swl.attn_sink_decode_paged_fp8(q.to(DEV), *pools, table, sl, sinks.to(DEV), W, 1.0, out)
        kd, vd, qd = (x.double().cpu().numpy() for x in (kb, vb, q))
        lo = max(0, n - W)
        for h in range(Hkv * G):
            x = kd[lo:, 0] @ qd[0, h]
            m = max(x.max(), 0.0)
            p = np.exp(x - m)
            den = p.sum() + np.exp(-m)
            o, mag = p @ vd[lo:, 0] / den, p @ np.abs(vd[lo:, 0]) / den
            top = (np.abs(kd[lo:, 0]) @ np.abs(qd[0, h])).max()
            got = out[0, h].double().cpu().numpy()
            assert (np.abs(got - o) <= _tol(o, mag[None], np.array([top]), n - lo, D)[0]).all()
    assert swl.attn_sink_get_status() == 0


def test_two_graphs_at_once():
    """Two captured decodes that need workspace, replayed on two streams over one another."""
    cases = [_decode_case(96 + i, [3000 + 500 * i, 300, 2000], 64, 64, 2, 8, 128, FULL) for i in range(2)]
    graphs, outs, want, streams = [], [], [], []
    for c in cases:
        args = (c[0].to(DEV), *_pools(*c[1:5]), _i32(c[5]), _i32(c[6]), torch.from_numpy(c[7]).to(DEV), FULL, 0.1)
        want.append(torch.empty_like(args[0]))
        swl.attn_sink_decode_paged_fp8(*args, want[-1])
        outs.append([torch.zeros_like(args[0]) for _ in range(8)])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for o in outs[-1]:
                swl.attn_sink_decode_paged_fp8(*args, o)
        graphs.append((g, args))
        streams.append(torch.cuda.Stream())
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(x, w) for x in o)
            for x in o:
                x.zero_()
        torch.cuda.synchronize()
    assert swl.attn_sink_get_status() == 0


def test_decode_widest_window_of_whole_and_cut():
    for seqlens, MP in (([500, 70], 8), ([1400, 0, 900], 24)):
        c = _decode_case(98, seqlens, MP, 64, 2, 4, 128, FULL)
        np.testing.assert_array_equal(_decode(*c, WIDEST, 0.1), _decode(*c, FULL, 0.1))


def test_rows_whose_offsets_pass_32_bits():
    """k and v of 2.3e9 elements (4.7 GB): appended, and read back, at both ends."""
    T, Hkv, D, P = 1150003, 8, 256, 64
    pages = -(-T // P)
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=DEV)  # noqa: E731
    pools = (z(pages, P, Hkv, D).view(e4), z(pages, P, Hkv, D).view(e4), z(pages, Hkv, P).view(e8), z(pages, Hkv, P).view(e8))
    table, sl, cu = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=DEV)[None], _i32([T]), _i32([0, T])
    k, v = (torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    assert k.numel() > 1 << 31
    rng = np.random.default_rng(99)
    ends = [slice(0, 300), slice(T // 2, T // 2 + 300), slice(T - 300, T)]
    rows = [(_rows(rng, 300, Hkv, D), _rows(rng, 300, Hkv, D)) for _ in ends]
    for e, (a, b) in zip(ends, rows):
        k[e], v[e] = a.to(DEV), b.to(DEV)
    swl.attn_sink_cache_append_fp8(k, v, table, sl, cu, *pools)
    k.fill_(7), v.fill_(7)
    swl.attn_sink_cache_read_fp8(*pools, table, sl, cu, k, v)
    for e, ab in zip(ends, rows):
        for got, x in zip((k, v), ab):
            codes, scale = cache8.quantise(inputs.bits(x))
            np.testing.assert_array_equal(got[e].double().cpu().numpy(), cache8.E4M3[codes] * cache8.scales(scale)[..., None])
    between = torch.ones(T, dtype=torch.bool, device=DEV)
    for e in ends:
        between[e] = False
    at = between.nonzero()[:: 97, 0]
    assert not k[at].any() and not v[at].any()
    assert swl.attn_sink_get_status() == 0


def test_queries_whose_offsets_pass_32_bits():
    """q and out of 2.3e9 elements, each query beside its own key alone (W = 1)."""
    T, Hq, D = 70001, 128, 256
    g = torch.Generator(device=DEV).manual_seed(100)
    q = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV)
    k, v = (torch.randn(T, 4, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    assert q.numel() > 1 << 31
    ends = (0, T // 2, T - 50)
    for e in ends:
        q[e: e + 50] = torch.randn(50, Hq, D, generator=g, device=DEV).bfloat16()
    sinks = torch.linspace(-2, 3, Hq, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(Hq, T, device=DEV)
    cu = _i32([0, T])
    swl.attn_sink_fwd_extend(q, k, v, cu, cu, T, sinks, 1, 0.1, out, lse)
    torch.cuda.synchronize()
    assert swl.attn_sink_get_status() == 0
    for e in ends:
        x = [t[e: e + 50] for t in (q, k, v)]
        one = np.array([0, 50])
        ro, rl, mag, top = cache8.extend(*(inputs.bits(t.cpu()) for t in x), one, one, sinks.cpu().numpy(), 1, 0.1)
        assert (np.abs(out[e: e + 50].double().cpu().numpy() - ro) <= _tol_extend(ro, mag, top, 1, D)).all()
        assert (np.abs(lse[:, e: e + 50].double().cpu().numpy() - rl) <= _tol_lse(rl, top, 1, D)).all()


@pytest.mark.parametrize("terms", [1, 2])
def test_a_captured_call_of_either_number_of_terms(terms):
    q, k, v, cu_q, cu_k, sinks = _case(101, [5, 40], [2500, 1900], 2, 8, 128, tail=(0, 0))
    args = (q.to(DEV), k.to(DEV), v.to(DEV), _i32(cu_q), _i32(cu_k), 40, torch.from_numpy(sinks).to(DEV), FULL, 0.1, terms)
    want, got = torch.empty_like(q, device=DEV), torch.zeros_like(q, device=DEV)
    swl.attn_sink_fwd_extend_terms(*args, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        swl.attn_sink_fwd_extend_terms(*args, got)
    for _ in range(3):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert swl.attn_sink_get_status() == 0
