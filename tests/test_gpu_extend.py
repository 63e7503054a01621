"""attn_sink_fwd_extend on the GPU against the double-precision definition, and
the cache's calls together: a prompt attended to in chunks, quantised as it
goes, then decoded from.

Tolerance of an output: half a bf16 step, 2^-8 |o|, and relative to A = sum_j p_j
|v_j| / den: P in bf16 (2^-8), fp32 scores of D products of magnitude at most S
in all (D * 2^-24 * S in numerator and denominator), fp32 sums over n keys, the
exponentials' few 2^-22.  LSE: the scores' and the sum's part of that, and its
own rounding."""
import numpy as np
import pytest
import torch

import sliding_window_learned_b200 as swl
from oracle import cache8
from sliding_window_learned_b200 import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sliding_window_learned_b200 import build
    build.build()


def _tol(o, mag, top, n, D):
    c = 2.0 ** -8 + 2 * D * 2.0 ** -24 * top + 2 * n * 2.0 ** -24 + 2.0 ** -19
    return 2.0 ** -8 * np.abs(o) + c[..., None] * mag * 1.01 + 1e-37


def _tol_lse(lse, top, n, D):
    return D * 2.0 ** -24 * top.T + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(lse) + 2.0 ** -19


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _case(seed, lq, lk, Hkv, G, D, tail=(3, 5)):
    rng = np.random.default_rng(seed)
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]) for x in (lq, lk))
    T, Tk = int(cu_q[-1]) + tail[0], int(cu_k[-1]) + tail[1]
    q, k, v = (torch.from_numpy(rng.standard_normal(s)).bfloat16()
               for s in ((T, Hkv * G, D), (Tk, Hkv, D), (Tk, Hkv, D)))
    sinks = rng.uniform(-4, 8, Hkv * G).astype(np.float32)
    return q, k, v, cu_q, cu_k, sinks


def _run(q, k, v, cu_q, cu_k, sinks, W, scale, max_q=None, lse=True):
    T, Hq, D = q.shape
    out = torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    l = torch.full((Hq, T), 9.0, device=DEV) if lse else None
    swl.attn_sink_fwd_extend(q.to(DEV), k.to(DEV), v.to(DEV), _i32(cu_q), _i32(cu_k),
                             int(np.diff(cu_q).max(initial=0)) if max_q is None else max_q,
                             torch.from_numpy(sinks).to(DEV), W, scale, out, l)
    torch.cuda.synchronize()
    assert swl.attn_sink_get_status() == 0
    return out.double().cpu().numpy(), l.double().cpu().numpy() if lse else None


CASES = [  # queries, keys, Hkv, G, D, W
    ([1], [1], 1, 1, 64, 1 << 30),
    ([1, 1, 1], [1, 65, 300], 2, 4, 128, 1 << 30),
    ([128], [128 + 64], 1, 2, 128, 1 << 30),
    ([130, 0, 7, 200], [300, 40, 7, 200], 2, 2, 64, 50),
    ([100, 33], [612, 545], 1, 3, 128, 513),
    ([64, 150], [70, 151], 2, 1, 256, 100),
    ([17, 5], [1000, 0], 1, 2, 128, 1),
    ([140, 20], [5, 30], 1, 2, 64, 1 << 30),          # more queries than keys: rows that see nothing
    ([300], [130], 1, 1, 128, 64),                    # a whole query tile that sees nothing
    ([20, 3], [0, 0], 1, 2, 64, 7),                   # no key at all
    ([1] * 70, list(range(1, 71)), 1, 2, 64, 20),
    # heads that share a query tile: groups of every kind, tiles with unused rows
    ([60, 1], [90, 40], 1, 8, 64, 1 << 30),
    ([40], [41], 2, 7, 64, 17),
    ([9, 8, 10], [9, 80, 100], 1, 16, 64, 1 << 30),
    ([5, 2], [70, 2], 1, 37, 64, 60),
    ([3, 4], [70, 9], 1, 48, 64, 60),
    ([2], [5], 1, 130, 64, 60),
    # few queries, many keys: the keys are split
    ([1, 3], [3000, 700], 2, 2, 128, 1 << 30),
    ([2, 0, 1], [2500, 900, 0], 1, 5, 64, 1 << 30),
    ([30], [2000], 1, 3, 256, 1500),
    ([7, 20, 1], [600, 2100, 513], 1, 8, 128, 600),
    ([5], [4000], 2, 16, 64, 1 << 30),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_extend_against_the_definition(case):
    lq, lk, Hkv, G, D, W = CASES[case]
    q, k, v, cu_q, cu_k, sinks = _case(case, lq, lk, Hkv, G, D)
    scale = D ** -0.5
    ro, rl, mag, top = cache8.extend(q=inputs.bits(q), k=inputs.bits(k), v=inputs.bits(v), cu_q=cu_q, cu_k=cu_k,
                                     sinks=sinks, window=W, scale=scale)
    o, lse = _run(q, k, v, cu_q, cu_k, sinks, W, scale)
    n, T = min(W, max(lk)), int(cu_q[-1])
    assert (np.abs(o - ro) <= _tol(ro, mag, top, n, D))[:T].all(), np.abs(o - ro)[:T].max()
    assert (np.abs(lse - rl) <= _tol_lse(rl, top, n, D))[:, :T].all()
    assert (o[T:] == 9.0).all() and (lse[:, T:] == 9.0).all(), "rows of no sequence were written"


@pytest.mark.parametrize("lq,lk,Hkv,G,D,W", [
    ([1], [9], 1, 1, 64, 1 << 30), ([3, 1], [1000, 70], 1, 16, 128, 513), ([2, 2, 0, 3], [2, 300, 5, 65], 2, 5, 256, 100),
    ([16], [4000], 2, 8, 128, 1 << 30), ([5, 1], [3, 200], 1, 2, 64, 1 << 30), ([1] * 8, [2900] * 8, 4, 8, 64, 1 << 30)])
def test_extend_of_few_rows_rounds_the_weights_twice(lq, lk, Hkv, G, D, W):
    """At most 512 rows: P as two bf16 terms, 2^-16 off (2^-8 the rest, and 2^-8 of that)."""
    q, k, v, cu_q, cu_k, sinks = _case(60, lq, lk, Hkv, G, D, tail=(0, 5))
    assert q.shape[0] * Hkv * G <= 512
    ro, rl, mag, top = cache8.extend(q=inputs.bits(q), k=inputs.bits(k), v=inputs.bits(v), cu_q=cu_q, cu_k=cu_k,
                                     sinks=sinks, window=W, scale=D ** -0.5)
    o, lse = _run(q, k, v, cu_q, cu_k, sinks, W, D ** -0.5)
    n = min(W, max(lk))
    tol = _tol(ro, mag, top, n, D) - (2.0 ** -8 - 2.0 ** -16) * mag * 1.01
    assert (np.abs(o - ro) <= tol).all(), (np.abs(o - ro) / tol).max()
    assert (np.abs(lse - rl) <= _tol_lse(rl, top, n, D)).all()


@pytest.mark.parametrize("G", [1, 3])
def test_extend_without_earlier_keys_is_the_packed_forward(G):
    q, k, v, cu, _, sinks = _case(50, [200, 1, 77], [200, 1, 77], 2, G, 128, tail=(0, 0))
    a = _run(q, k, v, cu, cu, sinks, 65, 0.1)
    out, lse = torch.empty_like(q, device=DEV), torch.empty(2 * G, q.shape[0], device=DEV)
    swl.attn_sink_fwd_varlen(q.to(DEV), k.to(DEV), v.to(DEV), _i32(cu), 200, torch.from_numpy(sinks).to(DEV), 65, 0.1,
                             out, lse)
    # the same scores and key tiles; a row's running maximum may move at another
    # tile beside other rows, so P is rounded from another reference
    c = 2 * 2.0 ** -8 * np.abs(v.double().numpy()).max()
    assert np.abs(a[0] - out.double().cpu().numpy()).max() <= c
    assert np.abs(a[1] - lse.double().cpu().numpy()).max() <= 2.0 ** -19


def test_extend_workspace_failure_launches_nothing():
    q, k, v, cu_q, cu_k, sinks = _case(54, [2], [3000], 1, 2, 64, tail=(0, 0))     # (keys are split)
    out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device=DEV)
    args = (q.to(DEV), k.to(DEV), v.to(DEV), _i32(cu_q), _i32(cu_k), 2, torch.from_numpy(sinks).to(DEV), 1 << 30, 0.1, out)
    swl.attn_sink_fail_workspace_allocs(1)
    try:
        with pytest.raises(swl.AttnSinkError) as e:
            swl.attn_sink_fwd_extend(*args)
        assert e.value.code == -4 and (out == 9.0).all()
    finally:
        swl.attn_sink_fail_workspace_allocs(0)
    swl.attn_sink_fwd_extend(*args)
    assert torch.isfinite(out.float()).all() and (out != 9.0).any()


def test_extend_keeps_other_sequences_values_out():
    """The value rows of the next sequence (NaN, infinity) share this one's last key tile."""
    q, k, v, cu_q, cu_k, sinks = _case(51, [40, 30, 9], [70, 100, 9], 1, 2, 64)
    scale = 0.125
    good = _run(q, k, v, cu_q, cu_k, sinks, 1 << 30, scale)[0]
    v[70:170], v[179:] = float("nan"), float("inf")
    k[70:170] = float("nan")
    got = _run(q, k, v, cu_q, cu_k, sinks, 1 << 30, scale)[0]
    for rows in (slice(0, 40), slice(70, 79)):
        np.testing.assert_array_equal(got[rows], good[rows])
    assert np.isnan(got[40:70]).all()


def test_extend_only_needs_the_windows_keys():
    q, k, v, cu_q, cu_k, sinks = _case(52, [90], [700], 1, 2, 128, tail=(0, 0))
    W = 129
    full = _run(q, k, v, cu_q, cu_k, sinks, W, 0.1)
    keep = 90 + W - 1
    part = _run(q, k[-keep:], v[-keep:], cu_q, [0, keep], sinks, W, 0.1)
    # (other tiles of keys: the sums' order differs)
    n = 2 * 2.0 ** -24 * 200 + 2.0 ** -8
    assert (np.abs(part[0] - full[0]) <= 2 * n * np.abs(v.double().numpy()).max()).all()
    assert np.abs(part[1] - full[1]).max() < 1e-5


def test_extend_strided_no_lse_other_stream_and_malformed_offsets():
    q, k, v, cu_q, cu_k, sinks = _case(53, [50, 20], [80, 60], 2, 2, 64, tail=(0, 0))
    want = _run(q, k, v, cu_q, cu_k, sinks, 33, 0.1, lse=False, max_q=70)[0]
    kv = torch.zeros(k.shape[0], 3, 2, 64, dtype=torch.bfloat16, device=DEV)
    kv[:, 0], kv[:, 2] = k.to(DEV), v.to(DEV)
    qo = torch.zeros(q.shape[0], 2, 4, 64, dtype=torch.bfloat16, device=DEV)
    qo[:, 0] = q.to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    swl.attn_sink_fwd_extend(qo[:, 0], kv[:, 0], kv[:, 2], _i32(cu_q), _i32(cu_k), 50, torch.from_numpy(sinks).to(DEV),
                             33, 0.1, qo[:, 1], stream=s)
    s.synchronize()
    np.testing.assert_array_equal(qo[:, 1].double().cpu().numpy(), want)
    # offsets that decrease or pass T and Tk stay inside the tensors
    buf = torch.full((q.shape[0] + 2,) + q.shape[1:], 5.0, dtype=torch.bfloat16, device=DEV)
    for bad_q, bad_k in (([0, 90, 30], cu_k), (cu_q, [0, 500, 100]), ([-5, 60, 70], [30, 10, 140])):
        swl.attn_sink_fwd_extend(q.to(DEV), k.to(DEV), v.to(DEV), _i32(bad_q), _i32(bad_k), 70,
                                 torch.from_numpy(sinks).to(DEV), 33, 0.1, buf[1:-1])
        assert (buf[0] == 5.0).all() and (buf[-1] == 5.0).all()
    assert swl.attn_sink_get_status() == 0


def _tensors(B, MP, P, Hkv, D, NB):
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    z = lambda *s: torch.full(s, 0x7F, dtype=torch.uint8, device=DEV)  # noqa: E731  (NaN codes)
    return z(NB, P, Hkv, D).view(e4), z(NB, P, Hkv, D).view(e4), z(NB, Hkv, P).view(e8), z(NB, Hkv, P).view(e8)


@pytest.mark.parametrize("W", [90, 1 << 30])
def test_a_prompt_in_chunks_then_tokens(W):
    """Three sequences: prompt chunks through append, read and extend, then tokens
    through append and decode.  Every step against the definition on the same
    cache, whose contents are checked bit for bit as they grow."""
    rng = np.random.default_rng(60)
    B, MP, P, Hkv, G, D, scale = 3, 24, 16, 2, 3, 64, 0.125
    Hq, NB = Hkv * G, B * MP + 1
    pools = _tensors(B, MP, P, Hkv, D, NB)
    ref = [t.view(torch.uint8).cpu().numpy().copy() for t in pools]
    table = rng.permutation(NB)[: B * MP].reshape(B, MP).astype(np.int32)
    sinks = rng.uniform(-4, 8, Hq).astype(np.float32)
    tab, snk = _i32(table), torch.from_numpy(sinks).to(DEV)
    have = np.zeros(B, np.int64)

    def append(k, v, cu):
        swl.attn_sink_cache_append_fp8(k.to(DEV), v.to(DEV), tab, _i32(have), _i32(cu), *pools)
        cache8.append(inputs.bits(k), inputs.bits(v), table, have, cu, *ref)
        for g, r in zip(pools, ref):
            np.testing.assert_array_equal(g.view(torch.uint8).cpu().numpy(), r)

    for chunk in ([100, 33, 0], [64, 130, 1], [1, 90, 150]):
        cu = np.concatenate([[0], np.cumsum(chunk)])
        T = int(cu[-1])
        q = torch.from_numpy(rng.standard_normal((T, Hq, D))).bfloat16()
        k, v = (torch.from_numpy(rng.standard_normal((T, Hkv, D))).bfloat16() for _ in range(2))
        have += chunk
        append(k, v, cu)
        # the chunk's keys and what its window reaches before them, as the cache holds them
        span = np.where(np.array(chunk) > 0, np.minimum(have, np.array(chunk) + W - 1), 0)
        cu_k = np.concatenate([[0], np.cumsum(span)])
        kb, vb = (torch.empty(int(cu_k[-1]), Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        swl.attn_sink_cache_read_fp8(*pools, tab, _i32(have), _i32(cu_k), kb, vb)
        rk, rv = cache8.read(*ref, table, have, cu_k, int(cu_k[-1]))
        np.testing.assert_array_equal(kb.double().cpu().numpy(), rk)
        np.testing.assert_array_equal(vb.double().cpu().numpy(), rv)
        o, lse = _run(q, kb.cpu(), vb.cpu(), cu, cu_k, sinks, W, scale)
        ro, rl, mag, top = cache8.extend(inputs.bits(q), inputs.bits(kb.cpu()), inputs.bits(vb.cpu()), cu, cu_k, sinks,
                                         W, scale)
        assert (np.abs(o - ro) <= _tol(ro, mag, top, 400, D)).all()
        assert (np.abs(lse - rl) <= _tol_lse(rl, top, 400, D)).all()
    for _ in range(3):
        q = torch.from_numpy(rng.standard_normal((B, Hq, D))).bfloat16()
        k, v = (torch.from_numpy(rng.standard_normal((B, Hkv, D))).bfloat16() for _ in range(2))
        have += 1
        append(k, v, np.arange(B + 1))
        out = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=DEV)
        swl.attn_sink_decode_paged_fp8(q.to(DEV), *pools, tab, _i32(have), snk, W, scale, out)
        ro, mag, top = cache8.decode(inputs.bits(q), *ref, table, have, sinks, W, scale)
        assert (np.abs(out.double().cpu().numpy() - ro) <= _tol(ro, mag, top, 400, D)).all()
    assert swl.attn_sink_get_status() == 0


def test_captured_steps_replay_like_eager_ones():
    """append, read, extend and decode in one graph, and a second graph of the same
    calls; replayed in turn on refilled inputs, with an eager call between."""
    rng = np.random.default_rng(61)
    B, MP, P, Hkv, G, D, W = 3, 20, 16, 2, 4, 128, 100
    Hq = Hkv * G
    table = _i32(rng.permutation(B * MP).reshape(B, MP))
    cu, have = _i32([0, 30, 41, 42]), _i32([200, 11, 300])
    cu_k = _i32([0, 129, 140, 240])
    sinks = torch.randn(Hq, device=DEV)

    def state(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        pools = [t.view(torch.uint8).copy_(torch.randint(1, 100, t.shape, generator=g, device=DEV, dtype=torch.uint8)).
                 view(t.dtype) for t in _tensors(B, MP, P, Hkv, D, B * MP)]
        r = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
        return pools, r(42, Hkv, D), r(42, Hkv, D), r(42, Hq, D), r(B, Hq, D)

    def outputs():
        e = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        return e(240, Hkv, D), e(240, Hkv, D), e(42, Hq, D), torch.zeros(Hq, 42, device=DEV), e(B, Hq, D)

    def step(st, o, stream=None):
        pools, k, v, q, qd = st
        swl.attn_sink_cache_append_fp8(k, v, table, have, cu, *pools, stream=stream)
        swl.attn_sink_cache_read_fp8(*pools, table, have, cu_k, o[0], o[1], stream=stream)
        swl.attn_sink_fwd_extend(q, o[0], o[1], cu, cu_k, 30, sinks, W, 0.1, o[2], o[3], stream=stream)
        swl.attn_sink_decode_paged_fp8(qd, *pools, table, have, sinks, W, 0.1, o[4], stream=stream)

    st, outs = [state(1), state(2)], [outputs(), outputs()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(st[0], outs[0], side)
    torch.cuda.synchronize()
    graphs = []
    for s, o in zip(st, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(s, o, side)
        graphs.append(g)
    for turn in range(3):
        for i in (0, 1):
            new = state(10 + 2 * turn + i)
            for a, b in zip((*st[i][0], *st[i][1:]), (*new[0], *new[1:])):
                a.view(torch.uint8).copy_(b.view(torch.uint8))
            eager = outputs()
            step(new, eager)
            graphs[i].replay()
            torch.cuda.synchronize()
            for a, b in zip(outs[i], eager):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
            for a, b in zip(st[i][0], new[0]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert swl.attn_sink_get_status() == 0
