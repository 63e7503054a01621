"""Pins of the 8-bit paged cache's double-precision definition (CPU only):
against torch's own number formats, the bf16 paged decode of the same values
and the packed forward, and with planted mistakes that each pin must catch."""
import numpy as np
import pytest
import torch

import oracle
from oracle import cache8
from sliding_window_learned_b200 import inputs


def test_code_table_is_torchs():
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(cache8.E4M3, ref)
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e8m0fnu).double().numpy()
    np.testing.assert_array_equal(cache8.scales(np.arange(256, dtype=np.uint8)), ref)


def _rows(seed, n=64, D=64):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, D, generator=g) * torch.exp2(torch.randint(-60, 60, (n, 1), generator=g).float())).bfloat16()


def test_quantise_is_torchs_rounding_of_the_scaled_row():
    x = _rows(1)
    codes, byte = cache8.quantise(inputs.bits(x))
    e = byte.astype(np.int64) - 127
    top = x.double().abs().amax(-1).numpy()
    assert (top <= 448 * 2.0 ** e).all() and (top > 448 * 2.0 ** (e - 1)).all()
    ref = (x.double() / torch.from_numpy(2.0 ** e)[:, None]).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(codes, ref)
    # an error of at most half a step
    back = cache8.E4M3[codes] * 2.0 ** e[:, None]
    xd = x.double().numpy()
    assert (np.abs(back - xd) <= np.maximum(2.0 ** -4 * np.abs(xd), 2.0 ** -10 * 2.0 ** e[:, None])).all()


def test_quantise_at_the_edges():
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(6, 64)
    x[1, :3] = torch.tensor([448.0, -449.0, 1.0])
    x[2, :3] = torch.tensor([inf, 1.0, -inf])
    x[3, :2] = torch.tensor([nan, 2.0])
    x[4, :2] = torch.tensor([3.38e38, 1.0])                # beyond 448 * 2^119
    x[5, :2] = torch.tensor([2.0 ** -130, 2.0 ** -126])    # subnormal range
    codes, byte = cache8.quantise(inputs.bits(x.bfloat16()))
    assert byte[0] == 10 and (codes[0] == 0).all()
    assert byte[1] == 128 - 1                              # bf16 rounds 449 to 448: e = 0
    assert byte[2] == 127 - 8 and codes[2, 0] == 0x7F and codes[2, 2] == 0x7F
    assert cache8.E4M3[codes[2, 1]] * 2.0 ** -8 == 1.0
    assert byte[3] == 127 - 7 and codes[3, 0] == 0x7F
    assert byte[4] == 246 and cache8.E4M3[codes[4, 0]] == 448
    assert byte[5] == 10 and cache8.E4M3[codes[5, 1]] == 2.0 ** -9


def _pool_case(seed, B=3, MP=5, P=16, Hq=4, Hkv=2, D=64):
    rng = np.random.default_rng(seed)
    seqlens = np.array([70, 1, 33])[:B]
    NB = B * MP + 2
    table = rng.permutation(NB)[: B * MP].reshape(B, MP).astype(np.int32)
    x = torch.from_numpy(rng.standard_normal((2, NB, P, Hkv, D)) * 2.0 ** rng.integers(-3, 4, (2, NB, P, Hkv, 1)))
    kp, ks = cache8.quantise(inputs.bits(x[0].bfloat16()))
    vp, vs = cache8.quantise(inputs.bits(x[1].bfloat16()))
    q = torch.from_numpy(rng.standard_normal((B, Hq, D))).bfloat16()
    sinks = rng.uniform(-4, 8, Hq).astype(np.float32)
    return inputs.bits(q), kp, vp, ks.transpose(0, 2, 1).copy(), vs.transpose(0, 2, 1).copy(), table, seqlens, sinks


def _as_bf16(codes, byte):
    x = cache8.E4M3[codes] * cache8.scales(byte.transpose(0, 2, 1))[..., None]
    t = torch.from_numpy(x).bfloat16()
    assert (t.double().numpy() == x).all()                 # exact: what the read returns
    return inputs.bits(t)


@pytest.mark.parametrize("W", [1, 20, 1000])
def test_decode_equals_the_bf16_paged_decode_of_the_same_values(W):
    q, kp, vp, ks, vs, table, sl, sinks = _pool_case(5)
    ref, _ = oracle.decode_paged(q, _as_bf16(kp, ks), _as_bf16(vp, vs), table, sl, sinks, W, 0.125)
    got = cache8.decode(q, kp, vp, ks, vs, table, sl, sinks, W, 0.125)[0]
    np.testing.assert_allclose(got, ref, rtol=1e-12, atol=1e-13)
    # planted: value scales left out, a key scale off by one, the window off by one
    for bad in (cache8.decode(q, kp, vp, ks, np.full_like(vs, 127), table, sl, sinks, W, 0.125)[0],
                cache8.decode(q, kp, vp, ks + 1, vs, table, sl, sinks, W, 0.125)[0],
                cache8.decode(q, kp, vp, ks, vs, table, sl, sinks, W + 1, 0.125)[0] if W < 70 else ref + 1):
        assert np.abs(bad - ref).max() > 1e-3


def test_append_then_read_is_the_rounded_rows():
    _, kp, vp, ks, vs, table, _, _ = _pool_case(6)
    cu, sl = np.array([0, 40, 40, 57]), np.array([60, 9, 17])
    rng = np.random.default_rng(7)
    k = torch.from_numpy(rng.standard_normal((60, 2, 64))).bfloat16()
    v = torch.from_numpy(rng.standard_normal((60, 2, 64))).bfloat16()
    before = kp.copy()
    cache8.append(inputs.bits(k), inputs.bits(v), table, sl, cu, kp, vp, ks, vs)
    assert (kp != before).any(axis=(1, 2, 3)).sum() == 3 + 2     # pages 1-3 of sequence 0 (positions 20..59), two of sequence 2
    rk, rv = cache8.read(kp, vp, ks, vs, table, sl, cu, 60)
    c, s = cache8.quantise(inputs.bits(k))
    np.testing.assert_array_equal(rk[:57], (cache8.E4M3[c] * cache8.scales(s)[..., None])[:57])
    assert np.isnan(rk[57:]).all() and np.isfinite(rv[:57]).all()


def test_extend_without_earlier_keys_is_the_packed_forward():
    rng = np.random.default_rng(8)
    cu = np.array([0, 17, 17, 40])
    q = inputs.bits(torch.from_numpy(rng.standard_normal((40, 4, 64))).bfloat16())
    k, v = (inputs.bits(torch.from_numpy(rng.standard_normal((40, 2, 64))).bfloat16()) for _ in range(2))
    sinks = rng.uniform(-4, 8, 4).astype(np.float32)
    ro, rl = oracle.fwd_varlen(q, k, v, cu, sinks, 9, 0.125)
    o, lse, _, _ = cache8.extend(q, k, v, cu, cu, sinks, 9, 0.125)
    np.testing.assert_allclose(o, ro, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(lse, rl, rtol=1e-12)


def test_extend_continues_the_packed_forward():
    """The last rows of a sequence as a chunk give the whole forward's last rows;
    a chunk longer than its keys has rows that see nothing."""
    rng = np.random.default_rng(9)
    L, n = 50, 13
    q = inputs.bits(torch.from_numpy(rng.standard_normal((L, 2, 64))).bfloat16())
    k, v = (inputs.bits(torch.from_numpy(rng.standard_normal((L, 1, 64))).bfloat16()) for _ in range(2))
    sinks = np.array([1.0, -2.0], np.float32)
    ro, rl = oracle.fwd_varlen(q, k, v, np.array([0, L]), sinks, 20, 0.125)
    o, lse, _, _ = cache8.extend(q[L - n:], k, v, [0, n], [0, L], sinks, 20, 0.125)
    np.testing.assert_allclose(o, ro[L - n:], rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(lse, rl[:, L - n:], rtol=1e-12)
    o, lse, _, _ = cache8.extend(q[:n], k[:4], v[:4], [0, n], [0, 4], sinks, 20, 0.125)
    assert (o[:9] == 0).all() and (lse[:, :9] == sinks[:, None]).all() and (o[9:] != 0).any()
