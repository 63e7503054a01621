"""Decode over the 8-bit pages at the ends of its formats: scales that the append
may write (2^-117 .. 2^119) and queries that bring the logits back into range.
Each case in both forms, sequences finished whole and sequences cut over the SMs.
Tolerance as in test_gpu_cache_fp8."""
import numpy as np
import pytest
import torch

import sliding_window_learned_b200 as swl
from oracle import cache8
from sliding_window_learned_b200 import inputs
from test_gpu_cache_fp8 import DEV, _decode, _decode_case, _i32, _pools, _tol

pytestmark = pytest.mark.gpu
FULL = 1 << 30
FORMS = {"whole": ([500, 70, 193], 8, 64, 2, 4, 128), "whole, narrow": ([1000, 70], 16, 64, 1, 12, 64),
         "cut": ([1400, 70, 0, 900], 24, 64, 2, 4, 128),
         "cut, many parts": ([9000], 141, 64, 1, 2, 64), "cut, wide": ([700, 1, 640], 44, 16, 2, 3, 256)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sliding_window_learned_b200 import build
    build.build()


def _check(c, W, scale, n):
    D = c[0].shape[2]
    ref, mag, top = cache8.decode(inputs.bits(c[0]), *c[1:], W, scale)
    got = _decode(*c, W, scale)
    assert np.isfinite(ref).all() and np.isfinite(got).all()
    bad = ~(np.abs(got - ref) <= _tol(ref, mag, top, n, D))
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])
    return got


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("form", FORMS)
def test_the_largest_values(form, sink):
    """Value rows of up to 448 * 2^119: their sum passes f32, their mean does not."""
    seqlens, MP, P, Hkv, G, D = FORMS[form]
    c = list(_decode_case(31, seqlens, MP, P, Hkv, G, D, FULL))
    c[4] = np.where(c[4] == 255, 255, 246).astype(np.uint8)
    c[2] &= 0x7F                                           # (one sign: the mean is large)
    if not sink:
        c[7][:] = -np.inf
    got = _check(c, FULL, D ** -0.5, max(seqlens))
    assert sink or got.max() > 2.0 ** 124


@pytest.mark.parametrize("form", FORMS)
def test_the_smallest_values(form):
    seqlens, MP, P, Hkv, G, D = FORMS[form]
    c = list(_decode_case(32, seqlens, MP, P, Hkv, G, D, FULL))
    c[4] = np.where(c[4] == 255, 255, 10).astype(np.uint8)
    c[7][:] = -np.inf
    ref, mag, top = cache8.decode(inputs.bits(c[0]), *c[1:], FULL, D ** -0.5)
    got = _decode(*c, FULL, D ** -0.5)
    # (bf16's own subnormals start at 2^-126, their half step is 2^-134)
    assert (np.abs(got - ref) <= _tol(ref, mag, top, max(seqlens), D) - 1e-37 + 2.0 ** -134).all()


@pytest.mark.parametrize("key,query,scale", [
    (246, -121, None), (246, -126, None), (230, -104, None), (10, 116, None), (10, 118, None), (10, 124, 2.0 ** -10),
    (246, -121, 2.0 ** -3), (246, -110, 2.0 ** -14), (246, -121, 3.0), (60, 40, 2.0 ** 20), (246, -60, 2.0 ** -62)])
@pytest.mark.parametrize("form", FORMS)
def test_keys_and_queries_of_opposite_sizes(form, key, query, scale):
    """Scale bytes at the ends of the append's range, queries that make ordinary logits of them."""
    seqlens, MP, P, Hkv, G, D = FORMS[form]
    c = list(_decode_case(33, seqlens, MP, P, Hkv, G, D, FULL))
    rng = np.random.default_rng(34)
    low = rng.integers(-3, 1, c[3].shape) if key > 13 else rng.integers(0, 4, c[3].shape)
    c[3] = np.where(c[3] == 255, 255, key + low).astype(np.uint8)
    c[0] = torch.from_numpy(rng.standard_normal(c[0].shape) * 2.0 ** (query - 3)).bfloat16()
    _check(c, FULL, D ** -0.5 if scale is None else scale, max(seqlens))


def test_ordinary_heads_beside_extreme_ones():
    """One group's heads of queries from 2^-124 to 2^15 (logits of 2^21, which single out a key) over ordinary keys."""
    seqlens, MP, P, Hkv, G, D = [500, 70, 193], 8, 64, 1, 8, 128
    c = list(_decode_case(35, seqlens, MP, P, Hkv, G, D, FULL))
    rng = np.random.default_rng(36)
    q = rng.standard_normal(c[0].shape) * 2.0 ** np.array([-124, -63, -23, -3, -2, -1, 14, 15])[None, :, None]
    c[0] = torch.from_numpy(q).bfloat16()
    ref, mag, top = cache8.decode(inputs.bits(c[0]), *c[1:], FULL, D ** -0.5)
    got = _decode(*c, FULL, D ** -0.5)
    assert np.isfinite(got).all() and top[:, 7].max() > 2.0 ** 20
    assert (np.abs(got - ref) <= _tol(ref, mag, top, 500, D))[:, :6].all()


@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("at", [3, 62, -2])
@pytest.mark.parametrize("form", FORMS)
def test_one_key_far_above_the_others(form, at, sink):
    """One key's logit is 2^9 .. 2^25 (in powers of two), the others' at most a seventh of it:
    the output is that key's value row.  Exactly: the weight's rounding, 2^-11, is less than
    half a bf16 step, and a row of codes needs no more than four of bf16's eight bits."""
    seqlens, MP, P, Hkv, G, D = FORMS[form]
    c = list(_decode_case(38, seqlens, MP, P, Hkv, G, D, FULL))
    rng = np.random.default_rng(39)
    c[4] = np.where(c[4] == 255, 255, rng.integers(120, 134, c[4].shape)).astype(np.uint8)
    c[3] = np.where(c[3] == 255, 255, 127).astype(np.uint8)
    c[1] = np.where(c[1] == 0x7F, c[1], (c[1] & 0x80) | np.minimum(c[1] & 0x7F, 0x5F)).astype(np.uint8)   # |k| <= 60
    if not sink:
        c[7][:] = -np.inf
    sign = rng.integers(0, 2, (Hkv, D))
    t = at % seqlens[0]
    page, pos = int(c[5][0, t // P]), t % P
    c[1][page, pos] = 0x7E | (sign << 7).astype(np.uint8)                                                 # |k| = 448
    want = cache8.E4M3[c[2][page, pos]] * cache8.scales(c[4][page, :, pos])[:, None]
    dirs = np.repeat(1.0 - 2.0 * sign, G, 0)
    for log in range(9, 26):
        c[0][0] = torch.from_numpy(dirs * 2.0 ** log * np.log(2) / 448 / D).bfloat16()
        got = _decode(*c, FULL, 1.0)[0]
        np.testing.assert_array_equal(got, np.repeat(want, G, 0), err_msg=str(log))


def test_rows_read_back_at_the_ends_of_the_range_are_the_values_decoded():
    """Appended rows near bf16's ends, read back and decoded with one key visible: the
    decode gives that key's values exactly (no sink)."""
    rng = np.random.default_rng(37)
    Hkv, D, P = 2, 128, 16
    T = 16
    k = torch.zeros(T, Hkv, D, dtype=torch.bfloat16)
    v = torch.from_numpy(rng.standard_normal((T, Hkv, D)) * 2.0 ** rng.integers(-120, 124, (T, Hkv, 1))).bfloat16()
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=DEV)  # noqa: E731
    pools = (z(T, P, Hkv, D).view(e4), z(T, P, Hkv, D).view(e4), z(T, Hkv, P).view(e8), z(T, Hkv, P).view(e8))
    table, one, cu = _i32(np.arange(T)[:, None]), _i32([1] * T), _i32(np.arange(T + 1))
    swl.attn_sink_cache_append_fp8(k.to(DEV), v.to(DEV), table, one, cu, *pools)
    kb, vb = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
    swl.attn_sink_cache_read_fp8(*pools, table, one, cu, kb, vb)
    out = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
    q = torch.randn(T, Hkv, D, device=DEV).bfloat16()
    swl.attn_sink_decode_paged_fp8(q, *pools, table, one, torch.full((Hkv,), -float("inf"), device=DEV), 1, 0.1, out)
    assert torch.equal(out, vb)
