"""attn_sink_fwd_extend at sizes where the softmax's weights enter the product as one
bf16 term (more than 512 rows), with keys split and not, and with several units a CTA.

A call whose keys are split is one that needs workspace: it fails when the next
workspace allocation is made to fail.  Tolerances as in test_gpu_extend."""
import numpy as np
import pytest
import torch

import sliding_window_learned_b200 as swl
from oracle import cache8
from sliding_window_learned_b200 import inputs
from test_gpu_extend import DEV, _case, _i32, _run, _tol, _tol_lse

pytestmark = pytest.mark.gpu
FULL = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sliding_window_learned_b200 import build
    build.build()


def _is_split(q, k, v, cu_q, cu_k, sinks, W):
    swl.attn_sink_fail_workspace_allocs(1)
    try:
        swl.attn_sink_fwd_extend(q.to(DEV), k.to(DEV), v.to(DEV), _i32(cu_q), _i32(cu_k), int(np.diff(cu_q).max()),
                                 torch.from_numpy(sinks).to(DEV), W, 0.1, torch.empty_like(q, device=DEV))
        return False
    except swl.AttnSinkError as e:
        assert e.code == -4
        return True
    finally:
        swl.attn_sink_fail_workspace_allocs(0)


def _check(c, W, lk):
    q, k, v, cu_q, cu_k, sinks = c
    D, T = q.shape[2], int(cu_q[-1])
    assert q.shape[0] * q.shape[1] > 512
    ro, rl, mag, top = cache8.extend(inputs.bits(q), inputs.bits(k), inputs.bits(v), cu_q, cu_k, sinks, W, D ** -0.5)
    o, lse = _run(q, k, v, cu_q, cu_k, sinks, W, D ** -0.5)
    n = min(W, max(lk))
    assert (np.abs(o - ro) <= _tol(ro, mag, top, n, D))[:T].all(), np.abs(o - ro)[:T].max()
    assert (np.abs(lse - rl) <= _tol_lse(rl, top, n, D))[:, :T].all()
    assert (o[T:] == 9.0).all() and (lse[:, T:] == 9.0).all(), "rows of no sequence were written"
    return o, lse


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lq,lk,Hkv,G,W", [
    ([40], [4000], 2, 8, FULL), ([33, 0, 20], [3000, 70, 1900], 1, 16, 1700), ([100], [2500], 1, 7, FULL),
    ([60, 1], [30, 4000], 1, 9, FULL)])                        # (the first sequence sees fewer keys than it has rows)
def test_split_keys(lq, lk, Hkv, G, W, D):
    c = _case(70, lq, lk, Hkv, G, D)
    assert _is_split(*c, W)
    a = _check(c, W, lk)
    for x, y in zip(a, _run(*c, W, D ** -0.5)):
        np.testing.assert_array_equal(x, y)                    # the same every time


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lq,lk,Hkv,G,W", [
    ([300, 0, 70], [500, 40, 70], 1, 2, 129), ([90, 33], [100, 545], 2, 3, FULL), ([129, 1], [700, 66], 1, 8, 513),
    ([50, 7], [70, 900], 1, 16, FULL), ([200], [130], 1, 4, 64), ([20, 30], [0, 0], 2, 6, 7), ([9, 8], [70, 9], 1, 37, 60)])
def test_keys_that_are_not_split(lq, lk, Hkv, G, W, D):
    c = _case(71, lq, lk, Hkv, G, D)
    assert not _is_split(*c, W)
    _check(c, W, lk)


def _many(seed, D):
    """40 sequences of 16 kv heads: 640 tiles, at least two units for every CTA, of one to ten key tiles."""
    rng = np.random.default_rng(seed)
    lq = rng.integers(1, 31, 40)
    lk = np.maximum(rng.integers(0, 640, 40), rng.integers(0, 2, 40) * lq)
    lq[7], lk[8], lk[9] = 0, 0, 64
    return lq, lk, _case(seed, lq, lk, 16, 1, D)


@pytest.mark.parametrize("W", [100, FULL])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_several_units_a_cta(W, D):
    lq, lk, c = _many(72, D)
    assert not _is_split(*c, W)
    _check(c, W, lk)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("many", [False, True])
def test_other_sequences_values_stay_out(many, D):
    """NaN and infinities in the rows behind a sequence's last key, which share its last tile."""
    if many:
        lq, lk, (q, k, v, cu_q, cu_k, sinks) = _many(73, D)
    else:
        lq, lk = [40, 30, 9, 5], [70, 100, 9, 0]
        q, k, v, cu_q, cu_k, sinks = _case(73, lq, lk, 2, 8, D)
    assert q.shape[0] * q.shape[1] > 512
    good = _run(q, k, v, cu_q, cu_k, sinks, FULL, D ** -0.5)
    for b in range(1, len(lq), 2):
        rows = slice(int(cu_k[b]), int(cu_k[b + 1]))
        v[rows], k[rows] = float("nan") if b % 4 == 1 else float("inf"), float("nan")
    v[int(cu_k[-1]):] = float("inf")
    got = _run(q, k, v, cu_q, cu_k, sinks, FULL, D ** -0.5)
    for b in range(len(lq)):
        rows = slice(int(cu_q[b]), int(cu_q[b + 1]))
        if b % 2 == 0 or lk[b] == 0:
            np.testing.assert_array_equal(got[0][rows], good[0][rows])
            np.testing.assert_array_equal(got[1][:, rows], good[1][:, rows])
        else:
            sees = np.arange(lq[b]) + lk[b] - lq[b] >= 0
            assert np.isnan(got[0][rows][sees]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_other_sequences_values_stay_out_of_split_keys(D):
    lq, lk = [33, 30], [3001, 2900]
    q, k, v, cu_q, cu_k, sinks = _case(74, lq, lk, 1, 16, D)
    assert _is_split(q, k, v, cu_q, cu_k, sinks, FULL) and q.shape[0] * q.shape[1] > 512
    good = _run(q, k, v, cu_q, cu_k, sinks, FULL, D ** -0.5)
    v[3001:], k[3001:5901] = float("nan"), float("nan")
    got = _run(q, k, v, cu_q, cu_k, sinks, FULL, D ** -0.5)
    np.testing.assert_array_equal(got[0][:33], good[0][:33])
    np.testing.assert_array_equal(got[1][:, :33], good[1][:, :33])
    assert np.isnan(got[0][33:63]).all()
