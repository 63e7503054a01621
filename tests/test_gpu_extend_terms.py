"""attn_sink_fwd_extend_terms: the number of bf16 terms of the softmax's weights, said by
the caller, against the definition.  Tolerances as in test_gpu_extend, less the
weights' rounding where they have two terms (2^-8 the rest, and 2^-8 of that)."""
import numpy as np
import pytest
import torch

import sliding_window_learned_b200 as swl
from oracle import cache8
from sliding_window_learned_b200 import inputs
from test_gpu_extend import DEV, _case, _i32, _tol, _tol_lse

pytestmark = pytest.mark.gpu
FULL = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sliding_window_learned_b200 import build
    build.build()


def _run(q, k, v, cu_q, cu_k, sinks, W, scale, terms):
    out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((q.shape[1], q.shape[0]), 9.0, device=DEV)
    args = (q.to(DEV), k.to(DEV), v.to(DEV), _i32(cu_q), _i32(cu_k), int(np.diff(cu_q).max()),
            torch.from_numpy(sinks).to(DEV), W, scale)
    if terms is None:
        swl.attn_sink_fwd_extend(*args, out, lse)
    else:
        swl.attn_sink_fwd_extend_terms(*args, terms, out, lse)
    torch.cuda.synchronize()
    assert swl.attn_sink_get_status() == 0
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


@pytest.mark.parametrize("terms", [1, 2])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lq,lk,Hkv,G,W", [
    ([3, 1], [1000, 70], 1, 16, 513), ([40], [4000], 2, 8, FULL), ([200, 0, 70], [300, 5, 70], 1, 8, 129),
    ([20, 9] * 40, [70, 9] * 40, 8, 1, FULL)])
def test_either_number_of_terms_at_any_size(lq, lk, Hkv, G, W, D, terms):
    c = _case(80, lq, lk, Hkv, G, D)
    q, k, v, cu_q, cu_k, sinks = c
    ro, rl, mag, top = cache8.extend(inputs.bits(q), inputs.bits(k), inputs.bits(v), cu_q, cu_k, sinks, W, D ** -0.5)
    o, lse = _run(*c, W, D ** -0.5, terms)
    n, T = min(W, max(lk)), int(cu_q[-1])
    tol = _tol(ro, mag, top, n, D) - (terms == 2) * (2.0 ** -8 - 2.0 ** -16) * mag * 1.01
    assert (np.abs(o - ro) <= tol)[:T].all(), (np.abs(o - ro) / tol)[:T].max()
    assert (np.abs(lse - rl) <= _tol_lse(rl, top, n, D))[:, :T].all()
    assert (o[T:] == 9.0).all() and (lse[:, T:] == 9.0).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_row_does_not_depend_on_the_rows_beside_it(D):
    """One sequence alone and beside others (few keys: nothing is split), the same bits
    with one term and with two; without a say two up to 512 rows and one above."""
    lq, lk, Hkv, G = [20, 50, 33], [300, 90, 400], 1, 8
    q, k, v, cu_q, cu_k, sinks = _case(81, lq, lk, Hkv, G, D, tail=(0, 0))
    first = (q[:20], k[:300], v[:300], cu_q[:2], cu_k[:2], sinks)
    assert 20 * G <= 512 < q.shape[0] * G
    together, alone = {}, {}
    for terms in (None, 0, 1, 2):
        together[terms] = _run(q, k, v, cu_q, cu_k, sinks, FULL, 0.2, terms)
        alone[terms] = _run(*first, FULL, 0.2, terms)
    for terms in (1, 2):
        np.testing.assert_array_equal(together[terms][0][:20], alone[terms][0])
        np.testing.assert_array_equal(together[terms][1][:, :20], alone[terms][1])
    for terms in (None, 0):
        np.testing.assert_array_equal(together[terms][0], together[1][0])
        np.testing.assert_array_equal(alone[terms][0], alone[2][0])
    assert (alone[1][0] != alone[2][0]).any()
