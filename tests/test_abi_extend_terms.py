"""attn_sink_fwd_extend_terms without a GPU: its own argument and those it shares with
attn_sink_fwd_extend are refused on the host."""
import ctypes

import pytest
import torch

import sliding_window_learned_b200 as swl
from sliding_window_learned_b200 import abi
from test_abi_cache import F32, I32, _t, lib  # noqa: F401


def _call(lib, terms, **over):  # noqa: F811
    a = dict(q=_t([50, 8, 128]), k=_t([90, 2, 128]), v=_t([90, 2, 128]), cq=_t([4], I32), ck=_t([4], I32), mq=50,
             s=_t([8], F32), W=100, scale=0.1, out=_t([50, 8, 128]), lse=_t([8, 50], F32))
    a.update(over)
    r = lambda n: ctypes.byref(a[n]) if a[n] is not None else None  # noqa: E731
    return lib.attn_sink_fwd_extend_terms(r("q"), r("k"), r("v"), r("cq"), r("ck"), a["mq"], r("s"), a["W"], a["scale"],
                                          terms, r("out"), r("lse"), None)


@pytest.mark.parametrize("terms", [-1, 3, 1 << 20])
def test_other_numbers_of_terms_are_refused(lib, terms):  # noqa: F811
    assert _call(lib, terms) == abi.ATTN_EINVAL
    assert "terms" in abi.attn_sink_last_error()


@pytest.mark.parametrize("over", [dict(W=0), dict(q=None), dict(v=_t([91, 2, 128])), dict(mq=-1), dict(ck=_t([5], I32))])
def test_the_shared_arguments_are_checked(lib, over):  # noqa: F811
    assert _call(lib, 1, **over) == abi.ATTN_EINVAL


@pytest.mark.parametrize("terms", [0, 1, 2])
def test_no_work_is_no_error(lib, terms):  # noqa: F811
    assert _call(lib, terms, mq=0) == abi.ATTN_OK


def test_host_tensors_are_refused():
    t = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="one CUDA device"):
        swl.attn_sink_fwd_extend_terms(t, t, t, t, t, 2, t, 5, 0.1, 1, t)
    with pytest.raises(TypeError):
        abi._binding().fwd_extend_terms(None)
