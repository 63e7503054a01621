"""The C++ marshalling of the serving calls, without a GPU: what is not a tensor
on one CUDA device is refused before the library sees it."""
import pytest
import torch

import sliding_window_learned_b200 as swl
from sliding_window_learned_b200 import abi


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sliding_window_learned_b200 import build
    build.build()


def _args():
    t = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    return [t] * 9


@pytest.mark.parametrize("call", [
    lambda a: swl.attn_sink_cache_append_fp8(*a), lambda a: swl.attn_sink_cache_read_fp8(*a),
    lambda a: swl.attn_sink_decode_paged_fp8(*a[:8], 5, 0.1, a[8]),
    lambda a: swl.attn_sink_fwd_extend(*a[:5], 2, a[5], 5, 0.1, a[6], a[7])])
def test_host_tensors_and_other_objects_are_refused(call):
    with pytest.raises(ValueError, match="one CUDA device"):
        call(_args())
    for bad in (None, 3, "x"):
        with pytest.raises(TypeError):
            call([bad] + _args()[1:])


def test_wrong_numbers_of_arguments_are_refused():
    native = abi._binding()
    for name in ("cache_append", "cache_read", "decode_paged", "fwd_extend"):
        with pytest.raises(TypeError):
            getattr(native, name)(None)


def test_a_missing_binding_is_named(monkeypatch):
    import builtins
    real = builtins.__import__

    def no_binding(name, *a, **k):
        if a and a[2] and "_binding" in a[2]:
            raise ImportError("no such file")
        return real(name, *a, **k)

    monkeypatch.setattr(abi, "_native", None)
    monkeypatch.setattr(builtins, "__import__", no_binding)
    with pytest.raises(ImportError, match="_binding.so is not built"):
        abi._binding()
