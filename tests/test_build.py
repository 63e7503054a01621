"""The build step: the library does not need the binding's tools, and a binding built
against another torch is built again, or refused."""
import os

import pytest
import torch

from sliding_window_learned_b200 import abi, build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("stale", [False, True])
def test_the_library_is_built_where_the_binding_cannot_be(monkeypatch, stale):
    done = []

    def no_compiler(force=False):
        raise RuntimeError("binding build failed: no g++")

    monkeypatch.setattr(build, "_stale", lambda: stale)
    monkeypatch.setattr(build, "_build_library", lambda verbose: done.append(verbose), raising=False)
    monkeypatch.setattr(build, "build_binding", no_compiler)
    with pytest.warns(RuntimeWarning, match="no g\\+\\+"):
        assert build.build() == build.LIB
    assert len(done) == stale


class _Ran(Exception):
    pass


@pytest.fixture
def copy(monkeypatch, tmp_path):
    """The present binding under other paths, with a compiler that only says that it was called."""
    so, stamp = tmp_path / "_binding.so", tmp_path / "_build" / "binding.txt"
    stamp.parent.mkdir()
    so.write_bytes(b"")
    stamp.write_text(build.binding_for())
    monkeypatch.setattr(build, "BINDING", str(so))
    monkeypatch.setattr(build, "BINDING_STAMP", str(stamp))

    def run(*a, **k):
        raise _Ran

    monkeypatch.setattr(build.subprocess, "run", run)
    return so, stamp


def test_a_fresh_binding_is_kept(copy):
    assert build.build_binding() == str(copy[0])


def test_another_torch_builds_the_binding_again(copy, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "2.12.0+cu130")
    with pytest.raises(_Ran):
        build.build_binding()


def test_a_binding_of_unknown_origin_is_built_again(copy):
    copy[1].unlink()
    with pytest.raises(_Ran):
        build.build_binding()


def test_an_older_binding_is_built_again(copy):
    os.utime(copy[0], (0, 0))
    with pytest.raises(_Ran):
        build.build_binding()


def test_no_old_binding_stays_behind_a_failed_build(copy, monkeypatch):
    def none(*a, **k):
        raise FileNotFoundError("g++")

    monkeypatch.setattr(build.subprocess, "run", none)
    with pytest.raises(RuntimeError, match="binding build failed"):
        build.build_binding(force=True)
    assert not copy[0].exists()


def test_a_binding_for_another_torch_is_not_loaded(monkeypatch):
    monkeypatch.setattr(abi, "_native", None)
    assert abi._binding().built_for == build.binding_for()
    monkeypatch.setattr(abi, "_native", None)
    monkeypatch.setattr(torch, "__version__", "2.12.0+cu130")
    with pytest.raises(ImportError, match="was built for torch"):
        abi._binding()
