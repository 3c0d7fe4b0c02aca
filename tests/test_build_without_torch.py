"""The library needs nvcc only: on a machine without torch, g++ or Python's headers it is
built all the same, and the module beside it is left out."""
import importlib.metadata
import importlib.util
import os
import shutil
import sysconfig
import warnings

import pytest

from w4a16_moe_expert_sync_gb300 import build


@pytest.fixture
def built(monkeypatch, tmp_path):
    """What build() would compile, in order of its names."""
    seen = []
    monkeypatch.setattr(build, "_compile", lambda *a: seen.append("library"))
    monkeypatch.setattr(build, "_compile_calls", lambda: seen.append("module"))
    return seen


def _lack_torch(monkeypatch, tmp_path):
    find, version = importlib.util.find_spec, importlib.metadata.version

    def no_version(name):
        if name == "torch":
            raise importlib.metadata.PackageNotFoundError(name)
        return version(name)
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setattr(importlib.metadata, "version", no_version)


def _lack_gxx(monkeypatch, tmp_path):
    which = shutil.which
    monkeypatch.setattr(shutil, "which", lambda name, *a, **k: None if name == "g++" else
                        which(name, *a, **k))


def _lack_headers(monkeypatch, tmp_path):
    paths = sysconfig.get_paths
    monkeypatch.setattr(sysconfig, "get_paths",
                        lambda *a, **k: dict(paths(*a, **k), include=str(tmp_path)))


@pytest.mark.parametrize("lack", [_lack_torch, _lack_gxx, _lack_headers])
def test_the_library_is_built(built, monkeypatch, tmp_path, lack):
    lack(monkeypatch, tmp_path)
    with pytest.warns(UserWarning, match="only the library"):
        assert build.build(force=True) == build.LIB
    assert built == ["library"]


def test_both_are_built(built):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        build.build(force=True)
    assert sorted(built) == ["library", "module"]


def test_torch_without_metadata(monkeypatch):
    """A torch that is found but not installed as a package has a version all the same."""
    import torch

    def none(name):
        raise importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(importlib.metadata, "version", none)
    name = os.path.basename(build.calls_path())
    assert name.startswith("w4_calls_torch_") and name.endswith(".so")
    assert "".join(c if c.isalnum() else "_" for c in torch.__version__) in name


@pytest.mark.parametrize("lack", [_lack_torch, _lack_gxx, _lack_headers])
def test_the_build_entry_loads_what_was_built(built, monkeypatch, tmp_path, lack):
    import __graft_entry__
    import oracle
    import w4a16_moe_expert_sync_gb300 as w4
    from w4a16_moe_expert_sync_gb300 import _lib
    for module, name in ((oracle, "build"), (w4, "load_library"), (_lib, "_calls")):
        monkeypatch.setattr(module, name, lambda name=name: built.append(name))
    monkeypatch.setattr(build, "_stale", lambda *a: True)
    __graft_entry__.build()
    assert sorted(built) == ["_calls", "build", "library", "load_library", "module"]
    del built[:]
    lack(monkeypatch, tmp_path)
    with pytest.warns(UserWarning, match="only the library"):
        __graft_entry__.build()
    assert sorted(built) == ["build", "library", "load_library"]
