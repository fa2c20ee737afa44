"""CPU checks of the build where the extension module cannot be compiled, and of the
binding beside an extension module of another version."""

import os
import subprocess
import types

import pytest
import torch

from block_sparse_local_nb_b200 import binding, build


@pytest.mark.parametrize("how", ["no headers", "no compiler"])
def test_the_library_is_built_without_the_extension_module(how, tmp_path, monkeypatch):
    """Nothing of an earlier extension module stays, and the build says what will happen."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "CALL", str(tmp_path / "_call.so"))
    (tmp_path / "_call.so").write_text("an earlier one")
    monkeypatch.setattr(build, "_compile", lambda src, info: (src, ""))

    def run(cmd, **kw):
        if "nvcc" in cmd[0]:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("the library")
            return subprocess.CompletedProcess(cmd, 0, "", "")
        if how == "no compiler":
            raise FileNotFoundError(cmd[0])
        return subprocess.CompletedProcess(cmd, 1, "", "Python.h: No such file or directory")

    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.warns(UserWarning, match="ctypes"):
        assert build.build() == str(tmp_path / "lib.so")
    assert (tmp_path / "lib.so").read_text() == "the library"
    assert not os.path.exists(tmp_path / "_call.so")


@pytest.mark.parametrize("version", [None, -1, 0])  # without one, older, this one
def test_an_extension_module_of_another_version_is_not_called(built_lib, version, monkeypatch):
    import sys

    called = []
    stale = types.ModuleType("block_sparse_local_nb_b200._call")
    stale.nb_kv4_write = lambda *a: called.append(a) or 0
    if version is not None:
        stale.abi_version = built_lib.nb_abi_version() + version
    monkeypatch.setattr(binding, "_entries", {})
    monkeypatch.setitem(sys.modules, "block_sparse_local_nb_b200._call", stale)
    monkeypatch.setattr(sys.modules["block_sparse_local_nb_b200"], "_call", stale, raising=False)
    t = torch.empty(64)
    status = binding.nb_kv4_write(t, t, t, t, None, None, 1, 1, 1, 63, 4, 9, 1, stream=0, check=False)
    assert (status, len(called)) == ((0, 1) if version == 0 else (-2, 0))


def test_the_extension_module_has_the_library_s_version(built_lib):
    if not os.path.exists(build.CALL):
        build._build_call()
    from block_sparse_local_nb_b200 import _call

    assert _call.abi_version == built_lib.nb_abi_version()
