"""The build without what only the tensor layer needs: the C library is built all the same, and an extension module of
earlier sources does not stay behind. A stand-in for hipcc that only makes its output files; nothing in the tree is
touched."""

import stat
import types

import pytest

from fp8_fine_grained_fp8bq_amd import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    fake = tmp_path / "hipcc"
    fake.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\n: > "$2"\n')
    fake.chmod(fake.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("HIPCC", str(fake))
    for name, file in (("PKG", ""), ("LIB", "libfp8bq.so"), ("PROBE_LIB", "libfp8bq_probe.so"), ("TENSORS_LIB", "_tensors.so")):
        monkeypatch.setattr(b, name, str(tmp_path / file) if file else str(tmp_path))
    (tmp_path / "_tensors.so").write_text("earlier")
    return tmp_path


@pytest.mark.parametrize("missing", ["torch", "torch for ROCm", "g++"])
def test_the_c_library_is_built_without(missing, tree, monkeypatch, capfd):
    if missing == "torch":
        monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    elif missing == "torch for ROCm":
        monkeypatch.setattr(b.importlib.util, "find_spec",
                            lambda name: types.SimpleNamespace(submodule_search_locations=[str(tree)]))
    else:
        (tree / "lib").mkdir()
        (tree / "lib" / "libc10_hip.so").write_text("")
        monkeypatch.setattr(b.importlib.util, "find_spec",
                            lambda name: types.SimpleNamespace(submodule_search_locations=[str(tree)]))
        monkeypatch.setattr(b.shutil, "which", lambda name: None)
    assert b.build() == str(tree / "libfp8bq.so")
    assert (tree / "libfp8bq.so").exists() and (tree / "libfp8bq_probe.so").exists()
    assert not (tree / "_tensors.so").exists()
    assert "_tensors.so not built" in capfd.readouterr().err


def test_the_extension_is_built_where_torch_is():
    pytest.importorskip("torch")
    cmd = b.tensors_command("out.so")
    if not cmd:
        pytest.skip("no torch for ROCm or no g++ here")
    assert cmd[0] == "g++" and "out.so" in cmd and "-l:libfp8bq.so" in cmd
