"""The order of the build, with commands in place of the compilers (no GPU, nothing
compiled): the C library is whole wherever hipcc works, and a binding that does not
compile is reported afterwards."""
import os
import subprocess

import pytest

from segmented_top_selection_amd import build as b


@pytest.fixture
def folder(tmp_path, monkeypatch):
    hipcc = tmp_path / "hipcc"  # writes its output's name into its output
    hipcc.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do\n  if [ "$1" = -o ]; then echo "$2" > "$2"; fi\n'
                     "  shift\ndone\n")
    hipcc.chmod(0o755)
    monkeypatch.setenv("HIPCC", str(hipcc))
    for name in ("LIB", "PROBE_LIB", "BINDING_LIB"):
        monkeypatch.setattr(b, name, str(tmp_path / name))
    monkeypatch.setattr(b, "OBJ_DIR", str(tmp_path / "objects"))
    return tmp_path


def test_the_library_is_linked_where_the_binding_does_not_compile(folder, monkeypatch):
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(subprocess.CalledProcessError) as e:
        b.build()
    assert e.value.cmd[0] == "false"
    assert (folder / "LIB").exists() and not (folder / "BINDING_LIB").exists()


def test_the_library_is_linked_where_there_is_no_compiler_for_the_binding(folder, monkeypatch):
    monkeypatch.setenv("CXX", str(folder / "missing"))
    with pytest.raises(OSError):
        b.build()
    assert (folder / "LIB").exists()


def test_the_library_is_linked_where_there_is_no_torch(folder, monkeypatch):
    def command(out):
        raise ImportError("no torch")
    monkeypatch.setattr(b, "binding_command", command)
    with pytest.raises(ImportError):
        b.build()
    assert (folder / "LIB").exists()


def test_a_source_that_does_not_compile_leaves_the_library_as_it_was(folder, monkeypatch):
    monkeypatch.setenv("CXX", str(folder / "hipcc"))
    assert b.build() == str(folder / "LIB") and (folder / "BINDING_LIB").exists()
    before = os.stat(folder / "LIB")
    monkeypatch.setenv("HIPCC", "false")
    with pytest.raises(subprocess.CalledProcessError):
        b.build()
    assert os.stat(folder / "LIB").st_mtime_ns == before.st_mtime_ns
