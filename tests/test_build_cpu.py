"""The build without the compiled part of the binding: what keeps g++ from building it is no
reason not to build the library.  (nvcc is a script that writes empty files here.)"""
import os
import shutil
import stat

import pytest
import torch

from layout_folding_gb300 import build as lfbuild


@pytest.fixture
def place(monkeypatch, tmp_path):
    """A build folder of its own, with headers that are there and an nvcc that always succeeds."""
    nvcc = shutil.which(lfbuild.NVCC)
    if nvcc is None or lfbuild._binding_command("out") is None:
        pytest.skip("no headers of PyTorch, Python or CUDA here")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    (tmp_path / "cuda" / "bin").mkdir(parents=True)
    os.symlink(include, tmp_path / "cuda" / "include")
    script = tmp_path / "cuda" / "bin" / "nvcc"
    script.write_text('#!/bin/sh\nwhile [ $# -gt 1 ]; do [ "$1" = -o ] && : > "$2"; shift; done\n')
    script.chmod(script.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(lfbuild, "NVCC", str(script))
    monkeypatch.setattr(lfbuild, "OBJ_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(lfbuild, "LIB_DIR", str(tmp_path / "lib"))
    for name in ("LIB_PATH", "BINDING_PATH"):
        monkeypatch.setattr(lfbuild, name, str(tmp_path / "lib" / os.path.basename(getattr(lfbuild, name))))
    return tmp_path


def compiler(place, text):
    path = place / "cxx"
    path.write_text("#!/bin/sh\n" + text)
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


def files(place):
    return sorted(os.listdir(place / "lib"))


@pytest.mark.parametrize("cxx", ["/nonexistent/g++", "fails"])
def test_the_library_is_built_without_the_binding(place, monkeypatch, capfd, cxx):
    monkeypatch.setenv("CXX", compiler(place, "echo no such header >&2; exit 1\n") if cxx == "fails" else cxx)
    library, binding = os.path.basename(lfbuild.LIB_PATH), os.path.basename(lfbuild.BINDING_PATH)
    assert lfbuild.build() == lfbuild.LIB_PATH
    assert files(place) == [library]
    said = capfd.readouterr().err
    assert "the compiled part of the binding is not built" in said and ("no such header" in said) == (cxx == "fails")
    # one of an earlier build that could not be renewed goes; one that is up to date stays
    (place / "lib" / binding).write_text("old")
    lfbuild.build()
    assert files(place) == sorted([library, binding])
    lfbuild.build(force=True)
    assert files(place) == [library]


def test_only_what_is_out_of_date_is_built(place, monkeypatch):
    monkeypatch.setenv("CXX", compiler(place, 'while [ $# -gt 1 ]; do [ "$1" = -o ] && echo new > "$2"; shift; done\n'))
    assert not lfbuild.up_to_date()
    lfbuild.build()
    assert len(files(place)) == 2 and lfbuild.up_to_date()
    before = os.stat(lfbuild.LIB_PATH).st_mtime_ns
    os.remove(lfbuild.BINDING_PATH)
    assert not lfbuild.up_to_date()
    lfbuild.build()
    assert len(files(place)) == 2 and lfbuild.up_to_date() and os.stat(lfbuild.LIB_PATH).st_mtime_ns == before


def test_a_binding_for_another_torch_or_python_is_not_taken(place, monkeypatch):
    monkeypatch.setenv("CXX", compiler(place, 'while [ $# -gt 1 ]; do [ "$1" = -o ] && echo new > "$2"; shift; done\n'))
    lfbuild.build()
    other = os.path.basename(lfbuild.BINDING_PATH).replace(torch.__version__, "0.0.1")
    os.rename(lfbuild.BINDING_PATH, place / "lib" / other)
    assert other in files(place) and not lfbuild.up_to_date()
    lfbuild.build()
    assert lfbuild.up_to_date() and os.path.exists(lfbuild.BINDING_PATH) and other not in files(place)


def test_one_that_is_out_of_date_goes_where_none_can_be_built(place, monkeypatch):
    monkeypatch.setattr(lfbuild, "_binding_command", lambda out: None)  # (no headers)
    lfbuild.build()
    assert len(files(place)) == 1 and lfbuild.up_to_date()
    binding = place / "lib" / os.path.basename(lfbuild.BINDING_PATH)
    binding.write_text("old")
    os.utime(binding, (1, 1))
    assert not lfbuild.up_to_date()
    lfbuild.build()
    assert len(files(place)) == 1 and lfbuild.up_to_date()


def test_a_library_that_does_not_build_is_an_error(place, monkeypatch):
    monkeypatch.setenv("CXX", "/nonexistent/g++")
    script = place / "cuda" / "bin" / "nvcc"
    script.write_text("#!/bin/sh\nexit 1\n")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        lfbuild.build()
    assert not os.path.exists(lfbuild.LIB_PATH)
