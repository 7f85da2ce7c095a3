"""The build script with stand-in compilers: what is put in place when a part does not build."""
import os
import stat

import pytest

from fp8_mqa_logits_02_gb300 import nvcc_build


def compiler(path, fails=False):
    """A program that writes the file after -o, or fails."""
    path.write_text("#!/bin/sh\necho \"ran $0\"\n" + ("exit 1\n" if fails else
                    'while [ $# -gt 0 ]; do [ "$1" = -o ] && echo built > "$2"; shift; done\n'))
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


@pytest.fixture
def place(tmp_path, monkeypatch):
    for name in ("LIB", "DEBUG_LIB", "BINDING"):
        monkeypatch.setattr(nvcc_build, name, str(tmp_path / name))
    monkeypatch.setattr(nvcc_build, "nvcc_path", lambda: compiler(tmp_path / "nvcc"))
    monkeypatch.setenv("CXX", compiler(tmp_path / "cxx"))
    return tmp_path


def built(place):
    left = {p.name for p in place.iterdir()} - {"nvcc", "cxx"}
    assert left <= {"LIB", "DEBUG_LIB", "BINDING"}      # no temporaries
    return left


def test_everything_builds(place):
    assert nvcc_build.build() == nvcc_build.LIB
    assert built(place) == {"LIB", "DEBUG_LIB", "BINDING"}


@pytest.mark.parametrize("why", ["fails", "missing", "torch"])
def test_without_the_binding_the_libraries_are_there(place, why, monkeypatch):
    # a host compiler or torch headers that are not there: the C library needs neither
    (place / "BINDING").write_text("of other sources")
    os.utime(place / "BINDING", (0, 0))
    if why == "fails":
        compiler(place / "cxx", fails=True)
    elif why == "missing":
        monkeypatch.setenv("CXX", str(place / "no-such-compiler"))
    else:
        def gone():
            raise ImportError("no torch")
        monkeypatch.setattr(nvcc_build, "torch_dir", gone)
    with pytest.warns(UserWarning, match="paged operators are not available"):
        assert nvcc_build.build() == nvcc_build.LIB
    assert built(place) == {"LIB", "DEBUG_LIB"}


def test_a_library_that_does_not_build_raises(place, monkeypatch):
    monkeypatch.setattr(nvcc_build, "nvcc_path", lambda: compiler(place / "nvcc", fails=True))
    with pytest.raises(RuntimeError, match="compiling LIB"):
        nvcc_build.build()
    assert built(place) == {"BINDING"}


def test_only_one_library(place):
    assert nvcc_build.build(debug=False) == nvcc_build.LIB
    assert built(place) == {"LIB", "BINDING"}
    assert nvcc_build.build(debug=True) == nvcc_build.DEBUG_LIB
    assert built(place) == {"LIB", "DEBUG_LIB", "BINDING"}
