"""The build's own logic, with a stand-in for nvcc that writes empty outputs: the library needs
nothing but nvcc, the Python module needs Python's headers and belongs to one Python."""
import os
import stat
import sysconfig

import pytest

import paged_kv_attention_photon_gb300 as P
from paged_kv_attention_photon_gb300 import _build as B

FAKE_NVCC = """#!/bin/sh
# notes its arguments; fails on the Python module if there is no Python.h on the include path
echo "$@" >> "$NVCC_LOG"
out= ; prev= ; binding= ; header=
for a in "$@"; do
  [ "$prev" = "-o" ] && out="$a"
  case "$a" in
    *binding.cpp) binding=1 ;;
    -I*) [ -e "${a#-I}/Python.h" ] && header=1 ;;
  esac
  prev="$a"
done
if [ -n "$binding" ] && [ -z "$header" ]; then echo "Python.h: No such file" >&2; exit 1; fi
if [ -n "$binding" ] && [ -n "$NVCC_BAD_BINDING" ]; then echo "error in binding.cpp" >&2; exit 1; fi
: > "$out"
"""


@pytest.fixture
def place(tmp_path, monkeypatch):
    """The build's outputs in a folder of their own; returns (that folder, the calls so far)."""
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(FAKE_NVCC)
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    log = tmp_path / "log"
    monkeypatch.setenv("NVCC", str(nvcc))
    monkeypatch.setenv("NVCC_LOG", str(log))
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(B, "LIB_PATH", str(tmp_path / B.LIB_NAME))
    monkeypatch.setattr(B, "BINDING_PATH", str(tmp_path / os.path.basename(B.BINDING_PATH)))
    include = tmp_path / "include"
    include.mkdir()
    (include / "Python.h").write_text("")
    monkeypatch.setattr(B.sysconfig, "get_paths", lambda: {"include": str(include)})
    return tmp_path, lambda: log.read_text().splitlines() if log.exists() else []


def test_builds_the_library_without_pythons_headers(place):
    folder, calls = place
    os.remove(folder / "include" / "Python.h")
    assert B.build() == B.LIB_PATH
    assert os.path.exists(B.LIB_PATH) and not os.path.exists(B.BINDING_PATH)
    n = len(calls())
    assert B.up_to_date() and B.build() == B.LIB_PATH and len(calls()) == n
    (folder / "include" / "Python.h").write_text("")     # installed later: the module alone is built
    assert not B.up_to_date()
    B.build()
    assert os.path.exists(B.BINDING_PATH) and len(calls()) == n + 1


def test_a_module_that_does_not_compile_leaves_the_library(place, monkeypatch):
    monkeypatch.setenv("NVCC_BAD_BINDING", "1")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        B.build()
    assert os.path.exists(B.LIB_PATH) and not B.up_to_date()


def test_the_module_belongs_to_one_python(place):
    folder, calls = place
    assert B.BINDING_PATH.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    B.build()
    n = len(calls())
    B.build()
    assert len(calls()) == n
    # another Python's module is not taken for this one's
    os.rename(B.BINDING_PATH, folder / "_binding.cpython-399-other.so")
    (folder / "_binding.so").write_text("")
    assert not B.up_to_date()
    B.build()
    assert len(calls()) == n + 1 and os.path.exists(B.BINDING_PATH)


def test_calls_without_the_module_say_so(place, monkeypatch):
    monkeypatch.setattr(P, "_calls", None)
    monkeypatch.setattr(P, "_load", lambda: None)
    with pytest.raises(ImportError, match="headers"):
        P._native()
