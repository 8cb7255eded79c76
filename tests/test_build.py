"""CPU tests of the build's parts, with compilers that only write their output
file: what is built without torch, and what is rebuilt when."""
import os
import stat

import pytest

from residual_add_rmsnorm_vec_gb300 import build as b

COMPILER = """#!/bin/sh
echo "$@" >> {log}
case "$*" in *{failing}*) echo refused >&2; exit 1;; esac
while [ $# -gt 1 ]; do [ "$1" = -o ] && echo built > "$2"; shift; done
exit 0
"""


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """A build folder of its own; set(failing) makes commands with that text fail."""
    def compilers(failing="no such text"):
        for name in ("nvcc", "g++"):
            path = tmp_path / name
            path.write_text(COMPILER.format(log=tmp_path / "log", failing=failing.replace(" ", "\\ ")))
            path.chmod(path.stat().st_mode | stat.S_IXUSR)

    compilers()
    monkeypatch.setenv("PATH", f"{tmp_path}{os.pathsep}{os.environ['PATH']}")
    monkeypatch.setenv("NVCC", str(tmp_path / "nvcc"))
    out = tmp_path / "out"
    for name in ("LIB_PATH", "CHECKED_PATH", "ATTN_PATH", "FAST_PATH", "HOSTCOST_PATH"):
        monkeypatch.setattr(b, name, str(out / os.path.basename(getattr(b, name))))
    monkeypatch.setattr(b, "BUILD_DIR", str(out))
    monkeypatch.setattr(b, "log", lambda: (tmp_path / "log").read_text(), raising=False)
    return compilers


def without_torch(monkeypatch):
    find = b.importlib.util.find_spec
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_everything_is_built_and_then_up_to_date(fake):
    assert not b.up_to_date()
    assert b.build() == b.LIB_PATH
    for path in (b.LIB_PATH, b.ATTN_PATH, b.FAST_PATH, b.HOSTCOST_PATH):
        assert os.path.exists(path)
    assert b.up_to_date()


def test_the_c_libraries_need_no_torch(fake, monkeypatch):
    without_torch(monkeypatch)
    assert b.build() == b.LIB_PATH
    for path in (b.LIB_PATH, b.ATTN_PATH, b.HOSTCOST_PATH):
        assert os.path.exists(path)
    assert not os.path.exists(b.FAST_PATH) and "attn_fast" not in b.log()
    assert b.up_to_date()


def test_the_c_libraries_are_linked_although_the_module_fails(fake):
    fake(failing="attn_fast")
    with pytest.raises(RuntimeError, match="attn_fast"):
        b.build()
    for path in (b.LIB_PATH, b.ATTN_PATH, b.HOSTCOST_PATH):
        assert os.path.exists(path)
    assert not os.path.exists(b.FAST_PATH) and not b.up_to_date()
    fake()
    b.build()
    assert b.up_to_date()


def test_the_module_of_another_torch_is_not_taken(fake, monkeypatch):
    assert os.path.basename(b.FAST_PATH) == os.path.basename(b.fast_path())
    b.build()
    have = b.importlib.metadata.version("torch")
    assert have in b.fast_path() and b.sysconfig.get_config_var("SOABI") in b.fast_path()
    monkeypatch.setattr(b.importlib.metadata, "version", lambda name: "99.0")
    monkeypatch.setattr(b, "FAST_PATH", b.fast_path())
    assert not b.up_to_date()
    b.build()
    assert os.path.exists(b.FAST_PATH) and b.up_to_date()


def test_the_checked_library_is_the_row_norms(fake, monkeypatch):
    # files of the attention path are no part of it and do not make it stale
    assert b.build(checked=True) == b.CHECKED_PATH
    assert "csrc_attn" not in b.log() and "attn_fast" not in b.log()
    time = os.path.getmtime
    later = lambda part: lambda f: time(f) + (1e6 if part in str(f) else 0)
    for part in ("csrc_attn", "rmsnorm_attn.h", "attn_fast.cpp", "host_cost.cu"):
        monkeypatch.setattr(b.os.path, "getmtime", later(part))
        assert b.up_to_date(checked=True), part
    for part in (os.sep + "csrc" + os.sep, "rmsnorm.h", "build.py"):
        monkeypatch.setattr(b.os.path, "getmtime", later(part))
        assert not b.up_to_date(checked=True), part
    monkeypatch.setattr(b.os.path, "getmtime", time)
    b.build()
    for part in ("csrc_attn", "rmsnorm_attn.h", "attn_fast.cpp", "host_cost.cu", os.sep + "csrc" + os.sep):
        monkeypatch.setattr(b.os.path, "getmtime", later(part))
        assert not b.up_to_date(), part
