"""When the build is taken as current: not under another interpreter, another torch or other flags."""
import importlib.metadata
import os
import sysconfig

import pytest

from paged_kv_cache_275_gb300 import build


@pytest.fixture
def built(tmp_path, monkeypatch):
    """A build directory whose binaries are newer than every source."""
    monkeypatch.delenv("PKV_NVCC_FLAGS", raising=False)
    for name in ("LIB", "BINDING", "STAMP"):
        monkeypatch.setattr(build, name, tmp_path / name)
    later = max(p.stat().st_mtime for p in build._inputs()) + 100
    for p in (build.LIB, build.BINDING):
        p.write_bytes(b"")
        os.utime(p, (later, later))
    build.STAMP.write_text(build._stamp())


def test_current(built):
    assert not build.needs_build()


def test_another_interpreter(built, monkeypatch):
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var",
                        lambda name: "cpython-399-other" if name == "SOABI" else real(name))
    assert build.needs_build()


def test_another_torch(built, monkeypatch):
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0.1")
    assert build.needs_build()


def test_other_flags(built, monkeypatch):
    monkeypatch.setenv("PKV_NVCC_FLAGS", "-DPKV_D128_WARPS=6")
    assert build.needs_build()


@pytest.mark.parametrize("name", ["LIB", "BINDING"])
def test_a_missing_binary(built, name):
    getattr(build, name).unlink()
    assert build.needs_build()
