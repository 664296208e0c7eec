"""The build without torch, and what makes the extension be built anew.  No GPU."""
import ctypes
import importlib.util
import os
import subprocess
import sys
import sysconfig

import pytest

from paged_kv_cache_218_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_the_library_is_built_without_torch(tmp_path, monkeypatch, capsys):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libpa.so"))
    monkeypatch.setattr(build, "PYCALL", str(tmp_path / "_pycall.so"))
    assert build.build() == str(tmp_path / "libpa.so")
    assert ctypes.CDLL(build.LIB).pa_version() >= 1 << 16
    assert os.listdir(tmp_path) == ["libpa.so"]
    assert "_pycall" in capsys.readouterr().err


def test_the_binding_says_what_it_misses():
    code = ("import sys; sys.modules['paged_kv_cache_218_gb300._pycall'] = None\n"
            "try:\n    from paged_kv_cache_218_gb300 import binding\n"
            "except ImportError as e:\n    print(e)")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and "_pycall is missing" in r.stdout, r.stderr


def test_the_extension_belongs_to_an_interpreter_and_a_torch(tmp_path, monkeypatch):
    """A torch of another version is another one, however old its files are."""
    assert build.PYCALL.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert not build._Extension(build._torch(), "nvcc").stale
    version = tmp_path / "version.py"
    version.write_text("__version__ = '1'")
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "PYCALL", str(tmp_path / "_pycall.so"))
    ext = build._Extension(str(tmp_path), "nvcc")
    assert ext.stale

    def link(cmd, **kw):
        assert cmd == ext.link
        with open(ext.tmp, "w"):
            pass

    monkeypatch.setattr(build.subprocess, "run", link)
    ext.finish()
    assert not build._Extension(str(tmp_path), "nvcc").stale
    version.write_text("__version__ = '0'")
    os.utime(version, (0, 0))
    assert build._Extension(str(tmp_path), "nvcc").stale
