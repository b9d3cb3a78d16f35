"""The build's dealings with the Python binding (nothing is compiled here)."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

from precision_attention_fa4fp4_gb300 import build as b


@pytest.fixture(scope="module")
def built():
    return b.build()


def header():
    return os.path.join(os.path.dirname(b.HERE), "include", "fa4fp4.h")


def test_library_builds_without_torch(built, tmp_path):
    """The library's build where torch is not installed: from a copy of the tree
    whose objects are fresh, with the libraries removed."""
    root = tmp_path / "tree"
    package = root / os.path.basename(b.HERE)
    shutil.copytree(b.HERE, package, ignore=shutil.ignore_patterns("__pycache__"))
    shutil.copytree(os.path.join(os.path.dirname(b.HERE), "include"), root / "include")
    for name in (os.path.basename(b.BINDING), os.path.basename(b.LIB)):
        os.remove(package / name)
    code = ("import sys, runpy; sys.modules['torch'] = None; sys.argv = ['build.py']; "
            f"runpy.run_path({str(package / 'build.py')!r}, run_name='__main__')")
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
    assert "torch is not installed" in run.stderr
    assert (package / os.path.basename(b.LIB)).exists() and not (package / os.path.basename(b.BINDING)).exists()


def test_binding_is_for_one_python_and_one_torch(built, monkeypatch, tmp_path):
    assert b.BINDING.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and os.path.exists(b.BINDING)
    assert b._binding_commands(False, header())[:2] == (None, None)
    with open(b.STAMP) as f:
        stamp = f.read()
    for other in (stamp.replace("torch ", "torch 0."), stamp.replace("cpython-3", "cpython-2"), "2.11.0"):
        path = tmp_path / "stamp"
        path.write_text(other)
        monkeypatch.setattr(b, "STAMP", str(path))
        compile_, link, against = b._binding_commands(False, header())
        assert compile_ and link and against == stamp
