"""Building the Python module on top of the library: without what it needs the
library is built all the same, and layer.py makes every call itself."""
import os
import subprocess

import pytest

from gated_delta_rule_55_amd import build


@pytest.fixture
def old(tmp_path, monkeypatch):
    """A module that an earlier build left, perhaps of another library."""
    out = tmp_path / "_fast.so"
    out.write_text("old")
    monkeypatch.setattr(build, "FAST_OUT", str(out))
    return out


@pytest.mark.parametrize("missing", ["g++", "Python.h", "torch"])
def test_no_module_without_its_tools(old, monkeypatch, capsys, missing):
    if missing == "g++":
        monkeypatch.setattr(build.shutil, "which", lambda name: None)
    elif missing == "Python.h":
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": "/nowhere"})
    else:
        monkeypatch.setattr(build, "_torch_root", lambda: None)
    assert build.build_fast() is None
    assert not old.exists() and missing in capsys.readouterr().out


def test_an_error_in_its_source_is_an_error(old, monkeypatch):
    monkeypatch.setattr(build, "_fast_command", lambda: ["false"])
    with pytest.raises(subprocess.CalledProcessError):
        build.build_fast()


def test_it_is_built_where_all_is_there(old):
    if build._fast_missing():
        pytest.skip(build._fast_missing())
    if not os.path.exists(build.OUT):
        pytest.skip("libkda.so not built")
    assert build.build_fast() == str(old) and os.path.getsize(old) > 10000
