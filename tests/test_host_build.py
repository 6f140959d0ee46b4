"""The build without what only the torch extension needs: libkvp.so is built all the same.
nvcc is faked; no compiler runs."""

import os
import subprocess
import sysconfig
import types

import pytest

from paged_kv_cache_319_b200 import build


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """A build into tmp_path whose compiler writes its output file and records its command."""
    torch, python = tmp_path / "torch", tmp_path / "python"
    (torch / "include" / "ATen").mkdir(parents=True)
    (torch / "include" / "ATen" / "dlpack.h").write_text("struct DLPackExchangeAPI;")
    python.mkdir()
    (python / "Python.h").write_text("")
    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "LIB", str(tmp_path / "libkvp.so"))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_torch_calls.so"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(subprocess, "run", run)
    spec = types.SimpleNamespace(submodule_search_locations=[str(torch)])
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: spec)
    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(python)})
    return types.SimpleNamespace(torch=torch, python=python, runs=runs)


def test_both_libraries_are_built(fake):
    assert build.build() == build.LIB
    assert len(fake.runs) == 2 and os.path.exists(build.LIB) and os.path.exists(build.CALLS)
    assert build.up_to_date()
    build.build()
    assert len(fake.runs) == 2
    os.remove(build.CALLS)
    assert not build.up_to_date()


@pytest.mark.parametrize("missing", ["torch", "header", "table", "python"])
def test_the_library_is_built_without_what_the_extension_needs(fake, missing, monkeypatch, capsys):
    header = fake.torch / "include" / "ATen" / "dlpack.h"
    if missing == "torch":
        monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    elif missing == "header":
        header.unlink()
    elif missing == "table":
        header.write_text("struct DLTensor;")
    else:
        (fake.python / "Python.h").unlink()
    with open(build.CALLS, "w"):
        pass
    assert build.build() == build.LIB
    assert len(fake.runs) == 1 and os.path.exists(build.LIB)
    assert not os.path.exists(build.CALLS)  # one of another build is not left beside it
    assert "_torch_calls.so is not built" in capsys.readouterr().err
    assert build.up_to_date()
    build.build()
    assert len(fake.runs) == 1


def test_a_compiler_error_in_the_extension_is_one(fake, monkeypatch):
    good = subprocess.run

    def run(cmd, **kw):
        r = good(cmd, **kw)
        r.returncode = int(build.CALLS_SOURCE in cmd)
        return r

    monkeypatch.setattr(subprocess, "run", run)
    with pytest.raises(RuntimeError):
        build.build()
