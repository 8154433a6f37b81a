"""The build of the compiled Python calls beside the library, on the host."""
import functools
import os
import subprocess

import pytest
import torch

import varlen_paged_kv_gb300 as pa
from varlen_paged_kv_gb300 import build, step


@pytest.fixture()
def tree(tmp_path, monkeypatch):
    """The build's outputs in a folder of the test's own; compilers that only leave their output."""
    monkeypatch.setattr(build, "LIB", str(tmp_path / os.path.basename(build.LIB)))
    monkeypatch.setattr(build, "binding_path", functools.partial(build.binding_path, str(tmp_path)))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    commands = []

    def run(cmd, **kw):
        commands.append(cmd)
        broken = os.path.basename(cmd[0]) == "g++" and run.broken
        if not broken:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, int(broken), "", "no headers" if broken else "")

    run.broken = False
    run.commands = commands
    monkeypatch.setattr(build.subprocess, "run", run)
    return run


def test_the_library_is_built_where_the_compiled_calls_cannot_be(tree):
    build.build()  # both
    binding = build.binding_path()
    assert os.path.exists(build.LIB) and os.path.exists(binding)
    tree.broken = True
    os.utime(binding, (0, 0))  # older than its source
    with pytest.warns(RuntimeWarning, match="no headers"):
        assert build.build() == build.LIB  # (the library is up to date)
    assert os.path.exists(build.LIB) and not os.path.exists(binding)
    with pytest.warns(RuntimeWarning, match="no headers"):
        build.build(force=True)
    assert os.path.exists(build.LIB)


def test_the_library_is_built_where_there_is_no_torch(tree, monkeypatch):
    def absent():
        raise ImportError("no torch")

    monkeypatch.setattr(build, "binding_path", absent)
    with pytest.warns(RuntimeWarning, match="no torch"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB)


def test_the_calls_are_made_in_python_where_the_compiled_ones_are_missing(monkeypatch, tmp_path):
    build.build()
    monkeypatch.setattr(step, "_fast", None)
    monkeypatch.setattr(step, "__file__", str(tmp_path / "step.py"))  # (no binding beside it)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.warns(RuntimeWarning, match="compiled calls"), pytest.raises(ValueError, match="CUDA"):
        pa.build_block_tables(i, i, i, i.reshape(2, 1), i, i, block_size=16, num_tokens=1)
    h = torch.zeros(2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):  # (and no second warning)
        pa.qk_norm_rope(h, h, i, num_heads=1, kv_num_heads=1)


def test_the_compiled_calls_are_those_of_this_torch(tree, monkeypatch):
    """A binding compiled against another torch is neither taken for current nor loaded."""
    def compiled():
        n = sum(os.path.basename(c[0]) == "g++" for c in tree.commands)
        tree.commands.clear()
        return n

    build.build()
    assert compiled() == 1
    build.build()
    assert compiled() == 0  # up to date
    build.build(force=True)
    assert compiled() == 1
    mine = build.binding_path()
    monkeypatch.setattr(torch, "__version__", "2.0.0+other")
    assert build.binding_path() != mine and not os.path.exists(build.binding_path())
    monkeypatch.setattr(step, "_fast", None)
    monkeypatch.setattr(step, "__file__", os.path.join(os.path.dirname(mine), "step.py"))
    with pytest.warns(RuntimeWarning, match="compiled calls"):
        assert step._load_fast().select_pages(1, 2) is None
    build.build()
    assert compiled() == 1
