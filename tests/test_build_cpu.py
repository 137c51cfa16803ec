"""What is built anew, and when.  Fake compilers, no GPU."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from sparse_attention_indexer_uint32_gb300 import build as build_mod


@pytest.fixture
def commands(monkeypatch):
    """The compilers' command lines, none of which runs, where everything is built already."""
    build_mod.build()
    run = []
    monkeypatch.setattr(build_mod.subprocess, "run", lambda cmd, **kw: run.append(cmd) or type("Done", (), dict(returncode=0, stderr="")))
    monkeypatch.setattr(build_mod.os, "replace", lambda *a: None)
    return run


def test_nothing_to_do(commands):
    assert build_mod.build() == build_mod.LIBRARY and commands == []


@pytest.mark.parametrize("what", ["torch", "python"])
def test_module_of_another_version_is_not_taken(commands, monkeypatch, what):
    """It reads objects whose layout is the version's own; the library does not."""
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "9.9.9")
    else:
        known = build_mod.sysconfig.get_config_var
        monkeypatch.setattr(build_mod.sysconfig, "get_config_var", lambda x: "cpython-999" if x == "SOABI" else known(x))
    build_mod.build()
    assert len(commands) == 1 and any(x.endswith("tensor_calls.cpp") for x in commands[0])


def test_library_without_the_module(commands, monkeypatch, tmp_path):
    """A module that cannot be compiled is said, once the library is there."""
    monkeypatch.setattr(build_mod, "LIBRARY", str(tmp_path / "lib.so"))
    done = type("Done", (), dict(returncode=0, stderr=""))
    fails = type("Fails", (), dict(returncode=1, stderr="no such header"))
    monkeypatch.setattr(build_mod.subprocess, "run",
                        lambda cmd, **kw: commands.append(cmd) or (fails if any(x.endswith("tensor_calls.cpp") for x in cmd) else done))
    with pytest.raises(RuntimeError, match="tensor_calls.cpp"):
        build_mod.build(force=True)
    assert any(cmd[-1] == "-lcudart" for cmd in commands)  # the link


CODE = """
import sys, warnings
sys.path.insert(0, sys.argv[1])
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    from sparse_attention_indexer_uint32_gb300 import _lib, api
assert _lib.__file__.startswith(sys.argv[1]), _lib.__file__
assert [w for w in seen if w.category is RuntimeWarning and "_tensor_calls" in str(w.message)], seen
import torch
assert _lib.topk_attend_workspace_bytes(2, 1, 16) > 0
x = torch.zeros(2, 128, dtype=torch.bfloat16)
i = torch.zeros(2, dtype=torch.int32)
for call in (lambda: api.index_append(x, i, x),
             lambda: api.index_scores(x[:, None], torch.zeros(2, 1), x, i, i[:, None], 16, out=torch.zeros(2, 16)),
             lambda: api.attend_shared(torch.zeros(2, 1, 1, 576).half(), torch.zeros(2, 576).half(), i, i[:, None], i, i[:1], 16, 0.1,
                                       out=torch.zeros(2, 1, 1, 512).half(), workspace=x)):
    try:
        call()
    except ValueError as e:
        assert "on a GPU" in str(e), e
    else:
        raise AssertionError("no refusal")
"""


@pytest.mark.parametrize("module", ["missing", "broken"])
def test_package_without_the_module(tmp_path, module):
    """The library and every call of it stay, through ctypes."""
    build_mod.build()
    package = tmp_path / "sparse_attention_indexer_uint32_gb300"
    package.mkdir()
    for name in os.listdir(build_mod.PKG):
        if name.endswith(".py") or name == "libtopkidx.so":
            (package / name).symlink_to(os.path.join(build_mod.PKG, name))
    if module == "broken":
        (package / os.path.basename(build_mod.tensor_calls_path())).write_bytes(b"not a module")
    res = subprocess.run([sys.executable, "-c", CODE, str(tmp_path)], capture_output=True, text=True, cwd=tmp_path)
    assert res.returncode == 0, res.stderr
