"""What is built anew, and when.  Fake compilers, no GPU."""
from __future__ import annotations

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
