"""The tensor calls make the tensors' GPU the current one where it is not: the
library launches on the current one.  Fake devices and a fake library, no GPU."""
from __future__ import annotations

import contextlib

import pytest
import torch

from sparse_attention_indexer_uint32_gb300 import build as build_mod


@pytest.fixture
def api(monkeypatch):
    build_mod.build()
    from sparse_attention_indexer_uint32_gb300 import api

    state = dict(current=0, calls=[])

    @contextlib.contextmanager
    def device(gpu):
        before, state["current"] = state["current"], gpu
        yield
        state["current"] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(api, "_current_device", lambda: state["current"])
    api_state = state

    class Library:
        def __getattr__(self, name):
            def fn(*args):
                api_state["calls"].append((name, api_state["current"]))
                return 0

            return fn

    monkeypatch.setattr(api, "_c", Library())
    monkeypatch.setattr(api._lib, "topk_plan", lambda *a: Library().topk_plan(*a))
    monkeypatch.setattr(api._lib, "topk_transform", lambda *a: Library().topk_transform(*a))
    monkeypatch.setattr(api._lib, "stream_handle", lambda stream, index: 0)
    api.state = state
    return api


class On(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""

    gpu = 1

    def get_device(self):
        return self.gpu


def on(gpu, t):
    t = t.as_subclass(On)
    t.gpu = gpu
    return t


def every_call(api, gpu):
    bf = dict(dtype=torch.bfloat16)
    z = lambda *shape, **kw: on(gpu, torch.zeros(*shape, **kw))  # noqa: E731
    i32 = lambda *shape: z(*shape, dtype=torch.int32)  # noqa: E731
    tables = api.BlockTables(i32(3), i32(4), i32(8), i32(8), i32(8), i32(2))
    api.block_tables(i32(3), i32(3), i32(5), i32(3, 4), 16, 8, out=tables)
    api.cache_append(z(3, 576, **bf), i32(3), z(9, 576, **bf))
    api.attend_selected(z(3, 2, 576, **bf), z(9, 576, **bf), i32(3, 4), 0.1, out=z(3, 2, 512, **bf), lse=z(3, 2),
                        workspace=z(1 << 20, dtype=torch.uint8).repeat(4))
    api.attend_paged(z(3, 1, 2, 576, **bf), z(9, 576, **bf), i32(3), i32(3, 4), 16, 0.1, out=z(3, 1, 2, 512, **bf),
                     lse=z(3, 1, 2), workspace=z(1 << 20, dtype=torch.uint8).repeat(4))
    api.attend_prompt(z(5, 2, 192, **bf), z(6, 2, 128, **bf), z(6, 64, **bf), z(6, 2, 128, **bf), i32(2), i32(2), 0.1,
                      out=z(5, 2, 128, **bf), lse=z(5, 2))
    api.topk_transform(z(3, 64), i32(3), i32(3, 4), 16, 8, out=i32(3, 8))


NAMES = ["topk_block_tables", "topk_cache_append", "topk_attend_selected", "topk_attend_paged", "topk_attend_prompt",
         "topk_plan", "topk_transform"]


@pytest.mark.parametrize("gpu", [0, 1, 5])
def test_launched_where_the_tensors_are(api, gpu):
    every_call(api, gpu)
    assert api.state["calls"] == [(name, gpu) for name in NAMES]
    assert api.state["current"] == 0  # as it was
