"""The index calls and attention behind a shared prompt where the compiled module
is not there: the same results, and the same refusals."""
from __future__ import annotations

import types

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, SCALE = torch.bfloat16, 0.07


@pytest.fixture
def api(monkeypatch):
    from sparse_attention_indexer_uint32_gb300 import _lib, api

    none = types.SimpleNamespace(index_append=lambda *a: False, index_scores=lambda *a: False, attend_shared=lambda *a: False)
    api.with_module = lambda: monkeypatch.setattr(api, "_calls", _lib.tensor_calls)
    api.without = lambda: monkeypatch.setattr(api, "_calls", none)
    yield api
    del api.with_module, api.without


def randn(*shape, dtype=BF):
    return torch.randn(shape, device="cuda").to(dtype)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def both(api, call, fresh):
    """What the call makes of fresh outputs, with the module and without it."""
    results = []
    for way in (api.with_module, api.without):
        way()
        to = fresh()
        call(*to)
        results.append(to)
    assert all(torch.equal(a, b) for a, b in zip(*results))
    return results[0]


def test_same_results(api):
    rows, slots, weight, bias = randn(5, 192)[:, 32:160], i32([4, 0, -1, 7, 2]), randn(128), randn(128)
    turn, positions, before = torch.randn(10, 64, device="cuda"), i32([1, 2, 3, 0, 9]), randn(8, 160)
    for more in ({}, dict(norm_weight=weight), dict(norm_weight=weight, norm_bias=bias, eps=1e-3),
                 dict(cos_sin=turn, positions=positions, interleaved=True, rope_last=True), dict(cos_sin=turn, positions=positions)):
        cache, = both(api, lambda c: api.index_append(rows, slots, c[:, :128], **more), lambda: [before.clone()])
        assert not torch.equal(cache, before)
    q, heads, keys = randn(7, 10, 128)[:, ::2], torch.randn(7, 8, device="cuda")[:, 1:6], randn(6 * 32, 136)[:, :128]
    lens, table, cu = i32([40, 90]), i32([[0, 1, 2, 9], [3, 4, 5, 9]])[:, :3], i32([0, 2, 7])
    scores, = both(api, lambda out: api.index_scores(q, heads, keys, lens, table, 32, cu_q=cu, max_seq_len=93, out=out),
                   lambda: [torch.zeros(7, 100, device="cuda")])
    assert scores[6, :90].any() and not scores[:, 90:].any()
    x, latent, pages, common = randn(2, 3, 16, 576)[:, :2], randn(10 * 64, 576), i32([6, 7]), i32([100])
    room = torch.empty(api._shared_workspace_bytes(2, 2, 16), dtype=torch.uint8, device="cuda")
    rows = i32([[9, 6, 0, 1, 2], [9, 7, 3, 4, 5]])
    out, lse = both(api, lambda out, lse: api.attend_shared(x, latent, i32([200, 300]), rows, pages, common, 64, SCALE, out=out,
                                                            lse=lse, workspace=room),
                    lambda: [torch.zeros(2, 2, 16, 512, dtype=BF, device="cuda"), torch.zeros(2, 2, 16, device="cuda")])
    assert out.any() and lse.any()
