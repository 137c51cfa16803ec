"""The binding's functions of the C names, called as the header lists their
arguments, against the tensor calls."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, SCALE = torch.bfloat16, 0.07


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_uint32_gb300 import _lib

    return _lib


@pytest.fixture(scope="module")
def api(lib):
    from sparse_attention_indexer_uint32_gb300 import api

    return api


def randn(*shape, dtype=BF):
    return torch.randn(shape, device="cuda").to(dtype)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def empty(*shape, dtype=torch.int32):
    return torch.full(shape, 77, dtype=dtype, device="cuda")


def test_block_tables(lib, api):
    context, new, free = i32([3, 0, 9]), i32([4, 2, 0]), i32([11, 12, 13, 14])
    table = i32([[1, 0, 0, 0], [0, 0, 0, 0], [2, 3, 4, 0]])
    other = table.clone()
    want = api.block_tables(context, new, free, other, 4, 8)
    seq, cu, slots, positions, rows, status = empty(3), empty(4), empty(8), empty(8), empty(8), empty(2)
    lib.topk_block_tables(context, new, 3, 4, free, 4, table, 4, 4, 8, seq, cu, slots, positions, rows, status)
    for got, x in zip((seq, cu, slots, positions, rows, status, table), (*want, other)):
        assert torch.equal(got, x)
    slots = empty(8)
    lib.topk_block_tables(context, new, 3, 4, None, 0, table, 4, 4, 8, seq, cu, slots, None, None, status)
    assert status.tolist() == [0, lib.TOPK_TABLES_NO_PAGES]


@pytest.mark.parametrize("interleaved", [False, True])
def test_cache_append(lib, api, interleaved):
    rows, weight, slots, positions = randn(5, 640), randn(512), i32([4, 0, -1, 7, 2]), i32([1, 2, 3, 0, 9])
    turn = torch.randn(10, 64, device="cuda")
    a, b = empty(8, 600, dtype=BF), empty(8, 600, dtype=BF)
    api.cache_append(rows[:, :576], slots, a[:, :576], weight, 1e-5, turn, positions, interleaved)
    lib.topk_cache_append(rows, 640, 5, weight, 1e-5, turn, 10, positions, interleaved, slots, b, 600, 8, lib.TOPK_BF16)
    assert torch.equal(a, b)


def test_attend_selected_and_paged(lib, api):
    cache, lens = randn(500, 576), i32([300, 40, 0])
    q, slots = randn(3, 16, 576), i32(torch.randint(0, 500, (3, 50)))
    want = api.attend_selected(q, cache, slots, SCALE, seq_lens=lens)
    need = lib.topk_attend_workspace_bytes(3, 2, 16)
    workspace = empty(need, dtype=torch.uint8)
    out, lse = empty(3, 16, 512, dtype=BF), empty(3, 16, dtype=torch.float32)
    lib.topk_attend_selected(q, 16 * 576, 576, cache, 576, 500, slots, 50, lens, 3, 16, 50, SCALE, lib.TOPK_BF16, out, lse,
                             workspace)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    q, table = randn(3, 2, 16, 576), i32(torch.randperm(31)[:30].reshape(3, 10))
    lens = i32([150, 40, 0])
    want = api.attend_paged(q, cache, lens, table, 16, SCALE)
    out, lse = empty(3, 2, 16, 512, dtype=BF), empty(3, 2, 16, dtype=torch.float32)
    lib.topk_attend_paged(q, 32 * 576, 16 * 576, 576, cache, 576, 500, lens, table, 10, 16, 160, 3, 2, 16, SCALE,
                          lib.TOPK_BF16, out, lse, workspace)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    out.fill_(77)  # without a place for the log-sum-exp
    lib.topk_attend_paged(q, 32 * 576, 16 * 576, 576, cache, 576, 500, lens, table, 10, 16, 160, 3, 2, 16, SCALE,
                          lib.TOPK_BF16, out, None, workspace)
    assert torch.equal(out, want[0])


def test_attend_prompt(lib, api):
    q, up, rope, cu_q, cu_k = randn(30, 3, 192), randn(44, 3, 256), randn(44, 64), i32([0, 10, 30]), i32([0, 12, 44])
    for causal in (True, False):
        want = api.attend_prompt(q, up[..., :128], rope, up[..., 128:], cu_q, cu_k, SCALE, causal=causal)
        for lse in (empty(30, 3, dtype=torch.float32), None):
            out = empty(30, 3, 128, dtype=BF)
            lib.topk_attend_prompt(q, 576, 192, up, 768, 256, rope, 64, up[..., 128:], 768, 256, cu_q, cu_k, 2, 30, 44, 3,
                                   SCALE, causal, lib.TOPK_BF16, out, lse)
            assert torch.equal(out, want[0]) and (lse is None or torch.equal(lse, want[1]))
