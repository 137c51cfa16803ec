"""Refusals of the index append, index score and shared-prompt attention entry
points: found on the host before any CUDA call (fake pointers, never
dereferenced), and the tensor-level checks of the conveniences."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_indexer_uint32_gb300 import build as build_mod
from tests.test_attend_abi_cpu import BIG, FAKE, caller


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    from sparse_attention_indexer_uint32_gb300 import _lib

    return _lib


@pytest.fixture(scope="module")
def api(lib):
    from sparse_attention_indexer_uint32_gb300 import api

    return api


def test_index_append_refusals(lib):
    call = caller(lib.library().topk_index_append, rows=FAKE, row_stride=128, tokens=4, weight=FAKE, bias=FAKE, eps=1e-6,
                  cos_sin=FAKE, num_positions=10, positions=FAKE, interleaved=0, rope_last=0, slots=FAKE, cache=FAKE,
                  slot_stride=128, num_slots=9, dtype=lib.TOPK_BF16, stream=None)
    for bad in (dict(rows=None), dict(row_stride=127), dict(row_stride=120), dict(tokens=-1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(weight=None), dict(num_positions=0),
                dict(positions=None), dict(slots=None), dict(cache=None), dict(slot_stride=120), dict(num_slots=0),
                dict(dtype=2), dict(dtype=-1), dict(row_stride=BIG), dict(slot_stride=BIG)):
        assert call(**bad) == lib.TOPK_EINVAL, bad
    for bad in (dict(rows=FAKE + 8), dict(row_stride=132), dict(weight=FAKE + 2), dict(bias=FAKE + 8), dict(cos_sin=FAKE + 4),
                dict(positions=FAKE + 1), dict(slots=FAKE + 2), dict(cache=FAKE + 8), dict(slot_stride=130)):
        assert call(**bad) == lib.TOPK_EALIGN, bad


def test_index_scores_refusals(lib):
    call = caller(lib.library().topk_index_scores, q=FAKE, q_token_stride=64 * 128, q_head_stride=128, weights=FAKE,
                  weights_stride=64, cache=FAKE, slot_stride=128, num_slots=100, seq_lens=FAKE, page_table=FAKE,
                  page_table_stride=4, page_size=64, max_seq_len=256, cu_q=FAKE, batch=3, total_q=6, heads=64,
                  dtype=lib.TOPK_BF16, scores=FAKE, scores_stride=256, stream=None)
    for bad in (dict(q=None), dict(weights=None), dict(cache=None), dict(seq_lens=None), dict(page_table=None),
                dict(scores=None), dict(batch=0), dict(total_q=-1), dict(heads=0), dict(heads=257), dict(dtype=3),
                dict(num_slots=0), dict(page_size=48), dict(page_size=0), dict(max_seq_len=-1), dict(page_table_stride=3),
                dict(slot_stride=120), dict(slot_stride=BIG), dict(q_token_stride=120), dict(q_head_stride=64),
                dict(weights_stride=63), dict(scores_stride=255), dict(cu_q=None, total_q=7),
                dict(total_q=1 << 24, max_seq_len=1 << 20, page_table_stride=1 << 20, scores_stride=1 << 20)):
        assert call(**bad) == lib.TOPK_EINVAL, bad
    for bad in (dict(q=FAKE + 8), dict(cache=FAKE + 2), dict(weights=FAKE + 2), dict(seq_lens=FAKE + 1),
                dict(page_table=FAKE + 2), dict(cu_q=FAKE + 2), dict(scores=FAKE + 2), dict(q_token_stride=64 * 128 + 4),
                dict(q_head_stride=132), dict(slot_stride=132)):
        assert call(**bad) == lib.TOPK_EALIGN, bad


def test_attend_shared_refusals(lib):
    call = caller(lib.library().topk_attend_shared, q=FAKE, q_row_stride=32 * 576, q_query_stride=16 * 576,
                  q_head_stride=576, cache=FAKE, slot_stride=576, num_slots=100, seq_lens=FAKE, page_table=FAKE,
                  page_table_stride=4, shared_pages=FAKE, num_shared_pages=2, shared_len=FAKE, page_size=64,
                  max_seq_len=256, batch=3, queries=2, heads=16, scale=0.1, dtype=lib.TOPK_FP16, out=FAKE, lse=None,
                  workspace=FAKE, workspace_bytes=1 << 34, stream=None)
    for bad in (dict(q=None), dict(cache=None), dict(seq_lens=None), dict(page_table=None), dict(shared_pages=None),
                dict(num_shared_pages=-1), dict(shared_len=None), dict(page_size=63), dict(max_seq_len=-1),
                dict(page_table_stride=3), dict(batch=0), dict(queries=0), dict(heads=0), dict(heads=1 << 30),
                dict(scale=float("nan")), dict(dtype=5), dict(out=None), dict(workspace=None), dict(num_slots=0),
                dict(slot_stride=570), dict(q_row_stride=-8), dict(q_query_stride=100), dict(slot_stride=BIG)):
        assert call(**bad) == lib.TOPK_EINVAL, bad
    for bad in (dict(q=FAKE + 8), dict(cache=FAKE + 2), dict(out=FAKE + 8), dict(workspace=FAKE + 4), dict(lse=FAKE + 2),
                dict(seq_lens=FAKE + 2), dict(page_table=FAKE + 2), dict(shared_pages=FAKE + 1), dict(shared_len=FAKE + 2),
                dict(q_row_stride=32 * 576 + 4), dict(q_query_stride=16 * 576 + 1), dict(q_head_stride=580), dict(slot_stride=580)):
        assert call(**bad) == lib.TOPK_EALIGN, bad
    assert call(workspace_bytes=8) == lib.TOPK_ENOSPACE
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1 << 20, 1, 1 << 11), (1, 1 << 20, 1 << 11)):
        assert lib.topk_attend_shared_workspace_bytes(*bad) == 0
    assert lib.topk_attend_shared_workspace_bytes(1, 1, 1) >= 16


BF = dict(dtype=torch.bfloat16)
I32 = torch.zeros(3, dtype=torch.int32)
TABLE = torch.zeros(3, 4, dtype=torch.int32)


def append(api, rows=torch.zeros(3, 128, **BF), slots=I32, cache=torch.zeros(10, 128, **BF), **more):
    api.index_append(rows, slots, cache, **more)


def score(api, q=torch.zeros(6, 2, 128, **BF), weights=torch.zeros(6, 2), cache=torch.zeros(10, 128, **BF), seq_lens=I32,
          page_table=TABLE, page_size=16, **more):
    api.index_scores(q, weights, cache, seq_lens, page_table, page_size, **more)


def shared(api, q=torch.zeros(3, 1, 2, 576, **BF), cache=torch.zeros(10, 576, **BF), seq_lens=I32, page_table=TABLE,
           pages=I32, length=I32[:1], **more):
    api.attend_shared(q, cache, seq_lens, page_table, pages, length, 16, 0.1, **more)


def test_cpu_tensors_are_refused(api):
    for call in (append, score, shared):
        with pytest.raises(ValueError, match="on a GPU"):
            call(api)


@pytest.mark.parametrize("call,match,bad", [
    (append, "rows", dict(rows=torch.zeros(3, 128))),
    (append, "128", dict(rows=torch.zeros(3, 64, **BF))),
    (append, "rows", dict(rows=torch.zeros(128, 3, **BF).t())),
    (append, "slots", dict(slots=I32[:2])),
    (append, "slots", dict(slots=I32.long())),
    (append, "cache", dict(cache=torch.zeros(10, 128))),
    (append, "norm_weight", dict(norm_weight=torch.zeros(127, **BF))),
    (append, "norm_bias", dict(norm_bias=torch.zeros(128))),
    (append, "cos_sin", dict(cos_sin=torch.zeros(5, 32), positions=I32)),
    (append, "positions", dict(cos_sin=torch.zeros(5, 64), positions=I32[:1])),
    (append, "requires a gradient", dict(rows=torch.zeros(3, 128, **BF).requires_grad_())),
    (append, "requires a gradient", dict(norm_bias=torch.zeros(128, **BF).requires_grad_())),
    (score, "q must be", dict(q=torch.zeros(6, 2, 128))),
    (score, "q and page_table", dict(q=torch.zeros(6, 128, **BF))),
    (score, "128", dict(q=torch.zeros(6, 2, 64, **BF))),
    (score, "weights", dict(weights=torch.zeros(6, 3))),
    (score, "weights", dict(weights=torch.zeros(6, 2, **BF))),
    (score, "cache", dict(cache=torch.zeros(10, 128, dtype=torch.float16))),
    (score, "seq_lens", dict(seq_lens=I32[:2])),
    (score, "page_table", dict(page_table=TABLE.long())),
    (score, "cu_q", dict(cu_q=I32)),
    (score, "without cu_q", dict(q=torch.zeros(5, 2, 128, **BF), weights=torch.zeros(5, 2))),
    (score, "max_seq_len", dict(max_seq_len=65)),
    (score, "out", dict(out=torch.zeros(6, 63))),
    (score, "out", dict(out=torch.zeros(5, 64))),
    (score, "out", dict(out=torch.zeros(6, 64, dtype=torch.float64))),
    (score, "requires a gradient", dict(weights=torch.zeros(6, 2, requires_grad=True))),
    (score, "requires a gradient", dict(cache=torch.zeros(10, 128, **BF).requires_grad_())),
    (shared, "q and page_table", dict(q=torch.zeros(3, 2, 576, **BF))),
    (shared, "q must be", dict(q=torch.zeros(3, 1, 2, 576))),
    (shared, "576", dict(q=torch.zeros(3, 1, 2, 512, **BF))),
    (shared, "shared_pages", dict(pages=I32.long())),
    (shared, "shared_pages", dict(pages=torch.zeros(6, dtype=torch.int32)[::2])),
    (shared, "shared_len", dict(length=I32)),
    (shared, "shared_len", dict(length=torch.zeros(1))),
    (shared, "seq_lens", dict(seq_lens=I32[:2])),
    (shared, "out", dict(out=torch.zeros(3, 1, 2, 576, **BF))),
    (shared, "lse", dict(lse=torch.zeros(3, 1, 2, **BF))),
    (shared, "requires a gradient", dict(q=torch.zeros(3, 1, 2, 576, **BF).requires_grad_())),
])
def test_tensor_checks(api, call, match, bad):
    with pytest.raises(ValueError, match=match):
        call(api, **bad)


def test_max_seq_len_of_shared_rows(api):
    with pytest.raises(ValueError, match="max_seq_len"):
        api.attend_shared(torch.zeros(3, 1, 2, 576, **BF), torch.zeros(10, 576, **BF), I32, TABLE, I32, I32[:1], 16, 0.1,
                          max_seq_len=65)
