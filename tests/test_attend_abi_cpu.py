"""Refusals of the block-table, cache-append and attention entry points: found
on the host before any CUDA call (fake pointers, never dereferenced), and the
tensor-level checks of the conveniences."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_indexer_uint32_gb300 import build as build_mod

FAKE = 1 << 20
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    from sparse_attention_indexer_uint32_gb300 import _lib

    return _lib


@pytest.fixture(scope="module")
def api(lib):
    from sparse_attention_indexer_uint32_gb300 import api

    return api


def caller(fn, **ok):
    names = list(ok)

    def call(**over):
        assert set(over) <= set(names)
        return fn(*({**ok, **over}[n] for n in names))

    return call


def test_block_tables_refusals(lib):
    call = caller(lib.library().topk_block_tables, context=FAKE, new=FAKE, batch=4, page_size=64, free=FAKE, num_free=3,
                  table=FAKE, stride=8, pages=8, max_tokens=16, seq=FAKE, cu=FAKE, slots=FAKE, positions=None, rows=None,
                  status=FAKE, stream=None)
    for bad in (dict(context=None), dict(new=None), dict(batch=0), dict(page_size=48), dict(page_size=0),
                dict(free=None), dict(num_free=-1), dict(table=None), dict(stride=7), dict(pages=0), dict(max_tokens=-1),
                dict(seq=None), dict(cu=None), dict(slots=None), dict(status=None),
                dict(batch=1 << 20, pages=1 << 11, stride=1 << 11)):
        assert call(**bad) == lib.TOPK_EINVAL, bad
    for name in ("context", "new", "free", "table", "seq", "cu", "slots", "positions", "rows", "status"):
        assert call(**{name: FAKE + 2}) == lib.TOPK_EALIGN, name


def test_cache_append_refusals(lib):
    call = caller(lib.library().topk_cache_append, rows=FAKE, row_stride=576, tokens=4, weight=FAKE, eps=1e-6,
                  cos_sin=FAKE, num_positions=10, positions=FAKE, interleaved=0, slots=FAKE, cache=FAKE, slot_stride=576,
                  num_slots=9, dtype=lib.TOPK_BF16, stream=None)
    for bad in (dict(rows=None), dict(row_stride=575), dict(row_stride=568), dict(tokens=-1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(num_positions=0), dict(positions=None),
                dict(slots=None), dict(cache=None), dict(slot_stride=570), dict(num_slots=0), dict(dtype=2),
                dict(dtype=-1), dict(row_stride=BIG)):
        assert call(**bad) == lib.TOPK_EINVAL, bad
    for bad in (dict(rows=FAKE + 8), dict(row_stride=580), dict(weight=FAKE + 2), dict(cos_sin=FAKE + 4),
                dict(positions=FAKE + 1), dict(slots=FAKE + 2), dict(cache=FAKE + 8), dict(slot_stride=578)):
        assert call(**bad) == lib.TOPK_EALIGN, bad


LATENT = dict(q=FAKE, cache=FAKE, slot_stride=576, num_slots=100, heads=16, scale=0.1, out=FAKE, lse=FAKE,
              workspace=FAKE, workspace_bytes=1 << 34)


def test_attend_refusals(lib):
    c, ok = lib.library(), LATENT
    selected = caller(c.topk_attend_selected, q=ok["q"], q_row_stride=16 * 576, q_head_stride=576, cache=ok["cache"],
                      slot_stride=576, num_slots=100, indices=FAKE, indices_stride=32, seq_lens=None, rows=3, heads=16,
                      k=32, scale=0.1, dtype=lib.TOPK_BF16, out=FAKE, lse=None, workspace=FAKE, workspace_bytes=1 << 34,
                      stream=None)
    paged = caller(c.topk_attend_paged, q=ok["q"], q_row_stride=32 * 576, q_query_stride=16 * 576, q_head_stride=576,
                   cache=ok["cache"], slot_stride=576, num_slots=100, seq_lens=FAKE, page_table=FAKE,
                   page_table_stride=4, page_size=64, max_seq_len=256, batch=3, queries=2, heads=16, scale=0.1,
                   dtype=lib.TOPK_FP16, out=FAKE, lse=None, workspace=FAKE, workspace_bytes=1 << 34, stream=None)
    shared = (dict(q=None), dict(cache=None), dict(slot_stride=570), dict(num_slots=0), dict(heads=0), dict(out=None),
              dict(scale=float("nan")), dict(dtype=5), dict(workspace=None), dict(q_row_stride=-8),
              dict(heads=(1 << 30)), dict(slot_stride=BIG))
    for call, more in ((selected, (dict(indices=None), dict(indices_stride=31), dict(rows=0), dict(k=0))),
                       (paged, (dict(seq_lens=None), dict(page_table=None), dict(page_table_stride=3),
                                dict(page_size=63), dict(max_seq_len=-1), dict(batch=0), dict(queries=0)))):
        for bad in shared + more:
            assert call(**bad) == lib.TOPK_EINVAL, bad
        for bad in (dict(q=FAKE + 8), dict(cache=FAKE + 2), dict(out=FAKE + 8), dict(workspace=FAKE + 4),
                    dict(lse=FAKE + 2), dict(q_row_stride=16 * 576 + 4), dict(q_head_stride=580), dict(slot_stride=580)):
            assert call(**bad) == lib.TOPK_EALIGN, bad
        assert call(workspace_bytes=8) == lib.TOPK_ENOSPACE
    assert selected(indices=FAKE + 2) == lib.TOPK_EALIGN
    assert paged(page_table=FAKE + 2) == lib.TOPK_EALIGN
    assert paged(q_query_stride=577) == lib.TOPK_EALIGN
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1 << 20, 1, 1 << 11), (1, 1 << 20, 1 << 11)):
        assert lib.topk_attend_workspace_bytes(*bad) == 0
    assert lib.topk_attend_workspace_bytes(1, 1, 1) >= 16


def test_attend_prompt_refusals(lib):
    call = caller(lib.library().topk_attend_prompt, q=FAKE, q_token_stride=3 * 192, q_head_stride=192, k_nope=FAKE,
                  k_token_stride=3 * 256, k_head_stride=256, k_rope=FAKE, k_rope_stride=64, v=FAKE, v_token_stride=768,
                  v_head_stride=256, cu_q=FAKE, cu_k=FAKE, batch=2, total_q=10, total_k=12, heads=3, scale=0.1, causal=1,
                  dtype=lib.TOPK_BF16, out=FAKE, lse=None, stream=None)
    for bad in (dict(q=None), dict(k_nope=None), dict(k_rope=None), dict(v=None), dict(cu_q=None), dict(cu_k=None),
                dict(batch=0), dict(total_q=-1), dict(total_k=-1), dict(heads=0), dict(scale=float("nan")),
                dict(dtype=3), dict(out=None), dict(total_q=1 << 30), dict(q_token_stride=-8), dict(k_rope_stride=-64),
                dict(v_token_stride=BIG)):
        assert call(**bad) == lib.TOPK_EINVAL, bad
    for bad in (dict(q=FAKE + 2), dict(k_nope=FAKE + 8), dict(k_rope=FAKE + 4), dict(v=FAKE + 8), dict(out=FAKE + 8),
                dict(lse=FAKE + 1), dict(cu_q=FAKE + 2), dict(cu_k=FAKE + 2), dict(q_token_stride=577),
                dict(q_head_stride=196), dict(k_token_stride=772), dict(k_head_stride=257), dict(k_rope_stride=68),
                dict(v_token_stride=772), dict(v_head_stride=260)):
        assert call(**bad) == lib.TOPK_EALIGN, bad


def test_read_attend_flags_refusal(lib):
    assert lib.library().topk_read_attend_flags(None, 0, None) == lib.TOPK_EINVAL


def test_cpu_tensors_are_refused(api):
    i32, bf = torch.zeros(3, dtype=torch.int32), dict(dtype=torch.bfloat16)
    cache, table = torch.zeros(10, 576, **bf), torch.zeros(3, 4, dtype=torch.int32)
    calls = (lambda: api.block_tables(i32, i32, i32, table, 16, 8),
             lambda: api.cache_append(torch.zeros(3, 576, **bf), i32, cache),
             lambda: api.attend_selected(torch.zeros(3, 2, 576, **bf), cache, table, 0.1),
             lambda: api.attend_paged(torch.zeros(3, 1, 2, 576, **bf), cache, i32, table, 16, 0.1),
             lambda: api.attend_prompt(torch.zeros(5, 2, 192, **bf), torch.zeros(6, 2, 128, **bf),
                                       torch.zeros(6, 64, **bf), torch.zeros(6, 2, 128, **bf), i32, i32, 0.1))
    for call in calls:
        with pytest.raises(ValueError, match="on a GPU"):
            call()


def test_tensor_checks(api):
    """The conveniences name the argument that is wrong (CPU tensors: nothing reaches a kernel)."""
    i32 = torch.zeros(3, dtype=torch.int32)
    bf = dict(dtype=torch.bfloat16)
    cache = torch.zeros(10, 576, **bf)
    with pytest.raises(ValueError, match="new_lens"):
        api.block_tables(i32, i32[:2], i32, torch.zeros(3, 4, dtype=torch.int32), 16, 8)
    with pytest.raises(ValueError, match="page_table"):
        api.block_tables(i32, i32, i32, torch.zeros(3, 4), 16, 8)
    with pytest.raises(ValueError, match="rows"):
        api.cache_append(torch.zeros(3, 576), i32, cache)
    with pytest.raises(ValueError, match="576"):
        api.cache_append(torch.zeros(3, 512, **bf), i32, cache)
    with pytest.raises(ValueError, match="slots"):
        api.cache_append(torch.zeros(4, 576, **bf), i32, cache)
    with pytest.raises(ValueError, match="cache"):
        api.cache_append(torch.zeros(3, 576), i32, torch.zeros(10, 576))
    q = torch.zeros(3, 16, 576, **bf)
    with pytest.raises(ValueError, match="indices"):
        api.attend_selected(q, cache, torch.zeros(3, 8), 0.1)
    with pytest.raises(ValueError, match="q and indices"):
        api.attend_selected(q, cache, torch.zeros(2, 8, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError, match="cache"):
        api.attend_selected(q, cache.to(torch.float16), torch.zeros(3, 8, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError, match="q must be"):
        api.attend_selected(q.float(), cache.float(), torch.zeros(3, 8, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError, match="q rows"):
        api.attend_selected(torch.zeros(3, 576, 16, **bf).transpose(1, 2), cache, torch.zeros(3, 8, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError, match="out"):
        api.attend_selected(q, cache, torch.zeros(3, 8, dtype=torch.int32), 0.1, out=torch.zeros(3, 16, 576, **bf))
    with pytest.raises(ValueError, match="seq_lens"):
        api.attend_selected(q, cache, torch.zeros(3, 8, dtype=torch.int32), 0.1, seq_lens=i32[:2])
    with pytest.raises(ValueError, match="q and page_table"):
        api.attend_paged(q, cache, i32, torch.zeros(3, 8, dtype=torch.int32), 16, 0.1)
    with pytest.raises(ValueError, match="max_seq_len"):
        api.attend_paged(q[:, None], cache, i32, torch.zeros(3, 8, dtype=torch.int32), 16, 0.1, max_seq_len=129)
    pq, kn, kr, v = (torch.zeros(*s, **bf) for s in ((5, 2, 192), (6, 2, 128), (6, 64), (6, 2, 128)))
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_rope"):
        api.attend_prompt(pq, kn, kr[:5], v, cu, cu, 0.1)
    with pytest.raises(ValueError, match="k_nope"):
        api.attend_prompt(pq, kn[:, :1], kr, v, cu, cu, 0.1)
    with pytest.raises(ValueError, match="cu_k"):
        api.attend_prompt(pq, kn, kr, v, cu, torch.zeros(3, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError, match="lse"):
        api.attend_prompt(pq, kn, kr, v, cu, cu, 0.1, lse=torch.zeros(5, 2, **bf))
