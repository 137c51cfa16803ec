"""Scores as index_scores returns them, handed to the selection."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
INDEX = 128


@pytest.fixture(scope="module")
def api():
    from sparse_attention_indexer_uint32_gb300 import api

    return api


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def inputs(seed, batch, total, heads, pages, page):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    table = torch.randperm(batch * pages, generator=g, device="cuda").to(torch.int32).reshape(batch, pages)
    cache = randn(batch * pages * page, INDEX).to(torch.bfloat16)
    return randn(total, heads, INDEX).to(torch.bfloat16), randn(total, heads), cache, table


def check(scores, lens, table, page, k, slots, raw):
    """Rows whose k best positions are `raw`, and these positions' slots."""
    for r, n in enumerate(lens):
        row, m = scores[r, :n].double(), min(n, k)
        at = raw[r, :m].long()
        assert at.unique().numel() == m and (m == 0 or (0 <= int(at.min()) and int(at.max()) < n)), r
        if m:
            assert (row[at] >= row.topk(m).values.min()).all(), r
        assert torch.equal(slots[r, :m].long(), table[r].long()[at // page] * page + at % page), r
        assert (raw[r, m:] == -1).all() and (slots[r, m:] == -1).all(), r


@pytest.mark.parametrize("pages,page", [(5, 1), (7, 1), (3, 2), (4, 2), (5, 4)])
def test_rows_padded_past_the_last_page(api, pages, page):
    lens = [pages * page, 1, 0, pages * page - 1]
    q, weights, cache, table = inputs(1, 4, 4, 8, pages, page)
    out = api.index_scores(q, weights, cache, i32(lens), table, page)
    assert out.shape == (4, (pages * page + 3) // 4 * 4)
    for k in (3, 64):
        slots, raw, _ = api.topk_transform(out, i32(lens), table, page, k, want_raw=True)
        check(out, lens, table, page, k, slots, raw)
