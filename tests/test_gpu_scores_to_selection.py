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


@pytest.mark.parametrize("page", [2, 64])
def test_several_queries_a_request(api, page):
    """The selection takes a length and a row of pages for each row of scores: those of the row's request, and what
    its query sees."""
    new, past = [5, 1, 0, 130, 3], [400, 77, 20, 0, 0]
    lens, pages = [a + b for a, b in zip(new, past)], -(-407 // page)
    q, weights, cache, table = inputs(2, 5, sum(new), 16, pages, page)
    cu = torch.tensor([0] + new).cumsum(0)
    out = api.index_scores(q, weights, cache, i32(lens), table, page, cu_q=i32(cu))
    # As a program has it, on the GPU and without a host read of lengths.
    of = torch.repeat_interleave(torch.arange(5, device="cuda"), i32(new), output_size=sum(new))
    seen = (i32(lens) - i32(cu[1:]))[of] + torch.arange(1, sum(new) + 1, device="cuda", dtype=torch.int32)
    rows = table[of]
    slots, raw, _ = api.topk_transform(out, seen, rows, page, 50, want_raw=True)
    expected = [n - m + 1 + i for n, m in zip(lens, new) for i in range(m)]
    assert seen.tolist() == expected
    check(out, expected, rows, page, 50, slots, raw)


def test_a_length_of_its_own(api):
    """Lengths above a max_seq_len that both calls are given: nothing past it is looked at."""
    q, weights, cache, table = inputs(3, 3, 3, 8, 10, 64)
    lens = [640, 70, 69]
    out = api.index_scores(q, weights, cache, i32(lens), table, 64, max_seq_len=70)
    assert out.shape == (3, 72)
    out[:, 70:] = float("inf")
    slots, raw, _ = api.topk_transform(out, i32(lens), table, 64, 80, max_seq_len=70, want_raw=True)
    check(out, [70, 70, 69], table, 64, 80, slots, raw)
