"""What length the selection is called with when none is given: a fake library, no GPU."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_indexer_uint32_gb300 import build as build_mod


@pytest.fixture
def calls(monkeypatch):
    build_mod.build()
    from sparse_attention_indexer_uint32_gb300 import api

    made = {}
    monkeypatch.setattr(api._lib, "topk_plan", lambda lens, batch, most, *a: made.__setitem__("plan", most))
    monkeypatch.setattr(api._lib, "topk_transform",
                        lambda scores, stride, lens, batch, most, *a: made.__setitem__("transform", (stride, most)))

    def run(row, pages, page, most=None):
        made.clear()
        i32 = dict(dtype=torch.int32)
        api.topk_transform(torch.zeros(3, row), torch.zeros(3, **i32), torch.zeros(3, pages, **i32), page, 4, max_seq_len=most)
        return made["plan"], *made["transform"]

    return run


@pytest.mark.parametrize("row,pages,page,most", [
    (8, 5, 1, 5), (8, 3, 2, 6),   # rows of scores padded to a multiple of 4, past the last page
    (8, 8, 1, 8), (64, 4, 16, 64),
    (60, 4, 16, 60),              # narrower than the pages
])
def test_length_where_none_is_given(calls, row, pages, page, most):
    assert calls(row, pages, page) == (most, row, most)


def test_a_length_that_is_given_stays(calls):
    assert calls(8, 5, 1, 4) == (4, 8, 4)
    assert calls(8, 5, 1, 8) == (8, 8, 8)  # past the pages: the library refuses it
