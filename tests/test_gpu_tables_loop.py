"""A decode loop in which one step's lengths are the next step's context."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_serve import i32, plain_tables

pytestmark = pytest.mark.gpu


def test_two_results_in_turn():
    from sparse_attention_indexer_uint32_gb300 import api

    page, batch, width = 4, 300, 6
    context = [(7 * b) % 17 for b in range(batch)]
    new = [b % 3 for b in range(batch)]
    ids = torch.randperm(2 * batch * width).tolist()
    table = [ids[b * width:(b + 1) * width] for b in range(batch)]
    free, pair = ids[batch * width:], [None, None]
    dev_table, lens, dev_free = i32(table), i32(context), i32(free)
    for step in range(4):
        pair[step % 2] = got = api.block_tables(lens, i32(new), dev_free, dev_table, page, sum(new), out=pair[step % 2])
        want = plain_tables(context, new, free, table, page, sum(new))
        for name, x in zip(got._fields, want):
            assert getattr(got, name).tolist() == x, (step, name)
        assert dev_table.tolist() == table
        context, lens, free = want[0], got.seq_lens, free[want[5][0]:]
        dev_free = dev_free[want[5][0]:]
    before = [t.clone() for t in pair[1]], dev_table.clone()
    with pytest.raises(ValueError, match="out.seq_lens must not lie over context_lens"):
        api.block_tables(pair[1].seq_lens, i32(new), dev_free, dev_table, page, sum(new), out=pair[1])
    assert all(torch.equal(a, b) for a, b in zip(before[0], pair[1])) and torch.equal(before[1], dev_table)


def test_lengths_between_the_tables_rows():
    """A wide buffer with the pages of each row, and the lengths in the gap behind the first row."""
    from sparse_attention_indexer_uint32_gb300 import api

    wide = torch.zeros(3, 12, dtype=torch.int32, device="cuda")
    context, new = wide[0, 4:7], wide[0, 7:10]
    new.fill_(5)
    got = api.block_tables(context, new, i32(range(1, 7)), wide[:, :4], 4, 15)
    assert got.seq_lens.tolist() == [5, 5, 5] and got.status.tolist() == [6, 0]
    assert wide[:, :4].tolist() == [[1, 2, 0, 0], [3, 4, 0, 0], [5, 6, 0, 0]]
