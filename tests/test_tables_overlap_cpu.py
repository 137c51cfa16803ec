"""Block tables whose outputs lie over their inputs are refused on the host: a
step's lengths are read again after the next ones are written."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_indexer_uint32_gb300 import build as build_mod

BATCH, PAGES, STRIDE, FREE, TOKENS = 4, 8, 20, 5, 16


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    from sparse_attention_indexer_uint32_gb300 import _lib

    return _lib


def place(**over):
    """Addresses (in int32 values from a base) of every argument, far apart unless given."""
    at = dict(context=0, new=1000, free=2000, table=3000, seq=4000, cu=5000, slots=6000, positions=7000, rows=8000,
              status=9000)
    assert set(over) <= set(at)
    return {n: (1 << 20) + 4 * x for n, x in {**at, **over}.items()}


def call(lib, num_free=FREE, max_tokens=TOKENS, **over):
    a = place(**over)
    return lib.library().topk_block_tables(a["context"], a["new"], BATCH, 64, a["free"], num_free, a["table"],
                                           STRIDE, PAGES, max_tokens, a["seq"], a["cu"], a["slots"], a["positions"],
                                           a["rows"], a["status"], None)


LENGTHS = dict(context=BATCH, new=BATCH, free=FREE)
OUTPUTS = dict(seq=BATCH, cu=BATCH + 1, slots=TOKENS, positions=TOKENS, rows=TOKENS, status=2)


@pytest.mark.parametrize("out", OUTPUTS)
@pytest.mark.parametrize("source", LENGTHS)
def test_outputs_over_lengths_and_list(lib, out, source):
    at = 1000 * list(LENGTHS).index(source)
    for offset in (0, LENGTHS[source] - 1, 1 - OUTPUTS[out]):  # the same place, the last value, the first
        assert call(lib, **{out: at + offset}) == lib.TOPK_EINVAL, offset


@pytest.mark.parametrize("out,n", [*OUTPUTS.items(), *LENGTHS.items()])
def test_anything_over_the_table(lib, out, n):
    """Rows of 8 pages, 20 apart; what lies between two rows may be anybody's."""
    for row in range(BATCH):
        for offset in (0, PAGES - 1, 1 - n):
            assert call(lib, **{out: 3000 + row * STRIDE + offset}) == lib.TOPK_EINVAL, (row, offset)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real: nothing may be launched on them")
def test_neighbours_are_taken(lib):
    """Arrays that touch, or lie between the table's rows, get past the check (and end at the missing GPU)."""
    refused = (lib.TOPK_EINVAL, lib.TOPK_EALIGN)
    for out, n in OUTPUTS.items():
        for source, m in LENGTHS.items():
            at = 1000 * list(LENGTHS).index(source)
            for offset in (m, -n):
                assert call(lib, **{out: at + offset}) not in refused, (out, source, offset)
    for name, n in {**OUTPUTS, **LENGTHS}.items():
        for at in (3000 - n, 3000 + (BATCH - 1) * STRIDE + PAGES):
            assert call(lib, **{name: at}) not in refused, (name, at)
        if n <= STRIDE - PAGES:
            for at in (3000 + PAGES, 3000 + 2 * STRIDE - n):
                assert call(lib, **{name: at}) not in refused, (name, at)
    # A list and token arrays without a value lie over nothing.
    assert call(lib, max_tokens=0, slots=0, positions=1000, rows=3000) not in refused
    assert call(lib, num_free=0, free=4000) not in refused


def test_the_message_names_the_pair(lib):
    from sparse_attention_indexer_uint32_gb300 import api

    flat = torch.zeros(100, dtype=torch.int32)
    step = api.BlockTables(flat[:3], flat[10:14], flat[20:30], flat[30:40], flat[40:50], flat[50:52])
    new, free, table = flat[60:63], flat[70:75], flat[80:92].reshape(3, 4)
    api._check_overlap(flat[95:98], new, free, table, step)
    with pytest.raises(ValueError, match="out.seq_lens must not lie over context_lens"):
        api._check_overlap(step.seq_lens, new, free, table, step)
    with pytest.raises(ValueError, match="page_table must not lie over free_pages"):
        api._check_overlap(flat[95:98], new, table[1], table, step)
