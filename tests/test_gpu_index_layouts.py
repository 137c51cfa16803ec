"""Scores with every number of columns a query has and in both forms of a chunk:
one product of several queries, and two products from one place in shared
memory.  Which of them a call takes follows from its sizes, so the sizes here are
held against the rule."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_index import INDEX, api, i32, paged, randn, run  # noqa: F401 - a fixture

pytestmark = pytest.mark.gpu
TILE, COLUMNS = 128, 256  # keys of a tile; columns of a product


def chunk(batch, total, heads, max_len, sms):
    """Queries of a product and log2 of a chunk's, as launch_index_scores has them."""
    log2_heads = max(4, (heads - 1).bit_length())
    most, log2 = 8 - log2_heads, 0
    while log2 <= most and batch << log2 < total:
        log2 += 1
    tiles = lambda x: ((total + (1 << x) - 1 >> x) + (batch if x else 0)) * -(-max_len // TILE)  # noqa: E731
    while log2 > 0 and 2 * tiles(log2) < 3 * sms:
        log2 -= 1
    return 1 << most, log2


def scores(api, heads, new, past, two, dtype, page=64):  # noqa: F811
    lens = [a + b for a, b in zip(new, past)]
    width = -(-max(lens) // page)
    total = sum(new) + 1  # a row behind the last request
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    product, log2 = chunk(len(new), total, heads, width * page, sms)
    assert 1 << log2 == (2 if two else 1) * product, (product, log2)
    cache, table = paged(heads, len(new), width, page, dtype)
    run(api, randn(heads + 1, total, heads, INDEX, dtype=dtype), randn(heads + 2, total, heads, dtype=torch.float32), cache,
        i32(lens), table, page, cu=i32([0] + torch.tensor(new).cumsum(0).tolist()))


HEADS = [5, 16, 24, 32, 48, 64, 100, 128, 200, 256]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads", HEADS)
def test_two_products(api, heads, dtype):  # noqa: F811
    one = COLUMNS // (1 << max(4, (heads - 1).bit_length()))  # queries of a product
    # The last chunks: a second product of one query; a first one alone, not full; whole.
    new = [2 * one * (150 // one) + one + 1, 2 * one + max(one - 1, 1), 2 * one * (90 // one), 0, 2 * one + 1]
    scores(api, heads, new, [1700, 2900, 0, 77, 130], True, dtype)


@pytest.mark.parametrize("heads", [h for h in HEADS if h <= 128])
def test_products_of_several_queries(api, heads):  # noqa: F811
    one = COLUMNS // (1 << max(4, (heads - 1).bit_length()))
    new = [one, one - 1, 1, one, one, one - 1, one]
    scores(api, heads, new, [4000, 2900, 127, 0, 1000, 513, 128], False, torch.bfloat16)


def test_a_piece_among_single_queries(api):  # noqa: F811
    """Chunks go by the mean number of queries: this piece is cut in many, and single queries get room for four."""
    new = [1] * 40 + [200] + [1] * 20
    lens = [97 * i % 3000 + 1 for i in range(60)]
    past = lens[:40] + [2000] + lens[40:]
    cache, table = paged(1, 61, 50, 64, torch.bfloat16)
    run(api, randn(2, 260, 64, INDEX), randn(3, 260, 64, dtype=torch.float32), cache, i32([a + b for a, b in zip(new, past)]),
        table, 64, cu=i32([0] + torch.tensor(new).cumsum(0).tolist()))


@pytest.mark.parametrize("heads", [5, 64, 256])
def test_more_queries_than_positions(api, heads):  # noqa: F811
    """A request's first queries see nothing, whole chunks of them; others beside it see what they see."""
    new, lens = [700, 40, 3, 300, 90], [100, 7, 3000, 0, 2900]
    cache, table = paged(1, 5, 48, 64, torch.bfloat16)
    total = sum(new)
    run(api, randn(2, total, heads, INDEX), randn(3, total, heads, dtype=torch.float32), cache, i32(lens), table, 64,
        cu=i32([0] + torch.tensor(new).cumsum(0).tolist()))
