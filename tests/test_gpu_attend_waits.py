"""The attention kernels' bounded waits: none gave up in the tests of the files
before this one, and one that does ends its call with the flag set and leaves
the next call right.  Under a limit of up to 100 us a block takes no wait that
is not over; a longer one runs out by the clock.  Nothing faults."""
from __future__ import annotations

import pytest
import torch

from tests.parity_util import tuning

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_uint32_gb300 import _lib

    return _lib


@pytest.fixture(scope="module")
def api(lib):
    from sparse_attention_indexer_uint32_gb300 import api

    return api


def randn(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def selected(api, rows, heads, k):
    q, cache = randn(1, rows, heads, 576), randn(2, 200000, 576)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    slots = i32(torch.randint(0, 200000, (rows, k), generator=g, device="cuda"))
    return lambda: api.attend_selected(q, cache, slots, SCALE)[:2]


def paged(api, batch, queries, heads, length, page):
    pages = -(-length // page)
    q, cache = randn(4, batch, queries, heads, 576, dtype=torch.float16), randn(5, batch * pages * page, 576, dtype=torch.float16)
    table = i32(torch.randperm(batch * pages, device="cuda").reshape(batch, pages))
    lens = i32([length - 37 * r for r in range(batch)])
    return lambda: api.attend_paged(q, cache, lens, table, page, SCALE)[:2]


def paged_by_rows(api):
    """Queries whose heads are not next to their neighbours': copied a row at a time."""
    q, cache = randn(6, 6, 3, 50, 576)[:, :, :40], randn(7, 6 * 1024, 576)
    table, lens = i32(torch.arange(96, device="cuda").reshape(6, 16)), i32([1024, 3, 700, 0, 1000, 90])
    return lambda: api.attend_paged(q, cache, lens, table, 64, SCALE)[:2]


def prompt(api, lq, lk, heads):
    q, up, rope = randn(8, lq, heads, 192), randn(9, lk, heads, 256), randn(10, lk, 64)
    marks = i32([0, lq]), i32([0, lk])
    return lambda: api.attend_prompt(q, up[..., :128], rope, up[..., 128:], *marks, SCALE)


CALLS = {
    "selected, 128 heads": lambda api: selected(api, 100, 128, 1000),
    "selected, 16 heads": lambda api: selected(api, 300, 16, 500),
    "selected, several groups of rows": lambda api: selected(api, 20, 300, 700),
    "paged, 128 heads": lambda api: paged(api, 9, 1, 128, 9000, 64),
    "paged, 16 heads": lambda api: paged(api, 90, 2, 16, 4000, 16),
    "paged, small pages": lambda api: paged(api, 9, 1, 64, 900, 4),
    "paged, queries by rows": paged_by_rows,
    "prompt": lambda api: prompt(api, 3000, 4000, 8),
    "prompt, shared pieces": lambda api: prompt(api, 200, 6000, 2),
}


def test_no_wait_gave_up_before(lib):
    assert lib.topk_read_attend_flags(clear=True) == 0


@pytest.mark.parametrize("name", CALLS)
def test_a_wait_that_gives_up_and_the_next_call(lib, api, name):
    call = CALLS[name](api)
    want = call()
    assert lib.topk_read_attend_flags() == 0
    seen = 0
    for _ in range(4):  # everything may be there at the first look
        with tuning(wait_limit_us=1):
            call()
        seen |= lib.topk_read_attend_flags(clear=True)
        if seen:
            break
    assert seen == lib.TOPK_FLAG_TIMEOUT
    for limit in (0, 60000000):
        with tuning(wait_limit_us=limit):
            got = call()
        assert lib.topk_read_attend_flags() == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# Long pieces of work, whose queries (or, for prompts, whose place) the next
# piece waits for longer than 100 us: that wait runs out by the clock, while
# copies and products are under way.
LONG = {
    "selected": lambda api: selected(api, 8, 128, 150000),
    "paged, 128 heads": lambda api: paged(api, 16, 1, 128, 80000, 64),
    # (two places for queries: runs of three rows)
    "paged, 16 heads": lambda api: paged(api, 150, 1, 16, 20000, 64),
    "prompt": lambda api: prompt(api, 20000, 40000, 4),
}


@pytest.mark.parametrize("name", LONG)
def test_a_wait_that_runs_out_in_mid_run(lib, api, name):
    call = LONG[name](api)
    want = call()
    assert lib.topk_read_attend_flags() == 0
    with tuning(wait_limit_us=101):
        call()
    assert lib.topk_read_attend_flags(clear=True) == lib.TOPK_FLAG_TIMEOUT
    got = call()
    assert lib.topk_read_attend_flags() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
