"""The bounded waits of the index scores and of attention behind a shared
prompt: one that gives up ends its call with the flag set and leaves the next
call right.  Under a limit of up to 100 us a block takes no wait that is not
over; a longer one runs out by the clock.  Nothing faults."""
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


def scores(api, batch, queries, heads, length, page, dtype=torch.bfloat16):
    pages = -(-length // page)
    q, weights = randn(1, batch * queries, heads, 128, dtype=dtype), randn(2, batch * queries, heads, dtype=torch.float32)
    cache = randn(3, batch * pages * page, 128, dtype=dtype)
    table = i32(torch.randperm(batch * pages, device="cuda").reshape(batch, pages))
    lens = i32([max(0, length - 37 * r) for r in range(batch)])

    def call():
        out = torch.zeros(batch * queries, pages * page, device="cuda")
        return (api.index_scores(q, weights, cache, lens, table, page, out=out),)

    return call


def shared(api, batch, queries, heads, common, own, page, dtype=torch.bfloat16):
    pages, width = -(-common // page), -(-(common + own) // page)
    q, cache = randn(4, batch, queries, heads, 576, dtype=dtype), randn(5, (pages + batch * width) * page, 576, dtype=dtype)
    ids = i32(torch.randperm(pages + batch * width, device="cuda"))
    table, lens = ids[pages:].reshape(batch, width).contiguous(), i32([common + max(0, own - 37 * r) for r in range(batch)])
    return lambda: api.attend_shared(q, cache, lens, table, ids[:pages], i32([common]), page, SCALE)[:2]


CALLS = {
    "scores, one query": lambda api: scores(api, 40, 1, 64, 9000, 64),
    "scores, many requests": lambda api: scores(api, 700, 2, 16, 900, 16),
    "scores, a prompt": lambda api: scores(api, 1, 900, 64, 4000, 64, torch.float16),
    "scores, 200 heads": lambda api: scores(api, 3, 40, 200, 3000, 32),
    "scores, small pages": lambda api: scores(api, 9, 3, 40, 1500, 2),
    "shared, 128 heads": lambda api: shared(api, 9, 1, 128, 5000, 2000, 64),
    "shared, 16 heads": lambda api: shared(api, 40, 2, 16, 9000, 700, 32, torch.float16),
    "shared, few rows": lambda api: shared(api, 3, 1, 16, 6000, 300, 64),
    "shared, small pages": lambda api: shared(api, 20, 1, 32, 700, 300, 4),
}


def run(lib, call, limit):
    with tuning(wait_limit_us=limit):
        got = call()
    return got, lib.topk_read_attend_flags(clear=True)


@pytest.mark.parametrize("name", CALLS)
def test_a_wait_that_gives_up_and_the_next_call(lib, api, name):
    call = CALLS[name](api)
    lib.topk_read_attend_flags(clear=True)
    want, flags = run(lib, call, 0)
    assert flags == 0
    # (everything may be there at the first look)
    assert any(run(lib, call, 1)[1] == lib.TOPK_FLAG_TIMEOUT for _ in range(4))
    for limit in (0, 60000000):
        got, flags = run(lib, call, limit)
        assert flags == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


# The queries of a block's next piece wait longer than 100 us for its place: of
# requests those of the fourth for the second's end (about 300 tiles of 0.75 us).
LONG = {
    "scores, requests": lambda api: scores(api, 600, 1, 64, 40000, 64),
    "scores, a prompt": lambda api: scores(api, 1, 2048, 64, 60000, 64),
    "shared": lambda api: shared(api, 64, 1, 16, 200000, 2000, 64),
}


@pytest.mark.parametrize("name", LONG)
def test_a_wait_that_runs_out_in_mid_run(lib, api, name):
    call = LONG[name](api)
    lib.topk_read_attend_flags(clear=True)
    want, flags = run(lib, call, 0)
    assert flags == 0
    assert run(lib, call, 101)[1] == lib.TOPK_FLAG_TIMEOUT
    got, flags = run(lib, call, 0)
    assert flags == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
