"""The indexer's side of a step: keys appended to their paged cache, and scores
over it, against plain 64-bit forms."""
from __future__ import annotations

import math

import pytest
import torch

from tests.attend_util import check
from tests.index_util import INDEX, ROPE, append, check_scores

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def api():
    from sparse_attention_indexer_uint32_gb300 import api

    return api


def randn(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def perm(seed, n):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32)


def turns(n):
    angle = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(ROPE // 2, device="cuda", dtype=torch.float64) / (ROPE // 2))
    return torch.cat((angle.cos(), angle.sin()), 1).float()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [1, 2, 17, 301, 2433, 40000])
@pytest.mark.parametrize("interleaved,rope_last", [(False, False), (True, False), (False, True), (True, True)])
def test_append(api, dtype, tokens, interleaved, rope_last):
    n = tokens + 13
    wide = randn(1, tokens, INDEX + 24, dtype=dtype)
    rows = wide[:, 8:8 + INDEX] + 3  # a mean that is not zero
    rows = torch.cat((rows, wide[:, :24]), 1)[:, :INDEX]
    slots, cos_sin = perm(2, n)[:tokens].clone(), turns(500)
    slots[::7] = -1
    if tokens > 5:
        slots[3], slots[4] = n, 2 ** 31 - 1  # not in the cache
    positions = i32(torch.arange(tokens) * 37 % 500)
    if tokens > 20:
        positions[15], positions[16] = 500, -1  # not in the table of angles: not written
    weight, bias = 1 + randn(3, INDEX, dtype=dtype) / 8, randn(4, INDEX, dtype=dtype) / 8
    store = randn(5, n, 2 * INDEX, dtype=dtype)
    before = store.clone()
    api.index_append(rows, slots, store[:, :INDEX], norm_weight=weight, norm_bias=bias, eps=1e-5, cos_sin=cos_sin,
                     positions=positions, interleaved=interleaved, rope_last=rope_last)
    keep = (slots >= 0) & (slots < n) & (positions >= 0) & (positions < 500)
    want, bound = append(rows[keep], weight, bias, 1e-5, cos_sin, positions[keep], interleaved, rope_last)
    check(store[slots[keep].long(), :INDEX], want, bound, "rows")
    left = torch.ones(n, dtype=torch.bool, device="cuda")
    left[slots[keep].long()] = False
    assert torch.equal(store[left], before[left]) and torch.equal(store[:, INDEX:], before[:, INDEX:])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("norm,bias,rope", [(False, False, False), (True, False, False), (False, False, True), (True, True, False)])
def test_append_parts(api, dtype, norm, bias, rope):
    tokens = 77
    rows, cache = randn(1, tokens, INDEX, dtype=dtype) * 5, torch.zeros(tokens, INDEX, dtype=dtype, device="cuda")
    rows[3] = 0  # no spread: the norm gives the bias
    rows[4] = 2
    w, b = randn(2, INDEX, dtype=dtype) if norm else None, randn(3, INDEX, dtype=dtype) if bias else None
    cos_sin, positions = (turns(80), i32(torch.arange(tokens))) if rope else (None, None)
    api.index_append(rows, i32(torch.arange(tokens)), cache, norm_weight=w, norm_bias=b, cos_sin=cos_sin, positions=positions)
    want, bound = append(rows, w, b, 1e-6, cos_sin, positions, False, False)
    check(cache, want, bound, "rows")
    if not norm and not rope:
        assert torch.equal(cache, rows)


def test_append_nothing_and_special_rows(api):
    cache = randn(1, 9, INDEX)
    before = cache.clone()
    api.index_append(torch.empty(0, INDEX, dtype=torch.bfloat16, device="cuda"), i32([]), cache)
    assert torch.equal(cache, before)
    rows = randn(2, 4, INDEX)
    rows[1, 5], rows[2, 9] = math.nan, math.inf
    api.index_append(rows, i32([0, 1, 2, 3]), cache, norm_weight=torch.ones(INDEX, dtype=torch.bfloat16, device="cuda"))
    want, bound = append(rows[[0, 3]], torch.ones(INDEX, device="cuda"), None, 1e-6, None, None, False, False)
    check(cache[[0, 3]], want, bound, "rows beside those with a NaN and an infinity")
    assert cache[1:3].isnan().all() and torch.equal(cache[4:], before[4:])


def test_append_replayed_and_on_another_stream(api):
    tokens, n = 300, 400
    rows, slots, cos_sin = randn(1, tokens, INDEX), perm(2, n)[:tokens].clone(), turns(500)
    positions, weight, bias = i32(torch.arange(tokens)), 1 + randn(3, INDEX) / 8, randn(4, INDEX) / 8
    more = dict(norm_weight=weight, norm_bias=bias, cos_sin=cos_sin, positions=positions)
    cache, other = torch.zeros(n, INDEX, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, INDEX, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    api.index_append(rows, slots, other, stream=stream, **more)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        api.index_append(rows, slots, cache, **more)
    for seed in (7, 8):
        rows.copy_(randn(seed, tokens, INDEX))
        slots.copy_(perm(seed, n)[:tokens])
        positions.copy_(perm(seed + 10, 500)[:tokens])
        graph.replay()
        torch.cuda.synchronize()
        want, bound = append(rows, weight, bias, 1e-6, cos_sin, positions, False, False)
        check(cache[slots.long()], want, bound, "rows")
    assert other.any()


def paged(seed, batch, width, page, dtype, spare=3, slot_room=INDEX):
    cache = randn(seed, (batch * width + spare) * page, slot_room, dtype=dtype)[:, :INDEX]
    return cache, perm(seed + 1, batch * width + spare)[: batch * width].reshape(batch, width)


def run(api, q, weights, cache, lens, table, page, cu=None, max_len=None, room=0, **more):
    most = table.shape[1] * page if max_len is None else max_len
    out = torch.full((q.shape[0], most + room), 7.0, device="cuda")
    before = out.clone()
    got = api.index_scores(q, weights, cache, lens, table, page, cu_q=cu, max_seq_len=max_len, out=out, **more)
    assert got is out
    check_scores(q, weights, cache, lens, table, page, out, before, cu, max_len)
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", [1, 3, 8, 16, 17, 32, 40, 64, 65, 100, 128, 200, 256])
@pytest.mark.parametrize("queries", [1, 3])
def test_scores_heads(api, dtype, heads, queries):
    lens = i32([0, 1, 127, 128, 129, 300])
    cache, table = paged(1, 6, 5, 64, dtype)
    run(api, randn(3, 6 * queries, heads, INDEX, dtype=dtype), randn(4, 6 * queries, heads, dtype=torch.float32), cache, lens,
        table, 64)


@pytest.mark.parametrize("page", [1, 2, 8, 16, 32, 64, 128, 256, 1024])
def test_scores_pages(api, page):
    width = max(1, 1500 // page)
    lens = i32([1, width * page, min(700, width * page), 13])
    cache, table = paged(1, 4, width, page, torch.bfloat16, slot_room=INDEX + 8)
    run(api, randn(3, 8, 24, INDEX), randn(4, 8, 24, dtype=torch.float32), cache, lens, table, page, room=5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,new,past", [
    (64, [1, 9, 300, 0, 17], [0, 200, 100, 40, 1000]), (16, [700], [0]), (100, [33, 5], [0, 257]), (48, [64, 1, 1, 40], [130, 0, 600, 9]),
    (4, [500, 129], [3, 1100]), (130, [5, 9], [100, 7]), (64, [1024], [512])])
def test_scores_ragged(api, dtype, heads, new, past):
    page = 32
    lens = [a + b for a, b in zip(new, past)]
    cu = i32([0] + torch.tensor(new).cumsum(0).tolist())
    cache, table = paged(1, len(new), (max(lens) + page - 1) // page, page, dtype)
    total = sum(new) + 2  # two rows behind the last request
    run(api, randn(3, total, heads, INDEX, dtype=dtype), randn(4, total, heads, dtype=torch.float32), cache, i32(lens), table, page,
        cu=cu)


def test_scores_many_requests(api):
    """More requests than threads, with empty ones among them."""
    b = 1500
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(-3, 70, (b,), generator=g)
    cache, table = paged(1, b, 4, 16, torch.bfloat16)
    run(api, randn(3, b, 8, INDEX), randn(4, b, 8, dtype=torch.float32), cache, i32(lens), table, 16)


def test_scores_long(api):
    lens, page = i32([40000, 9]), 64
    cache, table = paged(1, 2, 625, page, torch.float16)
    run(api, randn(3, 2, 64, INDEX, dtype=torch.float16), randn(4, 2, 64, dtype=torch.float32), cache, lens, table, page)


def test_scores_strides_and_limits(api):
    cache, table = paged(1, 3, 8, 16, torch.bfloat16, slot_room=3 * INDEX)
    q = randn(2, 6, 12, 3 * INDEX)[:, ::2, INDEX:2 * INDEX]  # [6, 6, 128], wide strides
    weights = randn(3, 6, 20, dtype=torch.float32)[:, 3:9]
    lens = i32([500, 90, 4])  # the first is past max_seq_len
    wide = torch.cat((table, table), 1)[:, :8]
    run(api, q, weights, cache, lens, wide, 16, max_len=100, room=3)
    # Heads before tokens.
    q = randn(5, 4, 6, INDEX).transpose(0, 1)
    run(api, q, randn(6, 6, 4, dtype=torch.float32), cache, i32([40, 128, 1]), table, 16)


def test_scores_pages_out_of_the_cache(api):
    cache, table = paged(1, 2, 10, 16, torch.bfloat16)
    table = table.clone()
    table[0, 2], table[0, 5], table[1, 0] = -1, cache.shape[0] // 16, 2 ** 31 - 1
    run(api, randn(2, 4, 16, INDEX), randn(3, 4, 16, dtype=torch.float32), cache, i32([160, 33]), table, 16)
    # A page that the cache's end cuts.
    run(api, randn(2, 4, 16, INDEX), randn(3, 4, 16, dtype=torch.float32), cache[: cache.shape[0] - 7], i32([160, 33]), table, 16)
    lens, tables = i32([60, 0]), i32([[-1] * 4] * 2)  # nothing of it is there
    run(api, randn(2, 2, 16, INDEX), randn(3, 2, 16, dtype=torch.float32), cache, lens, tables, 16)


def test_scores_what_is_not_seen_may_be_anything(api):
    cache, table = paged(1, 2, 4, 64, torch.bfloat16)
    lens = i32([70, 130])
    rest = torch.ones(cache.shape[0], dtype=torch.bool, device="cuda")
    for b in range(2):
        t = torch.arange(int(lens[b]), device="cuda")
        rest[table[b].long()[t // 64] * 64 + t % 64] = False
    cache[rest] = math.nan
    run(api, randn(2, 2, 64, INDEX), randn(3, 2, 64, dtype=torch.float32), cache, lens, table, 64)
    # A key that is seen and holds a NaN: its own score only.
    cache[int(table[1, 1]) * 64 + 3, 5] = math.nan
    out = run(api, randn(2, 2, 64, INDEX), randn(3, 2, 64, dtype=torch.float32), cache, lens, table, 64)
    assert out[1].isnan().sum() == 1


def test_scores_large_offsets(api):
    """Rows of the cache, and of the result, past 2^31 values."""
    page, n = 64, (2 ** 31 // INDEX + 4096) // 64 * 64
    cache = torch.empty(n, INDEX, dtype=torch.bfloat16, device="cuda")
    table = i32([[n // page - 1, 3], [n // page - 2, n // page - 5]])
    for p in table.flatten().tolist():
        cache[p * page:(p + 1) * page] = randn(p % 1000, page, INDEX)
    q, weights = randn(1, 2, 64, INDEX), randn(2, 2, 64, dtype=torch.float32)
    small = cache[torch.cat([torch.arange(p * page, (p + 1) * page, device="cuda") for p in table.flatten().tolist()])]
    want = api.index_scores(q, weights, small, i32([100, 128]), i32([[0, 1], [2, 3]]), page)
    got = api.index_scores(q, weights, cache, i32([100, 128]), table, page)
    assert torch.equal(got[0, :100], want[0, :100]) and torch.equal(got[1], want[1])
    del cache
    out = torch.empty(2, 2 ** 31 + 8, device="cuda")
    api.index_scores(q, weights, small, i32([100, 128]), i32([[0, 1], [2, 3]]), page, max_seq_len=128, out=out)
    assert torch.equal(out[0, :100], want[0, :100]) and torch.equal(out[1, :128], want[1])


def test_scores_default_result_feeds_the_selection(api):
    b, page, k = 3, 64, 100
    lens = i32([37, 500, 640])
    cache, table = paged(1, b, 10, page, torch.bfloat16)
    q, weights = randn(2, b, 32, INDEX), randn(3, b, 32, dtype=torch.float32)
    out = api.index_scores(q, weights, cache, lens, table, page)
    assert out.shape == (b, 640) and out.dtype == torch.float32
    slots, raw, _ = api.topk_transform(out, lens, table, page, k, want_raw=True)
    for r in range(b):
        n = min(int(lens[r]), k)
        order = out[r, : int(lens[r])].double()
        floor = order.topk(n).values.min()
        assert (order[raw[r, :n].long()] >= floor).all() and (raw[r, n:] == -1).all() and raw[r, :n].unique().numel() == n


def test_scores_nothing(api):
    cache, table = paged(1, 2, 2, 16, torch.bfloat16)
    none = api.index_scores(torch.empty(0, 4, INDEX, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 4, device="cuda"), cache,
                            i32([3, 4]), table, 16)
    assert none.shape == (0, 32)
    run(api, randn(2, 2, 4, INDEX), randn(3, 2, 4, dtype=torch.float32), cache, i32([0, -5]), table, 16)
    out = torch.full((2, 4), 7.0, device="cuda")
    api.index_scores(randn(2, 2, 4, INDEX), randn(3, 2, 4, dtype=torch.float32), cache, i32([3, 3]), table, 16, max_seq_len=0, out=out)
    assert (out == 7).all()


def test_scores_offsets_that_are_not_in_order(api):
    """Offsets outside the queries are clamped; a request that ends before it begins has none."""
    cache, table = paged(1, 4, 8, 16, torch.bfloat16)
    run(api, randn(2, 9, 8, INDEX), randn(3, 9, 8, dtype=torch.float32), cache, i32([100, 128, 60, 77]), table, 16, cu=i32([-4, 3, 9, 5, 5]))


@pytest.mark.parametrize("heads", [7, 16, 64])
def test_scores_of_infinite_keys(api, heads):
    """Infinities in a key go to its own score, and padding columns add nothing to them."""
    cache, table = paged(1, 1, 4, 64, torch.bfloat16)
    q, weights = randn(2, 2, heads, INDEX).abs(), randn(3, 2, heads, dtype=torch.float32).abs() + 1
    at = table[0].long()[:, None].mul(64).add(torch.arange(64, device="cuda")).flatten()
    cache[at[3], 7], cache[at[9], 8] = math.inf, -math.inf  # (no query value is zero)
    out = run(api, q, weights, cache, i32([200]), table, 64)
    assert (out[:, 3] == math.inf).all() and (out[:, 9] == 0).all() and not out[:, :199].isnan().any()


def test_scores_replayed_with_other_lengths(api):
    page, b = 32, 3
    cache, table = paged(1, b, 40, page, torch.bfloat16)
    q, weights, lens = randn(2, 2 * b, 64, INDEX), randn(3, 2 * b, 64, dtype=torch.float32), i32([1, 1, 1])
    out = torch.full((2 * b, 40 * page), 7.0, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        api.index_scores(q, weights, cache, lens, table, page, out=out)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        api.index_scores(q, weights, cache, lens, table, page, out=out)
    for now in ([5, 1280, 700], [0, 3, 129]):
        out.fill_(7.0)
        lens.copy_(i32(now))
        before = out.clone()
        graph.replay()
        torch.cuda.synchronize()
        check_scores(q, weights, cache, lens, table, page, out, before)


def test_scores_on_two_streams(api):
    page, b = 64, 5
    cache, table = paged(1, b, 30, page, torch.float16)
    lens = i32([1900, 3, 700, 64, 1000])
    sets = [(randn(10 + i, b, 16, INDEX, dtype=torch.float16), randn(20 + i, b, 16, dtype=torch.float32)) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [torch.full((b, 30 * page), 7.0, device="cuda") for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for (q, w), s, out in zip(sets, streams, outs):
            api.index_scores(q, w, cache, lens, table, page, out=out, stream=s)
    torch.cuda.synchronize()
    for (q, w), out in zip(sets, outs):
        check_scores(q, w, cache, lens, table, page, out, torch.full_like(out, 7.0))


def test_scores_into_new_memory_on_another_stream(api):
    page = 64
    cache, table = paged(1, 3, 10, page, torch.float16)
    q, w, lens = randn(2, 6, 24, INDEX, dtype=torch.float16), randn(3, 6, 24, dtype=torch.float32), i32([600, 1, 77])
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for s in (stream, stream.cuda_stream, None):
        out = api.index_scores(q, w, cache, lens, table, page, max_seq_len=630, stream=s)
        torch.cuda.synchronize()
        assert out.shape == (6, 632)
        before = out.clone()
        for i in range(6):  # (what is not seen is whatever the memory held)
            before[i, : int(lens[i // 2]) - (1 - i % 2)] = 0
        check_scores(q, w, cache, lens, table, page, out, before, max_len=630)


def test_scores_equal_calls_give_equal_bits(api):
    cache, table = paged(1, 7, 30, 64, torch.bfloat16)
    args = (randn(2, 7, 64, INDEX), randn(3, 7, 64, dtype=torch.float32), cache, i32([1900, 3, 700, 64, 1000, 1, 1920]), table, 64)
    first = torch.zeros(7, 1920, device="cuda")
    api.index_scores(*args, out=first)
    for _ in range(3):
        again = torch.zeros_like(first)
        api.index_scores(*args, out=again)
        assert torch.equal(first, again)
