"""Attention over the latent cache (selected slots, whole rows through the page
table) and for prompts, against a plain 64-bit implementation, at the sizes and
masks where such kernels go wrong."""
from __future__ import annotations

import math

import pytest
import torch

from tests.attend_util import attend, check

pytestmark = pytest.mark.gpu

LATENT, WIDTH, SCALE = 512, 576, 192 ** -0.5
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


def check_selected(q, cache, indices, lens, out, lse, scale=SCALE):
    for r in range(q.shape[0]):
        idx = indices[r, : max(0, int(lens[r]))] if lens is not None else indices[r]
        idx = idx[(idx >= 0) & (idx < cache.shape[0])].long()
        kv = cache[idx]
        o, l, ob, lb = attend(q[r], kv, kv[:, :LATENT], scale, q.dtype)
        check(out[r], o, ob, f"out of row {r}")
        check(lse[r], l, lb, f"lse of row {r}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,heads,k", [
    (1, 1, 1), (1, 128, 2), (3, 16, 5), (2, 64, 63), (2, 65, 64), (2, 128, 65), (1, 127, 127), (2, 128, 128),
    (3, 100, 129), (2, 128, 300), (5, 24, 512), (1, 128, 2048), (1, 8, 4099), (200, 16, 200), (90, 128, 260),
    (2, 129, 70), (1, 300, 130)])
def test_selected(api, dtype, rows, heads, k):
    n = 5000
    q, cache = randn(1, rows, heads, WIDTH, dtype=dtype), randn(2, n, WIDTH, dtype=dtype)
    g = torch.Generator(device="cuda")
    g.manual_seed(rows * 1000 + k)
    indices = i32(torch.randint(0, n, (rows, k), generator=g, device="cuda"))
    out, lse, _ = api.attend_selected(q, cache, indices, SCALE)
    check_selected(q, cache, indices, None, out, lse)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k", [1, 60, 128, 500])
def test_selected_masks(api, dtype, k):
    """Rows with no index, one at the end, -1 in between, indices past the cache, repeated ones, and lengths of zero,
    one, below zero and past k; slots that nobody selected hold NaN and infinities."""
    n, rows = 1000, 12
    q, cache = randn(3, rows, 40, WIDTH, dtype=dtype), randn(4, n, WIDTH, dtype=dtype)
    cache[500:750] = math.nan
    cache[750:] = math.inf
    cache[0] = -math.inf
    g = torch.Generator(device="cuda")
    g.manual_seed(k)
    indices = i32(torch.randint(1, 500, (rows, k), generator=g, device="cuda"))
    indices[0] = -1
    indices[1, :-1] = -1
    indices[2, ::2] = -1
    indices[3, : k // 2] = n
    indices[4, : k // 2] = -(2 ** 31)
    indices[5, k // 2:] = 2 ** 31 - 1
    indices[6] = 7
    lens = i32([k, k, k, k, k, k, k, 0, 1, -5, k + 100, k // 2])
    indices[11, k // 2:] = 600  # past its length: not looked at
    out, lse, ws = api.attend_selected(q, cache, indices, SCALE, seq_lens=lens)
    check_selected(q, cache, indices, lens, out, lse)
    assert (out[7] == 0).all() and (lse[7] == -math.inf).all()
    again = api.attend_selected(q, cache, indices, SCALE, seq_lens=lens, workspace=ws)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("dtype", DTYPES)
def test_selected_strides_and_large_scores(api, dtype):
    """Query heads and cache rows that are slices of wider tensors; scores whose exponents span the range, the largest
    last (the running maximum rises tile by tile) or first; a negative and a zero scale."""
    q = randn(5, 6, 20, WIDTH + 64, dtype=dtype)[:, 2:18, 64:]
    cache = randn(6, 900, 2 * WIDTH, dtype=dtype)[:, WIDTH:]
    for order in (1, -1):
        grow = torch.linspace(0.0, 4.0, 900, device="cuda")[::order] if order == 1 else torch.linspace(4.0, 0.0, 900, device="cuda")
        cache.copy_((randn(7, 1, WIDTH).float() * grow[:, None]).to(dtype))
        for scale in (0.05, -0.05, 0.0):
            indices = i32(torch.arange(900, device="cuda").repeat(6, 1))
            out, lse, _ = api.attend_selected(q, cache, indices, scale)
            check_selected(q, cache, indices, None, out, lse, scale)


def test_selected_long_cache(api):
    """Element offsets past 2^32: the cache's last slots."""
    n = 2 ** 23
    cache = torch.zeros(n, WIDTH, dtype=torch.bfloat16, device="cuda")
    cache[-600:] = randn(8, 600, WIDTH)
    q = randn(9, 2, 128, WIDTH)
    indices = i32(torch.stack((torch.arange(n - 600, n, device="cuda"), torch.arange(0, n, n // 600, device="cuda")[:600])))
    out, lse, _ = api.attend_selected(q, cache, indices, SCALE)
    check_selected(q, cache, indices, None, out, lse)


def check_paged(q, cache, lens, table, page, out, lse, most=None):
    b, n, h, _ = q.shape
    for r in range(b):
        length = min(max(0, int(lens[r])), table.shape[1] * page if most is None else most)
        t = torch.arange(length, device="cuda")
        slot = table[r].long()[t // page] * page + t % page
        for i in range(n):
            s = slot[: max(0, length - (n - 1 - i))]
            kv = cache[s[(s >= 0) & (s < cache.shape[0])]]
            o, l, ob, lb = attend(q[r, i], kv, kv[:, :LATENT], SCALE, q.dtype)
            check(out[r, i], o, ob, f"out of row {r}, query {i}")
            check(lse[r, i], l, lb, f"lse of row {r}, query {i}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("queries,heads,page,most", [
    (1, 128, 64, 700), (1, 16, 1, 130), (2, 16, 16, 300), (3, 20, 32, 257), (4, 16, 128, 1000), (5, 128, 64, 200),
    (2, 100, 64, 129), (8, 16, 256, 900), (1, 7, 2, 64), (9, 15, 64, 140)])
def test_paged(api, dtype, queries, heads, page, most):
    batch = 9
    pages = -(-most // page)
    g = torch.Generator(device="cuda")
    g.manual_seed(most)
    table = torch.randperm(batch * pages + 3, generator=g, device="cuda")[: batch * pages].reshape(batch, pages)
    cache = randn(11, (batch * pages + 3) * page, WIDTH, dtype=dtype)
    lens = i32(torch.randint(0, most + 1, (batch,), generator=g, device="cuda"))
    lens[0], lens[1], lens[2], lens[3] = 0, 1, most, most + 50
    lens[4] = min(most, max(queries - 1, 2))
    table = i32(table)
    # What lies past the lengths is stale: not a number.
    t = torch.arange(pages * page, device="cuda")
    for r in range(batch):
        s = table[r].long()[t // page] * page + t % page
        cache[s[max(0, int(lens[r])):]] = math.nan
    q = randn(12, batch, queries, heads, WIDTH, dtype=dtype)
    out, lse, _ = api.attend_paged(q, cache, lens, table, page, SCALE, max_seq_len=most)
    check_paged(q, cache, lens, table, page, out, lse, most)


def test_paged_pages_out_of_range(api):
    """Pages that are negative, past the cache, or whose product passes 32 bits hide their positions."""
    page, cache = 64, randn(13, 40 * 64, WIDTH)
    table = i32(torch.arange(36, device="cuda").reshape(4, 9))
    table[0, 2], table[1, 0], table[2, 8], table[3] = -1, 40, 2 ** 31 - 1, -1
    table[1, 3] = -(2 ** 31)
    lens = i32([9 * 64, 9 * 64 - 5, 9 * 64, 9 * 64])
    q = randn(14, 4, 1, 128, WIDTH)
    out, lse, _ = api.attend_paged(q, cache, lens, table, page, SCALE)
    check_paged(q, cache, lens, table, page, out, lse)
    assert (out[3] == 0).all() and (lse[3] == -math.inf).all()


def test_paged_long_rows_share_blocks(api):
    """Rows of very different lengths, the work cut inside rows."""
    page, lens = 64, i32([20000, 3, 0, 7001, 1, 12345])
    pages = -(-20000 // page)
    table = i32(torch.randperm(6 * pages, device="cuda").reshape(6, pages))
    cache = randn(15, 6 * pages * page, WIDTH)
    q = randn(16, 6, 1, 128, WIDTH)
    out, lse, ws = api.attend_paged(q, cache, lens, table, page, SCALE)
    check_paged(q, cache, lens, table, page, out, lse)
    out2, lse2, _ = api.attend_paged(q, cache, lens, table, page, SCALE, workspace=ws)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def check_prompt(q, kn, kr, v, cu_q, cu_k, causal, out, lse, scale=SCALE):
    for r in range(len(cu_q) - 1):
        a, b = slice(cu_q[r], cu_q[r + 1]), slice(cu_k[r], cu_k[r + 1])
        nq, nk = a.stop - a.start, b.stop - b.start
        for h in range(q.shape[1]):
            k = torch.cat((kn[b, h], kr[b]), 1)
            if not causal:
                o, l, ob, lb = attend(q[a, h], k, v[b, h], scale, q.dtype)
                check(out[a, h], o, ob, f"out of request {r}, head {h}")
                check(lse[a, h], l, lb, f"lse of request {r}, head {h}")
                continue
            # Few queries each with a prefix of its own: the first, the last, those around multiples of 128, some others.
            at = {0, 1, nq - 1, nq // 2, nq // 3} | {i + d for i in range(128, nq + 1, 128) for d in (-1, 0)}
            for i in sorted(x for x in at if 0 <= x < nq):
                n = max(0, nk - (nq - 1 - i))
                t = a.start + i
                o, l, ob, lb = attend(q[t:t + 1, h], k[:n], v[b, h][:n], scale, q.dtype)
                check(out[t:t + 1, h], o, ob, f"out of request {r}, head {h}, query {i}")
                check(lse[t:t + 1, h], l, lb, f"lse of request {r}, head {h}, query {i}")


def prompt_inputs(seed, lq, lk, heads, dtype, gap=0):
    """Requests' tensors with `gap` tokens of NaN and infinities before, between and after them."""
    cu_q, cu_k = [gap], [gap]
    total_q, total_k = gap + sum(lq) + gap, gap + sum(lk) + gap
    for n in lq:
        cu_q.append(cu_q[-1] + n)
    for n in lk:
        cu_k.append(cu_k[-1] + n)
    q = randn(seed, total_q, heads, 192, dtype=dtype)
    up, kr = randn(seed + 1, total_k, heads, 256, dtype=dtype), randn(seed + 2, total_k, 64, dtype=dtype)
    if gap:
        q[:gap], q[-gap:] = math.nan, math.inf
        up[:gap], up[-gap:], kr[:gap], kr[-gap:] = math.nan, math.inf, math.inf, math.nan
    return q, up[..., :128], kr, up[..., 128:], cu_q, cu_k


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,heads", [
    ([1], [1], 1), ([1], [300], 3), ([2], [2], 2), ([127], [127], 1), ([128], [128], 2), ([129], [129], 1),
    ([257], [257], 1), ([300, 1, 64, 0, 128], [300, 1, 64, 0, 128], 3), ([5, 200], [700, 333], 2),
    ([600], [601], 1), ([130, 7], [40, 0], 2), ([0, 0, 3], [0, 9, 3], 1), ([1000], [1500], 1)])
def test_prompt(api, dtype, causal, lq, lk, heads):
    """Lengths around the tiles, requests with no query or no key, fewer keys than queries (rows that see nothing),
    and NaN or infinities in the tokens that belong to no request."""
    q, kn, kr, v, cu_q, cu_k = prompt_inputs(21, lq, lk, heads, dtype, gap=5)
    out = torch.full((q.shape[0], heads, 128), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((q.shape[0], heads), 7.0, device="cuda")
    api.attend_prompt(q, kn, kr, v, i32(cu_q), i32(cu_k), SCALE, causal=causal, out=out, lse=lse)
    check_prompt(q, kn, kr, v, cu_q, cu_k, causal, out, lse)
    for t in (out, lse):  # tokens of no request are not written
        assert (t[:5] == 7).all() and (t[-5:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_prompt_neighbours_do_not_leak(api, dtype):
    """A request's keys hold NaN: only its own queries see them."""
    lens = [130, 70, 200]
    q, kn, kr, v, cu_q, cu_k = prompt_inputs(31, lens, lens, 2, dtype)
    for t in (kn, kr, v):
        t[cu_k[1]:cu_k[2]] = math.nan
    out, lse = api.attend_prompt(q, kn, kr, v, i32(cu_q), i32(cu_k), SCALE)
    assert torch.isnan(out[cu_q[1]:cu_q[2]]).all()
    for r in (0, 2):
        check_prompt(q, kn, kr, v, [cu_q[r], cu_q[r + 1]], [cu_k[r], cu_k[r + 1]], True, out, lse)


@pytest.mark.parametrize("dtype", DTYPES)
def test_prompt_strides_and_large_scores(api, dtype):
    """Heads before tokens, slices of wider rows, one head for all (stride 0), scores that grow along the keys."""
    t, heads = 400, 3
    q = randn(41, heads, t, 200, dtype=dtype).transpose(0, 1)[..., 8:]
    kn = randn(42, t, 1, 128, dtype=dtype).expand(t, heads, 128)
    kr = randn(43, t, 128, dtype=dtype)[:, 64:]
    v = randn(44, heads, t, 136, dtype=dtype).transpose(0, 1)[..., :128]
    kr *= torch.linspace(0, 8, t, device="cuda")[:, None].to(dtype)
    for scale in (0.3, -0.3, 0.0):
        out, lse = api.attend_prompt(q, kn, kr, v, i32([0, t]), i32([0, t]), scale)
        check_prompt(q, kn, kr, v, [0, t], [0, t], True, out, lse, scale)


def test_prompt_offsets_out_of_range(api):
    """Offsets below zero, past the tensors or decreasing are clamped: nothing outside is read or written."""
    q, kn, kr, v, _, _ = prompt_inputs(51, [300], [300], 1, torch.bfloat16)
    out = torch.full((300, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(300, 1, device="cuda")
    api.attend_prompt(q, kn, kr, v, i32([-7, 100, 50, 1000]), i32([-9, 120, 40, 5000]), SCALE, out=out, lse=lse)
    check_prompt(q, kn, kr, v, [0, 100], [0, 120], True, out, lse)


def test_other_stream_and_graph(api):
    """The calls run on the stream they are given, and replay from a graph."""
    q, cache = randn(61, 3, 128, WIDTH), randn(62, 3000, WIDTH)
    indices = i32(torch.arange(1500, device="cuda").repeat(3, 1))
    pq, kn, kr, v, cu_q, cu_k = prompt_inputs(63, [200], [200], 2, torch.bfloat16)
    cu_q, cu_k = i32(cu_q), i32(cu_k)
    want = api.attend_selected(q, cache, indices, SCALE)
    want_p = api.attend_prompt(pq, kn, kr, v, cu_q, cu_k, SCALE)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = api.attend_selected(q, cache, indices, SCALE, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out, lse, ws = torch.zeros_like(want[0]), torch.zeros_like(want[1]), want[2]
    out_p, lse_p = torch.zeros_like(want_p[0]), torch.zeros_like(want_p[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.attend_selected(q, cache, indices, SCALE, out=out, lse=lse, workspace=ws)
        api.attend_prompt(pq, kn, kr, v, cu_q, cu_k, SCALE, out=out_p, lse=lse_p)
    for _ in range(3):
        out.zero_()
        out_p.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(out_p, want_p[0])
        assert torch.equal(lse, want[1]) and torch.equal(lse_p, want_p[1])


def test_selection_feeds_attention(api):
    """topk_transform's slots into attend_selected, against attention over the oracle's choice of positions."""
    import oracle
    from sparse_attention_indexer_uint32_gb300 import workloads

    wl = workloads.random_case(seed=91, batch=5, min_len=1, max_len=3000, k=256, page_size=64, dist="normal")
    scores, lens = torch.from_numpy(wl.scores).cuda(), torch.from_numpy(wl.seq_lens).cuda()
    table = torch.from_numpy(wl.page_table).cuda()
    cache = randn(92, (int(table.max()) + 1) * 64, WIDTH)
    q = randn(93, 5, 16, WIDTH)
    slots, _, _ = api.topk_transform(scores, lens, table, 64, wl.k)
    out, lse, _ = api.attend_selected(q, cache, slots, SCALE, seq_lens=lens)
    want, _, _ = oracle.topk_transform(wl.scores, wl.seq_lens, wl.page_table, wl.page_size, wl.k)
    check_selected(q, cache, torch.from_numpy(want).cuda(), None, out, lse)


def test_prompt_without_keys_and_many_requests(api):
    """No key at all; more requests than the 32 that are put in order of their length."""
    q, kn, kr, v, cu_q, cu_k = prompt_inputs(71, [200, 3], [0, 0], 2, torch.bfloat16)
    out, lse = api.attend_prompt(q, kn, kr, v, i32(cu_q), i32(cu_k), SCALE)
    assert (out == 0).all() and (lse == -math.inf).all()
    lens = [(7 * r) % 60 for r in range(70)]
    q, kn, kr, v, cu_q, cu_k = prompt_inputs(72, lens, lens[::-1], 1, torch.float16)
    out, lse = api.attend_prompt(q, kn, kr, v, i32(cu_q), i32(cu_k), SCALE, causal=False)
    check_prompt(q, kn, kr, v, cu_q, cu_k, False, out, lse)


def test_selected_odd_heads_in_parts(api):
    """Rows that several blocks share, with numbers of heads that are no multiple of four."""
    cache = randn(81, 9000, WIDTH, dtype=torch.float16)
    for heads in (1, 7, 33, 63, 65, 127):
        q = randn(82, 2, heads, WIDTH, dtype=torch.float16)
        indices = i32(torch.randperm(9000, device="cuda")[:3001].repeat(2, 1))
        out, lse, _ = api.attend_selected(q, cache, indices, SCALE)
        check_selected(q, cache, indices, None, out, lse)


def test_query_layouts_of_several_queries(api):
    """Queries whose heads are not next to their neighbours' (copied a row at a time) and heads before queries."""
    page, batch = 64, 3
    table = i32(torch.arange(batch * 5, device="cuda").reshape(batch, 5))
    cache, lens = randn(83, batch * 5 * page, WIDTH), i32([300, 2, 190])
    wide = randn(84, batch, 3, 12, WIDTH)
    for q in (wide[:, :, :10], wide.transpose(1, 2)[:, :6]):
        out, lse, _ = api.attend_paged(q, cache, lens, table, page, SCALE)
        check_paged(q, cache, lens, table, page, out, lse)


def test_no_wait_gave_up(api):
    """The flag word of the attention kernels, after everything above."""
    from sparse_attention_indexer_uint32_gb300 import _lib

    assert _lib.topk_read_attend_flags() == 0
    assert _lib.topk_read_attend_flags(clear=True) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("paged", [False, True])
def test_short_rows_after_rows_of_nan(api, dtype, paged):
    """Rows that end anywhere in a tile and follow, in the same block, rows whose cache entries are all NaN."""
    page, lens = 64, [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 79, 80, 81, 112, 113, 127, 128, 129, 145]
    batch = 2 * 8 * len(lens)
    cache = randn(101, 64 * page, WIDTH, dtype=dtype)
    cache[32 * page:] = math.nan
    seen = [lens[r // 2 % len(lens)] if r % 2 else 256 for r in range(batch)]
    q = randn(102, batch, 16, WIDTH, dtype=dtype)
    first = torch.tensor([0 if r % 2 else 32 for r in range(batch)], device="cuda")[:, None]
    table = i32(first + torch.arange(4, device="cuda")[None] * 5 + torch.arange(batch, device="cuda")[:, None] % 7)
    slots = i32((table[..., None] * page + torch.arange(page, device="cuda")).reshape(batch, -1))
    if paged:
        out, lse, _ = api.attend_paged(q[:, None], cache, i32(seen), table, page, SCALE)
        out, lse = out[:, 0], lse[:, 0]
    else:
        out, lse, _ = api.attend_selected(q, cache, slots, SCALE, seq_lens=i32(seen))
    assert torch.isnan(out[::2]).all() and torch.isnan(lse[::2]).all()
    for r in range(1, batch, 2):
        k = cache[slots[r, :seen[r]].long()]
        o, l, ob, lb = attend(q[r], k, k[:, :512], SCALE, dtype)
        check(out[r], o, ob, f"out of row {r}")
        check(lse[r], l, lb, f"lse of row {r}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,heads", [
    ([1], [5000], 1), ([1], [257], 2), ([100], [2049], 16), ([300, 2], [4100, 130], 2), ([1, 17, 256], [2049, 700, 3], 3),
    ([257], [1500], 1), ([700], [600], 1), ([200, 0, 3], [0, 900, 1281], 5), ([129], [3000], 30)])
def test_prompt_few_queries_long_keys(api, dtype, causal, lq, lk, heads):
    """Calls with few pieces of work, whose keys several blocks share: parts with no, one or some of the steps, rows
    that see nothing of a part, requests with too few keys to share beside long ones."""
    q, kn, kr, v, cu_q, cu_k = prompt_inputs(111, lq, lk, heads, dtype, gap=5)
    out = torch.full((q.shape[0], heads, 128), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((q.shape[0], heads), 7.0, device="cuda")
    api.attend_prompt(q, kn, kr, v, i32(cu_q), i32(cu_k), SCALE, causal=causal, out=out, lse=lse)
    check_prompt(q, kn, kr, v, cu_q, cu_k, causal, out, lse)
    for t in (out, lse):
        assert (t[:5] == 7).all() and (t[-5:] == 7).all()
    again = api.attend_prompt(q, kn, kr, v, i32(cu_q), i32(cu_k), SCALE, causal=causal)
    assert torch.equal(out[5:-5], again[0][5:-5]) and torch.equal(lse[5:-5], again[1][5:-5])


def test_prompt_parts_of_infinities(api):
    """Keys that several blocks share: scores of -inf and +inf, and NaN, in one part of the keys only."""
    q, kn, kr, v, cu_q, cu_k = prompt_inputs(121, [3], [3000], 1, torch.float16)
    q[:, 0, 0] = 1
    for bad in (-math.inf, math.inf, math.nan):
        keys = kn.clone()
        keys[1500, 0, 0] = bad
        out, lse = api.attend_prompt(q, keys, kr, v, i32(cu_q), i32(cu_k), SCALE, causal=False)
        if bad == -math.inf:  # as if the key were not there
            rest = [i for i in range(3000) if i != 1500]
            check_prompt(q, kn[rest], kr[rest], v[rest], [0, 3], [0, 2999], False, out, lse)
        else:
            assert torch.isnan(out).all() and not torch.isfinite(lse).any()


def test_prompt_few_queries_in_graph(api):
    """Pieces that several blocks share, replayed from a graph on another stream with other inputs and lengths."""
    q, kn, kr, v, cu_q, cu_k = prompt_inputs(131, [70], [2500], 2, torch.bfloat16)
    marks_q, marks_k = i32(cu_q), i32(cu_k)
    out, lse = api.attend_prompt(q, kn, kr, v, marks_q, marks_k, SCALE)  # looks up the device
    out.zero_(), lse.zero_()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        api.attend_prompt(q, kn, kr, v, marks_q, marks_k, SCALE, out=out, lse=lse, stream=stream)
    for length in (2500, 1111, 300):
        marks_k[1] = length
        q.neg_()
        graph.replay()
        check_prompt(q, kn, kr, v, cu_q, [0, length], True, out, lse)
