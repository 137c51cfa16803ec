"""Latent attention for requests whose first positions are the same, against a
plain 64-bit implementation and against attention over whole rows."""
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


class Batch:
    """Requests of these lengths behind a prompt of `shared` positions; the rows' entries below it are -1."""

    def __init__(self, lens, shared, queries, heads, page, dtype, seed=0, width=None, room=WIDTH):
        b = len(lens)
        self.page, self.shared, self.lens = page, i32([shared]), i32(lens)
        common = max(1, (shared + page - 1) // page)
        width = width or max(1, (max(lens) + page - 1) // page)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        ids = torch.randperm(common + b * width + 2, generator=g, device="cuda").to(torch.int32)
        self.cache = randn(seed + 1, ids.numel() * page, room, dtype=dtype)[:, :WIDTH]
        self.pages, self.table = ids[:common].clone(), ids[common:common + b * width].reshape(b, width).clone()
        self.table[:, : shared // page] = -1
        self.q = randn(seed + 2, b, queries, heads, WIDTH, dtype=dtype)

    def rows(self, r, n, shared):
        """The rows of the cache that the first n positions of request r have, those that are there."""
        assert n <= self.table.shape[1] * self.page
        t = torch.arange(n, device="cuda")
        page = torch.where(t < shared, self.pages.long()[(t // self.page).clamp(max=self.pages.numel() - 1)], self.table[r].long()[t // self.page])
        slot = page * self.page + t % self.page
        return slot, (slot >= 0) & (slot < self.cache.shape[0])

    def run(self, api, **more):
        return api.attend_shared(self.q, self.cache, self.lens, self.table, self.pages, self.shared, self.page, SCALE, **more)

    def check(self, out, lse, max_len=None, scale=SCALE):
        b, queries = self.q.shape[:2]
        most = self.table.shape[1] * self.page if max_len is None else max_len
        shared = min(max(int(self.shared), 0), most, self.pages.numel() * self.page)
        for r in range(b):
            n = min(max(int(self.lens[r]), 0), most)
            for i in range(queries):
                slot, good = self.rows(r, max(0, n - (queries - 1 - i)), shared)
                kv = self.cache[slot[good]]
                o, l, ob, lb = attend(self.q[r, i], kv, kv[:, :LATENT], scale, self.q.dtype)
                check(out[r, i], o, ob, f"out of request {r}, query {i}")
                check(lse[r, i], l, lb, f"lse of request {r}, query {i}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,shared,queries,heads,page", [
    ([1], 0, 1, 1, 64),                                # one position, nothing shared
    ([1], 1, 1, 1, 16),                                # one position, shared
    ([300, 257, 256], 256, 1, 16, 64),                 # one that has nothing of its own
    ([200, 130, 131, 140], 129, 1, 16, 64),            # the prompt ends inside a page
    ([700, 650, 900, 641], 640, 3, 16, 32),
    ([513, 514, 700], 512, 2, 128, 128),
    ([1300, 1290], 1285, 5, 100, 16),
    ([40, 41, 42, 43, 44, 45, 46, 47, 48], 33, 1, 20, 16),
    ([300] * 40, 290, 1, 8, 64),                       # more rows than one tile of queries
    ([2100, 2049], 2048, 1, 64, 256),
    ([130, 90, 20, 0, 129], 128, 2, 16, 16),           # some shorter than the prompt
    ([5, 3], 2000, 1, 16, 64),                         # all shorter than it
    ([900, 3000], 100, 1, 32, 64),                     # own positions outnumber the shared
])
def test_shared(api, dtype, lens, shared, queries, heads, page):
    x = Batch(lens, shared, queries, heads, page, dtype, width=None if max(lens) >= shared else (shared + page - 1) // page)
    out, lse, _ = x.run(api)
    x.check(out, lse)


@pytest.mark.parametrize("page", [1, 2, 8, 16, 32, 64, 128, 512])
@pytest.mark.parametrize("shared", [100, 511])
def test_page_sizes(api, page, shared):
    x = Batch([shared + 1, shared + 77, shared + 300], shared, 2, 24, page, torch.bfloat16, room=WIDTH + 8)
    out, lse, _ = x.run(api)
    x.check(out, lse)


def test_as_whole_rows(api):
    """Rows that hold the common pages too: both calls see the same positions."""
    x = Batch([1500, 1025, 1100, 2000], 1024, 2, 16, 64, torch.bfloat16)
    x.table[:, :16] = x.pages[:16]
    out, lse, _ = x.run(api)
    x.check(out, lse)
    whole, whole_lse, _ = api.attend_paged(x.q, x.cache, x.lens, x.table, 64, SCALE)
    assert (out.float() - whole.float()).abs().max() < 2.0 ** -5 and (lse - whole_lse).abs().max() < 2.0 ** -16


def test_rows_that_see_nothing(api):
    x = Batch([0, 1, 2, 300], 256, 4, 16, 64, torch.float16)
    x.lens[0] = -3
    out, lse, _ = x.run(api)
    x.check(out, lse)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all() and (lse[1, :3] == -math.inf).all()


@pytest.mark.parametrize("shared", [-5, 10 ** 9, 2 ** 31 - 1])
def test_lengths_are_clamped(api, shared):
    """A shared length below 0, or past its pages."""
    x = Batch([192, 250, 2000], 192, 1, 16, 64, torch.bfloat16, width=4)
    x.table = i32(torch.arange(12).reshape(3, 4))
    x.shared.fill_(shared)
    out, lse, _ = x.run(api)
    x.check(out, lse)
    y, y_lse, _ = x.run(api, max_seq_len=100)
    x.check(y, y_lse, max_len=100)


def test_pages_out_of_the_cache(api):
    x = Batch([700, 800, 500], 300, 2, 16, 64, torch.bfloat16)
    x.pages[1], x.pages[3] = -1, x.cache.shape[0] // 64
    x.table[1, 6], x.table[2, 7] = -7, 2 ** 31 - 1
    out, lse, _ = x.run(api)
    x.check(out, lse)
    x.cache = x.cache[: x.cache.shape[0] - 9]  # a page that the cache's end cuts
    out, lse, _ = x.run(api)
    x.check(out, lse)
    x.pages.fill_(-1)
    x.table.fill_(-1)
    out, lse, _ = x.run(api)
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [16, 64, 8])
def test_what_is_not_seen_may_be_anything(api, dtype, page):
    """Slots behind each length, and those of a request's first own page before its own positions, hold NaN."""
    x = Batch([333, 401, 330], 329, 1, 32, page, dtype)
    keep = torch.zeros(x.cache.shape[0], dtype=torch.bool, device="cuda")
    for r, n in enumerate(x.lens.tolist()):
        slot, good = x.rows(r, n, 329)
        keep[slot[good]] = True
    x.cache[~keep] = math.nan
    out, lse, _ = x.run(api)
    x.check(out, lse)


@pytest.mark.parametrize("page,shared", [(64, 192), (64, 200), (16, 208), (8, 100), (256, 300)])
def test_entries_below_the_prompt_may_be_anything(api, page, shared):
    x = Batch([shared + 70, shared + 1, shared, 500], shared, 1, 16, page, torch.bfloat16)
    out, lse, _ = x.run(api)
    x.check(out, lse)
    below = shared // page
    for value in (0, x.cache.shape[0] // page, 2 ** 31 - 1, -2 ** 31):
        x.table[:, :below] = value
        again, again_lse, _ = x.run(api)
        assert torch.equal(again, out) and torch.equal(again_lse, lse)


def test_no_positions_at_all(api):
    x = Batch([5, 70], 64, 2, 16, 64, torch.bfloat16)
    out, lse, _ = x.run(api, max_seq_len=0)
    assert (out == 0).all() and (lse == -math.inf).all()
    x.shared.zero_()
    x.lens.zero_()
    out, lse, _ = x.run(api)
    assert (out == 0).all() and (lse == -math.inf).all()
    x.pages = x.pages[:0]  # no list: nothing is shared, and every position is a row's own
    x.lens.copy_(i32([5, 70]))
    x.table = i32(torch.arange(4).reshape(2, 2))
    x.shared.fill_(64)
    out, lse, _ = x.run(api)
    for r, n in enumerate((5, 70)):
        for i in range(2):
            kv = x.cache[x.table[r, 0] * 64:][: n - 1 + i]
            o, l, ob, lb = attend(x.q[r, i], kv, kv[:, :LATENT], SCALE, x.q.dtype)
            check(out[r, i], o, ob, f"request {r}, query {i}")
            check(lse[r, i], l, lb, f"request {r}, query {i}")


def test_large_scores_on_either_side(api):
    """The maximum in the prompt for some rows, far above or below what is their own."""
    x = Batch([600, 700, 640], 512, 1, 64, 64, torch.bfloat16)
    x.cache[x.pages.long()[:, None].mul(64).add(torch.arange(64, device="cuda")).flatten()] *= 6
    out, lse, _ = x.run(api)
    x.check(out, lse)
    x = Batch([600, 700, 640], 512, 1, 64, 64, torch.float16)
    own = x.table[:, 8:].long()[..., None].mul(64).add(torch.arange(64, device="cuda")).flatten()
    x.cache[own] *= 6
    out, lse, _ = x.run(api)
    x.check(out, lse)


@pytest.mark.parametrize("scale", [-0.07, 0.0, 1.5])
def test_scales(api, scale):
    x = Batch([300, 290, 400], 256, 1, 16, 64, torch.bfloat16)
    out, lse, _ = api.attend_shared(x.q, x.cache, x.lens, x.table, x.pages, x.shared, 64, scale)
    x.check(out, lse, scale=scale)


def test_query_layouts(api):
    x = Batch([300, 290, 400], 256, 2, 6, 64, torch.bfloat16)
    whole = x.q
    for q in (randn(9, 3, 2, 6, 2 * WIDTH)[..., 64:64 + WIDTH], randn(9, 2, 3, 6, WIDTH).transpose(0, 1),
              randn(9, 3, 6, 2, WIDTH).transpose(1, 2), randn(9, 6, 2, 3, WIDTH).permute(2, 1, 0, 3)):
        x.q = q
        assert q.shape == whole.shape
        out, lse, _ = x.run(api)
        x.check(out, lse)


def test_many_requests(api):
    """More requests than a block has threads."""
    g = torch.Generator().manual_seed(3)
    lens = (torch.randint(0, 90, (700,), generator=g) + 40).tolist()
    x = Batch(lens, 64, 1, 4, 16, torch.bfloat16)
    out, lse, _ = x.run(api)
    x.check(out, lse)


def test_workspace_and_outputs_are_reused(api):
    x = Batch([300, 290, 400], 256, 1, 16, 64, torch.bfloat16)
    out, lse, workspace = x.run(api)
    workspace.view(torch.float32).fill_(math.nan)
    out2, lse2, again = x.run(api, out=torch.full_like(out, math.nan), lse=torch.full_like(lse, math.nan), workspace=workspace)
    assert again is workspace and torch.equal(out, out2) and torch.equal(lse, lse2)
    y = Batch([900, 290], 128, 2, 128, 64, torch.bfloat16)
    out, lse, more = y.run(api, workspace=workspace)  # one that is too small is left alone
    y.check(out, lse)
    assert more is workspace or more.numel() > workspace.numel()


def test_replayed_with_other_lengths(api):
    x = Batch([1, 1, 1, 1], 0, 2, 16, 64, torch.bfloat16, width=30)
    x.pages, x.table = i32(torch.arange(20)), i32(torch.arange(x.table.numel()).reshape(4, 30))
    x.cache = randn(4, 140 * 64, WIDTH)
    out, lse, workspace = x.run(api)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        x.run(api, out=out, lse=lse, workspace=workspace)
    for shared, lens in ((0, [5, 0, 1900, 64]), (1000, [1003, 1900, 1001, 1700]), (1280, [1280, 3, 1281, 1920])):
        x.shared.fill_(shared)
        x.lens.copy_(i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        x.check(out, lse)


def test_two_graphs_share_a_workspace(api):
    """Replayed in turn on one stream, with other shapes each."""
    sets = [Batch([900, 700, 650], 640, 1, 64, 64, torch.bfloat16), Batch([300] * 9, 200, 2, 16, 32, torch.float16, seed=9)]
    first = [x.run(api) for x in sets]
    workspace = max((w for _, _, w in first), key=lambda w: w.numel())
    outs = [(torch.empty_like(o), torch.empty_like(l)) for o, l, _ in first]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    for x, (out, lse) in zip(sets, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            x.run(api, out=out, lse=lse, workspace=workspace)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (o, l, _), (out, lse) in zip(first, outs):
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_on_two_streams(api):
    sets = [Batch([900, 1290, 700], 640, 1, 16, 64, torch.bfloat16, seed=s) for s in (0, 50)]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    results = []
    for _ in range(4):
        results = [x.run(api, stream=s) for x, s in zip(sets, streams)]
    torch.cuda.synchronize()
    for x, (out, lse, _) in zip(sets, results):
        x.check(out, lse)


def test_equal_calls_give_equal_bits(api):
    x = Batch([5000, 4100, 4999, 6000], 4096, 1, 64, 64, torch.bfloat16)
    first, first_lse, workspace = x.run(api)
    for _ in range(3):
        out, lse, _ = x.run(api, workspace=workspace)
        assert torch.equal(out, first) and torch.equal(lse, first_lse)


def test_large_offsets(api):
    """Rows of the cache past 2^31 values."""
    page, n = 64, (2 ** 31 // WIDTH + 4096) // 64 * 64
    x = Batch([200, 140], 100, 1, 16, page, torch.bfloat16)
    small, ids = x.cache, torch.cat((x.pages, x.table.flatten()))
    ids = ids[ids >= 0].unique().long()
    far = n // page - 1 - torch.arange(int(ids.max()) + 1, device="cuda")
    want, want_lse, _ = x.run(api)
    x.check(want, want_lse)
    cache = torch.empty(n, WIDTH, dtype=torch.bfloat16, device="cuda")
    for p in ids.tolist():
        cache[int(far[p]) * page:(int(far[p]) + 1) * page] = small[p * page:(p + 1) * page]
    move = lambda t: torch.where(t < 0, t, far[t.long().clamp(min=0)].to(torch.int32))  # noqa: E731
    x.cache, x.pages, x.table = cache, move(x.pages), move(x.table)
    out, lse, _ = x.run(api)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
