"""Block tables and the cache append, against plain loops and 64-bit arithmetic."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from sparse_attention_indexer_uint32_gb300 import api

    return api


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def plain_tables(context, new, free, table, page, max_tokens):
    """Python whole numbers, request by request."""
    pages = lambda n: -(-n // page)  # noqa: E731
    width = len(table[0])
    room, limit = width * page, 2 ** 31 - 1
    flags, taken, cu, seq = 0, 0, [0], []
    slots, positions, rows = [], [], []
    for b, (c, n) in enumerate(zip(context, new)):
        if c < 0 or n < 0:
            flags |= 1
        c, n = max(c, 0), max(n, 0)
        if c + n > room:
            flags |= 2
        seq.append(min(c + n, room, limit))
        for col in range(pages(min(c, room)), pages(min(c + n, room))):
            table[b][col] = free[taken] if taken < len(free) else -1
            taken += 1
        for p in range(c, c + min(n, max(0, max_tokens - len(slots)))):
            col = p // page
            slot = table[b][col] * page + p % page if p < room and table[b][col] >= 0 else -1
            slots.append(slot if slot <= limit else -1)
            positions.append(min(p, limit))
            rows.append(b)
        cu.append(min(cu[-1] + n, limit))
    if taken > len(free):
        flags |= 4
    if sum(max(n, 0) for n in new) > max_tokens:
        flags |= 8
    pad = [-1] * (max_tokens - len(slots))
    return seq, cu, slots + pad, positions + pad, rows + pad, [min(taken, len(free)), flags]


def run_tables(api, context, new, free, table, page, max_tokens, **kw):
    dev_table = i32(table)
    got = api.block_tables(i32(context), i32(new), i32(free), dev_table, page, max_tokens, **kw)
    table = [list(r) for r in table]
    want = plain_tables(context, new, free, table, page, max_tokens)
    for name, x in zip(got._fields, want):
        assert getattr(got, name).tolist() == x, name
    assert dev_table.tolist() == table
    return got


@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("batch,most", [(1, 1), (1, 700), (7, 1), (33, 150), (1000, 3), (4096, 1), (4097, 2), (9000, 3)])
def test_tables(api, page, batch, most):
    g = torch.Generator()
    g.manual_seed(batch + page)
    context = torch.randint(0, 300, (batch,), generator=g).tolist()
    new = torch.randint(0, most + 1, (batch,), generator=g).tolist()
    width = -(-(300 + most) // page)
    held = batch * width
    ids = torch.randperm(2 * held + 5, generator=g).tolist()
    table = [ids[b * width:(b + 1) * width] for b in range(batch)]
    got = run_tables(api, context, new, ids[held:], table, page, sum(new) + 11)
    # Buffers of an earlier call are taken again.
    run_tables(api, context, new, ids[held:], table, page, sum(new) + 11, out=got)


def test_tables_edges(api):
    page = 4
    table = [[10 * b + c for c in range(5)] for b in range(6)]
    free = [100, 101, 102, 103]
    # Negative lengths, a row longer than its table, a held page that is -1, contexts at and inside a page's end.
    table[5][1] = -1
    run_tables(api, [-3, 4, 18, 25, 3, 6], [2, -1, 9, 2, 1, 3], free, table, page, 40)
    # The list of free pages ends; the room for tokens ends; there is none of either; no token at all.
    run_tables(api, [0, 0, 0, 0, 0, 0], [9, 9, 9, 9, 9, 9], free, table, page, 60)
    run_tables(api, [0, 0, 0, 0, 0, 0], [3, 3, 3, 3, 3, 3], free, table, page, 7)
    run_tables(api, [1, 2, 3, 4, 5, 6], [1, 1, 1, 1, 1, 1], [], table, page, 0)
    run_tables(api, [1, 2, 3, 4, 5, 6], [0, 0, 0, 0, 0, 0], free, table, page, 5)


def test_tables_large_numbers(api):
    """Sums and positions past 31 bits, pages whose slots would be."""
    top = 2 ** 31 - 1
    run_tables(api, [top, top - 1, 5], [top, 3, top], [7, 2 ** 30, 9], [[1, 2 ** 21, 3, 4]] * 3, 2 ** 10, 6)
    run_tables(api, [2 ** 30, 2 ** 31 - 2], [1, 2], [3, 1], [[0, 1, 2, 3], [0, 1, -1, 3]], 2 ** 30, 4)


def test_tables_strided(api):
    """Rows of a wider table: what lies between them stays."""
    wide = torch.full((3, 12), 55, dtype=torch.int32, device="cuda")
    got = api.block_tables(i32([0, 3, 8]), i32([5, 5, 0]), i32([1, 2, 3, 4, 5]), wide[:, 2:6], 4, 10)
    assert got.status.tolist() == [3, 0]
    want = torch.full((3, 12), 55, dtype=torch.int32)
    want[0, 2], want[0, 3], want[1, 3] = 1, 2, 3
    assert torch.equal(wide.cpu(), want)


@pytest.mark.parametrize("dtype,unit,small", [(torch.bfloat16, 2.0 ** -8, 0.0), (torch.float16, 2.0 ** -11, 2.0 ** -25)])
@pytest.mark.parametrize("tokens", [1, 9, 1000])
@pytest.mark.parametrize("norm,turn", [(True, "half"), (True, "interleaved"), (False, "half"), (True, None), (False, None)])
def test_append(api, dtype, unit, small, tokens, norm, turn):
    """Against 64 bits: one rounding of the output (unit), and 32-bit arithmetic before it (2^-20 of the terms)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    n, positions_n = 2 * tokens + 3, 50
    wide = torch.randn(tokens, 640, generator=g, device="cuda").to(dtype)
    rows = wide[:, 64:]
    weight = torch.randn(512, generator=g, device="cuda").to(dtype) if norm else None
    angle = torch.rand(positions_n, 32, generator=g, device="cuda") * 6.28
    cos_sin = torch.cat((angle.cos(), angle.sin()), 1).contiguous() if turn else None
    slots = torch.randperm(n, generator=g, device="cuda")[:tokens].to(torch.int32)
    positions = torch.randint(0, positions_n, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    skip = torch.zeros(tokens, dtype=torch.bool, device="cuda")
    if tokens > 8:
        slots[1], slots[2], slots[3] = -1, n, 2 ** 31 - 1
        skip[1:4] = True
        if turn:
            positions[4], positions[5] = -1, positions_n
            skip[4:6] = True
        rows[6] = 0  # a row of zeros stays zeros
    if tokens > 8:
        rows[7] *= 100
    cache_wide = torch.randn(n, 600, generator=g, device="cuda").to(dtype)
    cache = cache_wide[:, 8:584]
    before = cache_wide.clone()
    api.cache_append(rows, slots, cache, norm_weight=weight, eps=1e-5, cos_sin=cos_sin,
                     positions=positions if turn else None, interleaved=turn == "interleaved")
    x = rows[~skip].double()
    c, r = x[:, :512], x[:, 512:]
    if norm:
        c = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * weight.double()
    terms = torch.cat((c, r), 1).abs()
    if turn:
        f = cos_sin.double()[positions[~skip].long()]
        cos, sin = f[:, :32], f[:, 32:]
        a, b = (r[:, 0::2], r[:, 1::2]) if turn == "interleaved" else (r[:, :32], r[:, 32:])
        y0, y1 = a * cos - b * sin, a * sin + b * cos
        size = a.abs() + b.abs()
        join = (lambda u, v: torch.stack((u, v), 2).flatten(1)) if turn == "interleaved" else (lambda u, v: torch.cat((u, v), 1))
        r = join(y0, y1)
        terms[:, 512:] = join(size, size)
    want = torch.cat((c, r), 1)
    at = slots[~skip].long()
    off = (cache[at].double() - want).abs() - (unit * want.abs() + 2.0 ** -20 * terms + small)
    assert off.max().item() <= 0
    # Nothing else changed: other slots, and the columns around the cache's rows.
    after = cache_wide.clone()
    after[at, 8:584] = before[at, 8:584]
    assert torch.equal(after, before)


def test_append_large_values(api):
    """A square sum past the type's own range, and NaN that stays in its row."""
    rows = torch.full((3, 576), 60000.0, device="cuda").to(torch.float16)
    rows[1] = math.nan
    rows[2] = 1e-7
    cache = torch.zeros(3, 576, dtype=torch.float16, device="cuda")
    api.cache_append(rows, i32([0, 1, 2]), cache, norm_weight=torch.ones(512, device="cuda", dtype=torch.float16), eps=0.0)
    assert (cache[0, :512] == 1).all() and torch.isnan(cache[1]).all()
    assert (cache[2, :512] == 1).all()


def test_append_no_tokens(api):
    cache = torch.zeros(4, 576, dtype=torch.bfloat16, device="cuda")
    api.cache_append(torch.zeros(0, 576, dtype=torch.bfloat16, device="cuda"), i32([]), cache)
    assert (cache == 0).all()


def test_step_feeds_step(api):
    """Tables, append and attention in a row: what was appended through the slot map is what the table finds."""
    page, heads = 16, 16
    context, new = [0, 20, 5], [18, 3, 1]
    table = i32([[9, 9, 9], [2, 3, 9], [6, 9, 9]])
    step = api.block_tables(i32(context), i32(new), i32([5, 0, 1, 4]), table, page, 30)
    cache = torch.randn(8 * page, 576, device="cuda").to(torch.bfloat16)
    rows = torch.randn(30, 576, device="cuda").to(torch.bfloat16)
    api.cache_append(rows, step.slots, cache)
    at = 0
    for b, n in enumerate(new):
        for j in range(n):
            p = context[b] + j
            assert torch.equal(cache[int(table[b, p // page]) * page + p % page], rows[at])
            at += 1
    q = torch.randn(3, 1, heads, 576, device="cuda").to(torch.bfloat16)
    out, lse, _ = api.attend_paged(q, cache, step.seq_lens, table, page, 0.07)
    from tests.test_gpu_attend import LATENT
    from tests.attend_util import attend, check

    for b in range(3):
        t = torch.arange(context[b] + new[b], device="cuda")
        kv = cache[table[b].long()[t // page] * page + t % page]
        o, l, ob, lb = attend(q[b, 0], kv, kv[:, :LATENT], 0.07, q.dtype)
        check(out[b, 0], o, ob, "out")
        check(lse[b, 0], l, lb, "lse")
