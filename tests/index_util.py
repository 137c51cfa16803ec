"""Plain 64-bit forms of the indexer's operators for the tests, with bounds on
what 32-bit sums and two-byte outputs may be off.

Append: the mean of 128 values is off by at most 7 roundings of the mean of
their sizes (a tree of depth 7), which moves each normed value by that times
r |w|; centring, the squares' tree, the root (2 ulp), the two products and the
bias add at most 20 roundings of |z w| + |b|, the rotation 3 of each pair's
size.  All are within 32 * 2^-24 = 2^-19 of (mean|x| r |w| + size of the pair),
and the output is rounded once (u, and 2^-25 absolute in fp16).

Scores: a dot product of d = 128 exact products summed in 32 bits in any order,
rounded or cut off, is off by at most (d + 4) 2^-23 sum|q k|; max(., 0) widens
nothing; the weighted sum of H of them adds (H + 4) 2^-24 sum|w max|.
"""
from __future__ import annotations

import math

import torch

from tests.attend_util import UNIT

INDEX, ROPE = 128, 64


def append(rows, weight, bias, eps, cos_sin, positions, interleaved, rope_last):
    """The rows as they are stored, in 64 bits, and how far they may be off."""
    x = rows.double()
    size = x.abs()
    spread = torch.zeros_like(x)
    if weight is not None:
        mean = x.mean(1, keepdim=True)
        r = 1 / ((x - mean).square().mean(1, keepdim=True) + eps).sqrt()
        spread = size.mean(1, keepdim=True) * r * weight.double().abs()
        x = (x - mean) * r * weight.double()
        size = x.abs()
        if bias is not None:
            x = x + bias.double()
            size = size + bias.double().abs()
    size = size + spread
    if cos_sin is not None:
        at = slice(INDEX - ROPE, INDEX) if rope_last else slice(0, ROPE)
        turn = cos_sin[positions.long()].double()
        c, s = turn[:, :32], turn[:, 32:]

        def rotate(y, c, s, back):
            a, b = (y[:, 0::2], y[:, 1::2]) if interleaved else (y[:, :32], y[:, 32:])
            a, b = a * c + b * back, a * s + b * c
            return torch.stack((a, b), 2).flatten(1) if interleaved else torch.cat((a, b), 1)

        # Of the sizes nothing cancels.
        both = rotate(x[:, at], c, s, -s), rotate(size[:, at], c.abs(), s.abs(), s.abs())
        x, size = x.clone(), size.clone()
        x[:, at], size[:, at] = both
    u = UNIT[rows.dtype]
    small = 2.0 ** -25 if rows.dtype == torch.float16 else 0.0
    return x, (u * x.abs() + 2.0 ** -19 * size + small) * 1.01


def scores(q, weights, keys):
    """q [m, h, d], weights [m, h], keys [n, d] -> ([m, n] scores, bounds) in 64 bits."""
    q, w, k = q.double(), weights.double(), keys.double()
    dot = torch.einsum("mhd,nd->mhn", q, k)
    top = torch.where(dot > 0, dot, torch.where(dot.isnan(), dot, 0.0))
    off = torch.einsum("mh,mhn->mn", w.abs(), torch.einsum("mhd,nd->mhn", q.abs(), k.abs()))
    total = torch.einsum("mh,mhn->mn", w, top)
    wide = torch.einsum("mh,mhn->mn", w.abs(), top)
    return total, ((q.shape[2] + 4) * 2.0 ** -23 * off + (q.shape[1] + 4) * 2.0 ** -24 * wide) * 1.01


def gather(cache, table, page, n):
    """Rows of the first n positions through a page-table row, and which of them have a slot in the cache."""
    assert n <= table.shape[0] * page
    t = torch.arange(n, device=cache.device)
    slot = table.long()[t // page] * page + t % page
    good = (slot >= 0) & (slot < cache.shape[0])
    return cache[torch.where(good, slot, 0)], good


def check_scores(q, weights, cache, lens, table, page, out, before, cu=None, max_len=None):
    """Every row of `out`: what its query sees against the plain form, the rest as it was `before`."""
    total, b = q.shape[0], lens.shape[0]
    cu = [i * (total // b) for i in range(b + 1)] if cu is None else [min(max(int(c), 0), total) for c in cu]
    expected = before.clone().double()
    bound = torch.zeros_like(expected)
    for r in range(b):
        n = min(int(lens[r]), table.shape[1] * page if max_len is None else max_len)
        if cu[r + 1] <= cu[r] or n <= 0:
            continue
        keys, good = gather(cache, table[r], page, n)
        want, off = scores(q[cu[r]:cu[r + 1]], weights[cu[r]:cu[r + 1]], keys)
        want[:, ~good], off[:, ~good] = -math.inf, 0.0
        for i in range(cu[r + 1] - cu[r]):
            seen = max(0, n - (cu[r + 1] - cu[r] - 1 - i))
            expected[cu[r] + i, :seen], bound[cu[r] + i, :seen] = want[i, :seen], off[i, :seen]
    got = out.double()
    assert torch.equal(got.isnan(), expected.isnan()), "other values are NaN"
    fine = torch.isfinite(expected)
    rest = ~fine & ~expected.isnan()
    assert torch.equal(got[rest], expected[rest]), "infinities differ"
    off = ((got - expected).abs() - bound)[fine]
    if off.numel():
        assert off.max().item() <= 0, f"{off.max().item():.3g} past its bound, {(off > 0).sum().item()} of {off.numel()}"
