"""Rows in fp16 with one dominant slot whose values are zero and thousands of
slots far below it: the output is the tail's alone.

Bound, derived as in attend_util but for small weights: the largest weight of a
row is stored at 2^7 to 2^15, so the sum of the weights is at least 2^7 in
that unit; a stored weight is off by 2^-11 of itself where it is normal (from
2^-14 on) and by 2^-25 below, which is 2^-32 of the sum.  The output itself is
rounded once (2^-11 of itself, 2^-25 absolute):

|o' - o| <= (2^-11 + 2 (ds + dx) + 2^-16) sum p|v| + 2^-11 |o| + 2^-32 sum|v| + 2^-25.
"""
from __future__ import annotations

import pytest
import torch

from tests.attend_util import check

pytestmark = pytest.mark.gpu
F16, U = torch.float16, 2.0 ** -11


@pytest.fixture(scope="module")
def api():
    from sparse_attention_indexer_uint32_gb300 import api

    return api


def expected(score, v, terms):
    """Plain 64-bit output and log-sum-exp of one row, with their bounds; terms: values summed in a score."""
    lse = torch.logsumexp(score, 0)
    p = torch.exp(score - lse)
    out = p @ v
    ds, dx = score.abs().max() * (terms + 4) * 2.0 ** -24, (score.abs().max() + lse.abs()) * 2.0 ** -22
    bound = (U + 2 * (ds + dx) + 2.0 ** -16) * (p @ v.abs()) + U * out.abs() + 2.0 ** -32 * v.abs().sum(0) + 2.0 ** -25
    return out, lse, bound, ds + dx + 2.0 ** -20 + 2.0 ** -22 * lse.abs()


def rows_of(count, width, at):
    """Scores (one rotary value, scale 1) e^-15 to e^-21 below that of slot `at`, values around 1; its own are zero."""
    g = torch.Generator(device="cuda")
    g.manual_seed(count + at)
    score = -15 - 6 * torch.rand(count, generator=g, device="cuda")
    value = 1 + 0.25 * torch.randn(count, width, generator=g, device="cuda")
    score[at], value[at] = 0, 0
    return score.to(F16), value.to(F16)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("batch,length", [(100, 2000), (1, 60000), (3, 130)])
@pytest.mark.parametrize("place", [0.0, 0.5, 1.0])
def test_cache(api, paged, batch, length, place):
    page, heads, at = 16, 16, int(place * (length - 1))
    score, value = rows_of(length, 512, at)
    cache = torch.zeros(-(-length // page) * page, 576, dtype=F16, device="cuda")
    cache[:length, :512], cache[:length, 512] = value, score
    q = torch.zeros(batch, heads, 576, dtype=F16, device="cuda")
    q[..., 512] = 1
    lens = torch.full((batch,), length, dtype=torch.int32, device="cuda")
    if paged:
        table = torch.arange(cache.shape[0] // page, dtype=torch.int32, device="cuda").repeat(batch, 1)
        out, lse, _ = api.attend_paged(q[:, None], cache, lens, table, page, 1.0)
        out, lse = out[:, 0], lse[:, 0]
    else:
        slots = torch.arange(length, dtype=torch.int32, device="cuda").repeat(batch, 1)
        out, lse, _ = api.attend_selected(q, cache, slots, 1.0, seq_lens=lens)
    o, l, ob, lb = expected(score.double(), value.double(), 576)
    check(out, o.expand(out.shape), ob.expand(out.shape), "out")
    check(lse, l.expand(lse.shape), lb.expand(lse.shape), "lse")


@pytest.mark.parametrize("queries,heads,length", [(300, 2, 3000), (1, 1, 9000), (3, 1, 130)])
@pytest.mark.parametrize("place", [0.0, 0.5, 1.0])
def test_prompt(api, queries, heads, length, place):
    at = int(place * (length - 1))
    score, value = rows_of(length, 128, at)
    q = torch.zeros(queries, heads, 192, dtype=F16, device="cuda")
    q[..., 128] = 1
    k_nope, k_rope = torch.zeros(length, heads, 128, dtype=F16, device="cuda"), torch.zeros(length, 64, dtype=F16, device="cuda")
    k_rope[:, 0] = score
    v = value[:, None].expand(length, heads, 128).contiguous()
    marks = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (queries, length)]
    out, lse = api.attend_prompt(q, k_nope, k_rope, v, *marks, 1.0, causal=False)
    o, l, ob, lb = expected(score.double(), value.double(), 192)
    check(out, o.expand(out.shape), ob.expand(out.shape), "out")
    check(lse, l.expand(lse.shape), lb.expand(lse.shape), "lse")


def test_steps_up_to_the_head(api):
    """Scores that rise by 8 and a little more in base 2 from tile to tile: weights near the type's largest."""
    length = 128 * 12
    step = torch.arange(length, device="cuda") // 128
    for rise in (5.5, 5.6, 10.4):  # 7.9, 8.1 and 15.004 in base 2
        cache = torch.zeros(length, 576, dtype=F16, device="cuda")
        cache[:, :512] = 1 + 0.25 * torch.randn(length, 512, device="cuda")
        cache[:, 512] = step * rise
        q = torch.zeros(1, 16, 576, dtype=F16, device="cuda")
        q[..., 512] = 1
        slots = torch.arange(length, dtype=torch.int32, device="cuda")[None]
        out, lse, _ = api.attend_selected(q, cache, slots, 1.0)
        o, l, ob, lb = expected(cache[:, 512].double(), cache[:, :512].double(), 576)
        check(out[0], o.expand(out[0].shape), ob.expand(out[0].shape), f"out, {rise}")
        check(lse[0], l.expand(lse[0].shape), lb.expand(lse[0].shape), f"lse, {rise}")
