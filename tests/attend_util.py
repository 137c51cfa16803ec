"""Plain 64-bit attention for the tests, with bounds on what two-byte weights
and outputs and 32-bit sums may be off.

For one query: s_j = scale q.k_j, p = softmax(s), o = sum p_j v_j.  With u the
unit roundoff of the two-byte type:

* a score summed in 32 bits is off by at most ds = (d + 4) 2^-24 scale
  sum|q k_j| (any order of d additions, and the scale), and by 2^-22 relative
  to the exponent's argument in its own rounding; both change the weights by a
  factor of at most 1 + 2 (ds + dx) (numerator and sum);
* each weight is rounded once to the type (u relative, and in fp16 2^-25
  absolute where it is below the normal range, against a sum of at least
  2^-9: the running maximum may lag by up to 8 in the exponent's base-2 unit,
  in either direction of a row's joined parts, before it is raised);
* the output is rounded once (u relative, 2^-25 absolute in fp16).

So |o' - o| <= (u + 2 (ds + dx) + 2^-16) sum p|v| + u |o| + 2^-25 (sum|v| + 1),
the 2^-16 covering the 32-bit sums over the weights, and
|lse' - lse| <= ds + dx + 2^-20 + 2^-22 |lse|.
"""
from __future__ import annotations

import math

import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def attend(q, k, v, scale, dtype):
    """q [m, d], k [n, d], v [n, e] -> (out, lse, out_bound, lse_bound) in 64 bits; n may be 0."""
    m, e = q.shape[0], v.shape[1]
    if k.shape[0] == 0:
        zero = torch.zeros(m, e, dtype=torch.float64, device=q.device)
        none = torch.full((m,), -math.inf, dtype=torch.float64, device=q.device)
        return zero, none, zero, torch.zeros_like(none)
    q, k, v = q.double(), k.double(), v.double()
    s = q @ k.t() * scale
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    out = p @ v
    ds = (q.abs() @ k.abs().t() * abs(scale)).amax(1) * (q.shape[1] + 4) * 2.0 ** -24
    dx = (s.abs().amax(1) + lse.abs()) * 2.0 ** -22
    u = UNIT[dtype]
    small = 2.0 ** -25 if dtype == torch.float16 else 0.0
    bound = (u + 2 * (ds + dx) + 2.0 ** -16)[:, None] * (p @ v.abs()) + u * out.abs() + small * (v.abs().sum(0) + 1)
    return out, lse, bound * 1.01, ds + dx + 2.0 ** -20 + 2.0 ** -22 * lse.abs()


def check(got, want, bound, what):
    got, want = got.double(), want.double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: other values are finite"
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine], want[~fine]), f"{what}: infinities differ"
    off = ((got - want).abs() - bound)[fine]
    if off.numel():
        worst = off.max().item()
        assert worst <= 0, f"{what}: {worst:.3g} past its bound, {(off > 0).sum().item()} of {off.numel()} values"
