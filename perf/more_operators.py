"""Measured cases of the indexer's side of a serving step, and of batches that
share a prompt: the append of the indexer's keys to their paged cache, the
indexer's scores over that cache (which the selection takes), and latent
attention for requests whose first tokens are the same.

``run`` computes a pass with elementary torch operations in 32 bits, or, where
``own`` is true, with the framework's entry points.  An index key holds 128
values, 64 of them rotary; a latent row holds 512 values and 64 rotary ones.
"""
import math

import torch

own = False

INDEX, ROPE, LATENT, NOPE = 128, 64, 512, 128
WIDTH = LATENT + ROPE
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # The keys of a decode step of 64 requests.
        {"name": "index_append_decode64", "op": "append", "tokens": 64, "slots": 65536, "dtype": "bf16", "interleaved": True, "rope_last": False},
        # The keys of a prefill step of 65536 tokens, some of them without a slot.
        {"name": "index_append_prompt65536", "op": "append", "tokens": 65536, "slots": 131072, "dtype": "fp16", "interleaved": False, "rope_last": True},
        # A small decode step: 4 requests of 8192 tokens.
        {"name": "scores_small4", "op": "scores", "batch": 4, "queries": 1, "heads": 64, "min_len": 8192, "max_len": 8192, "page_size": 64, "dtype": "bf16"},
        # One request of the longest context.
        {"name": "scores_one1m", "op": "scores", "batch": 1, "queries": 1, "heads": 64, "min_len": 1048576, "max_len": 1048576, "page_size": 64, "dtype": "bf16"},
        # A decode batch of 128 ragged requests.
        {"name": "scores_ragged128", "op": "scores", "batch": 128, "queries": 1, "heads": 64, "min_len": 1024, "max_len": 32768, "page_size": 128, "dtype": "bf16"},
        # 32 requests that verify 4 proposed tokens each, 32 heads, lengths from empty on.
        {"name": "scores_verify32", "op": "scores", "batch": 32, "queries": 4, "heads": 32, "min_len": 0, "max_len": 16384, "page_size": 64, "dtype": "fp16"},
        # The second half of a prompt of 8192 tokens.
        {"name": "scores_prompt4096", "op": "prompt", "batch": 1, "heads": 64, "max_new": 4096, "max_past": 4096, "page_size": 64, "dtype": "bf16"},
        # Pieces of 8 prompts after what is cached of them already, 16 heads.
        {"name": "scores_pieces8", "op": "prompt", "batch": 8, "heads": 16, "max_new": 509, "max_past": 4096, "page_size": 32, "dtype": "fp16"},
        # 4 requests behind a short common prompt: a launch's latency.
        {"name": "shared_few4", "op": "shared", "batch": 4, "queries": 1, "heads": 16, "shared": 2048, "min_own": 1, "max_own": 130, "page_size": 64, "dtype": "bf16"},
        # 64 requests with the 16 heads of one of 8 shards behind one long document.
        {"name": "shared_document64", "op": "shared", "batch": 64, "queries": 1, "heads": 16, "shared": 32768, "min_own": 1, "max_own": 2048, "page_size": 64, "dtype": "bf16"},
        # 16 requests with all 128 heads, and as much of their own on average as they share.
        {"name": "shared_heads128", "op": "shared", "batch": 16, "queries": 1, "heads": 128, "shared": 8192, "min_own": 4096, "max_own": 12288, "page_size": 64, "dtype": "bf16"},
        # 32 requests that verify 4 proposed tokens each; the common prompt ends inside a page.
        {"name": "shared_verify32", "op": "shared", "batch": 32, "queries": 4, "heads": 16, "shared": 16000, "min_own": 4, "max_own": 777, "page_size": 128, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("append", "scores", "prompt", "shared", "scores", "prompt", "shared"))
    dtype, page = rng.choice(("bf16", "fp16")), rng.choice((16, 32, 64, 128))
    if op == "append":
        tokens = _log(rng, 1, 65536)
        return {"op": op, "tokens": tokens, "slots": 2 * tokens, "dtype": dtype, "interleaved": rng.random() < 0.5, "rope_last": rng.random() < 0.5}
    if op == "scores":
        heads, queries = rng.choice((4, 8, 16, 24, 32, 64, 100, 128)), rng.choice((1, 1, 2, 3, 5))
        most = _log(rng, 1, 1048576)
        batch = _log(rng, 1, max(1, min(256, 2 ** 21 // most, 2 ** 28 // (most * heads * queries))))
        return {"op": op, "batch": batch, "queries": queries, "heads": heads, "min_len": rng.choice((0, 1, most)), "max_len": most, "page_size": page, "dtype": dtype}
    if op == "prompt":
        heads, batch = rng.choice((4, 16, 24, 32, 64)), rng.choice((1, 2, 3, 5, 8))
        new = _log(rng, 1, max(64, 4096 // batch))
        return {"op": op, "batch": batch, "heads": heads, "max_new": new, "max_past": rng.choice((0, _log(rng, 1, 4096 // batch))), "page_size": page, "dtype": dtype}
    heads, queries = rng.choice((8, 16, 20, 64, 128)), rng.choice((1, 1, 2, 3, 5))
    batch = _log(rng, 1, min(64, 4096 // (heads * queries)))
    shared = _log(rng, 1, 32768)
    most = _log(rng, queries, min(16384, 2 ** 18 // batch))
    return {"op": op, "batch": batch, "queries": queries, "heads": heads, "shared": shared, "min_own": rng.choice((queries, most)), "max_own": most, "page_size": page, "dtype": dtype}


def _spread(count, lo, hi):
    """Lengths spread evenly from lo to hi, one alone hi."""
    return [lo + (hi - lo) * i // (count - 1) for i in range(count)] if count > 1 else [hi]


def _lengths(g, count, lo, hi):
    """Those lengths, in an order of the seed's."""
    return torch.tensor(_spread(count, lo, hi), dtype=torch.int32)[torch.randperm(count, generator=g)]


def _pages(n, page):
    return (n + page - 1) // page


def prepare(case, seed):
    g, h = torch.Generator(), torch.Generator(device="cuda")
    g.manual_seed(seed)
    h.manual_seed(seed + 1)
    dev, dtype, op = torch.device("cuda"), DTYPES[case["dtype"]], case["op"]
    randn = lambda *shape, dtype=dtype: torch.randn(shape, generator=h, device=dev, dtype=dtype)  # noqa: E731
    perm = lambda n: torch.randperm(n, generator=h, device=dev).to(torch.int32)  # noqa: E731
    s = {"case": dict(case)}
    if op == "append":
        t, n = case["tokens"], case["slots"]
        # The keys are a slice of a wider projection's output.
        wide = randn(t, INDEX + 64)
        slots = perm(n)[:t].clone()
        if t > 16:
            slots[torch.rand(t, generator=h, device=dev) < 0.02] = -1
        positions = torch.randint(0, 16384, (t,), generator=h, device=dev, dtype=torch.int32)
        angle = torch.arange(16384, device=dev, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(ROPE // 2, device=dev, dtype=torch.float64) / (ROPE // 2))
        s.update(rows=wide[:, :INDEX], slots=slots, positions=positions, weight=(1 + 0.1 * randn(INDEX, dtype=torch.float32)).to(dtype),
                 bias=(0.1 * randn(INDEX, dtype=torch.float32)).to(dtype), cos_sin=torch.cat((angle.cos(), angle.sin()), 1).float(), eps=1e-6,
                 # One row past the cache takes what has no slot in the plain form.
                 store=randn(n + 1, INDEX), n=n)
        s["cache"] = s["store"][:n]
        return s
    heads, b, page = case["heads"], case["batch"], case["page_size"]
    if op in ("scores", "prompt"):
        if op == "scores":
            lens = _lengths(g, b, case["min_len"], case["max_len"])
            new = torch.full((b,), case["queries"], dtype=torch.int32)
        else:
            new = _lengths(g, b, 1, case["max_new"])
            lens = new + _lengths(g, b, 0, case["max_past"])
        cu = torch.cat((torch.zeros(1, dtype=torch.int32), new.cumsum(0).to(torch.int32)))
        # As long as the requests may get, whatever lengths they have now.
        most = case["max_len"] if op == "scores" else case["max_new"] + case["max_past"]
        width, total = max(1, _pages(most, page)), int(cu[-1])
        # A page table of a layer: the requests' pages in any order.
        s.update(cache=randn(b * width * page, INDEX), table=perm(b * width).reshape(b, width), lens=lens.to(dev), page=page, most=most,
                 cu=None if op == "scores" else cu.to(dev), first=cu.to(dev), longest=int(new.max()),
                 q=randn(total, heads, INDEX), weights=randn(total, heads, dtype=torch.float32) * (INDEX * heads) ** -0.5)
        # The selection reads a row's scores up to the row's length only.
        s["out"] = torch.full((total, _pages(most, 4) * 4), -math.inf, device=dev)
        return s
    shared = case["shared"]
    lens = shared + _lengths(g, b, case["min_own"], case["max_own"])
    width, common = _pages(int(lens.max()), page), _pages(shared, page)
    ids = perm(common + b * width)
    table = ids[common:].reshape(b, width).clone()
    # Every request's row begins with the whole pages that all of them share.
    table[:, : shared // page] = ids[: shared // page]
    s.update(cache=randn((common + b * width) * page, WIDTH), table=table, pages=ids[:common].contiguous(), lens=lens.to(dev),
             shared=torch.tensor([shared], dtype=torch.int32, device=dev), n=shared, page=page, scale=(NOPE + ROPE) ** -0.5,
             q=randn(b, case["queries"], heads, WIDTH), workspace=None,
             out=torch.empty(b, case["queries"], heads, LATENT, dtype=dtype, device=dev),
             lse=torch.empty(b, case["queries"], heads, dtype=torch.float32, device=dev))
    return s


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from sparse_attention_indexer_uint32_gb300 import api

    op = s["case"]["op"]
    if op == "append":
        api.index_append(s["rows"], s["slots"], s["cache"], norm_weight=s["weight"], norm_bias=s["bias"], eps=s["eps"], cos_sin=s["cos_sin"],
                         positions=s["positions"], interleaved=s["case"]["interleaved"], rope_last=s["case"]["rope_last"])
        return s["cache"]
    if op == "shared":
        out, lse, s["workspace"] = api.attend_shared(s["q"], s["cache"], s["lens"], s["table"], s["pages"], s["shared"], s["page"], s["scale"],
                                                     out=s["out"], lse=s["lse"], workspace=s["workspace"])
        return {"out": out, "lse": lse}
    return api.index_scores(s["q"], s["weights"], s["cache"], s["lens"], s["table"], s["page"], cu_q=s["cu"], max_seq_len=s["most"], out=s["out"])


def _parts(score, seen, v):
    """Largest score, sum of weights and weighted values of one part of the keys."""
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    return top[..., 0], p.sum(-1), torch.matmul(p, v)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "append":
        x = s["rows"].float()
        x = x - x.mean(1, keepdim=True)
        x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + s["eps"]) * s["weight"].float() + s["bias"].float()
        r, rest = (x[:, INDEX - ROPE:], x[:, : INDEX - ROPE]) if case["rope_last"] else (x[:, :ROPE], x[:, ROPE:])
        cs = s["cos_sin"][s["positions"].long()]
        cos, sin = cs[:, : ROPE // 2], cs[:, ROPE // 2:]
        a, b = (r[:, 0::2], r[:, 1::2]) if case["interleaved"] else (r[:, : ROPE // 2], r[:, ROPE // 2:])
        a, b = a * cos - b * sin, a * sin + b * cos
        r = torch.stack((a, b), 2).flatten(1) if case["interleaved"] else torch.cat((a, b), 1)
        x = torch.cat((rest, r) if case["rope_last"] else (r, rest), 1)
        s["store"][torch.where(s["slots"] < 0, s["n"], s["slots"]).long()] = x.to(s["store"].dtype)
        return s["cache"]
    page = s["page"]
    if op == "shared":
        b, n, h, _ = s["q"].shape
        q, limit = s["q"].float(), s["lens"][:, None] - (n - 1) + torch.arange(n, device="cuda")[None, :]
        pos = torch.arange(s["n"], device="cuda")
        kv = s["cache"][s["pages"].long()[pos // page] * page + pos % page].float()
        score = torch.matmul(q.reshape(b * n * h, WIDTH), kv.t()) * s["scale"]
        seen = (pos[None, None, :] < limit[:, :, None])[:, :, None, :].expand(b, n, h, -1).reshape(b * n * h, -1)
        m0, l0, o0 = (x.reshape(b, n, h, *x.shape[1:]) for x in _parts(score, seen, kv[:, :LATENT]))
        pos = torch.arange(s["n"], s["table"].shape[1] * page, device="cuda")
        kv = s["cache"][s["table"].long()[:, pos // page] * page + pos % page].float()
        score = torch.matmul(q.reshape(b, n * h, WIDTH), kv.transpose(1, 2)) * s["scale"]
        seen = (pos[None, None, :] < limit[:, :, None])[:, :, None, :].expand(b, n, h, -1).reshape(b, n * h, -1)
        m1, l1, o1 = (x.reshape(b, n, h, *x.shape[2:]) for x in _parts(score, seen, kv[..., :LATENT]))
        top = torch.maximum(m0, m1)
        base = torch.where(top == -math.inf, 0.0, top)
        f0, f1 = torch.exp(m0 - base), torch.exp(m1 - base)
        total = l0 * f0 + l1 * f1
        out = (o0 * f0[..., None] + o1 * f1[..., None]) / torch.where(total == 0, 1.0, total)[..., None]
        return {"out": out.to(s["q"].dtype), "lse": torch.log(total) + base}
    # Queries by request, as many rows for each as the longest one has.
    b, n, heads, first = s["lens"].shape[0], s["longest"], case["heads"], s["first"].long()
    total, pos = s["q"].shape[0], torch.arange(s["most"], device="cuda")
    kv = s["cache"][s["table"].long()[:, pos // page] * page + pos % page].float()
    at = (first[:-1, None] + torch.arange(n, device="cuda")[None, :]).clamp(max=total - 1)
    score = torch.matmul(s["q"][at].float().reshape(b, n * heads, INDEX), kv.transpose(1, 2)).clamp_(min=0.0)
    score = torch.matmul(s["weights"][at][:, :, None, :], score.reshape(b, n, heads, -1))[:, :, 0]
    i = torch.arange(total, device="cuda")
    row = torch.searchsorted(first, i, right=True) - 1
    limit = s["lens"][row] - (first[row + 1] - 1 - i)
    out = s["out"][:, : s["most"]]
    out.copy_(torch.where(pos[None, :] < limit[:, None], score[row, i - first[row]], out))
    return s["out"]


def work(case):
    op = case["op"]
    if op == "append":
        return {"bytes": case["tokens"] * (4 * INDEX + 4 * ROPE + 8), "flops": case["tokens"] * (7 * INDEX + 3 * ROPE)}
    b, heads = case["batch"], case["heads"]
    if op == "shared":
        own_rows, n = sum(_spread(b, case["min_own"], case["max_own"])), case["queries"]
        m = b * n * heads
        return {"bytes": (case["shared"] + own_rows) * (2 * WIDTH + 4 / case["page_size"]) + m * (2 * WIDTH + 2 * LATENT + 4),
                "flops": 2 * (case["shared"] * b + own_rows) * n * heads * (WIDTH + LATENT)}
    if op == "scores":
        lens, n = _spread(b, case["min_len"], case["max_len"]), case["queries"]
        keys, queries = sum(lens), b * n
        pairs = sum(max(0, x - i) for x in lens for i in range(n))
    else:
        new, past = _spread(b, 1, case["max_new"]), sum(_spread(b, 0, case["max_past"]))
        keys, queries = sum(new) + past, sum(new)
        # A query sees what is cached before its prompt's piece, and the piece up to itself.
        pairs = sum(new) * past // b + sum(x * (x + 1) // 2 for x in new)
    return {"bytes": keys * (2 * INDEX + 4 / case["page_size"]) + queries * heads * (2 * INDEX + 4) + 4 * pairs,
            "flops": pairs * heads * (2 * INDEX + 3)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "append":
        keep = s["slots"] >= 0
        x, f = s["rows"][keep].double(), s["cos_sin"].double()[s["positions"][keep].long()]
        x = (x - x.mean(1)[:, None]) / (x.var(1, correction=0) + s["eps"]).sqrt()[:, None]
        x = torch.addcmul(s["bias"].double(), x, s["weight"].double())
        turn = slice(INDEX - ROPE, INDEX) if case["rope_last"] else slice(0, ROPE)
        pair = x[:, turn].reshape(-1, ROPE // 2, 2) if case["interleaved"] else x[:, turn].reshape(-1, 2, ROPE // 2).transpose(1, 2)
        pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * torch.complex(f[:, : ROPE // 2], f[:, ROPE // 2:]))
        x[:, turn] = pair.flatten(1) if case["interleaved"] else pair.transpose(1, 2).flatten(1)
        want = s["cache"].double()
        want[s["slots"][keep].long()] = x
        return want
    page = s["page"]
    if op == "shared":
        b, n, h, _ = s["q"].shape
        out = torch.zeros(b, n, h, LATENT, dtype=torch.float64, device="cuda")
        lse = torch.zeros(b, n, h, dtype=torch.float64, device="cuda")
        for r, length in enumerate(s["lens"].tolist()):
            at = torch.arange(length, device="cuda")
            pages = torch.where(at < s["n"], s["pages"].long()[(at // page).clamp(max=s["pages"].shape[0] - 1)], s["table"][r].long()[at // page])
            kv = s["cache"][pages * page + at % page].double()
            for i in range(n):
                seen = kv[: max(0, length - (n - 1 - i))]
                score = torch.einsum("hd,td->ht", s["q"][r, i].double(), seen) * s["scale"]
                lse[r, i] = torch.logsumexp(score, 1)
                out[r, i] = torch.einsum("ht,td->hd", torch.softmax(score, 1), seen[:, :LATENT])
        return {"out": out, "lse": lse}
    want = s["out"].double()
    first = s["first"].tolist()
    for r, length in enumerate(s["lens"].tolist()):
        at = torch.arange(length, device="cuda")
        k = s["cache"][s["table"][r].long()[at // page] * page + at % page].double()
        for i in range(first[r], first[r + 1], 128):
            j = min(i + 128, first[r + 1])
            dot = torch.einsum("qhd,td->qht", s["q"][i:j].double(), k)
            score = (torch.where(dot > 0, dot, 0.0) * s["weights"][i:j].double()[:, :, None]).sum(1)
            last = length - (first[r + 1] - 1 - torch.arange(i, j, device="cuda"))
            want[i:j, :length] = torch.where(at[None, :] < last[:, None], score, want[i:j, :length])
    return want
