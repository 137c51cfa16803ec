"""Measured cases of the operators around the selection: the block tables and
slot maps a step starts from, the append of its latent rows to the paged
cache, and latent attention over that cache (selected positions, whole rows
through the page table, and the expanded form for prompts).

``run`` computes a pass with elementary torch operations in 32 bits, or, where
``own`` is true, with the framework's entry points.  A latent row holds 512
values and 64 rotary ones; the expanded form has 128 + 64 values per query and
key head and 128 per value head.
"""
import math

import torch

own = False

LATENT, ROPE, NOPE, VDIM = 512, 64, 128, 128
WIDTH = LATENT + ROPE
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # One decode step of 32 requests, a new token each, 64K of context at most: a launch's latency.
        {"name": "tables_decode32", "op": "tables", "batch": 32, "max_context": 65536, "max_new": 1, "page_size": 64},
        # A mixed step of 4096 requests: prompts' chunks of up to 512 tokens beside short ones, pages of 64.
        {"name": "tables_mixed4096", "op": "tables", "batch": 4096, "max_context": 32768, "max_new": 512, "page_size": 64},
        # The rows of a decode step of 64 requests.
        {"name": "append_decode64", "op": "append", "tokens": 64, "slots": 65536, "dtype": "bf16", "interleaved": True},
        # The rows of a prefill step of 65536 tokens, some of them without a slot.
        {"name": "append_prompt65536", "op": "append", "tokens": 65536, "slots": 131072, "dtype": "fp16", "interleaved": False},
        # One request of long context, its 2048 selected positions, all 128 heads on the GPU.
        {"name": "selected_one", "op": "selected", "rows": 1, "heads": 128, "k": 2048, "min_len": 65536, "max_len": 65536, "page_size": 64, "dtype": "bf16"},
        # A wide decode step (or a piece of a prompt): 128 rows with 2048 positions each.
        {"name": "selected_wide", "op": "selected", "rows": 128, "heads": 128, "k": 2048, "min_len": 8192, "max_len": 8192, "page_size": 64, "dtype": "bf16"},
        # The decode batch's 2048 rows with k = 512 and the 16 heads of one of 8 shards; rows from empty to 4096 long.
        {"name": "selected_heads16", "op": "selected", "rows": 2048, "heads": 16, "k": 512, "min_len": 0, "max_len": 4096, "page_size": 64, "dtype": "fp16"},
        # Whole rows of 16 requests of up to 131072 tokens, one query each.
        {"name": "paged_long16", "op": "paged", "batch": 16, "queries": 1, "heads": 128, "min_len": 32768, "max_len": 131072, "page_size": 64, "dtype": "bf16"},
        # 64 requests that verify 4 proposed tokens each, 16 heads, ragged lengths from empty on, pages of 128.
        {"name": "paged_verify64", "op": "paged", "batch": 64, "queries": 4, "heads": 16, "min_len": 0, "max_len": 8192, "page_size": 128, "dtype": "fp16"},
        # A few short prompts together.
        {"name": "prompt_short4", "op": "prompt", "batch": 4, "heads": 16, "max_new": 300, "max_past": 0, "causal": True, "dtype": "bf16"},
        # One prompt of 8192 tokens.
        {"name": "prompt_one8192", "op": "prompt", "batch": 1, "heads": 32, "max_new": 8192, "max_past": 0, "causal": True, "dtype": "bf16"},
        # Pieces of 8 prompts after what is cached of them already (up to 4096 tokens each).
        {"name": "prompt_pieces8", "op": "prompt", "batch": 8, "heads": 16, "max_new": 1024, "max_past": 4096, "causal": True, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("tables", "append", "selected", "paged", "prompt", "selected", "paged", "prompt"))
    dtype = rng.choice(("bf16", "fp16"))
    page = rng.choice((16, 32, 64, 128))
    if op == "tables":
        batch, new = _log(rng, 1, 4096), _log(rng, 1, 4096)
        return {"op": op, "batch": batch, "max_context": _log(rng, 64, 32768), "max_new": min(new, max(1, 2 ** 21 // batch)), "page_size": page}
    if op == "append":
        tokens = _log(rng, 1, 65536)
        return {"op": op, "tokens": tokens, "slots": 2 * tokens, "dtype": dtype, "interleaved": rng.random() < 0.5}
    if op == "selected":
        heads, k = rng.choice((8, 16, 24, 32, 64, 100, 128)), _log(rng, 1, 2048)
        rows = _log(rng, 1, max(1, min(2048, 2 ** 18 // k, 2 ** 25 // (k * heads))))
        most = _log(rng, k, max(k, min(65536, 2 ** 20 // rows)))
        return {"op": op, "rows": rows, "heads": heads, "k": k, "min_len": rng.choice((0, 1, most)), "max_len": most, "page_size": page, "dtype": dtype}
    if op == "paged":
        heads, queries = rng.choice((8, 16, 20, 64, 128)), rng.choice((1, 1, 2, 3, 5))
        most = _log(rng, 1, 131072)
        batch = _log(rng, 1, max(1, min(256, 2 ** 20 // most, 2 ** 27 // (most * heads * queries))))
        return {"op": op, "batch": batch, "queries": queries, "heads": heads, "min_len": rng.choice((0, 1, most)), "max_len": most, "page_size": page, "dtype": dtype}
    heads, batch = rng.choice((1, 3, 8, 16, 32)), rng.choice((1, 2, 3, 5, 8))
    new = _log(rng, 1, max(64, 8192 // batch))
    past = rng.choice((0, 0, _log(rng, 1, 8192 // batch)))
    return {"op": op, "batch": batch, "heads": heads, "max_new": new, "max_past": past, "causal": rng.random() < 0.75, "dtype": dtype}


def _spread(count, lo, hi):
    """Lengths spread evenly from lo to hi, one alone hi."""
    return [lo + (hi - lo) * i // (count - 1) for i in range(count)] if count > 1 else [hi]


def _lengths(g, count, lo, hi):
    """Those lengths, in an order of the seed's."""
    return torch.tensor(_spread(count, lo, hi), dtype=torch.int32)[torch.randperm(count, generator=g)]


def _generators(seed):
    g, h = torch.Generator(), torch.Generator(device="cuda")
    g.manual_seed(seed)
    h.manual_seed(seed + 1)
    return g, h


def _pages(n, page):
    return (n + page - 1) // page


def prepare(case, seed):
    g, h = _generators(seed)
    dev = torch.device("cuda")
    op = case["op"]
    randn = lambda *shape, dtype=torch.float32: torch.randn(shape, generator=h, device=dev, dtype=dtype)  # noqa: E731
    perm = lambda n: torch.randperm(n, generator=h, device=dev).to(torch.int32)  # noqa: E731
    s = {"case": dict(case)}
    if op == "tables":
        b, page = case["batch"], case["page_size"]
        context = _lengths(g, b, 0, case["max_context"])
        new = _lengths(g, b, 1 if case["max_new"] == 1 else 0, case["max_new"])
        width = _pages(case["max_context"] + case["max_new"], page)
        have = _pages(context, page)
        total = int(new.sum())
        need = int((_pages(context + new, page) - have).sum())
        held = b * width
        ids = perm(held + need)
        table = ids[:held].reshape(b, width).clone()
        table[torch.arange(width, device=dev)[None, :] >= have.to(dev)[:, None]] = -1
        # A step's buffers have room to spare, and so has the list of free pages.
        s.update(context=context.to(dev), new=new.to(dev), table=table, free=ids[held:].contiguous() if need else perm(1),
                 page=page, tokens=total + total // 8 + 7, outs=None)
        return s
    dtype = DTYPES[case["dtype"]]
    if op == "append":
        t, n = case["tokens"], case["slots"]
        # The rows are a slice of a wider projection's output.
        wide = randn(t, WIDTH + 192, dtype=dtype)
        slots = perm(n)[:t].clone()
        if t > 16:
            slots[torch.rand(t, generator=h, device=dev) < 0.02] = -1
        positions = torch.randint(0, 16384, (t,), generator=h, device=dev, dtype=torch.int32)
        angle = torch.arange(16384, device=dev, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(ROPE // 2, device=dev, dtype=torch.float64) / (ROPE // 2))
        s.update(rows=wide[:, 192:], slots=slots, positions=positions, weight=(1 + 0.1 * randn(LATENT)).to(dtype),
                 cos_sin=torch.cat((angle.cos(), angle.sin()), 1).float(), eps=1e-6, interleaved=case["interleaved"],
                 # One row past the cache takes what has no slot in the plain form.
                 store=randn(n + 1, WIDTH, dtype=dtype), n=n)
        s["cache"] = s["store"][:n]
        return s
    if op in ("selected", "paged"):
        page, heads = case["page_size"], case["heads"]
        b = case["rows"] if op == "selected" else case["batch"]
        lens = _lengths(g, b, case["min_len"], case["max_len"]).to(dev)
        width = _pages(case["max_len"], page)
        table = perm(b * width).reshape(b, width)
        s.update(cache=randn(b * width * page, WIDTH, dtype=dtype), lens=lens, scale=(NOPE + ROPE) ** -0.5, page=page, workspace=None)
        if op == "selected":
            k, most = case["k"], case["max_len"]
            at = torch.rand((b, most), generator=h, device=dev)
            at = torch.where(torch.arange(most, device=dev)[None, :] < lens[:, None], at, -1.0)
            top = at.topk(k, 1, sorted=False)
            idx = torch.where(top.values >= 0, top.indices, -1)
            # The selection writes its positions first and -1 in the slots past them.
            idx = idx.gather(1, (idx < 0).to(torch.uint8).sort(dim=1, stable=True).indices)
            slot = table.long().gather(1, idx.clamp(min=0) // page) * page + idx.clamp(min=0) % page
            s.update(q=randn(b, heads, WIDTH, dtype=dtype), indices=torch.where(idx >= 0, slot, -1).to(torch.int32))
        else:
            s.update(q=randn(b, case["queries"], heads, WIDTH, dtype=dtype), table=table)
        s["out"] = torch.empty(s["q"].shape[:-1] + (LATENT,), dtype=dtype, device=dev)
        s["lse"] = torch.empty(s["q"].shape[:-1], dtype=torch.float32, device=dev)
        return s
    heads, b = case["heads"], case["batch"]
    new, past = _lengths(g, b, 1, case["max_new"]), _lengths(g, b, 0, case["max_past"])
    zero = torch.zeros(1, dtype=torch.int32)
    cu_q = torch.cat((zero, new.cumsum(0).to(torch.int32)))
    cu_k = torch.cat((zero, (new + past).cumsum(0).to(torch.int32)))
    tq, tk = int(cu_q[-1]), int(cu_k[-1])
    # Keys and values are the two parts of one up-projection's output; the rotary part is one row for all heads.
    up = randn(tk, heads, NOPE + VDIM, dtype=dtype)
    s.update(q=randn(tq, heads, NOPE + ROPE, dtype=dtype), k_nope=up[..., :NOPE], k_rope=randn(tk, ROPE, dtype=dtype), v=up[..., NOPE:],
             cu_q=cu_q.to(dev), cu_k=cu_k.to(dev), scale=(NOPE + ROPE) ** -0.5, causal=case["causal"],
             out=torch.empty(tq, heads, VDIM, dtype=dtype, device=dev), lse=torch.empty(tq, heads, dtype=torch.float32, device=dev))
    return s


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from sparse_attention_indexer_uint32_gb300 import api

    op = s["case"]["op"]
    if op == "tables":
        s["outs"] = r = api.block_tables(s["context"], s["new"], s["free"], s["table"], s["page"], s["tokens"], out=s["outs"])
        return {"table": s["table"], "seq_lens": r.seq_lens, "cu_new": r.cu_new, "slots": r.slots, "positions": r.positions, "rows": r.rows}
    if op == "append":
        api.cache_append(s["rows"], s["slots"], s["cache"], norm_weight=s["weight"], eps=s["eps"], cos_sin=s["cos_sin"],
                         positions=s["positions"], interleaved=s["interleaved"])
        return s["cache"]
    if op == "selected":
        out, lse, s["workspace"] = api.attend_selected(s["q"], s["cache"], s["indices"], s["scale"], seq_lens=s["lens"],
                                                       out=s["out"], lse=s["lse"], workspace=s["workspace"])
    elif op == "paged":
        out, lse, s["workspace"] = api.attend_paged(s["q"], s["cache"], s["lens"], s["table"], s["page"], s["scale"],
                                                    out=s["out"], lse=s["lse"], workspace=s["workspace"])
    else:
        out, lse = api.attend_prompt(s["q"], s["k_nope"], s["k_rope"], s["v"], s["cu_q"], s["cu_k"], s["scale"],
                                     causal=s["causal"], out=s["out"], lse=s["lse"])
    return {"out": out, "lse": lse}


def _softmax_parts(score, seen):
    """Weights (rows that see nothing: zeros) and log-sum-exp of masked scores."""
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total), (torch.log(total) + top)[..., 0]


def _run_plain(s):
    op = s["case"]["op"]
    if op == "tables":
        return _plain_tables(s)
    if op == "append":
        x = s["rows"].float()
        c, r = x[:, :LATENT], x[:, LATENT:]
        c = c * torch.rsqrt((c * c).mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
        cs = s["cos_sin"][s["positions"].long()]
        cos, sin = cs[:, : ROPE // 2], cs[:, ROPE // 2:]
        a, b = (r[:, 0::2], r[:, 1::2]) if s["interleaved"] else (r[:, : ROPE // 2], r[:, ROPE // 2:])
        a, b = a * cos - b * sin, a * sin + b * cos
        r = torch.stack((a, b), 2).flatten(1) if s["interleaved"] else torch.cat((a, b), 1)
        s["store"][torch.where(s["slots"] < 0, s["n"], s["slots"]).long()] = torch.cat((c, r), 1).to(s["store"].dtype)
        return s["cache"]
    dtype = s["q"].dtype
    if op == "selected":
        idx = s["indices"].long()
        kv = s["cache"][idx.clamp(min=0)].float()
        score = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * s["scale"]
        p, lse = _softmax_parts(score, (idx >= 0)[:, None, :])
        return {"out": torch.matmul(p, kv[..., :LATENT]).to(dtype), "lse": lse}
    if op == "paged":
        b, n, h, _ = s["q"].shape
        width, page = s["table"].shape[1], s["page"]
        pos = torch.arange(width * page, device="cuda")
        slot = s["table"].long()[:, pos // page] * page + pos % page
        kv = s["cache"][slot].float()
        score = torch.matmul(s["q"].float().reshape(b, n * h, WIDTH), kv.transpose(1, 2)).reshape(b, n, h, -1) * s["scale"]
        limit = s["lens"][:, None] - (n - 1) + torch.arange(n, device="cuda")[None, :]
        p, lse = _softmax_parts(score, (pos[None, None, :] < limit[:, :, None])[:, :, None, :])
        out = torch.matmul(p.reshape(b, n * h, -1), kv[..., :LATENT])
        return {"out": out.reshape(b, n, h, LATENT).to(dtype), "lse": lse}
    q, k_nope, k_rope, v = (s[x].float() for x in ("q", "k_nope", "k_rope", "v"))
    score = torch.matmul(q[..., :NOPE].transpose(0, 1), k_nope.permute(1, 2, 0))
    score += torch.matmul(q[..., NOPE:].transpose(0, 1), k_rope.t())
    score *= s["scale"]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    i, j = torch.arange(q.shape[0], device="cuda"), torch.arange(v.shape[0], device="cuda")
    ri, rj = torch.searchsorted(cu_q, i, right=True) - 1, torch.searchsorted(cu_k, j, right=True) - 1
    # The last query of a request sees its last key.
    last = i - cu_q[ri + 1] + cu_k[ri + 1] if s["causal"] else cu_k[ri + 1] - 1
    p, lse = _softmax_parts(score, ((ri[:, None] == rj[None, :]) & (j[None, :] <= last[:, None]))[None])
    return {"out": torch.matmul(p, v.transpose(0, 1)).transpose(0, 1).to(dtype), "lse": lse.t().contiguous()}


def _plain_tables(s):
    context, new, page, table = s["context"].long(), s["new"].long(), s["page"], s["table"]
    b, width = table.shape
    total = context + new
    have = (context + page - 1) // page
    need = (total + page - 1) // page - have
    ends = need.cumsum(0)
    col = torch.arange(width, device="cuda")[None, :]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    at = (ends - need)[:, None] + col - have[:, None]
    table.copy_(torch.where(fresh, s["free"][at.clamp(0, s["free"].numel() - 1)], table))
    cu = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), new.cumsum(0)))
    t = torch.arange(s["tokens"], device="cuda")
    live = t < cu[-1]
    row = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=b - 1)
    pos = context[row] + t - cu[row]
    slot = table[row, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return {"table": table, "seq_lens": i32(total), "cu_new": i32(cu), "slots": i32(torch.where(live, slot, -1)),
            "positions": i32(torch.where(live, pos, -1)), "rows": i32(torch.where(live, row, -1))}


def work(case):
    op = case["op"]
    if op == "tables":
        b, page = case["batch"], case["page_size"]
        new = sum(_spread(b, 1 if case["max_new"] == 1 else 0, case["max_new"]))
        # Lengths in; lengths, offsets and three values a token out; a page read and written for each new one.
        return {"bytes": 16 * b + 12 * (new + new // 8 + 7) + 8 * new / page, "flops": 0}
    if op == "append":
        return {"bytes": case["tokens"] * (4 * WIDTH + 4 * ROPE + 8), "flops": case["tokens"] * (4 * LATENT + 3 * ROPE)}
    if op == "selected":
        n = sum(min(x, case["k"]) for x in _spread(case["rows"], case["min_len"], case["max_len"]))
        m = case["rows"] * case["heads"]
        return {"bytes": n * (2 * WIDTH + 4) + m * (2 * WIDTH + 2 * LATENT + 4), "flops": 2 * n * case["heads"] * (WIDTH + LATENT)}
    if op == "paged":
        n = sum(_spread(case["batch"], case["min_len"], case["max_len"]))
        m = case["batch"] * case["queries"] * case["heads"]
        return {"bytes": n * (2 * WIDTH + 4 / case["page_size"]) + m * (2 * WIDTH + 2 * LATENT + 4),
                "flops": 2 * n * case["heads"] * case["queries"] * (WIDTH + LATENT)}
    b, h = case["batch"], case["heads"]
    new, past = _spread(b, 1, case["max_new"]), sum(_spread(b, 0, case["max_past"]))
    pairs = sum(new) * past / b + sum(x * x for x in new) / (2 if case["causal"] else 1)
    rows = sum(new) + past
    return {"bytes": 2 * (h * (sum(new) * (NOPE + ROPE + VDIM + 2) + rows * (NOPE + VDIM)) + rows * ROPE),
            "flops": 2 * pairs * h * (NOPE + ROPE + VDIM)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "tables":
        return None  # whole numbers only
    if op == "append":
        keep = s["slots"] >= 0
        x, f = s["rows"][keep].double(), s["cos_sin"].double()[s["positions"][keep].long()]
        latent = x[:, :LATENT] / (x[:, :LATENT].square().mean(1) + s["eps"]).sqrt()[:, None] * s["weight"].double()
        pair = x[:, LATENT:].reshape(-1, ROPE // 2, 2) if s["interleaved"] else x[:, LATENT:].reshape(-1, 2, ROPE // 2).transpose(1, 2)
        turned = torch.view_as_complex(pair.contiguous()) * torch.complex(f[:, : ROPE // 2], f[:, ROPE // 2:])
        turned = torch.view_as_real(turned)
        turned = turned.flatten(1) if s["interleaved"] else turned.transpose(1, 2).flatten(1)
        want = s["cache"].double()
        want[s["slots"][keep].long()] = torch.cat((latent, turned), 1)
        return want
    outs, lses = [], []

    def attend(q, k, v):
        """q [m, h, d], k [n, (h,) d], v [n, (h,) e] of 64 bits: their outputs and log-sum-exps."""
        if not k.shape[0]:
            return q.new_zeros(q.shape[0], q.shape[1], v.shape[-1]), q.new_full(q.shape[:2], -math.inf)
        score = (torch.einsum("mhd,nhd->mhn", q, k) if k.dim() == 3 else torch.einsum("mhd,nd->mhn", q, k)) * s["scale"]
        lse = torch.logsumexp(score, -1)
        p = torch.exp(score - lse[..., None])
        return (torch.einsum("mhn,nhe->mhe", p, v) if v.dim() == 3 else torch.einsum("mhn,ne->mhe", p, v)), lse

    if op == "selected":
        for r in range(case["rows"]):
            idx = s["indices"][r]
            kv = s["cache"][idx[idx >= 0].long()].double()
            o, l = attend(s["q"][r:r + 1].double(), kv, kv[:, :LATENT])
            outs.append(o)
            lses.append(l)
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    if op == "paged":
        for r, n in enumerate(s["lens"].tolist()):
            at = torch.arange(n, device="cuda")
            kv = s["cache"][s["table"][r].long()[at // s["page"]] * s["page"] + at % s["page"]].double()
            for i in range(case["queries"]):
                m = max(0, n - (case["queries"] - 1 - i))
                o, l = attend(s["q"][r, i:i + 1].double(), kv[:m], kv[:m, :LATENT])
                outs.append(o)
                lses.append(l)
        shape = (case["batch"], case["queries"], case["heads"])
        return {"out": torch.cat(outs).reshape(*shape, LATENT), "lse": torch.cat(lses).reshape(shape)}
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    for r in range(case["batch"]):
        a, b = slice(cu_q[r], cu_q[r + 1]), slice(cu_k[r], cu_k[r + 1])
        nq, nk = a.stop - a.start, b.stop - b.start
        # Scores that a query may not see are left out of the sums by -inf.
        hide = torch.ones(nq, nk, dtype=torch.bool, device="cuda").triu(nk - nq + 1) if s["causal"] else None
        for h in range(case["heads"]):
            k = torch.cat((s["k_nope"][b, h], s["k_rope"][b]), 1).double()
            score = s["q"][a, h].double() @ k.t() * s["scale"]
            if hide is not None:
                score.masked_fill_(hide, -math.inf)
            lse[a, h] = torch.logsumexp(score, 1)
            out[a, h] = torch.exp(score - lse[a, h][:, None]) @ s["v"][b, h].double()
    return {"out": out, "lse": lse}
