"""The serving step's calls in a row: what comes out is attention over what went in."""
from __future__ import annotations

import pytest
import torch

from tests.attend_util import attend, check

pytestmark = pytest.mark.gpu


def test_steps():
    from sparse_attention_indexer_uint32_gb300 import serve_step as s

    layer = s.Layer(batch=5, pages_per_row=8, page_size=32, seed=3)
    new = torch.tensor([100, 1, 32, 0, 65], dtype=torch.int32, device="cuda")
    total = int(new.sum())
    q, out, lse, step = layer.prompt(new, total)
    layer.take_pages(step)
    assert step.status.tolist() == [4 + 1 + 1 + 0 + 3, 0] and layer.lens.tolist() == new.tolist()
    latent = layer.cache[step.slots.long()]
    up = torch.einsum("tl,lhd->thd", latent[:, : s.LATENT], layer.up)
    cu = step.cu_new.tolist()
    for r in range(5):
        for i in {cu[r], (cu[r] + cu[r + 1]) // 2, cu[r + 1] - 1} if cu[r + 1] > cu[r] else ():
            k = torch.cat((up[cu[r]:i + 1, 2, : s.NOPE], latent[cu[r]:i + 1, s.LATENT:]), 1)
            o, l, ob, lb = attend(q[i:i + 1, 2], k, up[cu[r]:i + 1, 2, s.NOPE:], s.SCALE, q.dtype)
            check(out[i:i + 1, 2], o, ob, f"prompt {r}, token {i}")
            check(lse[i:i + 1, 2], l, lb, f"prompt {r}, token {i}")
    for _ in range(2):
        q, selected, whole, step = layer.decode(k=128)
        layer.take_pages(step)
        for r, n in enumerate(layer.lens.tolist()):
            t = torch.arange(n, device="cuda")
            kv = layer.cache[layer.table[r].long()[t // 32] * 32 + t % 32]
            o, _, ob, _ = attend(q[r], kv, kv[:, : s.LATENT], s.SCALE, q.dtype)
            check(whole[r], o, ob, f"row {r}")
            if n <= 128:  # every position is selected
                check(selected[r], o, ob, f"row {r}, selected")


def test_main_runs(capsys):
    from sparse_attention_indexer_uint32_gb300 import serve_step

    serve_step.main()
    assert capsys.readouterr().out.count("decode:") == 3
