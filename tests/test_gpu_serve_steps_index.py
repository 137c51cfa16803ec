"""The serving step's indexer and its rows behind a common prompt: what comes out
of the calls in a row is what the plain forms give on what went in."""
from __future__ import annotations

import pytest
import torch

from tests.attend_util import attend, check
from tests.index_util import check_scores

pytestmark = pytest.mark.gpu


def test_scores_of_a_step():
    from sparse_attention_indexer_uint32_gb300 import serve_step as s

    layer = s.Layer(batch=4, pages_per_row=8, page_size=32, seed=5)
    new = torch.tensor([120, 1, 0, 65], dtype=torch.int32, device="cuda")
    _, _, _, step = layer.prompt(new, int(new.sum()))
    layer.take_pages(step)
    for _ in range(2):
        _, _, _, step = layer.decode(k=64)
        layer.take_pages(step)
        q, weights, scores = layer.scored
        before = scores.clone()
        for r, n in enumerate(layer.lens.tolist()):
            before[r, :n] = 0  # what is seen is compared, the rest is as it is
        check_scores(q, weights, layer.index_cache, layer.lens, layer.table, 32, scores, before)
        # Normed, then rotated: the mean of the squares is 1, but for each value's rounding (2^-8 of itself).
        square = layer.index_cache[step.slots.long()].double().square().mean(1)
        assert ((square - 1).abs() < 2.0 ** -6).all()


def test_common_prompt():
    from sparse_attention_indexer_uint32_gb300 import serve_step as s

    layer = s.Layer(batch=5, pages_per_row=8, page_size=32, seed=6)
    layer.common_prompt(pages=3)
    for _ in range(3):
        q, shared, _, step = layer.decode_shared()
        layer.take_pages(step)
        for r, n in enumerate(layer.lens.tolist()):
            t = torch.arange(n, device="cuda")
            kv = layer.cache[layer.table[r].long()[t // 32] * 32 + t % 32]
            o, _, ob, _ = attend(q[r], kv, kv[:, : s.LATENT], s.SCALE, q.dtype)
            check(shared[r], o, ob, f"row {r}")
    assert layer.lens.tolist() == [99] * 5
