"""Tensors that require a gradient: refused while gradients are recorded, taken as they are otherwise."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
def test_parameters_without_recording(off):
    from sparse_attention_indexer_uint32_gb300 import api

    q = torch.randn(3, 16, 576, device="cuda").to(torch.bfloat16)
    cache = torch.randn(200, 576, device="cuda").to(torch.bfloat16)
    slots = torch.randint(0, 200, (3, 40), device="cuda", dtype=torch.int32)
    rows, at = cache[:4].clone(), torch.arange(100, 104, device="cuda", dtype=torch.int32)
    weight = torch.rand(512, device="cuda").to(torch.bfloat16)
    want = api.attend_selected(q, cache, slots, 0.1)
    kept = cache.clone()
    api.cache_append(rows, at, kept, norm_weight=weight)
    leaf, parameter, place = q.clone().requires_grad_(), torch.nn.Parameter(weight.clone()), cache.clone()
    with pytest.raises(ValueError, match="q requires a gradient"):
        api.attend_selected(leaf, cache, slots, 0.1)
    with pytest.raises(ValueError, match="norm_weight requires a gradient"):
        api.cache_append(rows, at, place, norm_weight=parameter)
    assert torch.equal(place, cache)
    with off():
        got = api.attend_selected(leaf, cache, slots, 0.1)
        api.cache_append(rows, at, place, norm_weight=parameter)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(place, kept)
