"""The calls around the selection have no backward pass: a tensor that requires
a gradient is refused where gradients are recorded (CPU tensors: the refusal
comes before the one of their device)."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_indexer_uint32_gb300 import build as build_mod

BF = dict(dtype=torch.bfloat16)


@pytest.fixture(scope="module")
def api():
    build_mod.build()
    from sparse_attention_indexer_uint32_gb300 import api

    return api


def tensors():
    i32 = torch.zeros(3, dtype=torch.int32)
    return {
        "cache_append": dict(rows=torch.zeros(3, 576, **BF), slots=i32, cache=torch.zeros(10, 576, **BF),
                             norm_weight=torch.ones(512, **BF), cos_sin=torch.zeros(4, 64), positions=i32),
        "attend_selected": dict(q=torch.zeros(3, 2, 576, **BF), cache=torch.zeros(10, 576, **BF),
                                indices=torch.zeros(3, 4, dtype=torch.int32), scale=0.1,
                                out=torch.zeros(3, 2, 512, **BF), lse=torch.zeros(3, 2)),
        "attend_paged": dict(q=torch.zeros(3, 1, 2, 576, **BF), cache=torch.zeros(10, 576, **BF), seq_lens=i32,
                             page_table=torch.zeros(3, 4, dtype=torch.int32), page_size=16, scale=0.1,
                             out=torch.zeros(3, 1, 2, 512, **BF), lse=torch.zeros(3, 1, 2)),
        "attend_prompt": dict(q=torch.zeros(5, 2, 192, **BF), k_nope=torch.zeros(6, 2, 128, **BF),
                              k_rope=torch.zeros(6, 64, **BF), v=torch.zeros(6, 2, 128, **BF),
                              cu_q=i32, cu_k=i32, scale=0.1, out=torch.zeros(5, 2, 128, **BF), lse=torch.zeros(5, 2)),
    }


CASES = [(call, name) for call, args in tensors().items() for name, t in args.items()
         if isinstance(t, torch.Tensor) and t.dtype != torch.int32]


@pytest.mark.parametrize("call,name", CASES)
def test_refused(api, call, name):
    args = tensors()[call]
    args[name].requires_grad_()
    with pytest.raises(ValueError, match=f"{name} requires a gradient"):
        getattr(api, call)(**args)
    with torch.no_grad(), pytest.raises(ValueError, match="on a GPU"):  # as without a gradient
        getattr(api, call)(**args)
