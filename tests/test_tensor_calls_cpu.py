"""The compiled module answers whatever it is given with True or False: what is
not a right call's argument is left to the checks in Python."""
from __future__ import annotations

import pytest
import torch

from sparse_attention_indexer_uint32_gb300 import build as build_mod


@pytest.fixture(scope="module")
def calls():
    build_mod.build()
    from sparse_attention_indexer_uint32_gb300 import _lib

    return _lib.tensor_calls


I32, F32 = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 3)
BF = torch.zeros(3, 128, dtype=torch.bfloat16)
ODD = (None, "x", 1 << 80, -1, 1.5, object(), [], I32, F32, BF, torch.zeros(0), torch.nn.Parameter(F32),
       torch.zeros(2, 2).to_sparse(), torch.empty(3, 128, device="meta", dtype=torch.bfloat16))


@pytest.mark.parametrize("name,count", [("index_append", 11), ("index_scores", 10), ("attend_shared", 13)])
def test_odd_arguments(calls, name, count):
    call = getattr(calls, name)
    assert call() is False and call(*[None] * (count + 1)) is False
    for x in ODD:
        assert call(*[x] * count) is False
    for i in range(count):
        for x in ODD:
            args = [BF] * count
            args[i] = x
            assert call(*args) is False


def test_tensors_on_the_cpu(calls):
    q, cache, table = torch.zeros(3, 2, 128, dtype=torch.bfloat16), torch.zeros(64, 128, dtype=torch.bfloat16), torch.zeros(3, 4, dtype=torch.int32)
    assert calls.index_append(BF, I32, cache, None, None, 1e-6, None, None, False, False, None) is False
    assert calls.index_scores(q, torch.zeros(3, 2), cache, I32, table, 16, None, None, torch.zeros(3, 64), None) is False
    assert calls.attend_shared(torch.zeros(3, 1, 2, 576, dtype=torch.bfloat16), torch.zeros(64, 576, dtype=torch.bfloat16), I32, table,
                               I32, I32[:1], 16, 0.1, None, torch.zeros(3, 1, 2, 512, dtype=torch.bfloat16), torch.zeros(3, 1, 2),
                               torch.zeros(1 << 20), None) is False


def test_bind_takes_addresses(calls):
    with pytest.raises(TypeError):
        calls.bind(1, 2)
    with pytest.raises(TypeError):
        calls.bind("a", "b", "c", "d")
