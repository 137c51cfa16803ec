"""An empty table of angles is refused, not taken for none."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,width", [("cache_append", 576), ("index_append", 128)])
def test_empty_table_of_angles(name, width):
    from sparse_attention_indexer_uint32_gb300 import _lib, api

    i32 = dict(dtype=torch.int32, device="cuda")
    rows, cache = torch.randn(4, width, device="cuda").half(), torch.zeros(9, width, device="cuda").half()
    slots, turn = torch.arange(4, **i32), torch.randn(10, 64, device="cuda")
    with pytest.raises(ValueError, match="cos_sin"):
        getattr(api, name)(rows, slots, cache, cos_sin=turn[:0], positions=slots)
    assert not cache.any()
    if name == "index_append":
        assert _lib.tensor_calls.index_append(rows, slots, cache, None, None, 1e-6, turn[:0], slots, False, False, None) is False
    getattr(api, name)(rows, slots, cache, cos_sin=turn[:4], positions=slots)
    assert cache[:4].any() and not cache[4:].any()
