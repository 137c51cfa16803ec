"""Tables of angles that the append calls refuse: an empty one has no address, and
would pass for none at all.  Fake devices and a fake library, no GPU."""
from __future__ import annotations

import pytest
import torch

from tests.test_current_device_cpu import api, on  # noqa: F401 - a fixture


@pytest.mark.parametrize("gpu", [0, 1])
@pytest.mark.parametrize("name,width", [("cache_append", 576), ("index_append", 128)])
@pytest.mark.parametrize("shape", [(0, 64), (64,), (), (3, 64, 1)])
def test_angles(api, name, width, gpu, shape):  # noqa: F811
    bf = dict(dtype=torch.bfloat16)
    z = lambda *s, **kw: on(gpu, torch.zeros(s, **kw))  # noqa: E731
    args = z(3, width, **bf), z(3, dtype=torch.int32), z(9, width, **bf)
    positions = z(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="cos_sin"):
        getattr(api, name)(*args, cos_sin=z(*shape), positions=positions)
    assert api.state["calls"] == []
    getattr(api, name)(*args, cos_sin=z(1, 64), positions=positions)
    assert api.state["calls"] == [("topk_" + name, gpu)]
