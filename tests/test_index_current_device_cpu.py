"""The index calls and attention behind a shared prompt make the tensors' GPU
the current one where it is not.  Fake devices and a fake library, no GPU."""
from __future__ import annotations

import pytest
import torch

from tests.test_current_device_cpu import api, on  # noqa: F401 - a fixture


@pytest.mark.parametrize("gpu", [0, 1, 5])
def test_launched_where_the_tensors_are(api, gpu):  # noqa: F811
    bf = dict(dtype=torch.bfloat16)
    z = lambda *shape, **kw: on(gpu, torch.zeros(*shape, **kw))  # noqa: E731
    i32 = lambda *shape: z(*shape, dtype=torch.int32)  # noqa: E731
    api.index_append(z(3, 128, **bf), i32(3), z(9, 128, **bf), norm_weight=z(128, **bf), norm_bias=z(128, **bf))
    api.index_scores(z(6, 2, 128, **bf), z(6, 2), z(9, 128, **bf), i32(3), i32(3, 4), 16, out=z(6, 64))
    room = api._shared_workspace_bytes(3, 1, 2)
    api.attend_shared(z(3, 1, 2, 576, **bf), z(9, 576, **bf), i32(3), i32(3, 4), i32(2), i32(1), 16, 0.1,
                      out=z(3, 1, 2, 512, **bf), lse=z(3, 1, 2), workspace=z(room, dtype=torch.uint8))
    assert api.state["calls"] == [(name, gpu) for name in ("topk_index_append", "topk_index_scores", "topk_attend_shared")]
    assert api.state["current"] == 0  # as it was


def test_tensors_on_two_gpus_are_refused(api):  # noqa: F811
    bf = dict(dtype=torch.bfloat16)
    z = lambda gpu, *shape, **kw: on(gpu, torch.zeros(*shape, **kw))  # noqa: E731
    i32 = lambda gpu, *shape: z(gpu, *shape, dtype=torch.int32)  # noqa: E731
    # (fake devices differ in get_device only: what is checked is that no call is made)
    for call in (lambda: api.index_append(z(1, 3, 128, **bf), i32(0, 3), z(1, 9, 128, **bf)),
                 lambda: api.index_scores(z(1, 6, 2, 128, **bf), z(1, 6, 2), z(1, 9, 128, **bf), i32(1, 3), i32(0, 3, 4), 16),
                 lambda: api.attend_shared(z(1, 3, 1, 2, 576, **bf), z(1, 9, 576, **bf), i32(1, 3), i32(1, 3, 4), i32(1, 2),
                                           i32(0, 1), 16, 0.1)):
        with pytest.raises(ValueError):
            call()
    assert api.state["calls"] == []
