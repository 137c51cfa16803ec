"""Which parts a row has stands in the workspace, for every group of rows and in
each call, also where there are none: the join reads nothing else for it."""
from __future__ import annotations

import math

import pytest
import torch

from tests.test_gpu_attend_shared import Batch, api, i32  # noqa: F401 - a fixture

pytestmark = pytest.mark.gpu
ROWS = 128  # (request, query, head) rows of a group


@pytest.mark.parametrize("queries,heads,dtype", [(1, 4, torch.bfloat16), (2, 100, torch.float16), (3, 128, torch.bfloat16)])
@pytest.mark.parametrize("page", [8, 64])
@pytest.mark.parametrize("shared,lens", [
    (0, [0, 70, 0, 300, 1]),         # nothing is shared, and some have nothing at all
    (200, [200, 70, 0, 300, 201]),   # some have nothing of their own
    (200, [200, 200, 200, 3, 0]),    # nobody has
    (0, [0, 0, 0, 0, 0]),
])
def test_records(api, queries, heads, dtype, page, shared, lens):  # noqa: F811
    x = Batch(lens, shared, queries, heads, page, dtype, width=(320 + page - 1) // page)
    _, _, workspace = x.run(api)
    b, each = len(lens), queries * heads
    groups = [-(-b * each // ROWS)] + [-(-each // ROWS)] * b
    records = workspace.view(torch.int32)[: 2 * sum(groups)].view(-1, 2)
    records.fill_(-3)
    out, lse, _ = x.run(api, workspace=workspace)
    x.check(out, lse)
    have = [shared > 0] + [n > shared for n in lens]
    for i, (n, there) in enumerate(zip(groups, have)):
        mine = records[sum(groups[:i]):sum(groups[:i + 1])]
        assert (mine[:, 1] >= 1).all() and (mine[:, 0] >= 0).all() if there else (mine == 0).all(), (i, mine)


def test_lengths_that_change_after_the_call(api):  # noqa: F811
    """What comes behind the call in its stream may write the lengths it was given."""
    x = Batch([900, 700, 650, 0], 640, 1, 16, 64, torch.bfloat16)
    lens, shared = x.lens.clone(), x.shared.clone()
    want, want_lse, workspace = x.run(api)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    for _ in range(50):
        out.fill_(math.nan)
        x.lens.copy_(lens)
        x.shared.copy_(shared)
        x.run(api, out=out, lse=lse, workspace=workspace)
        x.lens.copy_(i32([1, 2, 3, 640]))
        x.shared.copy_(i32([0]))
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
