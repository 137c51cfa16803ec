"""Behind a shared prompt: queries whose (query, head) rows have one stride while
the requests do not follow one another, and the join's widths in both types."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_attend_shared import WIDTH, Batch, api, randn  # noqa: F401 - a fixture

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("queries", [1, 2])
@pytest.mark.parametrize("batch,heads", [
    (3, 6),    # up to 64 (request, query, head) rows: 32 a block
    (4, 24),   # more, of which each request has fewer
    (3, 70),   # each request has more too
])
@pytest.mark.parametrize("page", [8, 64])
def test_requests_apart(api, queries, batch, heads, page):  # noqa: F811
    x = Batch([300, 290, 400, 256][:batch], 256, queries, heads, page, torch.bfloat16)
    x.q = randn(9, batch, queries + 1, heads, WIDTH)[:, :queries]
    out, lse, _ = x.run(api)
    x.check(out, lse)


# Rows up to 767: 4 values a warp; to 2047: 8; more: 16.
@pytest.mark.parametrize("requests", [150, 300, 700])
def test_joins_in_fp16(api, requests):  # noqa: F811
    g = torch.Generator().manual_seed(3)
    lens = (torch.randint(0, 90, (requests,), generator=g) + 40).tolist()
    x = Batch(lens, 64, 1, 4, 16, torch.float16)
    out, lse, _ = x.run(api)
    x.check(out, lse)
