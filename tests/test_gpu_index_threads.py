"""The index calls and attention behind a shared prompt from several threads at
once, each on a stream of its own: the compiled module lets the others run while
it calls the library."""
from __future__ import annotations

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def randn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def step(api, seed, stream):
    """A step's inputs, and a function that runs it into new outputs."""
    page, b = 64, 3
    cache, latent = randn(seed, 40 * page, 128), randn(seed + 1, 40 * page, 576)
    table, lens = i32(torch.randperm(36, generator=torch.Generator().manual_seed(seed)).reshape(b, 12)), i32([700, 193, 512 + seed])
    q, weights, keys = randn(seed + 2, b, 16, 128), randn(seed + 3, b, 16).float(), randn(seed + 4, 50, 128)
    x, pages, common = randn(seed + 5, b, 1, 16, 576), i32([36, 37, 38]), i32([192])
    room = torch.empty(api._shared_workspace_bytes(b, 1, 16), dtype=torch.uint8, device="cuda")
    slots = i32(torch.arange(50) * 3)

    def run():
        appended, scores = torch.zeros_like(cache), torch.zeros(b, 768, device="cuda")
        out, lse = torch.zeros(b, 1, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(b, 1, 16, device="cuda")
        api.index_append(keys, slots, appended, stream=stream)
        api.index_scores(q, weights, cache, lens, table, page, out=scores, stream=stream)
        api.attend_shared(x, latent, lens, table, pages, common, page, 0.07, out=out, lse=lse, workspace=room, stream=stream)
        return appended, scores, out, lse

    return run


def test_threads():
    from sparse_attention_indexer_uint32_gb300 import _lib, api

    streams = [torch.cuda.Stream() for _ in range(4)]
    steps = [step(api, 10 * i, s) for i, s in enumerate(streams)]
    torch.cuda.synchronize()
    want = []
    for s, run in zip(streams, steps):
        with torch.cuda.stream(s):
            want.append(run())
        s.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                results = [steps[i]() for _ in range(40)]
            streams[i].synchronize()
            wrong.extend(i for r in results for a, b in zip(r, want[i]) if not torch.equal(a, b))
        except Exception as e:  # noqa: BLE001 - said by the assertion
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert wrong == [] and all(t.any() for w in want for t in w) and _lib.topk_read_attend_flags() == 0
