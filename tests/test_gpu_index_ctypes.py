"""The index calls and attention behind a shared prompt where the compiled module
is not there: the same results, and the same refusals."""
from __future__ import annotations

import types

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, SCALE = torch.bfloat16, 0.07


@pytest.fixture
def api(monkeypatch):
    from sparse_attention_indexer_uint32_gb300 import _lib, api

    none = types.SimpleNamespace(index_append=lambda *a: False, index_scores=lambda *a: False, attend_shared=lambda *a: False)
    api.with_module = lambda: monkeypatch.setattr(api, "_calls", _lib.tensor_calls)
    api.without = lambda: monkeypatch.setattr(api, "_calls", none)
    yield api
    del api.with_module, api.without


def randn(*shape, dtype=BF):
    return torch.randn(shape, device="cuda").to(dtype)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def both(api, call, fresh):
    """What the call makes of fresh outputs, with the module and without it."""
    results = []
    for way in (api.with_module, api.without):
        way()
        to = fresh()
        call(*to)
        results.append(to)
    assert all(torch.equal(a, b) for a, b in zip(*results))
    return results[0]


def test_same_results(api):
    rows, slots, weight, bias = randn(5, 192)[:, 32:160], i32([4, 0, -1, 7, 2]), randn(128), randn(128)
    turn, positions, before = torch.randn(10, 64, device="cuda"), i32([1, 2, 3, 0, 9]), randn(8, 160)
    for more in ({}, dict(norm_weight=weight), dict(norm_weight=weight, norm_bias=bias, eps=1e-3),
                 dict(cos_sin=turn, positions=positions, interleaved=True, rope_last=True), dict(cos_sin=turn, positions=positions)):
        cache, = both(api, lambda c: api.index_append(rows, slots, c[:, :128], **more), lambda: [before.clone()])
        assert not torch.equal(cache, before)
    q, heads, keys = randn(7, 10, 128)[:, ::2], torch.randn(7, 8, device="cuda")[:, 1:6], randn(6 * 32, 136)[:, :128]
    lens, table, cu = i32([40, 90]), i32([[0, 1, 2, 9], [3, 4, 5, 9]])[:, :3], i32([0, 2, 7])
    scores, = both(api, lambda out: api.index_scores(q, heads, keys, lens, table, 32, cu_q=cu, max_seq_len=93, out=out),
                   lambda: [torch.zeros(7, 100, device="cuda")])
    assert scores[6, :90].any() and not scores[:, 90:].any()
    x, latent, pages, common = randn(2, 3, 16, 576)[:, :2], randn(10 * 64, 576), i32([6, 7]), i32([100])
    room = torch.empty(api._shared_workspace_bytes(2, 2, 16), dtype=torch.uint8, device="cuda")
    rows = i32([[9, 6, 0, 1, 2], [9, 7, 3, 4, 5]])
    out, lse = both(api, lambda out, lse: api.attend_shared(x, latent, i32([200, 300]), rows, pages, common, 64, SCALE, out=out,
                                                            lse=lse, workspace=room),
                    lambda: [torch.zeros(2, 2, 16, 512, dtype=BF, device="cuda"), torch.zeros(2, 2, 16, device="cuda")])
    assert out.any() and lse.any()


def arguments():
    x = types.SimpleNamespace(
        rows=randn(4, 128), cache=randn(64, 128), slots=i32([0, 3, 5, 8]), w=randn(128), turn=torch.randn(10, 64, device="cuda"),
        positions=i32([1, 2, 3, 0]), q=randn(4, 3, 128), hw=torch.randn(4, 3, device="cuda"), lens=i32([30, 16]),
        table=i32([[0, 1], [2, 3]]), out=torch.zeros(4, 32, device="cuda"), x=randn(2, 1, 3, 576), latent=randn(64, 576), pages=i32([3]),
        common=i32([16]), to=randn(2, 1, 3, 512), lse=torch.zeros(2, 1, 3, device="cuda"),
        room=torch.zeros(1 << 26, dtype=torch.uint8, device="cuda"))
    right = dict(
        index_append=dict(rows=x.rows, slots=x.slots, cache=x.cache, norm_weight=x.w, norm_bias=x.w, eps=1e-6, cos_sin=x.turn,
                          positions=x.positions),
        index_scores=dict(q=x.q, weights=x.hw, cache=x.cache, seq_lens=x.lens, page_table=x.table, page_size=16, out=x.out),
        attend_shared=dict(q=x.x, cache=x.latent, seq_lens=x.lens, page_table=x.table, shared_pages=x.pages, shared_len=x.common,
                           page_size=16, scale=0.1, out=x.to, lse=x.lse, workspace=x.room))
    return x, right


WRONG = [
    ("index_append", [
        lambda x: dict(rows=x.rows.half()), lambda x: dict(rows=x.rows[0]), lambda x: dict(rows=x.rows[:, :64]),
        lambda x: dict(rows=x.rows.t().contiguous().t()), lambda x: dict(rows=x.rows.cpu()),
        lambda x: dict(rows=x.rows.float(), cache=x.cache.float()), lambda x: dict(slots=x.slots.long()),
        lambda x: dict(slots=x.slots[:3]), lambda x: dict(slots=x.slots.cpu()), lambda x: dict(slots=i32(range(8))[::2]),
        lambda x: dict(cache=x.cache[:, :64]), lambda x: dict(cache=x.cache.half()), lambda x: dict(norm_weight=None),
        lambda x: dict(norm_weight=x.w.float()), lambda x: dict(norm_weight=x.w[:64]), lambda x: dict(norm_bias=x.w[::2]),
        lambda x: dict(eps=-1.0), lambda x: dict(eps=float("nan")), lambda x: dict(eps=float("inf")),
        lambda x: dict(cos_sin=x.turn[:, :32]), lambda x: dict(cos_sin=x.turn.double()), lambda x: dict(cos_sin=x.turn[:0]),
        lambda x: dict(cos_sin=x.turn[0]), lambda x: dict(cos_sin=x.turn[0, 0]), lambda x: dict(positions=None),
        lambda x: dict(positions=x.positions[:2]), lambda x: dict(positions=x.positions.long()),
        lambda x: dict(rows=randn(4, 132)[:, 4:])]),
    ("index_scores", [
        lambda x: dict(page_size=0), lambda x: dict(page_size=-16), lambda x: dict(page_size=12),
        lambda x: dict(max_seq_len=33), lambda x: dict(max_seq_len=-1), lambda x: dict(max_seq_len=-1, out=None),
        lambda x: dict(page_size=-16, out=None), lambda x: dict(page_size=0, out=None), lambda x: dict(out=x.out[:, :31]),
        lambda x: dict(out=x.out[:3]), lambda x: dict(out=x.out.t()), lambda x: dict(out=x.out.half()),
        lambda x: dict(out=x.out[0]), lambda x: dict(cu_q=i32([0, 1])), lambda x: dict(cu_q=i32([0, 1, 4]).long()),
        lambda x: dict(weights=x.hw.half()), lambda x: dict(weights=x.hw[:, :2]), lambda x: dict(weights=x.hw[:, 0]),
        lambda x: dict(weights=x.hw[:, :1].expand(4, 3)), lambda x: dict(weights=x.hw[:1].expand(4, 3)),
        lambda x: dict(q=x.q[:3], weights=x.hw[:3], out=x.out[:3]), lambda x: dict(q=x.q[0]), lambda x: dict(q=x.q.float()),
        lambda x: dict(q=x.q[..., :64]), lambda x: dict(q=x.q[:1].expand(4, 3, 128)), lambda x: dict(seq_lens=x.lens[:1]),
        lambda x: dict(seq_lens=x.lens.long()), lambda x: dict(page_table=x.table.float()),
        lambda x: dict(page_table=x.table[0]), lambda x: dict(page_table=x.table.cpu()), lambda x: dict(cache=x.cache[:, :64]),
        lambda x: dict(cache=x.cache.half()), lambda x: dict(cache=x.cache[:0]), lambda x: dict(cache=x.cache[0]),
        lambda x: dict(q=randn(4, 257, 128), weights=torch.randn(4, 257, device="cuda")),
        lambda x: dict(out=x.out[:1].expand(4, 32))]),
    ("attend_shared", [
        lambda x: dict(page_size=0), lambda x: dict(page_size=24), lambda x: dict(max_seq_len=33),
        lambda x: dict(max_seq_len=-1), lambda x: dict(q=x.x[0]), lambda x: dict(q=x.x.float()),
        lambda x: dict(q=x.x[..., :512]), lambda x: dict(cache=x.latent.half()), lambda x: dict(cache=x.latent[:, :512]),
        lambda x: dict(cache=x.latent[0]), lambda x: dict(seq_lens=i32([1, 2, 3])), lambda x: dict(seq_lens=x.lens.long()),
        lambda x: dict(page_table=x.table[:1]), lambda x: dict(page_table=x.table.float()),
        lambda x: dict(shared_pages=x.pages.long()), lambda x: dict(shared_len=i32([1, 2])),
        lambda x: dict(shared_len=x.common.long()), lambda x: dict(scale=float("nan")), lambda x: dict(out=x.to[:, :, :2]),
        lambda x: dict(out=x.to.half()), lambda x: dict(lse=x.lse.double()), lambda x: dict(lse=x.lse[:1]),
        lambda x: dict(workspace=x.room.cpu())]),
]


@pytest.mark.parametrize("name,at", [(name, i) for name, changes in WRONG for i in range(len(changes))])
def test_same_refusals(api, name, at):
    """What is wrong is said by the checks, in the same words, and nothing is written."""
    from sparse_attention_indexer_uint32_gb300._lib import TopkError

    x, right = arguments()
    change = dict(WRONG)[name][at](x)
    kept = [t.clone() for t in (x.cache, x.out, x.to, x.lse)]
    said = []
    for way in (api.with_module, api.without):
        way()
        with pytest.raises((ValueError, TopkError)) as e:
            getattr(api, name)(**{**right[name], **change})
        said.append(str(e.value))
    assert said[0] == said[1]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, (x.cache, x.out, x.to, x.lse)))


def test_right_calls(api):
    _, right = arguments()
    for way in (api.with_module, api.without):
        way()
        for name, args in right.items():
            getattr(api, name)(**args)
    torch.cuda.synchronize()
