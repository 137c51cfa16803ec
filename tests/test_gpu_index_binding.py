"""The binding's functions of the C names for the index calls and attention
behind a shared prompt, called as the header lists their arguments, against the
tensor calls; and tensors that require a gradient."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, SCALE = torch.bfloat16, 0.07


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_indexer_uint32_gb300 import _lib

    return _lib


@pytest.fixture(scope="module")
def api(lib):
    from sparse_attention_indexer_uint32_gb300 import api

    return api


def randn(*shape, dtype=BF):
    return torch.randn(shape, device="cuda").to(dtype)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("interleaved,rope_last", [(False, True), (True, False)])
def test_index_append(lib, api, interleaved, rope_last):
    rows, weight, bias, slots = randn(5, 192), randn(128), randn(128), i32([4, 0, -1, 7, 2])
    turn, positions = torch.randn(10, 64, device="cuda"), i32([1, 2, 3, 0, 9])
    a, b = randn(8, 160), None
    b = a.clone()
    api.index_append(rows[:, :128], slots, a[:, :128], weight, bias, 1e-5, turn, positions, interleaved, rope_last)
    lib.topk_index_append(rows, 192, 5, weight, bias, 1e-5, turn, 10, positions, interleaved, rope_last, slots, b, 160, 8,
                          lib.TOPK_BF16)
    assert torch.equal(a, b)


def test_index_scores(lib, api):
    q, weights, cache = randn(7, 5, 128), torch.randn(7, 5, device="cuda"), randn(6 * 32, 128)
    lens, table, cu = i32([40, 90]), i32([[0, 1, 2], [3, 4, 5]]), i32([0, 2, 7])
    a, b = torch.zeros(7, 100, device="cuda"), torch.zeros(7, 100, device="cuda")
    api.index_scores(q, weights, cache, lens, table, 32, cu_q=cu, out=a)
    lib.topk_index_scores(q, 5 * 128, 128, weights, 5, cache, 128, 192, lens, table, 3, 32, 96, cu, 2, 7, 5, lib.TOPK_BF16, b, 100)
    assert torch.equal(a, b) and a[6, :90].any() and not a[:, 90:].any()


def test_attend_shared(lib, api):
    q, cache = randn(2, 1, 16, 576), randn(10 * 64, 576)
    lens, table, pages, common = i32([200, 300]), i32([[9, 9, 0, 1, 2], [9, 9, 3, 4, 5]]), i32([6, 7]), i32([128])
    want, want_lse, _ = api.attend_shared(q, cache, lens, table, pages, common, 64, SCALE)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    room = torch.empty(lib.topk_attend_shared_workspace_bytes(2, 1, 16), dtype=torch.uint8, device="cuda")
    for place in (lse, None):
        out.zero_()
        lib.topk_attend_shared(q, 16 * 576, 16 * 576, 576, cache, 576, 640, lens, table, 5, pages, 2, common, 64, 320, 2, 1, 16,
                               SCALE, lib.TOPK_BF16, out, place, room)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # Nothing is shared: no list is needed, and it is attention over whole rows.
    common.zero_()
    lib.topk_attend_shared(q, 16 * 576, 16 * 576, 576, cache, 576, 640, lens, table, 5, None, 0, common, 64, 320, 2, 1, 16, SCALE,
                           lib.TOPK_BF16, out, lse, room)
    whole, whole_lse, _ = api.attend_paged(q, cache, lens, table, 64, SCALE)
    # Two roundings of the output and one of each weight, 2^-8 of values up to 4 or so.
    assert (out.float() - whole.float()).abs().max() < 2.0 ** -5 and (lse - whole_lse).abs().max() < 2.0 ** -16


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
def test_parameters_without_recording(api, off):
    rows, cache, weight = randn(4, 128), randn(9, 128), torch.nn.Parameter(randn(128))
    place, kept = cache.clone(), cache.clone()
    at = i32([0, 3, 5, 8])
    api.index_append(rows, at, kept, norm_weight=weight.detach())
    with pytest.raises(ValueError, match="norm_weight requires a gradient"):
        api.index_append(rows, at, place, norm_weight=weight)
    assert torch.equal(place, cache)
    q, w = randn(2, 3, 128), torch.randn(2, 3, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="weights requires a gradient"):
        api.index_scores(q, w, cache, i32([9, 9]), i32([[0], [0]]), 16)
    want = api.index_scores(q, w.detach(), cache, i32([9, 9]), i32([[0], [0]]), 16)
    with off():
        api.index_append(rows, at, place, norm_weight=weight)
        got = api.index_scores(q, w, cache, i32([9, 9]), i32([[0], [0]]), 16)
    assert torch.equal(place, kept) and torch.equal(got[:, :9], want[:, :9])


def test_right_calls_are_made_from_tensors(lib, api):
    """The compiled module makes a right call and leaves a wrong one, or one elsewhere, to the checks."""
    calls = lib.tensor_calls
    rows, cache, slots = randn(4, 192)[:, :128], randn(64, 128), i32([0, 3, 5, 8])
    turn, positions, w = torch.randn(10, 64, device="cuda"), i32([1, 2, 3, 0]), randn(128)
    assert calls.index_append(rows, slots, cache, w, w, 1e-6, turn, positions, True, False, None) is True
    assert calls.index_append(rows, slots, cache, None, None, 1, None, None, 0, 1, torch.cuda.current_stream().cuda_stream) is True
    assert calls.index_append(rows, slots, cache, None, w, 1e-6, None, None, False, False, None) is False  # a bias alone
    assert calls.index_append(rows, slots, cache, w, w, float("nan"), None, None, False, False, None) is False
    assert calls.index_append(rows, slots, cache, w, w, "x", None, None, False, False, None) is False
    assert calls.index_append(rows, slots.long(), cache, w, w, 1e-6, None, None, False, False, None) is False
    assert calls.index_append(rows, slots[:3], cache, w, w, 1e-6, None, None, False, False, None) is False
    assert calls.index_append(rows.half(), slots, cache, w, w, 1e-6, None, None, False, False, None) is False
    assert calls.index_append(rows, slots.cpu(), cache, w, w, 1e-6, None, None, False, False, None) is False
    assert calls.index_append(rows, slots, cache, w, w.float(), 1e-6, None, None, False, False, None) is False
    assert calls.index_append(rows, slots, cache, w, w[::2], 1e-6, None, None, False, False, None) is False
    assert calls.index_append(rows, slots, cache, w, w, 1e-6, turn[:, :32], positions, False, False, None) is False
    parameter = torch.nn.Parameter(w.clone())
    assert calls.index_append(rows, slots, cache, parameter, None, 1e-6, None, None, False, False, None) is False
    with torch.no_grad():
        assert calls.index_append(rows, slots, cache, parameter, None, 1e-6, None, None, False, False, None) is True
    q, hw, lens, table, out = randn(4, 3, 128), torch.randn(4, 3, device="cuda"), i32([30, 16]), i32([[0, 1], [2, 3]]), torch.zeros(4, 32, device="cuda")
    scores = lambda q=q, hw=hw, cache=cache, lens=lens, table=table, page=16, cu=None, most=None, out=out: calls.index_scores(  # noqa: E731
        q, hw, cache, lens, table, page, cu, most, out, None)
    assert scores() is True and scores(cu=i32([0, 1, 4]), most=20, out=torch.zeros(4, 20, device="cuda")) is True
    for bad in (dict(page=0), dict(page=12), dict(page=1 << 70), dict(most=33), dict(most=-1), dict(out=out[:, :31]), dict(out=out.t()),
                dict(cu=i32([0, 1])), dict(hw=hw.half()), dict(q=q[:3], hw=hw[:3], out=out[:3]), dict(lens=lens[:1]),
                dict(table=table.float()), dict(out=None), dict(q=q.float()), dict(cache=cache[:, :64])):
        assert scores(**bad) is False, bad
    x, latent, pages, common = randn(2, 1, 3, 576), randn(64, 576), i32([3]), i32([16])
    to, lse = randn(2, 1, 3, 512), torch.zeros(2, 1, 3, device="cuda")
    room = torch.zeros(lib.topk_attend_shared_workspace_bytes(2, 1, 3), dtype=torch.uint8, device="cuda")
    shared = lambda x=x, latent=latent, lens=lens, table=table, pages=pages, common=common, page=16, scale=0.1, most=None, to=to, lse=lse, room=room: (  # noqa: E731
        calls.attend_shared(x, latent, lens, table, pages, common, page, scale, most, to, lse, room, None))
    assert shared() is True and shared(most=20) is True and shared(pages=pages[:0]) is True
    for bad in (dict(room=room[:-1]), dict(room=None), dict(lse=None), dict(lse=lse.double()), dict(to=to[:, :, :2]), dict(most=33),
                dict(common=i32([1, 2])), dict(common=16), dict(pages=pages.long()), dict(scale=None), dict(page=24),
                dict(x=x[..., :512]), dict(latent=latent.half()), dict(lens=i32([1, 2, 3]))):
        assert shared(**bad) is False, bad
