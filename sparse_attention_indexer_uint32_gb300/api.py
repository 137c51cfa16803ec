"""Tensor-level conveniences over the C ABI (allocation and marshalling only)."""
from __future__ import annotations

import functools
from typing import NamedTuple

import torch

from . import _lib

# The current device's index, without the look at CUDA's state around it, which
# a tensor on a GPU has set up, where this torch has that call.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _there(fn, gpu: int):
    """The function with the tensors' GPU as the current one, on which the library launches."""
    def call(*args):
        with torch.cuda.device(gpu):
            return fn(*args)

    return call


def plan(seq_lens: torch.Tensor, max_seq_len: int, workspace: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """Runs ``topk_plan`` and returns the (possibly newly allocated) workspace."""
    batch = seq_lens.shape[0]
    need = _lib.topk_plan_workspace_bytes(batch)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=seq_lens.device)
    gpu = seq_lens.get_device()
    run = _lib.topk_plan if gpu < 0 or _current_device() == gpu else _there(_lib.topk_plan, gpu)
    run(seq_lens, batch, max_seq_len, workspace, stream)
    return workspace


def topk_transform(scores: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor, page_size: int,
                   k: int, max_seq_len: int | None = None, want_raw: bool = False,
                   workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   raw_out: torch.Tensor | None = None, stream=None):
    """Plans (unless a planned ``workspace`` is given) and runs the transform.

    ``scores``: float32 cuda [batch, row_stride] (row-contiguous); ``seq_lens``:
    int32 cuda [batch]; ``page_table``: int32 cuda [batch, pages].  Without
    ``max_seq_len`` a row has what its scores and its pages both hold: rows of
    scores may be padded past the last page.  Returns ``(out, raw_or_None,
    workspace)``.
    """
    batch, row_stride = scores.shape
    if max_seq_len is None:
        max_seq_len = min(row_stride, page_table.shape[1] * page_size)
    if scores.stride(1) != 1 or page_table.stride(1) != 1:
        raise ValueError("scores and page_table rows must be contiguous")
    if workspace is None:
        workspace = plan(seq_lens, max_seq_len, stream=stream)
    if out is None:
        out = torch.empty((batch, k), dtype=torch.int32, device=scores.device)
    if want_raw and raw_out is None:
        raw_out = torch.empty((batch, k), dtype=torch.int32, device=scores.device)
    gpu = scores.get_device()
    run = _lib.topk_transform if gpu < 0 or _current_device() == gpu else _there(_lib.topk_transform, gpu)
    run(scores, scores.stride(0), seq_lens, batch, max_seq_len, page_table, page_table.stride(0), page_size, k, out,
        raw_out if want_raw else None, workspace, stream)
    return out, (raw_out if want_raw else None), workspace


_DTYPES = {torch.bfloat16: _lib.TOPK_BF16, torch.float16: _lib.TOPK_FP16}
_LATENT, _ROPE, _NOPE, _VALUE = _lib.TOPK_LATENT_DIM, _lib.TOPK_ROPE_DIM, _lib.TOPK_NOPE_DIM, _lib.TOPK_VALUE_DIM
_WIDTH = _LATENT + _ROPE
_INDEX = _lib.TOPK_INDEX_DIM
_INDEX_ROW, _VALUES_ROW = (_INDEX,), (_LATENT,)
_I32, _F32 = torch.int32, torch.float32
_c = _lib.library()
_calls = _lib.tensor_calls


# The calls below look their arguments over twice at most: one condition that
# is true of every right call (a few microseconds), and, where it is not, the
# checks that say which argument is wrong.  None of them has a backward pass:
# where gradients are being recorded, tensors that require one are refused.  The
# attention calls do not wait for their kernels: topk_read_attend_flags of the
# binding says afterwards whether a bounded wait of one gave up, which makes
# that call's output void.  The index calls and attention behind a shared prompt
# are tried by a compiled module first, which returns whether it made the call:
# what it does not take (results to allocate, another GPU than the current one,
# arguments that are wrong) goes on here.


def _same(dtype: torch.dtype, device: torch.device, **tensors) -> None:
    """Raises unless the tensors (None is skipped) are of this type, on this GPU, with contiguous rows."""
    for name, t in tensors.items():
        if t is None:
            continue
        if t.dtype != dtype or t.device != device:
            raise ValueError(f"{name} must be {dtype} on {device}: got {t.dtype} on {t.device}")
        if t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} rows must be contiguous")


def _whole(shape: tuple, **tensors) -> None:
    """Raises unless the tensors (None is skipped) are contiguous and of this shape."""
    for name, t in tensors.items():
        if t is not None and (tuple(t.shape) != tuple(shape) or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous of shape {tuple(shape)}: got {tuple(t.shape)}")


def _no_grad(**tensors) -> None:
    """Raises where a gradient would be lost: the calls have no backward pass, and their results are detached."""
    if torch.is_grad_enabled():
        for name, t in tensors.items():
            if t is not None and t.requires_grad:
                raise ValueError(f"{name} requires a gradient and the call has no backward pass: detach it, or call under "
                                 "torch.no_grad()")


def _on_gpu(t: torch.Tensor) -> None:
    if not t.is_cuda:
        raise ValueError(f"the tensors must be on a GPU: got {t.device}")


def _dtype(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float16: got {t.dtype}")
    return code


def _empty(shape: tuple, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """New memory for a call on ``stream``: out of that stream's own pool, so that nothing else uses it meanwhile."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _lib.stream_handle(stream, device.index)
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _is(t: torch.Tensor, dtype: torch.dtype, gpu: int, shape: tuple) -> bool:
    return t.dtype is dtype and t.get_device() == gpu and t.shape == shape and t.is_contiguous()


_grad_enabled = torch.is_grad_enabled


def _any_grad(a: torch.Tensor, b: torch.Tensor, c: torch.Tensor | None, d: torch.Tensor | None) -> bool:
    return (a.requires_grad or b.requires_grad or (c is not None and c.requires_grad)
            or (d is not None and d.requires_grad))


def _line(t: torch.Tensor, n: int, gpu: int) -> bool:
    """n int32 values in a row."""
    return t.dtype is _I32 and t.numel() == n and t.get_device() == gpu and t.is_contiguous()


class BlockTables(NamedTuple):
    """Outputs of :func:`block_tables` (int32 cuda); ``status`` holds the pages taken and the flag bits."""

    seq_lens: torch.Tensor  # [batch]
    cu_new: torch.Tensor  # [batch + 1]
    slots: torch.Tensor  # [max_tokens], -1 past the last new token
    positions: torch.Tensor  # [max_tokens]
    rows: torch.Tensor  # [max_tokens]
    status: torch.Tensor  # [2]


def _check_tables(context_lens, new_lens, free_pages, page_table, max_tokens, out):
    dev = context_lens.device
    _same(_I32, dev, context_lens=context_lens, new_lens=new_lens, free_pages=free_pages, page_table=page_table)
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be [batch, pages]: got {tuple(page_table.shape)}")
    batch = page_table.shape[0]
    _whole((batch,), context_lens=context_lens, new_lens=new_lens)
    _whole((free_pages.numel(),), free_pages=free_pages)
    if out is not None:
        _same(_I32, dev, **out._asdict())
        _whole((batch,), seq_lens=out.seq_lens)
        _whole((batch + 1,), cu_new=out.cu_new)
        _whole((max_tokens,), slots=out.slots, positions=out.positions, rows=out.rows)
        _whole((2,), status=out.status)
    _on_gpu(context_lens)


def _check_overlap(context_lens, new_lens, free_pages, page_table, out):
    """Names the pair where an output, or the table, lies over an input (the C call refuses it)."""
    def span(t):
        last = sum((n - 1) * s for n, s in zip(t.shape, t.stride())) if t.numel() else -1
        return t.data_ptr(), t.data_ptr() + 4 * (last + 1)

    inputs = dict(context_lens=context_lens, new_lens=new_lens, free_pages=free_pages)
    table = dict(page_table=page_table)
    for name, t in {**{f"out.{n}": x for n, x in out._asdict().items()}, **table}.items():
        a, b = span(t)
        for other, x in {**inputs, **({} if t is page_table else table)}.items():
            c, d = span(x)
            if a < d and c < b:
                raise ValueError(f"{name} must not lie over {other} (the result of one call and the lengths of the next: "
                                 "take two results in turn)")


def block_tables(context_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
                 page_table: torch.Tensor, page_size: int, max_tokens: int, out: BlockTables | None = None,
                 stream=None) -> BlockTables:
    """Runs ``topk_block_tables``: writes the new pages into ``page_table`` ([batch, pages], in place) and returns
    the step's lengths, offsets and slot map (in ``out``, where the result of an earlier call is given).  ``out`` must
    not hold this call's inputs: where ``seq_lens`` becomes the next step's ``context_lens``, two results are taken
    in turn."""
    gpu, shape = context_lens.get_device(), page_table.shape
    batch, num_free = shape[0] if shape else 0, free_pages.numel()
    if not (gpu >= 0 and len(shape) == 2 and page_table.dtype is _I32 and page_table.get_device() == gpu
            and (shape[1] <= 1 or page_table.stride(1) == 1) and _line(context_lens, batch, gpu)
            and _line(new_lens, batch, gpu) and _line(free_pages, num_free, gpu)
            and (out is None or (_line(out[0], batch, gpu) and _line(out[1], batch + 1, gpu)
                                 and _line(out[2], max_tokens, gpu) and _line(out[3], max_tokens, gpu)
                                 and _line(out[4], max_tokens, gpu) and _line(out[5], 2, gpu)))):
        _check_tables(context_lens, new_lens, free_pages, page_table, max_tokens, out)
    pages = shape[1]
    if out is None:
        # One allocation; the token arrays start on 16 bytes, where the kernel writes four values at once.
        room = (max_tokens + 3) // 4 * 4
        buf = _empty((3 * room + 2 * batch + 3,), _I32, context_lens.device, stream)
        at = 3 * room
        out = BlockTables(buf[at:at + batch], buf[at + batch:at + 2 * batch + 1], buf[:max_tokens],
                          buf[room:room + max_tokens], buf[2 * room:2 * room + max_tokens], buf[at + 2 * batch + 1:])
    status = (_c.topk_block_tables if _current_device() == gpu else _there(_c.topk_block_tables, gpu))(
        context_lens.data_ptr(), new_lens.data_ptr(), batch, page_size, free_pages.data_ptr(), num_free,
        page_table.data_ptr(), page_table.stride(0) if batch > 1 else pages, pages, max_tokens, out[0].data_ptr(),
        out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(), out[4].data_ptr(), out[5].data_ptr(),
        _lib.stream_handle(stream, gpu))
    if status:
        if status == _lib.TOPK_EINVAL:
            _check_overlap(context_lens, new_lens, free_pages, page_table, out)
        _lib.check("topk_block_tables", status)
    return out


def _check_angles(cos_sin):
    # (an empty table has no address: the library would take it for none)
    if cos_sin is not None and (cos_sin.dim() != 2 or cos_sin.shape[0] < 1 or cos_sin.shape[1] != _ROPE
                                or not cos_sin.is_contiguous()):
        raise ValueError(f"cos_sin must be contiguous [1 position or more, {_ROPE}]: got {tuple(cos_sin.shape)}")


def _check_append(rows, slots, cache, norm_weight, cos_sin, positions):
    dev = cache.device
    _dtype(cache, "cache")
    _same(cache.dtype, dev, rows=rows, cache=cache, norm_weight=norm_weight)
    _same(_I32, dev, slots=slots, positions=positions)
    _same(_F32, dev, cos_sin=cos_sin)
    if rows.dim() != 2 or cache.dim() != 2 or rows.shape[1] != _WIDTH or cache.shape[1] != _WIDTH:
        raise ValueError(f"rows and cache must be [.., {_WIDTH}]: got {tuple(rows.shape)} and {tuple(cache.shape)}")
    _whole((rows.shape[0],), slots=slots, positions=positions)
    _whole((_LATENT,), norm_weight=norm_weight)
    _check_angles(cos_sin)
    _no_grad(rows=rows, cache=cache, norm_weight=norm_weight, cos_sin=cos_sin)
    _on_gpu(cache)


def cache_append(rows: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor,
                 norm_weight: torch.Tensor | None = None, eps: float = 1e-6, cos_sin: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, interleaved: bool = False, stream=None) -> None:
    """Runs ``topk_cache_append``: ``rows`` [tokens, 576] (512 latent values, 64 rotary ones) to ``slots`` of
    ``cache`` [num_slots, 576], normed by ``norm_weight`` [512] and rotated by ``cos_sin`` (float32
    [num_positions, 64]: cosines, sines) at ``positions``, where these are given."""
    gpu, dtype, shape, places = cache.get_device(), cache.dtype, rows.shape, cache.shape
    code, tokens = _DTYPES.get(dtype), shape[0] if shape else 0
    positions_n = cos_sin.shape[0] if cos_sin is not None and cos_sin.dim() else 0
    if not (gpu >= 0 and code is not None and rows.dtype is dtype and rows.get_device() == gpu and len(shape) == 2
            and len(places) == 2 and shape[1] == _WIDTH == places[1] and rows.stride(1) == 1 == cache.stride(1)
            and _line(slots, tokens, gpu) and (positions is None or _line(positions, tokens, gpu))
            and (norm_weight is None or _is(norm_weight, dtype, gpu, (_LATENT,)))
            and (cos_sin is None or (positions_n > 0 and _is(cos_sin, _F32, gpu, (positions_n, _ROPE))))
            and not (_grad_enabled() and _any_grad(rows, cache, norm_weight, cos_sin))):
        _check_append(rows, slots, cache, norm_weight, cos_sin, positions)
    status = (_c.topk_cache_append if _current_device() == gpu else _there(_c.topk_cache_append, gpu))(
        rows.data_ptr(), rows.stride(0) if tokens > 1 else _WIDTH, tokens,
        None if norm_weight is None else norm_weight.data_ptr(), eps, None if cos_sin is None else cos_sin.data_ptr(),
        positions_n, None if positions is None else positions.data_ptr(), interleaved,
        slots.data_ptr(), cache.data_ptr(), cache.stride(0) if places[0] > 1 else _WIDTH, places[0], code,
        _lib.stream_handle(stream, gpu))
    if status:
        _lib.check("topk_cache_append", status)


def _check_index_append(rows, slots, cache, norm_weight, norm_bias, cos_sin, positions):
    dev = cache.device
    _dtype(cache, "cache")
    _same(cache.dtype, dev, rows=rows, cache=cache, norm_weight=norm_weight, norm_bias=norm_bias)
    _same(_I32, dev, slots=slots, positions=positions)
    _same(_F32, dev, cos_sin=cos_sin)
    if rows.dim() != 2 or cache.dim() != 2 or rows.shape[1] != _INDEX or cache.shape[1] != _INDEX:
        raise ValueError(f"rows and cache must be [.., {_INDEX}]: got {tuple(rows.shape)} and {tuple(cache.shape)}")
    _whole((rows.shape[0],), slots=slots, positions=positions)
    _whole((_INDEX,), norm_weight=norm_weight, norm_bias=norm_bias)
    _check_angles(cos_sin)
    _no_grad(rows=rows, cache=cache, norm_weight=norm_weight, norm_bias=norm_bias, cos_sin=cos_sin)
    _on_gpu(cache)


def index_append(rows: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor,
                 norm_weight: torch.Tensor | None = None, norm_bias: torch.Tensor | None = None, eps: float = 1e-6,
                 cos_sin: torch.Tensor | None = None, positions: torch.Tensor | None = None, interleaved: bool = False,
                 rope_last: bool = False, stream=None) -> None:
    """Runs ``topk_index_append``: the indexer's keys ``rows`` [tokens, 128] to ``slots`` of their ``cache``
    [num_slots, 128], layer-normed by ``norm_weight`` and ``norm_bias`` [128] and, in their first 64 values (the last
    with ``rope_last``), rotated by ``cos_sin`` (as in :func:`cache_append`) at ``positions``, where these are given."""
    if _calls.index_append(rows, slots, cache, norm_weight, norm_bias, eps, cos_sin, positions, interleaved, rope_last,
                           None if stream is None else _lib.stream_handle(stream, 0)):
        return
    gpu, dtype, shape, places, steps, slot_steps = (cache.get_device(), cache.dtype, rows.shape, cache.shape, rows.stride(),
                                                    cache.stride())
    code, tokens, positions_n = _DTYPES.get(dtype), shape[0] if shape else 0, 0
    line = (tokens,)
    right = (gpu >= 0 and code is not None and rows.dtype is dtype and rows.get_device() == gpu and len(shape) == 2
             and len(places) == 2 and shape[1] == _INDEX == places[1] and steps[1] == 1 == slot_steps[1]
             and slots.dtype is _I32 and slots.shape == line and slots.get_device() == gpu and slots.is_contiguous())
    if positions is not None:
        right = (right and positions.dtype is _I32 and positions.shape == line and positions.get_device() == gpu
                 and positions.is_contiguous())
        positions_at = positions.data_ptr()
    else:
        positions_at = None
    weight_at = bias_at = turns_at = None
    if norm_weight is not None:
        right = (right and norm_weight.dtype is dtype and norm_weight.shape == _INDEX_ROW and norm_weight.get_device() == gpu
                 and norm_weight.is_contiguous())
        weight_at = norm_weight.data_ptr()
    if norm_bias is not None:
        right = (right and norm_bias.dtype is dtype and norm_bias.shape == _INDEX_ROW and norm_bias.get_device() == gpu
                 and norm_bias.is_contiguous())
        bias_at = norm_bias.data_ptr()
    if cos_sin is not None:
        turns = cos_sin.shape
        positions_n = turns[0] if turns else 0
        right = (right and cos_sin.dtype is _F32 and len(turns) == 2 and positions_n > 0 and turns[1] == _ROPE
                 and cos_sin.get_device() == gpu and cos_sin.is_contiguous())
        turns_at = cos_sin.data_ptr()
    if not right or (_grad_enabled() and (_any_grad(rows, cache, norm_weight, norm_bias)
                                          or (cos_sin is not None and cos_sin.requires_grad))):
        _check_index_append(rows, slots, cache, norm_weight, norm_bias, cos_sin, positions)
    status = (_c.topk_index_append if _current_device() == gpu else _there(_c.topk_index_append, gpu))(
        rows.data_ptr(), steps[0] if tokens > 1 else _INDEX, tokens, weight_at, bias_at, eps, turns_at, positions_n,
        positions_at, interleaved, rope_last, slots.data_ptr(), cache.data_ptr(), slot_steps[0] if places[0] > 1 else _INDEX,
        places[0], code, _lib.stream_handle(stream, gpu))
    if status:
        _lib.check("topk_index_append", status)


def _check_index_scores(q, weights, cache, seq_lens, page_table, page_size, cu_q, max_seq_len, out):
    dev = q.device
    _dtype(q, "q")
    if q.dim() != 3 or page_table.dim() != 2:
        raise ValueError(f"q and page_table must be [tokens, heads, ..] and [batch, pages]: got {tuple(q.shape)} and "
                         f"{tuple(page_table.shape)}")
    (total, heads, width), batch = q.shape, page_table.shape[0]
    _same(q.dtype, dev, q=q, cache=cache)
    if width != _INDEX or cache.dim() != 2 or cache.shape[1] != _INDEX:
        raise ValueError(f"q and cache must be [.., {_INDEX}]: got {tuple(q.shape)} and {tuple(cache.shape)}")
    _same(_F32, dev, weights=weights, out=out)
    if tuple(weights.shape) != (total, heads):
        raise ValueError(f"weights must be {(total, heads)}: got {tuple(weights.shape)}")
    _same(_I32, dev, seq_lens=seq_lens, page_table=page_table, cu_q=cu_q)
    _whole((batch,), seq_lens=seq_lens)
    _whole((batch + 1,), cu_q=cu_q)
    if cu_q is None and (batch == 0 or total % batch):
        raise ValueError(f"without cu_q the {total} queries must be as many for each of the {batch} requests")
    if max_seq_len is not None and max_seq_len > page_table.shape[1] * page_size:
        raise ValueError(f"max_seq_len {max_seq_len} is over {page_table.shape[1]} pages of {page_size}")
    if out is not None:
        most = page_table.shape[1] * page_size if max_seq_len is None else max_seq_len
        if out.dim() != 2 or out.shape[0] != total or out.shape[1] < most:
            raise ValueError(f"out must be [{total}, {most} or more]: got {tuple(out.shape)}")
    _no_grad(q=q, weights=weights, cache=cache, out=out)
    _on_gpu(q)


def index_scores(q: torch.Tensor, weights: torch.Tensor, cache: torch.Tensor, seq_lens: torch.Tensor,
                 page_table: torch.Tensor, page_size: int, cu_q: torch.Tensor | None = None,
                 max_seq_len: int | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Runs ``topk_index_scores``: the scores that :func:`topk_transform` selects from, of the index queries ``q``
    [tokens, heads, 128] with ``weights`` [tokens, heads] (float32) over the keys ``cache`` [num_slots, 128] of their
    requests, through ``page_table`` [batch, pages].  ``cu_q`` [batch + 1]: the requests' queries, their newest
    tokens (None: as many for each).  Returns ``out`` [tokens, max_seq_len or more] (float32; new memory has
    max_seq_len rounded up to a multiple of 4), of which each query's row is written up to what it sees: the last
    query of a request ``seq_lens`` positions, each one before it one less.  Where lengths may be above a
    ``max_seq_len`` given here, the selection is given it too."""
    if out is not None and _calls.index_scores(q, weights, cache, seq_lens, page_table, page_size, cu_q, max_seq_len, out,
                                               None if stream is None else _lib.stream_handle(stream, 0)):
        return out
    gpu, dtype, shape, listed, places, steps = q.get_device(), q.dtype, q.shape, page_table.shape, cache.shape, q.stride()
    w_steps, slot_steps, table_steps = weights.stride(), cache.stride(), page_table.stride()
    code = _DTYPES.get(dtype)
    right = (gpu >= 0 and code is not None and len(shape) == 3 and len(listed) == 2 and shape[2] == _INDEX
             and steps[2] == 1 and cache.dtype is dtype and cache.get_device() == gpu and len(places) == 2
             and places[1] == _INDEX and slot_steps[1] == 1 and weights.dtype is _F32 and weights.get_device() == gpu
             and weights.shape == shape[:2] and (w_steps[1] == 1 or shape[1] <= 1)
             and page_table.dtype is _I32 and page_table.get_device() == gpu
             and (table_steps[1] == 1 or listed[1] <= 1) and seq_lens.dtype is _I32 and seq_lens.get_device() == gpu
             and seq_lens.shape == listed[:1] and seq_lens.is_contiguous()
             and (_line(cu_q, listed[0] + 1, gpu) if cu_q is not None else listed[0] > 0 and shape[0] % listed[0] == 0))
    if right:
        most = listed[1] * page_size
        if max_seq_len is None:
            most = min(most, 2 ** 31 - 1)
        else:
            right, most = max_seq_len <= most, max_seq_len
    if right and out is not None:
        sides, out_steps = out.shape, out.stride()
        right = (out.dtype is _F32 and out.get_device() == gpu and len(sides) == 2 and sides[0] == shape[0]
                 and sides[1] >= most and (out_steps[1] == 1 or sides[1] <= 1))
    if not right or (_grad_enabled() and _any_grad(q, weights, cache, out)):
        _check_index_scores(q, weights, cache, seq_lens, page_table, page_size, cu_q, max_seq_len, out)
    total, heads, _ = shape
    batch, slots = listed[0], places[0]
    if out is None:
        out = _empty((total, max(most + 3, 0) // 4 * 4), _F32, q.device, stream)  # (what is below 0 the library refuses)
        out_steps = out.stride()
    many = total > 1
    status = (_c.topk_index_scores if _current_device() == gpu else _there(_c.topk_index_scores, gpu))(
        q.data_ptr(), steps[0] if many else _INDEX, steps[1] if heads > 1 else _INDEX, weights.data_ptr(),
        w_steps[0] if many else heads, cache.data_ptr(), slot_steps[0] if slots > 1 else _INDEX, slots,
        seq_lens.data_ptr(), page_table.data_ptr(), table_steps[0] if batch > 1 else listed[1], page_size, most,
        None if cu_q is None else cu_q.data_ptr(), batch, total, heads, code, out.data_ptr(),
        out_steps[0] if many else most, _lib.stream_handle(stream, gpu))
    if status:
        _lib.check("topk_index_scores", status)
    return out


def _check_attend(q, cache, out, lse):
    """What the cache attentions share."""
    _dtype(q, "q")
    _same(q.dtype, q.device, q=q, cache=cache, out=out)
    if q.shape[-1] != _WIDTH or cache.dim() != 2 or cache.shape[1] != _WIDTH:
        raise ValueError(f"q and cache must be [.., {_WIDTH}]: got {tuple(q.shape)} and {tuple(cache.shape)}")
    _whole((*q.shape[:-1], _LATENT), out=out)
    _same(_F32, q.device, lse=lse)
    _whole(q.shape[:-1], lse=lse)
    _no_grad(q=q, cache=cache, out=out, lse=lse)
    _on_gpu(q)


def _fits(q, cache, places, out, lse, gpu, dtype, lead) -> bool:
    """Whether they are what the cache attentions take; ``lead``: q's dimensions but the last."""
    return (gpu >= 0 and not (_grad_enabled() and _any_grad(q, cache, out, lse)) and cache.dtype is dtype and cache.get_device() == gpu and len(places) == 2
            and places[1] == _WIDTH and cache.stride(1) == 1
            and (out is None or _is(out, dtype, gpu, lead + (_LATENT,)))
            and (lse is None or _is(lse, _F32, gpu, lead)))


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(batch: int, queries: int, heads: int) -> int:
    return _lib.topk_attend_workspace_bytes(batch, queries, heads)


def _attend_workspace(workspace, batch, queries, heads, device, stream):
    """The workspace and its bytes."""
    return _room(workspace, _workspace_bytes(batch, queries, heads), device, stream)


def _room(workspace, need, device, stream):
    """The workspace, a new one where it is too small, and its bytes."""
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on {device}: got {workspace.device}")
        room = workspace.numel() * workspace.element_size()
        if room >= need:
            return workspace, room
    return _empty((need,), torch.uint8, device, stream), need


def attend_selected(q: torch.Tensor, cache: torch.Tensor, indices: torch.Tensor, scale: float,
                    seq_lens: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Runs ``topk_attend_selected``: ``q`` [rows, heads, 576] over the slots ``indices`` [rows, k] (int32, as
    :func:`topk_transform` writes them) of ``cache`` [num_slots, 576].  ``seq_lens`` [rows], where given, bounds
    the slots looked at.  Returns ``(out [rows, heads, 512], lse [rows, heads], workspace)``; the workspace serves
    later calls on the same stream."""
    gpu, dtype, shape, listed, places, steps = q.get_device(), q.dtype, q.shape, indices.shape, cache.shape, q.stride()
    code = _DTYPES.get(dtype)
    if not (code is not None and len(shape) == 3 and len(listed) == 2 and listed[0] == shape[0]
            and shape[2] == _WIDTH and steps[2] == 1 and indices.dtype is _I32 and indices.get_device() == gpu
            and (listed[1] <= 1 or indices.stride(1) == 1)
            and (seq_lens is None or _line(seq_lens, shape[0], gpu))
            and _fits(q, cache, places, out, lse, gpu, dtype, (shape[0], shape[1]))):
        if q.dim() != 3 or indices.dim() != 2 or indices.shape[0] != q.shape[0]:
            raise ValueError(f"q and indices must be [rows, heads, ..] and [rows, k]: got {tuple(q.shape)} and "
                             f"{tuple(indices.shape)}")
        _dtype(q, "q")
        _same(_I32, q.device, indices=indices, seq_lens=seq_lens)
        _whole(shape[:1], seq_lens=seq_lens)
        _check_attend(q, cache, out, lse)
    rows, heads, _ = shape
    if out is None:
        out = _empty((rows, heads, _LATENT), dtype, q.device, stream)
    if lse is None:
        lse = _empty((rows, heads), _F32, q.device, stream)
    workspace, room = _attend_workspace(workspace, rows, 1, heads, q.device, stream)
    slots = places[0]
    status = (_c.topk_attend_selected if _current_device() == gpu else _there(_c.topk_attend_selected, gpu))(
        q.data_ptr(), steps[0] if rows > 1 else _WIDTH, steps[1] if heads > 1 else _WIDTH, cache.data_ptr(),
        cache.stride(0) if slots > 1 else _WIDTH, slots, indices.data_ptr(),
        indices.stride(0) if rows > 1 else listed[1], None if seq_lens is None else seq_lens.data_ptr(), rows, heads,
        listed[1], scale, code, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), room,
        _lib.stream_handle(stream, gpu))
    if status:
        _lib.check("topk_attend_selected", status)
    return out, lse, workspace


def attend_paged(q: torch.Tensor, cache: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor,
                 page_size: int, scale: float, max_seq_len: int | None = None, out: torch.Tensor | None = None,
                 lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Runs ``topk_attend_paged``: ``q`` [batch, queries, heads, 576], the newest tokens' queries, over each
    request's positions through ``page_table`` [batch, pages].  Returns ``(out [batch, queries, heads, 512],
    lse [batch, queries, heads], workspace)``."""
    gpu, dtype, shape, listed, places, steps = q.get_device(), q.dtype, q.shape, page_table.shape, cache.shape, q.stride()
    code = _DTYPES.get(dtype)
    if not (code is not None and len(shape) == 4 and len(listed) == 2 and listed[0] == shape[0]
            and shape[3] == _WIDTH and steps[3] == 1 and page_table.dtype is _I32 and page_table.get_device() == gpu
            and (listed[1] <= 1 or page_table.stride(1) == 1) and _line(seq_lens, shape[0], gpu)
            and _fits(q, cache, places, out, lse, gpu, dtype, (shape[0], shape[1], shape[2]))):
        if q.dim() != 4 or page_table.dim() != 2 or page_table.shape[0] != q.shape[0]:
            raise ValueError(f"q and page_table must be [batch, queries, heads, ..] and [batch, pages]: got "
                             f"{tuple(q.shape)} and {tuple(page_table.shape)}")
        _dtype(q, "q")
        _same(_I32, q.device, seq_lens=seq_lens, page_table=page_table)
        _whole(shape[:1], seq_lens=seq_lens)
        if max_seq_len is not None and max_seq_len > listed[1] * page_size:
            raise ValueError(f"max_seq_len {max_seq_len} is over {listed[1]} pages of {page_size}")
        _check_attend(q, cache, out, lse)
    batch, queries, heads, _ = shape
    if max_seq_len is None:
        max_seq_len = min(listed[1] * page_size, 2 ** 31 - 1)
    elif max_seq_len > listed[1] * page_size:
        raise ValueError(f"max_seq_len {max_seq_len} is over {listed[1]} pages of {page_size}")
    if out is None:
        out = _empty((batch, queries, heads, _LATENT), dtype, q.device, stream)
    if lse is None:
        lse = _empty((batch, queries, heads), _F32, q.device, stream)
    workspace, room = _attend_workspace(workspace, batch, queries, heads, q.device, stream)
    slots = places[0]
    status = (_c.topk_attend_paged if _current_device() == gpu else _there(_c.topk_attend_paged, gpu))(
        q.data_ptr(), steps[0] if batch > 1 else _WIDTH, steps[1] if queries > 1 else _WIDTH,
        steps[2] if heads > 1 else _WIDTH, cache.data_ptr(), cache.stride(0) if slots > 1 else _WIDTH, slots,
        seq_lens.data_ptr(), page_table.data_ptr(), page_table.stride(0) if batch > 1 else listed[1], page_size,
        max_seq_len, batch, queries, heads, scale, code, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), room,
        _lib.stream_handle(stream, gpu))
    if status:
        _lib.check("topk_attend_paged", status)
    return out, lse, workspace


@functools.lru_cache(maxsize=1024)
def _shared_workspace_bytes(batch: int, queries: int, heads: int) -> int:
    return _lib.topk_attend_shared_workspace_bytes(batch, queries, heads)


def attend_shared(q: torch.Tensor, cache: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor,
                  shared_pages: torch.Tensor, shared_len: torch.Tensor, page_size: int, scale: float,
                  max_seq_len: int | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None):
    """Runs ``topk_attend_shared``: :func:`attend_paged` for requests whose first ``shared_len`` [1] positions are the
    same, which are read once for all through ``shared_pages`` [pages]; those after them through each request's row of
    ``page_table``.  ``seq_lens`` counts both.  Returns ``(out [batch, queries, heads, 512], lse [batch, queries,
    heads], workspace)``."""
    if workspace is not None and out is not None and _calls.attend_shared(
            q, cache, seq_lens, page_table, shared_pages, shared_len, page_size, scale, max_seq_len, out, lse, workspace,
            None if stream is None else _lib.stream_handle(stream, 0)):
        return out, lse, workspace
    gpu, dtype, shape, listed, places, steps = q.get_device(), q.dtype, q.shape, page_table.shape, cache.shape, q.stride()
    code, common, slot_steps, table_steps = _DTYPES.get(dtype), shared_pages.numel(), cache.stride(), page_table.stride()
    right = (gpu >= 0 and code is not None and len(shape) == 4 and len(listed) == 2 and listed[0] == shape[0]
             and shape[3] == _WIDTH and steps[3] == 1 and cache.dtype is dtype and cache.get_device() == gpu
             and len(places) == 2 and places[1] == _WIDTH and slot_steps[1] == 1 and page_table.dtype is _I32
             and page_table.get_device() == gpu and (table_steps[1] == 1 or listed[1] <= 1)
             and seq_lens.dtype is _I32 and seq_lens.get_device() == gpu and seq_lens.shape == listed[:1]
             and seq_lens.is_contiguous() and _line(shared_pages, common, gpu) and _line(shared_len, 1, gpu))
    if right and out is not None:
        right = out.dtype is dtype and out.get_device() == gpu and out.shape == shape[:3] + _VALUES_ROW and out.is_contiguous()
    if right and lse is not None:
        right = lse.dtype is _F32 and lse.get_device() == gpu and lse.shape == shape[:3] and lse.is_contiguous()
    if not right or (_grad_enabled() and _any_grad(q, cache, out, lse)):
        if q.dim() != 4 or page_table.dim() != 2 or page_table.shape[0] != q.shape[0]:
            raise ValueError(f"q and page_table must be [batch, queries, heads, ..] and [batch, pages]: got "
                             f"{tuple(q.shape)} and {tuple(page_table.shape)}")
        _dtype(q, "q")
        _same(_I32, q.device, seq_lens=seq_lens, page_table=page_table, shared_pages=shared_pages, shared_len=shared_len)
        _whole(shape[:1], seq_lens=seq_lens)
        _whole((common,), shared_pages=shared_pages)
        _whole((1,), shared_len=shared_len.reshape(-1))
        if max_seq_len is not None and max_seq_len > listed[1] * page_size:
            raise ValueError(f"max_seq_len {max_seq_len} is over {listed[1]} pages of {page_size}")
        _check_attend(q, cache, out, lse)
    batch, queries, heads, _ = shape
    if max_seq_len is None:
        max_seq_len = min(listed[1] * page_size, 2 ** 31 - 1)
    elif max_seq_len > listed[1] * page_size:
        raise ValueError(f"max_seq_len {max_seq_len} is over {listed[1]} pages of {page_size}")
    if out is None:
        out = _empty((batch, queries, heads, _LATENT), dtype, q.device, stream)
    if lse is None:
        lse = _empty((batch, queries, heads), _F32, q.device, stream)
    workspace, room = _room(workspace, _shared_workspace_bytes(batch, queries, heads), q.device, stream)
    slots = places[0]
    status = (_c.topk_attend_shared if _current_device() == gpu else _there(_c.topk_attend_shared, gpu))(
        q.data_ptr(), steps[0] if batch > 1 else _WIDTH, steps[1] if queries > 1 else _WIDTH,
        steps[2] if heads > 1 else _WIDTH, cache.data_ptr(), slot_steps[0] if slots > 1 else _WIDTH, slots,
        seq_lens.data_ptr(), page_table.data_ptr(), table_steps[0] if batch > 1 else listed[1],
        shared_pages.data_ptr(), common, shared_len.data_ptr(), page_size, max_seq_len, batch, queries, heads, scale, code,
        out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), room, _lib.stream_handle(stream, gpu))
    if status:
        _lib.check("topk_attend_shared", status)
    return out, lse, workspace


def _check_prompt(q, k_nope, k_rope, v, cu_q, cu_k, out, lse):
    dev = q.device
    _dtype(q, "q")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError(f"q and v must be [tokens, heads, ..]: got {tuple(q.shape)} and {tuple(v.shape)}")
    (total_q, heads, _), total_k = q.shape, v.shape[0]
    for name, t, shape in (("q", q, (total_q, heads, _NOPE + _ROPE)), ("k_nope", k_nope, (total_k, heads, _NOPE)),
                           ("k_rope", k_rope, (total_k, _ROPE)), ("v", v, (total_k, heads, _VALUE))):
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {shape}: got {tuple(t.shape)}")
    _whole(cu_q.shape[:1], cu_q=cu_q, cu_k=cu_k)
    _whole((total_q, heads, _VALUE), out=out)
    _whole((total_q, heads), lse=lse)
    _same(q.dtype, dev, q=q, k_nope=k_nope, k_rope=k_rope, v=v, out=out)
    _same(_I32, dev, cu_q=cu_q, cu_k=cu_k)
    _same(_F32, dev, lse=lse)
    _no_grad(q=q, k_nope=k_nope, k_rope=k_rope, v=v, out=out, lse=lse)
    _on_gpu(q)


def attend_prompt(q: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                  cu_k: torch.Tensor, scale: float, causal: bool = True, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, stream=None):
    """Runs ``topk_attend_prompt``: ``q`` [total_q, heads, 192], ``k_nope`` [total_k, heads, 128], ``k_rope``
    [total_k, 64], ``v`` [total_k, heads, 128], requests by the offsets ``cu_q`` and ``cu_k`` [batch + 1].
    Returns ``(out [total_q, heads, 128], lse [total_q, heads])``."""
    gpu, dtype, shape, marks = q.get_device(), q.dtype, q.shape, cu_q.shape
    code, tokens = _DTYPES.get(dtype), k_rope.shape[0] if k_rope.dim() else 0
    q_step, k_step, r_step, v_step = q.stride(), k_nope.stride(), k_rope.stride(), v.stride()
    if not (gpu >= 0 and code is not None and len(shape) == 3 and shape[2] == _NOPE + _ROPE
            and k_nope.dtype is dtype and k_nope.get_device() == gpu and k_nope.shape == (tokens, shape[1], _NOPE)
            and v.dtype is dtype and v.get_device() == gpu and v.shape == (tokens, shape[1], _VALUE)
            and k_rope.dtype is dtype and k_rope.get_device() == gpu and k_rope.shape == (tokens, _ROPE)
            and q_step[2] == k_step[2] == r_step[1] == v_step[2] == 1
            and len(marks) == 1 and _line(cu_q, marks[0], gpu) and _line(cu_k, marks[0], gpu)
            and (out is None or _is(out, dtype, gpu, (shape[0], shape[1], _VALUE)))
            and (lse is None or _is(lse, _F32, gpu, (shape[0], shape[1])))
            and not (_grad_enabled() and (_any_grad(q, k_nope, out, lse) or k_rope.requires_grad or v.requires_grad))):
        _check_prompt(q, k_nope, k_rope, v, cu_q, cu_k, out, lse)
    total_q, heads, _ = shape
    if out is None:
        out = _empty((total_q, heads, _VALUE), dtype, q.device, stream)
    if lse is None:
        lse = _empty((total_q, heads), _F32, q.device, stream)
    # The stride of a dimension of one entry means nothing.
    many_q, many_k, many_heads = total_q > 1, tokens > 1, heads > 1
    status = (_c.topk_attend_prompt if _current_device() == gpu else _there(_c.topk_attend_prompt, gpu))(
        q.data_ptr(), q_step[0] if many_q else _NOPE + _ROPE, q_step[1] if many_heads else _NOPE + _ROPE,
        k_nope.data_ptr(), k_step[0] if many_k else _NOPE, k_step[1] if many_heads else _NOPE, k_rope.data_ptr(),
        r_step[0] if many_k else _ROPE, v.data_ptr(), v_step[0] if many_k else _VALUE,
        v_step[1] if many_heads else _VALUE, cu_q.data_ptr(), cu_k.data_ptr(), marks[0] - 1, total_q, tokens, heads,
        scale, causal, code, out.data_ptr(), lse.data_ptr(), _lib.stream_handle(stream, gpu))
    if status:
        _lib.check("topk_attend_prompt", status)
    return out, lse
