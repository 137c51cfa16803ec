"""Tensor-level conveniences over the C ABI (allocation and marshalling only)."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib


def plan(seq_lens: torch.Tensor, max_seq_len: int, workspace: torch.Tensor | None = None,
         stream=None) -> torch.Tensor:
    """Runs ``topk_plan`` and returns the (possibly newly allocated) workspace."""
    batch = seq_lens.shape[0]
    need = _lib.topk_plan_workspace_bytes(batch)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=seq_lens.device)
    _lib.topk_plan(seq_lens, batch, max_seq_len, workspace, stream)
    return workspace


def topk_transform(scores: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor, page_size: int,
                   k: int, max_seq_len: int | None = None, want_raw: bool = False,
                   workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   raw_out: torch.Tensor | None = None, stream=None):
    """Plans (unless a planned ``workspace`` is given) and runs the transform.

    ``scores``: float32 cuda [batch, row_stride] (row-contiguous); ``seq_lens``:
    int32 cuda [batch]; ``page_table``: int32 cuda [batch, pages].  Returns
    ``(out, raw_or_None, workspace)``.
    """
    batch, row_stride = scores.shape
    if max_seq_len is None:
        max_seq_len = row_stride
    if scores.stride(1) != 1 or page_table.stride(1) != 1:
        raise ValueError("scores and page_table rows must be contiguous")
    if workspace is None:
        workspace = plan(seq_lens, max_seq_len, stream=stream)
    if out is None:
        out = torch.empty((batch, k), dtype=torch.int32, device=scores.device)
    if want_raw and raw_out is None:
        raw_out = torch.empty((batch, k), dtype=torch.int32, device=scores.device)
    _lib.topk_transform(scores, scores.stride(0), seq_lens, batch, max_seq_len, page_table, page_table.stride(0),
                        page_size, k, out, raw_out if want_raw else None, workspace, stream)
    return out, (raw_out if want_raw else None), workspace


_DTYPES = {torch.bfloat16: _lib.TOPK_BF16, torch.float16: _lib.TOPK_FP16}


def _same(dtype: torch.dtype, device: torch.device, **tensors) -> None:
    """Raises unless the tensors (None is skipped) are of this type, on this device, with contiguous rows."""
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


def _step(t: torch.Tensor, dim: int, least: int) -> int:
    """Stride of a dimension; `least` where there is one entry, whose stride means nothing."""
    return t.stride(dim) if t.shape[dim] > 1 else least


def _dtype(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16 or float16: got {t.dtype}")
    return code


class BlockTables(NamedTuple):
    """Outputs of :func:`block_tables` (int32 cuda); ``status`` holds the pages taken and the flag bits."""

    seq_lens: torch.Tensor  # [batch]
    cu_new: torch.Tensor  # [batch + 1]
    slots: torch.Tensor  # [max_tokens], -1 past the last new token
    positions: torch.Tensor  # [max_tokens]
    rows: torch.Tensor  # [max_tokens]
    status: torch.Tensor  # [2]


def block_tables(context_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
                 page_table: torch.Tensor, page_size: int, max_tokens: int, out: BlockTables | None = None,
                 stream=None) -> BlockTables:
    """Runs ``topk_block_tables``: writes the new pages into ``page_table`` ([batch, pages], in place) and returns
    the step's lengths, offsets and slot map (in ``out``, where the result of an earlier call is given)."""
    dev, i32 = context_lens.device, torch.int32
    batch, pages = page_table.shape
    _same(i32, dev, context_lens=context_lens, new_lens=new_lens, free_pages=free_pages, page_table=page_table)
    _whole((batch,), context_lens=context_lens, new_lens=new_lens)
    if out is None:
        buf = torch.empty(2 * batch + 3 + 3 * max_tokens, dtype=i32, device=dev)
        out = BlockTables(*buf.split([batch, batch + 1, max_tokens, max_tokens, max_tokens, 2]))
    else:
        _same(i32, dev, **out._asdict())
        _whole((batch,), seq_lens=out.seq_lens)
        _whole((batch + 1,), cu_new=out.cu_new)
        _whole((max_tokens,), slots=out.slots, positions=out.positions, rows=out.rows)
        _whole((2,), status=out.status)
    _lib.topk_block_tables(context_lens, new_lens, batch, page_size, free_pages, free_pages.numel(), page_table,
                           _step(page_table, 0, pages), pages, max_tokens, *out, stream)
    return out


def cache_append(rows: torch.Tensor, slots: torch.Tensor, cache: torch.Tensor,
                 norm_weight: torch.Tensor | None = None, eps: float = 1e-6, cos_sin: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, interleaved: bool = False, stream=None) -> None:
    """Runs ``topk_cache_append``: ``rows`` [tokens, 576] (512 latent values, 64 rotary ones) to ``slots`` of
    ``cache`` [num_slots, 576], normed by ``norm_weight`` [512] and rotated by ``cos_sin`` (float32
    [num_positions, 64]: cosines, sines) at ``positions``, where these are given."""
    dev, width = cache.device, _lib.TOPK_LATENT_DIM + _lib.TOPK_ROPE_DIM
    code, tokens = _dtype(cache, "cache"), rows.shape[0]
    _same(cache.dtype, dev, rows=rows, cache=cache, norm_weight=norm_weight)
    _same(torch.int32, dev, slots=slots, positions=positions)
    _same(torch.float32, dev, cos_sin=cos_sin)
    if rows.dim() != 2 or cache.dim() != 2 or rows.shape[1] != width or cache.shape[1] != width:
        raise ValueError(f"rows and cache must be [.., {width}]: got {tuple(rows.shape)} and {tuple(cache.shape)}")
    _whole((tokens,), slots=slots, positions=positions)
    _whole((_lib.TOPK_LATENT_DIM,), norm_weight=norm_weight)
    if cos_sin is not None:
        _whole((cos_sin.shape[0], _lib.TOPK_ROPE_DIM), cos_sin=cos_sin)
    _lib.topk_cache_append(rows, _step(rows, 0, width), tokens, norm_weight, eps, cos_sin,
                           0 if cos_sin is None else cos_sin.shape[0], positions, interleaved, slots, cache,
                           _step(cache, 0, width), cache.shape[0], code, stream)


def _attend_outputs(q, cache, batch, queries, heads, out, lse, workspace):
    """Checks (or allocates) what both cache attentions share."""
    dev = q.device
    _same(q.dtype, dev, q=q, cache=cache, out=out)
    width, latent = _lib.TOPK_LATENT_DIM + _lib.TOPK_ROPE_DIM, _lib.TOPK_LATENT_DIM
    if q.shape[-1] != width or cache.dim() != 2 or cache.shape[1] != width:
        raise ValueError(f"q and cache must be [.., {width}]: got {tuple(q.shape)} and {tuple(cache.shape)}")
    if out is None:
        out = torch.empty((*q.shape[:-1], latent), dtype=q.dtype, device=dev)
    else:
        _whole((*q.shape[:-1], latent), out=out)
    if lse is None:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=dev)
    else:
        _same(torch.float32, dev, lse=lse)
        _whole(q.shape[:-1], lse=lse)
    need = _lib.topk_attend_workspace_bytes(batch, queries, heads)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    return out, lse, workspace


def attend_selected(q: torch.Tensor, cache: torch.Tensor, indices: torch.Tensor, scale: float,
                    seq_lens: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Runs ``topk_attend_selected``: ``q`` [rows, heads, 576] over the slots ``indices`` [rows, k] (int32, as
    :func:`topk_transform` writes them) of ``cache`` [num_slots, 576].  ``seq_lens`` [rows], where given, bounds
    the slots looked at.  Returns ``(out [rows, heads, 512], lse [rows, heads], workspace)``."""
    if q.dim() != 3 or indices.dim() != 2 or indices.shape[0] != q.shape[0]:
        raise ValueError(f"q and indices must be [rows, heads, ..] and [rows, k]: got {tuple(q.shape)} and "
                         f"{tuple(indices.shape)}")
    code, (rows, heads, _) = _dtype(q, "q"), q.shape
    _same(torch.int32, q.device, indices=indices, seq_lens=seq_lens)
    _whole((rows,), seq_lens=seq_lens)
    out, lse, workspace = _attend_outputs(q, cache, rows, 1, heads, out, lse, workspace)
    _lib.topk_attend_selected(q, _step(q, 0, 0), _step(q, 1, 0), cache, _step(cache, 0, cache.shape[1]), cache.shape[0],
                              indices, _step(indices, 0, indices.shape[1]), seq_lens, rows, heads, indices.shape[1], scale, code, out, lse,
                              workspace, stream)
    return out, lse, workspace


def attend_paged(q: torch.Tensor, cache: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor,
                 page_size: int, scale: float, max_seq_len: int | None = None, out: torch.Tensor | None = None,
                 lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Runs ``topk_attend_paged``: ``q`` [batch, queries, heads, 576], the newest tokens' queries, over each
    request's positions through ``page_table`` [batch, pages].  Returns ``(out [batch, queries, heads, 512],
    lse [batch, queries, heads], workspace)``."""
    if q.dim() != 4 or page_table.dim() != 2 or page_table.shape[0] != q.shape[0]:
        raise ValueError(f"q and page_table must be [batch, queries, heads, ..] and [batch, pages]: got "
                         f"{tuple(q.shape)} and {tuple(page_table.shape)}")
    code, (batch, queries, heads, _) = _dtype(q, "q"), q.shape
    _same(torch.int32, q.device, seq_lens=seq_lens, page_table=page_table)
    _whole((batch,), seq_lens=seq_lens)
    if max_seq_len is None:
        max_seq_len = min(page_table.shape[1] * page_size, 2 ** 31 - 1)
    elif max_seq_len > page_table.shape[1] * page_size:
        raise ValueError(f"max_seq_len {max_seq_len} is over {page_table.shape[1]} pages of {page_size}")
    out, lse, workspace = _attend_outputs(q, cache, batch, queries, heads, out, lse, workspace)
    _lib.topk_attend_paged(q, _step(q, 0, 0), _step(q, 1, 0), _step(q, 2, 0), cache, _step(cache, 0, cache.shape[1]),
                           cache.shape[0], seq_lens, page_table, _step(page_table, 0, page_table.shape[1]), page_size, max_seq_len, batch, queries, heads,
                           scale, code, out, lse, workspace, stream)
    return out, lse, workspace


def attend_prompt(q: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                  cu_k: torch.Tensor, scale: float, causal: bool = True, out: torch.Tensor | None = None,
                  lse: torch.Tensor | None = None, stream=None):
    """Runs ``topk_attend_prompt``: ``q`` [total_q, heads, 192], ``k_nope`` [total_k, heads, 128], ``k_rope``
    [total_k, 64], ``v`` [total_k, heads, 128], requests by the offsets ``cu_q`` and ``cu_k`` [batch + 1].
    Returns ``(out [total_q, heads, 128], lse [total_q, heads])``."""
    code, dev = _dtype(q, "q"), q.device
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError(f"q and v must be [tokens, heads, ..]: got {tuple(q.shape)} and {tuple(v.shape)}")
    (total_q, heads, _), total_k = q.shape, v.shape[0]
    _same(q.dtype, dev, q=q, k_nope=k_nope, k_rope=k_rope, v=v, out=out)
    _same(torch.int32, dev, cu_q=cu_q, cu_k=cu_k)
    nope, rope, value = _lib.TOPK_NOPE_DIM, _lib.TOPK_ROPE_DIM, _lib.TOPK_VALUE_DIM
    for name, t, shape in (("q", q, (total_q, heads, nope + rope)), ("k_nope", k_nope, (total_k, heads, nope)),
                           ("k_rope", k_rope, (total_k, rope)), ("v", v, (total_k, heads, value))):
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {shape}: got {tuple(t.shape)}")
    _whole(cu_q.shape[:1], cu_q=cu_q, cu_k=cu_k)
    if out is None:
        out = torch.empty((total_q, heads, value), dtype=q.dtype, device=dev)
    else:
        _whole((total_q, heads, value), out=out)
    if lse is None:
        lse = torch.empty((total_q, heads), dtype=torch.float32, device=dev)
    else:
        _same(torch.float32, dev, lse=lse)
        _whole((total_q, heads), lse=lse)
    _lib.topk_attend_prompt(q, _step(q, 0, nope + rope), _step(q, 1, nope + rope), k_nope, _step(k_nope, 0, nope),
                            _step(k_nope, 1, nope), k_rope, _step(k_rope, 0, rope), v, _step(v, 0, value),
                            _step(v, 1, value), cu_q, cu_k, cu_q.shape[0] - 1, total_q, total_k, heads, scale, causal,
                            code, out, lse, stream)
    return out, lse
