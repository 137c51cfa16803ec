"""One serving step of a sparse-attention layer, from request lengths to outputs.

``python -m sparse_attention_indexer_uint32_gb300.serve_step`` runs a few
steps of a small batch with random weights and prints what each one did.  A
step goes through the library's calls in the order in which a program makes
them, all on one stream and without a host read in between:

* ``block_tables``: pages for the new tokens, their slots and positions;
* ``cache_append``: the tokens' latent rows, normed and rotated, to those slots;
* prompts: ``attend_prompt`` on the keys and values expanded from the latents;
* decoding: ``topk_transform`` on the indexer's scores, ``attend_selected`` on
  the slots it wrote, or, for rows no longer than ``k``, ``attend_paged`` on
  the whole row (both are computed here and agree on such rows).
"""
from __future__ import annotations

import torch

from . import _lib, api

HEADS, LATENT, ROPE, NOPE, VALUE = 16, 512, 64, 128, 128
SCALE = (NOPE + ROPE) ** -0.5


class Layer:
    """Cache, tables and random weights of one layer for a fixed batch."""

    def __init__(self, batch: int, pages_per_row: int, page_size: int, seed: int = 0, dtype=torch.bfloat16):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g, self.dtype, self.batch, self.page_size = g, dtype, batch, page_size
        i32 = dict(dtype=torch.int32, device="cuda")
        pages = batch * pages_per_row
        self.cache = torch.zeros(pages * page_size, LATENT + ROPE, dtype=dtype, device="cuda")
        self.table = torch.full((batch, pages_per_row), -1, **i32)
        self.free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.lens = torch.zeros(batch, **i32)
        self.norm = torch.ones(LATENT, dtype=dtype, device="cuda")
        angle = torch.arange(pages_per_row * page_size, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(ROPE // 2, device="cuda") / (ROPE // 2))
        self.cos_sin = torch.cat((angle.cos(), angle.sin()), 1).float()
        self.up = torch.randn(LATENT, HEADS, NOPE + VALUE, generator=g, device="cuda").to(dtype) * LATENT ** -0.5
        self.outs = self.workspace = None

    def randn(self, *shape) -> torch.Tensor:
        return torch.randn(shape, generator=self.g, device="cuda").to(self.dtype)

    def append(self, new_lens: torch.Tensor, max_tokens: int):
        """Tables, slots and cached rows of the new tokens; returns the step's offsets and the rows' slots."""
        step = api.block_tables(self.lens, new_lens, self.free, self.table, self.page_size, max_tokens)
        rows = self.randn(max_tokens, LATENT + ROPE)
        api.cache_append(rows, step.slots, self.cache, norm_weight=self.norm, cos_sin=self.cos_sin,
                         positions=step.positions)
        # The pages that were handed out leave the list: the host learns how
        # many between steps.
        self.lens = step.seq_lens
        return step

    def take_pages(self, step) -> None:
        self.free = self.free[int(step.status[0]):].contiguous()

    def prompt(self, new_lens: torch.Tensor, total: int):
        """New prompts for empty rows: (q, out, lse, step) of ``total`` tokens."""
        step = self.append(new_lens, total)
        latent = self.cache[step.slots.long()]
        up = torch.einsum("tl,lhd->thd", latent[:, :LATENT], self.up)
        q = self.randn(total, HEADS, NOPE + ROPE)
        out, lse = api.attend_prompt(q, up[..., :NOPE], latent[:, LATENT:], up[..., NOPE:], step.cu_new, step.cu_new,
                                     SCALE)
        return q, out, lse, step

    def decode(self, k: int):
        """One token for every row: (q, attention over the selected slots, over the whole rows, step)."""
        step = self.append(torch.ones_like(self.lens), self.batch)
        width = self.table.shape[1] * self.page_size
        scores = torch.randn(self.batch, width, generator=self.g, device="cuda")
        slots, _, _ = api.topk_transform(scores, self.lens, self.table, self.page_size, k)
        q = self.randn(self.batch, HEADS, LATENT + ROPE)
        selected, _, self.workspace = api.attend_selected(q, self.cache, slots, SCALE, seq_lens=self.lens,
                                                          workspace=self.workspace)
        whole, _, self.workspace = api.attend_paged(q[:, None], self.cache, self.lens, self.table, self.page_size, SCALE,
                                                    workspace=self.workspace)
        return q, selected, whole[:, 0], step


def main() -> None:
    layer = Layer(batch=4, pages_per_row=16, page_size=64)
    new = torch.tensor([300, 17, 64, 129], dtype=torch.int32, device="cuda")
    _, out, _, step = layer.prompt(new, int(new.sum()))
    layer.take_pages(step)
    print("prompts: lengths", layer.lens.tolist(), "pages", int(step.status[0]), "output", tuple(out.shape))
    for _ in range(3):
        _, selected, whole, step = layer.decode(k=256)
        layer.take_pages(step)
        short = layer.lens <= 256
        gap = (selected[short].float() - whole[short].float()).abs().max().item()
        print("decode: lengths", layer.lens.tolist(), "pages", int(step.status[0]), "selected", tuple(selected.shape),
              f"rows that were selected whole differ by {gap:.1e}")
    # Where the host waits anyway: a wait of a kernel that gave up makes the
    # outputs of its call void.
    if _lib.topk_read_attend_flags(clear=True):
        raise RuntimeError("a wait of an attention kernel gave up")


if __name__ == "__main__":
    main()
