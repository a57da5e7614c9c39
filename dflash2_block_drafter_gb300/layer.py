"""A drafter layer around its sublayers, as a sequence of library calls over preallocated buffers.

``LayerRunner`` is the layer that ``TailRunner`` leaves open (there the sublayers' outputs are given):
attention over a 4-bit context cache and the gated feed-forward block, each between its conv site's
prepare and finish (MAX DFlash2TransformerBlock; dflash2.ts #block):

    a, coef = conv_prepare(norm(x));  q, k, v = a Wqkv^T           # the block's own rows; positions(q, k)
    o = attention(q; the context's cached rows, k, v)              # bidirectional inside the block
    x = x + conv_finish(o Wo^T, coef)                              # and the MLP site's RMSNorm
    a, coef = conv_prepare(n);  h = act(a Wg^T) * (a Wu^T)
    x = x + conv_finish(h Wd^T, coef)

The context's rows enter the cache with ``append_context`` once their tokens are verified (the pages
project them from the target's hidden states; here they are given); ``ContextPages`` keeps their pages, on the device. The RMSNorm of each head of q and k and the
rotary positions, which the pages put between projection and attention, are the caller's: ``positions(q, k)``
may change both in place there; without it neither is applied.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Callable, Optional

import torch

from . import (dflash2_conv_finish, dflash2_conv_prepare, dflash2_conv_prepare_workspace_bytes, dflash2_gated_ffn,
               dflash2_gated_ffn_workspace_bytes, dflash2_kv4_append, dflash2_kv4_attention,
               dflash2_kv4_attention_workspace_bytes, dflash2_kv4_cache, dflash2_kv4_plan, dflash2_proj,
               dflash2_proj_workspace_bytes)
from .tail import SiteWeights, capture


@dataclass
class LayerWeights:
    attn_site: SiteWeights
    w_qkv: torch.Tensor   # [(q_heads + 2 kv_heads) head_dim, H] bf16
    w_o: torch.Tensor     # [H, q_heads head_dim]
    mlp_site: SiteWeights
    w_gate: torch.Tensor  # [F, H]
    w_up: torch.Tensor    # [F, H]
    w_down: torch.Tensor  # [H, F]


class ContextPages:
    """Page table, lengths and free pages of B sequences over a cache of num_pages pages, kept on the device
    (``dflash2_kv4_plan`` in place). One serves every layer whose caches have the same pages."""

    def __init__(self, B: int, num_pages: int, max_pages: int, page_size: int = 64, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.num_pages, self.page_size = num_pages, page_size
        self.table = torch.full((B, max_pages), -1, **i32)
        self.lengths = torch.zeros(B, **i32)
        self.free = torch.arange(num_pages, **i32)
        self.state = torch.tensor([0, num_pages], **i32)
        self.offsets = torch.zeros(B + 1, **i32)

    def gain(self, change: torch.Tensor, rows: int = 0, place: Optional[torch.Tensor] = None, slots=None, positions=None):
        """change [B]: tokens that each sequence gains, or (negative) drops from its end. Returns (slots, positions) of the
        new tokens' rows: `rows` packed ones, or place's [B, G]. A sequence for which no page was free keeps its length."""
        *_, slots, positions = dflash2_kv4_plan(
            self.lengths, change, self.table, self.free, self.state, self.page_size, self.num_pages, rows=rows, place=place,
            ctx_out=self.lengths, state_out=self.state, offsets=self.offsets, slots=slots, positions=positions)
        return slots, positions


class LayerRunner:
    """A drafter layer for B blocks of G rows over a paged 4-bit context cache (bf16)."""

    def __init__(self, weights: LayerWeights, B: int, G: int, q_heads: int, kv_heads: int, head_dim: int,
                 num_pages: int, max_pages: int, page_size: int = 64, group_size: int = 16, eps: float = 1e-6,
                 window: int = 0, act: str = "silu", device="cuda"):
        w = weights
        self.w, self.B, self.G, self.eps, self.act, self.window = w, B, G, eps, act, window
        self.gs, self.page_size, self.scale = group_size, page_size, head_dim ** -0.5
        H, F, M = w.w_o.shape[0], w.w_gate.shape[0], B * G
        nq, nk = q_heads * head_dim, kv_heads * head_dim
        if tuple(w.w_qkv.shape) != (nq + 2 * nk, H):
            raise ValueError(f"w_qkv must be [{nq + 2 * nk}, {H}], got {tuple(w.w_qkv.shape)}")
        new = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=device)
        ws = lambda n: torch.empty(max(n, 256), dtype=torch.uint8, device=device)
        self.cache = dflash2_kv4_cache(num_pages, kv_heads, head_dim, page_size, device)
        self.a, self.n, self.x, self.mid = (new(B, G, H) for _ in range(4))
        self.y = new(B, G, H)
        self.coef = new(B, G, 2, H // group_size)
        self.qkv = new(B, G, nq + 2 * nk)
        self.q = self.qkv[..., :nq].unflatten(-1, (q_heads, head_dim))
        self.k = self.qkv[..., nq:nq + nk].unflatten(-1, (kv_heads, head_dim))
        self.v = self.qkv[..., nq + nk:].unflatten(-1, (kv_heads, head_dim))
        self.o = new(B, G, q_heads, head_dim)
        self.h = new(M, F)
        self.conv_ws = ws(dflash2_conv_prepare_workspace_bytes(B, G, H, group_size, torch.bfloat16))
        # (the projections run one after the other on one stream and share a workspace)
        self.proj_ws = ws(max(dflash2_proj_workspace_bytes(M, nq + 2 * nk, H), dflash2_proj_workspace_bytes(M, H, nq),
                              dflash2_proj_workspace_bytes(M, H, F)))
        self.attn_ws = ws(dflash2_kv4_attention_workspace_bytes(B, G, q_heads, kv_heads, head_dim, page_size, max_pages))
        self.ffn_ws = ws(dflash2_gated_ffn_workspace_bytes(M, H, F, False))

    def append_context(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor):
        """Quantise verified context rows [T, kv_heads, head_dim] into cache slots [T] (int64)."""
        dflash2_kv4_append(k, v, slots, self.cache, self.page_size)

    def forward(self, x: torch.Tensor, page_table: torch.Tensor, ctx_len: torch.Tensor,
                positions: Optional[Callable[[torch.Tensor, torch.Tensor], None]] = None) -> torch.Tensor:
        """x [B, G, H] -> the layer's output residual stream [B, G, H] (self.x); x is left unchanged.
        page_table [B, max_pages] and ctx_len [B] (int32) say where each sequence's context lies."""
        w, M = self.w, self.B * self.G
        s = w.attn_site
        dflash2_conv_prepare(x, s.norm_w, self.eps, s.w_kp, s.base, self.gs, out=self.a, coef1=self.coef,
                             workspace=self.conv_ws)
        dflash2_proj(self.a.view(M, -1), w.w_qkv, out=self.qkv, workspace=self.proj_ws)
        if positions is not None:
            positions(self.q, self.k)
        dflash2_kv4_attention(self.q, self.cache, page_table, ctx_len, self.page_size, self.scale, k_new=self.k,
                              v_new=self.v, window=self.window, out=self.o, workspace=self.attn_ws)
        dflash2_proj(self.o.view(M, -1), w.w_o, out=self.y, workspace=self.proj_ws)
        dflash2_conv_finish(self.y, self.coef, s.base, self.gs, residual=x, out=self.mid, next_norm_w=w.mlp_site.norm_w,
                            eps=self.eps, next_n=self.n)
        s = w.mlp_site
        dflash2_conv_prepare(self.n, None, self.eps, s.w_kp, s.base, self.gs, out=self.a, coef1=self.coef,
                             workspace=self.conv_ws)
        dflash2_gated_ffn(self.a.view(M, -1), w.w_gate, w.w_up, act=self.act, out=self.h, workspace=self.ffn_ws)
        dflash2_proj(self.h, w.w_down, out=self.y, workspace=self.proj_ws)
        dflash2_conv_finish(self.y, self.coef, s.base, self.gs, residual=self.mid, out=self.x)
        return self.x

    def capture(self, *args, **kwargs) -> "torch.cuda.CUDAGraph":
        """One ``forward`` as a CUDA graph (see ``tail.capture``); lengths and pages are read at replay."""
        return capture(self.forward, *args, **kwargs)
