"""One decode step of a mixture-of-experts layer on the library's kernels.

Attention over a paged E4M3 cache, the router, the low-latency dispatch in FP8
and the experts with 4-bit weights (or 8-bit, expert_bits=8), as a serving loop
runs them:

    keys, values, queries -> kv_append (rotation, quantisation) -> kv_attention
    -> route -> low_latency_dispatch -> receive hook
    -> expert_linear (gate and up, gated) -> expert_linear (down)
    -> low_latency_combine

With 8-bit weights the first product leaves its rows in FP8, with a scale for
each 128 channels, as the second takes them (expert_linear_fp8).

Every workspace is made once and kept. Projections and the router's logits are
plain torch products. Run it for random weights and a few steps:

    python examples/moe_decode_step.py
"""
from __future__ import annotations

import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_ep_get_dispatch_gb300 as ep  # noqa: E402


@dataclasses.dataclass
class Config:
    tokens: int = 16         # sequences of the batch, one token each
    ranks: int = 4           # expert-parallel ranks (partitions of this GPU)
    experts: int = 32
    topk: int = 4
    hidden: int = 1024
    inner: int = 512         # of an expert
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    page_size: int = 16
    max_len: int = 256
    expert_bits: int = 4     # of the experts' weights: 4 (E2M1) or 8 (E4M3)


class MoELayer:
    """Random weights of one layer, its cache and its workspaces."""

    def __init__(self, cfg: Config, device="cuda", seed: int = 0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.cfg = c = cfg

        def normal(*shape, scale=1.0):
            return (torch.randn(shape, generator=g, device=device) * scale).to(torch.bfloat16)

        def codes(*shape):
            return torch.randint(0, 256, shape, generator=g, device=device, dtype=torch.uint8)

        heads = c.q_heads + 2 * c.kv_heads
        self.w_qkv = normal(heads * c.head_dim, c.hidden, scale=c.hidden ** -0.5)
        self.w_out = normal(c.hidden, c.q_heads * c.head_dim, scale=(c.q_heads * c.head_dim) ** -0.5)
        self.w_router = normal(c.experts, c.hidden, scale=c.hidden ** -0.5)
        if c.expert_bits == 4:
            # E2M1 codes have a mean square of about 9: scales of 2^-7 keep products of order one.
            self.w_up, self.s_up = codes(c.experts, 2 * c.inner, c.hidden // 2), \
                torch.full((c.experts, 2 * c.inner, c.hidden // 32), 120, dtype=torch.uint8, device=device)
            self.w_down, self.s_down = codes(c.experts, c.hidden, c.inner // 2), \
                torch.full((c.experts, c.hidden, c.inner // 32), 120, dtype=torch.uint8, device=device)
        else:
            def blocks(rows, cols):
                """E4M3 codes of normal values, and a scale for each 128 x 128 of them."""
                w = torch.randn(c.experts, rows, cols, generator=g, device=device) * 100.0
                scale = torch.full((c.experts, rows // 128, cols // 128), 0.01 * cols ** -0.5, device=device)
                return w.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), scale
            self.w_up, self.s_up = blocks(2 * c.inner, c.hidden)
            self.w_down, self.s_down = blocks(c.hidden, c.inner)
        pages = c.max_len // c.page_size
        table = torch.arange(c.tokens * pages, dtype=torch.int32, device=device).view(c.tokens, pages)
        self.cache = ep.new_kv_cache(c.tokens * pages, c.kv_heads, c.page_size, c.head_dim, table)
        angle = torch.arange(c.max_len, device=device)[:, None] * \
            10000.0 ** (-2.0 * torch.arange(c.head_dim // 2, device=device) / c.head_dim)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float()
        # Workspaces: zero-filled once.
        n = -(-c.tokens // c.ranks)
        self.ll_ws = torch.zeros(ep.ep_ll_workspace_bytes(c.tokens, c.topk, c.experts, c.ranks, n), dtype=torch.uint8,
                                 device=device)
        self.attend_ws = ep.kv_attention_workspace(
            torch.empty(c.tokens, c.q_heads, c.head_dim, dtype=torch.bfloat16, device=device), self.cache)
        self.max_rows = c.tokens * c.topk
        x8 = torch.empty(c.experts, n * c.ranks, c.hidden, dtype=torch.uint8, device=device)
        if c.expert_bits == 4:
            self.up_ws = ep.expert_linear_workspace(x8, self.w_up, self.max_rows)
            self.down_ws = ep.expert_linear_workspace(
                torch.empty(c.experts, 1, c.inner, dtype=torch.bfloat16, device=device), self.w_down, self.max_rows)
        else:  # one after the other on a stream, the products may share a workspace
            self.up_ws = self.down_ws = ep.expert_linear_fp8_workspace(x8, self.w_up, self.max_rows)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def step(self, x: torch.Tensor, seq_lens: torch.Tensor) -> torch.Tensor:
        """x [tokens, hidden] bf16; seq_lens [tokens] int32, this token included. Returns [tokens, hidden]."""
        c, st = self.cfg, self.status
        qkv = (x @ self.w_qkv.t()).view(c.tokens, -1, c.head_dim)
        q, k, v = qkv.split([c.q_heads, c.kv_heads, c.kv_heads], 1)
        q = ep.kv_append(k, v, self.cache, seq_lens, rope=self.rope, q=q, q_out=q, status=st)  # q rotated in place
        o = ep.kv_attention(q, self.cache, seq_lens, workspace=self.attend_ws, status=st)
        h = x + o.view(c.tokens, -1) @ self.w_out.t()
        idx, weights = ep.route(h.float() @ self.w_router.float().t(), c.topk)
        (rx, rs), count, handle, hook = ep.low_latency_dispatch(
            h, idx, -(-c.tokens // c.ranks), c.experts, c.ranks, use_fp8=True, use_ue8m0=True, workspace=self.ll_ws,
            status=st)
        hook()
        if c.expert_bits == 4:
            y = ep.expert_linear(rx, self.w_up, self.s_up, count, x_scale=rs, glu=True, max_rows=self.max_rows,
                                 workspace=self.up_ws, status=st)
            y = ep.expert_linear(y, self.w_down, self.s_down, count, max_rows=self.max_rows, workspace=self.down_ws,
                                 status=st)
        else:
            y, ys = ep.expert_linear_fp8(rx, rs, self.w_up, self.s_up, count, glu=True, use_fp8=True,
                                         max_rows=self.max_rows, workspace=self.up_ws, status=st)
            y = ep.expert_linear_fp8(y, ys, self.w_down, self.s_down, count, max_rows=self.max_rows,
                                     workspace=self.down_ws, status=st)
        return h + ep.low_latency_combine(y, weights, handle, status=st)


def main(expert_bits: int = 4) -> None:
    cfg = Config(expert_bits=expert_bits)
    layer = MoELayer(cfg)
    x = torch.randn(cfg.tokens, cfg.hidden, device="cuda").to(torch.bfloat16)
    lens = torch.zeros(cfg.tokens, dtype=torch.int32, device="cuda")
    for i in range(20):
        lens += 1
        y = layer.step(x, lens)
        x = (y / y.float().pow(2).mean(-1, keepdim=True).sqrt()).to(torch.bfloat16)
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0, ep.ep_error_string(int(layer.status.item()))
    print(f"20 decode steps of {cfg.tokens} sequences, {expert_bits}-bit experts: outputs finite {bool(torch.isfinite(y).all())}, "
          f"rms {y.float().pow(2).mean().sqrt().item():.3f}")


if __name__ == "__main__":
    for bits in (4, 8):
        main(bits)
