"""One decode step of a mixture-of-experts layer on the library's kernels.

Attention over a paged E4M3 cache, the router, the low-latency dispatch in FP8
and the experts with 4-bit weights, as a serving loop runs them:

    keys, values, queries -> kv_append (rotation, quantisation) -> kv_attention
    -> router -> low_latency_dispatch -> receive hook
    -> expert_linear (gate and up, gated) -> expert_linear (down)
    -> low_latency_combine

Every workspace is made once and kept. Projections and the router's scores are
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
        # E2M1 codes have a mean square of about 9: scales of 2^-7 keep products of order one.
        self.w_up, self.s_up = codes(c.experts, 2 * c.inner, c.hidden // 2), \
            torch.full((c.experts, 2 * c.inner, c.hidden // 32), 120, dtype=torch.uint8, device=device)
        self.w_down, self.s_down = codes(c.experts, c.hidden, c.inner // 2), \
            torch.full((c.experts, c.hidden, c.inner // 32), 120, dtype=torch.uint8, device=device)
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
        self.up_ws = ep.expert_linear_workspace(x8, self.w_up, self.max_rows)
        self.down_ws = ep.expert_linear_workspace(
            torch.empty(c.experts, 1, c.inner, dtype=torch.bfloat16, device=device), self.w_down, self.max_rows)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def step(self, x: torch.Tensor, seq_lens: torch.Tensor) -> torch.Tensor:
        """x [tokens, hidden] bf16; seq_lens [tokens] int32, this token included. Returns [tokens, hidden]."""
        c, st = self.cfg, self.status
        qkv = (x @ self.w_qkv.t()).view(c.tokens, -1, c.head_dim)
        q, k, v = qkv.split([c.q_heads, c.kv_heads, c.kv_heads], 1)
        q = ep.kv_append(k, v, self.cache, seq_lens, rope=self.rope, q=q, q_out=q, status=st)  # q rotated in place
        o = ep.kv_attention(q, self.cache, seq_lens, workspace=self.attend_ws, status=st)
        h = x + o.view(c.tokens, -1) @ self.w_out.t()
        scores, idx = torch.topk(h.float() @ self.w_router.float().t(), c.topk)
        weights = scores.softmax(-1)
        (rx, rs), count, handle, hook = ep.low_latency_dispatch(
            h, idx, -(-c.tokens // c.ranks), c.experts, c.ranks, use_fp8=True, use_ue8m0=True, workspace=self.ll_ws,
            status=st)
        hook()
        y = ep.expert_linear(rx, self.w_up, self.s_up, count, x_scale=rs, glu=True, max_rows=self.max_rows,
                             workspace=self.up_ws, status=st)
        y = ep.expert_linear(y, self.w_down, self.s_down, count, max_rows=self.max_rows, workspace=self.down_ws,
                             status=st)
        return h + ep.low_latency_combine(y, weights, handle, status=st)


def main() -> None:
    cfg = Config()
    layer = MoELayer(cfg)
    x = torch.randn(cfg.tokens, cfg.hidden, device="cuda").to(torch.bfloat16)
    lens = torch.zeros(cfg.tokens, dtype=torch.int32, device="cuda")
    for i in range(20):
        lens += 1
        y = layer.step(x, lens)
        x = (y / y.float().pow(2).mean(-1, keepdim=True).sqrt()).to(torch.bfloat16)
    torch.cuda.synchronize()
    assert int(layer.status.item()) == 0, ep.ep_error_string(int(layer.status.item()))
    print(f"20 decode steps of {cfg.tokens} sequences: outputs finite {bool(torch.isfinite(y).all())}, "
          f"rms {y.float().pow(2).mean().sqrt().item():.3f}")


if __name__ == "__main__":
    main()
