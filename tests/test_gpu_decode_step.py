"""The decode-step example against the same layer written with elementary torch operations."""
import importlib.util
import os
import sys

import pytest
import torch

import decode_reference as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__ as g
    g.build()
    spec = importlib.util.spec_from_file_location("moe_decode_step", os.path.join(ROOT, "examples", "moe_decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = m  # dataclasses look their module up
    spec.loader.exec_module(m)
    return m


def weights_of(codes, scales):
    return torch.stack([torch.from_numpy(R.weights(c, s)) for c, s in zip(codes.cpu().numpy(), scales.cpu().numpy())]).cuda()


def test_steps_agree_with_plain_torch(example):
    cfg = example.Config(tokens=8, experts=8, topk=2, hidden=256, inner=128, ranks=2, max_len=64)
    layer = example.MoELayer(cfg, seed=3)
    up, down = weights_of(layer.w_up, layer.s_up), weights_of(layer.w_down, layer.s_down)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    lens = torch.zeros(cfg.tokens, dtype=torch.int32, device="cuda")
    past_k, past_v = [], []
    for step in range(20):
        lens += 1
        x = torch.randn(cfg.tokens, cfg.hidden, generator=g, device="cuda").to(torch.bfloat16)
        y = layer.step(x, lens)
        # the plain layer, without quantising the cache or the dispatched rows
        qkv = (x @ layer.w_qkv.t()).view(cfg.tokens, -1, cfg.head_dim).double()
        q, k, v = qkv.split([cfg.q_heads, cfg.kv_heads, cfg.kv_heads], 1)
        h = cfg.head_dim // 2
        c, s = layer.rope[step, :h].double(), layer.rope[step, h:].double()
        q, k = (torch.cat([t[..., :h] * c - t[..., h:] * s, t[..., h:] * c + t[..., :h] * s], -1) for t in (q, k))
        past_k.append(k)
        past_v.append(v)
        rep = cfg.q_heads // cfg.kv_heads
        K, V = (torch.stack(t, 1).repeat_interleave(rep, 2) for t in (past_k, past_v))
        p = (torch.einsum("thd,tjhd->thj", q, K) * cfg.head_dim ** -0.5).softmax(-1)
        o = torch.einsum("thj,tjhd->thd", p, V).reshape(cfg.tokens, -1)
        a = x.double() + o @ layer.w_out.double().t()
        scores, idx = torch.topk(a @ layer.w_router.double().t(), cfg.topk + 1)
        w = scores[:, :cfg.topk].softmax(-1)
        clear = (scores[:, cfg.topk - 1] - scores[:, cfg.topk]) > 0.05  # the choice of experts does not hang on rounding
        want = a.clone()
        for t in range(cfg.tokens):
            for j in range(cfg.topk):
                e = idx[t, j]
                z = up[e] @ a[t]
                z = torch.nn.functional.silu(z[:cfg.inner]) * z[cfg.inner:]
                want[t] += w[t, j] * (down[e] @ z)
        # E4M3 keeps 4 bits: an error of a few percent of the row's norm
        off = (y.double() - want).norm(dim=1) / want.norm(dim=1)
        assert clear.sum() >= 2 and (off[clear] < 0.08).all(), off
    assert int(layer.status.item()) == 0


def test_example_runs(example, capsys):
    example.main()
    assert "finite True" in capsys.readouterr().out
