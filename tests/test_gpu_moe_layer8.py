"""The router, the dispatch, the 8-bit experts and the combine together: a decode step, and a layer's gradients."""
import importlib.util
import os
import sys

import numpy as np
import pytest
import torch

import combine_ep_get_dispatch_gb300 as ep
import experts_reference as X

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


def value(codes, scale):
    """[experts, rows, cols] E4M3 codes and scales of 128 x 128 blocks -> values in 64 bits."""
    w = codes.view(torch.float8_e4m3fn).double()
    s = scale.double().repeat_interleave(128, 1)[:, :w.shape[1]].repeat_interleave(128, 2)
    return w * s


def blocks(g, experts, rows, cols):
    w = torch.randn(experts, rows, cols, generator=g, device="cuda") * 100.0
    scale = torch.rand(experts, -(-rows // 128), cols // 128, generator=g, device="cuda") + 0.5
    return w.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), scale * 0.01 * cols ** -0.5


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_decode_step8", os.path.join(ROOT, "examples", "moe_decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = m  # dataclasses look their module up
    spec.loader.exec_module(m)
    return m


def test_example_runs_with_8_bit_experts(example, capsys):
    example.main(8)
    out = capsys.readouterr().out
    assert "8-bit" in out and "finite True" in out


def test_decode_experts_agree_with_plain_torch():
    """Routing in groups with a bias, low-latency dispatch, both products, combine, for a batch of tokens."""
    g = torch.Generator(device="cuda").manual_seed(1)
    N, E, K, R, H, I = 32, 16, 4, 4, 512, 256
    x = torch.randn(N, H, generator=g, device="cuda").to(torch.bfloat16)
    z = torch.randn(N, E, generator=g, device="cuda")
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    up, s_up = blocks(g, E, 2 * I, H)
    down, s_down = blocks(g, E, H, I)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(score="sigmoid", groups=4, topk_groups=2, scale=2.5)
    idx, w = ep.route(z, K, bias=bias, **args)
    (rx, rs), count, handle, _ = ep.low_latency_dispatch(x, idx, N // R, E, R, use_fp8=True, use_ue8m0=True,
                                                         return_recv_hook=False, status=st)
    y, ys = ep.expert_linear_fp8(rx, rs, up, s_up, count, glu=True, use_fp8=True, use_ue8m0=True, max_rows=N * K, status=st)
    y = ep.expert_linear_fp8(y, ys, down, s_down, count, max_rows=N * K, status=st)
    out = ep.low_latency_combine(y, w, handle, status=st)
    assert int(st.item()) == 0
    ri, rw, _ = X.route(z.cpu().numpy(), K, bias.cpu().numpy(), "sigmoid", 4, 2, 2, True, 2.5)
    assert np.array_equal(idx.cpu().numpy(), ri)
    wu, wd, xd = value(up, s_up), value(down, s_down), x.double()
    want = torch.zeros(N, H, dtype=torch.float64, device="cuda")
    for t in range(N):
        for k in range(K):
            a, b = (wu[ri[t, k]] @ xd[t]).chunk(2)
            want[t] += rw[t, k] * (wd[ri[t, k]] @ (torch.nn.functional.silu(a) * b))
    # E4M3 keeps 4 bits: x and the gated values are each off by at most 2^-4, and by 2^-5 on average, in directions of
    # their own; gate and up both carry x's
    off = (out.double() - want).norm(dim=1) / want.norm(dim=1)
    assert (off < 3 * 2.0 ** -5).all(), off


def test_gradients_through_a_layer():
    """x and the router's logits: the kernels' chain against autograd of the same layer in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(2)
    N, E, K, R, H, I = 67, 8, 3, 2, 256, 384
    x = torch.randn(N, H, generator=g, device="cuda").to(torch.bfloat16)
    z = torch.randn(N, E, generator=g, device="cuda")
    up, s_up = blocks(g, E, I, H)
    down, s_down = blocks(g, E, H, I)
    dout = torch.randn(N, H, generator=g, device="cuda").to(torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def quantize(t):
        q = torch.empty(t.shape, dtype=torch.uint8, device="cuda")
        s = torch.empty(t.shape[0], t.shape[1] // 128, device="cuda")
        ep.ep_fp8_quantize(t, q, s)
        return q, s
    # forward: route, dispatch, up, relu, down, combine
    idx, w = ep.route(z, K, scale=1.5)
    lay, res = ep.get_layout_and_dispatch(x, idx, E, R, w, use_fp8=True, with_rank=False, status=st)
    n, off = lay.num_tokens_per_expert, lay.expert_offset
    h = ep.expert_linear_fp8(res.expert_x, res.expert_scales, up, s_up, n, off, status=st)
    y = ep.expert_linear_fp8(*quantize(h.relu()), down, s_down, n, off, status=st)
    out = ep.combine(y, lay, w, status=st)
    # backward
    dy, dw = ep.combine_backward(dout, lay, y, w, status=st)
    dh = ep.expert_linear_fp8_backward(*quantize(dy), down, s_down, n, off, status=st)
    dx_rows = ep.expert_linear_fp8_backward(*quantize(dh * (h > 0)), up, s_up, n, off, status=st)
    dx = ep.dispatch_backward(dx_rows, lay, status=st)
    dz = ep.route_backward(dw, z, idx, scale=1.5, status=st)
    assert int(st.item()) == 0
    # the same in 64 bits
    wu, wd = value(up, s_up), value(down, s_down)
    xr, zr = x.double().requires_grad_(), z.double().requires_grad_()
    p = zr.softmax(1).gather(1, idx.long())
    p = 1.5 * p / p.sum(1, keepdim=True)
    hr = torch.einsum("nkoh,nh->nko", wu[idx.long()], xr).relu()
    ref = (torch.einsum("nkho,nko->nkh", wd[idx.long()], hr) * p[..., None]).sum(1)
    ref.backward(dout.double())

    def rel(a, b):
        return ((a.double() - b).norm() / b.norm()).item()
    # values in E4M3 are off by at most 2^-4 of themselves, 2^-5 on average: two of them on the way to out, two to dz
    # (x and h, by way of y), and to dx two of its own (dy, dh) and the signs of h that x's errors turn: of the
    # values near 0, under 2^-5 of them, each worth its whole gradient: sqrt(2^-5) of the norm at the very most
    assert rel(out, ref.detach()) < 2 * 2.0 ** -5
    assert rel(dz, zr.grad) < 4 * 2.0 ** -5
    assert rel(dx, xr.grad) < 2 * 2.0 ** -5 + 2.0 ** -2.5


def test_a_captured_step_of_routing_dispatch_and_products():
    """The whole decode path in a graph, replayed on other tokens: the same bits as eager calls."""
    g = torch.Generator(device="cuda").manual_seed(3)
    N, E, K, R, H, I = 24, 8, 2, 2, 256, 128
    up, s_up = blocks(g, E, 2 * I, H)
    down, s_down = blocks(g, E, H, I)
    ws = torch.zeros(ep.ep_ll_workspace_bytes(N, K, E, R, N // R), dtype=torch.uint8, device="cuda")
    work = ep.expert_linear_fp8_workspace(torch.empty(E, N, H, dtype=torch.uint8, device="cuda"), up, N * K)

    def step(x, z):
        idx, w = ep.route(z, K)
        (rx, rs), count, handle, _ = ep.low_latency_dispatch(x, idx, N // R, E, R, return_recv_hook=False, workspace=ws)
        y, ys = ep.expert_linear_fp8(rx, rs, up, s_up, count, glu=True, use_fp8=True, max_rows=N * K, workspace=work)
        y = ep.expert_linear_fp8(y, ys, down, s_down, count, max_rows=N * K, workspace=work)
        return ep.low_latency_combine(y, w, handle)

    def inputs():
        return torch.randn(N, H, generator=g, device="cuda").to(torch.bfloat16), torch.randn(N, E, generator=g, device="cuda")
    x, z = inputs()
    step(x, z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, z)
    for _ in range(3):
        nx, nz = inputs()
        x.copy_(nx)
        z.copy_(nz)
        graph.replay()
        got = out.clone()
        assert torch.equal(got, step(nx, nz))
