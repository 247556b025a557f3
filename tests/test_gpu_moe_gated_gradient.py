"""Back through a gated product: its gate outside, and the gradient of gates and ups together through the weights as one matrix."""
import numpy as np
import pytest
import torch

import combine_ep_get_dispatch_gb300 as ep
import decode_reference as R
import experts_reference as X

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,inner", [(256, 128), (384, 384)])
def test_gradient_through_gates_and_ups(K, inner):
    import __graft_entry__ as build
    build.build()
    g = torch.Generator(device="cuda").manual_seed(K + inner)
    counts, E = [5, 0, 17], 3
    n, M = sum(counts), 2 * inner

    def codes(*shape):
        v = (torch.randn(*shape, generator=g, device="cuda") * 100.0).clamp(-448.0, 448.0)
        return v.to(torch.float8_e4m3fn).view(torch.uint8)
    w, x = codes(E, M, K), codes(n, K)
    ws = torch.exp(0.3 * torch.randn(E, M // 128, K // 128, generator=g, device="cuda")) * (0.01 * K ** -0.5)
    xs = torch.exp(0.3 * torch.randn(n, K // 128, generator=g, device="cuda")) * 0.01
    count = torch.tensor(counts, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 5, 5], dtype=torch.int32, device="cuda")
    dh = torch.randn(n, inner, generator=g, device="cuda")
    gu = ep.expert_linear_fp8(x, xs, w, ws, count, off).float()
    a, b = gu.chunk(2, 1)
    s = torch.sigmoid(a)
    dgu = torch.cat([dh * b * s * (1 + a * (1 - s)), dh * a * s], 1).to(torch.bfloat16)
    q, qs = torch.empty(n, M, dtype=torch.uint8, device="cuda"), torch.empty(n, M // 128, device="cuda")
    ep.ep_fp8_quantize(dgu, q, qs)
    dx = ep.expert_linear_fp8_backward(q, qs, w, ws, count, off).double().cpu().numpy()
    h = ep.expert_linear_fp8(x, xs, w, ws, count, off, glu=True).double().cpu().numpy()
    # autograd of the gated product in 64 bits
    expert = np.repeat([0, 2], [5, 17])
    value = [R.TABLE[w[e].cpu().numpy()] * X.blocks(ws[e].double().cpu().numpy(), M, K) for e in range(E)]
    xv = R.TABLE[x.cpu().numpy()] * xs.double().cpu().numpy().repeat(128, axis=1)
    for e in (0, 2):
        rows = expert == e
        xr = torch.from_numpy(xv[rows]).requires_grad_()
        p, u = (xr @ torch.from_numpy(value[e]).t()).chunk(2, 1)
        p.retain_grad(), u.retain_grad()
        y = torch.nn.functional.silu(p) * u
        y.backward(dh[torch.from_numpy(rows).cuda()].double().cpu())
        # h: one rounding; dx: of gates and ups in BF16 (2^-8 of either, which silu' < 1.1, silu'' < 0.5 and the other
        # factor carry on), of their gradient in BF16 and E4M3 (2^-4 of a value, or 2^-10 of its block's scale), and dx's
        want = y.detach().numpy()
        assert (np.abs(h[rows] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -16 * (np.abs(xv[rows]) @ np.abs(value[e]).T).max()).all()
        P, U, D = (v.detach().abs().numpy() for v in (p, u, dh[torch.from_numpy(rows).cuda()].double().cpu()))
        d = np.concatenate([p.grad.numpy(), u.grad.numpy()], 1)
        lost = np.concatenate([D * (1.1 * 2.0 ** -8 * U + 0.5 * U * 2.0 ** -8 * P), D * 1.1 * 2.0 ** -8 * P], 1)
        top = (np.abs(d) + lost).reshape(d.shape[0], -1, 128).max(2).repeat(128, axis=1) / 448
        lost += (2.0 ** -4 + 2.0 ** -8) * (np.abs(d) + lost) + 2.0 ** -10 * top
        dxw = xr.grad.numpy()
        tol = (lost * 1.05) @ np.abs(value[e]) + 2.0 ** -8 * np.abs(dxw) * 1.05
        off_by = np.abs(dx[rows] - dxw)
        assert (off_by <= tol).all(), (off_by / tol).max()
        # and as a whole much nearer: errors of E4M3, 2^-5 on average, in directions of their own
        assert np.linalg.norm(dx[rows] - dxw) < 2.0 ** -4 * np.linalg.norm(dxw)
