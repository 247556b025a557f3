"""The gradient of the experts' 8-bit products against differences of the product, large against its roundings.

Rows of x that hold one channel each give the product's derivative in that
channel with nothing beside it: y(x) - y(0) is that term alone, off by its own
rounding to BF16, not by that of a whole output.
"""
import numpy as np
import pytest
import torch

import combine_ep_get_dispatch_gb300 as ep
import decode_reference as R
import experts_reference as X

K, M, COUNTS, ROWS = 256, 384, [3, 2], 5   # inputs, outputs, rows of the gradient of two experts
VALUE = 0.75                               # what a channel is raised by


class Inputs:
    def __init__(self, ue8m0):
        g = torch.Generator().manual_seed(31)

        def codes(*shape):
            v = (torch.randn(*shape, generator=g) * 60.0).clamp(-448.0, 448.0)
            return v.to(torch.float8_e4m3fn).view(torch.uint8)
        self.w, self.gy = codes(2, M, K), codes(ROWS, M)
        self.ws = torch.exp(0.2 * torch.randn(2, M // 128, K // 128, generator=g)) / 60.0
        if ue8m0:
            self.gs = torch.randint(119, 122, (ROWS, M // 128), generator=g, dtype=torch.uint8)
            scale = 2.0 ** (self.gs.numpy().astype(np.float64) - 127)
        else:
            self.gs = torch.exp(0.2 * torch.randn(ROWS, M // 128, generator=g)) / 60.0
            scale = self.gs.numpy().astype(np.float64)
        self.expert = np.repeat([0, 1], COUNTS)
        self.g = R.TABLE[self.gy.numpy()] * scale.repeat(128, axis=1)
        self.weights = [R.TABLE[self.w[e].numpy()] * X.blocks(self.ws[e].numpy().astype(np.float64), M, K) for e in (0, 1)]
        # a row for each channel and expert: 1.5 times the scale 0.5
        self.x = torch.zeros(2, K, K, dtype=torch.uint8)
        self.x[:, torch.arange(K), torch.arange(K)] = 0x3C
        self.xs = torch.full((2, K, K // 128), 0.5)

    def slack(self, r):
        """What <g, y(x) - y(0)> and dx * VALUE of row r can differ by: BF16's half steps, and fp32 sums (experts_reference)."""
        terms = np.abs(self.g[r]) @ np.abs(self.weights[self.expert[r]])            # of each channel
        dx = np.abs(self.g[r] @ self.weights[self.expert[r]])
        sums = (M / 32 + 8) * 2.0 ** -22 * terms
        return VALUE * (2.0 ** -8 * terms + 2.0 ** -22 * terms + 2.0 ** -8 * (dx + sums) + sums)


@pytest.mark.parametrize("ue8m0", [False, True])
def test_the_differences_are_large_against_their_slack(ue8m0):
    """Before any kernel runs: a gradient of 0, of the wrong sign or of the next channel is outside for nearly all."""
    c = Inputs(ue8m0)
    assert R.TABLE[0x3C] * 0.5 == VALUE
    for r in range(ROWS):
        dx, slack = c.g[r] @ c.weights[c.expert[r]] * VALUE, c.slack(r)
        assert (np.abs(dx) > 4 * slack).mean() > 0.7
        assert (np.abs(np.roll(dx, 1) - dx) > slack).mean() > 0.9
        other = c.g[r] @ c.weights[1 - c.expert[r]] * VALUE
        assert (np.abs(other - dx) > slack).mean() > 0.9


@pytest.mark.gpu
@pytest.mark.parametrize("ue8m0", [False, True])
def test_gradient_of_every_channel(ue8m0):
    import __graft_entry__ as g
    g.build()
    c = Inputs(ue8m0)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    w, ws = c.w.cuda(), c.ws.cuda()
    dx = ep.expert_linear_fp8_backward(c.gy.cuda(), c.gs.cuda(), w, ws, ints(COUNTS), ints([0, COUNTS[0]]))
    y = ep.expert_linear_fp8(c.x.cuda(), c.xs.cuda(), w, ws, ints([K, K]))
    none = ep.expert_linear_fp8(torch.zeros_like(c.x).cuda(), c.xs.cuda(), w, ws, ints([K, K]))
    assert (none == 0).all()
    dx, dy = dx.double().cpu().numpy(), (y - none).double().cpu().numpy()
    for r in range(ROWS):
        by_differences, slack = dy[c.expert[r]] @ c.g[r], c.slack(r)
        off = np.abs(by_differences - VALUE * dx[r])
        assert (off <= slack).all(), (off / slack).max()
        assert (np.abs(by_differences) > 4 * slack).mean() > 0.7
