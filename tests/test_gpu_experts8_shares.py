"""The experts' 8-bit products in calls of few units: shared by several blocks, or one block's each, by sizes and rows."""
import numpy as np
import pytest
import torch

import combine_ep_get_dispatch_gb300 as ep
import decode_reference as R
import experts_reference as X

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("K", [512, 1024, 2048, 4096, 7168, 16384])
@pytest.mark.parametrize("rows", [1, 8, 9, 33])
def test_units_shared_and_whole(K, rows):
    """Sums in parts and in one give the formula's values, the same bits each time, on one workspace for all."""
    g = torch.Generator(device="cuda").manual_seed(K + rows)
    wide = 256 * 76
    w = (torch.randn(wide, K, generator=g, device="cuda") * 60.0).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    ws = torch.exp(0.3 * torch.randn(wide // 128, K // 128, generator=g, device="cuda")) * (K ** -0.5 / 60.0)
    x = (torch.randn(rows, K, generator=g, device="cuda") * 100.0).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    xs = torch.exp(0.3 * torch.randn(rows, K // 128, generator=g, device="cuda")) / 100.0
    count, off = (torch.tensor([v], dtype=torch.int32, device="cuda") for v in (rows, 0))
    space = torch.zeros(ep.ep_expert_linear_fp8_workspace_bytes(1, rows), dtype=torch.uint8, device="cuda")
    value = R.TABLE[x.cpu().numpy()] * xs.double().cpu().numpy().repeat(128, axis=1)
    rng = np.random.default_rng(K + rows)
    for units in (1, 19, 20, 38, 39, 48, 60, 64, 68, 76):
        outs = 256 * units
        args = (x, xs, w[:outs].unsqueeze(0), ws[:outs // 128].unsqueeze(0), count, off)
        y = ep.expert_linear_fp8(*args, workspace=space)
        for _ in range(3):
            assert torch.equal(ep.expert_linear_fp8(*args, workspace=space), y)
        at = np.sort(rng.choice(outs, 96, replace=False))
        scale = ws[:outs // 128].double().cpu().numpy()[at // 128].repeat(128, axis=1)
        X.check_bf16(y.double().cpu().numpy()[:, at], *X.product(value, R.TABLE[w[torch.from_numpy(at).cuda()].cpu().numpy()] * scale, False))
