"""The sigmoid's gradient of confident experts, against the formula in 64 bits and a bound that shrinks with it."""
import numpy as np
import pytest
import torch

import combine_ep_get_dispatch_gb300 as ep
import experts_reference as X


def sigmoid(z):
    z = z.astype(np.float64)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def backward(z, idx, dw, ds, renormalize, scale):
    """(dz, bound of fp32's error) of tokens z [N, E]; s (1 - s) without a difference: 1 - s(z) is s(-z)."""
    N, E = z.shape
    s, slope = sigmoid(z), sigmoid(z) * sigmoid(-z)
    g = np.zeros((N, E)) if ds is None else ds.astype(np.float64).copy()
    size = np.abs(g)
    for t in range(N):
        chosen = s[t, idx[t]]
        d = dw[t].astype(np.float64)
        S = chosen.sum() + X.TINY if renormalize else 1.0
        mean, spread = ((d * chosen).sum() / S, (np.abs(d) * chosen).sum() / S) if renormalize else (0.0, 0.0)
        for k, e in enumerate(idx[t]):
            g[t, e] += scale / S * (d[k] - mean)
            size[t, e] += abs(scale) / S * (abs(d[k]) + spread)
    # The slope is e / (1 + e)^2, e = exp(-|z|): 2^-22 of e, twice 2^-24 + 2^-23 of the reciprocal, two products:
    # under 2^-20. What it multiplies has scores off by under 2^-18 each, two of them, and two sums: 2^-16 in all.
    return slope * g, 2.0 ** -16 * slope * size


def cases(dtype, seed, N=24, E=96, K=6):
    g = torch.Generator().manual_seed(seed)
    z = torch.rand(N, E, generator=g) * 60.0 - 30.0
    z[:8] = z[:8].abs()                                        # experts that are all sure of the token
    z[8] = torch.linspace(10.0, 30.0, E)
    z = z.to(dtype)
    idx = z.float().topk(K, dim=1)[1].to(torch.int32)
    idx[9:12, 0] = torch.arange(3, dtype=torch.int32)          # and some that the choice would not have taken
    return z, idx, torch.randn(N, K, generator=g), torch.randn(N, E, generator=g) * 0.1


def assert_near(got, want, err, rounding):
    tol = rounding * np.abs(want) + err * (1 + rounding) + 2.0 ** -125
    off = np.abs(got - want)
    assert (off <= tol).all(), (off / tol).max()


@pytest.mark.parametrize("renormalize", [False, True])
def test_reference_by_differences(renormalize):
    """Of s(-|z|), which has the slope of s(z) and loses nothing next to 1."""
    z, idx, dw, ds = (v[7:10].double().numpy() for v in cases(torch.float32, 1, E=12, K=3))
    idx = idx.astype(np.int64)
    dz, _ = backward(z, idx, dw, ds, renormalize, 1.5)
    h = 1e-3
    for t in range(3):
        chosen = sigmoid(z[t, idx[t]])
        S = chosen.sum() + X.TINY if renormalize else 1.0
        for e in range(12):
            low = -np.abs(z[t, e:e + 1])
            ds_dz = (sigmoid(low + h) - sigmoid(low - h))[0] / (2 * h)
            dL_ds = float(ds[t, e])  # and the weights' derivatives in s, by the quotient rule
            for k in range(3):
                for j in range(3):
                    if idx[t, j] == e:
                        dw_ds = 1.5 / S * (k == j) - (1.5 * chosen[k] / S ** 2 if renormalize else 0.0)
                        dL_ds += float(dw[t, k]) * dw_ds
            # central differences of an exponential: h^2 / 6 of it, and 2^-52 / h
            assert abs(ds_dz * dL_ds - dz[t, e]) <= 1e-6 * abs(dz[t, e]) + 1e-30


def test_the_bound_sees_a_difference_from_one():
    """s (1 - s) in fp32 is outside the bound from 10 on, and nothing at all from 18 on; e / (1 + e)^2 is inside."""
    z, idx, dw, ds = cases(torch.float32, 2)
    want, err = backward(z.numpy(), idx.numpy(), dw.numpy(), ds.numpy(), False, 1.0)
    s = (1.0 / (1.0 + torch.exp(-z))).numpy()
    e = torch.exp(-z.abs()).numpy()
    r = np.float32(1.0) / (np.float32(1.0) + e)
    g = ds.clone()
    for k in range(idx.shape[1]):
        g.scatter_add_(1, idx[:, k:k + 1].long(), dw[:, k:k + 1])
    g = g.numpy()
    assert s.dtype == r.dtype == np.float32
    assert_near((e * r * r * g).astype(np.float64), want, err, 2.0 ** -24)
    bad = np.abs(s * (np.float32(1.0) - s) * g - want) > 2.0 ** -24 * np.abs(want) + err
    assert bad[8].mean() > 0.9 and ((s * (np.float32(1.0) - s) * g)[8, 40:] == 0).all()


@pytest.fixture(scope="module")
def built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("scores", [False, True])
@pytest.mark.parametrize("E,K", [(96, 6), (1, 1), (40, 32), (61, 5), (256, 8), (300, 7), (1024, 8)])
def test_gradient_of_confident_experts(built, dtype, renormalize, scores, E, K):
    z, idx, dw, ds = cases(dtype, E + K, E=E, K=K) if E > 8 else \
        (torch.linspace(-30, 30, 24)[:, None].to(dtype), torch.zeros(24, 1, dtype=torch.int32), torch.ones(24, 1),
         torch.ones(24, 1))
    ds = ds if scores else None
    got = ep.route_backward(dw.cuda(), z.cuda(), idx.cuda(), score="sigmoid", renormalize=renormalize, scale=2.5,
                            grad_scores=None if ds is None else ds.cuda())
    want, err = backward(z.double().numpy(), idx.numpy(), dw.numpy(), None if ds is None else ds.numpy(), renormalize, 2.5)
    assert got.dtype == dtype
    assert_near(got.double().cpu().numpy(), want, err, 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24)


@pytest.mark.gpu
def test_gradient_of_masked_and_extreme_logits(built):
    """Infinities, a NaN and logits past fp32's exponentials move nothing, whatever their gradient; the others stay right."""
    inf = float("inf")
    z = torch.tensor([[inf, -inf, float("nan"), 300.0, -300.0, 20.0, -20.0, 0.0]], device="cuda")
    idx = torch.tensor([[0, 1, 5, 6]], dtype=torch.int32, device="cuda")
    dw, ds = torch.ones(1, 4, device="cuda"), torch.full((1, 8), 3.0, device="cuda")
    for last in (3.0, inf, float("nan")):
        ds[0, :5] = last
        got = ep.route_backward(dw, z, idx, score="sigmoid", renormalize=False, grad_scores=ds)[0].double().cpu()
        assert (got[:5] == 0).all()
        slope = sigmoid(np.array([20.0, -20.0, 0.0])) * sigmoid(np.array([-20.0, 20.0, 0.0]))
        assert np.allclose(got[5:].numpy(), slope * np.array([4.0, 4.0, 3.0]), rtol=2.0 ** -16, atol=0)
