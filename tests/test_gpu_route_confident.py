"""The router's gradient where one expert has nearly all of a token, against the formula in 64 bits.

A score next to 1 is alone in its sums: ds_i - sum_j s_j ds_j and dw_k - sum_j w'_j dw_j
are then differences of nearly equal numbers. As sums over the others,
sum_j s_j (ds_i - ds_j), they lose nothing, and the bound here is made of those.
"""
import numpy as np
import pytest
import torch

import combine_ep_get_dispatch_gb300 as ep
import experts_reference as X


def parts(z, kind):
    """Scores and slopes of one token; both small where they are."""
    z = z.astype(np.float64)
    s = X.scores(z, kind)
    with np.errstate(over="ignore"):
        return s, s / (1.0 + np.exp(z))  # (the slope of a sigmoid)


def backward(z, idx, dw, ds, kind, renormalize, scale):
    """(dz, bound of fp32's error) of tokens z [N, E]."""
    N, E = z.shape
    dz, err = np.zeros((N, E)), np.zeros((N, E))
    for t in range(N):
        s, slope = parts(z[t], kind)
        g = np.zeros(E) if ds is None else ds[t].astype(np.float64).copy()
        size, d, c = np.abs(g), dw[t].astype(np.float64), s[idx[t]]
        S = c.sum() + X.TINY if renormalize else 1.0
        for k, e in enumerate(idx[t]):
            if renormalize:  # dw_k - sum_j w'_j dw_j, of which sum_j w'_j falls short of 1 by 1e-20 / S
                v = (c / S * (d[k] - d)).sum() + d[k] * (X.TINY / S)
                m = np.delete(c / S * (abs(d[k]) + np.abs(d)), k).sum() + abs(d[k]) * (X.TINY / S)
            else:
                v, m = d[k], abs(d[k])
            g[e] += scale / S * v
            size[e] += abs(scale) / S * m
        if kind == "sigmoid":
            dz[t], err[t] = slope * g, slope * size
        else:
            dz[t] = s * (s * (g[:, None] - g)).sum(1)
            pairs = s * (size[:, None] + size)
            np.fill_diagonal(pairs, 0.0)
            err[t] = s * pairs.sum(1)
    # As for any logits (experts_reference): scores off by under 2^-18 of themselves (arguments up to 60 apart
    # among it), three of them in a term, and two sums.
    return dz, 2.0 ** -16 * err


def cases(dtype, seed, N=26, E=96, K=6):
    """Tokens whose best expert is ahead by 0 to 25, at any place among the chosen."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(N, E, generator=g)
    best = torch.randint(0, E, (N,), generator=g)
    z[torch.arange(N), best] = z.amax(1) + torch.linspace(0.0, 25.0, N)
    z = z.to(dtype)
    idx = z.float().topk(K, dim=1)[1]
    idx = idx.gather(1, torch.rand(N, K, generator=g).argsort(1)).to(torch.int32)
    return z, idx, torch.randn(N, K, generator=g), torch.randn(N, E, generator=g) * 0.1


def assert_near(got, want, err, rounding):
    tol = rounding * np.abs(want) + err * (1 + rounding) + 2.0 ** -125
    off = np.abs(got - want)
    assert (off <= tol).all(), (off / tol).max()


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_reference_is_the_formula(kind, renormalize):
    """Where nothing cancels, what experts_reference says; and everywhere the softmax's gradients add up to nothing."""
    z, idx, dw, ds = (v.numpy() for v in cases(torch.float32, 1, E=20, K=4))
    dz, err = backward(z, idx, dw, ds, kind, renormalize, 1.5)
    want, slack = X.route_backward(z, idx, dw, ds, kind, renormalize, 1.5)
    assert np.allclose(dz[:4], want[:4], rtol=1e-11, atol=1e-14)
    assert (np.abs(dz - want) <= 2.0 ** -30 * slack + 1e-300).all()
    assert (err <= slack * (1 + 1e-9) + 1e-300).all() or kind == "softmax"  # no wider a bound than that
    if kind == "softmax":
        assert (np.abs(dz.sum(1)) <= 1e-15 * np.abs(dz).sum(1) + 1e-16).all()


@pytest.mark.parametrize("renormalize", [False, True])
def test_the_bound_sees_a_difference_of_equal_numbers(renormalize):
    """The formula as written, in fp32, is outside for tokens that are sure."""
    z, idx, dw, ds = cases(torch.float32, 2)
    want, err = backward(z.numpy(), idx.numpy(), dw.numpy(), ds.numpy(), "softmax", renormalize, 1.0)
    s = torch.softmax(z, 1)
    at = idx.long()
    c = s.gather(1, at)
    d = dw
    if renormalize:
        S = c.sum(1, keepdim=True) + 1e-20
        d = (dw - (dw * c / S).sum(1, keepdim=True)) / S
    g = ds.scatter_add(1, at, d)
    plain = s * (g - (s * g).sum(1, keepdim=True))
    off = np.abs(plain.double().numpy() - want) - (2.0 ** -24 * np.abs(want) + err)
    assert (off.max(1) > 0)[16:].mean() > 0.7


@pytest.fixture(scope="module")
def built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("scores", [False, True])
@pytest.mark.parametrize("E,K", [(96, 6), (2, 1), (40, 32), (61, 5), (256, 8), (300, 7), (1024, 8)])
def test_gradient_of_tokens_that_are_sure(built, dtype, kind, renormalize, scores, E, K):
    z, idx, dw, ds = cases(dtype, E + K, E=E, K=K)
    ds = ds if scores else None
    got = ep.route_backward(dw.cuda(), z.cuda(), idx.cuda(), score=kind, renormalize=renormalize, scale=2.5,
                            grad_scores=None if ds is None else ds.cuda())
    want, err = backward(z.double().numpy(), idx.numpy(), dw.numpy(), None if ds is None else ds.numpy(), kind,
                         renormalize, 2.5)
    assert_near(got.double().cpu().numpy(), want, err, 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("spread", [0.01, 0.3])
@pytest.mark.parametrize("E,K", [(448, 4), (992, 3), (1024, 9)])
def test_gradient_of_tokens_that_are_sure_of_nothing(built, dtype, kind, renormalize, spread, E, K):
    """Scores of a thousandth, and a few large gradients among zeros: those stay as near to 0 as they are."""
    g = torch.Generator().manual_seed(E + K)
    N = 40
    z = (torch.randn(N, E, generator=g) * spread).to(dtype)
    idx = torch.rand(N, E, generator=g).argsort(1)[:, :K].to(torch.int32)
    idx[:20, 0] = z[:20].float().argmax(1)     # the best among the chosen, twice where it was
    dw = torch.randn(N, K, generator=g)
    got = ep.route_backward(dw.cuda(), z.cuda(), idx.cuda(), score=kind, renormalize=renormalize)
    want, err = backward(z.double().numpy(), idx.numpy(), dw.numpy(), None, kind, renormalize, 1.0)
    assert_near(got.double().cpu().numpy(), want, err, 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24)
