"""The router and its gradient against their formulas in 64 bits."""
import numpy as np
import pytest
import torch

import combine_ep_get_dispatch_gb300 as ep
import experts_reference as X

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def check(z, topk, bias=None, score="softmax", groups=1, topk_groups=None, group_best=2, renormalize=True, scale=1.0,
          **kw):
    """z, bias: CPU tensors."""
    topk_groups = groups if topk_groups is None else topk_groups
    zd = kw.pop("z_device", None)
    zd = z.cuda() if zd is None else zd
    idx, w, s = ep.route(zd, topk, bias=None if bias is None else bias.cuda(), score=score, groups=groups,
                         topk_groups=topk_groups, group_best=group_best, renormalize=renormalize, scale=scale,
                         return_scores=True, **kw)
    want, ww, ws = X.route(z.double().numpy(), topk, None if bias is None else bias.numpy(), score, groups, topk_groups,
                           group_best, renormalize, scale)
    assert idx.dtype == torch.int32 and np.array_equal(idx.cpu().numpy(), want)
    # a score is off by under 2^-18 of itself, a sum of them too; below fp32's smallest number it is 0
    assert (np.abs(f64(w) - ww) <= 2.0 ** -16 * ww + 2.0 ** -125 * abs(scale)).all()
    assert (np.abs(f64(s) - ws) <= 2.0 ** -17 * ws + 2.0 ** -125).all()
    return idx, w


SHAPES = [  # tokens, experts, topk, groups, topk_groups
    (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (7, 8, 2, 1, 1), (5, 60, 4, 6, 2), (33, 256, 8, 8, 4), (3, 33, 32, 1, 1),
    (64, 128, 6, 4, 1), (2, 1024, 8, 32, 3), (9, 512, 10, 16, 16), (4, 300, 7, 3, 2), (6, 24, 5, 24, 7), (11, 31, 31, 1, 1),
]


@pytest.mark.parametrize("N,E,K,G,kept", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route(N, E, K, G, kept, score, biased, dtype):
    g = torch.Generator().manual_seed(N * E + K)
    z = (torch.randn(N, E, generator=g) * 1.5).to(dtype)
    bias = torch.randn(E, generator=g) * 0.1 if biased else None
    for best in (1, 2):
        check(z, K, bias, score, G, kept, best, renormalize=best == 2, scale=2.5 if biased else 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,kept", [(1, 1), (8, 4)])
def test_choices_closer_than_fp32_can_tell(score, G, kept):
    """Biases that make up for the scores to half an ulp: only 64 bits see the order."""
    g = torch.Generator().manual_seed(5)
    E = 64
    z = (torch.randn(1, E, generator=g) * 1.5).repeat(40, 1)
    bias = torch.from_numpy((0.75 - X.scores(z[0].numpy(), score)).astype(np.float32))
    z += torch.randn(40, E, generator=g) * 1e-7
    check(z, 8, bias, score, G, kept, 2)
    check(z, 8, None, score, G, kept, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,kept", [(40, 1, 1), (256, 8, 4), (300, 3, 2), (512, 1, 1), (1000, 8, 3), (1024, 32, 9)])
@pytest.mark.parametrize("tied", [12, 45])
def test_some_choices_closer_than_fp32_can_tell(score, E, G, kept, tied):
    """Of each token's experts some are the best by far and equal to half an ulp, few enough to compare or too many."""
    g = torch.Generator().manual_seed(E + tied)
    z = (torch.randn(1, E, generator=g) * 0.5).repeat(24, 1)
    bias = torch.randn(E, generator=g) * 0.01
    top = torch.randperm(E, generator=g)[:min(tied, E)]
    bias[top] = torch.from_numpy((3.0 - X.scores(z[0].numpy(), score)).astype(np.float32))[top]
    z += torch.randn(24, E, generator=g) * 1e-7
    check(z, 8, bias, score, G, kept, 2)
    check(z, 32, bias, score, G, kept, 1, renormalize=False)
    check(z.to(torch.bfloat16), 8, bias, score, G, kept, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sums_of_groups_closer_than_fp32_can_tell(score):
    """Groups with the same two best logits in another order, and with neighbours of them."""
    z = torch.full((16, 32), -4.0)
    for t in range(16):
        for g in range(4):
            z[t, 8 * g + (t + g) % 8] = 1.0
            z[t, 8 * g + (t + 3 * g + 1) % 8] = 0.5
        z[t, 8 * (t % 4) + 5] += 2.0 ** -22 * (t % 3)
    check(z, 4, None, score, 4, 2, 2)
    check(z, 4, torch.zeros(32), score, 4, 2, 2)


def test_ties_go_to_the_lower_index():
    z = torch.zeros(3, 70)
    z[1, 1::2] = 1.0
    z[2] = -0.0
    z[2, ::3] = 0.0
    for bias in (None, torch.zeros(70)):
        for score in ("softmax", "sigmoid"):
            idx, _ = check(z, 6, bias, score)
            assert idx[0].tolist() == list(range(6)) and idx[1].tolist() == [1, 3, 5, 7, 9, 11]
            assert idx[2].tolist() == list(range(6))
    check(z[:, :64], 6, torch.zeros(64), "sigmoid", 8, 3)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("G,kept", [(1, 1), (4, 2)])
def test_masked_experts(score, biased, G, kept):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    g = torch.Generator().manual_seed(9)
    z = torch.randn(12, 32, generator=g)
    z[0] = -inf                    # nothing left
    z[1] = nan
    z[2] = low                     # masked by the type's lowest value: still there
    z[3, 3:] = -inf                # fewer than are asked for
    z[4, :30] = low
    z[5, 7] = inf
    z[6, [4, 20]] = inf
    z[7, ::2] = nan
    z[8, :16] = -inf               # whole groups masked
    z[9, 1:] = -inf
    z[10] = -200.0                 # a sigmoid that fp32 rounds to 0
    bias = None
    if biased:
        bias = torch.randn(32, generator=g) * 0.1
        bias[11], bias[12], bias[13] = -inf, nan, inf
    idx, w = check(z, 6, bias, score, G, kept)
    assert (idx[:2] == -1).all() and (w[:2] == 0).all()
    check(z, 6, bias, score, G, kept, 1, renormalize=False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_a_wider_tensor(dtype):
    g = torch.Generator().manual_seed(10)
    wide = (torch.randn(9, 101, generator=g)).to(dtype)
    check(wide[:, 3:67], 5, None, "softmax", 8, 2, z_device=wide.cuda()[:, 3:67])
    check(wide[::2, 1:33], 5, torch.zeros(32), "sigmoid", z_device=wide.cuda()[::2, 1:33])
    check(wide[:1, 1:33], 5, z_device=wide.cuda()[:1, 1:33])


def test_no_tokens_and_given_outputs():
    idx, w = ep.route(torch.empty(0, 16, device="cuda"), 4)
    assert idx.shape == w.shape == (0, 4)
    assert ep.route_backward(w, torch.empty(0, 16, device="cuda"), idx).shape == (0, 16)
    z = torch.randn(5, 16, device="cuda")
    idx, w = torch.empty(5, 3, dtype=torch.int32, device="cuda"), torch.empty(5, 3, device="cuda")
    a, b = ep.route(z, 3, topk_idx=idx, topk_weights=w)
    assert a is idx and b is w and torch.equal(a.long(), z.topk(3)[1])


def test_many_tokens():
    g = torch.Generator().manual_seed(12)
    check(torch.randn(3001, 256, generator=g) * 1.5, 8, torch.randn(256, generator=g) * 0.1, "sigmoid", 8, 4, scale=2.5)


# ---------------------------------------------------------------- gradient --
def check_backward(z, idx, dw, ds, score, renormalize, scale, z_device=None, **kw):
    zd = z.cuda() if z_device is None else z_device
    got = ep.route_backward(dw.cuda(), zd, idx.cuda(), score=score, renormalize=renormalize, scale=scale,
                            grad_scores=None if ds is None else ds.cuda(), **kw)
    want, err = X.route_backward(z.double().numpy(), idx.numpy(), dw.numpy(), None if ds is None else ds.numpy(), score,
                                 renormalize, scale)
    assert got.dtype == z.dtype and got.shape == z.shape
    rounding = 2.0 ** -8 if z.dtype == torch.bfloat16 else 2.0 ** -24
    off = np.abs(f64(got) - want)
    tol = rounding * np.abs(want) + err * (1 + rounding) + 2.0 ** -125
    assert (off <= tol).all(), (off / tol).max()
    return got


@pytest.mark.parametrize("N,E,K,G,kept", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward(N, E, K, G, kept, score, renormalize, dtype):
    g = torch.Generator().manual_seed(N + E + K)
    z = (torch.randn(N, E, generator=g) * 1.5).to(dtype)
    idx = ep.route(z.cuda(), K, score=score, groups=G, topk_groups=kept)[0].cpu()
    dw, ds = torch.randn(N, K, generator=g), torch.randn(N, E, generator=g) * 0.1
    check_backward(z, idx, dw, None, score, renormalize, 2.5)
    check_backward(z, idx, dw, ds, score, renormalize, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_backward_of_missing_repeated_and_bad_indices(score, renormalize):
    g = torch.Generator().manual_seed(3)
    z = torch.randn(5, 40, generator=g)
    idx = torch.tensor([[-1, -1, -1], [3, -1, 39], [7, 7, 1], [40, 2, -2], [0, 1, 2]], dtype=torch.int32)
    dw = torch.randn(5, 3, generator=g)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = check_backward(z, idx, dw, None, score, renormalize, 1.5, status=st)
    assert int(st.item()) == ep.EP_ST_BAD_INDEX and (got[0] == 0).all()
    st.zero_()
    check_backward(z[[0, 1, 2, 4]], idx[[0, 1, 2, 4]], dw[[0, 1, 2, 4]], None, score, renormalize, 1.5, status=st)
    assert int(st.item()) == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_of_masked_logits(score):
    """Masked experts get no gradient, and a NaN no other's."""
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(4)
    z = torch.randn(6, 32, generator=g)
    z[0] = -inf
    z[1, 5:] = -inf
    z[2, ::2] = nan
    z[3] = torch.finfo(torch.float32).min
    z[4, 3] = torch.finfo(torch.float32).min
    idx = ep.route(z.cuda(), 4, score=score)[0].cpu()
    dw, ds = torch.randn(6, 4, generator=g), torch.randn(6, 32, generator=g)
    got = check_backward(z, idx, dw, ds, score, True, 1.0)
    assert torch.isfinite(got).all() and (got[0] == 0).all() and (got[1, 5:] == 0).all() and (got[2, ::2] == 0).all()


def test_backward_of_rows_of_a_wider_tensor():
    g = torch.Generator().manual_seed(6)
    wide = torch.randn(9, 101, generator=g)
    z = wide[::2, 3:67]
    idx = ep.route(z.cuda(), 5)[0].cpu()
    out = torch.full((5, 64), 9.0, device="cuda")
    assert check_backward(z, idx, torch.randn(5, 5, generator=g), None, "softmax", True, 1.0,
                          z_device=wide.cuda()[::2, 3:67], out=out) is out


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_in_a_graph_and_on_another_stream(score):
    g = torch.Generator(device="cuda").manual_seed(7)
    z = torch.randn(50, 96, generator=g, device="cuda")
    bias = torch.randn(96, generator=g, device="cuda") * 0.1
    dw = torch.randn(50, 6, generator=g, device="cuda")
    args = dict(bias=bias, score=score, groups=6, topk_groups=3)
    want = ep.route(z, 6, **args)
    grad = ep.route_backward(dw, z, want[0], score=score)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    made = ep.route(z, 6, **args, stream=side)
    back = ep.route_backward(dw, z, made[0], score=score, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(made[0], want[0]) and torch.equal(made[1], want[1]) and torch.equal(back, grad)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        idx, w = ep.route(z, 6, **args)
        d = ep.route_backward(dw, z, idx, score=score)
    z.copy_(torch.randn(50, 96, generator=g, device="cuda"))
    graph.replay()
    want = ep.route(z, 6, **args)
    assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
    assert torch.equal(d, ep.route_backward(dw, z, idx, score=score))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,kept,K", [(32, 8, 5, 20), (32, 4, 3, 20), (60, 6, 4, 32), (24, 12, 8, 12)])
@pytest.mark.parametrize("best", [1, 2])
def test_groups_whose_biases_add_up_past_fp32(score, E, G, kept, K, best):
    """Biases of the type's lowest and largest values: a sum of two has no fp32, and is none of "no expert is left"."""
    g = torch.Generator().manual_seed(14)
    z, size = torch.randn(16, E, generator=g) * 1.5, E // G
    low, most = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    for value in (low, most, low / 2, most / 2):
        bias = torch.randn(E, generator=g) * 0.1
        bias[size:-size] = value           # all groups but two
        check(z, K, bias, score, G, kept, best)
        bias[::2] *= 0.999                 # and values that differ
        check(z, K, bias, score, G, kept, best)
        bias[:] = value                    # every group
        check(z, K, bias, score, G, kept, best)
    bias[:size], bias[size:] = low, float("-inf")
    check(z, K, bias, score, G, kept, best)
