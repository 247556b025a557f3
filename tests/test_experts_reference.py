"""The references of the router and the 8-bit experts, against closed forms and differences."""
import numpy as np
import pytest

import experts_reference as X


def test_scores_of_known_logits():
    z = np.array([np.log(1.0), np.log(2.0), np.log(5.0)])
    assert np.allclose(X.scores(z, "softmax"), [1 / 8, 2 / 8, 5 / 8])
    assert np.allclose(X.scores(z, "sigmoid"), [1 / 2, 2 / 3, 5 / 6])
    with np.errstate(invalid="ignore"):
        assert np.allclose(X.scores(np.array([np.inf, 0.0, np.inf]), "softmax"), [0.5, 0, 0.5])
        assert np.allclose(X.scores(np.array([np.nan, 0.0, -np.inf]), "softmax"), [0, 1, 0])
        assert (X.scores(np.array([-np.inf] * 2), "softmax") == 0).all()


def test_choice_by_groups_and_bias():
    z = np.array([[3.0, -9.0, 2.0, 2.0, 1.0, 0.9, 0.0, 2.9]])
    # best single experts: groups 0, 1 (tie of 2.0s behind), 3; best pairs: 1, 3, 2
    one = X.route(z, 2, None, "sigmoid", 4, 2, 1, True, 1.0)[0]
    assert one.tolist() == [[0, 7]]
    two = X.route(z, 2, None, "sigmoid", 4, 1, 2, True, 1.0)[0]
    assert two.tolist() == [[2, 3]]
    idx, w, s = X.route(z, 8, np.array([0, 5.0, 0, 0, 0, 0, 0, -np.inf]), "sigmoid", 1, 1, 2, False, 2.0)
    assert idx.tolist() == [[1, 0, 2, 3, 4, 5, 6, -1]] and w[0, -1] == 0 and np.allclose(w[0, 0], 2 * s[0, 1])


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_by_differences(kind, renormalize):
    rng = np.random.default_rng(1)
    z = rng.normal(size=(2, 9))
    idx = np.array([[3, 0, 8], [5, -1, 5]])
    dw, ds = rng.normal(size=(2, 3)), rng.normal(size=(2, 9))

    def loss(z):
        total = 0.0
        for t in range(2):
            on = idx[t] >= 0
            total += (dw[t][on] * X.weights_of(z[t], idx[t][on], kind, renormalize, 1.5)).sum()
            total += (ds[t] * X.scores(z[t], kind)).sum()
        return total
    dz, _ = X.route_backward(z, idx, dw, ds, kind, renormalize, 1.5)
    h = 1e-5
    for t in range(2):
        for e in range(9):
            up, down = z.copy(), z.copy()
            up[t, e] += h
            down[t, e] -= h
            # central differences: h^2 of the third derivative (under 10), and rounding over h
            assert abs((loss(up) - loss(down)) / (2 * h) - dz[t, e]) < 1e-8


def test_blocks_of_scales():
    s = np.arange(6.0).reshape(3, 2)
    b = X.blocks(s, 300, 200)
    assert b.shape == (300, 200) and b[0, 0] == 0 and b[127, 128] == 1 and b[128, 0] == 2 and b[299, 199] == 5
    b = X.blocks(np.arange(4.0).reshape(4, 1), 2 * 136, 128, parts=2)  # each half starts a block of its own
    assert b[135, 0] == 1 and b[136, 0] == 2 and b[136 + 128, 0] == 3


def test_a_products_bound_holds_for_fp32_sums():
    rng = np.random.default_rng(2)
    x, w = rng.normal(size=(5, 256)).astype(np.float32), rng.normal(size=(8, 256)).astype(np.float32)
    y, err = X.product(x.astype(np.float64), w.astype(np.float64), False)
    assert (np.abs(x @ w.T - y) <= err).all()
    X.check_bf16(y * (1 + 2.0 ** -8), y, err)
    with pytest.raises(AssertionError):
        X.check_bf16(y * (1 + 2.0 ** -6), y, err)
