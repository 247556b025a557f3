"""The router and the 8-bit experts in 64 bits, from their formulas (numpy, loops)."""
import numpy as np

import decode_reference as R

TINY = float(np.float32(1e-20))


# ------------------------------------------------------------------ router --
def scores(z: np.ndarray, kind: str) -> np.ndarray:
    """One token's scores; a NaN scores 0 and has no part in the softmax."""
    z = z.astype(np.float64)
    ok = ~np.isnan(z)
    s = np.zeros(z.shape)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            s[ok] = 1.0 / (1.0 + np.exp(-z[ok]))
            return s
        top = z[ok].max() if ok.any() else -np.inf
        if top == -np.inf:
            return s
        e = np.where(z[ok] == top, 1.0, np.exp(np.where(z[ok] == top, 0.0, z[ok] - top)))
    s[ok] = e / e.sum()
    return s


def route(z, topk, bias, kind, groups, topk_groups, best, renormalize, scale):
    """(indices, weights, scores) of tokens z [N, E] (any float type)."""
    N, E = z.shape
    size = E // groups
    idx, w, all_s = np.full((N, topk), -1), np.zeros((N, topk)), np.zeros((N, E))
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    for t in range(N):
        zt = z[t].astype(np.float64)
        s = scores(zt, kind)
        all_s[t] = s
        can = (zt > -np.inf) & (b > -np.inf)
        c = np.where(can, s + b, -np.inf)
        key = c if bias is not None else np.where(can, zt, -np.inf)  # without a bias the logits order as the scores do
        if topk_groups < groups:
            of = []
            for g in range(groups):
                v = (c if best == 2 or bias is not None else key)[g * size:(g + 1) * size]
                v = np.sort(v[v > -np.inf])[::-1][:best]
                of.append(v.sum() if v.size else -np.inf)
            keep = [g for g in sorted(range(groups), key=lambda g: (-of[g], g))[:topk_groups] if of[g] > -np.inf]
            for e in range(E):
                if e // size not in keep:
                    key = key.copy()
                    key[e] = -np.inf
        order = sorted(np.flatnonzero(key > -np.inf), key=lambda e: (-key[e], e))[:topk]
        idx[t, :len(order)] = order
        v = s[order]
        w[t, :len(order)] = scale * (v / (v.sum() + TINY) if renormalize else v)
    return idx, w, all_s


def weights_of(z, idx, kind, renormalize, scale):
    """Differentiable part alone: the weights of a given choice, for one token."""
    s = scores(z, kind)[idx]
    return scale * (s / (s.sum() + TINY) if renormalize else s)


def route_backward(z, idx, dw, ds, kind, renormalize, scale):
    """(dz, bound of what fp32 scores and sums can be off) for tokens z [N, E]."""
    N, E = z.shape
    dz, mag = np.zeros((N, E)), np.zeros((N, E))
    for t in range(N):
        s = scores(z[t], kind)
        g = np.zeros(E) if ds is None else ds[t].astype(np.float64).copy()
        size = np.abs(g)
        on = [k for k in range(idx.shape[1]) if 0 <= idx[t, k] < E]
        S = s[idx[t, on]].sum() + TINY if renormalize else 1.0
        d = dw[t].astype(np.float64)
        mean = (d[on] * s[idx[t, on]]).sum() / S if renormalize else 0.0
        spread = (np.abs(d[on]) * s[idx[t, on]]).sum() / S if renormalize else 0.0
        for k in on:
            g[idx[t, k]] += scale / S * (d[k] - mean)
            size[idx[t, k]] += abs(scale) / S * (abs(d[k]) + spread)
        if kind == "sigmoid":
            dz[t], mag[t] = s * (1 - s) * g, s * size
        else:
            dz[t], mag[t] = s * (g - (s * g).sum()), s * (size + (s * size).sum())
    # A score is off by under 2^-18 of itself (an exponential of 2 ulp, its argument rounded, sums of up to 37
    # steps, a division); a gradient has three such factors and two more sums.
    return dz, 2.0 ** -16 * mag


# ----------------------------------------------------------------- experts --
def blocks(scale: np.ndarray, rows: int, cols: int, parts: int = 1) -> np.ndarray:
    """Scales of 128 x 128 blocks -> one for each of [rows, cols]; `parts` of the rows have blocks of their own."""
    half = rows // parts
    s = scale.reshape(parts, -1, scale.shape[1]).repeat(128, axis=1)[:, :half].reshape(rows, -1)
    return s.repeat(128, axis=1)[:, :cols]


def product(x, w, glu):
    """y [rows, out] of x [rows, in], w [out, in] (values), and a bound of its error before it is rounded.

    Products of E4M3 values are exact; a step's four sums and what joins the
    steps are fp32: under in / 32 + 8 sums of relative error 2^-22, of sum |x w|.
    """
    y = x @ w.T
    err = (x.shape[1] / 32 + 8) * 2.0 ** -22 * (np.abs(x) @ np.abs(w).T)
    if not glu:
        return y, err
    h = y.shape[1] // 2
    g, u, eg, eu = y[:, :h], y[:, h:], err[:, :h], err[:, h:]
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    # |silu'| < 1.1; the exponential and the division cost a few 2^-23
    return silu * u, 1.1 * eg * (np.abs(u) + eu) + (np.abs(silu) + 1.1 * eg) * eu + 2.0 ** -20 * np.abs(silu * u)


def check_bf16(got, y, err):
    tol = (2.0 ** -8 * np.abs(y) + err) * 1.01 + 2.0 ** -130
    off = np.abs(got - y)
    assert (off <= tol).all(), (off / tol).max()


def check_fp8(codes, scale, y, err, power_of_two):
    """E4M3 rows and their scales against values y known within err."""
    rows, n = y.shape
    b, e = y.reshape(rows, -1, 128), err.reshape(rows, -1, 128)
    top, slack = np.abs(b).max(2), e.max(2)
    lo, hi = np.maximum(top - slack, 0) / 448 * (1 - 2.0 ** -22), (top + slack) / 448 * (1 + 2.0 ** -22)
    if power_of_two:
        assert (np.frexp(scale[scale > 0])[0] == 0.5).all()
        hi = hi * 2
    assert ((lo <= scale) & (scale <= hi)).all()
    s = scale[..., None]
    got = R.TABLE[codes].reshape(rows, -1, 128) * s
    # half a step of the code, relative to the value, or of the finest step
    tol = (2.0 ** -4 * (np.abs(b) + e) + e + 2.0 ** -10 * s) * 1.01
    off = np.abs(got - b)
    assert (off <= tol).all(), (off / tol).max()
