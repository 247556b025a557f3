"""The decode step's operators in 64 bits, from their formulas (numpy, loops)."""
import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_table() -> np.ndarray:
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(float) - 10))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


TABLE = e4m3_table()
_POS = TABLE[:127]  # 0 .. 448, ascending


def e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest code (ties to the even code), saturating; NaN -> 0x7F."""
    a = np.minimum(np.abs(np.asarray(v, dtype=np.float64)), 448.0)
    nan = np.isnan(a)
    a = np.where(nan, 0.0, a)
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = code | np.where(np.signbit(v), 128, 0)
    return np.where(nan, 127, code).astype(np.uint8)


def pow2_above(v: float) -> float:
    m, e = np.frexp(v)
    return float(2.0 ** (e - 1) if m == 0.5 else 2.0 ** e)


def block_scale(x: np.ndarray) -> float:
    """x fp32: the smallest power of two >= fl(amax / 448) of the finite values, at least 2^-100."""
    a = np.abs(x[np.isfinite(x)])
    amax = np.float32(a.max() if a.size else 0.0)
    return pow2_above(max(float(np.float32(amax / np.float32(448.0))), 2.0 ** -100))


def rotate(x: np.ndarray, row: np.ndarray, interleaved: bool, dtype=np.float32) -> np.ndarray:
    """x [heads, D]; row [rot]: cosines then sines. In fp32 every product and sum is rounded on its own."""
    y = x.astype(dtype)
    rot = row.shape[0]
    h = rot // 2
    c, s = row[:h].astype(dtype), row[h:].astype(dtype)
    ia = np.arange(h) * 2 if interleaved else np.arange(h)
    ib = ia + 1 if interleaved else ia + h
    a, b = y[:, ia].copy(), y[:, ib].copy()
    with np.errstate(invalid="ignore"):
        y[:, ia] = a * c - b * s
        y[:, ib] = b * c + a * s
    return y


def append(cache: dict, lens, cu, k, v, rope, interleaved) -> None:
    """cache: k, v codes [pages, KH, P, D], k_scale, v_scale [pages, KH], table; changed in place."""
    P = cache["k"].shape[2]
    for b, length in enumerate(lens):
        n = cu[b + 1] - cu[b]
        start = length - n
        if n == 0:
            continue
        for j in range(start // P, (length - 1) // P + 1):
            page = cache["table"][b, j]
            lo, hi = max(start, j * P), min(length, (j + 1) * P)
            held = lo - j * P
            rows = range(cu[b] + lo - start, cu[b] + hi - start)
            for name, src in (("k", k), ("v", v)):
                new = np.stack([rotate(src[t], rope[start + t - cu[b]], interleaved)
                                if name == "k" and rope is not None else src[t] for t in rows], 1)  # [KH, rows, D]
                for h in range(new.shape[0]):
                    s = block_scale(new[h])
                    codes, old = cache[name][page, h], float(cache[name + "_scale"][page, h])
                    if held:
                        s = max(s, old)
                        if s > old:
                            codes[:held] = e4m3(TABLE[codes[:held]] * (old / s))
                    codes[held:held + hi - lo] = e4m3(new[h].astype(np.float64) / s)
                    cache[name + "_scale"][page, h] = s


def attention(cache: dict, lens, cu, q, scale, window):
    """out, lse and what bounds their errors.

    For each row: sum_j p_j |v_j|; max_j scale sum |q k_j|; and the largest p_j
    times its value block's scale, times the sum of the value codes'
    magnitudes, which 2^-40 of is what weights too small for fp16 can lose.
    """
    T, QH, D = q.shape
    P, KH = cache["k"].shape[2], cache["k"].shape[1]
    G = QH // KH
    out, lse = np.zeros((T, QH, D)), np.full((T, QH), -np.inf)
    pv, mag, small = np.zeros((T, QH, D)), np.zeros((T, QH)), np.zeros((T, QH, D))
    pages = cache["k"].shape[0]
    for b, length in enumerate(lens):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            last = length - n + i
            lo = max(0, last + 1 - window) if window else 0
            js = [j for j in range(lo, min(last + 1, cache["table"].shape[1] * P))
                  if 0 <= cache["table"][b, j // P] < pages]
            if not js:
                continue
            js = np.array(js)
            page = cache["table"][b, js // P]
            for h in range(QH):
                k = TABLE[cache["k"][page, h // G, js % P]] * cache["k_scale"][page, h // G][:, None]
                v = TABLE[cache["v"][page, h // G, js % P]] * cache["v_scale"][page, h // G][:, None]
                qq = q[cu[b] + i, h].astype(np.float64)
                s = scale * (k @ qq)
                m = s.max()
                e = np.exp(s - m)
                p = e / e.sum()
                out[cu[b] + i, h] = p @ v
                lse[cu[b] + i, h] = m + np.log(e.sum())
                pv[cu[b] + i, h] = p @ np.abs(v)
                vs = cache["v_scale"][page, h // G].astype(np.float64)
                small[cu[b] + i, h] = (p * vs).max() * (np.abs(v) / vs[:, None]).sum(0)
                mag[cu[b] + i, h] = abs(scale) * np.max(np.abs(k) @ np.abs(qq) + 2.0 ** -4 * np.abs(k).sum(1) * np.abs(qq).max())
    return out, lse, pv, mag, small


def weights(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """[out, in/2] codes and [out, in/32] UE8M0 bytes -> [out, in] values."""
    w = np.empty((codes.shape[0], codes.shape[1] * 2))
    w[:, 0::2], w[:, 1::2] = E2M1[codes & 15], E2M1[codes >> 4]
    return w * np.repeat(2.0 ** (scales.astype(float) - 127), 32, axis=1)


def expert_product(x: np.ndarray, w: np.ndarray, glu: bool):
    """y and a bound of its error before the rounding to BF16, for x [rows, in], w [out, in].

    Sums are fp32: at most in / 32 + 8 partial sums of relative error 2^-22
    each, of sum |x w|. A BF16 x enters with an error of at most 2^-22 of the
    largest magnitude among its 32 neighbours.
    """
    y = x @ w.T
    top = np.abs(x).reshape(x.shape[0], -1, 32).max(2).repeat(32, axis=1)
    err = (x.shape[1] / 32 + 8) * 2.0 ** -22 * (np.abs(x) @ np.abs(w).T) + 2.0 ** -22 * (top @ np.abs(w).T)
    if not glu:
        return y, err
    h = y.shape[1] // 2
    g, u, eg, eu = y[:, :h], y[:, h:], err[:, :h], err[:, h:]
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    # |silu'| < 1.1; the exponential and the division cost a few 2^-23
    return silu * u, 1.1 * eg * (np.abs(u) + eu) + (np.abs(silu) + 1.1 * eg) * eu + 2.0 ** -20 * np.abs(silu * u)
