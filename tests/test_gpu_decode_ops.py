"""Cache append, cache attention and the experts' 4-bit products against their formulas in 64 bits.

Tolerances come from the formats: BF16 results are within half a step (2^-8) of
the value, E4M3 codes are those of the fp32 value (compared as they are), softmax
weights enter their products with 11 bits, sums are fp32 (see
decode_reference). fp16 weights relative to 2^15 have a smallest step of
2^-39 of the largest.
"""
import numpy as np
import pytest
import torch

import combine_ep_get_dispatch_gb300 as ep
import decode_reference as R
from helpers import status_value, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


def new_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rope_table(rows, rot):
    ang = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(rot // 2) * 2.0 / max(rot, 1))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def random_cache(rng, lens, P, KH, D, spare=3, nan_tail=True):
    """Codes of every kind in the tokens held, NaN codes and NaN scales wherever no sequence holds a token."""
    pages = [-(-int(n) // P) for n in lens]
    total = sum(pages) + spare
    ids = rng.permutation(total)
    table = np.full((len(lens), max(pages + [1]) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n]
        at += n
    c = dict(table=table)
    for name in "kv":
        codes = rng.integers(0, 254, (total, KH, P, D))
        codes = np.where(codes >= 127, codes + 1, codes).astype(np.uint8)
        scale = 2.0 ** rng.integers(-9, -5, (total, KH))
        if nan_tail:
            codes[ids[at:]], scale[ids[at:]] = 0x7F, np.nan
            for b, n in enumerate(lens):
                if n % P:
                    codes[table[b, pages[b] - 1], :, n % P:] = 0xFF
        c[name], c[name + "_scale"] = codes, scale.astype(np.float32)
    return c


def device_cache(c):
    return ep.KVCache(*(to_dev(c[n]) for n in ("k", "v", "k_scale", "v_scale", "table")))


# ------------------------------------------------------------------- append --
APPENDS = [
    # D, P, KH, QH, rot, interleaved, [(earlier tokens, new tokens)]
    (128, 64, 8, 16, 128, False, [(1000, 1)]),
    (128, 64, 3, 5, 128, False, [(0, 1), (63, 1), (64, 1), (5, 1)]),
    (64, 16, 2, 2, 64, False, [(0, 1), (15, 1), (16, 1), (31, 1), (40, 1)]),
    (64, 16, 1, 7, 32, True, [(3, 20), (0, 0), (16, 1), (0, 33), (7, 0), (15, 2)]),
    (128, 32, 2, 4, 64, True, [(31, 70), (0, 5)]),
    (128, 128, 4, 4, 16, False, [(100, 300), (0, 129), (127, 1)]),
    (64, 128, 5, 10, 0, False, [(2, 131), (0, 17)]),
    (128, 16, 17, 17, 128, False, [(0, 40)]),
    (128, 64, 1, 2, 128, False, [(10, 15), (60, 20), (0, 12)]),
    (64, 32, 3, 3, 64, True, [(31, 13), (1, 30), (0, 64)]),
    (64, 64, 2, 1, 32, False, [(7, 130)]),
    (64, 16, 64, 1, 64, False, [(15, 3), (0, 0), (16, 1), (5, 11), (31, 2), (14, 5)] * 3),   # few tokens, many heads
    (128, 16, 60, 1, 32, True, [(15, 3), (9, 9), (16, 1), (0, 1), (31, 2), (14, 5)] * 3),
    (64, 16, 2, 2, 64, False, [(9, 90), (0, 17), (30, 3)]),
    (64, 128, 3, 2, 64, True, [(9, 90), (100, 40)]),
    (128, 16, 4, 2, 128, False, [(3, 20), (0, 0), (16, 1), (0, 33), (7, 0), (15, 2)]),   # a warp a block
    (128, 128, 2, 3, 64, True, [(100, 60), (0, 3), (5, 2), (127, 1), (3, 9), (0, 1), (1, 2), (8, 1), (60, 1)]),
    (64, 64, 3, 1, 32, False, [(60, 60), (0, 3), (5, 2), (127, 1), (3, 9), (0, 1), (1, 2), (8, 1), (60, 1)]),
]


@pytest.mark.parametrize("D,P,KH,QH,rot,inter,seqs", APPENDS)
@pytest.mark.parametrize("fused", [False, True])
def test_append(D, P, KH, QH, rot, inter, seqs, fused):
    rng = np.random.default_rng(D + P + len(seqs))
    lens = [s + n for s, n in seqs]
    cu = np.concatenate([[0], np.cumsum([n for _, n in seqs])])
    T = int(cu[-1])
    c = random_cache(rng, lens, P, KH, D)
    # heads whose new values are far above, near and far below what the block holds
    size = 10.0 ** rng.integers(-3, 4, (1, QH + 2 * KH, 1))
    qkv = bf16(rng.normal(size=(T, QH + 2 * KH, D)) * size).cuda()
    q, k, v = qkv[:, :QH], qkv[:, QH:QH + KH], qkv[:, QH + KH:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    rope = rope_table(max(lens), rot) if rot else None
    want = {n: a.copy() for n, a in c.items()}
    hq, hk, hv = (t.float().cpu().numpy() for t in (q, k, v))
    R.append(want, lens, cu, hk, hv, rope, inter)
    cache, st = device_cache(c), new_status()
    one_each = all(n == 1 for _, n in seqs)
    args = dict(cu_tokens=None if one_each else to_dev(cu.astype(np.int32)), interleaved=inter,
                rope=None if rope is None else to_dev(rope), status=st)
    lens_d = to_dev(np.array(lens, np.int32))
    for _ in range(2):  # the second call finds the first one's blocks and changes nothing
        out = ep.kv_append(k, v, cache, lens_d, q=q, **args)
        for name in ("k", "v", "k_scale", "v_scale"):
            assert np.array_equal(getattr(cache, name).cpu().numpy(), want[name], equal_nan=name.endswith("scale")), name
    ref = hq.copy()
    if rot:
        for b, (s, n) in enumerate(seqs):
            for i in range(n):
                ref[cu[b] + i] = R.rotate(hq[cu[b] + i], rope[s + i], inter)
    assert torch.equal(out.cpu(), torch.from_numpy(ref).to(torch.bfloat16))
    assert status_value(st) == 0
    # in place, and against 64 bits: half a step of BF16 and the three fp32 roundings
    ep.kv_append(k, v, cache, lens_d, q=q, q_out=q, **args)
    assert torch.equal(q, out)
    if rot:
        for b, (s, n) in enumerate(seqs):
            for i in range(n):
                x = R.rotate(hq[cu[b] + i], rope[s + i], inter, np.float64)
                top = np.abs(hq[cu[b] + i]).max(1, keepdims=True)
                assert (np.abs(f64(out[cu[b] + i]) - x) <= 2.0 ** -8 * np.abs(x) + 2.0 ** -21 * top).all()


def test_append_keeps_values_within_a_code_of_their_own():
    """Appended one by one, every cached value stays within one E4M3 step at its block's scale of what was appended."""
    rng = np.random.default_rng(3)
    P, KH, D, n = 32, 2, 64, 80
    x = rng.normal(size=(n, KH, D)) * np.exp(0.05 * np.arange(n))[:, None, None]
    x = f64(bf16(x))
    table = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    cache = ep.new_kv_cache(3, KH, P, D, table)
    d = bf16(x).cuda()
    for i in range(n):
        ep.kv_append(d[i:i + 1], d[i:i + 1], cache, torch.tensor([i + 1], dtype=torch.int32, device="cuda"))
    got = R.TABLE[cache.v.cpu().numpy()] * f64(cache.v_scale)[:, :, None, None]
    got = got.transpose(0, 2, 1, 3).reshape(-1, KH, D)[:n]
    scale = f64(cache.v_scale).repeat(P, 0)[:n]
    # each of a block's re-encodings moves a value by at most half a step; steps double from one to the next
    step = np.maximum(2.0 ** (np.floor(np.log2(np.abs(x) + 1e-300)) - 3), scale[:, :, None] * 2.0 ** -9)
    assert (np.abs(got - x) <= step * (1 + 2.0 ** -10)).all()
    assert torch.equal(cache.k, cache.v)


def test_append_of_infinities_and_nan():
    c = dict(k=np.zeros((1, 1, 16, 64), np.uint8), v=np.zeros((1, 1, 16, 64), np.uint8),
             k_scale=np.ones((1, 1), np.float32), v_scale=np.ones((1, 1), np.float32), table=np.zeros((1, 1), np.int32))
    x = np.ones((2, 1, 64))
    x[0, 0, :3], x[1, 0, 63] = (np.inf, -np.inf, np.nan), 7.0
    k = bf16(x).cuda()
    cache = device_cache(c)
    ep.kv_append(k, k, cache, torch.tensor([2], dtype=torch.int32, device="cuda"),
                 cu_tokens=torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
    R.append(c, [2], [0, 2], x.astype(np.float32), x.astype(np.float32), None, False)
    assert c["k_scale"][0, 0] == 2.0 ** -6 and c["k"][0, 0, 0, :3].tolist() == [0x7E, 0xFE, 0x7F]
    assert np.array_equal(cache.k.cpu().numpy(), c["k"]) and np.array_equal(cache.v_scale.cpu().numpy(), c["v_scale"])
    # nothing finite, and zeros: the smallest scale
    z = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    ep.kv_append(z * float("inf"), z, cache, torch.ones(1, dtype=torch.int32, device="cuda"))
    assert cache.v_scale.item() == cache.k_scale.item() == 2.0 ** -100 and not cache.v[0, 0, 0].any()


def append_and_compare(c, lens, cu, T, KH, D, rope, expect, touched, table_ok=True):
    """The given (wrong) call flags `expect` and writes only the sequences in `touched`."""
    rng = np.random.default_rng(5)
    k = rng.normal(size=(T, KH, D)).astype(np.float32)
    k = bf16(k).float().numpy()
    want = {n: a.copy() for n, a in c.items()}
    for b in touched:
        sub = dict(want, table=want["table"][b:b + 1])
        R.append(sub, [lens[b]], [0, cu[b + 1] - cu[b]], k[cu[b]:cu[b + 1]], k[cu[b]:cu[b + 1]], rope, False)
    cache, st = device_cache(c), new_status()
    q = bf16(k).cuda()
    out = torch.full_like(q, 9.0)
    ep.kv_append(q, q, cache, to_dev(np.array(lens, np.int32)), cu_tokens=to_dev(np.array(cu, np.int32)),
                 rope=None if rope is None else to_dev(rope), q=q, q_out=out, status=st)
    assert status_value(st) == expect
    for name in ("k", "v", "k_scale", "v_scale"):
        assert np.array_equal(getattr(cache, name).cpu().numpy(), want[name], equal_nan=name.endswith("scale")), name
    written = np.zeros(T, bool)
    for b in touched:
        written[cu[b]:cu[b + 1]] = True
    if table_ok:
        assert (out[torch.from_numpy(~written)] == 9.0).all()


def test_append_reports_what_it_skips():
    rng = np.random.default_rng(4)
    KH, D, P = 2, 64, 16
    c = random_cache(rng, [20, 40, 9], P, KH, D)
    cu = [0, 4, 10, 13]
    rope = rope_table(64, 64)
    append_and_compare(c, [20, 40, 9], cu, 13, KH, D, rope, 0, [0, 1, 2])
    append_and_compare(c, [3, 40, 9], cu, 13, KH, D, rope, ep.EP_ST_BAD_INDEX, [1, 2])       # shorter than its tokens
    append_and_compare(c, [20, 40, 9], cu, 13, KH, D, rope[:39], ep.EP_ST_BAD_INDEX, [0, 2])  # beyond the table
    append_and_compare(c, [20, 40, 4 * P + 1], cu, 13, KH, D, None, ep.EP_ST_CAPACITY, [0, 1])
    # out of order: sequence 1 ends before it starts, and sequence 2's eleven tokens exceed its length
    append_and_compare(c, [20, 40, 9], [0, 4, 2, 13], 13, KH, D, None, ep.EP_ST_BAD_INDEX, [0])
    for bad in (-1, c["k"].shape[0], 1 << 30):
        t = c["table"].copy()
        t[1, 2] = bad  # the page of positions 32..47: where sequence 1's tokens 34..39 go
        append_and_compare(dict(c, table=t), [20, 40, 9], cu, 13, KH, D, None, ep.EP_ST_BAD_INDEX, [0, 2], False)


def test_append_reports_every_list_out_of_order():
    """Also where the sequence that is out of order has no page of its own in the call."""
    rng = np.random.default_rng(17)
    c = random_cache(rng, [200, 200, 200], 16, 1, 64)
    for cu in ([0, 100, 10, 110], [110, 110, 110, 110], [-5, -5, -5, 0], [0, 111, 111, 111], [500, 2, 3, 4]):
        cache, st = device_cache(c), new_status()
        k = torch.zeros(110, 1, 64, dtype=torch.bfloat16, device="cuda")
        ep.kv_append(k, k, cache, to_dev(np.array([200, 200, 200], np.int32)), cu_tokens=to_dev(np.array(cu, np.int32)),
                     status=st)
        assert status_value(st) == (0 if cu[0] == 110 else ep.EP_ST_BAD_INDEX), cu


def test_append_nothing():
    cache = ep.new_kv_cache(2, 2, 16, 64, torch.zeros((0, 4), dtype=torch.int32, device="cuda"))
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    ep.kv_append(k, k, cache, torch.zeros(0, dtype=torch.int32, device="cuda"), q=k)


# ---------------------------------------------------------------- attention --
ATTENDS = [
    # D, P, KH, QH, [(length, new)], window
    (128, 64, 8, 64, [(1, 1), (64, 1), (65, 1), (1000, 1)], 0),
    (128, 64, 1, 16, [(5000, 1)], 0),
    (64, 16, 2, 2, [(0, 1), (1, 1), (16, 1), (17, 1), (33, 1), (700, 1)], 0),
    (64, 16, 3, 15, [(40, 3), (2, 2), (0, 0), (300, 1), (17, 5)], 0),
    (128, 32, 4, 32, [(333, 4), (4, 4), (2, 4), (900, 4)], 0),   # (2, 4): two tokens before the sequence's start
    (128, 128, 2, 32, [(513, 3), (128, 2)], 0),
    (128, 64, 2, 16, [(200, 70), (64, 64), (600, 9)], 0),
    (64, 32, 1, 1, [(450, 33)], 0),
    (64, 16, 2, 8, [(100, 1), (700, 1), (3, 1)], 50),
    (128, 16, 1, 8, [(100, 40), (450, 3), (9, 9)], 17),
    (128, 64, 2, 10, [(777, 2), (65, 1)], 1),
    (64, 128, 2, 40, [(300, 2), (129, 1)], 0),
    (128, 16, 16, 16, [(130, 1)] * 9, 0),
]


def check_attention(c, lens, cu, q, scale, window, got, lse):
    ref, rl, pv, mag, small = R.attention(c, lens, cu, q, scale, window)
    weight = 2.0 ** -11 + 2.0 ** -19 * mag[..., None]          # of a softmax weight: 11 bits, and its score's error
    tol = 2.0 ** -8 * np.abs(ref) * 1.01 + (weight + 2.0 ** -16) * pv * 1.01 + 2.0 ** -40 * small + 2.0 ** -130
    err = np.abs(f64(got) - ref)
    assert (err <= tol).all(), (err / tol).max()
    if lse is not None:
        l = f64(lse)
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(l), empty)
        e = np.abs(l[~empty] - rl[~empty])
        assert (e <= 2.0 ** -19 * mag[~empty] + 2.0 ** -21 * (np.abs(rl[~empty]) + 16)).all()
        assert not f64(got)[empty].any()


@pytest.mark.parametrize("D,P,KH,QH,seqs,window", ATTENDS)
def test_attention(D, P, KH, QH, seqs, window):
    rng = np.random.default_rng(D * P + QH)
    lens = [n for n, _ in seqs]
    cu = np.concatenate([[0], np.cumsum([n for _, n in seqs])])
    T = int(cu[-1])
    c = random_cache(rng, lens, P, KH, D)
    q = bf16(rng.normal(size=(T, QH, D)) * 10.0 ** rng.integers(-2, 2, (T, QH, 1))).cuda()
    wide = torch.zeros(T, QH + 3, D, dtype=torch.bfloat16, device="cuda")
    wide[:, :QH] = q
    cache, st = device_cache(c), new_status()
    ws = ep.kv_attention_workspace(q, cache)
    one_each = all(n == 1 for _, n in seqs)
    args = dict(cu_tokens=None if one_each else to_dev(cu.astype(np.int32)), scale=0.05, window=window, workspace=ws,
                status=st)
    lens_d = to_dev(np.array(lens, np.int32))
    out, lse = ep.kv_attention(q, cache, lens_d, return_lse=True, **args)
    check_attention(c, lens, cu, f64(q), 0.05, window, out, lse)
    assert status_value(st) == 0
    # the same again from strided queries, without lse, on the used workspace: the same bits
    again = ep.kv_attention(wide[:, :QH], cache, lens_d, **args)
    assert torch.equal(again, out)


@pytest.mark.parametrize("D,P,KH,G,n,window", [(64, 16, 16, 1, 1, 0), (128, 64, 16, 1, 1, 0), (64, 32, 16, 8, 2, 0),
                                               (128, 32, 8, 8, 4, 70), (64, 128, 8, 12, 5, 0)])
def test_attention_of_many_short_sequences(D, P, KH, G, n, window):
    """Several units a block, of one chunk of tokens to ten, in any order."""
    rng = np.random.default_rng(D + P + n)
    seqs = 96 if n == 1 else 40 if n == 2 else 20
    lens = [int(x) for x in np.floor(np.exp(rng.uniform(0, np.log(330), seqs)))]
    c = random_cache(rng, lens, P, KH, D)
    q = bf16(rng.normal(size=(seqs * n, KH * G, D))).cuda()
    cu = np.arange(seqs + 1) * n
    out, lse = ep.kv_attention(q, device_cache(c), to_dev(np.array(lens, np.int32)), cu_tokens=to_dev(cu.astype(np.int32)),
                               scale=0.1, window=window, return_lse=True)
    check_attention(c, lens, cu, f64(q), 0.1, window, out, lse)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_attention_scales(scale):
    rng = np.random.default_rng(8)
    c = random_cache(rng, [150], 32, 1, 64)
    q = bf16(rng.normal(size=(1, 4, 64))).cuda()
    out, lse = ep.kv_attention(q, device_cache(c), torch.tensor([150], dtype=torch.int32, device="cuda"), scale=scale,
                               return_lse=True)
    check_attention(c, [150], [0, 1], f64(q), scale, 0, out, lse)


def test_attention_of_blocks_with_far_apart_scales():
    """Value and key scales that differ by 2^60 from page to page; large and tiny queries."""
    rng = np.random.default_rng(9)
    for ks, vs, qs in ((1, 30, 1.0), (6, 0, 1.0), (0, 30, 1e30), (0, 0, 1e-30)):
        c = random_cache(rng, [200], 16, 2, 128, nan_tail=False)
        c["k_scale"] *= 2.0 ** rng.integers(-ks, ks + 1, c["k_scale"].shape).astype(np.float32)
        c["v_scale"] *= 2.0 ** rng.integers(-vs, vs + 1, c["v_scale"].shape).astype(np.float32)
        q = bf16(rng.normal(size=(1, 8, 128)) * qs).cuda()
        scale = 0.02 / qs
        out, lse = ep.kv_attention(q, device_cache(c), torch.tensor([200], dtype=torch.int32, device="cuda"),
                                   scale=scale, return_lse=True)
        check_attention(c, [200], [0, 1], f64(q), scale, 0, out, lse)


@pytest.mark.parametrize("unseen", [0.0, 2.0 ** -100, 2.0 ** 120, np.inf, np.nan])
def test_attention_never_uses_the_scales_of_pages_it_does_not_see(unseen):
    """Pages of 16 that the window leaves out, the first one of a chunk of tokens that it does not."""
    rng = np.random.default_rng(18)
    lens = [50, 61, 16 * 41 + 9]
    c = random_cache(rng, lens, 16, 2, 64)
    c["v_scale"] *= 2.0 ** 9   # blocks of magnitudes above 448: exponents above zero
    for b, n in enumerate(lens):
        for j in range((n - 10) // 16):
            page = c["table"][b, j]
            c["k"][page] = c["v"][page] = 0x7F
            c["k_scale"][page] = c["v_scale"][page] = unseen
    q = bf16(rng.normal(size=(3, 8, 64))).cuda()
    out, lse = ep.kv_attention(q, device_cache(c), to_dev(np.array(lens, np.int32)), scale=0.1, window=10, return_lse=True)
    check_attention(c, lens, [0, 1, 2, 3], f64(q), 0.1, 10, out, lse)


@pytest.mark.parametrize("first", [True, False])
def test_attention_of_zero_value_blocks_beside_large_ones(first):
    """A block of zeros has the smallest scale, 2^-100; its tokens count in the normaliser as any others."""
    rng = np.random.default_rng(19)
    c = random_cache(rng, [64], 16, 1, 64)
    zeros, large = c["table"][0, :2] if first else c["table"][0, [2, 0]]
    c["v"][zeros], c["v_scale"][zeros] = 0, 2.0 ** -100
    c["v_scale"][large] = 2.0 ** 19   # magnitudes up to 2^28
    q = bf16(rng.normal(size=(1, 4, 64))).cuda()
    out, lse = ep.kv_attention(q, device_cache(c), to_dev(np.array([64], np.int32)), scale=0.05, return_lse=True)
    check_attention(c, [64], [0, 1], f64(q), 0.05, 0, out, lse)


def test_attention_masks_bad_pages_and_reports_them():
    rng = np.random.default_rng(10)
    c = random_cache(rng, [200, 100], 16, 2, 64)
    c["table"][0, 3], c["table"][0, 7], c["table"][1, 0] = -1, 1 << 20, c["k"].shape[0]
    q = bf16(rng.normal(size=(2, 4, 64))).cuda()
    st = new_status()
    out, lse = ep.kv_attention(q, device_cache(c), to_dev(np.array([200, 100], np.int32)), return_lse=True, status=st)
    check_attention(c, [200, 100], [0, 1, 2], f64(q), 64 ** -0.5, 0, out, lse)
    assert status_value(st) == ep.EP_ST_BAD_INDEX
    # every page bad: an empty row
    c["table"][:] = -1
    out, lse = ep.kv_attention(q, device_cache(c), to_dev(np.array([200, 100], np.int32)), return_lse=True, status=st)
    assert torch.isneginf(lse).all() and not out.any()
    # longer than the table holds: the rest is masked
    c = random_cache(rng, [64, 30], 16, 2, 64)
    c["table"] = np.ascontiguousarray(c["table"][:, :3])
    st = new_status()
    out, lse = ep.kv_attention(q, device_cache(c), to_dev(np.array([64, 30], np.int32)), return_lse=True, status=st)
    check_attention(c, [64, 30], [0, 1, 2], f64(q), 64 ** -0.5, 0, out, lse)
    assert status_value(st) == ep.EP_ST_CAPACITY


def test_attention_of_tokens_outside_cu_tokens():
    """A list out of order: flagged; its tokens, and those past the list's end, are empty rows."""
    rng = np.random.default_rng(11)
    c = random_cache(rng, [50, 60, 70], 16, 1, 64)
    q = bf16(rng.normal(size=(9, 2, 64))).cuda()
    st = new_status()
    out, lse = ep.kv_attention(q, device_cache(c), to_dev(np.array([50, 60, 70], np.int32)),
                               cu_tokens=to_dev(np.array([0, 2, 4, 7], np.int32)), return_lse=True, status=st)
    check_attention(c, [50, 60, 70], [0, 2, 4, 7], f64(q)[:7], 0.125, 0, out[:7], lse[:7])
    assert torch.isneginf(lse[7:]).all() and not out[7:].any() and status_value(st) == 0
    for cu in ([0, 2, 1, 7], [0, 2, 4, 99], [-3, 2, 4, 7]):
        st = new_status()
        ep.kv_attention(q, device_cache(c), to_dev(np.array([50, 60, 70], np.int32)),
                        cu_tokens=to_dev(np.array(cu, np.int32)), return_lse=True, status=st)
        assert status_value(st) == ep.EP_ST_BAD_INDEX


def test_cache_offsets_beyond_32_bits():
    """The last pages of a cache of more than 2^32 bytes a side, appended to and read."""
    rng = np.random.default_rng(12)
    P, KH, D = 128, 8, 128
    pages = (1 << 32) // (P * KH * D) + 3
    big = [torch.empty((pages, KH, P, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((pages, KH), dtype=torch.float32, device="cuda") for _ in range(2)]
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    cache = ep.KVCache(*big, *scales, table)
    n = 200
    kv = bf16(rng.normal(size=(n, 2 * KH, D))).cuda()
    lens, cu = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    ep.kv_append(kv[:, :KH], kv[:, KH:], cache, lens, cu_tokens=cu)
    c = dict(k=np.zeros((2, KH, P, D), np.uint8), v=np.zeros((2, KH, P, D), np.uint8),
             k_scale=np.zeros((2, KH), np.float32), v_scale=np.zeros((2, KH), np.float32), table=np.array([[1, 0]]))
    h = kv.float().cpu().numpy()
    R.append(c, [n], [0, n], h[:, :KH], h[:, KH:], None, False)
    assert np.array_equal(cache.k[-2:].cpu().numpy()[1], c["k"][1])
    assert np.array_equal(cache.v[-2:].cpu().numpy()[0][:, :n - P], c["v"][0][:, :n - P])
    q = bf16(rng.normal(size=(2, 16, D))).cuda()
    out, lse = ep.kv_attention(q, cache, lens, cu_tokens=torch.tensor([0, 2], dtype=torch.int32, device="cuda"),
                               return_lse=True)
    check_attention(c, [n], [0, 2], f64(q), D ** -0.5, 0, out, lse)


@pytest.mark.parametrize("D,P,window", [(64, 16, 0), (128, 32, 0), (128, 64, 40)])
def test_attention_keeps_nan_to_the_tokens_that_see_it(D, P, window):
    """NaN codes among the newest tokens (and where a window ends) reach the rows that attend to them, no others."""
    rng = np.random.default_rng(19)
    n, length = 6, 83
    c = random_cache(rng, [length], P, 1, D)
    for at, ch in ((length - 3, 5), (length - 1, 0), (length - n - 38, 17)):
        c["v"][c["table"][0, at // P], 0, at % P, ch] = 0x7F
    c["k"][c["table"][0, (length - 2) // P], 0, (length - 2) % P, 9] = 0xFF
    q = bf16(rng.normal(size=(n, 4, D))).cuda()
    out, lse = ep.kv_attention(q, device_cache(c), torch.tensor([length], dtype=torch.int32, device="cuda"),
                               cu_tokens=torch.tensor([0, n], dtype=torch.int32, device="cuda"), window=window,
                               scale=0.05, return_lse=True)
    with np.errstate(invalid="ignore"):
        ref, rl, *_ = R.attention(c, [length], [0, n], f64(q), 0.05, window)
    assert np.isnan(ref).any() and not np.isnan(ref[0]).all() and np.isnan(rl[-1]).all()
    assert np.array_equal(np.isnan(f64(out)), np.isnan(ref)) and np.array_equal(np.isnan(f64(lse)), np.isnan(rl))
    fine = ~np.isnan(ref)
    assert np.allclose(f64(out)[fine], ref[fine], rtol=2.0 ** -7, atol=2.0 ** -9)


@pytest.mark.parametrize("D,KH,G,n", [(128, 1, 8, 1), (64, 3, 5, 1), (128, 2, 8, 4), (64, 1, 16, 5)])
def test_attention_of_a_long_sequence_over_many_blocks(D, KH, G, n):
    """One sequence whose parts are joined in two levels, against fp64 torch on its dequantised cache."""
    rng = np.random.default_rng(20)
    length, P = 40001, 64
    pages = -(-length // P)
    table = torch.from_numpy(rng.permutation(pages).astype(np.int32))[None].cuda()
    codes = [torch.randint(0, 127, (pages, KH, P, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    for t in codes:
        t |= torch.randint(0, 2, t.shape, dtype=torch.uint8, device="cuda") << 7
    scales = [torch.exp2(torch.randint(-8, -5, (pages, KH), device="cuda").float()) for _ in range(2)]
    cache = ep.KVCache(*codes, *scales, table)
    q = bf16(rng.normal(size=(n, KH * G, D))).cuda()
    args = dict(cu_tokens=torch.tensor([0, n], dtype=torch.int32, device="cuda"), scale=0.02, return_lse=True,
                workspace=ep.kv_attention_workspace(q, cache))
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")
    out, lse = ep.kv_attention(q, cache, lens, **args)
    k, v = (t[table[0].long()].view(torch.float8_e4m3fn).double() * s[table[0].long()].double()[..., None, None]
            for t, s in zip(codes, scales))
    k, v = (x.permute(1, 0, 2, 3).reshape(KH, -1, D)[:, :length] for x in (k, v))
    for i in range(n):
        stop = length - n + i + 1
        sc = torch.einsum("hgd,hjd->hgj", q[i].double().view(KH, G, D), k[:, :stop]) * 0.02
        z = torch.logsumexp(sc, -1)
        w = (sc - z[..., None]).exp()
        ref = torch.einsum("hgj,hjd->hgd", w, v[:, :stop]).reshape(-1, D)
        mag = torch.einsum("hgj,hjd->hgd", w, v[:, :stop].abs()).reshape(-1, D)
        # weights keep 11 bits and scores 2^-19 of at most 64; the result rounds to BF16
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2.0 ** -13) * mag
        assert ((out[i].double() - ref).abs() <= tol * 1.01).all()
        assert ((lse[i].double() - z.reshape(-1)).abs() <= 2.0 ** -13).all()
    for _ in range(3):  # the same bits whichever block comes last
        again, lse2 = ep.kv_attention(q, cache, lens, **args)
        assert torch.equal(again, out) and torch.equal(lse2, lse)


def test_attention_on_another_stream():
    rng = np.random.default_rng(13)
    c = random_cache(rng, [900], 64, 2, 128)
    q = bf16(rng.normal(size=(1, 16, 128))).cuda()
    cache, lens = device_cache(c), torch.tensor([900], dtype=torch.int32, device="cuda")
    want = ep.kv_attention(q, cache, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = ep.kv_attention(q, cache, lens)
    b = ep.kv_attention(q, cache, lens, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


# ------------------------------------------------------------------ experts --
LINEARS = [
    # in, out, rows of each expert, glu
    (128, 8, [1], False),
    (128, 16, [1], True),
    (256, 136, [3, 0, 1], False),
    (384, 72, [2, 9], False),
    (256, 272, [5, 0, 8, 17], True),
    (1152, 200, [64, 1, 65], False),
    (512, 96, [130, 2, 300], True),
    (2048, 128, [1] * 20, False),
    (7168, 256, [4, 0, 1, 33], True),
    (896, 640, [0, 0, 0, 7], False),
    # clusters of two and four blocks, whole and with an idle end; odd numbers of 128 inputs
    (256, 256, [4, 5, 3, 4], False),
    (640, 1168, [9, 2, 0, 7, 12], False),
    (384, 512, [30, 25, 11], True),
    (256, 1024, [130, 40], False),
    (384, 2080, [200, 0, 90, 191, 193], False),
    (896, 528, [150, 100], True),
]


def linear_case(rng, K, M, counts, fp8, regions, spare=2):
    E = len(counts)
    codes = rng.integers(0, 256, (E, M, K // 2)).astype(np.uint8)
    scales = rng.integers(115, 131, (E, M, K // 32)).astype(np.uint8)
    cap = (max(counts) + spare) if regions else 0
    if regions:
        first = np.arange(E) * cap
        total = E * cap
    else:  # segments padded by `spare` rows
        first = np.cumsum([0] + [c + spare for c in counts])
        total = int(first[-1])
    if fp8:
        x = rng.integers(0, 254, (total, K))
        x = np.where(x >= 127, x + 1, x).astype(np.uint8)
        xs = rng.integers(117, 124, (total, K // 128)).astype(np.uint8)
        value = R.TABLE[x] * np.repeat(2.0 ** (xs.astype(float) - 127), 128, axis=1)
        xd, xsd = to_dev(x), to_dev(xs)
    else:
        xd = bf16(rng.normal(size=(total, K)) * np.exp(rng.normal(size=(total, K)) * 2)).cuda()
        value, xsd = f64(xd), None
    if regions:
        xd = xd.view(E, cap, K)
        xsd = None if xsd is None else xsd.view(E, cap, K // 128)
    return codes, scales, first, xd, xsd, value


@pytest.mark.parametrize("K,M,counts,glu", LINEARS)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("regions", [False, True])
def test_expert_linear(K, M, counts, glu, fp8, regions):
    rng = np.random.default_rng(K + M + len(counts))
    codes, scales, first, x, xs, value = linear_case(rng, K, M, counts, fp8, regions)
    outs = M // 2 if glu else M
    y = torch.full((*x.shape[:-1], outs), 77.0, dtype=torch.bfloat16, device="cuda")
    st = new_status()
    w, ws_ = to_dev(codes), to_dev(scales)
    work = ep.expert_linear_workspace(x, w, max_rows=sum(counts))
    args = dict(row_count=to_dev(np.array(counts, np.int32)),
                row_offset=None if regions else to_dev(first.astype(np.int32)), x_scale=xs, glu=glu,
                max_rows=sum(counts), workspace=work, status=st)
    ep.expert_linear(x, w, ws_, out=y, **args)
    got = f64(y).reshape(-1, outs)
    received = np.zeros(got.shape[0], bool)
    for e, n in enumerate(counts):
        if n == 0:
            continue
        rows = slice(first[e], first[e] + n)
        received[rows] = True
        ref, err = R.expert_product(value[rows], R.weights(codes[e], scales[e]), glu)
        tol = (2.0 ** -8 * np.abs(ref) + err) * 1.01 + 2.0 ** -130
        off = np.abs(got[rows] - ref)
        assert (off <= tol).all(), (e, (off / tol).max())
    assert (got[~received] == 77.0).all()
    assert status_value(st) == 0
    first_y = y.clone()
    ep.expert_linear(x, w, ws_, out=y, **args)  # the used workspace: the same bits
    assert torch.equal(y, first_y)


def test_expert_linear_reads_bf16_rows_to_the_last_bit():
    """Rows with one nonzero, times a power-of-two weight: every BF16 value comes back as it is."""
    bits = np.arange(1 << 15, dtype=np.uint32)
    v = (bits << 16).view(np.float32)
    v = v[np.isfinite(v) & ((v >= 2.0 ** -100) | (v == 0))][:: 7]
    v = v[v < 2.0 ** 100]
    n, K = v.size, 128
    x = np.zeros((n, K), np.float32)
    x[np.arange(n), np.arange(n) % K] = v * np.where(np.arange(n) % 2, 1, -1)
    codes = np.full((1, 8, K // 2), 0x22, np.uint8)  # ones
    y = ep.expert_linear(bf16(x).cuda(), to_dev(codes), to_dev(np.full((1, 8, K // 32), 127, np.uint8)),
                         torch.tensor([n], dtype=torch.int32, device="cuda"),
                         row_offset=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert np.array_equal(f64(y), np.repeat(x.sum(1, keepdims=True), 8, 1).astype(np.float64))


def test_expert_linear_of_infinities_and_nan():
    """A row with an infinity or a NaN gives no finite output; its neighbours are as they were."""
    rng = np.random.default_rng(14)
    codes, scales, first, x, _, value = linear_case(rng, 256, 24, [6], False, False)
    codes |= 0x11  # no zero weights
    args = dict(row_count=torch.tensor([6], dtype=torch.int32, device="cuda"), row_offset=to_dev(first[:1].astype(np.int32)))
    want = ep.expert_linear(x, to_dev(codes), to_dev(scales), **args)[:6]
    x[1, 5], x[4, 200], x[4, 3] = float("nan"), float("inf"), float("-inf")
    got = ep.expert_linear(x, to_dev(codes), to_dev(scales), **args)[:6]
    assert not torch.isfinite(got[[1, 4]]).any()
    keep = [0, 2, 3, 5]
    assert torch.equal(got[keep], want[keep])


def test_expert_linear_reports_rows_it_skips():
    rng = np.random.default_rng(15)
    codes, scales, first, x, _, value = linear_case(rng, 256, 24, [4, 4], False, True, spare=0)
    w, s = to_dev(codes), to_dev(scales)
    y = torch.full((2, 4, 24), 5.0, dtype=torch.bfloat16, device="cuda")
    want = ep.expert_linear(x, w, s, to_dev(np.array([4, 4], np.int32)))

    def run(counts, **kw):
        st = new_status()
        y.fill_(5.0)
        ep.expert_linear(kw.pop("x", x), w, s, to_dev(np.array(counts, np.int32)), out=kw.pop("out", y), status=st, **kw)
        return status_value(st)

    assert run([9, 2]) == ep.EP_ST_CAPACITY                 # more than a region holds
    assert torch.equal(y[0], want[0]) and torch.equal(y[1, :2], want[1, :2]) and (y[1, 2:] == 5.0).all()
    flat = x.view(8, -1)
    out = y.view(8, -1)
    assert run([4, 4], x=flat, out=out, row_offset=to_dev(np.array([0, 6], np.int32))) == ep.EP_ST_CAPACITY
    assert torch.equal(y[0], want[0])
    assert run([4, 4], max_rows=5) == ep.EP_ST_CAPACITY     # more than max_rows in all
    assert torch.equal(y[0], want[0])
    assert run([-3, 2]) == 0
    assert (y[0] == 5.0).all() and torch.equal(y[1, :2], want[1, :2])
    assert run([0, 0]) == 0 and (y == 5.0).all()


def test_expert_linear_weights_beyond_32_bits():
    """An expert whose weights start past 2^32 bytes."""
    rng = np.random.default_rng(16)
    E, M, K = 150, 8192, 7168
    w = torch.empty((E, M, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, M, K // 32), dtype=torch.uint8, device="cuda")
    codes = rng.integers(0, 256, (M, K // 2)).astype(np.uint8)
    scales = rng.integers(118, 124, (M, K // 32)).astype(np.uint8)
    w[-1], s[-1] = to_dev(codes), to_dev(scales)
    x = bf16(rng.normal(size=(3, K))).cuda()
    count = torch.zeros(E, dtype=torch.int32, device="cuda")
    count[-1] = 3
    y = ep.expert_linear(x, w, s, count, row_offset=torch.zeros(E, dtype=torch.int32, device="cuda"))
    at = rng.choice(M, 64, replace=False)
    ref, err = R.expert_product(f64(x), R.weights(codes[at], scales[at]), False)
    assert (np.abs(f64(y)[:, at] - ref) <= (2.0 ** -8 * np.abs(ref) + err) * 1.01).all()


def test_expert_linear_in_a_graph_and_on_another_stream():
    rng = np.random.default_rng(17)
    codes, scales, first, x, _, _ = linear_case(rng, 512, 64, [3, 1, 20], False, False)
    w, s, off = to_dev(codes), to_dev(scales), to_dev(first.astype(np.int32))
    n = to_dev(np.array([3, 1, 20], np.int32))
    work = ep.expert_linear_workspace(x, w)
    want = ep.expert_linear(x, w, s, n, off, workspace=work)
    y = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ep.expert_linear(x, w, s, n, off, out=y, workspace=work)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ep.expert_linear(x, w, s, n, off, out=y, workspace=work)
    rows = torch.cat([torch.arange(f, f + c) for f, c in zip(first, [3, 1, 20])]).cuda()
    y.zero_()
    graph.replay()
    assert torch.equal(y[rows], want[rows])
    x.mul_(2.0)
    graph.replay()
    assert torch.equal(y[rows], want[rows] * 2)
