"""The decode-step operators around the dispatch, as cases to measure.

Three operators: appending keys and values to a paged E4M3 cache with the
position rotation on the way, attention over that cache, and the experts'
products with 4-bit weights. ``run`` computes a case either in its plain form
(elementary torch operations in 32 bits, rounded once at the end) or, where
``own`` is true, by the calls a user makes of the package.

Lengths and expert loads are spread by rule and only permuted by the seed, so
that ``work`` knows them; values come from the seed alone.
"""
import math
import random

import numpy as np
import torch

own = False

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
MIN_SCALE = 2.0 ** -100  # smallest scale of a cache block


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one request's decode step: a single token, bound by latency
        dict(name="append_one", op="append", seqs=1, new=1, ragged=False, context=1000, q_heads=64, kv_heads=8,
             dim=128, rot=128, interleaved=False, page=64),
        # a decode batch of requests of all ages
        dict(name="append_decode", op="append", seqs=256, new=1, ragged=True, context=700, q_heads=64, kv_heads=8,
             dim=128, rot=128, interleaved=False, page=64),
        # a few prompts of very different lengths entering at once
        dict(name="append_prompts", op="append", seqs=5, new=9000, ragged=True, context=0, q_heads=32, kv_heads=4,
             dim=128, rot=128, interleaved=False, page=128),
        # drafted tokens of many requests; small heads, partial rotation of interleaved pairs, small pages
        dict(name="append_drafts", op="append", seqs=33, new=9, ragged=True, context=300, q_heads=16, kv_heads=16,
             dim=64, rot=32, interleaved=True, page=16),
        # the large decode batch: the cache read bounds everything
        dict(name="attend_decode", op="attend", seqs=128, new=1, ragged=False, context=8192, q_heads=64, kv_heads=8,
             dim=128, page=64, window=0),
        # one long document: a single row of work to split over the whole GPU
        dict(name="attend_long", op="attend", seqs=1, new=1, ragged=False, context=131072, q_heads=64, kv_heads=4,
             dim=128, page=64, window=0),
        # verifying four drafted tokens for requests of mixed lengths
        dict(name="attend_verify", op="attend", seqs=24, new=4, ragged=True, context=30011, q_heads=32, kv_heads=4,
             dim=128, page=32, window=0),
        # short chats, one query head a cache head, a sliding window: latency counts
        dict(name="attend_chats", op="attend", seqs=48, new=1, ragged=True, context=700, q_heads=16, kv_heads=16,
             dim=64, page=16, window=512),
        # one token's eight experts: a matrix-vector product each
        dict(name="experts_one_token", op="experts", tokens=1, topk=8, experts=256, inner=7168, outer=4096, glu=True,
             fp8=False, regions=False),
        # the 128-token decode batch, gate and up projections of every expert
        dict(name="experts_up", op="experts", tokens=128, topk=8, experts=256, inner=7168, outer=4096, glu=True,
             fp8=False, regions=False),
        # the same batch's down projection, in the low-latency receive regions
        dict(name="experts_down", op="experts", tokens=128, topk=8, experts=256, inner=2048, outer=7168, glu=False,
             fp8=False, regions=True),
        # the 4096-token FP8 batch: about 128 rows an expert, the largest
        dict(name="experts_fp8", op="experts", tokens=4096, topk=8, experts=256, inner=7168, outer=4096, glu=True,
             fp8=True, regions=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["append", "attend", "experts"])
    if op == "experts":
        fp8 = rng.random() < 0.35
        experts = rng.choice([1, 8, 60, 128, 256])
        topk = 1 if experts == 1 else rng.choice([1, 2, 6, 8])
        most = max(1, experts * (100 if fp8 else 12) // topk)
        glu = rng.random() < 0.5
        return dict(op=op, tokens=_log(rng, 1, min(2048, most)), topk=topk, experts=experts,
                    inner=rng.choice([128 * _log(rng, 2, 20), 896 * _log(rng, 1, 8)]),
                    outer=16 * _log(rng, 30, 190) if glu else 8 * _log(rng, 30, 250), glu=glu, fp8=fp8,
                    regions=rng.random() < 0.5)
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = dict(q_heads=kv_heads * rng.choice([1, 2, 4, 5, 8, 16 if kv_heads < 16 else 4]), kv_heads=kv_heads,
                 dim=dim, page=rng.choice([16, 32, 64, 128]))
    if op == "append":
        seqs = _log(rng, 1, 200)
        return dict(op=op, seqs=seqs, new=_log(rng, 1, max(1, 8000 // seqs)), ragged=rng.random() < 0.7,
                    context=rng.choice([0, _log(rng, 1, 1000)]), rot=rng.choice([16, 32, 64, dim]),
                    interleaved=rng.random() < 0.4, **heads)
    seqs = _log(rng, 1, 200)
    return dict(op=op, seqs=seqs, new=rng.choice([1, 1, 1, 2, 3, 5]), ragged=rng.random() < 0.7,
                context=_log(rng, 8, min(131072, 4000000 // (seqs * kv_heads))), **heads,
                window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]))


def _spread(case):
    """Context lengths and new tokens of the sequences, before the seed's permutation."""
    B = case["seqs"]
    at = np.linspace(0.0, 1.0, B) if B > 1 else np.ones(1)
    ctx = np.full(B, case["context"], dtype=np.int64)
    new = np.full(B, case["new"], dtype=np.int64)
    if case["ragged"]:
        ctx = np.floor(np.exp(at * math.log(case["context"] + 1.0)) - 0.5).astype(np.int64)
        if case["op"] == "append":
            new = np.maximum(1, np.floor(np.exp(at[::-1] * math.log(case["new"] + 0.5)))).astype(np.int64)
    if case["op"] == "attend":  # the context holds the new tokens
        ctx = np.maximum(ctx, new)
    return ctx, new


def _loads(case):
    """Rows of each expert, before the seed's permutation."""
    r = np.random.RandomState(11)
    E, K = case["experts"], case["topk"]
    picks = np.argsort(r.random_sample((case["tokens"], E)) if case["tokens"] * E < 1 << 22
                       else r.standard_normal((case["tokens"], E)).astype(np.float32), axis=1)[:, :K]
    return np.bincount(picks.reshape(-1), minlength=E).astype(np.int64)


def work(case):
    if case["op"] == "experts":
        n = _loads(case)
        rows, active = int(n.sum()), int((n > 0).sum())
        M, K = case["outer"], case["inner"]
        x = K + K // 128 if case["fp8"] else 2 * K
        return {"bytes": active * (M * K // 2 + M * K // 32) + rows * x + rows * (M // 2 if case["glu"] else M) * 2
                + 8 * case["experts"], "flops": 2 * rows * M * K}
    ctx, new = _spread(case)
    D, QH, KH = case["dim"], case["q_heads"], case["kv_heads"]
    T = int(new.sum())
    if case["op"] == "append":
        return {"bytes": T * ((2 * QH + KH * 2) * D * 2 + KH * 2 * D + case["rot"] * 4 + 8), "flops": T * (QH + KH) * D * 3}
    seen = ctx if not case["window"] else np.minimum(ctx, case["window"] + new - 1)
    rows = int((seen * new).sum())
    return {"bytes": int(seen.sum()) * KH * 2 * D + T * QH * D * 4 + 4 * QH * T, "flops": 4 * rows * QH * D}


# -------------------------------------------------------------------- inputs
def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _e4m3(v):
    """fp32 -> E4M3 bytes, to nearest even, saturating."""
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _value(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float32)


def _ue8m0(b):
    """UE8M0 bytes (not 0) -> the powers of two they stand for."""
    return (b.to(torch.int32) << 23).view(torch.float32)


def _pow2_above(v):
    """The smallest power of two that is not below v > 0."""
    m, e = torch.frexp(v)
    return torch.ldexp(torch.ones_like(v), e - (m == 0.5).to(e.dtype))


def prepare(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 17)
    perm = np.random.RandomState(seed % (1 << 31))

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def ints(a):
        return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)

    if case["op"] == "experts":
        n = perm.permutation(_loads(case))
        E, M, K, rows = case["experts"], case["outer"], case["inner"], int(n.sum())
        s = {"case": case,
             "codes": torch.randint(0, 256, (E, M, K // 2), generator=g, device=dev, dtype=torch.uint8),
             "scales": torch.randint(117, 122, (E, M, K // 32), generator=g, device=dev, dtype=torch.uint8),
             "count": ints(n)}
        cap = -(-int(n.max()) // 8) * 8 if case["regions"] else 0
        off = np.concatenate([[0], np.cumsum(n)])
        s["offset"] = None if cap else ints(off)
        # what a dispatch knows of each row: its expert, and its place among that expert's rows
        expert = np.repeat(np.arange(E), n)
        place = np.arange(rows) - off[:-1][expert]
        s["at"] = torch.tensor(expert * cap + place if cap else np.arange(rows), device=dev)
        active = np.flatnonzero(n)
        s["active"] = torch.tensor(active, device=dev)
        s["row_expert"] = torch.tensor(np.searchsorted(active, expert), device=dev)
        s["row_place"] = torch.tensor(place, device=dev)
        s["most"] = int(n.max())
        total = E * cap if cap else rows
        x = torch.zeros(total, K, dtype=torch.bfloat16, device=dev)
        x[s["at"]] = (normal(rows, K) * torch.exp(0.5 * normal(rows, 1))).to(torch.bfloat16)
        s["x_scale"] = None
        if case["fp8"]:  # as the FP8 dispatch delivers rows, with one scale byte for 128 channels
            b = x.float().view(total, K // 128, 128)
            sc = _pow2_above((b.abs().amax(2) / 448.0).clamp_min(2.0 ** -120))
            s["x_scale"] = (torch.frexp(sc)[1] + 126).to(torch.uint8)
            x = _e4m3(b / sc[..., None]).view(total, K)
        s["x"] = x
        shape = (total, M // 2 if case["glu"] else M)
        s["out"] = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
        if cap:
            s["x"] = s["x"].view(E, cap, K)
            s["x_scale"] = None if s["x_scale"] is None else s["x_scale"].view(E, cap, K // 128)
            s["out"] = s["out"].view(E, cap, shape[1])
        return s

    ctx, new = _spread(case)
    order = perm.permutation(len(ctx))
    ctx, new = ctx[order], new[order]
    length = ctx + new if case["op"] == "append" else ctx
    B, P, D, QH, KH = case["seqs"], case["page"], case["dim"], case["q_heads"], case["kv_heads"]
    T = int(new.sum())
    pages = -(-length // P)
    total = int(pages.sum())
    most = int(pages.max())
    ids = perm.permutation(total)  # pages of a sequence lie anywhere in the cache
    table = np.full((B, most), -1, dtype=np.int64)
    col = np.arange(total) - np.repeat(np.cumsum(pages) - pages, pages)
    table[np.repeat(np.arange(B), pages), col] = ids
    cu = np.concatenate([[0], np.cumsum(new)])
    s = {"case": case, "page_table": ints(table), "seq_lens": ints(length), "most": int(length.max()),
         "cu": None if case["new"] == 1 else ints(cu)}
    # what earlier tokens left in the cache: codes that reach near the top of the range, scales a power of two
    for name in "kv":
        v = normal(total, KH, P, D) if total * KH * P * D < 1 << 27 else None
        if v is None:  # large caches: bytes of both signs, exponents up to the largest (bits 0x7F and 0xFF are NaN)
            c = torch.randint(0, 254, (total, KH, P, D), generator=g, device=dev, dtype=torch.uint8)
            c = torch.where(c >= 127, c + 1, c)
            s[name] = c
        else:
            s[name] = _e4m3(v * 100.0)
        s[name + "_scale"] = torch.ldexp(torch.ones(total, KH, device=dev),
                                         torch.randint(-7, -4, (total, KH), generator=g, device=dev).to(torch.int32))
    if case["op"] == "append":
        qkv = (normal(T, QH + 2 * KH, D) * 1.5).to(torch.bfloat16)  # one fused projection's output
        s["q"], s["new_k"], s["new_v"] = qkv[:, :QH], qkv[:, QH:QH + KH], qkv[:, QH + KH:]
        at = torch.arange(s["most"], device=dev, dtype=torch.float64)
        angle = at[:, None] * 10000.0 ** (-2.0 * torch.arange(case["rot"] // 2, device=dev, dtype=torch.float64) / case["rot"])
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
        s["q_out"] = torch.empty(T, QH, D, dtype=torch.bfloat16, device=dev)
        return s
    s["q"] = normal(T, QH, D).to(torch.bfloat16)
    s["sm_scale"] = 1.0 / math.sqrt(D) / 4.0
    return s


# ----------------------------------------------------------------- own calls
def _run_own(s):
    import combine_ep_get_dispatch_gb300 as ep

    case = s["case"]
    if case["op"] == "experts":
        if "ws" not in s:
            s["ws"] = ep.expert_linear_workspace(s["x"], s["codes"], max_rows=s["at"].numel())
        return ep.expert_linear(s["x"], s["codes"], s["scales"], s["count"], s["offset"], x_scale=s["x_scale"],
                                glu=case["glu"], out=s["out"], max_rows=s["at"].numel(), workspace=s["ws"])
    if "cache" not in s:
        s["cache"] = ep.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["page_table"])
    cache = s["cache"]
    if case["op"] == "append":
        q = ep.kv_append(s["new_k"], s["new_v"], cache, s["seq_lens"], cu_tokens=s["cu"], rope=s["rope"], q=s["q"],
                         q_out=s["q_out"], interleaved=case["interleaved"])
        return {"q": q, "k": cache.k.view(torch.float8_e4m3fn), "v": cache.v.view(torch.float8_e4m3fn),
                "k_scale": cache.k_scale, "v_scale": cache.v_scale}
    if "ws" not in s:
        s["ws"] = ep.kv_attention_workspace(s["q"], cache)
    out, lse = ep.kv_attention(s["q"], cache, s["seq_lens"], cu_tokens=s["cu"], scale=s["sm_scale"],
                               window=case["window"], return_lse=True, workspace=s["ws"])
    return {"out": out, "lse": lse}


# --------------------------------------------------------------- plain forms
def _places(s, T):
    """Sequence and position of each new token."""
    lens = s["seq_lens"].long()
    i = torch.arange(T, device=lens.device)
    if s["cu"] is None:
        return i, lens - 1
    cu = s["cu"].long()
    b = torch.searchsorted(cu, i, right=True) - 1
    return b, lens[b] - cu[b + 1] + i


def _rotate(x, rope, pos, interleaved):
    h = rope.shape[1] // 2
    c, sn = rope[pos, None, :h], rope[pos, None, h:]
    x = x.to(torch.float32)
    head, rest = x[..., :2 * h], x[..., 2 * h:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        return torch.cat([torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2), rest], -1)
    a, b = head[..., :h], head[..., h:]
    return torch.cat([a * c - b * sn, b * c + a * sn, rest], -1)


def _plain_append(s):
    case = s["case"]
    T, P = s["q"].shape[0], case["page"]
    b, pos = _places(s, T)
    lens = s["seq_lens"].long()
    page = s["page_table"].long()[b, pos // P]
    start = lens - (1 if s["cu"] is None else (s["cu"][1:] - s["cu"][:-1]).long())  # earlier tokens of a sequence
    first = s["page_table"].long().gather(1, (start // P)[:, None])[:, 0]           # the page that may hold some
    held = torch.arange(P, device=b.device) < (start % P)[:, None]                  # its earlier rows
    q = _rotate(s["q"], s["rope"], pos, case["interleaved"]).to(torch.bfloat16)
    ks = [_rotate(s["new_k"], s["rope"], pos, case["interleaved"]), s["new_v"].to(torch.float32)]
    s["k"], s["k_scale"] = _plain_blocks(s["k"], s["k_scale"], ks[0], page, pos % P, first, held)
    s["v"], s["v_scale"] = _plain_blocks(s["v"], s["v_scale"], ks[1], page, pos % P, first, held)
    return {"q": q, "k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_blocks(codes, scale, x, page, row, first, held):
    KH = codes.shape[1]
    amax = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    most = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand(-1, KH), amax, "amax")
    need = torch.where(most > 0, _pow2_above((most / 448.0).clamp_min(MIN_SCALE)), MIN_SCALE)
    keep = held.any(1)
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=scale.device)
    touched[page] = True
    old = scale
    kept = torch.zeros_like(scale)
    kept[first] = torch.where(keep[:, None], scale[first], 0.0)
    scale = torch.where(touched[:, None], torch.maximum(need, kept), scale)
    before = codes[first]
    again = _e4m3(_value(before) * (old[first] / scale[first])[..., None, None])
    codes[first] = torch.where(held[:, None, :, None], again, before)
    codes[page, :, row] = _e4m3(x / scale[page][..., None])
    return codes, scale


def _plain_attend(s):
    case = s["case"]
    T, QH, D = s["q"].shape
    KH, P = case["kv_heads"], case["page"]
    B, n = case["seqs"], case["new"]
    pages = s["page_table"].long().clamp_min(0)
    q = s["q"].to(torch.float32).view(B, n, KH, QH // KH, D)
    k = _value(s["k"][pages]) * s["k_scale"][pages][..., None, None]   # [B, pages, KH, P, D]
    k = k.permute(0, 2, 1, 3, 4).reshape(B, KH, -1, D)
    rows = q.permute(0, 2, 1, 3, 4).reshape(B, KH, -1, D)
    sc = (rows @ k.transpose(2, 3) * s["sm_scale"]).view(B, KH, n, QH // KH, -1)
    del k
    j = torch.arange(sc.shape[-1], device=sc.device)
    pos = s["seq_lens"].long()[:, None] - n + torch.arange(n, device=sc.device)      # [B, n]
    seen = j <= pos[..., None]
    if case["window"]:
        seen = seen & (j > pos[..., None] - case["window"])
    sc = sc.masked_fill(~seen[:, None, :, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = (sc - top).exp()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0]
    v = _value(s["v"][pages]) * s["v_scale"][pages][..., None, None]
    v = v.permute(0, 2, 1, 3, 4).reshape(B, KH, -1, D)
    out = (p.view(B, KH, -1, p.shape[-1]) @ v).view(B, KH, n, QH // KH, D) / total
    out = out.permute(0, 2, 1, 3, 4).reshape(T, QH, D).to(torch.bfloat16)
    return {"out": out, "lse": lse.permute(0, 2, 1, 3).reshape(T, QH)}


def _plain_experts(s):
    case = s["case"]
    K = case["inner"]
    pairs = torch.tensor(E2M1, device=s["count"].device)
    pairs = torch.stack([pairs.repeat(16), pairs.repeat_interleave(16)], 1)        # byte -> (low, high)
    codes, scales = s["codes"][s["active"]], s["scales"][s["active"]]
    A, M = codes.shape[:2]
    w = pairs.index_select(0, codes.view(-1).to(torch.int32)).view(A, M, K // 32, 32)
    w *= _ue8m0(scales)[..., None]
    w = w.view(A, M, K)
    x = s["x"].reshape(-1, K)[s["at"]]
    if case["fp8"]:
        sc = _ue8m0(s["x_scale"].reshape(-1, K // 128)[s["at"]])
        x = (_value(x).view(-1, K // 128, 128) * sc[..., None]).view(-1, K)
    padded = torch.zeros(A, s["most"], K, device=w.device)
    padded[s["row_expert"], s["row_place"]] = x.to(torch.float32)
    y = (padded @ w.transpose(1, 2))[s["row_expert"], s["row_place"]]
    if case["glu"]:
        g, u = y[:, :M // 2], y[:, M // 2:]
        y = g / (1.0 + (-g).exp()) * u
    s["out"].view(-1, y.shape[1])[s["at"]] = y.to(torch.bfloat16)
    return s["out"]


def run(state):
    if own:
        return _run_own(state)
    return {"append": _plain_append, "attend": _plain_attend, "experts": _plain_experts}[state["case"]["op"]](state)


# --------------------------------------------------------- values in 64 bits
def _nearest_e4m3(v):
    """float64 -> the nearest E4M3 value (ties to even), saturating."""
    e = (torch.frexp(v.abs().clamp_min(2.0 ** -20))[1] - 1).to(v.dtype)
    step = torch.exp2(e.clamp_min(-6.0) - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    dev = _dev()
    if case["op"] == "experts":
        K, M = case["inner"], case["outer"]
        half = torch.tensor(E2M1, dtype=torch.float64, device=dev)
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=dev).view(-1, s["out"].shape[-1])
        x = s["x"].reshape(-1, K)
        for a, e in enumerate(s["active"].tolist()):
            c = s["codes"][e].long()
            w = torch.empty(M, K, dtype=torch.float64, device=dev)
            w[:, 0::2], w[:, 1::2] = half[c & 15], half[c >> 4]
            w = w * torch.exp2(s["scales"][e].double() - 127.0).repeat_interleave(32, 1)
            at = s["at"][s["row_expert"] == a]
            r = x[at]
            if case["fp8"]:
                r = r.view(torch.float8_e4m3fn).double() * torch.exp2(
                    s["x_scale"].reshape(-1, K // 128)[at].double() - 127.0).repeat_interleave(128, 1)
            y = r.double() @ w.t()
            if case["glu"]:
                y = torch.sigmoid(y[:, :M // 2]) * y[:, :M // 2] * y[:, M // 2:]
            out[at] = y
        return out.view(s["out"].shape)
    P, D, KH = case["page"], case["dim"], case["kv_heads"]
    lens = s["seq_lens"].tolist()
    cu = list(range(len(lens) + 1)) if s["cu"] is None else s["cu"].tolist()
    table = s["page_table"].tolist()
    if case["op"] == "append":
        h = case["rot"] // 2

        def turn(x, p0, p1):
            x = x.double()
            c, sn = s["rope"][p0:p1, None, :h].double(), s["rope"][p0:p1, None, h:].double()
            y = x.clone()
            ia = torch.arange(h, device=dev) * 2 if case["interleaved"] else torch.arange(h, device=dev)
            ib = ia + 1 if case["interleaved"] else ia + h
            y[..., ia] = x[..., ia] * c - x[..., ib] * sn
            y[..., ib] = x[..., ib] * c + x[..., ia] * sn
            return y

        q = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
        res = {"q": q}
        for name in "kv":
            res[name] = s[name].view(torch.float8_e4m3fn).double()
            res[name + "_scale"] = s[name + "_scale"].double()
        for b, length in enumerate(lens):
            n = cu[b + 1] - cu[b]
            p0 = length - n
            rows = slice(cu[b], cu[b + 1])
            q[rows] = turn(s["q"][rows], p0, length)
            new = {"k": turn(s["new_k"][rows], p0, length), "v": s["new_v"][rows].double()}
            for blk in range(p0 // P, (length - 1) // P + 1):
                page, lo = table[b][blk], max(p0, blk * P)
                hi = min(length, blk * P + P)
                for name in "kv":
                    x = new[name][lo - p0:hi - p0].permute(1, 0, 2)                # [KH, rows, D]
                    need = (x.abs().amax((1, 2)) / 448.0).clamp_min(MIN_SCALE)
                    m, ex = torch.frexp(need)                                      # a power of two has m = 0.5
                    need = torch.exp2((ex - (m == 0.5).to(ex.dtype)).double())
                    codes, sc = res[name][page], res[name + "_scale"][page]
                    held = lo - blk * P
                    if held:
                        need = torch.maximum(need, sc)
                        codes[:, :held] = _nearest_e4m3(codes[:, :held] * (sc / need)[:, None, None])
                    codes[:, held:held + hi - lo] = _nearest_e4m3(x / need[:, None, None])
                    res[name + "_scale"][page] = need
        return res
    T, QH, _ = s["q"].shape
    out = torch.zeros(T, QH, D, dtype=torch.float64, device=dev)
    lse = torch.full((T, QH), -math.inf, dtype=torch.float64, device=dev)
    for b, length in enumerate(lens):
        n = cu[b + 1] - cu[b]
        ids = torch.tensor(table[b][:-(-length // P)], device=dev)
        kv = []
        for name in "kv":
            x = s[name][ids].view(torch.float8_e4m3fn).double() * s[name + "_scale"][ids].double()[..., None, None]
            kv.append(x.permute(1, 0, 2, 3).reshape(KH, -1, D)[:, :length])
        for i in range(n):
            last = length - n + i
            lo = max(0, last + 1 - case["window"]) if case["window"] else 0
            k, v = (x[:, lo:last + 1] for x in kv)
            sc = torch.einsum("hgd,hjd->hgj", s["q"][cu[b] + i].double().view(KH, -1, D), k) * s["sm_scale"]
            z = torch.logsumexp(sc, -1)
            lse[cu[b] + i] = z.reshape(-1)
            out[cu[b] + i] = torch.einsum("hgj,hjd->hgd", torch.exp(sc - z[..., None]), v).reshape(QH, D)
    return {"out": out, "lse": lse}
