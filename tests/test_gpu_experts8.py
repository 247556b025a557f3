"""The experts' products with 8-bit weights, and their gradient, against their formulas in 64 bits."""
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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def new_status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def codes_of(rng, *shape):
    c = rng.integers(0, 254, shape)
    return np.where(c >= 127, c + 1, c).astype(np.uint8)  # every code but the NaNs


class Case:
    """Random rows, weights and scales of experts with these counts, and their values."""

    def __init__(self, seed, K, M, counts, regions=False, ue8m0=False, glu=False, transposed=False, spare=2):
        rng = np.random.default_rng(seed)
        E = len(counts)
        self.counts, self.glu, self.transposed, self.outs = counts, glu, transposed, M // 2 if glu else M
        parts = 2 if glu else 1
        shape = (E, K, M) if transposed else (E, M, K)
        grid = (E, K // 128, M // 128) if transposed else (E, parts * -(-(M // parts) // 128), K // 128)
        w, ws = codes_of(rng, *shape), np.exp(rng.normal(size=grid) * 2 - 12).astype(np.float32)
        if regions:
            cap = max(counts) + spare
            self.first, total = np.arange(E) * cap, E * cap
        else:
            self.first = np.cumsum([0] + [c + spare for c in counts])
            total = int(self.first[-1])
        x = codes_of(rng, total, K)
        if ue8m0:
            xs = rng.integers(115, 125, (total, K // 128)).astype(np.uint8)
            xv = 2.0 ** (xs.astype(float) - 127)
        else:
            xs = np.exp(rng.normal(size=(total, K // 128)) - 6).astype(np.float32)
            xv = xs.astype(np.float64)
        self.value = R.TABLE[x] * xv.repeat(128, axis=1)
        self.weights = [R.TABLE[w[e]] * X.blocks(ws[e].astype(np.float64), *shape[1:], parts) for e in range(E)]
        if transposed:
            self.weights = [v.T for v in self.weights]
        self.w, self.ws, self.x, self.xs = dev(w), dev(ws), dev(x), dev(xs)
        self.total, self.row_count = total, ints(counts)
        self.row_offset = None if regions else ints(self.first.tolist())
        if regions:
            self.x, self.xs = self.x.view(E, cap, K), self.xs.view(E, cap, K // 128)

    def run(self, **kw):
        args = dict(row_offset=self.row_offset, max_rows=sum(self.counts)) | kw
        count = args.pop("row_count", self.row_count)
        x, xs = args.pop("x", self.x), args.pop("x_scale", self.xs)
        if self.transposed:
            return ep.expert_linear_fp8_backward(x, xs, self.w, self.ws, count, **args)
        return ep.expert_linear_fp8(x, xs, self.w, self.ws, count, glu=self.glu, **args)

    def rows(self):
        """(expert, its rows) of those that have any."""
        return [(e, slice(f, f + n)) for e, (f, n) in enumerate(zip(self.first, self.counts)) if n]

    def expect(self, e, rows):
        return X.product(self.value[rows], self.weights[e], self.glu)

    def received(self):
        r = np.zeros(self.total, bool)
        for _, rows in self.rows():
            r[rows] = True
        return r


SHAPES = [
    # in, out, rows of each expert, glu
    (128, 8, [1], False),
    (128, 16, [1], True),
    (256, 136, [3, 0, 1], False),
    (384, 72, [2, 9], False),
    (256, 272, [5, 0, 8, 17], True),
    (640, 304, [31, 1, 0, 33], True),
    (1152, 200, [64, 1, 65], False),
    (512, 96, [130, 2, 300], True),
    (2048, 128, [1] * 20, False),
    (7168, 256, [4, 0, 1, 33], True),
    (896, 640, [0, 0, 0, 7], False),
    (384, 2080, [200, 0, 90, 191, 193], False),
    (256, 1032, [128, 129, 127, 256], False),
    (128, 4096, [260, 1], True),
]


@pytest.mark.parametrize("K,M,counts,glu", SHAPES)
@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("regions", [False, True])
def test_product(K, M, counts, glu, ue8m0, regions):
    c = Case(K + M, K, M, counts, regions, ue8m0, glu)
    st = new_status()
    y = torch.full((*c.x.shape[:-1], c.outs), 77.0, dtype=torch.bfloat16, device="cuda")
    ws = ep.expert_linear_fp8_workspace(c.x, c.w, max_rows=sum(counts))
    c.run(out=y, workspace=ws, status=st)
    got = f64(y).reshape(-1, c.outs)
    for e, rows in c.rows():
        X.check_bf16(got[rows], *c.expect(e, rows))
    assert (got[~c.received()] == 77.0).all()
    assert int(st.item()) == 0
    first = y.clone()
    c.run(out=y, workspace=ws)  # the used workspace: the same bits
    assert torch.equal(y, first)


FP8_SHAPES = [
    (128, 128, [1], False),
    (128, 256, [3, 2], True),
    (384, 384, [5, 0, 40], False),
    (640, 768, [130, 2, 17], True),
    (7168, 512, [1] * 8, True),
    (256, 1280, [300, 129], False),
    (384, 768, [300, 131, 0, 250], True),
]


@pytest.mark.parametrize("K,M,counts,glu", FP8_SHAPES)
@pytest.mark.parametrize("form", ["fp32", "round", "ue8m0"])
@pytest.mark.parametrize("regions", [False, True])
def test_product_in_fp8(K, M, counts, glu, form, regions):
    c = Case(K + M + 1, K, M, counts, regions, False, glu)
    st = new_status()
    lead = c.x.shape[:-1]
    out = torch.full((*lead, c.outs), 0x11, dtype=torch.uint8, device="cuda")
    scale = torch.full((*lead, c.outs // 128), 3, dtype=torch.uint8 if form == "ue8m0" else torch.float32, device="cuda")
    y, s = c.run(use_fp8=True, round_scale=form == "round", use_ue8m0=form == "ue8m0", out=out, out_scale=scale, status=st)
    assert y is out and s is scale and int(st.item()) == 0
    codes, s = y.cpu().numpy().reshape(c.total, -1), s.cpu().numpy().reshape(c.total, -1)
    value = 2.0 ** (s.astype(float) - 127) if form == "ue8m0" else s.astype(np.float64)
    for e, rows in c.rows():
        X.check_fp8(codes[rows], value[rows], *c.expect(e, rows), form != "fp32")
    rest = ~c.received()
    assert (codes[rest] == 0x11).all() and (s[rest] == 3).all()


BACK = [
    (128, 128, [1]),
    (256, 384, [3, 0, 1]),
    (640, 128, [33, 64, 2]),
    (384, 896, [130, 2, 300]),
    (7168, 256, [4, 0, 1, 33]),
    (1024, 2048, [1] * 12),
]


@pytest.mark.parametrize("M,K,counts", BACK)
@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("regions", [False, True])
def test_gradient(M, K, counts, ue8m0, regions):
    """M outputs' gradients against a product's formula with the weights transposed."""
    c = Case(M + K + 2, M, K, counts, regions, ue8m0, transposed=True)
    st = new_status()
    y = torch.full((*c.x.shape[:-1], c.outs), 77.0, dtype=torch.bfloat16, device="cuda")
    assert c.run(out=y, status=st) is y
    got = f64(y).reshape(-1, c.outs)
    for e, rows in c.rows():
        X.check_bf16(got[rows], *c.expect(e, rows))
    assert (got[~c.received()] == 77.0).all() and int(st.item()) == 0
    codes, s = c.run(use_fp8=True)
    for e, rows in c.rows():
        X.check_fp8(codes.cpu().numpy().reshape(c.total, -1)[rows], f64(s).reshape(c.total, -1)[rows],
                    *c.expect(e, rows), False)


def test_gradient_agrees_with_differences_of_the_product():
    """<g, y(x + d) - y(x)> = <dx, d> for a change d of one channel; the product is linear, so a whole step will do."""
    c = Case(5, 256, 384, [3, 2])
    back = Case(6, 384, 256, [3, 2], transposed=True)
    back.w, back.ws = c.w, c.ws
    back.weights = [w.T for w in c.weights]
    dx = f64(back.run())
    y0 = f64(c.run())
    rng = np.random.default_rng(7)
    for e, rows in c.rows():
        w = c.weights[e]
        for row in range(rows.start, rows.stop):
            k = int(rng.integers(0, 256))
            x = c.x.clone()
            x[row, k] ^= 0x80  # the channel's sign
            d = -2 * c.value[row, k]
            dy = f64(c.run(x=x))[row] - y0[row]
            g = back.value[row]
            # what the two BF16 results, their sums, and dx can be off
            mag = np.abs(c.value[row]) @ np.abs(w).T
            slack = (np.abs(g) * (2 * 2.0 ** -8 + 2.0 ** -16) * mag).sum() + abs(d) * (2.0 ** -8 + 2.0 ** -16) * (np.abs(g) @ np.abs(w[:, k]))
            assert abs(g @ dy - dx[row, k] * d) <= slack


@pytest.mark.parametrize("transposed", [False, True])
def test_nan_stays_in_its_row(transposed):
    c = Case(8, 256, 256, [9, 4], transposed=transposed)
    want = c.run()
    x, xs = c.x.clone(), c.xs.clone()
    x[2, 100] = 0x7F
    xs[7, 1] = float("nan")
    got = c.run(x=x, x_scale=xs)
    keep = [0, 1, 3, 4, 5, 6, 8] + list(range(11, 15))  # (9 and 10 lie between the segments)
    assert torch.equal(got[keep], want[keep])
    assert not torch.isfinite(got[[2, 7]]).any()


def test_zero_rows_and_zero_scales():
    """A row of zeros, as the dispatch quantises it (scale 0): zero results, with the scale 0 in FP8."""
    c = Case(9, 256, 256, [4])
    c.x[1], c.xs[1] = 0, 0
    assert (c.run()[1] == 0).all()
    y, s = c.run(use_fp8=True)
    assert (s[1] == 0).all() and ((y[1] & 0x7F) == 0).all() and (s[[0, 2, 3]] > 0).all()


def test_fp8_results_of_all_sizes():
    """Scales from 2^-120 to 2^118, and rows of zeros of either sign beside them: the rule of ep_fp8_quantize."""
    K = M = 128
    w = torch.zeros((1, M, K), dtype=torch.uint8, device="cuda")
    w[0, torch.arange(M), torch.arange(K)] = 0x38                 # the identity
    ws = torch.ones((1, 1, 1), device="cuda")
    powers = torch.arange(-120, 119, 7, device="cuda")
    n = powers.numel()
    x = dev(codes_of(np.random.default_rng(24), n, K))
    x[::5, 3] = 0x80
    xs = torch.ldexp(torch.ones(n, device="cuda"), powers)[:, None]
    count, off = ints([n]), ints([0])
    y = ep.expert_linear_fp8(x, xs, w, ws, count, off)            # exact: E4M3 times a power of two
    for kw in (dict(), dict(round_scale=True), dict(use_ue8m0=True)):
        q, s = ep.expert_linear_fp8(x, xs, w, ws, count, off, use_fp8=True, **kw)
        want, ws_ = torch.empty_like(q), torch.empty_like(s)
        ep.ep_fp8_quantize(y, want, ws_, ep.fp8_flags(True, **kw))
        assert torch.equal(s, ws_)
        # a sum of zeros is +0, whatever their signs
        same = (q == want) | ((q & 0x7F) == 0) & ((want & 0x7F) == 0)
        assert same.all()


def test_reports_rows_it_skips():
    c = Case(15, 256, 24, [4, 4], regions=True, spare=0)
    want = c.run(max_rows=8)
    y = torch.empty_like(want)

    def run(counts, **kw):
        st = new_status()
        y.fill_(5.0)
        c.run(row_count=ints(counts), out=kw.pop("out", y), status=st, **({"max_rows": 8} | kw))
        return int(st.item())

    assert run([9, 2]) == ep.EP_ST_CAPACITY                 # more than a region holds
    assert torch.equal(y[0], want[0]) and torch.equal(y[1, :2], want[1, :2]) and (y[1, 2:] == 5.0).all()
    flat = dict(x=c.x.view(8, -1), x_scale=c.xs.view(8, -1), out=y.view(8, -1))
    assert run([4, 4], row_offset=ints([0, 6]), **flat) == ep.EP_ST_CAPACITY
    assert torch.equal(y[0], want[0])
    assert run([4, 4], row_offset=ints([-1, 4]), **flat) == ep.EP_ST_CAPACITY
    assert torch.equal(y[1], want[1]) and (y[0] == 5.0).all()
    assert run([4, 4], max_rows=5) == ep.EP_ST_CAPACITY     # more than max_rows in all
    assert torch.equal(y[0], want[0])
    assert run([-3, 2]) == 0
    assert (y[0] == 5.0).all() and torch.equal(y[1, :2], want[1, :2])
    assert run([0, 0]) == 0 and (y == 5.0).all()


def test_more_rows_than_the_tiles_were_sized_for():
    """All rows on one expert of many: its tiles are small, and many."""
    c = Case(16, 512, 520, [0, 0, 150] + [0] * 37)
    got = f64(c.run())
    (e, rows), = c.rows()
    X.check_bf16(got[rows], *c.expect(e, rows))


def test_weights_beyond_32_bits():
    rng = np.random.default_rng(17)
    E, M, K = 80, 8192, 7168
    w = torch.empty((E, M, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, M // 128, K // 128), device="cuda")
    codes, scales = codes_of(rng, M, K), np.exp(rng.normal(size=(M // 128, K // 128)) - 12).astype(np.float32)
    w[-1], s[-1] = dev(codes), dev(scales)
    x = codes_of(rng, 3, K)
    xs = np.exp(rng.normal(size=(3, K // 128)) - 6).astype(np.float32)
    count = torch.zeros(E, dtype=torch.int32, device="cuda")
    count[-1] = 3
    off = torch.zeros(E, dtype=torch.int32, device="cuda")
    y = ep.expert_linear_fp8(dev(x), dev(xs), w, s, count, off)
    at = rng.choice(M, 64, replace=False)
    value = R.TABLE[x] * xs.astype(np.float64).repeat(128, axis=1)
    wv = R.TABLE[codes] * X.blocks(scales.astype(np.float64), M, K)
    X.check_bf16(f64(y)[:, at], *X.product(value, wv[at], False))
    # ... and read along the other axis
    g, gs = codes_of(rng, 3, M), np.exp(rng.normal(size=(3, M // 128)) - 6).astype(np.float32)
    dx = ep.expert_linear_fp8_backward(dev(g), dev(gs), w, s, count, off)
    at = rng.choice(K, 64, replace=False)
    X.check_bf16(f64(dx)[:, at], *X.product(R.TABLE[g] * gs.astype(np.float64).repeat(128, axis=1), wv[:, at].T, False))


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_and_results_beyond_32_bits(fp8):
    """Rows whose codes, and whose results, start past 2^32 bytes."""
    rng = np.random.default_rng(23)
    K, M, total, at = 8192, 9216, 600_000, 599_000
    codes, scales = codes_of(rng, M, K), np.exp(rng.normal(size=(M // 128, K // 128)) - 12).astype(np.float32)
    x = torch.empty((total, K), dtype=torch.uint8, device="cuda")
    xs = torch.empty((total, K // 128), device="cuda")
    rows, row_scales = codes_of(rng, 5, K), np.exp(rng.normal(size=(5, K // 128)) - 6).astype(np.float32)
    x[at:at + 5], xs[at:at + 5] = dev(rows), dev(row_scales)
    made = ep.expert_linear_fp8(x, xs, dev(codes[None]), dev(scales[None]), ints([5]), ints([at]), use_fp8=fp8, max_rows=5)
    pick = np.sort(rng.choice(M // 128, 2, replace=False))[:, None] * 128 + np.arange(128)  # whole blocks of outputs
    value = R.TABLE[rows] * row_scales.astype(np.float64).repeat(128, axis=1)
    y, err = X.product(value, (R.TABLE[codes] * X.blocks(scales.astype(np.float64), M, K))[pick.reshape(-1)], False)
    if not fp8:
        X.check_bf16(f64(made[at:at + 5])[:, pick.reshape(-1)], y, err)
        return
    X.check_fp8(made[0][at:at + 5].cpu().numpy()[:, pick.reshape(-1)], f64(made[1][at:at + 5])[:, pick[:, 0] // 128], y, err,
                False)


@pytest.mark.parametrize("transposed", [False, True])
def test_in_a_graph_and_on_another_stream(transposed):
    c = Case(18, 512, 256, [3, 1, 20], transposed=transposed)
    rows = np.flatnonzero(c.received())
    ws = ep.expert_linear_fp8_workspace(c.x, c.w)
    want = c.run(workspace=ws, max_rows=None)[rows]
    side = torch.cuda.Stream()
    made = c.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(made[rows], want)
    y = torch.zeros((c.total, c.outs), dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=y, workspace=ws, max_rows=None)
    graph.replay()
    assert torch.equal(y[rows], want)
    c.xs.mul_(2.0)
    c.row_count.copy_(ints([2, 1, 11]))
    y.zero_()
    graph.replay()
    keep = [0, 1, *range(c.first[1], c.first[1] + 1), *range(c.first[2], c.first[2] + 11)]
    at = np.searchsorted(rows, keep)
    assert torch.equal(y[keep], want[at] * 2) and (y.float().abs().sum(1) > 0).sum() == len(keep)


def test_calls_at_once_with_workspaces_of_their_own():
    """Two calls that share all their inputs, on two streams, each with a workspace."""
    c = Case(19, 2048, 1024, [40, 3, 77, 0, 128])
    want = c.run()
    rows = np.flatnonzero(c.received())
    sides = [torch.cuda.Stream() for _ in range(2)]
    work = [ep.expert_linear_fp8_workspace(c.x, c.w, sum(c.counts)) for _ in sides]
    torch.cuda.synchronize()
    made = [[c.run(stream=s, workspace=w) for _ in range(5)] for s, w in zip(sides, work)]
    torch.cuda.synchronize()
    for m in made:
        assert all(torch.equal(y[rows], want[rows]) for y in m)


def test_many_units_and_blocks():
    """More units than blocks, an expert's tiles over several of them, and long runs that end inside a unit."""
    counts = [257, 0, 1, 130, 64, 15, 16, 17] * 3
    c = Case(20, 1408, 1288, counts)
    got = f64(c.run())
    for e, rows in c.rows():
        X.check_bf16(got[rows], *c.expect(e, rows))


@pytest.mark.parametrize("rows", [1, 40, 128])
def test_every_number_of_units(rows):
    """Units that are fewer than the blocks, whole and cut, about as many, and a few more."""
    for outs in (256, 256 * 20, 256 * 57, 256 * 58, 256 * 151, 256 * 152 + 8, 256 * 160):
        c = Case(rows + outs, 640, outs, [rows])
        got = f64(c.run())
        at = np.random.default_rng(outs).choice(outs, min(outs, 200), replace=False)
        y, err = X.product(c.value[:rows], c.weights[0][at], False)
        X.check_bf16(got[:rows, at], y, err)


@pytest.mark.parametrize("K,M,counts,transposed", [
    (128, 128, "many", False), (16384, 24, [2, 9], False), (16384, 256, [1, 33], True), (128, 16384, [17, 3], False),
    (256, 128, "many", True)])
def test_largest_sizes(K, M, counts, transposed):
    """As many experts, and as many inputs, as there may be."""
    if counts == "many":
        counts = np.random.default_rng(5).integers(0, 3, ep.EP_MAX_EXPERTS).tolist()
    c = Case(K + M + 40, K, M, counts, transposed=transposed)
    got = f64(c.run())
    for e, rows in c.rows():
        X.check_bf16(got[rows], *c.expect(e, rows))


def test_one_workspace_for_calls_of_all_sizes():
    """Calls one after the other, of other shapes and with nothing to do, leave a shared workspace as it was."""
    cases = [Case(30, 1024, 768, [9, 0, 200, 41]), Case(31, 256, 4096, [3] * 9), Case(32, 2048, 512, [70, 140], transposed=True)]
    ws = torch.zeros(max(ep.ep_expert_linear_fp8_workspace_bytes(9, 1000), *(
        ep.ep_expert_linear_fp8_workspace_bytes(len(c.counts), sum(c.counts)) for c in cases)), dtype=torch.uint8, device="cuda")
    want = [c.run()[np.flatnonzero(c.received())] for c in cases]
    for _ in range(3):
        for c, w in zip(cases, want):
            assert torch.equal(c.run(workspace=ws)[np.flatnonzero(c.received())], w)
            c.run(workspace=ws, row_count=torch.zeros_like(c.row_count))


def test_nothing_to_do():
    c = Case(21, 128, 128, [2])
    assert c.run(x=c.x[:0], x_scale=c.xs[:0], max_rows=0).shape == (0, 128)
    y = torch.full((c.total, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    c.run(out=y, max_rows=0)
    assert (y == 5.0).all()


@pytest.mark.parametrize("n", [7, 40])
def test_fp8_results_that_are_no_numbers(n):
    """Rows with infinities, NaN and the smallest numbers: the rule of ep_fp8_quantize, few rows and many."""
    K = M = 128
    w = torch.zeros((1, M, K), dtype=torch.uint8, device="cuda")
    w[0, torch.arange(M), torch.arange(K)] = 0x38                 # the identity
    ws = torch.ones((1, 1, 1), device="cuda")
    x = dev(codes_of(np.random.default_rng(25), n, K))
    powers = torch.tensor([127, -126, 120, 119, -125, 0, 124], device="cuda").repeat(6)[:n]
    xs = torch.ldexp(torch.ones(n, device="cuda"), powers)[:, None]
    x[1::7, :] &= 0x81                                            # a smallest code, or zero
    y = ep.expert_linear_fp8(x, xs, w, ws, ints([n]), ints([0]))
    with np.errstate(over="ignore", invalid="ignore"):
        v = (R.TABLE[x.cpu().numpy()] * f64(xs)).astype(np.float32)   # exact, or past fp32
        m = np.abs(v).max(1)
        for form, kw in (("fp32", dict()), ("round", dict(round_scale=True)), ("ue8m0", dict(use_ue8m0=True))):
            q, s = ep.expert_linear_fp8(x, xs, w, ws, ints([n]), ints([0]), use_fp8=True, **kw)
            scale = m / np.float32(448)
            if form != "fp32":
                f, e = np.frexp(scale)
                scale = np.where(np.isfinite(scale), np.ldexp(np.float32(1), e - (f == 0.5)), scale)
            if form == "ue8m0":
                scale = np.maximum(scale, np.float32(2.0 ** -127))
            got = f64(s)[:, 0]
            if form == "ue8m0":
                got = np.where(got == 255, np.inf, 2.0 ** (got - 127))
            assert np.array_equal(got, scale.astype(np.float64))
            want = torch.from_numpy(v / scale[:, None].astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
            q = q.cpu()
            nan = ((q & 0x7F) == 0x7F) & ((want & 0x7F) == 0x7F)
            assert ((q == want) | nan | ((q & 0x7F) == 0) & ((want & 0x7F) == 0)).all()
            codes, scales = torch.empty_like(q, device="cuda"), torch.empty_like(s)
            ep.ep_fp8_quantize(y, codes, scales, ep.fp8_flags(True, **kw))
            rows = torch.from_numpy(np.nonzero((f64(y) == v).all(1))[0])  # those that BF16 holds
            assert rows.numel() >= 4 * (n // 7) and torch.equal(scales.cpu()[rows], s.cpu()[rows])
            codes = codes.cpu()[rows]
            assert ((codes == q[rows]) | nan[rows] | ((codes & 0x7F) == 0) & ((q[rows] & 0x7F) == 0)).all()
