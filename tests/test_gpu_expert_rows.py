"""What a BF16 row of the experts' products keeps of a value beside a larger one."""
import numpy as np
import pytest
import torch

import combine_ep_get_dispatch_gb300 as ep
import decode_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


@pytest.mark.parametrize("power", [0, -60, 70])
@pytest.mark.parametrize("largest", [225.0, 226.0, 300.0, 448.0, 224.0, 1.0])
def test_values_beside_a_large_one(largest, power):
    """Every BF16 value from 2^-24 of the largest of its 32 neighbours up to it, read through a weight of one.

    With s the power of two at or above largest / 448, a value enters as multiples of 2^-13 s or coarser ones that
    hold it: exactly from 2^-13 of the largest on (2^-6 s has 8 bits above that step), within half a step of 2^-13 s
    below. Results have 8 bits at most, so that their rounding adds nothing.
    """
    bits = np.arange(0x7F80, dtype=np.uint32)  # finite
    v = (bits << 16).view(np.float32).astype(np.float64)
    v = v[(v >= 2.0 ** -24 * largest) & (v <= largest)]
    v = np.concatenate([v, np.zeros(-v.size % 31)]).reshape(-1, 31)
    v[:, ::2] *= -1
    n = v.shape[0]
    x = np.zeros((n, 128))
    x[:, 0], x[:, 1:32] = largest, v
    codes = np.zeros((1, 32, 64), np.uint8)  # output o reads input o
    codes[0, np.arange(32), np.arange(32) // 2] = np.where(np.arange(32) % 2, 0x20, 0x02)
    xd = torch.from_numpy((x * 2.0 ** power).astype(np.float32)).to(torch.bfloat16).cuda()
    y = ep.expert_linear(xd, torch.from_numpy(codes).cuda(), torch.full((1, 32, 4), 127, dtype=torch.uint8, device="cuda"),
                         torch.tensor([n], dtype=torch.int32, device="cuda"),
                         row_offset=torch.zeros(1, dtype=torch.int32, device="cuda"))
    got = y.float().cpu().numpy().astype(np.float64) * 2.0 ** -power
    s = R.pow2_above(largest / 448.0)
    off = np.abs(got[:, 1:] - v)
    assert (got[:, 0] == largest).all()
    assert not off[np.abs(v) >= 2.0 ** -13 * largest].any()
    assert (off <= 2.0 ** -14 * s).all() and 2.0 ** -14 * s <= 2.0 ** -21.8 * largest


# Many units a block, in the order that lets blocks work on one expert's output tiles together.
MANY = [
    # in, out, rows of each expert, glu
    (128, 1024, [40, 0, 70, 33] * 16, False),
    (256, 3216, [190, 64, 0, 0, 100, 5] * 4, True),
    (384, 2056, [250, 33, 97] * 7, False),       # several tiles of rows
    (640, 648, [80] * 61, False),
]


@pytest.mark.parametrize("K,M,counts,glu", MANY)
@pytest.mark.parametrize("fp8", [False, True])
def test_many_rows_of_many_experts(K, M, counts, glu, fp8):
    rng = np.random.default_rng(K + M)
    E = len(counts)
    codes = rng.integers(0, 256, (E, M, K // 2)).astype(np.uint8)
    scales = rng.integers(118, 124, (E, M, K // 32)).astype(np.uint8)
    first = np.cumsum([0] + counts)[:-1]
    n = int(sum(counts)) + 3
    if fp8:
        x = rng.integers(0, 254, (n, K))
        x = np.where(x >= 127, x + 1, x).astype(np.uint8)
        xs = rng.integers(117, 124, (n, K // 128)).astype(np.uint8)
        value = R.TABLE[x] * np.repeat(2.0 ** (xs.astype(float) - 127), 128, axis=1)
        xd, xsd = torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda()
    else:
        xd, xsd = torch.from_numpy(rng.normal(size=(n, K)).astype(np.float32)).to(torch.bfloat16).cuda(), None
        value = xd.float().cpu().numpy().astype(np.float64)
    outs = M // 2 if glu else M
    y = torch.full((n, outs), 77.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    w, s = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    args = dict(row_count=torch.tensor(counts, dtype=torch.int32, device="cuda"), x_scale=xsd, glu=glu, status=st,
                row_offset=torch.from_numpy(first.astype(np.int32)).cuda(), max_rows=sum(counts),
                workspace=ep.expert_linear_workspace(xd, w, max_rows=sum(counts)))
    ep.expert_linear(xd, w, s, out=y, **args)
    got = y.float().cpu().numpy().astype(np.float64)
    for e, c in enumerate(counts):
        if c == 0:
            continue
        rows = slice(first[e], first[e] + c)
        ref, err = R.expert_product(value[rows], R.weights(codes[e], scales[e]), glu)
        off, tol = np.abs(got[rows] - ref), (2.0 ** -8 * np.abs(ref) + err) * 1.01 + 2.0 ** -130
        assert (off <= tol).all(), (e, (off / tol).max())
    assert (got[-3:] == 77.0).all() and int(st.item()) == 0
    first_y = y.clone()
    ep.expert_linear(xd, w, s, out=y, **args)  # the used workspace: the same bits
    assert torch.equal(y, first_y)


def test_few_rows_of_long_units():
    """Units of 40 and more steps take that order too, with two steps a stage; an odd number of steps."""
    rng = np.random.default_rng(7)
    counts, K, M = [5, 0, 3, 1] * 12, 5248, 1032
    E, n = len(counts), sum(counts)
    w = rng.integers(0, 256, (E, M, K // 2)).astype(np.uint8)
    s = rng.integers(118, 124, (E, M, K // 32)).astype(np.uint8)
    x = torch.from_numpy(rng.normal(size=(n, K)).astype(np.float32)).to(torch.bfloat16)
    first = np.cumsum([0] + counts)[:-1]
    y = ep.expert_linear(x.cuda(), torch.from_numpy(w).cuda(), torch.from_numpy(s).cuda(),
                         torch.tensor(counts, dtype=torch.int32, device="cuda"),
                         row_offset=torch.from_numpy(first.astype(np.int32)).cuda())
    got, value = y.float().cpu().numpy().astype(np.float64), x.float().numpy().astype(np.float64)
    for e, c in enumerate(counts):
        if c:
            rows = slice(first[e], first[e] + c)
            ref, err = R.expert_product(value[rows], R.weights(w[e], s[e]), False)
            assert (np.abs(got[rows] - ref) <= (2.0 ** -8 * np.abs(ref) + err) * 1.01 + 2.0 ** -130).all(), e
