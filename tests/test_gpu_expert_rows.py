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
