"""The 64-bit reference of the decode step's operators against independent facts (CPU)."""
import numpy as np
import torch

import decode_reference as R


def test_e4m3_agrees_with_torch_on_codes_midpoints_and_random_values():
    pos = R.TABLE[:127]
    mid = (pos[1:] + pos[:-1]) / 2
    v = np.concatenate([pos, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9),
                        np.random.default_rng(0).normal(size=20000) * 50])
    v = np.concatenate([v, -v]).astype(np.float32)
    want = torch.from_numpy(v).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3(v), want)
    assert R.e4m3(np.array([np.nan]))[0] == 127 and R.e4m3(np.array([np.inf, -np.inf, 1e9])).tolist() == [126, 254, 126]


def test_block_scale_is_the_smallest_power_of_two():
    for a, s in ((448.0, 1.0), (449.0, 2.0), (7.0, 2.0 ** -6), (7.03125, 2.0 ** -5), (0.0, 2.0 ** -100),
                 (np.inf, 2.0 ** -100), (1e-38, 2.0 ** -100)):
        assert R.block_scale(np.array([a, -0.0], dtype=np.float32)) == s


def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(1)
    ang = np.arange(40)[:, None] * 10000.0 ** (-np.arange(8) / 8)
    rope = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    a, b = rng.normal(size=(1, 32)), rng.normal(size=(1, 32))
    for inter in (False, True):
        ra = [R.rotate(a, rope[p], inter, np.float64) for p in range(40)]
        rb = [R.rotate(b, rope[p], inter, np.float64) for p in range(40)]
        assert np.allclose((ra[7] * rb[12]).sum(), (ra[20] * rb[25]).sum())
        assert np.allclose(np.linalg.norm(ra[39]), np.linalg.norm(a))
        assert np.array_equal(ra[5][:, 16:], a[:, 16:])


def test_attention_of_equal_keys_averages_the_values():
    rng = np.random.default_rng(2)
    cache = dict(k=np.full((2, 1, 16, 64), 0x38, np.uint8), v=rng.integers(0, 127, (2, 1, 16, 64)).astype(np.uint8),
                 k_scale=np.ones((2, 1)), v_scale=np.array([[1.0], [4.0]]), table=np.array([[1, 0]]))
    out, lse, *_ = R.attention(cache, [20], [0, 1], np.ones((1, 2, 64)), 0.125, 0)
    v = np.concatenate([R.TABLE[cache["v"][1, 0]] * 4, R.TABLE[cache["v"][0, 0, :4]]])
    assert np.allclose(out[0, 1], v.mean(0)) and np.allclose(lse, np.log(20) + 8)
    assert np.allclose(R.attention(cache, [20], [0, 1], np.ones((1, 2, 64)), 0.125, 4)[0][0, 0], v[16:].mean(0))


def test_expert_product_of_unit_rows_reads_the_weights():
    codes = np.array([[0x21, 0x7F] + [0] * 14], np.uint8)  # 0.5, 1, -6, 6
    w = R.weights(codes, np.array([[128]], np.uint8))
    assert w[0, :4].tolist() == [1.0, 2.0, -12.0, 12.0] and not w[0, 4:].any()
    y, err = R.expert_product(np.eye(32), w, False)
    assert np.array_equal(y[:, 0], w[0]) and (err >= 0).all()
