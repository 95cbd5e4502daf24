"""The 4-bit oracle against things other than itself: exact rationals, torch's E4M3 conversion,
closed forms of attention, and hand-written page moves."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import fp4


def _nearest_by_rationals(x: float, values):
    best = min(range(len(values)), key=lambda i: (abs(Fraction(x) - Fraction(float(values[i]))), i % 2))
    return best


def test_e2m1_rounding_at_and_around_every_halfway_point():
    mids = [(a + b) / 2 for a, b in zip(fp4.E2M1, fp4.E2M1[1:])]
    xs = [0.0, 1e-30, 6.0, 7.5, 1e30]
    for v in list(fp4.E2M1) + mids:
        xs += [v, np.nextafter(np.float32(v), np.float32(100)), np.nextafter(np.float32(v), np.float32(-0.0))]
    xs = np.abs(np.array(xs, np.float32))
    got = fp4.nearest_code(np.minimum(xs.astype(np.float64), 6.0), fp4.E2M1)
    assert got.tolist() == [_nearest_by_rationals(min(float(x), 6.0), fp4.E2M1) for x in xs]
    # ties go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    assert fp4.E2M1[fp4.nearest_code(np.array(mids), fp4.E2M1)].tolist() == [0, 1, 1, 2, 2, 4, 4]


def test_e4m3_rounding_is_torchs():
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.rand(20000, generator=g) * 448, torch.exp2(torch.rand(20000, generator=g) * 18 - 12),
                   torch.tensor(fp4.E4M3, dtype=torch.float32),
                   torch.tensor((fp4.E4M3[1:] + fp4.E4M3[:-1]) / 2, dtype=torch.float32)]).clamp(max=448)
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp4.nearest_code(x.double().numpy(), fp4.E4M3), want)


@pytest.mark.parametrize("s", [1.0, 0.05, -0.3, 1e-20, 7e20])
def test_error_of_a_group_is_within_its_steps(s):
    # |value - x|: half a step of E2M1 at x/d is at most 1 (between 4 and 6) below 6, and the
    # largest element may lie above 6*d by E4M3's rounding of the scale, at most 2^-4 of it in the
    # normal range; float32 rounding of quotients and products adds less than 2^-20 of x.
    r = np.random.default_rng(2)
    x = (r.standard_normal((64, 2, 64)) * abs(s) * np.exp(r.standard_normal((64, 1, 1)))).astype(np.float32)
    codes, scales = fp4.quantize(x, s)
    v = fp4.code_values(codes).reshape(64, 2, 4, 16) * fp4.scale_values(scales)[..., None] * float(np.float32(s))
    v = v.reshape(x.shape)
    g = np.abs(x.reshape(64, 2, 4, 16)).max(-1, keepdims=True)
    bound = np.broadcast_to(g / 6 * (1 + 2.0 ** -4), (64, 2, 4, 16)).reshape(x.shape) * (1 + 2.0 ** -18)
    assert np.all(np.abs(v - x) <= bound)
    assert np.all((v == 0) | (np.sign(v) == np.sign(x)))


def test_corner_groups():
    x = np.zeros((5, 1, 64), np.float32)
    x[0] = -0.0                     # zeros of either sign: code 0
    x[1, 0, 3] = np.nan             # the first group is NaN, the others are not
    x[2, 0, :2] = [np.inf, -3.0]    # infinite: magnitude 6 of scale 448, the rest zero
    x[3, 0, 0] = -1e-12             # a scale that rounds to zero: the sign is kept
    x[4, 0, :3] = [6.0, 0.25, 0.75]
    codes, scales = fp4.quantize(x, 1.0)
    assert not codes[0].any() and not scales[0].any()
    assert scales[1, 0].tolist() == [0x7F, 0, 0, 0] and not codes[1].any()
    assert scales[2, 0, 0] == 0x7E and codes[2, 0, 0] == 0x87  # 6 and -0
    assert scales[3, 0, 0] == 0 and codes[3, 0, 0] == 0x08
    assert scales[4, 0, 0] == 0x38 and codes[4, 0, :2].tolist() == [0x07, 0x02]  # ties to even


def test_write_places_rows_and_leaves_the_rest():
    r = np.random.default_rng(3)
    codes = np.full((3, 8, 2, 32), 0x5A, np.uint8)
    scales = np.full((3, 2, 8, 4), 0x7F, np.uint8)
    x = r.standard_normal((4, 2, 64)).astype(np.float32)
    assert fp4.write(x, codes, scales, np.array([9, -1, 23, 24]), 0.5)  # 24 is out of range
    assert not fp4.write(x[:1], codes, scales, np.array([-1]), 0.5)
    for i, slot in ((0, 9), (2, 23)):
        c, b = fp4.quantize(x[i], 0.5)
        assert np.array_equal(codes[slot // 8, slot % 8], c) and np.array_equal(scales[slot // 8, :, slot % 8], b)
        back = fp4.dequant(codes, scales, np.array([slot]), 0.5)
        assert np.array_equal(back[0], (fp4.rows(codes, scales, np.array([slot]))[0] * 0.5).astype(np.float32))
    codes[1, 1] = codes[2, 7] = 0x5A
    scales[1, :, 1] = scales[2, :, 7] = 0x7F
    assert (codes == 0x5A).all() and (scales == 0x7F).all()


def test_attention_closed_forms():
    r = np.random.default_rng(4)
    kc = r.integers(0, 256, (4, 8, 2, 32)).astype(np.uint8)
    vc = r.integers(0, 256, (4, 8, 2, 32)).astype(np.uint8)
    kg = r.integers(0, 0x40, (4, 2, 8, 4)).astype(np.uint8)
    vg = r.integers(0, 0x40, (4, 2, 8, 4)).astype(np.uint8)
    bt = np.array([[2, 0, 3], [1, -1, -1]], np.int32)
    q = r.standard_normal((2, 4, 64))
    qsl = np.array([0, 1, 2])
    vals = lambda slots: fp4.rows(vc, vg, np.array(slots))  # noqa: E731
    one, _ = fp4.attention(q, qsl, kc, vc, kg, vg, bt, [1, 1], 0.3, 0.5)
    assert np.allclose(one[0, :2], 0.5 * vals([16])[0, 0]) and np.allclose(one[1, 2:], 0.5 * vals([8])[0, 1])
    mean, w = fp4.attention(0 * q, qsl, kc, vc, kg, vg, bt, [19, 8], 0.3, 0.5)
    slots = list(range(16, 24)) + list(range(8)) + [24, 25, 26]
    assert np.allclose(mean[0, 0], 0.5 * vals(slots)[:, 0].mean(0))
    assert np.allclose(w[0, 0], 0.5 * np.abs(vals(slots)[:, 0]).mean(0))
    # two new tokens: the first does not see the second, NaN or not
    vg[2, :, 5] = 0x7F
    two, _ = fp4.attention(q, np.array([0, 2, 2]), kc, vc, kg, vg, bt, [6, 0], 0.3, 0.5)
    assert np.isfinite(two[0]).all() and np.isnan(two[1]).all()


def test_page_moves():
    c = np.arange(8, dtype=np.uint8)[:, None].repeat(16, 1)
    a = c.copy()
    assert not fp4.copy_blocks([a], [1, 1, 5, -1], [0, 2, 5, 3])
    assert a[:, 0].tolist() == [1, 1, 1, 3, 4, 5, 6, 7]
    a = c.copy()
    assert fp4.copy_blocks([a], [1, 2, 3, 0], [4, 4, 5, 8])  # 4 twice, 8 outside
    assert a[:, 0].tolist() == [0, 1, 2, 3, 4, 3, 6, 7]
    a = c.copy()
    assert fp4.copy_blocks([a], [1, 2], [2, 3])  # the second reads what the first writes
    assert a[:, 0].tolist() == [0, 1, 1, 3, 4, 5, 6, 7]
    a = c.copy()
    bt = np.array([[7, 3, 9], [7, 5, 6]], np.int32)  # 7 shared
    new, n, flagged = fp4.compact([a], bt, [20, 9], 8)
    assert (n, flagged) == (3, True)  # 9 is outside
    # used {3, 5, 7}: 3 -> 0, 5 -> 1, 7 -> 2
    assert new.tolist() == [[2, 0, -1], [2, 1, -1]]
    assert a[:, 0].tolist() == [3, 5, 7, 3, 4, 5, 6, 7]


def test_attention_of_a_sequence_whose_blocks_are_all_outside():
    r = np.random.default_rng(5)
    kc, kg = r.integers(0, 256, (2, 8, 1, 32)).astype(np.uint8), r.integers(0, 0x40, (2, 1, 8, 4)).astype(np.uint8)
    q = r.standard_normal((3, 2, 64))
    bt = np.array([[-1, 2], [0, 1], [2, 1]], np.int32)
    out, weight = fp4.attention(q, np.arange(4), kc, kc, kg, kg, bt, [16, 16, 8], 0.3, 0.5)
    assert not out[0].any() and not weight[0].any() and out[1].any() and not out[2].any()
