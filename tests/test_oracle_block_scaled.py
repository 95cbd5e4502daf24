"""The oracle of the cache with block scales and of rotary positions, pinned to things other than itself."""
import math

import numpy as np
import pytest

import oracle
from oracle import block_scaled as bso


def test_encode_is_the_fp8_oracles():
    u = np.arange(65536, dtype=np.uint32)
    y = (u << 16).view(np.float32)
    assert np.array_equal(bso.encode(y), oracle.e4m3_encode_array(y))
    assert np.array_equal(bso.decode(np.arange(256, dtype=np.uint8)), oracle.e4m3_decode_all(), equal_nan=True)


@pytest.mark.parametrize("a", [0.0, 1e-30, 447.9, 448.0, 448.1, 1.0, 0.875, 0.876, 3.4028234663852886e38])
def test_power_holds_and_half_of_it_does_not(a):
    p = bso.power_for(a)
    assert math.frexp(p)[0] == 0.5 and 448 * p >= a
    assert p == 2.0 ** -60 or 448 * p / 2 < a


def test_one_call_a_block_is_the_fp8_store_at_that_scale():
    r = np.random.default_rng(0)
    x = (r.standard_normal((16, 2, 64)) * [[[1.0], [100.0]]]).astype(np.float32)
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)  # (bf16, as the other oracle takes them)
    x = (bits.astype(np.uint32) << 16).view(np.float32)
    codes, scales = np.zeros((1, 16, 2, 64), np.uint8), np.zeros((1, 4), np.float32)
    assert bso.write(x, codes, scales, np.arange(16)) == (False, False)
    for h in range(2):
        s = float(scales[0, h])
        assert 224 * s < np.abs(x[:, h]).max() <= 448 * s
        kc, vc = np.zeros((1, 16, 1, 64), np.uint8), np.zeros((1, 16, 1, 64), np.uint8)
        rows = np.ascontiguousarray(bits[:, h:h + 1])
        assert oracle.reshape_and_cache(rows, rows, kc, vc, np.arange(16), 16, s, s) == 0
        assert np.array_equal(codes[:, :, h:h + 1], kc)


def test_growth_by_powers_of_two_keeps_normal_values():
    """Token by token with rising magnitudes: what is read back is what the last scale alone would give, as long
    as values stay out of the range's bottom."""
    x = (2.0 ** np.arange(8)[:, None, None] * np.linspace(1, 1.9, 64)).astype(np.float32)
    codes, scales = np.zeros((1, 16, 1, 64), np.uint8), np.zeros((1, 4), np.float32)
    for i in range(8):
        bso.write(x[i:i + 1], codes, scales, np.array([i]))
    once, s1 = np.zeros((1, 16, 1, 64), np.uint8), np.zeros((1, 4), np.float32)
    bso.write(x, once, s1, np.arange(8))
    assert np.array_equal(codes[:, :8], once[:, :8]) and np.array_equal(scales, s1)


def test_a_first_token_starts_the_block_anew():
    codes, scales = np.full((1, 16, 1, 64), 0x7E, np.uint8), np.full((1, 4), 64.0, np.float32)
    bso.write(np.ones((1, 1, 64), np.float32), codes, scales, np.array([0]))
    assert scales[0, 0] == 2.0 ** -8 and (codes[0, 1:] == 0x7E).all()
    assert (bso.dequant(codes, scales, np.array([0])) == 1.0).all()


def test_attention_of_equal_scales_is_the_fp8_oracles():
    r = np.random.default_rng(1)
    kc, vc = (oracle.e4m3_encode_array(r.standard_normal((4, 16, 2, 64)).astype(np.float32) * 4).reshape(4, 16, 2, 64) for _ in "kv")
    q = r.standard_normal((2, 4, 64)).astype(np.float32)
    qb = (q.view(np.uint32) >> 16).astype(np.uint16)
    qf = (qb.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    bt, lens = np.array([[2, 0], [1, 3]], np.int32), np.array([20, 31], np.int32)
    want, st = oracle.paged_decode_attention(qb, kc, vc, bt, lens, 0.125, 0.5)
    scales = [np.full((4, 4), s, np.float32) for s in (0.125, 0.5)]
    got, weight, _ = bso.attention(qf, np.arange(3), kc, vc, *scales, bt, lens)
    assert st == 0 and np.abs(got - want).max() < 1e-6 and (weight >= np.abs(got) - 1e-12).all()


def test_attention_without_a_mask_sees_the_last_token_first():
    kc = np.zeros((1, 16, 1, 64), np.uint8)
    vc = np.zeros((1, 16, 1, 64), np.uint8)
    vc[0, 2] = 0x38  # 1.0
    scales = np.ones((1, 4), np.float32)
    q = np.ones((5, 1, 64))
    out, _, _ = bso.attention(q, np.array([0, 5]), kc, vc, scales, scales, np.array([[0]]), [3], causal=False)
    assert np.allclose(out, 1 / 3)  # more queries than tokens
    out, _, _ = bso.attention(q[:3], np.array([0, 3]), kc, vc, scales, scales, np.array([[0]]), [3])
    assert np.allclose(out[:2], 0) and np.allclose(out[2], 1 / 3)


def test_rotary_of_angles_and_layouts():
    x = np.random.default_rng(2).standard_normal((3, 2, 32))
    f = [1.0, 0.5, 0.25, 0.125, 0.1, 0.05, 0.025, 0.0125]
    y = bso.rotary(x, [0, 7, -7], f)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 16:], x[..., 16:])
    z = (x[1, :, :8] + 1j * x[1, :, 8:16]) * np.exp(1j * 7 * np.array(f))
    assert np.allclose(y[1, :, :8], z.real) and np.allclose(y[1, :, 8:16], z.imag)
    back = bso.rotary(y, [0, 7, -7], f, transpose=True)
    assert np.allclose(back, x)
    z = bso.rotary(x, [0, 7, -7], f, interleaved=True, magnitude=2.0)
    assert np.allclose(z[1, :, 0:16:2], 2 * (x[1, :, 0:16:2] * np.cos(7 * np.array(f)) - x[1, :, 1:16:2] * np.sin(7 * np.array(f))))
    assert abs(bso.angle(3, math.pi / 2) - 1.5 * math.pi) < 1e-12
    assert abs(bso.angle(10 ** 9, 0.001) - math.fmod(1e6, 2 * math.pi)) < 1e-9
