"""kv.rotary_frequencies against the schemes' definitions, values between the bounds included (CPU only)."""
import math

import numpy as np
import pytest

import fp8_paged_kv_reshape_gb300 as kv


def frequencies(rot_dim, base, **more):
    f, magnitude = kv.rotary_frequencies(rot_dim, base, device="cpu", **more)
    return f.numpy(), magnitude, base ** (-np.arange(rot_dim // 2) * 2.0 / rot_dim)


# rounding: a power and some products of float64
def close(a, b):
    return np.allclose(a, b, rtol=1e-13, atol=0)


@pytest.mark.parametrize("factor, length, low, high", [(8.0, 8192, 1.0, 4.0), (16.0, 4096, 1.0, 32.0), (4.0, 100, 0.5, 3.0)])
def test_parts_by_turns(factor, length, low, high):
    f, magnitude, plain = frequencies(128, 500000.0, scaling="parts", factor=factor, original_len=length, low_turns=low, high_turns=high)
    wave = 2 * math.pi / plain  # positions of a turn
    smooth = (length / wave - low) / (high - low)
    want = np.where(wave < length / high, plain, np.where(wave > length / low, plain / factor, (1 - smooth) * plain / factor + smooth * plain))
    assert close(f, want) and ((f < plain) & (f > plain / factor)).any()
    assert magnitude == 0.1 * math.log(factor) + 1


def test_parts_by_pairs():
    """At base 10000, 4096 positions and 128 dims a pair makes 32 turns at index 20.9 and one at 45.03: kept up to 20, slowed from 46."""
    f, magnitude, plain = frequencies(128, 10000.0, scaling="parts", factor=16.0, original_len=4096, ramp="pairs")
    assert close(f[:21], plain[:21]) and close(f[46:], plain[46:] / 16)
    j = np.arange(20, 47)
    keep = (46 - j) / 26
    assert close(f[20:47], plain[20:47] * keep + plain[20:47] / 16 * (1 - keep))
    assert magnitude == 0.1 * math.log(16.0) + 1
    # bounds outside the head: all slowed, all kept
    f, _, plain = frequencies(16, 10000.0, scaling="parts", factor=4.0, original_len=6, ramp="pairs")
    assert close(f[1:], plain[1:] / 4)
    f, _, plain = frequencies(16, 10000.0, scaling="parts", factor=4.0, original_len=1 << 40, low_turns=2.0 ** 10, high_turns=2.0 ** 11, ramp="pairs")
    assert close(f, plain)


def test_a_magnitude_of_the_models_own():
    for scaling in (None, "linear", "base", "parts"):
        f, magnitude, _ = frequencies(64, 10000.0, scaling=scaling, factor=8.0, original_len=512, magnitude=1.0)
        assert magnitude == 1.0
        g, _, _ = frequencies(64, 10000.0, scaling=scaling, factor=8.0, original_len=512)
        assert np.array_equal(f, g)


def test_refusals():
    for kw in (dict(ramp="other"), dict(magnitude=math.inf), dict(magnitude=math.nan),
               dict(scaling="parts", original_len=64, ramp="pairs", base=1.0), dict(scaling="parts", original_len=64, ramp="pairs", low_turns=0.0)):
        with pytest.raises(ValueError):
            kv.rotary_frequencies(**{**dict(rot_dim=64, device="cpu"), **kw})
