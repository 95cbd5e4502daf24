"""More of the rotary positions, beside test_gpu_rotary.py, whose bound of an output holds here."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_rotary import check, dev

pytestmark = pytest.mark.gpu

kv = pytest.importorskip("fp8_paged_kv_reshape_gb300")


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("rot", [16, 128, 256])
def test_frequencies_without_an_angle(rot, interleaved):
    """NaN, infinities and numbers from 2^54 on: their pairs are NaN and the call says so; the largest that do have one."""
    r = np.random.default_rng(rot)
    pos = np.array([0, 1, 5, -7, 2 ** 31 - 1, -2 ** 31 + 1, 100003])
    x = torch.from_numpy(r.standard_normal((len(pos), 3, 256))).float().cuda()
    good = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    good[[0, 3, rot // 2 - 1]] = [np.nextafter(2.0 ** 54, 0), -2.0 ** 53 - 2, 2.0 ** 31 + 0.5]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, _ = kv.rotary_embedding(x, None, dev(pos), dev(good), interleaved, status=st)
    assert int(st.item()) == 0
    check(y, x, pos, good, interleaved)
    bad = good.copy()
    at = {0: math.nan, 2: math.inf, 5: -math.inf, rot // 2 - 1: 2.0 ** 54, rot // 2 - 2: -1e300}
    for j, f in at.items():
        bad[j] = f
    z, _ = kv.rotary_embedding(x, None, dev(pos), dev(bad), interleaved, status=st)
    assert int(st.item()) == kv.DEV_BAD_SCALE
    nan = torch.zeros_like(x, dtype=torch.bool)
    for j in at:
        nan[..., [2 * j, 2 * j + 1] if interleaved else [j, j + rot // 2]] = True
    assert torch.equal(torch.isnan(z), nan)
    assert torch.equal(z[~nan], y[~nan])
