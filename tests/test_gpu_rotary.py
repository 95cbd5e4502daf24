"""Rotary positions on the GPU against the oracle.

Bound of an output, with m the magnitude and (a, b) the pair: angles are within 2^-27 turn, sinpif and cospif
within 2 ulp, magnitude, product and fused multiply-add a rounding each: |m| (|a| + |b|) * (2 pi 2^-27 + 2 * 2^-23 +
3 * 2^-24), under 12 * 2^-24 of it; then half a step of the output's type.
"""
import math

import numpy as np
import pytest
import torch

from oracle import block_scaled as bso

pytestmark = pytest.mark.gpu

kv = pytest.importorskip("fp8_paged_kv_reshape_gb300")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(got, x, positions, freq, interleaved=False, magnitude=1.0, transpose=False):
    rot = 2 * len(freq)
    xd = x.double().cpu().numpy()
    want = bso.rotary(xd, positions, freq, interleaved, magnitude, transpose)
    size = np.zeros(xd.shape)
    if interleaved:
        both = np.abs(xd[..., 0:rot:2]) + np.abs(xd[..., 1:rot:2])
        size[..., 0:rot:2] = size[..., 1:rot:2] = both
    else:
        both = np.abs(xd[..., :rot // 2]) + np.abs(xd[..., rot // 2:rot])
        size[..., :rot // 2] = size[..., rot // 2:rot] = both
    step = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    err = np.abs(got.double().cpu().numpy() - want)
    bound = (12 * 2.0 ** -24 * abs(magnitude) * size + step * np.abs(want)) * (1 + 2.0 ** -7)
    assert (err <= bound).all(), (err - bound).max()
    assert torch.equal(got[..., rot:], x[..., rot:])


SHAPES = [(1, 1, 1, 64, 64), (7, 4, 2, 64, 64), (33, 32, 8, 128, 128), (5, 64, 8, 128, 32), (300, 16, 4, 256, 64), (9, 14, 2, 64, 32),
          (12, 40, 8, 128, 96), (65, 5, 1, 80, 80), (3, 16, 16, 64, 16), (4, 3, 0, 256, 256), (2, 7, 1, 24, 16), (2000, 2, 1, 128, 112)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("n, n_q, n_k, hd, rot", SHAPES)
def test_matches_the_oracle(dtype, interleaved, n, n_q, n_k, hd, rot):
    r = np.random.default_rng(n + rot)
    q = torch.from_numpy(r.standard_normal((n, n_q, hd))).to(dtype).cuda()
    k = torch.from_numpy(r.standard_normal((n, n_k, hd))).to(dtype).cuda() if n_k else None
    pos = r.integers(0, 100000, n)
    freq, _ = kv.rotary_frequencies(rot)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q2, k2 = kv.rotary_embedding(q, k, dev(pos), freq, interleaved, status=st)
    assert int(st.item()) == 0
    check(q2, q, pos, freq.cpu().numpy(), interleaved)
    if n_k:
        check(k2, k, pos, freq.cpu().numpy(), interleaved)
    else:
        assert k2 is None


def test_far_negative_and_odd_positions_and_frequencies():
    r = np.random.default_rng(1)
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31 + 1, 123456789, -987654321, 2 ** 20, 3])
    freq = np.array([1.0, 0.1, 1e-9, 0.0, -0.7, math.pi, 2 * math.pi, 1234.5678])
    x = torch.from_numpy(r.standard_normal((len(pos), 3, 32))).float().cuda()
    for interleaved in (False, True):
        y, _ = kv.rotary_embedding(x, None, dev(pos), dev(freq), interleaved)
        check(y, x, pos, freq, interleaved)


def test_positions_out_of_range_leave_their_rows():
    x = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(x, 7.0)
    freq, _ = kv.rotary_frequencies(64)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.rotary_embedding(x, None, dev(np.array([1, 2 ** 31, -2 ** 31, 2])), freq, query_out=out, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == kv.DEV_BAD_SLOT
    assert bool((out[1:3] == 7).all()) and not bool((out[[0, 3]] == 7).any())


@pytest.mark.parametrize("scaling, kw", [(None, {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
                                         ("parts", dict(factor=16.0, original_len=4096)),
                                         ("parts", dict(factor=8.0, original_len=8192, low_turns=1.0, high_turns=4.0))])
def test_scaled_frequencies(scaling, kw):
    freq, mag = kv.rotary_frequencies(128, 500000.0, scaling, **kw)
    f, factor = freq.cpu().numpy(), kw.get("factor", 1.0)
    plain = 500000.0 ** (-np.arange(64) / 64)
    if scaling == "linear":
        assert np.allclose(f, plain / factor, rtol=1e-14)
    elif scaling == "base":
        assert np.allclose(f[0], 1) and np.allclose(f[-1], plain[-1] / factor, rtol=1e-12)
    elif scaling == "parts":
        turns = kw["original_len"] * plain / (2 * math.pi)
        fast, slow = turns >= kw.get("high_turns", 32.0), turns <= kw.get("low_turns", 1.0)
        assert fast.any() and slow.any()
        assert np.allclose(f[fast], plain[fast], rtol=1e-14) and np.allclose(f[slow], plain[slow] / factor, rtol=1e-14)
        assert (np.diff(f) < 0).all() and (f <= plain).all() and (f >= plain / factor * (1 - 1e-12)).all()
        assert mag == 0.1 * math.log(factor) + 1
    else:
        assert np.allclose(f, plain, rtol=1e-14)
    x = torch.randn(20, 4, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    pos = np.arange(20) * 6000
    y, _ = kv.rotary_embedding(x, None, dev(pos), freq, magnitude=mag)
    check(y, x, pos, f, magnitude=mag)


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
def test_transpose_is_the_gradient(interleaved):
    """<g, R x> = <R^T g, x>, and R^T g is the difference quotient of <g, R x>."""
    r = np.random.default_rng(2)
    x, g = (torch.from_numpy(r.standard_normal((6, 2, 48))).float().cuda() for _ in "xg")
    pos, (freq, _) = dev(r.integers(0, 5000, 6)), kv.rotary_frequencies(32)
    kw = dict(interleaved=interleaved, magnitude=1.25)
    turn = lambda t, **more: kv.rotary_embedding(t, None, pos, freq, **kw, **more)[0].double()  # noqa: E731
    back = turn(g, transpose=True)
    check(back.float(), g, pos.cpu().numpy(), freq.cpu().numpy(), interleaved, 1.25, transpose=True)
    # each product is within 12 * 2^-24 * 1.25 * (|a| + |b|): over 576 elements of size under 5 each
    assert abs(float((g.double() * turn(x)).sum() - (back * x.double()).sum())) < 576 * 12 * 2.0 ** -24 * 1.25 * 10 * 5
    h = 2.0 ** -3
    for i in range(0, 48, 5):
        d = torch.zeros_like(x)
        d[3, 1, i] = h
        slope = float((g.double() * (turn(x + d) - turn(x - d))).sum()) / (2 * h)
        # two evaluations of 48 elements, each off by 12 * 2^-24 * 1.25 * 10, times |g| < 5, over 2 h
        assert abs(slope - float(back[3, 1, i])) < 2 * 2 * 48 * 12 * 2.0 ** -24 * 1.25 * 10 * 5 / (2 * h)
    again = turn(turn(x).float(), transpose=True)  # magnitude^2 times what is rotated; the rest is copied
    assert float((again[..., :32] / 1.25 ** 2 - x[..., :32].double()).abs().max()) < 1e-5
    assert torch.equal(again[..., 32:], x[..., 32:].double())


def test_fused_rows_in_place_and_apart():
    r = np.random.default_rng(3)
    n, n_q, n_k, hd = 40, 6, 2, 64
    fused = torch.from_numpy(r.standard_normal((n, (n_q + 2 * n_k) * hd))).bfloat16().cuda()
    keep = fused.clone()
    q = fused[:, :n_q * hd].unflatten(1, (n_q, hd))
    k = fused[:, n_q * hd:(n_q + n_k) * hd].unflatten(1, (n_k, hd))
    q0, k0 = q.clone(), k.clone()
    pos, (freq, _) = r.integers(0, 1000, n), kv.rotary_frequencies(32)
    a, b = kv.rotary_embedding(q, k, dev(pos), freq)
    assert torch.equal(fused, keep) and a.is_contiguous() and b.is_contiguous()
    check(a, q0, pos, freq.cpu().numpy())
    qo, ko = kv.rotary_embedding(q, k, dev(pos), freq, query_out=q, key_out=k)
    assert qo.data_ptr() == q.data_ptr() and torch.equal(q, a) and torch.equal(k, b)
    assert torch.equal(fused[:, (n_q + n_k) * hd:], keep[:, (n_q + n_k) * hd:])  # V as it was
    for bad in (fused[:, 8:8 + n_q * hd].unflatten(1, (n_q, hd)), fused[1:, :1]):
        with pytest.raises(ValueError):
            kv.rotary_embedding(q, k, dev(pos), freq, query_out=bad)
    with pytest.raises(ValueError):
        kv.rotary_embedding(q, k, dev(pos), freq, key_out=q[:, :n_k])


def test_infinities_stay_in_their_pair():
    x = torch.ones(2, 1, 64, device="cuda")
    x[0, 0, 3], x[1, 0, 40] = math.inf, math.nan
    freq, _ = kv.rotary_frequencies(64)
    y, _ = kv.rotary_embedding(x, None, dev(np.array([5, 5])), freq)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 0, [3, 35]] = True
    want[1, 0, [8, 40]] = True
    assert torch.equal(bad, want)


def test_captured_and_on_another_stream():
    r = np.random.default_rng(4)
    x = torch.from_numpy(r.standard_normal((100, 8, 128))).bfloat16().cuda()
    pos = dev(r.integers(0, 9000, 100))
    freq, _ = kv.rotary_frequencies(128)
    first, _ = kv.rotary_embedding(x, None, pos, freq)
    out = torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.rotary_embedding(x, None, pos, freq, query_out=out)
    g.replay()
    assert torch.equal(out, first)
    pos.add_(17)
    g.replay()
    check(out, x, pos.cpu().numpy(), freq.cpu().numpy())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again, _ = kv.rotary_embedding(x, None, pos, freq, stream=side)
    side.synchronize()
    assert torch.equal(again, out)


def test_no_tokens():
    freq, _ = kv.rotary_frequencies(64)
    q, k = kv.rotary_embedding(torch.empty(0, 2, 64, device="cuda"), torch.empty(0, 1, 64, device="cuda"),
                               torch.empty(0, dtype=torch.int64, device="cuda"), freq)
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)
