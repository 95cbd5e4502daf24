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


def leaf(r, *shape, dtype=torch.float32):
    return torch.from_numpy(r.standard_normal(shape)).to(dtype).cuda().requires_grad_()


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_inputs_that_require_a_gradient_get_one(dtype, interleaved):
    """The gradient is the transposed map's, bit for bit what the call itself gives, and that one the oracle's."""
    r = np.random.default_rng(5)
    q, k = leaf(r, 9, 4, 48, dtype=dtype), leaf(r, 9, 2, 48, dtype=dtype)
    pos = r.integers(0, 5000, 9)
    freq, _ = kv.rotary_frequencies(32)
    how = dict(interleaved=interleaved, magnitude=1.25)
    with torch.no_grad():
        plain = kv.rotary_embedding(q, k, dev(pos), freq, **how)
    assert not plain[0].requires_grad and not plain[1].requires_grad
    outs = kv.rotary_embedding(q, k, dev(pos), freq, **how)
    assert all(torch.equal(a, b) for a, b in zip(outs, plain))
    # a gradient that is expanded, one that lies askew in a larger buffer
    gq = torch.from_numpy(r.standard_normal((9, 1, 48))).to(dtype).cuda().expand(9, 4, 48)
    gk = torch.from_numpy(r.standard_normal(9 * 2 * 48 + 1)).to(dtype).cuda()[1:].view(9, 2, 48)
    dq, dk = torch.autograd.grad(outs, (q, k), (gq, gk))
    with torch.no_grad():
        wq, wk = kv.rotary_embedding(gq.contiguous(), gk.clone(), dev(pos), freq, transpose=True, **how)
    assert torch.equal(dq, wq) and torch.equal(dk, wk)
    for d, g in ((dq, gq), (dk, gk)):
        check(d, g, pos, freq.cpu().numpy(), interleaved, 1.25, transpose=True)


def test_gradients_of_one_side_of_none_and_of_gradients():
    r = np.random.default_rng(6)
    pos, (freq, _) = dev(r.integers(0, 5000, 7)), kv.rotary_frequencies(32)
    q, k = leaf(r, 7, 2, 32), leaf(r, 7, 1, 32)
    g = torch.from_numpy(r.standard_normal((7, 1, 32))).float().cuda()
    back = lambda t: kv.rotary_embedding(t, None, pos, freq, transpose=True)[0]  # noqa: E731
    (dk,) = torch.autograd.grad(kv.rotary_embedding(q.detach(), k, pos, freq)[1], k, g)
    assert torch.equal(dk, back(g))
    dq, dk = torch.autograd.grad(kv.rotary_embedding(q, k, pos, freq)[1], (q, k), g, allow_unused=True)
    assert dq is None and torch.equal(dk, back(g))
    y, none = kv.rotary_embedding(k, None, pos, freq)
    assert none is None
    (dk,) = torch.autograd.grad(y, k, g, retain_graph=True)
    assert torch.equal(dk, back(g))
    # the gradient of <h, R^T g> by g is R h
    g.requires_grad_()
    (dk,) = torch.autograd.grad(y, k, g, create_graph=True)
    h = torch.from_numpy(r.standard_normal((7, 1, 32))).float().cuda()
    (dg,) = torch.autograd.grad(dk, g, h)
    assert torch.equal(dg, kv.rotary_embedding(h, None, pos, freq)[0])
    # a position out of range: no gradient to that row
    far = pos.clone()
    far[3] = 2 ** 31
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    junk = torch.full((64, 7, 1, 32), 7.0, device="cuda")  # (what the allocator gives out next)
    del junk
    (dk,) = torch.autograd.grad(kv.rotary_embedding(k, None, far, freq, status=st)[0], k, g.detach())
    want = back(g.detach())
    want[3] = 0
    assert torch.equal(dk, want) and int(st.item()) == kv.DEV_BAD_SLOT


def test_calls_that_have_no_graph_are_refused():
    r = np.random.default_rng(7)
    pos, (freq, _) = dev(r.integers(0, 5000, 4)), kv.rotary_frequencies(32)
    q, k = leaf(r, 4, 2, 32), leaf(r, 4, 1, 32)
    for more in (dict(query_out=torch.empty_like(q)), dict(key_out=torch.empty_like(k)), dict(query_out=q.detach())):
        with pytest.raises(ValueError):
            kv.rotary_embedding(q, k, pos, freq, **more)
        with torch.no_grad():
            kv.rotary_embedding(q, k, pos, freq, **more)
    with pytest.raises(ValueError):
        kv.rotary_embedding(q.detach(), None, pos, freq.clone().requires_grad_())


def test_a_training_step_on_another_stream():
    """Rotate, scores, a loss: its gradients are those of the same written in torch."""
    r = np.random.default_rng(8)
    n, hd = 33, 64
    q, k = leaf(r, n, 4, hd), leaf(r, n, 2, hd)
    pos, (freq, mag) = dev(np.arange(n) * 17), kv.rotary_frequencies(hd, scaling="parts", factor=4.0, original_len=256)
    t = (pos.double()[:, None] * freq)[:, None]
    c, s = t.cos() * mag, t.sin() * mag

    def turned(x):
        a, b = x.double().chunk(2, -1)
        return torch.cat([a * c - b * s, a * s + b * c], -1)

    def loss(a, b):
        return torch.einsum("ihd,jhd->ijh", a, b.repeat_interleave(2, 1)).softmax(1).square().sum()

    want = torch.autograd.grad(loss(turned(q), turned(k)), (q, k))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a, b = kv.rotary_embedding(q, k, pos, freq, magnitude=mag)
        got = torch.autograd.grad(loss(a.double(), b.double()), (q, k))
    torch.cuda.current_stream().wait_stream(side)
    # Rotated values are off by 13 * 2^-24 of |a| + |b| <= 10, so scores of 64 products of values below 7 by 64 * 2 * 7 * 8e-6 =
    # 7e-3 in the worst case; a softmax weight moves by that of itself, and the gradients, sums of such weights times values, with it.
    for w, g in zip(want, got):
        assert float((w - g).abs().max()) <= 4 * 7e-3 * float(w.abs().max())
