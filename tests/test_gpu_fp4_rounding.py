"""What the 4-bit attention keeps of its softmax weights: they enter the products as fp16, and nothing before
them is rounded to fewer than float32's bits."""
import math

import numpy as np
import pytest
import torch

from oracle import fp4
from tests.test_gpu_fp4 import dev, scalar

pytestmark = pytest.mark.gpu

kv = pytest.importorskip("fp8_paged_kv_reshape_gb300")

# n_q, n_kv, head_dim, new tokens, sequences: 80 of one row tile are not split, one is
ROUTES = [
    (4, 1, 64, 1, 2), (16, 1, 128, 1, 2), (4, 1, 128, 4, 2), (8, 1, 256, 1, 2),   # up to 16 score rows
    (20, 1, 64, 1, 80), (8, 1, 128, 5, 80), (4, 1, 256, 30, 80),                  # one row tile
    (20, 1, 128, 1, 1), (17, 1, 64, 2, 1), (9, 1, 256, 1, 1),
    (4, 1, 64, 75, 80), (3, 1, 128, 100, 40),                                     # two row tiles of 128
    (4, 1, 64, 75, 1), (3, 1, 128, 100, 1),
]


def one_and_many(n_q, hd, n, seqs, length, top, x, ks=1.0):
    """A token whose score is x (log2) above the others', with values of zero; the others' values are 1 and 1.5
    under scales of 1 to 1.875.  Returns the outputs and the oracle's, [new tokens, n_q, hd]."""
    bs = 16
    nb = -(-length // bs)
    kc, vc = (np.full((nb, bs, 1, hd // 2), b, np.uint8) for b in (0x22, 0x32))  # 1.0; 1.0 and 1.5
    kg, vg = (np.full((nb, 1, bs, hd // 16), 0x38, np.uint8) for _ in "kv")
    kc[top // bs, top % bs], vc[top // bs, top % bs] = 0x33, 0                   # 1.5; 0
    vg[..., :] += (np.arange(hd // 16) % 8).astype(np.uint8)
    q = torch.ones(seqs * n, n_q, hd, dtype=torch.bfloat16)
    qsl = (np.arange(seqs + 1) * n).astype(np.int32)
    bt = np.arange(nb, dtype=np.int32)[None].repeat(seqs, 0)
    lens = np.full(seqs, length, np.int32)
    sm = float(np.float32(x * math.log(2) / (hd / 2) / abs(ks)))
    if ks < 0:  # the other way round, so that the same token is highest
        q = -q
    args = [dev(a) for a in (kc, vc, kg, vg, bt, lens)] + [scalar(ks), scalar(1.0), sm]
    out = kv.paged_decode_attention_fp4(q.cuda(), *args) if n == 1 else \
        kv.paged_attention_multi_fp4(q.cuda(), dev(qsl), n, *args)
    got = out.double().cpu().numpy().reshape(seqs, n, n_q, hd)
    assert np.array_equal(got, got[:1].repeat(seqs, 0))
    ref, _ = fp4.attention(q[:n].double().numpy(), np.array([0, n]), kc, vc, kg, vg, bt, lens[:1], ks, 1.0, sm)
    return got[0], ref


@pytest.mark.parametrize("n_q, n_kv, hd, n, seqs", ROUTES)
def test_weights_are_rounded_once(n_q, n_kv, hd, n, seqs):
    """All weights but the highest are 2^-x of it, x from 8 to 14 and next to halfway between two fp16 numbers, so
    that the exponent rounded to fp16 would move all of them by 0.96 * 2^-8 log2 and the outputs by 2^-8.6.

    The weights are fp16 numbers of 11 bits here: 2^-11.  The scores are float32 sums of at most 256 products
    of equal size, below 3 * 14 log2: (256 + 4) * 2^-24 * 42 < 2^-10.5 at worst and, as the sums of ones that they
    are, exact but for their scaling: 42 * 2^-22 < 2^-16 log2.  So 2^-10.5 of the value covers both, and the
    output's own rounding is half a step of its binade."""
    length = 600
    for x in 8 + 0.375 * np.arange(16) + 0.96 * 2.0 ** -8:
        for ks in (1.0, -0.5):
            got, ref = one_and_many(n_q, hd, n, seqs, length, 0, x, ks)
            half = 2.0 ** (np.floor(np.log2(ref * (1 + 2.0 ** -10))) - 8)
            over = np.abs(got - ref) - (half + 2.0 ** -10.5 * ref)
            assert over.max() <= 0, (x, ks, (np.abs(got - ref) / ref).max())


@pytest.mark.parametrize("length", [200, 5000])
@pytest.mark.parametrize("n_q, n_kv, hd, n, seqs", ROUTES)
def test_a_tail_of_small_weights_counts_on_every_route(n_q, n_kv, hd, n, seqs, length):
    """Weights 2^-25.5 of the highest, whose values are zero: the outputs are the tail's share alone.

    The highest weight of a row is 2^7 at least, so the others are 2^-18.5 at least, 45 of fp16's smallest
    steps: half a step is 2^-6.5 of them.  The output's rounding adds 2^-8 and the scores 2^-10.5 as above, with
    77 for 42 log2: within 2^-6 in all."""
    for top in (0, length // 2) if n == 1 else (0,):
        got, ref = one_and_many(n_q, hd, n, seqs, length, top, 25.5)
        assert np.abs(got / ref - 1).max() < 2.0 ** -6, top


@pytest.mark.parametrize("n_q, n_kv, hd, n, seqs", ROUTES)
def test_scores_rising_along_the_keys(n_q, n_kv, hd, n, seqs):
    """The highest score comes up by a step every 64 tokens, so the weights' reference moves with it (or lags): by
    3 log2 (six tiles reach past what a reference may lag behind), by 14, by 15.5 and by 40.

    Each output dim belongs to one token class of 64, with value 1, so that its output is that class's
    share.  The classes' weights are fp16 numbers (2^-11 each) above 2^-14 of 2^7, and the class shares of a row
    differ by powers 2^-step; shares below 2^-20 are not compared closely.  bf16: 2^-8."""
    bs, length = 16, 64 * 9 + 5
    nb = -(-length // bs)
    cls = np.arange(length) // 64
    for step in (3.0, 14.0, 15.5, 40.0):
        kc = np.zeros((nb, bs, 1, hd // 2), np.uint8)
        kg, vg = (np.full((nb, 1, bs, hd // 16), 0x38, np.uint8) for _ in "kv")
        vc = np.zeros((nb, bs, 1, hd // 2), np.uint8)
        for t in range(length):
            kc[t // bs, t % bs, 0, 0] = 0x02                     # dim 0 is 1 under a scale of 1 + class
            kg[t // bs, 0, t % bs, 0] = (0x00, 0x38, 0x40, 0x44, 0x48, 0x4A, 0x4C, 0x4E, 0x50, 0x51)[cls[t]]
            vc[t // bs, t % bs, 0, cls[t]] = 0x22                # dims 2c, 2c + 1
        q = torch.zeros(seqs * n, n_q, hd, dtype=torch.bfloat16)
        q[..., 0] = 1.0
        qsl = (np.arange(seqs + 1) * n).astype(np.int32)
        bt = np.arange(nb, dtype=np.int32)[None].repeat(seqs, 0)
        lens = np.full(seqs, length, np.int32)
        args = [dev(a) for a in (kc, vc, kg, vg, bt, lens)] + [scalar(1.0), scalar(1.0), step * math.log(2)]
        out = kv.paged_decode_attention_fp4(q.cuda(), *args) if n == 1 else \
            kv.paged_attention_multi_fp4(q.cuda(), dev(qsl), n, *args)
        got = out.double().cpu().numpy().reshape(seqs, n, n_q, hd)
        assert np.array_equal(got, got[:1].repeat(seqs, 0))
        ref, _ = fp4.attention(q[:n].double().numpy(), np.array([0, n]), kc, vc, kg, vg, bt, lens[:1], 1.0, 1.0,
                               step * math.log(2))
        # (2^-16 of float32 error in scores of up to 360 log2)
        near = np.where(ref > 2.0 ** -20, (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13) * ref, 2.0 ** -6 * ref + 2.0 ** -30)
        assert np.all(np.abs(got[0] - ref) <= near), step


@pytest.mark.parametrize("n_q, n_kv, hd, n, seqs", ROUTES)
def test_small_queries_are_multiples_of_2_to_the_minus_24(n_q, n_kv, hd, n, seqs):
    """q of multiples of 2^-24 (here up to 2^-17) enters exactly; with a softmax scale that makes
    scores of order 1 the outputs are those of the same q times 2^20, to the bit: every product, sum and scaled
    score is a power of two apart."""
    r = np.random.default_rng(n_q + hd)
    bs, length = 16, 700
    nb = -(-length // bs)
    caches = [r.integers(0, 256, (nb, bs, 1, hd // 2)).astype(np.uint8) for _ in "kv"]
    caches += [r.integers(0x28, 0x38, (nb, 1, bs, hd // 16)).astype(np.uint8) for _ in "kv"]
    q = torch.from_numpy(r.integers(-128, 129, (seqs * n, n_q, hd)) * 2.0 ** -24).bfloat16().cuda()
    args = [dev(a) for a in caches] + [dev(np.arange(nb, dtype=np.int32)[None].repeat(seqs, 0)),
                                       dev(np.full(seqs, length, np.int32)), scalar(1.0), scalar(1.0)]
    qsl = dev((np.arange(seqs + 1) * n).astype(np.int32))
    small, large = (kv.paged_decode_attention_fp4(x, *args, sm) if n == 1 else
                    kv.paged_attention_multi_fp4(x, qsl, n, *args, sm)
                    for x, sm in ((q, 2.0 ** 14), (q * 2.0 ** 20, 2.0 ** -6)))
    assert torch.equal(small, large) and bool(torch.isfinite(small).all())
    assert len(torch.unique(small)) > 100
