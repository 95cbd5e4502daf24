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
