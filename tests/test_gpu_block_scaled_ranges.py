"""Attention over the FP8 cache with block scales where scales and scores lie far apart, against the oracle.

Bounds are those of test_gpu_block_scaled.py, but for what a small weight may be off by: the weights softmax * vs that meet V are
fp16 with a row's highest at 2^7 at least, so one below 2^-14 is off by 2^-25, 2^-32 of the highest, and a V code is 448 at most.
With H the highest softmax * vs among the tokens that the row sees: L * 2^-32 * H * 448.  |log2 vs| is up to 120 here, and the reference
that scores are taken against up to 15 from the highest: scores in the log2 domain are numbers of at most 1.45 S + 150.  The row's sum
may lose 2^-24 of itself where small weights leave a float's range; a term of it is a float, 2^-149 at least, and the highest one
2^(7 - 120): L * 2^-36 of the sum.
"""
import numpy as np
import pytest
import torch

from oracle import block_scaled as bso
from tests.test_gpu_block_scaled import ROUTES, build, multi, run

pytestmark = pytest.mark.gpu

kv = pytest.importorskip("fp8_paged_kv_reshape_gb300")


def highest(c, causal):
    """[rows, n_q]: the highest softmax * vs of the tokens that a row sees (0: none)."""
    n_q, hd = c["q"].shape[1:]
    bs, n_kv = c["kc"].shape[1:3]
    group, q, out = n_q // n_kv, c["q"].double().numpy(), np.zeros(c["q"].shape[:2])
    for i, length in enumerate(c["lengths"]):
        r0, n = int(c["qsl"][i]), int(c["qsl"][i + 1] - c["qsl"][i])
        t = np.arange(length)
        blk = c["bt"][i, t // bs]
        for h in range(n_kv):
            k = bso.decode(c["kc"][blk, t % bs, h]) * c["ks"][blk, h, None].astype(np.float64)
            for j in range(n):
                sees = length - n + j + 1 if causal else length
                if sees < 1:
                    continue
                x = q[r0 + j, h * group:(h + 1) * group] @ k[:sees].T / np.sqrt(hd)
                p = np.exp(x - x.max(-1, keepdims=True))
                out[r0 + j, h * group:(h + 1) * group] = (p / p.sum(-1, keepdims=True) * c["vs"][blk[:sees], h]).max(-1)
    return out


def check(got, c, causal=True, more=0.0):
    """more: by how much scores may be off besides."""
    hd, longest = c["q"].shape[2], max(c["lengths"])
    ref, weight, reach = bso.attention(c["q"].double().numpy(), c["qsl"], c["kc"], c["vc"], c["ks"], c["vs"], c["bt"], c["lengths"],
                                       causal)
    g = got.double().cpu().numpy()
    d = (hd + 8) * 2.0 ** -24 * (1.45 * reach + 150) + 2.0 ** -21 + more
    d = d + 2.0 ** -24 + longest * 2.0 ** -36  # (the row's sum)
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * d[..., None] + 2 * (longest / 16 + 16) * 2.0 ** -23) * weight \
        + (longest * 2.0 ** -32 * 448 * highest(c, causal))[..., None] + 1e-37
    over = np.abs(g - ref) - bound
    assert np.isfinite(g).all() and over.max() <= 0, (over.max(), np.abs(g - ref).max())


def no_large_codes(c):
    """V codes of 128 at most, so that values under a scale of 2^120 are floats."""
    c["vc"] = np.where((c["vc"] & 0x7F) > 0x70, (c["vc"] & 0x80) | 0x70, c["vc"]).astype(np.uint8)
    return c


LENGTHS = [[300, 77], [3000, 260, 16]]
ORDERS = {"small first": lambda i, n: i >= n // 2, "large first": lambda i, n: i < n // 2, "in turn": lambda i, n: i % 2 == 0,
          "large last": lambda i, n: i == n - 1, "large alone": lambda i, n: i == n // 3, "small alone": lambda i, n: i != n // 3}


def two_scales(order, lengths, small, large):
    """For build(): each sequence's blocks at one of two scales."""
    def scale(r, shape):
        n = [-(-x // 16) for x in lengths]
        return np.concatenate([np.where(ORDERS[order](np.arange(m), m), large, small) for m in n])[:, None] * np.ones(shape)
    return scale


@pytest.mark.parametrize("n_q, n_kv, hd, qlen", ROUTES)
@pytest.mark.parametrize("order", ORDERS)
def test_small_and_large_scales_share_a_row(order, n_q, n_kv, hd, qlen):
    """V scales 60 octaves apart; causal rows that see the small ones alone have those to give back."""
    lengths = LENGTHS[0]
    c = build(n_q, n_kv, hd, 16, lengths, [min(qlen, n) for n in lengths], 41, scale=two_scales(order, lengths, 2.0 ** -40, 2.0 ** 20))
    c["ks"][c["ks"] > 0] = 2.0 ** -8
    for causal in (True, False):
        check(run(multi, c, qlen, causal=causal), c, causal)


@pytest.mark.parametrize("n_q, n_kv, hd, qlen", ROUTES)
@pytest.mark.parametrize("small, octaves", [(2.0 ** -30, 30), (2.0 ** -60, 40), (2.0 ** -60, 55)])
def test_small_scales_hold_the_highest_scores(small, octaves, n_q, n_kv, hd, qlen):
    """A block of a small V scale takes nearly all of the softmax, the others, `octaves` lower in score, nearly all of the output."""
    lengths = [128, 60]
    c = build(n_q, n_kv, hd, 16, lengths, [min(qlen, n) for n in lengths], 44, scale=two_scales("small alone", lengths, 1.0, small))
    c["q"] = torch.ones_like(c["q"])
    for i in (0, 1):
        n = -(-lengths[i] // 16)
        c["kc"][c["bt"][i, :n]] = 0x00
        c["kc"][c["bt"][i, n // 3]] = 0x38  # 1.0
    # a score of hd / sqrt(hd) * ks nats against 0: ks the power of two below, and q what is left
    nats = octaves * np.log(2) / np.sqrt(hd)
    ks = 2.0 ** np.floor(np.log2(nats))
    c["ks"][c["ks"] > 0] = ks
    c["q"] = (c["q"] * (nats / ks)).bfloat16()
    for causal in (True, False):
        check(run(multi, c, qlen, causal=causal), c, causal)


@pytest.mark.parametrize("n_q, n_kv, hd, qlen", ROUTES)
@pytest.mark.parametrize("lengths", LENGTHS, ids=["whole", "split"])
@pytest.mark.parametrize("order", ORDERS)
def test_smallest_and_largest_scales_share_a_row(order, lengths, n_q, n_kv, hd, qlen):
    """V scales of 2^-60 and of 2^120 in one sequence: what the small ones hold adds nothing to the output, but their tokens' weights
    belong to the row's sum."""
    c = no_large_codes(build(n_q, n_kv, hd, 16, lengths, [min(qlen, n) for n in lengths], 41,
                             scale=two_scales(order, lengths, 2.0 ** -60, 2.0 ** 120)))
    c["ks"][c["ks"] > 0] = 2.0 ** -8
    for causal in (True, False):
        check(run(multi, c, qlen, causal=causal), c, causal)


@pytest.mark.parametrize("n_q, n_kv, hd, qlen", ROUTES)
@pytest.mark.parametrize("low, high", [(-60, 1), (-30, 31), (-60, 121), (-30, 121)])
def test_scales_and_scores_far_apart(low, high, n_q, n_kv, hd, qlen):
    """Scales at random, over the whole range too, with scores that lie up to a hundred octaves apart."""
    for lengths, seed in ((LENGTHS[0], 42), (LENGTHS[1], 43)):
        c = no_large_codes(build(n_q, n_kv, hd, 16, lengths, [min(qlen, n) for n in lengths], seed,
                                 scale=lambda r, shape: np.exp2(r.integers(low, high, shape))))
        live = c["ks"] > 0
        c["ks"][live] = np.exp2(np.random.default_rng(seed).integers(-7, 1, int(live.sum())))
        check(run(multi, c, qlen), c)


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("rows", [17, 31, 33, 65, 97, 127, 129, 161, 225])
def test_part_filled_warps_of_split_calls(rows, hd):
    """One sequence whose keys are split over CTAs, with any number of rows in the last warp that has some."""
    c = build(1, 1, hd, 16, [2100], [rows], 45)
    check(run(multi, c, rows), c)
    check(run(multi, c, rows, causal=False), c, False)


@pytest.mark.parametrize("n_q, n_kv, hd, qlen", ROUTES)
@pytest.mark.parametrize("octaves", [9, 11, 13, 16])
def test_small_elements_of_a_query_row_with_a_large_one(octaves, n_q, n_kv, hd, qlen):
    """One element 2^octaves times the row's others, over keys that are 0 there, so that the small elements make the scores."""
    lengths = [300, 77]
    c = build(n_q, n_kv, hd, 16, lengths, [min(qlen, n) for n in lengths], 46)
    q = c["q"].double().numpy()
    q[..., 5] = 0
    q[..., 5] = np.exp2(np.floor(np.log2(np.abs(q).max(-1))) + octaves)
    c["q"] = torch.from_numpy(q).bfloat16()
    c["kc"][..., 5] = 0
    # Up to 16 score columns (8 at head_dim 256) q is fp16, off by 2^-25 below 2^-14.  Beyond, scaled to a largest element of 2^7: an E4M3
    # number leaves 8 last places of a bf16's 8 bits, which E5M2's 3 bits hold, while the first is normal, from 2^-6 = 2^-13 of the
    # largest on; below, what it leaves is 2^-10 at most and E5M2's half step there 2^-14, 2^-21 of the largest.
    q = np.abs(c["q"].double().numpy())
    top = q.max(-1, keepdims=True)
    off = np.where(q >= top * 2.0 ** -13, 0.0, 2.0 ** -21 * top) if qlen >= 30 else np.full(q.shape, 2.0 ** -25)
    k = np.abs(bso.decode(c["kc"])) * c["ks"][:, None, :n_kv, None]  # [block, token, head, dim]
    k = np.repeat(np.nan_to_num(k[c["bt"][c["bt"] >= 0]]).max((0, 1)), n_q // n_kv, 0)
    check(run(multi, c, qlen), c, more=1.45 / np.sqrt(hd) * (off * k).sum(-1))


@pytest.mark.parametrize("n_q, n_kv, hd, qlen", [r for r in ROUTES if r[3] >= 30] + [(20, 1, 128, 1), (36, 4, 256, 1)])
@pytest.mark.parametrize("octaves", [20, 100, 126])
def test_long_chunks_and_wide_groups_take_rows_of_any_size(octaves, n_q, n_kv, hd, qlen):
    """A row 2^octaves times as large, with scales and sm_scale as much smaller, gives the same to the bit: all of these are powers of
    two.  (126: elements up to 2^127, the largest binade.)"""
    lengths = [300, 77]
    c = build(n_q, n_kv, hd, 16, lengths, [min(qlen, n) for n in lengths], 47)
    c["q"] = c["q"].clamp(-2, 2)
    sm = float(np.float32(1 / np.sqrt(hd)))
    want = run(multi, c, qlen, sm_scale=sm)
    check(want, c)
    c["q"] = (c["q"].double() * 2.0 ** octaves).bfloat16()
    c["ks"] *= np.float32(2.0 ** -20)
    assert bool(torch.isfinite(c["q"]).all())
    assert torch.equal(run(multi, c, qlen, sm_scale=sm * 2.0 ** (20 - octaves)), want)


@pytest.mark.parametrize("n_q, n_kv, hd, qlen", [r for r in ROUTES if r[3] < 30])
def test_query_elements_past_fp16_in_a_few_columns(n_q, n_kv, hd, qlen):
    """They are infinities there: the row is NaN where a score is (here some are positive, some negative), the others stay."""
    lengths = [300, 77]
    c = build(n_q, n_kv, hd, 16, lengths, [min(qlen, n) for n in lengths], 48)
    c["q"][0, 1, 7] = 65280.0  # bf16's largest below 65504
    want = run(multi, c, qlen)
    c["q"][0, 1, 7] = 2.0 ** 17
    c["q"][-1, 0, 3] = -2.0 ** 100
    got = run(multi, c, qlen)
    assert bool(torch.isnan(got[0, 1]).all()) and bool(torch.isnan(got[-1, 0]).all())
    got[0, 1], got[-1, 0] = want[0, 1], want[-1, 0]
    assert torch.equal(got, want)
