"""Attention over the 4-bit cache where every token of every tile counts, over many tiles of one CTA and
at the borders between CTAs.

Random inputs of long sequences hardly show a tile that is lost or counted twice: thousands of small weights
average out.  Here either all weights are equal and each output dim counts the tokens of its own classes of
eight, so that eight tokens more or less move some dim by a few percent, or one token of a row has all the
weight (a needle), and needles lie in every tile.

Bounds.  Counts: equal weights are powers of two and their float32 sums exact, so an output is off by its
rounding to bf16, half a step, at most 2^-8 of the value, and by the float32 quotient and merges, together
below 2^-18 of it.  Needles: all other weights of a row sum to less than 2^-20 of the needle's (asserted), with
values of at most 6.
"""
import math

import numpy as np
import pytest
import torch

from oracle import fp4
from tests.test_gpu_fp4 import check_attention, dev, scalar, status

pytestmark = pytest.mark.gpu

kv = pytest.importorskip("fp8_paged_kv_reshape_gb300")


# n_q, n_kv, head_dim, block, sequences, new tokens of each, shortest and longest
WIDE = [  # more row tiles than half the SMs: each CTA goes through all the keys
    (20, 1, 64, 8, 80, 1, 600, 2300),      # one row tile (17 to 128 score rows), stages of 64 keys
    (4, 1, 128, 32, 78, 8, 600, 2300),
    (24, 8, 128, 16, 11, 7, 1300, 2300),
    (9, 1, 256, 8, 78, 1, 600, 1600),
    (4, 1, 256, 128, 78, 5, 600, 1600),
    (4, 2, 256, 256, 40, 20, 600, 1600),
    (4, 1, 64, 16, 78, 40, 900, 2300),     # two row tiles of 128, 128 keys a time
    (2, 1, 128, 8, 40, 150, 900, 2300),
    (2, 1, 128, 64, 40, 130, 900, 2300),
]
FEW = [  # fewer: the keys are split, over many tiles of a part
    (24, 8, 64, 16, 9, 7, 2800, 3300),
    (32, 8, 128, 8, 9, 5, 2800, 3300),
    (16, 8, 256, 32, 9, 5, 1300, 3300),
    (16, 4, 64, 32, 18, 40, 2800, 3300),
    (8, 4, 128, 16, 17, 70, 2800, 3300),
    (20, 1, 128, 16, 1, 1, 20011, 20011),
]
DECODE = [  # up to 16 score rows: chunks of 32 keys, in ranges of equal length over the CTAs
    (8, 2, 64, 16, 3, 1, 9000, 20011),
    (32, 8, 128, 16, 3, 1, 9000, 20011),
    (32, 2, 128, 8, 2, 1, 9000, 20011),
    (8, 2, 256, 16, 3, 1, 9000, 20011),
    (4, 1, 64, 64, 300, 1, 100, 900),
    (32, 8, 128, 32, 5, 4, 3000, 9000),
    (4, 4, 64, 8, 5, 3, 3000, 9000),
    (4, 2, 256, 16, 5, 4, 3000, 9000),
]


def shared_case(n_kv, hd, bs, seqs, n, lo, hi, seed):
    """One row of pages that all sequences read (a common prefix of each length), and their lengths."""
    r = np.random.default_rng(seed)
    lens = r.integers(lo, hi + 1, seqs)
    lens[0], lens[-1] = hi, lo if seqs > 1 else hi
    pages = -(-hi // bs)
    nb = pages + 3
    row = r.permutation(nb)[:pages].astype(np.int32)
    bt = np.full((seqs, pages), -1, np.int32)
    for i, length in enumerate(lens):
        bt[i, :-(-int(length) // bs)] = row[:-(-int(length) // bs)]
    qsl = (np.arange(seqs + 1) * n).astype(np.int32)
    return r, lens, row, nb, bt, qsl


def place(x, row, nb, bs):
    """Values [tokens, n_kv, hd] that E2M1 holds, under scales of 1, into pages; slots without a token are NaN."""
    n, n_kv, hd = x.shape
    codes = np.full((nb, bs, n_kv, hd // 2), 0x5A, np.uint8)
    scales = np.full((nb, n_kv, bs, hd // 16), 0x7F, np.uint8)
    c = fp4.nearest_code(np.abs(x), fp4.E2M1).astype(np.uint8) + 8 * (x < 0).astype(np.uint8)
    t = np.arange(n)
    codes[row[t // bs], t % bs] = c[..., 0::2] | (c[..., 1::2] << 4)
    scales[row[t // bs], :, t % bs] = 0x38
    return codes, scales


def call(q, qsl, n, kc, vc, kg, vg, bt, lens, ks, vs, sm, st):
    args = [dev(a) for a in (kc, vc, kg, vg, bt, lens.astype(np.int32))]
    if n == 1:
        return kv.paged_decode_attention_fp4(q.cuda(), *args, scalar(ks), scalar(vs), sm, status=st)
    return kv.paged_attention_multi_fp4(q.cuda(), dev(qsl), n, *args, scalar(ks), scalar(vs), sm, status=st)


@pytest.mark.parametrize("n_q, n_kv, hd, bs, seqs, n, lo, hi", WIDE + FEW + DECODE)
def test_each_dim_counts_its_tokens(n_q, n_kv, hd, bs, seqs, n, lo, hi):
    r, lens, row, nb, bt, qsl = shared_case(n_kv, hd, bs, seqs, n, lo, hi, hd + seqs + hi)
    split = kv.paged_attention_fp4_workspace_size(seqs, n_q, n_kv, hd, n, bt.shape[1], bs) > 0
    assert split == ((n_q, n_kv, hd, bs, seqs, n, lo, hi) not in WIDE)
    t = np.arange(hi)
    v = np.zeros((hi, n_kv, hd))
    for h in range(n_kv):
        v[t, h, (t // 8 + 5 * h) % hd] = 1.0
    kc, kg = place(r.choice([-1.0, 1.0, 2.0], (hi, n_kv, hd)), row, nb, bs)
    vc, vg = place(v, row, nb, bs)
    st = status()
    out = call(torch.zeros(seqs * n, n_q, hd, dtype=torch.bfloat16), qsl, n, kc, vc, kg, vg, bt, lens, 0.5, 3.0, 0.0, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    got = out.double().cpu().numpy().reshape(seqs, n, n_kv, n_q // n_kv, hd)
    seen = v.cumsum(0)  # per head and dim, over the tokens up to t
    last = lens[:, None] - n + np.arange(n)
    want = 3.0 * seen[last] / (last + 1.0)[..., None, None]
    assert np.all(np.abs(got - want[:, :, :, None]) <= (2.0 ** -8 + 2.0 ** -18) * want[:, :, :, None])


@pytest.mark.parametrize("n_q, n_kv, hd, bs, seqs, n, lo, hi", WIDE + FEW + DECODE)
def test_every_row_finds_its_needle(n_q, n_kv, hd, bs, seqs, n, lo, hi):
    r, lens, row, nb, bt, qsl = shared_case(n_kv, hd, bs, seqs, n, lo, hi, hd + seqs + hi + 1)
    k = r.choice([-1.0, 1.0], (hi, n_kv, hd))
    v = r.choice(np.concatenate([fp4.E2M1[1:], -fp4.E2M1[1:]]), (hi, n_kv, hd))
    kc, kg = place(k, row, nb, bs)
    vc, vg = place(v, row, nb, bs)
    group = n_q // n_kv
    last = lens[:, None] - n + np.arange(n)
    # needles: the rows of all sequences spread over what they see, the first and the last token among them
    at = (last[..., None] * np.linspace(0, 1, seqs * n * n_q).reshape(seqs, n, n_q).clip(0, 1)).round().astype(np.int64)
    at[0, 0, 0], at[-1, -1, -1] = 0, last[-1, -1]
    kvh = np.arange(n_q) // group
    q = torch.from_numpy(k[at, kvh]).reshape(seqs * n, n_q, hd).bfloat16()
    sm = 0.5 if hd == 64 else 0.25
    # the other scores are at most `high` (checked on some rows): e^(high - hd) of each, hi of them
    for i in r.integers(0, seqs, 8):
        s = k[:lens[i], kvh[0]] @ k[at[i, 0, 0], kvh[0]]
        s[at[i, 0, 0]] = -math.inf
        assert np.exp(sm * (s - hd)).sum() < 2.0 ** -20
    st = status()
    out = call(q, qsl, n, kc, vc, kg, vg, bt, lens, 1.0, 1.0, sm, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    got = out.double().cpu().numpy().reshape(seqs, n, n_q, hd)
    want = v[at, kvh]
    assert np.abs(got - want).max() <= 6 * (2.0 ** -8 + 2.0 ** -19)


@pytest.mark.parametrize("n_q, n_kv, hd, bs, seqs, n, lo, hi", WIDE + FEW)
def test_nan_and_bad_blocks_late_in_the_keys(n_q, n_kv, hd, bs, seqs, n, lo, hi):
    """A NaN of V near the end (which some rows of a chunk see), one in the middle, one of K for the longest
    sequences only, and a block outside the pool, all past the first turn of a ring of stages; a few sequences
    are compared with the oracle, all of them for which outputs are NaN."""
    r, lens, row, nb, bt, qsl = shared_case(n_kv, hd, bs, seqs, n, lo, hi, hd + seqs + hi + 2)
    kc, vc = (r.integers(0, 256, (nb, bs, n_kv, hd // 2)).astype(np.uint8) for _ in "kv")
    kg, vg = (r.integers(0x28, 0x38, (nb, n_kv, bs, hd // 16)).astype(np.uint8) for _ in "kv")
    i = int(np.argsort(lens)[seqs // 2]) if seqs > 1 else 0
    late, middle = int(lens[i]) - 1 - n // 2, max(int(lens[i]) // 2, 560)
    vg[row[late // bs], 0, late % bs, 1] = 0x7F
    vg[row[middle // bs], n_kv - 1, middle % bs, hd // 16 - 1] = 0xFF
    top = hi - 3
    kg[row[top // bs], 0, top % bs, 0] = 0x7F
    bad = int(np.argsort(lens)[0])
    bt[bad, 530 // bs] = nb + 7
    q = torch.from_numpy(r.standard_normal((seqs * n, n_q, hd))).bfloat16()
    st = status()
    out = call(q, qsl, n, kc, vc, kg, vg, bt, lens, 0.05, 0.04, 0.0, st)
    torch.cuda.synchronize()
    assert int(st.item()) == kv.DEV_BAD_BLOCK
    for s in {0, i, bad, seqs - 1}:
        rows = slice(s * n, (s + 1) * n)
        check_attention(out[rows], (q[rows], np.array([0, n]), kc, vc, kg, vg, bt[s:s + 1]), [int(lens[s])], ks=0.05,
                        vs=0.04, one_tile=True)
    # token t is seen by a row when it is not past the row's own, and its block is there
    last = (lens[:, None] - n + np.arange(n)).reshape(-1)
    there = np.ones((seqs, hi), bool)
    there[bad, 530 // bs * bs:(530 // bs + 1) * bs] = False
    there = there.repeat(n, 0)
    group = n_q // n_kv
    nan = np.zeros((seqs * n, n_q, hd), bool)
    nan[:, :group, 16:32] |= ((last >= late) & there[:, late])[:, None, None]
    nan[:, n_q - group:, hd - 16:] |= ((last >= middle) & there[:, middle])[:, None, None]
    nan[:, :group] |= ((last >= top) & there[:, top])[:, None, None]
    assert np.array_equal(torch.isnan(out).cpu().numpy(), nan)


@pytest.mark.parametrize("n_q, n_kv, hd, n, length, others", [
    (4, 2, 64, 1, 90, 2), (32, 8, 128, 1, 5000, 2), (8, 2, 256, 3, 700, 1), (20, 1, 128, 1, 900, 1), (20, 1, 128, 1, 900, 90),
    (8, 2, 256, 20, 900, 1), (4, 1, 64, 75, 900, 1), (4, 1, 128, 75, 900, 50)])
def test_sequences_whose_blocks_are_all_outside_the_pool(n_q, n_kv, hd, n, length, others):
    """Their rows are zero, and the other sequences are as without them."""
    bs, seqs = 16, others + 2
    r, lens, row, nb, bt, qsl = shared_case(n_kv, hd, bs, seqs, n, length, length, 3)
    bt[0], bt[-1] = nb + 1, -1
    kc, vc = (r.integers(0, 256, (nb, bs, n_kv, hd // 2)).astype(np.uint8) for _ in "kv")
    kg, vg = (r.integers(0x28, 0x38, (nb, n_kv, bs, hd // 16)).astype(np.uint8) for _ in "kv")
    q = torch.from_numpy(r.standard_normal((seqs * n, n_q, hd))).bfloat16()
    st = status()
    out = call(q, qsl, n, kc, vc, kg, vg, bt, lens, 0.05, 0.04, 0.0, st)
    torch.cuda.synchronize()
    assert int(st.item()) == kv.DEV_BAD_BLOCK
    assert bool((out[:n] == 0).all()) and bool((out[-n:] == 0).all())
    for s in {1, seqs - 2}:
        rows = slice(s * n, (s + 1) * n)
        check_attention(out[rows], (q[rows], np.array([0, n]), kc, vc, kg, vg, bt[s:s + 1]), [length], ks=0.05, vs=0.04)


def test_more_head_groups_than_the_grid_holds_are_refused():
    """65537 kv heads, a prime: a group of CTAs for each."""
    n_kv, bs, hd = 65537, 8, 64
    c = torch.zeros(1, bs, n_kv, hd // 2, dtype=torch.uint8, device="cuda")
    g = torch.zeros(1, n_kv, bs, hd // 16, dtype=torch.uint8, device="cuda")
    q = torch.zeros(1, n_kv, hd, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(kv.KvFp8Error) as e:
        kv.paged_decode_attention_fp4(q, c, c, g, g, dev(np.zeros((1, 1), np.int32)), dev(np.array([8], np.int32)))
    assert e.value.status == kv.ERR_UNSUPPORTED
    assert int(torch.ones(3, device="cuda").sum().item()) == 3  # and no error is left behind
