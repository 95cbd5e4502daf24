"""The 4-bit cache on the GPU against the oracle: bytes bit for bit, attention within derived bounds.

Bounds of attention (all relative to A = sum p|v| / sum p of the row and dim, unless said):
  * the bf16 result is off by at most half a step, 2^-8 of the value;
  * the weights enter the products as fp16: 2^-11 of each, so 2^-11 A, and 2^-25 absolute below
    2^-14, so at most L * 2^-25 * max|v| (the largest weight of a row is 1, the sum at least 1);
  * the scores are float32 sums of hd exact products, off by at most (hd + 4) * 2^-24 of
    sum |q k|, which moves a weight by that relative amount, in numerator and denominator; the
    inputs here keep sum |q k| * scale below 64, so (256 + 4) * 2^-24 * 64 * 2 < 2^-8 * 0.6 at
    hd 256 and 2^-9 * 0.6 at 128: 2^-8 A covers it with exp2's and the merge's float32 errors;
  * the one-row-tile kernel rounds the exponent's argument to fp16 (at most 2^3 above the running
    maximum, falling towards smaller weights): 0.69 * 2^3 * 2^-11 < 2^-8 of a weight, in numerator
    and row sum: 2^-7 A.
"""
import math

import numpy as np
import pytest
import torch

from oracle import fp4

pytestmark = pytest.mark.gpu

kv = pytest.importorskip("fp8_paged_kv_reshape_gb300")

KS, VS = 0.05, 0.04


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def scalar(x, dtype=torch.float32):
    return torch.tensor([x], dtype=dtype, device="cuda")


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def empty_cache(nb, bs, n_kv, hd):
    """Sentinel bytes; an unwritten scale is NaN, so anything that reads one shows it."""
    return np.full((nb, bs, n_kv, hd // 2), 0x5A, np.uint8), np.full((nb, n_kv, bs, hd // 16), 0x7F, np.uint8)


# ---------------------------------------------------------------- writer

def check_write(k, v, slots, nb, bs, ks, vs, scale_dtype=torch.float32, want_status=0):
    n_kv, hd = k.shape[1:]
    sides = []
    for x, s in ((k, ks), (v, vs)):
        c, g = empty_cache(nb, bs, n_kv, hd)
        sc = 1.0 if s is None else float(torch.tensor([s], dtype=scale_dtype).float())
        fp4.write(x.float().cpu().numpy(), c, g, slots, sc)
        sides.append((c, g))
    got = [[dev(a) for a in empty_cache(nb, bs, n_kv, hd)] for _ in range(2)]
    st = status()
    kv.reshape_and_cache_fp4(k, v, got[0][0], got[1][0], got[0][1], got[1][1], dev(slots),
                             None if ks is None else scalar(ks, scale_dtype),
                             None if vs is None else scalar(vs, scale_dtype), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == want_status
    for (c, g), (gc, gg) in zip(sides, got):
        assert np.array_equal(gg.cpu().numpy(), g)
        assert np.array_equal(gc.cpu().numpy(), c)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n, n_kv, hd, bs", [(1, 1, 64, 8), (7, 2, 64, 16), (33, 5, 64, 32), (100, 8, 128, 16),
                                             (65, 3, 256, 64), (17, 12, 128, 128), (40, 1, 256, 256), (300, 33, 64, 8)])
def test_write_matches_the_oracle(dtype, n, n_kv, hd, bs):
    r = np.random.default_rng(n)
    nb = n // bs + 2
    slots = r.permutation(nb * bs)[:n].astype(np.int64)
    slots[r.random(n) < 0.1] = -1
    x = torch.from_numpy(r.standard_normal((2, n, n_kv, hd)) * 1.5).to(dtype).cuda()
    check_write(x[0], x[1], slots, nb, bs, KS, VS)


@pytest.mark.parametrize("scale_dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("ks, vs", [(None, None), (-0.3, 2.0), (1e-20, 3e19), (1e-37, 1e37), (1e-3, -1e-3)])
def test_write_scales(scale_dtype, ks, vs):
    r = np.random.default_rng(5)
    x = torch.from_numpy(r.standard_normal((2, 64, 2, 64)) * np.exp(3 * r.standard_normal((2, 64, 1, 1)))).float()
    x[1] *= abs(vs or 1) if abs(vs or 1) < 1e30 else 1.0
    check_write(x[0].cuda(), x[1].cuda(), np.arange(64), 4, 16, ks, vs, scale_dtype)


def test_write_strides_and_alignment():
    r = np.random.default_rng(6)
    for dtype, pads in ((torch.bfloat16, (0, 8, 16)), (torch.float32, (0, 4, 8))):
        for pad in pads:  # a slice of a fused row: 16-byte aligned starts and strides, 32 or not
            wide = torch.from_numpy(r.standard_normal((20, 3 * 256 + pad))).to(dtype).cuda()
            k = wide[:, pad:pad + 256].unflatten(1, (4, 64))
            v = wide[:, 256 + pad:512 + pad].unflatten(1, (4, 64))
            check_write(k, v, r.permutation(32)[:20].astype(np.int64), 2, 16, KS, VS)


def test_write_corner_values():
    x = torch.zeros(2, 8, 1, 64)
    big = torch.finfo(torch.float32).max
    x[0, 0] = -0.0
    x[0, 1, 0, :20] = torch.tensor([math.nan, 1.0] * 10)
    x[0, 2, 0, :6] = torch.tensor([math.inf, -math.inf, 1.0, -big, 0.0, -0.0])
    x[0, 3, 0, :4] = torch.tensor([1e-12, -1e-12, 1e-44, -1e-44])
    x[0, 4, 0, :3] = torch.tensor([big, -big, 1.0])
    x[0, 5, 0, 16:24] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x[0, 6, 0, 16:24] = -x[0, 5, 0, 16:24]
    x[0, 7] = torch.linspace(-3000, 3000, 64)
    x[1] = x[0].flip(0) * 0.5
    for s in (1.0, -1.0, 1e-30, 1e30, 0.05):
        check_write(x[0].cuda(), x[1].cuda(), np.arange(8), 1, 8, s, 1.0)
        check_write(x[0].bfloat16().cuda(), x[1].bfloat16().cuda(), np.arange(8), 1, 8, s, 1.0)


@pytest.mark.parametrize("s", [1.0, 0.05, -0.7])
def test_write_every_bf16_magnitude_under_every_group_scale(s):
    """Groups of all finite bf16 values near and below their maximum: 15 neighbours of every halfway point
    under group maxima over eight octaves."""
    tops = torch.arange(0x3F80 - 512, 0x3F80 + 512, dtype=torch.int16).view(torch.bfloat16).float()
    r = torch.rand(len(tops), 4, 15, generator=torch.Generator().manual_seed(7))
    x = torch.cat([tops[:, None, None].expand(-1, 4, 1), tops[:, None, None] * r], -1).reshape(-1, 1, 64)
    x = x * torch.where(torch.rand(x.shape, generator=torch.Generator().manual_seed(8)) < 0.5, -1.0, 1.0)
    grid = (tops[:, None] * torch.arange(1, 65)[None, :] / 64).reshape(-1, 1, 64)
    x = torch.cat([x, grid]).bfloat16().cuda()
    n = x.shape[0]
    check_write(x, -x, np.arange(n), n // 16, 16, s, 1.0)


def test_write_bad_slots_and_scales():
    x = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    check_write(x, x, np.array([3, 32, -2, 7]), 2, 16, KS, VS, want_status=kv.DEV_BAD_SLOT)
    for bad in (0.0, math.nan, math.inf):
        caches = [dev(a) for _ in range(2) for a in empty_cache(2, 16, 2, 64)]
        st = status()
        kv.reshape_and_cache_fp4(x, x, caches[0], caches[2], caches[1], caches[3], dev(np.arange(4)),
                                 scalar(1.0), scalar(bad), status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == kv.DEV_BAD_SCALE
        assert all(bool((c == v).all()) for c, v in zip(caches, (0x5A, 0x7F, 0x5A, 0x7F)))


# ---------------------------------------------------------------- rows read back

@pytest.mark.parametrize("dst", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n, n_kv, hd, bs", [(1, 1, 64, 8), (50, 5, 64, 16), (200, 8, 128, 32), (31, 9, 256, 8)])
def test_dequant_matches_the_oracle(dst, n, n_kv, hd, bs):
    r = np.random.default_rng(n)
    nb = 6
    codes = r.integers(0, 256, (nb, bs, n_kv, hd // 2)).astype(np.uint8)
    scales = r.integers(0, 256, (nb, n_kv, bs, hd // 16)).astype(np.uint8)  # NaN and negative ones too
    slots = r.integers(-1, nb * bs, n)  # some twice
    slots[0] = nb * bs
    for s in (None, -0.3, 1e30):
        st = status()
        out = kv.dequant_fp4(dev(codes), dev(scales), dev(slots), dst, None if s is None else scalar(s), status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == kv.DEV_BAD_SLOT
        want = torch.from_numpy(fp4.dequant(codes, scales, slots, s or 1.0)).to(dst)
        assert torch.equal(torch.isnan(out.cpu()), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(out.cpu()), torch.nan_to_num(want))


def test_dequant_unaligned_destination_and_bad_scale():
    codes, scales = empty_cache(2, 16, 2, 64)
    scales[:] = 0x38
    buf = torch.full((4 * 128 + 8,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = buf[8:].view(4, 2, 64)  # 16-byte, not 32-byte aligned
    kv.dequant_fp4(dev(codes), dev(scales), dev(np.array([0, 5, -1, 31])), out=out)
    assert torch.equal(out.cpu(), torch.from_numpy(fp4.dequant(codes, scales, np.array([0, 5, -1, 31]), 1.0)).bfloat16())
    assert bool((buf[:8] == 9).all())
    st = status()
    out.fill_(7)
    kv.dequant_fp4(dev(codes), dev(scales), dev(np.arange(4)), scale=scalar(0.0), out=out, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == kv.DEV_BAD_SCALE and bool((out == 7).all())


# ---------------------------------------------------------------- attention

def build(n_q, n_kv, hd, bs, lengths, qlens, seed, spare=3):
    """Caches in which every slot that no sequence holds has NaN scales, tables with -1 past each sequence."""
    r = np.random.default_rng(seed)
    need = [-(-n // bs) for n in lengths]
    nb = sum(need) + spare
    perm = r.permutation(nb).astype(np.int32)
    bt = np.full((len(lengths), max(1, max(need))), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        bt[i, :n] = perm[at:at + n]
        at += n
    slots = np.concatenate([bt[i, np.arange(n) // bs].astype(np.int64) * bs + np.arange(n) % bs
                            for i, n in enumerate(lengths)] + [np.zeros(0, np.int64)]).astype(np.int64)
    kc, kg = empty_cache(nb, bs, n_kv, hd)
    vc, vg = empty_cache(nb, bs, n_kv, hd)
    for c, g, s in ((kc, kg, KS), (vc, vg, VS)):
        fp4.write(r.standard_normal((len(slots), n_kv, hd)).astype(np.float32), c, g, slots, s)
    qsl = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    q = torch.from_numpy(r.standard_normal((int(qsl[-1]), n_q, hd))).bfloat16()
    return q, qsl, kc, vc, kg, vg, bt


def bound(ref, weight, lengths, vmax, one_tile=False):
    n = max(list(lengths) + [1])
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -8 + (2.0 ** -7 if one_tile else 0)) * weight \
        + n * 2.0 ** -25 * vmax + 1e-30


def check_attention(got, case, lengths, ks=KS, vs=VS, sm=0.0, one_tile=False):
    q, qsl, kc, vc, kg, vg, bt = case
    ref, weight = fp4.attention(q.double().numpy(), qsl, kc, vc, kg, vg, bt, lengths, ks, vs, sm)
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(ref))
    fine = ~np.isnan(ref)
    held = fp4.rows(vc, vg, np.arange(vc.shape[0] * vc.shape[1]))
    vmax = abs(vs) * np.nanmax(np.abs(held), initial=0.0)
    over = np.abs(g - ref)[fine] - bound(ref, weight, lengths, vmax, one_tile)[fine]
    assert over.size == 0 or over.max() <= 0, (over.max(), np.abs(g - ref)[fine].max())


def decode(case, lengths, ks=KS, vs=VS, **more):
    q, _, kc, vc, kg, vg, bt = case
    return kv.paged_decode_attention_fp4(q.cuda(), dev(kc), dev(vc), dev(kg), dev(vg), dev(bt),
                                         dev(np.array(lengths, np.int32)), scalar(ks), scalar(vs), **more)


def multi(case, lengths, qmax, ks=KS, vs=VS, **more):
    q, qsl, kc, vc, kg, vg, bt = case
    return kv.paged_attention_multi_fp4(q.cuda(), dev(qsl), qmax, dev(kc), dev(vc), dev(kg), dev(vg), dev(bt),
                                        dev(np.array(lengths, np.int32)), scalar(ks), scalar(vs), **more)


DECODE = [
    # n_q, n_kv, head_dim, block, lengths
    (4, 2, 64, 16, [17, 33, 64, 100]),
    (2, 2, 64, 8, [1, 7, 8, 9, 0, 24]),
    (32, 8, 128, 16, [1000, 1, 16, 15, 0, 257]),
    (8, 1, 128, 32, [31, 32, 33, 500]),
    (64, 8, 128, 8, [12, 200, 3]),
    (48, 4, 128, 64, [63, 65, 300]),          # 12 heads a group: two score tiles
    (16, 1, 64, 256, [255, 257, 600]),        # 16 heads a group
    (12, 12, 64, 16, [90, 5]),                # two head groups of six
    (32, 4, 256, 16, [1, 250, 77]),           # 8 heads a group at head_dim 256
    (7, 7, 256, 8, [40, 13]),
    (20, 1, 128, 16, [70, 0, 129]),           # 20 heads a group: the tensor-core kernel
    (36, 4, 256, 32, [65, 10]),               # 9 heads at head_dim 256: the tensor-core kernel
    (128, 1, 64, 16, [200]),
]


@pytest.mark.parametrize("n_q, n_kv, hd, bs, lengths", DECODE)
def test_decode_matches_the_oracle(n_q, n_kv, hd, bs, lengths):
    case = build(n_q, n_kv, hd, bs, lengths, [1] * len(lengths), n_q + hd + bs)
    st = status()
    out = decode(case, lengths, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_attention(out, case, lengths, one_tile=n_q // n_kv > (16 if hd < 256 else 8))


@pytest.mark.parametrize("hd, n_q, n_kv", [(64, 8, 2), (128, 32, 8), (128, 32, 2), (256, 8, 2)])
def test_decode_long_sequences_split_over_the_grid(hd, n_q, n_kv):
    lengths = [20011, 1, 9000]
    case = build(n_q, n_kv, hd, 16, lengths, [1, 1, 1], 11)
    check_attention(decode(case, lengths), case, lengths)


def test_decode_scales_and_softmax_scale():
    lengths = [50, 20]
    case = build(8, 2, 128, 16, lengths, [1, 1], 12)
    for ks, vs, sm in ((-0.05, 0.04, 0.0), (0.05, -2.0, 0.3), (1e-4, 1e4, 0.01)):
        check_attention(decode(case, lengths, ks, vs, sm_scale=sm), case, lengths, ks, vs, sm)
    for bad in (0.0, math.inf, math.nan):
        st = status()
        out = torch.full((2, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        decode(case, lengths, bad, VS, out=out, status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == kv.DEV_BAD_SCALE and bool((out == 7).all())


MULTI = [
    # n_q, n_kv, head_dim, block, lengths, query counts
    (4, 4, 64, 16, [4, 30, 257], [4, 4, 4]),
    (32, 8, 128, 16, [1000, 17, 4, 5], [4, 1, 3, 4]),
    (8, 8, 128, 8, [100, 16, 40], [16, 16, 9]),
    (4, 2, 256, 64, [129, 300], [4, 2]),
    (8, 2, 64, 32, [50, 80, 0], [0, 3, 0]),
    (32, 8, 128, 16, [300, 64, 21], [20, 64, 21]),      # one row tile, 80 rows and more
    (16, 2, 128, 16, [500, 129, 40], [130, 129, 1]),    # two row tiles
    (8, 2, 64, 8, [300, 77], [200, 77]),
    (4, 1, 64, 64, [400], [300]),
    (6, 2, 256, 16, [150, 33], [60, 33]),
    (24, 8, 64, 256, [513, 260], [100, 260]),
    (8, 1, 128, 128, [1, 700], [1, 70]),
]


def route_one_tile(n_q, n_kv, hd, qmax):
    cols = qmax * (n_q // n_kv)
    return cols > (8 if hd == 256 else 16) and (hd == 256 or cols <= 128)


@pytest.mark.parametrize("n_q, n_kv, hd, bs, lengths, qlens", MULTI)
def test_multi_matches_the_oracle(n_q, n_kv, hd, bs, lengths, qlens):
    case = build(n_q, n_kv, hd, bs, lengths, qlens, n_q + hd + bs)
    st = status()
    out = multi(case, lengths, max(qlens), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_attention(out, case, lengths, one_tile=route_one_tile(n_q, n_kv, hd, max(qlens)))


@pytest.mark.parametrize("n", [255, 256, 257, 700])
@pytest.mark.parametrize("longest", [250, 300])
def test_many_short_sequences(n, longest):
    """Both plans of the split, and sequences taken whole; some empty, some without queries."""
    r = np.random.default_rng(n + longest)
    lengths = r.integers(0, longest + 1, n)
    lengths[5] = longest
    lengths = lengths.tolist()
    case = build(4, 2, 64, 16, lengths, [1] * n, 26)
    st = status()
    out = decode(case, lengths, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_attention(out, case, lengths)
    qlens = np.minimum(r.integers(0, 4, n), lengths).tolist()
    case = build(4, 2, 64, 16, lengths, qlens, 27)
    out = multi(case, lengths, 3, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_attention(out, case, lengths)


SPLIT = [
    # few rows on long contexts: the tensor-core kernels' keys are split
    # n_q, n_kv, head_dim, block, lengths, new tokens, width of the tables beyond the longest
    (14, 2, 64, 32, [3000], [37], 0),             # 259 rows: two tiles of 256
    (14, 2, 64, 16, [4000, 700, 30], [9, 18, 2], 0),
    (8, 2, 128, 16, [2500], [5], 0),
    (24, 8, 128, 8, [3000, 100], [60, 60], 3000),  # wide tables
    (4, 4, 128, 64, [1300], [300], 0),            # the first rows see 1001 keys
    (16, 4, 256, 8, [2100], [8], 0),
    (6, 2, 256, 32, [1000, 515, 0, 256], [40, 100, 0, 256], 500),
]


@pytest.mark.parametrize("n_q, n_kv, hd, bs, lengths, qlens, wide", SPLIT)
def test_multi_with_split_keys(n_q, n_kv, hd, bs, lengths, qlens, wide):
    case = list(build(n_q, n_kv, hd, bs, lengths, qlens, 41))
    case[6] = np.concatenate([case[6], np.full((len(lengths), wide), -1, np.int32)], 1)
    assert kv.paged_attention_fp4_workspace_size(len(lengths), n_q, n_kv, hd, max(qlens), case[6].shape[1], bs) > 0
    check_attention(multi(tuple(case), lengths, max(qlens)), tuple(case), lengths, one_tile=True)


@pytest.mark.parametrize("n_q, n_kv, hd, lengths", [(20, 1, 128, [3000, 0, 129]), (64, 2, 64, [5000]), (36, 4, 256, [1500, 10])])
def test_decode_of_wide_groups_with_split_keys(n_q, n_kv, hd, lengths):
    case = build(n_q, n_kv, hd, 16, lengths, [1] * len(lengths), 42)
    check_attention(decode(case, lengths), case, lengths, one_tile=True)


def test_split_keys_nan_bad_blocks_and_a_workspace_of_the_callers():
    lengths, n = [2000], 40
    for side, hd, n_q in (("k", 128, 8), ("v", 128, 8), ("v", 256, 4), ("v", 64, 4)):
        case = build(n_q, 2, hd, 16, lengths, [n], 43)
        q, qsl, kc, vc, kg, vg, bt = case
        (vg if side == "v" else kg)[bt[0, 1980 // 16], 1, 1980 % 16, 2] = 0x7F  # seen by the last 20 rows
        check_attention(multi(case, lengths, n), case, lengths, one_tile=True)
    case = list(build(8, 2, 128, 16, lengths, [n], 44))
    case[6] = case[6].copy()
    case[6][0, 20] = -5
    st, need = status(), kv.paged_attention_fp4_workspace_size(1, 8, 2, 128, n, 125, 16)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    got = multi(tuple(case), lengths, n, workspace=ws[:need], status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == kv.DEV_BAD_BLOCK and bool((ws[need:] == 0xFF).all())
    check_attention(got, tuple(case), lengths, one_tile=True)
    with pytest.raises(kv.KvFp8Error):
        multi(tuple(case), lengths, n, workspace=ws[:need - 16])


@pytest.mark.parametrize("length", [200, 5000])  # taken whole, and split
@pytest.mark.parametrize("hd, n_q, n", [(64, 4, 1), (128, 8, 1), (128, 16, 1), (256, 8, 1), (64, 8, 2), (128, 4, 2)])
def test_a_tail_of_small_weights_beside_one_large(hd, n_q, n, length):
    """Weights 2^-25.5 of the highest, whose value is zero: the output is the tail's share alone.

    The weights are off by 2^-25 in fp16 at 2^7 times their ratio, so by 2^-6.5 of themselves, and the
    output's rounding by 2^-8 more: within 2^-6, the float32 errors of scores near 77 included."""
    bs = 16
    nb = -(-length // bs)
    codes = np.full((nb, bs, 1, hd // 2), 0x22, np.uint8)       # 1.0
    kc, vc = codes.copy(), codes.copy()
    kc[0, 0], vc[0, 0] = 0x33, 0                                # 1.5 and 0 at token 0
    one = np.full((nb, 1, bs, hd // 16), 0x38, np.uint8)
    q = torch.ones(n, n_q, hd, dtype=torch.bfloat16)
    case = (q, np.array([0, n], np.int32), kc, vc, one, one.copy(), np.arange(nb, dtype=np.int32)[None])
    sm = 25.5 * math.log(2) / (hd / 2)
    got = multi(case, [length], n, 1.0, 1.0, sm_scale=sm) if n > 1 else decode(case, [length], 1.0, 1.0, sm_scale=sm)
    ref, _ = fp4.attention(q.double().numpy(), case[1], kc, vc, one, one, case[6], [length], 1.0, 1.0, sm)
    assert np.abs(got.double().cpu().numpy() / ref - 1).max() < 2.0 ** -6


def test_multi_of_one_query_each_is_decode():
    lengths = [333, 17, 1200]
    case = build(32, 8, 128, 16, lengths, [1, 1, 1], 4)
    assert torch.equal(multi(case, lengths, 1), decode(case, lengths))


@pytest.mark.parametrize("n_q, n_kv, hd, bs, length, n", [(8, 2, 64, 16, 50, 4), (32, 8, 128, 16, 70, 4), (8, 8, 128, 8, 40, 16),
                                                          (4, 2, 256, 16, 60, 4), (32, 8, 128, 16, 70, 20),
                                                          (16, 2, 128, 16, 200, 100), (8, 2, 64, 16, 150, 120), (4, 2, 256, 16, 60, 30)])
def test_a_nan_reaches_exactly_the_rows_and_dims_that_see_it(n_q, n_kv, hd, bs, length, n):
    """NaN in V of a token that only the last few queries see, then in K, then in the last token alone."""
    for side, tok in (("v", length - 2), ("k", length - 2), ("v", length - 1), ("v", 3)):
        case = build(n_q, n_kv, hd, bs, [length, 20], [n, 1], 21)
        q, qsl, kc, vc, kg, vg, bt = case
        (vg if side == "v" else kg)[bt[0, tok // bs], n_kv - 1, tok % bs, 1] = 0x7F
        out = multi(case, [length, 20], n)
        check_attention(out, case, [length, 20], one_tile=route_one_tile(n_q, n_kv, hd, n))
        seen = ~torch.isfinite(out.float()).all(-1).all(-1)
        assert bool(seen.any()) and not bool(seen[-1])


def test_long_chunks_of_caches_full_of_nans():
    """NaN groups all over V, at every row's last tokens among them: each row sees its own."""
    r = np.random.default_rng(45)
    for n_q, hd, lengths, qlens in ((8, 128, [700, 90], [200, 90]), (4, 64, [1500], [30]), (4, 256, [600], [70])):
        case = build(n_q, 2, hd, 16, lengths, qlens, 46)
        vg, bt = case[5], case[6]
        for s, length in enumerate(lengths):
            for t in r.integers(max(0, length - max(qlens) - 20), length, 12):
                vg[bt[s, t // 16], r.integers(2), t % 16, r.integers(hd // 16)] = 0x7F
        check_attention(multi(case, lengths, max(qlens)), case, lengths, one_tile=True)


def test_decode_nan_in_a_split_sequence():
    lengths = [9000, 40]
    for side in ("k", "v"):
        case = build(8, 2, 128, 16, lengths, [1, 1], 22)
        q, qsl, kc, vc, kg, vg, bt = case
        (vg if side == "v" else kg)[bt[0, 5000 // 16], 1, 5000 % 16, 2] = 0x7F
        check_attention(decode(case, lengths), case, lengths)


def test_bad_blocks_lengths_and_query_rows_are_flagged():
    lengths = [40, 60, 20]
    case = build(8, 2, 64, 16, lengths, [1, 1, 1], 23)
    bad = list(case)
    bad[6] = case[6].copy()
    bad[6][1, 2] = case[2].shape[0]  # tokens 32..47 of sequence 1 have no block
    st = status()
    out = decode(tuple(bad), lengths, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == kv.DEV_BAD_BLOCK
    check_attention(out, tuple(bad), lengths)
    st = status()  # a length above the tables (clamped), a negative one (empty)
    out = decode(case, [40, 9999, -3], status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == kv.DEV_BAD_BLOCK
    assert bool((out[2] == 0).all())
    case = build(8, 2, 64, 16, [40, 40], [2, 2], 24)
    for qmax in (4, 30):  # both kernels
        st = status()
        out = torch.full((4, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        bad = list(case)
        bad[1] = np.array([0, 2, 9], np.int32)
        multi(tuple(bad), [40, 40], qmax, out=out, status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == kv.DEV_BAD_BLOCK and bool((out[2:] == 7).all())
        check_attention(out[:2], (case[0][:2], np.array([0, 2]), *case[2:6], case[6][:1]), [40],
                        one_tile=qmax > 4)


@pytest.mark.parametrize("n_q, hd, length, qmax", [(4, 64, 100, 2), (8, 128, 900, 2), (8, 128, 2000, 40), (8, 128, 300, 200)])
def test_rows_behind_the_last_sequence_are_left(n_q, hd, length, qmax):
    """A padded batch: sequences of no new tokens, query rows that no sequence has, an empty sequence."""
    lengths, qlens = [length, 0, length], [qmax, 0, 0]
    case = list(build(n_q, 2, hd, 16, lengths, qlens, 27))
    q = case[0]
    padded = torch.cat([q, torch.full((5, n_q, hd), math.nan).bfloat16()])
    out = torch.full(padded.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    st = status()
    multi((padded, *case[1:]), lengths, qmax, out=out, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and bool((out[qmax:] == 7).all())
    check_attention(out[:qmax], case, lengths, one_tile=True)


def test_streams_and_graphs():
    """A call on another stream, two calls at once with workspaces of their own, and a captured write and
    read replayed on new inputs."""
    lengths = [2000, 130]
    case = build(32, 8, 128, 16, lengths, [1, 1], 25)
    q, _, kc, vc, kg, vg, bt = case
    t = [dev(a) for a in (kc, vc, kg, vg, bt)]
    lens, ks, vs, qc = dev(np.array(lengths, np.int32)), scalar(KS), scalar(VS), q.cuda()
    want = kv.paged_decode_attention_fp4(qc, *t, lens, ks, vs)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(10):
        outs += [kv.paged_decode_attention_fp4(qc, *t, lens, ks, vs, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)

    row = torch.from_numpy(np.random.default_rng(1).standard_normal((2, 2, 8, 128))).bfloat16().cuda()
    new, slot = row[0].clone(), dev(np.array([int(bt[i, (n - 1) // 16]) * 16 + (n - 1) % 16 for i, n in enumerate(lengths)]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.reshape_and_cache_fp4(new, new, t[0], t[1], t[2], t[3], slot, ks, vs)
        got = kv.paged_decode_attention_fp4(qc, *t, lens, ks, vs)
    for i in (0, 1, 0):
        new.copy_(row[i])
        g.replay()
        torch.cuda.synchronize()
        first = got.clone()
        host = [a.cpu().numpy() for a in t]
        check_attention(first, (q, np.arange(3), host[0], host[1], host[2], host[3], bt), lengths)
        assert torch.equal(kv.paged_decode_attention_fp4(qc, *t, lens, ks, vs), first)


def test_a_captured_chunk_with_split_keys():
    """A short chunk on a long context captured with its workspace from the graph's memory, replayed between
    eager calls on another stream; the current device's streams are the callers' own."""
    lengths = [3000]
    case = build(32, 8, 128, 16, lengths, [16], 28)
    q, qsl, kc, vc, kg, vg, bt = case
    t = [dev(a) for a in (kc, vc, kg, vg, bt)]
    lens, start, ks, vs, qc = dev(np.array(lengths, np.int32)), dev(qsl), scalar(KS), scalar(VS), q.cuda()
    call = lambda **more: kv.paged_attention_multi_fp4(qc, start, 16, *t, lens, ks, vs, **more)
    want = call()
    check_attention(want, case, lengths, one_tile=True)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        got = call()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(5):
        got.zero_()
        g.replay()
        outs += [call(stream=side), got.clone()]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_large_offsets():
    """Blocks past 2^31 bytes of codes (and 2^28 of scales) from the start of the pool."""
    bs, n_kv, hd = 256, 8, 128
    nb = (1 << 32) // (bs * n_kv * hd // 2) + 3
    kc, vc = (torch.empty(nb, bs, n_kv, hd // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    kg, vg = (torch.empty(nb, n_kv, bs, hd // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    r = np.random.default_rng(3)
    bt = np.array([[nb - 1, 0, nb // 2 + 1]], np.int32)
    length = 600
    slots = bt[0, np.arange(length) // bs].astype(np.int64) * bs + np.arange(length) % bs
    x = torch.from_numpy(r.standard_normal((2, length, n_kv, hd))).bfloat16().cuda()
    kv.reshape_and_cache_fp4(x[0], x[1], kc, vc, kg, vg, dev(slots), scalar(KS), scalar(VS))
    back = kv.dequant_fp4(kc, kg, dev(slots), torch.float32, scalar(KS))
    small_c, small_g = empty_cache(3, bs, n_kv, hd)
    vs_c, vs_g = empty_cache(3, bs, n_kv, hd)
    fp4.write(x[0].float().cpu().numpy(), small_c, small_g, np.arange(length), KS)
    fp4.write(x[1].float().cpu().numpy(), vs_c, vs_g, np.arange(length), VS)
    assert np.array_equal(back.cpu().numpy(), fp4.dequant(small_c, small_g, np.arange(length), KS))
    for n in (1, 40):
        q = torch.from_numpy(r.standard_normal((n, 16, hd))).bfloat16()
        out = kv.paged_attention_multi_fp4(q.cuda(), dev(np.array([0, n], np.int32)), n, kc, vc, kg, vg, dev(bt),
                                           dev(np.array([length], np.int32)), scalar(KS), scalar(VS))
        case = (q, np.array([0, n]), small_c, vs_c, small_g, vs_g, np.arange(3, dtype=np.int32)[None])
        check_attention(out, case, [length], one_tile=n > 8)
    src = np.array([nb - 1, nb // 2 + 1], np.int32)
    kv.copy_blocks([kc, kg], dev(src), dev(np.array([1, nb - 2], np.int32)))
    assert torch.equal(kc[1], kc[nb - 1]) and torch.equal(kg[nb - 2], kg[nb // 2 + 1])
