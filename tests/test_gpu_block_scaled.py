"""The FP8 cache with block scales on the GPU against the oracle: codes and scales bit for bit, attention within
derived bounds.

Bounds of attention, for a row and dim, with A = sum p|v| / sum p and S the largest sm |q| . |k| of the row:
  * the bf16 result is off by at most half a step, 2^-8 of the value;
  * p * vs enters the product as fp16 (in long chunks with vs the largest of the token's 64 and V's codes times the rest,
    multiples of 2^-24 where 448 max(vs) is 2^15.8), 2^7 at least where it is highest: 2^-11 of each, so 2^-11 A, and
    2^-25 absolute below 2^-14, so 2^-32 of the highest p * vs: L * 2^-32 * max(vs) * 448 covers both, the row's sum
    being at least its highest p;
  * scores are float sums of hd exact products, (hd + 4) * 2^-24 S at most, and in the log2 domain they are
    multiplied, added to log2 vs and to the reference: three roundings of a number of at most 1.45 S + 80 (|log2 vs| <=
    60 here), with exp2's and log2's own 2^-22: a weight moves by at most d = (hd + 8) * 2^-24 (1.45 S + 80) +
    2^-21 of itself, in numerator and sum: 2 d A;
  * sums of L float terms, 16 at a time on the tensor cores, which may truncate (2^-23): (L / 16 + 16) * 2^-23 A, in
    numerator and sum: twice that.
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


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def stride_of(n_kv):
    return -(-n_kv // 4) * 4


def empty_cache(nb, bs, n_kv, hd, scale=0.0):
    """NaN codes, and scales of 0 (nothing written), so that anything that reads them shows."""
    return np.full((nb, bs, n_kv, hd), 0xFF, np.uint8), np.full((nb, stride_of(n_kv)), scale, np.float32)


# ---------------------------------------------------------------- writer

class Pool:
    """K and V sides on the GPU and as the oracle has them; every write is checked whole."""

    def __init__(self, nb, bs, n_kv, hd, fill=None):
        self.host = [empty_cache(nb, bs, n_kv, hd) for _ in "kv"]
        if fill is not None:
            for (c, s), seed in zip(self.host, (1, 2)):
                r = np.random.default_rng(seed)
                c[:] = r.integers(0, 256, c.shape)
                s[:] = fill(r, s.shape)
        self.gpu = [(dev(c), dev(s)) for c, s in self.host]

    def write(self, k, v, slots, want_status=0, **more):
        flags = 0
        for x, (c, s) in zip((k, v), self.host):
            bad_slot, bad_scale = bso.write(x.float().cpu().numpy(), c, s, slots)
            flags |= (kv.DEV_BAD_SLOT if bad_slot else 0) | (kv.DEV_BAD_SCALE if bad_scale else 0)
        st = status()
        (kc, ks), (vc, vs) = self.gpu
        kv.reshape_and_cache_block_scaled(k, v, kc, vc, ks, vs, dev(slots), status=st, **more)
        torch.cuda.synchronize()
        assert int(st.item()) == flags == want_status
        self.check()

    def check(self):
        for (c, s), (gc, gs) in zip(self.host, self.gpu):
            assert np.array_equal(gs.cpu().numpy(), s, equal_nan=True)
            assert np.array_equal(gc.cpu().numpy(), c)


def rows(r, n, n_kv, hd, dtype=torch.bfloat16, spread=2.0):
    """Rows whose magnitudes differ by token and head."""
    x = r.standard_normal((2, n, n_kv, hd)) * np.exp2(np.round(spread * r.standard_normal((2, n, n_kv, 1))))
    return torch.from_numpy(x).to(dtype).cuda()


SHAPES = [(1, 1, 64, 16), (7, 2, 64, 16), (33, 5, 64, 32), (100, 8, 128, 16), (65, 3, 256, 64), (17, 12, 128, 128),
          (40, 1, 256, 256), (512, 2, 64, 64), (513, 2, 64, 64), (700, 3, 128, 256), (1300, 1, 256, 32), (900, 33, 64, 16),
          (2000, 1, 64, 256), (600, 4, 128, 32)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n, n_kv, hd, bs", SHAPES)
def test_write_of_scattered_rows(dtype, n, n_kv, hd, bs):
    """Rows in any order over a pool that holds codes (NaN among them) under scales that are kept or raised."""
    r = np.random.default_rng(n)
    nb = n // bs + 3
    pool = Pool(nb, bs, n_kv, hd, fill=lambda r, shape: np.exp2(r.integers(-12, -3, shape)))
    slots = r.permutation(nb * bs)[:n].astype(np.int64)
    slots[r.random(n) < 0.1] = -1
    x = rows(r, n, n_kv, hd, dtype)
    pool.write(x[0], x[1], slots)
    x = rows(r, n, n_kv, hd, dtype, spread=4.0)
    pool.write(x[1], x[0], np.roll(slots, 3))


@pytest.mark.parametrize("n_kv, hd, bs, calls", [(2, 64, 16, [5, 1, 1, 30, 200, 1]), (8, 128, 32, [1] * 20 + [64]),
                                                 (5, 64, 64, [585, 1, 600]), (3, 256, 128, [100, 30, 1, 700]),
                                                 (1, 128, 256, [1, 255, 2, 513])])
def test_sequences_that_grow(n_kv, hd, bs, calls):
    """Three sequences appended to, call by call, their rows side by side or in turn."""
    r = np.random.default_rng(bs)
    total = sum(calls)
    per = -(-total // bs)
    ids = r.permutation(3 * per + 2)
    pool = Pool(3 * per + 2, bs, n_kv, hd)
    at = 0
    for i, n in enumerate(calls):
        pos = np.arange(at, at + n)
        slots = np.stack([ids[q * per + pos // bs] * bs + pos % bs for q in range(3)]).astype(np.int64)
        slots = (slots.T if i % 2 else slots).reshape(-1).copy()
        x = rows(r, 3 * n, n_kv, hd)
        pool.write(x[0], x[1], slots)
        at += n
    (kc, ks), _ = pool.gpu
    assert bool((ks[:, :n_kv].amax(1) > 0).sum() == 3 * per)


def test_write_strides_and_alignment():
    r = np.random.default_rng(6)
    for dtype, pads in ((torch.bfloat16, (0, 8, 16)), (torch.float32, (0, 4, 8))):
        for pad in pads:  # a slice of a fused row: 16-byte aligned starts and strides
            wide = torch.from_numpy(r.standard_normal((20, 3 * 256 + pad))).to(dtype).cuda()
            k = wide[:, pad:pad + 256].unflatten(1, (4, 64))
            v = wide[:, 256 + pad:512 + pad].unflatten(1, (4, 64))
            Pool(2, 16, 4, 64).write(k, v, r.permutation(32)[:20].astype(np.int64))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_write_corner_values(dtype):
    x = torch.zeros(16, 2, 64)
    big = torch.finfo(torch.float32).max
    x[0, 0] = -0.0
    x[1, 0, :20] = torch.tensor([math.nan, -math.nan] * 10)
    x[2, 0, :6] = torch.tensor([math.inf, -math.inf, 1.0, -2.0, 0.0, -0.0])
    x[3, 0, :4] = torch.tensor([1e-12, -1e-12, 1e-44, -1e-44])
    x[5, 0] = torch.linspace(-3000, 3000, 64)
    x[4, 1, :3] = torch.tensor([big, -big, 1.0])
    x = x.to(dtype).cuda()
    for slots in (np.arange(16), np.arange(16)[::-1].copy(), np.arange(16) * 16, np.arange(16) * 17 + 1):
        Pool(18, 16, 2, 64, fill=lambda r, shape: np.exp2(r.integers(-50, 60, shape))).write(x, x.flip(0), slots.astype(np.int64))
    # rows of one kind alone: zeros, NaN, infinities, denormals
    for v in (0.0, math.nan, math.inf, 1e-44, 2.0 ** -60 * 448):
        y = torch.full((3, 1, 64), v).to(dtype).cuda()
        Pool(1, 16, 1, 64).write(y, -y, np.array([0, 5, 6]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n, hd, bs, every", [(1300, 128, 256, 1), (1300, 64, 128, 3), (600, 256, 64, 1), (700, 128, 256, 14), (403, 128, 64, 1),
                                              (23, 256, 256, 1)])
def test_corner_values_among_many_rows(dtype, n, hd, bs, every):
    """Blocks with more rows than a warp holds, whole and with gaps, some of them with infinities, NaN or nothing but zeros; a
    block's last rows in a second call, under scales that they keep or raise."""
    r = np.random.default_rng(n + bs)
    x = rows(r, n, 2, hd, dtype, spread=5.0)
    x[:, :n // 3][torch.from_numpy(r.random((2, n // 3, 2, hd)) < 0.002).cuda()] = math.nan
    x[:, n // 4:n // 2][torch.from_numpy(r.random((2, n // 2 - n // 4, 2, hd)) < 0.002).cuda()] = -math.inf
    x[:, -n // 4:] = 0.0
    at = np.arange(n, dtype=np.int64) * every
    pool = Pool(-(-n * every // bs) + 1, bs, 2, hd)
    pool.write(x[0], x[1], r.permutation(n).astype(np.int64) * every)
    late = at % bs != 0
    pool.write(x[1][torch.from_numpy(late).cuda()].contiguous() * 2, x[0][torch.from_numpy(late).cuda()].contiguous() / 4, at[late])


def test_every_scale_boundary():
    """Block maxima around 448 times every power of two, under either type, and one binade of bf16 values whole."""
    tops = np.array([448.0 * 2.0 ** e * f for e in range(-75, 118, 3) for f in (1 - 2.0 ** -24, 1, 1 + 2.0 ** -23, 1.5)])
    n = len(tops)
    x = torch.from_numpy(tops).float()[:, None, None] * torch.linspace(-1, 1, 64)[None, None, :]
    pool = Pool(n, 16, 1, 64)
    pool.write(x.cuda(), (-x).cuda(), np.arange(n) * 16)
    pool = Pool(n, 16, 1, 64)
    pool.write(x.bfloat16().cuda(), x.flip(0).bfloat16().cuda(), np.arange(n) * 16)
    every = torch.arange(0, 0x7F80, dtype=torch.int16).view(torch.bfloat16)
    every = every[every.float().abs() < 2.0 ** 9].reshape(-1, 1, 64)
    m = len(every)
    pool = Pool(m // 16 + 1, 16, 1, 64, fill=lambda r, shape: np.exp2(r.integers(-6, 3, shape)))
    pool.write(every.cuda(), -every.cuda(), np.arange(m) + 1)


def test_scales_that_are_not_valid():
    for bad in (math.nan, math.inf, -1.0, 2.0 ** -61, 2.0 ** 121, 0.75, 1.0 + 2.0 ** -23):
        pool = Pool(2, 16, 2, 64, fill=lambda r, shape: np.where(np.arange(shape[1]) == 1, bad, 1.0) * np.ones(shape))
        x = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
        pool.write(x, x, np.array([3, 4, 20]), want_status=kv.DEV_BAD_SCALE)  # head 1 stays as it is
        pool.write(x, x, np.array([0, 16, 17]))                               # anew: what was there does not count


@pytest.mark.parametrize("n", [4, 600])
def test_bad_slots_and_padding(n):
    x = torch.ones(n, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = np.full(n, -1, np.int64)
    slots[:4] = [3, 32, -2, 7]
    Pool(2, 16, 2, 64).write(x, x, slots, want_status=kv.DEV_BAD_SLOT)
    Pool(2, 16, 2, 64).write(x, x, np.full(n, -1, np.int64))
    Pool(2, 16, 2, 64).write(x[:0], x[:0], slots[:0])


@pytest.mark.parametrize("n", [40, 1200])
def test_a_slot_named_twice_gets_one_of_its_rows_whole(n):
    r = np.random.default_rng(n)
    nb = n // 16 + 1
    x = rows(r, n, 4, 64, spread=0.0)
    slots = (np.arange(n) // 2 * 2).astype(np.int64)  # rows 2i and 2i + 1 at slot 2i
    (kc, ks), (vc, vs) = [(dev(c), dev(s)) for c, s in (empty_cache(nb, 16, 4, 64) for _ in "kv")]
    kv.reshape_and_cache_block_scaled(x[0], x[1], kc, vc, ks, vs, dev(slots))
    ids = dev(slots[::2].copy())
    for c, s, src in ((kc, ks, x[0]), (vc, vs, x[1])):
        got = kv.dequant_block_scaled(c, s, ids, torch.float32)
        step = 2.0 ** -4 * src.float().abs() + s[(ids // 16)][:, :4, None].repeat_interleave(2, 0)[:n] * 2.0 ** -10
        even = ((got - src[0::2].float()).abs() <= step[0::2]).flatten(1).all(1)
        odd = ((got - src[1::2].float()).abs() <= step[1::2]).flatten(1).all(1)
        assert bool((even | odd).all())
        pick = even if c is kc else pick
        assert bool((pick == even).all())  # K and V of the same row


@pytest.mark.parametrize("n", [64, 2048])
def test_write_captured_and_on_another_stream(n):
    r = np.random.default_rng(n)
    nb = n // 32 + 2
    slots = r.permutation(nb * 32)[:n].astype(np.int64)
    x = rows(r, n, 2, 128)
    pool = Pool(nb, 32, 2, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    (kc, ks), (vc, vs) = pool.gpu
    d_slots, k, v = dev(slots), x[0].clone(), x[1].clone()
    kv.reshape_and_cache_block_scaled(k, v, kc, vc, ks, vs, d_slots, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for xx, (c, s) in zip(x, pool.host):
        bso.write(xx.float().cpu().numpy(), c, s, slots)
    pool.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.reshape_and_cache_block_scaled(k, v, kc, vc, ks, vs, d_slots)
    for seed in (1, 2):
        y = rows(np.random.default_rng(seed), n, 2, 128, spread=3.0)
        new = np.random.default_rng(seed).permutation(nb * 32)[:n].astype(np.int64)
        k.copy_(y[0])
        v.copy_(y[1])
        d_slots.copy_(dev(new))
        g.replay()
        for yy, (c, s) in zip(y, pool.host):
            bso.write(yy.float().cpu().numpy(), c, s, new)
        torch.cuda.synchronize()
        pool.check()


def test_workspace_of_a_caller_may_hold_anything():
    n, nb = 700, 30
    r = np.random.default_rng(3)
    need = kv.reshape_and_cache_block_scaled_workspace_size(n, nb, 32)
    assert need >= nb * 32 * 4
    for fill in (0, 0xFF, 1):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        pool = Pool(nb, 32, 2, 64)
        for _ in range(2):
            x = rows(r, n, 2, 64)
            pool.write(x[0], x[1], r.permutation(nb * 32)[:n].astype(np.int64), workspace=ws)


# ---------------------------------------------------------------- rows read back

@pytest.mark.parametrize("dst", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n, n_kv, hd, bs", [(1, 1, 64, 16), (50, 5, 64, 16), (200, 8, 128, 32), (31, 9, 256, 16), (3001, 3, 128, 256)])
def test_dequant_matches_the_oracle(dst, n, n_kv, hd, bs):
    r = np.random.default_rng(n)
    nb = 6
    codes = r.integers(0, 256, (nb, bs, n_kv, hd)).astype(np.uint8)
    scales = np.exp2(r.integers(-60, 121, (nb, stride_of(n_kv)))).astype(np.float32)
    slots = r.integers(-1, nb * bs, n)  # some twice
    for bad in (0.0, math.nan, -1.0, 2.0 ** 121, 0.3):
        scales[2, 0] = bad
        slots[0] = nb * bs
        st = status()
        out = kv.dequant_block_scaled(dev(codes), dev(scales), dev(slots), dst, status=st)
        torch.cuda.synchronize()
        hit = ((slots[1:] >= 0) & (slots[1:] // bs == 2)).any()
        assert int(st.item()) == kv.DEV_BAD_SLOT | (kv.DEV_BAD_SCALE if hit else 0)
        want = torch.from_numpy(bso.dequant(codes, scales, slots)).to(dst)
        assert torch.equal(torch.isnan(out.cpu()), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(out.cpu()), torch.nan_to_num(want))


# ---------------------------------------------------------------- attention

def build(n_q, n_kv, hd, bs, lengths, qlens, seed, spare=3, scale=None):
    """Random codes (no NaN) in the tokens that sequences hold, NaN codes elsewhere; block scales over eight octaves;
    scales of blocks that no sequence holds 0; tables with -1 past each sequence."""
    r = np.random.default_rng(seed)
    need = [-(-n // bs) for n in lengths]
    nb = sum(need) + spare
    perm = r.permutation(nb).astype(np.int32)
    bt = np.full((len(lengths), max(1, max(need))), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        bt[i, :n] = perm[at:at + n]
        at += n
    used = perm[:at]
    slots = np.concatenate([bt[i, np.arange(n) // bs].astype(np.int64) * bs + np.arange(n) % bs
                            for i, n in enumerate(lengths)] + [np.zeros(0, np.int64)]).astype(np.int64)
    sides = []
    for lo in (-9, -6):
        c, s = empty_cache(nb, bs, n_kv, hd)
        x = r.standard_normal((len(slots), n_kv, hd)).astype(np.float32) * 60
        c[slots // bs, slots % bs] = bso.encode(x)
        s[used] = np.exp2(r.integers(lo, lo + 8, (len(used), s.shape[1]))) if scale is None else scale(r, (len(used), s.shape[1]))
        sides += [(c, s)]
    (kc, ks), (vc, vs) = sides
    qsl = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
    q = torch.from_numpy(r.standard_normal((int(qsl[-1]), n_q, hd)) / 4).bfloat16()
    return dict(q=q, qsl=qsl, kc=kc, vc=vc, ks=ks, vs=vs, bt=bt, lengths=list(lengths))


def check_attention(got, case, causal=True, sm=0.0, more=0.0):
    """more: by how much scores may be off besides."""
    c = case
    hd, longest = c["q"].shape[2], max(c["lengths"] + [1])
    ref, weight, reach = bso.attention(c["q"].double().numpy(), c["qsl"], c["kc"], c["vc"], c["ks"], c["vs"], c["bt"],
                                       c["lengths"], causal, sm)
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(ref))
    fine = ~np.isnan(ref)
    vs = c["vs"][bso.scale_ok(c["vs"])]
    d = (hd + 8) * 2.0 ** -24 * (1.45 * reach + 80) + 2.0 ** -21 + more
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * d[..., None] + 2 * (longest / 16 + 16) * 2.0 ** -23) * weight \
        + longest * 2.0 ** -32 * vs.max(initial=0.0) * 448 + 1e-37
    over = (np.abs(g - ref) - bound)[fine]
    assert over.size == 0 or over.max() <= 0, (over.max(), np.abs(g - ref)[fine].max())


def caches(c):
    return [dev(c[name]) for name in ("kc", "vc", "ks", "vs", "bt")] + [dev(np.array(c["lengths"], np.int32))]


def decode(c, **more):
    return kv.paged_decode_attention_block_scaled(c["q"].cuda(), *caches(c), **more)


def multi(c, qmax, **more):
    return kv.paged_attention_multi_block_scaled(c["q"].cuda(), dev(c["qsl"]), qmax, *caches(c), **more)


def run(call, *args, want_status=0, **more):
    st = status()
    out = call(*args, status=st, **more)
    torch.cuda.synchronize()
    assert int(st.item()) == want_status
    return out


DECODE = [
    # n_q, n_kv, head_dim, block, lengths
    (4, 2, 64, 16, [17, 33, 64, 100]),
    (2, 2, 64, 16, [1, 7, 8, 9, 0, 24]),
    (32, 8, 128, 16, [1000, 1, 16, 15, 0, 257]),
    (8, 1, 128, 32, [31, 32, 33, 500]),
    (64, 8, 128, 64, [12, 200, 3]),
    (48, 4, 128, 64, [63, 65, 300]),          # 12 heads a group: two score tiles
    (16, 1, 64, 256, [255, 257, 600]),        # 16 heads a group
    (12, 12, 64, 16, [90, 5]),                # two head groups of six
    (10, 5, 128, 128, [300, 77]),             # head groups of one
    (32, 4, 256, 16, [1, 250, 77]),           # 8 heads a group at head_dim 256
    (7, 7, 256, 32, [40, 13]),
    (20, 1, 128, 16, [70, 0, 129]),           # 20 heads a group: the tensor-core kernel
    (36, 4, 256, 32, [65, 10]),               # 9 heads at head_dim 256: the tensor-core kernel
    (128, 1, 64, 16, [200]),
]


@pytest.mark.parametrize("n_q, n_kv, hd, bs, lengths", DECODE)
def test_decode_matches_the_oracle(n_q, n_kv, hd, bs, lengths):
    c = build(n_q, n_kv, hd, bs, lengths, [1] * len(lengths), n_q + hd + bs)
    check_attention(run(decode, c), c)


@pytest.mark.parametrize("hd, n_q, n_kv", [(64, 8, 2), (128, 32, 8), (128, 32, 2), (256, 8, 2), (128, 3, 3)])
def test_decode_long_sequences_split_over_the_grid(hd, n_q, n_kv):
    c = build(n_q, n_kv, hd, 16, [20011, 1, 9000], [1, 1, 1], 11)
    check_attention(run(decode, c), c)


MULTI = [
    # n_q, n_kv, head_dim, block, lengths, query counts
    (4, 4, 64, 16, [4, 30, 257], [4, 4, 4]),
    (32, 8, 128, 16, [1000, 17, 4, 5], [4, 1, 3, 4]),
    (8, 8, 128, 32, [100, 16, 40], [16, 16, 9]),
    (4, 2, 256, 64, [129, 300], [4, 2]),
    (8, 2, 64, 32, [50, 80, 0], [0, 3, 0]),
    (32, 8, 128, 16, [300, 64, 21], [20, 64, 21]),      # one row tile, 80 rows and more
    (16, 2, 128, 16, [500, 129, 40], [130, 129, 1]),    # two row tiles
    (8, 2, 64, 16, [300, 77], [200, 77]),
    (4, 1, 64, 64, [400], [300]),
    (6, 2, 256, 16, [150, 33], [60, 33]),
    (24, 8, 64, 256, [513, 260], [100, 260]),
    (8, 1, 128, 128, [1, 700], [1, 70]),
]


@pytest.mark.parametrize("n_q, n_kv, hd, bs, lengths, qlens", MULTI)
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "all"])
def test_multi_matches_the_oracle(causal, n_q, n_kv, hd, bs, lengths, qlens):
    c = build(n_q, n_kv, hd, bs, lengths, qlens, n_q + hd + bs)
    check_attention(run(multi, c, max(qlens), causal=causal), c, causal)


@pytest.mark.parametrize("n_q, n_kv, hd, qlens", [(4, 4, 64, [9, 3]), (8, 2, 128, [40, 17]), (4, 1, 128, [150, 70]),
                                                  (6, 2, 256, [30, 8]), (16, 16, 64, [225, 150])])
def test_more_queries_than_tokens(n_q, n_kv, hd, qlens):
    """Cross attention to shorter states; causal, the queries before the first token see nothing."""
    c = build(n_q, n_kv, hd, 16, [5, 21], qlens, 3)
    check_attention(run(multi, c, max(qlens), causal=False), c, False)
    check_attention(run(multi, c, max(qlens), want_status=kv.DEV_BAD_BLOCK if qlens[0] > 5 or qlens[1] > 21 else 0), c)


@pytest.mark.parametrize("n_q, n_kv, hd, lengths, qlens", [
    (4, 1, 128, [7000, 300], [8, 8]), (16, 4, 64, [3000], [33]), (8, 2, 256, [5000, 40], [12, 12]), (32, 8, 128, [2500], [48]),
    (16, 16, 64, [1500], [150])])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "all"])
def test_few_row_tiles_split_their_keys(causal, n_q, n_kv, hd, lengths, qlens):
    c = build(n_q, n_kv, hd, 16, lengths, qlens, 5)
    check_attention(run(multi, c, max(qlens), causal=causal), c, causal)


@pytest.mark.parametrize("n", [255, 256, 257, 700])
@pytest.mark.parametrize("longest", [250, 300])
def test_many_short_sequences(n, longest):
    """Both plans of the split, and sequences taken whole; some empty, some without queries."""
    r = np.random.default_rng(n + longest)
    lengths = r.integers(0, longest + 1, n)
    lengths[5] = longest
    c = build(4, 2, 64, 16, lengths.tolist(), [1] * n, 26)
    check_attention(run(decode, c), c)
    qlens = np.minimum(r.integers(0, 4, n), lengths).tolist()
    c = build(4, 2, 64, 16, lengths.tolist(), qlens, 27)
    check_attention(run(multi, c, 3), c)
    qlens = r.integers(0, 5, n).tolist()  # more than a sequence has tokens, some
    c = build(4, 2, 64, 16, lengths.tolist(), qlens, 28)
    check_attention(run(multi, c, 4, causal=False), c, False)


ROUTES = [(8, 2, 128, 1), (8, 2, 64, 3), (16, 2, 128, 2), (4, 2, 256, 2), (8, 2, 128, 30), (8, 2, 128, 70), (8, 2, 64, 90), (4, 2, 256, 70)]


@pytest.mark.parametrize("n_q, n_kv, hd, qlen", ROUTES)
def test_scales_of_any_size(n_q, n_kv, hd, qlen):
    """V scales from 2^-60 to 2^60 side by side, K scales such that scores stay small; and all at one end."""
    lengths, qlens = [300, 77], [qlen, min(qlen, 77)]

    def mixed(r, shape):
        return np.exp2(r.integers(-60, 61, shape).astype(np.float64))

    for scale in (mixed, lambda r, shape: np.full(shape, 2.0 ** -60), lambda r, shape: np.full(shape, 2.0 ** 60)):
        c = build(n_q, n_kv, hd, 16, lengths, qlens, 7, scale=scale)
        live = c["ks"] > 0
        c["ks"][live] = np.exp2(np.random.default_rng(8).integers(-27, -5, int(live.sum())))
        check_attention(run(multi, c, qlen), c)


@pytest.mark.parametrize("n_q, n_kv, hd, qlen", ROUTES)
def test_scales_of_an_earlier_call_do_not_linger(n_q, n_kv, hd, qlen):
    """Calls with scales far apart one after the other, the last tiles cut off inside: nothing of a tile's shared memory
    that the tile did not fill may count."""
    for at in (2.0 ** 50, 2.0 ** -55, 1.0, 2.0 ** -60, 2.0 ** 60):
        c = build(n_q, n_kv, hd, 16, [300, 77, 129], [qlen, min(qlen, 77), min(qlen, 129)], 7, scale=lambda r, shape: np.full(shape, at))
        c["ks"][c["ks"] > 0] = 2.0 ** -27 if at < 1 else 2.0 ** -6
        check_attention(run(multi, c, qlen), c)


@pytest.mark.parametrize("n_q, n_kv, hd, qlen", ROUTES)
def test_bad_blocks_and_scales_hold_no_tokens(n_q, n_kv, hd, qlen):
    lengths, qlens = [300, 177, 140], [qlen, qlen, min(qlen, 140)]
    base = build(n_q, n_kv, hd, 16, lengths, qlens, 9)
    c = dict(base, bt=base["bt"].copy())
    c["bt"][0, 3], c["bt"][1, 0], c["bt"][1, 10] = -1, len(c["kc"]), 1 << 30
    c["bt"][2, :] = -5  # a sequence without any
    check_attention(run(multi, c, qlen, want_status=kv.DEV_BAD_BLOCK), c)
    for bad in (0.0, math.nan, -1.0, math.inf, 2.0 ** -61, 2.0 ** 121, 3.0):
        c = dict(base, ks=base["ks"].copy(), vs=base["vs"].copy())
        c["ks"][base["bt"][0, 2], 0] = bad
        c["vs"][base["bt"][0, 18], 1] = bad  # its last block
        c["vs"][base["bt"][2, :9], 0] = bad  # every block of a sequence, one head
        check_attention(run(multi, c, qlen, want_status=kv.DEV_BAD_SCALE), c)


@pytest.mark.parametrize("n_q, n_kv, hd, qlen", ROUTES)
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "all"])
def test_nan_reaches_what_sees_it(causal, n_q, n_kv, hd, qlen):
    lengths, qlens = [300, 140, 200], [qlen, min(qlen, 140), qlen]
    for side, at in (("kc", 299), ("vc", 299), ("vc", 298), ("vc", 200), ("vc", 130), ("vc", 3), ("kc", 40)):
        c = build(n_q, n_kv, hd, 16, lengths, qlens, 13)
        c[side][c["bt"][0, at // 16], at % 16, 1, 5] = 0x7F
        c[side][c["bt"][0, at // 16], at % 16, 0, hd - 1] = 0xFF
        t = max(0, 140 - qlen // 2 - 1)
        c[side][c["bt"][1, t // 16], t % 16, 0, 17] = 0xFF
        check_attention(run(multi, c, qlen, causal=causal), c, causal)


def test_softmax_scale_and_large_scores():
    c = build(8, 2, 128, 16, [500, 20], [1, 1], 12)
    for sm in (0.3, 0.01, 1e-30, 1e-38):
        check_attention(run(decode, c, sm_scale=sm), c, sm=sm)


def test_lengths_out_of_range_are_flagged():
    c = build(8, 2, 64, 16, [50, 20], [1, 1], 14)
    c["lengths"] = [-3, 10 ** 6]
    out = run(decode, c, want_status=kv.DEV_BAD_BLOCK)
    assert bool((out[0] == 0).all())
    c["lengths"] = [0, c["bt"].shape[1] * 16]
    c["bt"][1, 2:] = -1
    want = bso.attention(c["q"].double().numpy(), c["qsl"], c["kc"], c["vc"], c["ks"], c["vs"], c["bt"], c["lengths"])[0]
    assert np.array_equal(np.isnan(out.double().cpu().numpy()), np.isnan(want))


def test_query_rows_out_of_range():
    c = build(8, 2, 64, 16, [50, 20, 30], [2, 2, 2], 15)
    c["qsl"] = np.array([0, 2, 9, 6], np.int32)  # sequence 1 has seven, sequence 2 a negative count
    out = torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    for qmax in (2, 40):
        run(multi, c, qmax, out=out, want_status=kv.DEV_BAD_BLOCK)
        assert bool((out[2:] == 7).all())


@pytest.mark.parametrize("qlen", [1, 40])
def test_rows_behind_the_last_sequence_stay(qlen):
    c = build(8, 2, 128, 16, [100, 60], [qlen, qlen], 16)
    pad = torch.full((5, 8, 128), 3.0).bfloat16()
    c["q"] = torch.cat([c["q"], pad])
    out = torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    run(multi, c, qlen, out=out)
    assert bool((out[2 * qlen:] == 7).all())
    c["q"] = c["q"][:2 * qlen]
    check_attention(out[:2 * qlen], c)


@pytest.mark.parametrize("qlen", [1, 3, 40, 200])
def test_attention_repeats_itself_and_replays(qlen):
    c = build(8, 2, 128, 16, [3000, 260], [qlen, qlen], 17)
    q, rest, qsl = c["q"].cuda(), caches(c), dev(c["qsl"])
    first = kv.paged_attention_multi_block_scaled(q, qsl, qlen, *rest)
    out = torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.paged_attention_multi_block_scaled(q, qsl, qlen, *rest, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = kv.paged_attention_multi_block_scaled(q, qsl, qlen, *rest, stream=side)
    side.synchronize()
    assert torch.equal(again, first)
    q.mul_(-1)  # other inputs through the same graph
    g.replay()
    c["q"] = -c["q"]
    check_attention(out, c)


@pytest.mark.parametrize("n_q, n_kv, hd, qlen", ROUTES)
def test_query_rows_of_any_magnitude(n_q, n_kv, hd, qlen):
    """Rows of q down to denormals; rows with one element 2^4 to 2^12 times the others, over keys that are 0 there, so that the
    small elements make the scores; rows with a NaN."""
    lengths, qlens = [300, 77], [qlen, min(qlen, 77)]
    c = build(n_q, n_kv, hd, 16, lengths, qlens, 31)
    r = np.random.default_rng(32)
    q = c["q"].double().numpy()
    q *= np.exp2(r.choice([0.0, -3, -20, -110, -130], q.shape[:2]))[..., None]
    odd = r.random(q.shape[:2]) < 0.3
    q[odd, 5] = np.abs(q[odd]).max(-1) * np.exp2(r.integers(4, 13, int(odd.sum())))
    q[0, 1, 7] = math.nan
    c["q"] = torch.from_numpy(q).bfloat16()
    c["kc"][..., 5] = 0
    # In long chunks an element of q is the sum of two E4M3 numbers, the row scaled to a largest of [2^7, 2^8).  The first
    # leaves 4 bits of a bf16's 8, the last of them 2^-7 of the element's own power of two: the second holds
    # them from 2^-9 on, so elements from 2^-2, 2^-9 of the largest at least, are exact, and others off by half of
    # 2^-9, 2^-17 of the largest at most.  Elsewhere q is fp16: off by 2^-25 below 2^-14 at most.  A score is off by the
    # sum of those times |k|.
    q = np.abs(np.nan_to_num(c["q"].double().numpy()))
    top = q.max(-1, keepdims=True)
    off = np.where(q >= top * 2.0 ** -9, 0.0, 2.0 ** -17 * top) + 2.0 ** -25
    k = np.abs(bso.decode(c["kc"])) * c["ks"][:, None, :n_kv, None]  # [block, token, head, dim]
    k = np.repeat(np.nan_to_num(k[c["bt"][c["bt"] >= 0]]).max((0, 1)), n_q // n_kv, 0)
    check_attention(run(multi, c, qlen), c, more=1.45 / math.sqrt(hd) * (off * k).sum(-1))


def test_a_pool_past_32_bits():
    """Blocks that lie past 4 GB of codes give what the same blocks give at the front of a small pool."""
    n_kv, hd, bs = 8, 128, 16
    c = build(16, n_kv, hd, bs, [300, 77], [60, 60], 33)
    nb = len(c["kc"])
    at = (1 << 32) // (bs * n_kv * hd) + 5  # the blocks' place in the big pool
    small = caches(c)
    big = []
    for t in small[:4]:
        p = torch.empty((at + nb,) + t.shape[1:], dtype=t.dtype, device="cuda")
        p[at:] = t
        big.append(p)
    bt = torch.where(small[4] >= 0, small[4] + at, small[4])
    q, qsl = c["q"].cuda(), dev(c["qsl"])
    for n in (1, 60):  # a few columns, long chunks
        st = status()
        want = kv.paged_attention_multi_block_scaled(q[:2 * n], qsl // 60 * n, n, *small, status=st)
        got = kv.paged_attention_multi_block_scaled(q[:2 * n], qsl // 60 * n, n, *big[:4], bt, small[5], status=st)
        assert torch.equal(got, want) and int(st.item()) == 0
    x = (torch.randn(2000, n_kv, hd, device="cuda") * 30).bfloat16()
    slots = torch.randperm(nb * bs, device="cuda")
    for n in (200, min(2000, nb * bs)):  # both ways of finding a block's rows
        if n > 512:
            x, slots = x[:n], slots[:n]
        kv.reshape_and_cache_block_scaled(x[:n], -x[:n], *small[:4], slots[:n])
        kv.reshape_and_cache_block_scaled(x[:n], -x[:n], *big, slots[:n] + at * bs)
        for s, b in zip(small[:4], big):
            assert torch.equal(b[at:], s)
    assert torch.equal(kv.dequant_block_scaled(big[0], big[2], slots + at * bs), kv.dequant_block_scaled(small[0], small[2], slots))


def test_calls_on_two_streams_at_once():
    """Two streams with workspaces of their own, neither waiting for the other, give what one does."""
    cases = [build(8, 2, 128, 16, [3000, 260], [qlen, qlen], 34 + qlen) for qlen in (3, 200)]
    sets = [(c["q"].cuda(), dev(c["qsl"]), c["qsl"][1].item(), caches(c)) for c in cases]
    rows = [(torch.randn(600, 2, 128, device="cuda") * 3).bfloat16() for _ in sets]
    slots = torch.arange(600, device="cuda")
    want = [kv.paged_attention_multi_block_scaled(q, qsl, n, *rest) for q, qsl, n, rest in sets]
    pools = [[torch.zeros(40, 16, 2, 128, dtype=torch.uint8, device="cuda") for _ in range(2)] +
             [kv.block_scales(40, 2) for _ in range(2)] for _ in range(4)]
    for i in range(2):
        kv.reshape_and_cache_block_scaled(rows[i], rows[i], *pools[i], slots)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[], []]
    for _ in range(5):
        for i, (q, qsl, n, rest) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                kv.reshape_and_cache_block_scaled(rows[i], rows[i], *pools[2 + i], slots)
                outs[i].append(kv.paged_attention_multi_block_scaled(q, qsl, n, *rest))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])
        assert all(torch.equal(a, b) for a, b in zip(pools[i], pools[2 + i]))


# ---------------------------------------------------------------- together

def test_a_serving_loop():
    """Prompts rotated, written, attended to; a fork whose last page is copied on write; steps; pages compacted; the context
    shifted by reading keys back, turning them and writing them again."""
    r = np.random.default_rng(20)
    n_q, n_kv, hd, bs, nb = 8, 2, 64, 16, 40
    freq, mag = kv.rotary_frequencies(hd, 10000.0, "parts", 4.0, 64)
    pool = Pool(nb, bs, n_kv, hd)
    (kc, ks), (vc, vs) = pool.gpu
    ids = r.permutation(nb)
    tables = [list(ids[:4]), list(ids[4:8])]
    lens = [40, 25]

    def slots_of(seq, pos):
        return np.array([tables[seq][p // bs] * bs + p % bs for p in pos], np.int64)

    def step(seqs, counts):
        """New tokens of `seqs`, `counts` of each: rotate, write, attend."""
        pos = [np.arange(lens[s], lens[s] + n) for s, n in zip(seqs, counts)]
        n = sum(counts)
        qkv = torch.from_numpy(r.standard_normal((n, (n_q + 2 * n_kv) * hd))).bfloat16().cuda()
        q = qkv[:, :n_q * hd].unflatten(1, (n_q, hd))
        k = qkv[:, n_q * hd:(n_q + n_kv) * hd].unflatten(1, (n_kv, hd))
        v = qkv[:, (n_q + n_kv) * hd:].unflatten(1, (n_kv, hd))
        want = [torch.from_numpy(bso.rotary(x.double().cpu().numpy(), np.concatenate(pos), freq.cpu().numpy(), magnitude=mag))
                for x in (q, k)]
        q2, _ = kv.rotary_embedding(q, k, dev(np.concatenate(pos)), freq, magnitude=mag, key_out=k)
        for got, w in zip((q2, k), want):
            assert ((got.double().cpu() - w).abs() <= 2.0 ** -8 * w.abs() + 1e-5).all()
        pool.write(k, v, np.concatenate([slots_of(s, p) for s, p in zip(seqs, pos)]))
        for s, m in zip(seqs, counts):
            lens[s] += m
        most = max(len(tables[s]) for s in seqs)
        bt = np.array([tables[s] + [-1] * (most - len(tables[s])) for s in seqs], np.int32)
        c = dict(q=q2.cpu(), qsl=np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), kc=pool.host[0][0], ks=pool.host[0][1],
                 vc=pool.host[1][0], vs=pool.host[1][1], bt=bt, lengths=[lens[s] for s in seqs])
        out = multi(c, max(counts))
        check_attention(out, c)

    lens = [0, 0]
    step([0, 1], [40, 25])
    for _ in range(3):
        step([0, 1], [1, 1])
    tables.append(tables[0][:2] + [int(ids[8]), int(ids[9])])  # a fork of sequence 0, its last page copied
    lens.append(lens[0])
    kv.copy_blocks([kc, vc, ks, vs], dev(np.array([tables[0][2]], np.int32)), dev(np.array([tables[2][2]], np.int32)))
    for c, s in pool.host:
        c[tables[2][2]], s[tables[2][2]] = c[tables[0][2]], s[tables[0][2]]
    pool.check()
    step([0, 1, 2], [2, 1, 4])
    # sequence 1 ends; its pages go
    bt = np.array([tables[0], tables[2]], np.int32)
    lens_now = np.array([lens[0], lens[2]], np.int32)
    new, used = kv.compact_blocks([kc, vc, ks, vs], dev(bt), dev(lens_now), bs)
    old, new = [(c.copy(), s.copy()) for c, s in pool.host], new.cpu().numpy()
    for (c, s), (oc, os_) in zip(pool.host, old):
        for a, b in zip(bt.ravel(), new.ravel()):
            if b >= 0:
                c[b], s[b] = oc[a], os_[a]
    assert int(used.item()) == len({int(b) for b in new.ravel() if b >= 0})
    for seq, row in ((0, new[0]), (2, new[1])):
        keep = -(-lens[seq] // bs)
        free = [b for b in range(nb) if b not in set(new.ravel().tolist())]
        tables[seq] = [int(b) for b in row[:keep]] + free[4 * seq:4 * seq + 4]
    for (c, s), (gc, gs) in zip(pool.host, pool.gpu):
        live = new[new >= 0]
        assert np.array_equal(gc.cpu().numpy()[live], c[live]) and np.array_equal(gs.cpu().numpy()[live], s[live])
        c[:], s[:] = gc.cpu().numpy(), gs.cpu().numpy()
    step([0, 2], [1, 1])
    # a shift of sequence 0 by 16 positions: whole blocks turned back
    pos = np.arange(lens[0])
    slots = dev(slots_of(0, pos))
    k = kv.dequant_block_scaled(kc, ks, slots)
    v = kv.dequant_block_scaled(vc, vs, slots)
    plain, _ = kv.rotary_frequencies(hd, 10000.0, "parts", 4.0, 64)
    k2, _ = kv.rotary_embedding(k, None, torch.full((len(pos),), 16, device="cuda"), plain, transpose=True)
    pool.write(k2, v, slots_of(0, pos))
    step([0, 2], [1, 1])
