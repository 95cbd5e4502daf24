"""Page copies and compaction on the GPU against the oracle, byte for byte, and a serving sequence
that uses them with the 4-bit cache."""
import numpy as np
import pytest
import torch

from oracle import fp4

pytestmark = pytest.mark.gpu

kv = pytest.importorskip("fp8_paged_kv_reshape_gb300")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def pool(r, nb, shapes):
    return [r.integers(0, 256, (nb, *s)).astype(np.uint8) for s in shapes]


SHAPES = [[(16, 2, 64)], [(16,)], [(16, 8, 128), (16, 8, 128)], [(8, 1, 32), (1, 8, 4), (48,)],
          [(16, 2, 32), (2, 16, 4)] * 3, [(5000 * 16,), (1024,), (4096 + 32,)]]


def check_copy(caches, src, dst, st=None):
    got = [dev(c) for c in caches]
    st = status()
    kv.copy_blocks(got, dev(np.array(src, np.int32)), dev(np.array(dst, np.int32)), status=st)
    torch.cuda.synchronize()
    refused = fp4.copy_blocks(caches, list(src), list(dst))
    assert int(st.item()) == (kv.DEV_BAD_BLOCK if refused else 0)
    for g, c in zip(got, caches):
        assert np.array_equal(g.cpu().numpy(), c)
    return refused


@pytest.mark.parametrize("shapes", SHAPES)
@pytest.mark.parametrize("nb, n", [(1, 0), (2, 1), (33, 16), (200, 70)])
def test_copies(shapes, nb, n):
    r = np.random.default_rng(nb)
    ids = r.permutation(nb)[:2 * n].astype(np.int32)
    src, dst = ids[:n].copy(), ids[n:]
    if n > 4:
        src[3], src[4] = src[0], -1  # one source for several destinations; padding
    assert not check_copy(pool(r, nb, shapes), src, dst)


def test_many_copies_and_many_caches():
    r = np.random.default_rng(1)
    ids = r.permutation(20000).astype(np.int32)
    assert not check_copy(pool(r, 20000, [(16, 16)]), ids[:9000], ids[9000:18000])
    ids = r.permutation(64).astype(np.int32)
    assert not check_copy(pool(r, 64, [(16 * (1 + i % 5),) for i in range(kv.MAX_CACHES)]), ids[:30], ids[30:60])


@pytest.mark.parametrize("src, dst", [
    ([1, 2], [5, 5]),                      # one destination twice
    ([1, 1, 1], [5, 5, 5]),
    ([1, 5], [5, 7]),                      # a chain
    ([1, 2], [2, 1]),                      # a swap
    ([3, 1, 4], [3, 2, 4]),                # blocks onto themselves
    ([3, 6], [3, 3]),                      # a block onto itself and one onto it
    ([8, 1, -2, 0], [1, 8, 2, 3]),         # outside the pool
    ([-1, 4, -1], [2, -1, -1]),            # padding
    ([8, 5], [5, 6]),                      # a pair outside does not count against the others
    ([0, 7, 31, 32], [30, 33, 1, 2]),
])
def test_conflicting_and_outside_pairs(src, dst):
    r = np.random.default_rng(2)
    check_copy(pool(r, 8 if max(src + dst) <= 8 else 34, [(16, 2, 64), (2, 16, 4)]), src, dst)


def test_random_pairs_with_conflicts():
    r = np.random.default_rng(3)
    for nb in (31, 64, 1000):
        assert check_copy(pool(r, nb, [(64,)]), r.integers(-2, nb + 2, nb), r.integers(-2, nb + 2, nb))


def test_copy_refuses_a_pool_past_its_limit():
    big = torch.empty(900001, 16, dtype=torch.uint8, device="cuda")
    ids = dev(np.array([0], np.int32))
    with pytest.raises(kv.KvFp8Error) as e:
        kv.copy_blocks([big], ids, ids)
    assert e.value.status == kv.ERR_UNSUPPORTED
    big = big[:900000]
    big.zero_()
    big[5] = 3
    kv.copy_blocks([big], dev(np.array([5], np.int32)), dev(np.array([899999], np.int32)))
    assert bool((big[899999] == 3).all()) and int(big.sum()) == 2 * 48


def check_compact(caches, bt, lens, bs, in_place=False):
    got = [dev(c) for c in caches]
    t, st = dev(bt), status()
    new, used = kv.compact_blocks(got, t, dev(lens), bs, new_block_tables=t if in_place else None, status=st)
    torch.cuda.synchronize()
    want, n, flagged = fp4.compact(caches, bt, lens, bs)
    assert int(st.item()) == (kv.DEV_BAD_BLOCK if flagged else 0)
    assert int(used.item()) == n
    assert np.array_equal(new.cpu().numpy(), want)
    for g, c in zip(got, caches):
        assert np.array_equal(g.cpu().numpy(), c)
    if not in_place:
        assert np.array_equal(t.cpu().numpy(), bt)
    return want, n


def tables(r, nb, lens, bs, share=0.0):
    need = [-(-int(n) // bs) for n in lens]
    ids = r.permutation(nb)
    bt = r.integers(-5, nb + 5, (len(lens), max(need + [1]))).astype(np.int32)  # junk past the lengths
    at = 0
    for i, n in enumerate(need):
        bt[i, :n] = ids[at:at + n]
        at += n
        if i > 0 and r.random() < share:
            k = min(n, need[i - 1])
            bt[i, :k] = bt[i - 1, :k]
    return bt


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("nb, n, longest, share", [(1, 1, 16, 0), (33, 4, 90, 0), (33, 4, 90, 0.7), (70, 7, 160, 0.5),
                                                   (1025, 40, 400, 0.2), (40000, 300, 1600, 0.1), (64, 4, 256, 0)])
def test_compaction(nb, n, longest, share, in_place):
    r = np.random.default_rng(nb + n)
    lens = np.minimum(r.integers(0, longest + 1, n), nb * 16 // n).astype(np.int32)
    lens[0] = min(longest, nb * 16 // n)
    check_compact(pool(r, nb, [(16, 2), (32,)]), tables(r, nb, lens, 16, share), lens, 16, in_place)


def test_compaction_of_odd_pools():
    r = np.random.default_rng(9)
    for nb, ids in ((10, range(10)), (10, range(5)), (10, range(5, 10)), (33, [32]), (64, [63, 0]), (2048 * 32 + 1, [2048 * 32, 7])):
        bt = np.array([list(ids)], np.int32)
        check_compact(pool(r, nb, [(16,)]), bt, np.array([bt.shape[1] * 8], np.int32), 8)
    check_compact(pool(r, 10, [(16,)]), np.zeros((2, 3), np.int32), np.zeros(2, np.int32), 8)      # nothing used
    check_compact(pool(r, 10, [(16,)]), np.zeros((0, 3), np.int32), np.zeros(0, np.int32), 8)      # no sequences
    bt = np.array([[9, 3, 50], [-1, 4, 7]], np.int32)
    check_compact(pool(r, 10, [(16,)]), bt, np.array([24, 16], np.int32), 8)                       # ids outside
    check_compact(pool(r, 10, [(16,)]), bt % 10, np.array([99, -4], np.int32), 8)                  # lengths outside
    check_compact(pool(r, 10, [(16,)]), bt % 10, np.array([3, 2], np.int32), 1)                    # one token a block


def test_compaction_workspace_shared_in_order_and_captured():
    """One workspace for calls that follow one another, eager and captured, on changing tables."""
    r = np.random.default_rng(10)
    nb, bs, lens = 100, 16, np.array([160, 33, 300], np.int32)
    bt = dev(tables(r, nb, lens, bs))
    cache = dev(pool(r, nb, [(64,)])[0])
    ws = torch.full((kv.compact_blocks_workspace_size(nb),), 0xFF, dtype=torch.uint8, device="cuda")
    new, used = torch.empty_like(bt), torch.empty(1, dtype=torch.int32, device="cuda")
    args = dict(new_block_tables=new, num_used=used, workspace=ws)
    kv.compact_blocks([cache], bt, dev(lens), bs, **args)  # the kernels are loaded before the capture
    lens_t = dev(lens)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.compact_blocks([cache], bt, lens_t, bs, **args)
    for _ in range(3):
        host_bt, host = tables(r, nb, lens, bs), pool(r, nb, [(64,)])
        bt.copy_(dev(host_bt))
        cache.copy_(dev(host[0]))
        g.replay()
        torch.cuda.synchronize()
        want, n, _ = fp4.compact(host, host_bt, lens, bs)
        assert np.array_equal(new.cpu().numpy(), want) and int(used.item()) == n
        assert np.array_equal(cache.cpu().numpy(), host[0])


def test_unaligned_and_sixteen_byte_caches():
    r = np.random.default_rng(11)
    flat = torch.from_numpy(r.integers(0, 256, 50 * 96 + 16).astype(np.uint8)).cuda()
    c = flat[16:].view(50, 96)  # 16-byte, not 32-byte aligned
    host = c.cpu().numpy().copy()
    kv.copy_blocks([c], dev(np.array([1, 2], np.int32)), dev(np.array([40, 41], np.int32)))
    fp4.copy_blocks([host], [1, 2], [40, 41])
    assert np.array_equal(c.cpu().numpy(), host)


@pytest.mark.parametrize("fp4_cache", [True, False], ids=["fp4", "e4m3"])
def test_serving_a_fork(fp4_cache):
    """A prompt is written, the sequence forks (shared pages, its last page copied on write), both
    branches append and attend, the first ends, the pool is compacted and cut: what the second
    branch reads is unchanged to the bit at each step."""
    r = np.random.default_rng(12)
    n_q, n_kv, hd, bs, nb, n = 32, 8, 128, 16, 64, 100
    ids = r.permutation(nb).astype(np.int32)
    first, fork = ids[:8].copy(), ids[:8].copy()
    fork[6:] = ids[20:22]  # page 6 (tokens 96..) is copied, page 7 is new
    ks, vs = torch.tensor([0.05], device="cuda"), torch.tensor([0.04], device="cuda")
    shape = (nb, bs, n_kv, hd // 2 if fp4_cache else hd)
    caches = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    if fp4_cache:
        caches += [torch.full((nb, n_kv, bs, hd // 16), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def write(x, slots):
        fn = kv.reshape_and_cache_fp4 if fp4_cache else kv.reshape_and_cache
        fn(x[0], x[1], *caches, dev(np.asarray(slots, np.int64)), ks, vs, status=st)

    def attend(q, bt, lens):
        fn = kv.paged_decode_attention_fp4 if fp4_cache else kv.paged_decode_attention
        return fn(q, *caches, bt, dev(np.asarray(lens, np.int32)), ks, vs, status=st)

    def rows(count):
        return torch.from_numpy(r.standard_normal((2, count, n_kv, hd))).bfloat16().cuda()

    st = status()
    slot = lambda t, pos: int(t[pos // bs]) * bs + pos % bs  # noqa: E731
    write(rows(n), [slot(first, p) for p in range(n)])
    q = torch.from_numpy(r.standard_normal((2, n_q, hd))).bfloat16().cuda()
    alone = attend(q[:1], dev(first[None]), [n])
    kv.copy_blocks(caches, dev(first[6:7]), dev(fork[6:7]), status=st)
    same = attend(q[[0, 0]], dev(np.stack([first, fork])), [n, n])
    assert torch.equal(same[0], alone[0]) and torch.equal(same[1], alone[0])
    for pos in range(n, n + 14):  # both grow, onto page 7 of each
        write(rows(2), [slot(first, pos), slot(fork, pos)])
    bt = dev(np.stack([first, fork]))
    both = attend(q, bt, [n + 14, n + 14])
    assert not torch.equal(both[0], both[1])
    bt2, used = kv.compact_blocks(caches, bt, dev(np.array([0, n + 14], np.int32)), bs, status=st)
    torch.cuda.synchronize()
    assert int(used.item()) == 8 and sorted(bt2[1].tolist()) == list(range(8)) and bt2[0].tolist() == [-1] * 8
    caches = [c[:8].clone() for c in caches]  # the pool is cut
    after = attend(q[1:], bt2[1:].contiguous(), [n + 14])
    assert torch.equal(after[0], both[1])
    torch.cuda.synchronize()
    assert int(st.item()) == 0
