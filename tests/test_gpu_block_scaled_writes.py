"""More of the writer of the FP8 cache with block scales, beside test_gpu_block_scaled.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_block_scaled import Pool, dev, rows, status

pytestmark = pytest.mark.gpu

kv = pytest.importorskip("fp8_paged_kv_reshape_gb300")


@pytest.mark.parametrize("n_kv, hd, bs, n", [(8, 128, 16, 600), (2, 256, 64, 900), (1, 64, 256, 2000), (4, 64, 32, 300)])
def test_writes_past_32_bits(n_kv, hd, bs, n):
    """Rows into blocks that lie past 4 GB of codes give what the same rows give at the front of a small pool, which the oracle
    checks: calls of some hundred rows (searched) and longer ones (listed), with blocks of few rows, of more than a warp holds,
    and scales that are kept or raised."""
    r = np.random.default_rng(n)
    nb = -(-n // bs) + 3
    at = (1 << 32) // (bs * n_kv * hd) + 5
    listed = kv.reshape_and_cache_block_scaled_workspace_size(n, nb, bs) > 0
    assert listed == (n > 512)
    pool = Pool(nb, bs, n_kv, hd, fill=lambda r, shape: np.exp2(r.integers(-12, -3, shape)))
    big = []
    for t in (t for side in pool.gpu for t in side):
        p = torch.empty((at + nb,) + t.shape[1:], dtype=t.dtype, device="cuda")
        p[at:] = t
        big.append(p)
    kc, ks, vc, vs = big
    assert kc.numel() > 1 << 32
    for spread, slots in ((2.0, r.permutation(nb * bs)[:n]), (4.0, np.arange(n) + 1), (3.0, np.arange(n))):
        slots = slots.astype(np.int64)
        x = rows(r, n, n_kv, hd, spread=spread)
        pool.write(x[0], x[1], slots)
        st = status()
        kv.reshape_and_cache_block_scaled(x[0], x[1], kc, vc, ks, vs, dev(slots + at * bs), status=st)
        assert int(st.item()) == 0
        for (c, s), (bc, bsc) in zip(pool.gpu, ((kc, ks), (vc, vs))):
            assert torch.equal(bc[at:], c) and torch.equal(bsc[at:], s)
            got = kv.dequant_block_scaled(bc, bsc, dev(slots + at * bs), torch.float32)
            want = kv.dequant_block_scaled(c, s, dev(slots), torch.float32)
            assert torch.equal(got.view(torch.int32), want.view(torch.int32))


@pytest.mark.parametrize("dst", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n, n_kv, hd", [(1, 1, 64), (37, 3, 64), (700, 8, 128), (5, 2, 256)])
def test_rows_read_back_to_any_aligned_place(dst, n, n_kv, hd):
    """out at 16 bytes past a multiple of 32, and nothing beside it written."""
    r = np.random.default_rng(n)
    nb, bs = n // 16 + 2, 16
    codes = dev(r.integers(0, 0x7F, (nb, bs, n_kv, hd)).astype(np.uint8))
    scales = dev(np.exp2(r.integers(-20, 20, (nb, -(-n_kv // 4) * 4))).astype(np.float32))
    slots = dev(r.integers(0, nb * bs, n))
    want = kv.dequant_block_scaled(codes, scales, slots, dst)
    size, step = n * n_kv * hd, 16 // want.element_size()
    buffer = torch.full((size + 4 * step,), 7.0, dtype=dst, device="cuda")
    out = buffer[step:step + size].view(n, n_kv, hd)
    assert buffer.data_ptr() % 32 == 0 and out.data_ptr() % 32 == 16
    assert kv.dequant_block_scaled(codes, scales, slots, dst, out=out).data_ptr() == out.data_ptr()
    assert torch.equal(out, want) and bool((buffer[:step] == 7).all()) and bool((buffer[step + size:] == 7).all())
