"""The bounded waits of the attention kernels over block scales, made to run out on the GPU without any fault.

As in test_gpu_timeout.py: a test-only build of the library whose CTAs withhold the copy of their first chunk (no copy, no arrival)
and whose waits give up after about 1e5 cycles.  Every wait on that chunk runs out or sees that another did, copies that were issued
land (they take a few microseconds of the 50 that a wait lasts), tensor memory is released, and the call returns with
KVFP8_DEV_TIMEOUT; the next call is right.
"""
import ctypes
import time

import pytest
import torch

from tests.test_gpu_block_scaled import build, caches, dev

pytestmark = pytest.mark.gpu

kv = pytest.importorskip("fp8_paged_kv_reshape_gb300")
from fp8_paged_kv_reshape_gb300 import _build, binding  # noqa: E402

CASES = [
    # n_q, n_kv, head_dim, lengths, query tokens
    (4, 2, 64, [17, 100], 1),                # whole sequences
    (8, 2, 128, [3000, 260], 1),             # split over the grid
    (8, 2, 64, [40] * 299 + [300], 1),       # with a plan kernel
    (16, 2, 128, [700, 90], 2),              # 16 score columns
    (4, 2, 256, [700, 90], 2),
    (8, 2, 128, [100, 60], 20),              # one row tile, a tile of keys
    (8, 2, 128, [3000], 20),                 # split
    (8, 2, 64, [700, 300], 70),              # two row tiles, scores ahead
    (8, 2, 128, [700, 300], 70),             # a thread per row tile issuing
    (8, 2, 128, [5000], 200),                # split
    (4, 2, 256, [700, 300], 70),
]


@pytest.fixture(scope="module")
def withhold_lib():
    lib = ctypes.CDLL(_build.build_withhold_variant())  # its own symbols (RTLD_LOCAL)
    call = lib.kvfp8_paged_attention_multi_block_scaled
    call.argtypes = kv.LIB.kvfp8_paged_attention_multi_block_scaled.argtypes
    call.restype = ctypes.c_int
    return lib


@pytest.mark.parametrize("n_q, n_kv, hd, lengths, qlen", CASES)
def test_waits_run_out_and_the_next_call_is_correct(withhold_lib, n_q, n_kv, hd, lengths, qlen):
    qlens = [min(qlen, n) for n in lengths]
    c = build(n_q, n_kv, hd, 16, lengths, qlens, 51)
    q, qsl = c["q"].cuda(), dev(c["qsl"])
    kc, vc, ks, vs, bt, lens = caches(c)
    normal = lambda: kv.paged_attention_multi_block_scaled(q, qsl, qlen, kc, vc, ks, vs, bt, lens)  # noqa: E731
    want = normal()
    need = kv.paged_attention_block_scaled_workspace_size(len(lengths), n_q, n_kv, hd, qlen, bt.shape[1], 16)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    out, st = torch.zeros_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    rc = withhold_lib.kvfp8_paged_attention_multi_block_scaled(
        p(out), p(q), p(qsl), q.shape[0], qlen, 1, p(kc), p(vc), p(ks), p(vs), ks.shape[1], p(bt), bt.shape[1], p(lens), len(lengths),
        n_q, n_kv, hd, 16, kc.shape[0], 0.0, p(ws), need, p(st), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()  # the kernels ended
    assert rc == binding.OK and time.perf_counter() - t0 < 10.0
    assert int(st.item()) == kv.DEV_TIMEOUT
    assert torch.equal(normal(), want)
