"""Sizes at the edge of what the kernels index (CPU only): refused with their code before anything is launched."""
import ctypes

import pytest

import fp8_paged_kv_reshape_gb300 as kv
from fp8_paged_kv_reshape_gb300 import binding

P16 = ctypes.c_void_p(16)


def multi(fp4: bool, qmax, group, num_seqs, n_kv):
    caches = [P16] * (4 if fp4 else 2)
    fn = kv.LIB.kvfp8_paged_attention_multi_fp4 if fp4 else kv.LIB.kvfp8_paged_attention_multi
    # (a null output, which is refused after the sizes)
    return fn(None, P16, P16, 64, qmax, *caches, P16, 256, P16, num_seqs, n_kv * group, n_kv, 128, 16, 1024, 0.0, None, None,
              binding.F32, P16, 1 << 30, None, None)


@pytest.mark.parametrize("fp4", [True, False], ids=["fp4", "e4m3"])
@pytest.mark.parametrize("qmax, group, num_seqs, n_kv", [
    ((1 << 28) + 16, 16, 4, 8),      # 2^32 + 256 score rows per kv head: 256 in 32 bits
    (1 << 24, 128, 1, 1),            # 2^31
    ((1 << 31) - 1, 1, 1, 1),        # the last tile's end would pass 2^31
    ((1 << 31) - 1, 128, 1, 1),
    ((1 << 31) - 1, 128, 1 << 20, 1 << 10),  # 2^61 row tiles
    ((1 << 31) - 1, 128, (1 << 31) - 1, 128),  # past 64 bits
])
def test_score_rows_past_32_bits(fp4, qmax, group, num_seqs, n_kv):
    assert multi(fp4, qmax, group, num_seqs, n_kv) == binding.ERR_UNSUPPORTED


@pytest.mark.parametrize("fp4", [True, False], ids=["fp4", "e4m3"])
@pytest.mark.parametrize("qmax, group, num_seqs, n_kv", [(1 << 20, 128, 1, 1), (512, 16, 64, 8), ((1 << 24) - 4, 128, 1, 1)])
def test_large_chunks_below_that(fp4, qmax, group, num_seqs, n_kv):
    assert multi(fp4, qmax, group, num_seqs, n_kv) == binding.ERR_NULL


def test_a_batch_without_new_tokens_has_nothing_to_do():
    """No query rows: torch's empty tensors have null pointers."""
    call = lambda rows, q: kv.LIB.kvfp8_paged_attention_multi_fp4(  # noqa: E731
        q, q, P16, rows, 4, P16, P16, P16, P16, P16, 256, P16, 4, 32, 8, 128, 16, 1024, 0.0, None, None,
        binding.F32, P16, 1 << 30, None, None)
    assert call(0, None) == binding.OK
    assert call(1, None) == binding.ERR_NULL
