"""Host-side refusals of the 4-bit cache and page calls (CPU only): documented codes come back
before anything touches a GPU, and the binding checks what it passes on."""
import ctypes

import pytest
import torch

import fp8_paged_kv_reshape_gb300 as kv
from fp8_paged_kv_reshape_gb300 import binding

P16 = ctypes.c_void_p(16)


def _call(fn, args, over):
    args = dict(args)
    assert set(over) <= set(args), over
    args.update(over)
    return fn(*args.values())


def _write(**over):
    return _call(kv.LIB.kvfp8_reshape_and_cache_fp4, dict(
        key=P16, value=P16, src_dtype=binding.BF16, key_stride=1024, value_stride=1024, num_tokens=4,
        key_cache=P16, value_cache=P16, key_scales=P16, value_scales=P16, num_blocks=4, block_size=16,
        n_kv=8, head_dim=128, slot_mapping=P16, k_scale=None, v_scale=None, scale_dtype=binding.F32,
        status=None, stream=None), over)


def _read(**over):
    return _call(kv.LIB.kvfp8_dequant_fp4, dict(
        dst=P16, dst_dtype=binding.BF16, codes=P16, scales=P16, num_blocks=4, block_size=16, n_kv=8,
        head_dim=128, slot_mapping=P16, num_tokens=4, scale=None, scale_dtype=binding.F32, status=None,
        stream=None), over)


def _decode(**over):
    return _call(kv.LIB.kvfp8_paged_decode_attention_fp4, dict(
        out=P16, query=P16, key_cache=P16, value_cache=P16, key_scales=P16, value_scales=P16,
        block_tables=P16, max_blocks_per_seq=256, seq_lens=P16, num_seqs=4, n_q=32, n_kv=8, head_dim=128,
        block_size=16, num_blocks=1024, sm_scale=0.0, k_scale=None, v_scale=None, scale_dtype=binding.F32,
        workspace=P16, workspace_bytes=1 << 30, status=None, stream=None), over)


def _multi(**over):
    return _call(kv.LIB.kvfp8_paged_attention_multi_fp4, dict(
        out=P16, query=P16, qsl=P16, rows=16, qmax=4, key_cache=P16, value_cache=P16, key_scales=P16,
        value_scales=P16, block_tables=P16, max_blocks_per_seq=256, seq_lens=P16, num_seqs=4, n_q=32,
        n_kv=8, head_dim=128, block_size=16, num_blocks=1024, sm_scale=0.0, k_scale=None, v_scale=None,
        scale_dtype=binding.F32, workspace=P16, workspace_bytes=1 << 30, status=None, stream=None), over)


def _pages(fn, args, over, ptrs=(16, 4096), sizes=(1024, 64)):
    p = (ctypes.c_void_p * len(ptrs))(*ptrs)
    s = (ctypes.c_int64 * len(sizes))(*sizes)
    return _call(fn, dict(dict(caches=p, block_bytes=s, num_caches=len(ptrs), num_blocks=8), **args), over)


def _copy(ptrs=(16, 4096), sizes=(1024, 64), **over):
    return _pages(kv.LIB.kvfp8_copy_blocks, dict(src=P16, dst=P16, pairs=3, status=None, stream=None),
                  over, ptrs, sizes)


def _compact(ptrs=(16, 4096), sizes=(1024, 64), **over):
    return _pages(kv.LIB.kvfp8_compact_blocks, dict(
        block_size=16, tables=P16, most=4, seq_lens=P16, num_seqs=2, new_tables=P16, num_used=P16,
        workspace=P16, workspace_bytes=1 << 20, status=None, stream=None), over, ptrs, sizes)


@pytest.mark.parametrize("over, code", [
    (dict(src_dtype=7), binding.ERR_DTYPE), (dict(scale_dtype=-1), binding.ERR_DTYPE),
    (dict(num_tokens=-1), binding.ERR_SHAPE), (dict(head_dim=96), binding.ERR_SHAPE),
    (dict(block_size=24), binding.ERR_SHAPE), (dict(block_size=4), binding.ERR_SHAPE),
    (dict(num_blocks=0), binding.ERR_SHAPE), (dict(num_blocks=1 << 28, block_size=256), binding.ERR_SHAPE),
    (dict(key_stride=1016), binding.ERR_SHAPE), (dict(n_kv=1 << 14, key_stride=1 << 21, value_stride=1 << 21), binding.ERR_SHAPE),
    (dict(key=None), binding.ERR_NULL), (dict(value_scales=None), binding.ERR_NULL),
    (dict(slot_mapping=None), binding.ERR_NULL), (dict(key_scales=ctypes.c_void_p(24)), binding.ERR_ALIGN),
    (dict(value_stride=1028), binding.ERR_ALIGN), (dict(slot_mapping=ctypes.c_void_p(20)), binding.ERR_ALIGN),
    (dict(num_tokens=0, key=None), binding.OK)])
def test_write_refusals(over, code):
    assert _write(**over) == code


@pytest.mark.parametrize("over, code", [
    (dict(dst_dtype=3), binding.ERR_DTYPE), (dict(head_dim=32), binding.ERR_SHAPE),
    (dict(block_size=12), binding.ERR_SHAPE), (dict(num_tokens=-5), binding.ERR_SHAPE),
    (dict(n_kv=0), binding.ERR_SHAPE), (dict(dst=None), binding.ERR_NULL), (dict(scales=None), binding.ERR_NULL),
    (dict(codes=ctypes.c_void_p(8)), binding.ERR_ALIGN), (dict(num_tokens=0, dst=None), binding.OK)])
def test_read_refusals(over, code):
    assert _read(**over) == code


@pytest.mark.parametrize("over, code", [
    (dict(scale_dtype=2), binding.ERR_DTYPE), (dict(n_q=30), binding.ERR_SHAPE), (dict(head_dim=192), binding.ERR_SHAPE),
    (dict(block_size=512), binding.ERR_SHAPE), (dict(n_q=129 * 8), binding.ERR_UNSUPPORTED),
    (dict(sm_scale=float("nan")), binding.ERR_SCALE), (dict(query=None), binding.ERR_NULL),
    (dict(key_scales=None), binding.ERR_NULL), (dict(workspace=None), binding.ERR_NULL),
    (dict(value_scales=ctypes.c_void_p(8)), binding.ERR_ALIGN), (dict(out=ctypes.c_void_p(8)), binding.ERR_ALIGN),
    (dict(workspace_bytes=64), binding.ERR_WORKSPACE), (dict(num_seqs=0, query=None), binding.OK),
    (dict(n_kv=1 << 20, n_q=1 << 20, num_blocks=1 << 12), binding.ERR_SHAPE)])  # 2^32 (block, head) rows
def test_decode_refusals(over, code):
    assert _decode(**over) == code


@pytest.mark.parametrize("over, code", [
    (dict(qmax=0), binding.ERR_SHAPE), (dict(rows=-1), binding.ERR_SHAPE), (dict(max_blocks_per_seq=0), binding.ERR_SHAPE),
    (dict(head_dim=96), binding.ERR_SHAPE), (dict(qsl=None), binding.ERR_NULL), (dict(workspace=None), binding.ERR_NULL),
    (dict(qmax=64, workspace=None, workspace_bytes=0, value_scales=None), binding.ERR_NULL),
    (dict(qsl=ctypes.c_void_p(18)), binding.ERR_ALIGN), (dict(workspace_bytes=64), binding.ERR_WORKSPACE),
    (dict(n_q=129 * 8), binding.ERR_UNSUPPORTED), (dict(num_seqs=1 << 20, n_q=128 * 8, qmax=1 << 12), binding.ERR_UNSUPPORTED),
    # 2^64 row tiles
    (dict(num_seqs=1 << 20, n_q=1 << 20, n_kv=1 << 20, num_blocks=1, qmax=(1 << 31) - 1), binding.ERR_UNSUPPORTED),
    (dict(sm_scale=float("inf")), binding.ERR_SCALE), (dict(num_seqs=0, query=None), binding.OK)])
def test_multi_refusals(over, code):
    assert _multi(**over) == code


@pytest.mark.parametrize("over, code", [
    (dict(num_caches=0), binding.ERR_SHAPE), (dict(num_caches=129), binding.ERR_SHAPE),
    (dict(num_blocks=0), binding.ERR_SHAPE), (dict(num_blocks=(1 << 30) + 1), binding.ERR_SHAPE), (dict(pairs=-1), binding.ERR_SHAPE), (dict(pairs=1 << 31), binding.ERR_SHAPE),
    (dict(caches=None), binding.ERR_NULL), (dict(block_bytes=None), binding.ERR_NULL), (dict(src=None), binding.ERR_NULL),
    (dict(ptrs=(16, 0)), binding.ERR_NULL), (dict(sizes=(1024, 0)), binding.ERR_SHAPE),
    (dict(sizes=(1024, 24)), binding.ERR_ALIGN), (dict(ptrs=(16, 4104)), binding.ERR_ALIGN),
    (dict(dst=ctypes.c_void_p(18)), binding.ERR_ALIGN), (dict(pairs=0, src=None), binding.OK)])
def test_copy_refusals(over, code):
    assert _copy(**over) == code


@pytest.mark.parametrize("over, code", [
    (dict(block_size=0), binding.ERR_SHAPE), (dict(num_seqs=-1), binding.ERR_SHAPE), (dict(most=0), binding.ERR_SHAPE),
    (dict(most=1 << 30), binding.ERR_SHAPE), (dict(tables=None), binding.ERR_NULL), (dict(num_used=None), binding.ERR_NULL),
    (dict(workspace=None), binding.ERR_NULL), (dict(workspace=ctypes.c_void_p(24)), binding.ERR_ALIGN),
    (dict(new_tables=ctypes.c_void_p(18)), binding.ERR_ALIGN), (dict(workspace_bytes=16), binding.ERR_WORKSPACE),
    (dict(sizes=(1000, 64)), binding.ERR_ALIGN)])
def test_compact_refusals(over, code):
    assert _compact(**over) == code


def test_attention_workspace_follows_the_route():
    ws = kv.paged_attention_fp4_workspace_size
    assert ws(4, 32, 8, 128, 1, 256, 16) == kv.paged_decode_workspace_size(4, 32, 128) > 0
    assert ws(4, 32, 8, 128, 4, 256, 16) == kv.paged_attention_multi_workspace_size(4, 32, 8, 128, 4) > 0
    # 20 columns: tensor cores.  32 row tiles leave SMs idle, so their keys are split over four parts
    assert ws(4, 32, 8, 128, 5, 256, 16) == 32 * 4 * 128 * (128 + 1) * 4
    assert ws(4, 32, 8, 128, 5, 15, 16) == 0                                  # fewer than two parts of 128 keys
    assert ws(10, 32, 8, 128, 5, 256, 16) == 0 and ws(4, 32, 8, 128, 512, 256, 16) == 0  # enough row tiles
    assert ws(4, 32, 8, 128, 1, 16, 16) == 0 < ws(4, 32, 8, 128, 1, 17, 16)   # 256 tokens: not split
    assert ws(-1, 32, 8, 128, 1, 256, 16) == ws(4, 32, 8, 128, 1, 0, 16) == 0
    assert _decode(max_blocks_per_seq=16, workspace=None, workspace_bytes=0, num_blocks=0) == binding.ERR_SHAPE
    assert _decode(max_blocks_per_seq=17, workspace=None) == binding.ERR_NULL
    assert _multi(max_blocks_per_seq=16, workspace=None, workspace_bytes=0, qsl=None) == binding.ERR_NULL


def test_compact_workspace_size():
    assert kv.compact_blocks_workspace_size(0) == 0
    assert 0 < kv.compact_blocks_workspace_size(1) <= kv.compact_blocks_workspace_size(100000)


def test_binding_checks():
    """Shapes, types and devices are refused in Python (here every tensor is on the CPU, which is
    itself refused last)."""
    u8 = torch.uint8
    kc, kg = torch.zeros(4, 16, 2, 32, dtype=u8), torch.zeros(4, 2, 16, 4, dtype=u8)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    bt, sl = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    good = dict(key=k, value=k, key_cache=kc, value_cache=kc, key_scales=kg, value_scales=kg, slot_mapping=slots)
    for over in (dict(), dict(key_scales=kg[:, :, :8]), dict(key_cache=kc.float()), dict(value_cache=kc[..., :16]),
                 dict(slot_mapping=slots.int()), dict(slot_mapping=slots[:2]), dict(key=k.transpose(0, 1)),
                 dict(status=torch.zeros(1))):
        with pytest.raises(ValueError):
            kv.reshape_and_cache_fp4(**{**good, **over})
    with pytest.raises(TypeError):
        kv.reshape_and_cache_fp4(**{**good, "value": k.float()})
    for over in (dict(), dict(slot_mapping=slots.int()), dict(out=torch.zeros(2, 2, 64, dtype=torch.bfloat16)),
                 dict(scales=kg.transpose(1, 2))):
        with pytest.raises(ValueError):
            kv.dequant_fp4(**{**dict(cache=kc, scales=kg, slot_mapping=slots), **over})
    att = dict(query=q, key_cache=kc, value_cache=kc, key_scales=kg, value_scales=kg, block_tables=bt, seq_lens=sl)
    for over in (dict(), dict(seq_lens=sl.long()), dict(block_tables=bt[:2]), dict(query=q.float()),
                 dict(query=torch.zeros(3, 4, 128, dtype=torch.bfloat16)), dict(out=q[:2]),
                 dict(value_scales=kg.transpose(1, 2))):
        with pytest.raises(ValueError):
            kv.paged_decode_attention_fp4(**{**att, **over})
        with pytest.raises(ValueError):
            kv.paged_attention_multi_fp4(query_start_loc=torch.arange(4, dtype=torch.int32), max_query_len=1,
                                         **{**att, **over})
    with pytest.raises(ValueError):
        kv.paged_attention_multi_fp4(query_start_loc=torch.arange(3, dtype=torch.int32), max_query_len=1, **att)
    ids = torch.zeros(2, dtype=torch.int32)
    for caches, s, d in (([kc, kg], ids, ids), ([], ids, ids), ([kc, kg[:2]], ids, ids), ([kc] * 129, ids, ids),
                         ([kc, kc], ids, ids), ([kc.transpose(0, 1)], ids, ids)):
        with pytest.raises(ValueError):
            kv.copy_blocks(caches, s, d)
        with pytest.raises(ValueError):
            kv.compact_blocks(caches, bt, sl, 16)
