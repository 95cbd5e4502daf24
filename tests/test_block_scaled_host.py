"""Host-side refusals of the calls of the cache with block scales and of rotary positions (CPU only): documented codes
come back before anything touches a GPU, and the binding checks what it passes on."""
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
    return _call(kv.LIB.kvfp8_reshape_and_cache_block_scaled, dict(
        key=P16, value=P16, src_dtype=binding.BF16, key_stride=1024, value_stride=1024, num_tokens=4, key_cache=P16,
        value_cache=P16, key_scales=P16, value_scales=P16, scale_stride=8, num_blocks=4, block_size=16, n_kv=8, head_dim=128,
        slot_mapping=P16, workspace=P16, workspace_bytes=1 << 30, status=None, stream=None), over)


def _read(**over):
    return _call(kv.LIB.kvfp8_dequant_block_scaled, dict(
        dst=P16, dst_dtype=binding.BF16, codes=P16, scales=P16, scale_stride=8, num_blocks=4, block_size=16, n_kv=8,
        head_dim=128, slot_mapping=P16, num_tokens=4, status=None, stream=None), over)


def _decode(**over):
    return _call(kv.LIB.kvfp8_paged_decode_attention_block_scaled, dict(
        out=P16, query=P16, key_cache=P16, value_cache=P16, key_scales=P16, value_scales=P16, scale_stride=8,
        block_tables=P16, max_blocks_per_seq=256, seq_lens=P16, num_seqs=4, n_q=32, n_kv=8, head_dim=128, block_size=16,
        num_blocks=1024, sm_scale=0.0, workspace=P16, workspace_bytes=1 << 30, status=None, stream=None), over)


def _multi(**over):
    return _call(kv.LIB.kvfp8_paged_attention_multi_block_scaled, dict(
        out=P16, query=P16, qsl=P16, rows=16, qmax=4, causal=0, key_cache=P16, value_cache=P16, key_scales=P16,
        value_scales=P16, scale_stride=8, block_tables=P16, max_blocks_per_seq=256, seq_lens=P16, num_seqs=4, n_q=32, n_kv=8,
        head_dim=128, block_size=16, num_blocks=1024, sm_scale=0.0, workspace=P16, workspace_bytes=1 << 30, status=None,
        stream=None), over)


def _rotary(**over):
    return _call(kv.LIB.kvfp8_rotary_embedding, dict(
        query_out=P16, key_out=P16, query_out_stride=4096, key_out_stride=1024, query=P16, key=P16, query_stride=4096,
        key_stride=1024, dtype=binding.BF16, num_tokens=4, n_q=32, n_k=8, head_dim=128, rot_dim=128, interleaved=0,
        transpose=0, positions=P16, frequencies=P16, magnitude=1.0, status=None, stream=None), over)


@pytest.mark.parametrize("over, code", [
    (dict(src_dtype=7), binding.ERR_DTYPE), (dict(num_tokens=-1), binding.ERR_SHAPE), (dict(num_tokens=1 << 31), binding.ERR_SHAPE),
    (dict(head_dim=96), binding.ERR_SHAPE), (dict(block_size=8), binding.ERR_SHAPE), (dict(block_size=24), binding.ERR_SHAPE),
    (dict(block_size=512), binding.ERR_SHAPE), (dict(num_blocks=0), binding.ERR_SHAPE),
    (dict(num_blocks=1 << 28, block_size=256), binding.ERR_SHAPE), (dict(scale_stride=7), binding.ERR_SHAPE),
    (dict(scale_stride=10), binding.ERR_SHAPE), (dict(scale_stride=4), binding.ERR_SHAPE), (dict(key_stride=1016), binding.ERR_SHAPE),
    (dict(n_kv=1 << 14, scale_stride=1 << 14, key_stride=1 << 21, value_stride=1 << 21), binding.ERR_SHAPE),
    (dict(key=None), binding.ERR_NULL), (dict(value_scales=None), binding.ERR_NULL), (dict(slot_mapping=None), binding.ERR_NULL),
    (dict(num_tokens=600, workspace=None), binding.ERR_NULL), (dict(key_scales=ctypes.c_void_p(24)), binding.ERR_ALIGN),
    (dict(value_stride=1028), binding.ERR_ALIGN), (dict(slot_mapping=ctypes.c_void_p(20)), binding.ERR_ALIGN),
    (dict(num_tokens=600, workspace=ctypes.c_void_p(24)), binding.ERR_ALIGN),
    (dict(num_tokens=600, workspace_bytes=255), binding.ERR_WORKSPACE), (dict(num_tokens=0, key=None), binding.OK)])
def test_write_refusals(over, code):
    assert _write(**over) == code


@pytest.mark.parametrize("over, code", [
    (dict(dst_dtype=3), binding.ERR_DTYPE), (dict(head_dim=32), binding.ERR_SHAPE), (dict(block_size=8), binding.ERR_SHAPE),
    (dict(num_tokens=-5), binding.ERR_SHAPE), (dict(n_kv=0), binding.ERR_SHAPE), (dict(scale_stride=4), binding.ERR_SHAPE),
    (dict(dst=None), binding.ERR_NULL), (dict(scales=None), binding.ERR_NULL), (dict(codes=ctypes.c_void_p(8)), binding.ERR_ALIGN),
    (dict(scales=ctypes.c_void_p(20)), binding.ERR_ALIGN), (dict(num_tokens=0, dst=None), binding.OK)])
def test_read_refusals(over, code):
    assert _read(**over) == code


@pytest.mark.parametrize("over, code", [
    (dict(n_q=30), binding.ERR_SHAPE), (dict(head_dim=192), binding.ERR_SHAPE), (dict(block_size=8), binding.ERR_SHAPE),
    (dict(scale_stride=12, n_kv=16), binding.ERR_SHAPE), (dict(n_q=129 * 8), binding.ERR_UNSUPPORTED),
    (dict(sm_scale=float("nan")), binding.ERR_SCALE), (dict(query=None), binding.ERR_NULL), (dict(key_scales=None), binding.ERR_NULL),
    (dict(workspace=None), binding.ERR_NULL), (dict(value_scales=ctypes.c_void_p(8)), binding.ERR_ALIGN),
    (dict(out=ctypes.c_void_p(8)), binding.ERR_ALIGN), (dict(workspace_bytes=64), binding.ERR_WORKSPACE),
    (dict(num_seqs=0, query=None), binding.OK), (dict(num_seqs=0, scale_stride=3), binding.ERR_SHAPE)])
def test_decode_refusals(over, code):
    assert _decode(**over) == code


@pytest.mark.parametrize("over, code", [
    (dict(qmax=0), binding.ERR_SHAPE), (dict(rows=-1), binding.ERR_SHAPE), (dict(max_blocks_per_seq=0), binding.ERR_SHAPE),
    (dict(head_dim=96), binding.ERR_SHAPE), (dict(block_size=8), binding.ERR_SHAPE), (dict(qsl=None), binding.ERR_NULL),
    (dict(workspace=None), binding.ERR_NULL), (dict(qmax=64, workspace=None, workspace_bytes=0, value_scales=None), binding.ERR_NULL),
    (dict(qsl=ctypes.c_void_p(18)), binding.ERR_ALIGN), (dict(workspace_bytes=64), binding.ERR_WORKSPACE),
    (dict(n_q=129 * 8), binding.ERR_UNSUPPORTED), (dict(num_seqs=1 << 20, n_q=128 * 8, qmax=1 << 12), binding.ERR_UNSUPPORTED),
    (dict(sm_scale=float("inf")), binding.ERR_SCALE), (dict(num_seqs=0, query=None), binding.OK), (dict(rows=0, query=None), binding.OK)])
def test_multi_refusals(over, code):
    assert _multi(**over) == code


@pytest.mark.parametrize("over, code", [
    (dict(dtype=2), binding.ERR_DTYPE), (dict(num_tokens=-1), binding.ERR_SHAPE), (dict(n_q=0), binding.ERR_SHAPE), (dict(n_k=-1), binding.ERR_SHAPE),
    (dict(head_dim=132), binding.ERR_SHAPE), (dict(head_dim=264), binding.ERR_SHAPE), (dict(rot_dim=136), binding.ERR_SHAPE),
    (dict(rot_dim=24), binding.ERR_SHAPE), (dict(rot_dim=0), binding.ERR_SHAPE), (dict(query_stride=4088), binding.ERR_SHAPE),
    (dict(key_out_stride=1000), binding.ERR_SHAPE), (dict(magnitude=float("inf")), binding.ERR_SCALE),
    (dict(n_q=1 << 14, query_stride=1 << 21, query_out_stride=1 << 21), binding.ERR_SHAPE),
    (dict(key=None), binding.ERR_NULL), (dict(positions=None), binding.ERR_NULL), (dict(frequencies=None), binding.ERR_NULL),
    (dict(query=ctypes.c_void_p(8)), binding.ERR_ALIGN), (dict(key_stride=1028), binding.ERR_ALIGN),
    (dict(positions=ctypes.c_void_p(20)), binding.ERR_ALIGN), (dict(num_tokens=0, query=None), binding.OK)])
def test_rotary_refusals(over, code):
    assert _rotary(**over) == code


def test_workspace_sizes():
    assert kv.reshape_and_cache_block_scaled_workspace_size(512, 100, 16) == 0
    assert kv.reshape_and_cache_block_scaled_workspace_size(513, 100, 16) == 4 * (1600 + 100 + 2)
    assert kv.reshape_and_cache_block_scaled_workspace_size(513, 1 << 27, 16) == (1 << 33) + (1 << 29) + 8
    assert kv.reshape_and_cache_block_scaled_workspace_size(-1, 100, 16) == 0
    assert kv.paged_attention_block_scaled_workspace_size(4, 32, 8, 128, 1, 16, 16) == 0
    assert kv.paged_attention_block_scaled_workspace_size(4, 32, 8, 128, 1, 256, 16) > 0


def test_binding_checks():
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 16, 2, 64, dtype=torch.uint8)
    scales = kv.block_scales(2, 2, device="cpu")
    slots = torch.arange(4)
    ok = dict(key=k, value=k, key_cache=cache, value_cache=cache, key_scales=scales, value_scales=scales, slot_mapping=slots)
    assert scales.shape == (2, 4)
    for err, over in [(TypeError, dict(key=k.half(), value=k.half())), (TypeError, dict(value=k.float())),
                      (ValueError, dict(key=k[:3])), (ValueError, dict(key=k.transpose(1, 2), value=k.transpose(1, 2))),
                      (ValueError, dict(key_cache=cache[:, :, :1])), (ValueError, dict(key_scales=scales[:, :2])),
                      (ValueError, dict(key_scales=scales[:1])), (ValueError, dict(value_scales=scales.double())),
                      (ValueError, dict(value_scales=kv.block_scales(2, 5, device="cpu"))),
                      (ValueError, dict(slot_mapping=slots.int())), (ValueError, dict(slot_mapping=slots[:2])), (ValueError, {})]:
        with pytest.raises(err):  # (the last: not on a GPU)
            kv.reshape_and_cache_block_scaled(**{**ok, **over})
    with pytest.raises(TypeError):
        kv.dequant_block_scaled(cache, scales, slots, torch.float16)
    with pytest.raises(ValueError):
        kv.dequant_block_scaled(cache, scales[:, :3], slots)
    q, bt, lens = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for over in [dict(query=q.float()), dict(query=q[:, :, :32]), dict(block_tables=bt[:1]), dict(seq_lens=lens.long()),
                 dict(key_scales=scales[:, :2]), dict(out=q[:1]), {}]:
        with pytest.raises(ValueError):
            kv.paged_decode_attention_block_scaled(**{**dict(query=q, key_cache=cache, value_cache=cache, key_scales=scales,
                                                             value_scales=scales, block_tables=bt, seq_lens=lens), **over})
    pos, (freq, mag) = torch.arange(2), kv.rotary_frequencies(64, device="cpu")
    assert mag == 1.0 and freq.dtype == torch.float64
    for err, over in [(TypeError, dict(query=q.half())), (TypeError, dict(key=q.float())), (ValueError, dict(key=q[:1])),
                      (ValueError, dict(positions=pos.int())), (ValueError, dict(positions=pos[:1])), (ValueError, dict(frequencies=freq.float())),
                      (ValueError, dict(query_out=q[:, :2])), (ValueError, dict(key=None, key_out=q)), (ValueError, {})]:
        with pytest.raises(err):
            kv.rotary_embedding(**{**dict(query=q, key=q, positions=pos, frequencies=freq), **over})


def test_frequency_refusals():
    for kw in (dict(rot_dim=7), dict(rot_dim=0), dict(base=0.0), dict(factor=-1.0), dict(scaling="other"),
               dict(scaling="parts"), dict(scaling="parts", original_len=64, low_turns=4.0, high_turns=4.0)):
        with pytest.raises(ValueError):
            kv.rotary_frequencies(**{**dict(rot_dim=64, device="cpu"), **kw})
