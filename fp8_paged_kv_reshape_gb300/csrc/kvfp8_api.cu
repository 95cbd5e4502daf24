// The kvfp8 C ABI: host-side validation, then one enqueue on the caller's stream.
// Declarations, argument meanings and error behaviour: include/kvfp8.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/kvfp8.h"
#include "kvfp8_internal.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool dtype_ok(kvfp8_dtype t) { return t == KVFP8_BF16 || t == KVFP8_F32; }

kvfp8_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return KVFP8_OK;
    if (e == cudaErrorNotSupported) return KVFP8_ERR_UNSUPPORTED;
    return KVFP8_ERR_CUDA;
}

bool cache_dtype_ok(kvfp8_cache_dtype t) { return t == KVFP8_CACHE_E4M3 || t == KVFP8_CACHE_BF16; }

bool block_size_ok_for_decode(int32_t bs) {
    return bs == 8 || bs == 16 || bs == 32 || bs == 64 || bs == 128 || bs == 256;
}

// the 4-bit cache's shape rules, shared by its entry points
kvfp8_status check_fp4_cache(int32_t num_blocks, int32_t block_size, int32_t n_kv, int32_t head_dim) {
    if (num_blocks < 1 || n_kv < 1 || !block_size_ok_for_decode(block_size) ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return KVFP8_ERR_SHAPE;
    // tensor-map extents and row indices are 32 bits
    if (static_cast<int64_t>(num_blocks) * block_size > 0x7FFFFFFFLL ||
        static_cast<int64_t>(num_blocks) * n_kv > 0x7FFFFFFFLL || n_kv > (1 << 20))
        return KVFP8_ERR_SHAPE;
    return KVFP8_OK;
}

// the shape rules of the FP8 cache with block scales, shared by its entry points
kvfp8_status check_block_cache(int32_t num_blocks, int32_t block_size, int32_t n_kv, int32_t head_dim,
                               int32_t scale_stride) {
    if (num_blocks < 1 || n_kv < 1 || !block_size_ok_for_decode(block_size) || block_size < 16 ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256) || scale_stride < n_kv || scale_stride % 4 != 0)
        return KVFP8_ERR_SHAPE;
    if (static_cast<int64_t>(num_blocks) * block_size > 0x7FFFFFFFLL || static_cast<int64_t>(n_kv) * head_dim > (1 << 20))
        return KVFP8_ERR_SHAPE;
    return KVFP8_OK;
}

// tables whose width in tokens, rounded up to a tile of keys, is an int32 (the attention over block scales)
bool table_width_ok(int32_t max_blocks_per_seq, int32_t block_size) {
    return static_cast<int64_t>(max_blocks_per_seq) * block_size <= 0x7FFFFFFFLL - 127;
}

int32_t log2_of(int32_t x) {  // of a power of two
    int32_t n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

// the cache list of the page calls: KVFP8_OK with *out filled, or what is wrong with it
kvfp8_status make_cache_list(void *const *caches, const int64_t *block_bytes, int32_t num_caches,
                             int32_t num_blocks, kvfp8::CacheList *out) {
    if (num_caches < 1 || num_caches > KVFP8_MAX_CACHES || num_blocks < 1 || num_blocks > (1 << 30))
        return KVFP8_ERR_SHAPE;
    if (!caches || !block_bytes) return KVFP8_ERR_NULL;
    for (int32_t c = 0; c < num_caches; ++c) {
        if (block_bytes[c] < 1 || block_bytes[c] > (int64_t{1} << 40)) return KVFP8_ERR_SHAPE;
        if (!caches[c]) return KVFP8_ERR_NULL;
        if (!aligned16(caches[c]) || block_bytes[c] % 16 != 0) return KVFP8_ERR_ALIGN;
        out->ptr[c] = static_cast<uint8_t *>(caches[c]);
        out->block_bytes[c] = block_bytes[c];
    }
    out->count = num_caches;
    return KVFP8_OK;
}

}  // namespace

namespace kvfp8 {

kvfp8_status validate_decode(const void *out, const void *query, const uint8_t *key_cache,
                             const uint8_t *value_cache, const int32_t *block_tables,
                             int32_t max_blocks_per_seq, const int32_t *seq_lens,
                             int32_t num_seqs, int32_t n_q, int32_t n_kv, int32_t head_dim,
                             int32_t block_size, int32_t num_blocks, float sm_scale,
                             int scale_dtype, bool *nothing_to_do) {
    *nothing_to_do = false;
    if (!dtype_ok(static_cast<kvfp8_dtype>(scale_dtype))) return KVFP8_ERR_DTYPE;
    if (num_seqs < 0 || n_q < 1 || n_kv < 1 || n_q % n_kv != 0 || num_blocks < 1 ||
        max_blocks_per_seq < 1)
        return KVFP8_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return KVFP8_ERR_SHAPE;
    if (!block_size_ok_for_decode(block_size)) return KVFP8_ERR_SHAPE;
    if (n_q / n_kv > 128) return KVFP8_ERR_UNSUPPORTED;  // past the tensor-core kernel's rows
    if (static_cast<int64_t>(num_blocks) * block_size > 0x7FFFFFFFLL ||
        static_cast<int64_t>(max_blocks_per_seq) * block_size > 0x7FFFFFFFLL)
        return KVFP8_ERR_SHAPE;
    if (std::isnan(sm_scale) || std::isinf(sm_scale)) return KVFP8_ERR_SCALE;
    if (num_seqs == 0) {
        *nothing_to_do = true;
        return KVFP8_OK;
    }
    if (!out || !query || !key_cache || !value_cache || !block_tables || !seq_lens)
        return KVFP8_ERR_NULL;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) ||
        !aligned16(value_cache) || !aligned(block_tables, 4) || !aligned(seq_lens, 4))
        return KVFP8_ERR_ALIGN;
    return KVFP8_OK;
}

kvfp8_status launch_decode_validated(void *out, const void *query, const uint8_t *key_cache,
                                     const uint8_t *value_cache, const int32_t *block_tables,
                                     int32_t max_blocks_per_seq, const int32_t *seq_lens,
                                     int32_t num_seqs, int32_t n_q, int32_t n_kv,
                                     int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                     float sm_scale, const void *k_scale, const void *v_scale,
                                     int scale_dtype, void *workspace, uint32_t *status,
                                     kvfp8_stream_t stream) {
    DecodeArgs d;
    d.out = out;
    d.query = query;
    d.key_cache = key_cache;
    d.value_cache = value_cache;
    d.block_tables = block_tables;
    d.max_blocks_per_seq = max_blocks_per_seq;
    d.seq_lens = seq_lens;
    d.num_seqs = num_seqs;
    d.n_q = n_q;
    d.n_kv = n_kv;
    d.head_dim = head_dim;
    d.block_size = block_size;
    d.num_blocks = num_blocks;
    d.sm_scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt(static_cast<float>(head_dim));
    d.k_scale = k_scale;
    d.v_scale = v_scale;
    d.scale_dtype = scale_dtype;
    d.workspace = workspace;
    d.status = status;
    d.qsl = nullptr;
    d.qmax = 1;
    d.qrows = num_seqs;
    d.k_bf16 = 0;
    d.v_bf16 = 0;
    return from_cuda(launch_paged_decode(d, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace kvfp8

extern "C" {

kvfp8_status kvfp8_reshape_and_cache(const void *key, const void *value, kvfp8_dtype src_dtype,
                                     int64_t key_stride, int64_t value_stride, int64_t num_tokens,
                                     uint8_t *key_cache, uint8_t *value_cache, int32_t num_blocks,
                                     int32_t block_size, int32_t n_kv, int32_t head_dim,
                                     const int64_t *slot_mapping, const void *k_scale,
                                     const void *v_scale, kvfp8_dtype scale_dtype,
                                     uint32_t *status, kvfp8_stream_t stream) {
    if (!dtype_ok(src_dtype) || !dtype_ok(scale_dtype)) return KVFP8_ERR_DTYPE;
    if (num_tokens < 0 || num_blocks < 1 || block_size < 1 || block_size > 1024 || n_kv < 1 ||
        head_dim < 1)
        return KVFP8_ERR_SHAPE;
    const int64_t row = static_cast<int64_t>(n_kv) * head_dim;
    if (row % 8 != 0 || row > (1 << 20) || key_stride < row || value_stride < row)
        return KVFP8_ERR_SHAPE;
    if (num_tokens == 0) return KVFP8_OK;
    if (!key || !value || !key_cache || !value_cache || !slot_mapping) return KVFP8_ERR_NULL;
    const int64_t esz = src_dtype == KVFP8_F32 ? 4 : 2;
    if (!aligned16(key) || !aligned16(value) || !aligned16(key_cache) || !aligned16(value_cache) ||
        (key_stride * esz) % 16 != 0 || (value_stride * esz) % 16 != 0 || !aligned(slot_mapping, 8))
        return KVFP8_ERR_ALIGN;
    kvfp8::ReshapeArgs a;
    a.key = key;
    a.value = value;
    a.src_dtype = src_dtype;
    a.key_stride = key_stride;
    a.value_stride = value_stride;
    a.num_tokens = num_tokens;
    a.key_cache = key_cache;
    a.value_cache = value_cache;
    a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
    a.row_elems = static_cast<int32_t>(row);
    a.slot_mapping = slot_mapping;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.scale_dtype = scale_dtype;
    a.status = status;
    a.positions = nullptr;
    a.cos_sin = nullptr;
    a.max_pos = 0;
    a.rot = 0;
    a.neox = 0;
    a.head_dim = head_dim;
    a.k_bf16 = 0;
    a.v_bf16 = 0;
    return from_cuda(kvfp8::launch_reshape_and_cache(a, reinterpret_cast<cudaStream_t>(stream)));
}

kvfp8_status kvfp8_rope_reshape_and_cache(
    const void *key, const void *value, kvfp8_dtype src_dtype, int64_t key_stride,
    int64_t value_stride, int64_t num_tokens, uint8_t *key_cache, uint8_t *value_cache,
    int32_t num_blocks, int32_t block_size, int32_t n_kv, int32_t head_dim,
    const int64_t *slot_mapping, const int64_t *positions, const float *cos_sin_cache,
    int64_t max_position, int32_t rot_dim, int32_t is_neox, const void *k_scale,
    const void *v_scale, kvfp8_dtype scale_dtype, uint32_t *status, kvfp8_stream_t stream) {
    if (!dtype_ok(src_dtype) || !dtype_ok(scale_dtype)) return KVFP8_ERR_DTYPE;
    if (num_tokens < 0 || num_blocks < 1 || block_size < 1 || block_size > 1024 || n_kv < 1 ||
        max_position < 1)
        return KVFP8_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return KVFP8_ERR_SHAPE;
    if (rot_dim < 16 || rot_dim > head_dim || (rot_dim & (rot_dim - 1)) != 0) return KVFP8_ERR_SHAPE;
    const int64_t row = static_cast<int64_t>(n_kv) * head_dim;
    if (key_stride < row || value_stride < row) return KVFP8_ERR_SHAPE;
    if (row > 2048) return KVFP8_ERR_UNSUPPORTED;
    if (num_tokens == 0) return KVFP8_OK;
    if (!key || !value || !key_cache || !value_cache || !slot_mapping || !positions ||
        !cos_sin_cache)
        return KVFP8_ERR_NULL;
    const int64_t esz = src_dtype == KVFP8_F32 ? 4 : 2;
    if (!aligned16(key) || !aligned16(value) || !aligned16(key_cache) || !aligned16(value_cache) ||
        (key_stride * esz) % 16 != 0 || (value_stride * esz) % 16 != 0 ||
        !aligned(slot_mapping, 8) || !aligned(positions, 8) || !aligned16(cos_sin_cache))
        return KVFP8_ERR_ALIGN;
    kvfp8::ReshapeArgs a;
    a.key = key;
    a.value = value;
    a.src_dtype = src_dtype;
    a.key_stride = key_stride;
    a.value_stride = value_stride;
    a.num_tokens = num_tokens;
    a.key_cache = key_cache;
    a.value_cache = value_cache;
    a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
    a.row_elems = static_cast<int32_t>(row);
    a.slot_mapping = slot_mapping;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.scale_dtype = scale_dtype;
    a.status = status;
    a.positions = positions;
    a.cos_sin = cos_sin_cache;
    a.max_pos = max_position;
    a.rot = rot_dim;
    a.neox = is_neox ? 1 : 0;
    a.head_dim = head_dim;
    a.k_bf16 = 0;
    a.v_bf16 = 0;
    return from_cuda(kvfp8::launch_reshape_and_cache(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kvfp8_paged_decode_workspace_size(int32_t num_seqs, int32_t n_q, int32_t head_dim) {
    if (num_seqs < 0 || n_q < 1 || head_dim < 1) return 0;
    return kvfp8::decode_workspace_layout(num_seqs, n_q, head_dim).total;
}

kvfp8_status kvfp8_paged_decode_attention(void *out, const void *query, const uint8_t *key_cache,
                                          const uint8_t *value_cache, const int32_t *block_tables,
                                          int32_t max_blocks_per_seq, const int32_t *seq_lens,
                                          int32_t num_seqs, int32_t n_q, int32_t n_kv,
                                          int32_t head_dim, int32_t block_size,
                                          int32_t num_blocks, float sm_scale,
                                          const void *k_scale, const void *v_scale,
                                          kvfp8_dtype scale_dtype, void *workspace,
                                          size_t workspace_bytes, uint32_t *status,
                                          kvfp8_stream_t stream) {
    bool nothing_to_do = false;
    const kvfp8_status v = kvfp8::validate_decode(
        out, query, key_cache, value_cache, block_tables, max_blocks_per_seq, seq_lens, num_seqs,
        n_q, n_kv, head_dim, block_size, num_blocks, sm_scale, scale_dtype, &nothing_to_do);
    if (v != KVFP8_OK || nothing_to_do) return v;
    if (!workspace) return KVFP8_ERR_NULL;
    if (!aligned16(workspace)) return KVFP8_ERR_ALIGN;
    if (workspace_bytes < kvfp8_paged_decode_workspace_size(num_seqs, n_q, head_dim))
        return KVFP8_ERR_WORKSPACE;
    return kvfp8::launch_decode_validated(out, query, key_cache, value_cache, block_tables,
                                          max_blocks_per_seq, seq_lens, num_seqs, n_q, n_kv,
                                          head_dim, block_size, num_blocks, sm_scale, k_scale,
                                          v_scale, scale_dtype, workspace, status, stream);
}

size_t kvfp8_paged_attention_multi_workspace_size(int32_t num_seqs, int32_t n_q, int32_t n_kv,
                                                  int32_t head_dim, int32_t max_query_len) {
    if (num_seqs < 0 || n_q < 1 || n_kv < 1 || n_q % n_kv != 0 || head_dim < 1 || max_query_len < 1)
        return 0;
    if (!kvfp8::multi_uses_decode_kernel(n_q, n_kv, head_dim, max_query_len)) return 0;
    return kvfp8::decode_workspace_layout(num_seqs, n_q * max_query_len, head_dim).total;
}

kvfp8_status kvfp8_paged_attention_multi(
    void *out, const void *query, const int32_t *query_start_loc, int32_t num_query_rows,
    int32_t max_query_len, const uint8_t *key_cache, const uint8_t *value_cache, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t num_seqs, int32_t n_q,
    int32_t n_kv, int32_t head_dim, int32_t block_size, int32_t num_blocks, float sm_scale,
    const void *k_scale, const void *v_scale, kvfp8_dtype scale_dtype, void *workspace,
    size_t workspace_bytes, uint32_t *status, kvfp8_stream_t stream) {
    if (!dtype_ok(scale_dtype)) return KVFP8_ERR_DTYPE;
    if (num_seqs < 0 || n_q < 1 || n_kv < 1 || n_q % n_kv != 0 || max_query_len < 1 ||
        num_query_rows < 0 || num_blocks < 1 || max_blocks_per_seq < 1)
        return KVFP8_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return KVFP8_ERR_SHAPE;
    if (!block_size_ok_for_decode(block_size)) return KVFP8_ERR_SHAPE;
    const bool split_kv = kvfp8::multi_uses_decode_kernel(n_q, n_kv, head_dim, max_query_len);
    if (!split_kv && !kvfp8::prefill_takes(n_q, n_kv, max_query_len, num_seqs)) return KVFP8_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(num_blocks) * block_size > 0x7FFFFFFFLL ||
        static_cast<int64_t>(max_blocks_per_seq) * block_size > 0x7FFFFFFFLL)
        return KVFP8_ERR_SHAPE;
    if (std::isnan(sm_scale) || std::isinf(sm_scale)) return KVFP8_ERR_SCALE;
    if (num_seqs == 0) return KVFP8_OK;
    if (!out || !query || !query_start_loc || !key_cache || !value_cache || !block_tables ||
        !seq_lens || (split_kv && !workspace))
        return KVFP8_ERR_NULL;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) ||
        !aligned16(value_cache) || !aligned(block_tables, 4) || !aligned(seq_lens, 4) ||
        !aligned(query_start_loc, 4) || (split_kv && !aligned16(workspace)))
        return KVFP8_ERR_ALIGN;
    if (workspace_bytes <
        kvfp8_paged_attention_multi_workspace_size(num_seqs, n_q, n_kv, head_dim, max_query_len))
        return KVFP8_ERR_WORKSPACE;
    kvfp8::DecodeArgs d;
    d.out = out;
    d.query = query;
    d.key_cache = key_cache;
    d.value_cache = value_cache;
    d.block_tables = block_tables;
    d.max_blocks_per_seq = max_blocks_per_seq;
    d.seq_lens = seq_lens;
    d.num_seqs = num_seqs;
    d.n_q = n_q;
    d.n_kv = n_kv;
    d.head_dim = head_dim;
    d.block_size = block_size;
    d.num_blocks = num_blocks;
    d.sm_scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt(static_cast<float>(head_dim));
    d.k_scale = k_scale;
    d.v_scale = v_scale;
    d.scale_dtype = scale_dtype;
    d.workspace = workspace;
    d.status = status;
    d.qsl = query_start_loc;
    d.qmax = max_query_len;
    d.qrows = num_query_rows;
    d.k_bf16 = 0;
    d.v_bf16 = 0;
    return from_cuda(kvfp8::launch_paged_decode(d, reinterpret_cast<cudaStream_t>(stream)));
}

kvfp8_status kvfp8_reshape_and_cache_mixed(
    const void *key, const void *value, kvfp8_dtype src_dtype, int64_t key_stride,
    int64_t value_stride, int64_t num_tokens, void *key_cache, kvfp8_cache_dtype k_cache_dtype,
    void *value_cache, kvfp8_cache_dtype v_cache_dtype, int32_t num_blocks, int32_t block_size,
    int32_t n_kv, int32_t head_dim, const int64_t *slot_mapping, const void *k_scale,
    const void *v_scale, kvfp8_dtype scale_dtype, uint32_t *status, kvfp8_stream_t stream) {
    if (!dtype_ok(src_dtype) || !dtype_ok(scale_dtype) || !cache_dtype_ok(k_cache_dtype) ||
        !cache_dtype_ok(v_cache_dtype))
        return KVFP8_ERR_DTYPE;
    if (num_tokens < 0 || num_blocks < 1 || block_size < 1 || block_size > 1024 || n_kv < 1 ||
        head_dim < 1)
        return KVFP8_ERR_SHAPE;
    const int64_t row = static_cast<int64_t>(n_kv) * head_dim;
    if (row % 8 != 0 || key_stride < row || value_stride < row) return KVFP8_ERR_SHAPE;
    if (row > 2048) return KVFP8_ERR_UNSUPPORTED;
    if (num_tokens == 0) return KVFP8_OK;
    if (!key || !value || !key_cache || !value_cache || !slot_mapping) return KVFP8_ERR_NULL;
    const int64_t esz = src_dtype == KVFP8_F32 ? 4 : 2;
    if (!aligned16(key) || !aligned16(value) || !aligned16(key_cache) || !aligned16(value_cache) ||
        (key_stride * esz) % 16 != 0 || (value_stride * esz) % 16 != 0 || !aligned(slot_mapping, 8))
        return KVFP8_ERR_ALIGN;
    kvfp8::ReshapeArgs a;
    a.key = key;
    a.value = value;
    a.src_dtype = src_dtype;
    a.key_stride = key_stride;
    a.value_stride = value_stride;
    a.num_tokens = num_tokens;
    a.key_cache = static_cast<uint8_t *>(key_cache);
    a.value_cache = static_cast<uint8_t *>(value_cache);
    a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
    a.row_elems = static_cast<int32_t>(row);
    a.slot_mapping = slot_mapping;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.scale_dtype = scale_dtype;
    a.status = status;
    a.positions = nullptr;
    a.cos_sin = nullptr;
    a.max_pos = 0;
    a.rot = 0;
    a.neox = 0;
    a.head_dim = head_dim;
    a.k_bf16 = k_cache_dtype == KVFP8_CACHE_BF16 ? 1 : 0;
    a.v_bf16 = v_cache_dtype == KVFP8_CACHE_BF16 ? 1 : 0;
    return from_cuda(kvfp8::launch_reshape_and_cache(a, reinterpret_cast<cudaStream_t>(stream)));
}

kvfp8_status kvfp8_paged_decode_attention_mixed(
    void *out, const void *query, const void *key_cache, kvfp8_cache_dtype k_cache_dtype,
    const void *value_cache, kvfp8_cache_dtype v_cache_dtype, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t num_seqs, int32_t n_q,
    int32_t n_kv, int32_t head_dim, int32_t block_size, int32_t num_blocks, float sm_scale,
    const void *k_scale, const void *v_scale, kvfp8_dtype scale_dtype, void *workspace,
    size_t workspace_bytes, uint32_t *status, kvfp8_stream_t stream) {
    if (!cache_dtype_ok(k_cache_dtype) || !cache_dtype_ok(v_cache_dtype)) return KVFP8_ERR_DTYPE;
    if (k_cache_dtype == KVFP8_CACHE_E4M3 && v_cache_dtype == KVFP8_CACHE_E4M3)
        return kvfp8_paged_decode_attention(
            out, query, static_cast<const uint8_t *>(key_cache),
            static_cast<const uint8_t *>(value_cache), block_tables, max_blocks_per_seq, seq_lens,
            num_seqs, n_q, n_kv, head_dim, block_size, num_blocks, sm_scale, k_scale, v_scale,
            scale_dtype, workspace, workspace_bytes, status, stream);
    if (!dtype_ok(scale_dtype)) return KVFP8_ERR_DTYPE;
    if (num_seqs < 0 || n_q < 1 || n_kv < 1 || n_q % n_kv != 0 || num_blocks < 1 ||
        max_blocks_per_seq < 1)
        return KVFP8_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return KVFP8_ERR_SHAPE;
    if (!block_size_ok_for_decode(block_size)) return KVFP8_ERR_SHAPE;
    if (static_cast<int64_t>(num_blocks) * block_size > 0x7FFFFFFFLL ||
        static_cast<int64_t>(max_blocks_per_seq) * block_size > 0x7FFFFFFFLL)
        return KVFP8_ERR_SHAPE;
    if (k_cache_dtype == v_cache_dtype ||
        !kvfp8::mixed_uses_decode_kernel(n_q, n_kv, head_dim, 1))
        return KVFP8_ERR_UNSUPPORTED;
    if (std::isnan(sm_scale) || std::isinf(sm_scale)) return KVFP8_ERR_SCALE;
    if (num_seqs == 0) return KVFP8_OK;
    if (!out || !query || !key_cache || !value_cache || !block_tables || !seq_lens || !workspace)
        return KVFP8_ERR_NULL;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) ||
        !aligned16(value_cache) || !aligned(block_tables, 4) || !aligned(seq_lens, 4) ||
        !aligned16(workspace))
        return KVFP8_ERR_ALIGN;
    if (workspace_bytes < kvfp8_paged_decode_workspace_size(num_seqs, n_q, head_dim))
        return KVFP8_ERR_WORKSPACE;
    kvfp8::DecodeArgs d;
    d.out = out;
    d.query = query;
    d.key_cache = static_cast<const uint8_t *>(key_cache);
    d.value_cache = static_cast<const uint8_t *>(value_cache);
    d.block_tables = block_tables;
    d.max_blocks_per_seq = max_blocks_per_seq;
    d.seq_lens = seq_lens;
    d.num_seqs = num_seqs;
    d.n_q = n_q;
    d.n_kv = n_kv;
    d.head_dim = head_dim;
    d.block_size = block_size;
    d.num_blocks = num_blocks;
    d.sm_scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt(static_cast<float>(head_dim));
    d.k_scale = k_scale;
    d.v_scale = v_scale;
    d.scale_dtype = scale_dtype;
    d.workspace = workspace;
    d.status = status;
    d.qsl = nullptr;
    d.qmax = 1;
    d.qrows = num_seqs;
    d.k_bf16 = k_cache_dtype == KVFP8_CACHE_BF16 ? 1 : 0;
    d.v_bf16 = v_cache_dtype == KVFP8_CACHE_BF16 ? 1 : 0;
    return from_cuda(kvfp8::launch_paged_decode(d, reinterpret_cast<cudaStream_t>(stream)));
}

kvfp8_status kvfp8_paged_attention_multi_mixed(
    void *out, const void *query, const int32_t *query_start_loc, int32_t num_query_rows,
    int32_t max_query_len, const void *key_cache, kvfp8_cache_dtype k_cache_dtype,
    const void *value_cache, kvfp8_cache_dtype v_cache_dtype, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t num_seqs, int32_t n_q,
    int32_t n_kv, int32_t head_dim, int32_t block_size, int32_t num_blocks, float sm_scale,
    const void *k_scale, const void *v_scale, kvfp8_dtype scale_dtype, void *workspace,
    size_t workspace_bytes, uint32_t *status, kvfp8_stream_t stream) {
    if (!cache_dtype_ok(k_cache_dtype) || !cache_dtype_ok(v_cache_dtype)) return KVFP8_ERR_DTYPE;
    if (k_cache_dtype == KVFP8_CACHE_E4M3 && v_cache_dtype == KVFP8_CACHE_E4M3)
        return kvfp8_paged_attention_multi(
            out, query, query_start_loc, num_query_rows, max_query_len,
            static_cast<const uint8_t *>(key_cache), static_cast<const uint8_t *>(value_cache),
            block_tables, max_blocks_per_seq, seq_lens, num_seqs, n_q, n_kv, head_dim, block_size,
            num_blocks, sm_scale, k_scale, v_scale, scale_dtype, workspace, workspace_bytes, status,
            stream);
    if (!dtype_ok(scale_dtype)) return KVFP8_ERR_DTYPE;
    if (num_seqs < 0 || n_q < 1 || n_kv < 1 || n_q % n_kv != 0 || max_query_len < 1 ||
        num_query_rows < 0 || num_blocks < 1 || max_blocks_per_seq < 1)
        return KVFP8_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return KVFP8_ERR_SHAPE;
    if (!block_size_ok_for_decode(block_size)) return KVFP8_ERR_SHAPE;
    if (static_cast<int64_t>(num_blocks) * block_size > 0x7FFFFFFFLL ||
        static_cast<int64_t>(max_blocks_per_seq) * block_size > 0x7FFFFFFFLL)
        return KVFP8_ERR_SHAPE;
    if (k_cache_dtype == v_cache_dtype ||
        !kvfp8::mixed_uses_decode_kernel(n_q, n_kv, head_dim, max_query_len))
        return KVFP8_ERR_UNSUPPORTED;
    if (std::isnan(sm_scale) || std::isinf(sm_scale)) return KVFP8_ERR_SCALE;
    if (num_seqs == 0) return KVFP8_OK;
    if (!out || !query || !query_start_loc || !key_cache || !value_cache || !block_tables ||
        !seq_lens || !workspace)
        return KVFP8_ERR_NULL;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) ||
        !aligned16(value_cache) || !aligned(block_tables, 4) || !aligned(seq_lens, 4) ||
        !aligned(query_start_loc, 4) || !aligned16(workspace))
        return KVFP8_ERR_ALIGN;
    if (workspace_bytes <
        kvfp8_paged_attention_multi_workspace_size(num_seqs, n_q, n_kv, head_dim, max_query_len))
        return KVFP8_ERR_WORKSPACE;
    kvfp8::DecodeArgs d;
    d.out = out;
    d.query = query;
    d.key_cache = static_cast<const uint8_t *>(key_cache);
    d.value_cache = static_cast<const uint8_t *>(value_cache);
    d.block_tables = block_tables;
    d.max_blocks_per_seq = max_blocks_per_seq;
    d.seq_lens = seq_lens;
    d.num_seqs = num_seqs;
    d.n_q = n_q;
    d.n_kv = n_kv;
    d.head_dim = head_dim;
    d.block_size = block_size;
    d.num_blocks = num_blocks;
    d.sm_scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt(static_cast<float>(head_dim));
    d.k_scale = k_scale;
    d.v_scale = v_scale;
    d.scale_dtype = scale_dtype;
    d.workspace = workspace;
    d.status = status;
    d.qsl = query_start_loc;
    d.qmax = max_query_len;
    d.qrows = num_query_rows;
    d.k_bf16 = k_cache_dtype == KVFP8_CACHE_BF16 ? 1 : 0;
    d.v_bf16 = v_cache_dtype == KVFP8_CACHE_BF16 ? 1 : 0;
    return from_cuda(kvfp8::launch_paged_decode(d, reinterpret_cast<cudaStream_t>(stream)));
}

kvfp8_status kvfp8_dequant(void *dst, kvfp8_dtype dst_dtype, const uint8_t *src, int64_t n,
                           const void *scale, kvfp8_dtype scale_dtype, kvfp8_stream_t stream) {
    if (!dtype_ok(dst_dtype) || !dtype_ok(scale_dtype)) return KVFP8_ERR_DTYPE;
    if (n < 0) return KVFP8_ERR_SHAPE;
    if (n == 0) return KVFP8_OK;
    if (!dst || !src) return KVFP8_ERR_NULL;
    if (!aligned16(dst) || !aligned16(src)) return KVFP8_ERR_ALIGN;
    return from_cuda(kvfp8::launch_dequant(dst, dst_dtype, src, n, scale, scale_dtype,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

kvfp8_status kvfp8_reshape_and_cache_fp4(
    const void *key, const void *value, kvfp8_dtype src_dtype, int64_t key_stride,
    int64_t value_stride, int64_t num_tokens, uint8_t *key_cache, uint8_t *value_cache,
    uint8_t *key_scales, uint8_t *value_scales, int32_t num_blocks, int32_t block_size,
    int32_t n_kv, int32_t head_dim, const int64_t *slot_mapping, const void *k_scale,
    const void *v_scale, kvfp8_dtype scale_dtype, uint32_t *status, kvfp8_stream_t stream) {
    if (!dtype_ok(src_dtype) || !dtype_ok(scale_dtype)) return KVFP8_ERR_DTYPE;
    if (num_tokens < 0) return KVFP8_ERR_SHAPE;
    const kvfp8_status sh = check_fp4_cache(num_blocks, block_size, n_kv, head_dim);
    if (sh != KVFP8_OK) return sh;
    const int64_t row = static_cast<int64_t>(n_kv) * head_dim;
    if (row > (1 << 20) || key_stride < row || value_stride < row) return KVFP8_ERR_SHAPE;
    if (num_tokens == 0) return KVFP8_OK;
    if (!key || !value || !key_cache || !value_cache || !key_scales || !value_scales ||
        !slot_mapping)
        return KVFP8_ERR_NULL;
    const int64_t esz = src_dtype == KVFP8_F32 ? 4 : 2;
    if (!aligned16(key) || !aligned16(value) || !aligned16(key_cache) || !aligned16(value_cache) ||
        !aligned16(key_scales) || !aligned16(value_scales) || (key_stride * esz) % 16 != 0 ||
        (value_stride * esz) % 16 != 0 || !aligned(slot_mapping, 8))
        return KVFP8_ERR_ALIGN;
    kvfp8::Fp4WriteArgs a;
    a.src[0] = key;
    a.src[1] = value;
    a.stride[0] = key_stride;
    a.stride[1] = value_stride;
    a.codes[0] = key_cache;
    a.codes[1] = value_cache;
    a.scales[0] = key_scales;
    a.scales[1] = value_scales;
    a.scale[0] = k_scale;
    a.scale[1] = v_scale;
    a.src_dtype = src_dtype;
    a.scale_dtype = scale_dtype;
    a.num_tokens = num_tokens;
    a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
    a.block_size = block_size;
    a.n_kv = n_kv;
    a.head_dim = head_dim;
    a.slot_mapping = slot_mapping;
    a.status = status;
    return from_cuda(kvfp8::launch_reshape_and_cache_fp4(a, reinterpret_cast<cudaStream_t>(stream)));
}

kvfp8_status kvfp8_dequant_fp4(void *dst, kvfp8_dtype dst_dtype, const uint8_t *codes,
                               const uint8_t *scales, int32_t num_blocks, int32_t block_size,
                               int32_t n_kv, int32_t head_dim, const int64_t *slot_mapping,
                               int64_t num_tokens, const void *scale, kvfp8_dtype scale_dtype,
                               uint32_t *status, kvfp8_stream_t stream) {
    if (!dtype_ok(dst_dtype) || !dtype_ok(scale_dtype)) return KVFP8_ERR_DTYPE;
    if (num_tokens < 0) return KVFP8_ERR_SHAPE;
    const kvfp8_status sh = check_fp4_cache(num_blocks, block_size, n_kv, head_dim);
    if (sh != KVFP8_OK) return sh;
    if (static_cast<int64_t>(n_kv) * head_dim > (1 << 20)) return KVFP8_ERR_SHAPE;
    if (num_tokens == 0) return KVFP8_OK;
    if (!dst || !codes || !scales || !slot_mapping) return KVFP8_ERR_NULL;
    if (!aligned16(dst) || !aligned16(codes) || !aligned16(scales) || !aligned(slot_mapping, 8))
        return KVFP8_ERR_ALIGN;
    kvfp8::Fp4ReadArgs a;
    a.dst = dst;
    a.dst_dtype = dst_dtype;
    a.scale_dtype = scale_dtype;
    a.codes = codes;
    a.scales = scales;
    a.scale = scale;
    a.num_tokens = num_tokens;
    a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
    a.block_size = block_size;
    a.n_kv = n_kv;
    a.head_dim = head_dim;
    a.slot_mapping = slot_mapping;
    a.status = status;
    return from_cuda(kvfp8::launch_dequant_fp4(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kvfp8_paged_attention_fp4_workspace_size(int32_t num_seqs, int32_t n_q, int32_t n_kv,
                                                int32_t head_dim, int32_t max_query_len,
                                                int32_t max_blocks_per_seq, int32_t block_size) {
    if (num_seqs < 1 || n_q < 1 || n_kv < 1 || n_q % n_kv != 0 || max_query_len < 1 || max_blocks_per_seq < 1 ||
        block_size < 1)
        return 0;
    if (!kvfp8::multi_uses_decode_kernel(n_q, n_kv, head_dim, max_query_len))
        return kvfp8::fp4_prefill_workspace_size(num_seqs, n_q, n_kv, head_dim, max_query_len,
                                                 static_cast<int64_t>(max_blocks_per_seq) * block_size);
    if (kvfp8::decode_takes_sequences_whole(max_blocks_per_seq, block_size)) return 0;
    return kvfp8_paged_attention_multi_workspace_size(num_seqs, n_q, n_kv, head_dim, max_query_len);
}

kvfp8_status kvfp8_paged_decode_attention_fp4(
    void *out, const void *query, const uint8_t *key_cache, const uint8_t *value_cache,
    const uint8_t *key_scales, const uint8_t *value_scales, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t num_seqs, int32_t n_q,
    int32_t n_kv, int32_t head_dim, int32_t block_size, int32_t num_blocks, float sm_scale,
    const void *k_scale, const void *v_scale, kvfp8_dtype scale_dtype, void *workspace,
    size_t workspace_bytes, uint32_t *status, kvfp8_stream_t stream) {
    bool nothing_to_do = false;
    const kvfp8_status v = kvfp8::validate_decode(
        out, query, key_cache, value_cache, block_tables, max_blocks_per_seq, seq_lens, num_seqs,
        n_q, n_kv, head_dim, block_size, num_blocks, sm_scale, scale_dtype, &nothing_to_do);
    if (v != KVFP8_OK || nothing_to_do) return v;
    const kvfp8_status sh = check_fp4_cache(num_blocks, block_size, n_kv, head_dim);
    if (sh != KVFP8_OK) return sh;
    const size_t need = kvfp8_paged_attention_fp4_workspace_size(num_seqs, n_q, n_kv, head_dim, 1,
                                                                 max_blocks_per_seq, block_size);
    if (!key_scales || !value_scales || (need > 0 && !workspace)) return KVFP8_ERR_NULL;
    if (!aligned16(key_scales) || !aligned16(value_scales) || (need > 0 && !aligned16(workspace)))
        return KVFP8_ERR_ALIGN;
    if (workspace_bytes < need) return KVFP8_ERR_WORKSPACE;
    kvfp8::DecodeArgs d;
    d.out = out;
    d.query = query;
    d.key_cache = key_cache;
    d.value_cache = value_cache;
    d.key_scales = key_scales;
    d.value_scales = value_scales;
    d.block_tables = block_tables;
    d.max_blocks_per_seq = max_blocks_per_seq;
    d.seq_lens = seq_lens;
    d.num_seqs = num_seqs;
    d.n_q = n_q;
    d.n_kv = n_kv;
    d.head_dim = head_dim;
    d.block_size = block_size;
    d.num_blocks = num_blocks;
    d.sm_scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt(static_cast<float>(head_dim));
    d.k_scale = k_scale;
    d.v_scale = v_scale;
    d.scale_dtype = scale_dtype;
    d.workspace = workspace;
    d.status = status;
    d.qsl = nullptr;
    d.qmax = 1;
    d.qrows = num_seqs;
    d.k_bf16 = 0;
    d.v_bf16 = 0;
    return from_cuda(kvfp8::launch_paged_decode_fp4(d, reinterpret_cast<cudaStream_t>(stream)));
}

kvfp8_status kvfp8_paged_attention_multi_fp4(
    void *out, const void *query, const int32_t *query_start_loc, int32_t num_query_rows,
    int32_t max_query_len, const uint8_t *key_cache, const uint8_t *value_cache,
    const uint8_t *key_scales, const uint8_t *value_scales, const int32_t *block_tables,
    int32_t max_blocks_per_seq, const int32_t *seq_lens, int32_t num_seqs, int32_t n_q,
    int32_t n_kv, int32_t head_dim, int32_t block_size, int32_t num_blocks, float sm_scale,
    const void *k_scale, const void *v_scale, kvfp8_dtype scale_dtype, void *workspace,
    size_t workspace_bytes, uint32_t *status, kvfp8_stream_t stream) {
    if (!dtype_ok(scale_dtype)) return KVFP8_ERR_DTYPE;
    if (num_seqs < 0 || n_q < 1 || n_kv < 1 || n_q % n_kv != 0 || max_query_len < 1 ||
        num_query_rows < 0 || max_blocks_per_seq < 1)
        return KVFP8_ERR_SHAPE;
    const kvfp8_status sh = check_fp4_cache(num_blocks, block_size, n_kv, head_dim);
    if (sh != KVFP8_OK) return sh;
    const bool split_kv = kvfp8::multi_uses_decode_kernel(n_q, n_kv, head_dim, max_query_len);
    if (!split_kv && !kvfp8::prefill_takes(n_q, n_kv, max_query_len, num_seqs)) return KVFP8_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_blocks_per_seq) * block_size > 0x7FFFFFFFLL) return KVFP8_ERR_SHAPE;
    if (std::isnan(sm_scale) || std::isinf(sm_scale)) return KVFP8_ERR_SCALE;
    if (num_seqs == 0 || num_query_rows == 0) return KVFP8_OK;
    const size_t need = kvfp8_paged_attention_fp4_workspace_size(
        num_seqs, n_q, n_kv, head_dim, max_query_len, max_blocks_per_seq, block_size);
    if (!out || !query || !query_start_loc || !key_cache || !value_cache || !key_scales ||
        !value_scales || !block_tables || !seq_lens || (need > 0 && !workspace))
        return KVFP8_ERR_NULL;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) ||
        !aligned16(value_cache) || !aligned16(key_scales) || !aligned16(value_scales) ||
        !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) ||
        (need > 0 && !aligned16(workspace)))
        return KVFP8_ERR_ALIGN;
    if (workspace_bytes < need) return KVFP8_ERR_WORKSPACE;
    kvfp8::DecodeArgs d;
    d.out = out;
    d.query = query;
    d.key_cache = key_cache;
    d.value_cache = value_cache;
    d.key_scales = key_scales;
    d.value_scales = value_scales;
    d.block_tables = block_tables;
    d.max_blocks_per_seq = max_blocks_per_seq;
    d.seq_lens = seq_lens;
    d.num_seqs = num_seqs;
    d.n_q = n_q;
    d.n_kv = n_kv;
    d.head_dim = head_dim;
    d.block_size = block_size;
    d.num_blocks = num_blocks;
    d.sm_scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt(static_cast<float>(head_dim));
    d.k_scale = k_scale;
    d.v_scale = v_scale;
    d.scale_dtype = scale_dtype;
    d.workspace = workspace;
    d.status = status;
    d.qsl = query_start_loc;
    d.qmax = max_query_len;
    d.qrows = num_query_rows;
    d.k_bf16 = 0;
    d.v_bf16 = 0;
    return from_cuda(kvfp8::launch_paged_decode_fp4(d, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kvfp8_reshape_and_cache_block_scaled_workspace_size(int64_t num_tokens, int32_t num_blocks,
                                                           int32_t block_size) {
    if (num_blocks < 1 || block_size < 1) return 0;
    return kvfp8::block_write_workspace_size(num_tokens, num_blocks, block_size);
}

kvfp8_status kvfp8_reshape_and_cache_block_scaled(
    const void *key, const void *value, kvfp8_dtype src_dtype, int64_t key_stride,
    int64_t value_stride, int64_t num_tokens, uint8_t *key_cache, uint8_t *value_cache,
    float *key_scales, float *value_scales, int32_t scale_stride, int32_t num_blocks,
    int32_t block_size, int32_t n_kv, int32_t head_dim, const int64_t *slot_mapping,
    void *workspace, size_t workspace_bytes, uint32_t *status, kvfp8_stream_t stream) {
    if (!dtype_ok(src_dtype)) return KVFP8_ERR_DTYPE;
    if (num_tokens < 0 || num_tokens > 0x7FFFFFFFLL) return KVFP8_ERR_SHAPE;
    const kvfp8_status sh = check_block_cache(num_blocks, block_size, n_kv, head_dim, scale_stride);
    if (sh != KVFP8_OK) return sh;
    const int64_t row = static_cast<int64_t>(n_kv) * head_dim;
    if (key_stride < row || value_stride < row) return KVFP8_ERR_SHAPE;
    if (num_tokens == 0) return KVFP8_OK;
    const size_t need = kvfp8_reshape_and_cache_block_scaled_workspace_size(num_tokens, num_blocks, block_size);
    if (!key || !value || !key_cache || !value_cache || !key_scales || !value_scales || !slot_mapping ||
        (need > 0 && !workspace))
        return KVFP8_ERR_NULL;
    const int64_t esz = src_dtype == KVFP8_F32 ? 4 : 2;
    if (!aligned16(key) || !aligned16(value) || !aligned16(key_cache) || !aligned16(value_cache) ||
        !aligned16(key_scales) || !aligned16(value_scales) || !aligned(slot_mapping, 8) ||
        (need > 0 && !aligned16(workspace)) || key_stride * esz % 16 != 0 || value_stride * esz % 16 != 0)
        return KVFP8_ERR_ALIGN;
    if (workspace_bytes < need) return KVFP8_ERR_WORKSPACE;
    kvfp8::BlockWriteArgs a;
    a.src[0] = key;
    a.src[1] = value;
    a.stride[0] = key_stride;
    a.stride[1] = value_stride;
    a.codes[0] = key_cache;
    a.codes[1] = value_cache;
    a.scales[0] = key_scales;
    a.scales[1] = value_scales;
    a.scale_stride = scale_stride;
    a.src_dtype = src_dtype;
    a.num_tokens = num_tokens;
    a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
    a.block_shift = log2_of(block_size);
    a.n_kv = n_kv;
    a.head_dim = head_dim;
    a.slot_mapping = slot_mapping;
    a.row_of = need > 0 ? static_cast<int32_t *>(workspace) : nullptr;
    a.status = status;
    return from_cuda(kvfp8::launch_reshape_and_cache_block_scaled(a, reinterpret_cast<cudaStream_t>(stream)));
}

kvfp8_status kvfp8_dequant_block_scaled(void *dst, kvfp8_dtype dst_dtype, const uint8_t *codes, const float *scales,
                                        int32_t scale_stride, int32_t num_blocks, int32_t block_size,
                                        int32_t n_kv, int32_t head_dim, const int64_t *slot_mapping,
                                        int64_t num_tokens, uint32_t *status, kvfp8_stream_t stream) {
    if (!dtype_ok(dst_dtype)) return KVFP8_ERR_DTYPE;
    if (num_tokens < 0) return KVFP8_ERR_SHAPE;
    const kvfp8_status sh = check_block_cache(num_blocks, block_size, n_kv, head_dim, scale_stride);
    if (sh != KVFP8_OK) return sh;
    if (num_tokens == 0) return KVFP8_OK;
    if (!dst || !codes || !scales || !slot_mapping) return KVFP8_ERR_NULL;
    if (!aligned16(dst) || !aligned16(codes) || !aligned16(scales) || !aligned(slot_mapping, 8))
        return KVFP8_ERR_ALIGN;
    kvfp8::BlockReadArgs a;
    a.dst = dst;
    a.dst_dtype = dst_dtype;
    a.codes = codes;
    a.scales = scales;
    a.scale_stride = scale_stride;
    a.num_tokens = num_tokens;
    a.num_slots = static_cast<int64_t>(num_blocks) * block_size;
    a.block_shift = log2_of(block_size);
    a.n_kv = n_kv;
    a.head_dim = head_dim;
    a.head_shift = log2_of(head_dim / 16);
    a.slot_mapping = slot_mapping;
    a.status = status;
    return from_cuda(kvfp8::launch_dequant_block_scaled(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kvfp8_paged_attention_block_scaled_workspace_size(int32_t num_seqs, int32_t n_q, int32_t n_kv,
                                                         int32_t head_dim, int32_t max_query_len,
                                                         int32_t max_blocks_per_seq, int32_t block_size) {
    if (num_seqs < 1 || n_q < 1 || n_kv < 1 || n_q % n_kv != 0 || max_query_len < 1 || max_blocks_per_seq < 1 ||
        block_size < 1)
        return 0;
    if (!kvfp8::multi_uses_decode_kernel(n_q, n_kv, head_dim, max_query_len))
        return kvfp8::block_scaled_prefill_workspace_size(num_seqs, n_q, n_kv, head_dim, max_query_len,
                                                          static_cast<int64_t>(max_blocks_per_seq) * block_size);
    if (kvfp8::decode_takes_sequences_whole(max_blocks_per_seq, block_size)) return 0;
    return kvfp8_paged_attention_multi_workspace_size(num_seqs, n_q, n_kv, head_dim, max_query_len);
}

kvfp8_status kvfp8_paged_decode_attention_block_scaled(
    void *out, const void *query, const uint8_t *key_cache, const uint8_t *value_cache,
    const float *key_scales, const float *value_scales, int32_t scale_stride,
    const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *seq_lens,
    int32_t num_seqs, int32_t n_q, int32_t n_kv, int32_t head_dim, int32_t block_size,
    int32_t num_blocks, float sm_scale, void *workspace, size_t workspace_bytes, uint32_t *status,
    kvfp8_stream_t stream) {
    bool nothing_to_do = false;
    const kvfp8_status v = kvfp8::validate_decode(
        out, query, key_cache, value_cache, block_tables, max_blocks_per_seq, seq_lens, num_seqs,
        n_q, n_kv, head_dim, block_size, num_blocks, sm_scale, KVFP8_F32, &nothing_to_do);
    if (v != KVFP8_OK) return v;
    const kvfp8_status sh = check_block_cache(num_blocks, block_size, n_kv, head_dim, scale_stride);
    if (sh != KVFP8_OK) return sh;
    if (!table_width_ok(max_blocks_per_seq, block_size)) return KVFP8_ERR_SHAPE;
    if (nothing_to_do) return KVFP8_OK;
    const size_t need = kvfp8_paged_attention_block_scaled_workspace_size(num_seqs, n_q, n_kv, head_dim, 1,
                                                                          max_blocks_per_seq, block_size);
    if (!key_scales || !value_scales || (need > 0 && !workspace)) return KVFP8_ERR_NULL;
    if (!aligned16(key_scales) || !aligned16(value_scales) || (need > 0 && !aligned16(workspace)))
        return KVFP8_ERR_ALIGN;
    if (workspace_bytes < need) return KVFP8_ERR_WORKSPACE;
    kvfp8::DecodeArgs d = {};
    d.out = out;
    d.query = query;
    d.key_cache = key_cache;
    d.value_cache = value_cache;
    d.key_block_scales = key_scales;
    d.value_block_scales = value_scales;
    d.block_scale_stride = scale_stride;
    d.block_tables = block_tables;
    d.max_blocks_per_seq = max_blocks_per_seq;
    d.seq_lens = seq_lens;
    d.num_seqs = num_seqs;
    d.n_q = n_q;
    d.n_kv = n_kv;
    d.head_dim = head_dim;
    d.block_size = block_size;
    d.num_blocks = num_blocks;
    d.sm_scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt(static_cast<float>(head_dim));
    d.scale_dtype = KVFP8_F32;
    d.workspace = workspace;
    d.status = status;
    d.qmax = 1;
    d.qrows = num_seqs;
    return from_cuda(kvfp8::launch_paged_decode_block_scaled(d, reinterpret_cast<cudaStream_t>(stream)));
}

kvfp8_status kvfp8_paged_attention_multi_block_scaled(
    void *out, const void *query, const int32_t *query_start_loc, int32_t num_query_rows,
    int32_t max_query_len, int32_t causal, const uint8_t *key_cache, const uint8_t *value_cache,
    const float *key_scales, const float *value_scales, int32_t scale_stride,
    const int32_t *block_tables, int32_t max_blocks_per_seq, const int32_t *seq_lens,
    int32_t num_seqs, int32_t n_q, int32_t n_kv, int32_t head_dim, int32_t block_size,
    int32_t num_blocks, float sm_scale, void *workspace, size_t workspace_bytes, uint32_t *status,
    kvfp8_stream_t stream) {
    if (num_seqs < 0 || n_q < 1 || n_kv < 1 || n_q % n_kv != 0 || max_query_len < 1 ||
        num_query_rows < 0 || max_blocks_per_seq < 1)
        return KVFP8_ERR_SHAPE;
    const kvfp8_status sh = check_block_cache(num_blocks, block_size, n_kv, head_dim, scale_stride);
    if (sh != KVFP8_OK) return sh;
    const bool split_kv = kvfp8::multi_uses_decode_kernel(n_q, n_kv, head_dim, max_query_len);
    if (!split_kv && !kvfp8::prefill_takes(n_q, n_kv, max_query_len, num_seqs)) return KVFP8_ERR_UNSUPPORTED;
    if (!table_width_ok(max_blocks_per_seq, block_size)) return KVFP8_ERR_SHAPE;
    if (std::isnan(sm_scale) || std::isinf(sm_scale)) return KVFP8_ERR_SCALE;
    if (num_seqs == 0 || num_query_rows == 0) return KVFP8_OK;
    const size_t need = kvfp8_paged_attention_block_scaled_workspace_size(
        num_seqs, n_q, n_kv, head_dim, max_query_len, max_blocks_per_seq, block_size);
    if (!out || !query || !query_start_loc || !key_cache || !value_cache || !key_scales ||
        !value_scales || !block_tables || !seq_lens || (need > 0 && !workspace))
        return KVFP8_ERR_NULL;
    if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) ||
        !aligned16(value_cache) || !aligned16(key_scales) || !aligned16(value_scales) ||
        !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) ||
        (need > 0 && !aligned16(workspace)))
        return KVFP8_ERR_ALIGN;
    if (workspace_bytes < need) return KVFP8_ERR_WORKSPACE;
    kvfp8::DecodeArgs d = {};
    d.out = out;
    d.query = query;
    d.key_cache = key_cache;
    d.value_cache = value_cache;
    d.key_block_scales = key_scales;
    d.value_block_scales = value_scales;
    d.block_scale_stride = scale_stride;
    d.causal = causal != 0;
    d.block_tables = block_tables;
    d.max_blocks_per_seq = max_blocks_per_seq;
    d.seq_lens = seq_lens;
    d.num_seqs = num_seqs;
    d.n_q = n_q;
    d.n_kv = n_kv;
    d.head_dim = head_dim;
    d.block_size = block_size;
    d.num_blocks = num_blocks;
    d.sm_scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt(static_cast<float>(head_dim));
    d.scale_dtype = KVFP8_F32;
    d.workspace = workspace;
    d.status = status;
    d.qsl = query_start_loc;
    d.qmax = max_query_len;
    d.qrows = num_query_rows;
    return from_cuda(kvfp8::launch_paged_decode_block_scaled(d, reinterpret_cast<cudaStream_t>(stream)));
}

kvfp8_status kvfp8_rotary_embedding(void *query_out, void *key_out, int64_t query_out_stride,
                                    int64_t key_out_stride, const void *query, const void *key,
                                    int64_t query_stride, int64_t key_stride, kvfp8_dtype dtype,
                                    int64_t num_tokens, int32_t n_q, int32_t n_k, int32_t head_dim,
                                    int32_t rot_dim, int32_t interleaved, int32_t transpose,
                                    const int64_t *positions, const double *frequencies,
                                    float magnitude, uint32_t *status, kvfp8_stream_t stream) {
    if (!dtype_ok(dtype)) return KVFP8_ERR_DTYPE;
    if (num_tokens < 0 || num_tokens > 0x7FFFFFFFLL || n_q < 1 || n_k < 0 || head_dim < 16 || head_dim > 256 ||
        head_dim % 8 != 0 || rot_dim < 16 || rot_dim > head_dim || rot_dim % 16 != 0 ||
        static_cast<int64_t>(n_q) * head_dim > (1 << 20) || static_cast<int64_t>(n_k) * head_dim > (1 << 20))
        return KVFP8_ERR_SHAPE;
    const int64_t q_row = static_cast<int64_t>(n_q) * head_dim, k_row = static_cast<int64_t>(n_k) * head_dim;
    if (query_stride < q_row || query_out_stride < q_row || (n_k > 0 && (key_stride < k_row || key_out_stride < k_row)))
        return KVFP8_ERR_SHAPE;
    if (!std::isfinite(magnitude)) return KVFP8_ERR_SCALE;
    if (num_tokens == 0) return KVFP8_OK;
    if (!query_out || !query || (n_k > 0 && (!key_out || !key)) || !positions || !frequencies) return KVFP8_ERR_NULL;
    const int64_t esz = dtype == KVFP8_F32 ? 4 : 2;
    if (!aligned16(query_out) || !aligned16(query) || !aligned(positions, 8) || !aligned(frequencies, 8) ||
        query_stride * esz % 16 != 0 || query_out_stride * esz % 16 != 0 ||
        (n_k > 0 && (!aligned16(key_out) || !aligned16(key) || key_stride * esz % 16 != 0 ||
                     key_out_stride * esz % 16 != 0)))
        return KVFP8_ERR_ALIGN;
    kvfp8::RotaryArgs a;
    a.src[0] = query;
    a.src[1] = key;
    a.dst[0] = query_out;
    a.dst[1] = key_out;
    a.stride[0] = query_stride;
    a.stride[1] = key_stride;
    a.dst_stride[0] = query_out_stride;
    a.dst_stride[1] = key_out_stride;
    a.heads[0] = n_q;
    a.heads[1] = n_k;
    a.dtype = dtype;
    a.num_tokens = num_tokens;
    a.head_dim = head_dim;
    a.rot = rot_dim;
    a.interleaved = interleaved != 0;
    a.positions = positions;
    a.frequencies = frequencies;
    a.magnitude = magnitude;
    a.sin_magnitude = transpose ? -magnitude : magnitude;
    a.status = status;
    return from_cuda(kvfp8::launch_rotary(a, reinterpret_cast<cudaStream_t>(stream)));
}

kvfp8_status kvfp8_copy_blocks(void *const *caches, const int64_t *block_bytes, int32_t num_caches,
                               int32_t num_blocks, const int32_t *src_blocks,
                               const int32_t *dst_blocks, int64_t num_pairs, uint32_t *status,
                               kvfp8_stream_t stream) {
    kvfp8::CacheList list;
    const kvfp8_status v = make_cache_list(caches, block_bytes, num_caches, num_blocks, &list);
    if (v != KVFP8_OK) return v;
    if (num_pairs < 0 || num_pairs > 0x7FFFFFFFLL) return KVFP8_ERR_SHAPE;
    if (num_pairs == 0) return KVFP8_OK;
    if (!src_blocks || !dst_blocks) return KVFP8_ERR_NULL;
    if (!aligned(src_blocks, 4) || !aligned(dst_blocks, 4)) return KVFP8_ERR_ALIGN;
    return from_cuda(kvfp8::launch_copy_blocks(list, num_blocks, src_blocks, dst_blocks,
                                               static_cast<int32_t>(num_pairs), status,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

size_t kvfp8_compact_blocks_workspace_size(int32_t num_blocks) {
    return num_blocks < 1 ? 0 : kvfp8::compact_workspace_size(num_blocks);
}

kvfp8_status kvfp8_compact_blocks(void *const *caches, const int64_t *block_bytes,
                                  int32_t num_caches, int32_t num_blocks, int32_t block_size,
                                  const int32_t *block_tables, int32_t max_blocks_per_seq,
                                  const int32_t *seq_lens, int32_t num_seqs,
                                  int32_t *new_block_tables, int32_t *num_used, void *workspace,
                                  size_t workspace_bytes, uint32_t *status, kvfp8_stream_t stream) {
    kvfp8::CacheList list;
    const kvfp8_status v = make_cache_list(caches, block_bytes, num_caches, num_blocks, &list);
    if (v != KVFP8_OK) return v;
    if (block_size < 1 || num_seqs < 0 || max_blocks_per_seq < 1 || max_blocks_per_seq > (1 << 30) ||
        static_cast<int64_t>(max_blocks_per_seq) * block_size > 0x7FFFFFFFLL)
        return KVFP8_ERR_SHAPE;
    if (!num_used || !workspace ||
        (num_seqs > 0 && (!block_tables || !seq_lens || !new_block_tables)))
        return KVFP8_ERR_NULL;
    if (!aligned16(workspace) || !aligned(num_used, 4) || !aligned(block_tables, 4) ||
        !aligned(seq_lens, 4) || !aligned(new_block_tables, 4))
        return KVFP8_ERR_ALIGN;
    if (workspace_bytes < kvfp8::compact_workspace_size(num_blocks)) return KVFP8_ERR_WORKSPACE;
    return from_cuda(kvfp8::launch_compact_blocks(
        list, num_blocks, block_size, block_tables, max_blocks_per_seq, seq_lens, num_seqs,
        new_block_tables, num_used, workspace, status, reinterpret_cast<cudaStream_t>(stream)));
}

kvfp8_status kvfp8_check_scale_host(float s) {
    return (std::isfinite(s) && s != 0.0f) ? KVFP8_OK : KVFP8_ERR_SCALE;
}

const char *kvfp8_status_string(kvfp8_status s) {
    switch (s) {
        case KVFP8_OK: return "ok";
        case KVFP8_ERR_NULL: return "null pointer";
        case KVFP8_ERR_SHAPE: return "shape out of range";
        case KVFP8_ERR_DTYPE: return "unsupported dtype";
        case KVFP8_ERR_SCALE: return "scale must be finite and nonzero";
        case KVFP8_ERR_ALIGN: return "pointer or stride not 16-byte aligned";
        case KVFP8_ERR_WORKSPACE: return "workspace too small";
        case KVFP8_ERR_CUDA: return "CUDA error";
        case KVFP8_ERR_UNSUPPORTED: return "unsupported configuration";
    }
    return "unknown status";
}

}  // extern "C"
