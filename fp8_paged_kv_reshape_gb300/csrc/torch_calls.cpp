// The calls of the 4-bit cache, of the cache with block scales, of rotary positions and of pages on torch
// tensors: argument checks, allocation and the C call, for binding.py.
//
// These run once per layer and step, where a kernel takes a few microseconds, and the checks look at
// some fifty tensor attributes.  Read from Python each costs 0.06 to 0.15 us, the marshalling of twenty
// arguments 1.6 us and an allocation between launches 4 us; here a write takes 3.3 us of host time
// instead of 10.6, a decode call 6.5 instead of 18.2, copy_blocks 3.4 instead of 8.4, compact_blocks 10
// instead of 23.6.
//
// Tensors have to be on the current device; work goes to its current stream, outputs and workspaces
// come from that stream's memory.
#include <torch/extension.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <cstdlib>
#include <optional>
#include <utility>
#include <vector>

#include "../../include/kvfp8.h"

namespace {

using at::Tensor;
using Opt = std::optional<Tensor>;

// binding.py's, called with (code, call name).  Never destroyed: the interpreter goes first.
py::object &raise_status() {
    static py::object *f = new py::object;
    return *f;
}

void check(kvfp8_status rc, const char *what) {
    if (rc != KVFP8_OK) raise_status()(static_cast<int>(rc), what);
}

void *ptr(const Tensor &t) { return t.data_ptr(); }
void *ptr(const Opt &t) { return t ? t->data_ptr() : nullptr; }
template <typename T>
T *ptr(const Tensor &t) { return static_cast<T *>(t.data_ptr()); }
uint32_t *status_ptr(const Opt &t) { return static_cast<uint32_t *>(ptr(t)); }

// a kernel argument: sizes past 32 bits are refused, not cut
int32_t i32(int64_t x, const char *what) {
    TORCH_CHECK_VALUE(x <= INT32_MAX, what, " must be below 2^31");
    return static_cast<int32_t>(x);
}

// The current device, which every tensor of the call has to be on.
class Call {
public:
    explicit Call(const Tensor &first) : here_(first.get_device()), first_(first) {}  // (-1 on the CPU)
    Call &on(const Tensor &t) {
        TORCH_CHECK_VALUE(t.get_device() == here_, "tensors on different devices: ", t.device(), " and ",
                          first_.device());
        return *this;
    }
    Call &on(const Opt &t) { return t ? on(*t) : *this; }
    Call &start() {
        TORCH_CHECK_VALUE(here_ >= 0, "tensors must be CUDA tensors");
        const int current = c10::cuda::current_device();
        TORCH_CHECK_VALUE(here_ == current, "tensors on cuda:", here_, ", the current device is cuda:", current);
        return *this;
    }
    kvfp8_stream_t stream() const {
        return reinterpret_cast<kvfp8_stream_t>(c10::cuda::getCurrentCUDAStream(here_).stream());
    }
    Tensor empty(at::IntArrayRef sizes, at::ScalarType dtype) const {
        return at::empty(sizes, at::TensorOptions().dtype(dtype).device(c10::kCUDA, here_));
    }

private:
    c10::DeviceIndex here_;
    const Tensor &first_;
};

bool dense(const Tensor &t, at::ScalarType dtype) { return t.scalar_type() == dtype && t.is_contiguous(); }

// the scales' common type
kvfp8_dtype scale_type(const Opt &k, const Opt &v) {
    std::optional<at::ScalarType> dt;
    for (const Opt *s : {&k, &v}) {
        if (!*s) continue;
        const Tensor &t = **s;
        TORCH_CHECK_TYPE(t.numel() == 1 && t.is_cuda() && (t.scalar_type() == at::kFloat || t.scalar_type() == at::kBFloat16),
                         "scales must be 1-element CUDA float32 or bfloat16 tensors (or None)");
        TORCH_CHECK_TYPE(!dt || *dt == t.scalar_type(), "k_scale and v_scale must share one dtype");
        dt = t.scalar_type();
    }
    return dt == at::kBFloat16 ? KVFP8_BF16 : KVFP8_F32;
}

void check_status(const Opt &status) {
    TORCH_CHECK_VALUE(!status || (status->scalar_type() == at::kInt && status->numel() >= 1),
                      "status must be an int32 [1] tensor");
}

void check_workspace(const Opt &workspace) {
    TORCH_CHECK_VALUE(!workspace || workspace->is_contiguous(), "workspace must be contiguous");
}

void check_slots(const Tensor &slots, int64_t n) {
    TORCH_CHECK_VALUE(dense(slots, at::kLong) && slots.numel() == n,
                      "slot_mapping must be a contiguous int64 [num_tokens] tensor");
}

// the kernels index both for every sequence
void check_tables(const Tensor &tables, const Tensor &lens, int64_t num_seqs) {
    TORCH_CHECK_VALUE(dense(tables, at::kInt) && tables.dim() == 2 && tables.size(0) == num_seqs,
                      "block_tables must be a contiguous int32 [num_seqs, max_blocks] tensor");
    TORCH_CHECK_VALUE(dense(lens, at::kInt) && lens.numel() == num_seqs,
                      "seq_lens must be a contiguous int32 [num_seqs] tensor");
}

struct CacheShape {
    int32_t num_blocks, block_size, n_kv, head_dim;
    bool operator==(const CacheShape &o) const {
        return num_blocks == o.num_blocks && block_size == o.block_size && n_kv == o.n_kv && head_dim == o.head_dim;
    }
};

// one side of a 4-bit cache
CacheShape check_side(const Tensor &codes, const Tensor &scales) {
    TORCH_CHECK_VALUE(dense(codes, at::kByte) && codes.dim() == 4,
                      "4-bit codes must be contiguous uint8 [num_blocks, block_size, n_kv, head_dim/2]");
    const auto s = codes.sizes();
    TORCH_CHECK_VALUE(s[3] % 8 == 0 && dense(scales, at::kByte) &&
                          scales.sizes() == at::IntArrayRef({s[0], s[2], s[1], s[3] / 8}),
                      "their scales must be contiguous uint8 [num_blocks, n_kv, block_size, head_dim/16]");
    return {i32(s[0], "num_blocks"), i32(s[1], "block_size"), i32(s[2], "n_kv"), i32(2 * s[3], "head_dim")};
}

CacheShape check_caches(const Tensor &kc, const Tensor &vc, const Tensor &kg, const Tensor &vg) {
    const CacheShape shape = check_side(kc, kg);
    TORCH_CHECK_VALUE(check_side(vc, vg) == shape, "key and value caches must have one shape");
    return shape;
}

// ---------------------------------------------------------------- 4-bit cache

void reshape_and_cache_fp4(const Tensor &key, const Tensor &value, const Tensor &kc, const Tensor &vc,
                           const Tensor &kg, const Tensor &vg, const Tensor &slots, const Opt &k_scale,
                           const Opt &v_scale, const Opt &status) {
    const auto dt = key.scalar_type();
    TORCH_CHECK_TYPE(value.scalar_type() == dt && (dt == at::kBFloat16 || dt == at::kFloat),
                     "key and value must share one dtype, bfloat16 or float32");
    TORCH_CHECK_VALUE(key.dim() == 3 && value.sizes() == key.sizes(),
                      "key/value must be [num_tokens, n_kv, head_dim] with equal shapes");
    const int64_t n = key.size(0), n_kv = key.size(1), hd = key.size(2);
    for (const Tensor *t : {&key, &value})
        TORCH_CHECK_VALUE(n == 0 || (t->stride(2) == 1 && (n_kv == 1 || t->stride(1) == hd)),
                          "key/value inner dims [n_kv, head_dim] must be dense");
    const CacheShape c = check_caches(kc, vc, kg, vg);
    TORCH_CHECK_VALUE(c.n_kv == n_kv && c.head_dim == hd,
                      "the caches' n_kv and head_dim must be those of key and value");
    check_slots(slots, n);
    const kvfp8_dtype sdt = scale_type(k_scale, v_scale);
    check_status(status);
    Call call(key);
    call.on(value).on(kc).on(vc).on(kg).on(vg).on(slots).on(k_scale).on(v_scale).on(status).start();
    // (the stride of a single row is never used, and may be anything)
    const int64_t row = n_kv * hd, ks = n > 1 ? key.stride(0) : row, vs = n > 1 ? value.stride(0) : row;
    check(kvfp8_reshape_and_cache_fp4(ptr(key), ptr(value), dt == at::kFloat ? KVFP8_F32 : KVFP8_BF16, ks, vs, n,
                                      ptr<uint8_t>(kc), ptr<uint8_t>(vc), ptr<uint8_t>(kg), ptr<uint8_t>(vg),
                                      c.num_blocks, c.block_size, c.n_kv, c.head_dim, ptr<int64_t>(slots),
                                      ptr(k_scale), ptr(v_scale), sdt, status_ptr(status), call.stream()),
          "kvfp8_reshape_and_cache_fp4");
}

Tensor dequant_fp4(const Tensor &codes, const Tensor &scales, const Tensor &slots, bool to_bf16, const Opt &scale,
                   const Opt &out, const Opt &status) {
    const CacheShape c = check_side(codes, scales);
    TORCH_CHECK_VALUE(slots.dim() == 1, "slot_mapping must be a contiguous int64 [num_tokens] tensor");
    const int64_t n = slots.size(0);
    check_slots(slots, n);
    const auto dt = to_bf16 ? at::kBFloat16 : at::kFloat;
    const int64_t shape[3] = {n, c.n_kv, c.head_dim};
    TORCH_CHECK_VALUE(!out || (dense(*out, dt) && out->sizes() == at::IntArrayRef(shape)),
                      "out must be a contiguous dst_dtype [num_tokens, n_kv, head_dim] tensor");
    const kvfp8_dtype sdt = scale_type(scale, std::nullopt);
    check_status(status);
    Call call(codes);
    call.on(scales).on(slots).on(scale).on(out).on(status).start();
    Tensor dst = out ? *out : call.empty(shape, dt);
    check(kvfp8_dequant_fp4(ptr(dst), to_bf16 ? KVFP8_BF16 : KVFP8_F32, ptr<uint8_t>(codes), ptr<uint8_t>(scales),
                            c.num_blocks, c.block_size, c.n_kv, c.head_dim, ptr<int64_t>(slots), n, ptr(scale), sdt,
                            status_ptr(status), call.stream()),
          "kvfp8_dequant_fp4");
    return dst;
}

// Both attention calls (qsl: the multi-query form).
Tensor attention_fp4(const Tensor &query, const Opt &qsl, int64_t max_query_len, const Tensor &kc, const Tensor &vc,
                     const Tensor &kg, const Tensor &vg, const Tensor &tables, const Tensor &lens,
                     const Opt &k_scale, const Opt &v_scale, double sm_scale, const Opt &out, const Opt &workspace,
                     const Opt &status) {
    TORCH_CHECK_VALUE(dense(query, at::kBFloat16) && query.dim() == 3,
                      "query must be a contiguous bf16 [rows, n_q, head_dim] tensor");
    const int64_t num_seqs = qsl ? lens.numel() : query.size(0);
    TORCH_CHECK_VALUE(!qsl || (dense(*qsl, at::kInt) && qsl->numel() == num_seqs + 1),
                      "query_start_loc must be a contiguous int32 [num_seqs + 1] tensor");
    const CacheShape c = check_caches(kc, vc, kg, vg);
    TORCH_CHECK_VALUE(c.head_dim == query.size(2), "the caches' head_dim must be the query's");
    check_tables(tables, lens, num_seqs);
    TORCH_CHECK_VALUE(!out || (dense(*out, at::kBFloat16) && out->sizes() == query.sizes()),
                      "out must be a contiguous bf16 tensor shaped like query");
    check_workspace(workspace);
    const kvfp8_dtype sdt = scale_type(k_scale, v_scale);
    check_status(status);
    Call call(query);
    call.on(kc).on(vc).on(kg).on(vg).on(tables).on(lens).on(k_scale).on(v_scale).on(out).on(workspace).on(status);
    call.on(qsl).start();
    const int32_t seqs = i32(num_seqs, "num_seqs"), rows = i32(query.size(0), "query rows"),
                  n_q = i32(query.size(1), "n_q"), most = i32(tables.size(1), "max_blocks"),
                  qmax = i32(std::max<int64_t>(max_query_len, 0), "max_query_len");
    Tensor dst = out ? *out : call.empty(query.sizes(), at::kBFloat16);
    Opt ws = workspace;
    if (!ws) {
        const size_t need = kvfp8_paged_attention_fp4_workspace_size(seqs, n_q, c.n_kv, c.head_dim, qmax, most,
                                                                     c.block_size);
        if (need > 0) ws = call.empty({static_cast<int64_t>(need)}, at::kByte);
    }
    const size_t ws_bytes = ws ? ws->nbytes() : 0;
    if (qsl)
        check(kvfp8_paged_attention_multi_fp4(
                  ptr(dst), ptr(query), ptr<int32_t>(*qsl), rows, qmax, ptr<uint8_t>(kc), ptr<uint8_t>(vc),
                  ptr<uint8_t>(kg), ptr<uint8_t>(vg), ptr<int32_t>(tables), most, ptr<int32_t>(lens), seqs, n_q,
                  c.n_kv, c.head_dim, c.block_size, c.num_blocks, static_cast<float>(sm_scale), ptr(k_scale),
                  ptr(v_scale), sdt, ptr(ws), ws_bytes, status_ptr(status), call.stream()),
              "kvfp8_paged_attention_multi_fp4");
    else
        check(kvfp8_paged_decode_attention_fp4(
                  ptr(dst), ptr(query), ptr<uint8_t>(kc), ptr<uint8_t>(vc), ptr<uint8_t>(kg), ptr<uint8_t>(vg),
                  ptr<int32_t>(tables), most, ptr<int32_t>(lens), seqs, n_q, c.n_kv, c.head_dim, c.block_size,
                  c.num_blocks, static_cast<float>(sm_scale), ptr(k_scale), ptr(v_scale), sdt, ptr(ws), ws_bytes,
                  status_ptr(status), call.stream()),
              "kvfp8_paged_decode_attention_fp4");
    return dst;
}

Tensor paged_decode_attention_fp4(const Tensor &query, const Tensor &kc, const Tensor &vc, const Tensor &kg,
                                  const Tensor &vg, const Tensor &tables, const Tensor &lens, const Opt &k_scale,
                                  const Opt &v_scale, double sm_scale, const Opt &out, const Opt &workspace,
                                  const Opt &status) {
    return attention_fp4(query, std::nullopt, 1, kc, vc, kg, vg, tables, lens, k_scale, v_scale, sm_scale, out,
                         workspace, status);
}

Tensor paged_attention_multi_fp4(const Tensor &query, const Tensor &qsl, int64_t max_query_len, const Tensor &kc,
                                 const Tensor &vc, const Tensor &kg, const Tensor &vg, const Tensor &tables,
                                 const Tensor &lens, const Opt &k_scale, const Opt &v_scale, double sm_scale,
                                 const Opt &out, const Opt &workspace, const Opt &status) {
    return attention_fp4(query, qsl, max_query_len, kc, vc, kg, vg, tables, lens, k_scale, v_scale, sm_scale, out,
                         workspace, status);
}

// ---------------------------------------------------------------- FP8 cache with block scales

struct BlockCache {
    CacheShape shape;
    int32_t scale_stride;
};

// one side: codes and block scales
BlockCache check_block_side(const Tensor &codes, const Tensor &scales) {
    TORCH_CHECK_VALUE(dense(codes, at::kByte) && codes.dim() == 4,
                      "caches must be contiguous uint8 [num_blocks, block_size, n_kv, head_dim]");
    const auto s = codes.sizes();
    TORCH_CHECK_VALUE(dense(scales, at::kFloat) && scales.dim() == 2 && scales.size(0) == s[0] && scales.size(1) >= s[2] &&
                          scales.size(1) % 4 == 0,
                      "their scales must be contiguous float32 [num_blocks, n_kv rounded up to a multiple of 4]");
    return {{i32(s[0], "num_blocks"), i32(s[1], "block_size"), i32(s[2], "n_kv"), i32(s[3], "head_dim")},
            i32(scales.size(1), "the scales' row")};
}

BlockCache check_block_caches(const Tensor &kc, const Tensor &vc, const Tensor &ks, const Tensor &vs) {
    const BlockCache k = check_block_side(kc, ks), v = check_block_side(vc, vs);
    TORCH_CHECK_VALUE(k.shape == v.shape && k.scale_stride == v.scale_stride, "key and value caches must have one shape");
    return k;
}

void reshape_and_cache_block_scaled(const Tensor &key, const Tensor &value, const Tensor &kc, const Tensor &vc,
                                    const Tensor &ks, const Tensor &vs, const Tensor &slots, const Opt &workspace,
                                    const Opt &status) {
    const auto dt = key.scalar_type();
    TORCH_CHECK_TYPE(value.scalar_type() == dt && (dt == at::kBFloat16 || dt == at::kFloat),
                     "key and value must share one dtype, bfloat16 or float32");
    TORCH_CHECK_VALUE(key.dim() == 3 && value.sizes() == key.sizes(),
                      "key/value must be [num_tokens, n_kv, head_dim] with equal shapes");
    const int64_t n = key.size(0), n_kv = key.size(1), hd = key.size(2);
    for (const Tensor *t : {&key, &value})
        TORCH_CHECK_VALUE(n == 0 || (t->stride(2) == 1 && (n_kv == 1 || t->stride(1) == hd)),
                          "key/value inner dims [n_kv, head_dim] must be dense");
    const BlockCache b = check_block_caches(kc, vc, ks, vs);
    const CacheShape &c = b.shape;
    TORCH_CHECK_VALUE(c.n_kv == n_kv && c.head_dim == hd,
                      "the caches' n_kv and head_dim must be those of key and value");
    check_slots(slots, n);
    check_workspace(workspace);
    check_status(status);
    Call call(key);
    call.on(value).on(kc).on(vc).on(ks).on(vs).on(slots).on(workspace).on(status).start();
    Opt ws = workspace;
    if (!ws) {
        const size_t need = kvfp8_reshape_and_cache_block_scaled_workspace_size(n, c.num_blocks, c.block_size);
        if (need > 0) ws = call.empty({static_cast<int64_t>(need)}, at::kByte);
    }
    // (the stride of a single row is never used, and may be anything)
    const int64_t row = n_kv * hd, kst = n > 1 ? key.stride(0) : row, vst = n > 1 ? value.stride(0) : row;
    check(kvfp8_reshape_and_cache_block_scaled(
              ptr(key), ptr(value), dt == at::kFloat ? KVFP8_F32 : KVFP8_BF16, kst, vst, n, ptr<uint8_t>(kc),
              ptr<uint8_t>(vc), ptr<float>(ks), ptr<float>(vs), b.scale_stride, c.num_blocks, c.block_size, c.n_kv,
              c.head_dim, ptr<int64_t>(slots), ptr(ws), ws ? ws->nbytes() : 0, status_ptr(status), call.stream()),
          "kvfp8_reshape_and_cache_block_scaled");
}

Tensor dequant_block_scaled(const Tensor &codes, const Tensor &scales, const Tensor &slots, bool to_bf16, const Opt &out,
                            const Opt &status) {
    const BlockCache b = check_block_side(codes, scales);
    const CacheShape &c = b.shape;
    TORCH_CHECK_VALUE(slots.dim() == 1, "slot_mapping must be a contiguous int64 [num_tokens] tensor");
    const int64_t n = slots.size(0);
    check_slots(slots, n);
    const auto dt = to_bf16 ? at::kBFloat16 : at::kFloat;
    const int64_t shape[3] = {n, c.n_kv, c.head_dim};
    TORCH_CHECK_VALUE(!out || (dense(*out, dt) && out->sizes() == at::IntArrayRef(shape)),
                      "out must be a contiguous dst_dtype [num_tokens, n_kv, head_dim] tensor");
    check_status(status);
    Call call(codes);
    call.on(scales).on(slots).on(out).on(status).start();
    Tensor dst = out ? *out : call.empty(shape, dt);
    check(kvfp8_dequant_block_scaled(ptr(dst), to_bf16 ? KVFP8_BF16 : KVFP8_F32, ptr<uint8_t>(codes), ptr<float>(scales),
                                     b.scale_stride, c.num_blocks, c.block_size, c.n_kv, c.head_dim, ptr<int64_t>(slots),
                                     n, status_ptr(status), call.stream()),
          "kvfp8_dequant_block_scaled");
    return dst;
}

// Both attention calls (qsl: the multi-query form).
Tensor attention_block_scaled(const Tensor &query, const Opt &qsl, int64_t max_query_len, bool causal, const Tensor &kc,
                              const Tensor &vc, const Tensor &ks, const Tensor &vs, const Tensor &tables,
                              const Tensor &lens, double sm_scale, const Opt &out, const Opt &workspace,
                              const Opt &status) {
    TORCH_CHECK_VALUE(dense(query, at::kBFloat16) && query.dim() == 3,
                      "query must be a contiguous bf16 [rows, n_q, head_dim] tensor");
    const int64_t num_seqs = qsl ? lens.numel() : query.size(0);
    TORCH_CHECK_VALUE(!qsl || (dense(*qsl, at::kInt) && qsl->numel() == num_seqs + 1),
                      "query_start_loc must be a contiguous int32 [num_seqs + 1] tensor");
    const BlockCache b = check_block_caches(kc, vc, ks, vs);
    const CacheShape &c = b.shape;
    TORCH_CHECK_VALUE(c.head_dim == query.size(2), "the caches' head_dim must be the query's");
    check_tables(tables, lens, num_seqs);
    TORCH_CHECK_VALUE(!out || (dense(*out, at::kBFloat16) && out->sizes() == query.sizes()),
                      "out must be a contiguous bf16 tensor shaped like query");
    check_workspace(workspace);
    check_status(status);
    Call call(query);
    call.on(kc).on(vc).on(ks).on(vs).on(tables).on(lens).on(out).on(workspace).on(status).on(qsl).start();
    const int32_t seqs = i32(num_seqs, "num_seqs"), rows = i32(query.size(0), "query rows"),
                  n_q = i32(query.size(1), "n_q"), most = i32(tables.size(1), "max_blocks"),
                  qmax = i32(std::max<int64_t>(max_query_len, 0), "max_query_len");
    Tensor dst = out ? *out : call.empty(query.sizes(), at::kBFloat16);
    Opt ws = workspace;
    if (!ws) {
        const size_t need = kvfp8_paged_attention_block_scaled_workspace_size(seqs, n_q, c.n_kv, c.head_dim, qmax, most,
                                                                              c.block_size);
        if (need > 0) ws = call.empty({static_cast<int64_t>(need)}, at::kByte);
    }
    const size_t ws_bytes = ws ? ws->nbytes() : 0;
    if (qsl)
        check(kvfp8_paged_attention_multi_block_scaled(
                  ptr(dst), ptr(query), ptr<int32_t>(*qsl), rows, qmax, causal, ptr<uint8_t>(kc), ptr<uint8_t>(vc),
                  ptr<float>(ks), ptr<float>(vs), b.scale_stride, ptr<int32_t>(tables), most, ptr<int32_t>(lens), seqs, n_q,
                  c.n_kv, c.head_dim, c.block_size, c.num_blocks, static_cast<float>(sm_scale), ptr(ws), ws_bytes,
                  status_ptr(status), call.stream()),
              "kvfp8_paged_attention_multi_block_scaled");
    else
        check(kvfp8_paged_decode_attention_block_scaled(
                  ptr(dst), ptr(query), ptr<uint8_t>(kc), ptr<uint8_t>(vc), ptr<float>(ks), ptr<float>(vs), b.scale_stride,
                  ptr<int32_t>(tables), most, ptr<int32_t>(lens), seqs, n_q, c.n_kv, c.head_dim, c.block_size,
                  c.num_blocks, static_cast<float>(sm_scale), ptr(ws), ws_bytes, status_ptr(status), call.stream()),
              "kvfp8_paged_decode_attention_block_scaled");
    return dst;
}

Tensor paged_decode_attention_block_scaled(const Tensor &query, const Tensor &kc, const Tensor &vc, const Tensor &ks,
                                           const Tensor &vs, const Tensor &tables, const Tensor &lens, double sm_scale,
                                           const Opt &out, const Opt &workspace, const Opt &status) {
    return attention_block_scaled(query, std::nullopt, 1, true, kc, vc, ks, vs, tables, lens, sm_scale, out, workspace,
                                  status);
}

Tensor paged_attention_multi_block_scaled(const Tensor &query, const Tensor &qsl, int64_t max_query_len, const Tensor &kc,
                                          const Tensor &vc, const Tensor &ks, const Tensor &vs, const Tensor &tables,
                                          const Tensor &lens, bool causal, double sm_scale, const Opt &out,
                                          const Opt &workspace, const Opt &status) {
    return attention_block_scaled(query, qsl, max_query_len, causal, kc, vc, ks, vs, tables, lens, sm_scale, out, workspace,
                                  status);
}

// ---------------------------------------------------------------- rotary positions

// Rows of heads whose inner dims are dense; their stride (that of a single row is never used).
int64_t head_rows(const Tensor &t, const char *what) {
    const int64_t n = t.size(0), row = t.size(1) * t.size(2);
    TORCH_CHECK_VALUE(n == 0 || (t.stride(2) == 1 && (t.size(1) == 1 || t.stride(1) == t.size(2))), what,
                      "'s inner dims [heads, head_dim] must be dense");
    return n > 1 ? t.stride(0) : row;
}

// An output is its own input or apart from `other`.
void check_apart(const Tensor &out, const Tensor &other, bool may_be_same) {
    if (out.numel() == 0 || other.numel() == 0) return;
    if (may_be_same && out.data_ptr() == other.data_ptr() && (out.size(0) == 1 || out.stride(0) == other.stride(0))) return;
    auto end = [](const Tensor &t) {
        return ptr<char>(t) + ((t.size(0) - 1) * t.stride(0) + t.size(1) * t.size(2)) * t.element_size();
    };
    if (end(out) <= ptr<char>(other) || end(other) <= ptr<char>(out)) return;
    // slices of one fused row: the same stride, and apart within it
    const int64_t stride = out.stride(0) * out.element_size(), gap = std::abs(ptr<char>(out) - ptr<char>(other));
    const Tensor &low = ptr<char>(out) < ptr<char>(other) ? out : other, &high = &low == &out ? other : out;
    TORCH_CHECK_VALUE(out.stride(0) == other.stride(0) && gap >= low.size(1) * low.size(2) * low.element_size() &&
                          gap + high.size(1) * high.size(2) * high.element_size() <= stride,
                      "outputs must not overlap the inputs or each other (an output may be its own input)");
}

std::pair<Tensor, Opt> rotary_embedding(const Tensor &query, const Opt &key, const Tensor &positions,
                                        const Tensor &frequencies, bool interleaved, double magnitude, bool transpose,
                                        const Opt &query_out, const Opt &key_out, const Opt &status) {
    const auto dt = query.scalar_type();
    TORCH_CHECK_TYPE((dt == at::kBFloat16 || dt == at::kFloat) && (!key || key->scalar_type() == dt),
                     "query and key must share one dtype, bfloat16 or float32");
    TORCH_CHECK_VALUE(query.dim() == 3, "query must be [num_tokens, n_q, head_dim]");
    TORCH_CHECK_VALUE(!key || (key->dim() == 3 && key->size(0) == query.size(0) && key->size(2) == query.size(2)),
                      "key must be [num_tokens, n_k, head_dim] of query's tokens and head_dim");
    const int64_t n = query.size(0);
    TORCH_CHECK_VALUE(dense(positions, at::kLong) && positions.numel() == n,
                      "positions must be a contiguous int64 [num_tokens] tensor");
    TORCH_CHECK_VALUE(dense(frequencies, at::kDouble) && frequencies.dim() == 1,
                      "frequencies must be a contiguous float64 [rot_dim / 2] tensor");
    TORCH_CHECK_VALUE(!query_out || (query_out->scalar_type() == dt && query_out->sizes() == query.sizes()),
                      "query_out must have query's shape and dtype");
    TORCH_CHECK_VALUE(!key_out || (key && key_out->scalar_type() == dt && key_out->sizes() == key->sizes()),
                      "key_out must have key's shape and dtype");
    check_status(status);
    Call call(query);
    call.on(key).on(positions).on(frequencies).on(query_out).on(key_out).on(status).start();
    const int64_t q_stride = head_rows(query, "query"), k_stride = key ? head_rows(*key, "key") : 0;
    const Tensor q_to = query_out ? *query_out : call.empty(query.sizes(), dt);
    const Opt k_to = !key ? Opt() : key_out ? *key_out : Opt(call.empty(key->sizes(), dt));
    const int64_t q_to_stride = head_rows(q_to, "query_out"), k_to_stride = key ? head_rows(*k_to, "key_out") : 0;
    if (query_out) {
        check_apart(q_to, query, true);
        if (key) check_apart(q_to, *key, false);
    }
    if (key_out) {
        check_apart(*k_to, *key, true);
        check_apart(*k_to, query, false);
        check_apart(*k_to, q_to, false);
    }
    check(kvfp8_rotary_embedding(ptr(q_to), ptr(k_to), q_to_stride, k_to_stride, ptr(query), ptr(key), q_stride, k_stride,
                                 dt == at::kFloat ? KVFP8_F32 : KVFP8_BF16, n, i32(query.size(1), "n_q"),
                                 key ? i32(key->size(1), "n_k") : 0, i32(query.size(2), "head_dim"),
                                 i32(2 * frequencies.size(0), "rot_dim"), interleaved, transpose, ptr<int64_t>(positions),
                                 ptr<double>(frequencies), static_cast<float>(magnitude), status_ptr(status),
                                 call.stream()),
          "kvfp8_rotary_embedding");
    return {q_to, k_to};
}

// ---------------------------------------------------------------- pages

struct Caches {
    std::vector<void *> ptrs;
    std::vector<int64_t> block_bytes;
    int32_t num_blocks;

    explicit Caches(const std::vector<Tensor> &caches) {
        TORCH_CHECK_VALUE(!caches.empty() && caches.size() <= KVFP8_MAX_CACHES, "1 to ", KVFP8_MAX_CACHES, " caches");
        const int64_t nb = caches[0].dim() > 1 ? caches[0].size(0) : 0;
        num_blocks = i32(nb, "num_blocks");
        std::vector<std::pair<const char *, const char *>> spans;
        spans.reserve(caches.size());
        ptrs.reserve(caches.size());
        block_bytes.reserve(caches.size());
        for (const Tensor &c : caches) {
            const int64_t total = static_cast<int64_t>(c.nbytes());
            TORCH_CHECK_VALUE(c.dim() >= 2 && c.size(0) == nb && total > 0 && c.is_contiguous(),
                              "caches must be contiguous tensors [num_blocks, ...] of one num_blocks");
            ptrs.push_back(c.data_ptr());
            block_bytes.push_back(total / nb);
            spans.emplace_back(ptr<char>(c), ptr<char>(c) + total);
        }
        std::sort(spans.begin(), spans.end());
        for (size_t i = 1; i < spans.size(); ++i)
            TORCH_CHECK_VALUE(spans[i - 1].second <= spans[i].first, "caches must not overlap");
    }
    int32_t count() const { return static_cast<int32_t>(ptrs.size()); }
};

void copy_blocks(const std::vector<Tensor> &tensors, const Tensor &src, const Tensor &dst, const Opt &status) {
    const Caches c(tensors);
    for (const Tensor *t : {&src, &dst})
        TORCH_CHECK_VALUE(dense(*t, at::kInt) && t->dim() == 1,
                          "src_blocks and dst_blocks must be contiguous int32 [num_pairs] tensors");
    TORCH_CHECK_VALUE(src.numel() == dst.numel(), "src_blocks and dst_blocks must have one length");
    check_status(status);
    Call call(tensors[0]);
    for (const Tensor &t : tensors) call.on(t);
    call.on(src).on(dst).on(status).start();
    check(kvfp8_copy_blocks(c.ptrs.data(), c.block_bytes.data(), c.count(), c.num_blocks, ptr<int32_t>(src),
                            ptr<int32_t>(dst), src.numel(), status_ptr(status), call.stream()),
          "kvfp8_copy_blocks");
}

std::pair<Tensor, Tensor> compact_blocks(const std::vector<Tensor> &tensors, const Tensor &tables, const Tensor &lens,
                                         int64_t block_size, const Opt &new_tables, const Opt &num_used,
                                         const Opt &workspace, const Opt &status) {
    const Caches c(tensors);
    const int64_t num_seqs = lens.numel();
    check_tables(tables, lens, num_seqs);
    TORCH_CHECK_VALUE(!new_tables || (dense(*new_tables, at::kInt) && new_tables->sizes() == tables.sizes()),
                      "new_block_tables must be a contiguous int32 tensor shaped like block_tables");
    TORCH_CHECK_VALUE(!num_used || (num_used->scalar_type() == at::kInt && num_used->numel() == 1),
                      "num_used must be an int32 [1] tensor");
    check_workspace(workspace);
    check_status(status);
    Call call(tensors[0]);
    for (const Tensor &t : tensors) call.on(t);
    call.on(tables).on(lens).on(new_tables).on(num_used).on(workspace).on(status).start();
    const Tensor to = new_tables ? *new_tables : call.empty(tables.sizes(), at::kInt);
    const Tensor used = num_used ? *num_used : call.empty({1}, at::kInt);
    const Tensor ws = workspace ? *workspace
                                : call.empty({static_cast<int64_t>(kvfp8_compact_blocks_workspace_size(c.num_blocks))},
                                             at::kByte);
    check(kvfp8_compact_blocks(c.ptrs.data(), c.block_bytes.data(), c.count(), c.num_blocks,
                               i32(std::max<int64_t>(block_size, 0), "block_size"), ptr<int32_t>(tables),
                               i32(tables.size(1), "max_blocks"), ptr<int32_t>(lens), i32(num_seqs, "num_seqs"),
                               ptr<int32_t>(to), ptr<int32_t>(used), ptr(ws), ws.nbytes(), status_ptr(status),
                               call.stream()),
          "kvfp8_compact_blocks");
    return {to, used};
}

}  // namespace

PYBIND11_MODULE(kvfp8_torch, m) {
    // (wrapped, so that errors come out as the Python exceptions torch's own calls raise)
    m.def("reshape_and_cache_fp4", torch::wrap_pybind_function(reshape_and_cache_fp4));
    m.def("dequant_fp4", torch::wrap_pybind_function(dequant_fp4));
    m.def("paged_decode_attention_fp4", torch::wrap_pybind_function(paged_decode_attention_fp4));
    m.def("paged_attention_multi_fp4", torch::wrap_pybind_function(paged_attention_multi_fp4));
    m.def("reshape_and_cache_block_scaled", torch::wrap_pybind_function(reshape_and_cache_block_scaled));
    m.def("dequant_block_scaled", torch::wrap_pybind_function(dequant_block_scaled));
    m.def("paged_decode_attention_block_scaled", torch::wrap_pybind_function(paged_decode_attention_block_scaled));
    m.def("paged_attention_multi_block_scaled", torch::wrap_pybind_function(paged_attention_multi_block_scaled));
    m.def("rotary_embedding", torch::wrap_pybind_function(rotary_embedding));
    m.def("copy_blocks", torch::wrap_pybind_function(copy_blocks));
    m.def("compact_blocks", torch::wrap_pybind_function(compact_blocks));
    m.def("on_status", [](py::object f) { raise_status() = std::move(f); });
}
