// The 4-bit paged cache's writer and its rows read back, sm_103a.
//
// A group of 16 dims of a token's kv head is stored as 16 E2M1 codes and one E4M3 scale byte B;
// with the layer's scalar s the value of a dim is code * (B * s).  Writing a group:
//   a = max |x|,  B = E4M3((a / |s|) / 6),  d = B * |s|,  code = sign, E2M1(|x| / d)
// every quotient and product a float rounded to nearest even (the header gives the corner
// cases).  Both kernels are HBM streams: the writer reads 2 (bf16) or 4 bytes per element and
// writes 0.5625, the reader the reverse.
//
// A lane takes whole groups: a group's 16 source elements are 32 contiguous bytes of bf16 (one load),
// its codes one 8-byte store, and the maximum needs no exchange between lanes; four lanes' scale
// bytes leave as one word.  A row is spread over a power of two of lanes, at most 32, so short rows
// share a warp; a row of more than 32 groups gives each lane two, 32 apart (two loads and two
// independent conversions in flight; 32768 rows of 64 groups 60 to 38 us with the word stores), and
// passes of 64 groups go along gridDim.y.  gridDim.z is the side (K or V), so a warp has one layer
// scale.  Warps stride over the rows and hold the next row's elements, and the slot after it, while
// they convert the present one.
//
// 32768 rows of 8 heads of 128, bf16, both sides: the write 37.4 us (172 MB: 4.6 TB/s; twice the rows
// cost 5.3 TB/s more, the rest is start and end), a side read back 14.3 to 16.7 us (86 MB: 5.2 to 6.0
// TB/s).  The writer issues 182 instructions per 32 groups, 82 of them to the FMA pipe for the
// quotients: a warp waits as much for the pipes and its own dependencies as for memory.  Source
// rows staged by bulk copies in a ring of three per warp instead of in registers: 43 us.
//
// The quotient |x| / d has to be the float quotient, because halfway cases are common (a bf16 x
// over a d of few bits) and decide the code.  It takes the reciprocal-and-two-residuals divide
// of the 8-bit writer (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. R&D 34(1), 1990), in packed pairs; groups whose scale saturates
// or whose d is outside [2^-60, 2^60] divide element by element.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvfp8_device.cuh"
#include "kvfp8_e2m1.cuh"
#include "kvfp8_internal.h"

namespace kvfp8 {
namespace {

constexpr int kWarps = 8;  // per CTA

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// maxima that a NaN operand turns into NaN
__device__ __forceinline__ uint32_t max_abs_nan_bf16x2(uint32_t a, uint32_t b) {  // (of either sign)
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void ld_v8(const uint8_t *p, uint32_t *w) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}
__device__ __forceinline__ void ld_v4(const uint8_t *p, uint32_t *w) {
    asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p));
}
__device__ __forceinline__ void st_v8(uint8_t *p, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Sixteen elements of a source row as they lie in memory.
template <bool kF32>
struct Group16 {
    static constexpr int kWords = kF32 ? 16 : 8;
    uint32_t w[kWords];
    // kWide: 32-byte loads (p 32-byte aligned), else 16-byte ones
    template <bool kWide>
    __device__ __forceinline__ void load(const uint8_t *p) {
#pragma unroll
        for (int i = 0; i < kWords; i += 8) {
            if (kWide) {
                ld_v8(p + 4 * i, w + i);
            } else {
                ld_v4(p + 4 * i, w + i);
                ld_v4(p + 4 * i + 16, w + i + 4);
            }
        }
    }
    __device__ __forceinline__ void unpack(float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if (kF32) {
                x[i] = __uint_as_float(w[i]);
            } else {
                x[2 * i] = bf16lo(w[i]);
                x[2 * i + 1] = bf16hi(w[i]);
            }
        }
    }
    // max |x|, NaN if any element is
    __device__ __forceinline__ float amax() const {
        if (kF32) {
            float m = fabsf(__uint_as_float(w[0]));
#pragma unroll
            for (int i = 1; i < kWords; ++i) m = max_nan(m, fabsf(__uint_as_float(w[i])));
            return m;
        }
        uint32_t m = w[0];
#pragma unroll
        for (int i = 1; i < kWords; ++i) m = max_abs_nan_bf16x2(m, w[i]);
        return max_nan(fabsf(bf16lo(m)), fabsf(bf16hi(m)));
    }
};

// The layer scale of a side.  fast: |s| in [2^-50, 2^50], so that every d = B |s| that is not zero
// lies in [2^-60, 2^60], the range of the reciprocal divide.
struct LayerScale {
    float sa, y;    // |s|, RN(1 / |s|)
    uint32_t neg;   // 0x88888888 when s < 0
    bool fast;
    __device__ __forceinline__ explicit LayerScale(float s) {
        sa = fabsf(s);
        y = __frcp_rn(sa);
        neg = signbit(s) ? 0x88888888u : 0u;
        fast = sa >= 0x1p-50f && sa <= 0x1p50f;
    }
};

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    return __half2float(__ushort_as_half(static_cast<uint16_t>(f16x2_from_e4m3x2(byte) & 0xFFFFu)));
}

// Eight codes by plain divisions.  (By value: an array argument would put every group's elements on
// the stack.)
__device__ __noinline__ uint32_t quantize_slow8(float x0, float x1, float x2, float x3, float x4, float x5,
                                                float x6, float x7, float d) {
    const float x[8] = {x0, x1, x2, x3, x4, x5, x6, x7};
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float ax = fabsf(x[i]);
        const float m = isinf(ax) ? 6.f : d == 0.f ? 0.f : __fdiv_rn(ax, d);
        q[i] = x[i] < 0.f ? -m : m;
    }
    return e2m1x8_from_f32(q);
}
__device__ __noinline__ uint32_t scale_byte_slow(float a, float sa) {
    return isnan(a) ? 0x7Fu : e4m3x2_from_f32(__fdiv_rn(__fdiv_rn(a, sa), 6.f), 0.f) & 0xFFu;
}

// RN(x / d) for x >= 0 from y = RN(1 / d) by the two residual steps, wherever the quotient is in
// the range that decides an E4M3 code; NaN and a quotient that overflows on the way give 2^100.
__device__ __forceinline__ float quotient(float x, float d, float y) {
    const float q0 = x * y;
    const float q1 = fmaf(fmaf(q0, -d, x), y, q0);
    return fminf(fmaf(fmaf(q1, -d, x), y, q1), 0x1p100f);
}

// Sixteen elements -> their codes and the group's scale byte.  The rare groups (a scale that
// saturates or may, infinite or NaN elements, a layer scale out of range) all show byte 0x7E or
// !fast.
template <bool kF32>
__device__ __forceinline__ uint2 quantize16(const Group16<kF32> &g, const LayerScale &s, uint32_t &byte) {
    const float a = g.amax();
    byte = e4m3x2_from_f32(quotient(quotient(a, s.sa, s.y), 6.f, 0x1.555556p-3f), 0.f) & 0xFFu;  // RN(1/6)
    float x[16];
    g.unpack(x);
    uint2 c;
    if (__builtin_expect(byte == 0x7Eu || !s.fast, 0)) {
        byte = scale_byte_slow(a, s.sa);
        if (byte == 0x7Fu) return make_uint2(0u, 0u);  // a NaN among them
        const float d = __fmul_rn(e4m3_value(byte), s.sa);
        c.x = quantize_slow8(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], d);
        c.y = quantize_slow8(x[8], x[9], x[10], x[11], x[12], x[13], x[14], x[15], d);
    } else {
        // q0 = x*y, then two residual steps q += (x - q*d)*y.  d = 0 takes y = 0, which gives
        // zeros with the sign of x; x = -0 gives +0.
        const float d = __fmul_rn(e4m3_value(byte), s.sa);
        const float y = d == 0.f ? 0.f : __frcp_rn(d);
        const uint64_t y2 = pack2(y, y), nd2 = pack2(-d, -d);
        float q[16];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const uint64_t v = pack2(x[i], x[i + 1]);
            const uint64_t q0 = mul2(v, y2);
            const uint64_t q1 = fma2(fma2(q0, nd2, v), y2, q0);
            unpack2(fma2(fma2(q1, nd2, v), y2, q1), q[i], q[i + 1]);
        }
        c = make_uint2(e2m1x8_from_f32(q), e2m1x8_from_f32(q + 8));
    }
    return make_uint2(c.x ^ s.neg, c.y ^ s.neg);
}

// How rows map to lanes: gpr groups a row over 1 << lpr_log2 lanes.
struct RowMap {
    int32_t gpr, lpr_log2;
    int32_t gph_log2;    // log2 of the groups of a kv head
    int32_t bs_log2;
};

// kG: groups of a row per lane, 32 apart.
template <bool kF32, bool kWide, int kG>
__global__ void __launch_bounds__(32 * kWarps, kF32 ? 2 : 3)
write_fp4_kernel(const Fp4WriteArgs a, const RowMap m) {
    const int lane = threadIdx.x & 31, side = blockIdx.z;
    const float s0 = load_scale(a.scale[0], a.scale_dtype), s1 = load_scale(a.scale[1], a.scale_dtype);
    if (!scale_ok(s0) || !scale_ok(s1)) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && side == 0 && threadIdx.x == 0)
            flag(a.status, KVFP8_DEV_BAD_SCALE);
        return;
    }
    const LayerScale s(side == 0 ? s0 : s1);
    const int g = (blockIdx.y << 5) * kG + (lane & ((1 << m.lpr_log2) - 1));
    const int rpw = 32 >> m.lpr_log2;  // rows a warp takes at a time
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * rpw;
    int64_t t = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * rpw + (lane >> m.lpr_log2);
    // rows the warp's first lane sees (its lanes stay together: groups of four share a store)
    int64_t rounds = (a.num_tokens - (t - (lane >> m.lpr_log2)) + step - 1) / step;
    constexpr int kEsz = kF32 ? 4 : 2;
    const int64_t src_step = step * a.stride[side] * kEsz;
    const uint8_t *src = static_cast<const uint8_t *>(a.src[side]) + t * a.stride[side] * kEsz +
                         static_cast<int64_t>(g) * 16 * kEsz;
    const uint32_t row_codes = static_cast<uint32_t>(m.gpr) * 8;
    uint8_t *codes = a.codes[side] + static_cast<int64_t>(g) * 8;
    // scale bytes of group g: block (slot >> bs_log2), offset (slot & off_mask) of it
    uint8_t *scales = a.scales[side] + (static_cast<int64_t>(g >> m.gph_log2) << (m.bs_log2 + m.gph_log2)) +
                      (g & ((1 << m.gph_log2) - 1));
    const uint32_t block_scales = static_cast<uint32_t>(a.n_kv) << (m.bs_log2 + m.gph_log2);
    const int32_t off_mask = (1 << m.bs_log2) - 1;
    const uint32_t scales_32 = 32u << m.bs_log2;  // 32 groups further

    // The slot of row t (-1: not written).  A row is written when its slot is in range; -1 is
    // padding, anything else is flagged.
    const int64_t *slots = a.slot_mapping;
    auto slot_at = [&](int64_t i) -> int32_t {
        if (i >= a.num_tokens) return -1;
        const int64_t sl = __ldg(slots + i);
        if (sl >= 0 && sl < a.num_slots) return static_cast<int32_t>(sl);
        if (sl != -1 && g == 0 && side == 0) flag(a.status, KVFP8_DEV_BAD_SLOT);
        return -1;
    };
    auto load_row = [&](const uint8_t *p, int32_t slot, Group16<kF32> (&x)[kG]) {
#pragma unroll
        for (int k = 0; k < kG; ++k)
            if (slot >= 0 && g + 32 * k < m.gpr) x[k].template load<kWide>(p + k * 512 * kEsz);
    };
    int32_t slot = slot_at(t), slot_next = slot_at(t + step);
    Group16<kF32> cur[kG], nxt[kG];
    load_row(src, slot, cur);
    for (; rounds > 0; --rounds) {
        src += src_step;
        load_row(src, slot_next, nxt);
        t += step;
        const int32_t slot_after = slot_at(t + step);
        uint8_t *c_row = codes + static_cast<uint64_t>(static_cast<uint32_t>(slot)) * row_codes;
        uint8_t *s_row = scales + static_cast<uint64_t>(static_cast<uint32_t>(slot >> m.bs_log2)) * block_scales +
                         ((slot & off_mask) << m.gph_log2);
#pragma unroll
        for (int k = 0; k < kG; ++k) {
            const bool write = slot >= 0 && g + 32 * k < m.gpr;
            uint32_t byte = 0;
            if (write) *reinterpret_cast<uint2 *>(c_row + k * 256) = quantize16<kF32>(cur[k], s, byte);
            // four groups' scale bytes (of one head: it has 4, 8 or 16 groups) leave as one word
            byte |= __shfl_down_sync(0xFFFFFFFFu, byte, 1) << 8;
            byte |= __shfl_down_sync(0xFFFFFFFFu, byte, 2) << 16;
            if (write && (lane & 3) == 0) *reinterpret_cast<uint32_t *>(s_row + k * scales_32) = byte;
            cur[k] = nxt[k];
        }
        slot = slot_next;
        slot_next = slot_after;
    }
}

// Rows by slot, dequantized: the reader of the layout above, with the same split of a row.
template <bool kBF16Out, int kG>
__global__ void __launch_bounds__(32 * kWarps)
read_fp4_kernel(const Fp4ReadArgs a, const RowMap m, const int32_t wide) {
    const int lane = threadIdx.x & 31;
    const float s = load_scale(a.scale, a.scale_dtype);
    if (!scale_ok(s)) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) flag(a.status, KVFP8_DEV_BAD_SCALE);
        return;
    }
    const int g = (blockIdx.y << 5) * kG + (lane & ((1 << m.lpr_log2) - 1));
    if (g >= m.gpr) return;
    const int rpw = 32 >> m.lpr_log2;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * rpw;
    int64_t t = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * rpw + (lane >> m.lpr_log2);
    constexpr int kBytes = 16 * (kBF16Out ? 2 : 4);
    const int64_t row_bytes = static_cast<int64_t>(m.gpr) * kBytes;
    uint8_t *dst = static_cast<uint8_t *>(a.dst) + t * row_bytes + static_cast<int64_t>(g) * kBytes;
    const uint32_t row_codes = static_cast<uint32_t>(m.gpr) * 8;
    const uint8_t *codes = a.codes + static_cast<int64_t>(g) * 8;
    const uint8_t *scales = a.scales + (static_cast<int64_t>(g >> m.gph_log2) << (m.bs_log2 + m.gph_log2)) +
                            (g & ((1 << m.gph_log2) - 1));
    const uint32_t block_scales = static_cast<uint32_t>(a.n_kv) << (m.bs_log2 + m.gph_log2);
    const int32_t off_mask = (1 << m.bs_log2) - 1;
    const uint32_t scales_32 = 32u << m.bs_log2;  // 32 groups further

    // the slot of row t; -1 (and, flagged, anything out of range): the row reads as zeros
    auto slot_at = [&](int64_t i) -> int32_t {
        if (i >= a.num_tokens) return -1;
        const int64_t sl = __ldg(a.slot_mapping + i);
        if (sl >= 0 && sl < a.num_slots) return static_cast<int32_t>(sl);
        if (sl != -1 && g == 0) flag(a.status, KVFP8_DEV_BAD_SLOT);
        return -1;
    };
    auto fetch = [&](int32_t slot, uint2 (&c)[kG], uint32_t (&b)[kG]) {
        const uint8_t *cp = codes + static_cast<uint64_t>(static_cast<uint32_t>(slot)) * row_codes;
        const uint8_t *sp = scales + static_cast<uint64_t>(static_cast<uint32_t>(slot >> m.bs_log2)) * block_scales +
                            ((slot & off_mask) << m.gph_log2);
#pragma unroll
        for (int k = 0; k < kG; ++k) {
            c[k] = make_uint2(0u, 0u);
            b[k] = 0u;
            if (slot >= 0 && g + 32 * k < m.gpr) {
                c[k] = __ldg(reinterpret_cast<const uint2 *>(cp + k * 256));
                b[k] = __ldg(sp + k * scales_32);
            }
        }
    };
    int32_t slot_next = slot_at(t + step);
    uint2 c[kG], c_next[kG];
    uint32_t b[kG], b_next[kG];
    fetch(slot_at(t), c, b);
    for (; t < a.num_tokens; t += step, dst += step * row_bytes) {
        fetch(slot_next, c_next, b_next);
        slot_next = slot_at(t + 2 * step);
#pragma unroll
        for (int k = 0; k < kG; ++k) {
            const float d = __fmul_rn(e4m3_value(b[k]), s);
            uint32_t h[8], o[16];
            f16x2_from_e2m1x8(c[k].x, *reinterpret_cast<uint32_t(*)[4]>(h));
            f16x2_from_e2m1x8(c[k].y, *reinterpret_cast<uint32_t(*)[4]>(h + 4));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
                const float lo = __fmul_rn(v.x, d), hi = __fmul_rn(v.y, d);
                if (kBF16Out) {
                    o[i] = bf16x2_from_f32(lo, hi);
                } else {
                    o[2 * i] = __float_as_uint(lo);
                    o[2 * i + 1] = __float_as_uint(hi);
                }
            }
            if (g + 32 * k < m.gpr) {
                uint8_t *p = dst + k * 32 * kBytes;
#pragma unroll
                for (int i = 0; i < kBytes / 4; i += 8) {
                    if (wide) {
                        st_v8(p + 4 * i, o + i);
                    } else {
                        *reinterpret_cast<uint4 *>(p + 4 * i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        *reinterpret_cast<uint4 *>(p + 4 * i + 16) =
                            make_uint4(o[i + 4], o[i + 5], o[i + 6], o[i + 7]);
                    }
                }
            }
            c[k] = c_next[k];
            b[k] = b_next[k];
        }
    }
}

int log2_of(int32_t x) {  // of a power of two
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

RowMap row_map(int32_t n_kv, int32_t head_dim, int32_t block_size) {
    RowMap m;
    m.gpr = n_kv * (head_dim / 16);
    m.lpr_log2 = 0;
    while (m.lpr_log2 < 5 && (1 << m.lpr_log2) < m.gpr) ++m.lpr_log2;
    m.gph_log2 = log2_of(head_dim / 16);
    m.bs_log2 = log2_of(block_size);
    return m;
}

// CTAs along x: one wave of resident warps over all passes and sides, fewer for few rows
int rows_grid(int64_t tokens, const RowMap &m, int sms, int occ, int planes) {
    const int64_t rows_per_cta = static_cast<int64_t>(kWarps) * (32 >> m.lpr_log2);
    const int64_t want = (tokens + rows_per_cta - 1) / rows_per_cta;
    const int64_t wave = std::max<int64_t>(1, static_cast<int64_t>(sms) * occ / planes);
    return static_cast<int>(std::min(want, wave));
}

bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

template <bool kF32, bool kWide, int kG>
cudaError_t run_write(const Fp4WriteArgs &a, const RowMap &m, cudaStream_t stream) {
    DeviceFacts f;
    cudaError_t err = device_facts(&f);
    if (err != cudaSuccess) return err;
    auto kern = write_fp4_kernel<kF32, kWide, kG>;
    int occ = 0;
    if ((err = kernel_occupancy(kern, 32 * kWarps, 0, &occ)) != cudaSuccess) return err;
    const int passes = (m.gpr + 32 * kG - 1) / (32 * kG);
    const dim3 grid(rows_grid(a.num_tokens, m, f.sms, std::max(occ, 1), 2 * passes), passes, 2);
    kern<<<grid, 32 * kWarps, 0, stream>>>(a, m);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_reshape_and_cache_fp4(const Fp4WriteArgs &a, cudaStream_t stream) {
    const RowMap m = row_map(a.n_kv, a.head_dim, a.block_size);
    const bool f32 = a.src_dtype == KVFP8_F32;
    const int esz = f32 ? 4 : 2;
    const bool wide = aligned32(a.src[0]) && aligned32(a.src[1]) && a.stride[0] * esz % 32 == 0 &&
                      a.stride[1] * esz % 32 == 0;
    if (m.gpr <= 32) {
        if (f32) return wide ? run_write<true, true, 1>(a, m, stream) : run_write<true, false, 1>(a, m, stream);
        return wide ? run_write<false, true, 1>(a, m, stream) : run_write<false, false, 1>(a, m, stream);
    }
    if (f32) return wide ? run_write<true, true, 2>(a, m, stream) : run_write<true, false, 2>(a, m, stream);
    return wide ? run_write<false, true, 2>(a, m, stream) : run_write<false, false, 2>(a, m, stream);
}

cudaError_t launch_dequant_fp4(const Fp4ReadArgs &a, cudaStream_t stream) {
    DeviceFacts f;
    cudaError_t err = device_facts(&f);
    if (err != cudaSuccess) return err;
    const RowMap m = row_map(a.n_kv, a.head_dim, a.block_size);
    const bool bf16 = a.dst_dtype == KVFP8_BF16, two = m.gpr > 32;
    const int passes = (m.gpr + (two ? 63 : 31)) / (two ? 64 : 32);
    auto kern = bf16 ? (two ? read_fp4_kernel<true, 2> : read_fp4_kernel<true, 1>)
                     : (two ? read_fp4_kernel<false, 2> : read_fp4_kernel<false, 1>);
    int occ = 0;
    if ((err = kernel_occupancy(kern, 32 * kWarps, 0, &occ)) != cudaSuccess) return err;
    const dim3 grid(rows_grid(a.num_tokens, m, f.sms, std::max(occ, 1), passes), passes);
    kern<<<grid, 32 * kWarps, 0, stream>>>(a, m, aligned32(a.dst) ? 1 : 0);
    return cudaGetLastError();
}

}  // namespace kvfp8
