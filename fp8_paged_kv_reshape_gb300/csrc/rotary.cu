// Rotary positions on query and key heads, sm_103a.
//
// The pair j of a head (dims j and j + rot/2, or 2j and 2j+1) is turned by the angle
// position * frequency_j, both members scaled by `magnitude`; dims from rot on pass through:
//   a' = magnitude * (a cos - b sin),   b' = magnitude * (a sin + b cos)
//
// The angle is taken in turns as a 64-bit fraction: F = frequency / 2 pi in units of 2^-64 turn (its
// whole turns dropped, which positions being whole numbers allow), and position * F modulo 2^64
// drops the whole turns of the product exactly.  What is left is off by at most |position| * 2^-64 turn: far positions
// are as exact as near ones, at one 64-bit multiplication per pair and token.  The nearest quarter turn is
// then split off as an integer and sinpif / cospif see |x| <= 1/4.
//
// HBM-bound: each element is read and written once.  A warp takes a token's heads (or a part of them when
// there are few tokens): its lanes share out the token's sines over shared memory once, then each lane
// keeps the cosines and sines of its eight pairs in registers over all the heads.  Measured: 32768 tokens of 40 heads of 128
// bf16 122 us, 5.5 TB/s (the same accesses without the arithmetic take as long); 256 tokens 5.8 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvfp8_device.cuh"
#include "kvfp8_internal.h"

namespace kvfp8 {
namespace {

constexpr int kRotWarps = 8;
constexpr int kMaxPairs = 128;  // of a head (head_dim <= 256)

// (turns_of's shift: below 2^54)
__device__ __forceinline__ bool frequency_ok(double f) {
    return (static_cast<uint64_t>(__double_as_longlong(f)) >> 52 & 0x7FFu) < 1023u + 54u;
}

// frequency (radians a position) -> 2^-64 turns a position, whole turns dropped, within one unit: its 53 bits
// times 1 / 2 pi as a 128-bit fraction, shifted to where the exponent says.  (By float64 arithmetic the FP64
// pipe was busy for 16 us of each call: 2 results a clock and SM.)
__device__ __forceinline__ uint64_t turns_of(double f) {
    const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
    const int e = max(static_cast<int>((bits >> 52) & 0x7FFu), 1);
    uint64_t m = bits & ((1ull << 52) - 1);
    if ((bits >> 52) & 0x7FFu) m |= 1ull << 52;  // f = m 2^(e - 1075)
    constexpr uint64_t kHi = 0xA2F9836E4E441529ull, kLo = 0xFC2757D1F534DDC0ull;  // 2^66 / 2 pi, 128 bits
    uint64_t hi = __umul64hi(m, kHi);
    const uint64_t part = __umul64hi(m, kLo), lo = m * kHi + part;
    hi += lo < part;
    const int s = 1077 - e;  // the product, as 2^-64 turns, is (hi, lo) >> s
    uint64_t t = 0;
    if (s >= 64)
        t = s < 128 ? hi >> (s - 64) : 0;
    else if (s > 0)
        t = hi << (64 - s) | lo >> s;
    return bits >> 63 ? 0 - t : t;
}

// cosine and sine of phase * 2^-64 turns
__device__ __forceinline__ float2 cos_sin(uint64_t phase) {
    const uint64_t r = phase + (1ull << 61);
    const int quarter = static_cast<int>(r >> 62);
    const int64_t rest = static_cast<int64_t>(r & ((1ull << 62) - 1)) - (1ll << 61);  // within an eighth of a turn
    const float x = static_cast<float>(static_cast<int32_t>(rest >> 30)) * 0x1p-33f;   // half turns
    const float s = sinpif(x), c = cospif(x);
    const bool swap = quarter & 1;
    float cc = swap ? s : c, ss = swap ? c : s;
    if (quarter == 1 || quarter == 2) cc = -cc;
    if (quarter >= 2) ss = -ss;
    return make_float2(cc, ss);
}

// eight consecutive elements as floats, and back
template <bool kF32>
struct Eight {
    uint4 w[kF32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *p) {
#pragma unroll
        for (int i = 0; i < (kF32 ? 2 : 1); ++i) w[i] = static_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void store(void *p) const {
#pragma unroll
        for (int i = 0; i < (kF32 ? 2 : 1); ++i) static_cast<uint4 *>(p)[i] = w[i];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        if constexpr (kF32) {
            const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
        } else {
            const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = bf16lo(u[i]);
                f[2 * i + 1] = bf16hi(u[i]);
            }
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        if constexpr (kF32) {
            w[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
            w[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
        } else {
            w[0] = make_uint4(bf16x2_from_f32(f[0], f[1]), bf16x2_from_f32(f[2], f[3]), bf16x2_from_f32(f[4], f[5]),
                              bf16x2_from_f32(f[6], f[7]));
        }
    }
};

// One warp item: token `item / splits`, part `item % splits` of its heads.
template <bool kF32, bool kInterleaved>
__global__ void __launch_bounds__(32 * kRotWarps) rotary_kernel(const RotaryArgs a, int splits, int heads_per_split) {
    constexpr int kEsz = kF32 ? 4 : 2;
    constexpr int kBatch = kF32 ? 2 : 4;  // units of a lane in flight
    __shared__ float2 table[kRotWarps][kMaxPairs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pairs = a.rot / 2, units = a.rot / 16;  // a unit is eight pairs of a head
    const int at_once = 32 / units;                   // heads of a pass
    const int unit = lane % units, first = lane / units;
    const bool active = lane < at_once * units;
    const int heads = a.heads[0] + a.heads[1];
    uint64_t turns[kMaxPairs / 32];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kMaxPairs / 32; ++i) {
        const double f = lane + 32 * i < pairs ? a.frequencies[lane + 32 * i] : 0.;
        turns[i] = turns_of(f);
        bad |= !frequency_ok(f);
    }
    if (bad) flag(a.status, KVFP8_DEV_BAD_SCALE);
    const bool any_bad = __any_sync(0xFFFFFFFFu, bad);

    const int64_t items = a.num_tokens * splits, step = static_cast<int64_t>(gridDim.x) * kRotWarps;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * kRotWarps + warp; item < items; item += step) {
        const int64_t token = item / splits;
        const int h_lo = static_cast<int>(item - token * splits) * heads_per_split;
        const int h_hi = min(heads, h_lo + heads_per_split);
        const int64_t pos = a.positions[token];
        if (pos <= -(1ll << 31) || pos >= (1ll << 31)) {
            if (lane == 0) flag(a.status, KVFP8_DEV_BAD_SLOT);
            continue;
        }
        auto src = [&](int h, int dim) {  // dim of head h
            const int side = h >= a.heads[0];
            return static_cast<const char *>(a.src[side]) +
                   (token * a.stride[side] + (h - (side ? a.heads[0] : 0)) * a.head_dim + dim) * kEsz;
        };
        auto dst = [&](int h, int dim) {
            const int side = h >= a.heads[0];
            return static_cast<char *>(a.dst[side]) +
                   (token * a.dst_stride[side] + (h - (side ? a.heads[0] : 0)) * a.head_dim + dim) * kEsz;
        };
        const int d0 = kInterleaved ? 16 * unit : 8 * unit, d1 = kInterleaved ? d0 + 8 : d0 + a.rot / 2;
        Eight<kF32> x[kBatch][2];
        auto fetch = [&](int h0) {
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int h = h0 + b * at_once;
                if (active && h < h_hi) {
                    x[b][0].load(src(h, d0));
                    x[b][1].load(src(h, d1));
                }
            }
        };
        fetch(h_lo + first);
        __syncwarp();  // the previous item's table has been read
#pragma unroll
        for (int i = 0; i < kMaxPairs / 32; ++i)
            if (lane + 32 * i < pairs) {
                const float2 cs = cos_sin(static_cast<uint64_t>(pos) * turns[i]);
                table[warp][lane + 32 * i] = make_float2(cs.x * a.magnitude, cs.y * a.sin_magnitude);
            }
        if (any_bad)  // a pair without an angle becomes NaN (its frequency is looked up again: no register is spent on it)
            for (int i = lane; i < pairs; i += 32)
                if (!frequency_ok(a.frequencies[i])) table[warp][i] = make_float2(__uint_as_float(0x7FC00000u), __uint_as_float(0x7FC00000u));
        __syncwarp();
        float c[8], s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 cs = table[warp][8 * unit + j];
            c[j] = cs.x;
            s[j] = cs.y;
        }
        for (int h0 = h_lo + first; h0 < h_hi; h0 += kBatch * at_once) {
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int h = h0 + b * at_once;
                if (!active || h >= h_hi) continue;
                float p[8], q[8];
                x[b][0].get(p);
                x[b][1].get(q);
                if constexpr (kInterleaved) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float e = p[2 * j], o = p[2 * j + 1], g = q[2 * j], k = q[2 * j + 1];
                        p[2 * j] = fmaf(e, c[j], -o * s[j]);
                        p[2 * j + 1] = fmaf(e, s[j], o * c[j]);
                        q[2 * j] = fmaf(g, c[j + 4], -k * s[j + 4]);
                        q[2 * j + 1] = fmaf(g, s[j + 4], k * c[j + 4]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float e = p[j], o = q[j];
                        p[j] = fmaf(e, c[j], -o * s[j]);
                        q[j] = fmaf(e, s[j], o * c[j]);
                    }
                }
                x[b][0].set(p);
                x[b][1].set(q);
                x[b][0].store(dst(h, d0));
                x[b][1].store(dst(h, d1));
            }
            if (h0 + kBatch * at_once < h_hi) fetch(h0 + kBatch * at_once);
        }
        // dims that are not rotated, eight at a time
        const int rest = (a.head_dim - a.rot) / 8;
        for (int u = lane; u < rest * (h_hi - h_lo); u += 32) {
            const int h = h_lo + u / rest, d = a.rot + u % rest * 8;
            Eight<kF32> w;
            w.load(src(h, d));
            w.store(dst(h, d));
        }
    }
}

template <bool kF32, bool kInterleaved>
cudaError_t run_rotary(const RotaryArgs &a, cudaStream_t stream) {
    DeviceFacts f;
    cudaError_t err = device_facts(&f);
    if (err != cudaSuccess) return err;
    auto kern = rotary_kernel<kF32, kInterleaved>;
    int occ = 0;
    if ((err = kernel_occupancy(kern, 32 * kRotWarps, 0, &occ)) != cudaSuccess) return err;
    // few tokens: their heads go to several warps, a pass of heads at least to each
    const int heads = a.heads[0] + a.heads[1], at_once = 32 / (a.rot / 16);
    const int64_t warps = static_cast<int64_t>(f.sms) * std::max(occ, 1) * kRotWarps;
    const int most = (heads + at_once - 1) / at_once;
    const int splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, warps / std::max<int64_t>(a.num_tokens, 1))));
    const int per = (heads + splits - 1) / splits;
    const int used = (heads + per - 1) / per;
    const int64_t items = a.num_tokens * used;
    const int64_t ctas = std::min<int64_t>((items + kRotWarps - 1) / kRotWarps, static_cast<int64_t>(f.sms) * std::max(occ, 1));
    kern<<<static_cast<unsigned>(ctas), 32 * kRotWarps, 0, stream>>>(a, used, per);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a, cudaStream_t stream) {
    if (a.dtype == KVFP8_F32)
        return a.interleaved ? run_rotary<true, true>(a, stream) : run_rotary<true, false>(a, stream);
    return a.interleaved ? run_rotary<false, true>(a, stream) : run_rotary<false, false>(a, stream);
}

}  // namespace kvfp8
