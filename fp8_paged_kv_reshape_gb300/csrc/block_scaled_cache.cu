// The FP8 cache with a scale per block and kv head, sm_103a: rows written (the scales are made as they
// are written) and read back by slot.
//
// Writing.  A block's new scale takes the largest element of all of this call's rows in the block, so the
// rows of a block have to be found first: they may stand anywhere in the call.  A first kernel leaves
// row_of[slot] = row for every row; nothing initializes row_of, because a row that it names counts only if
// slot_mapping of that row is the slot, which holds exactly for the rows of this call whatever was there
// before.  Of a block's rows the one with the lowest offset leads; the CTA that meets it writes the block.
// (Calls of up to kDirectTokens rows look through slot_mapping instead: one launch.)
//
// A team of one to eight warps takes a (block, side, kv head): rows into registers, their maximum (of the
// integer bits: a positive float's order is its bits' order), the scale, the codes.  A scale made here is a
// power of two, so x / s is a multiplication, exact; and when a later call raises it, the
// block's older codes are multiplied by a power of two and lose nothing but what leaves the bottom of E4M3's
// range.  HBM-bound: rows are read once (blocks whose rows exceed a team's registers are read again, from L2).
#include <cuda_runtime.h>

#include <algorithm>

#include "kvfp8_block_scale.cuh"
#include "kvfp8_device.cuh"
#include "kvfp8_internal.h"

namespace kvfp8 {
namespace {

constexpr int kWarps = 8;            // of a CTA
constexpr int kDirectTokens = 512;   // rows up to which slot_mapping is searched instead of row_of
constexpr int kPasses = 8;           // 32 * 8 elements each, held by a lane
constexpr int kListWords = 4096;     // row lists of a CTA's leaders

__global__ void __launch_bounds__(256) mark_rows_kernel(const BlockWriteArgs a) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= a.num_tokens) return;
    const int64_t slot = a.slot_mapping[i];
    if (slot >= 0 && slot < a.num_slots) a.row_of[slot] = static_cast<int32_t>(i);
}

// The smallest k >= kMinScaleExp with 448 * 2^k >= a, as that power of two; a's bits, finite and not negative.
__device__ __forceinline__ float power_for(uint32_t bits) {
    // 448 = 1.75 * 2^8 (a denormal a ends at the floor as well)
    const int k = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(k, kMinScaleExp) + 127) << 23);
}

// four floats -> four codes; NaN comes out as 0x7F
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    return e4m3x2_from_f32(a, b) | e4m3x2_from_f32(c, d) << 16;
}

// `warps` warps of the CTA, number `id` of such teams, meet
__device__ __forceinline__ void team_sync(int id, int warps) {
    if (warps == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(32 * warps) : "memory");
}

// eight elements of a row, in 16 bytes (bf16) or 32 (float)
template <bool kF32>
struct Elems {
    uint32_t w[kF32 ? 8 : 4];
    __device__ __forceinline__ void load(const char *p) {
#pragma unroll
        for (int i = 0; i < (kF32 ? 2 : 1); ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (kF32 ? 8 : 4); ++i) w[i] = 0u;
    }
    // the largest magnitude's bits (bf16: in either half)
    __device__ __forceinline__ uint32_t top(uint32_t m) const {
#pragma unroll
        for (int i = 0; i < (kF32 ? 8 : 4); ++i)
            m = kF32 ? max(m, w[i] & 0x7FFFFFFFu) : __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        return m;
    }
    __device__ __forceinline__ float at(int i) const {
        if (kF32) return __uint_as_float(w[i]);
        return i & 1 ? bf16hi(w[i / 2]) : bf16lo(w[i / 2]);
    }
    // the largest finite magnitude's float bits
    __device__ __forceinline__ uint32_t finite_top(uint32_t m) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = __float_as_uint(at(i)) & 0x7FFFFFFFu;
            if (b < 0x7F800000u) m = max(m, b);
        }
        return m;
    }
};

template <int HD, bool kF32>
__global__ void __launch_bounds__(32 * kWarps) write_blocks_kernel(const BlockWriteArgs a, int rows_per_cta, int team_warps) {
    constexpr int kEsz = kF32 ? 4 : 2;
    constexpr int kLanes = HD / 8;         // lanes of a row
    constexpr int kRows = 32 / kLanes;     // rows of a pass
    extern __shared__ int32_t lists[];     // [rows_per_cta][block_size]: the leaders' rows by offset, -1 = none
    __shared__ int64_t leader[128];        // their blocks
    __shared__ int num_leaders;
    __shared__ uint32_t team_top[kWarps], team_odd[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bs = 1 << a.block_shift, n = static_cast<int>(a.num_tokens);
    if (threadIdx.x == 0) num_leaders = 0;
    __syncthreads();

    // the rows that lead a block, and their blocks' rows
    const int row0 = static_cast<int>(blockIdx.x) * rows_per_cta;
    for (int r = warp; r < rows_per_cta && row0 + r < n; r += kWarps) {
        const int i = row0 + r;
        const int64_t slot = a.slot_mapping[i];
        if (slot < 0 || slot >= a.num_slots) {
            if (slot != -1 && lane == 0 && blockIdx.y == 0) flag(a.status, KVFP8_DEV_BAD_SLOT);
            continue;
        }
        const int64_t block = slot >> a.block_shift, slot0 = block << a.block_shift;
        const int off = static_cast<int>(slot - slot0);
        if (off > 0 && i > 0 && a.slot_mapping[i - 1] == slot - 1) continue;  // a lower offset is written
        int32_t *list = lists + r * bs;
        if (a.row_of == nullptr) {
            for (int o = lane; o < bs; o += 32) list[o] = -1;
            __syncwarp();
            for (int j = lane; j < n; j += 32) {
                const int64_t s = a.slot_mapping[j];
                if (s >= slot0 && s < slot0 + bs) atomicMax(&list[s - slot0], j);
            }
            __syncwarp();
        }
        bool lower = false;
        for (int o = lane; o < bs; o += 32) {
            int j;
            if (a.row_of == nullptr) {
                j = list[o];
            } else {
                j = a.row_of[slot0 + o];
                if (static_cast<uint32_t>(j) >= static_cast<uint32_t>(n) || a.slot_mapping[j] != slot0 + o) j = -1;
                list[o] = j;
            }
            lower |= o < off && j >= 0;
        }
        __syncwarp();
        if (!__any_sync(0xFFFFFFFFu, lower) && list[off] == i && lane == 0) {
            const int k = atomicAdd(&num_leaders, 1);
            leader[k] = static_cast<int64_t>(r) << 32 | block;
        }
    }
    __syncthreads();

    const int teams = kWarps / team_warps, team = warp / team_warps, tw = warp % team_warps;
    const int tasks = 2 * a.n_kv;
    const int col = lane % kLanes;  // the lane's eight dims
    const int per_round = team_warps * kRows * kPasses;
    const int rounds = (bs + per_round - 1) / per_round;
    for (int li = 0; li < num_leaders; ++li) {
        const int64_t block = leader[li] & 0xFFFFFFFF;
        const int32_t *list = lists + (leader[li] >> 32) * bs;
        const bool anew = list[0] >= 0;
        for (int task = static_cast<int>(blockIdx.y) * teams + team; task < tasks; task += static_cast<int>(gridDim.y) * teams) {
            const int side = task >= a.n_kv, head = task - (side ? a.n_kv : 0);
            float *scale_at = a.scales[side] + block * a.scale_stride + head;
            const float old = anew ? 0.f : *scale_at;
            const char *src = static_cast<const char *>(a.src[side]) + (static_cast<int64_t>(head) * HD + col * 8) * kEsz;
            const int64_t row_bytes = a.stride[side] * kEsz;
            uint8_t *codes = a.codes[side] + ((block << a.block_shift) * a.n_kv + head) * HD;
            const int64_t code_row = static_cast<int64_t>(a.n_kv) * HD;

            Elems<kF32> x[kPasses];
            auto offset = [&](int round, int p) { return ((round * kPasses + p) * team_warps + tw) * kRows + lane / kLanes; };
            auto fetch = [&](int round) {
#pragma unroll
                for (int p = 0; p < kPasses; ++p) {
                    const int o = offset(round, p);
                    const int j = o < bs ? list[o] : -1;
                    if (j >= 0)
                        x[p].load(src + j * row_bytes);
                    else
                        x[p].zero();
                }
            };
            uint32_t top = 0;
            for (int round = 0; round < rounds; ++round) {
                fetch(round);
#pragma unroll
                for (int p = 0; p < kPasses; ++p) top = x[p].top(top);
            }
            if (!kF32) top = max(top & 0xFFFFu, top >> 16) << 16;
            top = __reduce_max_sync(0xFFFFFFFFu, top);
            if (team_warps > 1) {
                if (lane == 0) team_top[warp] = top;
                team_sync(team, team_warps);
                for (int w = 0; w < team_warps; ++w) top = max(top, team_top[team * team_warps + w]);
                team_sync(team, team_warps);  // (read before it is written again)
            }
            const bool odd = top >= 0x7F800000u;  // an infinity or NaN somewhere: the finite elements decide
            if (odd) {
                top = 0;
                for (int round = 0; round < rounds; ++round) {
                    if (rounds > 1) fetch(round);
#pragma unroll
                    for (int p = 0; p < kPasses; ++p) top = x[p].finite_top(top);
                }
                top = __reduce_max_sync(0xFFFFFFFFu, top);
                if (team_warps > 1) {
                    if (lane == 0) team_odd[warp] = top;
                    team_sync(team, team_warps);
                    for (int w = 0; w < team_warps; ++w) top = max(top, team_odd[team * team_warps + w]);
                    team_sync(team, team_warps);
                }
            }
            if (old != 0.f && !block_scale_ok(old)) {  // what the block holds has no meaning: left as it is
                if (lane == 0 && tw == 0) flag(a.status, KVFP8_DEV_BAD_SCALE);
                continue;
            }
            const float s = fmaxf(old, power_for(top));
            // 1 / s is exact where s is a power of two (always, but for scales that a user brought)
            const bool power = (__float_as_uint(s) & 0x7FFFFFu) == 0u;
            const float inv = 1.f / s;
            if (lane == 0 && tw == 0 && s != old) *scale_at = s;

            if (s > old && old > 0.f) {  // older codes under the new scale
                const float factor = old * inv;  // (s is a power of two here: exact, or below 2^-126 and all codes go to 0)
                constexpr int kPieces = HD / 16;
                for (int u = tw * 32 + lane; u < bs * kPieces; u += 32 * team_warps) {
                    const int o = u / kPieces;
                    if (list[o] >= 0) continue;
                    uint4 *at = reinterpret_cast<uint4 *>(codes + o * code_row + u % kPieces * 16);
                    const uint4 v = *at;
                    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __half2 lo = h2(f16x2_from_e4m3x2(w[i])), hi = h2(f16x2_from_e4m3x2_hi(w[i]));
                        const uint32_t nan = nan_byte_mask(w[i]), was = w[i];
                        w[i] = codes4(__fmul_rn(__low2float(lo), factor), __fmul_rn(__high2float(lo), factor),
                                      __fmul_rn(__low2float(hi), factor), __fmul_rn(__high2float(hi), factor));
                        w[i] = (w[i] & ~nan) | (was & nan);  // a NaN code stays as it is
                    }
                    *at = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            for (int round = 0; round < rounds; ++round) {
                if (rounds > 1) fetch(round);
#pragma unroll
                for (int p = 0; p < kPasses; ++p) {
                    const int o = offset(round, p);
                    if (o >= bs || list[o] < 0) continue;
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = power ? __fmul_rn(x[p].at(i), inv) : __fdiv_rn(x[p].at(i), s);
                    uint32_t w[2] = {codes4(y[0], y[1], y[2], y[3]), codes4(y[4], y[5], y[6], y[7])};
                    if (odd) {  // NaN: the element's sign and 0x7F
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t b = __float_as_uint(x[p].at(i));
                            if ((b & 0x7FFFFFFFu) > 0x7F800000u) {
                                const uint32_t code = 0x7Fu | (b >> 31) << 7;
                                w[i / 4] = (w[i / 4] & ~(0xFFu << (8 * (i % 4)))) | code << (8 * (i % 4));
                            }
                        }
                    }
                    *reinterpret_cast<uint2 *>(codes + o * code_row + col * 8) = make_uint2(w[0], w[1]);
                }
            }
        }
    }
}

// ---------------------------------------------------------------- rows read back

// A thread takes 16 codes of a row at a time, kUnits of them in flight.
template <bool kBF16>
__global__ void __launch_bounds__(256) read_blocks_kernel(const BlockReadArgs a) {
    constexpr int kUnits = 4;
    const int64_t pieces = static_cast<int64_t>(a.n_kv) * a.head_dim / 16;  // of a row
    const int64_t units = a.num_tokens * pieces, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    const int head_shift = a.head_shift;  // log2(head_dim / 16)
    for (int64_t u0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; u0 < units; u0 += kUnits * step) {
        int64_t slot[kUnits];
        int piece[kUnits];
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int64_t u = u0 + k * step;
            slot[k] = -1;
            if (u < units) {
                const int64_t row = u / pieces;
                piece[k] = static_cast<int>(u - row * pieces);
                slot[k] = a.slot_mapping[row];
                if (slot[k] < -1 || slot[k] >= a.num_slots) {
                    if (piece[k] == 0) flag(a.status, KVFP8_DEV_BAD_SLOT);
                    slot[k] = -1;
                }
            }
        }
        uint4 c[kUnits];
        float s[kUnits];
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            c[k] = make_uint4(0u, 0u, 0u, 0u);
            s[k] = 1.f;
            if (slot[k] >= 0) {
                c[k] = __ldg(reinterpret_cast<const uint4 *>(a.codes) + slot[k] * pieces + piece[k]);
                s[k] = __ldg(a.scales + (slot[k] >> a.block_shift) * a.scale_stride + (piece[k] >> head_shift));
                if (!block_scale_ok(s[k])) {
                    flag(a.status, KVFP8_DEV_BAD_SCALE);
                    c[k] = make_uint4(0u, 0u, 0u, 0u);
                    s[k] = 1.f;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int64_t u = u0 + k * step;
            if (u >= units) break;
            const uint32_t w[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
            uint32_t o[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const __half2 v = h2(i & 1 ? f16x2_from_e4m3x2_hi(w[i / 2]) : f16x2_from_e4m3x2(w[i / 2]));
                const float lo = __fmul_rn(__low2float(v), s[k]), hi = __fmul_rn(__high2float(v), s[k]);
                if (kBF16) {
                    o[i] = bf16x2_from_f32(lo, hi);
                } else {
                    o[2 * i] = __float_as_uint(lo);
                    o[2 * i + 1] = __float_as_uint(hi);
                }
            }
            uint4 *p = static_cast<uint4 *>(a.dst) + u * (kBF16 ? 2 : 4);
#pragma unroll
            for (int i = 0; i < (kBF16 ? 2 : 4); ++i) p[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
    }
}

template <int HD, bool kF32>
cudaError_t run_write(const BlockWriteArgs &a, cudaStream_t stream) {
    DeviceFacts f;
    cudaError_t err = device_facts(&f);
    if (err != cudaSuccess) return err;
    const int bs = 1 << a.block_shift;
    constexpr int kTeamRows = 32 / (HD / 8) * kPasses;
    const int team_warps = std::max(1, std::min(kWarps, bs / kTeamRows));
    // Rows a CTA looks at: 16 of the rows of a long call, one of a few hundred.
    const int rows_per_cta = static_cast<int>(
        std::max<int64_t>(1, std::min<int64_t>(std::min(128, std::max(1, kListWords / bs)), a.num_tokens / (4 * f.sms))));
    const int64_t ctas = (a.num_tokens + rows_per_cta - 1) / rows_per_cta;
    // the (side, head) tasks of a block over several CTAs where there are few blocks
    const int teams = kWarps / team_warps, most = (2 * a.n_kv + teams - 1) / teams;
    const int64_t blocks = std::max<int64_t>(1, a.num_tokens / bs);
    const int y = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({most, 8 * f.sms / blocks, 65535})));
    if (a.row_of != nullptr) {
        mark_rows_kernel<<<static_cast<unsigned>((a.num_tokens + 255) / 256), 256, 0, stream>>>(a);
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
    }
    write_blocks_kernel<HD, kF32><<<dim3(static_cast<unsigned>(ctas), y), 32 * kWarps, rows_per_cta * bs * sizeof(int32_t), stream>>>(
        a, rows_per_cta, team_warps);
    return cudaGetLastError();
}

}  // namespace

bool block_write_needs_rows(int64_t num_tokens) { return num_tokens > kDirectTokens; }

cudaError_t launch_reshape_and_cache_block_scaled(const BlockWriteArgs &a, cudaStream_t stream) {
    const bool f32 = a.src_dtype == KVFP8_F32;
    switch (a.head_dim) {
        case 64: return f32 ? run_write<64, true>(a, stream) : run_write<64, false>(a, stream);
        case 128: return f32 ? run_write<128, true>(a, stream) : run_write<128, false>(a, stream);
        case 256: return f32 ? run_write<256, true>(a, stream) : run_write<256, false>(a, stream);
        default: return cudaErrorNotSupported;
    }
}

cudaError_t launch_dequant_block_scaled(const BlockReadArgs &a, cudaStream_t stream) {
    DeviceFacts f;
    cudaError_t err = device_facts(&f);
    if (err != cudaSuccess) return err;
    auto kern = a.dst_dtype == KVFP8_BF16 ? read_blocks_kernel<true> : read_blocks_kernel<false>;
    int occ = 0;
    if ((err = kernel_occupancy(kern, 256, 0, &occ)) != cudaSuccess) return err;
    const int64_t units = a.num_tokens * a.n_kv * (a.head_dim / 16);
    const int64_t ctas = std::min<int64_t>((units + 255) / 256, static_cast<int64_t>(f.sms) * std::max(occ, 1));
    kern<<<static_cast<unsigned>(ctas), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kvfp8
