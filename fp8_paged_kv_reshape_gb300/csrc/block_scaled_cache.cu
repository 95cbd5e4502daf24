// The FP8 cache with a scale per block and kv head, sm_103a: rows written (the scales are made as they
// are written) and read back by slot.
//
// Writing.  A block's new scale takes the largest element of all of this call's rows in the block, so the
// rows of a block have to be found first: they may stand anywhere in the call.
//  * Calls of up to kDirectTokens rows: a CTA per row looks through slot_mapping for the other rows of its
//    row's block, and goes on if its row's offset is the lowest.  One launch.
//  * Longer ones: mark_rows_kernel leaves row_of[slot] = row for every row.  Nothing initializes row_of: a row that
//    it names counts only if slot_mapping of that row is the slot, which holds for the rows of this call alone, whatever
//    was there before.  find_blocks_kernel lets the row of a block's lowest offset check the block's
//    entries of row_of (-1 for those that do not count) and list the block; persistent grids of write_blocks_kernel
//    take the listed blocks.
// The unit of work is a (block, side, kv head), by one warp, or by a team of warps where the block has more rows of the
// call than a warp's registers hold (and part by part, what the team's do not): rows into registers, their maximum
// (of the integer bits: a positive float's order is its bits' order), the scale, the codes.  A scale made here is a
// power of two, so x / s is an exact multiplication, and when a later call raises it the block's older codes are
// multiplied by a power of two and lose nothing but what leaves the bottom of E4M3's range.
// Rows are read once (those past a team's registers, but for the last part, again from L2).  What bounds it: the loads' latency
// and the arithmetic of the codes, in turn, with the 24 warps an SM that registers leave (DRAM 53 % busy, issue 54 %); calls of a few
// thousand rows, their launches.  Measured, 32768 rows of 8 heads of 128 bf16, K and V: in blocks of 16 43 us for all
// three launches, of 256 68; a side read back 16 (6.2 TB/s, HBM-bound).  256 rows 8 us in one launch, behind one another.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvfp8_block_scale.cuh"
#include "kvfp8_device.cuh"
#include "kvfp8_internal.h"

namespace kvfp8 {
namespace {

constexpr int kWarps = 8;           // of a CTA
constexpr int kDirectTokens = 512;  // rows up to which slot_mapping is searched instead of row_of

// between the kernels of a long call (programmatic dependent launches)
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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
    static constexpr int kPieces = kF32 ? 2 : 1;
    uint4 v[kPieces];
    __device__ __forceinline__ void load(const char *p) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    // the largest magnitude's bits (bf16: in either half)
    __device__ __forceinline__ uint32_t top(uint32_t m) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            if constexpr (kF32)
                m = max(max(max(m, v[i].x & 0x7FFFFFFFu), max(v[i].y & 0x7FFFFFFFu, v[i].z & 0x7FFFFFFFu)), v[i].w & 0x7FFFFFFFu);
            else
                m = __vmaxu2(__vmaxu2(m, v[i].x & 0x7FFF7FFFu),
                             __vmaxu2(__vmaxu2(v[i].y & 0x7FFF7FFFu, v[i].z & 0x7FFF7FFFu), v[i].w & 0x7FFF7FFFu));
        }
        return m;
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (kF32) {
            const uint4 &q = v[i / 4];
            return __uint_as_float(i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w);
        } else {
            const uint32_t w = i / 2 == 0 ? v[0].x : i / 2 == 1 ? v[0].y : i / 2 == 2 ? v[0].z : v[0].w;
            return i % 2 ? bf16hi(w) : bf16lo(w);
        }
    }
    // the codes of these times inv, the inverse of a power of two (the products are the quotients)
    __device__ __forceinline__ uint2 codes(float inv) const {
        return make_uint2(codes4(__fmul_rn(at(0), inv), __fmul_rn(at(1), inv), __fmul_rn(at(2), inv), __fmul_rn(at(3), inv)),
                          codes4(__fmul_rn(at(4), inv), __fmul_rn(at(5), inv), __fmul_rn(at(6), inv), __fmul_rn(at(7), inv)));
    }
    // the codes of the NaN among these: the element's sign and 0x7F
    __device__ __forceinline__ void sign_nan(uint2 &w) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = __float_as_uint(at(i));
            if ((b & 0x7FFFFFFFu) > 0x7F800000u) {
                uint32_t &word = i < 4 ? w.x : w.y;
                word = (word & ~(0xFFu << (8 * (i % 4)))) | (0x7Fu | (b >> 31) << 7) << (8 * (i % 4));
            }
        }
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

// passes of 32 lanes x 8 elements that a warp holds: 4 KB
template <bool kF32>
__host__ __device__ constexpr int passes() { return kF32 ? 4 : 8; }
template <int HD, bool kF32>
__host__ __device__ constexpr int warp_rows() { return 32 / (HD / 8) * passes<kF32>(); }

constexpr int kMostHeld = 32;  // rows of 64 bf16
constexpr int kMostRows = 256;  // of a block

// Shared memory of the teams.
struct TeamTops {
    uint32_t all[kWarps], finite[kWarps];
    // a team's rows (offset, row): kMostHeld to a warp on its own, a block's to the others, which are kWarps / 2 at most
    int2 rows[kWarps / 2 * kMostRows];
    static_assert(kWarps * kMostHeld <= kWarps / 2 * kMostRows, "rows");
};

// A (block, side, head) and the team that has it.
struct Task {
    const char *src;         // this lane's eight dims of row 0
    uint8_t *codes;          // of the block's first token
    float *scale;
    const int32_t *list;     // the block's rows by offset, -1 = none
    const int2 *rows;        // those that there are (offset, row), one after the other
    int count;
    int64_t row_bytes;       // of src
    int32_t code_row;        // bytes from token to token
    int bs;
    int team, team_warps, tw, lane;

    // the maximum over the team's warps of one of each
    __device__ __forceinline__ uint32_t team_max(uint32_t v, uint32_t *slots) const {
        v = __reduce_max_sync(0xFFFFFFFFu, v);
        if (team_warps > 1) {
            if (lane == 0) slots[team * team_warps + tw] = v;
            team_sync(team, team_warps);
            for (int w = 0; w < team_warps; ++w) v = max(v, slots[team * team_warps + w]);
            team_sync(team, team_warps);  // (read before it is written again)
        }
        return v;
    }

    // The block's new scale for rows of this maximum (0: none, what the block holds has no meaning), with its older codes
    // under that.
    template <int HD>
    __device__ __forceinline__ float rescale(uint32_t top, float stored, uint32_t *status) const {
        const float old = list[0] >= 0 ? 0.f : stored;  // the first token starts the block anew
        if (old != 0.f && !block_scale_ok(old)) {
            if (lane == 0 && tw == 0) flag(status, KVFP8_DEV_BAD_SCALE);
            return 0.f;
        }
        const float s = fmaxf(old, power_for(top));
        if (lane == 0 && tw == 0 && s != stored) *scale = s;
        if (s == old || old == 0.f) return s;
        round_older<HD>(old * block_scale_inverse(s));  // (exact, or below 2^-126, where all codes go to 0)
        return s;
    }

    // The block's codes that the call does not write, times factor.
    template <int HD>
    __device__ __forceinline__ void round_older(float factor) const {
        constexpr int kPieces = HD / 16, kBatch = 4;
        const int step = 32 * team_warps;
        for (int u = tw * 32 + lane; u < bs * kPieces; u += kBatch * step) {
            uint4 v[kBatch];
            uint4 *at[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int o = (u + b * step) / kPieces;
                at[b] = o < bs && list[o] < 0
                            ? reinterpret_cast<uint4 *>(codes + static_cast<int64_t>(o) * code_row + (u + b * step) % kPieces * 16)
                            : nullptr;
                if (at[b] != nullptr) v[b] = *at[b];
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (at[b] == nullptr) continue;
                uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2 lo = h2(f16x2_from_e4m3x2(w[i])), hi = h2(f16x2_from_e4m3x2_hi(w[i]));
                    const uint32_t nan = nan_byte_mask(w[i]), was = w[i];
                    w[i] = codes4(__fmul_rn(__low2float(lo), factor), __fmul_rn(__high2float(lo), factor),
                                  __fmul_rn(__low2float(hi), factor), __fmul_rn(__high2float(hi), factor));
                    w[i] = (w[i] & ~nan) | (was & nan);  // a NaN code stays as it is
                }
                *at[b] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }

    // The rows' codes under s, any elements; rows are read, a few at a time.
    template <int HD, bool kF32>
    __device__ __forceinline__ void write_codes(float s) const {
        constexpr int kLanes = HD / 8, kRows = 32 / kLanes, kBatch = 4;
        const float inv = block_scale_inverse(s);
        const int step = team_warps * kRows;
        for (int e = tw * kRows + lane / kLanes; e < count; e += kBatch * step) {
            Elems<kF32> x[kBatch];
            int2 at[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                at[b] = e + b * step < count ? rows[e + b * step] : make_int2(0, -1);
                x[b].zero();
                if (at[b].y >= 0) x[b].load(src + at[b].y * row_bytes);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (at[b].y < 0) continue;
                uint2 w = x[b].codes(inv);
                x[b].sign_nan(w);
                *reinterpret_cast<uint2 *>(codes + static_cast<int64_t>(at[b].x) * code_row + lane % kLanes * 8) = w;
            }
        }
    }

    // The whole task, for rows that the team's registers do not hold or that have an infinity or NaN (the finite
    // elements decide the scale then).
    template <int HD, bool kF32>
    __device__ __noinline__ void write_streamed(float stored, uint32_t *slots, uint32_t *status) const {
        constexpr int kLanes = HD / 8, kRows = 32 / kLanes, kBatch = 4;
        uint32_t top = 0;
        const int step = team_warps * kRows;
        for (int e = tw * kRows + lane / kLanes; e < count; e += kBatch * step) {
            Elems<kF32> x[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                x[b].zero();
                if (e + b * step < count) x[b].load(src + rows[e + b * step].y * row_bytes);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) top = x[b].finite_top(top);
        }
        finish<HD, kF32>(team_max(top, slots), stored, status);
    }

    // What follows the maximum, for any scale.
    template <int HD, bool kF32>
    __device__ __noinline__ void finish(uint32_t top, float stored, uint32_t *status) const {
        const float s = rescale<HD>(top, stored, status);
        if (s != 0.f) write_codes<HD, kF32>(s);
    }
};

// first: the lane's entry of list (-1 past its end)
// kParts: rows past what the team's registers hold are taken part by part, and read twice.
template <int HD, bool kF32, bool kParts>
__device__ __forceinline__ void write_task(const BlockWriteArgs &a, TeamTops &tops, int64_t block, const int32_t *list,
                                           int task, int team, int team_warps, int tw, int lane, int first) {
    constexpr int kEsz = kF32 ? 4 : 2;
    constexpr int kLanes = HD / 8;      // lanes of a row
    constexpr int kRows = 32 / kLanes;  // rows of a pass
    constexpr int kPasses = passes<kF32>();
    const int side = task >= a.n_kv, head = task - (side ? a.n_kv : 0);
    Task t;
    t.src = static_cast<const char *>(a.src[side]) + (static_cast<int64_t>(head) * HD + lane % kLanes * 8) * kEsz;
    t.codes = a.codes[side] + ((block << a.block_shift) * a.n_kv + head) * HD;
    t.scale = a.scales[side] + block * a.scale_stride + head;
    t.list = list;
    t.row_bytes = a.stride[side] * kEsz;
    t.code_row = a.n_kv * HD;
    t.bs = 1 << a.block_shift;
    t.team = team;
    t.team_warps = team_warps;
    t.tw = tw;
    t.lane = lane;
    const float stored = *t.scale;
    // The block's rows, one after the other: each warp looks at all of them and stores its share.
    static_assert(warp_rows<HD, kF32>() <= kMostHeld, "rows");
    const int most = team_warps == 1 ? kMostHeld : kMostRows;
    int2 *rows = tops.rows + team * most;
    int count = 0;
    team_sync(team, team_warps);  // (the last task's have been read)
    for (int o0 = 0; o0 < t.bs; o0 += 32) {
        const int j = o0 == 0 ? first : o0 + lane < t.bs ? list[o0 + lane] : -1;
        const unsigned there = __ballot_sync(0xFFFFFFFFu, j >= 0);
        const int at = count + __popc(there & ((1u << lane) - 1u));
        if (j >= 0 && at < most && o0 / 32 % team_warps == tw) rows[at] = make_int2(o0 + lane, j);
        count += __popc(there);
    }
    team_sync(team, team_warps);
    t.rows = rows;
    t.count = count;
    // the registers hold a part of the rows at a time; pass p of this warp in part c: the lane's row (x: its offset, y:
    // itself, -1 = none)
    const int held = team_warps * warp_rows<HD, kF32>(), last = kParts ? (count - 1) / held : 0;
    auto row = [&](int c, int p) {
        const int e = c * held + (p * team_warps + tw) * kRows + lane / kLanes;
        return e < count ? rows[e] : make_int2(0, -1);
    };
    Elems<kF32> x[kPasses];
    auto load = [&](int c) {
        int j[kPasses];
#pragma unroll
        for (int p = 0; p < kPasses; ++p) j[p] = row(c, p).y;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            x[p].zero();
            if (j[p] >= 0) x[p].load(t.src + j[p] * t.row_bytes);
        }
    };
    uint32_t top = 0x7F800000u;
    if (kParts || count <= held) {
        top = 0;
#pragma unroll 1
        for (int c = 0; c <= last; ++c) {
            load(c);
#pragma unroll
            for (int p = 0; p < kPasses; ++p) top = x[p].top(top);
        }
        if (!kF32) top = max(top & 0xFFFFu, top >> 16) << 16;
        top = t.team_max(top, tops.all);
    }
    if (top >= 0x7F800000u) {
        t.write_streamed<HD, kF32>(stored, tops.finite, a.status);
        return;
    }
    // A block that starts anew, or whose scale holds the new rows; others (older codes to round again, a scale that
    // is not valid) read their rows again.
    const float old = list[0] >= 0 ? 0.f : stored, s = fmaxf(old, power_for(top));
    if (old != 0.f && !(s == old && block_scale_ok(old))) {
        t.finish<HD, kF32>(top, stored, a.status);
        return;
    }
    if (lane == 0 && tw == 0 && s != stored) *t.scale = s;
    const float inv = block_scale_inverse(s);
    auto store = [&](int c) {
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            const int2 at = row(c, p);
            if (at.y >= 0)
                *reinterpret_cast<uint2 *>(t.codes + static_cast<int64_t>(at.x) * t.code_row + lane % kLanes * 8) =
                    x[p].codes(inv);
        }
    };
    store(last);
    if constexpr (kParts) {
#pragma unroll 1
        for (int c = last - 1; c >= 0; --c) {  // from L2
            load(c);
            store(c);
        }
    }
}

// ---------------------------------------------------------------- short calls

// CTA x: row x, if it leads its block; CTAs y share the block's tasks out.  Four CTAs an SM leave 64 registers, which spill 16 to 40
// bytes in every instance; three leave 80, where only float rows spill.  One bf16 row of each of 256 sequences 5.2 us so and 5.5 with
// three, 256 rows of whole blocks 4.9 and 4.6, a single row 2.8 and 2.5.
template <int HD, bool kF32>
__global__ void __launch_bounds__(32 * kWarps, 4) write_rows_kernel(const __grid_constant__ BlockWriteArgs a) {
    __shared__ int32_t list[256];
    __shared__ TeamTops tops;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bs = 1 << a.block_shift, n = static_cast<int>(a.num_tokens);
    const int i = static_cast<int>(blockIdx.x);
    const int64_t slot = a.slot_mapping[i];
    int64_t others[kDirectTokens / (32 * kWarps)];  // slots of rows threadIdx.x + 256 k
#pragma unroll
    for (int k = 0; k < kDirectTokens / (32 * kWarps); ++k) {
        const int j = static_cast<int>(threadIdx.x) + 32 * kWarps * k;
        others[k] = j < n ? a.slot_mapping[j] : -1;
    }
    list[threadIdx.x] = -1;
    if (slot < 0 || slot >= a.num_slots) {
        if (slot != -1 && threadIdx.x == 0 && blockIdx.y == 0) flag(a.status, KVFP8_DEV_BAD_SLOT);
        return;
    }
    __syncthreads();
    const int64_t block = slot >> a.block_shift, slot0 = block << a.block_shift;
#pragma unroll
    for (int k = 0; k < kDirectTokens / (32 * kWarps); ++k)
        if (others[k] >= slot0 && others[k] < slot0 + bs)  // (of a slot named twice, its last row)
            atomicMax(&list[others[k] - slot0], static_cast<int>(threadIdx.x) + 32 * kWarps * k);
    __syncthreads();
    const int off = static_cast<int>(slot - slot0);
    int rows = 0;  // of the block
    bool leads = list[off] == i;
    for (int o = 0; o < bs; o += 32) {
        const bool there = o + lane < bs && list[o + lane] >= 0;
        rows += __popc(__ballot_sync(0xFFFFFFFFu, there));
        if (__any_sync(0xFFFFFFFFu, there && o + lane < off)) leads = false;
    }
    if (!leads) return;
    // a warp to a task, unless the rows there are fill several
    constexpr int kHeld = warp_rows<HD, kF32>();
    int team_warps = 1;
    if (rows > kHeld)
        while (team_warps < kWarps && team_warps * kHeld < rows) team_warps *= 2;
    const int teams = kWarps / team_warps, team = warp / team_warps;
    for (int task = static_cast<int>(blockIdx.y) * teams + team; task < 2 * a.n_kv; task += static_cast<int>(gridDim.y) * teams)
        write_task<HD, kF32, false>(a, tops, block, list, task, team, team_warps, warp % team_warps, lane, lane < bs ? list[lane] : -1);
}

// ---------------------------------------------------------------- long calls

// The workspace: row_of [num_slots], then the listed blocks [num_blocks], those whose rows a warp holds from the
// front, the others from the back, then the number of either.
__device__ __forceinline__ int32_t *listed_blocks(const BlockWriteArgs &a) { return a.row_of + a.num_slots; }
__device__ __forceinline__ int32_t *listed_counts(const BlockWriteArgs &a) {
    return listed_blocks(a) + (a.num_slots >> a.block_shift);
}

__global__ void __launch_bounds__(256) mark_rows_kernel(const __grid_constant__ BlockWriteArgs a) {
    pdl_trigger();  // the next kernel may be launched; it waits for what this one writes
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i < 2) listed_counts(a)[i] = 0;
    if (i >= a.num_tokens) return;
    const int64_t slot = a.slot_mapping[i];
    if (slot >= 0 && slot < a.num_slots)
        a.row_of[slot] = static_cast<int32_t>(i);
    else if (slot != -1)
        flag(a.status, KVFP8_DEV_BAD_SLOT);
}

// A warp takes rows_per_warp (at most 32) rows; those whose slot does not follow the slot of the row before may lead a
// block.
__global__ void __launch_bounds__(256) find_blocks_kernel(const __grid_constant__ BlockWriteArgs a, int held, int rows_per_warp) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t n = a.num_tokens;
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * rows_per_warp + lane;
    const int bs = 1 << a.block_shift;
    const bool mine = lane < rows_per_warp && i < n;
    const int64_t slot = mine ? a.slot_mapping[i] : -1, before = mine && i > 0 ? a.slot_mapping[i - 1] : -1;
    const bool may = slot >= 0 && slot < a.num_slots && ((slot & (bs - 1)) == 0 || before != slot - 1);
    for (unsigned left = __ballot_sync(0xFFFFFFFFu, may); left != 0u; left &= left - 1u) {
        const int from = __ffs(left) - 1;
        const int64_t s = __shfl_sync(0xFFFFFFFFu, slot, from);
        const int row = static_cast<int>(__shfl_sync(0xFFFFFFFFu, i, from));
        const int64_t slot0 = s & ~static_cast<int64_t>(bs - 1);
        constexpr int kMost = 8;  // 32 offsets each
        int j[kMost];
#pragma unroll
        for (int k = 0; k < kMost; ++k) j[k] = 32 * k + lane < bs ? a.row_of[slot0 + 32 * k + lane] : -1;
        int64_t names[kMost];  // the slot of the row that an entry names
#pragma unroll
        for (int k = 0; k < kMost; ++k)
            names[k] = static_cast<uint32_t>(j[k]) < static_cast<uint32_t>(n) ? a.slot_mapping[j[k]] : -1;
        int first = -1, rows = 0;  // the row at the lowest offset
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
            const bool counts = names[k] == slot0 + 32 * k + lane;
            const unsigned there = __ballot_sync(0xFFFFFFFFu, counts);
            const int row_k = __shfl_sync(0xFFFFFFFFu, j[k], there != 0u ? __ffs(there) - 1 : 0);
            if (rows == 0 && there != 0u) first = row_k;
            rows += __popc(there);
        }
        if (first != row) continue;
#pragma unroll
        for (int k = 0; k < kMost; ++k)
            if (32 * k + lane < bs && names[k] != slot0 + 32 * k + lane) a.row_of[slot0 + 32 * k + lane] = -1;
        if (lane == 0) {
            const int many = rows > held;
            const int at = atomicAdd(&listed_counts(a)[many], 1);
            listed_blocks(a)[many ? (a.num_slots >> a.block_shift) - 1 - at : at] = static_cast<int32_t>(slot0 >> a.block_shift);
        }
    }
}

// The listed blocks: those whose rows a warp holds, or (kMany, where blocks have room for more) the others, by teams.
// (A kernel each: with both in one, neither had the registers that it needs.  Three CTAs of the first an SM: 88 us for 32768
// rows and their read-back, 103 with four, whose 64 registers spill, 90 with two.)
template <int HD, bool kF32, bool kMany>
__global__ void __launch_bounds__(32 * kWarps, kMany ? 2 : 3) write_blocks_kernel(const __grid_constant__ BlockWriteArgs a, int team_warps) {
    __shared__ TeamTops tops;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const int tasks = 2 * a.n_kv, bs = 1 << a.block_shift;
    const int32_t *blocks = listed_blocks(a);
    const int num_blocks = static_cast<int>(a.num_slots >> a.block_shift), count = listed_counts(a)[kMany];
    int w = kMany ? 2 : 1;  // warps of a team: as many as hold the rows of such a block, on average at most
    if (kMany)
        while (w < team_warps && static_cast<int64_t>(w) * warp_rows<HD, kF32>() * count < a.num_tokens) w *= 2;
    const int teams = kWarps / w, team = warp / w;
    const int step = static_cast<int>(gridDim.x) * teams, start = static_cast<int>(blockIdx.x) * teams + team;
    // item (block of the list, task); the block's number and its rows are fetched two items and one ahead: each load's
    // address comes from the one before
    struct Item {
        int at, task;
    };
    auto next = [&](Item i) {
        i.at += step / tasks;
        i.task += step % tasks;
        if (i.task >= tasks) {
            i.task -= tasks;
            ++i.at;
        }
        return i;
    };
    auto block_of = [&](const Item &i) { return i.at < count ? blocks[kMany ? num_blocks - 1 - i.at : i.at] : 0; };
    auto list_of = [&](int block) { return a.row_of + (static_cast<int64_t>(block) << a.block_shift); };
    auto first_of = [&](const Item &i, int block) { return i.at < count && lane < bs ? list_of(block)[lane] : -1; };
    Item item = {start / tasks, start % tasks}, item1 = next(item);
    int block = block_of(item), block1 = block_of(item1), first = first_of(item, block);
#pragma unroll 1
    while (item.at < count) {
        const Item item2 = next(item1);
        const int block2 = block_of(item2), first1 = first_of(item1, block1);
        write_task<HD, kF32, kMany>(a, tops, block, list_of(block), item.task, team, kMany ? w : 1, kMany ? warp % w : 0, lane, first);
        item = item1, item1 = item2;
        block = block1, block1 = block2, first = first1;
    }
}

// ---------------------------------------------------------------- rows read back

// A thread takes 16 codes of a row at a time, kUnits of them in flight.  kWide: 32-byte stores.
template <bool kBF16, bool kWide>
__global__ void __launch_bounds__(256) read_blocks_kernel(const BlockReadArgs a) {
    constexpr int kUnits = 4;
    const uint32_t pieces = static_cast<uint32_t>(a.n_kv) * a.head_dim / 16;  // of a row
    const int64_t units = a.num_tokens * pieces, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    int64_t u = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    int64_t row = u / pieces;
    uint32_t piece = static_cast<uint32_t>(u - row * pieces);
    const int64_t row_step = step / pieces;
    const uint32_t piece_step = static_cast<uint32_t>(step - row_step * pieces);
    while (u < units) {
        int64_t slot[kUnits];
        uint32_t at[kUnits];
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            slot[k] = -1;
            at[k] = piece;
            if (u + k * step < units) {
                slot[k] = __ldg(a.slot_mapping + row);
                if (slot[k] < -1 || slot[k] >= a.num_slots) {
                    if (piece == 0) flag(a.status, KVFP8_DEV_BAD_SLOT);
                    slot[k] = -1;
                }
            }
            row += row_step;
            piece += piece_step;
            if (piece >= pieces) {
                piece -= pieces;
                ++row;
            }
        }
        uint4 c[kUnits];
        float s[kUnits];
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            c[k] = make_uint4(0u, 0u, 0u, 0u);
            s[k] = 1.f;
            if (slot[k] >= 0) {
                c[k] = __ldg(reinterpret_cast<const uint4 *>(a.codes) + slot[k] * pieces + at[k]);
                s[k] = __ldg(a.scales + (slot[k] >> a.block_shift) * a.scale_stride + (at[k] >> a.head_shift));
            }
        }
#pragma unroll
        for (int k = 0; k < kUnits; ++k, u += step) {
            if (u >= units) break;
            if (!block_scale_ok(s[k])) {
                flag(a.status, KVFP8_DEV_BAD_SCALE);
                c[k] = make_uint4(0u, 0u, 0u, 0u);
                s[k] = 1.f;
            }
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
            uint8_t *p = static_cast<uint8_t *>(a.dst) + u * (kBF16 ? 32 : 64);
#pragma unroll
            for (int i = 0; i < (kBF16 ? 8 : 16); i += 8) {
                if (kWide) {
                    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + 4 * i), "r"(o[i]),
                                 "r"(o[i + 1]), "r"(o[i + 2]), "r"(o[i + 3]), "r"(o[i + 4]), "r"(o[i + 5]), "r"(o[i + 6]),
                                 "r"(o[i + 7])
                                 : "memory");
                } else {
                    *reinterpret_cast<uint4 *>(p + 4 * i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    *reinterpret_cast<uint4 *>(p + 4 * i + 16) = make_uint4(o[i + 4], o[i + 5], o[i + 6], o[i + 7]);
                }
            }
        }
    }
}

template <int HD, bool kF32>
cudaError_t run_write(const BlockWriteArgs &a, cudaStream_t stream) {
    DeviceFacts f;
    cudaError_t err = device_facts(&f);
    if (err != cudaSuccess) return err;
    constexpr int kHeld = warp_rows<HD, kF32>();
    if (a.row_of == nullptr) {
        int team = 1;  // warps that a block's rows may fill
        while (team < kWarps && team * kHeld < std::min<int64_t>(a.num_tokens, 1 << a.block_shift)) team *= 2;
        const int64_t most = (2 * a.n_kv * team + kWarps - 1) / kWarps;  // CTAs that a block's tasks fill
        const int y = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({most, 12 * f.sms / a.num_tokens, 65535})));
        write_rows_kernel<HD, kF32><<<dim3(static_cast<unsigned>(a.num_tokens), y), 32 * kWarps, 0, stream>>>(a);
        return cudaGetLastError();
    }
    const unsigned by_row = static_cast<unsigned>((a.num_tokens + 255) / 256);
    mark_rows_kernel<<<by_row, 256, 0, stream>>>(a);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    // (a row that may lead costs a warp two reads one after the other: as many warps as the GPU holds)
    const int rows_per_warp = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(32, a.num_tokens / (32 * f.sms))));
    cfg.gridDim = dim3(static_cast<unsigned>((a.num_tokens + kWarps * rows_per_warp - 1) / (kWarps * rows_per_warp)));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((err = cudaLaunchKernelEx(&cfg, find_blocks_kernel, a, kHeld, rows_per_warp)) != cudaSuccess) return err;
    const int64_t warps = a.num_tokens * 2 * a.n_kv;  // a warp to a row's heads is the most there can be
    // (teams of up to eight: 19788 float rows in blocks of 64 71 us for 59, 32768 in blocks of 256 73 for 68)
    const int team_warps = std::max(1, std::min(4, (1 << a.block_shift) / kHeld));
    auto launch = [&](auto kern) {
        int occ = 0;
        if ((err = kernel_occupancy(kern, 32 * kWarps, 0, &occ)) != cudaSuccess) return err;
        const int64_t ctas = std::min<int64_t>((warps + kWarps - 1) / kWarps, static_cast<int64_t>(f.sms) * std::max(occ, 1));
        cfg.gridDim = dim3(static_cast<unsigned>(ctas));
        return cudaLaunchKernelEx(&cfg, kern, a, team_warps);
    };
    if ((err = launch(write_blocks_kernel<HD, kF32, false>)) != cudaSuccess || team_warps == 1) return err;
    return launch(write_blocks_kernel<HD, kF32, true>);
}

}  // namespace

size_t block_write_workspace_size(int64_t num_tokens, int32_t num_blocks, int32_t block_size) {
    if (num_tokens <= kDirectTokens) return 0;
    return (static_cast<size_t>(num_blocks) * block_size + num_blocks + 2) * sizeof(int32_t);
}

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
    const bool wide = (reinterpret_cast<uintptr_t>(a.dst) & 31u) == 0;
    auto kern = a.dst_dtype == KVFP8_BF16 ? (wide ? read_blocks_kernel<true, true> : read_blocks_kernel<true, false>)
                                          : (wide ? read_blocks_kernel<false, true> : read_blocks_kernel<false, false>);
    int occ = 0;
    if ((err = kernel_occupancy(kern, 256, 0, &occ)) != cudaSuccess) return err;
    const int64_t units = a.num_tokens * a.n_kv * (a.head_dim / 16);
    const int64_t ctas = std::min<int64_t>((units + 255) / 256, static_cast<int64_t>(f.sms) * std::max(occ, 1));
    kern<<<static_cast<unsigned>(ctas), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kvfp8
