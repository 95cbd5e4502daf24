// Attention over the FP8 cache with block scales for long query chunks and wide groups of heads, causal or
// not, sm_103a tensor cores (tcgen05) with accumulators in tensor memory:
//   s_t = sm_scale * ks(block of t) * q . dec(K_t),   out = sum_t softmax(s)_t * vs(block of t) * dec(V_t)
//
// Rows are (query token j, head g of the kv head's group) pairs, row = j*G + g; a CTA takes RT tiles of 128 rows of a
// (sequence, kv head) and goes over their keys in tiles of 128.  What bounds it is the chain of a row tile's scores,
// softmax and product with V, so the work beside it is kept small:
//  * K is not converted.  q is the sum of an E4M3 and an E5M2 number: with q scaled by a power of two per row, so that its largest
//    element lies in [128, 256), a = E4M3(q) leaves q - a of at most 8 of a bf16's last places, which 3 bits hold, so
//    b = E5M2(q - a) makes the sum exact as long as a is a normal number, within 2^13 of the row's largest.  Below, q - a is 2^-10 at
//    most and b off by 2^-14, 2^-21 of the largest.  K tiles arrive by TMA as the operand that the product takes
//    (kind::f8f6f4, twice the rate of f16: two products at half the time), products are exact, sums float.  (With b in E4M3, whose
//    smallest number is 2^-9, q was exact within 2^9 and to 2^-17 of the largest below, at the same times.)
//  * V meets fp16 weights, so it is converted to fp16 (exactly) and transposed: ldmatrix gives a lane four
//    dims of a key, which after the conversion are stored with stmatrix.trans as rows of V^T.
//  * ks multiplies the scores, 16 keys at a time (a block is 16 keys at least), in the multiplication that takes them
//    to the log2 domain.  vs goes into the exponent there: the weights that meet V's codes are 2^(s + log2 vs - m) with
//    m near the highest s + log2 vs that the row sees, within fp16's range whatever the scales, and the row's sum adds 16 keys'
//    weights times 1 / vs.  m lies 2^7 below the highest at the time, weights reach 2^15, so they keep 11 bits down to 2^-21 of
//    the highest and are above zero down to 2^-32.  (V's codes times their scale over the largest of 64 keys', and that one in
//    the exponent, lost what lies far below a scale that the row may not even see.)
//  * A row's 128 scores of a tile are read from tensor memory once and stay in its thread's registers from the maximum to
//    the weights, which takes 184 of them: warpgroups trade registers.  (Read twice, with 128 registers, 512 new
//    tokens of 16 sequences of 4096 took 612 us where this took 485; one pass half by half, whose sums tell when the reference
//    has to move and the half is done again, 587.)
//
// Measured: that case 450 us (778 TFLOP/s, the tensor pipe 38 % busy), 225 queries on 1500 states in 24 sequences, 16 heads
// of 64, 88 us.  A 128-key tile of two row tiles takes 4600 cycles: 2300 of products, 2400 of softmax.
//
// Two row tiles (head_dim 64 and 128, more than 128 rows) share K tiles and the converted V.  Where tensor memory has room for a
// score buffer more than row tiles (all but head_dim 128 with two), the next scores are computed meanwhile.
//
// NaN: a NaN code in K makes the key's scores NaN, which the masks keep from rows that do not see it.  One
// in V may reach all rows where all of them see the key.  Where not (the last tiles of a causal call), such codes are
// taken as 0, the CTA remembers that it met one, and at the end its rows look up which dims of the values
// they see are NaN (a slow scan that no finite cache runs).
//
// Every wait is bounded; one that runs out sets KVFP8_DEV_TIMEOUT, and tensor memory is always released.
#include "kvfp8_block_scale.cuh"
#include "prefill_common.cuh"

namespace kvfp8 {
namespace {

constexpr int kKeys = 128;  // of a tile
constexpr int kHalf = 64;   // V arrives and is converted in halves
constexpr int kConvWarps = 4;
constexpr float kHead = 7.f;  // see above
constexpr float kLag = 8.f;   // log2: how far scores may rise above the highest one when the reference was set

struct BlockPrefillArgs : PrefillCommon {
    const uint8_t *value_cache;
    const float *key_scales, *value_scales;  // [block][scale_stride], a kv head's at its index
    int32_t scale_stride;
    bool causal;  // else every query sees every cached token
    // parts a (sequence, kv head, row tiles)'s keys are cut into at most (gridDim.y), and the parts'
    // results, [CTA of the unsplit grid, in sequence order][part][row]
    int32_t splits;
    float *part_o, *part_lse;
};

template <int HD, int RT>
struct PbSmem {
    static constexpr int kSeg = HD < 128 ? HD : 128, kSegs = HD / kSeg;  // bytes of a TMA box row; of a key's head
    // Score buffers, taken in turns by the jobs (key tile i, row tile r), number RT * i + r.  One more than row tiles where
    // tensor memory has room: scores are ahead of the softmax then.
    static constexpr int kBufs = RT == 2 && HD == 128 ? 2 : RT + 1;
    static constexpr bool kAhead = kBufs > RT;
    static constexpr int kNK = HD == 64 ? 4 : HD == 128 ? 3 : 2;         // K tiles
    static constexpr int kNV = HD == 256 ? 2 : 4;                        // V^T halves
    static constexpr int kNS = HD == 64 ? 4 : HD == 128 ? 3 : 2;         // staged V halves
    // q: a row tile's two parts, 128 rows of [segment][row][kSeg] each
    static constexpr int kPart = 128 * HD;
    static constexpr int kQ = 0;
    static constexpr int kKBuf = kKeys * HD, kK = kQ + RT * 2 * kPart;   // [segment][128 keys][kSeg]
    static constexpr int kVBuf = HD * 128, kV = kK + kNK * kKBuf;        // [HD dims][64 keys] f16
    static constexpr int kStageBuf = kHalf * HD, kStage = kV + kNV * kVBuf;  // [segment][64 keys][kSeg]
    static constexpr int kInfo = kStage + kNS * kStageBuf;               // HalfInfo per V^T half
    static constexpr int kScales = kInfo + 80 * kNV;                     // [side][16 keys] per staged half
    static constexpr int kBars = kScales + 32 * kNS;
    // mbarriers
    static constexpr int kKFull = kBars, kKFree = kKFull + 16 * kNK;     // (a K tile's halves; a K tile)
    static constexpr int kVFull = kKFree + 8 * kNK, kVEmpty = kVFull + 8 * kNS;
    static constexpr int kVReady = kVEmpty + 8 * kNS, kVFree = kVReady + 8 * kNV;
    static constexpr int kQReady = kVFree + 8 * kNV;
    static constexpr int kSReady = kQReady + 8, kPReady = kSReady + 8 * kBufs;  // (per score buffer)
    static constexpr int kODone = kPReady + 8 * kBufs, kDrain = kODone + 32;  // (O of odd and even tiles: two may be under way)
    static constexpr int kMeta = kDrain + 16;                            // valid keys per staged half
    static constexpr int kMisc = kMeta + 8 * kNS;                        // tmem base, abort flag, NaN seen
    static constexpr int kTotal = kMisc + 16;
    static_assert(kTotal + 1024 <= 232448, "shared memory");
    // tensor memory: score buffers of 128 columns, then O of each row tile
    static constexpr uint32_t kTmemCols = 512;
    __host__ __device__ static constexpr uint32_t col_s(int b) { return static_cast<uint32_t>(128 * b); }
    __host__ __device__ static constexpr uint32_t col_o(int r) { return static_cast<uint32_t>(128 * kBufs + HD * r); }
    static_assert(128 * kBufs + RT * HD <= 512, "tensor memory");
};

// What the softmax takes of 64 keys, 16 at a time: scores times kmul (K's scales) and what its row says are in the log2 domain, weights
// carry vlog, their sum vinv (twice: the sum is two floats); the keys that are there.  far, of a tile's second half: the V scales
// so far are more than kSumSpan apart.
struct HalfInfo {
    float4 kmul, vlog, vinv[2];
    uint32_t mask[2], far, pad;
};
static_assert(sizeof(HalfInfo) == 80, "layout");

// P of keys 16k..16k+15 (f16 pairs, 8 columns): the first half of the 32 columns that held the scores of keys
// 32(k/2)..+31, so each 32-key chunk's P overwrites only its own scores
__host__ __device__ constexpr uint32_t col_p(int k) { return static_cast<uint32_t>(32 * (k >> 1) + 8 * (k & 1)); }

// ---------------------------------------------------------------- 8-bit operands

// D (TMEM) (+)= A x B, both 8-bit in shared memory
__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor, kind::f8f6f4: E4M3 or E5M2 A, E4M3 B, fp32 D, both K-major, M x N.
__host__ __device__ constexpr uint32_t f8_idesc(bool e5m2, int m, int n) {
    return (1u << 4) | (e5m2 ? 1u << 7 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
__device__ __forceinline__ uint32_t e5m2x2_from_f32(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Shared-memory matrix descriptor: K-major operand of SEG-byte rows (128 or 64) swizzled over them.
template <int SEG>
__device__ __forceinline__ uint64_t k_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (1ull << 16) |
           (static_cast<uint64_t>((8 * SEG) >> 4) << 32)  // 8 rows
           | (1ull << 46) | (SEG == 128 ? 2ull << 61 : 4ull << 61);
}

// ---------------------------------------------------------------- block scales

// The scales of 64 keys, taken apart by a whole warp: lane l has those of keys 16(l%4)..+15.
struct HalfScales {
    uint64_t keys;  // those whose block has valid scales of both sides
    float k, v;     // the lane's (1 without keys)

    // at: four K scales, then four V scales (stale where a group has no key in mask)
    __device__ __forceinline__ void load(const uint8_t *at, uint64_t mask, int lane) {
        const int g = lane & 3;
        const float ks = *reinterpret_cast<const float *>(at + 4 * g), vs = *reinterpret_cast<const float *>(at + 16 + 4 * g);
        const uint64_t group = mask & (0xFFFFull << (16 * g));
        const bool ok = group != 0ull && block_scale_ok(ks) && block_scale_ok(vs);
        keys = static_cast<uint64_t>(__reduce_or_sync(0xFFFFFFFFu, ok ? static_cast<uint32_t>(group) : 0u)) |
               static_cast<uint64_t>(__reduce_or_sync(0xFFFFFFFFu, ok ? static_cast<uint32_t>(group >> 32) : 0u)) << 32;
        k = ok ? ks : 1.f;
        v = ok ? vs : 1.f;
    }
};

// The dims d0..d0+31 (bit i: d0 + i) in which some value of tokens first..last of the sequence is NaN, for each
// lane's own last (negative: none); blocks out of range or without valid scales hold no tokens.  Called by
// whole warps: the tokens that every lane has are shared out over the lanes, the few after them are each lane's own.
template <int HD>
__device__ __noinline__ uint32_t nan_value_dims(const BlockPrefillArgs &a, int seq, int kvh, int d0, int first, int last) {
    const int32_t *bt = a.block_tables + static_cast<int64_t>(seq) * a.max_blocks_per_seq;
    uint32_t dims = 0;
    auto look = [&](int t) {
        const int32_t blk = bt[t / a.block_size];
        if (blk < 0 || blk >= a.num_blocks) return;
        const int64_t s = static_cast<int64_t>(blk) * a.scale_stride + kvh;
        if (!block_scale_ok(a.key_scales[s]) || !block_scale_ok(a.value_scales[s])) return;
        const uint32_t *row = reinterpret_cast<const uint32_t *>(
            a.value_cache + ((static_cast<int64_t>(blk) * a.block_size + t % a.block_size) * a.n_kv + kvh) * HD + d0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t nan = nan_byte_mask(row[i]) & 0x08040201u;
            dims |= ((nan | nan >> 8 | nan >> 16 | nan >> 24) & 0xFu) << (4 * i);
        }
    };
    const int lane = static_cast<int>(threadIdx.x & 31);
    const int all = __reduce_min_sync(0xFFFFFFFFu, last < 0 ? INT32_MAX : last);  // tokens first..all are every lane's
    if (all != INT32_MAX)
        for (int t = first + lane; t <= all; t += 32) look(t);
    dims = __reduce_or_sync(0xFFFFFFFFu, dims);
    if (last < 0) return 0u;
    for (int t = max(first, all + 1); t <= last; ++t) look(t);
    return dims;
}

// the largest of 16 scores
__device__ __forceinline__ float max16(const uint32_t *s) {
    auto v = [&](int c) { return __uint_as_float(s[c]); };
    const float a = max3f(max3f(v(0), v(1), v(2)), v(3), v(4)), b = max3f(max3f(v(5), v(6), v(7)), v(8), v(9));
    const float c = max3f(max3f(v(10), v(11), v(12)), v(13), v(14));
    return fmaxf(max3f(a, b, c), v(15));
}

// A warp's 32 rows of q (bf16 at q + the lane's row_at, or zeros where the lane has none) as an E4M3 part at part0 and an E5M2 part
// at part1 (rows row..row+31 of K-major operands).  Returns what a score of the lane's row is to be multiplied by.  HD/8 lanes
// share a row.  (A lane to a row took 13000 cycles of a CTA's 160000: lines apart, read twice.)
template <int HD, int SEG>
__device__ __forceinline__ float split_q_rows(const __nv_bfloat16 *q, int64_t row_at, bool row_ok, uint8_t *part0, uint8_t *part1, int row) {
    constexpr int kLanes = HD / 8, kAtOnce = 32 / kLanes, kBatch = 8;
    const int lane = static_cast<int>(threadIdx.x & 31), k = lane % kLanes;
    const uint32_t at = static_cast<uint32_t>((8 * k / SEG) * (128 * SEG) + (k & 1) * 8);
    float down = 1.f;
#pragma unroll 1
    for (int it0 = 0; it0 < kLanes; it0 += kBatch) {
        uint4 w[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int from = (it0 + b) * kAtOnce + lane / kLanes;
            const int64_t src = __shfl_sync(0xFFFFFFFFu, row_at, from);
            const bool there = __shfl_sync(0xFFFFFFFFu, row_ok, from);
            w[b] = there ? reinterpret_cast<const uint4 *>(q + src)[k] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const uint32_t x[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
            uint32_t top = __vmaxu2(__vmaxu2(x[0] & 0x7FFF7FFFu, x[1] & 0x7FFF7FFFu), __vmaxu2(x[2] & 0x7FFF7FFFu, x[3] & 0x7FFF7FFFu));
            top = max(top & 0xFFFFu, top >> 16);  // the largest magnitude's bits
#pragma unroll
            for (int d = 1; d < kLanes; d *= 2) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            // 2^(7 - e) of the largest's exponent e, kept where it and its inverse are floats
            const int e = min(max(static_cast<int>(top >> 7), 20), 254);
            const float up = __uint_as_float(static_cast<uint32_t>(261 - e) << 23);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = bf16lo(x[i]) * up, v = bf16hi(x[i]) * up;
                hi[i] = e4m3x2_from_f32(u, v);
                const float2 back = __half22float2(h2(f16x2_from_e4m3x2(hi[i])));
                lo[i] = e5m2x2_from_f32(u - back.x, v - back.y);
            }
            uint2 a = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            if (top >= 0x7F80u) a = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);  // an infinity or NaN: the whole row becomes NaN
            const uint32_t to = at + swz<SEG>(row + (it0 + b) * kAtOnce + lane / kLanes, 8 * k % SEG / 16);
            *reinterpret_cast<uint2 *>(part0 + to) = a;
            *reinterpret_cast<uint2 *>(part1 + to) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
            const float d = __shfl_sync(0xFFFFFFFFu, __uint_as_float(static_cast<uint32_t>(e - 7) << 23), lane % kAtOnce * kLanes);
            if (it0 + b == lane / kAtOnce) down = d;
        }
    }
    return down;
}

// what a row's scores are multiplied by, of 16 keys and its own (kept away from 0 and infinity, which would make a NaN of
// a score of infinity or 0)
__device__ __forceinline__ float score_mul(float kmul, float qmul) { return fminf(fmaxf(kmul * qmul, 0x1p-126f), 0x1p126f); }

// O of a warp's rows times factor
template <int HD>
__device__ __forceinline__ void scale_o(uint32_t at, float factor) {
#pragma unroll 1
    for (int c0 = 0; c0 < HD; c0 += 16) {
        uint32_t o[16];
        tmem_ld16(at + c0, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
        tmem_st16(at + c0, o);
    }
}

// A row's reference and sum (two fp32 halves); ok: no wait ran out.
struct FarRow {
    float m;
    uint64_t sum2;
    bool ok;
};

// The softmax of tiles i..ntiles - 1 where V scales are too far apart for the sum of weights times 1 / vs (see kSumSpan): 32 keys at a
// time, the sum's terms by themselves.  last: the last key, from the CTA's first tile on, that the row sees (a padding row: any).
// (In the loop that other caches run, behind a branch, this cost their calls 2 to 5 %.)
template <int HD, int RT>
__device__ __noinline__ FarRow far_tiles(uint32_t base, const uint8_t *bp, uint32_t lane_addr, int rt, int i, int ntiles, int rot, int last,
                                         float qmul, FarRow row) {
    using L = PbSmem<HD, RT>;
    const volatile int32_t *abort_flag = reinterpret_cast<const volatile int32_t *>(bp + L::kMisc + 4);
    auto wait = [&](int off, int k, int phase) {
        row.ok = __all_sync(0xFFFFFFFFu, mbar_wait(base + static_cast<uint32_t>(off + 8 * k), static_cast<uint32_t>(phase & 1), abort_flag));
        return row.ok;
    };
#pragma unroll 1
    for (; i < ntiles; ++i) {
        const int job = RT * i + rt, buf = job % L::kBufs, v0 = 2 * i % L::kNV;
        if (!wait(L::kVReady, v0, 2 * i / L::kNV) || !wait(L::kVReady, v0 + 1, 2 * i / L::kNV) || !wait(L::kSReady, buf, job / L::kBufs)) break;
        static_assert(L::kNV % 2 == 0, "a tile's halves are neighbours");
        tc_fence_after();
        const HalfInfo *in = reinterpret_cast<const HalfInfo *>(bp + L::kInfo) + v0;
        const uint32_t scol = lane_addr + L::col_s(buf);
        const int tile = i + rot >= ntiles ? i + rot - ntiles : i + rot;
        const int seen = last == INT32_MAX ? kKeys : last - tile * kKeys + 1;  // keys of the tile up to the row's last
        uint32_t x[32];
        float k[2], v[2];  // of 16 keys each
        auto load = [&](int c) {
            const HalfInfo &half = in[c >> 1];
            const float2 k2 = reinterpret_cast<const float2 *>(&half.kmul)[c & 1], v2 = reinterpret_cast<const float2 *>(&half.vlog)[c & 1];
            k[0] = score_mul(k2.x, qmul), k[1] = score_mul(k2.y, qmul), v[0] = v2.x, v[1] = v2.y;
            const int n = seen - 32 * c;
            const uint32_t bits = half.mask[c & 1] & (n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u);
            tmem_ld32(scol + 32 * c, x);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (!((bits >> e) & 1u)) x[e] = 0xFF800000u;  // -infinity
        };
        float mx = -INFINITY, down = 0.f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            load(c);
            mx = max3f(mx, fmaf(max16(x), k[0], v[0]), fmaf(max16(x + 16), k[1], v[1]));
        }
        if (mx > row.m + (kLag + kHead)) {
            down = row.m == -INFINITY ? 0.f : row.m - (mx - kHead);
            row.m = mx - kHead;
        }
        if (__any_sync(0xFFFFFFFFu, down != 0.f)) {
            if (L::kAhead) {  // (i > 0: the row had a reference)
                if (!wait(L::kODone, 2 * rt + ((i - 1) & 1), (i - 1) >> 1)) break;
                tc_fence_after();
            }
            scale_o<HD>(lane_addr + L::col_o(rt), ex2(down));
            const float root = ex2(0.5f * down);
            row.sum2 = mul_f32x2(mul_f32x2(row.sum2, pk2(root, root)), pk2(root, root));
        }
        const float msub = row.m == -INFINITY ? 0.f : row.m;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            load(c);
            uint32_t p[16];
#pragma unroll
            for (int w = 0; w < 16; ++w) {
                const float a0 = __uint_as_float(x[2 * w]), a1 = __uint_as_float(x[2 * w + 1]), shift = v[w >> 3] - msub;
                p[w] = f16x2_from_f32(ex2(fmaf(a0, k[w >> 3], shift)), ex2(fmaf(a1, k[w >> 3], shift)));
                row.sum2 = add_f32x2(row.sum2, pk2(ex2(fmaf(a0, k[w >> 3], -msub)), ex2(fmaf(a1, k[w >> 3], -msub))));
            }
            tmem_st16(scol + 32 * c, p);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(base + static_cast<uint32_t>(L::kPReady + 8 * buf));
    }
    return row;
}

// ---------------------------------------------------------------- the kernel

// One row tile: 10 warps have 168 registers each, of which the scores take 128, so the softmax looks V's scales up as it needs them, and 50
// to 85 bytes are spilled (128 rows of 8 sequences of 4096 at head_dim 256 152 us).
// Warps: 4 per row tile softmax (warp w reads TMEM lanes 32*(w%4)..+31, a row a thread), 4 converting V, one per
// row tile issuing products (the first allocates TMEM), one issuing copies.  Two row tiles: warpgroups trade registers, 128 a
// thread at the launch, so that the softmax keeps its scores (a warp without work makes up the last group).
template <int HD, int RT>
struct PbWarps {
    static constexpr int kIssue = PbSmem<HD, RT>::kAhead ? 1 : RT;  // threads that issue products
    static constexpr int kConv = 4 * RT, kMma = kConv + kConvWarps, kTma = kMma + kIssue, kAll = kMma + (RT == 2 ? 4 : 2);
    static constexpr int kSoftmaxRegs = 184, kConvRegs = 72, kIssueRegs = 72;
    static_assert(RT != 2 || 256 * kSoftmaxRegs + 128 * kConvRegs + 128 * kIssueRegs <= 512 * 128, "registers at launch");
};
template <int RT, int kRegs>
__device__ __forceinline__ void take_registers() {
    if constexpr (RT == 2) {
        if constexpr (kRegs > 128)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
    }
}

template <int HD, int RT, bool kSplit>
__global__ void __launch_bounds__(PbWarps<HD, RT>::kAll * 32, 1)
prefill_blocks_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                      const __grid_constant__ BlockPrefillArgs a) {
    using L = PbSmem<HD, RT>;
    using W = PbWarps<HD, RT>;
    constexpr int kRows = 128 * RT;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *bp = smem_raw + (base - raw);
    volatile uint64_t *meta = reinterpret_cast<volatile uint64_t *>(bp + L::kMeta);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bp + L::kMisc);
    volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(bp + L::kMisc + 4);
    volatile int32_t *nan_seen = reinterpret_cast<volatile int32_t *>(bp + L::kMisc + 8);
    auto bar = [&](int off, int i) { return base + static_cast<uint32_t>(off + 8 * i); };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // kv head fastest, then row tiles, then sequence (longest first): a (sequence, kv head)'s CTAs run side by side on
    // one K/V stream
    const int kvh = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.n_kv));
    const int ctile = static_cast<int>((blockIdx.x / static_cast<unsigned>(a.n_kv)) % static_cast<unsigned>(a.row_tiles));
    const int rank = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.n_kv * a.row_tiles));
    // (the K tiles are free scratch until the pipeline starts)
    const int seq = seq_of_rank(a.seq_lens, a.num_seqs, a.max_len, rank, reinterpret_cast<uint32_t *>(bp + L::kK));
    const int raw_nq = a.qsl ? a.qsl[seq + 1] - a.qsl[seq] : 1;
    const QueryRange qr = a.qsl ? query_range(a.qsl, seq, a.qmax, a.qrows) : QueryRange{seq, 1};
    const int Lraw = a.seq_lens[seq];
    const int Ls = min(max(Lraw, 0), a.max_len);
    if (ctile == 0 && kvh == 0 && tid == 0 && (!kSplit || blockIdx.y == 0) &&
        (qr.count != raw_nq || Lraw < 0 || Lraw > a.max_len || (a.qsl && a.causal && qr.count > Ls)))
        flag(a.status, KVFP8_DEV_BAD_BLOCK);
    const int nb = qr.count, G = a.group;
    const int row0 = ctile * kRows;  // first row of this CTA
    if (row0 >= nb * G) return;
    const int j_last = min(nb, (row0 + kRows + G - 1) / G) - 1;
    const int kend = a.causal ? Ls - nb + j_last + 1 : Ls;          // keys the CTA's last row may see
    const int all_see = a.causal ? Ls - nb + row0 / G + 1 : Ls;     // (the keys before it every row sees)
    int ntiles = kend > 0 ? (kend + kKeys - 1) / kKeys : 0;
    int tile_lo = 0;  // this CTA's key tiles: ntiles from tile_lo on
    if constexpr (kSplit) {
        const int parts = split_parts(a.splits, ntiles, kKeys);
        const int part = static_cast<int>(blockIdx.y);
        if (part >= parts) return;
        tile_lo = static_cast<int>(static_cast<int64_t>(part) * ntiles / parts);
        ntiles = static_cast<int>(static_cast<int64_t>(part + 1) * ntiles / parts) - tile_lo;
    }
    // each of the row tiles side by side starts its pass at its own key tile (the online softmax takes the keys in any
    // order), so they read different lines of the stream at any one time
    const int rot = ntiles > 0 ? static_cast<int>((static_cast<int64_t>(ctile) * ntiles) / a.row_tiles) % ntiles : 0;
    auto key_tile = [&](int i) { const int k = i + rot; return (k >= ntiles ? k - ntiles : k) + tile_lo; };

    if (ntiles == 0) {  // every row of the CTA sees no key: zero rows
        if (tid < kRows) {
            const int r = row0 + tid;
            if (r < nb * G) {
                uint4 *o = reinterpret_cast<uint4 *>(a.out + ((static_cast<int64_t>(qr.q0) + r / G) * a.n_q + kvh * G + r % G) * HD);
                for (int c = 0; c < HD / 8; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        return;
    }

    if (tid == 0) {
        for (int i = 0; i < L::kNK; ++i) {
            mbar_init(bar(L::kKFull, 2 * i), 1);
            mbar_init(bar(L::kKFull, 2 * i + 1), 1);
            mbar_init(bar(L::kKFree, i), W::kIssue);
        }
        for (int i = 0; i < L::kNS; ++i) {
            mbar_init(bar(L::kVFull, i), 1 + 32);  // the post, and every lane's scale copies
            mbar_init(bar(L::kVEmpty, i), kConvWarps);
        }
        for (int i = 0; i < L::kNV; ++i) {
            mbar_init(bar(L::kVReady, i), kConvWarps);
            mbar_init(bar(L::kVFree, i), W::kIssue);
        }
        mbar_init(bar(L::kQReady, 0), 4 * RT);
        for (int i = 0; i < L::kBufs; ++i) {
            mbar_init(bar(L::kSReady, i), 1);
            mbar_init(bar(L::kPReady, i), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(L::kODone, i), 1);
            mbar_init(bar(L::kODone, 2 + i), 1);
            mbar_init(bar(L::kDrain, i), 1);
        }
        *abort_flag = 0;
        *nan_seen = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == W::kMma) {
        tmem_alloc(base + L::kMisc, L::kTmemCols);
        tmem_relinquish();
    }
    if (warp == W::kTma && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmk)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmv)) : "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const volatile int32_t never = 0;

    if (warp >= W::kMma) {
      take_registers<RT, W::kIssueRegs>();
      if (warp == W::kTma) {
        // ------------------------------------------------------------ copies
        // half h of the key pass (64 keys of tile h/2): lane p < nbox copies K box p, lane nbox + p V box p
        const int32_t *bt = a.block_tables + static_cast<int64_t>(seq) * a.max_blocks_per_seq;
        const int bs = a.block_size, br = a.box_rows;
        const int lbs = __ffs(bs) - 1;
        const int nbox = kHalf / br;
        const bool k_lane = lane < nbox;
        const int p = k_lane ? lane : lane - nbox;
        const bool box_lane = lane < 2 * nbox;
        const CUtensorMap *map = k_lane ? &tmk : &tmv;
        int wbase = -(1 << 30);
        int32_t win = -1;  // the lane's block-table entry of the window from wbase on
        int issued = 0;
        bool aborted = false;
        for (int h = 0; h < 2 * ntiles; ++h) {
            const int i = h >> 1, hf = h & 1, kb = i % L::kNK, st = h % L::kNS;
            const int t0 = key_tile(i) * kKeys + hf * kHalf;
            if (t0 < kend) {
                const int e0 = t0 >> lbs, e1 = (min(kend, t0 + kHalf) - 1) >> lbs;
                if (e0 < wbase || e1 >= wbase + 32) {
                    wbase = e0;
                    win = wbase + lane < a.max_blocks_per_seq ? bt[wbase + lane] : -1;
                }
            }
            // this lane's box: its first key t, the block holding it, and whether it is copied (keys past kend are
            // left out; a bad block is flagged and left out)
            const int t = t0 + p * br;
            const int blk = __shfl_sync(0xFFFFFFFFu, win, ((t >> lbs) - wbase) & 31);
            const bool live = box_lane && t < kend;
            const bool good = live && blk >= 0 && blk < a.num_blocks;
            if (live && !good && k_lane) flag(a.status, KVFP8_DEV_BAD_BLOCK);
            uint64_t part = 0;
            if (good && k_lane) {
                const int nk = min(br, kend - t);
                part = (nk >= 64 ? ~0ull : ((1ull << nk) - 1)) << (p * br);
            }
            const uint64_t mask =
                static_cast<uint64_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(part))) |
                static_cast<uint64_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(part >> 32))) << 32;
            const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, good && k_lane));
            // and its scale: lanes 0-3 the K scales of 16 keys each, 4-7 the V scales
            const int ts = t0 + 16 * (lane & 3);
            const int sblk = __shfl_sync(0xFFFFFFFFu, win, ((ts >> lbs) - wbase) & 31);
            const uint32_t kfull = bar(L::kKFull, 2 * kb + hf), vfull = bar(L::kVFull, st);
            const bool withheld = kWithholdFirstChunk && h == 0;  // (test build: neither copies nor arrivals for the first half)
            if (lane == 0) {
                if ((hf == 0 && !mbar_wait(bar(L::kKFree, kb), ((i / L::kNK) & 1) ^ 1u, abort_flag)) ||
                    !mbar_wait(bar(L::kVEmpty, st), ((h / L::kNS) & 1) ^ 1u, abort_flag)) {
                    aborted = true;
                } else {
                    meta[st] = mask;
                    if (withheld) {
                    } else if (boxes > 0) {
                        mbar_arrive_tx(kfull, static_cast<uint32_t>(boxes * br * HD));
                        mbar_arrive_tx(vfull, static_cast<uint32_t>(boxes * br * HD));
                    } else {
                        mbar_arrive(kfull);
                        mbar_arrive(vfull);
                    }
                    ++issued;
                }
            }
            aborted = __shfl_sync(0xFFFFFFFFu, aborted, 0);
            if (aborted) break;
            __syncwarp();  // what lane 0 waited for (the buffers have been read) holds for every lane's copies
            if (good && !withheld) {  // the expected bytes are posted: each lane with a box copies it
                const int row = blk * bs + (t & (bs - 1));
                const uint32_t dst = k_lane ? base + L::kK + kb * L::kKBuf + static_cast<uint32_t>((hf * kHalf + p * br) * L::kSeg)
                                            : base + L::kStage + st * L::kStageBuf + static_cast<uint32_t>(p * br * L::kSeg);
                const uint32_t seg = static_cast<uint32_t>((k_lane ? kKeys : kHalf) * L::kSeg);
#pragma unroll
                for (int sgi = 0; sgi < L::kSegs; ++sgi)
                    tma_load_3d(dst + sgi * seg, map, 0, kvh * L::kSegs + sgi, row, k_lane ? kfull : vfull);
            }
            if (lane < 8 && ts < kend && sblk >= 0 && sblk < a.num_blocks && !withheld)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(base + L::kScales + 32 * st + 4 * lane),
                             "l"((lane < 4 ? a.key_scales : a.value_scales) + static_cast<int64_t>(sblk) * a.scale_stride + kvh)
                             : "memory");
            if (!withheld) asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(vfull) : "memory");
        }
        if (aborted) asm volatile("cp.async.wait_all;" ::: "memory");
        if (aborted && lane == 0) {
            flag(a.status, KVFP8_DEV_TIMEOUT);
            *abort_flag = 1;
            // let copies already issued land before the CTA's shared memory goes away
            for (int k = max(0, issued - max(L::kNS, 2 * L::kNK)); k < issued; ++k) {
                if (k >= issued - L::kNS) mbar_wait(bar(L::kVFull, k % L::kNS), (k / L::kNS) & 1, &never);
                mbar_wait(bar(L::kKFull, 2 * ((k >> 1) % L::kNK) + (k & 1)), ((k >> 1) / L::kNK) & 1, &never);
            }
        }
      } else if (warp < W::kMma + W::kIssue) {
        // ------------------------------------------------------------ products
        if (lane == 0) {
            const int own = warp - W::kMma;  // its row tile (kAhead: both)
            const uint32_t idesc_s[2] = {f8_idesc(false, 128, kKeys), f8_idesc(true, 128, kKeys)}, idesc_o = f16_idesc(128, HD);
            // operand descriptors computed once; each product adds its constant offset
            const uint64_t qdesc = k_desc<L::kSeg>(base + L::kQ), kdesc = k_desc<L::kSeg>(base + L::kK),
                           vdesc = sw128_desc(base + L::kV);
            auto wait = [&](int off, int i, int phase) {
                if (!mbar_wait(bar(off, i), static_cast<uint32_t>(phase & 1), abort_flag)) return false;
                tc_fence_after();
                return true;
            };
            auto k_there = [&](int i) {
                return wait(L::kKFull, 2 * (i % L::kNK), i / L::kNK) && wait(L::kKFull, 2 * (i % L::kNK) + 1, i / L::kNK);
            };
            auto issue_s = [&](int i, int r, int buf) {  // scores of tile i for row tile r
                const uint64_t kd = desc_at(kdesc, (i % L::kNK) * L::kKBuf);
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int k = 0; k < HD / 32; ++k) {
                        const int seg = 32 * k / L::kSeg, in = 32 * k % L::kSeg;
                        umma_f8(tmem + L::col_s(buf), desc_at(qdesc, (2 * r + part) * L::kPart + seg * (128 * L::kSeg) + in),
                                desc_at(kd, seg * (kKeys * L::kSeg) + in), idesc_s[part], part > 0 || k > 0 ? 1u : 0u);
                    }
                umma_commit(bar(L::kSReady, buf));
                if (!L::kAhead || r == RT - 1) umma_commit(bar(L::kKFree, i % L::kNK));
            };
            auto v_there = [&](int i) {
                return wait(L::kVReady, 2 * i % L::kNV, 2 * i / L::kNV) && wait(L::kVReady, (2 * i + 1) % L::kNV, (2 * i + 1) / L::kNV);
            };
            auto issue_o = [&](int i, int r, int buf) {  // O += P . V of tile i
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int vb = (2 * i + hf) % L::kNV;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_ts(tmem + L::col_o(r), tmem + L::col_s(buf) + col_p(4 * hf + k),
                                desc_at(vdesc, vb * L::kVBuf + k * 32), idesc_o, i > 0 || hf > 0 || k > 0 ? 1u : 0u);
                    if (!L::kAhead || r == RT - 1) umma_commit(bar(L::kVFree, vb));
                }
                umma_commit(bar(L::kODone, 2 * r + (i & 1)));
            };
            bool ok = wait(L::kQReady, 0, 0);
            if constexpr (L::kAhead) {
                // job n: O, then the scores of job n + kBufs into the buffer that P was read from
                const int jobs = RT * ntiles;
                auto scores = [&](int n) {
                    if (n % RT == 0 && !k_there(n / RT)) return false;
                    issue_s(n / RT, n % RT, n % L::kBufs);
                    return true;
                };
                for (int n = 0; n < min(L::kBufs, jobs) && ok; ++n) ok = scores(n);
                for (int n = 0; n < jobs && ok; ++n) {
                    ok = (n % RT != 0 || v_there(n / RT)) && wait(L::kPReady, n % L::kBufs, n / L::kBufs);
                    if (!ok) break;
                    issue_o(n / RT, n % RT, n % L::kBufs);
                    if (n + L::kBufs < jobs) ok = scores(n + L::kBufs);
                }
            } else {
                // O(i), then S(i+1) into the columns that P(i) was read from.  (One thread for both row tiles: 467 us where
                // this takes 446, the one's waits holding up the other's products.)
                ok = ok && k_there(0);
                if (ok) issue_s(0, own, own);
                for (int i = 0; i < ntiles && ok; ++i) {
                    ok = v_there(i) && wait(L::kPReady, own, i);
                    if (!ok) break;
                    issue_o(i, own, own);
                    if (i + 1 < ntiles) {
                        ok = k_there(i + 1);
                        if (ok) issue_s(i + 1, own, own);
                    }
                }
            }
            if (!ok) {
                flag(a.status, KVFP8_DEV_TIMEOUT);
                *abort_flag = 1;
            }
            // tensor memory is released when the products have finished, whoever gave up
            umma_commit(bar(L::kDrain, own));
            mbar_wait(bar(L::kDrain, own), 0, &never);
        }
      }
    } else if (warp >= W::kConv) {
        take_registers<RT, W::kConvRegs>();
        // ------------------------------------------------------------ V -> f16, transposed
        // A unit is 8 keys x 64 dims: one ldmatrix gives a lane four dims of one key in each of four 16-dim pieces; the
        // pairs of dims are stored transposed.  Lanes of the upper half of a key's dims swap their two pairs first, so that
        // the eight rows of V^T that a matrix goes to are different modulo 8 (different banks).
        constexpr int kUnits = 8 * (HD / 64) / kConvWarps;  // of a warp in a half
        const int cw = warp - W::kConv, t4 = lane & 3;
        const uint32_t swap = t4 < 2 ? 0x3210u : 0x1032u;
        // the row of V^T (past 64 dims' first, in the first two pieces) that this lane addresses for a store
        const int m = lane >> 3, c = lane & 7;
        const int store_dim = 16 * (m >> 1) + 4 * (c >> 1) + (c & 1) + 2 * ((m & 1) ^ (c >> 2));
        constexpr int kBatch = kUnits < 4 ? kUnits : 4;  // units whose codes are loaded together
        uint32_t r[kBatch][4];
        auto load = [&](uint32_t stage, int u0) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int un = cw + kConvWarps * (u0 + u), d0 = 64 * (un >> 3);
                const uint32_t addr = stage + static_cast<uint32_t>(d0 / L::kSeg * (kHalf * L::kSeg)) +
                                      swz<L::kSeg>(8 * (un & 7) + (lane & 7), d0 % L::kSeg / 16 + (lane >> 3));
                ldsm_x4(addr, r[u][0], r[u][1], r[u][2], r[u][3]);
            }
        };
        bool ok = true;
        uint32_t vtop = 0, vlow = ~0u;  // bits of the largest and the smallest V scale so far
        for (int h = 0; h < 2 * ntiles && ok; ++h) {
            const int st = h % L::kNS, vb = h % L::kNV;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kVFull, st), (h / L::kNS) & 1, abort_flag));
            if (!ok) break;
            const uint32_t stage = base + L::kStage + st * L::kStageBuf, vt = base + L::kV + vb * L::kVBuf;
            load(stage, 0);
            const uint64_t posted = meta[st];
            HalfScales sc;
            sc.load(bp + L::kScales + 32 * st, posted, lane);
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kVFree, vb), ((h / L::kNV) & 1) ^ 1u, abort_flag));
            if (!ok) break;
            if (cw == 0) {
                const bool has = (sc.keys >> (16 * (lane & 3)) & 0xFFFFull) != 0ull;
                vtop = max(vtop, __reduce_max_sync(0xFFFFFFFFu, has ? __float_as_uint(sc.v) : 0u));
                vlow = min(vlow, __reduce_min_sync(0xFFFFFFFFu, has ? __float_as_uint(sc.v) : ~0u));
            }
            if (cw == 0 && lane < 4) {
                HalfInfo *info = reinterpret_cast<HalfInfo *>(bp + L::kInfo) + vb;
                reinterpret_cast<float *>(&info->kmul)[lane] = sc.k;
                reinterpret_cast<float *>(&info->vlog)[lane] = static_cast<float>(static_cast<int>(__float_as_uint(sc.v) >> 23) - 127);
                const float inv = block_scale_inverse(sc.v);
                reinterpret_cast<float2 *>(info->vinv)[lane] = make_float2(inv, inv);
                if (lane == 0) {
                    if (sc.keys != posted) flag(a.status, KVFP8_DEV_BAD_SCALE);
                    info->mask[0] = static_cast<uint32_t>(sc.keys);
                    info->mask[1] = static_cast<uint32_t>(sc.keys >> 32);
                    info->far = vtop > vlow && (vtop - vlow) >> 23 > kSumSpan;
                }
            }
            const bool drop_nan = key_tile(h >> 1) * kKeys + ((h & 1) + 1) * kHalf > all_see;
#pragma unroll 1
            for (int u0 = 0; u0 < kUnits; u0 += kBatch) {
                if (u0 > 0) load(stage, u0);
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int un = cw + kConvWarps * (u0 + u), ko = un & 7, d0 = 64 * (un >> 3);
                    const bool there = (sc.keys >> (8 * ko + (lane >> 2))) & 1ull;
                    const uint32_t take = there ? swap : 0x4444u;
                    uint32_t f[8];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t w = __byte_perm(r[u][q], 0u, take);
                        if (drop_nan) {
                            const uint32_t nan = nan_byte_mask(w);
                            if (nan != 0u) *nan_seen = 1;
                            w &= ~nan;
                        }
                        f[2 * q] = f16x2_from_e4m3x2(w);
                        f[2 * q + 1] = f16x2_from_e4m3x2_hi(w);
                    }
                    const uint32_t to = vt + sw128(d0 + store_dim, ko);
                    stsm_x4_t(to, f[0], f[1], f[2], f[3]);
                    stsm_x4_t(to + 32 * 128, f[4], f[5], f[6], f[7]);
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(L::kVEmpty, st));
                mbar_arrive(bar(L::kVReady, vb));
            }
        }
        if (!ok && lane == 0) {
            flag(a.status, KVFP8_DEV_TIMEOUT);
            *abort_flag = 1;
        }
    } else {
        // ------------------------------------------------------------ softmax
        take_registers<RT, W::kSoftmaxRegs>();
        const int rt = RT == 2 ? warp >> 2 : 0;     // row tile
        const int r = row0 + tid;                   // this thread's row
        const bool row_ok = r < nb * G;
        const int jq = row_ok ? r / G : 0, gq = row_ok ? r % G : 0;
        const int64_t row_at = ((static_cast<int64_t>(qr.q0) + jq) * a.n_q + kvh * G + gq) * HD;
        const int pos = a.causal ? Ls - nb + jq : Ls - 1;  // last key position the row may see
        uint8_t *qp = bp + L::kQ + rt * 2 * L::kPart;
        // what the row's scores are multiplied by, but for K's scale (which comes last: q's and sm_scale alone stay well inside a float)
        const float qmul = split_q_rows<HD, L::kSeg>(a.query, row_at, row_ok, qp, qp + L::kPart, tid & 96) *
                           (a.sm_scale * 1.4426950408889634f);  // log2(e)
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kQReady, 0));
        const bool idle = row0 + (tid & ~31) >= nb * G;  // a warp of padding rows

        const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        float m_used = -INFINITY;
        uint64_t lsum2 = pk2(0.f, 0.f);  // the row sum, in two fp32 halves
        bool ok = true;
        int i = 0;
        for (; i < ntiles && ok; ++i) {
            const int job = RT * i + rt, buf = job % L::kBufs, turn = job / L::kBufs;
            const int v0 = 2 * i % L::kNV, v1 = (2 * i + 1) % L::kNV;
            const uint32_t scol = lane_addr + L::col_s(buf);
            if (idle) {  // whatever stands there: no other row takes part in these
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kSReady, buf), turn & 1, abort_flag));
                if (ok && lane == 0) mbar_arrive(bar(L::kPReady, buf));
                continue;
            }
            // the halves' keys and scales (stored with their V^T, which is there before the scores as a rule)
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kVReady, v0), (2 * i / L::kNV) & 1, abort_flag) &&
                                             mbar_wait(bar(L::kVReady, v1), ((2 * i + 1) / L::kNV) & 1, abort_flag));
            if (!ok) break;
            const HalfInfo *in[2] = {reinterpret_cast<const HalfInfo *>(bp + L::kInfo) + v0,
                                     reinterpret_cast<const HalfInfo *>(bp + L::kInfo) + v1};
            // the visible keys among columns 32c..32c+31
            const int seen = pos - key_tile(i) * kKeys + 1;  // keys of the tile up to the row's position
            auto visible = [&](int c) {
                const int n = seen - 32 * c;
                const uint32_t bits = in[c >> 1]->mask[c & 1] & (n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u);
                return row_ok ? bits : ~0u;  // (a padding row holds no warp back)
            };
            if (in[1]->far != 0u) break;
            const bool whole = __all_sync(0xFFFFFFFFu, (visible(0) & visible(1) & visible(2) & visible(3)) == ~0u);
            float mul[8], vheld[8];  // of 16 keys each
            // (one row tile: 168 registers do not hold the V scales as well)
            auto vlog = [&](int k) { return RT == 1 ? reinterpret_cast<const volatile float *>(&in[k >> 2]->vlog)[k & 3] : vheld[k]; };
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const float4 k4 = in[hf]->kmul, v4 = in[hf]->vlog;
                mul[4 * hf] = score_mul(k4.x, qmul);
                mul[4 * hf + 1] = score_mul(k4.y, qmul);
                mul[4 * hf + 2] = score_mul(k4.z, qmul);
                mul[4 * hf + 3] = score_mul(k4.w, qmul);
                vheld[4 * hf] = v4.x;
                vheld[4 * hf + 1] = v4.y;
                vheld[4 * hf + 2] = v4.z;
                vheld[4 * hf + 3] = v4.w;
            }
            // (not kAhead: with S(rt, i) O(rt, i-1) is done)
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kSReady, buf), turn & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
            uint32_t s[4][32];  // the row's scores of the tile, read once
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(scol + 32 * c, s[c]);
            tmem_wait_ld();
            if (!whole) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t bits = visible(c);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!((bits >> e) & 1u)) s[c][e] = 0xFF800000u;  // -infinity
                }
            }
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                mx = max3f(mx, fmaf(max16(s[c]), mul[2 * c], vlog(2 * c)), fmaf(max16(s[c] + 16), mul[2 * c + 1], vlog(2 * c + 1)));
            // the reference moves, and O is rescaled, only when the maximum has risen far above it (first visible keys: O
            // is still zero for this row, nothing to rescale)
            float factor = 1.f;
            if (mx > -INFINITY) {
                if (m_used == -INFINITY) {
                    m_used = mx - kHead;
                } else if (mx > m_used + (kLag + kHead)) {
                    factor = ex2(m_used - (mx - kHead));
                    m_used = mx - kHead;
                }
            }
            if (__any_sync(0xFFFFFFFFu, factor != 1.f)) {
                if (L::kAhead) {  // (i > 0: the row had a reference)
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kODone, 2 * rt + ((i - 1) & 1)), ((i - 1) >> 1) & 1, abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                }
                lsum2 = mul_f32x2(lsum2, pk2(factor, factor));
                scale_o<HD>(lane_addr + L::col_o(rt), factor);
            }
            // P = 2^(s + log2 vs - m) as f16 pairs, written over the first half of each 32 scores; its float values are summed
            const float msub = m_used == -INFINITY ? 0.f : m_used;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 inv = in[c >> 1]->vinv[c & 1];
                uint32_t p[16];
                uint64_t sum2[2];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float shift = vlog(2 * c + g) - msub;
                    const uint64_t shift2 = pk2(shift, shift), mul2 = pk2(mul[2 * c + g], mul[2 * c + g]);
                    sum2[g] = pk2(0.f, 0.f);
#pragma unroll
                    for (int w = 8 * g; w < 8 * g + 8; ++w) {
                        const float2 x = upk2(fma_f32x2(pk2u(s[c][2 * w], s[c][2 * w + 1]), mul2, shift2));
                        const float e0 = ex2(x.x), e1 = ex2(x.y);
                        p[w] = f16x2_from_f32(e0, e1);
                        sum2[g] = add_f32x2(sum2[g], pk2(e0, e1));
                    }
                }
                lsum2 = fma_f32x2(sum2[0], pk2(inv.x, inv.y), lsum2);
                lsum2 = fma_f32x2(sum2[1], pk2(inv.z, inv.w), lsum2);
                tmem_st16(scol + 32 * c, p);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kPReady, buf));
        }
        if (ok && !idle && i < ntiles) {
            const FarRow row = far_tiles<HD, RT>(base, bp, lane_addr, rt, i, ntiles, rot, row_ok ? pos - tile_lo * kKeys : INT32_MAX, qmul, {m_used, lsum2, true});
            m_used = row.m;
            lsum2 = row.sum2;
            ok = row.ok;
        }
        if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kODone, 2 * rt + ((ntiles - 1) & 1)), ((ntiles - 1) >> 1) & 1, abort_flag));
        if (ok && !idle) {
            tc_fence_after();
            const float2 ls = upk2(lsum2);
            const float lsum = ls.x + ls.y;
            const float inv = lsum == 0.f ? 0.f : 1.f / lsum;  // (a NaN sum makes the row NaN)
            // this row in the parts' results, when there are several
            const int64_t prow = kSplit ? ((((static_cast<int64_t>(seq) * a.row_tiles + ctile) * a.n_kv + kvh) * a.splits +
                                            blockIdx.y) * kRows) + tid : 0;
            if (kSplit && row_ok) a.part_lse[prow] = lsum == 0.f ? -INFINITY : m_used + __log2f(lsum);
            // what this row sees of the values that were taken out as NaN: from the first such half on
            const bool any_nan = *nan_seen != 0;
            const int key0 = kSplit ? tile_lo * kKeys : 0;
            const int nan_first = max(key0, max(all_see, 0) / kHalf * kHalf);
            const int nan_last = row_ok ? min(pos, key0 + ntiles * kKeys - 1) : -1;
            uint8_t *out_at = qp + (tid & 127) * 2 * HD;  // the lane's row
#pragma unroll 1
            for (int c0 = 0; c0 < HD; c0 += 32) {
                uint32_t nan = 0;
                if (any_nan) nan = nan_value_dims<HD>(a, seq, kvh, c0, nan_first, nan_last);
                __syncwarp();  // (tensor memory is read by whole warps; lanes part above and where rows are stored)
                uint32_t o[32];
                tmem_ld32(lane_addr + L::col_o(rt) + c0, o);
                tmem_wait_ld();
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    v[e] = (nan >> e) & 1u ? __uint_as_float(0x7FC00000u) : __uint_as_float(o[e]) * inv;
                if constexpr (kSplit) {
                    float4 *to = reinterpret_cast<float4 *>(a.part_o + prow * HD + c0);
                    if (row_ok) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) to[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    }
                } else {
                    // by way of the row tile's q, which no product reads any more: written a row a lane, read in rows
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint4 *>(out_at + (((c0 / 8 + e) ^ (lane & 7)) * 16)) =
                            make_uint4(bf16x2_from_f32(v[8 * e], v[8 * e + 1]), bf16x2_from_f32(v[8 * e + 2], v[8 * e + 3]),
                                       bf16x2_from_f32(v[8 * e + 4], v[8 * e + 5]), bf16x2_from_f32(v[8 * e + 6], v[8 * e + 7]));
                }
            }
            if constexpr (!kSplit) {
                constexpr int kLanes = HD / 8, kAtOnce = 32 / kLanes;  // lanes of a row, rows at once
                __syncwarp();
#pragma unroll 4
                for (int it = 0; it < kLanes; ++it) {
                    const int from = it * kAtOnce + lane / kLanes, k = lane % kLanes;
                    const int64_t to = __shfl_sync(0xFFFFFFFFu, row_at, from);
                    const bool there = __shfl_sync(0xFFFFFFFFu, row_ok, from);
                    const uint4 w = *reinterpret_cast<const uint4 *>(out_at + (from - lane) * 2 * HD + ((k ^ (from & 7)) * 16));
                    if (there) reinterpret_cast<uint4 *>(a.out + to)[k] = w;
                }
            }
        } else if (!ok && lane == 0) {
            flag(a.status, KVFP8_DEV_TIMEOUT);
            *abort_flag = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W::kMma) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// Joins the parts of each row: CTA (x, y) takes 256 / (HD / 4) rows of the row tiles x (tile_rows rows).
template <int HD>
__global__ void __launch_bounds__(256) join_blocks_kernel(const __grid_constant__ BlockPrefillArgs a, int tile_rows) {
    constexpr int kLanes = HD / 4;  // threads of a row, four dims each
    const int kvh = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.n_kv));
    const int tile = static_cast<int>((blockIdx.x / static_cast<unsigned>(a.n_kv)) % static_cast<unsigned>(a.row_tiles));
    const int seq = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.n_kv * a.row_tiles));
    const int lr = static_cast<int>(blockIdx.y) * (256 / kLanes) + static_cast<int>(threadIdx.x) / kLanes;
    const int d = static_cast<int>(threadIdx.x) % kLanes * 4;
    pdl_wait();  // the parts are visible from here on
    const QueryRange qr = a.qsl ? query_range(a.qsl, seq, a.qmax, a.qrows) : QueryRange{seq, 1};
    const int Ls = min(max(a.seq_lens[seq], 0), a.max_len);
    const int nb = qr.count, G = a.group, row0 = tile * tile_rows, r = row0 + lr;
    if (r >= nb * G) return;
    // the row tiles' parts, as their CTAs worked them out
    const int j_last = min(nb, (row0 + tile_rows + G - 1) / G) - 1;
    const int kend = a.causal ? Ls - nb + j_last + 1 : Ls;
    if (kend <= 0) return;  // zeroed by its CTA
    const int parts = split_parts(a.splits, (kend + kKeys - 1) / kKeys, kKeys);
    const int64_t p0 = static_cast<int64_t>(blockIdx.x) * a.splits * tile_rows + lr;
    PartMerge<true> mg;
    for (int c0 = 0; c0 < parts; c0 += 8) {
        float l[8];
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            l[i] = -INFINITY;
            if (c0 + i < parts) {
                const int64_t p = p0 + static_cast<int64_t>(c0 + i) * tile_rows;
                l[i] = a.part_lse[p];
                v[i] = *reinterpret_cast<const float4 *>(a.part_o + p * HD + d);
            }
        }
        mg.add8(l, v);
    }
    *reinterpret_cast<uint2 *>(a.out + ((static_cast<int64_t>(qr.q0) + r / G) * a.n_q + kvh * G + r % G) * HD + d) =
        mg.result(1.f);
}

// How a call is cut: the rows of a CTA, and the parts that fill the SMs.
struct BlockSplitPlan {
    int tile_rows = kPfRows, splits = 1;
    size_t lse_off = 0, total = 0;  // workspace
};
BlockSplitPlan block_split_plan(int32_t num_seqs, int32_t n_q, int32_t n_kv, int32_t head_dim, int32_t qmax, int64_t max_len) {
    BlockSplitPlan p;
    const int64_t group_rows = static_cast<int64_t>(qmax) * (n_q / n_kv);
    if (head_dim <= 128 && group_rows > kPfRows) p.tile_rows = 2 * kPfRows;
    const int64_t tiles = (group_rows + p.tile_rows - 1) / p.tile_rows;
    if (tiles > kSplitSms || tiles * n_kv > kSplitSms || tiles * n_kv * num_seqs > kSplitSms / 2) return p;
    const int64_t ctas = tiles * n_kv * num_seqs;
    p.splits = static_cast<int>(std::max<int64_t>(1, std::min(kSplitSms / ctas, max_len / kMinPartKeys)));
    if (p.splits == 1) return p;
    const size_t part_rows = static_cast<size_t>(ctas) * p.splits * p.tile_rows;
    p.lse_off = part_rows * head_dim * sizeof(float);
    p.total = p.lse_off + part_rows * sizeof(float);
    return p;
}

template <int HD, int RT>
cudaError_t run_row_tiles(const DecodeArgs &d, const BlockSplitPlan &sp, const CUtensorMap &tmk, const CUtensorMap &tmv,
                          BlockPrefillArgs a, cudaStream_t stream) {
    const size_t smem = PbSmem<HD, RT>::kTotal + 1024;
    constexpr int kThreads = PbWarps<HD, RT>::kAll * 32;
    auto kern = sp.splits > 1 ? prefill_blocks_kernel<HD, RT, true> : prefill_blocks_kernel<HD, RT, false>;
    cudaError_t err;
    int occ = 0;  // also raises the kernel's shared memory limit, once per device
    if ((err = kernel_occupancy(kern, kThreads, smem, &occ)) != cudaSuccess) return err;
    const int group_rows = d.qmax * a.group;  // (prefill_takes: below 2^31 - 511)
    a.row_tiles = (group_rows + 128 * RT - 1) / (128 * RT);
    const int64_t ctas = static_cast<int64_t>(d.num_seqs) * a.row_tiles * d.n_kv;
    kern<<<dim3(static_cast<unsigned>(ctas), sp.splits), kThreads, smem, stream>>>(tmk, tmv, a);
    if ((err = cudaGetLastError()) != cudaSuccess || sp.splits == 1) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 128 * RT / (256 / (HD / 4)));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_blocks_kernel<HD>, a, 128 * RT);
}

template <int HD>
cudaError_t run_prefill_blocks(const DecodeArgs &d, cudaStream_t stream) {
    constexpr int kSeg = HD < 128 ? HD : 128;
    const int box_rows = std::min(d.block_size, kHalf);
    const int64_t rows = static_cast<int64_t>(d.num_blocks) * d.block_size;
    CUtensorMap tmk, tmv;
    cudaError_t err;
    if ((err = encode_cache_map(&tmk, d.key_cache, rows, d.n_kv * HD, kSeg, box_rows)) != cudaSuccess ||
        (err = encode_cache_map(&tmv, d.value_cache, rows, d.n_kv * HD, kSeg, box_rows)) != cudaSuccess)
        return err;
    BlockPrefillArgs a = {};
    a.out = static_cast<__nv_bfloat16 *>(d.out);
    a.query = static_cast<const __nv_bfloat16 *>(d.query);
    a.qsl = d.qsl;
    a.qmax = d.qmax;
    a.qrows = d.qrows;
    a.block_tables = d.block_tables;
    a.max_blocks_per_seq = d.max_blocks_per_seq;
    a.seq_lens = d.seq_lens;
    a.num_seqs = d.num_seqs;
    a.n_q = d.n_q;
    a.n_kv = d.n_kv;
    a.group = d.n_q / d.n_kv;
    a.block_size = d.block_size;
    a.num_blocks = d.num_blocks;
    a.max_len = d.max_blocks_per_seq * d.block_size;
    a.sm_scale = d.sm_scale;
    a.status = d.status;
    a.box_rows = box_rows;
    a.value_cache = d.value_cache;
    a.key_scales = d.key_block_scales;
    a.value_scales = d.value_block_scales;
    a.scale_stride = d.block_scale_stride;
    a.causal = d.causal != 0;
    const BlockSplitPlan sp = block_split_plan(d.num_seqs, d.n_q, d.n_kv, HD, d.qmax, a.max_len);
    a.splits = sp.splits;
    a.part_o = static_cast<float *>(d.workspace);
    a.part_lse = reinterpret_cast<float *>(static_cast<uint8_t *>(d.workspace) + sp.lse_off);
    if constexpr (HD <= 128) {
        if (sp.tile_rows == 2 * kPfRows) return run_row_tiles<HD, 2>(d, sp, tmk, tmv, a, stream);
    }
    return run_row_tiles<HD, 1>(d, sp, tmk, tmv, a, stream);
}

}  // namespace

size_t block_scaled_prefill_workspace_size(int32_t num_seqs, int32_t n_q, int32_t n_kv, int32_t head_dim, int32_t qmax,
                                           int64_t max_len) {
    return block_split_plan(num_seqs, n_q, n_kv, head_dim, qmax, max_len).total;
}

cudaError_t launch_prefill_block_scaled(const DecodeArgs &d, cudaStream_t stream) {
    if (d.num_seqs == 0) return cudaSuccess;
    if (!prefill_takes(d.n_q, d.n_kv, d.qmax, d.num_seqs)) return cudaErrorNotSupported;
    switch (d.head_dim) {
        case 64: return run_prefill_blocks<64>(d, stream);
        case 128: return run_prefill_blocks<128>(d, stream);
        case 256: return run_prefill_blocks<256>(d, stream);
        default: return cudaErrorNotSupported;
    }
}

}  // namespace kvfp8
