// Causal multi-query attention over the FP8 (E4M3) cache for long query chunks (prefill),
// sm_103a tensor cores (tcgen05) with accumulators in tensor memory.
//
// What it computes is kvfp8_paged_attention_multi (llama.cpp "llama : Add FP8 KV-cache
// support (#28392)", tests/test-fp8.cpp check_fp8_attention: a batch of new tokens, each
// attending to every cached token up to its own position, on K/V rounded through the cache
// format).  The decode kernel covers up to 16 (query token, head) score columns per kv
// head; past that the rows form a real M dimension and the contraction is dense, so:
//
// Two kernels: prefill_kernel below (one row tile of 128 per CTA), and prefill2_kernel
// further down (two row tiles per CTA sharing each converted K/V tile), which takes the
// long chunks at head_dim 64 and 128.
//
//  * Work unit: one CTA per (sequence, kv head, tile of 128 score rows).  A row is a
//    (query token j, head g of the kv head's group) pair, row = j*G + g, so all rows of a
//    tile share one K/V stream.  Keys are visited in tiles of 64 up to the tile's last
//    causal position, each row tile starting at its own key tile (the online softmax takes
//    the keys in any order).  The grid runs kv head fastest, then row tile, then sequence.
//  * Warp-specialized, every stage overlapped with the others (14 warps):
//      - warp 13 issues the TMA loads of the FP8 K/V tiles (per-head-segment boxes of the
//        cache map, one lane per box) into a four-stage ring;
//      - warps 4-11 convert the tile's q rows bf16 -> f16 once, and each K tile
//        e4m3 -> f16, into the K-major 128-byte-swizzled operand layout, and each V tile
//        e4m3 -> f16 transposed (V^T: head dims as rows, keys along K), so both products
//        take K-major operands; K, V^T and the score buffers are triple-buffered;
//      - one thread of warp 12 issues S(i) = Q.K(i)^T (tcgen05.mma kind::f16, M = 128,
//        N = 64, fp32 in tensor memory) and then O += P(i-1).V(i-1) (A = P from tensor
//        memory, B = V^T from shared memory), so the next scores are computed while the
//        softmax works on the current ones.  Up to head_dim 128 V^T carries a row of ones,
//        so the same product also sums each row of P;
//      - warps 0-3 (one TMEM lane quarter each, one score row per thread) read S, apply
//        the causal mask and the online softmax (log2 domain), and write P (f16) back over
//        S.  O is rescaled in TMEM only when a row's running maximum grows by more than
//        2^8 (P <= 2^8 stays well inside fp16); at the end they divide by the row sum,
//        apply v_scale and store bf16.
//  * All waits are bounded (mbarriers with a clock64 limit); a wait that runs out sets
//    KVFP8_DEV_TIMEOUT.  Tensor memory is always released before the CTA exits.
#include "kvfp8_e2m1.cuh"
#include "prefill_common.cuh"

namespace kvfp8 {
namespace {

constexpr int kPfKeys = 64;    // keys per tile

// 2^x on an f16 pair (the tensor core takes P as f16)
__device__ __forceinline__ uint32_t ex2_f16x2(uint32_t x) {
    uint32_t r;
    asm("ex2.approx.f16x2 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ float f16lo_f32(uint32_t h) {
    float r;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(r) : "r"(h));
    return r;
}
__device__ __forceinline__ float f16hi_f32(uint32_t h) {
    float r;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.f32.f16 %0, u;\n\t}" : "=f"(r) : "r"(h));
    return r;
}
// the largest (kMax) or smallest of 64 scores, four independent chains of 3-input ops
template <bool kMax>
__device__ __forceinline__ float extreme64(const uint32_t (&s)[2][32]) {
    auto v = [&](int c) { return __uint_as_float(s[c >> 5][c & 31]); };
    auto op = [](float a, float b, float c) { return kMax ? max3f(a, b, c) : min3f(a, b, c); };
    float a0 = v(0), a1 = v(1), a2 = v(2), a3 = v(3);
#pragma unroll
    for (int c = 4; c < 60; c += 8) {
        a0 = op(a0, v(c), v(c + 1));
        a1 = op(a1, v(c + 2), v(c + 3));
        a2 = op(a2, v(c + 4), v(c + 5));
        a3 = op(a3, v(c + 6), v(c + 7));
    }
    a0 = op(a0, v(60), v(61));
    a1 = op(a1, v(62), v(63));
    return op(a0, a1, kMax ? fmaxf(a2, a3) : fminf(a2, a3));
}

// The 4-bit form's arguments are its own: carried along by the E4M3 kernels they cost the two-row-tile one
// 0.8 % (911 against 919 TFLOP/s on 512 new tokens of 64 sequences of 4096).
template <bool F4>
struct PrefillArgs : PrefillCommon {
    // (named by shared code, read by nothing)
    static constexpr int32_t splits = 1;
    static constexpr float *part_o = nullptr, *part_lse = nullptr;
};
template <>
struct PrefillArgs<true> : PrefillCommon {
    const uint8_t *key_scales, *value_scales;  // the groups' scale bytes
    // parts a (sequence, kv head, row tile)'s keys are cut into at most (gridDim.y), and the parts'
    // results, [CTA of the unsplit grid, in sequence order][part][row of the tile]
    int32_t splits;
    float *part_o, *part_lse;
};

// ---------------------------------------------------------------- the 4-bit cache
//
// F4: the cache holds E2M1 codes with an E4M3 scale byte per 16 dims instead of E4M3 bytes.  What
// fills the f16 operands differs: a stage holds the codes of its keys (boxes of one head's
// head_dim/2-byte rows) and their scale bytes (contiguous per block and head), and the conversion
// multiplies each fp16 pair of codes by its group's scale (exact: code * scale is an fp16 number).  So
// do the softmax weights' reference and rounding (kF4Head), and the split of the keys (kSplit).
//
// NaN: a scale byte 0x7F makes its 16 dims NaN.  In K that makes the key's scores NaN, which the
// masks keep from rows that do not see it.  In V it would reach every row of the tile (0 * NaN), so
// such scales are taken as 0, the CTA remembers that it met one, and at the end each of its rows
// looks up which groups of the values it sees are NaN (a slow scan that no finite cache runs).

// Weights are taken against a reference 2^7 below the row's highest score at the time (the E4M3 forms:
// that score), so they reach up to 2^15 and keep their 11 bits down to 2^-21 of the highest and are above
// zero down to 2^-32, as in the decode kernel over the same cache (paged_decode_fp4.cu).  fp16 weights
// move outputs by 0.0003 to 0.0006 of their norm, where rounding an output to bf16 moves it by 0.0016.
constexpr float kF4Head = 7.f;

// Conversion goes by units of 32 rows of 16 code bytes (8 keys x 4 chunks of 32 dims; 16 keys x 2 at
// head_dim 64; at 256 a key group has two units).  One ldmatrix gives a lane, per chunk, the codes of
// dims 8u..8u+7 of a key (u = lane % 4): as K they are one 16-byte piece of the key's operand row; as V
// the pairs of dims are stored transposed with stmatrix.  The dims of a 32-dim chunk are then permuted
// in V^T's rows, row 8j + 2a + b holding dim 8a + 2j + b, and so in O's columns: O's word (pair of
// columns) 4j + a is the output's word 4a + j.

// half k of an fp16 pair in both halves
template <int k>
__device__ __forceinline__ uint32_t half_pair(uint32_t x) {
    uint32_t r;
    if (k == 0)
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(r) : "r"(x));
    else
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(r) : "r"(x));
    return r;
}

template <int HD>
struct F4Unit {
    static constexpr int kPer64 = HD == 64 ? 4 : HD / 16;  // units of 64 keys
    static constexpr int kRow = HD / 2, kGph = HD / 16;
    uint32_t r[4];   // the lane's eight codes of chunk c(m), key(m), m = 0..3
    uint32_t bytes;  // their scale bytes

    __device__ __forceinline__ static int first_key(int unit) { return HD == 64 ? 16 * unit : HD == 128 ? 8 * unit : 8 * (unit >> 1); }
    // chunk of matrix m
    __device__ __forceinline__ static int chunk(int unit, int m) { return HD == 64 ? m & 1 : HD == 128 ? m : 4 * (unit & 1) + m; }
    // the key of row i of a matrix, past first_key: for K rows 2i, 2i + 1 are keys i and i + 4, so that
    // the stores of eight lanes (two rows) fall on different banks
    template <bool kK>
    __device__ __forceinline__ static int row_key(int i) { return kK ? (i >> 1) + 4 * (i & 1) : i; }
    template <bool kK>
    __device__ __forceinline__ static int key(int unit, int m, int lane) {
        return first_key(unit) + row_key<kK>(lane >> 2) + (HD == 64 ? 8 * (m >> 1) : 0);
    }

    // codes, scales: the stage's shared-memory addresses of this side; keys not in mask read as zeros
    template <bool kK>
    __device__ __forceinline__ void load(uint32_t codes, uint32_t scales, uint64_t mask, int unit, int lane) {
        const int m = lane >> 3, k = first_key(unit) + row_key<kK>(lane & 7) + (HD == 64 ? 8 * (m >> 1) : 0);
        const uint32_t addr = codes + swz<kRow>(k, chunk(unit, m));
        ldsm_x4(addr, r[0], r[1], r[2], r[3]);
        const int k0 = key<kK>(unit, 0, lane), k1 = key<kK>(unit, 2, lane);
        uint32_t w0, w1;  // scale bytes of the chunks of m = 0, 1 and of m = 2, 3
        if (HD == 64) {
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w0) : "r"(scales + k0 * kGph));
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w1) : "r"(scales + k1 * kGph));
        } else {
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(scales + k0 * kGph + 2 * chunk(unit, 0)));
        }
        if (!((mask >> k0) & 1ull)) w0 = 0u;
        if (!((mask >> k1) & 1ull)) w1 = 0u;
        bytes = __byte_perm(w0, w1, 0x6420u + 0x1111u * ((lane & 3) >> 1));
    }
    // the eight values of matrix m as fp16 pairs
    template <int m>
    __device__ __forceinline__ void values(uint32_t (&h)[4]) const {
        const uint32_t s = half_pair<m & 1>(m < 2 ? f16x2_from_e4m3x2(bytes) : f16x2_from_e4m3x2_hi(bytes));
        f16x2_from_e2m1x8(r[m], h);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = mul_f16x2(h[i], s);
    }
    // K: rows of the K-major operand blocks of 64 dims at dst, block_bytes apart
    template <int m>
    __device__ __forceinline__ void store_k1(uint32_t dst, uint32_t block_bytes, int unit, int lane) const {
        uint32_t h[4];
        values<m>(h);
        const int c = chunk(unit, m);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         dst + (c >> 1) * block_bytes + sw128(key<true>(unit, m, lane), 4 * (c & 1) + (lane & 3))),
                     "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                     : "memory");
    }
    __device__ __forceinline__ void store_k(uint32_t dst, uint32_t block_bytes, int unit, int lane) const {
        store_k1<0>(dst, block_bytes, unit, lane);
        store_k1<1>(dst, block_bytes, unit, lane);
        store_k1<2>(dst, block_bytes, unit, lane);
        store_k1<3>(dst, block_bytes, unit, lane);
    }
    // V: 8 keys of the V^T rows at dst (a key block's 64 keys)
    template <int m>
    __device__ __forceinline__ void store_v1(uint32_t dst, int unit, int lane) const {
        uint32_t h[4];
        values<m>(h);
        const int ko = first_key(unit) / 8 + (HD == 64 ? m >> 1 : 0);
        stsm_x4_t(dst + sw128(32 * chunk(unit, m) + lane, ko), h[0], h[1], h[2], h[3]);
    }
    __device__ __forceinline__ void store_v(uint32_t dst, int unit, int lane) const {
        store_v1<0>(dst, unit, lane);
        store_v1<1>(dst, unit, lane);
        store_v1<2>(dst, unit, lane);
        store_v1<3>(dst, unit, lane);
    }
    // NaN scales of V are taken as 0 and remembered
    __device__ __forceinline__ void drop_nan(volatile int32_t *nan_seen) {
        if ((((bytes & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0u) {
            bytes &= ~nan_byte_mask(bytes);
            *nan_seen = 1;
        }
    }
};
// the word of O's 32 columns that holds the output's dims 2w, 2w + 1 of the chunk
template <bool F4>
__host__ __device__ constexpr int o_word(int w) { return F4 ? 4 * (w & 3) + (w >> 2) : w; }

// The scale bytes of 64 keys from t0 on (K's at dst, V's side_bytes further), by all lanes of the
// TMA warp: 16-byte asynchronous copies, each of 1 to 4 keys of one block, whose completion every lane
// adds to the stage's barrier.  (As bulk copies they cost this warp one issue per block and side: 74
// against 69 us for 16 chunks of 32 tokens over 4096 keys in 16-token blocks, 105 against 84 in 8-token
// ones.)
// win: the lane window of block-table entries from wbase on.
template <int HD>
__device__ __forceinline__ void copy_scales(const PrefillArgs<true> &a, int kvh, int t0, int kend, int lbs, int32_t win,
                                            int wbase, uint32_t dst, uint32_t side_bytes, uint32_t bar, int lane) {
    constexpr int kGph = HD / 16, kKeys = 16 / kGph, kChunks = kPfKeys / kKeys;  // of a side
#pragma unroll
    for (int c = lane; c < 2 * kChunks; c += 32) {
        const int k = c % kChunks * kKeys, t = t0 + k;
        const int blk = __shfl_sync(0xFFFFFFFFu, win, ((t >> lbs) - wbase) & 31);
        if (t < kend && blk >= 0 && blk < a.num_blocks) {
            const uint8_t *src = (c < kChunks ? a.key_scales : a.value_scales) +
                                 (((static_cast<int64_t>(blk) * a.n_kv + kvh) << lbs) + (t & (a.block_size - 1))) * kGph;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             dst + (c < kChunks ? 0u : side_bytes) + static_cast<uint32_t>(k * kGph)),
                         "l"(src)
                         : "memory");
        }
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// The groups (bit g: dims 16g..16g+15) in which some value of tokens first..last of the sequence is NaN, for
// each lane's own last (negative: none); blocks out of range hold no tokens.  Called by whole warps: the
// tokens that every lane has are shared out over the lanes, the few after them are each lane's own.
template <int HD>
__device__ __noinline__ uint32_t nan_value_groups(const PrefillArgs<true> &a, int seq, int kvh, int first, int last) {
    const int32_t *bt = a.block_tables + static_cast<int64_t>(seq) * a.max_blocks_per_seq;
    uint32_t groups = 0;
    auto look = [&](int t) {
        const int32_t blk = bt[t / a.block_size];
        if (blk < 0 || blk >= a.num_blocks) return;
        const uint32_t *row = reinterpret_cast<const uint32_t *>(
            a.value_scales +
            ((static_cast<int64_t>(blk) * a.n_kv + kvh) * a.block_size + t % a.block_size) * (HD / 16));
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) {
            const uint32_t nan = nan_byte_mask(row[i]) & 0x08040201u;
            groups |= ((nan | nan >> 8 | nan >> 16 | nan >> 24) & 0xFu) << (4 * i);
        }
    };
    const int lane = static_cast<int>(threadIdx.x & 31);
    const int all = __reduce_min_sync(0xFFFFFFFFu, last < 0 ? INT32_MAX : last);  // tokens first..all are every lane's
    if (all != INT32_MAX)
        for (int t = first + lane; t <= all; t += 32) look(t);
    groups = __reduce_or_sync(0xFFFFFFFFu, groups);
    if (last < 0) return 0u;
    for (int t = max(first, all + 1); t <= last; ++t) look(t);
    return groups;
}

// Where the key one tile after key t lies: its block-table entry, and the row within that block.
struct KeyPlace {
    int entry, row;
};
__host__ __device__ constexpr KeyPlace next_tile_place(int t, int lbs) {
    return {(t + kPfKeys) >> lbs, (t + kPfKeys) & ((1 << lbs) - 1)};
}
static_assert(next_tile_place(0, 4).entry == 4 && next_tile_place(0, 4).row == 0 && next_tile_place(16, 4).entry == 5);
static_assert(next_tile_place(64, 6).entry == 2 && next_tile_place(64, 6).row == 0);
static_assert(next_tile_place(0, 7).entry == 0 && next_tile_place(0, 7).row == 64, "the second half of a block of 128");
static_assert(next_tile_place(64, 7).entry == 1 && next_tile_place(64, 7).row == 0);
static_assert(next_tile_place(128, 8).entry == 0 && next_tile_place(128, 8).row == 192);

__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *map, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// bf16 pair of dims d, d+1, NaN where the pair's group is in `groups`
__device__ __forceinline__ uint32_t nan_in(uint32_t w, uint32_t groups, int d) {
    return (groups >> (d >> 4)) & 1u ? 0x7FFF7FFFu : w;
}
// 32 dims from d0 on of a part's row, from O's columns, as float; NaN in `groups`
__device__ __forceinline__ void store_part(float *row, const uint32_t (&o)[32], float inv, uint32_t groups, int d0) {
#pragma unroll
    for (int w = 0; w < 16; w += 2) {  // dims 2w..2w+3
        const int e = 2 * o_word<true>(w), f = 2 * o_word<true>(w + 1);
        float4 v = make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                               __uint_as_float(o[f]) * inv, __uint_as_float(o[f + 1]) * inv);
        if ((groups >> ((d0 + 2 * w) >> 4)) & 1u) v.x = v.y = v.z = v.w = __uint_as_float(0x7FC00000u);
        *reinterpret_cast<float4 *>(row + d0 + 2 * w) = v;
    }
}

// Shared-memory plan (byte offsets from a 1024-aligned base).  Q is converted once; K and
// V^T (f16) have NB buffers, and so do the scores in tensor memory; the FP8 staging ring has
// NS stages.  At head_dim 256 the f16 buffers fill the shared memory: NB = 2, NS = 1.
template <int HD, bool F4>
struct PfSmem {
    static constexpr int kRow = F4 ? HD / 2 : HD;                  // cache bytes of a key's head
    static constexpr int kSeg = kRow >= 128 ? 128 : kRow;          // TMA box row (swizzle span)
    static constexpr int kSegs = kRow / kSeg;
    static constexpr int kNB = HD >= 256 ? 2 : 3;                  // f16 K/V^T and S buffers
    static constexpr int kNS = HD >= 256 ? 1 : F4 ? 8 : 4;         // staging stages
    static constexpr int kQ = 0;                                   // Q f16: HD/64 blocks x 128 rows x 128 B
    static constexpr int kKBuf = HD * 128;                         // one K f16 buffer: HD/64 x 64 rows x 128 B
    // Up to head_dim 128, V^T carries 16 more rows: a row of ones then zeros, so the O
    // product also accumulates each score row's sum of P (column HD of O) in fp32.  At 256
    // there is no room (the product's N would pass 256 and shared memory would overflow):
    // the softmax warps sum P themselves.
    static constexpr bool kSumCol = HD <= 128;
    static constexpr int kVRows = HD + (kSumCol ? 16 : 0);
    static constexpr int kVBuf = kVRows * 128;                     // one V^T f16 buffer: rows x 128 B
    static constexpr int kK = kQ + HD * 256;
    static constexpr int kV = kK + kNB * kKBuf;
    static constexpr int kStage = kV + kNB * kVBuf;                // fp8 K then V, per stage
    // F4: K codes, V codes, then the scale bytes of K and of V
    static constexpr int kScaleSide = F4 ? kPfKeys * (HD / 16) : 0;
    static constexpr int kScales = 2 * kPfKeys * kRow;
    static constexpr int kStageBytes = kScales + 2 * kScaleSide;
    static constexpr int kBars = kStage + kNS * kStageBytes;
    // mbarriers: full[NS], empty[NS], then per buffer kv_ready, kv_free, s_ready, p_ready,
    // and one to drain the tensor core on a timeout.  kv_free[b] completes when the products
    // of the buffer's tile are done (one commit after its O product covers its S product
    // too); it also tells that O is up to date.
    static constexpr int kFull = kBars, kEmpty = kFull + 8 * kNS, kKvReady = kEmpty + 8 * kNS;
    static constexpr int kKvFree = kKvReady + 8 * kNB, kSReady = kKvFree + 8 * kNB;
    static constexpr int kPReady = kSReady + 8 * kNB;
    static constexpr int kDrain = kPReady + 8 * kNB;
    static constexpr int kMeta = kDrain + 8;                       // valid-key mask per stage
    static constexpr int kBufMask = kMeta + 8 * kNS;               // valid-key mask per K/V buffer
    static constexpr int kMisc = kBufMask + 8 * kNB;               // tmem base, abort flag, NaN seen
    static constexpr int kTotal = kMisc + 16;
    // tensor memory: S[NB] (64 fp32 columns each; P as f16 over the first 32), then O
    static constexpr uint32_t kColO = 64 * kNB;
    static constexpr uint32_t kTmemCols = kColO + HD + 32 <= 256 ? 256 : 512;
};

// Warp roles (448 threads): warps 0-3 softmax + epilogue (TMEM lane quarters 0-3, one score
// row per thread), warps 4-11 conversion, warp 12 tensor-core issue (and TMEM allocation),
// warp 13 TMA.
constexpr int kPfConvWarps = 8;
constexpr int kPfMmaWarp = 4 + kPfConvWarps, kPfTmaWarp = kPfMmaWarp + 1;
constexpr int kPfWarps = kPfTmaWarp + 1;

template <int HD, bool F4, bool kSplit>
__global__ void __launch_bounds__(kPfWarps * 32, 1)
prefill_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
               const PrefillArgs<F4> a) {
    using L = PfSmem<HD, F4>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *bp = smem_raw + (base - raw);
    volatile uint64_t *meta = reinterpret_cast<volatile uint64_t *>(bp + L::kMeta);
    volatile uint64_t *buf_mask = reinterpret_cast<volatile uint64_t *>(bp + L::kBufMask);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bp + L::kMisc);
    volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(bp + L::kMisc + 4);
    volatile int32_t *nan_seen = reinterpret_cast<volatile int32_t *>(bp + L::kMisc + 8);
    auto bar = [&](int off, int i) { return base + static_cast<uint32_t>(off + 8 * i); };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // kv head fastest, then row tile, then sequence (longest first): the CTAs resident at one
    // time read every kv head's slice of the same cache rows, and a (sequence, kv head)'s row
    // tiles run together, so its K/V tiles are fetched from HBM once and re-read from L2
    const int kvh = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.n_kv));
    const int tile = static_cast<int>((blockIdx.x / static_cast<unsigned>(a.n_kv)) % static_cast<unsigned>(a.row_tiles));
    const int rank = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.n_kv * a.row_tiles));

    const float sk = load_scale(a.k_scale, a.scale_dtype);
    const float sv = load_scale(a.v_scale, a.scale_dtype);
    // the K buffers are free scratch until the pipeline starts
    const int seq = seq_of_rank(a.seq_lens, a.num_seqs, a.max_len, rank,
                                reinterpret_cast<uint32_t *>(bp + L::kK));
    if (!scale_ok(sk) || !scale_ok(sv)) {
        if (blockIdx.x == 0 && tid == 0) flag(a.status, KVFP8_DEV_BAD_SCALE);
        return;
    }
    // this sequence's query rows (qsl == nullptr: one query per sequence, row seq) and cached
    // length (flagged once, by its first CTA)
    const int raw_nq = a.qsl ? a.qsl[seq + 1] - a.qsl[seq] : 1;
    const QueryRange qr = a.qsl ? query_range(a.qsl, seq, a.qmax, a.qrows) : QueryRange{seq, 1};
    const int Lraw = a.seq_lens[seq];
    const int Ls = min(max(Lraw, 0), a.max_len);
    // (more new tokens than cached ones is an error of the multi-query form only: a decode
    // query on an empty sequence gives a zero row)
    if (tile == 0 && kvh == 0 && tid == 0 &&
        (qr.count != raw_nq || Lraw < 0 || Lraw > a.max_len || (a.qsl && qr.count > Ls)))
        flag(a.status, KVFP8_DEV_BAD_BLOCK);
    const int nb = qr.count, G = a.group;
    const int row0 = tile * kPfRows;                 // first score row of this tile
    if (row0 >= nb * G) return;                      // no rows here
    const int j_last = min(nb, (row0 + kPfRows + G - 1) / G) - 1;
    const int kend = Ls - nb + j_last + 1;           // keys the tile's last row may see
    int ntiles = kend > 0 ? (kend + kPfKeys - 1) / kPfKeys : 0;
    int tile_lo = 0;  // this CTA's key tiles: ntiles from tile_lo on
    if constexpr (kSplit) {
        const int parts = split_parts(a.splits, ntiles, kPfKeys);
        const int part = static_cast<int>(blockIdx.y);
        if (part >= parts) return;
        tile_lo = static_cast<int>(static_cast<int64_t>(part) * ntiles / parts);
        ntiles = static_cast<int>(static_cast<int64_t>(part + 1) * ntiles / parts) - tile_lo;
    }
    // The row tiles of one (sequence, kv head) run side by side on one K/V stream; each
    // starts its pass at its own key tile (the online softmax takes the keys in any order),
    // so they read different lines of the stream at any one time.
    const int rot = ntiles > 0 ? static_cast<int>((static_cast<int64_t>(tile) * ntiles) / a.row_tiles) % ntiles : 0;
    auto key_tile = [&](int i) { const int k = i + rot; return (k >= ntiles ? k - ntiles : k) + (kSplit ? tile_lo : 0); };

    if (ntiles == 0) {  // every row of the tile sees no key: zero rows
        if (tid < kPfRows) {
            const int r = row0 + tid;
            if (r < nb * G) {
                const int j = r / G, g = r % G;
                uint4 *o = reinterpret_cast<uint4 *>(
                    a.out + ((static_cast<int64_t>(qr.q0) + j) * a.n_q + kvh * G + g) * HD);
                for (int c = 0; c < HD / 8; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        return;
    }

    if (tid == 0) {
        for (int s = 0; s < L::kNS; ++s) {
            mbar_init(bar(L::kFull, s), F4 ? 33 : 1);  // F4: and every lane's scale copies
            mbar_init(bar(L::kEmpty, s), kPfConvWarps);
        }
        for (int b = 0; b < L::kNB; ++b) {
            mbar_init(bar(L::kKvReady, b), kPfConvWarps);
            mbar_init(bar(L::kKvFree, b), 1);
            mbar_init(bar(L::kSReady, b), 1);
            mbar_init(bar(L::kPReady, b), 4);
        }
        mbar_init(bar(L::kDrain, 0), 1);
        *abort_flag = 0;
        if (F4) *nan_seen = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kPfMmaWarp) {
        tmem_alloc(base + L::kMisc, L::kTmemCols);
        tmem_relinquish();
    }
    if (warp == kPfTmaWarp && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmk)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmv)) : "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const volatile int32_t never = 0;

    if (warp == kPfTmaWarp) {
        // ------------------------------------------------------------ TMA producer
        // The warp holds 32 block-table entries, one per lane (refreshed as the tiles move
        // past them).  A tile is nbox boxes of K and nbox of V: lane p < nbox works out K box
        // p and lane nbox + p V box p, side by side; lane 0 waits for a free stage and posts
        // the expected bytes, then every lane with a box issues its own copy.  (This warp
        // shares its scheduler with compute-heavy warps: its per-tile work is kept to a few
        // dozen instructions, with no division.)
        const int32_t *bt = a.block_tables + static_cast<int64_t>(seq) * a.max_blocks_per_seq;
        const int bs = a.block_size, br = a.box_rows;
        const int lbs = __ffs(bs) - 1;  // block_size is a power of two
        const int nbox = kPfKeys / br;
        const bool k_lane = lane < nbox;
        const int p = k_lane ? lane : lane - nbox;  // this lane's box within the tile
        const bool box_lane = lane < 2 * nbox;
        const CUtensorMap *map = k_lane ? &tmk : &tmv;
        const uint32_t side = k_lane ? 0u : static_cast<uint32_t>(kPfKeys * L::kRow);
        int wbase = -(1 << 30);
        int32_t win = -1;
        int issued = 0;
        bool aborted = false;
        for (int i = 0; i < ntiles; ++i) {
            const int st = i % L::kNS;
            const int t0 = key_tile(i) * kPfKeys;
            const int e0 = t0 >> lbs, e1 = (min(kend, t0 + kPfKeys) - 1) >> lbs;
            if (e0 < wbase || e1 >= wbase + 32) {  // next window of block-table entries
                wbase = e0;
                win = wbase + lane < a.max_blocks_per_seq ? bt[wbase + lane] : -1;
            }
            // this lane's box: its first key t, the block holding it, and whether it is
            // copied (keys past kend are left out; a bad block is flagged and left out)
            const int t = t0 + p * br;
            const int blk = __shfl_sync(0xFFFFFFFFu, win, ((t >> lbs) - wbase) & 31);
            const bool live = box_lane && t < kend;
            const bool good = live && blk >= 0 && blk < a.num_blocks;
            if (live && !good && k_lane) flag(a.status, KVFP8_DEV_BAD_BLOCK);
            const int row = blk * bs + (t & (bs - 1));
            uint64_t part = 0;
            if (good && k_lane) {
                const int nk = min(br, kend - t);
                part = (nk >= 64 ? ~0ull : ((1ull << nk) - 1)) << (p * br);
            }
            const uint64_t mask =
                static_cast<uint64_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(part))) |
                static_cast<uint64_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(part >> 32))) << 32;
            const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, good && k_lane));
            if (lane == 0) {
                if (!mbar_wait(bar(L::kEmpty, st), ((i / L::kNS) & 1) ^ 1u, abort_flag)) {
                    aborted = true;
                } else {
                    meta[st] = mask;
                    const uint32_t full = bar(L::kFull, st);
                    if (boxes > 0)
                        mbar_arrive_tx(full, static_cast<uint32_t>(boxes * 2 * br * L::kRow));
                    else
                        mbar_arrive(full);
                    ++issued;
                }
            }
            aborted = __shfl_sync(0xFFFFFFFFu, aborted, 0);
            if (aborted) break;
            __syncwarp();  // what lane 0 waited for (the stage has been read) holds for every lane's copies
            // the expected bytes are posted: each lane with a box copies it
            if (good) {
                const uint32_t full = bar(L::kFull, st);
                const uint32_t dst = base + L::kStage + st * L::kStageBytes + side +
                                     static_cast<uint32_t>(p * br * L::kSeg);
#pragma unroll
                for (int sgi = 0; sgi < L::kSegs; ++sgi)
                    tma_load_3d(dst + static_cast<uint32_t>(sgi * kPfKeys * L::kSeg), map, 0,
                                kvh * L::kSegs + sgi, row, full);
            }
            if constexpr (F4) {
                const uint32_t stage = base + L::kStage + st * L::kStageBytes;
                copy_scales<HD>(a, kvh, t0, kend, lbs, win, wbase, stage + L::kScales, L::kScaleSide,
                                bar(L::kFull, st), lane);
            }
            if constexpr (F4 && L::kNS == 1) {
                // one stage: the next copies start when this tile has been read, so their lines are brought
                // into L2 meanwhile, as far as the window of block-table entries goes (head_dim 256, 32 tokens
                // of 32 sequences on 4096: 150 to 124 us; two or three tiles ahead 127 and 128; with all lines
                // of the scale bytes 3 us less)
                const KeyPlace box = next_tile_place(t, lbs);
                const int next = __shfl_sync(0xFFFFFFFFu, win, (box.entry - wbase) & 31);
                if (box_lane && t + kPfKeys < kend && box.entry - wbase < 32 && next >= 0 && next < a.num_blocks) {
#pragma unroll
                    for (int sgi = 0; sgi < L::kSegs; ++sgi)
                        tma_prefetch_3d(map, 0, kvh * L::kSegs + sgi, next * bs + box.row);
                }
                // and the scale bytes, kLineKeys keys of a side by each of the first lanes
                constexpr int kLineKeys = 128 / (HD / 16), kLines = kPfKeys / kLineKeys;
                const int lt = t0 + lane % kLines * kLineKeys;
                const KeyPlace line = next_tile_place(lt, lbs);
                const int lblk = __shfl_sync(0xFFFFFFFFu, win, (line.entry - wbase) & 31);
                if (lane < 2 * kLines && lt + kPfKeys < kend && line.entry - wbase < 32 && lblk >= 0 && lblk < a.num_blocks)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(
                        (lane < kLines ? a.key_scales : a.value_scales) +
                        (((static_cast<int64_t>(lblk) * a.n_kv + kvh) << lbs) + line.row) * (HD / 16)));
            }
        }
        if (F4 && aborted) asm volatile("cp.async.wait_all;" ::: "memory");
        if (aborted && lane == 0) {
            flag(a.status, KVFP8_DEV_TIMEOUT);
            *abort_flag = 1;
            // let copies already issued land before the CTA's shared memory goes away
            for (int k = max(0, issued - L::kNS); k < issued; ++k)
                mbar_wait(bar(L::kFull, k % L::kNS), (k / L::kNS) & 1, &never);
        }
    } else if (warp == kPfMmaWarp) {
        // ------------------------------------------------------------ tensor-core issue
        // S(i) is issued before O(i-1), so the tensor core computes the next scores while the
        // softmax warps work on the current ones.
        if (lane == 0) {
            const uint32_t idesc_s = f16_idesc(kPfRows, kPfKeys), idesc_o = f16_idesc(kPfRows, L::kVRows);
            // operand descriptors computed once; each product adds its constant offset
            const uint64_t qdesc = sw128_desc(base + L::kQ), kdesc = sw128_desc(base + L::kK),
                           vdesc = sw128_desc(base + L::kV);
            bool ok = true;
            auto issue_o = [&](int t) {  // O += P(t) . V(t), then release tile t's buffers
                const int b = t % L::kNB;
                if (!mbar_wait(bar(L::kPReady, b), (t / L::kNB) & 1, abort_flag)) return false;
                tc_fence_after();
                const uint64_t vb = desc_at(vdesc, b * L::kVBuf);
#pragma unroll
                for (int k = 0; k < kPfKeys / 16; ++k)
                    umma_ts(tmem + L::kColO, tmem + 64 * b + 8 * k, desc_at(vb, k * 32), idesc_o,
                            (t > 0 || k > 0) ? 1u : 0u);
                umma_commit(bar(L::kKvFree, b));
                return true;
            };
            for (int i = 0; i < ntiles && ok; ++i) {
                const int b = i % L::kNB;
                ok = mbar_wait(bar(L::kKvReady, b), (i / L::kNB) & 1, abort_flag);
                // S(i) overwrites the buffer that held P(i-NB): O(i-NB) must have read it
                if (ok && i >= L::kNB)
                    ok = mbar_wait(bar(L::kKvFree, b), ((i / L::kNB) & 1) ^ 1u, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const uint64_t kb = desc_at(kdesc, b * L::kKBuf);
#pragma unroll
                for (int k = 0; k < HD / 16; ++k) {
                    const uint64_t ad = desc_at(qdesc, (k >> 2) * (kPfRows * 128) + (k & 3) * 32);
                    const uint64_t bd = desc_at(kb, (k >> 2) * (kPfKeys * 128) + (k & 3) * 32);
                    umma_ss(tmem + 64 * b, ad, bd, idesc_s, k > 0 ? 1u : 0u);
                }
                umma_commit(bar(L::kSReady, b));
                if (i >= 1) ok = issue_o(i - 1);
            }
            if (ok) ok = issue_o(ntiles - 1);
            if (!ok) {
                flag(a.status, KVFP8_DEV_TIMEOUT);
                *abort_flag = 1;
                // let the products already issued finish before tensor memory is released
                umma_commit(bar(L::kDrain, 0));
                mbar_wait(bar(L::kDrain, 0), 0, &never);
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ conversion warps
        const int ct = tid - 128;  // 0 .. 32*kPfConvWarps-1
        constexpr int kCT = 32 * kPfConvWarps;
        if (ct < kPfRows) {  // q rows -> f16, 128-byte-swizzled K-major blocks of 64 head dims; row ct
            const int r = row0 + ct;
            const bool row_ok = r < nb * G;
            const int jq = row_ok ? r / G : 0, gq = row_ok ? r % G : 0;
            const __nv_bfloat16 *qrow =
                a.query + ((static_cast<int64_t>(qr.q0) + jq) * a.n_q + kvh * G + gq) * HD;
#pragma unroll 4
            for (int c = 0; c < HD / 8; ++c) {
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (row_ok) w = *reinterpret_cast<const uint4 *>(qrow + 8 * c);
                uint4 h;
                h.x = f16x2_from_f32(bf16lo(w.x), bf16hi(w.x));
                h.y = f16x2_from_f32(bf16lo(w.y), bf16hi(w.y));
                h.z = f16x2_from_f32(bf16lo(w.z), bf16hi(w.z));
                h.w = f16x2_from_f32(bf16lo(w.w), bf16hi(w.w));
                *reinterpret_cast<uint4 *>(bp + L::kQ + (c >> 3) * (kPfRows * 128) + sw128(ct, c & 7)) = h;
            }
        }
        if (L::kSumCol) {  // V^T rows HD..HD+15 of every buffer: ones, then zeros
            for (int e = ct; e < L::kNB * 128; e += kCT) {
                const int bb = e >> 7, w = e & 127;  // 128 16-byte words per buffer
                const uint32_t one = w < 8 ? 0x3C003C00u : 0u;
                *reinterpret_cast<uint4 *>(bp + L::kV + bb * L::kVBuf + HD * 128 + 16 * w) =
                    make_uint4(one, one, one, one);
            }
        }
        bool ok = true;
        for (int i = 0; i < ntiles && ok; ++i) {
            const int st = i % L::kNS, b = i % L::kNB;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kFull, st), (i / L::kNS) & 1, abort_flag));
            // the buffer's previous tile (i-NB) has been through both products (F4: waited for below)
            if (!F4 && ok)
                ok = __all_sync(0xFFFFFFFFu,
                                mbar_wait(bar(L::kKvFree, b), ((i / L::kNB) & 1) ^ 1u, abort_flag));
            if (!ok) break;
            const uint64_t mask = meta[st];
            const uint8_t *kst = bp + L::kStage + st * L::kStageBytes;
            const uint8_t *vst = kst + kPfKeys * L::kRow;
            uint8_t *kdst0 = bp + L::kK + b * L::kKBuf;
            uint8_t *vdst = bp + L::kV + b * L::kVBuf;
            // K: 64 keys x HD/8 chunks of 8 fp8 -> one 16-byte f16 chunk (invalid keys: zeros);
            // eight consecutive threads take the eight chunks of one 64-dim block row, so each
            // quarter-warp's stores cover all 32 banks.
            // V^T by 8-key x 32-dim blocks: lane t converts dims (8j + 2(t%4), +1) of key t/4
            // (one e4m3 pair -> f16x2 per matrix j) and stmatrix.trans writes each dim's 8 keys
            // as one 16-byte row of V^T (head dims as rows, keys along K).
            // Every load of a round is issued before the first conversion, so their latencies
            // overlap (a store to shared memory would otherwise hold back the next load).
            constexpr int kKT = kPfKeys * (HD / 8) / kCT;                    // K tasks per thread
            constexpr int kVB = (kPfKeys / 8) * (HD / 32) / kPfConvWarps;    // V^T blocks per warp
            constexpr int kVG = kVB < 4 ? kVB : 4;                           // V^T blocks per round
            const int w4 = warp - 4;
            const uint32_t vbase = base + L::kV + b * L::kVBuf;
            const uint32_t vsel = static_cast<uint32_t>(2 * (lane & 3)) | static_cast<uint32_t>(2 * (lane & 3) + 1) << 4;
            uint2 kw[kKT];
            uint4 vw[kVG][2];
            auto v_load = [&](int g0) {
#pragma unroll
                for (int j = 0; j < kVG; ++j) {
                    const int blk = w4 + (g0 + j) * kPfConvWarps;
                    const int ko = blk % (kPfKeys / 8), dg = blk / (kPfKeys / 8);
                    const int key = ko * 8 + (lane >> 2);
                    const int sgi = (32 * dg) / L::kSeg, cc = ((32 * dg) % L::kSeg) >> 4;
                    const uint8_t *vrow = vst + sgi * kPfKeys * L::kSeg;
                    vw[j][0] = *reinterpret_cast<const uint4 *>(vrow + swz<L::kSeg>(key, cc));
                    vw[j][1] = *reinterpret_cast<const uint4 *>(vrow + swz<L::kSeg>(key, cc + 1));
                    if (!((mask >> key) & 1ull)) vw[j][0] = vw[j][1] = make_uint4(0u, 0u, 0u, 0u);
                }
            };
            auto v_store = [&](int g0) {
#pragma unroll
                for (int j = 0; j < kVG; ++j) {
                    const int blk = w4 + (g0 + j) * kPfConvWarps;
                    const int ko = blk % (kPfKeys / 8), dg = blk / (kPfKeys / 8);
                    const uint4 lo = vw[j][0], hi = vw[j][1];
                    const uint32_t wd[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    uint32_t r[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)  // bytes 8q + 2(t%4), +1 of the key's 32
                        r[q] = f16x2_from_e4m3x2(__byte_perm(wd[2 * q], wd[2 * q + 1], vsel));
                    const int n = 32 * dg + 8 * (lane >> 3) + (lane & 7);  // V^T row this lane addresses
                    stsm_x4_t(vbase + sw128(n, ko), r[0], r[1], r[2], r[3]);
                }
            };
            if constexpr (F4) {
                // K units, then V units, over the warps
                constexpr int kU = F4Unit<HD>::kPer64, kMine = 2 * kU / kPfConvWarps;
                const uint32_t codes = base + L::kStage + st * L::kStageBytes, scales = codes + L::kScales;
                F4Unit<HD> un[kMine];
#pragma unroll
                for (int j = 0; j < kMine; ++j) {
                    const int u = w4 + j * kPfConvWarps;
                    if (u < kU)
                        un[j].template load<true>(codes, scales, mask, u, lane);
                    else
                        un[j].template load<false>(codes + kPfKeys * L::kRow, scales + L::kScaleSide, mask, u - kU, lane);
                }
                // the codes are in registers: the stage is refilled while the tile's buffer is waited for
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::kEmpty, st));
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kKvFree, b), ((i / L::kNB) & 1) ^ 1u, abort_flag));
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < kMine; ++j) {
                    const int u = w4 + j * kPfConvWarps;
                    if (u < kU) {
                        un[j].store_k(base + L::kK + b * L::kKBuf, kPfKeys * 128, u, lane);
                    } else {
                        un[j].drop_nan(nan_seen);
                        un[j].store_v(vbase, u - kU, lane);
                    }
                }
            } else {
#pragma unroll
            for (int j = 0; j < kKT; ++j) {
                const int task = ct + j * kCT;
                const int key = task / (HD / 8), c = task % (HD / 8);  // dims 8c .. 8c+7
                const int sgi = (8 * c) / L::kSeg, within = (8 * c) % L::kSeg;
                kw[j] = *reinterpret_cast<const uint2 *>(kst + sgi * kPfKeys * L::kSeg +
                                                         swz<L::kSeg>(key, within >> 4) + (within & 8));
                if (!((mask >> key) & 1ull)) kw[j] = make_uint2(0u, 0u);
            }
            v_load(0);
#pragma unroll
            for (int j = 0; j < kKT; ++j) {
                const int task = ct + j * kCT;
                const int key = task / (HD / 8), c = task % (HD / 8);
                const uint2 w = kw[j];
                uint4 h;
                h.x = f16x2_from_e4m3x2(w.x);
                h.y = f16x2_from_e4m3x2_hi(w.x);
                h.z = f16x2_from_e4m3x2(w.y);
                h.w = f16x2_from_e4m3x2_hi(w.y);
                *reinterpret_cast<uint4 *>(kdst0 + (c >> 3) * (kPfKeys * 128) + sw128(key, c & 7)) = h;
            }
            v_store(0);
#pragma unroll
            for (int g0 = kVG; g0 < kVB; g0 += kVG) {
                v_load(g0);
                v_store(g0);
            }
            }
            if (ct == 0) buf_mask[b] = mask;  // for the softmax warps, released with kv_ready
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                if (!F4) mbar_arrive(bar(L::kEmpty, st));  // the FP8 stage may be refilled
                mbar_arrive(bar(L::kKvReady, b));    // K(i), V^T(i) (and Q) are ready
            }
        }
        if (!ok && lane == 0) {
            flag(a.status, KVFP8_DEV_TIMEOUT);
            *abort_flag = 1;
        }
    } else {
        // ------------------------------------------------------------ softmax warps
        const int r = row0 + tid;                   // this thread's score row (TMEM lane tid)
        const bool row_ok = r < nb * G;
        const int jq = row_ok ? r / G : 0, gq = row_ok ? r % G : 0;
        const int pos = Ls - nb + jq;               // last key position the row may see
        const float score_scale = a.sm_scale * sk * 1.4426950408889634f;  // log2(e)
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        constexpr float kHead = F4 ? kF4Head : 0.f;
        float m_used = -INFINITY, lsum = 0.f;
        bool ok = true;
        for (int i = 0; i < ntiles && ok; ++i) {
            const int b = i % L::kNB, ph = (i / L::kNB) & 1;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kSReady, b), ph, abort_flag));
            // the tile's valid-key mask (already complete: S(i) needed the same phase)
            if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kKvReady, b), ph, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const uint64_t mask = buf_mask[b];
            uint32_t s[2][32];
            tmem_ld32(lane_addr + 64 * b, s[0]);
            tmem_ld32(lane_addr + 64 * b + 32, s[1]);
            tmem_wait_ld();
            // causal mask, scale, running maximum (a key past the row's position, past the
            // sequence or in a bad block scores -inf; keys past kend are past every position).
            // A tile every row of the warp sees whole takes no mask: the maximum is taken on
            // the raw scores (the smallest when the scale is negative) and scaled once, and
            // the scale is applied inside the exponent's fma.
            const int k0 = key_tile(i) * kPfKeys;
            const int vis_n = row_ok ? min(kPfKeys, max(0, pos - k0 + 1)) : 0;  // keys 0..vis_n-1
            const uint64_t vis = mask & (vis_n >= 64 ? ~0ull : ((1ull << vis_n) - 1));
            float mx, mult;
            if (__all_sync(0xFFFFFFFFu, vis == ~0ull)) {
                mx = (score_scale >= 0.f ? extreme64<true>(s) : extreme64<false>(s)) * score_scale;
                mult = score_scale;
            } else {
                mx = -INFINITY;
                mult = 1.f;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float v = ((vis >> (32 * h + c)) & 1ull)
                                            ? __uint_as_float(s[h][c]) * score_scale
                                            : -INFINITY;
                        s[h][c] = __float_as_uint(v);
                        mx = fmaxf(mx, v);
                    }
            }
            // rescale O only when the maximum grew by more than 2^8 (first visible keys: O is
            // still zero for this row, nothing to rescale)
            float factor = 1.f;
            if (mx > -INFINITY) {
                if (m_used == -INFINITY) {
                    m_used = mx - kHead;
                } else if (mx > m_used + (8.f + kHead)) {
                    factor = ex2(m_used - (mx - kHead));
                    m_used = mx - kHead;
                }
            }
            if (__any_sync(0xFFFFFFFFu, factor != 1.f)) {
                // O(i-1) must be complete before O is rescaled (with its row-sum column)
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kKvFree, (i - 1) % L::kNB),
                                                       ((i - 1) / L::kNB) & 1, abort_flag));
                if (!ok) break;
                tc_fence_after();
                lsum *= factor;
#pragma unroll 1
                for (int c0 = 0; c0 < (L::kSumCol ? HD + 32 : HD); c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(lane_addr + L::kColO + c0, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * factor);
                    tmem_st32(lane_addr + L::kColO + c0, o);
                }
            }
            // P = 2^(s*mult - m) as f16 pairs over the first 32 columns of this S buffer.  E4M3: one
            // packed fma, one f16 pack and one f16x2 exp2 per pair (x <= 2^3 by the rescale rule, so
            // P <= 2^8; F4: 2^15).  F4: the exponent stays float and the weight is rounded, once: an fp16 exponent
            // of 8 to 16 moves a weight by up to 2^-8.5, a rounded weight by 2^-11.
            uint32_t p[32];
            const float msub = m_used == -INFINITY ? 0.f : m_used;
            const uint64_t mul2 = pk2(mult, mult), sub2 = pk2(-msub, -msub);
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                const int h = c >> 4, e = (2 * c) & 31;
                const float2 x = upk2(fma_f32x2(pk2u(s[h][e], s[h][e + 1]), mul2, sub2));
                p[c] = F4 ? f16x2_from_f32(ex2(x.x), ex2(x.y)) : ex2_f16x2(f16x2_from_f32(x.x, x.y));
                if (!L::kSumCol) lsum += f16lo_f32(p[c]) + f16hi_f32(p[c]);
            }
            tmem_st32(lane_addr + 64 * b, p);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kPReady, b));
        }
        if (ok)
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kKvFree, (ntiles - 1) % L::kNB),
                                                   ((ntiles - 1) / L::kNB) & 1, abort_flag));
        if (ok) {
            tc_fence_after();
            if (L::kSumCol) {  // the row's sum of P, accumulated by the O product
                uint32_t o[32];
                tmem_ld32(lane_addr + L::kColO + HD, o);
                tmem_wait_ld();
                lsum = __uint_as_float(o[0]);
            }
            const float inv = lsum > 0.f ? sv / lsum : 0.f;
            uint32_t nan_groups = 0;
            if constexpr (F4) {
                if (*nan_seen) {
                    const int key0 = kSplit ? tile_lo * kPfKeys : 0;  // of this part's keys
                    nan_groups = nan_value_groups<HD>(a, seq, kvh, key0,
                                                      row_ok ? kSplit ? min(pos, key0 + ntiles * kPfKeys - 1) : pos : -1);
                }
            }
            // this row in the parts' results, when there are several
            const int64_t prow = kSplit ? ((((static_cast<int64_t>(seq) * a.row_tiles + tile) * a.n_kv + kvh) * a.splits +
                                                     blockIdx.y) * kPfRows) + tid : 0;
            const float part_inv = !kSplit || lsum == 0.f ? 0.f : 1.f / lsum;
            if (kSplit && row_ok) a.part_lse[prow] = lsum == 0.f ? -INFINITY : m_used + __log2f(lsum);
            uint4 *orow = reinterpret_cast<uint4 *>(
                a.out + ((static_cast<int64_t>(qr.q0) + jq) * a.n_q + kvh * G + gq) * HD);
#pragma unroll 1
            for (int c0 = 0; c0 < HD; c0 += 32) {
                uint32_t o[32];
                tmem_ld32(lane_addr + L::kColO + c0, o);
                tmem_wait_ld();
                if constexpr (kSplit) {
                    if (row_ok) store_part(a.part_o + prow * HD, o, part_inv, nan_groups, c0);
                } else if (row_ok) {
#pragma unroll
                    for (int c = 0; c < 32; c += 8) {
                        uint4 w;
                        auto word = [&](int k) {  // output word k of the 32 dims
                            const int e = 2 * o_word<F4>(k);
                            return bf16x2_from_f32(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                        };
                        w.x = word(c / 2);
                        w.y = word(c / 2 + 1);
                        w.z = word(c / 2 + 2);
                        w.w = word(c / 2 + 3);
                        if (F4 && nan_groups != 0u) {
                            const int d = c0 + c;
                            w = make_uint4(nan_in(w.x, nan_groups, d), nan_in(w.y, nan_groups, d),
                                           nan_in(w.z, nan_groups, d), nan_in(w.w, nan_groups, d));
                        }
                        orow[(c0 + c) / 8] = w;
                    }
                }
            }
        } else if (lane == 0) {
            flag(a.status, KVFP8_DEV_TIMEOUT);
            *abort_flag = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kPfMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// ---------------------------------------------------------------- two row tiles per CTA
//
// For head_dim 64 and 128 when a (sequence, kv head) has more than 128 score rows: one CTA
// takes 256 rows as two row tiles that share every converted K/V tile, so the copies and
// the conversion are paid once per two tiles of tensor work.  Keys go in tiles of 128: the
// score product S = Q.K^T then has N = 128, where a kind::f16 product runs at the tensor
// core's full rate (at N = 64 the shared-memory reads of its two operands bound it to about
// two thirds of that), and each tile costs half as many products, commits and waits.
//
// Tensor memory (512 columns at head_dim 128): S[r] at 128*r (P written over its first 64
// columns as f16), O[r] at 256 + head_dim*r.  Each row tile has one score buffer: the tensor
// core runs the products one thread issues in order, and S(r, i+1) is issued after O(r, i),
// so the next scores land only after the product that reads P.  The two row tiles take
// turns: while one row tile's softmax works, the tensor core runs the other's O and next S.
// The commit that signals S(r, i) also covers O(r, i-1), so the softmax may rescale O as
// soon as its scores are ready.  The rows sum P themselves (fp32, in pairs).
//
// FP8 K/V arrive by TMA in halves of 64 keys (a staging ring of NS halves) and are converted
// into two f16 K buffers and two V^T buffers of 128 keys.  A K buffer is free once both row
// tiles' S products are done with it; a V^T buffer (and the valid-key masks stored with it)
// once both O products are.
//
// Warps (14): 0-3 softmax of row tile 0, 4-7 softmax of row tile 1 (warp w reads TMEM
// lanes 32*(w%4)..+31), 8-11 conversion, 12 tensor-core issue (and TMEM allocation), 13 TMA.
constexpr int kP2Rows = 2 * kPfRows;
constexpr int kP2Keys = 2 * kPfKeys;   // keys per tile; FP8 staging and conversion go by halves
constexpr int kP2ConvWarps = 4;
constexpr int kP2MmaWarp = 8 + kP2ConvWarps, kP2TmaWarp = kP2MmaWarp + 1;
constexpr int kP2Warps = kP2TmaWarp + 1;

template <int HD, bool F4>
struct Pf2Smem {
    static constexpr int kRow = F4 ? HD / 2 : HD;
    static constexpr int kSeg = kRow >= 128 ? 128 : kRow;
    static constexpr int kSegs = kRow / kSeg;
    static constexpr int kNS = HD < 128 ? (F4 ? 8 : 4) : F4 ? 3 : 2;  // staging halves
    static constexpr int kQTile = HD * 256;                        // one row tile of Q (f16)
    static constexpr int kQ = 0;
    // K f16: HD/64 blocks x 128 keys x 128 B; V^T f16: 2 key blocks x HD rows x 128 B
    static constexpr int kKBuf = HD * 256, kVBuf = HD * 256;
    static constexpr int kK = kQ + 2 * kQTile;
    static constexpr int kV = kK + 2 * kKBuf;
    static constexpr int kStage = kV + 2 * kVBuf;
    static constexpr int kScaleSide = F4 ? kPfKeys * (HD / 16) : 0;
    static constexpr int kScales = 2 * kPfKeys * kRow;             // K then V of 64 keys, then (F4)
    static constexpr int kStageBytes = kScales + 2 * kScaleSide;   // their scale bytes
    static constexpr int kBars = kStage + kNS * kStageBytes;
    // mbarriers: full[NS], empty[NS], then per buffer k_ready, v_ready, k_free, v_free, then
    // per row tile s_ready, p_ready, o_done, and one to drain the tensor core on a timeout
    static constexpr int kFull = kBars, kEmpty = kFull + 8 * kNS, kKReady = kEmpty + 8 * kNS;
    static constexpr int kVReady = kKReady + 16, kKFree = kVReady + 16, kVFree = kKFree + 16;
    static constexpr int kSReady = kVFree + 16, kPReady = kSReady + 16, kODone = kPReady + 16;
    static constexpr int kDrain = kODone + 16;
    static constexpr int kMeta = kDrain + 8;                       // valid-key mask per stage
    static constexpr int kBufMask = kMeta + 8 * kNS;               // per V^T buffer, two halves
    static constexpr int kMisc = kBufMask + 32;                    // tmem base, abort flag, NaN seen
    static constexpr int kTotal = kMisc + 16;
    static constexpr uint32_t kTmemCols = 512;
    __host__ __device__ static constexpr uint32_t col_s(int r) { return static_cast<uint32_t>(128 * r); }
    __host__ __device__ static constexpr uint32_t col_o(int r) { return static_cast<uint32_t>(256 + HD * r); }
    // P of keys 16k..16k+15 (f16 pairs, 8 columns): the first half of the 32 columns that
    // held the scores of keys 32(k/2)..+31, so each 32-key chunk's P overwrites only its own
    // scores
    __host__ __device__ static constexpr uint32_t col_p(int k) { return static_cast<uint32_t>(32 * (k >> 1) + 8 * (k & 1)); }
};

template <int HD, bool F4, bool kSplit>
__global__ void __launch_bounds__(kP2Warps * 32, 1)
prefill2_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                const PrefillArgs<F4> a) {
    using L = Pf2Smem<HD, F4>;
    static_assert(L::kTotal + 1024 <= 232448, "shared memory");
    static_assert(L::col_o(1) + HD <= L::kTmemCols, "tensor memory");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *bp = smem_raw + (base - raw);
    volatile uint64_t *meta = reinterpret_cast<volatile uint64_t *>(bp + L::kMeta);
    volatile uint64_t *buf_mask = reinterpret_cast<volatile uint64_t *>(bp + L::kBufMask);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bp + L::kMisc);
    volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(bp + L::kMisc + 4);
    volatile int32_t *nan_seen = reinterpret_cast<volatile int32_t *>(bp + L::kMisc + 8);
    auto bar = [&](int off, int i) { return base + static_cast<uint32_t>(off + 8 * i); };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kvh = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.n_kv));
    const int ctile = static_cast<int>((blockIdx.x / static_cast<unsigned>(a.n_kv)) % static_cast<unsigned>(a.row_tiles));
    const int rank = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.n_kv * a.row_tiles));

    const float sk = load_scale(a.k_scale, a.scale_dtype);
    const float sv = load_scale(a.v_scale, a.scale_dtype);
    // longest sequences first; the K buffers are free scratch until the pipeline starts
    const int seq = seq_of_rank(a.seq_lens, a.num_seqs, a.max_len, rank,
                                reinterpret_cast<uint32_t *>(bp + L::kK));
    if (!scale_ok(sk) || !scale_ok(sv)) {
        if (blockIdx.x == 0 && tid == 0) flag(a.status, KVFP8_DEV_BAD_SCALE);
        return;
    }
    const int raw_nq = a.qsl[seq + 1] - a.qsl[seq];
    const QueryRange qr = query_range(a.qsl, seq, a.qmax, a.qrows);
    const int Lraw = a.seq_lens[seq];
    const int Ls = min(max(Lraw, 0), a.max_len);
    if (ctile == 0 && kvh == 0 && tid == 0 &&
        (qr.count != raw_nq || Lraw < 0 || Lraw > a.max_len || qr.count > Ls))
        flag(a.status, KVFP8_DEV_BAD_BLOCK);
    const int nb = qr.count, G = a.group;
    const int row0 = ctile * kP2Rows;                 // first score row of this CTA
    if (row0 >= nb * G) return;
    const int j_last = min(nb, (row0 + kP2Rows + G - 1) / G) - 1;
    const int kend = Ls - nb + j_last + 1;            // keys the CTA's last row may see
    int ntiles = kend > 0 ? (kend + kP2Keys - 1) / kP2Keys : 0;
    int tile_lo = 0;  // this CTA's key tiles: ntiles from tile_lo on
    if constexpr (kSplit) {
        const int parts = split_parts(a.splits, ntiles, kP2Keys);
        const int part = static_cast<int>(blockIdx.y);
        if (part >= parts) return;
        tile_lo = static_cast<int>(static_cast<int64_t>(part) * ntiles / parts);
        ntiles = static_cast<int>(static_cast<int64_t>(part + 1) * ntiles / parts) - tile_lo;
    }
    const int rot = ntiles > 0 ? static_cast<int>((static_cast<int64_t>(ctile) * ntiles) / a.row_tiles) % ntiles : 0;
    auto key_tile = [&](int i) { const int k = i + rot; return (k >= ntiles ? k - ntiles : k) + (kSplit ? tile_lo : 0); };

    if (ntiles == 0) {  // every row of the CTA sees no key: zero rows
        if (tid < kP2Rows) {
            const int r = row0 + tid;
            if (r < nb * G) {
                const int j = r / G, g = r % G;
                uint4 *o = reinterpret_cast<uint4 *>(
                    a.out + ((static_cast<int64_t>(qr.q0) + j) * a.n_q + kvh * G + g) * HD);
                for (int c = 0; c < HD / 8; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        return;
    }

    if (tid == 0) {
        for (int s = 0; s < L::kNS; ++s) {
            mbar_init(bar(L::kFull, s), F4 ? 33 : 1);  // F4: and every lane's scale copies
            mbar_init(bar(L::kEmpty, s), kP2ConvWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(L::kKReady, b), kP2ConvWarps);
            mbar_init(bar(L::kVReady, b), kP2ConvWarps);
            mbar_init(bar(L::kKFree, b), 1);
            mbar_init(bar(L::kVFree, b), 1);
            mbar_init(bar(L::kSReady, b), 1);
            mbar_init(bar(L::kPReady, b), 4);
            mbar_init(bar(L::kODone, b), 1);
        }
        mbar_init(bar(L::kDrain, 0), 1);
        *abort_flag = 0;
        if (F4) *nan_seen = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kP2MmaWarp) {
        tmem_alloc(base + L::kMisc, L::kTmemCols);
        tmem_relinquish();
    }
    if (warp == kP2TmaWarp && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmk)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmv)) : "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const volatile int32_t never = 0;

    if (warp == kP2TmaWarp) {
        // ------------------------------------------------------------ TMA producer
        // half h of the key pass (64 keys of tile h/2): lane p < nbox fetches K box p, lane
        // nbox + p V box p
        const int32_t *bt = a.block_tables + static_cast<int64_t>(seq) * a.max_blocks_per_seq;
        const int bs = a.block_size, br = a.box_rows;
        const int lbs = __ffs(bs) - 1;
        const int nbox = kPfKeys / br;
        const bool k_lane = lane < nbox;
        const int p = k_lane ? lane : lane - nbox;
        const bool box_lane = lane < 2 * nbox;
        const CUtensorMap *map = k_lane ? &tmk : &tmv;
        const uint32_t side = k_lane ? 0u : static_cast<uint32_t>(kPfKeys * L::kRow);
        int wbase = -(1 << 30);
        int32_t win = -1;
        int issued = 0;
        bool aborted = false;
        for (int h = 0; h < 2 * ntiles; ++h) {
            const int st = h % L::kNS;
            const int t0 = key_tile(h >> 1) * kP2Keys + (h & 1) * kPfKeys;
            const int t = t0 + p * br;
            const bool any = t0 < kend;
            if (any) {
                const int e0 = t0 >> lbs, e1 = (min(kend, t0 + kPfKeys) - 1) >> lbs;
                if (e0 < wbase || e1 >= wbase + 32) {
                    wbase = e0;
                    win = wbase + lane < a.max_blocks_per_seq ? bt[wbase + lane] : -1;
                }
            }
            const int blk = __shfl_sync(0xFFFFFFFFu, win, ((t >> lbs) - wbase) & 31);
            const bool live = any && box_lane && t < kend;
            const bool good = live && blk >= 0 && blk < a.num_blocks;
            if (live && !good && k_lane) flag(a.status, KVFP8_DEV_BAD_BLOCK);
            const int row = blk * bs + (t & (bs - 1));
            uint64_t part = 0;
            if (good && k_lane) {
                const int nk = min(br, kend - t);
                part = (nk >= 64 ? ~0ull : ((1ull << nk) - 1)) << (p * br);
            }
            const uint64_t mask =
                static_cast<uint64_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(part))) |
                static_cast<uint64_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(part >> 32))) << 32;
            const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, good && k_lane));
            if (lane == 0) {
                if (!mbar_wait(bar(L::kEmpty, st), ((h / L::kNS) & 1) ^ 1u, abort_flag)) {
                    aborted = true;
                } else {
                    meta[st] = mask;
                    const uint32_t full = bar(L::kFull, st);
                    if (boxes > 0)
                        mbar_arrive_tx(full, static_cast<uint32_t>(boxes * 2 * br * L::kRow));
                    else
                        mbar_arrive(full);
                    ++issued;
                }
            }
            aborted = __shfl_sync(0xFFFFFFFFu, aborted, 0);
            if (aborted) break;
            __syncwarp();  // as in the one-row-tile kernel
            if (good) {
                const uint32_t full = bar(L::kFull, st);
                const uint32_t dst = base + L::kStage + st * L::kStageBytes + side +
                                     static_cast<uint32_t>(p * br * L::kSeg);
#pragma unroll
                for (int sgi = 0; sgi < L::kSegs; ++sgi)
                    tma_load_3d(dst + static_cast<uint32_t>(sgi * kPfKeys * L::kSeg), map, 0,
                                kvh * L::kSegs + sgi, row, full);
            }
            if constexpr (F4) {
                const uint32_t stage = base + L::kStage + st * L::kStageBytes;
                copy_scales<HD>(a, kvh, t0, kend, lbs, win, wbase, stage + L::kScales, L::kScaleSide,
                                bar(L::kFull, st), lane);
            }
        }
        if (F4 && aborted) asm volatile("cp.async.wait_all;" ::: "memory");
        if (aborted && lane == 0) {
            flag(a.status, KVFP8_DEV_TIMEOUT);
            *abort_flag = 1;
            for (int k = max(0, issued - L::kNS); k < issued; ++k)
                mbar_wait(bar(L::kFull, k % L::kNS), (k / L::kNS) & 1, &never);
        }
    }
    else if (warp == kP2MmaWarp) {
        // ------------------------------------------------------------ tensor-core issue
        // S(r, 0) for both row tiles, then per tile i and row tile r: O(r, i) once P(r, i) is
        // ready, then S(r, i+1) into the same columns.
        if (lane == 0) {
            const uint32_t idesc_s = f16_idesc(kPfRows, kP2Keys), idesc_o = f16_idesc(kPfRows, HD);
            // operand descriptors computed once; each product adds its constant offset
            const uint64_t qdesc = sw128_desc(base + L::kQ), kdesc = sw128_desc(base + L::kK),
                           vdesc = sw128_desc(base + L::kV);
            auto issue_s = [&](int i, int r) {
                const uint64_t qd = desc_at(qdesc, r * L::kQTile);
                const uint64_t kb = desc_at(kdesc, (i & 1) * L::kKBuf);
#pragma unroll
                for (int k = 0; k < HD / 16; ++k)
                    umma_ss(tmem + L::col_s(r), desc_at(qd, (k >> 2) * (kPfRows * 128) + (k & 3) * 32),
                            desc_at(kb, (k >> 2) * (kP2Keys * 128) + (k & 3) * 32), idesc_s,
                            k > 0 ? 1u : 0u);
                umma_commit(bar(L::kSReady, r));
            };
            auto issue_o = [&](int i, int r) {
                const uint64_t vb = desc_at(vdesc, (i & 1) * L::kVBuf);
#pragma unroll
                for (int k = 0; k < kP2Keys / 16; ++k)
                    umma_ts(tmem + L::col_o(r), tmem + L::col_s(r) + L::col_p(k),
                            desc_at(vb, (k >> 2) * (HD * 128) + (k & 3) * 32), idesc_o,
                            (i > 0 || k > 0) ? 1u : 0u);
            };
            bool ok = mbar_wait(bar(L::kKReady, 0), 0, abort_flag);
            if (ok) {
                tc_fence_after();
                issue_s(0, 0);
                issue_s(0, 1);
                umma_commit(bar(L::kKFree, 0));
            }
            for (int i = 0; i < ntiles && ok; ++i) {
                const int b = i & 1;
                ok = mbar_wait(bar(L::kVReady, b), (i >> 1) & 1, abort_flag);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (ok) ok = mbar_wait(bar(L::kPReady, r), i & 1, abort_flag);
                    if (ok && r == 0 && i + 1 < ntiles)
                        ok = mbar_wait(bar(L::kKReady, (i + 1) & 1), ((i + 1) >> 1) & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    issue_o(i, r);
                    if (i + 1 == ntiles) umma_commit(bar(L::kODone, r));
                    if (r == 1) umma_commit(bar(L::kVFree, b));
                    if (i + 1 < ntiles) {
                        issue_s(i + 1, r);
                        if (r == 1) umma_commit(bar(L::kKFree, (i + 1) & 1));
                    }
                }
            }
            if (!ok) {
                flag(a.status, KVFP8_DEV_TIMEOUT);
                *abort_flag = 1;
                // let the products already issued finish before tensor memory is released
                umma_commit(bar(L::kDrain, 0));
                mbar_wait(bar(L::kDrain, 0), 0, &never);
            }
        }
    }
    else if (warp >= 8) {
        // ------------------------------------------------------------ conversion warps
        const int ct = tid - 256;  // 0 .. 32*kP2ConvWarps-1
        constexpr int kCT = 32 * kP2ConvWarps;
        // q rows -> f16, 128-byte-swizzled K-major blocks of 64 head dims: rows ct and ct+128
#pragma unroll 1
        for (int rr = ct; rr < kP2Rows; rr += kCT) {
            const int r = row0 + rr;
            const bool row_ok = r < nb * G;
            const int jq = row_ok ? r / G : 0, gq = row_ok ? r % G : 0;
            const __nv_bfloat16 *qrow =
                a.query + ((static_cast<int64_t>(qr.q0) + jq) * a.n_q + kvh * G + gq) * HD;
            uint8_t *qt = bp + L::kQ + (rr / kPfRows) * L::kQTile;
            const int lr = rr % kPfRows;
#pragma unroll 4
            for (int c = 0; c < HD / 8; ++c) {
                uint4 w = make_uint4(0u, 0u, 0u, 0u);
                if (row_ok) w = *reinterpret_cast<const uint4 *>(qrow + 8 * c);
                uint4 h;
                h.x = f16x2_from_f32(bf16lo(w.x), bf16hi(w.x));
                h.y = f16x2_from_f32(bf16lo(w.y), bf16hi(w.y));
                h.z = f16x2_from_f32(bf16lo(w.z), bf16hi(w.z));
                h.w = f16x2_from_f32(bf16lo(w.w), bf16hi(w.w));
                *reinterpret_cast<uint4 *>(qt + (c >> 3) * (kPfRows * 128) + sw128(lr, c & 7)) = h;
            }
        }
        // K: a task is 8 dims of one key (8 FP8 bytes in, one 16-byte f16 chunk out); eight
        // consecutive threads take the eight chunks of one 64-dim block row, so each
        // quarter-warp's stores cover all 32 banks
        constexpr int kKT = kPfKeys * (HD / 8) / kCT;                    // K tasks per thread
        constexpr int kVB = (kPfKeys / 8) * (HD / 32) / kP2ConvWarps;    // V^T blocks per warp
        constexpr int kVG = kVB < 4 ? kVB : 4;                           // V^T blocks per round
        const int w8 = warp - 8;
        const uint32_t vsel = static_cast<uint32_t>(2 * (lane & 3)) | static_cast<uint32_t>(2 * (lane & 3) + 1) << 4;
        bool ok = true;
        for (int h = 0; h < 2 * ntiles && ok; ++h) {
            const int st = h % L::kNS, i = h >> 1, hf = h & 1, b = i & 1;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kFull, st), (h / L::kNS) & 1, abort_flag));
            // the K buffer's previous tile (i-2) is through both S products
            if (ok && hf == 0)
                ok = __all_sync(0xFFFFFFFFu,
                                mbar_wait(bar(L::kKFree, b), ((i >> 1) & 1) ^ 1u, abort_flag));
            if (!ok) break;
            const uint64_t mask = meta[st];
            const uint8_t *kst = bp + L::kStage + st * L::kStageBytes;
            const uint8_t *vst = kst + kPfKeys * L::kRow;
            // this half's 64 keys: rows 64*hf.. of every 64-dim block of the K buffer
            uint8_t *kdst0 = bp + L::kK + b * L::kKBuf + hf * (kPfKeys * 128);
            // and key block hf of the V^T buffer
            const uint32_t vbase = base + L::kV + b * L::kVBuf + hf * (HD * 128);
            uint4 vw[kVG][2];
            auto v_load = [&](int g0) {
#pragma unroll
                for (int q = 0; q < kVG; ++q) {
                    const int blk = w8 + (g0 + q) * kP2ConvWarps;
                    const int ko = blk % (kPfKeys / 8), dg = blk / (kPfKeys / 8);
                    const int key = ko * 8 + (lane >> 2);
                    const int sgi = (32 * dg) / L::kSeg, cc = ((32 * dg) % L::kSeg) >> 4;
                    const uint8_t *vrow = vst + sgi * kPfKeys * L::kSeg;
                    vw[q][0] = *reinterpret_cast<const uint4 *>(vrow + swz<L::kSeg>(key, cc));
                    vw[q][1] = *reinterpret_cast<const uint4 *>(vrow + swz<L::kSeg>(key, cc + 1));
                    if (!((mask >> key) & 1ull)) vw[q][0] = vw[q][1] = make_uint4(0u, 0u, 0u, 0u);
                }
            };
            auto v_store = [&](int g0) {
#pragma unroll
                for (int q = 0; q < kVG; ++q) {
                    const int blk = w8 + (g0 + q) * kP2ConvWarps;
                    const int ko = blk % (kPfKeys / 8), dg = blk / (kPfKeys / 8);
                    const uint4 lo = vw[q][0], hi = vw[q][1];
                    const uint32_t wd[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    uint32_t rv[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)  // bytes 8e + 2(t%4), +1 of the key's 32
                        rv[e] = f16x2_from_e4m3x2(__byte_perm(wd[2 * e], wd[2 * e + 1], vsel));
                    const int n = 32 * dg + 8 * (lane >> 3) + (lane & 7);
                    stsm_x4_t(vbase + sw128(n, ko), rv[0], rv[1], rv[2], rv[3]);
                }
            };
            constexpr int kU4 = F4Unit<HD>::kPer64 / kP2ConvWarps;  // F4: units a warp has of each side
            F4Unit<HD> uv[kU4];
            if constexpr (F4) {
                const uint32_t codes = base + L::kStage + st * L::kStageBytes, scales = codes + L::kScales;
                F4Unit<HD> uk[kU4];
#pragma unroll
                for (int q = 0; q < kU4; ++q) {
                    uk[q].template load<true>(codes, scales, mask, w8 + q * kP2ConvWarps, lane);
                    uv[q].template load<false>(codes + kPfKeys * L::kRow, scales + L::kScaleSide, mask,
                                               w8 + q * kP2ConvWarps, lane);
                }
#pragma unroll
                for (int q = 0; q < kU4; ++q)
                    uk[q].store_k(base + L::kK + b * L::kKBuf + hf * (kPfKeys * 128), kP2Keys * 128,
                                  w8 + q * kP2ConvWarps, lane);
            } else {
            // K: every load of the half before its conversions
            uint2 kw[kKT];
#pragma unroll
            for (int q = 0; q < kKT; ++q) {
                const int task = ct + q * kCT;
                const int key = task / (HD / 8), c = task % (HD / 8);
                const int sgi = (8 * c) / L::kSeg, within = (8 * c) % L::kSeg;
                kw[q] = *reinterpret_cast<const uint2 *>(kst + sgi * kPfKeys * L::kSeg +
                                                         swz<L::kSeg>(key, within >> 4) + (within & 8));
                if (!((mask >> key) & 1ull)) kw[q] = make_uint2(0u, 0u);
            }
#pragma unroll
            for (int q = 0; q < kKT; ++q) {
                const int task = ct + q * kCT;
                const int key = task / (HD / 8), c = task % (HD / 8);
                const uint2 w = kw[q];
                uint4 h;
                h.x = f16x2_from_e4m3x2(w.x);
                h.y = f16x2_from_e4m3x2_hi(w.x);
                h.z = f16x2_from_e4m3x2(w.y);
                h.w = f16x2_from_e4m3x2_hi(w.y);
                *reinterpret_cast<uint4 *>(kdst0 + (c >> 3) * (kP2Keys * 128) + sw128(key, c & 7)) = h;
            }
            }
            if (hf == 1) {  // both halves of the tile's K are in place
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::kKReady, b));
            }
            // the V^T buffer's previous tile (i-2) is through both O products
            if (hf == 0)
                ok = __all_sync(0xFFFFFFFFu,
                                mbar_wait(bar(L::kVFree, b), ((i >> 1) & 1) ^ 1u, abort_flag));
            if (!ok) break;
            if constexpr (F4) {
#pragma unroll
                for (int q = 0; q < kU4; ++q) {
                    uv[q].drop_nan(nan_seen);
                    uv[q].store_v(vbase, w8 + q * kP2ConvWarps, lane);
                }
            } else {
                v_load(0);
                v_store(0);
#pragma unroll
                for (int g0 = kVG; g0 < kVB; g0 += kVG) {
                    v_load(g0);
                    v_store(g0);
                }
            }
            if (ct == 0) buf_mask[2 * b + hf] = mask;  // for the softmax warps, released with v_ready
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(L::kEmpty, st));
                if (hf == 1) mbar_arrive(bar(L::kVReady, b));
            }
        }
        if (!ok && lane == 0) {
            flag(a.status, KVFP8_DEV_TIMEOUT);
            *abort_flag = 1;
        }
    }
    else {
        // ------------------------------------------------------------ softmax warps
        const int rt = warp >> 2;                   // row tile 0 or 1
        const int r = row0 + tid;                   // this thread's score row
        const bool row_ok = r < nb * G;
        const int jq = row_ok ? r / G : 0, gq = row_ok ? r % G : 0;
        const int pos = Ls - nb + jq;               // last key position the row may see
        const float score_scale = a.sm_scale * sk * 1.4426950408889634f;  // log2(e)
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t scol = lane_addr + L::col_s(rt);
        constexpr float kHead = F4 ? kF4Head : 0.f;
        float m_used = -INFINITY;
        uint64_t lsum2 = pk2(0.f, 0.f);  // the row sum, in two fp32 halves
        bool ok = true;
        for (int i = 0; i < ntiles && ok; ++i) {
            const int b = i & 1;
            // S(rt, i) is done, and with it O(rt, i-1)
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kSReady, rt), i & 1, abort_flag));
            // the tile's valid-key masks (stored with its V^T)
            if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kVReady, b), (i >> 1) & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const int k0 = key_tile(i) * kP2Keys;
            const int vis_n = row_ok ? min(kP2Keys, max(0, pos - k0 + 1)) : 0;
            const uint64_t vis0 = buf_mask[2 * b] & (vis_n >= 64 ? ~0ull : ((1ull << vis_n) - 1));
            const uint64_t vis1 = buf_mask[2 * b + 1] &
                                  (vis_n >= 128 ? ~0ull : vis_n <= 64 ? 0ull : ((1ull << (vis_n - 64)) - 1));
            const bool whole = __all_sync(0xFFFFFFFFu, (vis0 & vis1) == ~0ull);
            auto vis_bits = [&](int c) {  // the visible keys among columns 32c..32c+31
                return static_cast<uint32_t>((c < 2 ? vis0 : vis1) >> (32 * (c & 1)));
            };
            // pass 1: the row's maximum over the tile (raw extreme, scaled once, on a whole
            // tile).  Chunks 0 and 1, then 2 and 3, each pair loaded together; 2 and 3 stay in
            // registers for pass 2.
            uint32_t sa[32], sb[32];
            float mx = -INFINITY, ext = score_scale >= 0.f ? -INFINITY : INFINITY;
            auto chunk_max = [&](const uint32_t (&sc)[32], int c) {
                if (whole) {
                    ext = score_scale >= 0.f ? fmaxf(ext, extreme32<true>(sc)) : fminf(ext, extreme32<false>(sc));
                } else {
                    const uint32_t bits = vis_bits(c);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if ((bits >> e) & 1u) mx = fmaxf(mx, __uint_as_float(sc[e]) * score_scale);
                }
            };
            tmem_ld32(scol, sa);
            tmem_ld32(scol + 32, sb);
            tmem_wait_ld();
            chunk_max(sa, 0);
            chunk_max(sb, 1);
            tmem_ld32(scol + 64, sa);
            tmem_ld32(scol + 96, sb);
            tmem_wait_ld();
            chunk_max(sa, 2);
            chunk_max(sb, 3);
            if (whole) mx = ext * score_scale;
            float factor = 1.f;
            if (mx > -INFINITY) {
                if (m_used == -INFINITY) {
                    m_used = mx - kHead;
                } else if (mx > m_used + (8.f + kHead)) {
                    factor = ex2(m_used - (mx - kHead));
                    m_used = mx - kHead;
                }
            }
            if (__any_sync(0xFFFFFFFFu, factor != 1.f)) {
                // O(rt, i-1) is complete (covered by the commit of S(rt, i))
                lsum2 = mul_f32x2(lsum2, pk2(factor, factor));
#pragma unroll 1
                for (int c0 = 0; c0 < HD; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(lane_addr + L::col_o(rt) + c0, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * factor);
                    tmem_st32(lane_addr + L::col_o(rt) + c0, o);
                }
            }
            // pass 2: P = 2^(score - m) as f16 pairs, written over the first half of each
            // chunk's own scores; chunks 2 and 3 from registers, each followed by the reload
            // of chunk 0 or 1 into its registers
            const float msub = m_used == -INFINITY ? 0.f : m_used;
            const uint64_t sub2 = pk2(-msub, -msub);
            const float mult = whole ? score_scale : 1.f;
            const uint64_t mul2 = pk2(mult, mult);
            auto chunk_p = [&](uint32_t (&sc)[32], int c) {
                if (!whole) {
                    const uint32_t bits = vis_bits(c);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        sc[e] = __float_as_uint(((bits >> e) & 1u) ? __uint_as_float(sc[e]) * score_scale
                                                                    : -INFINITY);
                }
                // P = 2^x in fp32, rounded to f16 pairs for the product; the row sum adds the
                // fp32 values in packed pairs
                uint32_t p[16];
#pragma unroll
                for (int w = 0; w < 16; ++w) {
                    const float2 x = upk2(fma_f32x2(pk2u(sc[2 * w], sc[2 * w + 1]), mul2, sub2));
                    const float e0 = ex2(x.x), e1 = ex2(x.y);
                    p[w] = f16x2_from_f32(e0, e1);
                    lsum2 = add_f32x2(lsum2, pk2(e0, e1));
                }
                tmem_st16(scol + 32 * c, p);
            };
            chunk_p(sa, 2);
            tmem_ld32(scol, sa);       // chunk 0's scores: its columns are not written yet
            chunk_p(sb, 3);
            tmem_ld32(scol + 32, sb);  // chunk 1's
            tmem_wait_ld();
            chunk_p(sa, 0);
            chunk_p(sb, 1);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::kPReady, rt));
        }
        if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(L::kODone, rt), 0, abort_flag));
        if (ok) {
            tc_fence_after();
            const float2 ls = upk2(lsum2);
            const float lsum = ls.x + ls.y;
            const float inv = lsum > 0.f ? sv / lsum : 0.f;
            uint32_t nan_groups = 0;
            if constexpr (F4) {
                if (*nan_seen) {
                    const int key0 = kSplit ? tile_lo * kP2Keys : 0;  // of this part's keys
                    nan_groups = nan_value_groups<HD>(a, seq, kvh, key0,
                                                      row_ok ? kSplit ? min(pos, key0 + ntiles * kP2Keys - 1) : pos : -1);
                }
            }
            // this row in the parts' results, when there are several
            const int64_t prow = kSplit ? ((((static_cast<int64_t>(seq) * a.row_tiles + ctile) * a.n_kv + kvh) * a.splits +
                                                     blockIdx.y) * kP2Rows) + tid : 0;
            const float part_inv = !kSplit || lsum == 0.f ? 0.f : 1.f / lsum;
            if (kSplit && row_ok) a.part_lse[prow] = lsum == 0.f ? -INFINITY : m_used + __log2f(lsum);
            uint4 *orow = reinterpret_cast<uint4 *>(
                a.out + ((static_cast<int64_t>(qr.q0) + jq) * a.n_q + kvh * G + gq) * HD);
#pragma unroll 1
            for (int c0 = 0; c0 < HD; c0 += 32) {
                uint32_t o[32];
                tmem_ld32(lane_addr + L::col_o(rt) + c0, o);
                tmem_wait_ld();
                if constexpr (kSplit) {
                    if (row_ok) store_part(a.part_o + prow * HD, o, part_inv, nan_groups, c0);
                } else if (row_ok) {
#pragma unroll
                    for (int c = 0; c < 32; c += 8) {
                        uint4 w;
                        auto word = [&](int k) {  // output word k of the 32 dims
                            const int e = 2 * o_word<F4>(k);
                            return bf16x2_from_f32(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv);
                        };
                        w.x = word(c / 2);
                        w.y = word(c / 2 + 1);
                        w.z = word(c / 2 + 2);
                        w.w = word(c / 2 + 3);
                        if (F4 && nan_groups != 0u) {
                            const int d = c0 + c;
                            w = make_uint4(nan_in(w.x, nan_groups, d), nan_in(w.y, nan_groups, d),
                                           nan_in(w.z, nan_groups, d), nan_in(w.w, nan_groups, d));
                        }
                        orow[(c0 + c) / 8] = w;
                    }
                }
            }
        } else if (lane == 0) {
            flag(a.status, KVFP8_DEV_TIMEOUT);
            *abort_flag = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kP2MmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// Joins the parts of each row: CTA (x, y) takes 256 / (HD / 4) rows of row tile x (of tile_rows rows, keys in
// tiles of tile_keys).
template <int HD>
__global__ void __launch_bounds__(256) join_parts_kernel(const PrefillArgs<true> a, int tile_rows, int tile_keys) {
    constexpr int kLanes = HD / 4;  // threads of a row, four dims each
    const int kvh = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.n_kv));
    const int tile = static_cast<int>((blockIdx.x / static_cast<unsigned>(a.n_kv)) % static_cast<unsigned>(a.row_tiles));
    const int seq = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.n_kv * a.row_tiles));
    const int lr = static_cast<int>(blockIdx.y) * (256 / kLanes) + static_cast<int>(threadIdx.x) / kLanes;
    const int d = static_cast<int>(threadIdx.x) % kLanes * 4;
    pdl_wait();  // the parts are visible from here on
    const float sk = load_scale(a.k_scale, a.scale_dtype), sv = load_scale(a.v_scale, a.scale_dtype);
    if (!scale_ok(sk) || !scale_ok(sv)) return;
    const QueryRange qr = a.qsl ? query_range(a.qsl, seq, a.qmax, a.qrows) : QueryRange{seq, 1};
    const int Ls = min(max(a.seq_lens[seq], 0), a.max_len);
    const int nb = qr.count, G = a.group, row0 = tile * tile_rows, r = row0 + lr;
    if (r >= nb * G) return;
    // the row tile's parts, as its CTAs worked them out
    const int j_last = min(nb, (row0 + tile_rows + G - 1) / G) - 1;
    const int kend = Ls - nb + j_last + 1;
    if (kend <= 0) return;  // zeroed by its CTA
    const int parts = split_parts(a.splits, (kend + tile_keys - 1) / tile_keys, tile_keys);
    const int64_t p0 = static_cast<int64_t>(blockIdx.x) * a.splits * tile_rows + lr;
    PartMerge<> mg;
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
#pragma unroll
        for (int i = 0; i < 8; ++i) mg.add(l[i], v[i]);
    }
    *reinterpret_cast<uint2 *>(a.out + ((static_cast<int64_t>(qr.q0) + r / G) * a.n_q + kvh * G + r % G) * HD + d) =
        mg.result(sv);
}

// How the 4-bit form is cut: the row tiles' size, and the parts per row tile that fill the SMs.
struct SplitPlan {
    int tile_rows = kPfRows, tile_keys = kPfKeys, splits = 1;
    size_t part_rows = 0, lse_off = 0, total = 0;  // workspace
};
SplitPlan split_plan(int32_t num_seqs, int32_t n_q, int32_t n_kv, int32_t head_dim, int32_t qmax, int64_t max_len) {
    SplitPlan p;
    const int64_t group_rows = static_cast<int64_t>(qmax) * (n_q / n_kv);
    if (head_dim <= 128 && group_rows > kPfRows) {
        p.tile_rows = kP2Rows;
        p.tile_keys = kP2Keys;
    }
    const int64_t tiles = (group_rows + p.tile_rows - 1) / p.tile_rows;
    if (tiles > kSplitSms || tiles * n_kv > kSplitSms || tiles * n_kv * num_seqs > kSplitSms / 2) return p;
    const int64_t ctas = tiles * n_kv * num_seqs;
    p.splits = static_cast<int>(std::max<int64_t>(1, std::min(kSplitSms / ctas, max_len / kMinPartKeys)));
    if (p.splits == 1) return p;
    p.part_rows = static_cast<size_t>(ctas) * p.splits * p.tile_rows;
    p.lse_off = p.part_rows * head_dim * sizeof(float);
    p.total = p.lse_off + p.part_rows * sizeof(float);
    return p;
}

template <int HD>
cudaError_t join_parts(const PrefillArgs<true> &a, const SplitPlan &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.num_seqs * a.row_tiles * a.n_kv, p.tile_rows / (256 / (HD / 4)));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_parts_kernel<HD>, a, p.tile_rows, p.tile_keys);
}

template <int HD, bool F4>
cudaError_t run_prefill(const DecodeArgs &d, cudaStream_t stream) {
    using L = PfSmem<HD, F4>;
    const int row_bytes = d.n_kv * L::kRow;
    const int box_rows = d.block_size >= kPfKeys ? kPfKeys : d.block_size;  // whole tile when one block holds it
    const int64_t rows = static_cast<int64_t>(d.num_blocks) * d.block_size;
    CUtensorMap tmk, tmv;
    cudaError_t err;
    if ((err = encode_cache_map(&tmk, d.key_cache, rows, row_bytes, L::kSeg, box_rows)) != cudaSuccess)
        return err;
    if ((err = encode_cache_map(&tmv, d.value_cache, rows, row_bytes, L::kSeg, box_rows)) != cudaSuccess)
        return err;
    PrefillArgs<F4> a;
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
    a.k_scale = d.k_scale;
    a.v_scale = d.v_scale;
    a.scale_dtype = d.scale_dtype;
    a.status = d.status;
    a.box_rows = box_rows;
    SplitPlan sp;
    if constexpr (F4) {
        sp = split_plan(d.num_seqs, d.n_q, d.n_kv, HD, d.qmax, a.max_len);
        a.key_scales = d.key_scales;
        a.value_scales = d.value_scales;
        a.splits = sp.splits;
        a.part_o = static_cast<float *>(d.workspace);
        a.part_lse = reinterpret_cast<float *>(static_cast<uint8_t *>(d.workspace) + sp.lse_off);
    }
    auto launched = [&]() -> cudaError_t {
        const cudaError_t e = cudaGetLastError();
        if constexpr (F4) {
            if (e == cudaSuccess && sp.splits > 1) return join_parts<HD>(a, sp, stream);
        }
        return e;
    };
    const int group_rows = d.qmax * a.group;  // score rows of a kv head (prefill_takes: below 2^31 - 511)
    // more than one tile of 128 rows per kv head (a multi-query call): 256 rows per CTA
    if constexpr (HD <= 128) {
        if (d.qsl != nullptr && group_rows > kPfRows) {
            const size_t smem2 = Pf2Smem<HD, F4>::kTotal + 1024;
            auto kern2 = sp.splits > 1 ? prefill2_kernel<HD, F4, F4> : prefill2_kernel<HD, F4, false>;
            int occ2 = 0;  // also raises the kernel's shared memory limit, once per device
            if ((err = kernel_occupancy(kern2, kP2Warps * 32, smem2, &occ2)) != cudaSuccess)
                return err;
            a.row_tiles = (group_rows + kP2Rows - 1) / kP2Rows;
            const int64_t ctas = static_cast<int64_t>(d.num_seqs) * a.row_tiles * d.n_kv;
            kern2<<<dim3(static_cast<unsigned>(ctas), sp.splits), kP2Warps * 32, smem2, stream>>>(tmk, tmv, a);
            return launched();
        }
    }
    const size_t smem = L::kTotal + 1024;
    auto kern = sp.splits > 1 ? prefill_kernel<HD, F4, F4> : prefill_kernel<HD, F4, false>;
    int occ = 0;  // also raises the kernel's shared memory limit, once per device
    if ((err = kernel_occupancy(kern, kPfWarps * 32, smem, &occ)) != cudaSuccess) return err;
    a.row_tiles = (group_rows + kPfRows - 1) / kPfRows;
    const int64_t ctas = static_cast<int64_t>(d.num_seqs) * a.row_tiles * d.n_kv;
    kern<<<dim3(static_cast<unsigned>(ctas), sp.splits), kPfWarps * 32, smem, stream>>>(tmk, tmv, a);
    return launched();
}

}  // namespace

size_t fp4_prefill_workspace_size(int32_t num_seqs, int32_t n_q, int32_t n_kv, int32_t head_dim, int32_t qmax,
                                  int64_t max_len) {
    return split_plan(num_seqs, n_q, n_kv, head_dim, qmax, max_len).total;
}

bool prefill_takes(int32_t n_q, int32_t n_kv, int32_t max_query_len, int32_t num_seqs) {
    // score rows of a (sequence, kv head) are ints, up to the end of the last tile and a group of heads past it
    constexpr int64_t kMostRows = 0x80000000LL - 512;
    const int64_t rows = static_cast<int64_t>(max_query_len) * (n_q / n_kv);
    if (n_q / n_kv > kPfRows || rows > kMostRows) return false;
    return (rows + kPfRows - 1) / kPfRows <= 0x7FFFFFFFLL / n_kv / std::max(1, num_seqs);
}

cudaError_t launch_prefill_attention(const DecodeArgs &d, cudaStream_t stream) {
    if (d.num_seqs == 0) return cudaSuccess;
    if (d.k_bf16 || d.v_bf16) return cudaErrorNotSupported;
    if (!prefill_takes(d.n_q, d.n_kv, d.qmax, d.num_seqs)) return cudaErrorNotSupported;
    const bool f4 = d.key_scales != nullptr;
    switch (d.head_dim) {
        case 64: return f4 ? run_prefill<64, true>(d, stream) : run_prefill<64, false>(d, stream);
        case 128: return f4 ? run_prefill<128, true>(d, stream) : run_prefill<128, false>(d, stream);
        case 256: return f4 ? run_prefill<256, true>(d, stream) : run_prefill<256, false>(d, stream);
        default: return cudaErrorNotSupported;
    }
}

}  // namespace kvfp8
