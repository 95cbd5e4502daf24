// Paged attention over the FP8 cache with a scale per block and kv head, for up to 16 score columns per
// kv head (single queries, a few tokens to verify), sm_103a:
//   s_t = sm_scale * ks(block of t) * q . dec(K_t),   out = sum_t softmax(s)_t * vs(block of t) * dec(V_t)
//
// The split of the work, the plan, the ring of TMA stages with one producer warp and one consumer warp per
// kv head and the combine kernel are those of the other decode kernels (paged_decode_kernel.cuh,
// paged_decode_fp4.cu).  What is this cache's own:
//  * Block scales: chunks are 32 tokens and blocks 16 at least, so a 16-token tile has one K and one V
//    scale.  The producer's lanes fetch them with 4-byte asynchronous copies into the stage, completing on
//    its barrier with the codes.  ks multiplies the tile's scores.  vs goes into the exponent: the
//    weights that meet V are w_t = 2^(s_t + log2 vs - m), m near the highest s_t + log2 vs, so they fill
//    fp16's range by what they add to the output, whatever the scales; the row's sum adds w_t / vs in
//    float, one fused multiply-add per tile and column (and 2^(s_t - m) itself where scales are too far apart for that, kSumSpan).
//  * A code is an fp16 number: conversion is one cvt per two codes, and 8 warps of an SM have ~3000 cycles
//    for 32 tokens each at the HBM rate, of which they issue ~700.  HBM bounds it:
//    64 sequences of 4096 tokens, 32 / 8 heads of 128, 92 us (5.9 TB/s, 86 % of a copy's rate), 8 of 131072 at 8 columns 237
//    (95 %).  At 16 columns the chain of a chunk does (3000 cycles for two warps a scheduler, which 168 registers hold it to): four
//    new tokens of 32 sequences of 4096, 56 us.  (Two warps a head with half the columns each: 58, both convert all codes.)
//  * V (A operand, dims x tokens): ldmatrix.trans gives two tokens' codes of two dims, a byte permute makes
//    them pairs of tokens.  (The 4-bit kernel's product over (token, dim parity) needs no permute, but its zeros
//    would spread a NaN code to the dim beside it.)  Up to 4 score columns stand at the even columns of
//    a score tile, one to a lane, so no lane works on padding.
//  * NaN codes: tokens that no column sees are zeroed in V.  Where some columns see a token and others do not (the
//    last tokens of a causal call), its NaN codes are zeroed and the outputs that do see it are made NaN
//    from a product of indicators.
#include "kvfp8_block_scale.cuh"
#include "paged_decode_own_plan.cuh"

#include <type_traits>

namespace kvfp8 {
namespace {

constexpr int kTok = 32;  // tokens of a chunk: two 16-token tiles
// log2: how far scores may rise above the highest one when the reference m was set, and how far below that one
// m lies.  Weights reach 2^15 and keep their 11 bits down to 2^-21 of the highest.
constexpr float kLag = 8.f, kHead = 7.f;

struct BlockKernelArgs {
    KernelArgs k;
    const float *key_scales, *value_scales;
    int32_t scale_stride;
    int32_t causal;
    uint32_t code_box;     // bytes of a code box (hpc heads x box_rows tokens)
    uint32_t tile_off;     // from the first 16-token tile's codes to the second's
    uint32_t stage_bytes;  // K boxes, V boxes, then 32 scales: [side][box][8 heads]
};

struct BlockChunk {
    int32_t seq;
    int32_t tok0;
    uint32_t mask;  // bit t: token tok0 + t exists (within the length, in a block of the pool)
    int32_t flags;
};

// NV: tiles of 4 score columns per kv head (1, 2 or 4).  kv heads of a CTA: a stage is 32 KB then, three
// fit, and two CTAs share an SM.
template <int HD>
__host__ __device__ constexpr int bs_max_heads() { return HD == 64 ? 8 : HD == 128 ? 4 : 2; }
constexpr int kCtasPerSm = 2;

// A chunk in which some column does not see some token: what such tokens could spread through the product with V is taken out
// of the head's V codes in the stage, which start at `codes`.  (With a body of its own, unrolled like the common one, such a
// chunk, one per sequence, ran from a cold instruction cache: 10000 cycles where the common one takes 3000, 16 columns.)
template <int HD>
struct StagedValues {
    static constexpr int SEG = HD < 128 ? HD : 128, kPieces = SEG / 16;
    uint8_t *codes;
    uint32_t seg_bytes, tile_off;
    uint32_t mask;  // the tokens that are there

    __device__ __forceinline__ uint8_t *piece(int t, int seg) const { return codes + seg * seg_bytes + (t >> 4) * tile_off; }

    // Tokens that are not there become 0; NaN codes of the others do with zero_nan.  Whether there are any of those.
    __device__ __noinline__ bool clean(bool zero_nan) const {
        bool any = false;
#pragma unroll 1
        for (int i = static_cast<int>(threadIdx.x & 31); i < kTok * (HD / 16); i += 32) {
            const int t = i / kPieces % kTok;
            uint4 *at = reinterpret_cast<uint4 *>(piece(t, i / kPieces / kTok) + (t & 15) * SEG + i % kPieces * 16);
            const uint4 w = *at;
            if ((mask >> t) & 1u) {
                const uint4 n = make_uint4(nan_byte_mask(w.x), nan_byte_mask(w.y), nan_byte_mask(w.z), nan_byte_mask(w.w));
                if ((n.x | n.y | n.z | n.w) != 0u) {
                    any = true;
                    if (zero_nan) *at = make_uint4(w.x & ~n.x, w.y & ~n.y, w.z & ~n.z, w.w & ~n.w);
                }
            } else {
                *at = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (the next copy into the stage comes through the async proxy)
        return __any_sync(0xFFFFFFFFu, any);
    }

    // Which of the lane's outputs (column v, dim 16 p + 2 gid + r: bit 4 KP v + 2 p + r) see a NaN code; column v sees tokens
    // up to last[v].
    template <int NV>
    __device__ __noinline__ uint64_t nan_outputs(const int (&last)[NV]) const {
        constexpr int KP = HD / 32;
        const int gid = static_cast<int>(threadIdx.x & 31) >> 2;
        uint64_t bits = 0;
#pragma unroll 1
        for (int t = 0; t < kTok; ++t) {
            if (!((mask >> t) & 1u)) continue;
#pragma unroll 1
            for (int p = 0; p < 2 * KP; ++p) {
                const uint8_t *two = piece(t, 16 * p / SEG) + swz<SEG>(t & 15, 16 * p % SEG / 16) + 2 * gid;
                const uint64_t here = ((two[0] & 0x7F) == 0x7F ? 1u : 0u) | ((two[1] & 0x7F) == 0x7F ? 2u : 0u);
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if (t <= last[v]) bits |= here << (4 * KP * v + 2 * p);
            }
        }
        return bits;
    }
};

template <int HD, int NV, bool kMulti>
__global__ void __launch_bounds__(32 * (bs_max_heads<HD>() + 1), kCtasPerSm)
decode_blocks_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                     const BlockKernelArgs f) {
    const KernelArgs &a = f.k;
    constexpr int SEG = HD < 128 ? HD : 128;  // bytes of a TMA box row
    constexpr int SEGS = HD / SEG;            // of a token's head
    constexpr int KP = HD / 32;               // 32-dim chunks
    constexpr int NS = (NV + 1) / 2;          // score tiles of 8 columns

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);

    const int S = a.stages;
    const int hpc = a.hpc, h0 = static_cast<int>(blockIdx.y) * hpc;
    const uint32_t stage_bytes = f.stage_bytes;
    const uint32_t code_bytes = static_cast<uint32_t>(kTok * hpc * HD);  // of a side
    const uint32_t bars = base + static_cast<uint32_t>(S) * stage_bytes;  // full[S], empty[S]
    BlockChunk *meta = reinterpret_cast<BlockChunk *>(base_ptr + S * stage_bytes + 16 * S);
    volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(meta + S);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(bars + 8 * i, 1 + 32);  // the producer's post, and every lane's scale copies
            mbar_init(bars + 8 * (S + i), hpc);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == hpc && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmk)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmv)) : "memory");
    }
    if (warp == hpc && blockIdx.y == 0) {  // this CTA's slice of the block tables into L2
        const int64_t bytes = static_cast<int64_t>(a.num_seqs) * a.max_blocks_per_seq * 4;
        const int64_t per = (bytes + gridDim.x - 1) / gridDim.x;
        const char *tb = reinterpret_cast<const char *>(a.block_tables);
        for (int64_t off = blockIdx.x * per + lane * 128; off < min(bytes, (blockIdx.x + 1) * per);
             off += 32 * 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(tb + off));
    }
    pdl_wait();     // the plan grid's records and zeroed rows are visible from here on
    pdl_trigger();  // let the combine grid get launched; it waits for this grid to finish
    if (a.cta_plan != nullptr && a.cta_plan[blockIdx.x].lo >= a.cta_plan[blockIdx.x].hi) return;
    __syncthreads();

    if (warp == hpc) {
        // ------------------------------------------------------------ producer warp
        int64_t issued = 0;
        int stage = 0;
        uint32_t phase = 0;
        bool aborted = false;
        const CtaPlan rec = a.cta_plan != nullptr ? a.cta_plan[blockIdx.x] : own_plan<kTok>(a, lane);
        const int64_t chunk_lo = rec.lo, chunk_hi = rec.hi;
        int s = rec.s, L = rec.L;
        int64_t cs = rec.cs, ce = rec.ce;
        int wbase = -1 << 30;  // first block-table entry held in the lane window
        int32_t win = 0;
        if (chunk_lo < chunk_hi) prefetch_q<HD>(a, s, h0, lane);
        const int lbr = 31 - __clz(a.box_rows), lbs = 31 - __clz(a.block_size);  // powers of two
        // the scale that this lane copies: [side][box][head]
        const int sbox = (lane >> 3) & 1, shead = lane & 7;
        const float *scales = (lane < 16 ? f.key_scales : f.value_scales) + h0 + shead;
        for (int64_t x = chunk_lo; x < chunk_hi; ++x) {
            if (x >= ce) {
                while (x >= ce) {
                    ++s;
                    cs = ce;
                    ce = cs + seq_chunks<kTok>(a, s, L);
                }
                wbase = -1 << 30;
                prefetch_q<HD>(a, s, h0, lane);
            }
            // lane p < nloads has box p of the chunk (both sides)
            const int tok0 = static_cast<int>(x - cs) * kTok;
            const int nvalid = min(kTok, L - tok0);
            const int nloads = (nvalid + a.box_rows - 1) >> lbr;
            const int e0 = tok0 >> lbs, e1 = (tok0 + nvalid - 1) >> lbs;
            if (e0 < wbase || e1 >= wbase + 32) {
                wbase = e0;
                const int e = wbase + lane;
                win = (e < a.max_blocks_per_seq)
                          ? a.block_tables[static_cast<int64_t>(s) * a.max_blocks_per_seq + e]
                          : -1;
            }
            const int t = tok0 + (lane << lbr);
            const int blk = __shfl_sync(0xFFFFFFFFu, win, ((t >> lbs) - wbase) & 31);
            const bool mine = lane < nloads;
            const bool good = mine && blk >= 0 && blk < a.num_blocks;
            if (mine && !good) flag(a.status, KVFP8_DEV_BAD_BLOCK);
            uint32_t bits = 0;  // this box's tokens
            if (good) {
                const int first = lane << lbr, n = min(a.box_rows, nvalid - first);
                bits = (n == 32 ? ~0u : (1u << n) - 1u) << first;
            }
            const uint32_t mask = __reduce_or_sync(0xFFFFFFFFu, bits);
            const uint32_t goods = __ballot_sync(0xFFFFFFFFu, good);
            const int boxes = __popc(goods);
            const int sblk = __shfl_sync(0xFFFFFFFFu, blk, sbox);
            int32_t flags = 0;
            if (x == chunk_lo || x == cs) flags |= kFirst;
            if (x == chunk_hi - 1 || x == ce - 1) flags |= kLast;
            if (cs >= chunk_lo && ce <= chunk_hi) flags |= kDirect;
            const uint32_t full = bars + 8 * stage;
            const bool withheld = kWithholdFirstChunk && issued == 0;  // (test build: neither a copy nor an arrival for this stage)
            if (lane == 0) {
                if (!mbar_wait(bars + 8 * (S + stage), phase ^ 1u, abort_flag)) {
                    aborted = true;
                } else {
                    meta[stage] = BlockChunk{s, tok0, mask, flags};
                    if (withheld) {
                    } else if (boxes > 0)
                        mbar_arrive_tx(full, boxes * 2 * f.code_box);
                    else
                        mbar_arrive(full);
                }
            }
            aborted = __shfl_sync(0xFFFFFFFFu, aborted, 0);
            if (aborted) break;
            __syncwarp();  // what lane 0 waited for (the stage has been read) holds for every lane's copies
            const uint32_t st = base + static_cast<uint32_t>(stage) * stage_bytes;
            if (good && !withheld) {  // the expected bytes are posted: each lane copies its box
                const int row = (blk << lbs) + (t & (a.block_size - 1));
                tma_load_3d(st + lane * f.code_box, &tmk, 0, row, h0 * SEGS, full);
                tma_load_3d(st + code_bytes + lane * f.code_box, &tmv, 0, row, h0 * SEGS, full);
            }
            if (shead < hpc && (goods >> sbox) & 1u && !withheld)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(st + 2 * code_bytes + lane * 4),
                             "l"(scales + static_cast<int64_t>(sblk) * f.scale_stride)
                             : "memory");
            if (!withheld) asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
            ++issued;
            if (++stage == S) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!aborted) {
            if (lane == 0) {
                if (!mbar_wait(bars + 8 * (S + stage), phase ^ 1u, abort_flag))
                    aborted = true;
                else
                    meta[stage] = BlockChunk{0, 0, 0, kDone};
            }
            aborted = __shfl_sync(0xFFFFFFFFu, aborted, 0);
            if (!aborted) {  // 33 arrivals, as every phase takes
                mbar_arrive(bars + 8 * stage);
                if (lane == 0) mbar_arrive(bars + 8 * stage);
            }
        }
        if (a.cta_plan == nullptr && blockIdx.y == 0) finish_plan<HD, kTok>(a, lane, f.causal != 0);
        if (aborted) asm volatile("cp.async.wait_all;" ::: "memory");
        if (aborted && lane == 0) {
            flag(a.status, KVFP8_DEV_TIMEOUT);
            *abort_flag = 1;
            // let copies already issued land before the CTA's shared memory goes away
            const int64_t first = issued > S ? issued - S : 0;
            for (int64_t k = first; k < issued; ++k) {
                const volatile int32_t never = 0;
                mbar_wait(bars + 8 * static_cast<int>(k % S), static_cast<uint32_t>((k / S) & 1),
                          &never);
            }
        }
    } else if (warp < hpc) {
        // ------------------------------------------------------------ consumer warp
        const int kvh = h0 + warp;
        const int gid = lane >> 2, tig = lane & 3;
        const float score_scale = a.sm_scale * 1.4426950408889634f;  // log2(e)

        // The lane's score columns, v = 0..NV-1 (column x: query token x / group, head x % group), x at n =
        // x % 8 of score tile x / 8, so x = 8 (v / 2) + 2 tig + v % 2; NV = 1: x = tig, at n = 2 tig.
        auto column = [&](int v) { return NV == 1 ? tig : 8 * (v / 2) + 2 * tig + v % 2; };
        float o[NS][2 * KP][4];
        // dim 16p + 2 gid + r of column v
        auto at = [&](int v, int p, int r) -> float & { return o[v / 2][p][v % 2 + 2 * r]; };
        // per column: the reference (log2 domain, of s + log2 vs) the weights are taken against, and this
        // lane's part of the sum of weights / vs
        float m[NV], l[NV];
        float vtop = 0.f, vlow = 0.f;  // log2 of the largest and the smallest V scale so far
        uint32_t qb[2 * KP][NS][2];
        // multi-query form: the sequence's first query row, its query tokens, and the last cache position
        // that the first of them may see; one further each when causal
        int q0 = 0, nq = 1, first_lim = 0;

        // this lane's rows of a stage, for the first 16-token tile (the second: tile_off further); an 8-token
        // group is 8 SEG bytes, so a chunk further is an xor
        const uint32_t head_codes = static_cast<uint32_t>(warp * SEGS * a.box_rows * SEG);
        const uint32_t seg_bytes = static_cast<uint32_t>(a.box_rows * SEG);
        const uint32_t krow_off = head_codes + swz<SEG>((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
        const uint32_t vrow_off = code_bytes + head_codes + swz<SEG>(lane & 7, lane >> 3);
        const uint32_t scale_off = 2 * code_bytes + warp * 4;

        int stage = 0;
        uint32_t phase = 0;
        for (;;) {
            // every lane waits (acquire on the copies' bytes); the outcome is made warp-uniform
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(bars + 8 * stage, phase, abort_flag))) {
                if (lane == 0) {
                    flag(a.status, KVFP8_DEV_TIMEOUT);
                    *abort_flag = 1;
                }
                break;
            }
            BlockChunk mt = meta[stage];
            if (mt.flags & kDone) break;
            const uint32_t st = base + static_cast<uint32_t>(stage) * stage_bytes;

            if (mt.flags & kFirst) {
                if (kMulti) {
                    const QueryRange qr = query_range(a.qsl, mt.seq, a.rows_per_seq / a.n_q, a.qrows);
                    q0 = qr.q0;
                    nq = qr.count;
                    first_lim = min(max(a.seq_lens[mt.seq], 0), a.max_len) - (f.causal ? nq : 1);
                }
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const int x = NV == 1 ? gid >> 1 : 8 * s + gid;  // column gid of score tile s
                    const int jq = kMulti ? x / a.group : 0;
                    const int gq = kMulti ? x % a.group : x;
                    const bool qv = (kMulti ? jq < nq : x < a.group) && !(NV == 1 && (gid & 1));
                    const __nv_bfloat16 *qrow =
                        a.query +
                        ((static_cast<int64_t>(kMulti ? q0 + jq : mt.seq)) * a.n_q + kvh * a.group + gq) * HD;
#pragma unroll
                    for (int c = 0; c < 2 * KP; ++c) {
                        uint2 w = make_uint2(0u, 0u);
                        if (qv) w = *reinterpret_cast<const uint2 *>(qrow + 16 * c + 4 * tig);
                        qb[c][s][0] = f16x2_from_f32(bf16lo(w.x), bf16hi(w.x));
                        qb[c][s][1] = f16x2_from_f32(bf16lo(w.y), bf16hi(w.y));
                    }
                }
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    m[v] = -INFINITY;
                    l[v] = 0.f;
                }
                vtop = -INFINITY;
                vlow = INFINITY;
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int p = 0; p < 2 * KP; ++p)
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[s][p][r] = 0.f;
            }

            // the tiles' scales; a tile whose block has none that is valid is left out
            float kmul[2], vlog[2], vinv[2];
            {
                bool bad = false;
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    const uint32_t at_box = st + scale_off + (a.box_rows == 16 ? tt * 32 : 0);
                    float ks, vs;
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(ks) : "r"(at_box));
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vs) : "r"(at_box + 64));
                    const uint32_t tile = 0xFFFFu << (16 * tt);
                    const bool there = (mt.mask & tile) != 0u;
                    if (!(block_scale_ok(ks) && block_scale_ok(vs) && there)) {
                        bad |= there;
                        mt.mask &= ~tile;
                        ks = vs = 1.f;
                    }
                    // (kept away from 0 and infinity, which would make a NaN of a score of infinity or 0)
                    kmul[tt] = fminf(fmaxf(ks * score_scale, 0x1p-126f), 0x1p126f);
                    vlog[tt] = static_cast<float>(static_cast<int>(__float_as_uint(vs) >> 23) - 127);
                    vinv[tt] = block_scale_inverse(vs);
                }
                vtop = fmaxf(vtop, fmaxf(vlog[0], vlog[1]));
                vlow = fminf(vlow, fminf(vlog[0], vlog[1]));
                if (bad && lane == 0) flag(a.status, KVFP8_DEV_BAD_SCALE);
            }

            // partial: some column does not see some token of the chunk
            const bool partial = mt.mask != ~0u || (kMulti && mt.tok0 + kTok - 1 > first_lim);
            auto last_seen = [&](int v) {  // the last token of the chunk that column v sees (padding columns: none)
                if (!kMulti) return kTok - 1;
                const int j = column(v) / a.group;  // its query token
                return j < nq ? first_lim + (f.causal ? j : 0) - mt.tok0 : -1;
            };
            if (mt.mask != 0u) {
                uint64_t poison = 0;  // outputs that become NaN
                if (partial) {
                    const StagedValues<HD> values = {base_ptr + stage * stage_bytes + code_bytes + head_codes, seg_bytes, f.tile_off, mt.mask};
                    if (values.clean(false) && kMulti) {
                        int last[NV];
#pragma unroll
                        for (int v = 0; v < NV; ++v) last[v] = last_seen(v);
                        poison = values.template nan_outputs<NV>(last);
                        __syncwarp();  // (every lane has looked)
                        values.clean(true);
                    }
                    __syncwarp();
                }

                // ---- scores S^T[token][column] = K . q^T, tiles of 16 tokens
                float sacc[2][NS][4];
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    // two running sums, so that a product waits for the one before the last only
                    constexpr int kSums = NV <= 2 ? 2 : 1;
                    float part[kSums][NS][4];
#pragma unroll
                    for (int k = 0; k < kSums; ++k)
#pragma unroll
                        for (int s = 0; s < NS; ++s)
                            part[k][s][0] = part[k][s][1] = part[k][s][2] = part[k][s][3] = 0.f;
#pragma unroll
                    for (int c = 0; c < KP; ++c) {  // 32 dims: two 16-byte pieces of a row
                        const uint32_t addr = (st + krow_off + tt * f.tile_off + c * 32 / SEG * seg_bytes) ^
                                              static_cast<uint32_t>(c * 32 % SEG);
                        uint32_t r[4];
                        ldsm_x4(addr, r[0], r[1], r[2], r[3]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t a0 = f16x2_from_e4m3x2(r[2 * e]), a1 = f16x2_from_e4m3x2(r[2 * e + 1]);
                            const uint32_t a2 = f16x2_from_e4m3x2_hi(r[2 * e]), a3 = f16x2_from_e4m3x2_hi(r[2 * e + 1]);
#pragma unroll
                            for (int s = 0; s < NS; ++s)
                                mma16816(part[kSums == 2 ? e : 0][s], a0, a1, a2, a3, qb[2 * c + e][s][0],
                                         qb[2 * c + e][s][1]);
                        }
                    }
#pragma unroll
                    for (int s = 0; s < NS; ++s)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sacc[tt][s][i] = kSums == 2 ? part[0][s][i] + part[kSums - 1][s][i] : part[0][s][i];
                }

                // ---- weights 2^(s + log2 vs - m) per column.  m only has to be near the running maximum less
                // kHead: it moves when one passes it by more than kLag + kHead, so most chunks take no
                // maximum over the lanes and rescale nothing.  Tokens a column does not see get -inf.
                if (partial) {
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        const int last = last_seen(v);
#pragma unroll
                        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int row = 16 * tt + 8 * h + gid;
                                if (row > last || !((mt.mask >> row) & 1u)) sacc[tt][v / 2][v % 2 + 2 * h] = -INFINITY;
                            }
                    }
                }
                auto column_top = [&](int v) {  // this lane's highest of column v
                    const int s = v / 2, c = v % 2;
                    return fmaxf(fmaf(fmaxf(sacc[0][s][c], sacc[0][s][c + 2]), kmul[0], vlog[0]),
                                 fmaf(fmaxf(sacc[1][s][c], sacc[1][s][c + 2]), kmul[1], vlog[1]));
                };
                const bool far = vtop - vlow > kSumSpan;
                float top = far ? INFINITY : -INFINITY;  // the highest over its column's m
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    // (m starts at -inf, which any score passes; a column of -inf passes nothing)
                    top = fmaxf(top, column_top(v) - m[v]);
                if (__any_sync(0xFFFFFFFFu, top > kLag + kHead)) {
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        float x = column_top(v);
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16)) - kHead;
                        if (x > m[v]) {
                            // nothing but zeros (or a NaN, which stays) before the first score
                            const float down = m[v] == -INFINITY ? 0.f : m[v] - x;
                            const float alpha = ex2(down), root = ex2(0.5f * down);
                            m[v] = x;
                            l[v] = l[v] * root * root;  // (a sum of small scales' tokens may be as large as alpha is small)
#pragma unroll
                            for (int p = 0; p < 2 * KP; ++p) {
                                at(v, p, 0) *= alpha;
                                at(v, p, 1) *= alpha;
                            }
                        }
                    }
                    if (far) {  // the chunk's part of the sums by itself
#pragma unroll
                        for (int tt = 0; tt < 2; ++tt) {
                            vinv[tt] = 0.f;
#pragma unroll
                            for (int v = 0; v < NV; ++v) {
                                const float less = m[v] == -INFINITY ? 0.f : -m[v];
                                l[v] += ex2(fmaf(sacc[tt][v / 2][v % 2], kmul[tt], less)) + ex2(fmaf(sacc[tt][v / 2][v % 2 + 2], kmul[tt], less));
                            }
                        }
                    }
                }
                // Weights as B fragments of 16 tokens, through a register transpose.
                uint32_t pw[2][2][NS];  // tokens 16 tt + 8 h + 2 tig, + 1 of column gid
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    constexpr int kCols = NV == 1 ? 1 : 2;  // of the lane in a score tile
                    float p[2][2][2] = {};                  // [column][tt][h]
#pragma unroll
                    for (int k = 0; k < kCols; ++k) {
                        const int v = 2 * s + k;
                        // a column that has seen no score yet: -inf - 0 for every token
                        const float sub = m[v] == -INFINITY ? 0.f : m[v];
#pragma unroll
                        for (int tt = 0; tt < 2; ++tt) {
                            const float less = vlog[tt] - sub;
#pragma unroll
                            for (int h = 0; h < 2; ++h) p[k][tt][h] = ex2(fmaf(sacc[tt][s][k + 2 * h], kmul[tt], less));
                            l[v] = fmaf(p[k][tt][0] + p[k][tt][1], vinv[tt], l[v]);
                        }
                    }
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) pw[tt][h][s] = movm_t(f16x2_from_f32(p[0][tt][h], p[1][tt][h]));
                }

                // ---- O^T[dim][column] += V^T . P^T
                // Codes of tokens 2 tig, + 1 of half h (low and high 16 bits: dims 2 gid, +1 of a 16-dim
                // piece) of pieces 4 c4..4 c4 + 3 of a tile.
                auto value_codes = [&](int tt, int h, int c4, uint32_t (&r)[4]) {
                    const uint32_t addr = (st + vrow_off + tt * f.tile_off + h * (8 * SEG) + c4 * 64 / SEG * seg_bytes) ^
                                          static_cast<uint32_t>(c4 * 64 % SEG);
                    ldsm_x4_t(addr, r[0], r[1], r[2], r[3]);
                };
                // one 16-dim piece of 16 tokens (both halves), weights of score tile s
                auto product_tokens = [&](uint32_t lo, uint32_t hi, uint32_t b0, uint32_t b1, float (&acc)[4]) {
                    const uint32_t x = __byte_perm(lo, 0u, 0x3120), y = __byte_perm(hi, 0u, 0x3120);
                    mma16816(acc, f16x2_from_e4m3x2(x), f16x2_from_e4m3x2_hi(x), f16x2_from_e4m3x2(y),
                             f16x2_from_e4m3x2_hi(y), b0, b1);
                };
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
#pragma unroll
                    for (int c4 = 0; c4 < KP / 2; ++c4) {
                        uint32_t r[2][4];
                        value_codes(tt, 0, c4, r[0]);
                        value_codes(tt, 1, c4, r[1]);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int s = 0; s < NS; ++s)
                                product_tokens(r[0][e], r[1][e], pw[tt][0][s], pw[tt][1][s], o[s][4 * c4 + e]);
                    }
                }
                if (poison != 0) {
#pragma unroll
                    for (int v = 0; v < NV; ++v)
#pragma unroll
                        for (int p = 0; p < 2 * KP; ++p)
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                if ((poison >> (4 * KP * v + 2 * p + r)) & 1u) at(v, p, r) = __uint_as_float(0x7FC00000u);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + 8 * (S + stage));
            if (++stage == S) {
                stage = 0;
                phase ^= 1u;
            }

            if (mt.flags & kLast) {
                const bool direct = (mt.flags & kDirect) != 0;
                const int64_t pidx = static_cast<int64_t>(mt.seq) + blockIdx.x;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    float lt = l[v];
                    lt += __shfl_xor_sync(0xFFFFFFFFu, lt, 4);
                    lt += __shfl_xor_sync(0xFFFFFFFFu, lt, 8);
                    lt += __shfl_xor_sync(0xFFFFFFFFu, lt, 16);
                    const int x = column(v);
                    if (kMulti ? x / a.group >= nq : x >= a.group) continue;  // padding column
                    const int srow = kMulti ? x / a.group * a.n_q + kvh * a.group + x % a.group : kvh * a.group + x;
                    const int64_t orow_idx = kMulti ? static_cast<int64_t>(q0) * a.n_q + srow
                                                    : static_cast<int64_t>(mt.seq) * a.n_q + srow;
                    // zero where no token was visible; a NaN sum makes the row NaN
                    const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
                    for (int p = 0; p < 2 * KP; ++p) {
                        const int d = 16 * p + 2 * gid;
                        const float x0 = at(v, p, 0) * inv, x1 = at(v, p, 1) * inv;
                        if (direct)
                            *reinterpret_cast<uint32_t *>(a.out + orow_idx * HD + d) = bf16x2_from_f32(x0, x1);
                        else
                            *reinterpret_cast<float2 *>(a.part_o + (pidx * a.rows_per_seq + srow) * HD + d) =
                                make_float2(x0, x1);
                    }
                    if (!direct && gid == 0)
                        a.part_lse[pidx * a.rows_per_seq + srow] = lt == 0.f ? -INFINITY : m[v] + __log2f(lt);
                }
            }
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- host side

// Codes as a 3-D byte tensor (seg bytes, rows, segments of a row), boxes of box_rows x segs.
cudaError_t encode_blocks(CUtensorMap *map, const uint8_t *codes, int64_t rows, int row_bytes, int seg, int box_rows,
                          int segs) {
    auto enc = tensor_map_encoder();
    if (enc == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(seg), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(row_bytes / seg)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(seg)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(seg), static_cast<cuuint32_t>(box_rows),
                               static_cast<cuuint32_t>(segs)};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(codes), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle_of(seg), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int HD, int NV, bool kMulti>
cudaError_t run_blocks(const DecodeArgs &d, const DecodeWorkspace &ws, cudaStream_t stream) {
    DeviceFacts facts;
    cudaError_t err = device_facts(&facts);
    if (err != cudaSuccess) return err;
    const int sms = facts.sms, smem_optin = facts.smem_optin;
    constexpr int SEG = HD < 128 ? HD : 128;

    // kv heads per CTA: the largest divisor of n_kv up to the limit; the groups are a grid dimension
    int hpc = std::min(d.n_kv, bs_max_heads<HD>());
    while (d.n_kv % hpc != 0) --hpc;
    const int groups = d.n_kv / hpc;
    if (groups > 65535) return cudaErrorNotSupported;  // gridDim.y (a large prime n_kv)
    const int box_rows = std::min(d.block_size, kTok);
    BlockKernelArgs f;
    f.key_scales = d.key_block_scales;
    f.value_scales = d.value_block_scales;
    f.scale_stride = d.block_scale_stride;
    f.causal = d.causal;
    f.code_box = static_cast<uint32_t>(hpc * box_rows * HD);
    f.tile_off = box_rows == 32 ? 16 * SEG : f.code_box;
    f.stage_bytes = (2u * kTok * hpc * HD + 128u + 1023u) & ~1023u;
    // CTAs of fewer heads than the limit: as many as have that many warps in all
    const int ctas_per_sm = kCtasPerSm * (bs_max_heads<HD>() + 1) / (hpc + 1);
    constexpr int kMaxStages = 8;
    auto smem_for = [&](int st) { return static_cast<size_t>(st) * (f.stage_bytes + 32) + 16 + 1024; };
    const size_t sm_budget = static_cast<size_t>(smem_optin) + 1024;
    int stages = kMaxStages;
    while (stages > 2 && (smem_for(stages) + 1024) * ctas_per_sm > sm_budget) --stages;
    const size_t smem = smem_for(stages);
    if (smem > static_cast<size_t>(smem_optin)) return cudaErrorNotSupported;

    auto kern = decode_blocks_kernel<HD, NV, kMulti>;
    const int threads = 32 * (hpc + 1);
    int occ = 0;
    if ((err = kernel_occupancy(kern, threads, smem, &occ)) != cudaSuccess) return err;
    occ = std::max(1, std::min(occ, ctas_per_sm));
    const int num_ctas = std::max(1, std::min(sms * occ / groups, kMaxDecodeCtas));

    CUtensorMap tmk, tmv;
    const int64_t rows = static_cast<int64_t>(d.num_blocks) * d.block_size;
    const int row_bytes = d.n_kv * HD, segs = hpc * HD / SEG;
    if ((err = encode_blocks(&tmk, d.key_cache, rows, row_bytes, SEG, box_rows, segs)) != cudaSuccess ||
        (err = encode_blocks(&tmv, d.value_cache, rows, row_bytes, SEG, box_rows, segs)) != cudaSuccess)
        return err;

    uint8_t *w = static_cast<uint8_t *>(d.workspace);
    KernelArgs &k = f.k;
    k = KernelArgs{};
    k.out = static_cast<__nv_bfloat16 *>(d.out);
    k.query = static_cast<const __nv_bfloat16 *>(d.query);
    k.block_tables = d.block_tables;
    k.max_blocks_per_seq = d.max_blocks_per_seq;
    k.seq_lens = d.seq_lens;
    k.num_seqs = d.num_seqs;
    k.n_q = d.n_q;
    k.n_kv = d.n_kv;
    k.group = d.n_q / d.n_kv;
    k.hpc = hpc;
    k.block_size = d.block_size;
    k.num_blocks = d.num_blocks;
    k.max_len = d.max_blocks_per_seq * d.block_size;
    k.sm_scale = d.sm_scale;
    k.k_scale = k.v_scale = nullptr;  // (none per layer: the combine kernel multiplies by 1)
    k.scale_dtype = KVFP8_F32;
    k.cstart = reinterpret_cast<const int32_t *>(w + ws.cstart_off);
    k.cta_plan = reinterpret_cast<const CtaPlan *>(w + ws.cta_off);
    k.part_lse = reinterpret_cast<float *>(w + ws.lse_off);
    k.part_o = reinterpret_cast<float *>(w + ws.o_off);
    k.status = d.status;
    k.num_ctas = num_ctas;
    k.stages = stages;
    k.box_rows = box_rows;
    k.whole_box = 1;
    k.qsl = d.qsl;
    k.rows_per_seq = d.qmax * d.n_q;
    k.qrows = d.qrows;

    const bool whole = decode_takes_sequences_whole(d.max_blocks_per_seq, d.block_size);
    const bool own = whole || d.num_seqs <= kOwnPlanSeqs;
    if (own) {
        k.cta_plan = nullptr;
        if (whole) k.num_ctas = 0;
    } else {
        plan_kernel<kTok><<<1, 1024, 0, stream>>>(d.seq_lens, d.qsl, d.qmax, d.qrows, d.num_seqs, k.max_len, num_ctas,
                                                  reinterpret_cast<int32_t *>(w + ws.cstart_off),
                                                  reinterpret_cast<CtaPlan *>(w + ws.cta_off), k.out, d.n_q * HD,
                                                  d.status, d.causal != 0);
        if ((err = cudaGetLastError()) != cudaSuccess) return err;
    }

    // programmatic dependent launches, as for the 8-bit kernel
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(whole ? d.num_seqs : num_ctas, groups);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = own ? 0 : 1;  // (only a kernel of this call may be overtaken)
    if ((err = cudaLaunchKernelEx(&cfg, kern, tmk, tmv, f)) != cudaSuccess || whole) return err;

    constexpr int kRows = 256 / (HD / 4);  // of a CTA of the combine
    cudaLaunchConfig_t ccfg = cfg;
    ccfg.numAttrs = 1;
    ccfg.gridDim = dim3(d.num_seqs, (k.rows_per_seq + kRows - 1) / kRows);
    ccfg.dynamicSmemBytes = 0;
    const int64_t parts = (static_cast<int64_t>(num_ctas) + d.num_seqs) / std::max(1, d.num_seqs);
    // few, long sequences: a CTA per row, 512 threads over its parts, while that is one wave
    if (parts >= 32 && static_cast<int64_t>(d.num_seqs) * k.rows_per_seq <= 4 * sms) {
        constexpr int kSlices = 512 / (HD / 4);
        ccfg.gridDim = dim3(d.num_seqs, k.rows_per_seq);
        ccfg.blockDim = dim3(512);
        return cudaLaunchKernelEx(&ccfg, combine_kernel<HD, kSlices, 1, true>, k);
    }
    if (parts >= 32) {
        ccfg.blockDim = dim3(256 * 4);
        return cudaLaunchKernelEx(&ccfg, combine_kernel<HD, 4, kRows, true>, k);
    }
    if (parts >= 16) {
        ccfg.blockDim = dim3(256 * 2);
        return cudaLaunchKernelEx(&ccfg, combine_kernel<HD, 2, kRows, true>, k);
    }
    ccfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&ccfg, combine_kernel<HD, 1, kRows, true>, k);
}

template <int HD>
cudaError_t run_tiles(const DecodeArgs &d, const DecodeWorkspace &ws, int tiles, cudaStream_t stream) {
    const bool multi = d.qsl != nullptr;
    if (tiles <= 1) return multi ? run_blocks<HD, 1, true>(d, ws, stream) : run_blocks<HD, 1, false>(d, ws, stream);
    if (tiles <= 2) return multi ? run_blocks<HD, 2, true>(d, ws, stream) : run_blocks<HD, 2, false>(d, ws, stream);
    if constexpr (HD <= 128)
        return multi ? run_blocks<HD, 4, true>(d, ws, stream) : run_blocks<HD, 4, false>(d, ws, stream);
    return cudaErrorNotSupported;
}

}  // namespace

cudaError_t launch_paged_decode_block_scaled(const DecodeArgs &d, cudaStream_t stream) {
    if (d.num_seqs == 0) return cudaSuccess;
    if (!multi_uses_decode_kernel(d.n_q, d.n_kv, d.head_dim, d.qmax)) return launch_prefill_block_scaled(d, stream);
    const DecodeWorkspace ws = decode_workspace_layout(d.num_seqs, d.qmax * d.n_q, d.head_dim);
    const int tiles = (d.qmax * (d.n_q / d.n_kv) + 3) / 4;  // of 4 score columns
    switch (d.head_dim) {
        case 64: return run_tiles<64>(d, ws, tiles, stream);
        case 128: return run_tiles<128>(d, ws, tiles, stream);
        case 256: return run_tiles<256>(d, ws, tiles, stream);
        default: return cudaErrorNotSupported;
    }
}

}  // namespace kvfp8
