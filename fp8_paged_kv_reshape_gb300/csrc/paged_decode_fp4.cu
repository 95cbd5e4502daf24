// Paged decode attention over the 4-bit cache (E2M1 codes, an E4M3 scale per 16 dims), sm_103a:
//   s_t = sm_scale * k_scale * q . (code_K B_K)_t,   out = v_scale * softmax(s) . (code_V B_V)
//
// The split of the work, the plan and combine kernels, the ring of TMA stages with one producer
// warp and one consumer warp per kv head, and the online softmax are those of the 8-bit kernel
// (paged_decode_kernel.cuh).  What differs is what a chunk of 16 tokens holds and how a consumer
// makes tensor-core operands of it:
//  * 0.5625 bytes per element: per side a box of [heads][16 tokens][head_dim/2] code bytes
//    (swizzled over its 32-, 64- or 128-byte rows) and one of [heads][16 tokens][head_dim/16]
//    scale bytes, four TMA loads per chunk (eight when 8-token blocks cut it in two).
//  * code * B has at most 2 + 4 significant bits and lies between 2^-10 and 2688, so it is an
//    fp16 number: codes convert to fp16 pairs, one packed multiply applies the group's scale
//    exactly, and the products are those of fp16 mma.sync with fp32 accumulation.
//  * K (A operand, tokens x dims): ldmatrix gives a lane the 8 codes of dims 8t..8t+7 of a
//    32-dim chunk (t = lane % 4) for token rows lane/4 and +8; the k order of the two products
//    of a chunk is that order, for q too.  All 8 lie in one group of 16, so a lane needs one
//    scale per row and chunk.
//  * V (A operand, dims x tokens): ldmatrix.trans gives the 4 codes of dims 4g..4g+3 (g =
//    lane / 4) of two tokens; they are converted, regrouped into token pairs per dim (one byte
//    permute each) and multiplied by the tokens' scale pair.  A lane ends up with 4 consecutive
//    output dims per chunk.
//  * NaN: a scale byte of 0x7F makes its 16 dims NaN.  Tokens past the end have their V scales
//    zeroed.  In the multi-query form a chunk that some columns see only in part takes a second
//    look: NaN scales of V are zeroed too, and the outputs whose column does see the token are
//    made NaN from a product of indicators.
#include "paged_decode_kernel.cuh"

#include <type_traits>

namespace kvfp8 {
namespace {

constexpr int kTok = 32;  // tokens of a chunk: two 16-token tiles
constexpr float kLag = 8.f;  // log2: how far scores may rise above the reference maximum

struct Fp4KernelArgs {
    KernelArgs k;
    uint32_t code_box;         // bytes of one code box (hpc heads x box_rows tokens)
    uint32_t scale_box;        // smem bytes of one scale box, rounded up to 128
    uint32_t scale_box_bytes;  // bytes a scale box brings
    uint32_t stage_bytes;
    // Offsets within a side of a chunk's 8-token groups: group g starts at (g & 1) * x1 + (g >> 1)
    // * x2 past the head's first row (codes, scales).
    uint32_t c1, c2, s1, s2;
};

// A chunk's record: bit t of mask is set when token tok0 + t exists (within the length, in a
// block of the pool).
struct Fp4Chunk {
    int32_t seq;
    int32_t tok0;
    uint32_t mask;
    int32_t flags;
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <int N>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[N]) {
    static_assert(N == 1 || N == 2 || N == 4 || N == 8, "words");
    if constexpr (N == 1) {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
    } else if constexpr (N == 2) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "r"(addr + 4 * i));
    }
}

// 0x3C00 (fp16 one) in each half of an fp16 pair that is NaN
__device__ __forceinline__ uint32_t nan_ones(uint32_t h) {
    return ((h & 0x7FFFu) > 0x7C00u ? 0x3C00u : 0u) | ((h & 0x7FFF0000u) > 0x7C000000u ? 0x3C000000u : 0u);
}

// As for the 8-bit kernel: two CTAs per SM where the accumulators allow it.
template <int HD, int NT>
__host__ __device__ constexpr int fp4_ctas_per_sm() { return HD * NT <= 128 ? 2 : 1; }

template <int HD, int NT, bool kMulti>
__global__ void __launch_bounds__(kThreadsMax, fp4_ctas_per_sm<HD, NT>())
decode_fp4_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                  const __grid_constant__ CUtensorMap tmks, const __grid_constant__ CUtensorMap tmvs,
                  const Fp4KernelArgs f) {
    const KernelArgs &a = f.k;
    constexpr int SEG = HD / 2;    // code bytes of a token's kv head
    constexpr int GPH = HD / 16;   // scale bytes of it
    constexpr int KP = HD / 32;    // 32-dim chunks

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);

    const int S = a.stages;
    const int hpc = a.hpc, h0 = static_cast<int>(blockIdx.y) * hpc;
    const uint32_t stage_bytes = f.stage_bytes;
    // a stage: the chunk's K code boxes, V code boxes, K scale boxes, V scale boxes
    const uint32_t code_bytes = static_cast<uint32_t>(kTok * hpc * SEG);
    const uint32_t scales_off = 2 * code_bytes, vscales_off = scales_off + kTok / a.box_rows * f.scale_box;
    const uint32_t bars = base + static_cast<uint32_t>(S) * stage_bytes;  // full[S], empty[S]
    Fp4Chunk *meta = reinterpret_cast<Fp4Chunk *>(base_ptr + S * stage_bytes + 16 * S);
    volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(meta + S);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(bars + 8 * i, 1);
            mbar_init(bars + 8 * (S + i), hpc);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == hpc && lane == 0) {
        for (const CUtensorMap *t : {&tmk, &tmv, &tmks, &tmvs})
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(t)) : "memory");
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

    const float sk = load_scale(a.k_scale, a.scale_dtype);
    const float sv = load_scale(a.v_scale, a.scale_dtype);
    if (!scale_ok(sk) || !scale_ok(sv)) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) flag(a.status, KVFP8_DEV_BAD_SCALE);
        return;
    }
    const CtaPlan *rec = a.cta_plan + blockIdx.x;
    const int32_t pl_lo = rec->lo, pl_hi = rec->hi;
    if (pl_lo >= pl_hi) return;
    const int64_t chunk_lo = pl_lo, chunk_hi = pl_hi;
    __syncthreads();

    if (warp == hpc) {
        // ------------------------------------------------------------ producer warp
        int64_t issued = 0;
        int stage = 0;
        uint32_t phase = 0;
        bool aborted = false;
        int s = rec->s;  // sequence holding chunk_lo, its chunks and length (from the plan)
        int64_t cs = rec->cs, ce = rec->ce;
        int L = rec->L;
        int wbase = -1 << 30;  // first block-table entry held in the lane window
        int32_t win = 0;
        prefetch_q<HD>(a, s, h0, lane);
        const int lbr = 31 - __clz(a.box_rows), lbs = 31 - __clz(a.block_size);  // powers of two
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
            // lane p < nloads has box p of the chunk (every side and both arrays of it)
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
            const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, good));
            int32_t flags = 0;
            if (x == chunk_lo || x == cs) flags |= kFirst;
            if (x == chunk_hi - 1 || x == ce - 1) flags |= kLast;
            if (cs >= chunk_lo && ce <= chunk_hi) flags |= kDirect;
            const uint32_t full = bars + 8 * stage;
            if (lane == 0) {
                if (!mbar_wait(bars + 8 * (S + stage), phase ^ 1u, abort_flag)) {
                    aborted = true;
                } else {
                    meta[stage] = Fp4Chunk{s, tok0, mask, flags};
                    if (boxes > 0)
                        mbar_arrive_tx(full, boxes * 2 * (f.code_box + f.scale_box_bytes));
                    else
                        mbar_arrive(full);
                }
            }
            aborted = __shfl_sync(0xFFFFFFFFu, aborted, 0);
            if (aborted) break;
            if (good) {  // the expected bytes are posted: each lane copies its box
                const uint32_t st = base + static_cast<uint32_t>(stage) * stage_bytes;
                const int off = t & (a.block_size - 1), row = (blk << lbs) + off;
                const int sx = off * GPH / 4, sy = blk * a.n_kv + h0;
                tma_load_3d(st + lane * f.code_box, &tmk, 0, row, h0, full);
                tma_load_3d(st + code_bytes + lane * f.code_box, &tmv, 0, row, h0, full);
                tma_load_2d(st + scales_off + lane * f.scale_box, &tmks, sx, sy, full);
                tma_load_2d(st + vscales_off + lane * f.scale_box, &tmvs, sx, sy, full);
            }
            ++issued;
            if (++stage == S) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (!aborted) {
            if (lane == 0) {
                if (!mbar_wait(bars + 8 * (S + stage), phase ^ 1u, abort_flag)) {
                    aborted = true;
                } else {
                    meta[stage] = Fp4Chunk{0, 0, 0, kDone};
                    mbar_arrive(bars + 8 * stage);
                }
            }
            aborted = __shfl_sync(0xFFFFFFFFu, aborted, 0);
        }
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
        float score_scale = a.sm_scale * sk * 1.4426950408889634f;  // log2(e)
        if (score_scale == 0.f) score_scale = 0x1p-126f;  // underflow: equal weights, -inf stays -inf

        float o[KP][2][NT][4];
        // per score column: the reference maximum (log2 domain) the weights are taken against, and
        // this lane's part of the sum of weights
        float m[NT][2], l[NT][2];
        uint32_t qb[KP][NT][4];
        // multi-query form: per score column (query token j, head g) the last cache position it
        // may see, and its row within the sequence (-1: a padding column)
        int plim[NT][2], crow[NT][2];
        int q0 = 0, first_lim = 0;  // first_lim: the smallest plim of the sequence's columns

        // Offsets of this lane in a stage, for the first 16-token tile (the second: c2, s2 further).
        const uint32_t head_codes = static_cast<uint32_t>(warp * a.box_rows * SEG);
        const uint32_t head_scales = static_cast<uint32_t>(warp * a.box_rows * GPH);
        const uint32_t krow_off = head_codes + ((lane >> 3) & 1) * f.c1;
        const int kchunk_hi = lane >> 4;
        const uint32_t vrow_off = code_bytes + head_codes + (lane >> 4) * f.c1;
        const int vchunk_hi = (lane >> 3) & 1;
        const uint32_t ks_off = scales_off + head_scales + gid * GPH;
        const uint32_t vs_off = vscales_off + head_scales + 2 * tig * GPH;
        const uint32_t ksel = 0x6420u + 0x1111u * (tig >> 1);  // bytes of this lane's K groups
        const uint32_t vsel = 0x6240u + 0x1111u * (gid >> 2);  // (token, next token) of its V groups

        int stage = 0;
        uint32_t phase = 0;
        for (;;) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(bars + 8 * stage, phase, abort_flag))) {
                if (lane == 0) {
                    flag(a.status, KVFP8_DEV_TIMEOUT);
                    *abort_flag = 1;
                }
                break;
            }
            const Fp4Chunk mt = meta[stage];
            if (mt.flags & kDone) break;

            if (mt.flags & kFirst) {
                int nq = 1;
                if (kMulti) {
                    const QueryRange qr = query_range(a.qsl, mt.seq, a.rows_per_seq / a.n_q, a.qrows);
                    q0 = qr.q0;
                    nq = qr.count;
                    const int L = min(max(a.seq_lens[mt.seq], 0), a.max_len);
                    first_lim = L - nq;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int n = nt * 8 + 2 * tig + c;
                            const int j = n / a.group, g = n % a.group;
                            plim[nt][c] = j < nq ? L - nq + j : -1;
                            crow[nt][c] = j < nq ? j * a.n_q + kvh * a.group + g : -1;
                        }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    // column gid of n-tile nt: query token jq, head gq of the group
                    const int n = nt * 8 + gid;
                    const int jq = kMulti ? n / a.group : 0;
                    const int gq = kMulti ? n % a.group : n;
                    const bool qv = kMulti ? jq < nq : n < a.group;
                    const __nv_bfloat16 *qrow =
                        a.query +
                        ((static_cast<int64_t>(kMulti ? q0 + jq : mt.seq)) * a.n_q + kvh * a.group + gq) * HD;
#pragma unroll
                    for (int c = 0; c < KP; ++c) {
                        uint4 w = make_uint4(0u, 0u, 0u, 0u);
                        if (qv) w = *reinterpret_cast<const uint4 *>(qrow + 32 * c + 8 * tig);
                        qb[c][nt][0] = f16x2_from_f32(bf16lo(w.x), bf16hi(w.x));
                        qb[c][nt][1] = f16x2_from_f32(bf16lo(w.y), bf16hi(w.y));
                        qb[c][nt][2] = f16x2_from_f32(bf16lo(w.z), bf16hi(w.z));
                        qb[c][nt][3] = f16x2_from_f32(bf16lo(w.w), bf16hi(w.w));
                    }
                    m[nt][0] = m[nt][1] = -INFINITY;
                    l[nt][0] = l[nt][1] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < KP; ++e)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int r = 0; r < 4; ++r) o[e][j][nt][r] = 0.f;
            }

            const uint32_t st = base + static_cast<uint32_t>(stage) * stage_bytes;
            // kPartial: some column does not see some token of the chunk.  The common chunk has a body
            // without those tests: one basic block from the weights to the last product.
            auto chunk = [&](auto partial_tag) {
                constexpr bool kPartial = decltype(partial_tag)::value;

                // ---- scores S^T[token][head] = K . q^T, two tiles of 16 tokens
                float sacc[2][NT][4];
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    uint32_t sc_lo[KP / 2], sc_hi[KP / 2];  // bytes of this lane's groups, rows gid and +8
                    {
                        uint32_t wl[GPH / 4], wh[GPH / 4];
                        lds(st + ks_off + tt * f.s2, wl);
                        lds(st + ks_off + tt * f.s2 + f.s1, wh);
                        if constexpr (KP == 2) {
                            sc_lo[0] = __byte_perm(wl[0], 0u, ksel);
                            sc_hi[0] = __byte_perm(wh[0], 0u, ksel);
                        } else {
#pragma unroll
                            for (int i = 0; i < KP / 2; i += 2) {
                                const uint32_t bl = __byte_perm(wl[i], wl[i + 1], ksel);
                                const uint32_t bh = __byte_perm(wh[i], wh[i + 1], ksel);
                                sc_lo[i] = bl;
                                sc_lo[i + 1] = bl >> 16;
                                sc_hi[i] = bh;
                                sc_hi[i + 1] = bh >> 16;
                            }
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        sacc[tt][nt][0] = sacc[tt][nt][1] = sacc[tt][nt][2] = sacc[tt][nt][3] = 0.f;
#pragma unroll
                    for (int cp = 0; cp < KP / 2; ++cp) {
                        uint32_t r[4];
                        ldsm_x4(st + krow_off + tt * f.c2 + swz<SEG>(lane & 7, 2 * cp + kchunk_hi), r[0], r[1],
                                r[2], r[3]);
                        const uint32_t fl = f16x2_from_e4m3x2(sc_lo[cp]), fh = f16x2_from_e4m3x2(sc_hi[cp]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {  // chunk 2cp + e
                            const uint32_t sl = __byte_perm(fl, 0u, e ? 0x3232 : 0x1010);
                            const uint32_t sh = __byte_perm(fh, 0u, e ? 0x3232 : 0x1010);
                            uint32_t ka[4], kb[4];
                            f16x2_from_e2m1x8(r[2 * e], ka);
                            f16x2_from_e2m1x8(r[2 * e + 1], kb);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                ka[i] = hmul2(ka[i], sl);
                                kb[i] = hmul2(kb[i], sh);
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint32_t(&q)[4] = qb[2 * cp + e][nt];
                                mma16816(sacc[tt][nt], ka[0], kb[0], ka[1], kb[1], q[0], q[1]);
                                mma16816(sacc[tt][nt], ka[2], kb[2], ka[3], kb[3], q[2], q[3]);
                            }
                        }
                    }
                }

                // ---- weights 2^(score - m) per head column (log2 domain).  m only has to be near the
                // running maximum: it moves when a score passes it by more than kLag, so most chunks
                // take no maximum over the lanes and rescale nothing, and weights stay <= 2^kLag.
                // Tokens a column does not see get -inf (chunks with such tokens only).
                auto sees = [&](int row, int nt, int c) {  // row of the chunk
                    return ((mt.mask >> row) & 1u) != 0u && (!kMulti || mt.tok0 + row <= plim[nt][c]);
                };
                if constexpr (kPartial) {  // a score of -inf (whatever the scale's sign), a weight of 0
                    const float none = score_scale > 0.f ? -INFINITY : INFINITY;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    if (!sees(16 * tt + 8 * h + gid, nt, c)) sacc[tt][nt][c + 2 * h] = none;
                }
                float top = -INFINITY;  // the highest score over its column's m
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float a0 = sacc[0][nt][c], a1 = sacc[0][nt][c + 2];
                        const float a2 = sacc[1][nt][c], a3 = sacc[1][nt][c + 2];
                        const float x = score_scale > 0.f ? fmaxf(fmaxf(a0, a1), fmaxf(a2, a3))
                                                          : fminf(fminf(a0, a1), fminf(a2, a3));
                        // (m starts at -inf, which any score passes; a column of -inf passes nothing)
                        top = fmaxf(top, x * score_scale - m[nt][c]);
                    }
                if (__any_sync(0xFFFFFFFFu, top > kLag)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float a0 = sacc[0][nt][c], a1 = sacc[0][nt][c + 2];
                            const float a2 = sacc[1][nt][c], a3 = sacc[1][nt][c + 2];
                            float x = score_scale > 0.f ? fmaxf(fmaxf(a0, a1), fmaxf(a2, a3))
                                                        : fminf(fminf(a0, a1), fminf(a2, a3));
                            x *= score_scale;
                            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                            if (x > m[nt][c]) {
                                // nothing but zeros (or a NaN, which stays) before the first score
                                const float alpha = m[nt][c] == -INFINITY ? 1.f : ex2(m[nt][c] - x);
                                m[nt][c] = x;
                                l[nt][c] *= alpha;
#pragma unroll
                                for (int e = 0; e < KP; ++e)
#pragma unroll
                                    for (int j = 0; j < 2; ++j) {
                                        o[e][j][nt][c] *= alpha;
                                        o[e][j][nt][c + 2] *= alpha;
                                    }
                            }
                        }
                }
                uint32_t pb[2][NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        // a column that has seen no score yet: -inf - 0 for every token
                        const float sub = m[nt][c] == -INFINITY ? 0.f : m[nt][c];
#pragma unroll
                        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float p = ex2(fmaf(sacc[tt][nt][c + 2 * h], score_scale, -sub));
                                sacc[tt][nt][c + 2 * h] = p;
                            }
                        l[nt][c] += (sacc[0][nt][c] + sacc[0][nt][c + 2]) + (sacc[1][nt][c] + sacc[1][nt][c + 2]);
                    }
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                        for (int h = 0; h < 2; ++h)  // tokens 16 tt + 8 h ..+7
                            pb[tt][nt][h] = movm_t(f16x2_from_f32(sacc[tt][nt][2 * h], sacc[tt][nt][2 * h + 1]));
                }

                // ---- O^T[dim][head] += V^T . P^T
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    uint32_t vs_lo[KP], vs_hi[KP];  // scale pairs of tokens 2t, 2t+1 and 2t+8, 2t+9
                    {
                        uint32_t wl[GPH / 2], wh[GPH / 2];  // the two tokens' scale bytes
                        lds(st + vs_off + tt * f.s2, wl);
                        lds(st + vs_off + tt * f.s2 + f.s1, wh);
#pragma unroll
                        for (int i = 0; i < GPH / 4; ++i) {
                            const uint32_t bl = __byte_perm(wl[i], wl[i + GPH / 4], vsel);
                            const uint32_t bh = __byte_perm(wh[i], wh[i + GPH / 4], vsel);
                            vs_lo[2 * i] = f16x2_from_e4m3x2(bl);
                            vs_lo[2 * i + 1] = f16x2_from_e4m3x2_hi(bl);
                            vs_hi[2 * i] = f16x2_from_e4m3x2(bh);
                            vs_hi[2 * i + 1] = f16x2_from_e4m3x2_hi(bh);
                        }
                    }
                    if constexpr (kPartial) {
                        // tokens that are not there: scale 0
                        const uint32_t bits = mt.mask >> (16 * tt + 2 * tig);
                        const uint32_t mlo = (bits & 1u ? 0x0000FFFFu : 0u) | (bits & 2u ? 0xFFFF0000u : 0u);
                        const uint32_t mhi = (bits & 0x100u ? 0x0000FFFFu : 0u) | (bits & 0x200u ? 0xFFFF0000u : 0u);
#pragma unroll
                        for (int c = 0; c < KP; ++c) {
                            vs_lo[c] &= mlo;
                            vs_hi[c] &= mhi;
                        }
                        if (kMulti) {
                            // A column that does not see a token has weight 0 for it, and a NaN scale would
                            // make 0 * NaN of that.
                            uint32_t any = 0;
#pragma unroll
                            for (int c = 0; c < KP; ++c) any |= nan_ones(vs_lo[c]) | nan_ones(vs_hi[c]);
                            if (__any_sync(0xFFFFFFFFu, any != 0u)) {
                                uint32_t sb[NT][2];  // fp16 ones where the column sees the token
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int h = 0; h < 2; ++h) {
                                        const int row = 16 * tt + 8 * h + gid;
                                        sb[nt][h] = movm_t((sees(row, nt, 0) ? 0x3C00u : 0u) |
                                                           (sees(row, nt, 1) ? 0x3C000000u : 0u));
                                    }
#pragma unroll
                                for (int c = 0; c < KP; ++c) {
                                    const uint32_t nl = nan_ones(vs_lo[c]), nh = nan_ones(vs_hi[c]);
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt) {
                                        // NaN tokens per (dims of the lane's group, column)
                                        float cnt[4] = {0.f, 0.f, 0.f, 0.f};
                                        mma16816(cnt, nl, nl, nh, nh, sb[nt][0], sb[nt][1]);
#pragma unroll
                                        for (int r = 0; r < 4; ++r)
                                            if (cnt[r] > 0.f)
                                                o[c][0][nt][r] = o[c][1][nt][r] = __uint_as_float(0x7FC00000u);
                                    }
                                    vs_lo[c] &= ~(nl / 0x3C00u * 0xFFFFu);
                                    vs_hi[c] &= ~(nh / 0x3C00u * 0xFFFFu);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int cp = 0; cp < KP / 2; ++cp) {
                        uint32_t r[4];
                        ldsm_x4_t(st + vrow_off + tt * f.c2 + swz<SEG>(lane & 7, 2 * cp + vchunk_hi), r[0], r[1],
                                  r[2], r[3]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {  // chunk 2cp + e: tokens 0-7 in r[e], 8-15 in r[2+e]
                            uint32_t x[4], y[4];
                            f16x2_from_e2m1x8(r[e], x);
                            f16x2_from_e2m1x8(r[2 + e], y);
                            const uint32_t sl = vs_lo[2 * cp + e], sh = vs_hi[2 * cp + e];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {  // dims 4g + 2j, 4g + 2j + 1
                                const uint32_t a0 = hmul2(__byte_perm(x[j], x[j + 2], 0x5410), sl);
                                const uint32_t a1 = hmul2(__byte_perm(x[j], x[j + 2], 0x7632), sl);
                                const uint32_t a2 = hmul2(__byte_perm(y[j], y[j + 2], 0x5410), sh);
                                const uint32_t a3 = hmul2(__byte_perm(y[j], y[j + 2], 0x7632), sh);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma16816(o[2 * cp + e][j][nt], a0, a1, a2, a3, pb[tt][nt][0], pb[tt][nt][1]);
                            }
                        }
                    }
                }
            };
            if (mt.mask == ~0u && !(kMulti && mt.tok0 + kTok - 1 > first_lim))
                chunk(std::false_type{});
            else if (mt.mask != 0u)
                chunk(std::true_type{});
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
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float lt = l[nt][c];
                        lt += __shfl_xor_sync(0xFFFFFFFFu, lt, 4);
                        lt += __shfl_xor_sync(0xFFFFFFFFu, lt, 8);
                        lt += __shfl_xor_sync(0xFFFFFFFFu, lt, 16);
                        const int g = nt * 8 + 2 * tig + c;
                        if (kMulti ? crow[nt][c] < 0 : g >= a.group) continue;  // padding column
                        const int srow = kMulti ? crow[nt][c] : kvh * a.group + g;
                        const int64_t orow_idx = kMulti ? static_cast<int64_t>(q0) * a.n_q + srow
                                                        : static_cast<int64_t>(mt.seq) * a.n_q + srow;
                        // zero where no token was visible; a NaN sum makes the row NaN
                        const float inv = lt == 0.f ? 0.f : (direct ? sv : 1.f) / lt;
#pragma unroll
                        for (int e = 0; e < KP; ++e) {
                            const int d = 32 * e + 4 * gid;  // four consecutive dims
                            const float x0 = o[e][0][nt][c] * inv, x1 = o[e][0][nt][c + 2] * inv;
                            const float x2 = o[e][1][nt][c] * inv, x3 = o[e][1][nt][c + 2] * inv;
                            if (direct)
                                *reinterpret_cast<uint2 *>(a.out + orow_idx * HD + d) =
                                    make_uint2(bf16x2_from_f32(x0, x1), bf16x2_from_f32(x2, x3));
                            else
                                *reinterpret_cast<float4 *>(a.part_o + (pidx * a.rows_per_seq + srow) * HD + d) =
                                    make_float4(x0, x1, x2, x3);
                        }
                        if (!direct && gid == 0)
                            a.part_lse[pidx * a.rows_per_seq + srow] =
                                lt == 0.f ? -INFINITY : m[nt][c] + __log2f(lt);
                    }
                }
            }
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- host side

// Codes as a 3-D byte tensor (head_dim/2 bytes, rows, kv heads), boxes of box_rows x hpc heads.
cudaError_t encode_codes(CUtensorMap *map, const uint8_t *codes, int64_t rows, int n_kv, int seg,
                         int box_rows, int hpc) {
    auto enc = tensor_map_encoder();
    if (enc == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(seg), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(n_kv)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(n_kv) * seg, static_cast<cuuint64_t>(seg)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(seg), static_cast<cuuint32_t>(box_rows),
                               static_cast<cuuint32_t>(hpc)};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(codes), dims,
                           strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           swizzle_of(seg),
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Scales as a 2-D tensor of words of four bytes (a head's words of a block, block * n_kv + head).
// A box starts at a multiple of 8 tokens, so at a multiple of 32 bytes.
cudaError_t encode_scales(CUtensorMap *map, const uint8_t *scales, int64_t block_heads, int head_bytes,
                          int box_bytes, int hpc) {
    auto enc = tensor_map_encoder();
    if (enc == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(head_bytes / 4), static_cast<cuuint64_t>(block_heads)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(head_bytes)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_bytes / 4), static_cast<cuuint32_t>(hpc)};
    const cuuint32_t estr[2] = {1u, 1u};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t *>(scales), dims,
                           strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int HD, int NT, bool kMulti>
cudaError_t run_fp4(const DecodeArgs &d, const DecodeWorkspace &ws, cudaStream_t stream) {
    DeviceFacts facts;
    cudaError_t err = device_facts(&facts);
    if (err != cudaSuccess) return err;
    const int sms = facts.sms, smem_optin = facts.smem_optin;

    // kv heads per CTA: the largest divisor of n_kv up to 8; the groups are a grid dimension
    int hpc = std::min(d.n_kv, kMaxKvHeads);
    while (d.n_kv % hpc != 0) --hpc;
    const int groups = d.n_kv / hpc;
    const int box_rows = std::min(d.block_size, kTok);
    Fp4KernelArgs f;
    f.code_box = static_cast<uint32_t>(hpc * box_rows * (HD / 2));
    f.scale_box_bytes = static_cast<uint32_t>(hpc * box_rows * (HD / 16));
    f.scale_box = (f.scale_box_bytes + 127u) & ~127u;
    const uint32_t boxes = kTok / box_rows;
    f.stage_bytes = (2 * boxes * (f.code_box + f.scale_box) + 1023u) & ~1023u;
    // two 8-token groups a box of 16, four a box of 32, one a box of 8
    f.c1 = box_rows >= 16 ? 8 * (HD / 2) : f.code_box;
    f.c2 = box_rows == 32 ? 16 * (HD / 2) : box_rows == 16 ? f.code_box : 2 * f.code_box;
    f.s1 = box_rows >= 16 ? 8 * (HD / 16) : f.scale_box;
    f.s2 = box_rows == 32 ? 16 * (HD / 16) : box_rows == 16 ? f.scale_box : 2 * f.scale_box;
    const int ctas_per_sm = fp4_ctas_per_sm<HD, NT>();
    constexpr int kMaxStages = 8;
    auto smem_for = [&](int st) { return static_cast<size_t>(st) * (f.stage_bytes + 32) + 16 + 1024; };
    const size_t sm_budget = static_cast<size_t>(smem_optin) + 1024;
    int stages = kMaxStages;
    while (stages > 2 && (smem_for(stages) + 1024) * ctas_per_sm > sm_budget) --stages;
    const size_t smem = smem_for(stages);
    if (smem > static_cast<size_t>(smem_optin)) return cudaErrorNotSupported;

    auto kern = decode_fp4_kernel<HD, NT, kMulti>;
    const int threads = 32 * (hpc + 1);
    int occ = 0;
    if ((err = kernel_occupancy(kern, threads, smem, &occ)) != cudaSuccess) return err;
    occ = std::max(1, std::min(occ, ctas_per_sm));
    const int num_ctas = std::max(1, std::min(sms * occ / groups, kMaxDecodeCtas));

    CUtensorMap tmk, tmv, tmks, tmvs;
    const int64_t rows = static_cast<int64_t>(d.num_blocks) * d.block_size;
    const int64_t block_heads = static_cast<int64_t>(d.num_blocks) * d.n_kv;
    const int head_bytes = d.block_size * (HD / 16), box_bytes = box_rows * (HD / 16);
    if ((err = encode_codes(&tmk, d.key_cache, rows, d.n_kv, HD / 2, box_rows, hpc)) != cudaSuccess ||
        (err = encode_codes(&tmv, d.value_cache, rows, d.n_kv, HD / 2, box_rows, hpc)) != cudaSuccess ||
        (err = encode_scales(&tmks, d.key_scales, block_heads, head_bytes, box_bytes, hpc)) != cudaSuccess ||
        (err = encode_scales(&tmvs, d.value_scales, block_heads, head_bytes, box_bytes, hpc)) != cudaSuccess)
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
    k.k_scale = d.k_scale;
    k.v_scale = d.v_scale;
    k.scale_dtype = d.scale_dtype;
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

    plan_kernel<kTok><<<1, 1024, 0, stream>>>(d.seq_lens, d.qsl, d.qmax, d.qrows, d.num_seqs, k.max_len,
                                        num_ctas, reinterpret_cast<int32_t *>(w + ws.cstart_off),
                                        reinterpret_cast<CtaPlan *>(w + ws.cta_off), k.out,
                                        d.n_q * HD, d.status);
    if ((err = cudaGetLastError()) != cudaSuccess) return err;

    // programmatic dependent launches, as for the 8-bit kernel
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_ctas, groups);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((err = cudaLaunchKernelEx(&cfg, kern, tmk, tmv, tmks, tmvs, f)) != cudaSuccess) return err;

    constexpr int kHeadsPerCta = 256 / (HD / 4);
    cudaLaunchConfig_t ccfg = cfg;
    ccfg.gridDim = dim3(d.num_seqs, (k.rows_per_seq + kHeadsPerCta - 1) / kHeadsPerCta);
    ccfg.dynamicSmemBytes = 0;
    const int64_t parts = (static_cast<int64_t>(num_ctas) + d.num_seqs) / std::max(1, d.num_seqs);
    if (parts >= 32) {
        ccfg.blockDim = dim3(256 * 4);
        return cudaLaunchKernelEx(&ccfg, combine_kernel<HD, 4>, k);
    }
    if (parts >= 16) {
        ccfg.blockDim = dim3(256 * 2);
        return cudaLaunchKernelEx(&ccfg, combine_kernel<HD, 2>, k);
    }
    ccfg.blockDim = dim3(256);
    return cudaLaunchKernelEx(&ccfg, combine_kernel<HD, 1>, k);
}

}  // namespace

cudaError_t launch_paged_decode_fp4(const DecodeArgs &d, cudaStream_t stream) {
    if (d.num_seqs == 0) return cudaSuccess;
    if (!multi_uses_decode_kernel(d.n_q, d.n_kv, d.head_dim, d.qmax))
        return launch_prefill_attention(d, stream);
    const DecodeWorkspace ws = decode_workspace_layout(d.num_seqs, d.qmax * d.n_q, d.head_dim);
    const bool one = d.qmax * (d.n_q / d.n_kv) <= 8;  // n-tiles of 8 score columns
    if (d.qsl == nullptr) {
        switch (d.head_dim) {
            case 64: return one ? run_fp4<64, 1, false>(d, ws, stream) : run_fp4<64, 2, false>(d, ws, stream);
            case 128: return one ? run_fp4<128, 1, false>(d, ws, stream) : run_fp4<128, 2, false>(d, ws, stream);
            case 256: return one ? run_fp4<256, 1, false>(d, ws, stream) : cudaErrorNotSupported;
            default: return cudaErrorNotSupported;
        }
    }
    switch (d.head_dim) {
        case 64: return one ? run_fp4<64, 1, true>(d, ws, stream) : run_fp4<64, 2, true>(d, ws, stream);
        case 128: return one ? run_fp4<128, 1, true>(d, ws, stream) : run_fp4<128, 2, true>(d, ws, stream);
        case 256: return one ? run_fp4<256, 1, true>(d, ws, stream) : cudaErrorNotSupported;
        default: return cudaErrorNotSupported;
    }
}

}  // namespace kvfp8
