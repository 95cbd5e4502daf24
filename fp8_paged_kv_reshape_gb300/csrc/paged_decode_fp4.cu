// Paged decode attention over the 4-bit cache (E2M1 codes, an E4M3 scale per 16 dims), sm_103a:
//   s_t = sm_scale * k_scale * q . (code_K B_K)_t,   out = v_scale * softmax(s) . (code_V B_V)
//
// The split of the work, the combine kernel, the ring of TMA stages with one producer warp and one
// consumer warp per kv head are those of the 8-bit kernel (paged_decode_kernel.cuh).  A cached
// element is 0.5625 bytes, so at the HBM rate nearly twice as many elements a second have to be
// converted, and what a consumer does per element decides (an SM has 412 issue slots a scheduler for
// 16 tokens of a head at 6.8 TB/s; conversions, permutes and maxima go at half that rate):
//  * Chunks of 32 tokens: barriers, records and the softmax's bookkeeping are paid half as often.
//    Per side a box of [heads][tokens][head_dim/2] code bytes (swizzled over its 32-, 64- or 128-byte
//    rows) and one of [heads][tokens][head_dim/16] scale bytes; a block of less than 32 tokens is a
//    box, and lane p of the producer issues box p of each.
//  * code * B has at most 2 + 4 significant bits and lies between 2^-10 and 2688, so it is an
//    fp16 number: codes convert to fp16 pairs, one packed multiply applies the group's scale
//    exactly, and the products are those of fp16 mma.sync with fp32 accumulation.
//  * K (A operand, tokens x dims): ldmatrix gives a lane the 8 codes of dims 8t..8t+7 of a
//    32-dim chunk (t = lane % 4) for token rows lane/4 and +8; the k order of the two products
//    of a chunk is that order, for q too.  All 8 lie in one group of 16, so a lane needs one
//    scale per row and chunk.
//  * Weights are taken against a reference maximum that lags the running one (see below), so most
//    chunks need no maximum over lanes and rescale nothing.  They are rounded to fp16 for the product with V,
//    their sum is not: 11 bits, which moves outputs by 0.0004 of their norm (64 sequences of 4096; an
//    output's rounding to bf16 0.0016), where a second fp16 part would double those products.
//  * V (A operand, dims x tokens): ldmatrix.trans gives the 4 codes of dims 4g..4g+3 (g =
//    lane / 4) of two tokens, and conversion leaves them as pairs of dims, where a product over
//    tokens wants pairs of tokens.  Up to 8 score columns the product runs over (token, dim parity)
//    instead: rows are pairs of dims, and the other operand holds the weights at one parity and zeros
//    at the other, 4 columns to a tile of 8.  The four converted words of a lane are then an A
//    fragment as they are; without it each took a byte permute (127 against 113 us for 128 x 4096
//    tokens, 4 columns).  At 16 columns the doubled products would bind (384 of the 412 slots), and the
//    permutes are shared by two tiles: that form regroups.
//    A lane ends up with 4 consecutive output dims per 32-dim chunk.
//  * NaN: a scale byte of 0x7F makes its 16 dims NaN.  Tokens past the end have their V scales
//    zeroed.  In the multi-query form a chunk that some columns see only in part takes a second
//    look: NaN scales of V are zeroed too, and the outputs whose column does see the token are
//    made NaN from a product of indicators.
//
// 64 sequences of 4096 tokens, 32 / 8 heads of 128: 64.8 us a call (302 MB: 4.67 TB/s; the slope between
// 64 and 128 sequences is 6.4 TB/s, so the rest is start, tail and combine); 8 sequences of 33k to 131k
// tokens, 64 / 8 heads: 168 us (864 MB: 5.14 TB/s).  A warp's chain of 32 tokens takes ~1.5 us however few
// run beside it, so one or two kv heads, with 6 consumer warps an SM, stay at 1.3 to 2 TB/s.
#include "kvfp8_e2m1.cuh"
#include "paged_decode_kernel.cuh"

#include <type_traits>

namespace kvfp8 {
namespace {

constexpr int kTok = 32;  // tokens of a chunk: two 16-token tiles
constexpr float kLag = 8.f;  // log2: how far scores may rise above the highest one when the reference was set
// log2: the reference lies this far below that score, so that the weights fill fp16's range from its
// top (2^(kLag + kHead) = 2^15): a weight keeps its 11 bits down to 2^-21 of the highest and is above zero
// down to 2^-32, which counts where a long tail of small weights stands against a few large ones.
constexpr float kHead = 7.f;

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

// one half of an fp16 pair in both halves (an operand selector of the packed multiply)
__device__ __forceinline__ uint32_t bcast_lo(uint32_t x) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t bcast_hi(uint32_t x) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(r) : "r"(x));
    return r;
}

// A token's scale bytes (2 KP of them): those that sel picks (every second one, one per 32-dim
// chunk), four a word.
template <int KP>
__device__ __forceinline__ void lane_bytes(const uint32_t *w, uint32_t sel, uint32_t (&out)[(KP + 3) / 4]) {
#pragma unroll
    for (int i = 0; i < (KP + 3) / 4; ++i) out[i] = __byte_perm(w[2 * i], KP > 2 ? w[2 * i + 1] : 0u, sel);
}
// the scale of chunk c as an fp16 pair (the conversion of two chunks is shared)
template <int N>
__device__ __forceinline__ uint32_t chunk_scale(const uint32_t (&bytes)[N], int c) {
    const uint32_t b = bytes[c >> 2];
    const uint32_t two = c & 2 ? f16x2_from_e4m3x2_hi(b) : f16x2_from_e4m3x2(b);
    return c & 1 ? bcast_hi(two) : bcast_lo(two);
}

// Batches of up to kOwnPlanSeqs sequences take no plan kernel: each CTA's producer warp reads the
// lengths and works out its CTA's range with a warp scan, while the other warps set up (64 sequences:
// one launch and ~3 us less than the plan kernel in front).  CTA 0 leaves the chunk prefix for the
// combine kernel.  Where no sequence can be longer than kWholeTokens (the width of the block tables
// says so) nothing is split: one CTA per sequence and head group, no partial results, no workspace
// and no combine kernel (num_ctas = 0; four sequences of up to 100 tokens: 10.3 to 8.3 us).
constexpr int kOwnPlanSeqs = 256;
constexpr int kWholeTokens = 256;

__device__ __forceinline__ CtaPlan own_plan(const KernelArgs &a, int lane) {
    if (a.num_ctas == 0) {  // short sequences: CTA s takes sequence s whole
        CtaPlan p = {0, 0, static_cast<int32_t>(blockIdx.x), 0, 0, 0, 0, 0};
        p.hi = p.ce = seq_chunks<kTok>(a, p.s, p.L);
        return p;
    }
    constexpr int kRounds = kOwnPlanSeqs / 32;
    int n[kRounds];  // chunks of sequence 32 r + lane
    int sum = 0, L = 0;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int i = 32 * r + lane;
        n[r] = i < a.num_seqs ? seq_chunks<kTok>(a, i, L) : 0;
        sum += n[r];
    }
    const int T = __reduce_add_sync(0xFFFFFFFFu, sum);
    const int P = min(T, a.num_ctas), c = blockIdx.x;
    CtaPlan p = {0, 0, 0, 0, 0, 0, 0, 0};
    if (c < P) {
        p.lo = static_cast<int32_t>(static_cast<int64_t>(c) * T / P);
        p.hi = static_cast<int32_t>(static_cast<int64_t>(c + 1) * T / P);
    }
    const bool write = c == 0 && blockIdx.y == 0;
    int32_t *cstart = const_cast<int32_t *>(a.cstart);
    int run = 0;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        if (32 * r < a.num_seqs) {
            int x = n[r];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x += y;
            }
            const int before = run + x - n[r];
            if (write && 32 * r + lane < a.num_seqs) cstart[32 * r + lane] = before;
            const unsigned here = __ballot_sync(0xFFFFFFFFu, before <= p.lo && p.lo < before + n[r]);
            if (here != 0u) {
                const int from = __ffs(here) - 1;
                p.s = 32 * r + from;
                p.cs = __shfl_sync(0xFFFFFFFFu, before, from);
                p.ce = p.cs + __shfl_sync(0xFFFFFFFFu, n[r], from);
            }
            run += __shfl_sync(0xFFFFFFFFu, x, 31);
        }
    }
    if (write && lane == 0) cstart[a.num_seqs] = T;
    p.L = min(max(a.seq_lens[p.s], 0), a.max_len);
    return p;
}

// The plan kernel's other duties, by the producer warps once their copies are issued: the rows of
// sequences without chunks are zeroed, errors of lengths and query rows flagged.
template <int HD>
__device__ __forceinline__ void finish_plan(const KernelArgs &a, int lane) {
    const int qmax = a.rows_per_seq / a.n_q;
    for (int s = blockIdx.x; s < a.num_seqs; s += gridDim.x) {
        const int raw_len = a.seq_lens[s];
        int L;
        const int n = seq_chunks<kTok>(a, s, L);
        const QueryRange qr = a.qsl ? query_range(a.qsl, s, qmax, a.qrows) : QueryRange{s, 1};
        const int raw_nq = a.qsl ? a.qsl[s + 1] - a.qsl[s] : 1;
        if (lane == 0 && (raw_len < 0 || raw_len > a.max_len || qr.count != raw_nq || (a.qsl && qr.count > L)))
            flag(a.status, KVFP8_DEV_BAD_BLOCK);
        if (n > 0) continue;
        const int64_t row = static_cast<int64_t>(a.n_q) * HD;
        uint4 *rows = reinterpret_cast<uint4 *>(a.out + qr.q0 * row);
        for (int64_t k = lane; k < qr.count * row / 8; k += 32) rows[k] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// NV: output tiles of 4 score columns per kv head (1, 2 or 4).  kv heads (consumer warps) per CTA at
// most, and CTAs per SM, by the registers of the accumulators (HD * NV / 8 of a lane) and of q.  16
// columns at head_dim 128: eight warps of 168 registers that take 32 tokens at a time (55.0 us for 32
// sequences of 4 new tokens each) against twelve of 128 that take 16 and keep q in shared memory
// (57.4): independent work within a warp counts for more than warps here.
template <int HD, int NV>
__host__ __device__ constexpr int fp4_max_heads() { return HD == 128 && NV == 4 ? 8 : HD * NV >= 256 ? 4 : 8; }
template <int HD, int NV>
__host__ __device__ constexpr int fp4_ctas_per_sm() {
    return HD == 128 && NV == 4 ? 1 : HD <= 128 && HD * NV >= 256 ? 3 : 2;
}

template <int HD, int NV, bool kMulti>
__global__ void __launch_bounds__(32 * (fp4_max_heads<HD, NV>() + 1), fp4_ctas_per_sm<HD, NV>())
decode_fp4_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                  const __grid_constant__ CUtensorMap tmks, const __grid_constant__ CUtensorMap tmvs,
                  const Fp4KernelArgs f) {
    const KernelArgs &a = f.k;
    constexpr int SEG = HD / 2;    // code bytes of a token's kv head
    constexpr int GPH = HD / 16;   // scale bytes of it
    constexpr int KP = HD / 32;    // 32-dim chunks
    constexpr int NS = (NV + 1) / 2;  // score tiles of 8 columns
    constexpr bool kPair = NV <= 2;   // how V and the weights meet, see below

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
    if (a.cta_plan != nullptr && a.cta_plan[blockIdx.x].lo >= a.cta_plan[blockIdx.x].hi) return;
    __syncthreads();

    if (warp == hpc) {
        // ------------------------------------------------------------ producer warp
        int64_t issued = 0;
        int stage = 0;
        uint32_t phase = 0;
        bool aborted = false;
        // this CTA's chunks, the sequence holding the first, that one's chunks and length
        const CtaPlan rec = a.cta_plan != nullptr ? a.cta_plan[blockIdx.x] : own_plan(a, lane);
        const int64_t chunk_lo = rec.lo, chunk_hi = rec.hi;
        int s = rec.s, L = rec.L;
        int64_t cs = rec.cs, ce = rec.ce;
        int wbase = -1 << 30;  // first block-table entry held in the lane window
        int32_t win = 0;
        if (chunk_lo < chunk_hi) prefetch_q<HD>(a, s, h0, lane);
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
            __syncwarp();  // what lane 0 waited for (the stage has been read) holds for every lane's copies
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
        if (a.cta_plan == nullptr && blockIdx.y == 0) finish_plan<HD>(a, lane);
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
        // a negative scale's sign goes into q, so the highest product is always the highest score
        const uint32_t q_sign = score_scale < 0.f ? 0x80008000u : 0u;
        score_scale = fabsf(score_scale);
        if (score_scale == 0.f) score_scale = 0x1p-126f;  // underflow: equal weights, -inf stays -inf

        // The lane's score columns, v = 0..NV-1 (column x: query token x / group, head x % group).
        // kPair: x = 4v + tig, which is n = 2 tig + v % 2 of score tile v / 2.
        // Otherwise columns are in order, n = x % 8 of tile x / 8, so x = 8 (v / 2) + 2 tig + v % 2.
        auto column = [&](int v) { return kPair ? 4 * v + tig : 8 * (v / 2) + 2 * tig + v % 2; };
        float o[NV][KP][4];
        // dim 32c + 4 gid + r of column v
        auto at = [&](int v, int c, int r) -> float & {
            return kPair ? o[v][c][r] : o[(v & ~1) + (r >> 1)][c][(v & 1) + 2 * (r & 1)];
        };
        // per column: the reference (log2 domain) the weights are taken against, and this
        // lane's part of the sum of weights
        float m[NV], l[NV];
        uint32_t qb[KP][NS][4];
        // multi-query form: the sequence's first query row, its query tokens and the last cache position
        // the first of them may see
        int q0 = 0, nq = 1, first_lim = 0;

        // Offsets of this lane in a stage, for the first 16-token tile (the second: c2, s2 further).
        const uint32_t head_codes = static_cast<uint32_t>(warp * a.box_rows * SEG);
        const uint32_t head_scales = static_cast<uint32_t>(warp * a.box_rows * GPH);
        // (an 8-token group of a head is aligned to 8 SEG bytes, so a chunk pair further is an xor)
        const uint32_t krow_off = head_codes + ((lane >> 3) & 1) * f.c1 + swz<SEG>(lane & 7, lane >> 4);
        // V: at head_dim 64 one ldmatrix takes both halves of a tile (the matrices are half, chunk), else
        // four chunks of one half
        const uint32_t vrow_off =
            code_bytes + head_codes +
            (HD == 64 ? (lane >> 4) * f.c1 + swz<SEG>(lane & 7, (lane >> 3) & 1) : swz<SEG>(lane & 7, lane >> 3));
        const uint32_t ks_off = scales_off + head_scales + gid * GPH;
        const uint32_t vs_off = vscales_off + head_scales + 2 * tig * GPH;
        const uint32_t ksel = 0x6420u + 0x1111u * (tig >> 1);  // bytes of this lane's K groups
        const uint32_t vsel = 0x6420u + 0x1111u * (gid >> 2);  // and of its V groups
        // halves of a token pair's weights -> B fragment words (token, dim parity) of column gid
        const uint32_t bsel0 = gid & 1 ? 0x1044u : 0x4410u, bsel1 = gid & 1 ? 0x3244u : 0x4432u;

        int stage = 0;
        uint32_t phase = 0;
        for (;;) {
            // every lane waits (acquire on the TMA bytes); the outcome is made warp-uniform
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
                if (kMulti) {
                    const QueryRange qr = query_range(a.qsl, mt.seq, a.rows_per_seq / a.n_q, a.qrows);
                    q0 = qr.q0;
                    nq = qr.count;
                    first_lim = min(max(a.seq_lens[mt.seq], 0), a.max_len) - nq;
                }
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const int x = 8 * s + (kPair ? (gid >> 1) + 4 * (gid & 1) : gid);  // column gid of score tile s
                    const int jq = kMulti ? x / a.group : 0;
                    const int gq = kMulti ? x % a.group : x;
                    const bool qv = kMulti ? jq < nq : x < a.group;
                    const __nv_bfloat16 *qrow =
                        a.query +
                        ((static_cast<int64_t>(kMulti ? q0 + jq : mt.seq)) * a.n_q + kvh * a.group + gq) * HD;
#pragma unroll
                    for (int c = 0; c < KP; ++c) {
                        uint4 w = make_uint4(0u, 0u, 0u, 0u);
                        if (qv) w = *reinterpret_cast<const uint4 *>(qrow + 32 * c + 8 * tig);
                        qb[c][s][0] = f16x2_from_f32(bf16lo(w.x), bf16hi(w.x)) ^ q_sign;
                        qb[c][s][1] = f16x2_from_f32(bf16lo(w.y), bf16hi(w.y)) ^ q_sign;
                        qb[c][s][2] = f16x2_from_f32(bf16lo(w.z), bf16hi(w.z)) ^ q_sign;
                        qb[c][s][3] = f16x2_from_f32(bf16lo(w.w), bf16hi(w.w)) ^ q_sign;
                    }
                }
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    m[v] = -INFINITY;
                    l[v] = 0.f;
#pragma unroll
                    for (int c = 0; c < KP; ++c)
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[v][c][r] = 0.f;
                }
            }

            // kPartial: some column does not see some token of the chunk.  The common chunk has a body
            // without those tests: one basic block from the weights to the last product.
            auto chunk = [&](auto partial_tag) {
                constexpr bool kPartial = decltype(partial_tag)::value;
                const uint32_t st = base + static_cast<uint32_t>(stage) * stage_bytes;
                auto sees = [&](int row, int v) {  // row of the chunk
                    if (((mt.mask >> row) & 1u) == 0u) return false;
                    if (!kMulti) return true;
                    const int j = column(v) / a.group;  // its query token; padding columns see nothing
                    return j < nq && mt.tok0 + row <= first_lim + j;
                };

                // ---- scores S^T[token][column] = K . q^T, tiles of 16 tokens
                float sacc[2][NS][4];
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    // scale bytes of this lane's groups, rows gid and +8
                    uint32_t sl[(KP + 3) / 4], sh[(KP + 3) / 4];
                    {
                        uint32_t w[2][GPH / 4];
                        lds(st + ks_off + tt * f.s2, w[0]);
                        lds(st + ks_off + tt * f.s2 + f.s1, w[1]);
                        lane_bytes<KP>(w[0], ksel, sl);
                        lane_bytes<KP>(w[1], ksel, sh);
                    }
                    // kSums running sums, so that a product waits for the one before the last only (170.0
                    // against 171.7 us on eight long sequences; for 16 columns the registers cost more)
                    constexpr int kSums = NV <= 2 ? 2 : 1;
                    float part[kSums][NS][4];
#pragma unroll
                    for (int k = 0; k < kSums; ++k)
#pragma unroll
                        for (int s = 0; s < NS; ++s)
                            part[k][s][0] = part[k][s][1] = part[k][s][2] = part[k][s][3] = 0.f;
#pragma unroll
                    for (int cp = 0; cp < KP / 2; ++cp) {
                        uint32_t r[4];
                        ldsm_x4((st + krow_off + tt * f.c2) ^ (cp << 5), r[0], r[1], r[2], r[3]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {  // chunk 2cp + e
                            const uint32_t xl = chunk_scale(sl, 2 * cp + e), xh = chunk_scale(sh, 2 * cp + e);
                            uint32_t ka[4], kb[4];
                            f16x2_from_e2m1x8(r[2 * e], ka);
                            f16x2_from_e2m1x8(r[2 * e + 1], kb);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                ka[i] = hmul2(ka[i], xl);
                                kb[i] = hmul2(kb[i], xh);
                            }
#pragma unroll
                            for (int s = 0; s < NS; ++s) {
                                const uint32_t(&q)[4] = qb[2 * cp + e][s];
                                mma16816(part[0][s], ka[0], kb[0], ka[1], kb[1], q[0], q[1]);
                                mma16816(part[kSums - 1][s], ka[2], kb[2], ka[3], kb[3], q[2], q[3]);
                            }
                        }
                    }
#pragma unroll
                    for (int s = 0; s < NS; ++s)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sacc[tt][s][i] = kSums == 2 ? part[0][s][i] + part[kSums - 1][s][i] : part[0][s][i];
                }

                // ---- weights 2^(score - m) per column (log2 domain).  m only has to be near the running
                // maximum less kHead: it moves when a score passes it by more than kLag + kHead, so most
                // chunks take no maximum over the lanes and rescale nothing, and weights stay <= 2^(kLag +
                // kHead).  Tokens a column does not see get -inf.
                if constexpr (kPartial) {
#pragma unroll
                    for (int v = 0; v < NV; ++v)
#pragma unroll
                        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (!sees(16 * tt + 8 * h + gid, v)) sacc[tt][v / 2][v % 2 + 2 * h] = -INFINITY;
                }
                auto column_top = [&](int v) {  // this lane's highest score of column v
                    const int s = v / 2, c = v % 2;
                    return score_scale *
                           fmaxf(fmaxf(sacc[0][s][c], sacc[0][s][c + 2]), fmaxf(sacc[1][s][c], sacc[1][s][c + 2]));
                };
                float top = -INFINITY;  // the highest score over its column's m
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
                            const float alpha = m[v] == -INFINITY ? 1.f : ex2(m[v] - x);
                            m[v] = x;
                            l[v] *= alpha;
#pragma unroll
                            for (int c = 0; c < KP; ++c)
#pragma unroll
                                for (int r = 0; r < 4; ++r) at(v, c, r) *= alpha;
                        }
                    }
                }
                // Weights as B fragments, through a register transpose.  kPair: of 8 tokens for output tile
                // v, whose product runs over (token, dim parity): A's rows are pairs of dims as the
                // conversion leaves them, and column n of B has the weights of column 4v + n / 2 at the
                // parity n % 2, zeros at the other.  Otherwise of 16 tokens for score tile s.
                auto fragment = [&](uint32_t w, uint32_t (&b)[2]) {  // w: tokens 2 tig, +1 of column gid / 2
                    b[0] = __byte_perm(w, 0u, bsel0);
                    b[1] = __byte_perm(w, 0u, bsel1);
                };
                constexpr int NW = kPair ? NV : NS;
                uint32_t pw[2][2][NW];  // tokens 16 tt + 8 h + 2 tig, + 1
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    constexpr int kCols = kPair ? 1 : 2;  // columns of a word
                    float p[kCols][2][2];
#pragma unroll
                    for (int k = 0; k < kCols; ++k) {
                        const int v = kPair ? w : 2 * w + k;
                        // a column that has seen no score yet: -inf - 0 for every token
                        const float sub = m[v] == -INFINITY ? 0.f : m[v];
#pragma unroll
                        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                p[k][tt][h] = ex2(fmaf(sacc[tt][v / 2][v % 2 + 2 * h], score_scale, -sub));
                        l[v] += (p[k][0][0] + p[k][0][1]) + (p[k][1][0] + p[k][1][1]);
                    }
#pragma unroll
                    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            pw[tt][h][w] = movm_t(f16x2_from_f32(p[0][tt][h], p[kCols - 1][tt][h]));
                }

                // ---- O^T[dim][column] += V^T . P^T
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    // scale bytes of this lane's groups: tokens 8h + 2 tig and + 1
                    auto value_scales = [&](int h, uint32_t (&vs)[2][(KP + 3) / 4]) {
                        uint32_t w[GPH / 2];  // both tokens' bytes
                        lds(st + vs_off + tt * f.s2 + h * f.s1, w);
                        lane_bytes<KP>(w, vsel, vs[0]);
                        lane_bytes<KP>(w + GPH / 4, vsel, vs[1]);
                        if constexpr (kPartial) {
                            // Tokens that are not there: scale 0.  A column that does not see a token has
                            // weight 0 for it, and a NaN scale would make 0 * NaN of that, so NaN scales
                            // become 0 too and the outputs that do see the token are made NaN.
                            uint32_t nan[2][(KP + 3) / 4], any = 0;
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int i = 0; i < (KP + 3) / 4; ++i) {
                                    if (!((mt.mask >> (16 * tt + 8 * h + 2 * tig + k)) & 1u)) vs[k][i] = 0u;
                                    nan[k][i] = kMulti ? nan_byte_mask(vs[k][i]) : 0u;
                                    any |= nan[k][i];
                                }
                            if (!kMulti || !__any_sync(0xFFFFFFFFu, any != 0u)) return;
#pragma unroll
                            for (int v = 0; v < NV; ++v) {
                                uint32_t seen[2];  // fp16 ones where the column sees the token (at both parities)
                                fragment(movm_t(sees(16 * tt + 8 * h + gid, v) ? 0x3C003C00u : 0u), seen);
#pragma unroll
                                for (int c = 0; c < KP; ++c) {
                                    const uint32_t n0 = (nan[0][c >> 2] >> (8 * (c & 3))) & 1u ? 0x3C003C00u : 0u;
                                    const uint32_t n1 = (nan[1][c >> 2] >> (8 * (c & 3))) & 1u ? 0x3C003C00u : 0u;
                                    // NaN tokens that the lane's column v sees (every element the same count)
                                    float cnt[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma16816(cnt, n0, n0, n1, n1, seen[0], seen[1]);
#pragma unroll
                                    for (int r = 0; r < 4; ++r)
                                        if (cnt[0] > 0.f) at(v, c, r) = __uint_as_float(0x7FC00000u);
                                }
                            }
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int i = 0; i < (KP + 3) / 4; ++i) vs[k][i] &= ~nan[k][i];
                        }
                    };
                    // the codes of chunks 4 c4.. of half h (at head_dim 64 one load has both halves)
                    uint32_t r64[4];
                    if constexpr (HD == 64)
                        ldsm_x4_t(st + vrow_off + tt * f.c2, r64[0], r64[1], r64[2], r64[3]);
                    auto value_codes = [&](int h, int c4, uint32_t (&r)[4]) {
                        if constexpr (HD == 64) {
                            r[0] = r64[2 * h];
                            r[1] = r64[2 * h + 1];
                        } else {
                            ldsm_x4_t((st + vrow_off + tt * f.c2 + h * f.c1) ^ (c4 << 6), r[0], r[1], r[2], r[3]);
                        }
                    };
                    constexpr int kC = KP < 4 ? KP : 4;  // chunks of a load
                    if constexpr (kPair) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t vs[2][(KP + 3) / 4], pb[NV][2];
                            value_scales(h, vs);
#pragma unroll
                            for (int v = 0; v < NV; ++v) fragment(pw[tt][h][v], pb[v]);
#pragma unroll
                            for (int c4 = 0; c4 < (KP + 3) / 4; ++c4) {
                                uint32_t r[4];
                                value_codes(h, c4, r);
#pragma unroll
                                for (int e = 0; e < kC; ++e) {
                                    const int c = 4 * c4 + e;
                                    uint32_t x[4];  // token 2 tig: dims 4g, +1 and +2, +3; then token 2 tig + 1
                                    f16x2_from_e2m1x8(r[e], x);
                                    const uint32_t s0 = chunk_scale(vs[0], c), s1 = chunk_scale(vs[1], c);
                                    x[0] = hmul2(x[0], s0);
                                    x[1] = hmul2(x[1], s0);
                                    x[2] = hmul2(x[2], s1);
                                    x[3] = hmul2(x[3], s1);
#pragma unroll
                                    for (int v = 0; v < NV; ++v)
                                        mma16816(o[v][c], x[0], x[1], x[2], x[3], pb[v][0], pb[v][1]);
                                }
                            }
                        }
                    } else {
                        uint32_t vs[2][2][(KP + 3) / 4];
                        value_scales(0, vs[0]);
                        value_scales(1, vs[1]);
#pragma unroll
                        for (int c4 = 0; c4 < (KP + 3) / 4; ++c4) {
                            uint32_t r[2][4];
                            value_codes(0, c4, r[0]);
                            value_codes(1, c4, r[1]);
#pragma unroll
                            for (int e = 0; e < kC; ++e) {
                                const int c = 4 * c4 + e;
                                // per half: scaled dims (4g, +1), (4g + 2, +3) of token 2 tig, then of 2 tig + 1
                                uint32_t x[2][4];
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    f16x2_from_e2m1x8(r[h][e], x[h]);
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        x[h][i] = hmul2(x[h][i], chunk_scale(vs[h][i >> 1], c));
                                }
#pragma unroll
                                for (int j = 0; j < 2; ++j) {  // token pairs of dims 4g + 2j, 4g + 2j + 1
                                    const uint32_t a0 = __byte_perm(x[0][j], x[0][j + 2], 0x5410);
                                    const uint32_t a1 = __byte_perm(x[0][j], x[0][j + 2], 0x7632);
                                    const uint32_t a2 = __byte_perm(x[1][j], x[1][j + 2], 0x5410);
                                    const uint32_t a3 = __byte_perm(x[1][j], x[1][j + 2], 0x7632);
#pragma unroll
                                    for (int s = 0; s < NS; ++s)
                                        mma16816(o[2 * s + j][c], a0, a1, a2, a3, pw[tt][0][s], pw[tt][1][s]);
                                }
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
                    const float inv = lt == 0.f ? 0.f : (direct ? sv : 1.f) / lt;
#pragma unroll
                    for (int c = 0; c < KP; ++c) {
                        const int d = 32 * c + 4 * gid;
                        const float x0 = at(v, c, 0) * inv, x1 = at(v, c, 1) * inv;
                        const float x2 = at(v, c, 2) * inv, x3 = at(v, c, 3) * inv;
                        if (direct)
                            *reinterpret_cast<uint2 *>(a.out + orow_idx * HD + d) =
                                make_uint2(bf16x2_from_f32(x0, x1), bf16x2_from_f32(x2, x3));
                        else
                            *reinterpret_cast<float4 *>(a.part_o + (pidx * a.rows_per_seq + srow) * HD + d) =
                                make_float4(x0, x1, x2, x3);
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

template <int HD, int NV, bool kMulti>
cudaError_t run_fp4(const DecodeArgs &d, const DecodeWorkspace &ws, cudaStream_t stream) {
    DeviceFacts facts;
    cudaError_t err = device_facts(&facts);
    if (err != cudaSuccess) return err;
    const int sms = facts.sms, smem_optin = facts.smem_optin;

    // kv heads per CTA: the largest divisor of n_kv up to the limit; the groups are a grid dimension
    int hpc = std::min(d.n_kv, fp4_max_heads<HD, NV>());
    while (d.n_kv % hpc != 0) --hpc;
    const int groups = d.n_kv / hpc;
    if (groups > 65535) return cudaErrorNotSupported;  // gridDim.y (a large prime n_kv)
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
    // CTAs of fewer heads than the limit: as many as have that many warps in all (2 kv heads of 64, two
    // sequences of 102k tokens: 36 to 22 us; 64 of 4096: 26.8 to 19.3)
    const int ctas_per_sm = fp4_ctas_per_sm<HD, NV>() * (fp4_max_heads<HD, NV>() + 1) / (hpc + 1);
    constexpr int kMaxStages = 8;
    auto smem_for = [&](int st) { return static_cast<size_t>(st) * (f.stage_bytes + 32) + 16 + 1024; };
    const size_t sm_budget = static_cast<size_t>(smem_optin) + 1024;
    int stages = kMaxStages;
    while (stages > 2 && (smem_for(stages) + 1024) * ctas_per_sm > sm_budget) --stages;
    const size_t smem = smem_for(stages);
    if (smem > static_cast<size_t>(smem_optin)) return cudaErrorNotSupported;

    auto kern = decode_fp4_kernel<HD, NV, kMulti>;
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

    const bool whole = fp4_takes_sequences_whole(d.max_blocks_per_seq, d.block_size);
    const bool own_plan = whole || d.num_seqs <= kOwnPlanSeqs;
    if (own_plan) {
        k.cta_plan = nullptr;
        if (whole) k.num_ctas = 0;
    } else {
        plan_kernel<kTok><<<1, 1024, 0, stream>>>(d.seq_lens, d.qsl, d.qmax, d.qrows, d.num_seqs,
                                                  k.max_len, num_ctas,
                                                  reinterpret_cast<int32_t *>(w + ws.cstart_off),
                                                  reinterpret_cast<CtaPlan *>(w + ws.cta_off), k.out,
                                                  d.n_q * HD, d.status);
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
    cfg.numAttrs = own_plan ? 0 : 1;  // (only a kernel of this call may be overtaken)
    if ((err = cudaLaunchKernelEx(&cfg, kern, tmk, tmv, tmks, tmvs, f)) != cudaSuccess || whole) return err;

    constexpr int kHeadsPerCta = 256 / (HD / 4);
    cudaLaunchConfig_t ccfg = cfg;
    ccfg.numAttrs = 1;
    ccfg.gridDim = dim3(d.num_seqs, (k.rows_per_seq + kHeadsPerCta - 1) / kHeadsPerCta);
    ccfg.dynamicSmemBytes = 0;
    const int64_t parts = (static_cast<int64_t>(num_ctas) + d.num_seqs) / std::max(1, d.num_seqs);
    // few, long sequences: a CTA per row, 512 threads over its parts, while that is one wave (one sequence of
    // 98k tokens, 64 heads: 45.5 to 34 us; eleven of 539, 704 rows of 17 parts: 20.6 against 12.5)
    if (parts >= 32 && static_cast<int64_t>(d.num_seqs) * k.rows_per_seq <= 4 * sms) {
        constexpr int kSlices = 512 / (HD / 4);
        ccfg.gridDim = dim3(d.num_seqs, k.rows_per_seq);
        ccfg.blockDim = dim3(512);
        return cudaLaunchKernelEx(&ccfg, combine_kernel<HD, kSlices, 1>, k);
    }
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

template <int HD>
cudaError_t run_tiles(const DecodeArgs &d, const DecodeWorkspace &ws, int tiles, cudaStream_t stream) {
    const bool multi = d.qsl != nullptr;
    if (tiles <= 1) return multi ? run_fp4<HD, 1, true>(d, ws, stream) : run_fp4<HD, 1, false>(d, ws, stream);
    if (tiles <= 2) return multi ? run_fp4<HD, 2, true>(d, ws, stream) : run_fp4<HD, 2, false>(d, ws, stream);
    if constexpr (HD <= 128)
        return multi ? run_fp4<HD, 4, true>(d, ws, stream) : run_fp4<HD, 4, false>(d, ws, stream);
    return cudaErrorNotSupported;
}

}  // namespace

bool fp4_takes_sequences_whole(int32_t max_blocks_per_seq, int32_t block_size) {
    return static_cast<int64_t>(max_blocks_per_seq) * block_size <= kWholeTokens;
}

cudaError_t launch_paged_decode_fp4(const DecodeArgs &d, cudaStream_t stream) {
    if (d.num_seqs == 0) return cudaSuccess;
    if (!multi_uses_decode_kernel(d.n_q, d.n_kv, d.head_dim, d.qmax))
        return launch_prefill_attention(d, stream);
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
