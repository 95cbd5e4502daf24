// What the tensor-core (tcgen05) attention kernels for long query chunks share: PTX wrappers, operand
// descriptors, the order of the work and how keys are split over CTAs.
#pragma once

#include "paged_decode_kernel.cuh"

namespace kvfp8 {
namespace {

constexpr int kPfRows = 128;   // score rows per CTA (TMEM lanes)

// ---------------------------------------------------------------- tcgen05 wrappers

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
                 "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}
// D (TMEM) (+)= A (shared memory descriptor) x B (shared memory descriptor)
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D (TMEM) (+)= A (TMEM) x B (shared memory descriptor)
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// arrive on the mbarrier once every tcgen05.mma this thread issued before has completed
__device__ __forceinline__ void umma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// four 8x8 b16 matrices stored transposed: lane t gives (rows 2(t%4), 2(t%4)+1; column t/4)
// of matrix j in r[j], and the address of row t%8 of matrix t/8
__device__ __forceinline__ void stsm_x4_t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2,
                                          uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
                 "r"(r0), "r"(r1), "r"(r2), "r"(r3)
                 : "memory");
}

// generic-proxy shared-memory writes become visible to the tensor core (async proxy)
__device__ __forceinline__ void fence_proxy_async() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}

// Shared-memory matrix descriptor: K-major operand in the 128-byte swizzle layout (rows of
// 128 bytes, 16-byte chunks XOR-ed with row % 8, 8-row groups 1024 bytes apart).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu)  // start address
           | (1ull << 16)                                 // leading byte offset (unused here)
           | (static_cast<uint64_t>(1024 >> 4) << 32)     // stride byte offset: 8 rows
           | (1ull << 46)                                 // descriptor version
           | (2ull << 61);                                // 128-byte swizzle
}
// The descriptor of an address off bytes (a multiple of 16) past one whose descriptor is d:
// the start-address field is (address >> 4) in 14 bits, and every shared-memory address of
// a CTA is below 2^18, so the field never carries into the next one.
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t off) { return d + (off >> 4); }

// Instruction descriptor, kind::f16: f16 A and B, fp32 D, both K-major, M x N.
__host__ __device__ constexpr uint32_t f16_idesc(int m, int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
// byte offset of 16-byte chunk c of row r in a 128-byte-swizzled K-major block
__device__ __forceinline__ uint32_t sw128(int r, int c) {
    return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
}

// packed fp32 pairs (sm_100+ f32x2 arithmetic: two IEEE round-to-nearest operations)
__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint64_t pk2u(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ float2 upk2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float min3f(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// the largest (kMax) or smallest of 32 scores, four chains of 3-input ops
template <bool kMax>
__device__ __forceinline__ float extreme32(const uint32_t (&s)[32]) {
    auto v = [&](int c) { return __uint_as_float(s[c]); };
    auto op = [](float a, float b, float c) { return kMax ? max3f(a, b, c) : min3f(a, b, c); };
    float a0 = v(0), a1 = v(1), a2 = v(2), a3 = v(3);
#pragma unroll
    for (int c = 4; c < 28; c += 8) {
        a0 = op(a0, v(c), v(c + 1));
        a1 = op(a1, v(c + 2), v(c + 3));
        a2 = op(a2, v(c + 4), v(c + 5));
        a3 = op(a3, v(c + 6), v(c + 7));
    }
    a0 = op(a0, v(28), v(29));
    a1 = op(a1, v(30), v(31));
    return op(a0, a1, kMax ? fmaxf(a2, a3) : fminf(a2, a3));
}

struct PrefillCommon {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *query;
    const int32_t *qsl;
    int32_t qmax, qrows;
    const int32_t *block_tables;
    int32_t max_blocks_per_seq;
    const int32_t *seq_lens;
    int32_t num_seqs;
    int32_t n_q, n_kv, group, block_size, num_blocks, max_len;
    float sm_scale;
    const void *k_scale;
    const void *v_scale;
    int32_t scale_dtype;
    uint32_t *status;
    int32_t box_rows;
    int32_t row_tiles;  // tiles of 128 score rows per (sequence, kv head)
};
// Few row tiles (a short chunk or a wide group of heads on a long context) would leave most SMs idle, so
// their keys are cut: part p of a row tile takes key tiles [p n / parts, (p + 1) n / parts), leaves its
// normalized rows and their log2 sums of weights in the workspace, and a second kernel joins them.  A part
// is 128 keys at least (8 tokens on 1024, 32 / 8 heads of 128: 21.5 us unsplit, 16.4 / 12.7 / 11.1 with
// parts of 512 / 256 / 128; on 4096 17.6 / 15.0 / 16.0).  Nothing is split when more than half the SMs have
// a row tile: 80 to 216 tiles of equal lengths gained at most 7 % from any number of parts and lost up to
// 60 % (unequal ones were not measured).  (kSplit is an instance of its own: the few instructions cost the
// unsplit kernel of two row tiles 11 %, 531 against 478 us for 512 new tokens of 16 sequences of 4096.)
constexpr int kSplitSms = 152;
constexpr int kMinPartKeys = 128;
__host__ __device__ constexpr int split_parts(int splits, int key_tiles, int tile_keys) {
    const int most = key_tiles / (kMinPartKeys / tile_keys);
    return splits < most ? splits : most > 1 ? most : 1;
}

// ---------------------------------------------------------------- work order
//
// The CTAs of the sequences with the most keys go first.  The hardware starts CTAs in index
// order as SMs free up, so giving the low indices to the longest sequences keeps one of them
// from starting last and running alone at the end (longest-processing-time-first list
// scheduling; with lengths log-uniform over 16..32768 tokens, as in a serving mix, index
// order leaves the last SMs busy ~20 % past the mean).  Sequences are ranked by a bucket of
// their length, four buckets per octave (lengths in one bucket differ by less than 19 %),
// longest bucket first, and by index within a bucket.

__device__ __forceinline__ int length_bucket(int len, int max_len) {
    const int l = min(max(len, 0), max_len);
    if (l == 0) return 0;
    const int b = 31 - __clz(l);                                     // floor(log2 l), 0..30
    const int frac = b >= 2 ? (l >> (b - 2)) & 3 : (l << (2 - b)) & 3;  // next two bits
    return 1 + 4 * b + frac;                                         // 1..124
}

// The sequence of rank u (0 = longest).  Every thread of the CTA calls it (it synchronizes
// the CTA); scratch is 168 words of this CTA's shared memory, free until it returns.
__device__ __forceinline__ int seq_of_rank(const int32_t *seq_lens, int num_seqs, int max_len, int u,
                           uint32_t *scratch) {
    if (num_seqs <= 1) return u;
    uint32_t *cnt = scratch;                      // [128] sequences per bucket
    // bucket of rank u, rank within it, the result, and whether the result is final
    volatile uint32_t *pick = scratch + 128;
    volatile uint32_t *wsum = scratch + 136;      // [32] per-warp counts of one round
    const int tid = threadIdx.x, nthr = blockDim.x, warp = tid >> 5, lane = tid & 31;
    const int nwarps = nthr >> 5;
    // bucket of sequence tid, kept for the histogram and the first round of the scan
    const int my_bucket = tid < num_seqs ? length_bucket(seq_lens[tid], max_len) : -1;
    if (num_seqs <= nthr) {  // lengths all in one bucket (a batch of equal lengths): index order
        const int b0 = length_bucket(seq_lens[0], max_len);
        if (__syncthreads_and(tid >= num_seqs || my_bucket == b0)) return u;
    }
    for (int b = tid; b < 128; b += nthr) cnt[b] = 0u;
    if (tid == 0) {  // (u < num_seqs always finds its bucket; index order otherwise)
        pick[0] = 0u;
        pick[1] = 0u;
        pick[2] = static_cast<uint32_t>(u);
        pick[3] = 0u;
    }
    __syncthreads();
    for (int s = tid; s < num_seqs; s += nthr)
        atomicAdd(&cnt[s == tid ? my_bucket : length_bucket(seq_lens[s], max_len)], 1u);
    __syncthreads();
    if (warp == 0) {
        // lane l holds buckets 127-4l .. 124-4l, so lanes run longest first
        uint32_t c[4], tot = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            c[q] = cnt[127 - 4 * lane - q];
            tot += c[q];
        }
        uint32_t incl = tot;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += v;
        }
        uint32_t before = incl - tot;
        const uint32_t uu = static_cast<uint32_t>(u);
        if (uu >= before && uu < incl) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (uu < before + c[q]) {
                    pick[0] = static_cast<uint32_t>(127 - 4 * lane - q);
                    pick[1] = uu - before;
                    // every sequence in one bucket (a batch of equal lengths): index order
                    if (c[q] == static_cast<uint32_t>(num_seqs)) pick[3] = 1u;
                    break;
                }
                before += c[q];
            }
        }
    }
    __syncthreads();
    if (pick[3] != 0u) return u;
    const int B = static_cast<int>(pick[0]);
    const uint32_t k = pick[1];
    // the k-th sequence of bucket B in index order, nthr sequences a round
    uint32_t seen = 0;
    for (int s0 = 0; s0 < num_seqs; s0 += nthr) {
        const int s = s0 + tid;
        const int b = s0 == 0 ? my_bucket : (s < num_seqs ? length_bucket(seq_lens[s], max_len) : -1);
        const bool in = s < num_seqs && b == B;
        const uint32_t bal = __ballot_sync(0xFFFFFFFFu, in);
        if (lane == 0) wsum[warp] = static_cast<uint32_t>(__popc(bal));
        __syncthreads();
        uint32_t pre = seen, tot = 0;
        for (int w = 0; w < nwarps; ++w) {
            const uint32_t v = wsum[w];
            if (w < warp) pre += v;
            tot += v;
        }
        pre += static_cast<uint32_t>(__popc(bal & ((1u << lane) - 1u)));
        if (in && pre == k) pick[2] = static_cast<uint32_t>(s);
        seen += tot;
        __syncthreads();  // pick[2] is written; wsum may be reused
        if (seen > k) break;
    }
    return static_cast<int>(pick[2]);
}

}  // namespace
}  // namespace kvfp8
