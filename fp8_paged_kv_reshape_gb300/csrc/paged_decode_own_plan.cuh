// The plan of a split-KV decode grid worked out by its own producer warps, for kernels whose chunks are
// kTok tokens.
#pragma once

#include "paged_decode_kernel.cuh"

namespace kvfp8 {
namespace {

// Batches of up to kOwnPlanSeqs sequences take no plan kernel: each CTA's producer warp reads the
// lengths and works out its CTA's range with a warp scan, while the other warps set up (64 sequences:
// one launch and ~3 us less than the plan kernel in front).  CTA 0 leaves the chunk prefix for the
// combine kernel.  Where no sequence can be longer than kWholeTokens (the width of the block tables
// says so) nothing is split: one CTA per sequence and head group, no partial results, no workspace
// and no combine kernel (num_ctas = 0; four sequences of up to 100 tokens: 10.3 to 8.3 us).
constexpr int kOwnPlanSeqs = 256;
constexpr int kWholeTokens = 256;

template <int kTok>
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
// (causal: a sequence with more query rows than tokens is an error.)
template <int HD, int kTok>
__device__ __forceinline__ void finish_plan(const KernelArgs &a, int lane, bool causal) {
    const int qmax = a.rows_per_seq / a.n_q;
    for (int s = blockIdx.x; s < a.num_seqs; s += gridDim.x) {
        const int raw_len = a.seq_lens[s];
        int L;
        const int n = seq_chunks<kTok>(a, s, L);
        const QueryRange qr = a.qsl ? query_range(a.qsl, s, qmax, a.qrows) : QueryRange{s, 1};
        const int raw_nq = a.qsl ? a.qsl[s + 1] - a.qsl[s] : 1;
        if (lane == 0 && (raw_len < 0 || raw_len > a.max_len || qr.count != raw_nq || (a.qsl && causal && qr.count > L)))
            flag(a.status, KVFP8_DEV_BAD_BLOCK);
        if (n > 0) continue;
        const int64_t row = static_cast<int64_t>(a.n_q) * HD;
        uint4 *rows = reinterpret_cast<uint4 *>(a.out + qr.q0 * row);
        for (int64_t k = lane; k < qr.count * row / 8; k += 32) rows[k] = make_uint4(0u, 0u, 0u, 0u);
    }
}

}  // namespace
}  // namespace kvfp8
