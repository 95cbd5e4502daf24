// Pages of the paged caches: copying blocks and compacting a pool, sm_103a.
//
// Both move whole blocks of several device arrays (the K and V caches and scale arrays of one
// or more layers) and are bound by HBM: 2 bytes of traffic per byte moved.  The work is cut
// into segments of a block, one per warp at a time: 32 lanes x 32 bytes x up to 4 loads in
// flight, streamed past L1, so that a handful of small blocks still spreads over the SMs and a
// large copy keeps every SM's loads outstanding.
#include <cuda_runtime.h>

#include <algorithm>

#include "kvfp8_device.cuh"
#include "kvfp8_internal.h"

namespace kvfp8 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// The caches' segments: segment x of a block (0 <= x < seg0[count]) belongs to the cache c with
// seg0[c] <= x < seg0[c + 1] and starts (x - seg0[c]) * seg_bytes into its block.
struct SegMap {
    CacheList caches;
    int32_t seg0[KVFP8_MAX_CACHES + 1];
    int32_t seg_bytes;  // a multiple of 1024
};

__device__ __forceinline__ void ld_stream(const uint8_t *p, uint32_t (&w)[8]) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void st_stream(uint8_t *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// One warp copies bytes [0, n) (n a multiple of 16), 1024 or 4096 bytes a round.
// kWide: both sides are 32-byte aligned and n is a multiple of 32.
template <bool kWide>
__device__ __forceinline__ void copy_bytes(uint8_t *dst, const uint8_t *src, int64_t n, int lane) {
    if (kWide) {
        int64_t off = static_cast<int64_t>(lane) * 32;
        for (; off + 3 * 1024 < n; off += 4096) {
            uint32_t w[4][8];
#pragma unroll
            for (int k = 0; k < 4; ++k) ld_stream(src + off + 1024 * k, w[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k) st_stream(dst + off + 1024 * k, w[k]);
        }
        for (; off < n; off += 1024) {
            uint32_t w[8];
            ld_stream(src + off, w);
            st_stream(dst + off, w);
        }
    } else {
        for (int64_t off = static_cast<int64_t>(lane) * 16; off < n; off += 512)
            *reinterpret_cast<uint4 *>(dst + off) = __ldcs(reinterpret_cast<const uint4 *>(src + off));
    }
}

// Segment x of block `from` to block `to`.
template <bool kWide>
__device__ __forceinline__ void copy_segment(const SegMap &m, int32_t x, int32_t from, int32_t to, int lane) {
    int lo = 0, hi = m.caches.count;  // seg0[lo] <= x < seg0[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (m.seg0[mid] <= x) lo = mid; else hi = mid;
    }
    const int64_t bytes = m.caches.block_bytes[lo];
    const int64_t off = static_cast<int64_t>(x - m.seg0[lo]) * m.seg_bytes;
    uint8_t *base = m.caches.ptr[lo];
    copy_bytes<kWide>(base + to * bytes + off, base + from * bytes + off,
                      min(static_cast<int64_t>(m.seg_bytes), bytes - off), lane);
}

// kvfp8_copy_blocks.  Pairs that name one block twice would race, so each CTA first marks every
// pair's destination in a bitmap of the pool in shared memory (and in a second one the blocks
// that are a destination twice); a pair is carried out when its destination is not in the second
// and its source is in neither.  That costs each CTA one pass over the pairs (from L2, the loads of
// eight pairs a thread in flight together) and no memory of the caller's.
constexpr int kCopyThreads = 1024;

template <bool kWide>
__global__ void __launch_bounds__(kCopyThreads)
copy_blocks_kernel(const __grid_constant__ SegMap m, const int32_t num_blocks, const int32_t *src,
                   const int32_t *dst, const int32_t num_pairs, uint32_t *status) {
    extern __shared__ uint32_t marks[];
    const int words = (num_blocks + 31) >> 5;
    uint32_t *once = marks, *twice = marks + words;
    const int tid = threadIdx.x, lane = tid & 31;
    for (int i = tid; i < 2 * words; i += kCopyThreads) marks[i] = 0u;
    __syncthreads();
    auto inside = [&](int32_t b) { return b >= 0 && b < num_blocks; };
    constexpr int kBatch = 8;
    for (int64_t i0 = tid; i0 < num_pairs; i0 += kBatch * kCopyThreads) {
        int32_t s[kBatch], d[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int64_t i = i0 + k * kCopyThreads;
            s[k] = i < num_pairs ? __ldg(src + i) : -1;
            d[k] = i < num_pairs ? __ldg(dst + i) : -1;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (inside(s[k]) && inside(d[k])) {
                const uint32_t bit = 1u << (d[k] & 31);
                if (s[k] != d[k] && (atomicOr(&once[d[k] >> 5], bit) & bit) != 0u) atomicOr(&twice[d[k] >> 5], bit);
            } else if (blockIdx.x == 0 && s[k] != -1 && d[k] != -1) {
                flag(status, KVFP8_DEV_BAD_BLOCK);
            }
        }
    }
    __syncthreads();
    const int32_t segs = m.seg0[m.caches.count];
    const int64_t total = static_cast<int64_t>(num_pairs) * segs;
    // consecutive segments go to consecutive CTAs: a few blocks occupy every SM
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kCopyThreads / 32);
    for (int64_t it = blockIdx.x + static_cast<int64_t>(gridDim.x) * (tid >> 5); it < total; it += step) {
        const int64_t p = it / segs;
        const int32_t x = static_cast<int32_t>(it - p * segs);
        const int32_t s = __ldg(src + p), d = __ldg(dst + p);
        if (!inside(s) || !inside(d) || s == d) continue;
        if (((once[s >> 5] >> (s & 31)) | (twice[d >> 5] >> (d & 31))) & 1u) {
            if (x == 0 && lane == 0) flag(status, KVFP8_DEV_BAD_BLOCK);
            continue;
        }
        copy_segment<kWide>(m, x, s, d, lane);
    }
}

// ---------------------------------------------------------------- compaction
//
// The kernels of a call are chained as programmatic dependent launches: each grid is launched while
// its predecessor runs and waits for it.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Workspace: one bit per block (used), the exclusive count of used blocks before each word of
// it, the moves' sources and destinations in ascending order, and {U, moves}.
struct CompactWorkspace {
    size_t used, before, from, to, counts, total;
};

CompactWorkspace compact_layout(int32_t num_blocks) {
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    const size_t words = (static_cast<size_t>(num_blocks) + 31) / 32;
    CompactWorkspace w;
    w.used = 0;
    w.before = w.used + up(4 * words);
    w.from = w.before + up(4 * words);
    w.to = w.from + up(4 * (static_cast<size_t>(num_blocks) / 2 + 1));
    w.counts = w.to + up(4 * (static_cast<size_t>(num_blocks) / 2 + 1));
    w.total = w.counts + 256;
    return w;
}

struct CompactArgs {
    int32_t num_blocks, block_size, max_blocks_per_seq, num_seqs;
    const int32_t *tables;
    int32_t *new_tables;
    const int32_t *seq_lens;
    int32_t *num_used;
    uint32_t *used;
    int32_t *before, *from, *to, *counts;
    uint32_t *status;
};

// table entries of sequence s that hold tokens
__device__ __forceinline__ int32_t live_entries(const CompactArgs &a, int32_t s) {
    const int64_t most = static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size;
    const int64_t L = min(max(static_cast<int64_t>(a.seq_lens[s]), int64_t{0}), most);
    return static_cast<int32_t>((L + a.block_size - 1) / a.block_size);
}

// One bit per used block; errors are flagged here.  CTAs stride over the sequences (x) and
// their entries (y).
__global__ void __launch_bounds__(256) mark_kernel(const CompactArgs a) {
    pdl_trigger();
    for (int32_t s = blockIdx.x; s < a.num_seqs; s += gridDim.x) {
        const int32_t n = live_entries(a, s);
        if (blockIdx.y == 0 && threadIdx.x == 0 &&
            (a.seq_lens[s] < 0 ||
             a.seq_lens[s] > static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size))
            flag(a.status, KVFP8_DEV_BAD_BLOCK);
        const int32_t *row = a.tables + static_cast<int64_t>(s) * a.max_blocks_per_seq;
        for (int32_t e = blockIdx.y * 256 + threadIdx.x; e < n; e += gridDim.y * 256) {
            const int32_t b = row[e];
            if (b >= 0 && b < a.num_blocks)
                atomicOr(&a.used[b >> 5], 1u << (b & 31));
            else
                flag(a.status, KVFP8_DEV_BAD_BLOCK);
        }
    }
}

// sum over the CTA's 1024 threads, to all of them
__device__ __forceinline__ int32_t block_sum(int32_t v, int32_t *scratch) {
    v = __reduce_add_sync(0xFFFFFFFFu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_add_sync(0xFFFFFFFFu, scratch[threadIdx.x & 31]);
}

// The moves of word w of the bitmap, rank used blocks before it: every used id >= U is a source,
// every free id below U a destination, each in ascending order.  Returns the rank after the word.
__device__ __forceinline__ int32_t list_moves(const CompactArgs &a, int32_t w, uint32_t bits, int32_t rank,
                                              int32_t U, int32_t R) {
    const int32_t id0 = w * 32;
    if (id0 + 32 <= U) {  // holes only
        for (uint32_t f = ~bits; f != 0u; f &= f - 1u) {
            const int i = __ffs(f) - 1;
            a.to[id0 + i - rank - __popc(bits & ((1u << i) - 1u))] = id0 + i;
        }
        return rank + __popc(bits);
    }
    for (int i = 0; i < 32; ++i) {
        const int32_t id = id0 + i;
        if (id >= a.num_blocks) break;
        const bool is_used = (bits >> i) & 1u;
        if (is_used && id >= U) a.from[rank - R] = id;
        if (!is_used && id < U) a.to[id - rank] = id;
        rank += is_used;
    }
    return rank;
}
__device__ __forceinline__ void write_counts(const CompactArgs &a, int32_t U, int32_t R) {
    a.counts[0] = U;
    a.counts[1] = U - R;  // moves
    a.counts[2] = R;
    *a.num_used = U;
}

// Each CTA takes 1024 words of the bitmap.  It counts the used blocks of the whole pool (U), of
// the ids below U (R) and of the words before its own by reading the bitmap (a few KB per 32768
// blocks, from L2), then gives every used id >= U its move: source rank(id) - R, destination the
// free id below U of that rank.
__global__ void __launch_bounds__(1024) plan_moves_kernel(const CompactArgs a) {
    __shared__ int32_t scratch[32];
    pdl_trigger();
    pdl_wait();  // every mark is made
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t words = (a.num_blocks + 31) >> 5, w0 = blockIdx.x * 1024;
    int32_t all = 0, mine = 0;
    for (int32_t w = tid; w < words; w += 1024) {
        const int32_t c = __popc(a.used[w]);
        all += c;
        if (w < w0) mine += c;
    }
    const int32_t U = block_sum(all, scratch);
    const int32_t before_cta = block_sum(mine, scratch);
    int32_t low = 0;
    for (int32_t w = tid; w < words && w * 32 < U; w += 1024)
        low += __popc(a.used[w] & (U - w * 32 >= 32 ? ~0u : (1u << (U - w * 32)) - 1u));
    const int32_t R = block_sum(low, scratch);
    // exclusive count before this thread's word
    const int32_t w = w0 + tid;
    const uint32_t bits = w < words ? a.used[w] : 0u;
    const int32_t c = __popc(bits);
    int32_t x = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    int32_t tot = scratch[lane];
    const int32_t pre_warps = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? tot : 0);
    const int32_t before = before_cta + pre_warps + x - c;
    if (w < words) {
        a.before[w] = before;
        list_moves(a, w, bits, before, U, R);
    }
    if (blockIdx.x == 0 && tid == 0) write_counts(a, U, R);
}

// The same plan by one CTA with the bitmap in shared memory, for small pools and tables: one launch
// in the place of a memset and two kernels (33 sequences of up to 500 tokens: 10.3 against 12.4 us a
// call; 128 of up to 4096, 32768 entries: 160 against 153 us, so not for those).
constexpr int32_t kOneCtaBlocks = 32 * 1024, kOneCtaEntries = 16 * 1024;

__global__ void __launch_bounds__(1024) plan_one_cta_kernel(const CompactArgs a) {
    pdl_trigger();
    __shared__ uint32_t bits[kOneCtaBlocks / 32];
    __shared__ int32_t scratch[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t words = (a.num_blocks + 31) >> 5;
    for (int32_t w = tid; w < words; w += 1024) bits[w] = 0u;
    __syncthreads();
    // all entries in order, eight of a thread in flight; those past a sequence's length do not count
    const int32_t total = a.num_seqs * a.max_blocks_per_seq;
    constexpr int kBatch = 8;
    for (int32_t i0 = tid; i0 < total; i0 += kBatch * 1024) {
        int32_t b[kBatch], n[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int32_t i = i0 + k * 1024;
            b[k] = i < total ? a.tables[i] : 0;
            const int32_t s = i < total ? i / a.max_blocks_per_seq : 0;
            // entry e holds tokens when e * block_size < the length (no division by the block size)
            const int64_t first = static_cast<int64_t>(i - s * a.max_blocks_per_seq) * a.block_size;
            n[k] = i < total && first < a.seq_lens[s] ? 1 : 0;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (n[k] == 0) continue;
            if (b[k] >= 0 && b[k] < a.num_blocks)
                atomicOr(&bits[b[k] >> 5], 1u << (b[k] & 31));
            else
                flag(a.status, KVFP8_DEV_BAD_BLOCK);
        }
    }
    for (int32_t s = tid; s < a.num_seqs; s += 1024)
        if (a.seq_lens[s] < 0 || a.seq_lens[s] > static_cast<int64_t>(a.max_blocks_per_seq) * a.block_size)
            flag(a.status, KVFP8_DEV_BAD_BLOCK);
    __syncthreads();
    // a thread has per consecutive words
    const int32_t per = (words + 1023) / 1024, w0 = tid * per;
    int32_t mine = 0;
    for (int32_t w = w0; w < min(w0 + per, words); ++w) mine += __popc(bits[w]);
    const int32_t U = block_sum(mine, scratch);
    int32_t low = 0;
    for (int32_t w = w0; w < min(w0 + per, words) && w * 32 < U; ++w)
        low += __popc(bits[w] & (U - w * 32 >= 32 ? ~0u : (1u << (U - w * 32)) - 1u));
    const int32_t R = block_sum(low, scratch);
    int32_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    const int32_t tot = scratch[lane];
    int32_t rank = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? tot : 0) + x - mine;
    for (int32_t w = w0; w < min(w0 + per, words); ++w) {
        a.used[w] = bits[w];
        a.before[w] = rank;
        rank = list_moves(a, w, bits[w], rank, U, R);
    }
    if (tid == 0) write_counts(a, U, R);
}

// New tables, and the moves: no source is a destination (sources are >= U, destinations below).
template <bool kWide>
__global__ void __launch_bounds__(kThreads)
move_blocks_kernel(const __grid_constant__ SegMap m, const CompactArgs a) {
    pdl_wait();  // the plan is visible from here on
    const int32_t U = a.counts[0], moves = a.counts[1], R = a.counts[2];
    for (int32_t s = blockIdx.x; s < a.num_seqs; s += gridDim.x) {
        const int32_t n = live_entries(a, s);
        const int64_t row = static_cast<int64_t>(s) * a.max_blocks_per_seq;
        for (int32_t e = threadIdx.x; e < a.max_blocks_per_seq; e += kThreads) {
            int32_t b = e < n ? a.tables[row + e] : -1;
            if (b < 0 || b >= a.num_blocks) {
                b = -1;
            } else if (b >= U) {
                const int32_t rank = a.before[b >> 5] + __popc(a.used[b >> 5] & ((1u << (b & 31)) - 1u));
                b = a.to[rank - R];
            }
            a.new_tables[row + e] = b;
        }
    }
    const int32_t segs = m.seg0[m.caches.count];
    const int64_t total = static_cast<int64_t>(moves) * segs;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < total; it += step) {
        const int64_t p = it / segs;
        copy_segment<kWide>(m, static_cast<int32_t>(it - p * segs), a.from[p], a.to[p], threadIdx.x & 31);
    }
}

// ---------------------------------------------------------------- host side

bool wide_ok(const CacheList &c) {
    for (int i = 0; i < c.count; ++i)
        if ((reinterpret_cast<uintptr_t>(c.ptr[i]) & 31u) != 0 || c.block_bytes[i] % 32 != 0) return false;
    return true;
}

// Segments of 4 KiB when there are enough of them to give every resident warp a few, 1 KiB
// otherwise (a few blocks then spread over four times the warps).  False when a block has too
// many segments.
bool make_segments(const CacheList &c, int64_t pairs, int sms, SegMap *m) {
    m->caches = c;
    int64_t bytes = 0;
    for (int i = 0; i < c.count; ++i) bytes += c.block_bytes[i];
    m->seg_bytes = pairs >= static_cast<int64_t>(sms) * 64 / std::max<int64_t>(1, bytes / 4096) ? 4096 : 1024;
    int64_t at = 0;
    for (int i = 0; i < c.count; ++i) {
        m->seg0[i] = static_cast<int32_t>(at);
        at += (c.block_bytes[i] + m->seg_bytes - 1) / m->seg_bytes;
        if (at > 0x7FFFFFFFLL) return false;
    }
    m->seg0[c.count] = static_cast<int32_t>(at);
    return true;
}

}  // namespace

cudaError_t launch_copy_blocks(const CacheList &caches, int32_t num_blocks, const int32_t *src,
                               const int32_t *dst, int32_t num_pairs, uint32_t *status,
                               cudaStream_t stream) {
    DeviceFacts f;
    cudaError_t err = device_facts(&f);
    if (err != cudaSuccess) return err;
    if (num_blocks > KVFP8_MAX_COPY_BLOCKS) return cudaErrorNotSupported;
    const size_t smem = 8 * ((static_cast<size_t>(num_blocks) + 31) / 32);  // the two bitmaps
    if (smem > static_cast<size_t>(f.smem_optin)) return cudaErrorNotSupported;
    SegMap m;
    if (!make_segments(caches, num_pairs, f.sms, &m)) return cudaErrorNotSupported;
    auto kern = wide_ok(caches) ? copy_blocks_kernel<true> : copy_blocks_kernel<false>;
    int occ = 0;
    if ((err = kernel_occupancy(kern, kCopyThreads, smem, &occ)) != cudaSuccess) return err;
    const int64_t items = static_cast<int64_t>(num_pairs) * m.seg0[caches.count];
    const int grid = static_cast<int>(std::min<int64_t>(items, static_cast<int64_t>(f.sms) * std::max(occ, 1)));
    kern<<<grid, kCopyThreads, smem, stream>>>(m, num_blocks, src, dst, num_pairs, status);
    return cudaGetLastError();
}

size_t compact_workspace_size(int32_t num_blocks) { return compact_layout(num_blocks).total; }

cudaError_t launch_compact_blocks(const CacheList &caches, int32_t num_blocks, int32_t block_size,
                                  const int32_t *block_tables, int32_t max_blocks_per_seq,
                                  const int32_t *seq_lens, int32_t num_seqs,
                                  int32_t *new_block_tables, int32_t *num_used, void *workspace,
                                  uint32_t *status, cudaStream_t stream) {
    DeviceFacts f;
    cudaError_t err = device_facts(&f);
    if (err != cudaSuccess) return err;
    SegMap m;
    // the number of moves is known on the device only: at most half the pool
    if (!make_segments(caches, num_blocks / 2, f.sms, &m)) return cudaErrorNotSupported;
    const CompactWorkspace w = compact_layout(num_blocks);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    CompactArgs a;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.num_seqs = num_seqs;
    a.tables = block_tables;
    a.new_tables = new_block_tables;
    a.seq_lens = seq_lens;
    a.num_used = num_used;
    a.used = reinterpret_cast<uint32_t *>(ws + w.used);
    a.before = reinterpret_cast<int32_t *>(ws + w.before);
    a.from = reinterpret_cast<int32_t *>(ws + w.from);
    a.to = reinterpret_cast<int32_t *>(ws + w.to);
    a.counts = reinterpret_cast<int32_t *>(ws + w.counts);
    a.status = status;
    const int32_t words = (num_blocks + 31) / 32;
    const bool one_cta = num_blocks <= kOneCtaBlocks &&
                         static_cast<int64_t>(num_seqs) * max_blocks_per_seq <= kOneCtaEntries;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    if (one_cta) {
        plan_one_cta_kernel<<<1, 1024, 0, stream>>>(a);
    } else {
        if ((err = cudaMemsetAsync(a.used, 0, 4 * static_cast<size_t>(words), stream)) != cudaSuccess) return err;
        if (num_seqs > 0) {
            const dim3 grid(std::min(num_seqs, 4096), std::min((max_blocks_per_seq + 255) / 256, 64));
            mark_kernel<<<grid, 256, 0, stream>>>(a);
            if ((err = cudaGetLastError()) != cudaSuccess) return err;
        }
        cfg.gridDim = dim3((words + 1023) / 1024);
        cfg.blockDim = dim3(1024);
        cfg.numAttrs = num_seqs > 0 ? 1 : 0;  // (only a kernel of this call may be overtaken)
        err = cudaLaunchKernelEx(&cfg, plan_moves_kernel, a);
    }
    if (err != cudaSuccess || (err = cudaGetLastError()) != cudaSuccess) return err;
    auto kern = wide_ok(caches) ? move_blocks_kernel<true> : move_blocks_kernel<false>;
    int occ = 0;
    if ((err = kernel_occupancy(kern, kThreads, 0, &occ)) != cudaSuccess) return err;
    cfg.gridDim = dim3(f.sms * std::max(occ, 1));
    cfg.blockDim = dim3(kThreads);
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, m, a);
}

}  // namespace kvfp8
