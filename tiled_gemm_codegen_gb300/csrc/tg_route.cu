// Tokens sorted by expert and back: the stable counting sort of routing ids,
// the copy of token rows into expert order, the weighted sum of expert rows
// back into token order, and that sum's gradient.  Entry points and formulas:
// include/tg_gemm.h.
//
// All of it moves bytes (two flops a value): the bound is HBM for batches
// and launch latency for a few tokens.  Offsets of rows are 64-bit.
// Bandwidths below are the bytes a call cannot do without over its time, and
// their fraction of a plain copy's 6685 GB/s on the same GPU.
//
// The sort is a counting sort by expert, stable because an id's place is
//     offsets[e] + (ids of e in earlier blocks) + (in earlier warps of the
//     block) + (in earlier lanes and turns of the warp),
// with no atomic whose order shows.  How the counts reach everyone depends on
// their number: up to 1024 ids every block counts them all (64 ids: 1.9 us,
// 1000 x 5: 3.6), up to 16384 a cluster of eight blocks exchanges counts
// through distributed shared memory (5000 ids: 3.7 us), beyond that three launches over all SMs
// (32768: 7.1, 131072: 8.9, 262144: 12.4).  Latency bounds all three: the
// ids themselves are 1 MB at most there.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tg_gemm.h"
#include "tg_host_api.h"
#include "tg_ptx.cuh"

#define TG_API extern "C" __attribute__((visibility("default")))

namespace tg {
namespace {

constexpr int MAX_EXPERTS = 1024;
constexpr int SORT_BATCH = 4;                 // ids a thread ranks at once
constexpr int ONE_THREADS = 256;              // a block that ranks every id of a call
constexpr int ONE_IDS = ONE_THREADS * SORT_BATCH;
constexpr int PLACE_THREADS = 128;            // a block of the three-launch sort
constexpr int PLACE_IDS = PLACE_THREADS * SORT_BATCH;
constexpr int MAX_SORT_BLOCKS = 4096;         // columns of the count matrix

// The ids of one call and where its order goes.
struct SortArgs {
    const void *ids;
    int ids64;       // 8-byte ids
    int64_t ld_ids;
    int32_t n;       // T * k
    int32_t k, E;
    int32_t *offsets, *source, *slot;
    int32_t *counts;   // [E][blocks]: a block's ids of each expert, then those of the blocks before it
    int32_t *totals;   // [E]
    int32_t epad;      // E rounded up to 4
    int32_t blocks;    // blocks of the count and place kernels
    int32_t per_block; // ids of a block
};

// Rows copied into expert order, in bytes.
struct CopyArgs {
    const uint8_t *x;
    uint8_t *xs;
    int64_t ld_x, ld_xs;  // bytes
    int64_t row_bytes;
    int32_t T, k, E;
    const int32_t *offsets, *slot;
    int32_t chunks;       // 16-byte chunks a row can touch
};

// The expert of flat assignment f, or -1 (dropped: outside [0, E)).
__device__ __forceinline__ int32_t load_id(const SortArgs &a, int32_t f)
{
    int64_t at = f;
    if (a.ld_ids != a.k) at = static_cast<int64_t>(f / a.k) * a.ld_ids + f % a.k;
    if (a.ids64) {
        const int64_t v = static_cast<const int64_t *>(a.ids)[at];
        return v >= 0 && v < a.E ? static_cast<int32_t>(v) : -1;
    }
    const int32_t v = static_cast<const int32_t *>(a.ids)[at];
    return v >= 0 && v < a.E ? v : -1;
}

// Ranks of up to THREADS * SORT_BATCH ids inside their experts, in the order
// of the ids.  Warp w holds ids [w * seg, (w + 1) * seg), 32 consecutive ones
// at a time: an id's rank is the number of equal ids in lower lanes
// (match.any) plus the warp's count so far.  On return hist[w][e] is warp
// w's count.
struct Ranked {
    int32_t id[SORT_BATCH];
    int32_t rank[SORT_BATCH];
};

// Ids of a warp's segment: 32 times what the block's threads need each.
template <int THREADS>
__device__ __forceinline__ int32_t segment(int32_t n)
{
    return (n + THREADS - 1) / THREADS * 32;
}

template <int THREADS>
__device__ __forceinline__ void rank_ids(const SortArgs &a, int32_t base, int32_t n, int32_t *hist, Ranked &r)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t seg = segment<THREADS>(n);
#pragma unroll
    for (int b = 0; b < SORT_BATCH; ++b) {
        const int32_t i = warp * seg + b * 32 + lane;
        r.id[b] = (b * 32 < seg && i < n) ? load_id(a, base + i) : -1;
    }
    for (int i = threadIdx.x; i < THREADS / 32 * a.epad; i += THREADS) hist[i] = 0;
    __syncthreads();
    int32_t *mine = hist + warp * a.epad;
#pragma unroll
    for (int b = 0; b < SORT_BATCH; ++b) {
        if (b * 32 >= seg) break;
        const uint32_t peers = __match_any_sync(0xffffffffu, r.id[b]);
        const uint32_t before = peers & ((1u << lane) - 1u);
        const int32_t seen = r.id[b] >= 0 ? mine[r.id[b]] : 0;
        r.rank[b] = seen + __popc(before);
        __syncwarp();
        if (r.id[b] >= 0 && before == 0) mine[r.id[b]] = seen + __popc(peers);
        __syncwarp();
    }
    __syncthreads();
}

// hist[w][e] -> the count of the warps before w; returns expert e's total.
template <int WARPS>
__device__ __forceinline__ int32_t scan_warps(int32_t *hist, int32_t epad, int32_t e)
{
    int32_t v[WARPS], sum = 0;  // all loads before the first store: one latency, not WARPS of them
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v[w] = hist[w * epad + e];
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        hist[w * epad + e] = sum;
        sum += v[w];
    }
    return sum;
}

// Exclusive scan of v[0 .. E) in shared memory, in place; v[E] = the sum.
// Thread t owns PER consecutive entries.
template <int THREADS>
__device__ __forceinline__ void scan_experts(int32_t *v, int32_t E, int32_t *warp_sums)
{
    constexpr int PER = MAX_EXPERTS / THREADS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e0 = static_cast<int>(threadIdx.x) * PER;
    int32_t x[PER], mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        x[i] = e0 + i < E ? v[e0 + i] : 0;
        mine += x[i];
    }
    int32_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t t = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += t;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int32_t at = lane < warp ? warp_sums[lane] : 0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) at += __shfl_xor_sync(0xffffffffu, at, d);
    at += incl - mine;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (e0 + i <= E) v[e0 + i] = at;
        at += x[i];
    }
    if (E == MAX_EXPERTS && threadIdx.x == THREADS - 1) v[E] = at;  // otherwise the owner of entry E wrote it
    __syncthreads();
}

// How many ids of each expert a block's share holds.
__global__ void __launch_bounds__(PLACE_THREADS) sort_count_kernel(const SortArgs a)
{
    __shared__ int32_t hist[MAX_EXPERTS];
    for (int i = threadIdx.x; i < a.E; i += PLACE_THREADS) hist[i] = 0;
    __syncthreads();
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.per_block;
    const int64_t hi = lo + a.per_block < a.n ? lo + a.per_block : a.n;
#pragma unroll 4
    for (int64_t f = lo + threadIdx.x; f < hi; f += PLACE_THREADS) {
        const int32_t e = load_id(a, static_cast<int32_t>(f));
        if (e >= 0) atomicAdd(&hist[e], 1);  // integers: the order does not show
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.E; i += PLACE_THREADS) a.counts[static_cast<int64_t>(i) * a.blocks + blockIdx.x] = hist[i];
}

// A warp per expert: its counts become the sums of the blocks before.
__global__ void __launch_bounds__(128) sort_scan_kernel(const SortArgs a)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int32_t e = static_cast<int32_t>(blockIdx.x) * 4 + static_cast<int32_t>(threadIdx.x >> 5);
    if (e >= a.E) return;
    int32_t *row = a.counts + static_cast<int64_t>(e) * a.blocks;
    int32_t sum = 0;
    for (int32_t b0 = 0; b0 < a.blocks; b0 += 128) {
        int32_t v[4], mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t b = b0 + lane * 4 + i;
            v[i] = b < a.blocks ? __ldcg(row + b) : 0;
            mine += v[i];
        }
        int32_t incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t t = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += t;
        }
        int32_t at = sum + incl - mine;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t b = b0 + lane * 4 + i;
            if (b < a.blocks) row[b] = at;
            at += v[i];
        }
        sum += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) a.totals[e] = sum;
}

// Shared memory of a ranking block, hist[warps][epad] behind it.
struct SortSmem {
    int32_t base[MAX_EXPERTS + 4];   // next slot of each expert
    int32_t warp_sums[32];
};

// ------------------------------------------------------------ row copies
// The 16 bytes at p (any multiple of 2), which lie inside [lo, hi): one
// aligned load, or two and a shift; element by element where the aligned
// 16-byte words around them leave the span.
__device__ __forceinline__ uint4 load16_any(const uint8_t *p, const uint8_t *lo, const uint8_t *hi)
{
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
    if (off == 0) return *reinterpret_cast<const uint4 *>(p);
    const uint8_t *a = p - off;
    if (a >= lo && a + 32 <= hi) {
        const uint4 u = *reinterpret_cast<const uint4 *>(a);
        const uint4 v = *reinterpret_cast<const uint4 *>(a + 16);
        uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        if (off & 8u) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (off & 4u) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
        const uint32_t sh = (off & 2u) * 8u;
        return make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh),
                          __funnelshift_r(w[2], w[3], sh), __funnelshift_r(w[3], w[4], sh));
    }
    const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = static_cast<uint32_t>(h[2 * i]) | (static_cast<uint32_t>(h[2 * i + 1]) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One 16-byte-aligned chunk c of row `dst`, copied from row `src`.
__device__ __forceinline__ void copy_chunk(uint8_t *dst, const uint8_t *src, int64_t row_bytes, int64_t c,
                                           const uint8_t *lo, const uint8_t *hi)
{
    const int64_t mis = static_cast<int64_t>(reinterpret_cast<uintptr_t>(dst) & 15u);
    const int64_t b0 = c * 16 - mis;
    if (b0 >= 0 && b0 + 16 <= row_bytes) {
        *reinterpret_cast<uint4 *>(dst + b0) =
            src ? load16_any(src + b0, lo, hi) : make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const int64_t e0 = b0 > 0 ? b0 : 0, e1 = b0 + 16 < row_bytes ? b0 + 16 : row_bytes;
    for (int64_t b = e0; b < e1; b += 2)
        *reinterpret_cast<uint16_t *>(dst + b) = src ? *reinterpret_cast<const uint16_t *>(src + b) : uint16_t(0);
}

// x rows -> expert order, all rows 16-byte aligned multiples of 16 bytes: a
// thread reads 16 bytes of a token once and writes them to its k slots.
// Block (32 >> shift tokens per warp) x 8 warps; grid.y: segments of a row.
// Bound by HBM's writes (k times the reads), so a token's reads are not
// repeated for its k slots: 16384 tokens of 2048 bf16, k 8, 604 MB: 90.5 us,
// 6.67 TB/s (100%).  Copying inside the sort's last launch instead, so that it
// starts a launch earlier, made dispatch 118 us instead of 106: a block's
// copies then wait for its own ranks.
__global__ void __launch_bounds__(256) gather_aligned_kernel(const CopyArgs a, int shift)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * 8 + warp) * (32 >> shift) + (lane >> shift);
    const int64_t c = (static_cast<int64_t>(blockIdx.y) << shift) + (lane & ((1 << shift) - 1));
    const int64_t n = static_cast<int64_t>(a.T) * a.k;
    if (t < a.T && c < a.chunks) {
        const uint4 v = *reinterpret_cast<const uint4 *>(a.x + t * a.ld_x + c * 16);
        const int32_t *slot = a.slot + t * a.k;
#pragma unroll 4
        for (int j = 0; j < a.k; ++j) {
            const int32_t s = slot[j];
            if (s >= 0 && s < n) *reinterpret_cast<uint4 *>(a.xs + s * a.ld_xs + c * 16) = v;
        }
    }
    // rows behind the last expert: zeros
    const int64_t kept = max(0, a.offsets[a.E]);
    if (kept >= n) return;
    const int64_t tid = ((static_cast<int64_t>(blockIdx.y) * gridDim.x) + blockIdx.x) * 256 + threadIdx.x;
    const int64_t threads = static_cast<int64_t>(gridDim.x) * gridDim.y * 256;
    for (int64_t i = tid; i < (n - kept) * a.chunks; i += threads)
        *reinterpret_cast<uint4 *>(a.xs + (kept + i / a.chunks) * a.ld_xs + (i % a.chunks) * 16) =
            make_uint4(0u, 0u, 0u, 0u);
}

// The same for rows of any pitch and alignment: a thread writes one aligned
// 16-byte chunk of one slot's row, read through load16_any.  (A token's k
// slots lie differently to the 16-byte grid, so a read serves one of them; the
// others find it in L2.)
__global__ void __launch_bounds__(256) gather_any_kernel(const CopyArgs a, int shift)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t f = (static_cast<int64_t>(blockIdx.x) * 8 + warp) * (32 >> shift) + (lane >> shift);
    const int64_t c = (static_cast<int64_t>(blockIdx.y) << shift) + (lane & ((1 << shift) - 1));
    const int64_t n = static_cast<int64_t>(a.T) * a.k;
    const uint8_t *hi = a.x + (a.T - 1) * a.ld_x + a.row_bytes;
    if (f < n && c < a.chunks) {
        const int32_t s = a.slot[f];
        if (s >= 0 && s < n) copy_chunk(a.xs + s * a.ld_xs, a.x + (f / a.k) * a.ld_x, a.row_bytes, c, a.x, hi);
    }
    const int64_t kept = max(0, a.offsets[a.E]);
    if (kept >= n) return;
    const int64_t tid = ((static_cast<int64_t>(blockIdx.y) * gridDim.x) + blockIdx.x) * 256 + threadIdx.x;
    const int64_t threads = static_cast<int64_t>(gridDim.x) * gridDim.y * 256;
    for (int64_t i = tid; i < (n - kept) * a.chunks; i += threads)
        copy_chunk(a.xs + (kept + i / a.chunks) * a.ld_xs, nullptr, a.row_bytes, i % a.chunks, a.x, hi);
}

// The slots of a block's ids, PLACE_IDS at a time; the experts' starting slots
// come from the scan.
__global__ void __launch_bounds__(PLACE_THREADS) sort_place_kernel(const SortArgs a)
{
    __shared__ __align__(16) SortSmem sm;
    extern __shared__ int32_t hist[];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    for (int e = threadIdx.x; e < a.E; e += PLACE_THREADS) sm.base[e] = __ldcg(a.totals + e);
    __syncthreads();
    scan_experts<PLACE_THREADS>(sm.base, a.E, sm.warp_sums);
    const int32_t kept = sm.base[a.E];
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= a.E; e += PLACE_THREADS) a.offsets[e] = sm.base[e];
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += PLACE_THREADS)
        sm.base[e] += __ldcg(a.counts + static_cast<int64_t>(e) * a.blocks + blockIdx.x);
    // slots past the last kept assignment hold nothing
    for (int64_t s = kept + static_cast<int64_t>(blockIdx.x) * PLACE_THREADS + threadIdx.x; s < a.n;
         s += static_cast<int64_t>(gridDim.x) * PLACE_THREADS)
        a.source[s] = -1;
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.per_block;
    const int64_t hi = lo + a.per_block < a.n ? lo + a.per_block : a.n;
    constexpr int WARPS = PLACE_THREADS / 32;
    for (int64_t at = lo; at < hi; at += PLACE_IDS) {
        const int32_t n = static_cast<int32_t>(hi - at < PLACE_IDS ? hi - at : PLACE_IDS);
        Ranked r;
        rank_ids<PLACE_THREADS>(a, static_cast<int32_t>(at), n, hist, r);
        int32_t total[MAX_EXPERTS / PLACE_THREADS];
#pragma unroll
        for (int i = 0; i < MAX_EXPERTS / PLACE_THREADS; ++i) {
            const int e = static_cast<int>(threadIdx.x) + i * PLACE_THREADS;
            if (e < a.E) total[i] = scan_warps<WARPS>(hist, a.epad, e);
        }
        __syncthreads();
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int32_t seg = segment<PLACE_THREADS>(n);
#pragma unroll
        for (int b = 0; b < SORT_BATCH; ++b) {
            const int32_t i = warp * seg + b * 32 + lane;
            if (b * 32 >= seg || i >= n) continue;
            const int32_t f = static_cast<int32_t>(at) + i;
            int32_t s = -1;
            if (r.id[b] >= 0) {
                s = sm.base[r.id[b]] + hist[warp * a.epad + r.id[b]] + r.rank[b];
                a.source[s] = f;
            }
            a.slot[f] = s;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MAX_EXPERTS / PLACE_THREADS; ++i) {
            const int e = static_cast<int>(threadIdx.x) + i * PLACE_THREADS;
            if (e < a.E) sm.base[e] += total[i];
        }
        __syncthreads();
    }
}

// Up to CLUSTER_IDS ids in one launch: a cluster of CLUSTER blocks, each
// ranking CLUSTER_THREADS * SORT_BATCH of them.  Every block's counts by
// expert lie in its shared memory, where the others read them: the experts'
// offsets from all, the place of a block's own ids from the blocks before it.
constexpr int CLUSTER = 8;
constexpr int CLUSTER_THREADS = 512;
constexpr int CLUSTER_IDS = CLUSTER * CLUSTER_THREADS * SORT_BATCH;

__global__ void __launch_bounds__(CLUSTER_THREADS) sort_cluster_kernel(const SortArgs a)
{
    __shared__ __align__(16) SortSmem sm;
    __shared__ int32_t mine[MAX_EXPERTS];  // this block's counts
    extern __shared__ int32_t hist[];
    constexpr int WARPS = CLUSTER_THREADS / 32, EACH = MAX_EXPERTS / CLUSTER_THREADS;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int32_t rank = static_cast<int32_t>(ptx::cluster_ctarank());
    const int32_t share = (a.n + CLUSTER - 1) / CLUSTER;
    const int32_t lo = min(a.n, rank * share), n = min(a.n - lo, share);
    Ranked r;
    rank_ids<CLUSTER_THREADS>(a, lo, n, hist, r);
    for (int e = threadIdx.x; e < a.E; e += CLUSTER_THREADS) mine[e] = scan_warps<WARPS>(hist, a.epad, e);
    ptx::cluster_sync_all();
    int32_t before[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int e = static_cast<int>(threadIdx.x) + i * CLUSTER_THREADS;
        before[i] = 0;
        if (e >= a.E) continue;
        int32_t all = 0;
        const uint32_t at = ptx::smem_addr(mine + e);
#pragma unroll
        for (int32_t c = 0; c < CLUSTER; ++c) {
            const int32_t v = static_cast<int32_t>(ptx::ld_cluster_u32(ptx::map_to_cta(at, static_cast<uint32_t>(c))));
            all += v;
            if (c < rank) before[i] += v;
        }
        sm.base[e] = all;
    }
    ptx::cluster_sync_all();  // no block leaves while another still reads its counts
    scan_experts<CLUSTER_THREADS>(sm.base, a.E, sm.warp_sums);
    const int32_t kept = sm.base[a.E];
    if (rank == 0)
        for (int e = threadIdx.x; e <= a.E; e += CLUSTER_THREADS) a.offsets[e] = sm.base[e];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int e = static_cast<int>(threadIdx.x) + i * CLUSTER_THREADS;
        if (e < a.E) sm.base[e] += before[i];
    }
    __syncthreads();
    for (int32_t s = kept + rank * CLUSTER_THREADS + static_cast<int32_t>(threadIdx.x); s < a.n; s += CLUSTER * CLUSTER_THREADS)
        a.source[s] = -1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t seg = segment<CLUSTER_THREADS>(n);
#pragma unroll
    for (int b = 0; b < SORT_BATCH; ++b) {
        const int32_t i = warp * seg + b * 32 + lane;
        if (b * 32 >= seg || i >= n) continue;
        int32_t s = -1;
        if (r.id[b] >= 0) {
            s = sm.base[r.id[b]] + hist[warp * a.epad + r.id[b]] + r.rank[b];
            a.source[s] = lo + i;
        }
        a.slot[lo + i] = s;
    }
}

// The whole dispatch of at most ONE_IDS assignments in one launch: every
// block ranks all ids itself (they are few, and no block then waits for
// another), block 0 writes the order, and the blocks share the row copies.
// With c.x null only the order is written.  Bound by latency: one token of
// 2048 bf16 onto 8 of 64 experts, 2.7 us on the GPU.
__global__ void __launch_bounds__(ONE_THREADS) dispatch_one_kernel(const SortArgs a, const CopyArgs c)
{
    constexpr int THREADS = ONE_THREADS;
    __shared__ __align__(16) SortSmem sm;
    __shared__ int32_t source[THREADS * SORT_BATCH];
    extern __shared__ int32_t hist[];
    constexpr int WARPS = THREADS / 32;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    Ranked r;
    for (int i = threadIdx.x; i < a.n; i += THREADS) source[i] = -1;
    rank_ids<THREADS>(a, 0, a.n, hist, r);
    for (int e = threadIdx.x; e < a.E; e += THREADS) sm.base[e] = scan_warps<WARPS>(hist, a.epad, e);
    __syncthreads();
    scan_experts<THREADS>(sm.base, a.E, sm.warp_sums);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t seg = segment<THREADS>(a.n);
    const bool writes = blockIdx.x == 0;
#pragma unroll
    for (int b = 0; b < SORT_BATCH; ++b) {
        const int32_t f = warp * seg + b * 32 + lane;
        if (b * 32 >= seg || f >= a.n) continue;
        int32_t s = -1;
        if (r.id[b] >= 0) {
            s = sm.base[r.id[b]] + hist[warp * a.epad + r.id[b]] + r.rank[b];
            source[s] = f;
        }
        if (writes) a.slot[f] = s;
    }
    __syncthreads();
    if (writes) {
        for (int e = threadIdx.x; e <= a.E; e += THREADS) a.offsets[e] = sm.base[e];
        for (int i = threadIdx.x; i < a.n; i += THREADS) a.source[i] = source[i];
    }
    if (!c.x) return;
    const uint8_t *hi = c.x + (c.T - 1) * c.ld_x + c.row_bytes;
    // sorted rows in turn: a block's threads cover whole rows
    const int64_t first = static_cast<int64_t>(blockIdx.x) * THREADS + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x) * THREADS;
    int64_t s = first / c.chunks;
    int32_t ch = static_cast<int32_t>(first % c.chunks);
    const int64_t ds = step / c.chunks;
    const int32_t dch = static_cast<int32_t>(step % c.chunks);
#pragma unroll 2
    while (s < a.n) {
        const int32_t f = source[s];
        copy_chunk(c.xs + s * c.ld_xs, f >= 0 ? c.x + static_cast<int64_t>(f / a.k) * c.ld_x : nullptr, c.row_bytes, ch, c.x, hi);
        s += ds;
        ch += dch;
        if (ch >= c.chunks) {
            ch -= c.chunks;
            ++s;
        }
    }
}

// ------------------------------------------------------------ combine
struct CombineArgs {
    const void *ys;   // [S, D], ys_bf16 or fp32
    void *y;          // [T, D]
    int64_t ld_ys, ld_y;  // elements
    int64_t S, D;
    int32_t ys_bf16, y_bf16;
    const int32_t *slot;
    const float *weights;  // null: ones
    int64_t ld_w;
    int32_t T, k;
    int32_t chunks;  // 8-element chunks a row of y can touch
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <bool BF16>
__device__ __forceinline__ void store8_aligned(void *row, int64_t e0, const float (&f)[8])
{
    if constexpr (BF16) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(row) + e0) =
            make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    } else {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(row) + e0);
        p[0] = make_float4(f[0], f[1], f[2], f[3]);
        p[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// Elements [e0, e0 + 8) of a row of D at any alignment (elements outside
// [0, D) read as 0); [lo, hi) is the span of all rows.
__device__ __forceinline__ void load8_any(const void *row, bool bf16, int64_t e0, int64_t D, const uint8_t *lo,
                                          const uint8_t *hi, float (&f)[8])
{
    if (bf16) {
        const uint16_t *p = static_cast<const uint16_t *>(row);
        if (e0 >= 0 && e0 + 8 <= D) {
            unpack8(load16_any(reinterpret_cast<const uint8_t *>(p + e0), lo, hi), f);
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = e0 + i >= 0 && e0 + i < D ? __uint_as_float(static_cast<uint32_t>(p[e0 + i]) << 16) : 0.0f;
    } else {
        const float *p = static_cast<const float *>(row);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = e0 + i >= 0 && e0 + i < D ? p[e0 + i] : 0.0f;
    }
}

__device__ __forceinline__ void store8_any(void *row, bool bf16, int64_t e0, int64_t D, const float (&f)[8])
{
    if (bf16) {
        uint16_t *p = static_cast<uint16_t *>(row);
        if (e0 >= 0 && e0 + 8 <= D && (reinterpret_cast<uintptr_t>(p + e0) & 15u) == 0) {
            store8_aligned<true>(row, e0, f);
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e0 + i >= 0 && e0 + i < D) p[e0 + i] = __bfloat16_as_ushort(__float2bfloat16_rn(f[i]));
    } else {
        float *p = static_cast<float *>(row);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e0 + i >= 0 && e0 + i < D) p[e0 + i] = f[i];
    }
}

__device__ __forceinline__ const uint8_t *row_of(const void *base, int64_t row, int64_t ld, bool bf16)
{
    return static_cast<const uint8_t *>(base) + row * ld * (bf16 ? 2 : 4);
}

// Elements of `row` before its first 16-byte boundary, counted back: chunk c
// of the row covers elements [8c - lead, 8c - lead + 8).
__device__ __forceinline__ int64_t lead_of(const void *row, bool bf16)
{
    return bf16 ? static_cast<int64_t>((reinterpret_cast<uintptr_t>(row) & 15u) >> 1) : 0;
}

template <bool BF16>
struct Raw8;  // eight elements as loaded
template <>
struct Raw8<true> {
    uint4 v;
    __device__ __forceinline__ void load(const void *row, int64_t e0)
    {
        v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + e0));
    }
    __device__ __forceinline__ void get(float (&f)[8]) const { unpack8(v, f); }
};
template <>
struct Raw8<false> {
    float4 u, v;
    __device__ __forceinline__ void load(const void *row, int64_t e0)
    {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(row) + e0);
        u = __ldg(p);
        v = __ldg(p + 1);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w; f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
    }
};

// y[t] = sum_j w[t, j] ys[slot[t, j]], in the order of j, in fp32, rounded
// once.  A thread owns 8 elements of a token: KB rows' loads in flight, which
// is what keeps HBM busy at 48 registers and half the SM's warps.  16384
// tokens of 4096 bf16, k 4, 661 MB: 103 us, 6.42 TB/s (96%); five tokens of
// 1001: 2.5 us on the GPU.
template <bool YS_BF16, bool Y_BF16, int KB>
__global__ void __launch_bounds__(256) combine_aligned_kernel(const CombineArgs a, int shift)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * 8 + warp) * (32 >> shift) + (lane >> shift);
    const int64_t c = (static_cast<int64_t>(blockIdx.y) << shift) + (lane & ((1 << shift) - 1));
    if (t >= a.T || c >= a.chunks) return;
    const int32_t *slot = a.slot + t * a.k;
    const float *w = a.weights ? a.weights + t * a.ld_w : nullptr;
    float acc[8] = {};
    for (int j0 = 0; j0 < a.k; j0 += KB) {
        Raw8<YS_BF16> v[KB];
        uint32_t on = 0;
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const int32_t s = j0 + j < a.k ? __ldg(slot + j0 + j) : -1;
            if (s >= 0 && s < a.S) {
                on |= 1u << j;
                v[j].load(row_of(a.ys, s, a.ld_ys, YS_BF16), c * 8);
            }
        }
#pragma unroll
        for (int j = 0; j < KB; ++j)
            if (on >> j & 1u) {  // a dropped assignment adds nothing, whatever its weight
                const float wj = w ? __ldg(w + j0 + j) : 1.0f;
                float f[8];
                v[j].get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = fmaf(wj, f[i], acc[i]);
            }
    }
    store8_aligned<Y_BF16>(const_cast<uint8_t *>(row_of(a.y, t, a.ld_y, Y_BF16)), c * 8, acc);
}

// The same for any type, pitch and alignment, one row at a time.
__global__ void __launch_bounds__(256) combine_any_kernel(const CombineArgs a, int shift)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * 8 + warp) * (32 >> shift) + (lane >> shift);
    const int64_t c = (static_cast<int64_t>(blockIdx.y) << shift) + (lane & ((1 << shift) - 1));
    if (t >= a.T || c >= a.chunks) return;
    const int32_t *slot = a.slot + t * a.k;
    const float *w = a.weights ? a.weights + t * a.ld_w : nullptr;
    uint8_t *out = const_cast<uint8_t *>(row_of(a.y, t, a.ld_y, a.y_bf16));
    const int64_t e0 = c * 8 - lead_of(out, a.y_bf16);
    if (e0 >= a.D) return;
    const uint8_t *lo = static_cast<const uint8_t *>(a.ys);
    const uint8_t *hi = row_of(a.ys, a.S - 1, a.ld_ys, a.ys_bf16) + a.D * (a.ys_bf16 ? 2 : 4);
    float acc[8] = {};
#pragma unroll 2
    for (int j = 0; j < a.k; ++j) {
        const int32_t s = slot[j];
        if (s < 0 || s >= a.S) continue;
        float v[8];
        load8_any(row_of(a.ys, s, a.ld_ys, a.ys_bf16), a.ys_bf16, e0, a.D, lo, hi, v);
        const float wj = w ? w[j] : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(wj, v[i], acc[i]);
    }
    store8_any(out, a.y_bf16, e0, a.D, acc);
}

// ------------------------------------------------------------ gradient
struct GradArgs {
    const void *dy;  // [T, D]
    const void *ys;  // [S, D]
    void *dys;       // [S, D]
    float *dw;       // [T, k]
    int64_t ld_dy, ld_ys, ld_dys, ld_dw;
    int64_t S, D;
    int32_t dy_bf16, ys_bf16, dys_bf16;
    const int32_t *offsets, *slot;
    const float *weights;
    int64_t ld_w;
    int32_t T, k, E;
    int32_t chunks;
};

// Rows of dys behind the last expert: zeros (no assignment reads them).
__device__ __forceinline__ void zero_tail(const GradArgs &a)
{
    const int64_t kept = max(0, a.offsets[a.E]);
    if (kept >= a.S) return;
    const float zero[8] = {};
    for (int64_t s = kept + blockIdx.x; s < a.S; s += gridDim.x) {
        uint8_t *row = const_cast<uint8_t *>(row_of(a.dys, s, a.ld_dys, a.dys_bf16));
        const int64_t lead = lead_of(row, a.dys_bf16);
        for (int64_t c = threadIdx.x; c * 8 - lead < a.D; c += blockDim.x)
            store8_any(row, a.dys_bf16, c * 8 - lead, a.D, zero);
    }
}

// Sums of KB values over the block; thread 0 .. KB-1 return theirs.
template <int KB>
__device__ __forceinline__ float block_sums(float (&v)[KB], float (*part)[KB])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int j = 0; j < KB; ++j)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v[j] += __shfl_xor_sync(0xffffffffu, v[j], d);
    if (lane == 0) {
#pragma unroll
        for (int j = 0; j < KB; ++j) part[warp][j] = v[j];
    }
    __syncthreads();
    float sum = 0.0f;
    if (threadIdx.x < KB)
        for (int w = 0; w < warps; ++w) sum += part[w][threadIdx.x];
    __syncthreads();
    return sum;
}

// One block a token: dys[slot[t, j]] = w[t, j] dy[t] and
// dw[t, j] = <dy[t], ys[slot[t, j]]>.  dy is read once for KB assignments,
// whose rows of ys are loaded four at a time; all bf16 and 16-byte rows.  The
// dot products are summed lane by lane, warp by warp, in a fixed order.  Reads
// and writes share HBM about evenly, which costs it more than either alone:
// 8191 tokens of 2056, k 8, 568 MB: 99.5 us, 5.70 TB/s (85%); the kernel
// itself moves 520 MB, as dys partly stays in L2.
template <int KB>
__global__ void __launch_bounds__(512) combine_grad_aligned_kernel(const GradArgs a)
{
    constexpr int LB = KB < 4 ? KB : 4;
    __shared__ float part[16][KB];
    __shared__ int32_t s[KB];
    __shared__ float w[KB];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t t = blockIdx.x;
    const uint16_t *dy = static_cast<const uint16_t *>(a.dy) + t * a.ld_dy;
    for (int j0 = 0; j0 < a.k; j0 += KB) {
        if (threadIdx.x < KB) {
            const int j = j0 + static_cast<int>(threadIdx.x);
            const int32_t v = j < a.k ? a.slot[t * a.k + j] : -1;
            s[threadIdx.x] = v < a.S ? v : -1;
            w[threadIdx.x] = j < a.k && a.weights ? a.weights[t * a.ld_w + j] : 1.0f;
        }
        __syncthreads();
        float dot[KB] = {};
        for (int32_t c = threadIdx.x; c < a.chunks; c += static_cast<int32_t>(blockDim.x)) {
            float g[8];
            Raw8<true> d;
            d.load(dy, c * 8);
            uint4 raw[LB];
#pragma unroll
            for (int jb = 0; jb < KB; jb += LB) {
                if (a.dw) {
#pragma unroll
                    for (int j = 0; j < LB; ++j)
                        if (s[jb + j] >= 0)
                            raw[j] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.ys) +
                                                                           s[jb + j] * a.ld_ys + c * 8));
                }
                if (jb == 0) d.get(g);
#pragma unroll
                for (int j = 0; j < LB; ++j) {
                    if (s[jb + j] < 0) continue;
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = w[jb + j] * g[i];
                    store8_aligned<true>(static_cast<uint16_t *>(a.dys) + s[jb + j] * a.ld_dys, c * 8, o);
                    if (a.dw) {
                        float v[8];
                        unpack8(raw[j], v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dot[jb + j] = fmaf(g[i], v[i], dot[jb + j]);
                    }
                }
            }
        }
        if (a.dw) {
            const float sum = block_sums<KB>(dot, part);
            if (threadIdx.x < KB && j0 + threadIdx.x < a.k) a.dw[t * a.ld_dw + j0 + threadIdx.x] = sum;
        }
        if (j0 + KB < a.k) __syncthreads();  // s and w are written again
    }
    zero_tail(a);
}

// The same with a warp a token, for short rows (a block a token would be mostly
// its own start and barriers): 30946 tokens of 64 values, k 1: 32 -> 10.5 us.
constexpr int GRAD_WARP_CHUNKS = 64;

template <int KB>
__global__ void __launch_bounds__(256) combine_grad_warp_kernel(const GradArgs a)
{
    constexpr int LB = KB < 4 ? KB : 4;
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (t < a.T) {
        const uint16_t *dy = static_cast<const uint16_t *>(a.dy) + t * a.ld_dy;
        for (int j0 = 0; j0 < a.k; j0 += KB) {
            int32_t sl = -1;
            float wl = 1.0f;
            if (lane < KB && j0 + lane < a.k) {
                sl = a.slot[t * a.k + j0 + lane];
                if (sl >= a.S) sl = -1;
                if (a.weights) wl = a.weights[t * a.ld_w + j0 + lane];
            }
            int32_t s[KB];
            float w[KB], dot[KB];
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                s[j] = __shfl_sync(0xffffffffu, sl, j);
                w[j] = __shfl_sync(0xffffffffu, wl, j);
                dot[j] = 0.0f;
            }
            for (int32_t c = lane; c < a.chunks; c += 32) {
                float g[8];
                Raw8<true> d;
                d.load(dy, c * 8);
                uint4 raw[LB];
#pragma unroll
                for (int jb = 0; jb < KB; jb += LB) {
                    if (a.dw) {
#pragma unroll
                        for (int j = 0; j < LB; ++j)
                            if (s[jb + j] >= 0)
                                raw[j] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.ys) +
                                                                               s[jb + j] * a.ld_ys + c * 8));
                    }
                    if (jb == 0) d.get(g);
#pragma unroll
                    for (int j = 0; j < LB; ++j) {
                        if (s[jb + j] < 0) continue;
                        float o[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = w[jb + j] * g[i];
                        store8_aligned<true>(static_cast<uint16_t *>(a.dys) + s[jb + j] * a.ld_dys, c * 8, o);
                        if (a.dw) {
                            float v[8];
                            unpack8(raw[j], v);
#pragma unroll
                            for (int i = 0; i < 8; ++i) dot[jb + j] = fmaf(g[i], v[i], dot[jb + j]);
                        }
                    }
                }
            }
            if (a.dw) {
                float mine = 0.0f;
#pragma unroll
                for (int j = 0; j < KB; ++j) {
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
                    if (lane == j) mine = dot[j];
                }
                if (lane < KB && j0 + lane < a.k) a.dw[t * a.ld_dw + j0 + lane] = mine;
            }
        }
    }
    zero_tail(a);
}

// The same for any type, pitch and alignment: one row of dys at a time, by a
// warp (short rows) or a block.
template <bool WARP>
__global__ void __launch_bounds__(512) combine_grad_any_kernel(const GradArgs a)
{
    __shared__ float part[16][1];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int64_t t = WARP ? static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t first = WARP ? threadIdx.x & 31 : threadIdx.x, step = WARP ? 32 : blockDim.x;
    if (t < a.T) {
        const uint8_t *dy = row_of(a.dy, t, a.ld_dy, a.dy_bf16);
        const uint8_t *dy_lo = static_cast<const uint8_t *>(a.dy);
        const uint8_t *dy_hi = row_of(a.dy, a.T - 1, a.ld_dy, a.dy_bf16) + a.D * (a.dy_bf16 ? 2 : 4);
        const uint8_t *ys_lo = static_cast<const uint8_t *>(a.ys);
        const uint8_t *ys_hi = a.ys ? row_of(a.ys, a.S - 1, a.ld_ys, a.ys_bf16) + a.D * (a.ys_bf16 ? 2 : 4) : nullptr;
        for (int j = 0; j < a.k; ++j) {
            const int32_t s = a.slot[t * a.k + j];
            float dot[1] = {0.0f};
            if (s >= 0 && s < a.S) {
                const float w = a.weights ? a.weights[t * a.ld_w + j] : 1.0f;
                uint8_t *out = const_cast<uint8_t *>(row_of(a.dys, s, a.ld_dys, a.dys_bf16));
                const int64_t lead = lead_of(out, a.dys_bf16);
                for (int64_t c = first; c * 8 - lead < a.D; c += step) {
                    const int64_t e0 = c * 8 - lead;
                    float g[8], o[8];
                    load8_any(dy, a.dy_bf16, e0, a.D, dy_lo, dy_hi, g);
                    if (a.dw) {
                        float v[8];
                        load8_any(row_of(a.ys, s, a.ld_ys, a.ys_bf16), a.ys_bf16, e0, a.D, ys_lo, ys_hi, v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dot[0] = fmaf(g[i], v[i], dot[0]);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = w * g[i];
                    store8_any(out, a.dys_bf16, e0, a.D, o);
                }
            }
            if (a.dw) {
                if constexpr (WARP) {
                    __syncwarp();
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], d);
                    if (first == 0) a.dw[t * a.ld_dw + j] = dot[0];
                } else {
                    const float sum = block_sums<1>(dot, part);
                    if (threadIdx.x == 0) a.dw[t * a.ld_dw + j] = sum;
                }
            }
        }
    }
    zero_tail(a);
}

// ------------------------------------------------------------ host
template <class... P, class... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster, A... args)
{
    // Programmatic dependent launch: the kernel waits (griddepcontrol.wait)
    // before its first access to memory another kernel may write.
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// The shared-memory opt-in of a kernel, once per device (under the host
// mutex).
template <auto KERN>
cudaError_t opt_in(int dev, int bytes)
{
    static uint64_t configured = 0;
    if (dev < 64 && ((configured >> dev) & 1u)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) configured |= 1ull << dev;
    return e;
}

constexpr int64_t ROW_LIMIT = 1 << 22;            // elements of a row (segments fit grid.y)
constexpr int64_t PITCH_LIMIT = int64_t(1) << 40;

bool mult16(const void *p, int64_t pitch_bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && pitch_bytes % 16 == 0;
}

// log2 of the lanes that share a row of `chunks` chunks: 8, 16 or 32, the
// fewest idle (a warp takes 4, 2 or 1 rows); 32 for long rows, whose last
// segment is a small part.
int lanes_shift(int64_t chunks)
{
    int best = 5;
    if (chunks > 1024) return best;
    for (int s = 5; s >= 3; --s) {
        const int64_t used = (chunks + (1 << s) - 1) >> s << s;
        const int64_t have = (chunks + (1 << best) - 1) >> best << best;
        if (used < have) best = s;
    }
    return best;
}

struct Span {
    uintptr_t lo = 0, hi = 0;
};

Span span_of(const void *p, int64_t rows, int64_t ld, int64_t cols, int64_t bytes)
{
    if (!p || rows <= 0 || cols <= 0) return {};
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return {b, b + static_cast<uintptr_t>(((rows - 1) * ld + cols) * bytes)};
}

bool meets(const Span &a, const Span &b) { return a.lo < b.hi && b.lo < a.hi; }

bool counts_ok(int64_t T, int64_t k, int64_t E)
{
    return T >= 0 && k >= 1 && E >= 1 && k <= INT32_MAX && T <= INT32_MAX && E <= INT32_MAX && T * k <= INT32_MAX;
}

bool row_ok(const void *p, int64_t rows, int64_t ld, int64_t cols, int64_t bytes)
{
    if (rows == 0 || cols == 0) return true;
    return p != nullptr && ld >= cols && ld <= PITCH_LIMIT &&
           reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0;
}

CopyArgs copy_args(const void *x, int64_t ld_x, int64_t D, int32_t eb, void *xs, int64_t ld_xs, int64_t T, int64_t k,
                   int64_t E, const int32_t *offsets, const int32_t *slot, bool *aligned)
{
    CopyArgs c{};
    c.x = static_cast<const uint8_t *>(x);
    c.xs = static_cast<uint8_t *>(xs);
    c.ld_x = ld_x * eb;
    c.ld_xs = ld_xs * eb;
    c.row_bytes = D * eb;
    c.T = static_cast<int32_t>(T);
    c.k = static_cast<int32_t>(k);
    c.E = static_cast<int32_t>(E);
    c.offsets = offsets;
    c.slot = slot;
    *aligned = mult16(x, c.ld_x) && mult16(xs, c.ld_xs) && c.row_bytes % 16 == 0;
    c.chunks = static_cast<int32_t>(*aligned ? c.row_bytes / 16 : (c.row_bytes + 14 + 15) / 16);
    return c;
}

cudaError_t launch_gather(const CopyArgs &c, bool aligned, cudaStream_t s)
{
    const int sh = lanes_shift(c.chunks);
    const int64_t rows = aligned ? c.T : static_cast<int64_t>(c.T) * c.k;
    const int64_t per_block = 8 * (32 >> sh);
    const dim3 grid(static_cast<unsigned>((rows + per_block - 1) / per_block),
                    static_cast<unsigned>((c.chunks + (1 << sh) - 1) >> sh));
    return aligned ? launch(gather_aligned_kernel, grid, 256, 0, s, 1, c, sh) : launch(gather_any_kernel, grid, 256, 0, s, 1, c, sh);
}

// The sort (and, with x, the copy of the rows into expert order).
tg_status run_sort(const void *ids, int32_t id_bytes, int64_t ld_ids, int64_t T, int64_t k, int64_t E, int32_t *offsets,
                   int32_t *source, int32_t *slot, const void *x, int64_t ld_x, int64_t D, int32_t eb, void *xs,
                   int64_t ld_xs, cudaStream_t stream)
{
    if (!counts_ok(T, k, E) || (id_bytes != 4 && id_bytes != 8) || !offsets || !host_words_ok(offsets, source, slot))
        return TG_ERR_INVALID_ARG;
    const int64_t n = T * k;
    if (n > 0 && (!ids || !source || !slot || ld_ids < k || ld_ids > PITCH_LIMIT ||
                  reinterpret_cast<uintptr_t>(ids) % static_cast<uintptr_t>(id_bytes) != 0))
        return TG_ERR_INVALID_ARG;
    const bool copies = n > 0 && D > 0;
    if (D < 0 || (eb != 2 && eb != 4)) return TG_ERR_INVALID_ARG;
    if (copies && (!row_ok(x, T, ld_x, D, eb) || !row_ok(xs, n, ld_xs, D, eb))) return TG_ERR_INVALID_ARG;
    const Span in[2] = {span_of(ids, T, ld_ids, k, id_bytes), copies ? span_of(x, T, ld_x, D, eb) : Span{}};
    const Span out[4] = {span_of(offsets, 1, 0, E + 1, 4), span_of(source, 1, 0, n, 4), span_of(slot, 1, 0, n, 4),
                         copies ? span_of(xs, n, ld_xs, D, eb) : Span{}};
    for (int i = 0; i < 4; ++i) {
        for (const Span &r : in)
            if (meets(out[i], r)) return TG_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (meets(out[i], out[j])) return TG_ERR_INVALID_ARG;
    }
    if (E > MAX_EXPERTS || D > ROW_LIMIT) return TG_ERR_UNSUPPORTED;

    std::lock_guard<std::mutex> lock(host_mutex());
    HostStream hs;
    tg_status st = host_stream(stream, &hs);
    if (st != TG_OK) return st;
    SortArgs a{};
    a.ids = ids;
    a.ids64 = id_bytes == 8;
    a.ld_ids = ld_ids;
    a.n = static_cast<int32_t>(n);
    a.k = static_cast<int32_t>(k);
    a.E = static_cast<int32_t>(E);
    a.offsets = offsets;
    a.source = source;
    a.slot = slot;
    a.epad = static_cast<int32_t>((E + 3) / 4 * 4);
    bool aligned = false;
    CopyArgs c{};
    if (copies) c = copy_args(x, ld_x, D, eb, xs, ld_xs, T, k, E, offsets, slot, &aligned);
    const size_t warp_hist = static_cast<size_t>(a.epad) * 4;
    // Up to ONE_IDS assignments one launch does everything (1024 of 64
    // experts: 3.7 us, sorted by a cluster and copied by a second launch 5.8;
    // blocks of 1024 threads for 4096 of them take 7.7, the cluster 3.7).
    if (n <= ONE_IDS) {
        int64_t blocks = 1;
        if (copies) blocks = (n * c.chunks + ONE_THREADS - 1) / ONE_THREADS;
        if (blocks > 4 * hs.sms) blocks = 4 * hs.sms;
        return host_cuda_status(launch(dispatch_one_kernel, dim3(static_cast<unsigned>(blocks)), ONE_THREADS,
                                       ONE_THREADS / 32 * warp_hist, stream, 1, a, c));
    }
    // Up to CLUSTER_IDS one cluster sorts (5000 ids: 3.7 us); beyond, three
    // launches over all SMs: count, scan and place (32768: 7.1, 262144: 12.3).
    cudaError_t e;
    if (n <= CLUSTER_IDS) {
        constexpr int WARPS = CLUSTER_THREADS / 32;
        e = opt_in<sort_cluster_kernel>(hs.dev, WARPS * MAX_EXPERTS * 4);
        if (e == cudaSuccess)
            e = launch(sort_cluster_kernel, dim3(CLUSTER), CLUSTER_THREADS, WARPS * warp_hist, stream, CLUSTER, a);
    } else {
        a.per_block = PLACE_IDS;
        const int64_t least = (n + MAX_SORT_BLOCKS - 1) / MAX_SORT_BLOCKS;
        if (a.per_block < least) a.per_block = static_cast<int32_t>((least + PLACE_IDS - 1) / PLACE_IDS * PLACE_IDS);
        a.blocks = static_cast<int32_t>((n + a.per_block - 1) / a.per_block);
        void *arena = nullptr;
        st = host_arena(hs, (static_cast<size_t>(a.blocks) + 1) * a.E * 4, &arena);
        if (st != TG_OK) return st;
        a.counts = static_cast<int32_t *>(arena);
        a.totals = a.counts + static_cast<int64_t>(a.blocks) * a.E;
        const dim3 grid(static_cast<unsigned>(a.blocks));
        e = launch(sort_count_kernel, grid, PLACE_THREADS, 0, stream, 1, a);
        if (e == cudaSuccess) e = launch(sort_scan_kernel, dim3(static_cast<unsigned>((E + 3) / 4)), 128, 0, stream, 1, a);
        if (e == cudaSuccess) e = launch(sort_place_kernel, grid, PLACE_THREADS, PLACE_THREADS / 32 * warp_hist, stream, 1, a);
    }
    if (e == cudaSuccess && copies) e = launch_gather(c, aligned, stream);
    return host_cuda_status(e);
}

bool dtype_ok(int32_t t) { return t == TG_F32 || t == TG_BF16; }
int64_t dtype_bytes(int32_t t) { return t == TG_BF16 ? 2 : 4; }

template <bool YS_BF16, bool Y_BF16>
cudaError_t launch_combine(const CombineArgs &a, dim3 grid, int sh, cudaStream_t s)
{
    if (a.k <= 2) return launch(combine_aligned_kernel<YS_BF16, Y_BF16, 2>, grid, 256, 0, s, 1, a, sh);
    if (a.k <= 4) return launch(combine_aligned_kernel<YS_BF16, Y_BF16, 4>, grid, 256, 0, s, 1, a, sh);
    return launch(combine_aligned_kernel<YS_BF16, Y_BF16, 8>, grid, 256, 0, s, 1, a, sh);
}

}  // namespace
}  // namespace tg

using namespace tg;

TG_API tg_status tg_expert_sort(const void *ids, int32_t id_bytes, int64_t ld_ids, int64_t T, int64_t k, int64_t E,
                                int32_t *offsets, int32_t *source, int32_t *slot, tg_stream_t stream)
{
    return host_guard([&] {
        return run_sort(ids, id_bytes, ld_ids, T, k, E, offsets, source, slot, nullptr, 0, 0, 2, nullptr, 0,
                        reinterpret_cast<cudaStream_t>(stream));
    });
}

TG_API tg_status tg_expert_dispatch(const void *ids, int32_t id_bytes, int64_t ld_ids, int64_t T, int64_t k, int64_t E,
                                    int32_t *offsets, int32_t *source, int32_t *slot, const void *x, int64_t ld_x,
                                    int64_t D, int32_t dtype, void *xs, int64_t ld_xs, tg_stream_t stream)
{
    return host_guard([&] {
        if (!dtype_ok(dtype)) return TG_ERR_INVALID_ARG;
        return run_sort(ids, id_bytes, ld_ids, T, k, E, offsets, source, slot, x, ld_x, D,
                        static_cast<int32_t>(dtype_bytes(dtype)), xs, ld_xs, reinterpret_cast<cudaStream_t>(stream));
    });
}

TG_API tg_status tg_expert_gather(const void *x, int64_t ld_x, int64_t D, int32_t dtype, int64_t T, int64_t k, int64_t E,
                                  const int32_t *offsets, const int32_t *slot, void *xs, int64_t ld_xs,
                                  tg_stream_t stream)
{
    return host_guard([&] {
        if (!counts_ok(T, k, E) || D < 0 || !dtype_ok(dtype)) return TG_ERR_INVALID_ARG;
        const int64_t n = T * k, eb = dtype_bytes(dtype);
        if (n == 0 || D == 0) return TG_OK;
        if (!offsets || !slot || !host_words_ok(offsets, slot) || !row_ok(x, T, ld_x, D, eb) || !row_ok(xs, n, ld_xs, D, eb))
            return TG_ERR_INVALID_ARG;
        const Span out = span_of(xs, n, ld_xs, D, eb);
        if (meets(out, span_of(x, T, ld_x, D, eb)) || meets(out, span_of(offsets, 1, 0, E + 1, 4)) ||
            meets(out, span_of(slot, 1, 0, n, 4)))
            return TG_ERR_INVALID_ARG;
        if (D > ROW_LIMIT) return TG_ERR_UNSUPPORTED;
        bool aligned = false;
        const CopyArgs c = copy_args(x, ld_x, D, static_cast<int32_t>(eb), xs, ld_xs, T, k, E, offsets, slot, &aligned);
        return host_cuda_status(launch_gather(c, aligned, reinterpret_cast<cudaStream_t>(stream)));
    });
}

TG_API tg_status tg_expert_combine(const void *ys, int64_t ld_ys, int32_t ys_type, int64_t S, const int32_t *slot,
                                   const float *weights, int64_t ld_w, int64_t T, int64_t k, int64_t D, void *y,
                                   int64_t ld_y, int32_t y_type, tg_stream_t stream_)
{
    return host_guard([&] {
        cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
        if (!counts_ok(T, k, 1) || S < 0 || S > INT32_MAX || D < 0 || !dtype_ok(ys_type) || !dtype_ok(y_type))
            return TG_ERR_INVALID_ARG;
        if (T == 0 || D == 0) return TG_OK;
        const int64_t yb = dtype_bytes(y_type), ysb = dtype_bytes(ys_type);
        if (!slot || !host_words_ok(slot, weights) || !row_ok(ys, S, ld_ys, D, ysb) || !row_ok(y, T, ld_y, D, yb) || (weights && ld_w < k) ||
            (weights && ld_w > PITCH_LIMIT))
            return TG_ERR_INVALID_ARG;
        const Span out = span_of(y, T, ld_y, D, yb);
        if (meets(out, span_of(ys, S, ld_ys, D, ysb)) || meets(out, span_of(slot, 1, 0, T * k, 4)) ||
            meets(out, span_of(weights, T, ld_w, k, 4)))
            return TG_ERR_INVALID_ARG;
        if (D > ROW_LIMIT) return TG_ERR_UNSUPPORTED;
        CombineArgs a{};
        a.ys = ys;
        a.y = y;
        a.ld_ys = ld_ys;
        a.ld_y = ld_y;
        a.S = S;
        a.D = D;
        a.ys_bf16 = ys_type == TG_BF16;
        a.y_bf16 = y_type == TG_BF16;
        a.slot = slot;
        a.weights = weights;
        a.ld_w = ld_w;
        a.T = static_cast<int32_t>(T);
        a.k = static_cast<int32_t>(k);
        const bool aligned = D % 8 == 0 && mult16(ys, ld_ys * ysb) && mult16(y, ld_y * yb);
        a.chunks = static_cast<int32_t>(aligned ? D / 8 : (D + 7 + 7) / 8);
        const int sh = lanes_shift(a.chunks);
        const int64_t per_block = 8 * (32 >> sh);
        const dim3 grid(static_cast<unsigned>((T + per_block - 1) / per_block),
                        static_cast<unsigned>((a.chunks + (1 << sh) - 1) >> sh));
        cudaError_t e;
        if (!aligned)
            e = launch(combine_any_kernel, grid, 256, 0, stream, 1, a, sh);
        else if (a.ys_bf16)
            e = a.y_bf16 ? launch_combine<true, true>(a, grid, sh, stream) : launch_combine<true, false>(a, grid, sh, stream);
        else
            e = a.y_bf16 ? launch_combine<false, true>(a, grid, sh, stream) : launch_combine<false, false>(a, grid, sh, stream);
        return host_cuda_status(e);
    });
}

TG_API tg_status tg_expert_combine_grad(const void *dy, int64_t ld_dy, int32_t dy_type, const void *ys, int64_t ld_ys,
                                        int32_t ys_type, const int32_t *offsets, const int32_t *slot,
                                        const float *weights, int64_t ld_w, int64_t T, int64_t k, int64_t E, int64_t D,
                                        void *dys, int64_t ld_dys, int32_t dys_type, float *dweights, int64_t ld_dw,
                                        tg_stream_t stream_)
{
    return host_guard([&] {
        cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
        if (!counts_ok(T, k, E) || D < 0 || !dtype_ok(dy_type) || !dtype_ok(ys_type) || !dtype_ok(dys_type))
            return TG_ERR_INVALID_ARG;
        const int64_t n = T * k;
        if (n == 0) return TG_OK;
        const int64_t b_dy = dtype_bytes(dy_type), b_ys = dtype_bytes(ys_type), b_dys = dtype_bytes(dys_type);
        if (!offsets || !slot || !host_words_ok(offsets, slot, weights, dweights) || !row_ok(dy, T, ld_dy, D, b_dy) || !row_ok(dys, n, ld_dys, D, b_dys) ||
            (dweights && !row_ok(ys, n, ld_ys, D, b_ys)) || (weights && (ld_w < k || ld_w > PITCH_LIMIT)) ||
            (dweights && (ld_dw < k || ld_dw > PITCH_LIMIT)))
            return TG_ERR_INVALID_ARG;
        const Span in[5] = {span_of(dy, T, ld_dy, D, b_dy), dweights ? span_of(ys, n, ld_ys, D, b_ys) : Span{},
                            span_of(slot, 1, 0, n, 4), span_of(offsets, 1, 0, E + 1, 4), span_of(weights, T, ld_w, k, 4)};
        const Span o1 = span_of(dys, n, ld_dys, D, b_dys), o2 = span_of(dweights, T, ld_dw, k, 4);
        if (meets(o1, o2)) return TG_ERR_INVALID_ARG;
        for (const Span &r : in)
            if (meets(o1, r) || meets(o2, r)) return TG_ERR_INVALID_ARG;
        if (D > ROW_LIMIT) return TG_ERR_UNSUPPORTED;
        GradArgs a{};
        a.dy = dy;
        a.ys = dweights ? ys : nullptr;
        a.dys = dys;
        a.dw = dweights;
        a.ld_dy = ld_dy;
        a.ld_ys = ld_ys;
        a.ld_dys = ld_dys;
        a.ld_dw = ld_dw;
        a.S = n;
        a.D = D;
        a.dy_bf16 = dy_type == TG_BF16;
        a.ys_bf16 = ys_type == TG_BF16;
        a.dys_bf16 = dys_type == TG_BF16;
        a.offsets = offsets;
        a.slot = slot;
        a.weights = weights;
        a.ld_w = ld_w;
        a.T = static_cast<int32_t>(T);
        a.k = static_cast<int32_t>(k);
        a.E = static_cast<int32_t>(E);
        const bool aligned = a.dy_bf16 && a.dys_bf16 && (!dweights || a.ys_bf16) && D % 8 == 0 &&
                             mult16(dy, ld_dy * 2) && mult16(dys, ld_dys * 2) && (!dweights || mult16(ys, ld_ys * 2));
        a.chunks = static_cast<int32_t>(aligned ? D / 8 : (D + 7 + 7) / 8);
        // one turn of the block's threads over a row where 512 of them
        // suffice, else turns of 256
        int threads = a.chunks <= 512 ? static_cast<int>((a.chunks + 31) / 32 * 32) : 256;
        if (threads < 32) threads = 32;
        const dim3 grid(static_cast<unsigned>(T)), warps(static_cast<unsigned>((T + 7) / 8));
        const bool narrow = a.chunks <= GRAD_WARP_CHUNKS;
        cudaError_t e;
        if (!aligned)
            e = narrow ? launch(combine_grad_any_kernel<true>, warps, 256, 0, stream, 1, a)
                       : launch(combine_grad_any_kernel<false>, grid, threads, 0, stream, 1, a);
        else if (k <= 2)
            e = narrow ? launch(combine_grad_warp_kernel<2>, warps, 256, 0, stream, 1, a)
                       : launch(combine_grad_aligned_kernel<2>, grid, threads, 0, stream, 1, a);
        else if (k <= 4)
            e = narrow ? launch(combine_grad_warp_kernel<4>, warps, 256, 0, stream, 1, a)
                       : launch(combine_grad_aligned_kernel<4>, grid, threads, 0, stream, 1, a);
        else
            e = narrow ? launch(combine_grad_warp_kernel<8>, warps, 256, 0, stream, 1, a)
                       : launch(combine_grad_aligned_kernel<8>, grid, threads, 0, stream, 1, a);
        return host_cuda_status(e);
    });
}
