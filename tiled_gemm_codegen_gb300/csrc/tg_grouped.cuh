// Persistent, warp-specialised grouped GEMM for sm_103a: one product per
// group of consecutive rows, the groups' bounds on the device.
//
//   rows mode    D[s][:] = act(alpha * A[s][:] B[g] + bias[g]) for the rows s of group g: the rows
//                are ragged.  The tile is computed transposed - the columns of B[g] are the
//                MMA's M (256 or 128 of them), the rows of A its N - because N is a field
//                of each instruction: a group's last tile takes as many rows as are left,
//                rounded up to 32, where an M of 256 would compute 128 rows of padding a
//                group on average (uneven groups of 1024 rows, 2048 x 4096: an eighth
//                of the work).  A tile's box of A may start at any row; rows past the
//                group's end are loaded but never stored (a row of D depends on its
//                own row of A alone).
//   wgrad mode   D[g] = alpha * A[rows g]^T B[rows g]: the contraction is ragged.  Both operands
//                are read as stored (MN-major), 64 rows a k-block; the rows past the
//                group's end in its last k-block (its fringe) belong to the next
//                group, so a fixer warp overwrites them with zeros in shared memory
//                before the MMA may read them (in both operands: 0 x NaN is NaN).
//                A fringe's copies complete on the slot's fringe barrier, on which
//                only the fixer waits; it then arrives on the slot's full barrier
//                in the producer's place, so the MMA's own wait is one and the same.
//
// Roles, rings and the bounded waits are those of gemm_kernel (tg_kernel.cuh):
// warp 0 loads, warp 1 issues tcgen05.mma, warps 2..9 drain tensor memory;
// wgrad mode adds warp 10, the fixer, which runs as far ahead of the MMA as
// the ring allows.  PAIR: a cluster of two CTAs computes one tile, each half
// of its M, and loads half of its N.  Eight warps drain (two for each lane
// quadrant, taking boxes in turn), because short contractions leave little but
// the stores to do.  Every box of D is 32 rows of 128 bytes: in rows mode with
// bf16 a warp's 32 lanes are half of that, so the warps of two neighbouring
// quadrants fill two boxes together, one while the other is stored.
//
// Where there are few tiles, workers share a tile's contraction (a group of more
// rows between more of them): each writes its fp32 partial tile to scratch, and the last to
// arrive adds them in the order of k, as gemm_kernel's split-K does.
//
// What bounds it, measured (bf16 in and out, cold L2):
//   32768 rows of 32 even groups, 2048 x 4096: 314 us in short runs (1751
//     TFLOP/s, 91% of the 1931 of a plain library product in short runs; tensor
//     pipe 88-95% active), 363-387 us when run for seconds, where the
//     board's power limit lowers the clock (library: 1740 TFLOP/s).
//   64 rows of 40 of 64 experts, 2048 x 1408: 37.3-37.8 us, 231 MB of weights at
//     6.1 TB/s (92% of a plain copy): HBM.
//   5003 rows of 11 groups, 1400 x 1000, weights N x K: 28.3 us; about a
//     hundred pair tiles on 76 pairs are two turns, of which the second is a
//     third full, and a tile of 22 k-blocks is half start and stores.  (Pair tiles
//     of 128 rows: 30.8.)
//   wgrad, 32768 rows of 16 groups, 2048 x 2048: 174 us short (1580
//     TFLOP/s, 82%), 189-198 sustained: MN-major operands and fringe blocks.
//   wgrad, 1003 rows of 7 of 8 groups, 640 x 384, fp32: 5.7-6.2 us on the GPU:
//     latency (start, two or three k-blocks, stores of 7.9 MB).
//
// The list of tiles depends on offsets the host has not seen: every warp
// walks it by itself, 32 groups at a time with a lane for each (a group's
// tile count, a warp scan, a ballot), so that no table in shared memory and
// no second kernel is needed.
#pragma once

#include "tg_kernel.cuh"
#include "tg_sync.cuh"

namespace tg {

// Orders this thread's accesses before and after it for the whole cluster.
__device__ __forceinline__ void fence_acq_rel_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

struct GroupedParams {
    const int32_t *offsets;  // [groups + 1]
    int32_t groups;
    int32_t S;               // rows of the ragged operands
    int32_t M;               // wgrad mode: rows of D[g] (columns of A)
    int32_t N, K;            // K: rows mode only
    int32_t k_blocks;        // rows mode: ceil(K / BK)
    int32_t tiles_m;         // wgrad mode: tiles of M
    int32_t tiles_n;         // tiles of D's columns
    int32_t group_m;         // tiles of rows a raster strip
    int32_t b_k;             // rows mode: 1 = B stored N x K
    int32_t b_shared;        // rows mode: 1 = every group has the same B
    int32_t epi_tma;
    void *D;
    int64_t ldd, strideD;
    int32_t out_bf16, act;
    float alpha;
    const float *bias;
    int64_t bias_stride;
    int32_t splits;          // workers that share a tile, at most
    int32_t part_blocks;     // k-blocks a share has, about: a tile has as many shares as that takes
    float *partials;         // splits > 1: [tile][CTA of the pair][splits][BM x BN]
    int32_t *counters;       // splits > 1: arrivals per [tile][CTA], zero between calls
    uint32_t *err;
    uint64_t timeout_ns;
    int32_t debug_stall;     // watchdog self-test
};

// One tile: group, first row of the group and the row behind it (rows mode:
// rows of A and D; wgrad mode: rows of the contraction), tile coordinates.
struct GroupUnit {
    int32_t g, row0, row1, tm, tn, k_blocks;
    int32_t kb0, kb1;      // this worker's k-blocks of it
    int32_t part, nparts;
    int32_t tile;
};

// A warp's walk through the tiles (or shares of tiles) in order.  Lane l holds
// group base + l: its bounds and the number of tiles up to and including it.  Bounds are
// clamped to [0, S] and never fall, whatever offsets holds, so that no row
// is out of range and the number of tiles is bounded.
struct GroupWalk {
    int32_t base;      // group of lane 0
    int32_t lo, hi;    // lane: bounds of its group
    int32_t incl;      // lane: tiles of the chunk up to its group
    int32_t before;    // tiles before the chunk
    int32_t total;     // tiles of the chunk
    int32_t last;      // the bound before the next chunk
};

// The shares of a tile of so many k-blocks.
__device__ __forceinline__ int32_t shares_of(const GroupedParams &p, int32_t k_blocks)
{
    return p.splits > 1 ? max(1, min(p.splits, (k_blocks + p.part_blocks - 1) / p.part_blocks)) : 1;
}

template <int TILE_R, bool WGRAD>  // rows mode: rows of A a tile takes
__device__ __forceinline__ void walk_load(const GroupedParams &p, int32_t base, GroupWalk &w)
{
    const int lane = static_cast<int>(threadIdx.x & 31);
    const int32_t g = base + lane;
    int32_t hi = g < p.groups ? __ldg(p.offsets + g + 1) : 0;
    hi = max(0, min(hi, p.S));
    hi = max(hi, w.last);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, hi, d);
        if (lane >= d) hi = max(hi, o);
    }
    int32_t lo = __shfl_up_sync(0xffffffffu, hi, 1);
    if (lane == 0) lo = w.last;
    int32_t units = 0;
    if (g < p.groups)
        units = WGRAD ? p.tiles_m * p.tiles_n * shares_of(p, (hi - lo + BK - 1) / BK)
                      : (hi - lo + TILE_R - 1) / TILE_R * p.tiles_n * shares_of(p, p.k_blocks);
    int32_t incl = units;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    w.base = base;
    w.lo = lo;
    w.hi = hi;
    w.incl = incl;
    w.total = __shfl_sync(0xffffffffu, incl, 31);
    w.last = __shfl_sync(0xffffffffu, hi, 31);
}

template <int TILE_R, bool WGRAD>
__device__ __forceinline__ void walk_begin(const GroupedParams &p, GroupWalk &w)
{
    w.before = 0;
    w.last = max(0, min(__ldg(p.offsets), p.S));
    if (!WGRAD || p.splits > 1) walk_load<TILE_R, WGRAD>(p, 0, w);
}

// Item t of the list - a tile, or a share of one - where t never falls from
// call to call; false past the end.  Shares are counted group by group, each
// group's own number, so that none of the list is empty and workers, which
// take every n-th, have equal numbers.  (As tile x most shares, empty ones
// skipped, a quarter of the workers got them all where most shares and
// workers have a common factor: wgrad, 32768 rows of 8 groups, 256 x 1000:
// 98 us instead of 35.)  A group's first shares of all its tiles come first:
// they read the same rows.
template <int TILE_R, bool WGRAD>
__device__ __forceinline__ bool walk_to(const GroupedParams &p, int64_t t64, GroupWalk &w, GroupUnit &u)
{
    if (t64 > INT32_MAX) return false;
    const int32_t t = static_cast<int32_t>(t64);
    int32_t r, tiles_m;
    u.part = 0;
    u.nparts = 1;
    if (WGRAD && p.splits == 1) {
        tiles_m = p.tiles_m;
        const int32_t per = tiles_m * p.tiles_n;
        u.g = t / per;
        if (u.g >= p.groups) return false;
        r = t - u.g * per;
        u.row0 = max(0, min(__ldg(p.offsets + u.g), p.S));
        u.row1 = max(u.row0, min(__ldg(p.offsets + u.g + 1), p.S));
        u.k_blocks = (u.row1 - u.row0 + BK - 1) / BK;
    } else {
        while (t >= w.before + w.total) {
            if (w.base + 32 >= p.groups) return false;
            w.before += w.total;
            walk_load<TILE_R, WGRAD>(p, w.base + 32, w);
        }
        const int32_t at = t - w.before;
        const int idx = __popc(__ballot_sync(0xffffffffu, at >= w.incl));
        u.g = w.base + idx;
        u.row0 = __shfl_sync(0xffffffffu, w.lo, idx);
        u.row1 = __shfl_sync(0xffffffffu, w.hi, idx);
        int32_t before = __shfl_sync(0xffffffffu, w.incl, idx > 0 ? idx - 1 : 0);
        if (idx == 0) before = 0;
        r = at - before;
        tiles_m = WGRAD ? p.tiles_m : (u.row1 - u.row0 + TILE_R - 1) / TILE_R;
        u.k_blocks = WGRAD ? (u.row1 - u.row0 + BK - 1) / BK : p.k_blocks;
        if (p.splits > 1) {
            u.nparts = shares_of(p, u.k_blocks);
            const int32_t per = tiles_m * p.tiles_n;
            u.part = r / per;
            r -= u.part * per;
            u.tile = WGRAD ? u.g * per + r : (w.before + before) / u.nparts + r;
        }
    }
    const int32_t strip = p.group_m * p.tiles_n;
    const int32_t first = r / strip * p.group_m;
    const int32_t in = r % strip, rows = min(tiles_m - first, p.group_m);
    u.tm = first + in % rows;
    u.tn = in / rows;
    u.kb0 = static_cast<int32_t>(static_cast<int64_t>(u.part) * u.k_blocks / u.nparts);
    u.kb1 = static_cast<int32_t>(static_cast<int64_t>(u.part + 1) * u.k_blocks / u.nparts);
    return true;
}

// rows mode: the MMA's N for a tile, its rows rounded up to 32 (16 a CTA of a
// pair).
template <int BN>
__device__ __forceinline__ int32_t rows_n(const GroupUnit &u)
{
    return min(BN, (u.row1 - u.row0 - u.tm * BN + 31) / 32 * 32);
}

// alpha, bias and activation on 32 values (of one column of D in rows mode,
// whose bias is `bias`).
__device__ __forceinline__ void grouped_epilogue(const GroupedParams &p, uint32_t (&v)[32], float bias)
{
    float x[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) x[j] = __fmul_rn(p.alpha, __uint_as_float(v[j]));
    if (p.bias) {
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = __fadd_rn(x[j], bias);
    }
    switch (p.act) {
        case 1:
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = activation(x[j], 1);
            break;
        case 2:
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = activation(x[j], 2);
            break;
        case 3:
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = activation(x[j], 3);
            break;
        default:
            break;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(x[j]);
}

constexpr int GROUPED_EPI_WARPS = 8;
// A box of D in shared memory: 32 rows of 128 bytes with the 128-byte swizzle.
constexpr int EPI_ROWS = 32, EPI_ROW_BYTES = 128;

constexpr int GROUPED_THREADS = 64 + 32 * GROUPED_EPI_WARPS;  // rows mode
constexpr int GROUPED_WGRAD_THREADS = GROUPED_THREADS + 32;   // and the fixer warp

template <int BN, int STAGES, bool PAIR, bool WGRAD>
__global__ void __launch_bounds__(WGRAD ? GROUPED_WGRAD_THREADS : GROUPED_THREADS, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmD, const GroupedParams p)
{
    using G = Geometry<BN, PAIR>;
    constexpr int TILE_M = PAIR ? 2 * BM : BM;  // the MMA's M
    constexpr int TILE_R = WGRAD ? TILE_M : BN; // rows of D a tile takes
    constexpr int B_BOXES = G::B_COLS / 64;
    constexpr uint32_t BOX_BYTES = BK * 64 * 2;                    // 64 k x 64 columns, 8 KB
    constexpr uint32_t EPI_BOX_BYTES = EPI_CHUNK * EPI_CHUNK * 4;  // 4 KB
    constexpr uint32_t EPI_WARPS_TOTAL = (PAIR ? 2 : 1) * GROUPED_EPI_WARPS;
    static_assert(GROUPED_EPI_WARPS * EPI_BOX_BYTES <= G::EPI_BYTES, "epilogue boxes");
    static_assert(!WGRAD || BN % 64 == 0, "wgrad mode loads 64-column boxes");
    constexpr uint32_t TMEM_ALLOC = static_cast<uint32_t>(G::TMEM_COLS);
    static_assert(8 * (4 * STAGES + 6) + 24 <= G::BAR_BYTES, "barrier area");

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sA = raw + pad;
    const uint32_t sB = sA + STAGES * G::A_STAGE;
    const uint32_t sE = sB + STAGES * G::B_STAGE;
    uint8_t *bar_area = smem + STAGES * G::STAGE + G::EPI_BYTES;
    const uint32_t bar0 = ptx::smem_addr(bar_area);
    // barrier k at bar0 + 8k: [0, S) full, [S, 2S) empty, 2S+{0,1} tfull,
    // 2S+{2,3} tempty, 2S+4 mma-done; wgrad mode: from 2S+5 fringe[S] (this
    // CTA's copies of a group's last, partial k-block landed) and pfix[S]
    // (pair, on the leader's: the peer has zeroed its share of it).
    const uint32_t done_bar = bar0 + 8u * (2 * STAGES + 4);
    const uint32_t stall_bar = bar0 + 8u * (4 * STAGES + 5);  // never completed
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_area + 8 * (4 * STAGES + 6));
    volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(tmem_slot + 1);
    volatile int32_t *last_flag = reinterpret_cast<volatile int32_t *>(tmem_slot + 2);
    uint32_t *issued_slot = tmem_slot + 4;  // k-blocks this CTA's producer loaded; then a bit for
                                            // each slot whose last load was a fringe
    auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (STAGES + s); };
    auto tfull_bar = [&](uint32_t b) { return bar0 + 8u * (2 * STAGES + b); };
    auto tempty_bar = [&](uint32_t b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
    auto fringe_bar = [&](uint32_t s) { return bar0 + 8u * (2 * STAGES + 5 + s); };
    auto pfix_bar = [&](uint32_t s) { return bar0 + 8u * (3 * STAGES + 5 + s); };

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = static_cast<int>(threadIdx.x & 31);
    const uint32_t rank = PAIR ? ptx::cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    const int64_t worker = PAIR ? (blockIdx.x >> 1) : blockIdx.x;
    const int64_t n_workers = PAIR ? (gridDim.x >> 1) : gridDim.x;

    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < STAGES; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
            if constexpr (WGRAD) {
                ptx::mbar_init(fringe_bar(s), 1);
                ptx::mbar_init(pfix_bar(s), 1);
            }
        }
        for (uint32_t b = 0; b < 2; ++b) {
            ptx::mbar_init(tfull_bar(b), 1);
            ptx::mbar_init(tempty_bar(b), EPI_WARPS_TOTAL);
        }
        ptx::mbar_init(done_bar, 1);
        ptx::mbar_init(stall_bar, 1);
        *abort_flag = 0;
        issued_slot[0] = issued_slot[1] = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        if (WGRAD ? p.S > 0 : p.k_blocks > 0) {  // else there is nothing to load, and no map
            ptx::prefetch_tensormap(&tmA);
            ptx::prefetch_tensormap(&tmB);
        }
        if (p.epi_tma) ptx::prefetch_tensormap(&tmD);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            ptx::tmem_alloc_pair(ptx::smem_addr(tmem_slot), TMEM_ALLOC);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(ptx::smem_addr(tmem_slot), TMEM_ALLOC);
            ptx::tmem_relinquish();
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) ptx::cluster_sync_all();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    ptx::griddep_wait();
    const uint32_t peer_abort =
        PAIR ? ptx::map_to_cta(ptx::smem_addr(const_cast<int32_t *>(abort_flag)), rank ^ 1u) : 0u;
    const Watchdog wd{p.timeout_ns, abort_flag, p.err, peer_abort};

    GroupWalk walk;
    GroupUnit w;
    walk_begin<TILE_R, WGRAD>(p, walk);

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        uint32_t it = 0;
        uint32_t fringe = 0, fringe_phase = 0;  // bit s: slot s's last load; parity of its next fringe
        bool ok = true;
        const uint32_t full0 = PAIR ? ptx::map_to_cta(full_bar(0), 0u) : full_bar(0);
        const uint32_t fringe0 = PAIR ? ptx::map_to_cta(fringe_bar(0), rank) : fringe_bar(0);
        for (int64_t t = worker; ok && walk_to<TILE_R, WGRAD>(p, t, walk, w); t += n_workers) {
            if (!dbg_ok(w.g >= 0 && w.g < p.groups && w.row0 >= 0 && w.row0 <= w.row1 && w.row1 <= p.S && w.tm >= 0 &&
                            w.tn >= 0 && w.tn < p.tiles_n,
                        CHK_UNIT, wd))
                break;
            // this CTA's part of the MMA's M and N operands
            int32_t m0, n0;
            if constexpr (WGRAD) {
                m0 = w.tm * TILE_M + static_cast<int32_t>(rank) * BM;
                n0 = w.tn * BN + static_cast<int32_t>(rank) * G::B_COLS;
            } else {
                m0 = w.tn * TILE_M + static_cast<int32_t>(rank) * BM;
                n0 = w.row0 + w.tm * BN + static_cast<int32_t>(rank) * (rows_n<BN>(w) / 2);
            }
            for (int32_t kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                const uint32_t s = it % STAGES;
                const uint32_t ph = (it / STAGES) & 1u;
                const int r = wait_bounded_warp(empty_bar(s), ph ^ 1u, wd);
                if (r != WAIT_OK) {
                    if (r == WAIT_TIMEOUT && lane == 0) raise_abort(wd, ERR_TIMEOUT_PRODUCER);
                    ok = false;
                    break;
                }
                const bool partial = WGRAD && w.row1 - w.row0 < (kb + 1) * BK;
                if constexpr (WGRAD) {
                    fringe = partial ? fringe | (1u << s) : fringe & ~(1u << s);
                    if (partial) fringe_phase ^= 1u << s;
                }
                if (ptx::elect_one()) {
                    uint32_t fb;
                    if (partial) {
                        ptx::mbar_arrive_expect_tx(fringe_bar(s), G::STAGE);
                        fb = fringe0 + 8u * s;
                    } else if constexpr (PAIR) {
                        if (leader) ptx::mbar_arrive_expect_tx(full_bar(s), 2 * G::STAGE);
                        fb = full0 + 8u * s;
                    } else {
                        ptx::mbar_arrive_expect_tx(full_bar(s), G::STAGE);
                        fb = full_bar(s);
                    }
                    auto load = [&](uint32_t dst, const CUtensorMap *map, int32_t c0, int32_t c1, int32_t c2) {
                        if constexpr (PAIR)
                            ptx::tma_load_3d_pair(dst, map, fb, c0, c1, c2);
                        else
                            ptx::tma_load_3d(dst, map, fb, c0, c1, c2);
                    };
                    const uint32_t a_dst = sA + s * G::A_STAGE;
                    const uint32_t b_dst = sB + s * G::B_STAGE;
                    if constexpr (WGRAD) {
                        const int32_t k0 = w.row0 + kb * BK;
                        load(a_dst, &tmA, m0, k0, 0);
                        load(a_dst + BOX_BYTES, &tmA, m0 + 64, k0, 0);
#pragma unroll
                        for (int j = 0; j < B_BOXES; ++j) load(b_dst + j * BOX_BYTES, &tmB, n0 + 64 * j, k0, 0);
                    } else {
                        const int32_t z = p.b_shared ? 0 : w.g;
                        if (!p.b_k) {  // B[g] is K x N: 64 k x 64 columns, twice
                            load(a_dst, &tmB, m0, kb * BK, z);
                            load(a_dst + BOX_BYTES, &tmB, m0 + 64, kb * BK, z);
                        } else {  // stored N x K: 128 columns x 64 k
                            load(a_dst, &tmB, kb * BK, m0, z);
                        }
                        load(b_dst, &tmA, kb * BK, n0, 0);
                    }
                }
                __syncwarp();
            }
        }
        if (lane == 0) {
            issued_slot[0] = it;
            issued_slot[1] = fringe;
            const uint32_t first = it > STAGES ? it - STAGES : 0u;
            for (uint32_t j = first; j < it; ++j) {
                const uint32_t s = j % STAGES;
                if ((fringe >> s) & 1u) {  // its copies, on this CTA's own barrier
                    if (!wait_drain(fringe_bar(s), ((fringe_phase >> s) & 1u) ^ 1u, wd)) break;
                } else if constexpr (!PAIR) {
                    if (!wait_drain(full_bar(s), (j / STAGES) & 1u, wd)) break;
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (!PAIR || leader) {
            // ------------------------------------------------ MMA issuer
            const bool m_mn = WGRAD || p.b_k == 0;  // the M operand's M is contiguous (N's only in wgrad mode)
            uint32_t idesc = instr_desc_bf16<TILE_M, BN>(m_mn, WGRAD);
            const uint64_t a_desc0 = smem_desc_sw128(0, m_mn ? BK * 128 : 16, 1024);
            const uint64_t b_desc0 = smem_desc_sw128(0, WGRAD ? BK * 128 : 16, 1024);
            const uint32_t a_step = m_mn ? 2048u : 32u;
            const uint32_t b_step = WGRAD ? 2048u : 32u;
            uint32_t it = 0, n = 0;
            bool ok = true;
            for (int64_t t = worker; ok && walk_to<TILE_R, WGRAD>(p, t, walk, w); t += n_workers) {
                if (w.kb0 == w.kb1) continue;  // the epilogue writes an empty sum itself
                const uint32_t buf = n & 1u;
                const uint32_t tph = (n >> 1) & 1u;
                ++n;
                int r = wait_bounded_warp(tempty_bar(buf), tph ^ 1u, wd);
                if (r != WAIT_OK) {
                    if (r == WAIT_TIMEOUT && lane == 0) raise_abort(wd, ERR_TIMEOUT_MMA);
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t d_tmem = tmem_base + buf * BN;
                if constexpr (!WGRAD)
                    idesc = (idesc & ~(0x3Fu << 17)) | (static_cast<uint32_t>(rows_n<BN>(w)) >> 3 << 17);
                for (int32_t kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                    const uint32_t s = it % STAGES;
                    const uint32_t ph = (it / STAGES) & 1u;
                    r = wait_bounded_warp(full_bar(s), ph, wd);
                    if (r != WAIT_OK) {
                        if (r == WAIT_TIMEOUT && lane == 0) raise_abort(wd, ERR_TIMEOUT_MMA);
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    if (ptx::elect_one()) {
                        const uint32_t a_addr = sA + s * G::A_STAGE;
                        const uint32_t b_addr = sB + s * G::B_STAGE;
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk) {
                            const uint64_t ad = a_desc0 | (((a_addr + kk * a_step) >> 4) & 0x3FFFu);
                            const uint64_t bd = b_desc0 | (((b_addr + kk * b_step) >> 4) & 0x3FFFu);
                            const uint32_t acc = (kb > w.kb0 || kk > 0) ? 1u : 0u;
                            if constexpr (PAIR)
                                ptx::mma_bf16_pair(d_tmem, ad, bd, idesc, acc);
                            else
                                ptx::mma_bf16(d_tmem, ad, bd, idesc, acc);
                        }
                        if constexpr (PAIR)
                            ptx::mma_commit_pair_multicast(empty_bar(s), 0x3);
                        else
                            ptx::mma_commit(empty_bar(s));
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (ptx::elect_one()) {
                    if constexpr (PAIR)
                        ptx::mma_commit_pair_multicast(tfull_bar(buf), 0x3);
                    else
                        ptx::mma_commit(tfull_bar(buf));
                }
                __syncwarp();
            }
            if (ptx::elect_one()) {
                if constexpr (PAIR)
                    ptx::mma_commit_pair_multicast(done_bar, 0x1);
                else
                    ptx::mma_commit(done_bar);
                wait_drain(done_bar, 0, wd);
            }
            __syncwarp();
        }
    } else if (WGRAD && warp == 2 + GROUPED_EPI_WARPS) {
        // ------------------------------------------------ fixer
        if constexpr (WGRAD) {
            uint32_t it = 0;
            uint32_t phase = 0;  // bit s: parity of the slot's next fringe
            const uint32_t pfix_leader0 = PAIR ? ptx::map_to_cta(pfix_bar(0), 0u) : 0u;
            for (int64_t t = worker; walk_to<TILE_R, WGRAD>(p, t, walk, w); t += n_workers) {
                it += static_cast<uint32_t>(w.kb1 - w.kb0);
                const int32_t tail = (w.row1 - w.row0) % BK;
                // (no tail: also an empty group; the fringe is in the last share)
                if (tail == 0 || w.kb0 == w.kb1 || w.kb1 != w.k_blocks) continue;
                const uint32_t s = (it - 1) % STAGES;
                int r = wait_bounded_warp(fringe_bar(s), (phase >> s) & 1u, wd);
                if (r != WAIT_OK) {
                    if (r == WAIT_TIMEOUT && lane == 0) raise_abort(wd, ERR_TIMEOUT_PRODUCER);
                    break;
                }
                // k row r of a 64-column box is its bytes [128 r, 128 r + 128)
                for (int box = 0; box < 2 + B_BOXES; ++box) {
                    const uint32_t at = box < 2 ? sA + s * G::A_STAGE + box * BOX_BYTES
                                                : sB + s * G::B_STAGE + (box - 2) * BOX_BYTES;
                    for (uint32_t b = tail * 128u + lane * 16u; b < BOX_BYTES; b += 512u)
                        ptx::st_shared_v4(at + b, 0u, 0u, 0u, 0u);
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if constexpr (PAIR) {
                    if (!leader) {
                        if (lane == 0) ptx::mbar_arrive_cluster(pfix_leader0 + 8u * s);
                    } else {
                        r = wait_bounded_warp(pfix_bar(s), (phase >> s) & 1u, wd);
                        if (r != WAIT_OK) {
                            if (r == WAIT_TIMEOUT && lane == 0) raise_abort(wd, ERR_TIMEOUT_PRODUCER);
                            break;
                        }
                        fence_acq_rel_cluster();
                    }
                }
                if (leader && lane == 0) ptx::mbar_arrive(full_bar(s));
                phase ^= 1u << s;
                __syncwarp();
            }
        }
    } else {
        // ------------------------------------------------ epilogue
        const int q = warp & 3;              // tensor-memory lane quadrant of this warp
        const int turn = (warp - 2) >> 2;    // which of the quadrant's two warps
        const bool duo = !WGRAD && p.out_bf16;  // two quadrants' warps share boxes
        const int sub = q & 1;                  // duo: the half of a box row that is this warp's
        const uint32_t duo_bar = 2u + static_cast<uint32_t>((warp - 2) >> 1);
        const uint32_t boxes = duo ? sE + static_cast<uint32_t>((warp - 2) >> 1) * 2u * EPI_BOX_BYTES
                                   : sE + static_cast<uint32_t>(warp - 2) * EPI_BOX_BYTES;
        uint32_t box = boxes;
        const uint32_t tempty_leader0 = PAIR ? ptx::map_to_cta(tempty_bar(0), 0u) : tempty_bar(0);
        const bool plain = p.alpha == 1.0f && !p.bias && p.act == 0;
        const int size = p.out_bf16 ? 2 : 4;
        const int width = EPI_ROW_BYTES / size;
        // Address of 16-byte unit u of box row r.
        auto unit_at = [&](int r, int u) { return box + r * EPI_ROW_BYTES + ((u ^ (r & 7)) << 4); };

        // The next box may be written: its last TMA store has read it.  A duo
        // has two boxes in turn and lets the other one's store run on, which
        // counts on one bulk group a box (see flush).
        auto box_free = [&]() {
            if (duo) {
                box = box == boxes ? boxes + EPI_BOX_BYTES : boxes;
                if (p.epi_tma && sub == 0 && lane == 0) ptx::bulk_wait_group_read<1>();
                ptx::named_barrier_sync(duo_bar, 64);
            } else {
                if (p.epi_tma && lane == 0) ptx::bulk_wait_group_read<0>();
                __syncwarp();
            }
        };
        // The box -> rows row0 .. of D (those before `limit`), columns col0 ..
        // `whole`: a TMA store may write all of its rows (the tensor's own end
        // clips a box, a group's end does not).
        auto flush = [&](int32_t row0, int32_t limit, bool whole, int32_t col0, int32_t g) {
            const int32_t cols = min(width, p.N - col0);
            // (a box that the row's end cuts off its 16 bytes goes out plainly:
            // a TMA store would write on to the next 16-byte boundary)
            const bool tma = p.epi_tma && whole && (cols == width || p.N % (16 / size) == 0);
            if (tma) ptx::fence_proxy_async_smem();
            if (duo)
                ptx::named_barrier_sync(duo_bar, 64);
            else
                __syncwarp();
            if (tma) {
                if (lane == 0 && (!duo || sub == 0)) {
                    ptx::tma_store_3d(&tmD, box, col0, row0, WGRAD ? g : 0);
                    ptx::bulk_commit_group();
                }
                return;
            }
            // a plain box commits a group too, an empty one: without it the one
            // group that box_free leaves running could be of the box it hands out
            if (duo && p.epi_tma && sub == 0 && lane == 0) ptx::bulk_commit_group();
            const int32_t nrows = min(EPI_ROWS, limit - row0);
            const int r_first = duo ? sub : 0, r_step = duo ? 2 : 1;  // duo: every other row (or four) each
            uint8_t *dst = static_cast<uint8_t *>(p.D) +
                           ((WGRAD ? static_cast<int64_t>(g) * p.strideD : 0) + static_cast<int64_t>(row0) * p.ldd + col0) * size;
            const int64_t pitch = p.ldd * size;
            if (p.epi_tma) {  // rows of D on 16 bytes
                const int per = 16 / size, u = lane & 7, n = min(per, cols - u * per);
#pragma unroll 2
                for (int r = r_first * 4 + (lane >> 3); r < nrows; r += 4 * r_step) {
                    uint32_t v[4];
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                                 : "r"(unit_at(r, u))
                                 : "memory");
                    uint8_t *o = dst + r * pitch + u * 16;
                    if (n == per) {
                        *reinterpret_cast<uint4 *>(o) = make_uint4(v[0], v[1], v[2], v[3]);
                    } else if (p.out_bf16) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (e < n) reinterpret_cast<uint16_t *>(o)[e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (e < n) reinterpret_cast<uint32_t *>(o)[e] = v[e];
                    }
                }
            } else {  // an element a lane
                for (int c = lane; c < cols; c += 32) {
                    const int u = c * size >> 4, in = c * size & 15;
                    uint8_t *o = dst + c * size + r_first * pitch;
#pragma unroll 8
                    for (int r = r_first; r < nrows; r += r_step, o += r_step * pitch) {
                        if (p.out_bf16)
                            *reinterpret_cast<uint16_t *>(o) = ld_shared_u16(unit_at(r, u) + in);
                        else
                            *reinterpret_cast<float *>(o) = ld_shared_f32(unit_at(r, u) + in);
                    }
                }
            }
            if (!duo) __syncwarp();  // the box may be written again
        };
        // 32 values of lane `lane` into the box.  rows mode: one column of its
        // 32 rows; wgrad mode: row `lane`, columns from `at`.
        auto stage = [&](const uint32_t (&v)[32], int at) {
            if constexpr (WGRAD) {
                if (p.out_bf16) {
                    uint32_t h[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) h[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        ptx::st_shared_v4(unit_at(lane, at / 8 + u), h[4 * u], h[4 * u + 1], h[4 * u + 2], h[4 * u + 3]);
                } else {
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        ptx::st_shared_v4(unit_at(lane, u), v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
                }
            } else if (p.out_bf16) {
                const int u = sub * 4 + (lane >> 3), in = (lane & 7) * 2;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const uint16_t h = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v[j])));
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(unit_at(j, u) + in), "h"(h) : "memory");
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(unit_at(j, lane >> 2) + (lane & 3) * 4), "r"(v[j]) : "memory");
            }
        };
        auto release_tmem = [&](uint32_t buf) {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR)
                    ptx::mbar_arrive_cluster(tempty_leader0 + 8u * buf);
                else
                    ptx::mbar_arrive(tempty_bar(buf));
            }
        };

        bool ok = true;
        if (p.debug_stall) {  // watchdog self-test: a barrier that nothing completes
            const int r = wait_bounded(stall_bar, 0, wd);
            if (r == WAIT_TIMEOUT) raise_abort(wd, ERR_TIMEOUT_EPILOGUE);
            ok = agree(r == WAIT_OK, 1, 32 * GROUPED_EPI_WARPS);
        }
        uint32_t n = 0;
        const int per_box = WGRAD && p.out_bf16 ? 2 : 1;  // 32-column pieces of the accumulator a box takes
        for (int64_t t = worker; ok && walk_to<TILE_R, WGRAD>(p, t, walk, w); t += n_workers) {
            // Accumulator column `32 c` and this warp's lanes in D.
            const int32_t lanes0 = (WGRAD ? w.tm : w.tn) * TILE_M + static_cast<int32_t>(rank) * BM + q * 32;
            const int32_t box0 = duo ? lanes0 - 32 * sub : lanes0;  // the box's first lane
            const int32_t cols0 = WGRAD ? w.tn * BN : w.row0 + w.tm * BN;
            const int32_t end = WGRAD ? p.N : min(w.row1, cols0 + BN);  // of the accumulator's columns
            const int32_t limit = WGRAD ? p.M : end;                     // of D's rows
            const int32_t pieces = (min(BN, end - cols0) + 31) / 32;
            const bool lanes_in = box0 < (WGRAD ? p.M : p.N);  // uniform in a warp (and in a duo)
            const float bias = !WGRAD && p.bias && lanes0 + lane < p.N
                                   ? __ldg(p.bias + static_cast<int64_t>(w.g) * p.bias_stride + lanes0 + lane)
                                   : 0.0f;
            auto put = [&](int c) {
                const int32_t row0 = WGRAD ? lanes0 : cols0 + 32 * c;
                flush(row0, limit, row0 + EPI_ROWS <= limit || limit == (WGRAD ? p.M : p.S), WGRAD ? cols0 + 32 * c : box0, w.g);
            };
            uint32_t va[32], vb[32];
            if (w.k_blocks == 0) {  // the empty sum
#pragma unroll
                for (int j = 0; j < 32; ++j) va[j] = 0u;
                if (!plain) grouped_epilogue(p, va, bias);
                for (int c = turn * per_box; lanes_in && c < pieces; c += 2 * per_box) {
                    box_free();
                    stage(va, 0);
                    if (per_box == 2) stage(va, 32);
                    put(c);
                }
                continue;
            }
            const uint32_t buf = n & 1u;
            const uint32_t tph = (n >> 1) & 1u;
            ++n;
            // (the warps that meet at barriers below leave together)
            const int r = wait_bounded(tfull_bar(buf), tph, wd);
            if (r == WAIT_TIMEOUT) raise_abort(wd, ERR_TIMEOUT_EPILOGUE);
            if (!(p.splits > 1 ? agree(r == WAIT_OK, 1, 32 * GROUPED_EPI_WARPS) : agree(r == WAIT_OK, duo_bar, 64))) break;
            ptx::tc_fence_after();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * BN;
            if (w.nparts > 1) {
                // The partial tile -> scratch [piece][column quad][lane][4
                // columns]: 16 coalesced bytes a thread.
                constexpr int64_t PART4 = BM * BN / 4;  // float4s a part
                const int64_t half = static_cast<int64_t>(w.tile) * (PAIR ? 2 : 1) + rank;
                float4 *parts = reinterpret_cast<float4 *>(p.partials) + half * p.splits * PART4 + q * 32 + lane;
                float4 *mine = parts + w.part * PART4;
                for (int c = turn; lanes_in && c < pieces; c += 2) {
                    ptx::tmem_load_32cols(taddr + c * 32, va);
#pragma unroll
                    for (int j4 = 0; j4 < 8; ++j4)
                        __stcg(mine + (c * 8 + j4) * BM,
                               make_float4(__uint_as_float(va[4 * j4]), __uint_as_float(va[4 * j4 + 1]),
                                           __uint_as_float(va[4 * j4 + 2]), __uint_as_float(va[4 * j4 + 3])));
                }
                release_tmem(buf);
                __threadfence();
                ptx::named_barrier_sync(1, 32 * GROUPED_EPI_WARPS);
                if (warp == 2 && lane == 0) {
                    const int32_t old = atomicAdd(p.counters + half, 1);
                    *last_flag = old == w.nparts - 1 ? 1 : 0;
                    if (old == w.nparts - 1) atomicExch(p.counters + half, 0);  // ready for the next call
                }
                ptx::named_barrier_sync(1, 32 * GROUPED_EPI_WARPS);
                if (*last_flag) {
                    __threadfence();
                    for (int c0 = turn * per_box; lanes_in && c0 < pieces; c0 += 2 * per_box) {
                        box_free();
                        for (int c = c0; c < min(pieces, c0 + per_box); ++c) {
                            float4 acc[8];
#pragma unroll
                            for (int j4 = 0; j4 < 8; ++j4) acc[j4] = __ldcg(parts + (c * 8 + j4) * BM);
#pragma unroll 2
                            for (int s = 1; s < w.nparts; ++s) {
                                float4 t4[8];
#pragma unroll
                                for (int j4 = 0; j4 < 8; ++j4) t4[j4] = __ldcg(parts + s * PART4 + (c * 8 + j4) * BM);
#pragma unroll
                                for (int j4 = 0; j4 < 8; ++j4) {
                                    acc[j4].x += t4[j4].x; acc[j4].y += t4[j4].y;
                                    acc[j4].z += t4[j4].z; acc[j4].w += t4[j4].w;
                                }
                            }
#pragma unroll
                            for (int j4 = 0; j4 < 8; ++j4) {
                                va[4 * j4] = __float_as_uint(acc[j4].x);
                                va[4 * j4 + 1] = __float_as_uint(acc[j4].y);
                                va[4 * j4 + 2] = __float_as_uint(acc[j4].z);
                                va[4 * j4 + 3] = __float_as_uint(acc[j4].w);
                            }
                            if (!plain) grouped_epilogue(p, va, bias);
                            stage(va, (c - c0) * 32);
                        }
                        put(c0);
                    }
                }
                ptx::named_barrier_sync(1, 32 * GROUPED_EPI_WARPS);  // the flag may be written again
                continue;
            }
            // The next pieces' loads are on their way while these are stored.
            const int step = 2 * per_box;
            int c = turn * per_box;
            if (lanes_in && c < pieces) {
                ptx::tmem_load_32cols_async(taddr + c * 32, va);
                if (per_box == 2 && c + 1 < pieces) ptx::tmem_load_32cols_async(taddr + c * 32 + 32, vb);
            } else {
                release_tmem(buf);
            }
            for (; lanes_in && c < pieces; c += step) {
                box_free();
                ptx::tmem_wait_ld(va);
                if (!plain) grouped_epilogue(p, va, bias);
                stage(va, 0);
                if (per_box == 2 && c + 1 < pieces) {
                    ptx::tmem_wait_ld(vb);
                    if (!plain) grouped_epilogue(p, vb, bias);
                    stage(vb, 32);
                }
                if (c + step < pieces) {
                    ptx::tmem_load_32cols_async(taddr + (c + step) * 32, va);
                    if (per_box == 2 && c + step + 1 < pieces) ptx::tmem_load_32cols_async(taddr + (c + step) * 32 + 32, vb);
                } else {
                    release_tmem(buf);
                }
                put(c);
            }
        }
        if constexpr (!WGRAD) {
            // Rows of no group: zeros.  16-byte stores where D's rows allow.
            const int32_t first = max(0, min(__ldg(p.offsets), p.S));
            GroupWalk end = walk;
            while (end.base + 32 < p.groups) {
                end.before += end.total;
                walk_load<TILE_R, WGRAD>(p, end.base + 32, end);
            }
            const bool vec = (reinterpret_cast<uintptr_t>(p.D) & 15u) == 0 && p.ldd * size % 16 == 0;
            const int64_t w0 = static_cast<int64_t>(blockIdx.x) * GROUPED_EPI_WARPS + (warp - 2);
            const int64_t nw = static_cast<int64_t>(gridDim.x) * GROUPED_EPI_WARPS;
            for (int64_t i = w0; i < static_cast<int64_t>(first) + (p.S - end.last); i += nw) {
                const int64_t row = i < first ? i : end.last + (i - first);
                uint8_t *dst = static_cast<uint8_t *>(p.D) + row * p.ldd * size;
                const int64_t bytes = static_cast<int64_t>(p.N) * size;
                const int64_t body = vec ? bytes / 16 * 16 : 0;
                for (int64_t b = lane * 16; b < body; b += 512)
                    *reinterpret_cast<uint4 *>(dst + b) = make_uint4(0u, 0u, 0u, 0u);
                for (int64_t b = body + lane * 2; b < bytes; b += 64) *reinterpret_cast<uint16_t *>(dst + b) = 0;
            }
        }
        if (lane == 0) ptx::bulk_wait_group_read<0>();
        __syncwarp();
    }

    __syncthreads();
    if constexpr (PAIR) {
        // as gemm_kernel: neither CTA leaves while copies, MMAs or arrivals
        // of the other may still reach it; an abort's unequal issue counts
        // are settled first
        ptx::cluster_sync_all();
        if (leader && warp == 0 && lane == 0) {
            const uint32_t i_l = *issued_slot;
            const uint32_t i_p = ptx::ld_cluster_u32(ptx::map_to_cta(ptx::smem_addr(issued_slot), 1u));
            const uint32_t hi = i_l > i_p ? i_l : i_p;
            const uint32_t lo = hi > STAGES ? hi - STAGES : 0u;
            const uint32_t fringe_l = issued_slot[1];
            const uint32_t fringe_p = ptx::ld_cluster_u32(ptx::map_to_cta(ptx::smem_addr(issued_slot + 1), 1u));
            for (uint32_t j = lo; j < hi; ++j) {
                const uint32_t s = j % STAGES;
                // a fringe brings no bytes here (each CTA waited for its own)
                if (((j < i_l ? fringe_l : fringe_p) >> s) & 1u) continue;
                if (j < i_l && j >= i_p)
                    ptx::mbar_complete_tx(full_bar(s), G::STAGE);
                else if (j >= i_l && j < i_p)
                    ptx::mbar_arrive_expect_tx(full_bar(s), G::STAGE);
                if (!wait_drain(full_bar(s), (j / STAGES) & 1u, wd)) break;
            }
        }
        ptx::cluster_sync_all();
    }
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after();
        if constexpr (PAIR)
            ptx::tmem_dealloc_pair(tmem_base, TMEM_ALLOC);
        else
            ptx::tmem_dealloc(tmem_base, TMEM_ALLOC);
    }
}

}  // namespace tg
