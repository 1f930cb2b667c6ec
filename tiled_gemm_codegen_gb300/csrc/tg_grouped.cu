// Entry points of the grouped GEMM (include/tg_gemm.h): argument checks, the
// tile choice, tensor maps and launches of grouped_kernel (tg_grouped.cuh).
#include <algorithm>
#include <cuda.h>
#include <cuda_runtime.h>

#include "tg_gemm.h"
#include "tg_grouped.cuh"
#include "tg_host_api.h"
#include "tg_tiles.h"

#define TG_API extern "C" __attribute__((visibility("default")))

namespace tg {
namespace {

using GroupedKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const GroupedParams);

struct Shape {
    GroupedKernel kern;
    int bn, smem, threads;
    bool pair;
};

template <int BN, int STAGES, bool PAIR, bool WGRAD>
Shape shape()
{
    constexpr int smem = Geometry<BN, PAIR>::smem_bytes(STAGES);
    static_assert(smem <= SMEM_LIMIT, "shared memory budget");
    return {grouped_kernel<BN, STAGES, PAIR, WGRAD>, BN, smem, WGRAD ? GROUPED_WGRAD_THREADS : GROUPED_THREADS, PAIR};
}

cudaLaunchConfig_t config(const Shape &k, int grid, cudaStream_t s, cudaLaunchAttribute (&attr)[2])
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(k.threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(k.smem);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = k.pair ? 2 : 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

// Launches `shapes[which]` with at most `units` workers.  The shared-memory
// opt-in and the number of co-resident pairs are looked up once per device
// (under the host mutex).
struct ShapeState {
    uint64_t configured = 0;
    int pairs[64] = {};
};

cudaError_t launch_shape(const Shape &k, ShapeState &st, const HostStream &hs, int64_t units, const CUtensorMap &ta,
                         const CUtensorMap &tb, const CUtensorMap &td, const GroupedParams &p)
{
    cudaLaunchAttribute attr[2];
    const bool known = hs.dev < 64 && ((st.configured >> hs.dev) & 1u);
    int pairs = known ? st.pairs[hs.dev] : 0;
    if (!known) {
        cudaError_t e = cudaFuncSetAttribute(k.kern, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
        if (e != cudaSuccess) return e;
        if (k.pair) {
            cudaLaunchConfig_t cfg = config(k, 2, hs.stream, attr);
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&pairs, k.kern, &cfg);
            if (e != cudaSuccess) return e;
            if (pairs < 1) return cudaErrorInvalidConfiguration;
        }
        if (hs.dev < 64) {
            st.pairs[hs.dev] = pairs;
            st.configured |= 1ull << hs.dev;
        }
    }
    int64_t workers = k.pair ? pairs : hs.sms;
    if (workers > units) workers = units;
    if (workers < 1) workers = 1;
    const cudaLaunchConfig_t cfg = config(k, static_cast<int>(workers) * (k.pair ? 2 : 1), hs.stream, attr);
    return cudaLaunchKernelEx(&cfg, k.kern, ta, tb, td, p);
}

// Copies the operands that TMA cannot address to aligned scratch.
// (part_bytes of the scratch in front of the copies are for partial tiles.)
tg_status realign(const HostStream &hs, Operand &a, Operand &b, size_t part_bytes, float **partials)
{
    if (!a.pack && !b.pack && !part_bytes) return TG_OK;
    void *arena = nullptr;
    tg_status st = host_arena(hs, part_bytes + pack_bytes(a) + pack_bytes(b), &arena);
    if (st != TG_OK) return st;
    *partials = static_cast<float *>(arena);
    if (!a.pack && !b.pack) return TG_OK;
    HostPack ja, jb;
    uint8_t *at = static_cast<uint8_t *>(arena) + part_bytes;
    auto move = [&](Operand &o, HostPack &j) {
        if (!o.pack) return;
        j = HostPack{o.p, at, o.rows, o.cols, o.ld, o.nb, o.stride};
        at += pack_bytes(o);
        o.p = j.dst;
        o.ld = cdiv(o.cols, 64) * 64;
        o.stride = o.rows * o.ld;
    };
    const bool pa = a.pack, pb = b.pack;
    move(a, ja);
    move(b, jb);
    return host_cuda_status(host_pack(hs, pa ? &ja : nullptr, pb ? &jb : nullptr));
}

// The options that apply here: cta_pair (1 or 2), force_pack, timeout_ns,
// debug_stall (1), b_col_major; everything else has to be 0.
bool options_ok(const tg_options *o, bool wgrad)
{
    if (!o) return true;
    return !o->block_n && !o->stages && !o->split_k && !o->epilogue && !o->max_ctas && (o->debug_stall == 0 || o->debug_stall == 1) && !o->stream_k &&
           !o->operands && !o->trace_buffer && !o->a_col_major && !o->direct && o->cta_pair >= 0 && o->cta_pair <= 2 &&
           (!wgrad || !o->b_col_major);
}

tg_status run_grouped(bool wgrad, Operand a, Operand b, bool b_k, void *D, const int32_t *offsets, int64_t groups, int64_t S,
                      int64_t M, int64_t N, int64_t K, int64_t ldd, int64_t strideD, const tg_epilogue *ep,
                      const tg_options *opt, cudaStream_t stream)
{
    const bool out_bf16 = ep && ep->out_type == TG_BF16;
    const int64_t eb = out_bf16 ? 2 : 4;
    std::lock_guard<std::mutex> lock(host_mutex());
    HostStream hs;
    tg_status st = host_stream(stream, &hs);
    if (st != TG_OK) return st;

    const int64_t hit = groups < S ? groups : S;  // groups that have rows, at most
    // Tiles: 256 x 256 for a pair or 128 x 128 for one CTA, whichever is
    // quicker by tiles_cost; rows mode takes 128 columns x 32 rows where groups
    // have few (the ring is then deeper: weights are the traffic).
    bool pair = N > 128 && (wgrad ? M > 128 : S > 32 * hit) &&
                tiles_cost(wgrad, true, S, M, N, K, groups, hs.sms) < tiles_cost(wgrad, false, S, M, N, K, groups, hs.sms);
    if (opt && opt->cta_pair) pair = opt->cta_pair == 2;
    const bool few = !wgrad && !pair && S <= 32 * hit;
    const int64_t tile_m = pair ? 256 : 128, bn = pair ? 256 : few ? 32 : 128;
    const int64_t tiles_n = cdiv(N, wgrad ? bn : tile_m);
    const int64_t tiles_m = cdiv(M, tile_m);
    const int64_t row_tiles = S / bn + hit;  // rows mode: at most, over all groups
    const int64_t units = wgrad ? groups * tiles_m * tiles_n : row_tiles * tiles_n;
    if (units > INT32_MAX) return TG_ERR_UNSUPPORTED;

    GroupedParams p{};
    p.offsets = offsets;
    p.groups = static_cast<int32_t>(groups);
    p.S = static_cast<int32_t>(S);
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.K = static_cast<int32_t>(K);
    p.k_blocks = static_cast<int32_t>(cdiv(K, BK));
    p.tiles_m = static_cast<int32_t>(tiles_m);
    p.tiles_n = static_cast<int32_t>(tiles_n);
    p.group_m = 8;
    p.b_k = b_k ? 1 : 0;
    p.D = D;
    p.ldd = ldd;
    p.strideD = strideD;
    p.out_bf16 = out_bf16 ? 1 : 0;
    p.alpha = ep ? ep->alpha : 1.0f;
    if (ep && !wgrad) {
        p.act = ep->activation;
        p.bias = ep->bias;
        p.bias_stride = ep->bias_stride;
    }
    p.err = hs.err;
    p.timeout_ns = opt && opt->timeout_ns ? opt->timeout_ns : HOST_TIMEOUT_NS;
    p.debug_stall = opt ? opt->debug_stall : 0;

    const int64_t depth = wgrad ? cdiv(S / groups, BK) : cdiv(K, BK);
    const int64_t share = share_of(wgrad, pair, units, depth, hs.sms);
    const int64_t splits = share == 0 ? 1 : std::min<int64_t>(SPLIT_MOST, cdiv(wgrad ? cdiv(S, BK) : depth, share));
    p.part_blocks = static_cast<int32_t>(share);
    p.splits = static_cast<int32_t>(splits);
    const int64_t part_tiles = splits > 1 ? units * (pair ? 2 : 1) : 0;
    const size_t part_bytes = static_cast<size_t>(part_tiles) * splits * BM * bn * 4;

    const bool reads = S > 0 && (wgrad || K > 0);
    if (b.nb > 1 && b.stride == 0) {  // one matrix for every group
        b.nb = 1;
        p.b_shared = 1;
    }
    CUtensorMap ta{}, tb{}, td{};
    if (reads) {
        const bool force = opt && opt->force_pack;
        a.pack = force || !tma_ok(a.p, a.ld, 0, 2);
        b.pack = force || !tma_ok(b.p, b.ld, b.nb > 1 ? b.stride : 0, 2);
        if ((st = realign(hs, a, b, part_bytes, &p.partials)) != TG_OK) return st;
        // rows mode: A is the MMA's N operand (this CTA's rows x 64 k), B[g] its
        // M operand (64 k x 64 columns, or 128 columns x 64 k)
        const uint32_t a_box1 = wgrad ? BK : static_cast<uint32_t>(pair ? bn / 2 : bn);
        const uint32_t b_box1 = b_k ? BM : BK;
        if (!host_encode_3d(&ta, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.p, a.cols, a.rows, a.nb, a.ld * 2, problem_stride(a), 64,
                            a_box1, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !host_encode_3d(&tb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, b.p, b.cols, b.rows, b.nb, b.ld * 2, problem_stride(b), 64,
                            b_box1, CU_TENSOR_MAP_SWIZZLE_128B))
            return TG_ERR_CUDA;
    }
    if (tma_ok(D, ldd, wgrad && groups > 1 ? strideD : 0, eb)) {
        const Operand d{D, wgrad ? M : S, N, ldd, wgrad ? groups : 1, strideD};
        const uint64_t s2 = static_cast<uint64_t>(d.nb > 1 ? strideD * eb : cdiv(d.rows * ldd * eb, 16) * 16);
        p.epi_tma = host_encode_3d(&td, out_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, D, d.cols,
                                   d.rows, d.nb, ldd * eb, s2, static_cast<uint32_t>(EPI_ROW_BYTES / eb), EPI_ROWS,
                                   CU_TENSOR_MAP_SWIZZLE_128B)
                        ? 1
                        : 0;
    }
    static const Shape shapes[5] = {shape<128, 6, false, false>(), shape<256, 6, true, false>(),
                                    shape<128, 6, false, true>(), shape<256, 6, true, true>(), shape<32, 9, false, false>()};
    static ShapeState states[5];
    const int which = few ? 4 : (wgrad ? 2 : 0) + (pair ? 1 : 0);
    if (splits > 1 && (st = host_counters(hs, static_cast<size_t>(part_tiles) * 4, &p.counters)) != TG_OK) return st;
    return host_cuda_status(launch_shape(shapes[which], states[which], hs, units * splits, ta, tb, td, p));
}

}  // namespace
}  // namespace tg

using namespace tg;

TG_API tg_status tg_gemm_grouped(const void *A, const void *B, void *D, const int32_t *offsets, int64_t groups, int64_t S,
                                 int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t strideB, int64_t ldd,
                                 const tg_epilogue *ep, tg_stream_t stream, const tg_options *opt)
{
    return host_guard([&] {
        if (groups < 1 || groups > GROUPED_EXTENT || !extent_ok(S) || !extent_ok(N) || !extent_ok(K)) return TG_ERR_INVALID_ARG;
        if (!options_ok(opt, false)) return TG_ERR_INVALID_ARG;
        const bool b_k = opt && opt->b_col_major;
        const int64_t b_rows = b_k ? N : K, b_cols = b_k ? K : N;
        if (!pitch_ok(lda, K) || !pitch_ok(ldb, b_cols) || !pitch_ok(ldd, N) || strideB < 0 || strideB > PITCH_LIMIT ||
            !span_ok(1, 0, S, lda) || !span_ok(groups, strideB, b_rows, ldb) || !span_ok(1, 0, S, ldd))
            return TG_ERR_INVALID_ARG;
        if (ep && ((ep->out_type != TG_F32 && ep->out_type != TG_BF16) || ep->activation < TG_ACT_NONE ||
                   ep->activation > TG_ACT_SILU || ep->residual || (ep->bias && ep->bias_stride < 0)))
            return TG_ERR_INVALID_ARG;
        if (S == 0 || N == 0) return TG_OK;
        if (!offsets || !D || (K > 0 && (!A || !B))) return TG_ERR_INVALID_ARG;
        const int64_t eb = ep && ep->out_type == TG_BF16 ? 2 : 4;
        if (reinterpret_cast<uintptr_t>(D) % eb || reinterpret_cast<uintptr_t>(A) % 2 || reinterpret_cast<uintptr_t>(B) % 2 ||
            !host_words_ok(offsets, ep ? ep->bias : nullptr))
            return TG_ERR_INVALID_ARG;
        const Bytes d = bytes_of(D, 1, 0, S, ldd, N, eb);
        if (meets(d, bytes_of(A, 1, 0, S, lda, K, 2)) || meets(d, bytes_of(B, groups, strideB, b_rows, ldb, b_cols, 2)) ||
            meets(d, bytes_of(offsets, 1, 0, 1, 0, groups + 1, 4)))
            return TG_ERR_INVALID_ARG;
        return run_grouped(false, Operand{A, S, K, lda, 1, 0}, Operand{B, b_rows, b_cols, ldb, groups, strideB}, b_k, D, offsets,
                           groups, S, 0, N, K, ldd, 0, ep, opt, reinterpret_cast<cudaStream_t>(stream));
    });
}

TG_API tg_status tg_gemm_grouped_wgrad(const void *A, const void *B, void *D, const int32_t *offsets, int64_t groups, int64_t S,
                                       int64_t M, int64_t N, int64_t lda, int64_t ldb, int64_t ldd, int64_t strideD,
                                       const tg_epilogue *ep, tg_stream_t stream, const tg_options *opt)
{
    return host_guard([&] {
        if (groups < 1 || groups > GROUPED_EXTENT || !extent_ok(S) || !extent_ok(M) || !extent_ok(N)) return TG_ERR_INVALID_ARG;
        if (!options_ok(opt, true)) return TG_ERR_INVALID_ARG;
        if (!pitch_ok(lda, M) || !pitch_ok(ldb, N) || !pitch_ok(ldd, N) || strideD < 0 || strideD > PITCH_LIMIT ||
            !span_ok(1, 0, S, lda) || !span_ok(1, 0, S, ldb) || !span_ok(groups, strideD, M, ldd))
            return TG_ERR_INVALID_ARG;
        if (ep && ((ep->out_type != TG_F32 && ep->out_type != TG_BF16) || ep->activation != TG_ACT_NONE || ep->residual ||
                   ep->bias))
            return TG_ERR_INVALID_ARG;
        if (M == 0 || N == 0) return TG_OK;
        if (groups > 1 && strideD < (M - 1) * ldd + N) return TG_ERR_INVALID_ARG;
        if (!offsets || !D || (S > 0 && (!A || !B))) return TG_ERR_INVALID_ARG;
        const int64_t eb = ep && ep->out_type == TG_BF16 ? 2 : 4;
        if (reinterpret_cast<uintptr_t>(D) % eb || reinterpret_cast<uintptr_t>(A) % 2 || reinterpret_cast<uintptr_t>(B) % 2 ||
            !host_words_ok(offsets))
            return TG_ERR_INVALID_ARG;
        const Bytes d = bytes_of(D, groups, strideD, M, ldd, N, eb);
        if (meets(d, bytes_of(A, 1, 0, S, lda, M, 2)) || meets(d, bytes_of(B, 1, 0, S, ldb, N, 2)) ||
            meets(d, bytes_of(offsets, 1, 0, 1, 0, groups + 1, 4)))
            return TG_ERR_INVALID_ARG;
        return run_grouped(true, Operand{A, S, M, lda, 1, 0}, Operand{B, S, N, ldb, 1, 0}, false, D, offsets, groups, S, M, N, 0,
                           ldd, strideD, ep, opt, reinterpret_cast<cudaStream_t>(stream));
    });
}
