// Products with 4-bit weights and group scales for a few rows of 16-bit
// activations (single tokens), dense or per group of rows (experts).  Entry
// point and formula: include/tg_gemm.h.
//
// The weights are the traffic (half a byte each, read once), so the bound is
// HBM; at that rate an SM has to turn about 47 codes a clock into products.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "tg_gemm.h"
#include "tg_host_api.h"
#include "tg_ptx.cuh"

#define TG_API extern "C" __attribute__((visibility("default")))

namespace tg {
namespace {

struct W4Args {
    const uint16_t *x;      // [S, K] bf16
    const uint8_t *w;       // [groups][N][K / 2] packed codes
    const uint8_t *scales;  // [groups][N][runs]: bf16 (int4) or E8M0 bytes (e2m1)
    const uint8_t *zeros;   // [groups][N][runs] or null
    const int32_t *offsets; // [groups + 1] or null: one group of all rows
    void *y;                // [S, N]
    int64_t ldx;            // elements
    int64_t ldw, stride_w;  // bytes
    int64_t lds, stride_s;  // elements
    int64_t ldz, stride_z;
    int64_t ldy;
    int32_t groups, S, N, K, runs, run;  // run: codes of a scale (32, 64, 128)
    int32_t y_bf16;
};

// Group number `nth` among those with rows, and its rows; false past the
// last.  Whole warps; bounds are clamped to [0, S].
__device__ __forceinline__ bool nth_group(const W4Args &a, int32_t nth, int32_t &g, int32_t &lo, int32_t &hi)
{
    if (!a.offsets) {
        g = 0;
        lo = 0;
        hi = a.S;
        return nth == 0;
    }
    const int lane = static_cast<int>(threadIdx.x & 31);
    for (int32_t base = 0; base < a.groups; base += 32) {
        const int32_t e = base + lane;
        int32_t l = 0, h = 0;
        if (e < a.groups) {
            l = max(0, min(__ldg(a.offsets + e), a.S));
            h = max(l, min(__ldg(a.offsets + e + 1), a.S));
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, h > l);
        const int32_t count = __popc(mask);
        if (nth >= count) {
            nth -= count;
            continue;
        }
        const bool mine = h > l && __popc(mask & ((1u << lane) - 1u)) == nth;
        const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        g = base + src;
        lo = __shfl_sync(0xffffffffu, l, src);
        hi = __shfl_sync(0xffffffffu, h, src);
        return true;
    }
    return false;
}

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// 2^(e - 127), e = 255: NaN (the encoding of a float's exponent, but for
// e = 0, whose 2^-127 is a subnormal).
__device__ __forceinline__ float e8m0_value(uint32_t e)
{
    return e == 255u ? __uint_as_float(0x7fc00000u) : e == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23);
}

// The value of an E2M1 code: sign, two exponent bits (bias 1), one mantissa bit.
__device__ __forceinline__ float e2m1_value(uint32_t q)
{
    const uint32_t e = (q >> 1) & 3u, m = q & 1u;
    const float v = e == 0u ? 0.5f * static_cast<float>(m) : static_cast<float>((2u + m) << e) * 0.25f;
    return (q & 8u) ? -v : v;
}

__device__ __forceinline__ void store_y(const W4Args &a, int64_t row, int64_t n, float v)
{
    if (a.y_bf16)
        static_cast<__nv_bfloat16 *>(a.y)[row * a.ldy + n] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(a.y)[row * a.ldy + n] = v;
}

// Rows of no group: zeros in columns [n0, n1).
__device__ __forceinline__ void zero_rows(const W4Args &a, int32_t n0, int32_t n1)
{
    if (!a.offsets) return;
    const int32_t first = max(0, min(__ldg(a.offsets), a.S));
    const int32_t last = max(first, min(__ldg(a.offsets + a.groups), a.S));
    for (int32_t i = 0; i < first + (a.S - last); ++i) {
        const int64_t row = i < first ? i : last + (i - first);
        for (int32_t n = n0 + static_cast<int32_t>(threadIdx.x); n < n1; n += static_cast<int32_t>(blockDim.x))
            store_y(a, row, n, 0.0f);
    }
}

// Any layout and alignment: a warp per column n, a lane per byte of codes,
// four rows at a time.  (code - zero) * scale and its product with an
// activation are exact in fp32 (5 + 8 and 8 bits), so only the sum rounds.
constexpr int ANY_COLS = 8;

template <bool E2M1>
__global__ void __launch_bounds__(ANY_COLS * 32) w4_any_kernel(const W4Args a)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int32_t n0 = static_cast<int32_t>(blockIdx.x) * ANY_COLS;
    const int32_t n = n0 + static_cast<int32_t>(threadIdx.x >> 5);
    if (blockIdx.y == 0) zero_rows(a, n0, min(n0 + ANY_COLS, a.N));
    int32_t g, lo, hi;
    if (!nth_group(a, static_cast<int32_t>(blockIdx.y), g, lo, hi) || n >= a.N) return;
    const uint8_t *w = a.w + g * a.stride_w + n * a.ldw;
    const int64_t s0 = g * a.stride_s + n * a.lds, z0 = g * a.stride_z + n * a.ldz;
    for (int32_t r0 = lo; r0 < hi; r0 += 4) {
        float acc[4] = {};
        for (int32_t b = lane; b < a.K / 2; b += 32) {
            const uint32_t q = w[b];
            const int32_t r = 2 * b / a.run;
            float v0, v1;
            if constexpr (E2M1) {
                const float s = e8m0_value(a.scales[s0 + r]);
                v0 = e2m1_value(q & 15u) * s;
                v1 = e2m1_value(q >> 4) * s;
            } else {
                const float s = bf16_value(reinterpret_cast<const uint16_t *>(a.scales)[s0 + r]);
                const float z = a.zeros ? static_cast<float>(a.zeros[z0 + r] & 15u) : 8.0f;
                v0 = (static_cast<float>(q & 15u) - z) * s;
                v1 = (static_cast<float>(q >> 4) - z) * s;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (r0 + i < hi) {
                    const uint16_t *x = a.x + (r0 + i) * a.ldx + 2 * b;
                    acc[i] = fmaf(v0, bf16_value(x[0]), acc[i]);
                    acc[i] = fmaf(v1, bf16_value(x[1]), acc[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], d);
            if (lane == 0 && r0 + i < hi) store_y(a, r0 + i, n, acc[i]);
        }
    }
}

template <class... P, class... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

constexpr int64_t LIMIT = INT32_MAX - 1024;
constexpr int64_t PITCH_LIMIT = int64_t(1) << 40;

struct Bytes {
    uintptr_t lo = 0, hi = 0;
};
Bytes bytes_of(const void *p, int64_t nb, int64_t stride, int64_t rows, int64_t ld, int64_t cols, int64_t size)
{
    if (!p || nb < 1 || rows < 1 || cols < 1) return {};
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return {b, b + static_cast<uintptr_t>(((nb - 1) * stride + (rows - 1) * ld + cols) * size)};
}
bool meets(const Bytes &a, const Bytes &b) { return a.lo < b.hi && b.lo < a.hi; }

bool pitch_ok(int64_t ld, int64_t cols, int64_t stride)
{
    return ld >= cols && ld <= PITCH_LIMIT && stride >= 0 && stride <= PITCH_LIMIT;
}

}  // namespace
}  // namespace tg

using namespace tg;

TG_API tg_status tg_gemv_w4(const void *x, int64_t ldx, const void *W, int64_t ldw, int64_t strideW, const void *scales,
                            int64_t ld_s, int64_t stride_s, const uint8_t *zeros, int64_t ld_z, int64_t stride_z,
                            int32_t format, int32_t group_size, const int32_t *offsets, int64_t groups, int64_t S, int64_t N,
                            int64_t K, void *y, int64_t ldy, int32_t y_type, tg_stream_t stream)
{
    return host_guard([&] {
        if (groups < 1 || groups > LIMIT || S < 0 || S > LIMIT || N < 0 || N > LIMIT || K < 0 || K > LIMIT || K % 2 != 0)
            return TG_ERR_INVALID_ARG;
        if ((format != TG_W4_INT4 && format != TG_W4_E2M1) || (y_type != TG_F32 && y_type != TG_BF16)) return TG_ERR_INVALID_ARG;
        if (format == TG_W4_E2M1 ? (group_size != 32 || zeros) : (group_size != 32 && group_size != 64 && group_size != 128))
            return TG_ERR_INVALID_ARG;
        const int64_t runs = (K + group_size - 1) / group_size;
        if (!pitch_ok(ldx, K, 0) || !pitch_ok(ldw, K, strideW) || ldw % 2 != 0 || strideW % 2 != 0 || !pitch_ok(ld_s, runs, stride_s) ||
            (zeros && !pitch_ok(ld_z, runs, stride_z)) || !pitch_ok(ldy, N, 0))
            return TG_ERR_INVALID_ARG;
        if (groups > 1 && !offsets) return TG_ERR_INVALID_ARG;
        if (S == 0 || N == 0) return TG_OK;
        if (!y || (K > 0 && (!x || !W || !scales))) return TG_ERR_INVALID_ARG;
        const int64_t yb = y_type == TG_BF16 ? 2 : 4, sb = format == TG_W4_E2M1 ? 1 : 2;
        if (reinterpret_cast<uintptr_t>(y) % yb || reinterpret_cast<uintptr_t>(x) % 2 || reinterpret_cast<uintptr_t>(scales) % sb)
            return TG_ERR_INVALID_ARG;
        const Bytes out = bytes_of(y, 1, 0, S, ldy, N, yb);
        if (meets(out, bytes_of(x, 1, 0, S, ldx, K, 2)) || meets(out, bytes_of(W, groups, strideW / 2, N, ldw / 2, K / 2, 1)) ||
            meets(out, bytes_of(scales, groups, stride_s, N, ld_s, runs, sb)) ||
            meets(out, bytes_of(zeros, groups, stride_z, N, ld_z, runs, 1)) || meets(out, bytes_of(offsets, 1, 0, 1, 0, groups + 1, 4)))
            return TG_ERR_INVALID_ARG;
        W4Args a{};
        a.x = static_cast<const uint16_t *>(x);
        a.w = static_cast<const uint8_t *>(W);
        a.scales = static_cast<const uint8_t *>(scales);
        a.zeros = zeros;
        a.offsets = offsets;
        a.y = y;
        a.ldx = ldx;
        a.ldw = ldw / 2;
        a.stride_w = strideW / 2;
        a.lds = ld_s;
        a.stride_s = stride_s;
        a.ldz = ld_z;
        a.stride_z = stride_z;
        a.ldy = ldy;
        a.groups = static_cast<int32_t>(groups);
        a.S = static_cast<int32_t>(S);
        a.N = static_cast<int32_t>(N);
        a.K = static_cast<int32_t>(K);
        a.runs = static_cast<int32_t>(runs);
        a.run = group_size;
        a.y_bf16 = y_type == TG_BF16;
        const int64_t used = offsets ? (groups < S ? groups : S) : 1;  // groups with rows, at most
        if (used > 65535) return TG_ERR_UNSUPPORTED;
        const dim3 grid(static_cast<unsigned>((N + ANY_COLS - 1) / ANY_COLS), static_cast<unsigned>(used));
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        return host_cuda_status(format == TG_W4_E2M1 ? launch(w4_any_kernel<true>, grid, ANY_COLS * 32, 0, s, a)
                                                     : launch(w4_any_kernel<false>, grid, ANY_COLS * 32, 0, s, a));
    });
}
