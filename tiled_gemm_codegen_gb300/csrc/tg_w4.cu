// Products with 4-bit weights and group scales for a few rows of 16-bit
// activations (single tokens), dense or per group of rows (experts).  Entry
// point and formula: include/tg_gemm.h.
//
// The weights are the traffic (half a byte each, read once), so the bound is
// HBM; at that rate an SM has to turn about 47 codes a clock into products.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "tg_gemm.h"
#include "tg_host_api.h"
#include "tg_ptx.cuh"
#include "tg_sync.cuh"

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

// A run's scale f and its zero; s and z: where they lie.  A code's weight is
// code_value * f, which is exact in fp32, but past its largest value for the
// largest f; `late` is the part of f that goes on after the activation instead:
// all of it from 2^64, where only a product that overflows itself still does.
template <bool E2M1>
struct W4Run {
    float f, late, zero;
    __device__ __forceinline__ W4Run(const W4Args &a, int64_t s, int64_t z)
    {
        if constexpr (E2M1) {
            f = e8m0_value(a.scales[s]);
            zero = 0.0f;
        } else {
            f = bf16_value(reinterpret_cast<const uint16_t *>(a.scales)[s]);
            zero = a.zeros ? static_cast<float>(a.zeros[z] & 15u) : 8.0f;
        }
        late = fabsf(f) > 0x1p64f ? f : 1.0f;
        if (late != 1.0f) f = 1.0f;
    }
    __device__ __forceinline__ float weight(uint32_t q) const  // without `late`
    {
        if constexpr (E2M1)
            return e2m1_value(q) * f;
        else
            return (static_cast<float>(q) - zero) * f;
    }
};

__device__ __forceinline__ void store_y(const W4Args &a, int64_t row, int64_t n, float v)
{
    if (a.y_bf16)
        static_cast<__nv_bfloat16 *>(a.y)[row * a.ldy + n] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(a.y)[row * a.ldy + n] = v;
}

// Rows of no group: zeros in columns [n0, n1).
__device__ __forceinline__ void zero_rows(const W4Args &a, int32_t n0, int32_t n1, int32_t threads)
{
    if (!a.offsets) return;
    const int32_t first = max(0, min(__ldg(a.offsets), a.S));
    const int32_t last = max(first, min(__ldg(a.offsets + a.groups), a.S));
    for (int32_t i = 0; i < first + (a.S - last); ++i) {
        const int64_t row = i < first ? i : last + (i - first);
        for (int32_t n = n0 + static_cast<int32_t>(threadIdx.x); n < n1; n += threads)
            store_y(a, row, n, 0.0f);
    }
}

// Any layout and alignment: a warp per column n, eight codes a lane and turn,
// four rows at a time.  (code - zero) * scale and its product with an
// activation are exact in fp32 (5 + 8 and 8 bits), so only the sum rounds.
// Bound by its conversions and multiply-adds: 6 rows of 1964 codes (982-byte
// rows) x 2976, int4: 28.1 us.
constexpr int ANY_COLS = 8;

// The four bytes at p, of which the first `n` exist: one or two aligned words
// where they lie inside [lo, hi), else byte by byte.
__device__ __forceinline__ uint32_t load4_any(const uint8_t *p, int n, const uint8_t *lo, const uint8_t *hi)
{
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 3u);
    const uint8_t *a = p - off;
    if (n == 4 && a >= lo && a + 8 <= hi) {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(a);
        return off ? __funnelshift_r(w[0], w[1], 8 * off) : w[0];
    }
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) v |= static_cast<uint32_t>(p[i]) << (8 * i);
    return v;
}

template <bool E2M1>
__global__ void __launch_bounds__(ANY_COLS * 32) w4_any_kernel(const W4Args a)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int32_t n0 = static_cast<int32_t>(blockIdx.x) * ANY_COLS;
    const int32_t n = n0 + static_cast<int32_t>(threadIdx.x >> 5);
    if (blockIdx.y == 0) zero_rows(a, n0, min(n0 + ANY_COLS, a.N), static_cast<int32_t>(blockDim.x));
    int32_t g, lo, hi;
    if (!nth_group(a, static_cast<int32_t>(blockIdx.y), g, lo, hi) || n >= a.N) return;
    const uint8_t *w = a.w + g * a.stride_w + n * a.ldw;
    const uint8_t *w_lo = a.w, *w_hi = a.w + (a.groups - 1) * a.stride_w + (a.N - 1) * a.ldw + a.K / 2;
    const int64_t s0 = g * a.stride_s + n * a.lds, z0 = g * a.stride_z + n * a.ldz;
    const bool x4 = ((reinterpret_cast<uintptr_t>(a.x) | static_cast<uintptr_t>(2 * a.ldx)) & 3u) == 0;
    for (int32_t r0 = lo; r0 < hi; r0 += 4) {
        float acc[4] = {};
#pragma unroll 2
        for (int32_t k = lane * 8; k < a.K; k += 256) {
            const int32_t left = min(8, a.K - k);
            const uint32_t q = load4_any(w + k / 2, left / 2, w_lo, w_hi);
            const int32_t r = k / a.run;
            float v[8];
            const W4Run<E2M1> run(a, s0 + r, z0 + r);
#pragma unroll
            for (int b = 0; b < 8; ++b) v[b] = run.weight(q >> (4 * b) & 15u);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (r0 + i >= hi) break;
                const uint16_t *x = a.x + (r0 + i) * a.ldx + k;
                if (run.late != 1.0f) {
                    for (int b = 0; b < left; ++b) acc[i] = fmaf(run.weight(q >> (4 * b) & 15u) * bf16_value(x[b]), run.late, acc[i]);
                } else if (x4 && left == 8) {
                    uint32_t h[4];
#pragma unroll
                    for (int b = 0; b < 4; ++b) h[b] = __ldg(reinterpret_cast<const uint32_t *>(x) + b);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        acc[i] = fmaf(v[2 * b], __uint_as_float(h[b] << 16), acc[i]);
                        acc[i] = fmaf(v[2 * b + 1], __uint_as_float(h[b] & 0xffff0000u), acc[i]);
                    }
                } else {
#pragma unroll
                    for (int b = 0; b < 8; ++b)
                        if (b < left) acc[i] = fmaf(v[b], bf16_value(x[b]), acc[i]);
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

// Whole warp: <x[row], w_g[n]> over [k0, k1) value by value, for any values.
template <bool E2M1>
__device__ __forceinline__ float row_dot(const W4Args &a, int32_t g, int32_t n, int32_t row, int32_t k0, int32_t k1)
{
    const uint8_t *w = a.w + g * a.stride_w + n * a.ldw;
    const int64_t s0 = g * a.stride_s + n * a.lds, z0 = g * a.stride_z + n * a.ldz;
    const uint16_t *x = a.x + row * a.ldx;
    float acc = 0.0f;
    for (int32_t b = k0 / 2 + static_cast<int32_t>(threadIdx.x & 31); b < k1 / 2; b += 32) {
        const uint32_t q = w[b];
        const W4Run<E2M1> run(a, s0 + 2 * b / a.run, z0 + 2 * b / a.run);
        acc = fmaf(run.weight(q & 15u) * bf16_value(x[2 * b]), run.late, acc);
        acc = fmaf(run.weight(q >> 4) * bf16_value(x[2 * b + 1]), run.late, acc);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
    return acc;
}

// ------------------------------------------------------------ tile kernel
// For weights and activations whose rows lie on 4 bytes but not on TMA's 16.
// A CTA computes W4_ROWS weight rows x up to 8 activation rows.  Its warps
// share the rows and split K: a warp takes every WARPS-th step of 256 codes
// (128 bytes of each weight row), so that together they read long pieces of
// each row, and their fp32 sums are added in a fixed order at the end.
//
// The product is mma.sync m16n8k16 (bf16 in, fp32 sums) with the weights as
// the 16-row operand: its operands are registers, so a code goes from its
// staged word to the tensor core without another trip through shared memory,
// which a tcgen05 operand would need; at one to eight rows the tensor work is
// a small part of either's rate and HBM is the bound.
//
// A sum over k may take its terms in any order, so the k index of an operand
// slot is chosen to suit the packing: within 32 consecutive codes lane (g, c)
// = (lane / 4, lane % 4) owns the eight codes of one 32-bit word, c of the
// four, and slots (2c, 2c + 1), (2c + 8, 2c + 9) of two k steps are its nibble
// pairs (0, 4), (1, 5) and (2, 6), (3, 7) - the pairs that one mask of the
// word leaves in the two halves of a register.  The activations are paired
// the same way.
//
// A code becomes bf16 exactly: 0x4300 | q is 128 + q, minus 128 + z (the integer
// as mantissa bits of a constant that is then subtracted, the usual conversion by
// a magic number; for weights of few bits see Kim et al., arXiv 2211.10017); an E2M1
// code's three low bits sit on bf16's exponent and mantissa as its value times
// 2^-126 (0.5 is a subnormal), and a product by 2^126 restores it.  The sum of
// a group of codes is multiplied by its scale once, in fp32.
//
// Weights, activations, scales and zeros of a step travel through a ring of
// STAGES slots per warp by cp.async; no warp waits for another before the end.
// 4 rows of 7800 codes (3900-byte rows) x 6401, int4 with zeros by 64: 23 us,
// 27 MB at 1.2 TB/s: a copy instruction moves a quarter of what 16-byte rows
// would allow.
constexpr int W4_WARPS = 8;                // 4 where the ring holds eight activation rows
constexpr int W4_STAGES = 3;
constexpr int W4_MT = 2;                   // 16-row blocks a warp
constexpr int W4_ROWS = 16 * W4_MT;
constexpr int W4_STEP = 256;               // codes of a step
constexpr int W4_PITCH = W4_STEP / 2 + 16; // staged weight row: the 8 rows of a load fall in 32 different banks
constexpr int W4_XPITCH = 2 * W4_STEP + 64;

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Plain loads (not volatile): the compiler may move them ahead of the
// products before them, though not across the waits, which clobber memory.
__device__ __forceinline__ uint32_t lds32(const uint8_t *a) { return *reinterpret_cast<const uint32_t *>(a); }
__device__ __forceinline__ uint4 lds128(const uint8_t *a) { return *reinterpret_cast<const uint4 *>(a); }
__device__ __forceinline__ uint32_t lds_u16(const uint8_t *a) { return *reinterpret_cast<const uint16_t *>(a); }
__device__ __forceinline__ uint32_t lds_u8(const uint8_t *a) { return *a; }

// d (+)= a b; the first product of a sum takes no accumulator.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool first)
{
    if (first)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A constant the compiler keeps in a register: (w & mask) | magic is one
// instruction with one immediate and one register operand, two with two
// immediates.
__device__ __forceinline__ uint32_t in_register(uint32_t v)
{
    uint32_t r;
    asm volatile("mov.b32 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
template <uint32_t MASK>
__device__ __forceinline__ uint32_t masked_or(uint32_t w, uint32_t c)  // (w & MASK) | c
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t bf2_sub(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Nibbles (i, i + 4) of a word as two bf16, i = 0 .. 3.  magic: 0x4300 twice
// (int4) or 2^126 twice (e2m1); zz: (128 + zero) twice.
template <bool E2M1>
__device__ __forceinline__ void decode(uint32_t w, uint32_t magic, uint32_t zz, uint32_t (&p)[4])
{
    if constexpr (E2M1) {
        p[0] = bf2_mul(masked_or<0x01C001C0u>(w << 6, (w << 12) & 0x80008000u), magic);
        p[1] = bf2_mul(masked_or<0x01C001C0u>(w << 2, (w << 8) & 0x80008000u), magic);
        p[2] = bf2_mul(masked_or<0x01C001C0u>(w >> 2, (w << 4) & 0x80008000u), magic);
        p[3] = bf2_mul(masked_or<0x01C001C0u>(w >> 6, w & 0x80008000u), magic);
    } else {
        p[0] = bf2_sub(masked_or<0x000F000Fu>(w, magic), zz);
        p[1] = bf2_sub(masked_or<0x000F000Fu>(w >> 4, magic), zz);
        p[2] = bf2_sub(masked_or<0x000F000Fu>(w >> 8, magic), zz);
        p[3] = bf2_sub(masked_or<0x000F000Fu>(w >> 12, magic), zz);
    }
}

__host__ __device__ constexpr int w4_warps(int xt) { return xt > 4 ? W4_WARPS / 2 : W4_WARPS; }

// Staged scale words of a row and step: its bytes from the 4-byte boundary
// before them.
template <bool E2M1, int RUN>
struct W4Layout {
    static constexpr int PER_STEP = W4_STEP / RUN;
    static constexpr int SB = E2M1 ? 1 : 2;
    static constexpr int S_WORDS = (PER_STEP * SB + 3) / 4 + 1;
    static constexpr int Z_WORDS = (PER_STEP + 3) / 4 + 1;
    static constexpr int stage(int xt, bool zeros)
    {
        return W4_ROWS * W4_PITCH + xt * W4_XPITCH + (W4_ROWS * 4 * (S_WORDS + (zeros ? Z_WORDS : 0)) + 15) / 16 * 16;
    }
    static constexpr int smem(int xt, bool zeros)  // the sums reuse the ring
    {
        return w4_warps(xt) * W4_STAGES * stage(xt, zeros);
    }
    static_assert(W4_STAGES * (W4_ROWS * W4_PITCH) >= W4_ROWS * 8 * 4, "room for a warp's sums");
};

// xt: activation rows the ring has room for (1 .. 8).
template <bool E2M1, int RUN, bool ZEROS>
__global__ void __launch_bounds__(W4_WARPS * 32, 1) w4_tile_kernel(const W4Args a, int xt)
{
    using L = W4Layout<E2M1, RUN>;
    extern __shared__ __align__(16) uint8_t smem[];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lg = lane >> 2, lc = lane & 3;
    const uint32_t magic = in_register(E2M1 ? 0x7E807E80u : 0x43004300u), eight = in_register(0x43084308u);
    const int warps = static_cast<int>(blockDim.x >> 5);
    const int32_t n0 = static_cast<int32_t>(blockIdx.x) * W4_ROWS;
    if (blockIdx.y == 0) zero_rows(a, n0, min(n0 + W4_ROWS, a.N), static_cast<int32_t>(blockDim.x));
    int32_t grp, lo, hi;
    if (!nth_group(a, static_cast<int32_t>(blockIdx.y), grp, lo, hi)) return;
    const uint8_t *w0 = a.w + grp * a.stride_w + n0 * a.ldw;
    const uint8_t *s0 = a.scales + (grp * a.stride_s + n0 * a.lds) * L::SB;
    const uint8_t *z0 = ZEROS ? a.zeros + grp * a.stride_z + n0 * a.ldz : nullptr;
    const int32_t rows = min(W4_ROWS, a.N - n0);
    const int stage = L::stage(xt, ZEROS);
    uint8_t *const ring_p = smem + warp * W4_STAGES * stage;
    const uint32_t ring = ptx::smem_addr(ring_p);
    const uint32_t off_x = W4_ROWS * W4_PITCH, off_s = off_x + xt * W4_XPITCH, off_z = off_s + W4_ROWS * 4 * L::S_WORDS;
    const int32_t steps = (a.K + W4_STEP - 1) / W4_STEP;
    const int32_t mine = steps > warp ? (steps - warp + warps - 1) / warps : 0;
    const int32_t row_bytes = a.K / 2;
    const int32_t s_bytes = a.runs * L::SB;

    for (int32_t r0 = lo; r0 < hi; r0 += xt) {
        const int32_t nx = min(xt, hi - r0);
        auto fill = [&](int32_t i) {  // step i of this warp -> slot i mod STAGES
            const uint32_t dst = ring + static_cast<uint32_t>(i % W4_STAGES * stage);
            const int32_t k0 = (warp + i * warps) * W4_STEP;
            for (int r = 0; r < rows; ++r) {
                const int32_t left = row_bytes - (k0 / 2 + lane * 4);
                cp_async4(dst + r * W4_PITCH + lane * 4, w0 + r * a.ldw + (left > 0 ? k0 / 2 + lane * 4 : 0), max(0, min(4, left)));
            }
            for (int t = 0; t < nx; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int32_t xl = 2 * min(a.K - k0, W4_STEP) - (j * 32 + lane) * 4;
                    cp_async4(dst + off_x + t * W4_XPITCH + (j * 32 + lane) * 4,
                              a.x + (r0 + t) * a.ldx + (xl > 0 ? k0 + (j * 32 + lane) * 2 : 0), max(0, min(4, xl)));
                }
            const int32_t at = k0 / RUN;
            for (int j = lane; j < W4_ROWS * L::S_WORDS; j += 32) {
                const int r = j / L::S_WORDS, word = j % L::S_WORDS;
                if (r < rows) {
                    const uint8_t *p = s0 + (r * a.lds + at) * L::SB;
                    const uint8_t *src = p - (reinterpret_cast<uintptr_t>(p) & 3u) + word * 4;
                    const int64_t left = (s0 + r * a.lds * L::SB + s_bytes) - src;
                    cp_async4(dst + off_s + j * 4, left > 0 ? src : a.scales, static_cast<int>(left < 0 ? 0 : left > 4 ? 4 : left));
                }
            }
            if constexpr (ZEROS) {
                for (int j = lane; j < W4_ROWS * L::Z_WORDS; j += 32) {
                    const int r = j / L::Z_WORDS, word = j % L::Z_WORDS;
                    if (r < rows) {
                        const uint8_t *p = z0 + r * a.ldz + at;
                        const uint8_t *src = p - (reinterpret_cast<uintptr_t>(p) & 3u) + word * 4;
                        const int64_t left = (z0 + r * a.ldz + a.runs) - src;
                        cp_async4(dst + off_z + j * 4, left > 0 ? src : a.zeros, static_cast<int>(left < 0 ? 0 : left > 4 ? 4 : left));
                    }
                }
            }
        };
        float acc[W4_MT][4] = {};
#pragma unroll
        for (int i = 0; i < W4_STAGES - 1; ++i) {
            if (i < mine) fill(i);
            cp_async_commit();
        }
        for (int32_t i = 0; i < mine; ++i) {
            if (i + W4_STAGES - 1 < mine) fill(i + W4_STAGES - 1);
            cp_async_commit();
            cp_async_wait<W4_STAGES - 1>();
            __syncwarp();
            const uint8_t *src = ring_p + i % W4_STAGES * stage;
            const int32_t k0 = (warp + i * warps) * W4_STEP;
            const int32_t at = k0 / RUN;
            const uint8_t *s_row[2 * W4_MT], *z_row[2 * W4_MT];
#pragma unroll
            for (int h = 0; h < 2 * W4_MT; ++h) {  // rows lg + 8h
                const int r = lg + 8 * h;
                s_row[h] = src + off_s + r * 4 * L::S_WORDS +
                           static_cast<uint32_t>(reinterpret_cast<uintptr_t>(s0 + (r * a.lds + at) * L::SB) & 3u);
                if constexpr (ZEROS)
                    z_row[h] = src + off_z + r * 4 * L::Z_WORDS + static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z0 + r * a.ldz + at) & 3u);
            }
#pragma unroll
            for (int j = 0; j < L::PER_STEP; ++j) {
                if (k0 + j * RUN >= a.K) break;
                float part[W4_MT][4];
                uint32_t zz[2 * W4_MT];
#pragma unroll
                for (int h = 0; h < 2 * W4_MT; ++h)
                    zz[h] = ZEROS ? (0x4300u | (lds_u8(z_row[h] + j) & 15u)) * 0x00010001u : eight;
#pragma unroll
                for (int b = 0; b < RUN / 32; ++b) {
                    const int blk = j * (RUN / 32) + b;
                    // (an operand column of no row repeats row 0's: its sums are not stored)
                    const uint4 xv = lds128(src + off_x + (lg < nx ? lg : 0) * W4_XPITCH + blk * 64 + lc * 16);
                    const uint32_t x0 = __byte_perm(xv.x, xv.z, 0x5410), x1 = __byte_perm(xv.x, xv.z, 0x7632);
                    const uint32_t x2 = __byte_perm(xv.y, xv.w, 0x5410), x3 = __byte_perm(xv.y, xv.w, 0x7632);
#pragma unroll
                    for (int m = 0; m < W4_MT; ++m) {
                        uint32_t u[4], v[4];
                        const uint8_t *wa = src + (m * 16 + lg) * W4_PITCH + blk * 16 + lc * 4;
                        decode<E2M1>(lds32(wa), magic, zz[2 * m], u);
                        decode<E2M1>(lds32(wa + 8 * W4_PITCH), magic, zz[2 * m + 1], v);
                        const uint32_t a0[4] = {u[0], v[0], u[1], v[1]}, a1[4] = {u[2], v[2], u[3], v[3]};
                        mma_16816(part[m], a0, x0, x1, b == 0);
                        mma_16816(part[m], a1, x2, x3, false);
                    }
                }
#pragma unroll
                for (int m = 0; m < W4_MT; ++m) {
                    float sa, sb;
                    if constexpr (E2M1) {
                        sa = e8m0_value(lds_u8(s_row[2 * m] + j));
                        sb = e8m0_value(lds_u8(s_row[2 * m + 1] + j));
                    } else {
                        sa = bf16_value(static_cast<uint16_t>(lds_u16(s_row[2 * m] + 2 * j)));
                        sb = bf16_value(static_cast<uint16_t>(lds_u16(s_row[2 * m + 1] + 2 * j)));
                    }
                    acc[m][0] = fmaf(sa, part[m][0], acc[m][0]);
                    acc[m][1] = fmaf(sa, part[m][1], acc[m][1]);
                    acc[m][2] = fmaf(sb, part[m][2], acc[m][2]);
                    acc[m][3] = fmaf(sb, part[m][3], acc[m][3]);
                }
            }
            __syncwarp();
        }
        cp_async_wait<0>();
        __syncthreads();
        // sums[warp][x row][weight row]; then added over the warps in order
        float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int m = 0; m < W4_MT; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sums[(warp * 8 + 2 * lc + (i & 1)) * W4_ROWS + m * 16 + lg + 8 * (i >> 1)] = acc[m][i];
        __syncthreads();
        for (int i = threadIdx.x; i < nx * W4_ROWS; i += static_cast<int>(blockDim.x)) {
            const int t = i / W4_ROWS, n = i % W4_ROWS;
            float sum = 0.0f;
            for (int v = 0; v < warps; ++v) sum += sums[(v * 8 + t) * W4_ROWS + n];
            // A group's sum may overflow before its scale brings it back: what is not
            // finite (a warp holds one activation row's) is summed value by value.
            for (uint32_t left = __ballot_sync(0xffffffffu, n < rows && !isfinite(sum)); left; left &= left - 1) {
                const int at = __ffs(left) - 1;
                const float v = row_dot<E2M1>(a, grp, n0 + at, r0 + t, 0, a.K);
                if (n == at) sum = v;
            }
            if (n < rows) store_y(a, r0 + t, n0 + n, sum);
        }
        if (r0 + xt < hi) __syncthreads();  // the ring is filled again
    }
}

// ------------------------------------------------------------ stream kernel
// The same product for weights that TMA can address.  K is cut into slices
// (one where that is best) whose activations fit shared memory; products of a
// slice are added by w4_join_kernel.  One CTA per SM walks a contiguous range
// of tiles (32 weight rows for each of its teams of `wk` warps, which share a
// slice of K step by step); a producer warp keeps `stages` TMA boxes of 32 rows x 256 codes in
// flight for each of them, across the ends of tiles, so the weights never stop
// and a step costs the others one wait and one arrival.  What a tile needs
// besides is loaded once or ahead: the activations of a group in the order
// the products want, the scales of the next tile by cp.async during this
// one.
//
// The arithmetic is the tile kernel's: a code becomes the exact bf16 value of q -
// z, or of E2M1, activations stay the bf16 they are, a group's products are summed
// in fp32 and multiplied by its scale once.  So nothing depends on the size of
// other values: weights of zero leave nothing of their activations, and infinities and
// NaN go through the products.  (fp16 operands take fewer steps apart - codes as
// subnormals, zero points as a difference of two sums - and 4 to 9% less time on
// int4, 1 to 3% on E2M1, but their error goes with sum |q x| and with the largest
// activation of 256: a channel of 2^40 over zero weights hid the others.)
// Rows with a finite magnitude from W4_LARGE are computed value by value, scale
// first.
//
// What bounds it is taking the codes apart (56% of issue slots).  Measured (calls
// on a graph, weights not in L2): 1 row, 8192 x 28672 int4 by 128, 121 MB: 28.8 us,
// a quarter of those 12.0: 5.4 TB/s between the two, and 6.4 us of start,
// first boxes, activations and last tiles; with zero points 31.4; E2M1,
// which has a scale for every 32 codes, 39.0.  32 rows over 20 of 64 experts, 2048 x
// 1408 E2M1, 31 MB: 19.4 us, of which the start and a CTA's few turns are
// most.  Tried: eight turns' activation loads in flight instead of four (3-4
// us slower, registers), E2M1's sign moved by a multiply-add instead of a
// shift and mask (no change), the hardware's E2M1 conversion (twice the time).
//
// A box lies in shared memory with the 128-byte swizzle (16-byte unit u of
// row r at u ^ (r mod 8)), which puts the words of a block's eight rows in 32
// different banks.
struct W4Stream {
    int32_t xt;        // activation rows a pass
    int32_t warps, wk; // warps of the CTA, and of a team
    int32_t stages;
    int32_t steps;     // of 256 codes, of a slice
    int32_t all_steps, slices;
    int32_t tiles_n;   // tiles of a group
    int32_t w_shared;  // every group has the same weights
    int32_t x_pitch;   // bytes of an activation row in shared memory
    int32_t s_words, z_words;  // staged words of a row's scales and zeros
    int32_t off_x, off_s, off_z, off_sum;  // bytes in shared memory after the rings
    int32_t s_vec;             // every row of scales starts on 4 bytes
    float *partials;           // slices > 1: [slice][S][N]
    uint32_t *err;
    uint64_t timeout_ns;
#ifdef TG_DEBUG_CHECKS
    int32_t stall;  // watchdog self-test: the first warp's boxes are never asked for
#endif
};

constexpr int W4S_ROWS = 32;
constexpr int W4S_BOX = W4S_ROWS * W4_STEP / 2;  // 4 KB
constexpr int W4S_WARPS = 16;
constexpr int W4S_STAGES = 4;
constexpr int W4S_STATIC = 2048;  // static shared memory, rounded up
constexpr int W4S_SLICES = 32;
constexpr int64_t W4S_SCRATCH = int64_t(64) << 20;  // of partial sums, at most

// Pass `nth` over the groups' rows, at most xt rows each: its group, first
// row and number of rows; false past the last.  Whole warps.
__device__ __forceinline__ bool nth_pass(const W4Args &a, int32_t xt, int32_t nth, int32_t &g, int32_t &r0, int32_t &nx)
{
    if (!a.offsets) {
        g = 0;
        r0 = nth * xt;
        nx = min(xt, a.S - r0);
        return r0 < a.S;
    }
    const int lane = static_cast<int>(threadIdx.x & 31);
    for (int32_t base = 0; base < a.groups; base += 32) {
        const int32_t e = base + lane;
        int32_t l = 0, h = 0;
        if (e < a.groups) {
            l = max(0, min(__ldg(a.offsets + e), a.S));
            h = max(l, min(__ldg(a.offsets + e + 1), a.S));
        }
        const int32_t passes = (h - l + xt - 1) / xt;
        int32_t incl = passes;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        const int32_t count = __shfl_sync(0xffffffffu, incl, 31);
        if (nth >= count) {
            nth -= count;
            continue;
        }
        const int src = __popc(__ballot_sync(0xffffffffu, nth >= incl));
        g = base + src;
        const int32_t first = nth - (__shfl_sync(0xffffffffu, incl, src) - __shfl_sync(0xffffffffu, passes, src));
        r0 = __shfl_sync(0xffffffffu, l, src) + first * xt;
        nx = min(xt, __shfl_sync(0xffffffffu, h, src) - r0);
        return true;
    }
    return false;
}

// All passes over the groups' rows.  Whole warps.
__device__ __forceinline__ int32_t count_passes(const W4Args &a, int32_t xt)
{
    if (!a.offsets) return (a.S + xt - 1) / xt;
    int32_t sum = 0;
    for (int32_t e = static_cast<int32_t>(threadIdx.x & 31); e < a.groups; e += 32) {
        const int32_t l = max(0, min(__ldg(a.offsets + e), a.S));
        const int32_t h = max(l, min(__ldg(a.offsets + e + 1), a.S));
        sum += (h - l + xt - 1) / xt;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    return sum;
}

// Shared memory at a + OFF, neither volatile nor a memory access to the
// compiler: the caller orders them by what a and the results hang on.
__device__ __forceinline__ uint32_t shared_u32(uint32_t a, int off)
{
    uint32_t v;
    asm("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a + off));
    return v;
}
__device__ __forceinline__ uint4 shared_u128(uint32_t a, int off)
{
    uint4 v;
    asm("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a + off));
    return v;
}

// Activations from this magnitude, as bf16 bits, may add up to more than fp32's
// largest before their group's scale brings them back: 2^116 where a group of
// 128 has weights up to 15, 2^119 for 32 up to 6.
template <bool E2M1>
constexpr int32_t W4_LARGE = (127 + (E2M1 ? 119 : 116)) << 7;

template <bool E2M1, int RUN, bool ZEROS>
__global__ void __launch_bounds__((W4S_WARPS + 1) * 32, 1)
    w4_stream_kernel(const __grid_constant__ CUtensorMap tmW, const W4Args a, const W4Stream p)
{
    constexpr int SB = E2M1 ? 1 : 2;
    constexpr int RUNS = W4_STEP / RUN;        // of a step
    constexpr int SW = (RUNS * 2 + 3) / 4;     // registers of a step's scales of a row, bf16
    constexpr int SBYTES = RUNS * SB;          // as staged
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * W4S_WARPS * W4S_STAGES];  // a warp's full, then its empty ones
    __shared__ int32_t aborted;
    // The row holds a finite magnitude from W4_LARGE.  Two sets in turn:
    // the next pass's is cleared while warps may still be storing the last tile
    // of this one, which read this one's.
    __shared__ int32_t x_odd[2][8];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t base = ptx::smem_addr(smem);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = static_cast<int>(threadIdx.x & 31);
    const int lg = lane >> 2, lc = lane & 3;
    const uint32_t magic = in_register(E2M1 ? 0x7E807E80u : 0x43004300u), eight = in_register(0x43084308u);
    const int team = warp / p.wk, part_k = warp % p.wk;
    const int teams = p.warps / p.wk;
    const int tile_rows = teams * W4S_ROWS;
    const uint32_t ring = base + static_cast<uint32_t>(warp * p.stages * W4S_BOX);
    const uint32_t bars0 = ptx::smem_addr(bars), bar0 = bars0 + 16u * W4S_STAGES * warp;
    const int threads = p.warps * 32;  // without the producer's
    if (warp < p.warps && lane == 0) {
        for (int s = 0; s < p.stages; ++s) {
            ptx::mbar_init(bar0 + 8u * s, 1);
            ptx::mbar_init(bar0 + 8u * (W4S_STAGES + s), 1);
        }
        ptx::fence_barrier_init();
    }
    if (threadIdx.x == 0) {
        aborted = 0;
        ptx::prefetch_tensormap(&tmW);
    }
    __syncthreads();
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    auto clear = [&]() {  // this CTA's share of the rows of no group
        for (int32_t n = static_cast<int32_t>(blockIdx.x) * 256; n < a.N; n += static_cast<int32_t>(gridDim.x) * 256)
            zero_rows(a, n, min(n + 256, a.N), threads);
    };
    const int64_t tiles = static_cast<int64_t>(count_passes(a, p.xt)) * p.slices * p.tiles_n;
    // (a 64-bit division costs some hundred cycles of every call's start)
    int64_t first, last;
    if (tiles <= 0xFFFFFFFFll / 1024 && gridDim.x < 1024) {
        const uint32_t n = static_cast<uint32_t>(tiles);
        first = blockIdx.x * n / gridDim.x;
        last = (blockIdx.x + 1) * n / gridDim.x;
    } else {
        first = blockIdx.x * tiles / gridDim.x;
        last = (blockIdx.x + 1) * tiles / gridDim.x;
    }
    if (first == last) {
        if (warp < p.warps) clear();
        return;
    }
    // A tile by its pass, slice and place in it, stepped without a division.
    struct At {
        int32_t left, pass, slice, n;
        __device__ __forceinline__ void next(const W4Stream &p)
        {
            --left;
            if (++n == p.tiles_n) {
                n = 0;
                if (++slice == p.slices) {
                    slice = 0;
                    ++pass;
                }
            }
        }
    };
    const int32_t first_slice = static_cast<int32_t>(first <= INT32_MAX ? static_cast<int32_t>(first) / p.tiles_n : first / p.tiles_n);
    const int32_t first_pass = p.slices == 1 ? first_slice : first_slice / p.slices;
    const At at0{static_cast<int32_t>(last - first), first_pass, first_slice - first_pass * p.slices,
                 static_cast<int32_t>(first - static_cast<int64_t>(first_slice) * p.tiles_n)};
    if (warp == p.warps) {
        // ------------------------------------------------ producer
        // Lane l keeps warp l's ring full: a box at a time, whenever the
        // warp has freed its slot.
        const bool used = lane < p.warps;
        const int l_team = lane / p.wk, l_part = lane % p.wk;
        const uint32_t l_ring = base + static_cast<uint32_t>(lane * p.stages * W4S_BOX);
        const uint32_t l_full = bars0 + 16u * W4S_STAGES * lane, l_empty = l_full + 8u * W4S_STAGES;
        int32_t pass = at0.pass - 1, g = 0;
        uint32_t slot = 0, parity = 1;
        uint64_t t0 = 0;
        bool ok = true;
        for (At at = at0; ok && at.left > 0; at.next(p)) {
            if (at.pass != pass) {
                int32_t r, n;
                nth_pass(a, p.xt, at.pass, g, r, n);
                if (p.w_shared) g = 0;
                pass = at.pass;
            }
            const int32_t step0 = at.slice * p.steps;
            const int32_t each = (min(p.steps, p.all_steps - step0) - l_part + p.wk - 1) / p.wk;
            const int32_t n0 = at.n * tile_rows + l_team * W4S_ROWS;
            int32_t i = used ? 0 : each;  // boxes of the tile asked for
            while (__any_sync(0xffffffffu, i < each)) {
                bool moved = false;
                if (i < each && ptx::mbar_try_wait(l_empty + 8u * slot, parity)) {
#ifdef TG_DEBUG_CHECKS
                    if (!p.stall || lane > 0)
#endif
                    {
                        ptx::mbar_arrive_expect_tx(l_full + 8u * slot, W4S_BOX);
                        ptx::tma_load_3d(l_ring + slot * W4S_BOX, &tmW, l_full + 8u * slot, (step0 + l_part + i * p.wk) * (W4_STEP / 2), n0, g);
                    }
                    ++i;
                    moved = true;
                    if (++slot == static_cast<uint32_t>(p.stages)) {
                        slot = 0;
                        parity ^= 1u;
                    }
                }
                if (__any_sync(0xffffffffu, moved)) {
                    t0 = 0;
                } else {
                    const uint64_t now = ptx::global_timer_ns();
                    if (t0 == 0) t0 = now;
                    const bool late = now - t0 > p.timeout_ns;
                    if (late && lane == 0) {
                        atomicCAS(p.err, 0u, static_cast<uint32_t>(ERR_TIMEOUT_PRODUCER));
                        *reinterpret_cast<volatile int32_t *>(&aborted) = 1;
                    }
                    if (__any_sync(0xffffffffu, late || *reinterpret_cast<volatile int32_t *>(&aborted) != 0)) {
                        ok = false;
                        break;
                    }
                }
            }
        }
        // every box asked for has landed (bounded) before the CTA may leave
        t0 = ptx::global_timer_ns();
        if (used) {
            for (int s = 0; s < p.stages; ++s) {
                // the slot's last copy completed the phase before the one its
                // next use would wait for: slots before `slot` were used once more
                const uint32_t done = static_cast<uint32_t>(s) < slot ? parity ^ 1u : parity;
                while (!ptx::mbar_try_wait(l_full + 8u * s, done))
                    if (ptx::global_timer_ns() - t0 > p.timeout_ns) break;
            }
        }
        return;
    }
    int32_t g_next, r0_next, nx_next;  // the pass of the next tile
    nth_pass(a, p.xt, at0.pass, g_next, r0_next, nx_next);

    // ---- scales and zeros of a tile -> buffer b; a thread's first word and
    // its step to the next are the same for every tile
    const int32_t slice_runs = min(a.runs, p.steps * RUNS);
    const int32_t s_used = (slice_runs * SB + 3) / 4 + (p.s_vec ? 0 : 1), z_used = ZEROS ? (slice_runs + 3) / 4 + 1 : 1;
    const int32_t s_r = static_cast<int32_t>(threadIdx.x) / s_used, s_w = static_cast<int32_t>(threadIdx.x) - s_r * s_used;
    const int32_t s_dr = threads / s_used, s_dw = threads - s_dr * s_used;
    const int32_t z_r = static_cast<int32_t>(threadIdx.x) / z_used, z_w = static_cast<int32_t>(threadIdx.x) - z_r * z_used;
    const int32_t z_dr = threads / z_used, z_dw = threads - z_dr * z_used;
    auto stage_scales = [&](int32_t n0, int32_t g, int32_t slice, int b) {
        const int32_t rows = min(tile_rows, a.N - n0), from = slice * p.steps * RUNS, runs = min(slice_runs, a.runs - from);
        auto copy = [&](const uint8_t *src0, int64_t pitch, int32_t bytes, const uint8_t *any, int32_t used, int32_t words, uint32_t dst,
                        int32_t r, int32_t w, int32_t dr, int32_t dw) {
            while (r < rows) {
                const uint8_t *row = src0 + r * pitch;
                const int32_t off = static_cast<int32_t>(reinterpret_cast<uintptr_t>(row) & 3u);
                const int32_t left = bytes + off - w * 4;
                cp_async4(dst + (r * words + w) * 4, left > 0 ? row - off + w * 4 : any, max(0, min(4, left)));
                r += dr;
                w += dw;
                if (w >= used) {
                    w -= used;
                    ++r;
                }
            }
        };
        copy(a.scales + (g * a.stride_s + n0 * a.lds + from) * SB, a.lds * SB, runs * SB, a.scales, s_used, p.s_words,
             base + p.off_s + b * tile_rows * p.s_words * 4, s_r, s_w, s_dr, s_dw);
        if constexpr (ZEROS)
            copy(a.zeros + g * a.stride_z + n0 * a.ldz + from, a.ldz, runs, a.zeros, z_used, p.z_words,
                 base + p.off_z + b * tile_rows * p.z_words * 4, z_r, z_w, z_dr, z_dw);
    };

    // ---- activations of a pass: eight consecutive ones paired as the codes of a
    // word are.  A warp takes the 256 of a row and step.
    int32_t odd_set = 0;  // the set of x_odd in use
    auto stage_x = [&](int32_t r0, int32_t nx, int32_t k0, int32_t steps) {
        const bool aligned = ((reinterpret_cast<uintptr_t>(a.x) | static_cast<uintptr_t>(2 * a.ldx)) & 15u) == 0;
        constexpr int U = 4;  // turns whose loads are in flight together
        const int32_t turns = nx * steps;
        for (int32_t i0 = warp; i0 < turns; i0 += U * p.warps) {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int32_t i = i0 + u * p.warps;
                v[u] = make_uint4(0u, 0u, 0u, 0u);
                if (i >= turns) continue;
                const int32_t t = i / steps, k = k0 + ((i - t * steps) * 32 + lane) * 8;
                const uint16_t *row = a.x + (r0 + t) * a.ldx + k;
                if (aligned && k + 8 <= a.K) {
                    v[u] = *reinterpret_cast<const uint4 *>(row);
                } else if (k < a.K) {
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[e] = k + e < a.K ? row[e] : 0u;
                    v[u] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int32_t i = i0 + u * p.warps;
                if (i >= turns) break;
                const int32_t t = i / steps, c = (i - t * steps) * 32 + lane;
                const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
                bool large = false;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int32_t lo = static_cast<int32_t>(w[e] & 0x7fffu), hi = static_cast<int32_t>(w[e] >> 16 & 0x7fffu);
                    large |= (lo >= W4_LARGE<E2M1> && lo < 0x7f80) || (hi >= W4_LARGE<E2M1> && hi < 0x7f80);
                }
                if (large) x_odd[odd_set][t] = 1;
                *reinterpret_cast<uint4 *>(smem + p.off_x + t * p.x_pitch + c * 16) =
                    make_uint4(__byte_perm(w[0], w[2], 0x5410), __byte_perm(w[0], w[2], 0x7632), __byte_perm(w[1], w[3], 0x5410),
                               __byte_perm(w[1], w[3], 0x7632));
            }
        }
    };

    At at = at0;
    int32_t g, r0, nx;  // the tile's pass
    stage_scales(at.n * tile_rows, g_next, at.slice, 0);
    uint32_t slot = 0, parity = 0;  // of the next box
    bool fresh = true;  // the tile's activations are not in shared memory yet
    for (int b = 0; at.left > 0; b ^= 1) {
        if (fresh) {
            odd_set ^= 1;
            if (threadIdx.x < 8) x_odd[odd_set][threadIdx.x] = 0;
            ptx::named_barrier_sync(1, threads);  // every warp is done with the old ones
            g = g_next;
            r0 = r0_next;
            nx = nx_next;
            stage_x(r0, nx, at.slice * p.steps * W4_STEP, min(p.steps, p.all_steps - at.slice * p.steps));
            cp_async_commit();
            cp_async_wait<0>();
            ptx::named_barrier_sync(1, threads);
        }
        const int32_t n0 = at.n * tile_rows, slice = at.slice, k0 = slice * p.steps * W4_STEP;
        // this warp's steps of the tile: part_k, part_k + wk, ...
        const int32_t mine = (min(p.steps, p.all_steps - slice * p.steps) - part_k + p.wk - 1) / p.wk;
        at.next(p);  // from here on the tile behind this one
        fresh = at.n == 0;
        if (at.left > 0) {
            if (fresh) nth_pass(a, p.xt, at.pass, g_next, r0_next, nx_next);
            stage_scales(at.n * tile_rows, fresh ? g_next : g, at.slice, b ^ 1);
        }
        cp_async_commit();
        float acc[2][4] = {};
        // scale and zero bytes of this team's rows lg + 8 h
        const uint8_t *s_row[4], *z_row[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int32_t r = team * W4S_ROWS + lg + 8 * h;
            const uintptr_t src = reinterpret_cast<uintptr_t>(a.scales) + static_cast<uintptr_t>((g * a.stride_s + (n0 + r) * a.lds) * SB);
            s_row[h] = smem + p.off_s + (b * tile_rows + r) * p.s_words * 4 + static_cast<uint32_t>(src & 3u);
            if constexpr (ZEROS) {
                const uintptr_t zsrc = reinterpret_cast<uintptr_t>(a.zeros) + static_cast<uintptr_t>(g * a.stride_z + (n0 + r) * a.ldz + slice * p.steps * RUNS);
                z_row[h] = smem + p.off_z + (b * tile_rows + r) * p.z_words * 4 + static_cast<uint32_t>(zsrc & 3u);
            }
        }
        // (an operand column of no row repeats row 0's: its sums are not stored)
        uint32_t x_step = base + p.off_x + (lg < nx ? lg : 0) * p.x_pitch + lc * 16 + part_k * (2 * W4_STEP);
        int32_t k_left = a.K - k0 - part_k * W4_STEP;  // codes from the step's first
        int32_t run0 = part_k * RUNS;
        for (int32_t i = 0; i < mine; ++i) {
            if (!ptx::mbar_try_wait(bar0 + 8u * slot, parity)) {
                const uint64_t t0 = ptx::global_timer_ns();
                while (!ptx::mbar_try_wait(bar0 + 8u * slot, parity)) {
                    if (*reinterpret_cast<volatile int32_t *>(&aborted)) break;
                    if (ptx::global_timer_ns() - t0 > p.timeout_ns) {
                        atomicCAS(p.err, 0u, static_cast<uint32_t>(ERR_TIMEOUT_PRODUCER));
                        *reinterpret_cast<volatile int32_t *>(&aborted) = 1;
                        break;
                    }
                }
            }
            __syncwarp();
            uint32_t w_lane = (ring + slot * W4S_BOX + lg * 128 + lc * 4) ^ static_cast<uint32_t>(lg << 4);
            // (the loads below are not volatile, so that they mix with the
            // products; they hang on w_lane, which exists from here on)
            asm volatile("" : "+r"(w_lane), "+r"(x_step)::"memory");
            // the step's scales, as bf16 pairs
            uint32_t sc[4][SW];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const uint8_t *src = s_row[h] + run0 * SB;
                uint32_t in[(SBYTES + 3) / 4];
                if (p.s_vec) {
                    if constexpr (SBYTES == 16) {
                        const uint4 v = lds128(src);
                        in[0] = v.x, in[1] = v.y, in[2] = v.z, in[3] = v.w;
                    } else if constexpr (SBYTES == 8) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(src);
                        in[0] = v.x, in[1] = v.y;
                    } else {
                        in[0] = lds32(src);
                    }
                } else {
#pragma unroll
                    for (int w = 0; w < SBYTES / 4; ++w) {
                        if constexpr (E2M1)
                            in[w] = lds_u8(src + 4 * w) | lds_u8(src + 4 * w + 1) << 8 | lds_u8(src + 4 * w + 2) << 16 | lds_u8(src + 4 * w + 3) << 24;
                        else
                            in[w] = lds_u16(src + 4 * w) | lds_u16(src + 4 * w + 2) << 16;
                    }
                }
#pragma unroll
                for (int w = 0; w < SW; ++w) {
                    if constexpr (E2M1) {
                        const __nv_bfloat162_raw v = __nv_cvt_e8m0x2_to_bf162raw(static_cast<__nv_fp8x2_storage_t>(in[w >> 1] >> (16 * (w & 1))));
                        sc[h][w] = static_cast<uint32_t>(v.x) | static_cast<uint32_t>(v.y) << 16;
                    } else {
                        sc[h][w] = in[w];
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < RUNS; ++j) {
                if (j > 0 && j * RUN >= k_left) break;
                float part[2][4];
                uint32_t zz[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) zz[h] = ZEROS ? (0x4300u | (lds_u8(z_row[h] + run0 + j) & 15u)) * 0x00010001u : eight;
#pragma unroll
                for (int q = 0; q < RUN / 32; ++q) {
                    const int blk = j * (RUN / 32) + q;
                    const uint4 xv = shared_u128(x_step, blk * 64);
                    const uint32_t wa = w_lane ^ static_cast<uint32_t>(blk << 4);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t u[4], v[4];
                        decode<E2M1>(shared_u32(wa, m * 2048), magic, zz[2 * m], u);
                        decode<E2M1>(shared_u32(wa, m * 2048 + 1024), magic, zz[2 * m + 1], v);
                        const uint32_t a0[4] = {u[0], v[0], u[1], v[1]}, a1[4] = {u[2], v[2], u[3], v[3]};
                        mma_16816(part[m], a0, xv.x, xv.y, q == 0);
                        mma_16816(part[m], a1, xv.z, xv.w, false);
                    }
                }
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const float sv = (j & 1) ? __uint_as_float(sc[h][j >> 1] & 0xffff0000u) : __uint_as_float(sc[h][j >> 1] << 16);
                    float &a0 = acc[h >> 1][2 * (h & 1)], &a1 = acc[h >> 1][2 * (h & 1) + 1];
                    a0 = fmaf(sv, part[h >> 1][2 * (h & 1)], a0);
                    a1 = fmaf(sv, part[h >> 1][2 * (h & 1) + 1], a1);
                }
            }
            x_step += p.wk * (2 * W4_STEP);
            k_left -= p.wk * W4_STEP;
            run0 += p.wk * RUNS;
            // the box has been read into these sums: its slot may be filled again
            asm volatile(""
                         : "+f"(acc[0][0]), "+f"(acc[0][1]), "+f"(acc[0][2]), "+f"(acc[0][3]), "+f"(acc[1][0]), "+f"(acc[1][1]), "+f"(acc[1][2]),
                           "+f"(acc[1][3])::"memory");
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar0 + 8u * (W4S_STAGES + slot));
            if (++slot == static_cast<uint32_t>(p.stages)) {
                slot = 0;
                parity ^= 1u;
            }
        }
        // sums[warp][x row][weight row], added over a team's warps in order
        float *sums = reinterpret_cast<float *>(smem + p.off_sum);
        ptx::named_barrier_sync(1, threads);  // the last tile's have been added
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int tok = 2 * lc + i;
            if (tok >= nx) continue;
            float *dst = sums + (warp * p.xt + tok) * W4S_ROWS + lg;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                dst[16 * m] = acc[m][i];
                dst[16 * m + 8] = acc[m][2 + i];
            }
        }
        cp_async_wait<0>();
        // The sums, and the next tile's scales, are there.  The warps leave as one
        // where a wait has run out: the producer may say so between two warps'
        // reads of it.  (It waits for the boxes on their way itself.)
        if (!agree(*reinterpret_cast<volatile int32_t *>(&aborted) == 0, 1, threads)) return;
        // A warp: the 32 weight rows of a team for one activation row a turn,
        // to y or, where there are more slices, to scratch.
        auto put = [&](int tok, int n, float v) {
            if (p.slices == 1)
                store_y(a, r0 + tok, n0 + n, v);
            else
                __stcg(p.partials + (static_cast<int64_t>(slice) * a.S + r0 + tok) * a.N + n0 + n, v);
        };
        for (int i = warp; i < teams * nx; i += p.warps) {
            const int tm = i / nx, tok = i - tm * nx, n = tm * W4S_ROWS + lane;
            if (x_odd[odd_set][tok]) {
                for (int r = 0; r < W4S_ROWS && n0 + tm * W4S_ROWS + r < a.N; ++r) {
                    const float v = row_dot<E2M1>(a, g, n0 + tm * W4S_ROWS + r, r0 + tok, k0, min(a.K, k0 + p.steps * W4_STEP));
                    if (lane == 0) put(tok, tm * W4S_ROWS + r, v);
                }
                continue;
            }
            if (n0 + n >= a.N) continue;
            const float *src = sums + (tm * p.wk * p.xt + tok) * W4S_ROWS + lane;
            float sum = 0.0f;
#pragma unroll 4
            for (int v = 0; v < p.wk; ++v) sum += src[v * p.xt * W4S_ROWS];
            put(tok, n, sum);
        }
    }
    clear();
}

// The slices' partial products, added in their order.
__global__ void __launch_bounds__(256) w4_join_kernel(const W4Args a, const float *partials, int32_t slices)
{
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int32_t n = static_cast<int32_t>(blockIdx.x) * 256 + static_cast<int32_t>(threadIdx.x);
    if (n >= a.N) return;
    const int32_t first = a.offsets ? max(0, min(__ldg(a.offsets), a.S)) : 0;
    const int32_t last = a.offsets ? max(first, min(__ldg(a.offsets + a.groups), a.S)) : a.S;
    for (int32_t r = first + static_cast<int32_t>(blockIdx.y); r < last; r += static_cast<int32_t>(gridDim.y)) {
        float sum = 0.0f;
#pragma unroll 4
        for (int32_t v = 0; v < slices; ++v) sum += __ldcg(partials + (static_cast<int64_t>(v) * a.S + r) * a.N + n);
        store_y(a, r, n, sum);
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

template <bool E2M1, int RUN, bool ZEROS>
cudaError_t launch_tile(const W4Args &a, int64_t used, int xt, int dev, cudaStream_t s)
{
    using L = W4Layout<E2M1, RUN>;
    auto kern = w4_tile_kernel<E2M1, RUN, ZEROS>;
    static std::atomic<unsigned long long> configured{0};  // the shared-memory opt-in, once per device
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (!bit || !(configured.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::smem(8, ZEROS) > L::smem(4, ZEROS) ? L::smem(8, ZEROS) : L::smem(4, ZEROS));
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    static_assert(L::smem(8, ZEROS) <= SMEM_LIMIT && L::smem(4, ZEROS) <= SMEM_LIMIT, "shared memory");
    const dim3 grid(static_cast<unsigned>((a.N + W4_ROWS - 1) / W4_ROWS), static_cast<unsigned>(used));
    return launch(kern, grid, w4_warps(xt) * 32, static_cast<size_t>(L::smem(xt, ZEROS)), s, a, xt);
}

cudaError_t launch_w4(const W4Args &a, bool e2m1, int64_t used, int xt, int dev, cudaStream_t s)
{
    if (e2m1) return launch_tile<true, 32, false>(a, used, xt, dev, s);
    if (a.zeros) {
        if (a.run == 32) return launch_tile<false, 32, true>(a, used, xt, dev, s);
        if (a.run == 64) return launch_tile<false, 64, true>(a, used, xt, dev, s);
        return launch_tile<false, 128, true>(a, used, xt, dev, s);
    }
    if (a.run == 32) return launch_tile<false, 32, false>(a, used, xt, dev, s);
    if (a.run == 64) return launch_tile<false, 64, false>(a, used, xt, dev, s);
    return launch_tile<false, 128, false>(a, used, xt, dev, s);
}

// The stream kernel's plan; false where no slice's activations fit.  `used`:
// the groups that have rows, at most.
bool plan_stream(const W4Args &a, bool e2m1, int64_t used, int sms, W4Stream &best_p, int &grid, size_t &smem)
{
    W4Stream p{};
    p.xt = 1;
    while (p.xt < 8 && p.xt < a.S) p.xt *= 2;
    p.all_steps = (a.K + W4_STEP - 1) / W4_STEP;
    const int sb = e2m1 ? 1 : 2, runs = W4_STEP / a.run;
    p.s_vec = (reinterpret_cast<uintptr_t>(a.scales) | static_cast<uintptr_t>(a.lds * sb) | static_cast<uintptr_t>(a.stride_s * sb)) % 4 == 0;
    // The passes to expect: rows that fall on groups at random leave some
    // groups empty (S of them reach groups (1 - (1 - 1/groups)^S)).
    const int64_t even = (a.S + p.xt - 1) / p.xt;
    double passes = static_cast<double>(even);
    if (a.offsets && a.groups > 1) {
        const double hit = a.groups * (1.0 - std::pow(1.0 - 1.0 / a.groups, static_cast<double>(a.S)));
        passes = std::fmax(passes, std::fmin(hit, static_cast<double>(used)));
    }
    // A CTA's time: for each of its tiles a turn of `warps` boxes for every
    // step a warp has, and the tile's end.  Measured on 28672 rows of 8192
    // codes (16 warps; teams of 16, 8, 4 and 2 warps: 31.6, 28.8, 35.1 and
    // 33.2 us): a turn costs about 1.5 times the end.  Fewer warps only shorten a
    // turn to a half, where latency is what is left of it, and a ring of
    // fewer than 32 boxes (128 KB) stretches it: the activations of a slice
    // of K take its room.  More slices mean a second launch that adds them,
    // activations staged for each (its share of the CTA's tiles) and partial
    // products.  Measured (us; 1, 2, 4 and 8 slices, int4): 8 rows of 9216
    // onto 8192 39, 24, 21, 21; 4 of 14336 onto 4096 21, 17, 15, 15; 8 of
    // 8192 onto 28672 44, 41, 38, 44; 1 of 8192 onto 28672 29, 30, 31, 36.
    double best = 0.0;
    for (int32_t slices = 1; slices <= W4S_SLICES && slices <= p.all_steps; slices *= 2) {
        p.steps = (p.all_steps + slices - 1) / slices;
        p.slices = (p.all_steps + p.steps - 1) / p.steps;
        if (p.slices != slices) continue;
        if (slices > 1 && static_cast<int64_t>(a.S) * a.N * slices * 4 > W4S_SCRATCH) break;
        if (p.steps > SMEM_LIMIT / (W4_STEP * 2)) continue;  // not one row of activations fits (and 32 bits hold what follows)
        p.x_pitch = p.steps * W4_STEP * 2 + 64;
        // A lane reads a step's scales of a row at once, 4 to 16 bytes: rows lie
        // an odd number of such pieces apart, in different banks.
        const int unit = (runs * sb + 3) / 4;
        const int pieces = (p.steps * unit + 1 + unit - 1) / unit | 1;
        p.s_words = pieces * unit;
        p.z_words = a.zeros ? (std::min(a.runs, p.steps * runs) + 3) / 4 + 1 : 0;
        for (p.warps = W4S_WARPS; p.warps >= 4; p.warps /= 2) {
            for (p.wk = 1; p.wk <= p.warps && p.wk <= p.steps; p.wk *= 2) {
                const int rows = p.warps / p.wk * W4S_ROWS;
                const int64_t room = SMEM_LIMIT - W4S_STATIC - 1024 - static_cast<int64_t>(p.xt) * p.x_pitch - 32 -  // (1 KB: alignment)
                                     2 * static_cast<int64_t>(rows) * (p.s_words + p.z_words) * 4 - p.warps * p.xt * W4S_ROWS * 4;
                if (room < 2 * p.warps * W4S_BOX) continue;
                p.tiles_n = static_cast<int32_t>((a.N + rows - 1) / rows);
                p.stages = static_cast<int32_t>(std::min<int64_t>(W4S_STAGES, room / (p.warps * W4S_BOX)));
                const double rounds = std::ceil(passes * slices * p.tiles_n / sms);
                const double starved = std::fmax(1.0, 32.0 / (p.warps * p.stages));
                const double turn = 1.5 * std::fmax(p.warps, 8) / 16.0 * starved;
                const double fresh = std::fmin(1.0 + rounds / p.tiles_n, rounds);
                const double cost = rounds * (turn * ((p.steps + p.wk - 1) / p.wk) + 1.0) + fresh * 0.015 * p.xt * p.steps + (slices > 1 ? 2.0 + 1.6e-6 * slices * a.S * a.N : 0.0);
                if (best != 0.0 && cost >= best) continue;
                best = cost;
                best_p = p;
                best_p.off_x = p.warps * p.stages * W4S_BOX;
                best_p.off_s = best_p.off_x + p.xt * p.x_pitch;
                best_p.off_z = best_p.off_s + 2 * rows * p.s_words * 4;
                best_p.off_sum = best_p.off_z + 2 * rows * p.z_words * 4;
                smem = static_cast<size_t>(best_p.off_sum + p.warps * p.xt * W4S_ROWS * 4 + 1024);
            }
        }
    }
    if (best == 0.0) return false;
    const int64_t n = std::max(a.offsets ? used : 0, even) * best_p.slices * best_p.tiles_n;
    grid = static_cast<int>(n < sms ? n : sms);
    return true;
}

template <bool E2M1, int RUN, bool ZEROS>
cudaError_t launch_stream(const CUtensorMap &tm, const W4Args &a, const W4Stream &p, int grid, size_t smem, int dev, cudaStream_t s)
{
    auto kern = w4_stream_kernel<E2M1, RUN, ZEROS>;
    static std::atomic<unsigned long long> configured{0};
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (!bit || !(configured.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT - W4S_STATIC);
        if (e != cudaSuccess) return e;
        configured.fetch_or(bit, std::memory_order_acq_rel);
    }
    return launch(kern, dim3(static_cast<unsigned>(grid)), (p.warps + 1) * 32, smem, s, tm, a, p);
}

cudaError_t launch_stream_of(bool e2m1, const CUtensorMap &tm, const W4Args &a, const W4Stream &p, int grid, size_t smem, int dev,
                             cudaStream_t s)
{
    if (e2m1) return launch_stream<true, 32, false>(tm, a, p, grid, smem, dev, s);
    if (a.zeros) {
        if (a.run == 32) return launch_stream<false, 32, true>(tm, a, p, grid, smem, dev, s);
        if (a.run == 64) return launch_stream<false, 64, true>(tm, a, p, grid, smem, dev, s);
        return launch_stream<false, 128, true>(tm, a, p, grid, smem, dev, s);
    }
    if (a.run == 32) return launch_stream<false, 32, false>(tm, a, p, grid, smem, dev, s);
    if (a.run == 64) return launch_stream<false, 64, false>(tm, a, p, grid, smem, dev, s);
    return launch_stream<false, 128, false>(tm, a, p, grid, smem, dev, s);
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

#ifdef TG_DEBUG_CHECKS
// What tg_gemv_w4_watchdog set for the calls after it (under the host mutex).
struct {
    int32_t stall = 0;
    uint64_t timeout_ns = 0;
} g_watchdog;
#endif

bool pitch_ok(int64_t ld, int64_t cols, int64_t stride)
{
    return ld >= cols && ld <= PITCH_LIMIT && stride >= 0 && stride <= PITCH_LIMIT;
}

}  // namespace
}  // namespace tg

using namespace tg;

#ifdef TG_DEBUG_CHECKS
// Of the checks build alone, as tg_gemv_w4 takes no options: the watchdog limit
// of later calls (0: the usual one) and whether their waits are made to run out.
TG_API void tg_gemv_w4_watchdog(int32_t stall, uint64_t timeout_ns)
{
    std::lock_guard<std::mutex> lock(host_mutex());
    g_watchdog.stall = stall;
    g_watchdog.timeout_ns = timeout_ns;
}
#endif

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
        if (reinterpret_cast<uintptr_t>(y) % yb || reinterpret_cast<uintptr_t>(x) % 2 || reinterpret_cast<uintptr_t>(scales) % sb ||
            !host_words_ok(offsets))
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
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        const bool e2m1 = format == TG_W4_E2M1;
        // Weights that TMA can address (16-byte rows; the activations may
        // have any alignment); 4-byte rows of both; anything else.
        const uintptr_t w_at = reinterpret_cast<uintptr_t>(W) | static_cast<uintptr_t>(a.ldw) | static_cast<uintptr_t>(a.stride_w);
        const uintptr_t x_at = reinterpret_cast<uintptr_t>(x) | static_cast<uintptr_t>(2 * ldx);
        const bool words = (reinterpret_cast<uintptr_t>(scales) | reinterpret_cast<uintptr_t>(zeros)) % 4 == 0;
        if (K > 0 && w_at % 16 == 0 && words) {
            std::lock_guard<std::mutex> lock(host_mutex());
            HostStream hs;
            const tg_status st = host_stream(s, &hs);
            if (st != TG_OK) return st;
            W4Stream p{};
            int grid = 0;
            size_t smem = 0;
            CUtensorMap tm;
            const uint64_t s2 = static_cast<uint64_t>(groups > 1 && a.stride_w > 0 ? a.stride_w : (N * a.ldw + 15) / 16 * 16);
            const bool shared_w = groups > 1 && a.stride_w == 0;
            if (plan_stream(a, e2m1, used, hs.sms, p, grid, smem) &&
                host_encode_3d(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, W, static_cast<uint64_t>(K / 2), static_cast<uint64_t>(N),
                               shared_w ? 1 : static_cast<uint64_t>(groups), static_cast<uint64_t>(a.ldw), s2, W4_STEP / 2, W4S_ROWS,
                               CU_TENSOR_MAP_SWIZZLE_128B)) {
                p.w_shared = shared_w;
                p.err = hs.err;
                p.timeout_ns = HOST_TIMEOUT_NS;
#ifdef TG_DEBUG_CHECKS
                p.stall = g_watchdog.stall;
                if (g_watchdog.timeout_ns) p.timeout_ns = g_watchdog.timeout_ns;
#endif
                if (p.slices > 1) {
                    void *scratch = nullptr;
                    const tg_status ws = host_arena(hs, static_cast<size_t>(p.slices) * S * N * 4, &scratch);
                    if (ws != TG_OK) return ws;
                    p.partials = static_cast<float *>(scratch);
                }
                cudaError_t e = launch_stream_of(e2m1, tm, a, p, grid, smem, hs.dev, s);
                if (e == cudaSuccess && p.slices > 1)
                    e = launch(w4_join_kernel, dim3(static_cast<unsigned>((N + 255) / 256), static_cast<unsigned>(S < 1024 ? S : 1024)), 256, 0, s,
                               a, p.partials, p.slices);
                return host_cuda_status(e);
            }
        }
        if (K > 0 && (w_at | x_at) % 4 == 0 && words) {
            int dev = 0;
            const cudaError_t e = cudaGetDevice(&dev);
            if (e != cudaSuccess) return host_cuda_status(e);
            int xt = 1;  // activation rows a pass: no more than there are
            while (xt < 8 && xt < S) xt *= 2;
            return host_cuda_status(launch_w4(a, e2m1, used, xt, dev, s));
        }
        const dim3 grid(static_cast<unsigned>((N + ANY_COLS - 1) / ANY_COLS), static_cast<unsigned>(used));
        return host_cuda_status(format == TG_W4_E2M1 ? launch(w4_any_kernel<true>, grid, ANY_COLS * 32, 0, s, a)
                                                     : launch(w4_any_kernel<false>, grid, ANY_COLS * 32, 0, s, a));
    });
}
