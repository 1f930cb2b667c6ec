// Host code that the products over ragged rows share (tg_grouped.cu,
// tg_block.cu): checks of extents and spans, operands that need a realigned
// copy, the choice of tiles and shares.  Not part of the public ABI.
#pragma once

#include <algorithm>
#include <cstdint>

#include "tg_internal.h"

namespace tg {

constexpr int64_t SPLIT_DEPTH = 12;  // k-blocks of a share at least (pairs: twice that)
constexpr int64_t SPLIT_MOST = 16;   // shares of a tile at most

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t GROUPED_EXTENT = INT32_MAX - 1024;  // a tile past the end stays in range
constexpr int64_t PITCH_LIMIT = int64_t(1) << 40;

inline bool tma_ok(const void *p, int64_t ld, int64_t stride, int64_t bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * bytes % 16 == 0 && stride * bytes % 16 == 0;
}

struct Operand {
    const void *p;
    int64_t rows, cols, ld, nb, stride;  // stored: nb matrices of rows x cols
    bool pack = false;
};

inline uint64_t problem_stride(const Operand &o)
{
    // any valid value where there is one matrix only
    return static_cast<uint64_t>(o.nb > 1 ? o.stride * 2 : cdiv(o.rows * o.ld * 2, 16) * 16);
}

inline size_t pack_bytes(const Operand &o)
{
    return o.pack ? static_cast<size_t>(cdiv(o.nb * o.rows * cdiv(o.cols, 64) * 64 * 2, 256) * 256) : 0;
}

struct Bytes {
    uintptr_t lo = 0, hi = 0;
};
inline Bytes bytes_of(const void *p, int64_t nb, int64_t stride, int64_t rows, int64_t ld, int64_t cols, int64_t size)
{
    if (!p || nb < 1 || rows < 1 || cols < 1) return {};
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return {b, b + static_cast<uintptr_t>(((nb - 1) * stride + (rows - 1) * ld + cols) * size)};
}
inline bool meets(const Bytes &a, const Bytes &b) { return a.lo < b.hi && b.lo < a.hi; }

inline bool extent_ok(int64_t v) { return v >= 0 && v <= GROUPED_EXTENT; }
inline bool pitch_ok(int64_t ld, int64_t cols) { return ld >= cols && ld <= PITCH_LIMIT; }
inline bool span_ok(int64_t nb, int64_t stride, int64_t rows, int64_t ld)
{
    return static_cast<__int128>(nb) * stride + static_cast<__int128>(rows) * ld < (static_cast<__int128>(1) << 56);
}

// Few tiles and a long contraction: workers share tiles.  The k-blocks of a
// share, or 0 where tiles are not shared: as many shares as there are workers
// for the average group's tiles (the one that arrives last adds them, 128 or
// 64 KB each, so a share is 24 or 12 k-blocks at least: with 16, 8 or 4 for 12,
// 22 short calls take 3%, 5% and 10% longer), and a longer group's
// tiles more of the same length.  (Two, three or four times as many, to even
// out groups of unknown lengths, measured the same or more: wgrad, 32768 rows
// of 8 groups, 256 x 1000: 35, 38, 46 and 49 us.)
inline int64_t share_of(bool wgrad, bool pair, int64_t units, int64_t depth, int sms)
{
    const int64_t workers = pair ? sms / 2 : sms;
    const int64_t least = pair ? 2 * SPLIT_DEPTH : SPLIT_DEPTH;
    if (depth < 2 * least || units >= (wgrad ? 2 * workers : workers)) return 0;
    return std::max(least, units <= workers ? cdiv(depth, workers / units) : cdiv(units * depth, workers));
}

// A measure of what a call takes with one-CTA tiles (128 x 128) or pairs (256 x
// 256): turns of the workers over the tiles (rows mode: those of groups that end
// anywhere in a tile) or shares, each a start, so much a k-block, and where tiles
// are shared the adding.  Its constants choose, they do not foretell: they were fitted,
// in microseconds, to the choice in 350 calls of both kinds (1 to 32 uneven groups of
// 64 to 4096 rows, rows mode K 64 to 4096 and N 256 to 4096, gradients 256 to 2048 x
// 256 to 4096), and a pair's start carries a part of its k-blocks (which take 0.33 at
// the tensor cores' measured rate, not 0.143), so that contractions deeper than those
// look too short in pairs.  The tiles it
// chooses take 0.4% longer than the better ones on average, those of a rule by
// size (256 rows and enough pair tiles to fill half the SMs) 4%, and up to half as
// long again: 8 groups of 256 rows, 4096 x 1000: 42.9 us in one-CTA tiles, 28.1
// in pairs; 32 of 192, 64 x 1000: 10.1, 15.4.
inline double tiles_cost(bool wgrad, bool pair, int64_t S, int64_t M, int64_t N, int64_t K, int64_t groups, int sms)
{
    const double start = pair ? 4.3 : 0.7, block = pair ? 0.143 : 0.27, adding = pair ? 9.5 : 2.1;
    const int64_t t = pair ? 256 : 128, workers = pair ? sms / 2 : sms;
    const int64_t hit = std::max<int64_t>(1, groups < S ? groups : S);
    const int64_t depth = wgrad ? cdiv(S / groups, BK) : cdiv(K, BK);
    int64_t units = cdiv(N, t);
    if (wgrad)
        units *= groups * cdiv(M, t);
    else
        units *= groups > 1 ? std::max(hit, S / t + (hit + 1) / 2) : cdiv(S, t);
    const int64_t share = share_of(wgrad, pair, units, depth, sms);
    if (share == 0) return static_cast<double>(cdiv(units, workers)) * (start + block * depth);
    return static_cast<double>(cdiv(units * cdiv(depth, share), workers)) * (start + block * share + (share < depth ? adding : 0.0));
}

}  // namespace tg
