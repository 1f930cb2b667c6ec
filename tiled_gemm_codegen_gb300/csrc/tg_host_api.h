// What the host library (tg_host.cu) offers the other entry-point files: the
// device's SM count, the per-stream workspace (scratch arena and error
// word), TMA descriptors and the realign pass.  Not part of the public ABI.
#pragma once

#include <mutex>

#include "tg_gemm.h"
#include "tg_internal.h"

namespace tg {

// Held by every call from its first use of the workspace tables to its last
// launch.
std::mutex &host_mutex();

// Watchdog limit of a call that sets none.
constexpr uint64_t HOST_TIMEOUT_NS = 2000000000ull;  // 2 s

// The calling thread's device as `stream` uses it.  Caller holds host_mutex.
struct HostStream {
    int dev = 0;
    int sms = 0;
    cudaStream_t stream = nullptr;
    uint32_t *err = nullptr;  // the stream's device error word
};
tg_status host_stream(cudaStream_t stream, HostStream *out);

// At least `bytes` of the stream's scratch arena (256-byte aligned; contents
// of earlier calls are stale; later calls on the stream reuse it).
tg_status host_arena(const HostStream &hs, size_t bytes, void **out);

// At least `bytes` of the stream's arrival counters, all zero (their kernel
// leaves them so; tg_device_error resets them after an abort).
tg_status host_counters(const HostStream &hs, size_t bytes, int32_t **out);

tg_status host_cuda_status(cudaError_t e);

// Whether arrays of 4-byte values (bounds, slots, weights, bias) lie on 4 bytes.
template <class... P>
bool host_words_ok(const P *...p)
{
    return ((reinterpret_cast<uintptr_t>(p) | ... | uintptr_t(0)) & 3u) == 0;
}

// A rank-3 tensor map (dim0 contiguous, dim1 rows, dim2 problems; strides in
// bytes; box {box0, box1, 1}); false if the driver refuses it.
bool host_encode_3d(CUtensorMap *m, CUtensorMapDataType dt, const void *base, uint64_t d0, uint64_t d1, uint64_t d2,
                    uint64_t stride1, uint64_t stride2, uint32_t box0, uint32_t box1, CUtensorMapSwizzle swz);

// One operand of a realign pass: nb matrices of rows x cols bf16 (row pitch
// ld, `stride` elements between matrices) -> dst, rows pack_pitch(cols) apart.
struct HostPack {
    const void *src = nullptr;
    void *dst = nullptr;
    int64_t rows = 0, cols = 0, ld = 0, nb = 0, stride = 0;
};
cudaError_t host_pack(const HostStream &hs, const HostPack *a, const HostPack *b);  // either may be null

// Runs an entry point's body; C++ exceptions (std::bad_alloc of the workspace
// tables) end here, before the C ABI.
template <class F>
tg_status host_guard(F &&f)
{
    try {
        return f();
    } catch (...) {
        return TG_ERR_OOM;
    }
}

}  // namespace tg
