// What the host sides of the paged operators and of a step's other operators share: a device's state,
// launches and their results, and the memory that the bounds-checking build holds accesses against.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <mutex>

#include "../../include/fp8_mqa_logits.h"
#include "paged_common.cuh"

namespace fp8mqa {

struct PagedDevice {
    std::mutex setting_up;
    int sm_count = 0;
    int32_t* status = nullptr;  // status word of the paged logits
    std::atomic<bool> ready{false};
    std::atomic<bool> wide_pages{false};  // the page tables' kernel may take all the shared memory that it wants
};

// The current device's state, set up by the first call that succeeds in it: what fails once (no memory
// left, a stream being captured) is tried again by the next call.
PagedDevice* paged_device(int* err);

// Launches a kernel that begins with griddepcontrol.wait: it is set up while the one before it ends.
// Its own result says whether it is under way (the runtime's last error may be an older one of the
// caller's).
template <class... Params, class... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                         const Args&... args)
{
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

inline bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Bytes of an element (of the two values that E2M1 keeps in one).
inline int64_t size_of(int32_t type)
{
    return type == FP8MQA_E4M3 || type == FP8MQA_E2M1 ? 1 : type == FP8MQA_F32 ? 4 : 2;
}

// What the bounds-checking build holds a launch's accesses against, from the call's arguments alone; in the
// library nothing of it is there.
#ifdef FP8MQA_DEBUG_BOUNDS
extern std::atomic<uint64_t> g_short[kMemKinds];  // bytes that a kind's memory is taken to be short of (tests)
#endif
inline void spans(PagedBounds& b, int kind, const void* from, int64_t bytes)
{
#ifdef FP8MQA_DEBUG_BOUNDS
    b.from[kind] = reinterpret_cast<uint64_t>(from);
    b.bytes[kind] = bytes > 0 ? uint64_t(bytes) - std::min(uint64_t(bytes), g_short[kind].load()) : 0;
#endif
}
inline PagedBounds bounds_for(const PagedDevice& st)
{
    PagedBounds b = {};
#ifdef FP8MQA_DEBUG_BOUNDS
    b.status = st.status;
#endif
    return b;
}
// Bytes from the first to past the last of n0 x n1 x n2 places, `size` bytes each, at strides in bytes.
inline int64_t extent(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t size)
{
    return n0 > 0 && n1 > 0 && n2 > 0 ? (n0 - 1) * s0 + (n1 - 1) * s1 + (n2 - 1) * s2 + size : 0;
}
// What an entry point returns for its launches' result; a refusal is not left behind for the caller's
// next look at the last error.
inline int launched(cudaError_t e)
{
    if (e == cudaSuccess) return FP8MQA_OK;
    cudaGetLastError();
    return FP8MQA_ERR_LAUNCH;
}

}  // namespace fp8mqa
