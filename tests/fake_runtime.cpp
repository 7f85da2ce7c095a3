// A stand-in for the CUDA runtime calls that the paged operators' host code makes, so that its
// behaviour on failing calls can be tested without a GPU: no kernel runs, no address is read.
// Linked with --wrap for each of the calls.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <cstring>

#include "paged_host.h"

namespace {
int g_launches, g_fail_launch, g_mallocs, g_fail_malloc;
cudaError_t g_last;
char g_grids[64][3 * sizeof(unsigned)];

cudaError_t result(cudaError_t e)
{
    if (e != cudaSuccess) g_last = e;
    return e;
}
}  // namespace

namespace fp8mqa {
uint64_t wait_limit_ns() { return 1000000000ull; }
bool encode_rows128(CUtensorMap*, const void*, uint64_t, uint64_t, uint32_t) { return true; }
}  // namespace fp8mqa

extern "C" {

// The n-th launch (or allocation) from now on fails; 0: none.  `last`: the runtime's last error.
void fake_set(int fail_launch, int fail_malloc, int last)
{
    g_launches = g_mallocs = 0;
    g_fail_launch = fail_launch;
    g_fail_malloc = fail_malloc;
    g_last = cudaError_t(last);
}
int fake_launches() { return g_launches; }
int fake_last() { return int(g_last); }
void fake_grid(int i, unsigned* xyz) { std::memcpy(xyz, g_grids[i], sizeof(g_grids[i])); }

cudaError_t __wrap_cudaGetDevice(int* dev)
{
    *dev = 0;
    return cudaSuccess;
}
cudaError_t __wrap_cudaDeviceGetAttribute(int* value, cudaDeviceAttr attr, int)
{
    *value = attr == cudaDevAttrComputeCapabilityMajor   ? 10
             : attr == cudaDevAttrComputeCapabilityMinor ? 3
                                                         : 152;
    return cudaSuccess;
}
cudaError_t __wrap_cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t __wrap_cudaMalloc(void** p, size_t n)
{
    if (++g_mallocs == g_fail_malloc) return result(cudaErrorMemoryAllocation);
    *p = std::calloc(1, n);
    return cudaSuccess;
}
cudaError_t __wrap_cudaFree(void* p)
{
    std::free(p);
    return cudaSuccess;
}
cudaError_t __wrap_cudaMemset(void* p, int c, size_t n)
{
    std::memset(p, c, n);
    return cudaSuccess;
}
cudaError_t __wrap_cudaMemcpy(void* to, const void* from, size_t n, cudaMemcpyKind)
{
    std::memcpy(to, from, n);
    return cudaSuccess;
}
cudaError_t __wrap_cudaGetLastError()
{
    const cudaError_t e = g_last;
    g_last = cudaSuccess;
    return e;
}
cudaError_t __wrap_cudaLaunchKernelExC(const cudaLaunchConfig_t* cfg, const void*, void**)
{
    const unsigned xyz[3] = {cfg->gridDim.x, cfg->gridDim.y, cfg->gridDim.z};
    if (g_launches < 64) std::memcpy(g_grids[g_launches], xyz, sizeof(xyz));
    return result(++g_launches == g_fail_launch ? cudaErrorLaunchOutOfResources : cudaSuccess);
}
}
