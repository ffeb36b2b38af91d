// The launchers of the products with 8-bit activations (csrc/fp8_gemm*.cu) over a stand-in for the CUDA runtime in which
// a kernel cannot be loaded at first, as when the device's memory is full: its attributes can be neither read nor set,
// and no launch of it succeeds. Prints two statuses per kernel, of such a call and of one after it.
#include <cuda_runtime_api.h>

#include <cstdio>
#include <map>

#include "fp8.h"

namespace {
bool full = false;
std::map<const void*, int> room;  // dynamic shared memory that a kernel may have
CUresult encode(...) { return CUDA_SUCCESS; }
}  // namespace

extern "C" {
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction() {}
void __cudaRegisterVar() {}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, cudaStream_t) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaSuccess; }
cudaError_t __cudaGetKernel(cudaKernel_t*, const void*) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t cudaGetDevice(int* d)
{
    *d = 0;
    return cudaSuccess;
}
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int)
{
    *v = a == cudaDevAttrMultiProcessorCount ? 152 : 227 * 1024;
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long, cudaDriverEntryPointQueryResult* q)
{
    *p = reinterpret_cast<void*>(encode);
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*)
{
    if (full) return cudaErrorMemoryAllocation;
    *a = cudaFuncAttributes{};
    a->numRegs = 168;
    a->sharedSizeBytes = 1024;
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v)
{
    if (full) return cudaErrorMemoryAllocation;
    if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) room[f] = v;
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int, size_t)
{
    *n = 1;
    return full ? cudaErrorMemoryAllocation : cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*)
{
    *n = 15;
    return full ? cudaErrorMemoryAllocation : cudaSuccess;
}
cudaError_t cudaMemcpyFromSymbol(void*, const void*, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaMemcpyToSymbol(const void*, const void*, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**)
{
    if (full) return cudaErrorMemoryAllocation;
    return c->dynamicSmemBytes > 48 * 1024 && static_cast<int>(c->dynamicSmemBytes) > room[f] ? cudaErrorInvalidValue : cudaSuccess;
}
}

int main()
{
    alignas(16) static uint8_t data[16];
    for (bool dual : {false, true})
        for (int64_t T : {1, 20, 50, 200, 4000}) {  // 16, 32 and 64 tokens, 128 x 128 tiles, pairs
            bqd::Fp8GemmArgs a{};
            a.w0 = a.w1 = a.x = data;
            a.M = T == 4000 ? 4096 : 256;
            a.K = 1024;
            a.T = T;
            a.y_type = BQD_BF16;
            full = true;
            const int first = static_cast<int>(bqd::launch_fp8_gemm(a, dual, nullptr));
            full = false;
            std::printf("%d %d\n", first, static_cast<int>(bqd::launch_fp8_gemm(a, dual, nullptr)));
        }
}
