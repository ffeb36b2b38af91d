// The launcher of token_logprobs (csrc/logprobs.cu) over a stand-in for the CUDA runtime that keeps kernel attributes
// for each device, as the runtime does: a cluster of more than 8 blocks is refused on a device where the kernel has not
// been allowed one. Prints one status per call, in the order of main().
#include <cuda_runtime_api.h>

#include <cstdio>
#include <set>
#include <utility>

#include "attn.h"

namespace {
int device = 0;
bool refuse_attribute = false;
std::set<std::pair<int, const void*>> wide;
unsigned cluster = 0;  // of the last launch
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
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t)
{
    cluster = 1;
    return cudaSuccess;
}

cudaError_t cudaGetDevice(int* d)
{
    *d = device;
    return cudaSuccess;
}
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int)
{
    *v = a == cudaDevAttrMultiProcessorCount ? 152 : 227 * 1024;
    return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*)
{
    *a = cudaFuncAttributes{};
    return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v)
{
    if (a != cudaFuncAttributeNonPortableClusterSizeAllowed) return cudaSuccess;
    if (refuse_attribute) return cudaErrorNotSupported;
    if (v) wide.insert({device, f});
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int, size_t)
{
    *n = 3;
    return cudaSuccess;
}
cudaError_t cudaMemcpyFromSymbol(void*, const void*, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaMemcpyToSymbol(const void*, const void*, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**)
{
    cluster = 1;
    for (unsigned i = 0; i < c->numAttrs; ++i)
        if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = c->attrs[i].val.clusterDim.x;
    return cluster > 8 && !wide.count({device, f}) ? cudaErrorInvalidClusterSize : cudaSuccess;
}
}

int main()
{
    auto call = [](int dev, int type, int64_t T) {
        device = dev;
        cluster = 0;
        bqd::LogprobArgs a{};
        a.T = T;
        a.V = 151936;
        a.pitch = a.V;
        const cudaError_t e = bqd::launch_token_logprobs(a, type, nullptr);
        std::printf("device %d type %d rows %d: status %d, cluster %u\n", dev, type, static_cast<int>(T),
                    static_cast<int>(e), cluster);
    };
    for (int type : {BQD_F32, BQD_BF16})
        for (int dev : {0, 1, 0, 5}) call(dev, type, 1);
    call(1, BQD_F32, 42);   // the most rows whose clusters are larger than 8
    call(1, BQD_F32, 400);  // no cluster
    refuse_attribute = true;
    call(2, BQD_F32, 1);
    refuse_attribute = false;
    call(2, BQD_F32, 1);
}
