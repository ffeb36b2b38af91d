// A kernel of a user's program, for tests of calls that may start while the kernel before them runs: it lets its
// successor start at once, stays for `ns` nanoseconds (at most 2^28 looks at the clock) and then writes its outputs,
// copies of up to four arrays. One block.
#include <cuda_runtime.h>

#include <cstdint>

struct Copies {
    void* to[4];
    const void* from[4];
    int64_t bytes[4];
};

__device__ __forceinline__ uint64_t now()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__global__ void early_writer_kernel(const Copies c, uint64_t ns)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint64_t t0 = now();
    for (uint32_t i = 0; i < (1u << 28) && now() - t0 < ns; ++i) {
    }
    for (int a = 0; a < 4; ++a)
        for (int64_t i = threadIdx.x; i < c.bytes[a]; i += blockDim.x)
            static_cast<uint8_t*>(c.to[a])[i] = static_cast<const uint8_t*>(c.from[a])[i];
}

extern "C" int early_writer(void** to, const void** from, const int64_t* bytes, int n, uint64_t ns, cudaStream_t s)
{
    Copies c = {};
    if (n < 0 || n > 4) return static_cast<int>(cudaErrorInvalidValue);
    for (int i = 0; i < n; ++i) {
        c.to[i] = to[i];
        c.from[i] = from[i];
        c.bytes[i] = bytes[i];
    }
    early_writer_kernel<<<1, 1024, 0, s>>>(c, ns);
    return static_cast<int>(cudaGetLastError());
}
