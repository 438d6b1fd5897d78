// A kernel that lets the next one on its stream begin launching at once and then
// runs for `ns` nanoseconds (a bounded loop) on one SM before it writes `n` values:
// for tests of kernels that are launched as programmatic dependents.
#include <cuda_runtime.h>
#include <stdint.h>

namespace {

__device__ uint64_t now() {
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

__global__ void producer(uint16_t *out, const uint16_t *from, int64_t n, uint64_t ns) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint64_t begin = now();
    for (int i = 0; i < 100000000 && now() - begin < ns; ++i) __nanosleep(1000);
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) out[i] = from[i];
}

}  // namespace

extern "C" int early_producer(uint16_t *out, const uint16_t *from, int64_t n, uint64_t ns,
                              cudaStream_t stream) {
    producer<<<1, 1024, 0, stream>>>(out, from, n, ns);
    return static_cast<int>(cudaGetLastError());
}
