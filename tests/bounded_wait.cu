// A wait on an mbarrier that nothing ever completes ends by itself with false, in
// the time that tensor_core.cuh states; one whose arrival comes late ends with
// true.  By one thread and by a whole warp.  Prints a line for each: warp or
// not, late or never, its answer and milliseconds.
#include <cstdio>
#include <cuda_runtime.h>

#include "../gradient_reduction_gb300/csrc/tensor_core.cuh"

__global__ void wait_for(int warp, int late, int* answer) {
    __shared__ __align__(8) unsigned long long bar;
    const uint32_t at = dpr::tc::smem_addr(&bar);
    if (threadIdx.x == 0) {
        dpr::tc::mbar_init(at, 1);
        dpr::tc::mbar_init_fence();
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        if (warp) answer[0] = dpr::tc::mbar_wait_warp(at, 0);
        else if (threadIdx.x == 0) answer[0] = dpr::tc::mbar_wait(at, 0);
    }
    if (threadIdx.x == 32 && late) {
        const long long start = clock64();
        while (clock64() - start < 2000000) {}       // about 1 ms
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(at) : "memory");
    }
}

int main() {
    int* answer;
    cudaEvent_t a, b;
    if (cudaMallocManaged(&answer, sizeof(int)) != cudaSuccess) return 2;
    cudaEventCreate(&a);
    cudaEventCreate(&b);
    for (int warp = 0; warp < 2; ++warp)
        for (int late = 1; late >= 0; --late) {
            *answer = -1;
            cudaEventRecord(a);
            wait_for<<<1, 64>>>(warp, late, answer);
            cudaEventRecord(b);
            if (cudaDeviceSynchronize() != cudaSuccess) return 3;
            float ms = 0;
            cudaEventElapsedTime(&ms, a, b);
            printf("%d %d %d %.1f\n", warp, late, *answer, ms);
        }
    return 0;
}
