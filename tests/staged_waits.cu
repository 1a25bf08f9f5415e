// The layer norm's backward kernels when one thread's wait is reported as run out:
// the source is compiled here with mbar_wait in a wrapper that waits in earnest
// and then, in one chosen thread, answers false once.  Prints a line for each
// case: its name and how many waits were counted.
#include <cstdio>
#include <vector>

#include "../gradient_reduction_gb300/csrc/tensor_core.cuh"

namespace dpr {
namespace tc {
struct Chosen {
    int block, thread, nth, seen;
};
__device__ Chosen g_chosen = {-1, 0, 0, 0};
__device__ __forceinline__ bool mbar_wait_reported(uint32_t bar, uint32_t parity) {
    const bool done = mbar_wait(bar, parity);
    if (int(blockIdx.x) == g_chosen.block && int(threadIdx.x) == g_chosen.thread && threadIdx.y == 0)
        if (++g_chosen.seen == g_chosen.nth) return false;
    return done;
}
}  // namespace tc
}  // namespace dpr
#define mbar_wait mbar_wait_reported
#include "../gradient_reduction_gb300/csrc/layernorm_backward.cu"
#undef mbar_wait
#include "../gradient_reduction_gb300/csrc/ops_host.cu"

namespace dpr {
bool programmatic_launch_enabled() { return true; }
dpr_status record_cuda_status(cudaError_t e) { return e == cudaSuccess ? DPR_OK : DPR_ERR_CUDA; }
}  // namespace dpr

namespace {

int failures() {
    unsigned int n = 0;
    return dpr::norm_wait_failures(&n) == cudaSuccess ? int(n) : -1;
}

// dx of dy = 1 in the first half of a row and -1 in the second, xhat = 0: dy itself.
bool run(const char* name, int64_t rows, int64_t width, int block, int thread, int nth) {
    const size_t n = size_t(rows * width);
    int64_t need = 0;
    if (dpr_layernorm_backward_workspace(rows, width, &need) != DPR_OK) return false;
    float *mean, *rstd, *dw, *db;
    uint16_t *x, *dy, *dx;
    void* ws;
    if (cudaMalloc(&x, 2 * n) || cudaMalloc(&dy, 2 * n) || cudaMalloc(&dx, 2 * n) ||
        cudaMalloc(&mean, 4 * rows) || cudaMalloc(&rstd, 4 * rows) || cudaMalloc(&dw, 4 * width) ||
        cudaMalloc(&db, 4 * width) || cudaMalloc(&ws, size_t(need)))
        return false;
    std::vector<uint16_t> d(n), got(n);
    for (size_t i = 0; i < n; ++i) d[i] = int64_t(i % size_t(width)) < width / 2 ? 0x3F80 : 0xBF80;
    const std::vector<float> ones(size_t(rows), 1.0f);
    cudaMemset(x, 0, 2 * n);
    cudaMemset(mean, 0, 4 * rows);
    cudaMemcpy(dy, d.data(), 2 * n, cudaMemcpyHostToDevice);
    cudaMemcpy(rstd, ones.data(), 4 * rows, cudaMemcpyHostToDevice);
    bool ok = true;
    for (int chosen = 1; chosen >= 0; --chosen) {   // a call after it is as if nothing had been
        const dpr::tc::Chosen c = {chosen ? block : -1, thread, nth, 0};
        cudaMemcpyToSymbol(dpr::tc::g_chosen, &c, sizeof(c));
        const int before = failures();
        if (dpr_layernorm_backward(dy, width, x, width, nullptr, rows, width, DPR_BF16, nullptr,
                                   DPR_BF16, mean, rstd, dx, width, dw, db, DPR_FP32, 0, ws, need,
                                   nullptr) != DPR_OK ||
            cudaDeviceSynchronize() != cudaSuccess)
            return false;
        const int counted = failures() - before;
        if (chosen) {
            printf("%s %d\n", name, counted);
        } else {
            cudaMemcpy(got.data(), dx, 2 * n, cudaMemcpyDeviceToHost);
            ok = counted == 0 && got == d;
        }
    }
    for (void* q : {(void*)x, (void*)dy, (void*)dx, (void*)mean, (void*)rstd, (void*)dw, (void*)db, ws})
        cudaFree(q);
    return ok;
}

}  // namespace

int main() {
    // one row a group, so that nothing is skipped after the answer: the row's load, and
    // (two CTAs a row) the other half's sums
    if (!run("none", 64, 1024, -1, 0, 0)) return 2;
    if (!run("thread", 64, 1024, 1, 37, 1)) return 3;
    if (!run("first-thread", 64, 1024, 1, 0, 1)) return 4;
    if (!run("pair-load", 3, 8208, 1, 100, 1)) return 5;
    if (!run("pair-sums", 3, 8208, 2, 100, 2)) return 6;
    // more rows than stages: the first thread asks for no more, the others' waits run out
    if (!run("first-thread-of-many", 16384, 1024, 1, 0, 1)) return 7;
    if (!run("first-thread-of-many-pairs", 1000, 8208, 2, 0, 3)) return 8;
    return 0;
}
