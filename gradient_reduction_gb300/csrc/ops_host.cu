// Launch and argument checks shared by the backward-pass operators.
#include <map>
#include <mutex>

#include "ops_kernels.h"

namespace dpr {

cudaError_t launch_grid(const void* kernel, dim3 grid, dim3 block, size_t smem, void** args,
                        cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const bool legacy = s == nullptr || s == cudaStreamLegacy || s == cudaStreamPerThread;
    cfg.attrs = attr;
    cfg.numAttrs = (!legacy && programmatic_launch_enabled()) ? 1 : 0;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

cudaError_t current_sm_count(int* sms) {
    static std::mutex mu;
    static std::map<int, int> cache;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    auto it = cache.find(dev);
    if (it == cache.end()) {
        int v = 0;
        e = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        it = cache.emplace(dev, v).first;
    }
    *sms = it->second;
    return cudaSuccess;
}

dpr_status check_matrix_size(int64_t rows, int64_t width) {
    if (rows < 0 || width < 1) return DPR_ERR_INVALID_ARG;
    if (rows > DPR_MAX_ROWS || width > DPR_MAX_WIDTH) return DPR_ERR_UNSUPPORTED;
    return DPR_OK;
}

dpr_status check_matrix(const void* p, int64_t stride, int64_t width, int dtype, bool written) {
    if (!p || stride < (written ? width : 0)) return DPR_ERR_INVALID_ARG;
    if (stride > (int64_t(1) << 30)) return DPR_ERR_UNSUPPORTED;
    if (!aligned(p, uintptr_t(dtype_size(dtype)))) return DPR_ERR_ALIGNMENT;
    return DPR_OK;
}

dpr_status check_checkpoint(const dpr_checkpoint* c, int64_t width) {
    if (!c->codes || !c->steps) return DPR_ERR_INVALID_ARG;
    if (c->code_stride < width || c->step_stride < ceil_div(width, DPR_CHECKPOINT_BLOCK))
        return DPR_ERR_INVALID_ARG;
    if (c->code_stride > (int64_t(1) << 30) || c->step_stride > (int64_t(1) << 30))
        return DPR_ERR_UNSUPPORTED;
    return DPR_OK;
}

void add_spans(const dpr_checkpoint& c, int64_t rows, int64_t width, std::vector<Span>* v) {
    v->push_back(span_of(c.codes, matrix_bytes(rows, width, c.code_stride, 1)));
    v->push_back(span_of(
        c.steps, matrix_bytes(rows, ceil_div(width, DPR_CHECKPOINT_BLOCK), c.step_stride, 1)));
}

}  // namespace dpr
