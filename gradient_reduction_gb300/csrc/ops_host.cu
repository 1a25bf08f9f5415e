// Launch and argument checks shared by the backward-pass operators.
#include <map>
#include <mutex>
#include <tuple>

#include "ops_kernels.h"

namespace dpr {

cudaError_t launch_grid(const void* kernel, dim3 grid, dim3 block, size_t smem, void** args,
                        cudaStream_t s, int cluster) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    if (cluster > 1) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = unsigned(cluster);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.numAttrs = 1;
    }
    const bool legacy = s == nullptr || s == cudaStreamLegacy || s == cudaStreamPerThread;
    cfg.attrs = attr;
    if (!legacy && programmatic_launch_enabled()) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

cudaError_t resident_blocks(const void* kernel, int threads, int64_t* blocks) {
    static std::mutex mu;
    static std::map<std::tuple<const void*, int, int>, int64_t> cache;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    try {
        std::lock_guard<std::mutex> lock(mu);
        const auto key = std::make_tuple(kernel, threads, dev);
        auto it = cache.find(key);
        if (it == cache.end()) {
            int sms = 0, per_sm = 0;
            e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
            if (e == cudaSuccess)
                e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, 0);
            if (e != cudaSuccess) return e;
            it = cache.emplace(key, int64_t(sms) * (per_sm < 1 ? 1 : per_sm)).first;
        }
        *blocks = it->second;
    } catch (...) {   // out of host memory: no exception leaves a C entry
        return cudaErrorMemoryAllocation;
    }
    return cudaSuccess;
}

cudaError_t allow_shared_memory(const void* kernel, int bytes, std::atomic<uint64_t>* done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (e != cudaSuccess || (dev < 64 && (done->load(std::memory_order_acquire) & bit))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done->fetch_or(bit, std::memory_order_release);
    return e;
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

}  // namespace dpr
