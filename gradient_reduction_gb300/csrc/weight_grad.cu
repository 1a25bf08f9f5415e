// A linear layer's weight gradient dW = dY^T X~ from the 8-bit checkpoint of
// X: a product of a [rows, out] and a [rows, in] matrix along their rows.
#include <algorithm>

#include "ops_device.cuh"
#include "ops_kernels.h"

namespace dpr {

struct WeightGradParams {
    const uint16_t* dy;
    int64_t dy_stride;
    dpr_checkpoint x;
    int64_t rows;
    int out_features;
    int in_features;
    void* dw;
    int64_t dw_stride;
    int dw_bf16;
    int accumulate;
};

namespace {

__device__ __forceinline__ void store_grad(const WeightGradParams& p, int o, int i, float v) {
    const int64_t at = int64_t(o) * p.dw_stride + i;
    if (p.dw_bf16) {
        uint16_t* d = static_cast<uint16_t*>(p.dw) + at;
        *d = to_bf16(p.accumulate ? __fadd_rn(bf_1(*d), v) : v);
    } else {
        float* d = static_cast<float*>(p.dw) + at;
        *d = p.accumulate ? __fadd_rn(*d, v) : v;
    }
}

// 64 x 64 outputs per block, 4 x 4 per thread, 16 rows at a time.
__global__ void __launch_bounds__(256) weight_grad_any(const __grid_constant__ WeightGradParams p) {
    __shared__ float a[16][64], b[16][64];
    grid_wait();
    grid_release();
    const int i0 = int(blockIdx.x) * 64, o0 = int(blockIdx.y) * 64;
    const int tx = int(threadIdx.x) & 15, ty = int(threadIdx.x) >> 4;
    float acc[4][4] = {};
    for (int64_t t0 = 0; t0 < p.rows; t0 += 16) {
        for (int q = int(threadIdx.x); q < 16 * 64; q += 256) {
            const int64_t t = t0 + q / 64;
            const int o = o0 + q % 64, i = i0 + q % 64;
            const bool in = t < p.rows;
            a[q / 64][q % 64] = in && o < p.out_features ? bf_1(p.dy[t * p.dy_stride + o]) : 0.0f;
            float v[1] = {0.0f};
            if (in && i < p.in_features) {
                CodeRaw<1> code;
                load_codes<1>(p.x.codes + t * p.x.code_stride + i, code);
                decode<1>(code, step_value(p.x.steps[t * p.x.step_stride + i / kBlockChannels]), v);
            }
            b[q / 64][q % 64] = v[0];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    acc[m][n] = __fmaf_rn(a[k][ty + 16 * m], b[k][tx + 16 * n], acc[m][n]);
        __syncthreads();
    }
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int o = o0 + ty + 16 * m, i = i0 + tx + 16 * n;
            if (o < p.out_features && i < p.in_features) store_grad(p, o, i, acc[m][n]);
        }
}

}  // namespace
}  // namespace dpr

using namespace dpr;

extern "C" {

dpr_status dpr_linear_weight_grad_workspace(int64_t rows, int64_t out_features,
                                            int64_t in_features, int64_t* bytes) {
    if (!bytes) return DPR_ERR_INVALID_ARG;
    *bytes = 0;
    dpr_status st = check_matrix_size(rows, out_features);
    if (st == DPR_OK) st = check_matrix_size(rows, in_features);
    if (st != DPR_OK) return st;
    return DPR_OK;
}

dpr_status dpr_linear_weight_grad(const void* dy, int64_t dy_stride, const dpr_checkpoint* x_ckpt,
                                  int64_t rows, int64_t out_features, int64_t in_features,
                                  void* dweight, int64_t dweight_stride, int dtype, int accumulate,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
    int64_t need = 0;
    dpr_status st = dpr_linear_weight_grad_workspace(rows, out_features, in_features, &need);
    if (st != DPR_OK) return st;
    if (!dtype_ok(dtype)) return DPR_ERR_INVALID_ARG;
    if ((st = check_matrix(dweight, dweight_stride, in_features, dtype, true)) != DPR_OK) return st;
    std::vector<Span> outs, ins;
    outs.push_back(span_of(dweight, matrix_bytes(out_features, in_features, dweight_stride,
                                                 dtype_size(dtype))));
    if (rows > 0) {
        if ((st = check_matrix(dy, dy_stride, out_features, DPR_BF16, false)) != DPR_OK) return st;
        if (!x_ckpt) return DPR_ERR_INVALID_ARG;
        if ((st = check_checkpoint(x_ckpt, in_features)) != DPR_OK) return st;
        if (need > 0) {
            if (!workspace || workspace_bytes < need) return DPR_ERR_INVALID_ARG;
            if (!aligned(workspace, 16)) return DPR_ERR_ALIGNMENT;
            outs.push_back(span_of(workspace, uint64_t(need)));
        }
        ins.push_back(span_of(dy, matrix_bytes(rows, out_features, dy_stride, 2)));
        add_spans(*x_ckpt, rows, in_features, &ins);
    }
    if (!pairwise_disjoint(outs) || any_overlap(outs, ins)) return DPR_ERR_ALIAS;

    WeightGradParams p = {};
    p.dy = static_cast<const uint16_t*>(dy); p.dy_stride = dy_stride;
    if (rows > 0) p.x = *x_ckpt;
    p.rows = rows; p.out_features = int(out_features); p.in_features = int(in_features);
    p.dw = dweight; p.dw_stride = dweight_stride;
    p.dw_bf16 = dtype == DPR_BF16; p.accumulate = accumulate != 0;
    if (ceil_div(out_features, 64) > 65535) return DPR_ERR_UNSUPPORTED;
    void* args[] = {&p};
    return record_cuda_status(launch_grid(
        (const void*)weight_grad_any,
        dim3(unsigned(ceil_div(in_features, 64)), unsigned(ceil_div(out_features, 64))), dim3(256),
        0, args, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
