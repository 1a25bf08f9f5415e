// Layer norm, forward: one pass over the activation, each row held in the
// registers of the threads that share it, mean and centred sum of squares
// taken one after the other from those registers (no cancellation, no second
// read).  Optionally the row's input and output also leave in the 8-bit
// checkpoint format while they are in registers.
#include <algorithm>

#include "ops_device.cuh"
#include "ops_kernels.h"

namespace dpr {

struct NormParams {
    const void* x;
    int64_t x_stride;
    const void* weight;     // NULL: ones
    const void* bias;       // NULL: zeros
    void* y;
    int64_t y_stride;
    float* mean;            // NULL: not stored
    float* rstd;
    dpr_checkpoint x_ckpt;  // codes NULL: none
    dpr_checkpoint y_ckpt;
    int64_t rows;
    int width;
    float eps;
    float inv_width;
    int param_bf16;
    int param_vec;          // weight and bias allow 16-byte accesses
};

namespace {

template <int V>
__device__ __forceinline__ void load_affine(const NormParams& p, int c, float (&w)[V],
                                            float (&b)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) { w[k] = 1.0f; b[k] = 0.0f; }
    if (p.weight) load_params<V>(p.weight, p.param_bf16, p.param_vec, c, w);
    if (p.bias) load_params<V>(p.bias, p.param_bf16, p.param_vec, c, b);
}

// blockDim.x threads (a multiple of 32) share a row, blockDim.y rows per
// block; each thread holds NV vectors of V elements, vector i at
// (i * blockDim.x + threadIdx.x) * V.
template <typename T, int V, int NV, bool kCkpt>
__global__ void __launch_bounds__(1024) norm_rows(const __grid_constant__ NormParams p) {
    __shared__ float s[2][32][32];
    grid_wait();
    grid_release();
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < p.rows;   // the barriers below are for the whole block
    const T* x = static_cast<const T*>(p.x) + (live ? row : 0) * p.x_stride;

    Raw<T, V> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * int(blockDim.x) + int(threadIdx.x)) * V;
        zero_raw(raw[i]);
        if (live && c < p.width) load_raw(x + c, raw[i]);
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[V];
        unpack(raw[i], f);
#pragma unroll
        for (int k = 0; k < V; ++k) sum = __fadd_rn(sum, f[k]);
    }
    const float mean = __fmul_rn(row_sum(sum, s[0]), p.inv_width);
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * int(blockDim.x) + int(threadIdx.x)) * V;
        if (c < p.width) {
            float f[V];
            unpack(raw[i], f);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float d = __fsub_rn(f[k], mean);
                sq = __fmaf_rn(d, d, sq);
            }
        }
    }
    const float var = __fmul_rn(row_sum(sq, s[1]), p.inv_width);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, p.eps)));
    if (threadIdx.x == 0 && live) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }

    T* y = static_cast<T*>(p.y) + (live ? row : 0) * p.y_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * int(blockDim.x) + int(threadIdx.x)) * V;
        const bool on = live && c < p.width;
        float f[V], w[V], b[V];
        unpack(raw[i], f);
        if (kCkpt && p.x_ckpt.codes)
            save_vector<V>(f, c, on, p.x_ckpt.codes + (live ? row : 0) * p.x_ckpt.code_stride,
                           p.x_ckpt.steps + (live ? row : 0) * p.x_ckpt.step_stride);
        Raw<T, V> out;
        zero_raw(out);
        if (on) {
            load_affine<V>(p, c, w, b);
#pragma unroll
            for (int k = 0; k < V; ++k)
                f[k] = __fmaf_rn(__fmul_rn(__fsub_rn(f[k], mean), rstd), w[k], b[k]);
            pack(f, out);
            store_raw(y + c, out);
        }
        if (kCkpt && p.y_ckpt.codes) {
            unpack(out, f);
            save_vector<V>(f, c, on, p.y_ckpt.codes + (live ? row : 0) * p.y_ckpt.code_stride,
                           p.y_ckpt.steps + (live ? row : 0) * p.y_ckpt.step_stride);
        }
    }
}

// Rows too long for registers: one block of 1024 threads per row, which
// reads the row three times (from L2 after the first).
template <typename T, int V>
__global__ void __launch_bounds__(1024) norm_long_rows(const __grid_constant__ NormParams p) {
    __shared__ float s[2][32][32];
    grid_wait();
    grid_release();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
    T* y = static_cast<T*>(p.y) + row * p.y_stride;
    const int first = int(threadIdx.x) * V, step = int(blockDim.x) * V;
    Raw<T, V> raw;
    float f[V], w[V], b[V];
    float sum = 0.0f;
    for (int c = first; c < p.width; c += step) {
        load_raw(x + c, raw);
        unpack(raw, f);
#pragma unroll
        for (int k = 0; k < V; ++k) sum = __fadd_rn(sum, f[k]);
    }
    const float mean = __fmul_rn(row_sum(sum, s[0]), p.inv_width);
    float sq = 0.0f;
    for (int c = first; c < p.width; c += step) {
        load_raw(x + c, raw);
        unpack(raw, f);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float d = __fsub_rn(f[k], mean);
            sq = __fmaf_rn(d, d, sq);
        }
    }
    const float var = __fmul_rn(row_sum(sq, s[1]), p.inv_width);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, p.eps)));
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    // the same trip count for every thread: the lanes of a block of channels
    // take its peak together
    for (int c0 = 0; c0 < p.width; c0 += step) {
        const int c = c0 + first;
        const bool on = c < p.width;
        zero_raw(raw);
        if (on) load_raw(x + c, raw);
        unpack(raw, f);
        if (p.x_ckpt.codes)
            save_vector<V>(f, c, on, p.x_ckpt.codes + row * p.x_ckpt.code_stride,
                           p.x_ckpt.steps + row * p.x_ckpt.step_stride);
        zero_raw(raw);
        if (on) {
            load_affine<V>(p, c, w, b);
#pragma unroll
            for (int k = 0; k < V; ++k)
                f[k] = __fmaf_rn(__fmul_rn(__fsub_rn(f[k], mean), rstd), w[k], b[k]);
            pack(f, raw);
            store_raw(y + c, raw);
        }
        if (p.y_ckpt.codes) {
            unpack(raw, f);
            save_vector<V>(f, c, on, p.y_ckpt.codes + row * p.y_ckpt.code_stride,
                           p.y_ckpt.steps + row * p.y_ckpt.step_stride);
        }
    }
}

template <typename T, int V, int NV>
cudaError_t launch_rows(const NormParams& p, int threads, int per_block, cudaStream_t s) {
    const bool ckpt = p.x_ckpt.codes || p.y_ckpt.codes;
    const void* k = ckpt ? (const void*)norm_rows<T, V, NV, true>
                         : (const void*)norm_rows<T, V, NV, false>;
    void* args[] = {const_cast<NormParams*>(&p)};
    return launch_grid(k, dim3(unsigned(ceil_div(p.rows, per_block))), dim3(threads, per_block), 0,
                       args, s);
}

template <typename T, int V>
cudaError_t launch_long(const NormParams& p, cudaStream_t s) {
    void* args[] = {const_cast<NormParams*>(&p)};
    return launch_grid((const void*)norm_long_rows<T, V>, dim3(unsigned(p.rows)), dim3(1024), 0,
                       args, s);
}

// Vectors per thread and threads per row: NV small while the row's vectors
// still fit 1024 threads; short rows share a block of 256 threads.
template <typename T, int V, int N1, int N2>
cudaError_t launch_forward(const NormParams& p, cudaStream_t s) {
    const int64_t vecs = ceil_div(p.width, V);
    if (vecs > 1024 * N2) return launch_long<T, V>(p, s);
    const int nv = vecs > 1024 * N1 ? N2 : N1;
    const int threads = int(round_up(ceil_div(vecs, nv), 32));
    const int per_block = std::max(1, 256 / threads);
    return nv == N1 ? launch_rows<T, V, N1>(p, threads, per_block, s)
                    : launch_rows<T, V, N2>(p, threads, per_block, s);
}

}  // namespace
}  // namespace dpr

using namespace dpr;

extern "C" dpr_status dpr_layernorm_forward(const void* x, int64_t x_stride, int64_t rows,
                                            int64_t width, int dtype, const void* weight,
                                            const void* bias, int param_dtype, float eps, void* y,
                                            int64_t y_stride, float* mean, float* rstd,
                                            const dpr_checkpoint* x_ckpt,
                                            const dpr_checkpoint* y_ckpt, void* stream) {
    dpr_status st = check_matrix_size(rows, width);
    if (st != DPR_OK) return st;
    if (!dtype_ok(dtype) || !dtype_ok(param_dtype) || !(eps >= 0.0f)) return DPR_ERR_INVALID_ARG;
    if (rows == 0) return DPR_OK;
    if ((st = check_matrix(x, x_stride, width, dtype, false)) != DPR_OK) return st;
    if ((st = check_matrix(y, y_stride, width, dtype, true)) != DPR_OK) return st;
    const int64_t ps = dtype_size(param_dtype), es = dtype_size(dtype);
    if (!aligned(weight, uintptr_t(ps)) || !aligned(bias, uintptr_t(ps)) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return DPR_ERR_ALIGNMENT;
    for (const dpr_checkpoint* c : {x_ckpt, y_ckpt})
        if (c && (st = check_checkpoint(c, width)) != DPR_OK) return st;

    std::vector<Span> outs, ins;
    const Span xs = span_of(x, matrix_bytes(rows, width, x_stride, es));
    outs.push_back(span_of(y, matrix_bytes(rows, width, y_stride, es)));
    if (mean) outs.push_back(span_of(mean, uint64_t(rows) * 4));
    if (rstd) outs.push_back(span_of(rstd, uint64_t(rows) * 4));
    for (const dpr_checkpoint* c : {x_ckpt, y_ckpt})
        if (c) add_spans(*c, rows, width, &outs);
    if (!pairwise_disjoint(outs)) return DPR_ERR_ALIAS;
    if (weight) ins.push_back(span_of(weight, uint64_t(width * ps)));
    if (bias) ins.push_back(span_of(bias, uint64_t(width * ps)));
    if (any_overlap(outs, ins)) return DPR_ERR_ALIAS;
    // x may be y itself; nothing else may overlap it
    if (y == x && y_stride == x_stride) outs.erase(outs.begin());
    if (any_overlap(outs, {xs})) return DPR_ERR_ALIAS;

    NormParams p = {};
    p.x = x; p.x_stride = x_stride;
    p.weight = weight; p.bias = bias;
    p.y = y; p.y_stride = y_stride;
    p.mean = mean; p.rstd = rstd;
    bool a32 = rows_aligned(x, x_stride, es, 32) && rows_aligned(y, y_stride, es, 32);
    bool a16 = rows_aligned(x, x_stride, es, 16) && rows_aligned(y, y_stride, es, 16);
    for (const dpr_checkpoint* c : {x_ckpt, y_ckpt}) {
        if (!c) continue;
        (c == x_ckpt ? p.x_ckpt : p.y_ckpt) = *c;
        a32 = a32 && rows_aligned(c->codes, c->code_stride, 1, 16);
        a16 = a16 && rows_aligned(c->codes, c->code_stride, 1, 8);
    }
    p.rows = rows; p.width = int(width);
    p.eps = eps; p.inv_width = 1.0f / float(width);
    p.param_bf16 = param_dtype == DPR_BF16;
    p.param_vec = aligned(weight, 16) && aligned(bias, 16);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (vector_elems(dtype, width, a32, a16)) {
        case 16: e = launch_forward<uint16_t, 16, 1, 2>(p, s); break;
        case 8:
            e = dtype == DPR_BF16 ? launch_forward<uint16_t, 8, 1, 4>(p, s)
                                  : launch_forward<float, 8, 1, 4>(p, s);
            break;
        default:
            e = dtype == DPR_BF16 ? launch_forward<uint16_t, 1, 4, 16>(p, s)
                                  : launch_forward<float, 1, 4, 16>(p, s);
    }
    return record_cuda_status(e);
}
