// RMS norm of the sum of an activation and the residual stream, forward: one
// pass, each row held in the registers of the threads that share it.
// Optionally the sum and the output also leave in the 8-bit checkpoint format
// while they are in registers.
#include <algorithm>

#include "ops_device.cuh"
#include "ops_kernels.h"

namespace dpr {

struct RmsParams {
    const void* x;
    int64_t x_stride;
    const void* residual;   // NULL: none
    int64_t residual_stride;
    const void* weight;     // NULL: ones
    void* h;                // NULL: not stored
    int64_t h_stride;
    void* y;                // NULL: not stored
    int64_t y_stride;
    float* rstd;            // NULL: not stored
    dpr_checkpoint h_ckpt;  // codes NULL: none
    dpr_checkpoint y_ckpt;
    int64_t rows;
    int width;
    float eps;
    float count;            // width
    float inv_width;        // its rounded reciprocal
    int param_bf16;
    int param_vec;          // bytes an access of the weight may take
};

namespace {

template <int V>
__device__ __forceinline__ void load_weight(const RmsParams& p, int c, float (&w)[V]) {
    if (p.weight) {
        load_params<V>(p.weight, p.param_bf16, p.param_vec, c, w);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) w[k] = 1.0f;
    }
}

// V elements of h = x + residual, rounded to T.
template <typename T, int V>
__device__ __forceinline__ void add_residual(Raw<T, V>& x, const Raw<T, V>& residual) {
    float a[V], b[V];
    unpack(x, a);
    unpack(residual, b);
#pragma unroll
    for (int k = 0; k < V; ++k) a[k] = __fadd_rn(a[k], b[k]);
    pack(a, x);
}

// blockDim.x threads share a row (see row_sum), NV vectors of V elements each;
// blockDim.y rows per block.  All of a row's loads are in flight before its sum.
// 16384 x 4096 bf16: 41.8 us (6.4 TB/s, 0.95 of the measured copy rate), with the
// residual 78 us (1.02), and with both checkpoints 98.5 us (1.01).  One row of 4096:
// 2.0 us.  Single elements (rows that start anywhere): 16384 x 1001 bf16 36 us, 0.54
// of the copy rate, by instructions.
template <typename T, int V, int NV, bool kCkpt>
__global__ void __launch_bounds__(V == 1 ? 1024 : 512)
rms_rows(const __grid_constant__ RmsParams p) {
    __shared__ float s[8][32];
    grid_wait();
    grid_release();
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < p.rows;   // the barrier below is for the whole block
    const int64_t r = live ? row : 0;
    const int width = live ? p.width : 0;
    const T* x = static_cast<const T*>(p.x) + r * p.x_stride;
    const T* residual = static_cast<const T*>(p.residual) + r * p.residual_stride;
    Raw<T, V> raw[NV], other[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = own_channel<V, NV>(i);
        zero_raw(raw[i]);
        if (c < width) load_raw(x + c, raw[i]);
    }
    if (p.residual) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = own_channel<V, NV>(i);
            zero_raw(other[i]);
            if (c < width) load_raw(residual + c, other[i]);
        }
        T* h = static_cast<T*>(p.h) + r * p.h_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = own_channel<V, NV>(i);
            add_residual(raw[i], other[i]);
            if (p.h && c < width) store_raw(h + c, raw[i]);
        }
    }
    float part[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[V];
        unpack(raw[i], f);
#pragma unroll
        for (int k = 0; k < V; ++k) part[k & 1] = __fmaf_rn(f[k], f[k], part[k & 1]);
    }
    if (kCkpt && p.h_ckpt.codes)
        save_row<T, V, NV>(raw, width, p.h_ckpt.codes + r * p.h_ckpt.code_stride,
                           p.h_ckpt.steps + r * p.h_ckpt.step_stride);
    const float sum = row_sum(__fadd_rn(part[0], part[1]), s);
    const float rstd = inverse_sqrt(__fadd_rn(divide(sum, p.count, p.inv_width), p.eps));
    if (threadIdx.x == 0 && live && p.rstd) p.rstd[row] = rstd;
    T* y = static_cast<T*>(p.y) + r * p.y_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = own_channel<V, NV>(i);
        if (c < width) {
            float f[V], w[V];
            unpack(raw[i], f);
            load_weight<V>(p, c, w);
#pragma unroll
            for (int k = 0; k < V; ++k) f[k] = __fmul_rn(__fmul_rn(f[k], rstd), w[k]);
            pack(f, raw[i]);
            if (p.y) store_raw(y + c, raw[i]);
        }
    }
    if (kCkpt && p.y_ckpt.codes)
        save_row<T, V, NV>(raw, width, p.y_ckpt.codes + r * p.y_ckpt.code_stride,
                           p.y_ckpt.steps + r * p.y_ckpt.step_stride);
}

// Rows too long for registers (more than 16384 channels): one block of 1024
// threads per row, which reads the row twice (from L2 the second time).
template <typename T, int V>
__global__ void __launch_bounds__(1024) rms_long_rows(const __grid_constant__ RmsParams p) {
    __shared__ float s[1][32];
    grid_wait();
    grid_release();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
    const T* residual = static_cast<const T*>(p.residual) + row * p.residual_stride;
    T* h = static_cast<T*>(p.h) + row * p.h_stride;
    T* y = static_cast<T*>(p.y) + row * p.y_stride;
    const int first = int(threadIdx.x) * V, step = int(blockDim.x) * V;
    Raw<T, V> raw[1], other;
    float f[V], w[V], sum = 0.0f;
    for (int c = first; c < p.width; c += step) {
        load_raw(x + c, raw[0]);
        if (p.residual) {
            load_raw(residual + c, other);
            add_residual(raw[0], other);
        }
        unpack(raw[0], f);
#pragma unroll
        for (int k = 0; k < V; ++k) sum = __fmaf_rn(f[k], f[k], sum);
    }
    sum = row_sum(sum, s);
    const float rstd = inverse_sqrt(__fadd_rn(divide(sum, p.count, p.inv_width), p.eps));
    if (threadIdx.x == 0 && p.rstd) p.rstd[row] = rstd;
    // the same trip count for every thread: the lanes of a block of channels
    // take its peak together
    for (int c0 = 0; c0 < p.width; c0 += step) {
        const int c = c0 + first;
        const bool on = c < p.width;
        zero_raw(raw[0]);
        if (on) {
            load_raw(x + c, raw[0]);
            if (p.residual) {
                load_raw(residual + c, other);
                add_residual(raw[0], other);
                if (p.h) store_raw(h + c, raw[0]);
            }
        }
        if (p.h_ckpt.codes)
            save_row<T, V, 1>(raw, p.width - c0, p.h_ckpt.codes + row * p.h_ckpt.code_stride + c0,
                              p.h_ckpt.steps + row * p.h_ckpt.step_stride + c0 / kBlockChannels);
        if (on) {
            unpack(raw[0], f);
            load_weight<V>(p, c, w);
#pragma unroll
            for (int k = 0; k < V; ++k) f[k] = __fmul_rn(__fmul_rn(f[k], rstd), w[k]);
            pack(f, raw[0]);
            if (p.y) store_raw(y + c, raw[0]);
        }
        if (p.y_ckpt.codes)
            save_row<T, V, 1>(raw, p.width - c0, p.y_ckpt.codes + row * p.y_ckpt.code_stride + c0,
                              p.y_ckpt.steps + row * p.y_ckpt.step_stride + c0 / kBlockChannels);
    }
}

template <typename T, int V, int NV>
cudaError_t launch_rows(const RmsParams& p, cudaStream_t s) {
    const bool ckpt = p.h_ckpt.codes || p.y_ckpt.codes;
    const RowShape f = row_shape(p.width, V * NV, V == 1 ? 32 : kBlockChannels / V, 256);
    const void* k = ckpt ? (const void*)rms_rows<T, V, NV, true>
                         : (const void*)rms_rows<T, V, NV, false>;
    void* args[] = {const_cast<RmsParams*>(&p)};
    return launch_grid(k, dim3(unsigned(ceil_div(p.rows, f.per_block))),
                       dim3(f.threads, f.per_block), 0, args, s);
}

template <typename T, int V>
cudaError_t launch_long(const RmsParams& p, cudaStream_t s) {
    void* args[] = {const_cast<RmsParams*>(&p)};
    return launch_grid((const void*)rms_long_rows<T, V>, dim3(unsigned(p.rows)), dim3(1024), 0,
                       args, s);
}

// Blocks of 256 threads, of as many rows as they hold: an SM begins a block every
// 0.4 us, so short rows in blocks of 128 threads took 40 us for 32768 x 1024 bf16
// instead of 22.  Channels per thread: in bf16 32, as many bytes as 16 in fp32
// (16384 x 4096, 16 and 32: 55.5 and 41.8 us; with the checkpoints 73.8 and 70.1; 512
// threads a block 44.6 and 95.6).  fp32 rows of 32 a thread are no faster, and with
// the checkpoints slower (8192 x 5120, 63 and 72 us).  Few rows wait for one row's
// latency: 1 x 4096 bf16 2.0 us with 16, 2.3 with 32.
constexpr int64_t kFewRows = 1024;
template <typename T, int V>
cudaError_t launch_forward(const RmsParams& p, cudaStream_t s) {
    const bool wide = sizeof(T) == 2 && p.rows >= kFewRows;
    if (p.width <= 512 * 16 && !wide) return launch_rows<T, V, 16 / V>(p, s);
    if (p.width <= 512 * 32) return launch_rows<T, V, 32 / V>(p, s);
    return launch_long<T, V>(p, s);
}

template <typename T>
cudaError_t launch_forward_any(const RmsParams& p, cudaStream_t s) {
    if (p.width <= 1024 * 8) return launch_rows<T, 1, 8>(p, s);
    if (p.width <= 1024 * 16) return launch_rows<T, 1, 16>(p, s);
    return launch_long<T, 1>(p, s);
}

}  // namespace
}  // namespace dpr

using namespace dpr;

extern "C" dpr_status dpr_rmsnorm_forward(const void* x, int64_t x_stride, const void* residual,
                                          int64_t residual_stride, int64_t rows, int64_t width,
                                          int dtype, const void* weight, int param_dtype, float eps,
                                          void* h, int64_t h_stride, void* y, int64_t y_stride,
                                          float* rstd, const dpr_checkpoint* h_ckpt,
                                          const dpr_checkpoint* y_ckpt, void* stream) {
    dpr_status st = check_matrix_size(rows, width);
    if (st != DPR_OK) return st;
    if (!dtype_ok(dtype) || !dtype_ok(param_dtype) || !(eps >= 0.0f)) return DPR_ERR_INVALID_ARG;
    if (rows == 0) return DPR_OK;
    if (h && !residual) return DPR_ERR_INVALID_ARG;
    if (!y && !y_ckpt) return DPR_ERR_INVALID_ARG;
    const int64_t ps = dtype_size(param_dtype), es = dtype_size(dtype);
    if ((st = check_matrix(x, x_stride, width, dtype, false)) != DPR_OK) return st;
    if (residual && (st = check_matrix(residual, residual_stride, width, dtype, false)) != DPR_OK)
        return st;
    if (h && (st = check_matrix(h, h_stride, width, dtype, true)) != DPR_OK) return st;
    if (y && (st = check_matrix(y, y_stride, width, dtype, true)) != DPR_OK) return st;
    if (!aligned(weight, uintptr_t(ps)) || !aligned(rstd, 4)) return DPR_ERR_ALIGNMENT;
    for (const dpr_checkpoint* c : {h_ckpt, y_ckpt})
        if (c && (st = check_checkpoint(c, width)) != DPR_OK) return st;

    // h and y may each be an input itself; nothing else that is written may overlap
    SpanList outs, ins;
    if (rstd) outs.add(rstd, uint64_t(rows) * 4);
    for (const dpr_checkpoint* c : {h_ckpt, y_ckpt})
        if (c) outs.add(*c, rows, width);
    if (weight) ins.add(weight, uint64_t(width * ps));
    struct Matrix { const void* p; int64_t stride; };
    for (const Matrix& in : {Matrix{x, x_stride}, Matrix{residual, residual_stride}}) {
        if (!in.p) continue;
        const Span is = span_of(in.p, matrix_bytes(rows, width, in.stride, es));
        if (outs.meets(is)) return DPR_ERR_ALIAS;
        for (const Matrix& out : {Matrix{h, h_stride}, Matrix{y, y_stride}}) {
            if (!out.p || (out.p == in.p && out.stride == in.stride)) continue;
            if (overlaps(is, span_of(out.p, matrix_bytes(rows, width, out.stride, es))))
                return DPR_ERR_ALIAS;
        }
    }
    if (h) outs.add(h, matrix_bytes(rows, width, h_stride, es));
    if (y) outs.add(y, matrix_bytes(rows, width, y_stride, es));
    if (!outs.disjoint() || outs.meets(ins)) return DPR_ERR_ALIAS;

    RmsParams p = {};
    p.x = x; p.x_stride = x_stride;
    p.residual = residual; p.residual_stride = residual_stride;
    p.weight = weight;
    p.h = h; p.h_stride = h_stride;
    p.y = y; p.y_stride = y_stride;
    p.rstd = rstd;
    bool a32 = rows_aligned(x, x_stride, es, 32), a16 = rows_aligned(x, x_stride, es, 16);
    for (const Matrix& m : {Matrix{residual, residual_stride}, Matrix{h, h_stride}, Matrix{y, y_stride}}) {
        if (!m.p) continue;
        a32 = a32 && rows_aligned(m.p, m.stride, es, 32);
        a16 = a16 && rows_aligned(m.p, m.stride, es, 16);
    }
    for (const dpr_checkpoint* c : {h_ckpt, y_ckpt}) {
        if (!c) continue;
        (c == h_ckpt ? p.h_ckpt : p.y_ckpt) = *c;
        a32 = a32 && rows_aligned(c->codes, c->code_stride, 1, 16);
        a16 = a16 && rows_aligned(c->codes, c->code_stride, 1, 8);
    }
    p.rows = rows; p.width = int(width);
    p.eps = eps; p.count = float(width); p.inv_width = 1.0f / float(width);
    p.param_bf16 = param_dtype == DPR_BF16;
    p.param_vec = param_access(weight, nullptr);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    const bool bf = dtype == DPR_BF16;
    switch (vector_elems(dtype, width, a32, a16)) {
        case 16: e = launch_forward<uint16_t, 16>(p, s); break;
        case 8: e = bf ? launch_forward<uint16_t, 8>(p, s) : launch_forward<float, 8>(p, s); break;
        default: e = bf ? launch_forward_any<uint16_t>(p, s) : launch_forward_any<float>(p, s);
    }
    return record_cuda_status(e);
}
