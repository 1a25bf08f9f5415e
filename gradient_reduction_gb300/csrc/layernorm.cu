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

// One block of up to 1024 threads (a multiple of 32) per row; each thread
// holds NV vectors of V elements, vector i at (i * blockDim.x + threadIdx.x) *
// V.
template <typename T, int V, int NV, bool kCkpt>
__global__ void __launch_bounds__(1024) norm_rows(const __grid_constant__ NormParams p) {
    __shared__ float s[2][1][32];
    grid_wait();
    grid_release();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.x_stride;

    Raw<T, V> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * int(blockDim.x) + int(threadIdx.x)) * V;
        zero_raw(raw[i]);
        if (c < p.width) load_raw(x + c, raw[i]);
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
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }

    T* y = static_cast<T*>(p.y) + row * p.y_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * int(blockDim.x) + int(threadIdx.x)) * V;
        const bool on = c < p.width;
        float f[V], w[V], b[V];
        unpack(raw[i], f);
        if (kCkpt && p.x_ckpt.codes)
            save_vector(raw[i], c, on, p.x_ckpt.codes + row * p.x_ckpt.code_stride,
                        p.x_ckpt.steps + row * p.x_ckpt.step_stride);
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
        if (kCkpt && p.y_ckpt.codes)
            save_vector(out, c, on, p.y_ckpt.codes + row * p.y_ckpt.code_stride,
                        p.y_ckpt.steps + row * p.y_ckpt.step_stride);
    }
}

// Rows of up to 512 threads x 16 channels: as norm_rows, but each block keeps
// its channels' weight and bias in registers over many rows (the blocks' rows
// are interleaved) and loads the next row while it works on one.
template <typename T, int V, int NV, bool kCkpt>
__global__ void __launch_bounds__(512) norm_many_rows(const __grid_constant__ NormParams p) {
    constexpr int E = V * NV;
    __shared__ float s[2][2][8][32];
    grid_wait();
    grid_release();
    const int tx = int(threadIdx.x), threads = int(blockDim.x);
    F2 w[E / 2], b[E / 2];
    {
        float fw[E], fb[E];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * threads + tx) * V;
            float v[V], u[V];
#pragma unroll
            for (int k = 0; k < V; ++k) { v[k] = 1.0f; u[k] = 0.0f; }
            if (c < p.width) load_affine<V>(p, c, v, u);
#pragma unroll
            for (int k = 0; k < V; ++k) { fw[i * V + k] = v[k]; fb[i * V + k] = u[k]; }
        }
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
            w[k] = f2(fw[2 * k], fw[2 * k + 1]);
            b[k] = f2(fb[2 * k], fb[2 * k + 1]);
        }
    }
    const int64_t stride = int64_t(gridDim.x) * blockDim.y;
    int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    Raw<T, V> next[NV];
    const auto load = [&](int64_t r) {
        const T* x = static_cast<const T*>(p.x) + r * p.x_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * threads + tx) * V;
            zero_raw(next[i]);
            if (r < p.rows && c < p.width) load_raw(x + c, next[i]);
        }
    };
    load(row);
    int turn = 0;
    // the same number of turns for every row of a block: the barriers are shared
    for (int64_t first = int64_t(blockIdx.x) * blockDim.y; first < p.rows;
         first += stride, row += stride, turn ^= 1) {
        const bool live = row < p.rows;
        Raw<T, V> raw[NV];
        F2 d[E / 2];
        F2 sum = f2(0.0f);
        {
            float f[E];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                raw[i] = next[i];
                float v[V];
                unpack(raw[i], v);
#pragma unroll
                for (int k = 0; k < V; ++k) f[i * V + k] = v[k];
            }
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                d[k] = f2(f[2 * k], f[2 * k + 1]);
                sum = add2(sum, d[k]);
            }
        }
        load(row + stride);
        if (kCkpt && p.x_ckpt.codes) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * threads + tx) * V;
                save_vector(raw[i], c, live && c < p.width,
                            p.x_ckpt.codes + (live ? row : 0) * p.x_ckpt.code_stride,
                            p.x_ckpt.steps + (live ? row : 0) * p.x_ckpt.step_stride);
            }
        }
        const float mean = __fmul_rn(row_sum(total(sum), s[turn][0]), p.inv_width);
        F2 sq = f2(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool on = (i * threads + tx) * V < p.width;
            if constexpr (V == 1) {
                // a pair is two vectors: the centred value of a channel past the end is 0
                if (i & 1) {
                    float lo, hi;
                    halves(add2(d[i / 2], f2(-mean)), lo, hi);
                    if (!on) hi = 0.0f;
                    if ((i - 1) * threads + tx >= p.width) lo = 0.0f;
                    d[i / 2] = f2(lo, hi);
                    sq = fma2(d[i / 2], d[i / 2], sq);
                }
            } else if (on) {
#pragma unroll
                for (int k = i * V / 2; k < (i + 1) * V / 2; ++k) {
                    d[k] = add2(d[k], f2(-mean));
                    sq = fma2(d[k], d[k], sq);
                }
            }
        }
        const float var = __fmul_rn(row_sum(total(sq), s[turn][1]), p.inv_width);
        const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, p.eps)));
        if (tx == 0 && live) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        float f[E];
#pragma unroll
        for (int k = 0; k < E / 2; ++k)
            halves(fma2(mul2(d[k], f2(rstd)), w[k], b[k]), f[2 * k], f[2 * k + 1]);
        T* y = static_cast<T*>(p.y) + (live ? row : 0) * p.y_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * threads + tx) * V;
            const bool on = live && c < p.width;
            float v[V];
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = on ? f[i * V + k] : 0.0f;
            Raw<T, V> out;
            pack(v, out);
            if (on) store_raw(y + c, out);
            if (kCkpt && p.y_ckpt.codes)
                save_vector(out, c, on, p.y_ckpt.codes + (live ? row : 0) * p.y_ckpt.code_stride,
                            p.y_ckpt.steps + (live ? row : 0) * p.y_ckpt.step_stride);
        }
    }
}

// Rows too long for registers: one block of 1024 threads per row, which
// reads the row three times (from L2 after the first).
template <typename T, int V>
__global__ void __launch_bounds__(1024) norm_long_rows(const __grid_constant__ NormParams p) {
    __shared__ float s[2][1][32];
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
            save_vector(raw, c, on, p.x_ckpt.codes + row * p.x_ckpt.code_stride,
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
        if (p.y_ckpt.codes)
            save_vector(raw, c, on, p.y_ckpt.codes + row * p.y_ckpt.code_stride,
                        p.y_ckpt.steps + row * p.y_ckpt.step_stride);
    }
}

template <typename T, int V, int NV>
cudaError_t launch_rows(const NormParams& p, int threads, cudaStream_t s) {
    const bool ckpt = p.x_ckpt.codes || p.y_ckpt.codes;
    const void* k = ckpt ? (const void*)norm_rows<T, V, NV, true>
                         : (const void*)norm_rows<T, V, NV, false>;
    void* args[] = {const_cast<NormParams*>(&p)};
    return launch_grid(k, dim3(unsigned(p.rows)), dim3(threads), 0, args, s);
}

template <typename T, int V>
cudaError_t launch_long(const NormParams& p, cudaStream_t s) {
    void* args[] = {const_cast<NormParams*>(&p)};
    return launch_grid((const void*)norm_long_rows<T, V>, dim3(unsigned(p.rows)), dim3(1024), 0,
                       args, s);
}

// 16 channels a thread up to 512 threads a row (norm_many_rows, blocks of at
// least 256 threads, 512 threads per SM); beyond that N1, then N2 vectors a
// thread of 1024 (norm_rows); then rows read three times.
constexpr int64_t kSms = 152;
template <typename T, int V, int N1, int N2>
cudaError_t launch_forward(const NormParams& p, cudaStream_t s) {
    constexpr int NV = 16 / V;
    if (p.width <= 512 * 16) {
        const int threads = int(round_up(ceil_div(p.width, V * NV), 32));
        const int per_block = std::max(1, 256 / threads);
        const int64_t resident = kSms * (512 / (threads * per_block));
        const int64_t blocks = std::min(resident, ceil_div(p.rows, per_block));
        const void* k = p.x_ckpt.codes || p.y_ckpt.codes ? (const void*)norm_many_rows<T, V, NV, true>
                                                         : (const void*)norm_many_rows<T, V, NV, false>;
        void* args[] = {const_cast<NormParams*>(&p)};
        return launch_grid(k, dim3(unsigned(blocks)), dim3(threads, per_block), 0, args, s);
    }
    const int64_t vecs = ceil_div(p.width, V);
    if (vecs > 1024 * N2) return launch_long<T, V>(p, s);
    const int nv = vecs > 1024 * N1 ? N2 : N1;
    const int threads = int(round_up(ceil_div(vecs, nv), 32));
    return nv == N1 ? launch_rows<T, V, N1>(p, threads, s) : launch_rows<T, V, N2>(p, threads, s);
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

    SpanList outs, ins;
    const Span xs = span_of(x, matrix_bytes(rows, width, x_stride, es));
    if (mean) outs.add(mean, uint64_t(rows) * 4);
    if (rstd) outs.add(rstd, uint64_t(rows) * 4);
    for (const dpr_checkpoint* c : {x_ckpt, y_ckpt})
        if (c) outs.add(*c, rows, width);
    // x may be y itself; nothing else may overlap it
    if (outs.meets(xs)) return DPR_ERR_ALIAS;
    const Span ys = span_of(y, matrix_bytes(rows, width, y_stride, es));
    if (!(y == x && y_stride == x_stride) && overlaps(xs, ys)) return DPR_ERR_ALIAS;
    outs.add(y, ys.hi - ys.lo);
    if (weight) ins.add(weight, uint64_t(width * ps));
    if (bias) ins.add(bias, uint64_t(width * ps));
    if (!outs.disjoint() || outs.meets(ins)) return DPR_ERR_ALIAS;

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
            e = dtype == DPR_BF16 ? launch_forward<uint16_t, 8, 2, 4>(p, s)
                                  : launch_forward<float, 8, 2, 4>(p, s);
            break;
        default:
            e = dtype == DPR_BF16 ? launch_forward<uint16_t, 1, 16, 16>(p, s)
                                  : launch_forward<float, 1, 16, 16>(p, s);
    }
    return record_cuda_status(e);
}
