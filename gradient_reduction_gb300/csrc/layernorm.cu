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
    float count;            // width
    float inv_width;        // its rounded reciprocal
    int param_bf16;
    int param_vec;          // bytes an access of weight and bias may take
};

namespace {

template <int V>
__device__ __forceinline__ void load_affine(const NormParams& p, int c, float (&w)[V],
                                            float (&b)[V]) {
    if (p.weight) {
        load_params<V>(p.weight, p.param_bf16, p.param_vec, c, w);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) w[k] = 1.0f;
    }
    if (p.bias) {
        load_params<V>(p.bias, p.param_bf16, p.param_vec, c, b);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) b[k] = 0.0f;
    }
}

// Vector accesses.  blockDim.x threads share a row (see row_sum), blockDim.y
// rows at a time per block, the blocks' rows interleaved; each thread holds NV
// vectors of V elements and loads those of its next row while it works on one.
// Reads x, writes y: 4 bytes an element in bf16.  16384 x 4096 bf16: 50.5 us,
// 5.3 TB/s (0.78 of the measured copy rate), with both checkpoints written 80 us,
// 5.1 TB/s; 16384 x 8192 fp32: 165 us, 6.5 TB/s.  What bounds bf16 is the
// row's chain of two sums across the threads and its instructions (16 warps an
// SM at 110 registers, 56% of the issue slots used), not memory: fewer channels
// a thread (16: 57 us) or more (64: spills) are slower, and so are registers
// capped for more warps (104: 54 us) and copies into shared memory ahead of time
// (62 us), which cost more than the registers.
template <typename T, int V, int NV, bool kCkpt>
__global__ void __launch_bounds__(512) norm_rows(const __grid_constant__ NormParams p) {
    __shared__ float s[2][2][8][32];
    grid_wait();
    grid_release();
    const int tx = int(threadIdx.x), threads = int(blockDim.x);
    const int64_t stride = int64_t(gridDim.x) * blockDim.y;
    int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const T* x = static_cast<const T*>(p.x) + row * p.x_stride + tx * V;
    T* y = static_cast<T*>(p.y) + row * p.y_stride + tx * V;
    const int64_t x_step = stride * p.x_stride, y_step = stride * p.y_stride;
    Raw<T, V> next[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (row < p.rows && (i * threads + tx) * V < p.width) load_raw(x + i * threads * V, next[i]);
        else zero_raw(next[i]);
    }
    int turn = 0;
    // rows that share a warp take the same number of turns: their lanes work together
    const int64_t end = threads < 32 ? p.rows + (threadIdx.y & (32 / threads - 1)) : p.rows;
    for (; row < end; row += stride, y += y_step, turn ^= 1) {
        const bool live = row < p.rows;
        F2 d[NV][V / 2];
        F2 part = f2(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack2(next[i], d[i]);
#pragma unroll
            for (int k = 0; k < V / 2; ++k) part = add2(part, d[i][k]);
            if (kCkpt && p.x_ckpt.codes) {
                const int64_t r = live ? row : 0;
                const int c = (i * threads + tx) * V;
                save_vector(next[i], d[i], c, live && c < p.width,
                            p.x_ckpt.codes + r * p.x_ckpt.code_stride,
                            p.x_ckpt.steps + r * p.x_ckpt.step_stride);
            }
        }
        x += x_step;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (row + stride < p.rows && (i * threads + tx) * V < p.width)
                load_raw(x + i * threads * V, next[i]);
            else zero_raw(next[i]);
        }
        const float mean = divide(row_sum(total(part), s[turn][0]), p.count, p.inv_width);
        part = f2(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((i * threads + tx) * V < p.width) {
#pragma unroll
                for (int k = 0; k < V / 2; ++k) {
                    d[i][k] = add2(d[i][k], f2(-mean));
                    part = fma2(d[i][k], d[i][k], part);
                }
            }
        const float var = divide(row_sum(total(part), s[turn][1]), p.count, p.inv_width);
        const float rstd = inverse_sqrt(__fadd_rn(var, p.eps));
        if (tx == 0 && live) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * threads + tx) * V;
            const bool on = live && c < p.width;
            Raw<T, V> raw;
            if (on) {
                float w[V], b[V];
                load_affine<V>(p, c, w, b);
#pragma unroll
                for (int k = 0; k < V / 2; ++k)
                    d[i][k] = fma2(mul2(d[i][k], f2(rstd)), f2(w[2 * k], w[2 * k + 1]),
                                   f2(b[2 * k], b[2 * k + 1]));
                pack2(d[i], raw);
                store_raw(y + i * threads * V, raw);
            } else {
                zero_raw(raw);
            }
            if (kCkpt && p.y_ckpt.codes) {
                const int64_t r = live ? row : 0;
                save_vector(raw, c, on, p.y_ckpt.codes + r * p.y_ckpt.code_stride,
                            p.y_ckpt.steps + r * p.y_ckpt.step_stride);
            }
        }
    }
}

// Single elements: as above, one row (or blockDim.y of them) per block, NV
// elements a thread in registers, at fixed distances (own_channel).  3001 x
// 1003 fp32: 7.1 us, 3.4 TB/s; 16384 x 1001 bf16: 27 us, bound by its loads and
// stores of single elements (54 us with both checkpoints, by quantising them).
// A persistent loop is slower (34 us): a block that ends makes room at once for
// one whose loads overlap the others' sums.
template <typename T, int NV, bool kCkpt>
__global__ void __launch_bounds__(1024) norm_rows_any(const __grid_constant__ NormParams p) {
    __shared__ float s[2][8][32];
    grid_wait();
    grid_release();
    const int tx = int(threadIdx.x);
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < p.rows;   // the barriers below are for the whole block
    const int64_t r = live ? row : 0;
    const int width = live ? p.width : 0;
    const T* x = static_cast<const T*>(p.x) + r * p.x_stride;
    Raw<T, 1> raw[NV];
    float d[NV], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = own_channel<1, NV>(i);
        zero_raw(raw[i]);
        if (c < width) load_raw(x + c, raw[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[1];
        unpack(raw[i], f);
        d[i] = f[0];
        sum = __fadd_rn(sum, d[i]);
    }
    const float mean = divide(row_sum(sum, s[0]), p.count, p.inv_width);
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        d[i] = own_channel<1, NV>(i) < width ? __fsub_rn(d[i], mean) : 0.0f;
        sq = __fmaf_rn(d[i], d[i], sq);
    }
    const float var = divide(row_sum(sq, s[1]), p.count, p.inv_width);
    const float rstd = inverse_sqrt(__fadd_rn(var, p.eps));
    if (tx == 0 && live) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    if (kCkpt && p.x_ckpt.codes)
        save_row<T, 1, NV>(raw, width, p.x_ckpt.codes + r * p.x_ckpt.code_stride,
                           p.x_ckpt.steps + r * p.x_ckpt.step_stride);
    T* y = static_cast<T*>(p.y) + r * p.y_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = own_channel<1, NV>(i);
        zero_raw(raw[i]);
        if (c < width) {
            float f[1], w[1], b[1];
            load_affine<1>(p, c, w, b);
            f[0] = __fmaf_rn(__fmul_rn(d[i], rstd), w[0], b[0]);
            pack(f, raw[i]);
            store_raw(y + c, raw[i]);
        }
    }
    if (kCkpt && p.y_ckpt.codes)
        save_row<T, 1, NV>(raw, width, p.y_ckpt.codes + r * p.y_ckpt.code_stride,
                           p.y_ckpt.steps + r * p.y_ckpt.step_stride);
}

// Rows too long for registers (more than 24576 channels, or 16384 single
// elements): one block of 1024 threads per row, which reads the row three
// times (from L2 after the first).
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
    const float mean = divide(row_sum(sum, s[0]), p.count, p.inv_width);
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
    const float var = divide(row_sum(sq, s[1]), p.count, p.inv_width);
    const float rstd = inverse_sqrt(__fadd_rn(var, p.eps));
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
        if (p.x_ckpt.codes) {
            const Raw<T, V> one[1] = {raw};
            save_row<T, V, 1>(one, p.width - c0, p.x_ckpt.codes + row * p.x_ckpt.code_stride + c0,
                              p.x_ckpt.steps + row * p.x_ckpt.step_stride + c0 / kBlockChannels);
        }
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
            const Raw<T, V> one[1] = {raw};
            save_row<T, V, 1>(one, p.width - c0, p.y_ckpt.codes + row * p.y_ckpt.code_stride + c0,
                              p.y_ckpt.steps + row * p.y_ckpt.step_stride + c0 / kBlockChannels);
        }
    }
}

constexpr int kBlock = 128;              // threads of a block, or one row's if more
// The same for single elements: a block lives for one row each of its threads,
// and with smaller blocks starting them takes the time (16384 x 1001 bf16 in
// blocks of 128, 256 and 512: 51, 32 and 27 us); the checkpoints' registers leave
// room for fewer of the large ones (100, 64 and 66 us when a checkpoint took more instructions).
constexpr int kBlockAny = 512;
constexpr int kBlockAnyCkpt = 256;
template <typename T, int V, int NV>
cudaError_t launch_rows(const NormParams& p, cudaStream_t s) {
    const RowShape f = row_shape(p.width, V * NV, kBlockChannels / V, kBlock);
    const void* k = p.x_ckpt.codes || p.y_ckpt.codes ? (const void*)norm_rows<T, V, NV, true>
                                                     : (const void*)norm_rows<T, V, NV, false>;
    int64_t resident = 0;
    const cudaError_t e = resident_blocks(k, f.threads * f.per_block, &resident);
    if (e != cudaSuccess) return e;
    void* args[] = {const_cast<NormParams*>(&p)};
    return launch_grid(k, dim3(unsigned(std::min(resident, ceil_div(p.rows, f.per_block)))),
                       dim3(f.threads, f.per_block), 0, args, s);
}

template <typename T, int NV>
cudaError_t launch_rows_any(const NormParams& p, cudaStream_t s) {
    const bool ckpt = p.x_ckpt.codes || p.y_ckpt.codes;
    const RowShape f = row_shape(p.width, NV, 32, ckpt ? kBlockAnyCkpt : kBlockAny);
    const void* k = ckpt ? (const void*)norm_rows_any<T, NV, true>
                         : (const void*)norm_rows_any<T, NV, false>;
    void* args[] = {const_cast<NormParams*>(&p)};
    return launch_grid(k, dim3(unsigned(ceil_div(p.rows, f.per_block))),
                       dim3(f.threads, f.per_block), 0, args, s);
}

template <typename T, int V>
cudaError_t launch_long(const NormParams& p, cudaStream_t s) {
    void* args[] = {const_cast<NormParams*>(&p)};
    return launch_grid((const void*)norm_long_rows<T, V>, dim3(unsigned(p.rows)), dim3(1024), 0,
                       args, s);
}

// Channels per thread: 32, so that a row's sums cross few threads; 48 where
// that lets an SM hold twice as many rows (8192 x 11008 bf16: 69 us against 89; in
// fp32 8 to 10 registers of a thread spill, in memory's shadow);
// one vector while 32 would leave the GPU short of threads.
template <typename T, int V>
cudaError_t launch_forward(const NormParams& p, cudaStream_t s) {
    const int64_t vecs = ceil_div(p.width, V);
    if (vecs <= 512 && p.rows * p.width < (1 << 22)) return launch_rows<T, V, 1>(p, s);
    const auto rows_per_sm = [&](int elems) {
        return 512 / std::max(row_shape(p.width, elems, kBlockChannels / V, 1).threads, 1);
    };
    if (p.width > 512 * 32 || (p.width > 4096 && rows_per_sm(48) >= 2 * rows_per_sm(32))) {
        if (p.width <= 512 * 48) return launch_rows<T, V, 48 / V>(p, s);
        return launch_long<T, V>(p, s);
    }
    return launch_rows<T, V, 32 / V>(p, s);
}

template <typename T>
cudaError_t launch_forward_any(const NormParams& p, cudaStream_t s) {
    // few rows: more threads for each (300 x 1003 fp32 3.5 -> 2.7 us; 3001 rows 8.6 -> 9.8)
    if (p.width <= 1024 * 4 && p.rows * p.width < (1 << 19)) return launch_rows_any<T, 4>(p, s);
    if (p.width <= 1024 * 8) return launch_rows_any<T, 8>(p, s);
    if (p.width <= 1024 * 16) return launch_rows_any<T, 16>(p, s);
    return launch_long<T, 1>(p, s);
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
    p.eps = eps; p.count = float(width); p.inv_width = 1.0f / float(width);
    p.param_bf16 = param_dtype == DPR_BF16;
    p.param_vec = param_access(weight, bias);
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
