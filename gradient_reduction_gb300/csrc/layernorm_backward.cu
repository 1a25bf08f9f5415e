// Layer norm, backward: dx needs two sums along every row, dweight and dbias
// one sum each down every column.
#include <algorithm>

#include "ops_device.cuh"
#include "ops_kernels.h"

namespace dpr {

struct NormGradParams {
    const void* dy;
    int64_t dy_stride;
    const void* x;            // the activation, or unused when ckpt.codes is set
    int64_t x_stride;
    dpr_checkpoint ckpt;
    const void* weight;       // NULL: ones
    const float* mean;
    const float* rstd;
    void* dx;
    int64_t dx_stride;
    float2* row_avg;          // [rows]: avg(g), avg(g * xhat)
    float* partial;           // [slices][2][width]: dweight and dbias of a slice of the rows
    int64_t rows;
    int width;
    int slices;
    int64_t slice_rows;       // rows per slice
    float inv_width;
    int param_bf16;
    int param_vec;
};

struct JoinParams {
    const float* partial;
    void* dweight;            // NULL: not wanted
    void* dbias;
    int width;
    int slices;
    int grad_bf16;
    int accumulate;
};

namespace {

// V elements of the row's x: the stored activation or its checkpoint.
template <typename T, int V, bool kSaved>
struct Source {
    Raw<T, V> raw;
    CodeRaw<V> codes;
    float step;

    __device__ __forceinline__ void load(const NormGradParams& p, int64_t row, int c) {
        if constexpr (kSaved) {
            load_codes<V>(p.ckpt.codes + row * p.ckpt.code_stride + c, codes);
            step = step_value(p.ckpt.steps[row * p.ckpt.step_stride + c / kBlockChannels]);
        } else {
            load_raw(static_cast<const T*>(p.x) + row * p.x_stride + c, raw);
        }
    }
    __device__ __forceinline__ void get(float (&f)[V]) const {
        if constexpr (kSaved) decode<V>(codes, step, f);
        else unpack(raw, f);
    }
};

// avg(g) and avg(g * xhat) of every row: blockDim.x threads per row.
template <typename T, int V, bool kSaved>
__global__ void __launch_bounds__(256) norm_grad_rows(const __grid_constant__ NormGradParams p) {
    __shared__ float s[2][32][32];
    grid_wait();
    grid_release();
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < p.rows;
    float a = 0.0f, b = 0.0f;
    if (live) {
        const float mean = p.mean[row], rstd = p.rstd[row];
        const T* dy = static_cast<const T*>(p.dy) + row * p.dy_stride;
        for (int c = int(threadIdx.x) * V; c < p.width; c += int(blockDim.x) * V) {
            Raw<T, V> rd;
            Source<T, V, kSaved> src;
            load_raw(dy + c, rd);
            src.load(p, row, c);
            float d[V], x[V], w[V];
            unpack(rd, d);
            src.get(x);
#pragma unroll
            for (int k = 0; k < V; ++k) w[k] = 1.0f;
            if (p.weight) load_params<V>(p.weight, p.param_bf16, p.param_vec, c, w);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float g = __fmul_rn(d[k], w[k]);
                a = __fadd_rn(a, g);
                b = __fmaf_rn(g, __fmul_rn(__fsub_rn(x[k], mean), rstd), b);
            }
        }
    }
    a = row_sum(a, s[0]);
    b = row_sum(b, s[1]);
    if (live && threadIdx.x == 0)
        p.row_avg[row] = make_float2(__fmul_rn(a, p.inv_width), __fmul_rn(b, p.inv_width));
}

// dx of a tile of 32 V columns by a slice of the rows, and the tile's column
// sums over the slice: threads (32, 8), row r of the slice at threadIdx.y =
// r % 8.
template <typename T, int V, bool kSaved>
__global__ void __launch_bounds__(256) norm_grad_columns(const __grid_constant__ NormGradParams p) {
    __shared__ float s[8][32 * V];
    grid_wait();
    grid_release();
    const int c = (int(blockIdx.x) * 32 + int(threadIdx.x)) * V;
    const bool on = c < p.width;
    const int64_t row0 = int64_t(blockIdx.y) * p.slice_rows;
    const int64_t row1 = min(row0 + p.slice_rows, p.rows);
    float dw[V], db[V], w[V];
#pragma unroll
    for (int k = 0; k < V; ++k) { dw[k] = 0.0f; db[k] = 0.0f; w[k] = 1.0f; }
    if (on) {
        if (p.weight) load_params<V>(p.weight, p.param_bf16, p.param_vec, c, w);
        for (int64_t row = row0 + threadIdx.y; row < row1; row += 8) {
            Raw<T, V> rd;
            Source<T, V, kSaved> src;
            load_raw(static_cast<const T*>(p.dy) + row * p.dy_stride + c, rd);
            src.load(p, row, c);
            const float mean = p.mean[row], rstd = p.rstd[row];
            const float2 avg = p.row_avg[row];
            float d[V], x[V];
            unpack(rd, d);
            src.get(x);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float h = __fmul_rn(__fsub_rn(x[k], mean), rstd);
                dw[k] = __fmaf_rn(d[k], h, dw[k]);
                db[k] = __fadd_rn(db[k], d[k]);
                const float g = __fsub_rn(__fmul_rn(d[k], w[k]), avg.x);
                d[k] = __fmul_rn(rstd, __fmaf_rn(-h, avg.y, g));
            }
            pack(d, rd);
            store_raw(static_cast<T*>(p.dx) + row * p.dx_stride + c, rd);
        }
    }
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        const int width = p.width, base = int(blockIdx.x) * 32 * V;
#pragma unroll
        for (int k = 0; k < V; ++k) s[threadIdx.y][threadIdx.x * V + k] = pass ? db[k] : dw[k];
        __syncthreads();
        for (int i = int(threadIdx.y) * 32 + int(threadIdx.x); i < 32 * V; i += 256) {
            float t = 0.0f;
#pragma unroll
            for (int y = 0; y < 8; ++y) t = __fadd_rn(t, s[y][i]);
            if (base + i < width)
                p.partial[(int64_t(blockIdx.y) * 2 + pass) * width + base + i] = t;
        }
        __syncthreads();
    }
}

// dweight and dbias from the slices' partial sums, added in slice order:
// 32 columns by 8 groups of slices per block; blockIdx.y picks the gradient.
__global__ void __launch_bounds__(256) norm_grad_join(const __grid_constant__ JoinParams p) {
    __shared__ float s[8][33];
    grid_wait();
    grid_release();
    void* out = blockIdx.y ? p.dbias : p.dweight;
    if (!out) return;
    const int c = int(blockIdx.x) * 32 + int(threadIdx.x);
    float t = 0.0f;
    if (c < p.width)
        for (int i = int(threadIdx.y); i < p.slices; i += 8)
            t = __fadd_rn(t, p.partial[(int64_t(i) * 2 + blockIdx.y) * p.width + c]);
    s[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.y != 0 || c >= p.width) return;
    t = 0.0f;
#pragma unroll
    for (int y = 0; y < 8; ++y) t = __fadd_rn(t, s[y][threadIdx.x]);
    if (p.grad_bf16) {
        uint16_t* o = static_cast<uint16_t*>(out) + c;
        *o = to_bf16(p.accumulate ? __fadd_rn(bf_1(*o), t) : t);
    } else {
        float* o = static_cast<float*>(out) + c;
        *o = p.accumulate ? __fadd_rn(*o, t) : t;
    }
}

// Slices of the rows: enough blocks for the GPU, at least 16 rows each.
constexpr int kMaxSlices = 256;
int slice_count(int64_t rows, int64_t width) {
    const int64_t tiles = ceil_div(width, 512);
    const int64_t want = std::max<int64_t>(1, (152 * 8) / tiles);
    return int(std::max<int64_t>(1, std::min<int64_t>({want, ceil_div(rows, 16), kMaxSlices})));
}

template <typename T, int V, bool kSaved>
cudaError_t launch_backward(NormGradParams& p, cudaStream_t s) {
    void* args[] = {&p};
    const int64_t vecs = ceil_div(p.width, V);
    const int threads = int(std::min<int64_t>(256, round_up(vecs, 32)));
    const int per_block = 256 / threads;
    cudaError_t e = launch_grid((const void*)norm_grad_rows<T, V, kSaved>,
                                dim3(unsigned(ceil_div(p.rows, per_block))),
                                dim3(threads, per_block), 0, args, s);
    if (e != cudaSuccess) return e;
    return launch_grid((const void*)norm_grad_columns<T, V, kSaved>,
                       dim3(unsigned(ceil_div(vecs, 32)), unsigned(p.slices)), dim3(32, 8), 0, args,
                       s);
}

template <typename T, int V>
cudaError_t launch_source(NormGradParams& p, cudaStream_t s) {
    return p.ckpt.codes ? launch_backward<T, V, true>(p, s) : launch_backward<T, V, false>(p, s);
}

}  // namespace
}  // namespace dpr

using namespace dpr;

extern "C" {

dpr_status dpr_layernorm_backward_workspace(int64_t rows, int64_t width, int64_t* bytes) {
    if (!bytes) return DPR_ERR_INVALID_ARG;
    *bytes = 0;
    const dpr_status st = check_matrix_size(rows, width);
    if (st != DPR_OK) return st;
    *bytes = round_up(rows * 8, 16) + int64_t(slice_count(rows, width)) * 2 * width * 4;
    return DPR_OK;
}

dpr_status dpr_layernorm_backward(const void* dy, int64_t dy_stride, const void* x,
                                  int64_t x_stride, const dpr_checkpoint* x_ckpt, int64_t rows,
                                  int64_t width, int dtype, const void* weight, int param_dtype,
                                  const float* mean, const float* rstd, void* dx,
                                  int64_t dx_stride, void* dweight, void* dbias, int grad_dtype,
                                  int accumulate, void* workspace, int64_t workspace_bytes,
                                  void* stream) {
    int64_t need = 0;
    dpr_status st = dpr_layernorm_backward_workspace(rows, width, &need);
    if (st != DPR_OK) return st;
    if (!dtype_ok(dtype) || !dtype_ok(param_dtype) || !dtype_ok(grad_dtype))
        return DPR_ERR_INVALID_ARG;
    const int64_t es = dtype_size(dtype), ps = dtype_size(param_dtype), gs = dtype_size(grad_dtype);
    if (!aligned(weight, uintptr_t(ps)) || !aligned(dweight, uintptr_t(gs)) ||
        !aligned(dbias, uintptr_t(gs)))
        return DPR_ERR_ALIGNMENT;
    std::vector<Span> outs, ins;
    if (dweight) outs.push_back(span_of(dweight, uint64_t(width * gs)));
    if (dbias) outs.push_back(span_of(dbias, uint64_t(width * gs)));
    if (weight) ins.push_back(span_of(weight, uint64_t(width * ps)));
    if (rows > 0) {
        if ((st = check_matrix(dy, dy_stride, width, dtype, false)) != DPR_OK) return st;
        if ((st = check_matrix(dx, dx_stride, width, dtype, true)) != DPR_OK) return st;
        if (x_ckpt) st = check_checkpoint(x_ckpt, width);
        else st = check_matrix(x, x_stride, width, dtype, false);
        if (st != DPR_OK) return st;
        if (!mean || !rstd || !workspace || workspace_bytes < need) return DPR_ERR_INVALID_ARG;
        if (!aligned(mean, 4) || !aligned(rstd, 4) || !aligned(workspace, 16))
            return DPR_ERR_ALIGNMENT;
        outs.push_back(span_of(workspace, uint64_t(need)));
        ins.push_back(span_of(mean, uint64_t(rows) * 4));
        ins.push_back(span_of(rstd, uint64_t(rows) * 4));
        if (x_ckpt) add_spans(*x_ckpt, rows, width, &ins);
        // dx may be dy or x itself; nothing else may overlap them
        const Span dxs = span_of(dx, matrix_bytes(rows, width, dx_stride, es));
        const Span dys = span_of(dy, matrix_bytes(rows, width, dy_stride, es));
        if (!(dx == dy && dx_stride == dy_stride) && overlaps(dxs, dys)) return DPR_ERR_ALIAS;
        if (!pairwise_disjoint(outs) || any_overlap(outs, {dys})) return DPR_ERR_ALIAS;
        if (!x_ckpt) {
            const Span xs = span_of(x, matrix_bytes(rows, width, x_stride, es));
            if (!(dx == x && dx_stride == x_stride) && overlaps(dxs, xs)) return DPR_ERR_ALIAS;
            if (any_overlap(outs, {xs})) return DPR_ERR_ALIAS;
        }
        outs.push_back(dxs);
    }
    if (!pairwise_disjoint(outs) || any_overlap(outs, ins)) return DPR_ERR_ALIAS;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    JoinParams j = {};
    j.dweight = dweight; j.dbias = dbias;
    j.width = int(width); j.grad_bf16 = grad_dtype == DPR_BF16; j.accumulate = accumulate != 0;
    cudaError_t e = cudaSuccess;
    if (rows > 0) {
        NormGradParams p = {};
        p.dy = dy; p.dy_stride = dy_stride;
        p.x = x; p.x_stride = x_stride;
        p.weight = weight;
        p.mean = mean; p.rstd = rstd;
        p.dx = dx; p.dx_stride = dx_stride;
        p.row_avg = static_cast<float2*>(workspace);
        p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + round_up(rows * 8, 16));
        p.rows = rows; p.width = int(width);
        p.slices = slice_count(rows, width);
        p.slice_rows = ceil_div(rows, p.slices);
        p.inv_width = 1.0f / float(width);
        p.param_bf16 = param_dtype == DPR_BF16;
        p.param_vec = aligned(weight, 16);
        bool a32 = rows_aligned(dy, dy_stride, es, 32) && rows_aligned(dx, dx_stride, es, 32);
        bool a16 = rows_aligned(dy, dy_stride, es, 16) && rows_aligned(dx, dx_stride, es, 16);
        if (x_ckpt) {
            p.ckpt = *x_ckpt;
            a32 = a32 && rows_aligned(x_ckpt->codes, x_ckpt->code_stride, 1, 16);
            a16 = a16 && rows_aligned(x_ckpt->codes, x_ckpt->code_stride, 1, 8);
        } else {
            a32 = a32 && rows_aligned(x, x_stride, es, 32);
            a16 = a16 && rows_aligned(x, x_stride, es, 16);
        }
        switch (vector_elems(dtype, width, a32, a16)) {
            case 16: e = launch_source<uint16_t, 16>(p, s); break;
            case 8:
                e = dtype == DPR_BF16 ? launch_source<uint16_t, 8>(p, s)
                                      : launch_source<float, 8>(p, s);
                break;
            default:
                e = dtype == DPR_BF16 ? launch_source<uint16_t, 1>(p, s)
                                      : launch_source<float, 1>(p, s);
        }
        if (e != cudaSuccess) return record_cuda_status(e);
        j.partial = p.partial; j.slices = p.slices;
    }
    if (dweight || dbias) {
        void* args[] = {&j};
        e = launch_grid((const void*)norm_grad_join, dim3(unsigned(ceil_div(width, 32)), 2),
                        dim3(32, 8), 0, args, s);
    }
    return record_cuda_status(e);
}

}  // extern "C"
