// Activation checkpoints in 8 bits: saving (a peak, a step and a code for
// each block of 32 channels) and restoring, each one pass over the data.
#include <algorithm>

#include "ops_device.cuh"
#include "ops_kernels.h"

namespace dpr {

struct CkptParams {
    void* x;                // saved from, or restored to
    int64_t stride;
    dpr_checkpoint c;
    int64_t rows;
    int width;
};

namespace {

// Both directions stream at the rate of memory: 16384 x 4096 bf16 is saved in
// 29.5 us (6.9 TB/s of 2 + 1 + 1/32 bytes an element) and restored in 30.4 us;
// 8192 x 11008 in 40.0 and 42.1 us.  Single elements (odd rows): 16384 x 1001 bf16
// in 13.1 and 13.8 us, bound by one-element accesses.
//
// blockDim.x threads along a row (a multiple of the lanes that hold a block
// of channels, so that its peak is found within a warp), NV vectors of V
// channels each per thread (own_channel), blockDim.y rows per block; blockIdx.y counts
// along the row.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads) checkpoint_save(const __grid_constant__ CkptParams p) {
    grid_wait();
    grid_release();
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const int first = int(blockIdx.y) * int(blockDim.x) * V * NV;
    const bool live = row < p.rows;
    const int64_t r = live ? row : 0;
    const T* x = static_cast<const T*>(p.x) + r * p.stride + first;
    const int width = live ? p.width - first : 0;   // may be short of this block's end
    Raw<T, V> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = own_channel<V, NV>(i);
        zero_raw(raw[i]);
        if (c < width) load_raw(x + c, raw[i]);
    }
    save_row<T, V, NV>(raw, width, p.c.codes + r * p.c.code_stride + first,
                       p.c.steps + r * p.c.step_stride + first / kBlockChannels);
}

template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads) checkpoint_load(const __grid_constant__ CkptParams p) {
    grid_wait();
    grid_release();
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= p.rows) return;
    const int first = int(blockIdx.y) * int(blockDim.x) * V * NV;
    const int width = p.width - first;
    const int8_t* from = p.c.codes + row * p.c.code_stride + first;
    const uint8_t* steps = p.c.steps + row * p.c.step_stride + first / kBlockChannels;
    T* x = static_cast<T*>(p.x) + row * p.stride + first;
    CodeRaw<V> codes[NV];
    float step[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = own_channel<V, NV>(i);
        if (c >= width) continue;
        load_codes<V>(from + c, codes[i]);
        step[i] = step_value(steps[c / kBlockChannels]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = own_channel<V, NV>(i);
        if (c >= width) continue;
        float f[V];
        decode<V>(codes[i], step[i], f);
        Raw<T, V> raw;
        pack(f, raw);
        store_raw(x + c, raw);
    }
}

template <typename T, int V, int NV>
cudaError_t launch(CkptParams& p, bool save, cudaStream_t s) {
    const void* k = save ? (const void*)checkpoint_save<T, V, NV>
                         : (const void*)checkpoint_load<T, V, NV>;
    const int lanes = V == 1 ? 32 : kBlockChannels / V;
    // the fewest pieces of a row that fit a block, of even size
    const int64_t pieces = ceil_div(p.width, int64_t(kThreads) * V * NV);
    const RowShape f = row_shape(ceil_div(p.width, pieces), V * NV, lanes, kThreads);
    void* args[] = {&p};
    return launch_grid(k, dim3(unsigned(ceil_div(p.rows, f.per_block)),
                               unsigned(ceil_div(p.width, int64_t(f.threads) * V * NV))),
                       dim3(f.threads, f.per_block), 0, args, s);
}

dpr_status run(void* x, int64_t stride, int64_t rows, int64_t width, int dtype,
               const dpr_checkpoint* c, bool save, void* stream) {
    dpr_status st = check_matrix_size(rows, width);
    if (st != DPR_OK) return st;
    if (!dtype_ok(dtype) || !c) return DPR_ERR_INVALID_ARG;
    if (rows == 0) return DPR_OK;
    if ((st = check_matrix(x, stride, width, dtype, !save)) != DPR_OK) return st;
    if ((st = check_checkpoint(c, width)) != DPR_OK) return st;
    const int64_t es = dtype_size(dtype);
    SpanList v;
    v.add(x, matrix_bytes(rows, width, stride, es));
    v.add(*c, rows, width);
    if (!v.disjoint()) return DPR_ERR_ALIAS;

    CkptParams p = {};
    p.x = x; p.stride = stride; p.c = *c; p.rows = rows; p.width = int(width);
    const bool a32 = rows_aligned(x, stride, es, 32) && rows_aligned(c->codes, c->code_stride, 1, 16);
    const bool a16 = rows_aligned(x, stride, es, 16) && rows_aligned(c->codes, c->code_stride, 1, 8);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    const bool bf = dtype == DPR_BF16;
    switch (vector_elems(dtype, width, a32, a16)) {
        case 16: e = launch<uint16_t, 16, 1>(p, save, s); break;
        case 8: e = bf ? launch<uint16_t, 8, 1>(p, save, s) : launch<float, 8, 1>(p, save, s); break;
        default: e = bf ? launch<uint16_t, 1, 8>(p, save, s) : launch<float, 1, 8>(p, save, s);
    }
    return record_cuda_status(e);
}

}  // namespace
}  // namespace dpr

using namespace dpr;

extern "C" {

dpr_status dpr_checkpoint_save(const void* x, int64_t x_stride, int64_t rows, int64_t width,
                               int dtype, const dpr_checkpoint* ckpt, void* stream) {
    return run(const_cast<void*>(x), x_stride, rows, width, dtype, ckpt, true, stream);
}

dpr_status dpr_checkpoint_load(const dpr_checkpoint* ckpt, int64_t rows, int64_t width, void* out,
                               int64_t out_stride, int dtype, void* stream) {
    return run(out, out_stride, rows, width, dtype, ckpt, false, stream);
}

}  // extern "C"
