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
    uint32_t per_row;       // thread slots per row, a multiple of the lanes of a block of channels
    uint64_t slots;
};

namespace {

// Slot q is V channels of row q / per_row.  A block of channels is 32 / V
// neighbouring slots, and slots come in order of lanes, so its lanes meet in
// one warp.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) checkpoint_save(const __grid_constant__ CkptParams p) {
    grid_wait();
    grid_release();
    const uint64_t q = uint64_t(blockIdx.x) * kThreads + threadIdx.x;
    const bool in = q < p.slots;
    const int64_t row = in ? int64_t(q / p.per_row) : 0;
    const int c = in ? int(q % p.per_row) * V : 0;
    const bool on = in && c < p.width;
    Raw<T, V> raw;
    zero_raw(raw);
    if (on) load_raw(static_cast<const T*>(p.x) + row * p.stride + c, raw);
    save_vector(raw, c, on, p.c.codes + row * p.c.code_stride, p.c.steps + row * p.c.step_stride);
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) checkpoint_load(const __grid_constant__ CkptParams p) {
    grid_wait();
    grid_release();
    const uint64_t q = uint64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (q >= p.slots) return;
    const int64_t row = int64_t(q / p.per_row);
    const int c = int(q % p.per_row) * V;
    if (c >= p.width) return;
    CodeRaw<V> codes;
    load_codes<V>(p.c.codes + row * p.c.code_stride + c, codes);
    const float step = step_value(p.c.steps[row * p.c.step_stride + c / kBlockChannels]);
    float f[V];
    decode<V>(codes, step, f);
    Raw<T, V> raw;
    pack(f, raw);
    store_raw(static_cast<T*>(p.x) + row * p.stride + c, raw);
}

template <int V>
cudaError_t launch(CkptParams& p, const void* kernel, cudaStream_t s) {
    p.per_row = uint32_t(round_up(ceil_div(p.width, V), kBlockChannels / V));
    p.slots = uint64_t(p.rows) * p.per_row;
    void* args[] = {&p};
    return launch_grid(kernel, dim3(unsigned((p.slots + kThreads - 1) / kThreads)), dim3(kThreads),
                       0, args, s);
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
    // a grid's blocks are counted in 31 bits
    if (rows * round_up(width, kBlockChannels) / kThreads > (int64_t(1) << 30))
        return DPR_ERR_UNSUPPORTED;

    CkptParams p = {};
    p.x = x; p.stride = stride; p.c = *c; p.rows = rows; p.width = int(width);
    const bool a32 = rows_aligned(x, stride, es, 32) && rows_aligned(c->codes, c->code_stride, 1, 16);
    const bool a16 = rows_aligned(x, stride, es, 16) && rows_aligned(c->codes, c->code_stride, 1, 8);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    const bool bf = dtype == DPR_BF16;
    switch (vector_elems(dtype, width, a32, a16)) {
        case 16:
            e = launch<16>(p, save ? (const void*)checkpoint_save<uint16_t, 16>
                                   : (const void*)checkpoint_load<uint16_t, 16>, s);
            break;
        case 8:
            e = launch<8>(p, save ? (bf ? (const void*)checkpoint_save<uint16_t, 8>
                                        : (const void*)checkpoint_save<float, 8>)
                                  : (bf ? (const void*)checkpoint_load<uint16_t, 8>
                                        : (const void*)checkpoint_load<float, 8>), s);
            break;
        default:
            e = launch<1>(p, save ? (bf ? (const void*)checkpoint_save<uint16_t, 1>
                                        : (const void*)checkpoint_save<float, 1>)
                                  : (bf ? (const void*)checkpoint_load<uint16_t, 1>
                                        : (const void*)checkpoint_load<float, 1>), s);
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
