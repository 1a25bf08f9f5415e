// Host-side pieces shared by the backward-pass operators (internal): launch
// with any block size, argument checks, and the selection of access widths.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/dpr_step.h"
#include "dpr_kernels.h"
#include "host_checks.h"

namespace dpr {

// As launch_kernel, with a block shape and dynamic shared memory.
// `cluster`: consecutive blocks that form a cluster (a divisor of grid.x).
cudaError_t launch_grid(const void* kernel, dim3 grid, dim3 block, size_t smem, void** args,
                        cudaStream_t s, int cluster = 1);

bool programmatic_launch_enabled();   // defined beside launch_kernel

// Waits that have run out in the layer norm's backward kernels.
cudaError_t norm_wait_failures(unsigned int* count);
// And in the RMS norm's, and in the products grouped by expert.
cudaError_t rms_wait_failures(unsigned int* count);
cudaError_t grouped_wait_failures(unsigned int* count);

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

inline bool dtype_ok(int d) { return d == DPR_BF16 || d == DPR_FP32; }
inline int64_t dtype_size(int d) { return d == DPR_BF16 ? 2 : 4; }

// Bytes from the first to one past the last element of a strided matrix.
inline uint64_t matrix_bytes(int64_t rows, int64_t width, int64_t stride, int64_t size) {
    return rows > 0 ? uint64_t((rows - 1) * stride + width) * uint64_t(size) : 0;
}

// Is every row start of the matrix a multiple of `a` bytes?
inline bool rows_aligned(const void* p, int64_t stride, int64_t size, int64_t a) {
    return aligned(p, uintptr_t(a)) && (stride * size) % a == 0;
}

dpr_status check_matrix_size(int64_t rows, int64_t width);
// `written`: the rows must not overlap (an input's may, down to stride 0 for
// a broadcast row).
dpr_status check_matrix(const void* p, int64_t stride, int64_t width, int dtype, bool written);
dpr_status check_checkpoint(const dpr_checkpoint* c, int64_t width);

// The few buffers of one call, without allocating.
struct SpanList {
    Span v[12];
    int n = 0;
    void add(const void* p, uint64_t bytes) { v[n++] = span_of(p, bytes); }
    // a checkpoint's codes and steps
    void add(const dpr_checkpoint& c, int64_t rows, int64_t width) {
        add(c.codes, matrix_bytes(rows, width, c.code_stride, 1));
        add(c.steps, matrix_bytes(rows, ceil_div(width, DPR_CHECKPOINT_BLOCK), c.step_stride, 1));
    }
    bool meets(const Span& s) const {
        for (int i = 0; i < n; ++i)
            if (overlaps(v[i], s)) return true;
        return false;
    }
    bool meets(const SpanList& o) const {
        for (int i = 0; i < o.n; ++i)
            if (meets(o.v[i])) return true;
        return false;
    }
    bool disjoint() const {
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < i; ++j)
                if (overlaps(v[i], v[j])) return false;
        return true;
    }
};

// Blocks of `threads` threads (no dynamic shared memory) that are resident on
// the current device at once; remembered per kernel and size.
cudaError_t resident_blocks(const void* kernel, int threads, int64_t* blocks);

// Allows `kernel` that much dynamic shared memory, once per device (`done`: a
// bit for each, the kernel's own).
cudaError_t allow_shared_memory(const void* kernel, int bytes, std::atomic<uint64_t>* done);

// The map of a tensor in memory that TMA reads in boxes: `rank` (2 or 3) sizes
// and box sizes in elements from the innermost on, strides in bytes (multiples
// of 16) from the second dimension on.  Outside the tensor zeros are read.
cudaError_t encode_tensor_map(CUtensorMap* map, CUtensorMapDataType type, const void* p, int rank,
                              const int64_t* dims, const int64_t* strides, const int* box,
                              CUtensorMapSwizzle swizzle);

// Threads that share a row of `width` channels at `elems` per thread, and rows
// per block of at least `block` threads: a power of two below 32 (at least
// `least`, the lanes that hold a block of channels), else a multiple of 32.
struct RowShape {
    int threads, per_block;
};
inline RowShape row_shape(int64_t width, int elems, int least, int block) {
    const int64_t need = ceil_div(width, elems);
    int threads = 1;
    if (need > 16 || least > 16) threads = int(round_up(need, 32));
    else
        while (threads < need || threads < least) threads *= 2;
    return RowShape{threads, threads >= block ? 1 : block / threads};
}

// Bytes an access of parameters may take (NULL allows any).
inline int param_access(const void* weight, const void* bias) {
    if (aligned(weight, 32) && aligned(bias, 32)) return 32;
    return aligned(weight, 16) && aligned(bias, 16) ? 16 : 1;
}

// Elements per access for an activation of `dtype` whose rows are `width`
// long: 32-byte accesses (16 bf16 or 8 fp32 elements) or 16-byte ones (8
// bf16) where every row start allows it, else single elements.
// `aligned32`, `aligned16`: whether every matrix of the call has such rows.
inline int vector_elems(int dtype, int64_t width, bool aligned32, bool aligned16) {
    if (dtype == DPR_FP32) return aligned32 && width % 8 == 0 ? 8 : 1;
    if (aligned32 && width % 16 == 0) return 16;
    if (aligned16 && width % 8 == 0) return 8;
    return 1;
}

}  // namespace dpr
