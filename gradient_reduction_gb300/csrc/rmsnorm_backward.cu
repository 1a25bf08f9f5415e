// RMS norm, backward: dx needs one sum along every row, dweight one down every
// column.  With n = h rstd and g = dy weight,
//   dx = dh + rstd (g - n avg(g n)),   dweight = sum_rows dy n.
// n, of about 1 in any row, comes first: rstd^3 avg(g h) takes as many operations,
// but its rstd^2 leaves fp32 for rows (and gradients) whose dx is well inside it.
//
// Rows of up to 8192 channels take one pass: the threads of a block own columns
// and keep their sums in registers over all of the block's rows; a second,
// small kernel joins the blocks' sums in a fixed order.  Rows of more than 512
// channels whose parts are 16-byte aligned are staged in shared memory
// (rms_grad_staged, in bf16 up to 16384 channels), the others loaded into
// registers a row ahead (rms_grad_rows).  What is left takes two passes, row
// sums first, then columns.
#include <algorithm>

#include "ops_device.cuh"
#include "ops_kernels.h"
#include "tensor_core.cuh"

namespace dpr {

struct RmsGradParams {
    const void* dy;
    int64_t dy_stride;
    const void* dh;           // NULL: none
    int64_t dh_stride;
    const void* h;            // or unused when ckpt.codes is set
    int64_t h_stride;
    dpr_checkpoint ckpt;
    const void* weight;       // NULL: ones
    const float* rstd;
    void* dx;
    int64_t dx_stride;
    float* row_avg;           // [rows]: avg(g n) (two passes)
    float* partial;           // [slices][partial_width]: dweight of a slice of the rows, or NULL
    int64_t rows;
    int width;
    int partial_width;        // width rounded up to 4
    int64_t slice_rows;       // rows per slice (two passes)
    int depth;                // rows of a group in flight (staged)
    float count;              // width
    float inv_width;          // its rounded reciprocal
    int param_bf16;
    int param_vec;
};

struct RmsJoinParams {
    const float* partial;
    void* dweight;
    int width;
    int partial_width;
    int slices;
    int grad_bf16;
    int accumulate;
};

namespace {

__device__ unsigned int g_wait_failures;

template <int V>
__device__ __forceinline__ void load_weight(const RmsGradParams& p, int c, float (&w)[V]) {
    if (p.weight) {
        load_params<V>(p.weight, p.param_bf16, p.param_vec, c, w);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) w[k] = 1.0f;
    }
}

// V elements of the row's h: the stored one or its checkpoint.
template <typename T, int V, bool kSaved>
struct RmsSource {
    Raw<T, V> raw;
    CodeRaw<V> codes;
    float step;

    __device__ __forceinline__ void load(const RmsGradParams& p, int64_t row, int c) {
        if constexpr (kSaved) {
            load_codes<V>(p.ckpt.codes + row * p.ckpt.code_stride + c, codes);
            step = step_value(p.ckpt.steps[row * p.ckpt.step_stride + c / kBlockChannels]);
        } else {
            load_raw(static_cast<const T*>(p.h) + row * p.h_stride + c, raw);
        }
    }
    __device__ __forceinline__ void zero() {
        if constexpr (kSaved) {
#pragma unroll
            for (int i = 0; i < int(sizeof(codes.w) / 4); ++i) codes.w[i] = 0;
            step = 0.0f;
        } else {
            zero_raw(raw);
        }
    }
    __device__ __forceinline__ void get(float (&f)[V]) const {
        if constexpr (kSaved) decode<V>(codes, step, f);
        else unpack(raw, f);
    }
};

// A block's column sums to its place among the partial sums: first over its
// rows-at-a-time, those that share a warp by exchanges, the others through
// `columns` ([groups - 1][threads * E] floats of shared memory).
template <int V, int NV>
__device__ __forceinline__ void store_columns(const RmsGradParams& p, F2 (&dw)[V * NV / 2],
                                              float* columns) {
    constexpr int E = V * NV;
    const int tx = int(threadIdx.x), threads = int(blockDim.x);
    if (!p.partial) return;
    int group = int(threadIdx.y), groups = int(blockDim.y);
    bool lead = true;
    if (threads < 32) {
        for (int d = threads; d < 32; d <<= 1) {
#pragma unroll
            for (int k = 0; k < E / 2; ++k)
                dw[k] = add2(dw[k], F2{__shfl_xor_sync(0xFFFFFFFFu, dw[k].v, d)});
        }
        const int thread = int(threadIdx.y) * threads + tx;
        group = thread >> 5;
        groups = threads * int(blockDim.y) >> 5;
        lead = (thread & 31) < threads;
    }
    if (groups > 1) {
        __syncthreads();
        if (group > 0 && lead) {
            float2* const mine = reinterpret_cast<float2*>(columns + (group - 1) * threads * E);
#pragma unroll
            for (int k = 0; k < E / 2; ++k) halves(dw[k], mine[k * threads + tx].x, mine[k * threads + tx].y);
        }
        __syncthreads();
        if (group > 0 || !lead) return;
        for (int y = 0; y + 1 < groups; ++y) {
            const float2* other = reinterpret_cast<const float2*>(columns + y * threads * E);
#pragma unroll
            for (int k = 0; k < E / 2; ++k)
                dw[k] = add2(dw[k], f2(other[k * threads + tx].x, other[k * threads + tx].y));
        }
    }
    float* to = p.partial + int64_t(blockIdx.x) * p.partial_width;
    float out[E];
#pragma unroll
    for (int k = 0; k < E / 2; ++k) halves(dw[k], out[2 * k], out[2 * k + 1]);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = own_channel<V, NV>(i);
        if (c < p.width) {
            if constexpr (V >= 4) {
#pragma unroll
                for (int k = 0; k < V; k += 4)
                    st_f4(to + c + k, out[i * V + k], out[i * V + k + 1], out[i * V + k + 2],
                          out[i * V + k + 3]);
            } else {
                to[c] = out[i];
            }
        }
    }
}

// blockDim.x threads (see row_sum; at most 512) share a row, NV vectors of V
// channels each; blockDim.y rows at a time per block, the blocks' rows
// interleaved.
template <typename T, int V, int NV, bool kSaved>
__global__ void __launch_bounds__(512) rms_grad_rows(const __grid_constant__ RmsGradParams p) {
    constexpr int E = V * NV;
    __shared__ float s[2][8][32];
    extern __shared__ float columns[];
    grid_wait();
    grid_release();
    // element i * V + k is half (i * V + k) & 1 of pair (i * V + k) / 2
    F2 w[E / 2], dw[E / 2];
    {
        float f[E];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = own_channel<V, NV>(i);
            float v[V] = {};
            if (c < p.width) load_weight<V>(p, c, v);
#pragma unroll
            for (int k = 0; k < V; ++k) f[i * V + k] = v[k];
        }
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
            w[k] = f2(f[2 * k], f[2 * k + 1]);
            dw[k] = f2(0.0f);
        }
    }
    const int64_t stride = int64_t(gridDim.x) * blockDim.y;
    int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    Raw<T, V> dy[NV], dh[NV];
    RmsSource<T, V, kSaved> h[NV];
    float rstd = 0.0f;
    const auto load = [&](int64_t r) {
        const bool live = r < p.rows;
        rstd = live ? p.rstd[r] : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = own_channel<V, NV>(i);
            if (live && c < p.width) {
                load_raw(static_cast<const T*>(p.dy) + r * p.dy_stride + c, dy[i]);
                h[i].load(p, r, c);
            } else {
                zero_raw(dy[i]);
                h[i].zero();
            }
        }
    };
    load(row);
    // the same number of turns for every row of a block: the barriers are shared
    int turn = 0;
    for (int64_t first = int64_t(blockIdx.x) * blockDim.y; first < p.rows;
         first += stride, row += stride, turn ^= 1) {
        F2 g[E / 2], x[E / 2];
        F2 sum = f2(0.0f);
        const F2 r = f2(rstd);
        const bool live = row < p.rows;
        {
            float d[E], f[E];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v[V];
                unpack(dy[i], v);
#pragma unroll
                for (int k = 0; k < V; ++k) d[i * V + k] = v[k];
                h[i].get(v);
#pragma unroll
                for (int k = 0; k < V; ++k) f[i * V + k] = v[k];
            }
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                // a channel past the row's end has d = 0 and x = 0
                const F2 dy2 = f2(d[2 * k], d[2 * k + 1]);
                x[k] = mul2(f2(f[2 * k], f[2 * k + 1]), r);
                g[k] = mul2(dy2, w[k]);
                sum = fma2(g[k], x[k], sum);
                dw[k] = fma2(dy2, x[k], dw[k]);
            }
        }
        if (p.dh) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = own_channel<V, NV>(i);
                zero_raw(dh[i]);
                if (live && c < p.width)
                    load_raw(static_cast<const T*>(p.dh) + row * p.dh_stride + c, dh[i]);
            }
        }
        load(row + stride);
        const float a = row_sum(total(sum), s[turn]);
        if (live) {
            const F2 minus = f2(-divide(a, p.count, p.inv_width));
            float d[E], r1, same;
            halves(r, r1, same);
#pragma unroll
            for (int k = 0; k < E / 2; ++k)
                halves(fma2(x[k], minus, g[k]), d[2 * k], d[2 * k + 1]);
            T* dx = static_cast<T*>(p.dx) + row * p.dx_stride;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = own_channel<V, NV>(i);
                if (c < p.width) {
                    float v[V];
                    if (p.dh) {
                        unpack(dh[i], v);
#pragma unroll
                        for (int k = 0; k < V; ++k) v[k] = __fmaf_rn(d[i * V + k], r1, v[k]);
                    } else {
#pragma unroll
                        for (int k = 0; k < V; ++k) v[k] = __fmul_rn(d[i * V + k], r1);
                    }
                    Raw<T, V> out;
                    pack(v, out);
                    store_raw(dx + c, out);
                }
            }
        }
    }
    store_columns<V, NV>(p, dw, columns);
}

__device__ __forceinline__ void load_shared(uint32_t at, uint32_t (&w)[4]) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
}
__device__ __forceinline__ void load_shared(uint32_t at, uint32_t (&w)[2]) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at));
}
__device__ __forceinline__ void load_shared(uint32_t at, uint32_t (&w)[1]) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at));
}

// Sum over the blockDim.x threads (64 to 512) that share threadIdx.y, with one
// barrier.  Two calls in a row need different `s`.
__device__ __forceinline__ float group_sum_all(float v, float (*s)[16]) {
    const int lane = int(threadIdx.x) & 31, nw = int(blockDim.x) >> 5, w = lane & 15;
    v = warp_sum(v);
    if (lane == 0) s[threadIdx.y][threadIdx.x >> 5] = v;
    row_barrier();
    return group_sum(w < nw ? s[threadIdx.y][w] : 0.0f, 16);
}

// As rms_grad_rows, for rows whose parts are 16-byte aligned.  One thread of
// each group of blockDim.x (at least 64) has its rows bulk-copied into shared
// memory, p.depth of them in all.  A thread owns 16-byte pieces of the row, piece i
// at i * blockDim.x + threadIdx.x; with 32 channels a thread there is no room for
// their weights in its registers, and it loads them for every row.
// 16384 x 4096 bf16 with dh and the join: 82 us, 6.5 TB/s (0.97 of the measured
// copy rate); from a checkpoint 80 us, 5.9 TB/s; without dh 67 and 73 us.  A row's
// chain of loads, sum, barrier and second half bounds the last three, with 16 warps an
// SM.  What was tried: dy and h unpacked again after the sum 91 and 96 us (22 and 31
// instructions an element); two rows a turn with their values in registers, the
// weights in shared memory, 86 and 111 us (fewer rows in flight).
constexpr int kMaxDepth = 8;
constexpr int kMaxGroups = 4;
template <typename T, bool kSaved, int NV>
__global__ void __launch_bounds__(512) rms_grad_staged(const __grid_constant__ RmsGradParams p) {
    constexpr int V = 16 / int(sizeof(T)), E = V * NV;
    __shared__ float s[2][kMaxGroups][16];
    __shared__ __align__(8) uint64_t bars[kMaxGroups][kMaxDepth];
    extern __shared__ __align__(16) uint8_t ring[];
    const int tx = int(threadIdx.x), threads = int(blockDim.x);
    const uint32_t full = tc::smem_addr(bars[threadIdx.y]);
    if (tx == 0) {
        for (int k = 0; k < p.depth; ++k) tc::mbar_init(full + 8 * k, 1);
        tc::mbar_init_fence();
    }
    __syncthreads();
    grid_wait();
    grid_release();
    const uint32_t dy_bytes = uint32_t(p.width) * sizeof(T);
    const uint32_t h_bytes = kSaved ? uint32_t(p.width) : dy_bytes;
    const uint32_t stage = dy_bytes + h_bytes + (p.dh ? dy_bytes : 0);
    const uint32_t mine = tc::smem_addr(ring) + threadIdx.y * p.depth * stage;
    const int rows = int(p.rows), stride = int(gridDim.x * blockDim.y);   // rows are counted in 30 bits
    const int row0 = int(blockIdx.x * blockDim.y + threadIdx.y);
    const auto fetch = [&](int64_t r, uint32_t k) {
        const void* h = kSaved ? static_cast<const void*>(p.ckpt.codes + r * p.ckpt.code_stride)
                               : static_cast<const T*>(p.h) + r * p.h_stride;
        const uint32_t to = mine + k * stage, bar = full + 8 * k;
        tc::mbar_expect(bar, stage);
        tc::bulk_load(to, static_cast<const T*>(p.dy) + r * p.dy_stride, dy_bytes, bar);
        tc::bulk_load(to + dy_bytes, h, h_bytes, bar);
        if (p.dh)
            tc::bulk_load(to + dy_bytes + h_bytes, static_cast<const T*>(p.dh) + r * p.dh_stride,
                          dy_bytes, bar);
        // a row's step bytes are a DRAM access of their own: asked for as early
        if constexpr (kSaved)
            for (int at = 0; at * kBlockChannels < p.width; at += 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.ckpt.steps + r * p.ckpt.step_stride + at));
    };
    uint32_t asked = 0;                 // rows fetched so far, by the first thread
    if (tx == 0)
        for (; asked < uint32_t(p.depth) && row0 + int(asked) * stride < rows; ++asked)
            fetch(row0 + int(asked) * stride, asked);

    constexpr bool kKeep = E <= 16;
    F2 w[kKeep ? E / 2 : 1], dw[E / 2];
    const auto weights = [&](int i, F2* to) {
        const int c = (i * threads + tx) * V;
        float v[V] = {};
        if (c < p.width) load_weight<V>(p, c, v);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) to[e] = f2(v[2 * e], v[2 * e + 1]);
    };
    if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < NV; ++i) weights(i, w + i * V / 2);
    }
#pragma unroll
    for (int k = 0; k < E / 2; ++k) dw[k] = f2(0.0f);
    // what does not come in 16-byte rows is loaded a turn ahead
    struct Small {
        float rstd, step[NV];
    };
    Small now, next;
    const auto load_small = [&](int64_t r, Small& m) {
        if (r >= rows) return;
        m.rstd = p.rstd[r];
        if constexpr (kSaved) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * threads + tx) * V;
                if (c < p.width)
                    m.step[i] = step_value(p.ckpt.steps[r * p.ckpt.step_stride + c / kBlockChannels]);
            }
        }
    };
    load_small(row0, now);
    T* dx = static_cast<T*>(p.dx) + row0 * p.dx_stride + tx * V;
    const int64_t dx_row = stride * p.dx_stride;
    uint32_t k = 0, parity = 0, last = 0;    // `last`: the stage of the turn before
    int turn = 0;
    bool ok = true;
    for (int row = row0; row < rows; row += stride, dx += dx_row, turn ^= 1) {
        F2 g[E / 2], n[E / 2];
        F2 sum = f2(0.0f);
        const F2 r2 = f2(now.rstd);
        const uint32_t at = mine + k * stage, first = k;
        if (ok) ok = tc::mbar_wait(full + 8 * k, parity);
        if (++k == uint32_t(p.depth)) { k = 0; parity ^= 1; }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t piece = uint32_t(i * threads + tx);
            if (int(piece) * V >= p.width) continue;
            Raw<T, V> raw;
            F2 d[V / 2], x[V / 2], mine_w[V / 2];
            if constexpr (kSaved) {
                CodeRaw<V> c;
                load_shared(at + dy_bytes + piece * V, c.w);
                decode2<V>(c, now.step[i], x);
            } else {
                load_shared(at + dy_bytes + piece * 16, raw.w);
                unpack2(raw, x);
            }
            load_shared(at + piece * 16, raw.w);
            unpack2(raw, d);
            if constexpr (!kKeep) weights(i, mine_w);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) {
                const int q = i * V / 2 + e;
                n[q] = mul2(x[e], r2);
                g[q] = mul2(d[e], kKeep ? w[kKeep ? q : 0] : mine_w[e]);
                sum = fma2(g[q], n[q], sum);
                dw[q] = fma2(d[e], n[q], dw[q]);
            }
        }
        load_small(row + stride, next);
        const float total_sum = group_sum_all(total(sum), s[turn]);
        // the whole group is past the turn before: its stage is free (after a failed
        // wait it is not known to be)
        if (tx == 0 && ok && row != row0 && row0 + int(asked) * stride < rows) {
            fetch(row0 + int(asked) * stride, last);
            ++asked;
        }
        last = first;
        const F2 minus = f2(-divide(total_sum, p.count, p.inv_width));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t piece = uint32_t(i * threads + tx);
            if (int(piece) * V >= p.width) continue;
            Raw<T, V> raw;
            F2 o[V / 2];
            if (p.dh) {
                load_shared(at + dy_bytes + h_bytes + piece * 16, raw.w);
                unpack2(raw, o);
#pragma unroll
                for (int e = 0; e < V / 2; ++e)
                    o[e] = fma2(fma2(n[i * V / 2 + e], minus, g[i * V / 2 + e]), r2, o[e]);
            } else {
#pragma unroll
                for (int e = 0; e < V / 2; ++e)
                    o[e] = mul2(fma2(n[i * V / 2 + e], minus, g[i * V / 2 + e]), r2);
            }
            pack2(o, raw);
            st_v4(dx + i * threads * V, make_uint4(raw.w[0], raw.w[1], raw.w[2], raw.w[3]));
        }
        now = next;
    }
    // One thread's wait may run out where the others' end, so the block counts it
    // as one, and lets what it has asked for land before the ring's memory is used
    // again or given up.
    if (__syncthreads_or(!ok)) {
        if (tx == 0) {
            if (threadIdx.y == 0) atomicAdd(&g_wait_failures, 1u);
            for (int j = 0; j < p.depth; ++j) {
                const uint32_t uses = asked / p.depth + (uint32_t(j) < asked % p.depth);
                if (uses > 0) tc::mbar_wait(full + 8 * j, (uses - 1) & 1);
            }
        }
        __syncthreads();
    }
    store_columns<V, NV>(p, dw, reinterpret_cast<float*>(ring));
}

// Two passes: avg(g n) of every row, blockDim.x threads per row.
template <typename T, int V, bool kSaved>
__global__ void __launch_bounds__(256) rms_grad_sums(const __grid_constant__ RmsGradParams p) {
    __shared__ float s[8][32];
    grid_wait();
    grid_release();
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < p.rows;
    float a = 0.0f;
    if (live) {
        const float rstd = p.rstd[row];
        const T* dy = static_cast<const T*>(p.dy) + row * p.dy_stride;
        for (int c = int(threadIdx.x) * V; c < p.width; c += int(blockDim.x) * V) {
            Raw<T, V> rd;
            RmsSource<T, V, kSaved> src;
            load_raw(dy + c, rd);
            src.load(p, row, c);
            float d[V], x[V], w[V];
            unpack(rd, d);
            src.get(x);
            load_weight<V>(p, c, w);
#pragma unroll
            for (int k = 0; k < V; ++k) a = __fmaf_rn(__fmul_rn(d[k], w[k]), __fmul_rn(x[k], rstd), a);
        }
    }
    a = row_sum(a, s);
    if (live && threadIdx.x == 0) p.row_avg[row] = divide(a, p.count, p.inv_width);
}

// dx of a tile of 32 V columns by a slice of the rows, and the tile's column
// sums over the slice: threads (32, 8), row r of the slice at threadIdx.y = r % 8.
template <typename T, int V, bool kSaved>
__global__ void __launch_bounds__(256) rms_grad_columns(const __grid_constant__ RmsGradParams p) {
    __shared__ float s[8][32 * V];
    grid_wait();
    grid_release();
    const int c = (int(blockIdx.x) * 32 + int(threadIdx.x)) * V;
    const int64_t row0 = int64_t(blockIdx.y) * p.slice_rows;
    const int64_t row1 = min(row0 + p.slice_rows, p.rows);
    float dw[V], w[V];
#pragma unroll
    for (int k = 0; k < V; ++k) dw[k] = 0.0f;
    if (c < p.width) {
        load_weight<V>(p, c, w);
        for (int64_t row = row0 + threadIdx.y; row < row1; row += 8) {
            Raw<T, V> rd, rh;
            RmsSource<T, V, kSaved> src;
            load_raw(static_cast<const T*>(p.dy) + row * p.dy_stride + c, rd);
            src.load(p, row, c);
            zero_raw(rh);
            if (p.dh) load_raw(static_cast<const T*>(p.dh) + row * p.dh_stride + c, rh);
            const float rstd = p.rstd[row], avg = p.row_avg[row];
            float d[V], x[V], add[V];
            unpack(rd, d);
            unpack(rh, add);
            src.get(x);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                x[k] = __fmul_rn(x[k], rstd);
                dw[k] = __fmaf_rn(d[k], x[k], dw[k]);
                const float v = __fmaf_rn(-x[k], avg, __fmul_rn(d[k], w[k]));
                d[k] = p.dh ? __fmaf_rn(v, rstd, add[k]) : __fmul_rn(v, rstd);
            }
            pack(d, rd);
            store_raw(static_cast<T*>(p.dx) + row * p.dx_stride + c, rd);
        }
    }
#pragma unroll
    for (int k = 0; k < V; ++k) s[threadIdx.y][threadIdx.x * V + k] = dw[k];
    __syncthreads();
    const int base = int(blockIdx.x) * 32 * V;
    for (int i = int(threadIdx.y) * 32 + int(threadIdx.x); i < 32 * V; i += 256) {
        float t = 0.0f;
#pragma unroll
        for (int y = 0; y < 8; ++y) t = __fadd_rn(t, s[y][i]);
        if (p.partial && base + i < p.width)
            p.partial[int64_t(blockIdx.y) * p.partial_width + base + i] = t;
    }
}

// dweight from the slices' partial sums, in a fixed order: 32 columns by
// blockDim.y groups of slices per block, a group's loads ten at a time, since
// their latency is what takes time.
__global__ void __launch_bounds__(1024) rms_grad_join(const __grid_constant__ RmsJoinParams p) {
    constexpr int kAhead = 10;
    __shared__ float s[32][33];
    grid_wait();
    grid_release();
    const int c = int(blockIdx.x) * 32 + int(threadIdx.x), groups = int(blockDim.y);
    float t = 0.0f;
    if (c < p.width) {
        const float* from = p.partial + c;
        for (int i = int(threadIdx.y); i < p.slices; i += kAhead * groups) {
            float v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int at = i + groups * j;
                v[j] = at < p.slices ? from[int64_t(at) * p.partial_width] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) t = __fadd_rn(t, v[j]);
        }
    }
    s[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.y != 0 || c >= p.width) return;
    t = 0.0f;
#pragma unroll 8
    for (int y = 0; y < groups; ++y) t = __fadd_rn(t, s[y][threadIdx.x]);
    if (p.grad_bf16) {
        uint16_t* o = static_cast<uint16_t*>(p.dweight) + c;
        *o = to_bf16(p.accumulate ? __fadd_rn(bf_1(*o), t) : t);
    } else {
        float* o = static_cast<float*>(p.dweight) + c;
        *o = p.accumulate ? __fadd_rn(*o, t) : t;
    }
}

constexpr int kSms = 152;
constexpr int kRowsWidth = 8192;         // longest rows of the one-pass kernels, but
constexpr int kStagedWidth = 16384;      // in bf16, staged
// fp32, 8192 rows with dh, staged and in registers: 2048 channels 50 and 55 us, 4096 89 and 107,
// 5120 106 and 105, 6144 166 and 119, 8192 188 and 155
constexpr int kStagedWidthFp32 = 4608;
constexpr int64_t kShared = 200 * 1024;  // of an SM, for staged rows

// How a call is done; the same for its workspace and its launch.
struct Shape {
    enum Kind { kStaged, kRows, kTwoPasses } kind;
    int nv;                  // vectors (pieces) a thread
    int depth;
    int threads, per_block;
    int64_t slices;          // blocks of the one-pass kernels
};

// Threads of a row for `elems` channels each, 512 threads per SM (the register
// file at 128 each), blocks of at least `block`.
void one_pass(Shape& q, int64_t rows, int64_t width, int elems, int least, int block) {
    const RowShape r = row_shape(width, elems, least, block);
    q.threads = r.threads;
    q.per_block = r.per_block;
    const int64_t resident = int64_t(kSms) * (512 / (r.threads * r.per_block));
    q.slices = std::max<int64_t>(1, std::min(resident, ceil_div(rows, r.per_block)));
}

// `v`: elements per access that every matrix allows; `pieces`: all of them may
// be read in 16-byte pieces.
Shape shape_of(int64_t rows, int64_t width, int dtype, bool saved, bool with_dh, int v, bool pieces) {
    Shape q = {};
    const int64_t es = dtype_size(dtype);
    if (pieces && width > 512 && width <= (dtype == DPR_BF16 ? kStagedWidth : kStagedWidthFp32)) {
        const int elems = width > kRowsWidth ? 32 : 16;
        // one block an SM for long rows, whose groups' column sums meet in shared
        // memory; few rows spread over more SMs in small blocks
        one_pass(q, rows, width, elems, 1, width > 2048 && rows >= kSms ? 512 : 256);
        const int64_t groups = 512 / (q.threads * q.per_block) * q.per_block;
        const int64_t row_bytes = width * (es + (saved ? 1 : es) + (with_dh ? es : 0));
        q.depth = int(std::min<int64_t>(kMaxDepth, kShared / (groups * row_bytes)));
        if (q.depth >= 2) {
            q.kind = Shape::kStaged;
            q.nv = int(elems * es / 16);
            return q;
        }
    }
    if (width <= kRowsWidth) {
        q.kind = Shape::kRows;
        // 16 single elements a thread spill, more so with codes and steps to hold
        q.nv = v == 16 ? 1
             : v == 8  ? (dtype == DPR_FP32 && width <= 4096 ? 1 : 2)
             : width <= 128 ? 4
             : width <= (saved ? 4096 : 256) ? 8 : 16;
        one_pass(q, rows, width, v * q.nv, v == 1 ? 32 : 1, 256);
        return q;
    }
    q.kind = Shape::kTwoPasses;
    // slices of the rows, enough blocks for the GPU, at least 16 rows each
    const int64_t want = std::max<int64_t>(1, (kSms * 8) / ceil_div(width, 512));
    q.slices = std::max<int64_t>(1, std::min<int64_t>({want, ceil_div(rows, 16), 256}));
    return q;
}

int64_t shape_bytes(const Shape& q, int64_t rows, int64_t width) {
    return (q.kind == Shape::kTwoPasses ? round_up(rows * 4, 16) : 0) +
           q.slices * round_up(width, 4) * 4;
}

template <typename T, bool kSaved, int NV>
cudaError_t launch_staged(RmsGradParams& p, const Shape& q, cudaStream_t s) {
    const size_t row_bytes = size_t(p.width) * (sizeof(T) + (kSaved ? 1 : sizeof(T)) + (p.dh ? sizeof(T) : 0));
    const size_t sums = size_t(q.per_block - 1) * q.threads * NV * 16 / sizeof(T) * 4;
    const void* k = (const void*)rms_grad_staged<T, kSaved, NV>;
    static std::atomic<uint64_t> allowed{0};   // of this kernel: one per instantiation
    const cudaError_t e = allow_shared_memory(k, int(kShared), &allowed);
    if (e != cudaSuccess) return e;
    void* args[] = {&p};
    return launch_grid(k, dim3(unsigned(q.slices)), dim3(q.threads, q.per_block),
                       std::max(size_t(q.per_block) * q.depth * row_bytes, sums), args, s);
}

template <typename T, bool kSaved>
cudaError_t launch_any_staged(RmsGradParams& p, const Shape& q, cudaStream_t s) {
    constexpr int kPieces = int(sizeof(T));     // of 16 channels
    if constexpr (sizeof(T) == 2)
        if (q.nv == 4) return launch_staged<T, kSaved, 4>(p, q, s);
    return launch_staged<T, kSaved, kPieces>(p, q, s);
}

template <typename T, int V, int NV, bool kSaved>
cudaError_t launch_rows(RmsGradParams& p, const Shape& q, cudaStream_t s) {
    const int groups = q.threads < 32 ? q.threads * q.per_block / 32 : q.per_block;
    void* args[] = {&p};
    // at most 15 * 32 * 16 floats: within the 48 KB every kernel may have
    return launch_grid((const void*)rms_grad_rows<T, V, NV, kSaved>, dim3(unsigned(q.slices)),
                       dim3(q.threads, q.per_block), size_t(groups - 1) * q.threads * V * NV * 4,
                       args, s);
}

template <typename T, int V, bool kSaved>
cudaError_t launch(RmsGradParams& p, const Shape& q, cudaStream_t s) {
    if (q.kind == Shape::kStaged) return launch_any_staged<T, kSaved>(p, q, s);
    if (q.kind == Shape::kRows) {
        if constexpr (V == 16) return launch_rows<T, 16, 1, kSaved>(p, q, s);
        else if constexpr (V == 8) {
            if constexpr (sizeof(T) == 4)
                if (q.nv == 1) return launch_rows<T, 8, 1, kSaved>(p, q, s);
            return launch_rows<T, 8, 2, kSaved>(p, q, s);
        } else {
            return q.nv == 4   ? launch_rows<T, 1, 4, kSaved>(p, q, s)
                   : q.nv == 8 ? launch_rows<T, 1, 8, kSaved>(p, q, s)
                               : launch_rows<T, 1, 16, kSaved>(p, q, s);
        }
    }
    p.slice_rows = ceil_div(p.rows, q.slices);
    void* args[] = {&p};
    const int64_t vecs = ceil_div(p.width, V);
    cudaError_t e = launch_grid((const void*)rms_grad_sums<T, V, kSaved>, dim3(unsigned(p.rows)),
                                dim3(256), 0, args, s);
    if (e != cudaSuccess) return e;
    return launch_grid((const void*)rms_grad_columns<T, V, kSaved>,
                       dim3(unsigned(ceil_div(vecs, 32)), unsigned(q.slices)), dim3(32, 8), 0, args,
                       s);
}

template <typename T, int V>
cudaError_t launch_source(RmsGradParams& p, const Shape& q, cudaStream_t s) {
    return p.ckpt.codes ? launch<T, V, true>(p, q, s) : launch<T, V, false>(p, q, s);
}

}  // namespace
}  // namespace dpr

using namespace dpr;

extern "C" {

dpr_status dpr_rmsnorm_backward_workspace(int64_t rows, int64_t width, int64_t* bytes) {
    if (!bytes) return DPR_ERR_INVALID_ARG;
    *bytes = 0;
    const dpr_status st = check_matrix_size(rows, width);
    if (st != DPR_OK) return st;
    // the most that any type and alignment asks for
    for (int dtype : {DPR_BF16, DPR_FP32})
        for (int saved = 0; saved < 2; ++saved)
            for (int dh = 0; dh < 2; ++dh)
                for (int v : {1, 8, 16})
                    for (int pieces = 0; pieces < 2; ++pieces)
                        if (v < 16 || dtype == DPR_BF16)
                            *bytes = std::max(*bytes, shape_bytes(shape_of(rows, width, dtype, saved, dh,
                                                                           v, pieces), rows, width));
    return DPR_OK;
}

dpr_status dpr_rmsnorm_backward(const void* dy, int64_t dy_stride, const void* dh,
                                int64_t dh_stride, const void* h, int64_t h_stride,
                                const dpr_checkpoint* h_ckpt, int64_t rows, int64_t width,
                                int dtype, const void* weight, int param_dtype, const float* rstd,
                                void* dx, int64_t dx_stride, void* dweight, int grad_dtype,
                                int accumulate, void* workspace, int64_t workspace_bytes,
                                void* stream) {
    int64_t need = 0;
    dpr_status st = dpr_rmsnorm_backward_workspace(rows, width, &need);
    if (st != DPR_OK) return st;
    if (!dtype_ok(dtype) || !dtype_ok(param_dtype) || !dtype_ok(grad_dtype))
        return DPR_ERR_INVALID_ARG;
    const int64_t es = dtype_size(dtype), ps = dtype_size(param_dtype), gs = dtype_size(grad_dtype);
    if (!aligned(weight, uintptr_t(ps)) || !aligned(dweight, uintptr_t(gs))) return DPR_ERR_ALIGNMENT;
    SpanList outs, ins;
    if (dweight) outs.add(dweight, uint64_t(width * gs));
    if (weight) ins.add(weight, uint64_t(width * ps));
    struct Matrix { const void* p; int64_t stride; };
    const Matrix from[3] = {{dy, dy_stride}, {dh, dh_stride}, {h_ckpt ? nullptr : h, h_stride}};
    if (rows > 0) {
        if ((st = check_matrix(dy, dy_stride, width, dtype, false)) != DPR_OK) return st;
        if (dh && (st = check_matrix(dh, dh_stride, width, dtype, false)) != DPR_OK) return st;
        if ((st = check_matrix(dx, dx_stride, width, dtype, true)) != DPR_OK) return st;
        if (h_ckpt) st = check_checkpoint(h_ckpt, width);
        else st = check_matrix(h, h_stride, width, dtype, false);
        if (st != DPR_OK) return st;
        if (!rstd || !workspace || workspace_bytes < need) return DPR_ERR_INVALID_ARG;
        if (!aligned(rstd, 4) || !aligned(workspace, 16)) return DPR_ERR_ALIGNMENT;
        outs.add(workspace, uint64_t(need));
        ins.add(rstd, uint64_t(rows) * 4);
        if (h_ckpt) ins.add(*h_ckpt, rows, width);
        // dx may be one of the matrices itself; nothing else may overlap them
        const Span dxs = span_of(dx, matrix_bytes(rows, width, dx_stride, es));
        for (const Matrix& m : from) {
            if (!m.p) continue;
            const Span ms = span_of(m.p, matrix_bytes(rows, width, m.stride, es));
            if (!(m.p == dx && m.stride == dx_stride) && overlaps(dxs, ms)) return DPR_ERR_ALIAS;
            if (outs.meets(ms)) return DPR_ERR_ALIAS;
        }
        outs.add(dx, dxs.hi - dxs.lo);
    }
    if (!outs.disjoint() || outs.meets(ins)) return DPR_ERR_ALIAS;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    RmsJoinParams j = {};
    j.dweight = dweight;
    j.width = int(width); j.grad_bf16 = grad_dtype == DPR_BF16; j.accumulate = accumulate != 0;
    cudaError_t e = cudaSuccess;
    if (rows > 0) {
        RmsGradParams p = {};
        p.dy = dy; p.dy_stride = dy_stride;
        p.dh = dh; p.dh_stride = dh_stride;
        p.h = h; p.h_stride = h_stride;
        p.weight = weight; p.rstd = rstd;
        p.dx = dx; p.dx_stride = dx_stride;
        p.rows = rows; p.width = int(width);
        p.partial_width = int(round_up(width, 4));
        p.count = float(width);
        p.inv_width = 1.0f / float(width);
        p.param_bf16 = param_dtype == DPR_BF16;
        p.param_vec = param_access(weight, nullptr);
        bool a32 = rows_aligned(dx, dx_stride, es, 32), a16 = rows_aligned(dx, dx_stride, es, 16);
        for (const Matrix& m : from) {
            if (!m.p) continue;
            a32 = a32 && rows_aligned(m.p, m.stride, es, 32);
            a16 = a16 && rows_aligned(m.p, m.stride, es, 16);
        }
        bool pieces = a16 && width * es % 16 == 0;
        if (h_ckpt) {
            p.ckpt = *h_ckpt;
            a32 = a32 && rows_aligned(h_ckpt->codes, h_ckpt->code_stride, 1, 16);
            a16 = a16 && rows_aligned(h_ckpt->codes, h_ckpt->code_stride, 1, 8);
            pieces = pieces && width % 16 == 0 &&
                     rows_aligned(h_ckpt->codes, h_ckpt->code_stride, 1, 16);
        }
        const int v = vector_elems(dtype, width, a32, a16);
        const Shape q = shape_of(rows, width, dtype, h_ckpt != nullptr, dh != nullptr, v, pieces);
        char* ws = static_cast<char*>(workspace);
        if (q.kind == Shape::kTwoPasses) {
            p.row_avg = reinterpret_cast<float*>(ws);
            ws += round_up(rows * 4, 16);
        }
        if (dweight) p.partial = reinterpret_cast<float*>(ws);
        p.depth = q.depth;
        switch (v) {
            case 16: e = launch_source<uint16_t, 16>(p, q, s); break;
            case 8:
                e = dtype == DPR_BF16 ? launch_source<uint16_t, 8>(p, q, s)
                                      : launch_source<float, 8>(p, q, s);
                break;
            default:
                e = dtype == DPR_BF16 ? launch_source<uint16_t, 1>(p, q, s)
                                      : launch_source<float, 1>(p, q, s);
        }
        if (e != cudaSuccess) return record_cuda_status(e);
        j.partial = p.partial; j.slices = int(q.slices); j.partial_width = p.partial_width;
    }
    if (dweight) {
        const int groups = j.slices > 128 ? 32 : j.slices > 64 ? 16 : 8;
        void* args[] = {&j};
        e = launch_grid((const void*)rms_grad_join, dim3(unsigned(ceil_div(width, 32))),
                        dim3(32, groups), 0, args, s);
    }
    return record_cuda_status(e);
}

}  // extern "C"

cudaError_t dpr::rms_wait_failures(unsigned int* count) {
    return cudaMemcpyFromSymbol(count, g_wait_failures, sizeof(*count));
}
