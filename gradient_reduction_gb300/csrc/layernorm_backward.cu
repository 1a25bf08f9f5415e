// Layer norm, backward: dx needs two sums along every row, dweight and dbias
// one sum each down every column.
//
// Rows of up to 8192 channels take one pass: the threads of a block own columns
// and keep their sums in registers over all of the block's rows; the blocks'
// sums are joined by a second, small kernel in a fixed order.  Rows of at most
// 512 channels, or whose parts are not 16-byte aligned, are loaded into
// registers a row ahead (norm_grad_fused), the others staged in shared memory
// (norm_grad_staged; fp32 rows too large for that, in registers).  Rows of up
// to 16384 channels whose parts are aligned take the staged kernel too, a row
// to two CTAs of a cluster, and so do some shorter ones (in_pairs).  All others take two passes, row sums first, then
// columns.
#include <algorithm>

#include "ops_device.cuh"
#include "ops_kernels.h"
#include "tensor_core.cuh"

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
    float* partial;           // [slices][2][partial_width]: dweight and dbias of a slice of the
                              // rows; NULL when neither is wanted
    int64_t rows;
    int width;
    int partial_width;        // width rounded up to 4
    int slices;
    int64_t slice_rows;       // rows per slice (two passes)
    int depth;                // rows of a group in flight (one pass, staged)
    float count;              // width
    float inv_width;          // its rounded reciprocal
    int param_bf16;
    int param_vec;
};

struct JoinParams {
    const float* partial;
    void* dweight;            // NULL: not wanted
    void* dbias;
    int width;
    int partial_width;
    int slices;
    int grad_bf16;
    int accumulate;
};

namespace {

constexpr int kMaxDepth = 6;             // rows of a group in shared memory, at most
__device__ unsigned int g_wait_failures;

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

// A block's column sums, first over its rows-at-a-time, to its place among the
// partial sums: rows that share a warp by exchanges, the others through
// `columns` ([groups - 1][2][threads * V * NV] floats of shared memory, see
// column_groups).  The block owns `width` columns from `base` on.
template <int V, int NV>
__device__ __forceinline__ void store_partial(const NormGradParams& p, F2 (&dw)[V * NV / 2],
                                              F2 (&db)[V * NV / 2], float* columns, int64_t slice,
                                              int base, int width) {
    constexpr int E = V * NV;
    const int tx = int(threadIdx.x), threads = int(blockDim.x);
    if (!p.partial) return;
    int group = int(threadIdx.y), groups = int(blockDim.y);
    bool lead = true;
    if (threads < 32) {
        for (int d = threads; d < 32; d <<= 1) {
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                dw[k] = add2(dw[k], F2{__shfl_xor_sync(0xFFFFFFFFu, dw[k].v, d)});
                db[k] = add2(db[k], F2{__shfl_xor_sync(0xFFFFFFFFu, db[k].v, d)});
            }
        }
        const int thread = int(threadIdx.y) * threads + tx;
        group = thread >> 5;
        groups = threads * int(blockDim.y) >> 5;
        lead = (thread & 31) < threads;
    }
    if (groups > 1) {
        __syncthreads();
        float2* const mine = reinterpret_cast<float2*>(columns + (group - 1) * 2 * threads * E);
        if (group > 0 && lead) {
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                float2& t = mine[k * threads + tx];
                halves(dw[k], t.x, t.y);
                float2& u = mine[(E / 2 + k) * threads + tx];
                halves(db[k], u.x, u.y);
            }
        }
        __syncthreads();
        if (group > 0 || !lead) return;
        for (int y = 0; y + 1 < groups; ++y) {
            const float2* other = reinterpret_cast<const float2*>(columns + y * 2 * threads * E);
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                const float2 u = other[k * threads + tx], v = other[(E / 2 + k) * threads + tx];
                dw[k] = add2(dw[k], f2(u.x, u.y));
                db[k] = add2(db[k], f2(v.x, v.y));
            }
        }
    }
    float* to = p.partial + slice * 2 * p.partial_width + base;
    float out_w[E], out_b[E];
#pragma unroll
    for (int k = 0; k < E / 2; ++k) {
        halves(dw[k], out_w[2 * k], out_w[2 * k + 1]);
        halves(db[k], out_b[2 * k], out_b[2 * k + 1]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = own_channel<V, NV>(i);
        if (c < width) {
            if constexpr (V >= 4) {
#pragma unroll
                for (int k = i * V; k < i * V + V; k += 4) {
                    float* at = to + c + k - i * V;
                    st_f4(at, out_w[k], out_w[k + 1], out_w[k + 2], out_w[k + 3]);
                    st_f4(at + p.partial_width, out_b[k], out_b[k + 1], out_b[k + 2], out_b[k + 3]);
                }
            } else {
                to[c] = out_w[i];
                to[p.partial_width + c] = out_b[i];
            }
        }
    }
}

// One pass: blockDim.x threads (see row_sum; at most 512) share a row, NV
// vectors of V channels each; blockDim.y rows at a time per block, the blocks'
// rows interleaved.  With the join: 65536 x 128 bf16 10.4 us, from a checkpoint
// 12.2 us (floors 7.4 and 6.2); 16384 x 8192 fp32 256 us, 6.3 TB/s; single
// elements, 3001 x 1003 fp32 10.7 us, 16384 x 1001 bf16 32 us.
template <typename T, int V, int NV, bool kSaved>
__global__ void __launch_bounds__(512) norm_grad_fused(const __grid_constant__ NormGradParams p) {
    constexpr int E = V * NV;
    __shared__ float2 s[2][8][32];
    extern __shared__ float columns[];           // [blockDim.y - 1][2][threads * E]
    grid_wait();
    grid_release();
    const int tx = int(threadIdx.x), threads = int(blockDim.x);
    // element i * V + k is half (i * V + k) & 1 of pair (i * V + k) / 2
    F2 w[E / 2], dw[E / 2], db[E / 2];
    {
        float f[E];
#pragma unroll
        for (int k = 0; k < E; ++k) f[k] = 1.0f;
        if (p.weight) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = own_channel<V, NV>(i);
                float v[V];
                if (c < p.width) {
                    load_params<V>(p.weight, p.param_bf16, p.param_vec, c, v);
#pragma unroll
                    for (int k = 0; k < V; ++k) f[i * V + k] = v[k];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
            w[k] = f2(f[2 * k], f[2 * k + 1]);
            dw[k] = f2(0.0f);
            db[k] = f2(0.0f);
        }
    }
    const int64_t stride = int64_t(gridDim.x) * blockDim.y;
    int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    Raw<T, V> dy[NV];
    Source<T, V, kSaved> x[NV];
    float mean = 0.0f, rstd = 0.0f;
    const auto load = [&](int64_t r) {
        const bool live = r < p.rows;
        mean = live ? p.mean[r] : 0.0f;
        rstd = live ? p.rstd[r] : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = own_channel<V, NV>(i);
            if (live && c < p.width) {
                load_raw(static_cast<const T*>(p.dy) + r * p.dy_stride + c, dy[i]);
                x[i].load(p, r, c);
            } else {
                zero_raw(dy[i]);
                x[i].zero();
            }
        }
    };
    load(row);
    // the same number of turns for every row of a block: the barriers are shared
    int turn = 0;
    for (int64_t first = int64_t(blockIdx.x) * blockDim.y; first < p.rows;
         first += stride, row += stride, turn ^= 1) {
        F2 g[E / 2], h[E / 2];
        F2 sum_g = f2(0.0f), sum_gh = f2(0.0f);
        const float r = rstd;
        {
            float d[E], f[E];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float v[V];
                unpack(dy[i], v);
#pragma unroll
                for (int k = 0; k < V; ++k) d[i * V + k] = v[k];
                x[i].get(v);
#pragma unroll
                for (int k = 0; k < V; ++k) f[i * V + k] = v[k];
            }
            const F2 minus_mean = f2(-mean), r2 = f2(r);
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                // a channel past the row's end has d = 0
                const F2 dk = f2(d[2 * k], d[2 * k + 1]);
                h[k] = mul2(add2(f2(f[2 * k], f[2 * k + 1]), minus_mean), r2);
                g[k] = mul2(dk, w[k]);
                sum_g = add2(sum_g, g[k]);
                sum_gh = fma2(g[k], h[k], sum_gh);
                dw[k] = fma2(dk, h[k], dw[k]);
                db[k] = add2(db[k], dk);
            }
        }
        load(row + stride);
        float a = total(sum_g), b = total(sum_gh);
        row_sums(a, b, s[turn]);
        if (row < p.rows) {
            const F2 minus_a = f2(-divide(a, p.count, p.inv_width)), r2 = f2(r);
            const F2 minus_b = f2(-divide(b, p.count, p.inv_width));
            float d[E];
#pragma unroll
            for (int k = 0; k < E / 2; ++k)
                halves(mul2(r2, fma2(h[k], minus_b, add2(g[k], minus_a))), d[2 * k], d[2 * k + 1]);
            T* dx = static_cast<T*>(p.dx) + row * p.dx_stride;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = own_channel<V, NV>(i);
                if (c < p.width) {
                    float v[V];
#pragma unroll
                    for (int k = 0; k < V; ++k) v[k] = d[i * V + k];
                    Raw<T, V> out;
                    pack(v, out);
                    store_raw(dx + c, out);
                }
            }
        }
    }
    store_partial<V, NV>(p, dw, db, columns, blockIdx.x, 0, p.width);
}

// Four sums over the blockDim.x threads (64 to 512) that share threadIdx.y;
// lane l of a warp ends up with sum l / 8 of the warp after six exchanges, and
// all four come back after one barrier.  `s` as for row_sums.
__device__ __forceinline__ void row_sums4(float (&v)[4], float (*s)[16][4]) {
    const int lane = int(threadIdx.x) & 31, warp = int(threadIdx.x) >> 5, nw = int(blockDim.x) >> 5;
    const bool upper = lane & 16, odd = lane & 8;
    const float k0 = __fadd_rn(upper ? v[2] : v[0],
                               __shfl_xor_sync(0xFFFFFFFFu, upper ? v[0] : v[2], 16));
    const float k1 = __fadd_rn(upper ? v[3] : v[1],
                               __shfl_xor_sync(0xFFFFFFFFu, upper ? v[1] : v[3], 16));
    float t = __fadd_rn(odd ? k1 : k0, __shfl_xor_sync(0xFFFFFFFFu, odd ? k0 : k1, 8));
    t = group_sum8(t);
    if ((lane & 7) == 0) s[threadIdx.y][warp][lane >> 3] = t;
    row_barrier();
    const int w = lane & 7;
    t = w < nw ? s[threadIdx.y][w][lane >> 3] : 0.0f;
    if (nw > 8) t = __fadd_rn(t, w + 8 < nw ? s[threadIdx.y][w + 8][lane >> 3] : 0.0f);
    t = group_sum8(t);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, t, 8 * i);
}

// As norm_grad_fused for rows of 513 channels up whose parts are 16-byte
// aligned.  One thread of each group of blockDim.x (at least 64) has its rows
// bulk-copied into shared memory, p.depth of them in all, so a row's loads
// cost the threads no registers and no address arithmetic.  The group takes
// two rows a turn: their sums share one barrier and most exchanges, and their
// chains of dependent instructions overlap.  Rows are read from shared memory
// twice, for the sums and for the rest, which leaves the registers to the
// column sums.  A thread owns 16 channels in 16-byte pieces, piece i at
// i * blockDim.x + threadIdx.x, which neighbours read without bank conflicts.
// 16384 x 4096 bf16 with the join: 68 us, 5.9 TB/s (0.87 of the measured copy
// rate); from a checkpoint 80 us, 4.2 TB/s.  There neither memory (48% of DRAM's
// peak) nor the issue slots (58%) are full: the codes are restored twice, 415
// instructions a warp and row against 333, and at the 16 warps an SM that its 128
// registers allow the latencies of a turn's two passes and the barrier between them
// show.  One row a turn in registers: 76 and 83 us; 8 channels a thread: 125 and
// 134 us; deeper staging or loads asked for earlier: no difference.
// kPair: a row to two CTAs of a cluster, which send each other their half's
// four sums.  8192 x 11008 bf16: 116 us (two passes: 166), from a checkpoint 138
// (154); 8192 x 12288: 118 and 144 us, 8192 x 12288 fp32: 207 us, 5.8 TB/s.  A
// turn waits once for the other CTA, with one CTA an SM to fill the gap.
template <typename T, bool kSaved, bool kPair>
__global__ void __launch_bounds__(512) norm_grad_staged(const __grid_constant__ NormGradParams p) {
    constexpr int V = 16 / int(sizeof(T)), NV = 16 / V, E = 16;
    __shared__ float s[2][4][16][4];
    __shared__ __align__(8) uint64_t bars[4][kMaxDepth];
    __shared__ __align__(16) float other[2][4];      // the other CTA's four sums
    __shared__ __align__(8) uint64_t sent[2];
    extern __shared__ __align__(16) uint8_t ring[];
    const int tx = int(threadIdx.x), threads = int(blockDim.x);
    const uint32_t full = tc::smem_addr(bars[threadIdx.y]);
    if (tx == 0) {
        for (int k = 0; k < p.depth; ++k) tc::mbar_init(full + 8 * k, 1);
        if constexpr (kPair)
            for (int k = 0; k < 2; ++k) tc::mbar_init(tc::smem_addr(&sent[k]), 1);
        tc::mbar_init_fence();
    }
    __syncthreads();
    if constexpr (kPair) tc::cluster_sync();
    grid_wait();
    grid_release();
    // this CTA's columns and the place of its rows among those of all
    const uint32_t rank = kPair ? tc::cluster_rank() : 0;
    const int base = int(rank) * threads * E;
    const int width = kPair && rank == 0 ? threads * E : p.width - base;
    const int64_t slice = kPair ? blockIdx.x >> 1 : blockIdx.x;
    const int64_t slices = kPair ? gridDim.x >> 1 : gridDim.x;
    const uint32_t dy_bytes = uint32_t(width) * sizeof(T);
    const uint32_t x_bytes = kSaved ? uint32_t(width) : dy_bytes;
    const uint32_t stage = dy_bytes + x_bytes;
    const uint32_t mine = tc::smem_addr(ring) + threadIdx.y * p.depth * stage;
    const int64_t stride = slices * blockDim.y;
    const int64_t row0 = slice * blockDim.y + threadIdx.y;
    const auto fetch = [&](int64_t r, uint32_t k) {
        const void* x = kSaved ? static_cast<const void*>(p.ckpt.codes + r * p.ckpt.code_stride + base)
                               : static_cast<const T*>(p.x) + r * p.x_stride + base;
        tc::mbar_expect(full + 8 * k, stage);
        tc::bulk_load(mine + k * stage, static_cast<const T*>(p.dy) + r * p.dy_stride + base, dy_bytes,
                      full + 8 * k);
        tc::bulk_load(mine + k * stage + dy_bytes, x, x_bytes, full + 8 * k);
        // a row's step bytes are a DRAM access of their own: asked for as early
        if constexpr (kSaved)
            for (int at = 0; at * kBlockChannels < width; at += 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.ckpt.steps +
                                                              r * p.ckpt.step_stride +
                                                              base / kBlockChannels + at));
    };
    uint32_t asked = 0;                 // rows fetched so far, by the first thread
    if (tx == 0)
        for (; asked < uint32_t(p.depth) && row0 + asked * stride < p.rows; ++asked)
            fetch(row0 + asked * stride, asked);

    F2 w[E / 2], dw[E / 2], db[E / 2];
    {
        float f[E];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * threads + tx) * V;
            float v[V];
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = 1.0f;
            if (p.weight && c < width)
                load_params<V>(p.weight, p.param_bf16, p.param_vec, base + c, v);
#pragma unroll
            for (int k = 0; k < V; ++k) f[i * V + k] = v[k];
        }
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
            w[k] = f2(f[2 * k], f[2 * k + 1]);
            dw[k] = f2(0.0f);
            db[k] = f2(0.0f);
        }
    }
    // what does not come in 16-byte rows is loaded a turn ahead
    struct Small {
        float mean, rstd, step[NV];
    };
    Small now[2], next[2];
    const uint8_t* steps = kSaved ? p.ckpt.steps + row0 * p.ckpt.step_stride + (base + tx * V) / kBlockChannels
                                  : nullptr;
    const int64_t step_turn = 2 * stride * p.ckpt.step_stride;
    const auto load_small = [&](int64_t r, int j, Small& m) {   // steps: of row r - j * stride
        if (r >= p.rows) return;
        m.mean = p.mean[r];
        m.rstd = p.rstd[r];
        if constexpr (kSaved) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if ((i * threads + tx) * V < width)
                    m.step[i] = step_value(
                        steps[j * stride * p.ckpt.step_stride + i * threads * V / kBlockChannels]);
        }
    };
    // a piece's dy and xhat from the stage at `at`
    const auto read = [&](uint32_t at, int i, const Small& m, F2 (&d)[V / 2], F2 (&h)[V / 2]) {
        Raw<T, V> raw;
        const uint32_t piece = uint32_t(i * threads + tx);
        load_shared(at + piece * 16, raw.w);
        unpack2(raw, d);
        const F2 minus_mean = f2(-m.mean), r2 = f2(m.rstd);
        if constexpr (kSaved) {
            CodeRaw<V> codes;
            load_shared(at + dy_bytes + piece * V, codes.w);
            codes2<V>(codes, h);
            // code * step is exact: one rounding, as subtracting from it
#pragma unroll
            for (int j = 0; j < V / 2; ++j) h[j] = mul2(fma2(h[j], f2(m.step[i]), minus_mean), r2);
        } else {
            load_shared(at + dy_bytes + piece * 16, raw.w);
            unpack2(raw, h);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) h[j] = mul2(add2(h[j], minus_mean), r2);
        }
    };
#pragma unroll
    for (int j = 0; j < 2; ++j) load_small(row0 + j * stride, j, now[j]);
    T* dx = static_cast<T*>(p.dx) + row0 * p.dx_stride + base + tx * V;
    const int64_t dx_row = stride * p.dx_stride;
    uint32_t k = 0, parity = 0, last = 0;    // `last`: the first stage of the turn before
    int turn = 0;
    uint32_t sent_parity = 0;
    bool ok = true;
    for (int64_t row = row0; row < p.rows; row += 2 * stride, dx += 2 * dx_row, turn ^= 1) {
        uint32_t at[2];
        float sums[4];
        const uint32_t first = k;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            F2 sum_g = f2(0.0f), sum_gh = f2(0.0f);
            at[j] = mine + k * stage;
            if (row + j * stride < p.rows) {
                if (ok) ok = tc::mbar_wait(full + 8 * k, parity);
                if (++k == uint32_t(p.depth)) { k = 0; parity ^= 1; }
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if ((i * threads + tx) * V >= width) continue;
                    F2 d[V / 2], h[V / 2];
                    read(at[j], i, now[j], d, h);
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) {
                        const F2 g = mul2(d[e], w[i * V / 2 + e]);
                        sum_g = add2(sum_g, g);
                        sum_gh = fma2(g, h[e], sum_gh);
                    }
                }
            }
            sums[2 * j] = total(sum_g);
            sums[2 * j + 1] = total(sum_gh);
        }
        if constexpr (kSaved) steps += step_turn;
#pragma unroll
        for (int j = 0; j < 2; ++j) load_small(row + (2 + j) * stride, j, next[j]);
        row_sums4(sums, s[turn]);
        if constexpr (kPair) {
            // The other half's sums arrive on this CTA's barrier.  A buffer is
            // free again two turns on: the other CTA sends those sums after it
            // has this CTA's of the turn between, which follow all reads here.
            const uint32_t to = tc::smem_addr(other[turn]), bar = tc::smem_addr(&sent[turn]);
            if (tx == 0 && ok) {
                tc::mbar_expect(bar, 16);
                tc::send4(tc::map_to(to, rank ^ 1), sums, tc::map_to(bar, rank ^ 1));
            }
            if (ok) ok = tc::mbar_wait(bar, sent_parity);
            sent_parity ^= uint32_t(turn);
#pragma unroll
            for (int j = 0; j < 4; ++j) sums[j] = __fadd_rn(sums[j], other[turn][j]);
        }
        // the whole group is past the turn before: its two stages are free (after a
        // failed wait they are not known to be)
        if (tx == 0 && ok && row != row0) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (row0 + asked * stride < p.rows) {
                    fetch(row0 + asked * stride, last);
                    ++asked;
                    if (++last == uint32_t(p.depth)) last = 0;
                }
        }
        last = first;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (row + j * stride >= p.rows) break;
            const F2 minus_a = f2(-divide(sums[2 * j], p.count, p.inv_width));
            const F2 minus_b = f2(-divide(sums[2 * j + 1], p.count, p.inv_width));
            const F2 r2 = f2(now[j].rstd);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if ((i * threads + tx) * V >= width) continue;
                F2 d[V / 2], h[V / 2];
                read(at[j], i, now[j], d, h);
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    const int q = i * V / 2 + e;
                    dw[q] = fma2(d[e], h[e], dw[q]);
                    db[q] = add2(db[q], d[e]);
                    d[e] = mul2(r2, fma2(h[e], minus_b, fma2(d[e], w[q], minus_a)));
                }
                Raw<T, V> out;
                pack2(d, out);
                st_v4(dx + j * dx_row + i * threads * V,
                      make_uint4(out.w[0], out.w[1], out.w[2], out.w[3]));
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) now[j] = next[j];
    }
    // One thread's wait may run out where the others' end, so the block counts it
    // as one, and lets what it has asked for land before the ring's memory is used
    // again or given up.
    const bool failed = __syncthreads_or(!ok);
    if (failed) {
        if (tx == 0) {
            if (threadIdx.y == 0) atomicAdd(&g_wait_failures, 1u);
            for (int j = 0; j < p.depth; ++j) {
                const uint32_t uses = asked / p.depth + (uint32_t(j) < asked % p.depth);
                if (uses > 0) tc::mbar_wait(full + 8 * j, (uses - 1) & 1);
            }
        }
        __syncthreads();
    }
    if constexpr (kPair) {
        tc::cluster_sync();    // neither CTA leaves while the other may send to it
        if (failed) {          // sums sent here that no wait has seen: some 50 us to land
            const long long start = clock64();
            while (clock64() - start < 100000) {}
        }
    }
    store_partial<V, NV>(p, dw, db, reinterpret_cast<float*>(ring), slice, base, width);
}

// Two passes (more than 16384 channels, or 8192 where rows are not aligned or a
// CTA's share of four rows is more than its shared memory): avg(g) and avg(g *
// xhat) of every row, blockDim.x threads per row.  dy and x are read twice, so
// 10 bytes an element in bf16 instead of 6: 8192 x 11008 bf16 would take 167 us,
// 155 from a checkpoint, about the 132 us that those bytes need.
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
        p.row_avg[row] = make_float2(divide(a, p.count, p.inv_width), divide(b, p.count, p.inv_width));
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
            if (p.partial && base + i < width)
                p.partial[(int64_t(blockIdx.y) * 2 + pass) * p.partial_width + base + i] = t;
        }
        __syncthreads();
    }
}

// dweight and dbias from the slices' partial sums, in a fixed order: 32
// columns by blockDim.y groups of slices per block, a group's loads ten at a
// time, since their latency is what takes time; blockIdx.y picks the gradient.
__global__ void __launch_bounds__(1024) norm_grad_join(const __grid_constant__ JoinParams p) {
    constexpr int kAhead = 10;
    __shared__ float s[32][33];
    grid_wait();
    grid_release();
    void* out = blockIdx.y ? p.dbias : p.dweight;
    if (!out) return;
    const int c = int(blockIdx.x) * 32 + int(threadIdx.x), groups = int(blockDim.y);
    float t = 0.0f;
    if (c < p.width) {
        const float* from = p.partial + int64_t(blockIdx.y) * p.partial_width + c;
        for (int i = int(threadIdx.y); i < p.slices; i += kAhead * groups) {
            float v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int at = i + groups * j;
                v[j] = at < p.slices ? from[int64_t(at) * 2 * p.partial_width] : 0.0f;
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
        uint16_t* o = static_cast<uint16_t*>(out) + c;
        *o = to_bf16(p.accumulate ? __fadd_rn(bf_1(*o), t) : t);
    } else {
        float* o = static_cast<float*>(out) + c;
        *o = p.accumulate ? __fadd_rn(*o, t) : t;
    }
}

// Groups of slices in the join: more loads in flight for many slices, small
// blocks for few.  With 8, 16 and 32 groups, both kernels together: 64 slices of
// 4096 channels 5.4, 5.8 and 7.6 us; 76 of 11008 117, 116 and 118 us; 256 of 4096
// 12.3, 9.6 and 8.6 us; 304 of 1024 19.0, 16.3 and 14.1 us.
int join_groups(int slices) { return slices > 128 ? 32 : slices > 64 ? 16 : 8; }

// Two passes: slices of the rows, enough blocks for the GPU, at least 16 rows
// each.
constexpr int kMaxSlices = 256;
int slice_count(int64_t rows, int64_t width) {
    const int64_t tiles = ceil_div(width, 512);
    const int64_t want = std::max<int64_t>(1, (152 * 8) / tiles);
    return int(std::max<int64_t>(1, std::min<int64_t>({want, ceil_div(rows, 16), kMaxSlices})));
}

// One pass: 16 channels a thread (8 for short fp32 rows), 512 threads a row at
// the most, blocks of at least `block` threads, 512 threads per SM (its 128
// registers a thread are the whole register file).
constexpr int kFusedWidth = 8192;
constexpr int kSms = 152;
struct FusedShape {
    int threads, per_block;
    int64_t blocks;
};
FusedShape fused_shape(int64_t rows, int64_t width, int v, int nv, int block = 256) {
    const RowShape r = row_shape(width, v * nv, v == 1 ? 32 : 1, block);
    const int64_t resident = int64_t(kSms) * (512 / (r.threads * r.per_block));
    return FusedShape{r.threads, r.per_block,
                      std::max<int64_t>(1, std::min(resident, ceil_div(rows, r.per_block)))};
}

// Groups of a block whose column sums meet in shared memory (store_partial).
int column_groups(const FusedShape& f) {
    return f.threads < 32 ? f.threads * f.per_block / 32 : f.per_block;
}

template <typename T, int V, int NV, bool kSaved>
cudaError_t launch_fused(NormGradParams& p, cudaStream_t s) {
    const FusedShape f = fused_shape(p.rows, p.width, V, NV);
    p.slices = int(f.blocks);
    void* args[] = {&p};
    // at most 7 * 2 * 32 * 16 floats: within the 48 KB every kernel may have
    const size_t smem = size_t(column_groups(f) - 1) * 2 * f.threads * V * NV * 4;
    return launch_grid((const void*)norm_grad_fused<T, V, NV, kSaved>, dim3(unsigned(f.blocks)),
                       dim3(f.threads, f.per_block), smem, args, s);
}

template <typename T, int V, bool kSaved>
cudaError_t launch_backward(NormGradParams& p, cudaStream_t s) {
    if (p.width <= kFusedWidth) {
        if constexpr (V == 16) return launch_fused<T, 16, 1, kSaved>(p, s);
        else if constexpr (V == 8 && sizeof(T) == 4)
            // 16 channels spill 26 registers a thread from x: 16384 x 8192 257 us, 0.92 of the floor
            return p.width <= 4096 ? launch_fused<T, 8, 1, kSaved>(p, s)
                                   : launch_fused<T, 8, 2, kSaved>(p, s);
        else if constexpr (V == 8) return launch_fused<T, 8, 2, kSaved>(p, s);
        // 16 single elements a thread spill, more so with codes and steps to hold:
        // 16384 x 1001 bf16 with 8 and 16: 40 and 32 us, from a checkpoint 35 and 49;
        // 9000 x 205: 9.4 and 10.6 us, 9.3 and 15
        else if (p.width <= 128) return launch_fused<T, 1, 4, kSaved>(p, s);
        else if (p.width <= (kSaved ? 4096 : 256)) return launch_fused<T, 1, 8, kSaved>(p, s);
        else return launch_fused<T, 1, 16, kSaved>(p, s);
    }
    p.slices = slice_count(p.rows, p.width);
    p.slice_rows = ceil_div(p.rows, p.slices);
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

// Rows of a group in shared memory, with all of an SM's groups in 200 KB; two
// turns' worth (4) at least, or the staged kernel is not for this width.
constexpr int64_t kShared = 200 * 1024;
int staged_depth(int64_t width, int64_t row_bytes) {
    const FusedShape f = fused_shape(1 << 20, width, 16, 1);
    const int64_t groups = 512 / (f.threads * f.per_block) * f.per_block;
    return int(std::min<int64_t>(kMaxDepth, kShared / (groups * row_bytes)));
}

// Two CTAs of a cluster share a row, the first takes threads * 16 channels of
// it: rows of 8193 to 16384 channels, and many rows of 4097 to 5120, of which one
// CTA an SM would leave over a third of the threads idle, while three halves fit
// (8192 x 5120 bf16: 56 -> 52 us, from a checkpoint 69 -> 59; 1000 rows 13.7 -> 14.5,
// 15.2 -> 15.1; 300 rows 9.0 -> 10.9, by the slices to be joined).
constexpr int kPairWidth = 16384;
bool in_pairs(int64_t rows, int64_t width) {
    return (width > kFusedWidth && width <= kPairWidth) ||
           (width > 4096 && width <= 5120 && rows >= 2048);
}
FusedShape pair_shape(int64_t rows, int64_t width) {
    const int threads = int(round_up(ceil_div(width, 32), 32));
    return FusedShape{threads, 1, std::min<int64_t>(kSms * (512 / threads) / 2, rows)};
}
int pair_depth(int64_t width, int64_t element_bytes) {
    const int threads = pair_shape(1, width).threads;
    return int(std::min<int64_t>(kMaxDepth, kShared / (512 / threads) /
                                                (int64_t(threads) * 16 * element_bytes)));
}

template <typename T, bool kSaved>
cudaError_t launch_pairs(NormGradParams& p, cudaStream_t s) {
    const FusedShape f = pair_shape(p.rows, p.width);
    const size_t element_bytes = sizeof(T) + (kSaved ? 1 : sizeof(T));
    const size_t row_bytes = size_t(f.threads) * 16 * element_bytes;
    p.slices = int(f.blocks);
    p.depth = pair_depth(p.width, element_bytes);
    const void* k = (const void*)norm_grad_staged<T, kSaved, true>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_shared_memory(k, int(kShared), &allowed);
    if (e != cudaSuccess) return e;
    void* args[] = {&p};
    return launch_grid(k, dim3(unsigned(2 * f.blocks)), dim3(f.threads), p.depth * row_bytes, args,
                       s, 2);
}

// Staged rows of 2049 channels up share an SM's one block where every SM gets
// one: its groups' column sums meet in shared memory, so half the slices are
// written and joined (1024 x 4096 bf16 11.8 -> 11.0 us, 8192 x 2560 30.5 -> 28.7).
// Fewer rows spread over more SMs in small blocks (64 x 4096: 5.6 us against 6.1),
// and shorter rows would put more groups behind one end (32768 x 768: 34 against
// 37).
template <typename T, bool kSaved>
cudaError_t launch_staged(NormGradParams& p, int depth, cudaStream_t s) {
    const FusedShape f =
        fused_shape(p.rows, p.width, 16, 1, p.width > 2048 && p.rows >= kSms ? 512 : 256);
    p.slices = int(f.blocks);
    p.depth = depth;
    const size_t sums = size_t(f.per_block - 1) * 2 * f.threads * 16 * 4;
    const size_t rows = size_t(f.per_block) * depth * p.width * (sizeof(T) + (kSaved ? 1 : sizeof(T)));
    const void* k = (const void*)norm_grad_staged<T, kSaved, false>;
    static std::atomic<uint64_t> allowed{0};   // of this kernel: one per instantiation
    const cudaError_t e = allow_shared_memory(k, int(kShared), &allowed);
    if (e != cudaSuccess) return e;
    void* args[] = {&p};
    return launch_grid(k, dim3(unsigned(f.blocks)), dim3(f.threads, f.per_block),
                       std::max(rows, sums), args, s);
}

template <typename T, int V>
cudaError_t launch_source(NormGradParams& p, cudaStream_t s) {
    if (V > 1 && in_pairs(p.rows, p.width)) {
        const bool saved = p.ckpt.codes != nullptr;
        const bool fits = pair_depth(p.width, sizeof(T) + (saved ? 1 : sizeof(T))) >= 4;
        if (fits && !saved) return launch_pairs<T, false>(p, s);
        if (fits && p.width % 16 == 0 && rows_aligned(p.ckpt.codes, p.ckpt.code_stride, 1, 16))
            return launch_pairs<T, true>(p, s);
    }
    // bulk copies take whole 16-byte pieces; more than 512 channels are at least
    // 64 threads a row, so at most the 4 groups a block that the kernel has room for
    if (V > 1 && p.width > 512 && p.width <= kFusedWidth) {
        const bool saved = p.ckpt.codes != nullptr;
        const int depth = staged_depth(p.width, p.width * int64_t(sizeof(T) + (saved ? 1 : sizeof(T))));
        if (depth >= 4 && !saved) return launch_staged<T, false>(p, depth, s);
        if (depth >= 4 && p.width % 16 == 0 && rows_aligned(p.ckpt.codes, p.ckpt.code_stride, 1, 16))
            return launch_staged<T, true>(p, depth, s);
    }
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
    // the most that any access width asks for: 32 threads upward share a row
    int64_t slices = slice_count(rows, width), sums = round_up(rows * 8, 16);
    if (width <= kFusedWidth) {
        slices = std::max({fused_shape(rows, width, 16, 1).blocks,
                           fused_shape(rows, width, 8, 1).blocks,
                           fused_shape(rows, width, 1, 4).blocks,
                           fused_shape(rows, width, 1, 8).blocks,
                           fused_shape(rows, width, 1, 16).blocks});
        sums = 0;
    }
    if (in_pairs(rows, width)) slices = std::max(slices, pair_shape(rows, width).blocks);
    *bytes = sums + slices * 2 * round_up(width, 4) * 4;
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
    SpanList outs, ins;
    if (dweight) outs.add(dweight, uint64_t(width * gs));
    if (dbias) outs.add(dbias, uint64_t(width * gs));
    if (weight) ins.add(weight, uint64_t(width * ps));
    if (rows > 0) {
        if ((st = check_matrix(dy, dy_stride, width, dtype, false)) != DPR_OK) return st;
        if ((st = check_matrix(dx, dx_stride, width, dtype, true)) != DPR_OK) return st;
        if (x_ckpt) st = check_checkpoint(x_ckpt, width);
        else st = check_matrix(x, x_stride, width, dtype, false);
        if (st != DPR_OK) return st;
        if (!mean || !rstd || !workspace || workspace_bytes < need) return DPR_ERR_INVALID_ARG;
        if (!aligned(mean, 4) || !aligned(rstd, 4) || !aligned(workspace, 16))
            return DPR_ERR_ALIGNMENT;
        outs.add(workspace, uint64_t(need));
        ins.add(mean, uint64_t(rows) * 4);
        ins.add(rstd, uint64_t(rows) * 4);
        if (x_ckpt) ins.add(*x_ckpt, rows, width);
        // dx may be dy or x itself; nothing else may overlap them
        const Span dxs = span_of(dx, matrix_bytes(rows, width, dx_stride, es));
        const Span dys = span_of(dy, matrix_bytes(rows, width, dy_stride, es));
        if (!(dx == dy && dx_stride == dy_stride) && overlaps(dxs, dys)) return DPR_ERR_ALIAS;
        if (outs.meets(dys)) return DPR_ERR_ALIAS;
        if (!x_ckpt) {
            const Span xs = span_of(x, matrix_bytes(rows, width, x_stride, es));
            if (!(dx == x && dx_stride == x_stride) && overlaps(dxs, xs)) return DPR_ERR_ALIAS;
            if (outs.meets(xs)) return DPR_ERR_ALIAS;
        }
        outs.add(dx, dxs.hi - dxs.lo);
    }
    if (!outs.disjoint() || outs.meets(ins)) return DPR_ERR_ALIAS;

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
        const int64_t sums = width <= kFusedWidth ? 0 : round_up(rows * 8, 16);
        if (dweight || dbias)
            p.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + sums);
        p.partial_width = int(round_up(width, 4));
        p.rows = rows; p.width = int(width);
        p.count = float(width);
        p.inv_width = 1.0f / float(width);
        p.param_bf16 = param_dtype == DPR_BF16;
        p.param_vec = param_access(weight, nullptr);
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
        j.partial = p.partial; j.slices = p.slices; j.partial_width = p.partial_width;
    }
    if (dweight || dbias) {
        void* args[] = {&j};
        e = launch_grid((const void*)norm_grad_join, dim3(unsigned(ceil_div(width, 32)), 2),
                        dim3(32, join_groups(j.slices)), 0, args, s);
    }
    return record_cuda_status(e);
}

}  // extern "C"

cudaError_t dpr::norm_wait_failures(unsigned int* count) {
    return cudaMemcpyFromSymbol(count, g_wait_failures, sizeof(*count));
}
