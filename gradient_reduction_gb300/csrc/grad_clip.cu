// The global norm of a list of gradients and their clipping.
//
// The norm is one read of every element, the clipping one more and a write; a
// plan holds the table of the tensors, so a call launches one kernel for each
// and copies nothing from the host.  Both kernels walk the list in tiles of 8192
// elements, each block a contiguous range of them, and the clipping walks its
// range backwards: what the norm read last is then still in L2.
//
// Sums.  Sixteen squares at a time are summed in fp32; such a sum between 2^-100
// and 2^60 is added to the thread's running sum, which is kept as an fp32 pair
// (the sum and what its roundings left out, as by Knuth's TwoSum), so that the
// error does not grow with the length.  Outside those limits (or not finite) the
// sixteen are squared again after scaling by a power of two, exactly, and added
// in fp64: nothing overflows or underflows.  fp64 throughout would take longer
// than memory does (about two operations a cycle and SM).
#include <algorithm>
#include <new>
#include <vector>

#include "ops_device.cuh"
#include "ops_kernels.h"

namespace dpr {

// One tensor of a plan.
struct GradSeg {
    const void* src;
    void* dst;
    int64_t numel;
    int64_t tile0;       // tiles of the tensors before
    int32_t head;        // elements before the first that is 32-byte aligned on both sides
    uint8_t src_bf16, dst_bf16;
    uint8_t wide;        // aligned together: 32-byte accesses behind the head
    uint8_t in_place;
};

struct GradParams {
    const GradSeg* segs;
    int n;
    int64_t tiles;
    double* partial;     // a block's sum of squares
    int partials;
    const float* given;  // clipping by a norm the device holds: else NULL
    float* norm;         // else where the norm goes
    float scale;
    float max_norm;
};

namespace {

constexpr int kUnit = 16;                        // elements a thread takes at a time
constexpr int kTileUnits = 512;
constexpr int64_t kGradTile = int64_t(kUnit) * kTileUnits;
constexpr int kGradThreads = 256;
constexpr int kBlocksPerSm = 4;
constexpr int kSmallThreads = 512;
constexpr int64_t kSmallTiles = 4;               // up to here one block does it all

__device__ __forceinline__ void load_unit(const void* p, bool bf16, int64_t at, float (&f)[kUnit]) {
    if (bf16) {
        Raw<uint16_t, 16> r;
        load_raw(static_cast<const uint16_t*>(p) + at, r);
        unpack(r, f);
    } else {
        Raw<float, 8> a, b;
        load_raw(static_cast<const float*>(p) + at, a);
        load_raw(static_cast<const float*>(p) + at + 8, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = __uint_as_float(a.w[i]);
            f[8 + i] = __uint_as_float(b.w[i]);
        }
    }
}

__device__ __forceinline__ void store_unit(void* p, bool bf16, int64_t at, const float (&f)[kUnit]) {
    if (bf16) {
        Raw<uint16_t, 16> r;
        pack(f, r);
        store_raw(static_cast<uint16_t*>(p) + at, r);
    } else {
        st_f8(static_cast<float*>(p) + at, f);
        st_f8(static_cast<float*>(p) + at + 8, f + 8);
    }
}

__device__ __forceinline__ float load_one(const void* p, bool bf16, int64_t at) {
    float f[1];
    if (bf16) {
        Raw<uint16_t, 1> r;
        load_raw(static_cast<const uint16_t*>(p) + at, r);
        unpack(r, f);
    } else {
        Raw<float, 1> r;
        load_raw(static_cast<const float*>(p) + at, r);
        unpack(r, f);
    }
    return f[0];
}

__device__ __forceinline__ void store_one(void* p, bool bf16, int64_t at, float f) {
    if (bf16) static_cast<uint16_t*>(p)[at] = to_bf16(f);
    else static_cast<float*>(p)[at] = f;
}

// A thread's sum of squares.
struct Squares {
    float hi = 0.0f, lo = 0.0f;
    double rest = 0.0;

    __device__ __forceinline__ void add(const float (&f)[kUnit]) {
        F2 part = f2(0.0f);
#pragma unroll
        for (int i = 0; i < kUnit / 2; ++i) {
            const F2 v = f2(f[2 * i], f[2 * i + 1]);
            part = fma2(v, v, part);
        }
        const float s = total(part);
        if (s >= 0x1p-100f && s <= 0x1p60f) {
            const float t = __fadd_rn(hi, s), b = __fsub_rn(t, hi);
            lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(s, b)));
            hi = t;
            return;
        }
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) any |= __float_as_uint(f[i]) << 1;
        if (any == 0) return;             // zeros
        // All below 2^-50 then, and 2^-53 at least after scaling; or (huge, infinite or NaN) one of
        // 2^28 at least, whose square is 2^-88 after scaling, and the largest squares' sum 2^116.
        const bool small = s < 1.0f;
        const float by = small ? 0x1p96f : 0x1p-72f;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const float v = __fmul_rn(f[i], by);
            sum = __fmaf_rn(v, v, sum);
        }
        rest += double(sum) * (small ? 0x1p-192 : 0x1p144);
    }
    __device__ __forceinline__ double value() const { return double(hi) + double(lo) + rest; }
};

// The block's sum of `v`, in every thread; kT threads.
template <int kT>
__device__ __forceinline__ double block_sum(double v, double* s) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < kT / 32; ++i) v += s[i];
    __syncthreads();
    return v;
}

// The tensor of a tile: the last one that starts at it or before.  Tensors
// without elements have no tile and share the next one's start.
__device__ __forceinline__ int find(const GradParams& p, int64_t tile) {
    int lo = 0, hi = p.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.segs[mid].tile0 <= tile) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Calls f(values, store) for a thread's parts of a tile; store(values) puts
// them where they go, once for each call of f.
template <int kT, bool kStore, typename F>
__device__ __forceinline__ void visit(const GradSeg& g, int64_t tile, F f) {
    const int tx = int(threadIdx.x);
    if (g.wide) {
        const int64_t units = (g.numel - g.head) / kUnit;
        constexpr int kPer = kTileUnits / kT;
        const int64_t u0 = tile * kTileUnits + tx;
        float v[kPer][kUnit];
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (u0 + k * kT < units) load_unit(g.src, g.src_bf16, g.head + (u0 + k * kT) * kUnit, v[k]);
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (u0 + k * kT < units) {
                f(v[k]);
                if constexpr (kStore)
                    store_unit(g.dst, g.dst_bf16, g.head + (u0 + k * kT) * kUnit, v[k]);
            }
        // the elements before and behind the units, with the first tile
        const int64_t behind = g.head + units * kUnit;
        if (tile == 0 && tx < g.head + int(g.numel - behind)) {
            const int64_t at = tx < g.head ? tx : behind + tx - g.head;
            float w[kUnit] = {};
            w[0] = load_one(g.src, g.src_bf16, at);
            f(w);
            if constexpr (kStore) store_one(g.dst, g.dst_bf16, at, w[0]);
        }
    } else {
        const int64_t first = tile * kGradTile;
#pragma unroll 1
        for (int64_t c = first; c < min(first + kGradTile, g.numel); c += kT * kUnit) {
            float w[kUnit];
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                const int64_t at = c + j * kT + tx;
                w[j] = at < g.numel ? load_one(g.src, g.src_bf16, at) : 0.0f;
            }
            f(w);
            if constexpr (kStore) {
#pragma unroll
                for (int j = 0; j < kUnit; ++j) {
                    const int64_t at = c + j * kT + tx;
                    if (at < g.numel) store_one(g.dst, g.dst_bf16, at, w[j]);
                }
            }
        }
    }
}

// A block's range of tiles.
__device__ __forceinline__ void range(const GradParams& p, int64_t& first, int64_t& last) {
    first = p.tiles * blockIdx.x / gridDim.x;
    last = p.tiles * (blockIdx.x + 1) / gridDim.x;
}

template <int kT>
__device__ __forceinline__ double sum_range(const GradParams& p) {
    int64_t first, last;
    range(p, first, last);
    Squares s;
    if (first < last) {
        int i = find(p, first);
        GradSeg g = p.segs[i];
        int64_t end = i + 1 < p.n ? p.segs[i + 1].tile0 : p.tiles;
        for (int64_t t = first; t < last; ++t) {
            while (t >= end) {
                g = p.segs[++i];
                end = i + 1 < p.n ? p.segs[i + 1].tile0 : p.tiles;
            }
            visit<kT, false>(g, t - g.tile0, [&](float (&v)[kUnit]) { s.add(v); });
        }
    }
    return s.value();
}

template <int kT>
__device__ __forceinline__ void scale_range(const GradParams& p, float norm) {
    // NaN stays NaN
    const float clip = norm <= p.max_norm ? 1.0f : __fdiv_rn(p.max_norm, norm);
    const float factor = __fmul_rn(p.scale, clip);
    int64_t first, last;
    range(p, first, last);
    if (first >= last) return;
    int i = find(p, last - 1);
    GradSeg g = p.segs[i];
    for (int64_t t = last - 1; t >= first; --t) {
        while (t < g.tile0) g = p.segs[--i];
        if (g.in_place && factor == 1.0f) continue;      // as they are
        visit<kT, true>(g, t - g.tile0, [&](float (&v)[kUnit]) {
#pragma unroll
            for (int k = 0; k < kUnit; ++k) v[k] = __fmul_rn(v[k], factor);
        });
    }
}

__device__ __forceinline__ float norm_of(double sum, float scale) {
    return float(double(scale) * sqrt(sum));
}

__global__ void __launch_bounds__(kGradThreads, kBlocksPerSm)
sum_squares(const __grid_constant__ GradParams p) {
    __shared__ double s[kGradThreads / 32];
    grid_wait();
    grid_release();
    const double v = block_sum<kGradThreads>(sum_range<kGradThreads>(p), s);
    if (threadIdx.x == 0) p.partial[blockIdx.x] = v;
}

// The sum of the blocks' sums, in the same order in every block.
__device__ __forceinline__ double join(const GradParams& p, double* s) {
    double v = 0.0;
    for (int i = int(threadIdx.x); i < p.partials; i += kGradThreads) v += p.partial[i];
    return block_sum<kGradThreads>(v, s);
}

__global__ void __launch_bounds__(kGradThreads) join_squares(const __grid_constant__ GradParams p) {
    __shared__ double s[kGradThreads / 32];
    grid_wait();
    grid_release();
    const double v = join(p, s);
    if (threadIdx.x == 0) *p.norm = norm_of(v, p.scale);
}

__global__ void __launch_bounds__(kGradThreads, kBlocksPerSm)
clip_grads(const __grid_constant__ GradParams p) {
    __shared__ double s[kGradThreads / 32];
    grid_wait();
    grid_release();
    float norm;
    if (p.given) {
        norm = *p.given;
    } else {
        norm = norm_of(join(p, s), p.scale);
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.norm = norm;
    }
    scale_range<kGradThreads>(p, norm);
}

// A few tiles: the norm and the clipping in one block.
template <bool kClip>
__global__ void __launch_bounds__(kSmallThreads) clip_few(const __grid_constant__ GradParams p) {
    __shared__ double s[kSmallThreads / 32];
    grid_wait();
    grid_release();
    const float norm = norm_of(block_sum<kSmallThreads>(sum_range<kSmallThreads>(p), s), p.scale);
    if (threadIdx.x == 0) *p.norm = norm;
    if constexpr (kClip) scale_range<kSmallThreads>(p, norm);
}

}  // namespace
}  // namespace dpr

namespace dpr {

// Spans by their start, with the furthest end of each and those before it.
struct SortedSpans {
    std::vector<Span> v;
    void finish() {
        std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
        for (size_t i = 1; i < v.size(); ++i) v[i].hi = std::max(v[i].hi, v[i - 1].hi);
    }
    bool meet(const Span& s) const {
        auto it = std::lower_bound(v.begin(), v.end(), s.hi,
                                   [](const Span& a, uintptr_t b) { return a.lo < b; });
        return it != v.begin() && (it - 1)->hi > s.lo;
    }
};

}  // namespace dpr

struct dpr_grad_plan {
    int device = 0;
    int64_t tiles = 0;
    int blocks = 0;                       // of a call
    std::vector<dpr::GradSeg> segs;
    dpr::GradSeg* d_segs = nullptr;
    dpr::SortedSpans outputs, all;        // what the plan's calls write, and all they touch
};

using namespace dpr;

namespace {

dpr_status check_device(const dpr_grad_plan* plan) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return record_cuda_status(e);
    return dev == plan->device ? DPR_OK : DPR_ERR_INVALID_ARG;
}

int64_t workspace_bytes_of(const dpr_grad_plan* plan) {
    return plan->tiles > kSmallTiles ? int64_t(plan->blocks) * 8 : 0;
}

dpr_status check_norm(const dpr_grad_plan* plan, float scale, const float* norm, bool given) {
    if (!plan || !norm) return DPR_ERR_INVALID_ARG;
    if (!(scale > 0.0f) || scale > 3.402823466e38f) return DPR_ERR_INVALID_ARG;
    if (!aligned(norm, 4)) return DPR_ERR_ALIGNMENT;
    return (given ? plan->outputs : plan->all).meet(span_of(norm, 4)) ? DPR_ERR_ALIAS : DPR_OK;
}

// The norm, and with `clip` the clipping.
dpr_status run(const dpr_grad_plan* plan, float scale, float max_norm, float* norm, bool clip,
               void* workspace, int64_t workspace_bytes, void* stream) {
    dpr_status st = check_norm(plan, scale, norm, false);
    if (st != DPR_OK) return st;
    if (clip && !(max_norm >= 0.0f)) return DPR_ERR_INVALID_ARG;
    const int64_t need = workspace_bytes_of(plan);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return DPR_ERR_INVALID_ARG;
        if (!aligned(workspace, 16)) return DPR_ERR_ALIGNMENT;
        if (plan->all.meet(span_of(workspace, uint64_t(need))) ||
            overlaps(span_of(workspace, uint64_t(need)), span_of(norm, 4)))
            return DPR_ERR_ALIAS;
    }
    if ((st = check_device(plan)) != DPR_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    GradParams p = {};
    p.segs = plan->d_segs; p.n = int(plan->segs.size()); p.tiles = plan->tiles;
    p.partial = static_cast<double*>(workspace); p.partials = plan->blocks;
    p.norm = norm; p.scale = scale; p.max_norm = max_norm;
    void* args[] = {&p};
    if (plan->tiles <= kSmallTiles)
        return record_cuda_status(launch_grid(
            clip ? (const void*)clip_few<true> : (const void*)clip_few<false>, dim3(1),
            dim3(kSmallThreads), 0, args, s));
    const dim3 grid(unsigned(plan->blocks));
    cudaError_t e = launch_grid((const void*)sum_squares, grid, dim3(kGradThreads), 0, args, s);
    if (e == cudaSuccess)
        e = clip ? launch_grid((const void*)clip_grads, grid, dim3(kGradThreads), 0, args, s)
                 : launch_grid((const void*)join_squares, dim3(1), dim3(kGradThreads), 0, args, s);
    return record_cuda_status(e);
}

}  // namespace

extern "C" {

dpr_status dpr_grad_plan_create(dpr_grad_plan** plan, int n, const void* const* src,
                                const int* src_dtype, void* const* dst, const int* dst_dtype,
                                const int64_t* numel, void* stream) {
    if (!plan) return DPR_ERR_INVALID_ARG;
    *plan = nullptr;
    if (n < 0 || n > DPR_MAX_GRADS) return DPR_ERR_INVALID_ARG;
    if (n > 0 && (!src || !src_dtype || !numel || (dst && !dst_dtype))) return DPR_ERR_INVALID_ARG;
    dpr_grad_plan* pl = new (std::nothrow) dpr_grad_plan();
    if (!pl) return DPR_ERR_CUDA;
    dpr_status st = DPR_OK;
    cudaError_t e = cudaSuccess;
    try {
        std::vector<Span> outs, ins;
        for (int i = 0; i < n && st == DPR_OK; ++i) {
            const int from = src_dtype[i], to = dst ? dst_dtype[i] : from;
            if (!dtype_ok(from) || !dtype_ok(to) || numel[i] < 0) st = DPR_ERR_INVALID_ARG;
            else if (numel[i] > DPR_MAX_ELEMS) st = DPR_ERR_UNSUPPORTED;
            if (st != DPR_OK || numel[i] == 0) continue;
            GradSeg g = {};
            g.src = src[i];
            g.dst = dst ? dst[i] : const_cast<void*>(src[i]);
            if (!g.src || !g.dst) { st = DPR_ERR_INVALID_ARG; continue; }
            const int64_t ss = dtype_size(from), ds = dtype_size(to);
            if (!aligned(g.src, uintptr_t(ss)) || !aligned(g.dst, uintptr_t(ds))) {
                st = DPR_ERR_ALIGNMENT;
                continue;
            }
            g.numel = numel[i];
            g.src_bf16 = from == DPR_BF16;
            g.dst_bf16 = to == DPR_BF16;
            g.in_place = g.dst == g.src && from == to;
            // the head that aligns the source aligns the destination too, or nothing does
            const uintptr_t a = reinterpret_cast<uintptr_t>(g.src), b = reinterpret_cast<uintptr_t>(g.dst);
            // (two bf16 misalignments are equal modulo 16 elements, an fp32 one modulo 8)
            for (int h = 0; h < kUnit && !g.wide; ++h)
                if ((a + h * ss) % 32 == 0 && (b + h * ds) % 32 == 0 && g.numel >= h + kUnit) {
                    g.wide = 1;
                    g.head = h;
                }
            g.tile0 = pl->tiles;
            pl->tiles += ceil_div(g.numel, kGradTile);
            pl->segs.push_back(g);
            const Span so = span_of(g.dst, uint64_t(g.numel) * uint64_t(ds));
            const Span si = span_of(g.src, uint64_t(g.numel) * uint64_t(ss));
            outs.push_back(so);
            if (!g.in_place) ins.push_back(si);
        }
        if (st == DPR_OK && (!pairwise_disjoint(outs) || any_overlap(outs, ins))) st = DPR_ERR_ALIAS;
        if (st == DPR_OK) {
            pl->outputs.v = outs;
            pl->all.v = std::move(outs);
            pl->all.v.insert(pl->all.v.end(), ins.begin(), ins.end());
            pl->outputs.finish();
            pl->all.finish();
            int sms = 0;
            e = cudaGetDevice(&pl->device);
            if (e == cudaSuccess)
                e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, pl->device);
            pl->blocks = int(std::min<int64_t>(pl->tiles, int64_t(sms) * kBlocksPerSm));
            if (e == cudaSuccess && !pl->segs.empty()) {
                e = upload(&pl->d_segs, pl->segs, static_cast<cudaStream_t>(stream));
                // one-time set-up: the plan is then usable on any stream
                if (e == cudaSuccess) e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
            }
        }
    } catch (...) {   // out of host memory
        e = cudaErrorMemoryAllocation;
    }
    if (st != DPR_OK || e != cudaSuccess) {
        if (pl->d_segs) cudaFree(pl->d_segs);
        delete pl;
        return st != DPR_OK ? st : record_cuda_status(e);
    }
    *plan = pl;
    return DPR_OK;
}

dpr_status dpr_grad_plan_destroy(dpr_grad_plan* plan) {
    if (!plan) return DPR_OK;
    cudaError_t e = cudaSuccess;
    if (plan->d_segs) e = cudaFree(plan->d_segs);
    delete plan;
    return record_cuda_status(e);
}

dpr_status dpr_grad_norm_workspace(const dpr_grad_plan* plan, int64_t* bytes) {
    if (!plan || !bytes) return DPR_ERR_INVALID_ARG;
    *bytes = workspace_bytes_of(plan);
    return DPR_OK;
}

dpr_status dpr_grad_norm(const dpr_grad_plan* plan, float scale, float* norm, void* workspace,
                         int64_t workspace_bytes, void* stream) {
    return run(plan, scale, 0.0f, norm, false, workspace, workspace_bytes, stream);
}

dpr_status dpr_grad_clip(const dpr_grad_plan* plan, float scale, float max_norm, const float* norm,
                         void* stream) {
    dpr_status st = check_norm(plan, scale, norm, true);
    if (st != DPR_OK) return st;
    if (!(max_norm >= 0.0f)) return DPR_ERR_INVALID_ARG;
    if ((st = check_device(plan)) != DPR_OK) return st;
    if (plan->tiles == 0) return DPR_OK;
    GradParams p = {};
    p.segs = plan->d_segs; p.n = int(plan->segs.size()); p.tiles = plan->tiles;
    p.given = norm; p.scale = scale; p.max_norm = max_norm;
    void* args[] = {&p};
    return record_cuda_status(launch_grid((const void*)clip_grads, dim3(unsigned(plan->blocks)),
                                          dim3(kGradThreads), 0, args,
                                          static_cast<cudaStream_t>(stream)));
}

dpr_status dpr_grad_norm_clip(const dpr_grad_plan* plan, float scale, float max_norm, float* norm,
                              void* workspace, int64_t workspace_bytes, void* stream) {
    return run(plan, scale, max_norm, norm, true, workspace, workspace_bytes, stream);
}

}  // extern "C"
