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
// than memory does (about two operations a cycle and SM).  Threads, blocks and
// partial sums are joined in a fixed order.
#include <algorithm>
#include <new>
#include <type_traits>
#include <vector>

#include "ops_device.cuh"
#include "ops_kernels.h"
#include "tensor_core.cuh"

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

// A block's range of tiles, with the tensors that hold its first and its last:
// one load, and the block's first data can be asked for.
struct GradRange {
    GradSeg first, last;
    int64_t tile, end;       // of the range
    int64_t first_end;       // tiles of the first tensor and those before
    int32_t first_index, last_index;
};

namespace {

constexpr int kUnit = 16;                        // elements a thread takes at a time
constexpr int kTileUnits = 512;
constexpr int64_t kGradTile = int64_t(kUnit) * kTileUnits;
constexpr int kGradThreads = 256;                // two units of a tile each
constexpr int kPer = kTileUnits / kGradThreads;
constexpr int kBlocksPerSm = 2;
constexpr int kFewThreads = 1024;                // four tiles in one block
constexpr int kFewTiles = kFewThreads / kGradThreads;
constexpr int kCluster = 8;
constexpr int64_t kSmallTiles = kFewTiles * kCluster;   // up to here one cluster does it all

// A unit as it is stored: 32 bytes of bf16, 64 of fp32.
template <bool kBf16>
struct Unit {
    uint32_t lo[8], hi[kBf16 ? 1 : 8];

    __device__ __forceinline__ void load(const void* p, int64_t at) {
        if constexpr (kBf16) {
            ld_v8(static_cast<const uint16_t*>(p) + at, lo);
        } else {
            ld_v8(static_cast<const float*>(p) + at, lo);
            ld_v8(static_cast<const float*>(p) + at + 8, hi);
        }
    }
    __device__ __forceinline__ void get(float (&f)[kUnit]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (kBf16) {
                f[2 * i] = bf_lo(lo[i]);
                f[2 * i + 1] = bf_hi(lo[i]);
            } else {
                f[i] = __uint_as_float(lo[i]);
                f[8 + i] = __uint_as_float(hi[i]);
            }
        }
    }
};

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

// A sum of squares: an fp32 pair, and in fp64 what does not fit its limits.
struct Sum {
    float hi, lo;
    double rest;

    __device__ __forceinline__ void add(float s) {
        const float t = __fadd_rn(hi, s), b = __fsub_rn(t, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(s, b)));
        hi = t;
    }
    __device__ __forceinline__ void add(const Sum& o) {
        add(o.hi);
        lo = __fadd_rn(lo, o.lo);
        if (o.rest != 0.0) rest += o.rest;      // fp64 only where there is something (NaN too)
    }
    // Adds the squares of a unit.  False where their fp32 sum is outside the limits,
    // which only `careful` takes: its fp64 and scaling, though a branch hardly taken, cost
    // the loop over 10^9 elements half of its loads in flight.
    template <bool kCareful>
    __device__ __forceinline__ bool squares(const float (&f)[kUnit]) {
        F2 part = f2(0.0f);
#pragma unroll
        for (int i = 0; i < kUnit / 2; ++i) {
            const F2 v = f2(f[2 * i], f[2 * i + 1]);
            part = fma2(v, v, part);
        }
        const float s = total(part);
        if (s >= 0x1p-100f && s <= 0x1p60f) {
            add(s);
            return true;
        }
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < kUnit; ++i) any |= __float_as_uint(f[i]) << 1;
        if (any == 0) return true;        // zeros
        if constexpr (kCareful) {
            // All below 2^-50 then, and 2^-53 at least after scaling; or (huge, infinite or NaN) one
            // of 2^28 at least, whose square is 2^-88 after scaling, and the largest squares' sum 2^116.
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
        return kCareful;
    }
};

struct GradParams {
    const GradSeg* segs;
    const GradRange* ranges;
    int n;
    int64_t tiles;
    Sum* partial;        // a block's sum of squares
    int partials;
    const float* given;  // clipping by a norm the device holds: else NULL
    float* norm;         // else where the norm goes
    float scale;
    float max_norm;
};

__device__ __forceinline__ Sum exchanged(const Sum& v, int d) {
    Sum o;
    o.hi = __shfl_xor_sync(0xFFFFFFFFu, v.hi, d);
    o.lo = __shfl_xor_sync(0xFFFFFFFFu, v.lo, d);
    o.rest = __shfl_xor_sync(0xFFFFFFFFu, v.rest, d);
    return o;
}

// The block's sum, in its first warp; kT threads.
template <int kT>
__device__ __forceinline__ Sum block_sum(Sum v, Sum* s) {
    const int lane = int(threadIdx.x) & 31;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v.add(exchanged(v, d));
    if (lane == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = lane < kT / 32 ? s[lane] : Sum{};
#pragma unroll
        for (int d = kT / 64; d > 0; d >>= 1) v.add(exchanged(v, d));
    }
    return v;
}

// The elements of a tensor before and behind its units go with its first tile,
// one to a thread; where this thread's is, or -1.
__device__ __forceinline__ int64_t edge_of(const GradSeg& g, int64_t tile, int tx) {
    if (tile != 0) return -1;
    const int64_t behind = g.head + (g.numel - g.head) / kUnit * kUnit;
    if (tx >= g.head + int(g.numel - behind)) return -1;
    return tx < g.head ? tx : behind + tx - g.head;
}

// Calls f(values) for a thread's parts of up to `count` tiles of a tensor (1 in
// fp32, 2 in bf16: 128 bytes of a thread in flight), and with kStore stores
// what it leaves.  One set of registers serves both types: with two, the loop
// takes 32 registers more and half the loads are in flight.
template <bool kStore, typename F>
__device__ __forceinline__ void visit_wide(const GradSeg& g, int64_t tile, int count, F f) {
    const int tx = int(threadIdx.x);
    const bool bf16 = g.src_bf16;
    // units from this thread's first one on, to the tensor's or the last tile's end
    const int left = int(min((g.numel - g.head) / kUnit - tile * kTileUnits, int64_t(count) * kTileUnits)) - tx;
    const int64_t first = g.head + (tile * kTileUnits + tx) * kUnit;
    const char* from = static_cast<const char*>(g.src) + first * (bf16 ? 2 : 4);
    uint32_t w[4][8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int k = bf16 ? q : q >> 1;         // of the thread's units
        const int at = bf16 ? q * kGradThreads * 32 : (q >> 1) * kGradThreads * 64 + (q & 1) * 32;
        if (k * kGradThreads < left) ld_v8(from + at, w[q]);
    }
    char* to = static_cast<char*>(g.dst) + first * (g.dst_bf16 ? 2 : 4);
    const int64_t step = kGradThreads * kUnit * (g.dst_bf16 ? 2 : 4);
    if (bf16) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q * kGradThreads < left) {
                float v[kUnit];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[2 * i] = bf_lo(w[q][i]);
                    v[2 * i + 1] = bf_hi(w[q][i]);
                }
                f(v);
                if constexpr (kStore) store_unit(to + q * step, g.dst_bf16, 0, v);
            }
    } else {
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (q * kGradThreads < left) {
                float v[kUnit];
#pragma unroll
                for (int i = 0; i < kUnit; ++i) v[i] = __uint_as_float(w[2 * q + i / 8][i % 8]);
                f(v);
                if constexpr (kStore) store_unit(to + q * step, g.dst_bf16, 0, v);
            }
    }
    const int64_t at = edge_of(g, tile, tx);
    if (at >= 0) {
        float v[kUnit] = {};
        v[0] = load_one(g.src, bf16, at);
        f(v);
        if constexpr (kStore) store_one(g.dst, g.dst_bf16, at, v[0]);
    }
}

template <bool kStore, typename F>
__device__ __forceinline__ void visit(const GradSeg& g, int64_t tile, int count, F f) {
    if (g.wide) {
        visit_wide<kStore>(g, tile, count, f);
        return;
    }
    const int tx = int(threadIdx.x);
    int64_t at = tile * kGradTile + tx;
    int left = int(min(g.numel - tile * kGradTile, count * kGradTile)) - tx;
#pragma unroll 1
    for (; left > -tx; left -= kGradThreads * kUnit, at += kGradThreads * kUnit) {
        float w[kUnit];
#pragma unroll
        for (int j = 0; j < kUnit; ++j)
            w[j] = j * kGradThreads < left ? load_one(g.src, g.src_bf16, at + j * kGradThreads) : 0.0f;
        f(w);
        if constexpr (kStore) {
#pragma unroll
            for (int j = 0; j < kUnit; ++j)
                if (j * kGradThreads < left) store_one(g.dst, g.dst_bf16, at + j * kGradThreads, w[j]);
        }
    }
}

// Tiles of a tensor in one visit.
__device__ __forceinline__ int together(const GradSeg& g) { return g.src_bf16 ? 2 : 1; }

template <bool kCareful>
__device__ __forceinline__ bool sum_range(const GradParams& p, Sum& s) {
    const GradRange& r = p.ranges[blockIdx.x];
    s = Sum{};
    bool ok = true;
    GradSeg g = r.first;
    int i = r.first_index;
    int64_t t = r.tile, seg_end = r.first_end;
    const int64_t end = r.end;
    while (t < end) {
        if (t >= seg_end) {
            g = p.segs[++i];
            seg_end = i + 1 < p.n ? p.segs[i + 1].tile0 : p.tiles;
        }
        const int n = int(min(int64_t(together(g)), min(seg_end, end) - t));
        visit<false>(g, t - g.tile0, n, [&](float (&v)[kUnit]) { ok &= s.squares<kCareful>(v); });
        t += n;
    }
    return ok;
}

__device__ __forceinline__ float factor_of(const GradParams& p, float norm) {
    // NaN stays NaN
    const float clip = norm <= p.max_norm ? 1.0f : __fdiv_rn(p.max_norm, norm);
    return __fmul_rn(p.scale, clip);
}

__device__ __forceinline__ void scale_range(const GradParams& p, float norm) {
    const float factor = factor_of(p, norm);
    const GradRange& r = p.ranges[blockIdx.x];
    GradSeg g = r.last;
    int i = r.last_index;
    const int64_t first = r.tile;
    int64_t t = r.end;                   // tiles from here on are done
    while (t > first) {
        if (t <= g.tile0) g = p.segs[--i];
        const int n = int(min(int64_t(together(g)), t - max(first, g.tile0)));
        t -= n;
        if (g.in_place && factor == 1.0f) continue;      // as they are
        visit<true>(g, t - g.tile0, n, [&](float (&v)[kUnit]) {
#pragma unroll
            for (int k = 0; k < kUnit; ++k) v[k] = __fmul_rn(v[k], factor);
        });
    }
}

// Both roundings are fp32's where the sum has no fp64 part.  fp64 takes the
// block long enough to show where every thread works the norm out (1024 threads
// with fp64 sums and roots: 9 us), so one does.
__device__ __forceinline__ float norm_of(const Sum& v, float scale) {
    if (v.rest == 0.0) return __fmul_rn(scale, __fsqrt_rn(__fadd_rn(v.hi, v.lo)));
    return float(double(scale) * sqrt(double(v.hi) + double(v.lo) + v.rest));
}

__global__ void __launch_bounds__(kGradThreads, kBlocksPerSm)
sum_squares(const __grid_constant__ GradParams p) {
    __shared__ Sum s[kGradThreads / 32];
    grid_wait();
    grid_release();
    Sum v;
    const bool ok = sum_range<false>(p, v);
    if (__syncthreads_or(!ok)) sum_range<true>(p, v);    // the block's range once more
    v = block_sum<kGradThreads>(v, s);
    if (threadIdx.x == 0) p.partial[blockIdx.x] = v;
}

// The norm from the blocks' sums, in the same order in every block; in every thread.
__device__ __forceinline__ float join(const GradParams& p) {
    __shared__ Sum s[kGradThreads / 32];
    __shared__ float norm;
    Sum v = {};
    for (int i = int(threadIdx.x); i < p.partials; i += kGradThreads) v.add(p.partial[i]);
    v = block_sum<kGradThreads>(v, s);
    if (threadIdx.x == 0) norm = norm_of(v, p.scale);
    __syncthreads();
    return norm;
}

__global__ void __launch_bounds__(kGradThreads) join_squares(const __grid_constant__ GradParams p) {
    grid_wait();
    grid_release();
    const float norm = join(p);
    if (threadIdx.x == 0) *p.norm = norm;
}

__global__ void __launch_bounds__(kGradThreads, kBlocksPerSm)
clip_grads(const __grid_constant__ GradParams p) {
    grid_wait();
    grid_release();
    float norm;
    if (p.given) {
        norm = *p.given;
    } else {
        norm = join(p);
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.norm = norm;
    }
    scale_range(p, norm);
}

// A few tiles: the norm and the clipping in one launch, of one block or one
// cluster of them, 256 threads to a tile, which keep it in registers between
// the two.  ranges[i] is tile i's.
template <bool kClip>
__global__ void __launch_bounds__(kFewThreads) clip_few(const __grid_constant__ GradParams p) {
    __shared__ Sum s[kFewThreads / 32];
    __shared__ Sum sums[kCluster];
    __shared__ float joined;
    grid_wait();
    grid_release();
    const int tx = int(threadIdx.x) & (kGradThreads - 1);
    const int64_t tile = int64_t(blockIdx.x) * kFewTiles + threadIdx.x / kGradThreads;
    GradSeg g = {};
    int64_t t = 0, edge = -1;
    float v[kPer][kUnit] = {}, one = 0.0f;
    Sum sq = {};
    if (tile < p.tiles) {
        g = p.ranges[tile].first;
        t = tile - g.tile0;
        if (g.wide) {
            const int64_t units = (g.numel - g.head) / kUnit;
            const auto load = [&](auto type) {
                Unit<decltype(type)::value> u[kPer];
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    const int64_t at = t * kTileUnits + k * kGradThreads + tx;
                    if (at < units) u[k].load(g.src, g.head + at * kUnit);
                }
#pragma unroll
                for (int k = 0; k < kPer; ++k)
                    if (t * kTileUnits + k * kGradThreads + tx < units) u[k].get(v[k]);
            };
            edge = edge_of(g, t, tx);
            if (edge >= 0) one = load_one(g.src, g.src_bf16, edge);
            if (g.src_bf16) load(std::true_type());
            else load(std::false_type());
        } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
#pragma unroll
                for (int j = 0; j < kUnit; ++j) {
                    const int64_t at = t * kGradTile + (k * kUnit + j) * kGradThreads + tx;
                    if (at < g.numel) v[k][j] = load_one(g.src, g.src_bf16, at);
                }
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) sq.squares<true>(v[k]);
        if (edge >= 0) {
            float w[kUnit] = {};
            w[0] = one;
            sq.squares<true>(w);
        }
    }
    Sum sum = block_sum<kFewThreads>(sq, s);
    const int blocks = int(gridDim.x);
    if (blocks > 1) {
        // every block's sum to every block, added in the order of the blocks
        tc::cluster_sync();
        if (threadIdx.x < 32) {
            sum.hi = __shfl_sync(0xFFFFFFFFu, sum.hi, 0);
            sum.lo = __shfl_sync(0xFFFFFFFFu, sum.lo, 0);
            sum.rest = __shfl_sync(0xFFFFFFFFu, sum.rest, 0);
            if (int(threadIdx.x) < blocks) {
                const uint32_t to = tc::map_to(tc::smem_addr(&sums[tc::cluster_rank()]), threadIdx.x);
                tc::send_double(to, __hiloint2double(__float_as_int(sum.lo), __float_as_int(sum.hi)));
                tc::send_double(to + 8, sum.rest);
            }
        }
        tc::cluster_sync();
        sum = sums[0];
        if (threadIdx.x == 0)
            for (int i = 1; i < blocks; ++i) sum.add(sums[i]);
    }
    if (threadIdx.x == 0) joined = norm_of(sum, p.scale);
    __syncthreads();
    const float norm = joined;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.norm = norm;
    if constexpr (kClip) {
        const float factor = factor_of(p, norm);
        if (tile >= p.tiles || (g.in_place && factor == 1.0f)) return;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
#pragma unroll
            for (int j = 0; j < kUnit; ++j) v[k][j] = __fmul_rn(v[k][j], factor);
        if (g.wide) {
            const int64_t units = (g.numel - g.head) / kUnit;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int64_t at = t * kTileUnits + k * kGradThreads + tx;
                if (at < units) store_unit(g.dst, g.dst_bf16, g.head + at * kUnit, v[k]);
            }
            if (edge >= 0) store_one(g.dst, g.dst_bf16, edge, __fmul_rn(one, factor));
        } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
#pragma unroll
                for (int j = 0; j < kUnit; ++j) {
                    const int64_t at = t * kGradTile + (k * kUnit + j) * kGradThreads + tx;
                    if (at < g.numel) store_one(g.dst, g.dst_bf16, at, v[k][j]);
                }
        }
    }
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
    dpr::GradRange* d_ranges = nullptr;   // of the blocks, or (few tiles) one for each tile
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
    return plan->tiles > kSmallTiles ? int64_t(plan->blocks) * int64_t(sizeof(Sum)) : 0;
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
    p.segs = plan->d_segs; p.ranges = plan->d_ranges;
    p.n = int(plan->segs.size()); p.tiles = plan->tiles;
    p.partial = static_cast<Sum*>(workspace); p.partials = plan->blocks;
    p.norm = norm; p.scale = scale; p.max_norm = max_norm;
    void* args[] = {&p};
    if (plan->tiles <= kSmallTiles) {
        int blocks = 1;
        while (blocks * kFewTiles < plan->tiles) blocks *= 2;
        return record_cuda_status(launch_grid(
            clip ? (const void*)clip_few<true> : (const void*)clip_few<false>, dim3(blocks),
            dim3(kFewThreads), 0, args, s, blocks));
    }
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
            if (pl->tiles <= kSmallTiles) pl->blocks = int(pl->tiles);
            std::vector<GradRange> ranges(size_t(pl->blocks));
            int at = 0;
            const int n_segs = int(pl->segs.size());
            for (int b = 0; b < pl->blocks; ++b) {
                GradRange& r = ranges[size_t(b)];
                r.tile = pl->tiles * b / pl->blocks;
                r.end = pl->tiles * (b + 1) / pl->blocks;
                const auto end_of = [&](int i) { return i + 1 < n_segs ? pl->segs[i + 1].tile0 : pl->tiles; };
                while (end_of(at) <= r.tile) ++at;
                r.first = pl->segs[at]; r.first_index = at; r.first_end = end_of(at);
                while (end_of(at) < r.end) ++at;
                r.last = pl->segs[at]; r.last_index = at;
            }
            if (e == cudaSuccess && !pl->segs.empty()) {
                e = upload(&pl->d_segs, pl->segs, static_cast<cudaStream_t>(stream));
                if (e == cudaSuccess)
                    e = upload(&pl->d_ranges, ranges, static_cast<cudaStream_t>(stream));
                // one-time set-up: the plan is then usable on any stream
                if (e == cudaSuccess) e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
            }
        }
    } catch (...) {   // out of host memory
        e = cudaErrorMemoryAllocation;
    }
    if (st != DPR_OK || e != cudaSuccess) {
        if (pl->d_segs) cudaFree(pl->d_segs);
        if (pl->d_ranges) cudaFree(pl->d_ranges);
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
    if (plan->d_ranges) {
        const cudaError_t f = cudaFree(plan->d_ranges);
        if (e == cudaSuccess) e = f;
    }
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
    p.segs = plan->d_segs; p.ranges = plan->d_ranges;
    p.n = int(plan->segs.size()); p.tiles = plan->tiles;
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
