// The global norm of a list of gradients and their clipping.
//
// The norm is one read of every element, the clipping one more and a write.  A
// plan holds the list cut into pieces, one record each, so a call copies
// nothing from the host.  The norm's blocks stride over the pieces; the clipping
// has a block for each and goes through them backwards: what the norm read last
// is then still in L2.  Both sweep memory in one order: with a contiguous range
// of pieces for each block, hundreds of places at a time, the clipping of 1.1e9
// bf16 gradients into fp32 took 1061 us instead of 940 (7.0 TB/s).  Norm and
// clipping of those: 1258 us; two reads and a write at the measured copy rate
// are 1301, L2's share 18.
//
// Sums.  Sixteen squares at a time are summed in fp32; such a sum between 2^-100
// and 2^60 is added to the thread's running sum, which is kept as an fp32 pair
// (the sum and what its roundings left out, as by Knuth's TwoSum), so that the
// error does not grow with the length.  A block that met a sum outside those limits
// (or not finite) goes through its pieces once more and squares such sixteen
// again after scaling by a power of two, exactly, adding them in fp64: nothing
// overflows or underflows.  fp64 throughout would take longer than memory does
// (about two operations a cycle and SM).  Threads, blocks and partial sums are
// joined in a fixed order.
#include <algorithm>
#include <new>
#include <vector>

#include "ops_device.cuh"
#include "ops_kernels.h"
#include "tensor_core.cuh"

namespace dpr {

// A piece of one tensor.  Wide: `count` units of 16 elements at 32-byte aligned
// addresses on both sides, with the tensor's `head` elements right before
// them and `tail` ones right behind.  Else `count` elements at any address.
struct alignas(32) GradPiece {
    const void* src;
    void* dst;
    int32_t count;
    uint8_t head, tail;
    uint8_t src_bf16, dst_bf16;
    uint8_t wide, in_place;
};

namespace {

constexpr int kUnit = 16;                        // elements a thread takes at a time
constexpr int kGradThreads = 256;
constexpr int kPer = 2;                          // units of a thread in a piece of fp32, half
                                                 // of those in one of bf16: 128 bytes in flight
constexpr int64_t kTile = int64_t(kGradThreads) * kPer * kUnit;   // elements of an fp32 piece
constexpr int kSumBlocksPerSm = 3;               // 2: 327 us for the norm above, 3: 308, 4: 311
constexpr int kFewThreads = 1024;                // four pieces in one block
constexpr int kFewPieces = kFewThreads / kGradThreads;
constexpr int kCluster = 8;
constexpr int64_t kFewTiles = kFewPieces * kCluster;   // of kTile: up to here one cluster does it all

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
    const GradPiece* pieces;
    int64_t n;
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

// The block's sum, in its first warp; of up to 1024 threads.
__device__ __forceinline__ Sum block_sum(Sum v, Sum* s) {
    const int lane = int(threadIdx.x) & 31;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v.add(exchanged(v, d));
    if (lane == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = lane < int(blockDim.x) >> 5 ? s[lane] : Sum{};
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v.add(exchanged(v, d));
    }
    return v;
}

// The elements of a wide piece in front of its units and behind them, one to a
// thread: where this thread's is (from the first unit on), or kNone.
constexpr int kNone = 1 << 30;
__device__ __forceinline__ int edge_of(const GradPiece& q, int tx) {
    if (tx < q.head) return tx - q.head;
    return tx < q.head + q.tail ? q.count * kUnit + tx - q.head : kNone;
}

// A thread's units of a wide piece as they are stored.  One set of registers
// serves both types: with two, the loop over the pieces takes 32 registers more
// and half the loads are in flight.
struct Loaded {
    uint32_t w[2 * kPer][8];

    __device__ __forceinline__ void load(const GradPiece& q, int tx) {
        const bool bf16 = q.src_bf16;
        const char* from = static_cast<const char*>(q.src) + tx * kUnit * (bf16 ? 2 : 4);
#pragma unroll
        for (int i = 0; i < 2 * kPer; ++i) {
            const int at = bf16 ? i * kGradThreads * 32 : (i >> 1) * kGradThreads * 64 + (i & 1) * 32;
            if ((bf16 ? i : i >> 1) * kGradThreads + tx < q.count) ld_v8(from + at, w[i]);
        }
    }
};

// Calls f(values) for a thread's parts of a piece and with kStore stores what
// it leaves.  `l`: what a wide piece's load gave.
template <bool kStore, typename F>
__device__ __forceinline__ void visit(const GradPiece& q, const Loaded& l, F f) {
    const int tx = int(threadIdx.x);
    const bool bf16 = q.src_bf16;
    if (q.wide) {
        const int left = q.count - tx;           // units from this thread's first one on
        char* to = static_cast<char*>(q.dst) + tx * kUnit * (q.dst_bf16 ? 2 : 4);
        const int step = kGradThreads * kUnit * (q.dst_bf16 ? 2 : 4);
        if (bf16) {
#pragma unroll
            for (int i = 0; i < 2 * kPer; ++i)
                if (i * kGradThreads < left) {
                    float v[kUnit];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        v[2 * j] = bf_lo(l.w[i][j]);
                        v[2 * j + 1] = bf_hi(l.w[i][j]);
                    }
                    f(v);
                    if constexpr (kStore) store_unit(to + i * step, q.dst_bf16, 0, v);
                }
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i * kGradThreads < left) {
                    float v[kUnit];
#pragma unroll
                    for (int j = 0; j < kUnit; ++j) v[j] = __uint_as_float(l.w[2 * i + j / 8][j % 8]);
                    f(v);
                    if constexpr (kStore) store_unit(to + i * step, q.dst_bf16, 0, v);
                }
        }
        const int at = edge_of(q, tx);
        if (at != kNone) {
            float v[kUnit] = {};
            v[0] = load_one(q.src, bf16, at);
            f(v);
            if constexpr (kStore) store_one(q.dst, q.dst_bf16, at, v[0]);
        }
        return;
    }
#pragma unroll 1
    for (int c = tx; c - tx < q.count; c += kGradThreads * kUnit) {
        float v[kUnit];
#pragma unroll
        for (int j = 0; j < kUnit; ++j)
            v[j] = c + j * kGradThreads < q.count ? load_one(q.src, bf16, c + j * kGradThreads) : 0.0f;
        f(v);
        if constexpr (kStore) {
#pragma unroll
            for (int j = 0; j < kUnit; ++j)
                if (c + j * kGradThreads < q.count) store_one(q.dst, q.dst_bf16, c + j * kGradThreads, v[j]);
        }
    }
}

template <bool kCareful>
__device__ __forceinline__ bool sum_pieces(const GradParams& p, Sum& s) {
    s = Sum{};
    bool ok = true;
    GradPiece next = p.pieces[blockIdx.x];
    for (int64_t i = blockIdx.x; i < p.n; i += gridDim.x) {
        const GradPiece q = next;
        if (i + gridDim.x < p.n) next = p.pieces[i + gridDim.x];
        Loaded l;
        if (q.wide) l.load(q, int(threadIdx.x));
        visit<false>(q, l, [&](float (&v)[kUnit]) { ok &= s.squares<kCareful>(v); });
    }
    return ok;
}

// What an element is multiplied by, in two steps: a factor below the normal numbers (of a
// step that diverged: a norm of 1e38 clipped to 0.01) has few digits or none, while the
// clipped gradients are normal numbers.  There 2^64 of it come second, and 2^-64 first,
// which is exact where the result is normal.
struct Factor {
    float first, second;
    __device__ __forceinline__ float times(float v) const { return __fmul_rn(__fmul_rn(v, first), second); }
    __device__ __forceinline__ bool one() const { return second == 1.0f; }   // then the first is 1 too
};

__device__ __forceinline__ Factor factor_of(const GradParams& p, float norm) {
    if (norm <= p.max_norm) return Factor{1.0f, p.scale};
    const float clip = __fdiv_rn(p.max_norm, norm), f = __fmul_rn(p.scale, clip);
    if (!(f < 0x1p-126f)) return Factor{1.0f, f};     // NaN stays NaN
    // clip itself is subnormal, or the scale is below 2^-58
    return Factor{0x1p-64f, __fmul_rn(p.scale, p.max_norm < 0x1p60f
                                                   ? __fdiv_rn(__fmul_rn(p.max_norm, 0x1p64f), norm)
                                                   : __fmul_rn(clip, 0x1p64f))};
}

// Both roundings are fp32's where the sum has no fp64 part.  fp64 takes the
// block long enough to show where every thread works the norm out (1024 threads
// with fp64 sums and roots: 9 us), so one does.
__device__ __forceinline__ float norm_of(const Sum& v, float scale) {
    if (v.rest == 0.0) return __fmul_rn(scale, __fsqrt_rn(__fadd_rn(v.hi, v.lo)));
    return float(double(scale) * sqrt(double(v.hi) + double(v.lo) + v.rest));
}

__global__ void __launch_bounds__(kGradThreads, kSumBlocksPerSm)
sum_squares(const __grid_constant__ GradParams p) {
    __shared__ Sum s[kGradThreads / 32];
    grid_wait();
    grid_release();
    Sum v;
    const bool ok = sum_pieces<false>(p, v);
    if (__syncthreads_or(!ok)) sum_pieces<true>(p, v);
    v = block_sum(v, s);
    if (threadIdx.x == 0) p.partial[blockIdx.x] = v;
}

// The norm from the blocks' sums, in the same order in every block; in every thread.
__device__ __forceinline__ float join(const GradParams& p) {
    __shared__ Sum s[kGradThreads / 32];
    __shared__ float norm;
    Sum v = {};
    for (int i = int(threadIdx.x); i < p.partials; i += kGradThreads) v.add(p.partial[i]);
    v = block_sum(v, s);
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

// A block for each piece, the last one first.
__global__ void __launch_bounds__(kGradThreads, 4) clip_pieces(const __grid_constant__ GradParams p) {
    grid_wait();
    grid_release();
    const GradPiece q = p.pieces[p.n - 1 - blockIdx.x];
    Loaded l;
    if (q.wide) l.load(q, int(threadIdx.x));     // in flight while the norm is
    float norm;
    if (p.given) {
        norm = *p.given;
    } else {
        norm = join(p);
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.norm = norm;
    }
    const Factor factor = factor_of(p, norm);
    if (q.in_place && factor.one()) return;      // as they are
    visit<true>(q, l, [&](float (&v)[kUnit]) {
#pragma unroll
        for (int k = 0; k < kUnit; ++k) v[k] = factor.times(v[k]);
    });
}

// A few pieces (of kTile elements at most): the norm and the clipping in one
// launch, of one block or one cluster of them, 256 threads to a piece, which
// keep it in registers between the two.  Four partitions of 1024 fp32 elements
// 3.8 us (6.2 in one block of 1024 threads).
template <bool kClip>
__global__ void __launch_bounds__(kFewThreads) clip_few(const __grid_constant__ GradParams p) {
    __shared__ Sum s[kFewThreads / 32];
    __shared__ Sum sums[kCluster];
    __shared__ float joined;
    grid_wait();
    grid_release();
    const int tx = int(threadIdx.x) & (kGradThreads - 1);
    const int64_t i = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) / kGradThreads;
    GradPiece q = {};
    int edge = kNone;
    float v[kPer][kUnit] = {}, one = 0.0f;
    Sum sq = {};
    if (i < p.n) {
        q = p.pieces[i];
        if (q.wide) {
            Loaded l;
            l.load(q, tx);       // at most kPer units a thread
            edge = edge_of(q, tx);
            if (edge != kNone) one = load_one(q.src, q.src_bf16, edge);
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                if (k * kGradThreads + tx < q.count) {
#pragma unroll
                    for (int j = 0; j < kUnit; ++j)
                        v[k][j] = !q.src_bf16 ? __uint_as_float(l.w[2 * k + j / 8][j % 8])
                                  : j & 1     ? bf_hi(l.w[k][j / 2]) : bf_lo(l.w[k][j / 2]);
                }
        } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
#pragma unroll
                for (int j = 0; j < kUnit; ++j) {
                    const int at = (k * kUnit + j) * kGradThreads + tx;
                    if (at < q.count) v[k][j] = load_one(q.src, q.src_bf16, at);
                }
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) sq.squares<true>(v[k]);
        if (edge != kNone) {
            float w[kUnit] = {};
            w[0] = one;
            sq.squares<true>(w);
        }
    }
    Sum sum = block_sum(sq, s);
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
            for (int b = 1; b < blocks; ++b) sum.add(sums[b]);
    }
    if (threadIdx.x == 0) joined = norm_of(sum, p.scale);
    __syncthreads();
    const float norm = joined;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.norm = norm;
    if constexpr (kClip) {
        const Factor factor = factor_of(p, norm);
        if (i >= p.n || (q.in_place && factor.one())) return;
#pragma unroll
        for (int k = 0; k < kPer; ++k)
#pragma unroll
            for (int j = 0; j < kUnit; ++j) v[k][j] = factor.times(v[k][j]);
        if (q.wide) {
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int at = k * kGradThreads + tx;
                if (at < q.count) store_unit(q.dst, q.dst_bf16, int64_t(at) * kUnit, v[k]);
            }
            if (edge != kNone) store_one(q.dst, q.dst_bf16, edge, factor.times(one));
        } else {
#pragma unroll
            for (int k = 0; k < kPer; ++k)
#pragma unroll
                for (int j = 0; j < kUnit; ++j) {
                    const int at = (k * kUnit + j) * kGradThreads + tx;
                    if (at < q.count) store_one(q.dst, q.dst_bf16, at, v[k][j]);
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
    int64_t n = 0;                        // pieces
    bool few = false;                     // one launch does it all
    int blocks = 0;                       // of the norm
    dpr::GradPiece* d_pieces = nullptr;
    dpr::SortedSpans outputs, all;        // what the plan's calls write, and all they touch
};

using namespace dpr;

namespace {

constexpr int64_t kJoinPieces = 152;            // up to here the clipping's blocks join the sums
// Of a list: more than the card's memory has room for.  (Pieces, a launch's blocks, are counted in
// 31 bits; these make 2^25, and one for each tensor.)
constexpr int64_t kMostElements = int64_t(1) << 38;

// One tensor of a plan.
struct Tensor {
    const void* src;
    void* dst;
    int64_t numel;
    bool src_bf16, dst_bf16;
};

// The pieces of a tensor, of up to `units` units; elements past 2^31 only ever
// show in the addresses.
void cut(const Tensor& t, int64_t units, std::vector<GradPiece>& out) {
    const int64_t ss = t.src_bf16 ? 2 : 4, ds = t.dst_bf16 ? 2 : 4;
    const uintptr_t a = reinterpret_cast<uintptr_t>(t.src), b = reinterpret_cast<uintptr_t>(t.dst);
    GradPiece q = {};
    q.src_bf16 = t.src_bf16;
    q.dst_bf16 = t.dst_bf16;
    q.in_place = a == b && t.src_bf16 == t.dst_bf16;
    // the head that aligns the source has to align the destination too
    int64_t head = 0;
    while (head < kUnit && !((a + head * ss) % 32 == 0 && (b + head * ds) % 32 == 0)) ++head;
    q.wide = head < kUnit && t.numel >= head + kUnit;
    if (!q.wide) head = 0;
    const int64_t step = q.wide ? kUnit : 1, total = (t.numel - head) / step;
    const int64_t most = q.wide ? units : kTile;
    for (int64_t i = 0; i < total; i += most) {
        const int64_t at = head + i * step;
        q.src = static_cast<const char*>(t.src) + at * ss;
        q.dst = static_cast<char*>(t.dst) + at * ds;
        q.count = int32_t(std::min(most, total - i));
        q.head = uint8_t(i == 0 ? head : 0);
        q.tail = uint8_t(i + most >= total ? t.numel - head - total * step : 0);
        out.push_back(q);
    }
}

dpr_status check_device(const dpr_grad_plan* plan) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return record_cuda_status(e);
    return dev == plan->device ? DPR_OK : DPR_ERR_INVALID_ARG;
}

int64_t workspace_bytes_of(const dpr_grad_plan* plan) {
    return plan->few ? 0 : int64_t(plan->blocks) * int64_t(sizeof(Sum));
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
        const Span ws = span_of(workspace, uint64_t(need));
        if (plan->all.meet(ws) || overlaps(ws, span_of(norm, 4))) return DPR_ERR_ALIAS;
    }
    if ((st = check_device(plan)) != DPR_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    GradParams p = {};
    p.pieces = plan->d_pieces; p.n = plan->n;
    p.partial = static_cast<Sum*>(workspace); p.partials = plan->blocks;
    p.norm = norm; p.scale = scale; p.max_norm = max_norm;
    void* args[] = {&p};
    if (plan->few) {
        // a piece to a block, up to four when a cluster has no more blocks
        int blocks = 1, each = 1;
        while (blocks * each < plan->n) (blocks < kCluster ? blocks : each) *= 2;
        return record_cuda_status(launch_grid(
            clip ? (const void*)clip_few<true> : (const void*)clip_few<false>, dim3(blocks),
            dim3(each * kGradThreads), 0, args, s, blocks));
    }
    cudaError_t e = launch_grid((const void*)sum_squares, dim3(unsigned(plan->blocks)),
                                dim3(kGradThreads), 0, args, s);
    // A few blocks of the clipping join the sums each for itself, which saves a launch (60 pieces:
    // 6.5 us against 7.5, and 2.7 us of host time); many read the norm (302: 11.8 us against 14.3).
    if (e == cudaSuccess && !(clip && plan->n <= kJoinPieces)) {
        e = launch_grid((const void*)join_squares, dim3(1), dim3(kGradThreads), 0, args, s);
        p.given = norm;
    }
    if (e == cudaSuccess && clip)
        e = launch_grid((const void*)clip_pieces, dim3(unsigned(plan->n)), dim3(kGradThreads), 0, args,
                        s);
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
        std::vector<Tensor> tensors;
        std::vector<Span> outs, ins;
        int64_t elements = 0, tiles = 0;
        for (int i = 0; i < n && st == DPR_OK; ++i) {
            const int from = src_dtype[i], to = dst ? dst_dtype[i] : from;
            if (!dtype_ok(from) || !dtype_ok(to) || numel[i] < 0) st = DPR_ERR_INVALID_ARG;
            else if (numel[i] > DPR_MAX_ELEMS || elements + numel[i] > kMostElements) st = DPR_ERR_UNSUPPORTED;
            if (st != DPR_OK || numel[i] == 0) continue;
            const Tensor t = {src[i], dst ? dst[i] : const_cast<void*>(src[i]), numel[i],
                              from == DPR_BF16, to == DPR_BF16};
            const int64_t ss = dtype_size(from), ds = dtype_size(to);
            if (!t.src || !t.dst) st = DPR_ERR_INVALID_ARG;
            else if (!aligned(t.src, uintptr_t(ss)) || !aligned(t.dst, uintptr_t(ds))) st = DPR_ERR_ALIGNMENT;
            if (st != DPR_OK) continue;
            tensors.push_back(t);
            elements += t.numel;
            tiles += ceil_div(t.numel, kTile);
            const Span so = span_of(t.dst, uint64_t(t.numel) * uint64_t(ds));
            const Span si = span_of(t.src, uint64_t(t.numel) * uint64_t(ss));
            outs.push_back(so);
            if (t.src != t.dst || from != to) ins.push_back(si);
        }
        if (st == DPR_OK && (!pairwise_disjoint(outs) || any_overlap(outs, ins))) st = DPR_ERR_ALIAS;
        if (st == DPR_OK) {
            pl->outputs.v = outs;
            pl->all.v = std::move(outs);
            pl->all.v.insert(pl->all.v.end(), ins.begin(), ins.end());
            pl->outputs.finish();
            pl->all.finish();
            pl->few = tiles <= kFewTiles;
            std::vector<GradPiece> pieces;
            const int64_t units = kTile / kUnit;
            for (const Tensor& t : tensors) cut(t, pl->few || !t.src_bf16 ? units : 2 * units, pieces);
            pl->n = int64_t(pieces.size());
            int sms = 0;
            e = cudaGetDevice(&pl->device);
            if (e == cudaSuccess)
                e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, pl->device);
            pl->blocks = int(std::min<int64_t>(pl->n, int64_t(sms) * kSumBlocksPerSm));
            if (e == cudaSuccess && pl->n > 0) {
                e = upload(&pl->d_pieces, pieces, static_cast<cudaStream_t>(stream));
                // one-time set-up: the plan is then usable on any stream
                if (e == cudaSuccess) e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
            }
        }
    } catch (...) {   // out of host memory
        e = cudaErrorMemoryAllocation;
    }
    if (st != DPR_OK || e != cudaSuccess) {
        if (pl->d_pieces) cudaFree(pl->d_pieces);
        delete pl;
        return st != DPR_OK ? st : record_cuda_status(e);
    }
    *plan = pl;
    return DPR_OK;
}

dpr_status dpr_grad_plan_destroy(dpr_grad_plan* plan) {
    if (!plan) return DPR_OK;
    cudaError_t e = cudaSuccess;
    if (plan->d_pieces) e = cudaFree(plan->d_pieces);
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
    if (plan->n == 0) return DPR_OK;
    GradParams p = {};
    p.pieces = plan->d_pieces; p.n = plan->n;
    p.given = norm; p.scale = scale; p.max_norm = max_norm;
    void* args[] = {&p};
    return record_cuda_status(launch_grid((const void*)clip_pieces, dim3(unsigned(plan->n)),
                                          dim3(kGradThreads), 0, args,
                                          static_cast<cudaStream_t>(stream)));
}

dpr_status dpr_grad_norm_clip(const dpr_grad_plan* plan, float scale, float max_norm, float* norm,
                              void* workspace, int64_t workspace_bytes, void* stream) {
    return run(plan, scale, max_norm, norm, true, workspace, workspace_bytes, stream);
}

}  // extern "C"
