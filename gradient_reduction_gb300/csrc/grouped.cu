// Linear layers of experts over tokens sorted by expert: the product, its input
// gradient and its weight gradients, on the tensor cores.
//
// A pair of CTAs computes a tile of 256 features (the M of the instruction, 128
// in each CTA) by up to 256 columns (N) with cta_group::2 instructions:
//   product          D[o][t] = sum_i W[o][i] x[t][i]    both operands along K
//   input gradient   D[i][t] = sum_o W[o][i] dy[t][o]   W along M, dy along K
//   weight gradient  D[i][o] = sum_t x[t][i] dy[t][o]   both along M and N
// The weights are the M side: an expert's tokens, of whatever number, are the N
// side, whose extent an instruction may choose in steps of 32, so few tokens
// waste little.  Features on the lanes of the accumulator also mean that a warp
// stores 32 consecutive elements of an output row straight from registers.
//
// Ragged edges: features and weights end with their tensor maps, which read
// zeros outside.  A tile of tokens reaches into the next expert's rows, whose
// columns of D are not stored.  The sum of a weight gradient runs along the
// tokens: there the rows behind the expert's last one are overwritten with
// zeros in shared memory, in both operands, since a NaN times 0 would not be 0.
//
// Sums run over 1024 elements in tensor memory, whose accumulation truncates,
// and are then added, rounded, to fp32 sums in registers.
//
// Weights whose rows are not 16-byte aligned cannot be loaded as they lie, but
// every eighth row of them can: eight rows further a row starts at the same place
// within 16 bytes.  So eight maps, each over its eighth of the rows, load pieces
// of rows with the (at most seven) elements in front of them, and eight warps
// move them to their places on the way (kForwardOdd, kInputGradOdd), as others
// restore checkpoints.
//
// A step of 64 takes 0.36 us with all pairs at work, the rate of the measured bf16
// matrix peak.  16384 tokens over 8 experts of 11008 x 4096: the product takes 0.80 ms
// in short bursts (1.85 PFLOP/s, 0.97 of the measured burst peak), 0.93 to 0.95 in
// a long loop, where the power limit sets the clock (a library product of as many
// operations, 0.86).  Few tokens: memory.  32 tokens, the same experts, 115 us, 6.3
// TB/s of weights (0.93 of the measured copy rate).  Weight gradients, 16384
// tokens, 8 experts of 4096 x 4096: fp32 305 us, from the checkpoint 370 (restoring
// takes 0.42 us a step); 16 tokens 88 us, the store at 6.1 TB/s.
//
// What did not pay: a chunk of 512 elements instead of 1024 in tensor memory; 24
// registers for the issuing warps; unaligned weights by 16-byte asynchronous copies of
// two warps (32 tokens over 8 experts of 11008 x 4095, 257 us against 152: their
// writes to shared memory, 24 to an instruction); outputs whose rows start anywhere
// stored through shared memory, as whole sectors (16 tokens, 4096 x 4095, fp32 208 ->
// 163 us, but bf16 96 -> 169, and spills for the others).
#include <type_traits>
#include <algorithm>
#include <atomic>

#include "ops_device.cuh"
#include "ops_kernels.h"
#include "tensor_core.cuh"

namespace dpr {

namespace {

enum Product { kForward, kInputGrad, kForwardOdd, kInputGradOdd, kWeightGrad, kWeightGradSaved };

constexpr int kTile = 256;               // features, and columns at most, of a tile
constexpr int kHalf = 128;               // of each CTA
constexpr int kDepth = 64;               // elements of the sum per step
constexpr int kChunk = 16;               // steps per accumulator
constexpr int kOperandBytes = kHalf * kDepth * 2;
constexpr int kGroupBytes = 64 * kDepth * 2;     // 64 channels of an operand along M or N
constexpr int kCodeBytes = kHalf * kDepth;
constexpr int kStepBytes = 16 * kDepth;  // 16 step bytes a token, 4 of them used
constexpr int kRawBytes = kHalf * (kDepth + 8) * 2;  // of a step's unaligned weights, at most
constexpr int kPiece = 16;               // rows of a load of part of a tile's tokens
constexpr int kSumWarps = 8;
constexpr int kRestoreWarps = 4;         // of each of the two groups
constexpr int kPairs = 76;               // of a GB300's 152 SMs

__host__ __device__ constexpr bool is_weight_grad(int kind) { return kind >= kWeightGrad; }
__host__ __device__ constexpr bool is_odd(int kind) { return kind == kForwardOdd || kind == kInputGradOdd; }
// Kinds whose M side is made on the way, by two more groups of warps.
__host__ __device__ constexpr bool is_made(int kind) { return kind == kWeightGradSaved || is_odd(kind); }
__host__ __device__ constexpr int stages(int kind) { return is_odd(kind) ? 4 : is_made(kind) ? 5 : 6; }
__host__ __device__ constexpr int threads(int kind) { return is_made(kind) ? 640 : 384; }
constexpr int smem_bytes(int kind) {
    return 1024 + stages(kind) * (2 * kOperandBytes + (is_odd(kind)    ? kRawBytes
                                                       : is_made(kind) ? kCodeBytes + kStepBytes
                                                                       : 0));
}
// Registers per thread after the split of those kernels (as in the weight
// gradient of one layer); together no more than the launch's.
constexpr int kIssueRegs = 40, kSumRegs = 160, kRestoreRegs = 56;
static_assert(kIssueRegs + 2 * kSumRegs + 2 * kRestoreRegs <= 5 * 96, "the block's registers");

}  // namespace

struct GroupedParams {
    CUtensorMap a;           // W, or x (or its codes): the M side
    CUtensorMap b;           // x or dy: the N side
    CUtensorMap b_piece;     // the same in pieces of kPiece rows (product, input gradient)
    CUtensorMap steps;
    const int32_t* offsets;
    int experts;
    int rows;
    int m_size;              // features along M
    int m_tiles;
    int n_size;              // weight gradients: features along N
    int n_tiles;
    int k_size;              // else: length of the sum
    void* out;
    int64_t out_stride;
    int64_t out_expert_stride;   // weight gradients
    int out_bf16;
    int accumulate;
    // work dealt out by steps: parts of tiles are summed here
    int slot_columns;        // columns of a part's room, which has kTile features
    float* partial;          // [2 * pairs][slot_columns][kTile]
    struct GroupedPart* parts;   // [2 * pairs]
};

// Weights whose rows are not aligned: rows j, j + 8, j + 16 and so on of all
// experts are map j's, which begins at the 16 bytes that hold row j's start.
struct GroupedOddParams : GroupedParams {
    CUtensorMap odd[8];
    int weight_rows;         // of an expert
    unsigned start, step;    // bytes behind 16 of row 0, and from row to row
};

// A part of a tile that begins its sum; the next pairs' first parts follow it.
struct GroupedPart {
    int64_t at;              // of the tile in the output, in elements
    int features, columns;
    int count;               // parts in all; 0: nothing to join
    int pad;
};

namespace {

__device__ unsigned int g_wait_failures;

// The experts' tokens and work, worked out by every block.
struct Experts {
    int edge[DPR_MAX_EXPERTS + 1];       // expert e has the rows edge[e] .. edge[e + 1] - 1
    int work0[DPR_MAX_EXPERTS + 1];      // of the experts before: tiles, or their steps
};

__host__ __device__ inline int tiles_of(int n) { return (n + kTile - 1) / kTile; }

// Steps of a tile of an expert; a tile without a step counts as one where
// steps are dealt out, for it has to be written.
template <int kKind>
__device__ __forceinline__ int steps_of(const GroupedParams& p, int count) {
    return ((is_weight_grad(kKind) ? count : p.k_size) + kDepth - 1) / kDepth;
}

// Offsets are limited to the rows there are and to no less than those before, so
// that whatever they hold no row has two experts and the work keeps its bounds.
template <int kKind, bool kSplit>
__device__ __forceinline__ int work_of_expert(const GroupedParams& p, int count) {
    const int n = p.m_tiles * (is_weight_grad(kKind) ? p.n_tiles : tiles_of(count));
    return kSplit ? n * max(steps_of<kKind>(p, count), 1) : n;
}

template <int kKind, bool kSplit>
__device__ void make_table(const GroupedParams& p, Experts& t) {
    const int lane = int(threadIdx.x) & 31;
    if (p.experts < 32) {                // an expert to a lane of the first warp
        if (threadIdx.x < 32) {
            int edge = lane <= p.experts ? min(max(p.offsets[lane], 0), p.rows) : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, edge, d);
                if (lane >= d) edge = max(edge, v);
            }
            const int count = __shfl_down_sync(0xFFFFFFFFu, edge, 1) - edge;
            const int mine = lane < p.experts ? work_of_expert<kKind, kSplit>(p, count) : 0;
            int upto = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, upto, d);
                if (lane >= d) upto += v;
            }
            if (lane <= p.experts) {
                t.edge[lane] = edge;
                t.work0[lane] = upto - mine;
            }
        }
        __syncthreads();
        return;
    }
    for (int e = int(threadIdx.x); e <= p.experts; e += int(blockDim.x))
        t.edge[e] = min(max(p.offsets[e], 0), p.rows);
    __syncthreads();
    if (threadIdx.x < 32) {              // a run of experts to a lane
        const int run = (p.experts + 32) / 32, first = lane * run;
        const int last = min(first + run, p.experts + 1);
        int top = 0;
        for (int e = first; e < last; ++e) top = max(top, t.edge[e]);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, top, d);
            if (lane >= d) top = max(top, v);
        }
        top = __shfl_up_sync(0xFFFFFFFFu, top, 1);
        if (lane == 0) top = 0;
        for (int e = first; e < last; ++e) t.edge[e] = top = max(top, t.edge[e]);
        __syncwarp();
        int sum = 0;
        for (int e = first; e < min(last, p.experts); ++e)
            sum += work_of_expert<kKind, kSplit>(p, t.edge[e + 1] - t.edge[e]);
        int before = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, before, d);
            if (lane >= d) before += v;
        }
        before -= sum;
        for (int e = first; e < last; ++e) {
            t.work0[e] = before;
            if (e < p.experts) before += work_of_expert<kKind, kSplit>(p, t.edge[e + 1] - t.edge[e]);
        }
    }
    __syncthreads();
}

struct Tile {
    int e;                   // advances from call to call
    int m, n;                // first feature, first column (row of the tokens, or feature)
    int columns;             // columns that are stored
    int size;                // columns of the instruction: the same up to a multiple of 32
    int steps;               // of the whole tile
    int first, last;         // those of this piece of work
    int next;                // where the work goes on
    int k, k_count;          // weight gradients: first token and how many
};

// A pair's work: every pairs-th tile, or a range of all tiles' steps.
struct Work {
    int begin, end;
    int step;                // pairs, or steps of a range
};
constexpr int kMinPart = 8;              // steps of a part, at least
template <bool kSplit>
__device__ __forceinline__ Work work_of(const GroupedParams& p, const Experts& t, int pair, int pairs) {
    const int total = t.work0[p.experts];
    if (!kSplit) return Work{pair, total, pairs};
    const int part = max((total + pairs - 1) / pairs, kMinPart);
    return Work{min(pair * part, total), min((pair + 1) * part, total), part};
}

// The piece of work at `at`; false when there is none.  An expert's tiles run in
// columns of 8 along N, so that the tiles at work at one time share inputs.
template <int kKind, bool kSplit>
__device__ __forceinline__ bool tile_at(const GroupedParams& p, const Experts& t, const Work& w, int at,
                                        Tile& s) {
    if (at >= w.end) return false;
    while (at >= t.work0[s.e + 1]) ++s.e;
    int local = at - t.work0[s.e];
    const int count = t.edge[s.e + 1] - t.edge[s.e];
    s.steps = steps_of<kKind>(p, count);
    if constexpr (kSplit) {
        const int each = max(s.steps, 1), tile = local / each;
        s.first = local - tile * each;
        s.next = min(at - s.first + each, w.end);
        s.last = min(s.first + s.next - at, s.steps);
        local = tile;
    } else {
        s.first = 0;
        s.last = s.steps;
        s.next = at + w.step;
    }
    const int n_tiles = is_weight_grad(kKind) ? p.n_tiles : tiles_of(count);
    const int group = local / (8 * p.m_tiles);
    const int rest = local - group * 8 * p.m_tiles;
    const int height = min(8, n_tiles - group * 8);
    s.m = rest / height * kTile;
    const int n = group * 8 + rest % height;
    if constexpr (is_weight_grad(kKind)) {
        s.n = n * kTile;
        s.columns = min(kTile, p.n_size - s.n);
        s.size = (s.columns + 31) & ~31;
        s.k = t.edge[s.e];
        s.k_count = count;
    } else {
        // an expert's tokens in tiles of even size
        s.size = ((count + n_tiles - 1) / n_tiles + 31) & ~31;
        s.n = t.edge[s.e] + n * s.size;
        s.columns = min(s.size, count - n * s.size);
        s.k = 0;
        s.k_count = p.k_size;
    }
    return true;
}

__device__ __forceinline__ void store_shared(uint32_t at, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c),
                 "r"(d) : "memory");
}

// The old values of a column that will be added to, all loads in flight together;
// bf16 as it is, in the lower half.
template <bool kBf16, int kN>
__device__ __forceinline__ void load_column(const char* q, int64_t stride, int count, float (&old)[kN]) {
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        old[j] = 0.0f;
        if (j < count) {
            if constexpr (kBf16) {
                uint32_t h;
                asm volatile("ld.global.u16 %0, [%1];" : "=r"(h) : "l"(q) : "memory");
                old[j] = __uint_as_float(h);
            } else {
                asm volatile("ld.global.f32 %0, [%1];" : "=f"(old[j]) : "l"(q) : "memory");
            }
        }
        q += stride;
        asm volatile("" : "+l"(q));
    }
}

__device__ __forceinline__ uint32_t select_word(uint32_t which, uint32_t yes, uint32_t no) {
    uint32_t r;
    asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\tselp.b32 %0, %2, %3, p;\n\t}"
        : "=r"(r) : "r"(which), "r"(yes), "r"(no));
    return r;
}

// The 16 bytes that begin 4 * `words` bytes and `bits` bits in 32: to w[0 .. 3].
// A word's choice is a select: lanes of one warp shift differently, and with the
// branches that a choice of four by ?: becomes a step of unaligned weights took
// 1.3 us instead of 0.47.
__device__ __forceinline__ void shift_words(uint32_t (&w)[8], uint32_t words, uint32_t bits) {
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = select_word(words & 2, w[k + 2], w[k]);
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = select_word(words & 1, w[k + 1], w[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], bits);
}

// Consecutive rows of the output at one column: `count` of a thread's kN sums,
// the rows `stride` bytes apart.  With kAdd the old values of 16 rows are
// loaded together.  The address advances step by step and is hidden from the
// compiler, which would otherwise compute all of them at once and spill the sums.
// `pause` (ns) keeps 16 rows from the next 16: all pairs store at about the same
// time, and the loads of the next tile wait behind their stores.
template <bool kBf16, bool kAdd, int kN>
__device__ __forceinline__ void store_column(char* d, int64_t stride, int count,
                                             const float (&sum)[kN], unsigned pause = 0) {
#pragma unroll
    for (int j0 = 0; j0 < kN; j0 += 16) {
        if (j0 >= count) break;
        if (pause) __nanosleep(pause);
        float old[16];
        if constexpr (kAdd) {
            const char* q = d;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                old[j] = 0.0f;
                if (j0 + j < count) {
                    if constexpr (kBf16) {
                        uint16_t h;
                        asm volatile("ld.global.u16 %0, [%1];" : "=h"(h) : "l"(q) : "memory");
                        old[j] = bf_1(h);
                    } else {
                        asm volatile("ld.global.f32 %0, [%1];" : "=f"(old[j]) : "l"(q) : "memory");
                    }
                }
                q += stride;
                asm volatile("" : "+l"(q));
            }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            if (j0 + j < count) {
                const float v = kAdd ? __fadd_rn(old[j], sum[j0 + j]) : sum[j0 + j];
                if constexpr (kBf16)
                    asm volatile("st.global.u16 [%0], %1;" ::"l"(d), "h"(to_bf16(v)) : "memory");
                else
                    asm volatile("st.global.f32 [%0], %1;" ::"l"(d), "f"(v) : "memory");
            }
            d += stride;
            asm volatile("" : "+l"(d));
        }
    }
}

template <int kKind>
using KindParams = std::conditional_t<is_odd(kKind), GroupedOddParams, GroupedParams>;

// Warps of a CTA: 0 issues the TMA loads, 1 the matrix instructions (first CTA
// only), 4-11 keep the sums and store them.  2 passes a loaded stage on to the
// first CTA (and writes the zeros behind an expert's last token); where the M
// side is made on the way 12-19 do, in two groups that take turns: they restore
// checkpoints, or move unaligned weights to their places.
template <int kKind, bool kSplit>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads(kKind), 1)
grouped_pairs(const __grid_constant__ KindParams<kKind> p) {
    constexpr bool kGrad = is_weight_grad(kKind);
    constexpr bool kSaved = kKind == kWeightGradSaved;
    constexpr bool kOdd = is_odd(kKind), kMade = is_made(kKind);
    constexpr bool kWeightAlongK = kKind == kForward || kKind == kForwardOdd;   // else along M
    // a load of unaligned weights: 72 x 16 of them, or 136 x 8
    constexpr int kOddRows = kWeightAlongK ? 16 : 8;
    constexpr int kOddPitch = ((kWeightAlongK ? kDepth : kHalf) + 8) * 2;
    constexpr int kStages = stages(kKind);
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[3 * kStages + 4];
    __shared__ uint32_t tmem_slot;
    __shared__ Experts table;
    __shared__ GroupedPart parts[2];             // what the pair's parts begin

    const uint32_t base = (tc::smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t a_at = base;                                  // [kStages], 1024-byte aligned
    const uint32_t b_at = base + kStages * kOperandBytes;        // [kStages]
    const uint32_t codes = base + 2 * kStages * kOperandBytes;   // [kStages], with checkpoints
    const uint32_t steps = codes + kStages * kCodeBytes;         // [kStages]
    const uint32_t pieces = codes;                               // [kStages], of unaligned weights
    const uint32_t bar0 = tc::smem_addr(bars);
    const auto full = [&](int s) { return bar0 + 8u * s; };                      // loads landed
    const auto free_ = [&](int s) { return bar0 + 8u * (kStages + s); };         // stage consumed
    const auto ready = [&](int s) { return bar0 + 8u * (2 * kStages + s); };     // in both CTAs
    const auto summed = [&](int a) { return bar0 + 8u * (3 * kStages + a); };
    const auto stored = [&](int a) { return bar0 + 8u * (3 * kStages + 2 + a); };

    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    const uint32_t rank = tc::cluster_rank();
    const int pairs = int(gridDim.x) >> 1, pair = int(blockIdx.x) >> 1;

    if (kSplit && threadIdx.x == 128) parts[0].count = parts[1].count = 0;
    if (warp == 0) {                     // a barrier to a lane
        if (lane < 3 * kStages + 4) {
            const int of = lane / kStages;
            tc::mbar_init(bar0 + 8u * lane,
                          of < 2                    ? 1
                          : of == 2                 ? (kMade ? 2 * kRestoreWarps : 2)
                          : lane < 3 * kStages + 2  ? 1
                                                    : 2 * kSumWarps);
        }
        tc::mbar_init_fence();
    }
    if (threadIdx.x == 64) {
        if (p.rows > 0) {                // else the maps are empty
            if constexpr (!kOdd) tc::tma_prefetch_map(&p.a);
            tc::tma_prefetch_map(&p.b);
        }
        if constexpr (!kGrad) tc::tma_prefetch_map(&p.b_piece);
        if constexpr (kSaved) tc::tma_prefetch_map(&p.steps);
        if constexpr (kOdd)
            for (int j = 0; j < 8; ++j) tc::tma_prefetch_map(&p.odd[j]);
    }
    if (warp == 1) tc::tmem_alloc(tc::smem_addr(&tmem_slot), 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_slot;
    grid_wait();
    grid_release();
    make_table<kKind, kSplit>(p, table);

    bool ok = true;
    Tile s;
    s.e = 0;
    const Work work = work_of<kSplit>(p, table, pair, pairs);
    if (warp < 4) {
        // The roles of the warps that give registers up are inside this branch: behind it the
        // compiler would count on all of the launch's again.
        if constexpr (kMade) tc::give_registers<kIssueRegs>();
        if (warp == 0) {
            if (tc::elect_one()) {
                int st = 0;
                uint32_t round = 0;
                for (int n = work.begin; ok && tile_at<kKind, kSplit>(p, table, work, n, s); n = s.next) {
                    const int m = s.m + int(rank) * kHalf;
                    const int half = s.size >> 1, c = s.n + int(rank) * half;
                    for (int k = s.first; k < s.last; ++k) {
                        if (!(ok = tc::mbar_wait(free_(st), (round & 1) ^ 1))) break;
                        const uint32_t a = a_at + st * kOperandBytes, b = b_at + st * kOperandBytes;
                        const int d = k * kDepth;
                        if constexpr (kGrad) {
                            const int t = s.k + d;
                            if constexpr (kSaved) {
                                tc::mbar_expect(full(st), kOperandBytes + kCodeBytes + kStepBytes);
                                tc::tma_load(codes + st * kCodeBytes, &p.a, m, t, full(st));
                                tc::tma_load(codes + st * kCodeBytes + kCodeBytes / 2, &p.a, m + 64, t,
                                             full(st));
                                tc::tma_load(steps + st * kStepBytes, &p.steps,
                                             (m / kBlockChannels) & ~15, t, full(st));
                            } else {
                                tc::mbar_expect(full(st), 2 * kOperandBytes);
                                tc::tma_load(a, &p.a, m, t, full(st));
                                tc::tma_load(a + kGroupBytes, &p.a, m + 64, t, full(st));
                            }
                            tc::tma_load(b, &p.b, c, t, full(st));
                            tc::tma_load(b + kGroupBytes, &p.b, c + 64, t, full(st));
                        } else {
                            tc::mbar_expect(full(st), (kOdd ? 8 * kOddRows * kOddPitch : kOperandBytes) +
                                                          half * kDepth * 2);
                            if constexpr (kOdd) {
                                const int row = s.e * p.weight_rows + (kWeightAlongK ? m : d);
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    tc::tma_load(pieces + st * kRawBytes + j * kOddRows * kOddPitch, &p.odd[j],
                                                 kWeightAlongK ? d : m, (row - j + 7) >> 3, full(st));
                            } else if constexpr (kKind == kForward) {
                                tc::tma_load(a, &p.a, d, m, s.e, full(st));
                            } else {
                                tc::tma_load(a, &p.a, m, d, s.e, full(st));
                                tc::tma_load(a + kGroupBytes, &p.a, m + 64, d, s.e, full(st));
                            }
                            if (half == kHalf) {
                                tc::tma_load(b, &p.b, d, c, full(st));
                            } else {
                                for (int r = 0; r < half; r += kPiece)
                                    tc::tma_load(b + r * kDepth * 2, &p.b_piece, d, c + r, full(st));
                            }
                        }
                        if (++st == kStages) { st = 0; ++round; }
                    }
                }
                // every load has landed and every signal of the matrix instructions has arrived
                // here before the CTA may leave: the last use of each stage
                const uint32_t total = round * kStages + st;
                for (int k = 0; k < kStages; ++k) {
                    const uint32_t uses = total / kStages + (uint32_t(k) < total % kStages);
                    if (uses == 0) continue;
                    ok &= tc::mbar_wait(full(k), (uses - 1) & 1);
                    if (ok) ok = tc::mbar_wait(free_(k), (uses - 1) & 1);
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            if (rank == 0 && tc::elect_one()) {
                constexpr bool kAlongM = !kWeightAlongK, kAlongN = kGrad;
                // 16 elements further along the sum
                constexpr uint32_t a_next = (kAlongM ? 2048 : 32) >> 4;
                constexpr uint32_t b_next = (kAlongN ? 2048 : 32) >> 4;
                const uint64_t a0 = kAlongM ? tc::operand(a_at, kGroupBytes, 1024)
                                            : tc::operand_along_k(a_at);
                const uint64_t b0 = kAlongN ? tc::operand(b_at, kGroupBytes, 1024)
                                            : tc::operand_along_k(b_at);
                uint32_t st = 0, round = 0, acc = 0, acc_round = 0;
                for (int n = work.begin; ok && tile_at<kKind, kSplit>(p, table, work, n, s); n = s.next) {
                    const uint32_t instruction = tc::bf16_instruction(kTile, s.size, kAlongM, kAlongN);
                    for (int left = s.last - s.first; ok && left > 0; left -= kChunk) {
                        if (!(ok = tc::mbar_wait(stored(acc), (acc_round & 1) ^ 1))) break;
                        const uint32_t d = tmem + acc * kTile;
                        bool add = false;
                        for (int k = min(left, kChunk); k > 0; --k) {
                            if (!(ok = tc::mbar_wait(ready(st), round & 1))) break;
                            tc::fence_after_sync();
                            const uint64_t a = a0 + st * (kOperandBytes >> 4);
                            const uint64_t b = b0 + st * (kOperandBytes >> 4);
#pragma unroll
                            for (int j = 0; j < kDepth / 16; ++j) {
                                tc::mma(d, a + j * a_next, b + j * b_next, instruction, add);
                                add = true;
                            }
                            tc::commit_both(free_(st));
                            if (++st == kStages) { st = 0; ++round; }
                        }
                        if (!ok) break;
                        tc::commit_both(summed(acc));
                        if (++acc == 2) { acc = 0; ++acc_round; }
                    }
                }
                // the other CTA's last signals have to land here before this one may leave
                for (uint32_t a = 0; a < 2; ++a) {
                    const uint32_t uses = acc_round + (a < acc);
                    if (ok && uses > 0) ok = tc::mbar_wait(stored(a), (uses - 1) & 1);
                }
            }
            __syncwarp();
        } else if (warp == 2 && !kMade) {
            int st = 0;
            uint32_t round = 0;
            for (int n = work.begin; ok && tile_at<kKind, kSplit>(p, table, work, n, s); n = s.next) {
                for (int k = s.first; k < s.last; ++k) {
                    if (!(ok = tc::mbar_wait_warp(full(st), round & 1))) break;
                    const int valid = s.k_count - k * kDepth;
                    if (kGrad && valid < kDepth) {
                        // rows of the step that belong to no token of the expert: 128 bytes in
                        // each group of 64 channels, whatever the order of the pieces in them
                        for (int r = valid + (lane >> 3); r < kDepth; r += 4) {
                            const uint32_t at = st * kOperandBytes + r * 128 + (lane & 7) * 16;
                            store_shared(a_at + at, 0, 0, 0, 0);
                            store_shared(a_at + at + kGroupBytes, 0, 0, 0, 0);
                            store_shared(b_at + at, 0, 0, 0, 0);
                            store_shared(b_at + at + kGroupBytes, 0, 0, 0, 0);
                        }
                        tc::fence_to_async();
                        __syncwarp();
                    }
                    if (lane == 0) tc::mbar_arrive_cluster(tc::map_to(ready(st), 0));
                    if (++st == kStages) { st = 0; ++round; }
                }
            }
        }
    } else if (warp < 4 + kSumWarps) {
        if constexpr (kMade) tc::take_registers<kSumRegs>();
        constexpr int kColumns = kTile / 2;
        const int quarter = warp & 3;               // the lanes this warp may read
        const int side = (warp - 4) >> 2;           // half of the columns
        int acc = 0;
        uint32_t acc_round = 0;
        float sum[kColumns];
        for (int n = work.begin; ok && tile_at<kKind, kSplit>(p, table, work, n, s); n = s.next) {
            const int half = s.size >> 1;           // a multiple of 16
            const int last = s.last;
            // A sum of one accumulator is added to the old values, loaded while it is being made:
            // rounded once, as by adding them behind it, but with a tile's loads in flight together
            // (16384 tokens, 32 experts of 4864 x 4096: fp32 1265 us without, 1069 with; bf16 1161
            // and 681).
            const bool preload = kGrad && !kSplit && p.accumulate && s.steps <= kChunk;
            if (preload && s.steps > 0) {
                const int f = s.m + int(rank) * kHalf + quarter * 32 + lane;
                const int count = f < p.m_size ? min(half, s.columns - side * half) : 0;
                const int64_t size = p.out_bf16 ? 2 : 4;
                const char* q = static_cast<const char*>(p.out) +
                                (int64_t(s.n + side * half) * p.out_stride + int64_t(s.e) * p.out_expert_stride + f) * size;
                if (p.out_bf16) load_column<true>(q, p.out_stride * size, count, sum);
                else load_column<false>(q, p.out_stride * size, count, sum);
            } else {
#pragma unroll
                for (int j = 0; j < kColumns; ++j) sum[j] = 0.0f;
            }
            for (int k = s.first; k < last; k += kChunk) {
                if (!(ok = tc::mbar_wait_warp(summed(acc), acc_round & 1))) break;
                tc::fence_after_sync();
                if (preload && p.out_bf16) {
#pragma unroll
                    for (int j = 0; j < kColumns; ++j) {
                        uint32_t v = __float_as_uint(sum[j]);
                        asm volatile("shl.b32 %0, %0, 16;" : "+r"(v));
                        sum[j] = __uint_as_float(v);
                    }
                }
                const uint32_t from = tmem + acc * kTile + side * half + (uint32_t(quarter) << 21);
#pragma unroll
                for (int c = 0; c < kColumns; c += 16) {
                    if (c < half) {
                        uint32_t v[16];
                        tc::tmem_load16(from + c, v);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            sum[c + j] = __fadd_rn(sum[c + j], __uint_as_float(v[j]));
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster(tc::map_to(stored(acc), 0));
                if (++acc == 2) { acc = 0; ++acc_round; }
            }
            if (!ok) break;
            // again: kept, it would cost the sums registers
            if constexpr (kSplit) tile_at<kKind, kSplit>(p, table, work, n, s);
            const int f = s.m + int(rank) * kHalf + quarter * 32 + lane;
            const int count = min(half, s.columns - side * half);
            int64_t at = int64_t(s.n) * p.out_stride;
            if constexpr (kGrad) at += int64_t(s.e) * p.out_expert_stride;
            if (kSplit && s.last - s.first < s.steps) {   // a part: its sums to the workspace
                const int slot = n == work.begin ? 0 : 1;
                float* to = p.partial + (int64_t(2 * pair + slot) * p.slot_columns + side * half) * kTile +
                            (f - s.m);
                store_column<false, false>(reinterpret_cast<char*>(to), kTile * 4, count, sum);
                if (s.first == 0 && threadIdx.x == 128) {
                    parts[slot].at = at + s.m;
                    parts[slot].features = min(kTile, p.m_size - s.m);
                    parts[slot].columns = s.columns;
                    parts[slot].count = 1 + (n + s.steps - work.end + work.step - 1) / work.step;
                }
            } else if (f < p.m_size && count > 0 && (s.steps > 0 || !p.accumulate)) {
                const int64_t size = p.out_bf16 ? 2 : 4;
                char* d = static_cast<char*>(p.out) + (at + int64_t(side * half) * p.out_stride + f) * size;
                const int64_t stride = p.out_stride * size;
                // fp32 tiles spread their stores over 4 us of the next one's sum, which has to take
                // longer; bf16's, and those of sums that wait for restored operands, are no
                // hindrance (16384 tokens, 8 experts of 4864 x 4096: 373 us without, 361 with)
                const bool more = kKind == kWeightGrad && s.steps >= kChunk && s.next < work.end;
                if (p.out_bf16) {
                    if (kGrad && p.accumulate && !preload) store_column<true, true>(d, stride, count, sum);
                    else store_column<true, false>(d, stride, count, sum);
                } else {
                    if (kGrad && p.accumulate && !preload) store_column<false, true>(d, stride, count, sum);
                    else store_column<false, false>(d, stride, count, sum, more ? 500 : 0);
                }
            }
        }
        if (kSplit && rank == 0 && threadIdx.x == 128) {
            p.parts[2 * pair] = parts[0];
            p.parts[2 * pair + 1] = parts[1];
        }
    } else if (kSaved && warp >= 12) {
        tc::give_registers<kRestoreRegs>();
        const int turn = (warp - 12) >> 2;          // of the two groups
        const int group = warp & 1;                 // 64 channels of the operand
        const int chunk = lane & 3;                 // 16 channels of those
        // 8 neighbouring lanes are 4 chunks of two rows: they read 128 consecutive bytes, and
        // as the 16-byte pieces of a row are permuted by the row's number, write all 32 banks
        const int row = ((warp & 2) << 4) + (lane >> 2);
        const uint32_t read = uint32_t(group * (kCodeBytes / 2) + row * 64 + chunk * 16);
        const uint32_t write = uint32_t(group * kGroupBytes + row * 128);
        const uint32_t piece0 = uint32_t((chunk * 2) ^ (row & 7)) * 16;
        const uint32_t piece1 = uint32_t((chunk * 2 + 1) ^ (row & 7)) * 16;
        uint32_t step0 = 0;                         // steps of the tiles before
        for (int n = work.begin; ok && tile_at<kKind, kSplit>(p, table, work, n, s); n = s.next) {
            const uint32_t block = uint32_t(((s.m + int(rank) * kHalf) / kBlockChannels & 15) +
                                            group * 2 + (chunk >> 1));
            const int count = s.last - s.first;
            for (int k = (step0 & 1) ^ turn; k < count; k += 2) {
                const uint32_t st = (step0 + k) % kStages, round = (step0 + k) / kStages;
                // The stage's use before this one was the other group's (their number is odd), and
                // loads may land out of order.  Until that use is over, `full` may still be in its
                // phase, and then this wait would take the one before it, long complete, for its own.
                bool landed = round > 0 && tc::mbar_passed(free_(st), (round & 1) ^ 1, full(st), round & 1);
                if (!__all_sync(0xFFFFFFFFu, landed))
                    landed = (round == 0 || tc::mbar_wait(free_(st), (round & 1) ^ 1)) &&
                             tc::mbar_wait(full(st), round & 1);
                if (!(ok = __all_sync(0xFFFFFFFFu, landed))) break;
                const int valid = s.k_count - (s.first + k) * kDepth;
                uint32_t w[4][4], step[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[h][0]), "=r"(w[h][1]), "=r"(w[h][2]), "=r"(w[h][3])
                                 : "r"(codes + st * kCodeBytes + read + h * 8 * 64));
                    asm volatile("ld.shared.u8 %0, [%1];"
                                 : "=r"(step[h])
                                 : "r"(steps + st * kStepBytes + (row + 8 * h) * 16 + block));
                    if (row + 8 * h >= valid) {     // behind the expert's last token
                        w[h][0] = w[h][1] = w[h][2] = w[h][3] = 0;
                        step[h] = 0;
                    }
                }
                const uint32_t at = a_at + st * kOperandBytes + write;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const uint32_t step2 = step[h] * 0x00800080u;   // the byte as a bf16 exponent
                    uint32_t v[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[2 * j] = restore_pair(__byte_perm(w[h][j], 0, 0x4140), step2);
                        v[2 * j + 1] = restore_pair(__byte_perm(w[h][j], 0, 0x4342), step2);
                    }
                    store_shared(at + piece0 + h * 8 * 128, v[0], v[1], v[2], v[3]);
                    store_shared(at + piece1 + h * 8 * 128, v[4], v[5], v[6], v[7]);
                }
                if (valid < kDepth) {
                    const uint32_t to = b_at + st * kOperandBytes + write;
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        if (row + 8 * h >= valid) {
                            store_shared(to + piece0 + h * 8 * 128, 0, 0, 0, 0);
                            store_shared(to + piece1 + h * 8 * 128, 0, 0, 0, 0);
                        }
                }
                tc::fence_to_async();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster(tc::map_to(ready(st), 0));
            }
            step0 += uint32_t(count);
        }
    } else if (kOdd && warp >= 12) {
        if constexpr (kOdd) {
            tc::give_registers<kRestoreRegs>();
            const int turn = (warp - 12) >> 2;
            // 16 bytes of a row a lane; 8 neighbouring lanes read and write 128 consecutive bytes of a
            // row, whose 16-byte pieces are permuted by the row's number where they are written
            constexpr int kLanes = kWeightAlongK ? 8 : 16, kRows = 128 / kLanes;
            const int at = int(threadIdx.x) & 127, row0 = at / kLanes, c = at % kLanes;
            const uint32_t write = uint32_t((c >> 3) * kGroupBytes + row0 * 128 + ((c ^ row0) & 7) * 16);
            uint32_t step0 = 0;                     // steps of the tiles before
            for (int n = work.begin; ok && tile_at<kKind, kSplit>(p, table, work, n, s); n = s.next) {
                const int count = s.last - s.first;
                for (int k = int(step0 & 1) ^ turn; k < count; k += 2) {
                    // the stages' number is even: a group always has the same ones and waits for each
                    // of their uses
                    const uint32_t st = (step0 + k) % kStages, round = (step0 + k) / kStages;
                    if (!(ok = tc::mbar_wait_warp(full(st), round & 1))) break;
                    const int d = (s.first + k) * kDepth;
                    const int first = s.e * p.weight_rows + (kWeightAlongK ? s.m + int(rank) * kHalf : d);
                    const int row = first + row0, j = row & 7;
                    const uint32_t read = pieces + st * kRawBytes +
                                          (j * kOddRows + (row >> 3) - ((first - j + 7) >> 3)) * kOddPitch + c * 16;
                    const uint32_t shift = (p.start + uint32_t(j) * p.step) & 15;
                    const uint32_t words = shift >> 2, bits = (shift & 3) * 8;
                    // rows of the sum behind the expert's last one
                    const int valid = kWeightAlongK ? kHalf : p.k_size - d;
                    const uint32_t to = a_at + st * kOperandBytes + write;
#pragma unroll 2
                    for (int i0 = 0; i0 < 8; i0 += 2) {     // two rows' loads in flight
                        uint32_t w[2][8];
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            uint32_t* v = w[h >> 1] + 4 * (h & 1);
                            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                                         : "r"(read + (i0 + (h >> 1)) * (kRows / 8) * kOddPitch + (h & 1) * 16));
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            shift_words(w[h], words, bits);
                            if ((i0 + h) * kRows + row0 >= valid) w[h][0] = w[h][1] = w[h][2] = w[h][3] = 0;
                            store_shared(to + (i0 + h) * kRows * 128, w[h][0], w[h][1], w[h][2], w[h][3]);
                        }
                    }
                    tc::fence_to_async();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive_cluster(tc::map_to(ready(st), 0));
                }
                step0 += uint32_t(count);
            }
        }
    }
    if (!ok) atomicAdd(&g_wait_failures, 1u);
    __syncwarp();
    // Nobody leaves while the other CTA may still signal or read this one: every signal has been
    // waited for by a thread of the CTA that it goes to, so this barrier need not order them.
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_meet();
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_free(tmem, 512);
}

// Tiles summed in parts: the parts in order, rounded once.  A block joins
// kJoinColumns columns of the tile that a part begins, a feature a thread.
constexpr int kJoinColumns = 8, kJoinAhead = 4;
__global__ void __launch_bounds__(kTile) grouped_join(const __grid_constant__ GroupedParams p) {
    grid_wait();
    grid_release();
    const int slot = int(blockIdx.x), column = int(blockIdx.y) * kJoinColumns, f = int(threadIdx.x);
    const GroupedPart q = p.parts[slot];
    if (q.count == 0 || column >= q.columns || f >= q.features) return;
    const int64_t room = int64_t(p.slot_columns) * kTile;
    float sum[kJoinColumns] = {};
    for (int i = 0; i < q.count; i += kJoinAhead) {
        float v[kJoinAhead][kJoinColumns];
#pragma unroll
        for (int a = 0; a < kJoinAhead; ++a) {
            // the first part may be its pair's last piece, every later one is its pair's first
            const int from = i + a == 0 ? slot : 2 * ((slot >> 1) + i + a);
            const float* part = p.partial + from * room + int64_t(column) * kTile + f;
#pragma unroll
            for (int c = 0; c < kJoinColumns; ++c)
                v[a][c] = i + a < q.count && column + c < q.columns ? part[c * kTile] : 0.0f;
        }
#pragma unroll
        for (int a = 0; a < kJoinAhead; ++a)
#pragma unroll
            for (int c = 0; c < kJoinColumns; ++c) sum[c] = __fadd_rn(sum[c], v[a][c]);
    }
#pragma unroll
    for (int c = 0; c < kJoinColumns; ++c) {
        if (column + c >= q.columns) break;
        const int64_t at = q.at + (column + c) * p.out_stride + f;
        if (p.out_bf16) {
            uint16_t* d = static_cast<uint16_t*>(p.out) + at;
            *d = to_bf16(p.accumulate ? __fadd_rn(bf_1(*d), sum[c]) : sum[c]);
        } else {
            float* d = static_cast<float*>(p.out) + at;
            *d = p.accumulate ? __fadd_rn(*d, sum[c]) : sum[c];
        }
    }
}

// An operand copied to 16-byte-aligned rows, for inputs that TMA cannot read.
// Row r is row r % inner of matrix r / inner.
struct Copy {
    const void* from;
    int64_t stride, outer;       // bytes, from row to row and from matrix to matrix
    void* to;
    int64_t to_stride;           // bytes, a multiple of 16
    int64_t rows, inner;
    int64_t row0;                // of the call's rows: the operands copied before
    int bytes;                   // of a row
    int weights;                 // matrix e is not read when expert e has no tokens
};
struct CopyParams {
    Copy op[3];
    int64_t rows;                // of all operands
    const int32_t* offsets;
    int tokens;
};

// A warp copies a row: 16 bytes a lane and turn, from the aligned 16 bytes that
// hold their beginning and (the next lane's) their end.  Only those that hold a
// byte of the row are read.  Behind the row, up to the next 16 bytes, follows
// what was there: TMA's maps end with the row.  All operands of a call in one
// launch: 2047 tokens, 5 x 1001 x 1003 from the checkpoint, 21.3 us with a launch for
// each and single elements.  No source is declared __restrict__: a programmatic
// launch lives while the grid before it writes.
constexpr int kCopyAhead = 4;            // loads of a lane in flight
__global__ void __launch_bounds__(kThreads) copy_rows(const __grid_constant__ CopyParams p) {
    grid_wait();
    grid_release();
    const int lane = int(threadIdx.x) & 31;
    const int64_t warps = int64_t(gridDim.x) * (kThreads / 32);
    for (int64_t r = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); r < p.rows; r += warps) {
        const Copy& c = r >= p.op[2].row0 ? p.op[2] : r >= p.op[1].row0 ? p.op[1] : p.op[0];
        const int64_t row = r - c.row0, e = row / c.inner;
        if (c.weights) {
            const int b = min(max(p.offsets[e], 0), p.tokens);
            if (min(p.offsets[e + 1], p.tokens) <= b) continue;
        }
        const char* from = static_cast<const char*>(c.from) + e * c.outer + (row - e * c.inner) * c.stride;
        char* to = static_cast<char*>(c.to) + row * c.to_stride;
        const int shift = int(reinterpret_cast<uintptr_t>(from) & 15);
        const char* base = from - shift;
        const int span = shift + c.bytes;        // bytes from the first aligned 16 on
        const uint32_t words = uint32_t(shift) >> 2, bits = uint32_t(shift & 3) * 8;
        for (int v0 = 0; v0 * 16 < c.bytes; v0 += 32 * kCopyAhead) {
            uint4 own[kCopyAhead], after[kCopyAhead];
#pragma unroll
            for (int j = 0; j < kCopyAhead; ++j) {
                const int v = v0 + j * 32 + lane;
                own[j] = after[j] = make_uint4(0, 0, 0, 0);
                if (v * 16 < span) own[j] = ld_v4(base + int64_t(v) * 16);
                if (lane == 31 && (v + 1) * 16 < span) after[j] = ld_v4(base + int64_t(v + 1) * 16);
            }
#pragma unroll
            for (int j = 0; j < kCopyAhead; ++j) {
                const int v = v0 + j * 32 + lane;
                uint32_t w[8] = {own[j].x, own[j].y, own[j].z, own[j].w};
                w[4] = __shfl_down_sync(0xFFFFFFFFu, own[j].x, 1);
                w[5] = __shfl_down_sync(0xFFFFFFFFu, own[j].y, 1);
                w[6] = __shfl_down_sync(0xFFFFFFFFu, own[j].z, 1);
                w[7] = __shfl_down_sync(0xFFFFFFFFu, own[j].w, 1);
                if (lane == 31) {
                    w[4] = after[j].x; w[5] = after[j].y; w[6] = after[j].z; w[7] = after[j].w;
                }
                shift_words(w, words, bits);
                if (v * 16 < c.bytes) st_v4(to + int64_t(v) * 16, make_uint4(w[0], w[1], w[2], w[3]));
            }
        }
    }
}

// Can TMA read these rows where they are?
bool tma_rows(const void* p, int64_t stride, int64_t size, int64_t width) {
    return aligned(p, 16) && stride >= width && stride * size % 16 == 0;
}

// An operand as the call gives it, and how it is read: where it is or copied.
struct Operand {
    const void* p;
    int64_t stride, outer;       // in elements; `outer` from matrix to matrix
    int64_t size, rows, inner, width;
    bool copy = false;
    int64_t bytes() const {      // in the workspace
        return copy ? round_up(rows * round_up(width, 16 / size) * size, 16) : 0;
    }
};

Operand operand(const void* p, int64_t stride, int64_t outer, int64_t size, int64_t matrices,
                int64_t inner, int64_t width) {
    Operand o{p, stride, outer, size, matrices * inner, inner, width};
    o.copy = o.rows > 0 && (!tma_rows(p, stride, size, width) ||
                            (matrices > 1 && (outer * size % 16 != 0 || outer < 0)));
    return o;
}

// The copies of a call's operands that TMA cannot read, into `ws`; the operands
// are then where they were copied to.
struct Copies {
    CopyParams p = {};
    int n = 0;

    void add(Operand& o, char*& ws, bool weights) {
        if (!o.copy) return;
        Copy& c = p.op[n++];
        c.from = o.p; c.stride = o.stride * o.size; c.outer = o.outer * o.size;
        o.stride = round_up(o.width, 16 / o.size);
        o.outer = o.inner * o.stride;
        o.p = ws;
        c.to = ws; c.to_stride = o.stride * o.size;
        c.rows = o.rows; c.inner = o.inner; c.row0 = p.rows;
        c.bytes = int(o.width * o.size);
        c.weights = weights;
        p.rows += o.rows;
        ws += o.bytes();
    }
    cudaError_t launch(const int32_t* offsets, int64_t tokens, cudaStream_t s) {
        if (n == 0) return cudaSuccess;
        for (int i = n; i < 3; ++i) p.op[i].row0 = INT64_MAX;
        p.offsets = offsets;
        p.tokens = int(tokens);
        void* args[] = {&p};
        return launch_grid((const void*)copy_rows,
                           dim3(unsigned(std::min<int64_t>(ceil_div(p.rows, kThreads / 32), 152 * 8))),
                           dim3(kThreads), 0, args, s);
    }
};

cudaError_t encode(CUtensorMap* map, const Operand& o, int box_x, int box_y) {
    const bool bytes = o.size == 1;
    const int64_t dims[2] = {o.width, o.rows}, strides[1] = {o.stride * o.size};
    const int box[2] = {box_x, box_y};
    return encode_tensor_map(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                             o.p, 2, dims, strides, box,
                             bytes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaError_t encode_experts(CUtensorMap* map, const Operand& o, int box_x, int box_y) {
    const int64_t experts = o.rows / o.inner;
    const int64_t outer = experts > 1 ? o.outer : o.inner * o.stride;
    const int64_t dims[3] = {o.width, o.inner, experts};
    const int64_t strides[2] = {o.stride * 2, outer * 2};
    const int box[3] = {box_x, box_y, 1};
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, o.p, 3, dims, strides, box,
                             CU_TENSOR_MAP_SWIZZLE_128B);
}

// How the work is dealt out, from what the host knows: `most` tiles at most,
// `tiles` of experts that have about as many tokens, of `steps` steps and `each`
// columns on average, `columns` at most.
struct Plan {
    bool split = false;
    int64_t pairs = 0, slot_columns = 0, partial_bytes = 0, part_bytes = 0;
    int64_t bytes() const { return partial_bytes + part_bytes; }
};

// Steps are dealt out, and parts of tiles joined by a second kernel, where whole
// tiles would take longer: pairs in different places of the sum share less in L2
// (kSplitSlow), and the parts' stores and the second kernel take kSplitCost steps more
// than the stores of whole tiles.  Tiles of few columns wait for memory, not for the
// tensor core: fewer pairs at once then go on faster (0.25 us a step against 0.36 with
// all of them).  Whole and dealt out: weight gradient of 16384 tokens, 200 x 512, 78 and
// 20 us, 2048 x 2560 (80 tiles of 256 steps) 147 and 124, 2048 x 4096 (128 tiles) 152
// and 206; product of 512 tokens, 4096 x 11008 (32 tiles of 172 steps), 52 and 45, of
// 1024 tokens, 4096 x 4096 (64 tiles of 64 steps), 24 and 35; of 32 tokens over 8 experts
// of 11008 x 4096, input gradient (128 tiles of few columns), 107 and 113.  More tiles:
// whole (4096 tokens, 8 experts of 4096 x 4096, 3.4 rounds, 86 and 129).
constexpr double kSplitSlow = 1.15, kSplitCost = 32;
Plan plan_work(int64_t most, int64_t tiles, double steps, int64_t columns, double each) {
    Plan q;
    q.pairs = std::min<int64_t>(most, kPairs);
    const double whole = double(ceil_div(tiles, kPairs)) * steps * (each <= 64 ? 0.7 : 1.0);
    const double dealt = std::max(double(tiles) * steps / kPairs, double(kMinPart));
    if (tiles < 2 * kPairs && whole > kSplitSlow * dealt + kSplitCost) {
        q.split = true;
        q.pairs = std::min<int64_t>(kPairs, std::max(most, int64_t(double(most) * steps / kMinPart)));
        q.slot_columns = std::min<int64_t>(kTile, round_up(columns, 32));
        q.partial_bytes = 2 * q.pairs * q.slot_columns * kTile * 4;
        q.part_bytes = 2 * q.pairs * int64_t(sizeof(GroupedPart));
    }
    return q;
}

Plan product_plan(int64_t rows, int64_t experts, int64_t to, int64_t from) {
    // at most: every expert's last tile may be short
    const int64_t short_ones = std::min(rows, experts), m = ceil_div(to, kTile);
    const int64_t n = rows / kTile + short_ones;
    return plan_work(m * n, m * std::max(ceil_div(rows, kTile), short_ones), double(ceil_div(from, kDepth)),
                     rows, double(rows) / double(n));
}

Plan grad_plan(int64_t rows, int64_t experts, int64_t out_features, int64_t in_features) {
    const int64_t tiles = experts * ceil_div(in_features, kTile) * ceil_div(out_features, kTile);
    return plan_work(tiles, tiles, double(rows) / double(experts * kDepth), out_features, kTile);
}

template <int kKind, bool kSplit>
cudaError_t launch_kernel(KindParams<kKind>& p, const Plan& q, cudaStream_t s) {
    static std::atomic<uint64_t> allowed{0};
    const void* k = (const void*)grouped_pairs<kKind, kSplit>;
    const cudaError_t e = allow_shared_memory(k, smem_bytes(kKind), &allowed);
    if (e != cudaSuccess) return e;
    void* args[] = {&p};
    return launch_grid(k, dim3(unsigned(2 * q.pairs)), dim3(threads(kKind)), smem_bytes(kKind), args, s);
}

template <int kKind>
cudaError_t launch_pairs(KindParams<kKind>& p, const Plan& q, char* ws, cudaStream_t s) {
    if (!q.split) return launch_kernel<kKind, false>(p, q, s);
    p.slot_columns = int(q.slot_columns);
    p.partial = reinterpret_cast<float*>(ws);
    p.parts = reinterpret_cast<GroupedPart*>(ws + q.partial_bytes);
    const cudaError_t e = launch_kernel<kKind, true>(p, q, s);
    if (e != cudaSuccess) return e;
    void* args[] = {static_cast<GroupedParams*>(&p)};
    return launch_grid((const void*)grouped_join,
                       dim3(unsigned(2 * q.pairs), unsigned(q.slot_columns / kJoinColumns)), dim3(kTile), 0,
                       args, s);
}

dpr_status check_sizes(int64_t rows, int64_t experts, int64_t out_features, int64_t in_features) {
    dpr_status st = check_matrix_size(rows, out_features);
    if (st == DPR_OK) st = check_matrix_size(rows, in_features);
    if (st != DPR_OK) return st;
    if (experts < 1) return DPR_ERR_INVALID_ARG;
    if (rows > DPR_MAX_GRAD_ROWS || experts > DPR_MAX_EXPERTS) return DPR_ERR_UNSUPPORTED;
    // tiles are counted in 31 bits
    const int64_t m = ceil_div(out_features, kTile), n = ceil_div(in_features, kTile);
    if (experts * m * n > (int64_t(1) << 30) ||
        (ceil_div(rows, kTile) + experts) * std::max(m, n) > (int64_t(1) << 30))
        return DPR_ERR_UNSUPPORTED;
    return DPR_OK;
}

// Elements from the first to one past the last of the experts' matrices.
int64_t experts_span(int64_t experts, int64_t outer, int64_t rows, int64_t stride, int64_t width) {
    return (experts - 1) * outer + (rows - 1) * stride + width;
}

dpr_status check_experts(const void* p, int64_t stride, int64_t outer, int64_t experts,
                         int64_t rows, int64_t width, int dtype, bool written) {
    const dpr_status st = check_matrix(p, stride, width, dtype, written);
    if (st != DPR_OK) return st;
    if (outer < 0 || (written && experts > 1 && outer < (rows - 1) * stride + width))
        return DPR_ERR_INVALID_ARG;
    // TMA's strides end at 2^40 bytes
    return outer > (int64_t(1) << 38) ? DPR_ERR_UNSUPPORTED : DPR_OK;
}

dpr_status check_workspace(const void* ws, int64_t bytes, int64_t need) {
    if (need == 0) return DPR_OK;
    if (!ws || bytes < need) return DPR_ERR_INVALID_ARG;
    return aligned(ws, 16) ? DPR_OK : DPR_ERR_ALIGNMENT;
}

// Unaligned weights are read as they lie where their rows follow one another
// through all experts, unless so many tokens read them that copying them once is
// faster.  8 experts of 11008 x 4095, product (input gradient): 32 tokens 152 us
// (155) as they lie, 404 (399) copied; 4096 tokens 329 (352) and 501 (509); 16384
// tokens 1090 (1229) and 1039 (1069).  Aligned weights take 115 us for 32 tokens.
constexpr int64_t kOddTokens = 1024;     // an expert, on average
bool read_odd(const Operand& w, int64_t rows) {
    const int64_t experts = w.rows / w.inner;
    return w.copy && w.width >= kDepth && w.stride >= w.width && w.stride < (int64_t(1) << 30) &&
           w.rows >= kDepth && w.rows < (int64_t(1) << 30) &&
           (experts == 1 || w.outer == w.inner * w.stride) && rows <= kOddTokens * experts;
}

cudaError_t encode_odd(GroupedOddParams& p, const Operand& w, bool along_k) {
    p.weight_rows = int(w.inner);
    p.start = unsigned(reinterpret_cast<uintptr_t>(w.p) & 15);
    p.step = unsigned(w.stride * 2 & 15);
    for (int j = 0; j < 8; ++j) {
        const char* row = static_cast<const char*>(w.p) + j * w.stride * 2;
        const int64_t front = reinterpret_cast<uintptr_t>(row) & 15;
        const int64_t dims[2] = {w.width + front / 2, ceil_div(w.rows - j, 8)}, strides[1] = {w.stride * 16};
        const int box[2] = {(along_k ? kDepth : kHalf) + 8, along_k ? 16 : 8};
        const cudaError_t e = encode_tensor_map(&p.odd[j], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, row - front, 2,
                                                dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// The operands of the product (x) or of the input gradient (dy).  The result is whether the
// weights, unaligned, are read as they lie.
bool operands(bool input_grad, const void* x, int64_t x_stride, int64_t rows, int64_t experts,
              const void* weight, int64_t weight_stride, int64_t expert_stride,
              int64_t out_features, int64_t in_features, Operand* a, Operand* b) {
    *a = operand(weight, weight_stride, expert_stride, 2, experts, out_features, in_features);
    *b = operand(x, x_stride, 0, 2, 1, rows, input_grad ? out_features : in_features);
    const bool odd = read_odd(*a, rows);
    if (odd) a->copy = false;
    return odd;
}

dpr_status product_workspace(bool input_grad, const void* x, int64_t x_stride, int64_t rows,
                             int64_t experts, const void* weight, int64_t weight_stride,
                             int64_t expert_stride, int64_t out_features, int64_t in_features,
                             int64_t* bytes) {
    if (!bytes) return DPR_ERR_INVALID_ARG;
    *bytes = 0;
    const dpr_status st = check_sizes(rows, experts, out_features, in_features);
    if (st != DPR_OK || rows == 0) return st;
    Operand a, b;
    operands(input_grad, x, x_stride, rows, experts, weight, weight_stride, expert_stride,
             out_features, in_features, &a, &b);
    *bytes = a.bytes() + b.bytes() +
             product_plan(rows, experts, input_grad ? in_features : out_features,
                          input_grad ? out_features : in_features).bytes();
    return DPR_OK;
}

dpr_status product(bool input_grad, const void* x, int64_t x_stride, int64_t rows,
                   const int32_t* offsets, int64_t experts, const void* weight,
                   int64_t weight_stride, int64_t expert_stride, int64_t out_features,
                   int64_t in_features, void* out, int64_t out_stride, int dtype, void* workspace,
                   int64_t workspace_bytes, void* stream) {
    int64_t need = 0;
    dpr_status st = product_workspace(input_grad, x, x_stride, rows, experts, weight, weight_stride,
                                      expert_stride, out_features, in_features, &need);
    if (st != DPR_OK) return st;
    if (!dtype_ok(dtype)) return DPR_ERR_INVALID_ARG;
    if (rows == 0) return DPR_OK;
    const int64_t from = input_grad ? out_features : in_features;
    const int64_t to = input_grad ? in_features : out_features;
    if ((st = check_matrix(x, x_stride, from, DPR_BF16, false)) != DPR_OK) return st;
    if ((st = check_matrix(out, out_stride, to, dtype, true)) != DPR_OK) return st;
    if ((st = check_experts(weight, weight_stride, expert_stride, experts, out_features,
                            in_features, DPR_BF16, false)) != DPR_OK) return st;
    if (!offsets) return DPR_ERR_INVALID_ARG;
    if (!aligned(offsets, 4)) return DPR_ERR_ALIGNMENT;
    if ((st = check_workspace(workspace, workspace_bytes, need)) != DPR_OK) return st;
    SpanList outs, ins;
    outs.add(out, matrix_bytes(rows, to, out_stride, dtype_size(dtype)));
    if (need > 0) outs.add(workspace, uint64_t(need));
    ins.add(x, matrix_bytes(rows, from, x_stride, 2));
    ins.add(weight, 2 * uint64_t(experts_span(experts, expert_stride, out_features, weight_stride,
                                              in_features)));
    ins.add(offsets, 4 * uint64_t(experts + 1));
    if (!outs.disjoint() || outs.meets(ins)) return DPR_ERR_ALIAS;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    Operand a, b;
    const bool odd = operands(input_grad, x, x_stride, rows, experts, weight, weight_stride, expert_stride,
                              out_features, in_features, &a, &b);
    GroupedOddParams p = {};
    p.offsets = offsets; p.experts = int(experts); p.rows = int(rows);
    p.m_size = int(to); p.m_tiles = int(ceil_div(to, kTile));
    p.k_size = int(from);
    p.out = out; p.out_stride = out_stride; p.out_bf16 = dtype == DPR_BF16;
    Copies copies;
    copies.add(a, ws, true);
    copies.add(b, ws, false);
    cudaError_t e = copies.launch(offsets, rows, s);
    if (e == cudaSuccess)
        e = odd ? encode_odd(p, a, !input_grad) : encode_experts(&p.a, a, 64, input_grad ? kDepth : kHalf);
    if (e == cudaSuccess) e = encode(&p.b, b, kDepth, kHalf);
    if (e == cudaSuccess) e = encode(&p.b_piece, b, kDepth, kPiece);
    if (e != cudaSuccess) return record_cuda_status(e);
    const Plan q = product_plan(rows, experts, to, from);
    if (odd)
        e = input_grad ? launch_pairs<kInputGradOdd>(p, q, ws, s) : launch_pairs<kForwardOdd>(p, q, ws, s);
    else
        e = input_grad ? launch_pairs<kInputGrad>(p, q, ws, s) : launch_pairs<kForward>(p, q, ws, s);
    return record_cuda_status(e);
}

// The operands of the weight gradients: x, or its codes and steps; dy.
void grad_operands(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride,
                   const dpr_checkpoint* c, int64_t rows, int64_t out_features,
                   int64_t in_features, Operand* a, Operand* steps, Operand* b) {
    *b = operand(dy, dy_stride, 0, 2, 1, rows, out_features);
    if (c) {
        *a = operand(c->codes, c->code_stride, 0, 1, 1, rows, in_features);
        *steps = operand(c->steps, c->step_stride, 0, 1, 1, rows,
                         ceil_div(in_features, kBlockChannels));
    } else {
        *a = operand(x, x_stride, 0, 2, 1, rows, in_features);
        *steps = operand(nullptr, 0, 0, 1, 0, 1, 1);
    }
}

}  // namespace

cudaError_t grouped_wait_failures(unsigned int* count) {
    return cudaMemcpyFromSymbol(count, g_wait_failures, sizeof(*count));
}

}  // namespace dpr

using namespace dpr;

extern "C" {

dpr_status dpr_grouped_linear_workspace(const void* x, int64_t x_stride, int64_t rows,
                                        int64_t experts, const void* weight,
                                        int64_t weight_stride, int64_t expert_stride,
                                        int64_t out_features, int64_t in_features, int64_t* bytes) {
    return product_workspace(false, x, x_stride, rows, experts, weight, weight_stride,
                             expert_stride, out_features, in_features, bytes);
}

dpr_status dpr_grouped_linear(const void* x, int64_t x_stride, int64_t rows,
                              const int32_t* offsets, int64_t experts, const void* weight,
                              int64_t weight_stride, int64_t expert_stride, int64_t out_features,
                              int64_t in_features, void* y, int64_t y_stride, int dtype,
                              void* workspace, int64_t workspace_bytes, void* stream) {
    return product(false, x, x_stride, rows, offsets, experts, weight, weight_stride, expert_stride,
                   out_features, in_features, y, y_stride, dtype, workspace, workspace_bytes,
                   stream);
}

dpr_status dpr_grouped_linear_input_grad_workspace(const void* dy, int64_t dy_stride, int64_t rows,
                                                   int64_t experts, const void* weight,
                                                   int64_t weight_stride, int64_t expert_stride,
                                                   int64_t out_features, int64_t in_features,
                                                   int64_t* bytes) {
    return product_workspace(true, dy, dy_stride, rows, experts, weight, weight_stride,
                             expert_stride, out_features, in_features, bytes);
}

dpr_status dpr_grouped_linear_input_grad(const void* dy, int64_t dy_stride, int64_t rows,
                                         const int32_t* offsets, int64_t experts,
                                         const void* weight, int64_t weight_stride,
                                         int64_t expert_stride, int64_t out_features,
                                         int64_t in_features, void* dx, int64_t dx_stride,
                                         int dtype, void* workspace, int64_t workspace_bytes,
                                         void* stream) {
    return product(true, dy, dy_stride, rows, offsets, experts, weight, weight_stride, expert_stride,
                   out_features, in_features, dx, dx_stride, dtype, workspace, workspace_bytes,
                   stream);
}

dpr_status dpr_grouped_linear_weight_grad_workspace(const void* dy, int64_t dy_stride,
                                                    const void* x, int64_t x_stride,
                                                    const dpr_checkpoint* x_ckpt, int64_t rows,
                                                    int64_t experts, int64_t out_features,
                                                    int64_t in_features, int64_t* bytes) {
    if (!bytes) return DPR_ERR_INVALID_ARG;
    *bytes = 0;
    const dpr_status st = check_sizes(rows, experts, out_features, in_features);
    if (st != DPR_OK || rows == 0) return st;
    Operand a, steps, b;
    grad_operands(dy, dy_stride, x, x_stride, x_ckpt, rows, out_features, in_features, &a, &steps,
                  &b);
    *bytes = a.bytes() + steps.bytes() + b.bytes() +
             grad_plan(rows, experts, out_features, in_features).bytes();
    return DPR_OK;
}

dpr_status dpr_grouped_linear_weight_grad(const void* dy, int64_t dy_stride, const void* x,
                                          int64_t x_stride, const dpr_checkpoint* x_ckpt,
                                          int64_t rows, const int32_t* offsets, int64_t experts,
                                          int64_t out_features, int64_t in_features, void* dweight,
                                          int64_t dweight_stride, int64_t expert_stride, int dtype,
                                          int accumulate, void* workspace, int64_t workspace_bytes,
                                          void* stream) {
    int64_t need = 0;
    dpr_status st = dpr_grouped_linear_weight_grad_workspace(
        dy, dy_stride, x, x_stride, x_ckpt, rows, experts, out_features, in_features, &need);
    if (st != DPR_OK) return st;
    if (!dtype_ok(dtype)) return DPR_ERR_INVALID_ARG;
    if ((st = check_experts(dweight, dweight_stride, expert_stride, experts, out_features,
                            in_features, dtype, true)) != DPR_OK) return st;
    if (!offsets) return DPR_ERR_INVALID_ARG;
    if (!aligned(offsets, 4)) return DPR_ERR_ALIGNMENT;
    SpanList outs, ins;
    outs.add(dweight, uint64_t(dtype_size(dtype)) *
                          uint64_t(experts_span(experts, expert_stride, out_features,
                                                dweight_stride, in_features)));
    ins.add(offsets, 4 * uint64_t(experts + 1));
    if (rows > 0) {
        if ((st = check_matrix(dy, dy_stride, out_features, DPR_BF16, false)) != DPR_OK) return st;
        st = x_ckpt ? check_checkpoint(x_ckpt, in_features)
                    : check_matrix(x, x_stride, in_features, DPR_BF16, false);
        if (st != DPR_OK) return st;
        if ((st = check_workspace(workspace, workspace_bytes, need)) != DPR_OK) return st;
        if (need > 0) outs.add(workspace, uint64_t(need));
        ins.add(dy, matrix_bytes(rows, out_features, dy_stride, 2));
        if (x_ckpt) ins.add(*x_ckpt, rows, in_features);
        else ins.add(x, matrix_bytes(rows, in_features, x_stride, 2));
    }
    if (!outs.disjoint() || outs.meets(ins)) return DPR_ERR_ALIAS;
    if (rows == 0 && accumulate) return DPR_OK;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    GroupedParams p = {};
    p.offsets = offsets; p.experts = int(experts); p.rows = int(rows);
    p.m_size = int(in_features); p.m_tiles = int(ceil_div(in_features, kTile));
    p.n_size = int(out_features); p.n_tiles = int(ceil_div(out_features, kTile));
    p.out = dweight; p.out_stride = dweight_stride; p.out_expert_stride = expert_stride;
    p.out_bf16 = dtype == DPR_BF16; p.accumulate = accumulate != 0;
    cudaError_t e = cudaSuccess;
    if (rows > 0) {       // without tokens no tile loads anything
        Operand a, steps, b;
        grad_operands(dy, dy_stride, x, x_stride, x_ckpt, rows, out_features, in_features, &a,
                      &steps, &b);
        Copies copies;
        copies.add(a, ws, false);
        copies.add(steps, ws, false);
        copies.add(b, ws, false);
        e = copies.launch(offsets, rows, s);
        if (e == cudaSuccess) e = encode(&p.a, a, 64, kDepth);
        if (e == cudaSuccess && x_ckpt) e = encode(&p.steps, steps, 16, kDepth);
        if (e == cudaSuccess) e = encode(&p.b, b, 64, kDepth);
        if (e != cudaSuccess) return record_cuda_status(e);
    }
    const Plan q = grad_plan(rows, experts, out_features, in_features);
    e = x_ckpt && rows > 0 ? launch_pairs<kWeightGradSaved>(p, q, ws, s)
                           : launch_pairs<kWeightGrad>(p, q, ws, s);
    return record_cuda_status(e);
}

}  // extern "C"
