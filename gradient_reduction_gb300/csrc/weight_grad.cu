// A linear layer's weight gradient dW = dY^T X~ from the 8-bit checkpoint of
// X, on the tensor cores.  The sum runs along the tokens, the slow dimension
// of both inputs, so both operands are "M/N-major": dY goes from memory to
// shared memory by TMA as it is, X~ is restored there from its codes on the
// way (exactly: a code times a power of two is a bf16 number).
//
// A pair of CTAs computes a tile of 256 in-features (the M of the
// instruction, 128 in each CTA) by 256 out-features (N) with cta_group::2
// instructions, so each CTA loads only half of the dY tile.  Restoring
// happens on the M side: 128 channels per CTA are restored once for 256
// out-features, 8192 codes per 64 tokens, against 512 cycles of matrix
// instructions.  With in-features on the lanes of the accumulator, a warp's
// store writes 32 consecutive elements of a row of dW straight from
// registers.
//
// The tensor core's fp32 accumulation truncates, an error that grows with the
// length of the sum (terms of both signs: 5.7e-6 relative after 8192 tokens,
// against 5.8e-7 for rounded fp32 sums).  So an accumulator runs over 1024 tokens
// only; then the other one goes on (two of 256 columns fill the tensor memory)
// while the first is added, rounded to nearest, to the tile's sums in the
// registers of eight warps: 5.4e-7, and 8.4e-7 for terms of one sign, where every
// truncation loses.
//
// Warps of a CTA: 0 issues the TMA loads, 1 the matrix instructions (first
// CTA only), 4-11 keep the sums and store them, 12-19 restore: two groups of
// four warps take turns, so that one group's latencies hide behind the other.
//
// Per step of 64 tokens a CTA reads 25 KB into its ring of five stages and
// takes 0.38 us, 0.354 us being the rate of the measured bf16 matrix peak under
// the power limit (0.36 without the restoring warps' wait for the stage's last
// use, which no run may do without).  8192 tokens, 4096 x 4096, fp32: 180 us with
// the join (1.53 PFLOP/s, 0.80 of the measured burst peak, 0.90 of the sustained
// one); 4096 tokens, 11008 x 4096, bf16: 229 us (1.61 PFLOP/s; 240 with two waits
// in turn instead of one look at both barriers first).  What is left is filling
// and draining (some 8 us), the join and the last, dealt-out tiles.
//
// What made it fast, 8192 tokens, 4096 x 4096, fp32: releasing arrivals at CTA
// scope 341 -> 230 us, one ring with one commit a step 230 -> 220, electing the
// issuing thread (tensor_core.cuh) 220 -> 173.  Separate rings for codes, dY and
// restored operands are slower (199 us): two more waits a step on the restoring
// path, and the codes queue behind dY in the TMA unit.
//
// Work: whole waves of tiles first, then the tokens of the tiles left over are
// dealt out evenly to all pairs; parts of a tile are summed in fp32 in the
// workspace and joined in token order by a second kernel.
#include <algorithm>
#include <atomic>

#include "ops_device.cuh"
#include "ops_kernels.h"
#include "tensor_core.cuh"

namespace dpr {

namespace {

constexpr int kTile = 256;               // in-features and out-features of a tile
constexpr int kHalf = 128;               // of each CTA
constexpr int kTokens = 64;              // per step of the main loop
constexpr int kStages = 5;               // ring of loaded inputs and restored operands
constexpr int kChunk = 16;               // main-loop steps per accumulator
constexpr int kDyBytes = kHalf * kTokens * 2;
constexpr int kCodeBytes = kHalf * kTokens;
constexpr int kStepBytes = 16 * kTokens; // 16 step bytes a token, 4 of them used
constexpr int kStageBytes = kDyBytes + kCodeBytes + kStepBytes;
constexpr int kOperandBytes = kHalf * kTokens * 2;
constexpr int kGroupBytes = 64 * kTokens * 2;   // 64 channels of an operand
constexpr int kSmemBytes = 1024 + kStages * (kOperandBytes + kStageBytes);
constexpr int kGradThreads = 640;
constexpr int kSumWarps = 8;
constexpr int kRestoreWarps = 4;         // of each of the two groups
// Registers per thread after the split (warpgroups: loads and matrix
// instructions, 2 of sums, 2 of restoring); together no more than the
// launch's 96 for each of five.
constexpr int kIssueRegs = 40, kSumRegs = 160, kRestoreRegs = 56;
static_assert(kIssueRegs + 2 * kSumRegs + 2 * kRestoreRegs <= 5 * 96, "the block's registers");

}  // namespace

struct WeightGradParams {
    CUtensorMap dy, codes, steps;
    void* dw;
    int64_t dw_stride;
    float* partial;          // [2 * pairs][256 out][256 in]
    int out_features;
    int in_features;
    int out_tiles;
    int in_tiles;
    int blocks;              // steps of the main loop per tile
    int waves;               // whole tiles per pair, before the dealt-out rest
    int rest_tiles;          // tiles dealt out: the last ones
    int64_t rest_chunk;      // steps per pair of those
    int dw_bf16;
    int accumulate;
};

namespace {

__device__ unsigned int g_wait_failures;

// A pair's piece of work: steps [first, last) of a tile.
struct Segment {
    int tile;
    int first, last;
    bool whole;
    int slot;                // of the partial sums, when not whole
};

// The n-th piece of pair `pair`; false when there is none.
__device__ __forceinline__ bool segment(const WeightGradParams& p, int pairs, int pair, int n,
                                        Segment& s) {
    if (n < p.waves) {
        s.tile = n * pairs + pair;
        s.first = 0; s.last = p.blocks; s.whole = true; s.slot = 0;
        return true;
    }
    if (p.rest_tiles == 0) return false;
    const int64_t total = int64_t(p.rest_tiles) * p.blocks;
    const int64_t begin = min(int64_t(pair) * p.rest_chunk, total);
    const int64_t end = min(begin + p.rest_chunk, total);
    if (begin >= end) return false;
    const int t = int(begin / p.blocks) + (n - p.waves);
    const int64_t t0 = int64_t(t) * p.blocks;
    if (t0 >= end) return false;
    s.tile = p.waves * pairs + t;
    s.first = int(max(begin - t0, int64_t(0)));
    s.last = int(min(end - t0, int64_t(p.blocks)));
    s.whole = s.first == 0 && s.last == p.blocks;
    s.slot = 2 * pair + (n - p.waves);
    return true;
}

// Tiles in columns of 8 out-tiles, so that the tiles of a wave share inputs.
__device__ __forceinline__ void tile_origin(const WeightGradParams& p, int tile, int& o, int& i) {
    const int group = tile / (8 * p.in_tiles);
    const int rest = tile - group * 8 * p.in_tiles;
    const int height = min(8, p.out_tiles - group * 8);
    i = rest / height * kTile;
    o = (group * 8 + rest % height) * kTile;
}

__device__ __forceinline__ void put_grad(const WeightGradParams& p, int64_t at, float v) {
    if (p.dw_bf16) {
        uint16_t* d = static_cast<uint16_t*>(p.dw) + at;
        *d = to_bf16(p.accumulate ? __fadd_rn(bf_1(*d), v) : v);
    } else {
        float* d = static_cast<float*>(p.dw) + at;
        *d = p.accumulate ? __fadd_rn(*d, v) : v;
    }
}

// Consecutive rows of dW at one column: `count` of a thread's kN sums, the
// rows `stride` bytes apart.  The address advances step by step (and is
// hidden from the compiler, which would otherwise compute all kN at once and
// spill the sums).  With kAdd every row's load waits for the store before it, kN
// times the latency of memory for a tile: 8192 tokens, 4096 x 4096, fp32 321 us
// against 172 without, 16 tokens 137 against 16.
template <bool kBf16, bool kAdd, int kN>
__device__ __forceinline__ void store_column(char* d, int64_t stride, int count,
                                             const float (&sum)[kN]) {
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        if (j < count) {
            float v = sum[j];
            if constexpr (kBf16) {
                uint16_t h;
                if constexpr (kAdd) {
                    asm volatile("ld.global.u16 %0, [%1];" : "=h"(h) : "l"(d) : "memory");
                    v = __fadd_rn(bf_1(h), v);
                }
                h = to_bf16(v);
                asm volatile("st.global.u16 [%0], %1;" ::"l"(d), "h"(h) : "memory");
            } else {
                if constexpr (kAdd) {
                    float old;
                    asm volatile("ld.global.f32 %0, [%1];" : "=f"(old) : "l"(d) : "memory");
                    v = __fadd_rn(old, v);
                }
                asm volatile("st.global.f32 [%0], %1;" ::"l"(d), "f"(v) : "memory");
            }
        }
        d += stride;
        asm volatile("" : "+l"(d));
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGradThreads, 1)
weight_grad_pairs(const __grid_constant__ WeightGradParams p) {
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[3 * kStages + 4];
    __shared__ uint32_t tmem_slot;

    const uint32_t base = (tc::smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t operands = base;                          // [kStages], 1024-byte aligned
    const uint32_t stages = base + kStages * kOperandBytes; // [kStages] dY
    const uint32_t codes = stages + kStages * kDyBytes;      // [kStages] codes
    const uint32_t steps = codes + kStages * kCodeBytes;     // [kStages] step bytes
    const uint32_t bar0 = tc::smem_addr(bars);
    const auto full = [&](int s) { return bar0 + 8u * s; };                         // loads landed
    const auto free_ = [&](int s) { return bar0 + 8u * (kStages + s); };            // stage consumed
    const auto ready = [&](int s) { return bar0 + 8u * (2 * kStages + s); };        // restored, both CTAs
    const auto summed = [&](int a) { return bar0 + 8u * (3 * kStages + a); };
    const auto stored = [&](int a) { return bar0 + 8u * (3 * kStages + 2 + a); };

    const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
    const uint32_t rank = tc::cluster_rank();
    const int pairs = int(gridDim.x) >> 1, pair = int(blockIdx.x) >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(full(s), 1);
            tc::mbar_init(free_(s), 1);
            tc::mbar_init(ready(s), 2 * kRestoreWarps);
        }
        for (int a = 0; a < 2; ++a) {
            tc::mbar_init(summed(a), 1);
            tc::mbar_init(stored(a), 2 * kSumWarps);
        }
        tc::mbar_init_fence();
        tc::tma_prefetch_map(&p.dy);
        tc::tma_prefetch_map(&p.codes);
        tc::tma_prefetch_map(&p.steps);
    }
    if (warp == 1) tc::tmem_alloc(tc::smem_addr(&tmem_slot), 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_slot;
    grid_wait();
    grid_release();

    bool ok = true;
    Segment s;
    if (warp < 4) tc::give_registers<kIssueRegs>();
    if (warp == 0) {
        if (tc::elect_one()) {
            int st = 0;
            uint32_t round = 0;
            for (int n = 0; ok && segment(p, pairs, pair, n, s); ++n) {
                int o, i;
                tile_origin(p, s.tile, o, i);
                o += int(rank) * kHalf;
                i += int(rank) * kHalf;
                for (int k = s.first; k < s.last; ++k) {
                    if (!(ok = tc::mbar_wait(free_(st), (round & 1) ^ 1))) break;
                    tc::mbar_expect(full(st), kStageBytes);
                    const int t = k * kTokens;
                    tc::tma_load(codes + st * kCodeBytes, &p.codes, i, t, full(st));
                    tc::tma_load(codes + st * kCodeBytes + kCodeBytes / 2, &p.codes, i + 64, t,
                                 full(st));
                    tc::tma_load(steps + st * kStepBytes, &p.steps, (i / kBlockChannels) & ~15, t,
                                 full(st));
                    tc::tma_load(stages + st * kDyBytes, &p.dy, o, t, full(st));
                    tc::tma_load(stages + st * kDyBytes + kGroupBytes, &p.dy, o + 64, t, full(st));
                    if (++st == kStages) { st = 0; ++round; }
                }
            }
            // every load has landed and every signal of the matrix instructions has arrived
            // here before the CTA may leave: the last use of each stage and buffer
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
            constexpr uint32_t instruction = tc::bf16_instruction(kTile, kTile);
            const uint64_t x0 = tc::operand(operands, kGroupBytes, 1024);
            const uint64_t y0 = tc::operand(stages, kGroupBytes, 1024);
            uint32_t st = 0, round = 0, acc = 0, acc_round = 0;
            for (int n = 0; ok && segment(p, pairs, pair, n, s); ++n) {
                for (int left = s.last - s.first; ok && left > 0; left -= kChunk) {
                    if (!(ok = tc::mbar_wait(stored(acc), (acc_round & 1) ^ 1))) break;
                    const uint32_t d = tmem + acc * kTile;
                    bool add = false;
                    for (int k = min(left, kChunk); k > 0; --k) {
                        if (!(ok = tc::mbar_wait(ready(st), round & 1))) break;
                        tc::fence_after_sync();
                        const uint64_t x = x0 + st * (kOperandBytes >> 4);
                        const uint64_t y = y0 + st * (kDyBytes >> 4);
#pragma unroll
                        for (int j = 0; j < kTokens / 16; ++j) {  // 16 tokens: 2048 bytes of a group
                            tc::mma(d, x + j * (2048 >> 4), y + j * (2048 >> 4), instruction, add);
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
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 12) {
        tc::take_registers<kSumRegs>();
        constexpr int kColumns = kTile / 2;
        const int quarter = warp & 3;               // the lanes this warp may read
        const int column = (warp - 4) / 4 * kColumns;
        const int ci = int(rank) * kHalf + quarter * 32 + lane;
        int acc = 0;
        uint32_t acc_round = 0;
        float sum[kColumns];
        for (int n = 0; ok && segment(p, pairs, pair, n, s); ++n) {
#pragma unroll
            for (int j = 0; j < kColumns; ++j) sum[j] = 0.0f;
            for (int k = s.first; k < s.last; k += kChunk) {
                if (!(ok = tc::mbar_wait_warp(summed(acc), acc_round & 1))) break;
                tc::fence_after_sync();
                const uint32_t from = tmem + acc * kTile + column + (uint32_t(quarter) << 21);
#pragma unroll
                for (int c = 0; c < kColumns; c += 16) {
                    uint32_t v[16];
                    tc::tmem_load16(from + c, v);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        sum[c + j] = __fadd_rn(sum[c + j], __uint_as_float(v[j]));
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster(tc::map_to(stored(acc), 0));
                if (++acc == 2) { acc = 0; ++acc_round; }
            }
            if (!ok) break;
            if (s.whole) {
                int o, i;
                tile_origin(p, s.tile, o, i);
                o += column;
                i += ci;
                if (i < p.in_features) {
                    const int64_t size = p.dw_bf16 ? 2 : 4;
                    char* d = static_cast<char*>(p.dw) + (int64_t(o) * p.dw_stride + i) * size;
                    const int64_t stride = p.dw_stride * size;
                    const int count = p.out_features - o;
                    if (p.dw_bf16) {
                        if (p.accumulate) store_column<true, true>(d, stride, count, sum);
                        else store_column<true, false>(d, stride, count, sum);
                    } else {
                        if (p.accumulate) store_column<false, true>(d, stride, count, sum);
                        else store_column<false, false>(d, stride, count, sum);
                    }
                }
            } else {
                float* d = p.partial + (int64_t(s.slot) * kTile + column) * kTile + ci;
                store_column<false, false>(reinterpret_cast<char*>(d), kTile * 4, kColumns, sum);
            }
        }
    } else if (warp >= 12) {
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
        uint32_t step0 = 0;                         // steps of the main loop before this segment
        for (int n = 0; ok && segment(p, pairs, pair, n, s); ++n) {
            int o, i;
            tile_origin(p, s.tile, o, i);
            const uint32_t block = uint32_t(((i + int(rank) * kHalf) / kBlockChannels & 15) +
                                            group * 2 + (chunk >> 1));
            const uint32_t count = uint32_t(s.last - s.first);
            for (uint32_t k = (step0 & 1) ^ uint32_t(turn); k < count; k += 2) {
                const uint32_t st = (step0 + k) % kStages, round = (step0 + k) / kStages;
                // The stage's use before this one was the other group's (their number is odd), and
                // loads may land out of order.  Until that use is over, `full` may still be in its
                // phase, and then this wait would take the one before it, long complete, for its own.
                bool landed = round > 0 && tc::mbar_passed(free_(st), (round & 1) ^ 1, full(st), round & 1);
                if (!__all_sync(0xFFFFFFFFu, landed))
                    landed = (round == 0 || tc::mbar_wait(free_(st), (round & 1) ^ 1)) &&
                             tc::mbar_wait(full(st), round & 1);
                if (!(ok = __all_sync(0xFFFFFFFFu, landed))) break;
                uint32_t w[4][4], step[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[h][0]), "=r"(w[h][1]), "=r"(w[h][2]), "=r"(w[h][3])
                                 : "r"(codes + st * kCodeBytes + read + h * 8 * 64));
                    asm volatile("ld.shared.u8 %0, [%1];"
                                 : "=r"(step[h])
                                 : "r"(steps + st * kStepBytes + (row + 8 * h) * 16 + block));
                }
                uint32_t v[4][8];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const uint32_t step2 = step[h] * 0x00800080u;   // the byte as a bf16 exponent
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[h][2 * j] = restore_pair(__byte_perm(w[h][j], 0, 0x4140), step2);
                        v[h][2 * j + 1] = restore_pair(__byte_perm(w[h][j], 0, 0x4342), step2);
                    }
                }
                const uint32_t at = operands + st * kOperandBytes + write;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     at + piece0 + h * 8 * 128),
                                 "r"(v[h][0]), "r"(v[h][1]), "r"(v[h][2]), "r"(v[h][3])
                                 : "memory");
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     at + piece1 + h * 8 * 128),
                                 "r"(v[h][4]), "r"(v[h][5]), "r"(v[h][6]), "r"(v[h][7])
                                 : "memory");
                }
                tc::fence_to_async();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_cluster(tc::map_to(ready(st), 0));
            }
            step0 += count;
        }
    }
    if (!ok) atomicAdd(&g_wait_failures, 1u);
    __syncwarp();
    // nobody leaves while the other CTA may still signal or read this one
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_free(tmem, 512);
}

// Up to four tokens: the product is an outer product or little more, and
// writing dW is all that takes time, which the tensor-core kernel's eight
// storing warps do more slowly (4 tokens, 4096 x 4096, fp32: 11.8 us here,
// 16.7 there; 2 tokens, 10038 x 2934: 28 and 51).  A block holds the tokens of
// 1024 in-features, 4 a thread, in registers, and walks over out-features 4 at
// a time, whose dY it keeps in shared memory.  Any strides and addresses.
// (With 16 tokens in registers the loads of the codes one by one take longer
// than the tensor-core kernel does: 38 us against 17.)
constexpr int kFew = 4;
constexpr int kFewThreads = 256, kFewOut = 64;
__global__ void __launch_bounds__(kFewThreads)
weight_grad_few(const __grid_constant__ WeightGradParams p, const uint16_t* dy, int64_t dy_stride,
                dpr_checkpoint x, int tokens) {
    __shared__ __align__(16) float d[kFew][kFewOut];
    grid_wait();
    grid_release();
    const int i0 = int(blockIdx.x) * 4 * kFewThreads + int(threadIdx.x);
    const int o0 = int(blockIdx.y) * kFewOut;
    for (int q = int(threadIdx.x); q < kFew * kFewOut; q += kFewThreads) {
        const int t = q / kFewOut, o = o0 + q % kFewOut;
        d[t][q % kFewOut] = t < tokens && o < p.out_features ? bf_1(dy[t * dy_stride + o]) : 0.0f;
    }
    float v[kFew][4];
#pragma unroll
    for (int t = 0; t < kFew; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * kFewThreads;
            v[t][j] = 0.0f;
            if (t < tokens && i < p.in_features) {
                CodeRaw<1> code;
                float f[1];
                load_codes<1>(x.codes + t * x.code_stride + i, code);
                decode<1>(code, step_value(x.steps[t * x.step_stride + i / kBlockChannels]), f);
                v[t][j] = f[0];
            }
        }
    __syncthreads();
    const int rows = min(kFewOut, p.out_features - o0);
    for (int r = 0; r < rows; r += 4) {
        float acc[4][4] = {};
#pragma unroll
        for (int t = 0; t < kFew; ++t) {
            const float4 a = *reinterpret_cast<const float4*>(&d[t][r]);
            const float w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[m][j] = __fmaf_rn(w[m], v[t][j], acc[m][j]);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (r + m < rows && i0 + j * kFewThreads < p.in_features)
                    put_grad(p, int64_t(o0 + r + m) * p.dw_stride + i0 + j * kFewThreads, acc[m][j]);
    }
}

// Tiles summed in parts: the parts in token order, then as put_grad.  A block
// joins two out-features of a dealt-out tile, 64 threads and 4 in-features a
// thread for each, so that a single tile still spreads over 128 SMs; the
// parts are loaded eight at a time (one by one the loads' latency made the
// join of 32 parts take 24 us).
constexpr int kJoinThreads = 128, kJoinRows = 2, kJoinAhead = 8;
__global__ void __launch_bounds__(kJoinThreads)
weight_grad_join(const __grid_constant__ WeightGradParams p, int pairs) {
    grid_wait();
    grid_release();
    const int t = int(blockIdx.x);
    const int64_t t0 = int64_t(t) * p.blocks;
    const int first = int(t0 / p.rest_chunk), last = int((t0 + p.blocks - 1) / p.rest_chunk);
    if (first == last) return;               // one pair summed it all
    int o, i;
    tile_origin(p, p.waves * pairs + t, o, i);
    const int row = int(blockIdx.y) * kJoinRows + (int(threadIdx.x) >> 6);
    const int column = int(threadIdx.x) & 63;
    if (o + row >= p.out_features) return;
    // the first pair's part may be its second piece, every later one's is its first
    const int slot0 = 2 * first + t - int(int64_t(first) * p.rest_chunk / p.blocks);
    const float* d = p.partial + int64_t(row) * kTile + column;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int q = first; q <= last; q += kJoinAhead) {
        float w[kJoinAhead][4];
#pragma unroll
        for (int a = 0; a < kJoinAhead; ++a) {
            if (q + a > last) break;
            const int slot = q + a == first ? slot0 : 2 * (q + a);
            const float* f = d + int64_t(slot) * kTile * kTile;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[a][j] = f[64 * j];
        }
#pragma unroll
        for (int a = 0; a < kJoinAhead; ++a) {
            if (q + a > last) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __fadd_rn(v[j], w[a][j]);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (i + column + 64 * j < p.in_features)
            put_grad(p, int64_t(o + row) * p.dw_stride + i + column + 64 * j, v[j]);
}

// Rows copied to 16-byte-aligned ones, for inputs that TMA cannot read; four
// loads of a thread in flight before its stores.  The source is not declared
// __restrict__: that allows loads that take memory to be unchanged as long as the
// kernel lives, and a programmatic launch lives while the grid before it writes.
template <typename T>
__global__ void __launch_bounds__(kThreads)
repack_rows(const T* from, int64_t from_stride, T* to, int64_t to_stride, int64_t rows, int width) {
    grid_wait();
    grid_release();
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* f = from + r * from_stride;
        T* t = to + r * to_stride;
        for (int c0 = int(threadIdx.x); c0 < width; c0 += 4 * kThreads) {
            T v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c0 + j * kThreads < width) v[j] = f[c0 + j * kThreads];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c0 + j * kThreads < width) t[c0 + j * kThreads] = v[j];
        }
    }
}

// dW = 0, for a call without tokens.
__global__ void __launch_bounds__(kThreads) zero_rows(const __grid_constant__ WeightGradParams p) {
    grid_wait();
    grid_release();
    for (int o = int(blockIdx.x); o < p.out_features; o += int(gridDim.x))
        for (int i = int(threadIdx.x); i < p.in_features; i += kThreads)
            put_grad(p, int64_t(o) * p.dw_stride + i, 0.0f);
}

// A [rows, width] tensor read in boxes of `box` elements by kTokens rows.
cudaError_t encode(CUtensorMap* map, CUtensorMapDataType type, int64_t size, const void* p,
                   int64_t stride, int64_t rows, int64_t width, int box,
                   CUtensorMapSwizzle swizzle) {
    const int64_t dims[2] = {width, rows}, strides[1] = {stride * size};
    const int boxes[2] = {box, kTokens};
    return encode_tensor_map(map, type, p, 2, dims, strides, boxes, swizzle);
}

struct Plan {
    int out_tiles, in_tiles, blocks;
    int waves, rest_tiles;
    int64_t rest_chunk;
    bool join;
    bool copy_dy, copy_x;            // repacked for TMA
    int64_t partial_bytes, dy_bytes, code_bytes, step_bytes;
};

constexpr int kPairs = 76;           // of a GB300's 152 SMs

// Can TMA read these rows where they are?
bool tma_rows(const void* p, int64_t stride, int64_t size, int64_t width) {
    return aligned(p, 16) && stride >= width && stride * size % 16 == 0;
}

Plan make_plan(const void* dy, int64_t dy_stride, const dpr_checkpoint* x, int64_t rows,
               int64_t out_features, int64_t in_features) {
    Plan q = {};
    if (rows <= kFew) return q;
    q.out_tiles = int(ceil_div(out_features, kTile));
    q.in_tiles = int(ceil_div(in_features, kTile));
    q.blocks = int(ceil_div(rows, kTokens));
    const int64_t tiles = int64_t(q.out_tiles) * q.in_tiles;
    q.waves = int(tiles / kPairs);
    q.rest_tiles = int(tiles % kPairs);
    // steps of the tiles left over, dealt out evenly; a part is at least 4 steps long
    const int64_t steps = int64_t(q.rest_tiles) * q.blocks;
    q.rest_chunk = std::min<int64_t>(q.blocks, std::max<int64_t>(ceil_div(steps, kPairs), 4));
    q.join = q.rest_tiles > 0 && q.rest_chunk < q.blocks;
    q.partial_bytes = q.join ? int64_t(2 * kPairs) * kTile * kTile * 4 : 0;
    q.copy_dy = !tma_rows(dy, dy_stride, 2, out_features);
    q.dy_bytes = q.copy_dy ? rows * round_up(out_features, 8) * 2 : 0;
    q.copy_x = !tma_rows(x->codes, x->code_stride, 1, in_features) ||
               !tma_rows(x->steps, x->step_stride, 1,
                         ceil_div(in_features, kBlockChannels));
    if (q.copy_x) {
        q.code_bytes = rows * round_up(in_features, 16);
        q.step_bytes = rows * round_up(ceil_div(in_features, kBlockChannels), 16);
    }
    return q;
}

dpr_status check_sizes(int64_t rows, int64_t out_features, int64_t in_features) {
    dpr_status st = check_matrix_size(rows, out_features);
    if (st == DPR_OK) st = check_matrix_size(rows, in_features);
    if (st != DPR_OK) return st;
    if (rows > DPR_MAX_GRAD_ROWS) return DPR_ERR_UNSUPPORTED;
    // tiles are counted in 31 bits
    if (ceil_div(out_features, kTile) * ceil_div(in_features, kTile) > (int64_t(1) << 30))
        return DPR_ERR_UNSUPPORTED;
    return DPR_OK;
}

template <typename T>
cudaError_t repack(const void* from, int64_t from_stride, void* to, int64_t to_stride, int64_t rows,
                   int width, cudaStream_t s) {
    const T* f = static_cast<const T*>(from);
    T* t = static_cast<T*>(to);
    void* args[] = {&f, &from_stride, &t, &to_stride, &rows, &width};
    return launch_grid((const void*)repack_rows<T>, dim3(unsigned(std::min<int64_t>(rows, 152 * 16))),
                       dim3(kThreads), 0, args, s);
}

}  // namespace
}  // namespace dpr

using namespace dpr;

extern "C" {

dpr_status dpr_linear_weight_grad_workspace(const void* dy, int64_t dy_stride,
                                            const dpr_checkpoint* x_ckpt, int64_t rows,
                                            int64_t out_features, int64_t in_features,
                                            int64_t* bytes) {
    if (!bytes) return DPR_ERR_INVALID_ARG;
    *bytes = 0;
    const dpr_status st = check_sizes(rows, out_features, in_features);
    if (st != DPR_OK || rows == 0) return st;
    if (!x_ckpt) return DPR_ERR_INVALID_ARG;
    const Plan q = make_plan(dy, dy_stride, x_ckpt, rows, out_features, in_features);
    *bytes = q.partial_bytes + round_up(q.dy_bytes, 16) + round_up(q.code_bytes, 16) + q.step_bytes;
    return DPR_OK;
}

dpr_status dpr_linear_weight_grad(const void* dy, int64_t dy_stride, const dpr_checkpoint* x_ckpt,
                                  int64_t rows, int64_t out_features, int64_t in_features,
                                  void* dweight, int64_t dweight_stride, int dtype, int accumulate,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
    int64_t need = 0;
    dpr_status st = dpr_linear_weight_grad_workspace(dy, dy_stride, x_ckpt, rows, out_features,
                                                     in_features, &need);
    if (st != DPR_OK) return st;
    if (!dtype_ok(dtype)) return DPR_ERR_INVALID_ARG;
    if ((st = check_matrix(dweight, dweight_stride, in_features, dtype, true)) != DPR_OK) return st;
    SpanList outs, ins;
    outs.add(dweight, matrix_bytes(out_features, in_features, dweight_stride, dtype_size(dtype)));
    if (rows > 0) {
        if ((st = check_matrix(dy, dy_stride, out_features, DPR_BF16, false)) != DPR_OK) return st;
        if ((st = check_checkpoint(x_ckpt, in_features)) != DPR_OK) return st;
        if (need > 0) {
            if (!workspace || workspace_bytes < need) return DPR_ERR_INVALID_ARG;
            if (!aligned(workspace, 16)) return DPR_ERR_ALIGNMENT;
            outs.add(workspace, uint64_t(need));
        }
        ins.add(dy, matrix_bytes(rows, out_features, dy_stride, 2));
        ins.add(*x_ckpt, rows, in_features);
    }
    if (!outs.disjoint() || outs.meets(ins)) return DPR_ERR_ALIAS;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    WeightGradParams p = {};
    p.out_features = int(out_features); p.in_features = int(in_features);
    p.dw = dweight; p.dw_stride = dweight_stride;
    p.dw_bf16 = dtype == DPR_BF16; p.accumulate = accumulate != 0;
    if (rows == 0) {
        if (accumulate) return DPR_OK;
        void* args[] = {&p};
        return record_cuda_status(launch_grid((const void*)zero_rows,
                                              dim3(unsigned(std::min<int64_t>(out_features, 1 << 16))),
                                              dim3(kThreads), 0, args, s));
    }

    if (rows <= kFew) {
        const uint16_t* d = static_cast<const uint16_t*>(dy);
        dpr_checkpoint x = *x_ckpt;
        int tokens = int(rows);
        void* args[] = {&p, &d, &dy_stride, &x, &tokens};
        return record_cuda_status(launch_grid(
            (const void*)weight_grad_few,
            dim3(unsigned(ceil_div(in_features, 4 * kFewThreads)),
                 unsigned(ceil_div(out_features, kFewOut))),
            dim3(kFewThreads), 0, args, s));
    }
    const Plan q = make_plan(dy, dy_stride, x_ckpt, rows, out_features, in_features);
    p.out_tiles = q.out_tiles; p.in_tiles = q.in_tiles; p.blocks = q.blocks;
    p.waves = q.waves; p.rest_tiles = q.rest_tiles; p.rest_chunk = q.rest_chunk;
    char* ws = static_cast<char*>(workspace);
    p.partial = reinterpret_cast<float*>(ws);
    ws += q.partial_bytes;
    dpr_checkpoint x = *x_ckpt;
    cudaError_t e = cudaSuccess;
    if (q.copy_dy) {
        const int64_t stride = round_up(out_features, 8);
        e = repack<uint16_t>(dy, dy_stride, ws, stride, rows, int(out_features), s);
        dy = ws; dy_stride = stride;
        ws += round_up(q.dy_bytes, 16);
    }
    if (q.copy_x && e == cudaSuccess) {
        const int64_t blocks = ceil_div(in_features, kBlockChannels);
        const int64_t cs = round_up(in_features, 16), ss = round_up(blocks, 16);
        e = repack<uint8_t>(x.codes, x.code_stride, ws, cs, rows, int(in_features), s);
        x.codes = reinterpret_cast<int8_t*>(ws); x.code_stride = cs;
        ws += round_up(q.code_bytes, 16);
        if (e == cudaSuccess)
            e = repack<uint8_t>(x.steps, x.step_stride, ws, ss, rows, int(blocks), s);
        x.steps = reinterpret_cast<uint8_t*>(ws); x.step_stride = ss;
    }
    if (e == cudaSuccess)
        e = encode(&p.dy, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dy, dy_stride, rows, out_features,
                   64, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = encode(&p.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, x.codes, x.code_stride, rows,
                   in_features, 64, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e == cudaSuccess)
        e = encode(&p.steps, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, x.steps, x.step_stride, rows,
                   ceil_div(in_features, kBlockChannels), 16, CU_TENSOR_MAP_SWIZZLE_NONE);
    static std::atomic<uint64_t> allowed{0};
    if (e == cudaSuccess)
        e = allow_shared_memory((const void*)weight_grad_pairs, kSmemBytes, &allowed);
    if (e != cudaSuccess) return record_cuda_status(e);
    void* args[] = {&p};
    // pairs without work are not launched, unless whole waves need all of them
    const int64_t busy = q.waves > 0 ? kPairs
                                     : ceil_div(int64_t(q.rest_tiles) * q.blocks, q.rest_chunk);
    e = launch_grid((const void*)weight_grad_pairs, dim3(unsigned(2 * busy)), dim3(kGradThreads),
                    kSmemBytes, args, s);
    if (e == cudaSuccess && q.join) {
        int pairs = int(busy);
        void* jargs[] = {&p, &pairs};
        e = launch_grid((const void*)weight_grad_join,
                        dim3(unsigned(q.rest_tiles), kTile / kJoinRows), dim3(kJoinThreads), 0,
                        jargs, s);
    }
    return record_cuda_status(e);
}

dpr_status dpr_device_wait_failures(uint32_t* count) {
    if (!count) return DPR_ERR_INVALID_ARG;
    unsigned int v = 0, w = 0, r = 0, g = 0;
    cudaError_t e = cudaDeviceSynchronize();   // a copy alone does not wait for non-blocking streams
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_wait_failures, sizeof(v));
    if (e == cudaSuccess) e = norm_wait_failures(&w);
    if (e == cudaSuccess) e = rms_wait_failures(&r);
    if (e == cudaSuccess) e = grouped_wait_failures(&g);
    *count = v + w + r + g;
    return record_cuda_status(e);
}

}  // extern "C"
