// Device-side helpers of the backward-pass operators: V-element accesses of
// bf16 and fp32 rows, sums over the threads that share a row, and the 8-bit
// checkpoint format (see dpr_checkpoint in dpr_ops.h).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "dpr_device.cuh"

namespace dpr {

constexpr int kBlockChannels = 32;   // channels that share a step

// --- two fp32 numbers per instruction (sm_100 and later) -----------------------
// Each half is rounded as the single operation is.

struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void halves(F2 p, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float total(F2 p) {
    float a, b;
    halves(p, a, b);
    return __fadd_rn(a, b);
}

// --- V consecutive elements of a row ----------------------------------------
// T is uint16_t (bf16 bits) or float.  V = 16 (bf16) and V = 8 (fp32) are
// 32-byte accesses, V = 8 (bf16) 16-byte ones, V = 1 single elements.

template <typename T, int V>
struct Raw {
    static constexpr int kWords = V * int(sizeof(T)) < 4 ? 1 : V * int(sizeof(T)) / 4;
    uint32_t w[kWords];
};

template <typename T, int V>
__device__ __forceinline__ void load_raw(const T* p, Raw<T, V>& r) {
    static_assert(V == 1 || r.kWords == 4 || r.kWords == 8, "16- or 32-byte accesses");
    if constexpr (V == 1) {
        if constexpr (sizeof(T) == 2) {
            uint16_t h;
            asm volatile("ld.global.u16 %0, [%1];" : "=h"(h) : "l"(p));
            r.w[0] = h;
        } else {
            asm volatile("ld.global.u32 %0, [%1];" : "=r"(r.w[0]) : "l"(p));
        }
    } else if constexpr (Raw<T, V>::kWords == 8) {
        ld_v8(p, r.w);
    } else {
        const uint4 v = ld_v4(p);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    }
}

template <typename T, int V>
__device__ __forceinline__ void zero_raw(Raw<T, V>& r) {
#pragma unroll
    for (int i = 0; i < Raw<T, V>::kWords; ++i) r.w[i] = 0;
}

template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& r, float (&f)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = __uint_as_float(r.w[i]);
    } else if constexpr (V == 1) {
        f[0] = bf_lo(r.w[0]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            f[2 * i] = bf_lo(r.w[i]);
            f[2 * i + 1] = bf_hi(r.w[i]);
        }
    }
}

// fp32 -> T, rounded to nearest even (identity for fp32).
template <typename T, int V>
__device__ __forceinline__ void pack(const float (&f)[V], Raw<T, V>& r) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) r.w[i] = __float_as_uint(f[i]);
    } else if constexpr (V == 1) {
        r.w[0] = to_bf16(f[0]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) r.w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_raw(T* p, const Raw<T, V>& r) {
    if constexpr (V == 1) {
        if constexpr (sizeof(T) == 2) *p = T(r.w[0]);
        else *reinterpret_cast<uint32_t*>(p) = r.w[0];
    } else if constexpr (Raw<T, V>::kWords == 8) {
        st_v8(p, r.w);
    } else {
        st_v4(p, make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]));
    }
}

// V elements as pairs.
template <typename T, int V>
__device__ __forceinline__ void unpack2(const Raw<T, V>& r, F2 (&f)[V / 2]) {
    float v[V];
    unpack(r, v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f[i] = f2(v[2 * i], v[2 * i + 1]);
}
template <typename T, int V>
__device__ __forceinline__ void pack2(const F2 (&f)[V / 2], Raw<T, V>& r) {
    float v[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) halves(f[i], v[2 * i], v[2 * i + 1]);
    pack(v, r);
}

// V parameter values (weight, bias), bf16 or fp32 by `is_bf16`; `vec`: how many
// bytes an access may take (32, 16 or one element).  32-byte accesses matter
// although the values come from L1: two 16-byte ones touch every sector twice.
// Volatile, so that none moves above the wait for the grid before.
__device__ __forceinline__ void ld_v8_cached(const void* p, uint32_t (&w)[8]) {
    asm volatile("ld.global.v8.u32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
          "=r"(w[7])
        : "l"(p));
}
template <int V>
__device__ __forceinline__ void load_params(const void* p, bool is_bf16, int vec, int64_t at,
                                            float (&f)[V]) {
    if (is_bf16) {
        const uint16_t* q = static_cast<const uint16_t*>(p) + at;
        if (V == 16 && vec == 32) {
            uint32_t w[8];
            ld_v8_cached(q, w);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                f[2 * i] = bf_lo(w[i & 7]);
                f[2 * i + 1] = bf_hi(w[i & 7]);
            }
        } else if (V >= 8 && vec >= 16) {
#pragma unroll
            for (int i = 0; i < V / 8; ++i) {
                const uint4 v = *reinterpret_cast<const uint4*>(q + 8 * i);
                f[8 * i + 0] = bf_lo(v.x); f[8 * i + 1] = bf_hi(v.x);
                f[8 * i + 2] = bf_lo(v.y); f[8 * i + 3] = bf_hi(v.y);
                f[8 * i + 4] = bf_lo(v.z); f[8 * i + 5] = bf_hi(v.z);
                f[8 * i + 6] = bf_lo(v.w); f[8 * i + 7] = bf_hi(v.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = bf_1(q[i]);
        }
    } else {
        const float* q = static_cast<const float*>(p) + at;
        if (V >= 8 && vec == 32) {
#pragma unroll
            for (int i = 0; i < V / 8; ++i) {
                uint32_t w[8];
                ld_v8_cached(q + 8 * i, w);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[8 * i + k] = __uint_as_float(w[k]);
            }
        } else if (V >= 4 && vec >= 16) {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const float4 v = *reinterpret_cast<const float4*>(q + 4 * i);
                f[4 * i + 0] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = q[i];
        }
    }
}

// First channel of the i-th of a thread's NV vectors: vectors of a row are
// dealt out thread by thread; single elements warp by warp, 32 NV channels
// each (blockDim.x a multiple of 32), which puts a thread's elements at fixed
// distances.  Either way the threads of a block of channels are neighbours.
template <int V, int NV>
__device__ __forceinline__ int own_channel(int i) {
    const int tx = int(threadIdx.x);
    if constexpr (V == 1) return (tx >> 5) * (32 * NV) + i * 32 + (tx & 31);
    else return (i * int(blockDim.x) + tx) * V;
}

// --- sums over the threads of a row -------------------------------------------

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

// Sum over each aligned group of `n` (a power of two) lanes.
__device__ __forceinline__ float group_sum(float v, int n) {
    for (int d = n >> 1; d > 0; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

__device__ __forceinline__ float group_sum8(float v) {
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

// The smallest power of two that is at least n (n = 1 .. 32).
__device__ __forceinline__ int power_of_two(int n) { return n <= 1 ? 1 : 2 << (31 - __clz(n - 1)); }

// Barrier of the blockDim.x (a multiple of 32) threads that share threadIdx.y;
// at most 15 of them.
__device__ __forceinline__ void row_barrier() {
    if (blockDim.y == 1) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(blockDim.x) : "memory");
}

// Sum of `v` over the blockDim.x threads that share threadIdx.y (a power of
// two below 32, or a multiple of 32 up to 1024); every one of them gets it.
// `s` has one row of 32 floats per threadIdx.y where that is a multiple.
// All of them call it.  Two calls in a row need different `s` (one barrier,
// none behind the reads).
__device__ __forceinline__ float row_sum(float v, float (*s)[32]) {
    if (blockDim.x < 32) return group_sum(v, int(blockDim.x));
    v = warp_sum(v);
    if (blockDim.x == 32) return v;
    const int nw = int(blockDim.x) >> 5, n = power_of_two(nw);
    const int lane = int(threadIdx.x) & 31, at = lane & (n - 1);
    if (lane == 0) s[threadIdx.y][threadIdx.x >> 5] = v;
    row_barrier();
    return group_sum(at < nw ? s[threadIdx.y][at] : 0.0f, n);
}

// The same for two sums at once.
__device__ __forceinline__ void row_sums(float& a, float& b, float2 (*s)[32]) {
    if (blockDim.x < 32) {
        a = group_sum(a, int(blockDim.x));
        b = group_sum(b, int(blockDim.x));
        return;
    }
    a = warp_sum(a);
    b = warp_sum(b);
    if (blockDim.x == 32) return;
    const int nw = int(blockDim.x) >> 5, n = power_of_two(nw);
    const int lane = int(threadIdx.x) & 31, at = lane & (n - 1);
    if (lane == 0) s[threadIdx.y][threadIdx.x >> 5] = make_float2(a, b);
    row_barrier();
    const float2 v = at < nw ? s[threadIdx.y][at] : make_float2(0.0f, 0.0f);
    a = group_sum(v.x, n);
    b = group_sum(v.y, n);
}

// 1 / sqrt(v) for v >= 0, all but correctly rounded: the hardware's
// approximation r, corrected by r (1 - v r^2) / 2 with the residual taken
// exactly to first order.  A relative error of rstd scales its whole row, and
// in fp32 turns codes of the row's checkpoint over, so the last bit counts.
// (0 gives infinity.)
__device__ __forceinline__ float inverse_sqrt(float v) {
    const float r = rsqrtf(v);
    const float h = __fmul_rn(v, r), low = __fmaf_rn(v, r, -h);
    const float e = __fmaf_rn(-low, r, __fmaf_rn(-h, r, 1.0f));
    const float better = __fmaf_rn(__fmul_rn(0.5f, r), e, r);
    return v > 1e-30f && v < 1e30f ? better : __fdiv_rn(1.0f, __fsqrt_rn(v));
}

// s / n, all but correctly rounded: the product with the rounded reciprocal,
// corrected by its remainder.
__device__ __forceinline__ float divide(float s, float n, float inverse) {
    const float q = __fmul_rn(s, inverse);
    const float better = __fmaf_rn(__fmaf_rn(-q, n, s), inverse, q);
    return fabsf(s) < 1e30f ? better : q;   // the remainder of a huge or infinite s is none
}

// --- the 8-bit format -----------------------------------------------------------

// The step byte of a block whose largest |x| has these fp32 bits (integer
// order is magnitude order, infinities and NaN above the rest).  For a peak in
// [2^k, 2^(k+1)) the smallest step keeping peak / step below 127.5 is
// 2^(k-6), or 2^(k-5) when the mantissa puts the peak at 127.5 * 2^(k-6) or
// above; steps are kept in [2^-126, 2^121] (the byte in [1, 248]).
__device__ __forceinline__ uint32_t step_byte(uint32_t peak) {
    if (peak >= 0x7F800000u) return 255u;
    if (peak == 0) return 0u;
    int b = int((peak + 0x00010000u) >> 23) - 6;   // carries into the exponent from 127.5/128 up
    return uint32_t(min(max(b, 1), 248));   // kTopByte
}

__device__ __forceinline__ float step_value(uint32_t byte) { return __uint_as_float(byte << 23); }

// 1 / step for bytes 1 .. 248; of no use (finite) for 0 and 255.
__device__ __forceinline__ float step_inverse(uint32_t byte) {
    return __uint_as_float((254u - min(byte, 248u)) << 23);
}

// x / step rounded to the nearest integer (ties to even), as the low byte of
// the result: x * inverse is exact or far below 1/2, and adding 1.5 * 2^23
// rounds it (once: a fused multiply-add) to an integer whose two's complement
// is the sum's low bits.
constexpr float kRoundInteger = 12582912.0f;
constexpr uint32_t kTopByte = 248;   // the largest step: codes may need limiting

// The low bytes of four such numbers.
__device__ __forceinline__ uint32_t pack_codes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The largest |x| of V elements, as fp32 bits.
template <typename T, int V>
__device__ __forceinline__ uint32_t peak_bits(const Raw<T, V>& r) {
    if constexpr (sizeof(T) == 4) {
        uint32_t peak = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) peak = max(peak, r.w[i] & 0x7FFFFFFFu);
        return peak;
    } else if constexpr (V == 1) {
        return (r.w[0] & 0x7FFFu) << 16;
    } else {
        uint32_t peak = 0;   // two bf16 magnitudes at a time
#pragma unroll
        for (int i = 0; i < V / 2; ++i) peak = __vmaxu2(peak, r.w[i] & 0x7FFF7FFFu);
        return max(peak << 16, peak & 0xFFFF0000u);
    }
}

// The code of x in a block with a step byte of kTopByte (limited to 127) or
// 255 (0), in the low byte.
__device__ __forceinline__ uint32_t encode_limited(float x, uint32_t byte) {
    const float top = __fmul_rn(127.0f, step_value(kTopByte));
    const float v = fminf(fmaxf(x, -top), top);
    const uint32_t q = __float_as_uint(__fmaf_rn(v, step_inverse(kTopByte), kRoundInteger));
    return byte == 255u ? 0u : q & 0xFFu;
}

// The code of one element in a block with this step byte, in the low byte.
template <typename T>
__device__ __forceinline__ uint32_t encode_one(const Raw<T, 1>& r, uint32_t byte) {
    float x[1];
    unpack(r, x);
    if (byte >= kTopByte) return encode_limited(x[0], byte);
    return __float_as_uint(__fmaf_rn(x[0], step_inverse(byte), kRoundInteger)) & 0xFFu;
}

// Saves V channels starting at channel c (a multiple of V) of one row, given
// as stored and as pairs.  The 32 / V threads of a block of channels are
// neighbouring lanes and all call it; channels at or past the row's end are
// zeros (`on` false: nothing stored).  `codes` and `steps` point at the row's
// start.
template <typename T, int V>
__device__ __forceinline__ void save_vector(const Raw<T, V>& raw, const F2 (&f)[V / 2], int c,
                                            bool on, int8_t* codes, uint8_t* steps) {
    uint32_t peak = peak_bits(raw);
#pragma unroll
    for (int d = 1; d < kBlockChannels / V; d <<= 1)
        peak = max(peak, __shfl_xor_sync(0xFFFFFFFFu, peak, d));
    const uint32_t byte = step_byte(peak);
    if (!on) return;
    uint32_t w[V / 4];
    if (byte < kTopByte) {
        const F2 inv = f2(step_inverse(byte)), round = f2(kRoundInteger);
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            float q[4];
            halves(fma2(f[2 * i], inv, round), q[0], q[1]);
            halves(fma2(f[2 * i + 1], inv, round), q[2], q[3]);
            w[i] = pack_codes(__float_as_uint(q[0]), __float_as_uint(q[1]), __float_as_uint(q[2]),
                              __float_as_uint(q[3]));
        }
    } else {   // numbers near the type's largest, or not finite
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            float x[4];
            halves(f[2 * i], x[0], x[1]);
            halves(f[2 * i + 1], x[2], x[3]);
            w[i] = pack_codes(encode_limited(x[0], byte), encode_limited(x[1], byte),
                              encode_limited(x[2], byte), encode_limited(x[3], byte));
        }
    }
    if constexpr (V == 16)
        st_v4(codes + c, make_uint4(w[0], w[1], w[2], w[3]));
    else
        *reinterpret_cast<uint2*>(codes + c) = make_uint2(w[0], w[1]);
    if ((c & (kBlockChannels - 1)) == 0) steps[c / kBlockChannels] = uint8_t(byte);
}

template <typename T, int V>
__device__ __forceinline__ void save_vector(const Raw<T, V>& raw, int c, bool on, int8_t* codes,
                                            uint8_t* steps) {
    F2 f[V / 2];
    unpack2(raw, f);
    save_vector(raw, f, c, on, codes, steps);
}

// Saves a thread's NV vectors of a row; nothing from `width` on.  Every thread calls it.
template <typename T, int V, int NV>
__device__ __forceinline__ void save_row(const Raw<T, V> (&raw)[NV], int width, int8_t* codes,
                                         uint8_t* steps) {
    if constexpr (V == 1) {
        // A warp's 32 lanes are a block of channels.  Lane i works out the step of
        // the warp's i-th block: every lane for all of them took 37 instructions
        // an element (16384 x 1001 bf16: 18 us).
        const int lane = int(threadIdx.x) & 31;
        uint32_t mine = 0, top = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t peak = __reduce_max_sync(0xFFFFFFFFu, peak_bits(raw[i]));
            if (lane == i) mine = peak;
            top = max(top, peak);
        }
        const uint32_t byte = step_byte(mine);
        const int first = own_channel<V, NV>(0) - lane;
        if (lane < NV && first + lane * kBlockChannels < width)
            steps[first / kBlockChannels + lane] = uint8_t(byte);
        if (step_byte(top) < kTopByte) {
            const float inv = step_inverse(byte);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = own_channel<V, NV>(i);
                float x[1];
                unpack(raw[i], x);
                const float q = __fmaf_rn(x[0], __shfl_sync(0xFFFFFFFFu, inv, i), kRoundInteger);
                if (c < width) codes[c] = int8_t(__float_as_uint(q));
            }
        } else {   // numbers near the type's largest, or not finite
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = own_channel<V, NV>(i);
                const uint32_t q = encode_one(raw[i], __shfl_sync(0xFFFFFFFFu, byte, i));
                if (c < width) codes[c] = int8_t(q);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = own_channel<V, NV>(i);
            save_vector(raw[i], c, c < width, codes, steps);
        }
    }
}

// Two codes, in the low bytes of the halves of `w`, as bf16: the seven low
// bits on top of 128, less 128 or (sign bit) 256, times the step.
__device__ __forceinline__ uint32_t restore_pair(uint32_t w, uint32_t step2) {
    const uint32_t low = (w & 0x007F007Fu) | 0x43004300u;
    const uint32_t base = (w & 0x00800080u) | 0x43004300u;
    uint32_t v, r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(low), "r"(base));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(step2));
    return r;
}

// V codes of a row.
template <int V>
struct CodeRaw {
    uint32_t w[V < 4 ? 1 : V / 4];
};

template <int V>
__device__ __forceinline__ void load_codes(const int8_t* p, CodeRaw<V>& r) {
    if constexpr (V == 1) {
        uint16_t h;
        asm volatile("ld.global.u8 %0, [%1];" : "=h"(h) : "l"(p));
        r.w[0] = h;
    } else if constexpr (V == 8) {
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                     : "=r"(r.w[0]), "=r"(r.w[1])
                     : "l"(p));
    } else {
        const uint4 v = ld_v4(p);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    }
}

// The codes as fp32 pairs: flipping a code's sign bit gives code + 128, which
// as the low byte of 2^23's bits is the float 2^23 + 128 + code.
template <int V>
__device__ __forceinline__ void codes2(const CodeRaw<V>& r, F2 (&f)[V / 2]) {
    float q[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        q[i] = __uint_as_float(__byte_perm(r.w[i / 4] ^ 0x80808080u, 0x4B000000u, 0x7650 + (i & 3)));
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f[i] = add2(f2(q[2 * i], q[2 * i + 1]), f2(-8388736.0f));
}
// code * step.
template <int V>
__device__ __forceinline__ void decode2(const CodeRaw<V>& r, float step, F2 (&f)[V / 2]) {
    codes2<V>(r, f);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f[i] = mul2(f[i], f2(step));
}
template <int V>
__device__ __forceinline__ void decode(const CodeRaw<V>& r, float step, float (&f)[V]) {
    if constexpr (V == 1) {
        const uint32_t bits = __byte_perm(r.w[0] ^ 0x80u, 0x4B000000u, 0x7650);
        f[0] = __fmul_rn(__fadd_rn(__uint_as_float(bits), -8388736.0f), step);
    } else {
        F2 p[V / 2];
        decode2<V>(r, step, p);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) halves(p[i], f[2 * i], f[2 * i + 1]);
    }
}

}  // namespace dpr
