// Device helpers of the row-wise operators (norm, routing): loads and stores
// of 8 consecutive elements at any element alignment, sums and maxima over the
// lanes that share a row, and the nearest-even MX block encoder.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

// ---------------------------------------------------------------- 8 elements
// A row of a caller's matrix starts at any multiple of its element size (odd
// widths, strides and offsets), so the 16-byte accesses carry only that
// alignment; gfx950 serves them at full width wherever they start.
typedef uint32_t u4_align2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f4_align4 __attribute__((ext_vector_type(4), aligned(4)));

// Elements p[0 .. min(n, 8) - 1] as binary32, zero beyond (n >= 1).
__device__ __forceinline__ void load_upto8(const uint16_t* p, int64_t n, float v[8]) {
    if (n >= 8) {
        const u4_align2 q = *reinterpret_cast<const u4_align2*>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(q[j] << 16);
            v[2 * j + 1] = __uint_as_float(q[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? __uint_as_float((uint32_t)p[j] << 16) : 0.0f;
    }
}

__device__ __forceinline__ void load_upto8(const float* p, int64_t n, float v[8]) {
    if (n >= 8) {
        const f4_align4 a = *reinterpret_cast<const f4_align4*>(p);
        const f4_align4 b = *reinterpret_cast<const f4_align4*>(p + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j < n ? p[j] : 0.0f;
    }
}

// Store min(n, 8) elements (BF16: one nearest-even rounding).
__device__ __forceinline__ void store_upto8(uint16_t* p, int64_t n, const float v[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
    if (n >= 8) {
        u4_align2 q = {w[0], w[1], w[2], w[3]};
        *reinterpret_cast<u4_align2*>(p) = q;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    }
}

__device__ __forceinline__ void store_upto8(float* p, int64_t n, const float v[8]) {
    if (n >= 8) {
        f4_align4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
        *reinterpret_cast<f4_align4*>(p) = a;
        *reinterpret_cast<f4_align4*>(p + 4) = b;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = v[j];
    }
}

// The value a store to T and a load back give.
template <typename T>
__device__ __forceinline__ float rounded_to(float v) {
    if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v) << 16);
    else return v;
}

// ---------------------------------------------------------------- row sums
// Reduction over an aligned group of 16 lanes, the result in every lane: two
// quad exchanges, then the mirror of each half row (lane i of 8 reads 7 - i:
// the other quad) and of the row (i of 16 reads 15 - i: the other half).  All
// 64 lanes must be active.
template <typename Op>
__device__ __forceinline__ float reduce16(float x, Op op) {
    x = op(x, lane_xor1(x));
    x = op(x, lane_xor2(x));
    x = op(x, quad_perm<0x141>(x));
    x = op(x, quad_perm<0x140>(x));
    return x;
}

// The value of the other one of a pair of rows of 16 (halves of 32) and the
// own one, in either order: exchanged between registers, without LDS.
__device__ __forceinline__ void row_pair(float x, float& a, float& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    a = __uint_as_float(r[0]);
    b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void half_pair(float x, float& a, float& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    a = __uint_as_float(r[0]);
    b = __uint_as_float(r[1]);
}

// As reduce16 over the 64 lanes of the wave.
template <typename Op>
__device__ __forceinline__ float reduce64(float x, Op op) {
    float a, b;
    row_pair(reduce16(x, op), a, b);
    half_pair(op(a, b), a, b);
    return op(a, b);
}

struct AddOp {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct MaxOp {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// A barrier of the workgroup for what lies in LDS alone: loads from memory
// that are under way stay so.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Sum over the TPR threads (16, 64, or whole workgroup of TPR threads) that
// share a row, in a fixed order, the result in every thread.  lds: TPR / 64
// floats that no other use of the current phase touches (TPR > 64); a second
// call must use other floats or follow a barrier.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* lds) {
    if constexpr (TPR == 16) return reduce16(x, AddOp());
    x = reduce64(x, AddOp());
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
        lds_barrier();
        x = 0.0f;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) x += lds[w];
    }
    return x;
}

// A binary64 value of another lane, by the same exchanges of its two words.
template <int CTRL>
__device__ __forceinline__ double quad_perm64(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    return __longlong_as_double((long long)((uint64_t)quad_perm<CTRL>((uint32_t)(b >> 32)) << 32 | quad_perm<CTRL>((uint32_t)b)));
}

// row_sum in binary64.
template <int TPR>
__device__ __forceinline__ double row_sum64(double x, double* lds) {
    x += quad_perm64<0xB1>(x);
    x += quad_perm64<0x4E>(x);
    x += quad_perm64<0x141>(x);
    x += quad_perm64<0x140>(x);
    if constexpr (TPR > 16) {
        const uint64_t b = (uint64_t)__double_as_longlong(x);
        auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
        auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false);
        x = __longlong_as_double((long long)((uint64_t)hi[0] << 32 | lo[0])) +
            __longlong_as_double((long long)((uint64_t)hi[1] << 32 | lo[1]));
        const uint64_t c = (uint64_t)__double_as_longlong(x);
        hi = __builtin_amdgcn_permlane32_swap((uint32_t)(c >> 32), (uint32_t)(c >> 32), false, false);
        lo = __builtin_amdgcn_permlane32_swap((uint32_t)c, (uint32_t)c, false, false);
        x = __longlong_as_double((long long)((uint64_t)hi[0] << 32 | lo[0])) +
            __longlong_as_double((long long)((uint64_t)hi[1] << 32 | lo[1]));
    }
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
        lds_barrier();
        x = 0.0;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) x += lds[w];
    }
    return x;
}

// ---------------------------------------------------------------- MX blocks
// Nearest-even MX codes of a lane's 8 consecutive elements, four lanes holding
// one 32-element block, and the block's scale byte (rules of include/nvfp4.h:
// s = floor(log2 amax) - emax clamped to [-127, 127], -127 for a zero block;
// y = v * 2^-s saturating at the largest element).  w: 2 words for E4M3, 1 for
// E2M1.
template <int ELEM>
__device__ __forceinline__ uint32_t mx_block_rne8(const float v[8], uint32_t w[2]) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
    m = fmaxf(m, lane_xor1(m));
    m = fmaxf(m, lane_xor2(m));
    constexpr int emax = ELEM == kMxE4M3 ? 8 : 2;
    // a normal amax has floor(log2) = exponent field - 127; a zero or
    // subnormal one (field 0) falls below the clamp
    const int s = max((int)(__float_as_uint(m) >> 23) - 127 - emax, -127);
    const float p2 = __uint_as_float((uint32_t)(127 - s) << 23);  // 2^-s, always normal
    if constexpr (ELEM == kMxE4M3) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = __builtin_amdgcn_fmed3f(v[4 * k + j] * p2, -448.0f, 448.0f);
            const uint32_t lo = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
            const uint32_t hi = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], 0, false);
            w[k] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);  // low halves of lo, then hi
        }
    } else {
        BlockScale bs;
        bs.byte = 0u;
        bs.R = p2;
        encode<false, 8>(v, bs, m, nullptr, w);
    }
    return (uint32_t)(s + 127);
}

}  // namespace nvfp4
