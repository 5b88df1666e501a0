// Products of a few BF16 or binary32 rows with 4-bit weights, for gfx950:
//   y[m][n] = s_t sum_k x[m][k] v[n][k] S[n][k]
// with v the E2M1 elements and S the block scales (NVFP4: E4M3 per 16 elements
// of a row or per 16x16 square, s_t the tensor scale; MXFP4: 2^s per 32
// elements, s_t = 1), and its routed form, in which every assignment of a
// token to an expert takes that expert's matrix.
//
// An element times its block scale has at most 6 significant bits, so it is a
// BF16 value exactly and the BF16 matrix cores form exact products with BF16
// x, summed in binary32.  A binary32 x is the exact sum of three BF16 values
// (its upper, middle and lower 8 significant bits), whose products go to the
// same accumulators.  One 16x16x32 MFMA then serves up to 16 rows of x at the
// cost of one, which is what bounds these products: the weights' bytes.
//
// A wave holds R tiles of 16 weight rows.  Lane l has weight row l % 16 (the
// MFMA's A operand) and x row l / 16's column of the B operand; group g = l / 16
// of a step of 128 k takes the 32 consecutive k from 32 g: 16 bytes of codes,
// its two (MX: one) scales, 32 elements of x, and four MFMAs.  The order of k
// inside an MFMA is the same for both operands and otherwise free.  The W
// waves of a workgroup take the steps in turn, so that together they stream
// whole rows, and their sums are added through LDS in a fixed order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch.hpp"
#include "nvfp4_device.hpp"
#include "row_device.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 v8b_t __attribute__((ext_vector_type(8)));
typedef __bf16 v2b_t __attribute__((ext_vector_type(2)));
typedef float v4f_t __attribute__((ext_vector_type(4)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
// codes start at any multiple of 8 bytes (a row of K / 2 bytes, K % 16 == 0)
typedef uint32_t u4_align8 __attribute__((ext_vector_type(4), aligned(8)));
typedef uint32_t u2_align8 __attribute__((ext_vector_type(2), aligned(8)));

enum { kFmtNv1D = 0, kFmtNv2D = 1, kFmtMx = 2 };

constexpr int kCols = 16;    // rows of x (MFMA columns) of one pass
constexpr int kStep = 128;   // k of one step

// Four E2M1 pairs (one dword) as 8 BF16 values times the scale s.
template <int FMT>
__device__ __forceinline__ v8b_t weights8(uint32_t w, float s) {
    u4_t r;
    if constexpr (FMT == kFmtMx) {  // a power of two: the convert's own scale operand
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = e2m1x2_unpack(w, j);  // times s: exact, the low half of the result zero
            r[j] = __builtin_amdgcn_perm(__float_as_uint(v.y * s), __float_as_uint(v.x * s), 0x07060302u);
        }
    }
    return __builtin_bit_cast(v8b_t, r);
}

// The upper halves of 8 binary32 values.
__device__ __forceinline__ v8b_t upper8(const float v[8]) {
    u4_t r;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        r[j] = __builtin_amdgcn_perm(__float_as_uint(v[2 * j + 1]), __float_as_uint(v[2 * j]), 0x07060302u);
    return __builtin_bit_cast(v8b_t, r);
}

__device__ __forceinline__ v4f_t mfma(v8b_t a, v8b_t b, v4f_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// One lane's share of a step: codes and scale bytes of its R weight rows and
// 32 elements of its x row.
template <bool XF32, int R>
struct Step {
    u4_t w[R];
    uint32_t s[R];
    u4_t x[XF32 ? 8 : 4];
};

// Where a lane reads: its R weight rows and its x row.
template <int R>
struct Lane {
    const uint8_t* codes[R];
    const uint8_t* scales[R];
    const void* x;
};

// The lane's share at k (n = K - k left of the row, >= 32; or 16, and the
// upper half is zero; or nothing).
template <int FMT, bool XF32, int R, bool TAIL>
__device__ __forceinline__ void load_step(const Lane<R>& a, int64_t k, int64_t n, Step<XF32, R>& st) {
    if constexpr (TAIL) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            st.w[i] = u4_t{0, 0, 0, 0};
            st.s[i] = 0;
        }
#pragma unroll
        for (int j = 0; j < (XF32 ? 8 : 4); ++j) st.x[j] = u4_t{0, 0, 0, 0};
        if (n <= 0) return;
    }
    const bool whole = !TAIL || n >= 32;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (whole) {
            st.w[i] = *reinterpret_cast<const u4_align8*>(a.codes[i] + k / 2);
        } else {
            const u2_align8 h = *reinterpret_cast<const u2_align8*>(a.codes[i] + k / 2);
            st.w[i][0] = h[0];
            st.w[i][1] = h[1];
        }
        if constexpr (FMT == kFmtMx) {
            st.s[i] = a.scales[i][k / 32];
        } else {
            st.s[i] = a.scales[i][k / 16];
            if (whole) st.s[i] |= (uint32_t)a.scales[i][k / 16 + 1] << 8;
        }
    }
    constexpr int per16 = XF32 ? 4 : 2;  // 16-byte pieces of 16 elements
#pragma unroll
    for (int j = 0; j < 2 * per16; ++j) {
        if (!whole && j >= per16) break;
        if constexpr (XF32)
            st.x[j] = __builtin_bit_cast(u4_t, *reinterpret_cast<const f4_align4*>(static_cast<const float*>(a.x) + k + 4 * j));
        else
            st.x[j] = *reinterpret_cast<const u4_align2*>(static_cast<const uint16_t*>(a.x) + k + 8 * j);
    }
}

template <int FMT, bool XF32, int R>
__device__ __forceinline__ void add_step(const Step<XF32, R>& st, v4f_t acc[R]) {
    float s[R][2];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if constexpr (FMT == kFmtMx) {
            s[i][0] = s[i][1] = __uint_as_float(st.s[i] << 23);
        } else {
            s[i][0] = __builtin_amdgcn_cvt_f32_fp8((int)st.s[i], 0);
            s[i][1] = __builtin_amdgcn_cvt_f32_fp8((int)st.s[i], 1);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (XF32) {
            float v[8], mid[8], low[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = __uint_as_float(st.x[2 * j + e / 4][e % 4]);
                mid[e] = v[e] - __uint_as_float(__float_as_uint(v[e]) & 0xFFFF0000u);
                low[e] = mid[e] - __uint_as_float(__float_as_uint(mid[e]) & 0xFFFF0000u);
            }
            const v8b_t b0 = upper8(v), b1 = upper8(mid), b2 = upper8(low);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const v8b_t a = weights8<FMT>(st.w[i][j], s[i][j >> 1]);
                acc[i] = mfma(a, b2, acc[i]);
                acc[i] = mfma(a, b1, acc[i]);
                acc[i] = mfma(a, b0, acc[i]);
            }
        } else {
            const v8b_t b = __builtin_bit_cast(v8b_t, st.x[j]);
#pragma unroll
            for (int i = 0; i < R; ++i) acc[i] = mfma(weights8<FMT>(st.w[i][j], s[i][j >> 1]), b, acc[i]);
        }
    }
}

// acc += the calling wave's steps (wave, wave + waves, ...) of rows of K.
template <int FMT, bool XF32, int R>
__device__ __forceinline__ void multiply(const Lane<R>& a, int64_t K, int wave, int waves, v4f_t acc[R]) {
    const int64_t full = K / kStep;
    const int k0 = 32 * ((threadIdx.x & 63) >> 4);
    for (int64_t t = wave; t < full; t += waves) {
        Step<XF32, R> st;
        load_step<FMT, XF32, R, false>(a, t * kStep + k0, 32, st);
        add_step<FMT, XF32, R>(st, acc);
    }
    if (K % kStep && full % waves == wave) {
        Step<XF32, R> st;
        const int64_t k = full * kStep + k0;
        load_step<FMT, XF32, R, true>(a, k, K - k, st);
        add_step<FMT, XF32, R>(st, acc);
    }
}

// gate sigmoid(gate) up.  With e = exp(-|gate|), sigmoid is 1 / (1 + e) or
// e / (1 + e); e goes in by its square root, once with each factor, so that
// nothing underflows or overflows before the result does.
__device__ __forceinline__ float swiglu32(float gate, float up) {
    const float root = expf(-0.5f * fabsf(gate)), tail = gate < 0.0f ? root : 1.0f;
    return (gate * tail) / (1.0f + root * root) * (up * tail);
}

__device__ __forceinline__ void store1(void* y, bool bf16, int64_t i, float v) {
    if (bf16) static_cast<uint16_t*>(y)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
    else static_cast<float*>(y)[i] = v;
}

// Workgroup (tile group blockIdx.x, blockIdx.y): R tiles of 16 weight rows
// against up to 16 rows of x: rows 16 blockIdx.y and on, or (EXPERT) those of
// all assignments that share the expert of assignment blockIdx.y, which is the
// first of them (other workgroups end at once).  SWIGLU: half of the tiles are
// gate rows, the others the up rows F further on.
template <int FMT, bool XF32, int R, bool SWIGLU, bool EXPERT>
__global__ void __launch_bounds__(512) k_gemv(const GemvArgs p) {
    constexpr int G = SWIGLU ? R / 2 : R;         // tiles of output columns
    constexpr int LDR = R * 16 + 4;               // floats of one x row's sums
    __shared__ __attribute__((aligned(16))) float sums[8 * kCols * LDR];
    __shared__ int list[EXPERT ? kMaxGemvAssignments : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int64_t outs = SWIGLU ? p.N / 2 : p.N, n0 = (int64_t)blockIdx.x * (16 * G);

    int64_t wrow0 = 0;  // first row of the matrix in the stack
    int columns;
    float ts = 1.0f;
    if constexpr (EXPERT) {
        const int first = blockIdx.y, id = p.ids[first];
        if (id < 0 || id >= p.experts) {  // no expert: its output is zero
            for (int o = threadIdx.x; o < 16 * G; o += blockDim.x)
                if (n0 + o < outs) store1(p.y, p.y_bf16, (int64_t)first * p.ldy + n0 + o, 0.0f);
            return;
        }
        columns = 0;
        for (int b = 0; b < p.assignments; b += 64) {
            const int a = b + lane;
            const bool same = a < p.assignments && p.ids[a] == id;
            const uint64_t m = __ballot(same);
            if (a < first && same) columns = -1;  // (an earlier one has them)
            if (__any(columns < 0)) return;       // the same in every wave
            if (wave == 0 && same) list[columns + __popcll(m & ((1ull << lane) - 1))] = a;
            columns += __popcll(m);
        }
        __syncthreads();
        wrow0 = (int64_t)id * p.N;
        ts = p.ts[id];
    } else {
        columns = (int)min((int64_t)kCols, p.m - (int64_t)blockIdx.y * kCols);
        if (p.ts) ts = p.ts[0];
    }

    Lane<R> a;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        // rows past the end repeat the last one; their sums are not stored
        const int64_t o = min(n0 + 16 * (i % G) + (lane & 15), outs - 1);
        const int64_t r = wrow0 + (i < G ? 0 : outs) + o;
        a.codes[i] = p.codes + r * (p.K / 2);
        a.scales[i] = p.scales + (FMT == kFmtNv2D ? (r / 16) * (p.K / 16) : r * (p.K / (FMT == kFmtMx ? 32 : 16)));
    }
    for (int c0 = 0; c0 < columns; c0 += kCols) {
        const int nc = min(columns - c0, kCols);
        // lanes past the last column repeat it; their sums are not stored
        const int c = min(lane & 15, nc - 1);
        const int64_t xr = EXPERT ? (p.x_per_assignment ? list[c0 + c] : list[c0 + c] / p.top_k)
                                  : (int64_t)blockIdx.y * kCols + c;
        a.x = XF32 ? static_cast<const void*>(static_cast<const float*>(p.x) + xr * p.ldx)
                   : static_cast<const void*>(static_cast<const uint16_t*>(p.x) + xr * p.ldx);
        v4f_t acc[R];
#pragma unroll
        for (int i = 0; i < R; ++i) acc[i] = v4f_t{0.0f, 0.0f, 0.0f, 0.0f};
        multiply<FMT, XF32, R>(a, p.K, wave, waves, acc);
        // accumulator r of lane l: weight row 4 (l / 16) + r, x row l % 16
        if ((lane & 15) < nc)
#pragma unroll
            for (int i = 0; i < R; ++i)
                *reinterpret_cast<v4f_t*>(sums + (wave * kCols + (lane & 15)) * LDR + 16 * i + 4 * (lane >> 4)) = acc[i];
        __syncthreads();
        for (int o = threadIdx.x; o < nc * 16 * G; o += blockDim.x) {
            const int cc = o / (16 * G), n = o % (16 * G);
            if (n0 + n >= outs) continue;
            float v = 0.0f, u = 0.0f;
            for (int w = 0; w < waves; ++w) {
                v += sums[(w * kCols + cc) * LDR + n];
                if constexpr (SWIGLU) u += sums[(w * kCols + cc) * LDR + 16 * G + n];
            }
            v *= ts;
            if constexpr (SWIGLU) v = swiglu32(v, u * ts);
            const int64_t yr = EXPERT ? list[c0 + cc] : (int64_t)blockIdx.y * kCols + cc;
            store1(p.y, p.y_bf16, yr * p.ldy + n0 + n, v);
        }
        __syncthreads();
    }
}

// y[t] = sum over j of weights[t][j] parts[t top_k + j], in order.
__global__ void __launch_bounds__(256) k_expert_sum(const float* __restrict__ parts, const float* __restrict__ weights,
                                                    int top_k, int64_t n, void* y, bool bf16, int64_t ldy) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
    if (i >= n) return;
    float v = 0.0f;
    for (int j = 0; j < top_k; ++j) v = __builtin_fmaf(weights[t * top_k + j], parts[(t * top_k + j) * n + i], v);
    store1(y, bf16, t * ldy + i, v);
}

inline int64_t v_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int FMT, bool XF32, bool SWIGLU, bool EXPERT>
hipError_t gemv_shaped(const GemvArgs& p, hipStream_t s) {
    constexpr int R = 2, G = SWIGLU ? 1 : 2;
    const int64_t outs = SWIGLU ? p.N / 2 : p.N;
    const int64_t rows_y = EXPERT ? p.assignments : v_cdiv(p.m, kCols);
    const int waves = (int)std::clamp<int64_t>(v_cdiv(p.K, kStep), 1, 8);
    hipLaunchKernelGGL((k_gemv<FMT, XF32, R, SWIGLU, EXPERT>), dim3((unsigned)v_cdiv(outs, 16 * G), (unsigned)rows_y),
                       dim3(64 * waves), 0, s, p);
    return hipGetLastError();
}

template <bool XF32>
hipError_t gemv_typed(const GemvArgs& p, bool swiglu, hipStream_t s) {
    if (p.mx) return gemv_shaped<kFmtMx, XF32, false, false>(p, s);
    if (p.scale_2d) {
        if (p.ids) return swiglu ? gemv_shaped<kFmtNv2D, XF32, true, true>(p, s) : gemv_shaped<kFmtNv2D, XF32, false, true>(p, s);
        return swiglu ? gemv_shaped<kFmtNv2D, XF32, true, false>(p, s) : gemv_shaped<kFmtNv2D, XF32, false, false>(p, s);
    }
    if (p.ids) return swiglu ? gemv_shaped<kFmtNv1D, XF32, true, true>(p, s) : gemv_shaped<kFmtNv1D, XF32, false, true>(p, s);
    return swiglu ? gemv_shaped<kFmtNv1D, XF32, true, false>(p, s) : gemv_shaped<kFmtNv1D, XF32, false, false>(p, s);
}

}  // namespace

hipError_t launch_gemv(const GemvArgs& p, bool swiglu, hipStream_t s) {
    if (p.m == 0 || p.N == 0) return hipSuccess;
    return p.x_bf16 ? gemv_typed<false>(p, swiglu, s) : gemv_typed<true>(p, swiglu, s);
}

hipError_t launch_expert_gemv(GemvArgs p, bool swiglu, const float* weights, float* ws, hipStream_t s) {
    if (p.assignments == 0 || p.N == 0) return hipSuccess;
    if (!weights) return launch_gemv(p, swiglu, s);
    // each assignment's product, then the tokens' weighted sums
    void* y = p.y;
    const bool bf16 = p.y_bf16;
    const int64_t ldy = p.ldy, outs = swiglu ? p.N / 2 : p.N;
    p.y = ws;
    p.y_bf16 = false;
    p.ldy = outs;
    const hipError_t e = launch_gemv(p, swiglu, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_expert_sum, dim3((unsigned)v_cdiv(outs, 256), (unsigned)(p.assignments / p.top_k)), dim3(256), 0,
                       s, ws, weights, p.top_k, outs, y, bf16, ldy);
    return hipGetLastError();
}

}  // namespace nvfp4
