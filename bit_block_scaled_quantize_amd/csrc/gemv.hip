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
// Two kernels: k_gemv4 for up to 4 rows of x (below), k_gemv for more.
//
// k_gemv: a wave holds R tiles of 16 weight rows and goes over K in units of
// 256, two steps of four MFMAs each.  Lane l has weight row l % 16 (the MFMA's
// A operand) and the x row l % 16 (B); group g = l / 16 takes the 32
// consecutive k from 32 g of a step: 16 bytes of codes, one load.  The order
// of k inside an MFMA is the same for both operands and otherwise free.  A
// row's scales of a unit come in one load, and x in whole rows of 512 bytes,
// laid down in LDS in the order in which the lanes read it (a wave's own part:
// no barrier): loading both by lane, 8 rows against 8192 x 8192 MXFP4 took
// 15.0 us, now 11.1.  The W waves of a workgroup take the units in turn, so
// that together they stream whole rows, the next unit's loads under way while
// one is multiplied, and their sums are added through LDS in a fixed order.
//
// Measured (a large copy: 5.07 TB/s) on one weight again and again, which the
// 256 MB memory-side cache then holds, and on 16 weights in turn, which it does
// not: one BF16 row, 20480 x 5120 with 16x16 scales, 11.9 to 12.7 us and 14.0 (3.8
// TB/s); 4 rows 15.4 and 16.6, binary32 24.9 and 26.3; 8 rows 19.6 and 21.5,
// binary32 29.7 and 31.5; 8 rows, 8192 x 8192 MXFP4, 10.3 to 11.1 and 13.2 (2.7
// TB/s).  Four tokens through 4 of 32 experts of 7168 / 2048, up with SwiGLU, down
// and weighted sum: 68 to 71 us (4.2 to 4.3 TB/s, from memory); one token 25.0.
// With more than 4 rows an NVFP4 weight costs 2.7 vector instructions, and binary32
// x three times the matrix instructions (its instances for SwiGLU and for experts
// keep 2 registers in scratch memory).
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
constexpr int kUnit = 256;   // k of one unit
constexpr int kRowBytes = kUnit * 2;  // of a unit of one row of x in LDS, as BF16

// scale bytes start anywhere
typedef uint32_t u4_align1 __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u2_align1 __attribute__((ext_vector_type(2), aligned(1)));

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

// What a lane loads for a unit: codes and scale bytes of its R weight rows,
// and XP pieces of 16 bytes of x.
template <int R, int XP>
struct Unit {
    u4_t w[2][R];
    u4_t s[R];  // NVFP4: the row's 16 scale bytes; MX: 8
    u4_t x[XP];
};

// Where a lane reads.  Piece i of x: of a BF16 row 2 i + lane / 32 the 8
// elements from 8 (lane % 32), of a binary32 row i the 4 from 4 lane.
template <int R, int XP>
struct Lane {
    const uint8_t* codes[R];   // of the lane's weight rows
    const uint8_t* scales[R];
    const char* x[XP];
};

// The lane's share of the unit at k0.  TAIL: the last one, of which n < 256 k
// (a multiple of 16) are left; what lies beyond is zero.
template <int FMT, bool XF32, int R, int XP, bool TAIL>
__device__ __forceinline__ void load_unit(const Lane<R, XP>& a, int64_t k0, int n, int rows, Unit<R, XP>& u) {
    const int lane = threadIdx.x & 63, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = 128 * h + 32 * g;
            const uint8_t* p = a.codes[i] + (k0 + k) / 2;
            if (!TAIL || k + 32 <= n) {
                u.w[h][i] = *reinterpret_cast<const u4_align8*>(p);
            } else {
                u.w[h][i] = u4_t{0, 0, 0, 0};
                if (k < n) {
                    const u2_align8 q = *reinterpret_cast<const u2_align8*>(p);
                    u.w[h][i][0] = q[0];
                    u.w[h][i][1] = q[1];
                }
            }
        }
        constexpr int per = FMT == kFmtMx ? 32 : 16;
        const uint8_t* p = a.scales[i] + k0 / per;
        if constexpr (TAIL) {
            u.s[i] = u4_t{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < kUnit / per; ++j)
                if (j < n / per) u.s[i][j / 4] |= (uint32_t)p[j] << (8 * (j % 4));
        } else if constexpr (FMT == kFmtMx) {
            const u2_align1 q = *reinterpret_cast<const u2_align1*>(p);
            u.s[i][0] = q[0];
            u.s[i][1] = q[1];
        } else {
            u.s[i] = *reinterpret_cast<const u4_align1*>(p);
        }
    }
    const int kx = XF32 ? 4 * lane : 8 * (lane & 31);
#pragma unroll
    for (int i = 0; i < XP; ++i) {
        u.x[i] = u4_t{0, 0, 0, 0};
        if ((XF32 ? i : 2 * i) < rows && (!TAIL || kx < n))
            u.x[i] = *reinterpret_cast<const u4_align2*>(a.x[i] + k0 * (XF32 ? 4 : 2));
    }
}

// Row c's 16-byte piece q of LDS: pieces are exchanged within each 16 of them
// by the row, so that the 16 rows of a lane group's read lie in all banks.
__device__ __forceinline__ int piece_at(int c, int q) { return c * kRowBytes + 16 * (q ^ (c & 15)); }

// Lays the unit's x down in the wave's part of LDS (`rows` rows of BF16; of
// binary32 x three planes of them: the upper, middle and lower 8 bits).
template <bool XF32, int R, int XP>
__device__ __forceinline__ void stage_x(const Unit<R, XP>& u, int rows, char* lds) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < XP; ++i) {
        if ((XF32 ? i : 2 * i) >= rows) continue;
        if constexpr (XF32) {
            char* at = lds + piece_at(i, lane >> 1) + 8 * (lane & 1);
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(u.x[i][j]);
#pragma unroll
            for (int plane = 0; plane < 3; ++plane) {
                uint2 q;
                q.x = __builtin_amdgcn_perm(__float_as_uint(v[1]), __float_as_uint(v[0]), 0x07060302u);
                q.y = __builtin_amdgcn_perm(__float_as_uint(v[3]), __float_as_uint(v[2]), 0x07060302u);
                *reinterpret_cast<uint2*>(at + plane * rows * kRowBytes) = q;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = v[j] - __uint_as_float(__float_as_uint(v[j]) & 0xFFFF0000u);
            }
        } else {
            const int c = 2 * i + (lane >> 5);
            if (c < rows) *reinterpret_cast<u4_t*>(lds + piece_at(c, lane & 31)) = u.x[i];
        }
    }
    // (other lanes of the wave read it: in order after the writes)
    asm volatile("" ::: "memory");
}

// acc += the unit's products with x row c of LDS.
template <int FMT, bool XF32, int R, int XP>
__device__ __forceinline__ void multiply_unit(const Unit<R, XP>& u, const char* lds, int rows, int c, v4f_t acc[R]) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float s[R][2];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if constexpr (FMT == kFmtMx) {
                s[i][0] = s[i][1] = __uint_as_float(((u.s[i][h] >> (8 * g)) & 0xFFu) << 23);
            } else {
                const int b = (int)((g < 2 ? u.s[i][2 * h] : u.s[i][2 * h + 1]) >> (16 * (g & 1)));
                s[i][0] = __builtin_amdgcn_cvt_f32_fp8(b, 0);
                s[i][1] = __builtin_amdgcn_cvt_f32_fp8(b, 1);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const char* at = lds + piece_at(c, 16 * h + 4 * g + j);
            v8b_t b[XF32 ? 3 : 1];
#pragma unroll
            for (int plane = 0; plane < (XF32 ? 3 : 1); ++plane)
                b[plane] = *reinterpret_cast<const v8b_t*>(at + plane * rows * kRowBytes);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const v8b_t w = weights8<FMT>(u.w[h][i][j], s[i][j >> 1]);
#pragma unroll
                for (int plane = XF32 ? 2 : 0; plane >= 0; --plane) acc[i] = mfma(w, b[plane], acc[i]);
            }
        }
    }
    asm volatile("" ::: "memory");
}

// acc += the calling wave's units (wave, wave + waves, ...) of rows of K; the
// next unit's loads are under way while one is multiplied.
template <int FMT, bool XF32, int R, int XP>
__device__ __forceinline__ void multiply(const Lane<R, XP>& a, int64_t K, int rows, int c, char* lds, int wave, int waves,
                                         v4f_t acc[R]) {
    const int full = (int)(K / kUnit);
    Unit<R, XP> even, odd;
    const auto load = [&](int t, Unit<R, XP>& u) {
        load_unit<FMT, XF32, R, XP, false>(a, (int64_t)t * kUnit, kUnit, rows, u);
    };
    const auto step = [&](int t, Unit<R, XP>& u, Unit<R, XP>& next) {
        if (t + waves < full) load(t + waves, next);
        __builtin_amdgcn_sched_barrier(0);
        stage_x<XF32, R, XP>(u, rows, lds);
        multiply_unit<FMT, XF32, R, XP>(u, lds, rows, c, acc);
    };
    int t = wave;
    if (t < full) load(t, even);
    while (t < full) {
        step(t, even, odd);
        t += waves;
        if (t >= full) break;
        step(t, odd, even);
        t += waves;
    }
    if (K % kUnit && full % waves == wave) {
        load_unit<FMT, XF32, R, XP, true>(a, (int64_t)full * kUnit, (int)(K % kUnit), rows, even);
        stage_x<XF32, R, XP>(even, rows, lds);
        multiply_unit<FMT, XF32, R, XP>(even, lds, rows, c, acc);
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

// The columns of a workgroup: rows of x and of y, numbered from 0.
struct Columns {
    int count;
    int64_t wrow0;  // first row of their matrix in the stack
    float ts;
};

// Dense: rows `most` blockIdx.y and on.  EXPERT: the assignments that share the
// expert of assignment blockIdx.y, which is the first of them (list, in order);
// false where it is not, or has no expert, which leaves its `width` outputs
// from n0 zero.
template <bool EXPERT>
__device__ __forceinline__ bool find_columns(const GemvArgs& p, int64_t n0, int width, int64_t outs, int most, int* list,
                                             Columns& c) {
    const int lane = threadIdx.x & 63;
    c.wrow0 = 0;
    c.ts = 1.0f;
    if constexpr (EXPERT) {
        const int first = blockIdx.y, id = p.ids[first];
        if (id < 0 || id >= p.experts) {
            for (int o = threadIdx.x; o < width; o += blockDim.x)
                if (n0 + o < outs) store1(p.y, p.y_bf16, (int64_t)first * p.ldy + n0 + o, 0.0f);
            return false;
        }
        c.count = 0;
        for (int b = 0; b < p.assignments; b += 64) {
            const int a = b + lane;
            const bool same = a < p.assignments && p.ids[a] == id;
            const uint64_t m = __ballot(same);
            if (__any(same && a < first)) return false;  // (an earlier one has them; the same in every wave)
            if (threadIdx.x < 64 && same) list[c.count + __popcll(m & ((1ull << lane) - 1))] = a;
            c.count += __popcll(m);
        }
        __syncthreads();
        c.wrow0 = (int64_t)id * p.N;
        c.ts = p.ts[id];
    } else {
        c.count = (int)min((int64_t)most, p.m - (int64_t)blockIdx.y * most);
        if (p.ts) c.ts = p.ts[0];
    }
    return true;
}

template <bool EXPERT>
__device__ __forceinline__ int64_t y_row(int most, const int* list, int c) {
    return EXPERT ? list[c] : (int64_t)blockIdx.y * most + c;
}

template <bool EXPERT>
__device__ __forceinline__ int64_t x_row(const GemvArgs& p, int most, const int* list, int c) {
    const int64_t y = y_row<EXPERT>(most, list, c);
    return EXPERT && !p.x_per_assignment ? y / p.top_k : y;
}

extern __shared__ __attribute__((aligned(16))) char gemv_lds[];

// Workgroup (tile group blockIdx.x, blockIdx.y): R tiles of 16 weight rows
// against up to p.rows (<= 16) rows of x at a time: rows p.rows blockIdx.y and
// on, or (EXPERT) those of all assignments that share the expert of assignment
// blockIdx.y, which is the first of them (other workgroups end at once).
// SWIGLU: half of the tiles are gate rows, the others the up rows F further on.
template <int FMT, bool XF32, int R, int XP, bool SWIGLU, bool EXPERT>
__global__ void __launch_bounds__(512) k_gemv(const GemvArgs p) {
    constexpr int G = SWIGLU ? R / 2 : R;  // tiles of output columns
    constexpr int LDR = R * 16 + 4;        // floats of one x row's sums
    __shared__ int list[EXPERT ? kMaxGemvAssignments : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int64_t outs = SWIGLU ? p.N / 2 : p.N, n0 = (int64_t)blockIdx.x * (16 * G);
    char* lds = gemv_lds + wave * (p.rows * kRowBytes * (XF32 ? 3 : 1));
    float* sums = reinterpret_cast<float*>(gemv_lds);

    Columns cols;
    if (!find_columns<EXPERT>(p, n0, 16 * G, outs, p.rows, list, cols)) return;
    Lane<R, XP> a;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        // rows past the end repeat the last one; their sums are not stored
        const int64_t o = min(n0 + 16 * (i % G) + (lane & 15), outs - 1);
        const int64_t r = cols.wrow0 + (i < G ? 0 : outs) + o;
        a.codes[i] = p.codes + r * (p.K / 2);
        a.scales[i] = p.scales + (FMT == kFmtNv2D ? (r / 16) * (p.K / 16) : r * (p.K / (FMT == kFmtMx ? 32 : 16)));
    }
    for (int c0 = 0; c0 < cols.count; c0 += p.rows) {
        const int nc = min(cols.count - c0, p.rows);
#pragma unroll
        for (int i = 0; i < XP; ++i) {
            const int c = min(XF32 ? i : 2 * i + (lane >> 5), nc - 1);
            const int64_t xr = x_row<EXPERT>(p, p.rows, list, c0 + c);
            a.x[i] = static_cast<const char*>(p.x) + (XF32 ? 4 * (xr * p.ldx + 4 * lane) : 2 * (xr * p.ldx + 8 * (lane & 31)));
        }
        v4f_t acc[R];
#pragma unroll
        for (int i = 0; i < R; ++i) acc[i] = v4f_t{0.0f, 0.0f, 0.0f, 0.0f};
        // (lanes past the last column repeat it; their sums are not stored)
        multiply<FMT, XF32, R, XP>(a, p.K, nc, min(lane & 15, nc - 1), lds, wave, waves, acc);
        __syncthreads();
        // accumulator r of lane l: weight row 4 (l / 16) + r, x row l % 16
        if ((lane & 15) < nc)
#pragma unroll
            for (int i = 0; i < R; ++i)
                *reinterpret_cast<v4f_t*>(sums + (wave * nc + (lane & 15)) * LDR + 16 * i + 4 * (lane >> 4)) = acc[i];
        __syncthreads();
        for (int o = threadIdx.x; o < nc * 16 * G; o += blockDim.x) {
            const int cc = o / (16 * G), n = o % (16 * G);
            if (n0 + n >= outs) continue;
            float v = 0.0f, u = 0.0f;
            for (int w = 0; w < waves; ++w) {
                v += sums[(w * nc + cc) * LDR + n];
                if constexpr (SWIGLU) u += sums[(w * nc + cc) * LDR + 16 * G + n];
            }
            v *= cols.ts;
            if constexpr (SWIGLU) v = swiglu32(v, u * cols.ts);
            store1(p.y, p.y_bf16, y_row<EXPERT>(p.rows, list, c0 + cc) * p.ldy + n0 + n, v);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- up to 4 rows of x
// v_mfma_f32_4x4x4: 16 separate products of 4 x 4 x 4.  Lane l has weight row
// l % 4 and x row l % 4 of product l / 4, whose k are its own: 32 of a unit of
// 512, 16 bytes of codes of each of R rows.  A product's k then lie within one
// scale block of each row, so the E4M3 scales (NVFP4) go to the four sums of a
// block, one multiply-add each, instead of to every weight, and the weights
// take the convert's output as it is: about one instruction a weight where
// the 16-column form takes 2.7.  (One token, 20480 x 5120, 16x16 scales:
// 12.0 us here, 15.8 there.)
constexpr int kWide = 512;

typedef short v4s_t __attribute__((ext_vector_type(4)));
typedef uint16_t h_align1 __attribute__((aligned(1)));

__device__ __forceinline__ v4f_t mfma4(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, v4f_t c) {
    return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(v4s_t, make_uint2(a0, a1)),
                                                  __builtin_bit_cast(v4s_t, make_uint2(b0, b1)), c, 0, 0, 0);
}

template <bool XF32, int R>
struct Wide {
    u4_t w[R];
    uint32_t s[R];
    u4_t x[XF32 ? 8 : 4];
};

template <int R>
struct WideLane {
    const uint8_t* codes[R];
    const uint8_t* scales[R];
    const void* x;
};

// The lane's share at k (n of the row are left: 32 or more; TAIL: or 16, or
// none; what lies beyond is zero).
template <int FMT, bool XF32, int R, bool TAIL>
__device__ __forceinline__ void load_wide(const WideLane<R>& a, int64_t k, int64_t n, Wide<XF32, R>& u) {
    if constexpr (TAIL) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            u.w[i] = u4_t{0, 0, 0, 0};
            u.s[i] = 0;
        }
#pragma unroll
        for (int j = 0; j < (XF32 ? 8 : 4); ++j) u.x[j] = u4_t{0, 0, 0, 0};
        if (n <= 0) return;
    }
    const bool whole = !TAIL || n >= 32;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (whole) {
            u.w[i] = *reinterpret_cast<const u4_align8*>(a.codes[i] + k / 2);
        } else {
            const u2_align8 h = *reinterpret_cast<const u2_align8*>(a.codes[i] + k / 2);
            u.w[i][0] = h[0];
            u.w[i][1] = h[1];
        }
        if constexpr (FMT == kFmtMx) u.s[i] = a.scales[i][k / 32];
        else if (whole) u.s[i] = *reinterpret_cast<const h_align1*>(a.scales[i] + k / 16);
        else u.s[i] = a.scales[i][k / 16];
    }
    constexpr int per16 = XF32 ? 4 : 2;  // 16-byte pieces of 16 elements
#pragma unroll
    for (int j = 0; j < 2 * per16; ++j) {
        if (whole || j < per16)
            u.x[j] = *reinterpret_cast<const u4_align2*>(static_cast<const char*>(a.x) + k * (XF32 ? 4 : 2) + 16 * j);
    }
}

// Eight weights times 2^s as four BF16 pairs.
__device__ __forceinline__ void pairs8(uint32_t w, float s, uint32_t r[4]) {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
}

template <int FMT, bool XF32, int R>
__device__ __forceinline__ void multiply_wide(const Wide<XF32, R>& u, v4f_t acc[R]) {
    constexpr int P = XF32 ? 3 : 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 16 k
        uint32_t x[P][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (XF32) {
                float v0 = __uint_as_float(u.x[4 * h + j / 2][2 * (j & 1)]);
                float v1 = __uint_as_float(u.x[4 * h + j / 2][2 * (j & 1) + 1]);
#pragma unroll
                for (int q = 0; q < 3; ++q) {  // upper, middle and lower 8 bits
                    x[q][j] = __builtin_amdgcn_perm(__float_as_uint(v1), __float_as_uint(v0), 0x07060302u);
                    v0 = v0 - __uint_as_float(__float_as_uint(v0) & 0xFFFF0000u);
                    v1 = v1 - __uint_as_float(__float_as_uint(v1) & 0xFFFF0000u);
                }
            } else {
                x[0][j] = u.x[2 * h + j / 4][j % 4];
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            uint32_t w[8];
            const float one = FMT == kFmtMx ? __uint_as_float(u.s[i] << 23) : 1.0f;
            pairs8(u.w[i][2 * h], one, w);
            pairs8(u.w[i][2 * h + 1], one, w + 4);
            v4f_t d = FMT == kFmtMx ? acc[i] : v4f_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = P - 1; q >= 0; --q)
#pragma unroll
                for (int j = 0; j < 8; j += 2) d = mfma4(w[j], w[j + 1], x[q][j], x[q][j + 1], d);
            if constexpr (FMT == kFmtMx) {
                acc[i] = d;
            } else {  // sum r of the block is weight row r's, whose scale lane r of the quad has
                const float s = h ? __builtin_amdgcn_cvt_f32_fp8((int)u.s[i], 1) : __builtin_amdgcn_cvt_f32_fp8((int)u.s[i], 0);
                acc[i][0] = __builtin_fmaf(group_lane<4>(s, 0), d[0], acc[i][0]);
                acc[i][1] = __builtin_fmaf(group_lane<4>(s, 1), d[1], acc[i][1]);
                acc[i][2] = __builtin_fmaf(group_lane<4>(s, 2), d[2], acc[i][2]);
                acc[i][3] = __builtin_fmaf(group_lane<4>(s, 3), d[3], acc[i][3]);
            }
        }
    }
}

// As multiply, by units of 512.
template <int FMT, bool XF32, int R>
__device__ __forceinline__ void multiply_all_wide(const WideLane<R>& a, int64_t K, int wave, int waves, v4f_t acc[R]) {
    const int full = (int)(K / kWide), k0 = 32 * ((threadIdx.x & 63) >> 2);
    Wide<XF32, R> even, odd;
    const auto load = [&](int t, Wide<XF32, R>& u) { load_wide<FMT, XF32, R, false>(a, (int64_t)t * kWide + k0, 32, u); };
    int t = wave;
    if (t < full) load(t, even);
    while (t < full) {
        if (t + waves < full) load(t + waves, odd);
        __builtin_amdgcn_sched_barrier(0);
        multiply_wide<FMT, XF32, R>(even, acc);
        if ((t += waves) >= full) break;
        if (t + waves < full) load(t + waves, even);
        __builtin_amdgcn_sched_barrier(0);
        multiply_wide<FMT, XF32, R>(odd, acc);
        t += waves;
    }
    if (K % kWide && full % waves == wave) {
        const int64_t k = (int64_t)full * kWide + k0;
        load_wide<FMT, XF32, R, true>(a, k, K - k, even);
        multiply_wide<FMT, XF32, R>(even, acc);
    }
}

// As k_gemv with R groups of 4 weight rows and up to 4 rows of x.
template <int FMT, bool XF32, int R, bool SWIGLU, bool EXPERT>
__global__ void __launch_bounds__(512) k_gemv4(const GemvArgs p) {
    constexpr int G = SWIGLU ? R / 2 : R;
    __shared__ __attribute__((aligned(16))) float sums[8][4][4][4 * R];  // wave, 16 lanes, x row, weight row
    __shared__ int list[EXPERT ? kMaxGemvAssignments : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int64_t outs = SWIGLU ? p.N / 2 : p.N, n0 = (int64_t)blockIdx.x * (4 * G);
    Columns cols;
    if (!find_columns<EXPERT>(p, n0, 4 * G, outs, 4, list, cols)) return;
    WideLane<R> a;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t o = min(n0 + 4 * (i % G) + (lane & 3), outs - 1);
        const int64_t r = cols.wrow0 + (i < G ? 0 : outs) + o;
        a.codes[i] = p.codes + r * (p.K / 2);
        a.scales[i] = p.scales + (FMT == kFmtNv2D ? (r / 16) * (p.K / 16) : r * (p.K / (FMT == kFmtMx ? 32 : 16)));
    }
    for (int c0 = 0; c0 < cols.count; c0 += 4) {
        const int nc = min(cols.count - c0, 4);
        const int64_t xr = x_row<EXPERT>(p, 4, list, c0 + min(lane & 3, nc - 1));
        a.x = static_cast<const char*>(p.x) + xr * p.ldx * (XF32 ? 4 : 2);
        v4f_t acc[R];
#pragma unroll
        for (int i = 0; i < R; ++i) acc[i] = v4f_t{0.0f, 0.0f, 0.0f, 0.0f};
        multiply_all_wide<FMT, XF32, R>(a, p.K, wave, waves, acc);
        // accumulator r of lane l: weight row r, x row l % 4; over the four
        // products of 16 lanes here, the others through LDS
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                acc[i][r] += quad_perm<0x128>(acc[i][r]);  // lane + 8 of 16
                acc[i][r] += quad_perm<0x124>(acc[i][r]);  // lane + 4
            }
            if ((lane & 12) == 0) *reinterpret_cast<v4f_t*>(&sums[wave][lane >> 4][lane & 3][4 * i]) = acc[i];
        }
        __syncthreads();
        for (int o = threadIdx.x; o < nc * 4 * G; o += blockDim.x) {
            const int cc = o / (4 * G), n = o % (4 * G);
            if (n0 + n >= outs) continue;
            float v = 0.0f, u = 0.0f;
            for (int w = 0; w < waves; ++w)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    v += sums[w][q][cc][n];
                    if constexpr (SWIGLU) u += sums[w][q][cc][4 * G + n];
                }
            v *= cols.ts;
            if constexpr (SWIGLU) v = swiglu32(v, u * cols.ts);
            store1(p.y, p.y_bf16, y_row<EXPERT>(4, list, c0 + cc) * p.ldy + n0 + n, v);
        }
        __syncthreads();
    }
}

// y[t] = sum over j of weights[t][j] parts[t top_k + j], in order, of the
// assignments that have an expert (whatever weight the others have).
__global__ void __launch_bounds__(256) k_expert_sum(const float* __restrict__ parts, const float* __restrict__ weights,
                                                    const int* __restrict__ ids, int experts, int top_k, int64_t n, void* y,
                                                    bool bf16, int64_t ldy) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
    if (i >= n) return;
    float v = 0.0f;
    for (int j = 0; j < top_k; ++j) {
        const int id = ids[t * top_k + j];
        const float sum = __builtin_fmaf(weights[t * top_k + j], parts[(t * top_k + j) * n + i], v);
        v = id >= 0 && id < experts ? sum : v;
    }
    store1(y, bf16, t * ldy + i, v);
}

inline int64_t v_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Up to 4 rows of x.  Waves of a workgroup: 1, 2, 4 or 8, as many as make 1280
// in all (5 a compute unit), but two unless there are more than 6 tiles a unit:
// longer streams a wave pay beyond that (one BF16 row: 20480 x 5120 with 1, 2, 4 waves 13.5,
// 12.0, 13.7 us; 8192 x 8192 with 3, 4, 5 11.9, 12.4, 14.3; 5120 x 20480 with 4,
// 5, 8 18.6, 22.1, 20.1; 13 experts' 7168 x 2048 with 1, 2, 4 24.6, 28.2, 36.6.
// On each side of the step, one wave and two, weights in turn: of 5120 columns 1536
// tiles 15.7 and 14.8, 1600 tiles 16.3 and 17.0; of 2048 columns 8.4 and 8.1, 8.5 and
// 9.5; of 8192 columns 25.9 and 24.2, 27.4 and 27.6).
template <int FMT, bool XF32, bool SWIGLU, bool EXPERT>
void gemv4_launch(const GemvArgs& p, hipStream_t s) {
    constexpr int R = 4, G = SWIGLU ? R / 2 : R;
    const int64_t tiles_x = v_cdiv(SWIGLU ? p.N / 2 : p.N, 4 * G), tiles_y = EXPERT ? p.assignments : v_cdiv(p.m, 4);
    const int64_t tiles = tiles_x * tiles_y, units = v_cdiv(p.K, kWide);
    int waves = tiles <= 1536 ? 2 : 1;
    while (waves < 8 && waves * tiles < 1280) waves *= 2;
    waves = (int)std::clamp<int64_t>(units, 1, waves);
    hipLaunchKernelGGL((k_gemv4<FMT, XF32, R, SWIGLU, EXPERT>), dim3((unsigned)tiles_x, (unsigned)tiles_y), dim3(64 * waves),
                       0, s, p);
}

// Up to 16 rows at a time, in 2 XP (of binary32 x, XP) pieces a lane.
template <int FMT, bool XF32, int XP, bool SWIGLU, bool EXPERT>
void gemv_launch(const GemvArgs& p, hipStream_t s) {
    constexpr int R = 2, G = SWIGLU ? R / 2 : R;
    const int64_t tiles_x = v_cdiv(SWIGLU ? p.N / 2 : p.N, 16 * G), tiles_y = EXPERT ? p.assignments : v_cdiv(p.m, p.rows);
    const int64_t wave_bytes = (int64_t)p.rows * std::max<int>(kRowBytes * (XF32 ? 3 : 1), (R * 16 + 4) * 4);
    // A compute unit holds 8 of these waves.  More workgroups than units: two
    // of 4 waves take turns (20480 x 5120, 8 BF16 rows: 20.8 us, one of 8 24.0;
    // binary32 31.2, 42.2); else all 8 (8192 x 8192 MXFP4: 11.1 us, 12.3 with 4).
    const int64_t most = tiles_x * tiles_y > 256 ? 4 : 8;
    const int waves = (int)std::clamp<int64_t>(v_cdiv(p.K, kUnit), 1, std::min<int64_t>(most, (EXPERT ? 61440 : 65536) / wave_bytes));
    hipLaunchKernelGGL((k_gemv<FMT, XF32, R, XP, SWIGLU, EXPERT>), dim3((unsigned)tiles_x, (unsigned)tiles_y),
                       dim3(64 * waves), (size_t)(waves * wave_bytes), s, p);
}

// Rows of x at a time: as many as there are (of a routed product, as many as
// there are tokens: more assignments to an expert take further rounds), up to
// 16, of binary32 x to 8 (registers).
template <int FMT, bool XF32, bool SWIGLU, bool EXPERT>
hipError_t gemv_shaped(GemvArgs p, hipStream_t s) {
    p.rows = (int)std::min<int64_t>(EXPERT ? p.assignments / p.top_k : p.m, XF32 ? 8 : kCols);
    // Two assignments or fewer to an expert on the average seldom make five; where
    // they do, each four of them read the expert's matrix again (64 tokens, one
    // expert each of 32, 7168 / 2048: spread 146 us, all on one expert 200, where
    // the 16-column form takes 91).
    if (p.rows <= 4 || (EXPERT && p.assignments <= 2 * p.experts)) {
        gemv4_launch<FMT, XF32, SWIGLU, EXPERT>(p, s);
    } else {
        if constexpr (!XF32) {
            if (p.rows <= 8) {
                gemv_launch<FMT, XF32, 4, SWIGLU, EXPERT>(p, s);
                return hipGetLastError();
            }
        }
        gemv_launch<FMT, XF32, 8, SWIGLU, EXPERT>(p, s);
    }
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
                       s, ws, weights, p.ids, p.experts, p.top_k, outs, y, bf16, ldy);
    return hipGetLastError();
}

}  // namespace nvfp4
