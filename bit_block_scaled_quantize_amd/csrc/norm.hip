// RMS norm with the residual's addition and an MX output, and its backward
// pass, for gfx950.
//
// Forward, per row of n elements:
//   h = round(x + residual)            (the row type: the residual stream as stored)
//   rstd = 1 / sqrt(sum h^2 / n + eps)
//   y = h * rstd * weight
// y is written in the row type, as MX codes and scales of the binary32 y, or
// both.  Backward, with g = dy * weight and xhat = h * rstd:
//   dx = rstd * (g - xhat * mean(g * xhat)) + dh
//   dweight = sum over rows of dy * xhat
// The forward sum joins groups of 8 squares in binary64, y uses what rstd's
// rounding to binary32 leaves too, and where a binary32 y lies on the border of
// two MX codes it is told which side it comes from: the codes are those of the
// formula's y, but for at most one in 10^7 of BF16 rows, whose groups of 8 are
// summed in binary32.  (8192 x 5120 with binary32 sums and y as (h * weight) * rstd: 77
// us, codes in 10^6 on the other side of a border; this: 84; with every square in
// binary64 and every y rounded to odd: 87.)  The backward sums are binary32.  All
// are in a fixed order.
//
// Both are HBM-bound streams.  A row's elements stay in registers between the
// sum and the outputs, so every array is read or written once: TPR threads
// share a row (16, 64, 256, 512 or 1024), each holding NC chunks of 8 consecutive
// elements (chunk i of thread t starts at 8 (i TPR + t)), so a wave's 16-byte
// accesses are contiguous and four lanes hold one 32-element MX block.  The widest
// rows are the exceptions: the forward kernel of BF16 rows past 16384 columns, four
// chunks a thread, keeps 44 of its values in scratch memory, and the backward
// kernel reads rows past 8192 columns twice, the second time from the cache.
// Measured (a large copy reaches 5.07 TB/s), BF16: forward with h, y and MXFP8
// codes, 8192 x 5120, 84 us or 4.51 TB/s; without the codes 67 (5.0); MXFP4
// without y 70; 2560 x 16384 with both 88, 1280 x 32768 114.  Binary32, 8192 x 5120:
// 130 (5.2), with codes 138.  Backward with dh, 16384 x 7168, 183 us or 5.13 TB/s,
// binary32 356; 2048 x 16384 67.5 (4.0), 1024 x 32768 89.6 (3.0).  Rows of zeros,
// whose every y passes by the border check, cost nothing that shows (86).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "launch.hpp"
#include "nvfp4_device.hpp"
#include "row_device.hpp"

namespace nvfp4 {

namespace {

// Chunks a thread: at most kNC (8192 x 5120 forward, with binary32 sums: 4 took
// 81.5 us, 2 76.9) but in the widest rows, which 1024 threads hold in kMaxNC.
constexpr int kNC = 2, kMaxNC = 4;

template <typename T>
struct NormFwd {
    const T* x;
    const T* residual;  // nullable
    const void* weight;
    T* h;               // nullable
    T* y;               // nullable
    uint8_t* codes;     // nullable
    uint8_t* scales;
    float* rstd;        // nullable
    int64_t rows, cols, ldx, ldr, ldh, ldy, groups, turns;
    double eps, inv_cols;
    bool w_bf16, mx_e2m1;
};

__device__ __forceinline__ void load_weight(const void* w, bool bf16, int64_t c, int64_t n, float v[8]) {
    if (bf16) load_upto8(static_cast<const uint16_t*>(w) + c, n, v);
    else load_upto8(static_cast<const float*>(w) + c, n, v);
}

// 8 elements as they lie in memory.
template <typename T>
struct Raw {
    uint32_t q[2 * sizeof(T)];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < (int)(2 * sizeof(T)); ++j) q[j] = 0;
    }
    // p[0 .. min(n, 8) - 1], zero beyond (n >= 1)
    __device__ __forceinline__ void load(const T* p, int64_t n) {
        constexpr int W = 2 * sizeof(T);
        if (n >= 8) {
#pragma unroll
            for (int k = 0; k < W / 4; ++k) {
                const u4_align2 u = *reinterpret_cast<const u4_align2*>(p + 16 / sizeof(T) * k);
#pragma unroll
                for (int j = 0; j < 4; ++j) q[4 * k + j] = u[j];
            }
        } else if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                q[j] = (2 * j < n ? (uint32_t)p[2 * j] : 0u) | (2 * j + 1 < n ? (uint32_t)p[2 * j + 1] << 16 : 0u);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = j < n ? __float_as_uint(p[j]) : 0u;
        }
    }
    __device__ __forceinline__ float value(int j) const {
        if constexpr (sizeof(T) == 2) return __uint_as_float((j & 1) ? q[j >> 1] & 0xFFFF0000u : q[j >> 1] << 16);
        else return __uint_as_float(q[j]);
    }
};

constexpr int block_of(int tpr) { return tpr > 256 ? tpr : 256; }

// 1 / sqrt(x): the hardware's binary64 approximation and one step of third order.
__device__ __forceinline__ double rsqrt64(double x) {
    const double r = __builtin_amdgcn_rsq(x);
    const double e = __builtin_fma(-(x * r), r, 1.0);
    return e == e ? __builtin_fma(r * e, __builtin_fma(e, 0.375, 0.5), r) : r;  // (an x of 0 or infinity)
}

// The sum of 8 squares, by halves: of BF16 values, whose squares are exact, in
// binary32, of binary32 ones in binary64.
template <typename T>
__device__ __forceinline__ double squares8(const float v[8]) {
    using S = typename std::conditional<sizeof(T) == 2, float, double>::type;
    S q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const S a = v[2 * j], b = v[2 * j + 1];
        if constexpr (sizeof(T) == 2) q[j] = __builtin_fmaf(b, b, a * a);
        else q[j] = __builtin_fma(b, b, a * a);
    }
    return (double)((q[0] + q[1]) + (q[2] + q[3]));
}

// h (hi + lo) w, within a hair of half a step of binary32.  The clamp changes
// no finite product: it keeps an infinite w's from turning inf into NaN.
__device__ __forceinline__ float scaled(float h, float hi, float lo, float w) {
    const float a = h * hi, ae = __builtin_fmaf(h, lo, __builtin_fmaf(h, hi, -a));
    return __builtin_fmaf(a, w, __builtin_amdgcn_fmed3f(ae * w, -3.402823466e38f, 3.402823466e38f));
}

// The values of scaled(), rounded to odd: of the two neighbours
// of one that is not exact, the one whose last bit is 1.  Rounding that again to
// an MX code goes as rounding the product itself would.
__device__ __forceinline__ void scaled_odd(const float h[8], float hi, float lo, const float w[8], float y[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a = h[j] * hi, ae = __builtin_fmaf(h[j], lo, __builtin_fmaf(h[j], hi, -a));
        const float rest = __builtin_fmaf(ae, w[j], __builtin_fmaf(a, w[j], -y[j]));
        const int b = (int)__float_as_uint(y[j]);
        const int away = ((b ^ (int)__float_as_uint(rest)) >> 31) | 1;  // -1: towards zero
        // (infinity and NaN leave a rest of infinity or NaN: they stay)
        if (__builtin_fabsf(rest) > 0.0f && __builtin_fabsf(rest) < 1e30f && y[j] != 0.0f && !(b & 1))
            y[j] = __uint_as_float((uint32_t)(b + away));
    }
}

template <typename T, int NC>
struct FwdRow {
    Raw<T> x[NC], residual[NC];
};

template <typename T, int TPR, int NC>
__device__ __forceinline__ void load_row(const NormFwd<T>& a, int64_t r, int t, FwdRow<T, NC>& b) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = 8 * ((int64_t)i * TPR + t), n = a.cols - c;
        b.x[i].clear();
        b.residual[i].clear();
        if (n > 0) {
            b.x[i].load(a.x + r * a.ldx + c, n);
            if (a.residual) b.residual[i].load(a.residual + r * a.ldr + c, n);
        }
    }
}

// Row group g takes rows g, g + groups, ...; with AHEAD the next row's elements
// are under way while the current row's sum goes round and its outputs leave.
template <typename T, int TPR, int NC, bool AHEAD>
__global__ void __launch_bounds__(block_of(TPR)) k_rmsnorm(const NormFwd<T> a) {
    __shared__ double red[2][TPR > 64 ? TPR / 64 : 1];
    const int t = threadIdx.x % TPR;
    const int64_t g = (int64_t)blockIdx.x * (block_of(TPR) / TPR) + threadIdx.x / TPR;
    const int64_t last = a.rows - 1;
    int buf = 0;
    FwdRow<T, NC> cur, next;
    load_row<T, TPR, NC>(a, min(g, last), t, cur);
    // every group of a workgroup makes the same number of turns; those past
    // the last row repeat it and store nothing
    for (int64_t k = 0; k < a.turns; ++k) {
        const int64_t row = g + k * a.groups, r = min(row, last);
        if constexpr (AHEAD) {
            if (k + 1 < a.turns) load_row<T, TPR, NC>(a, min(row + a.groups, last), t, next);
        }
        const bool live = row <= last;
        float v[NC][8];
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = 8 * ((int64_t)i * TPR + t), n = a.cols - c;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = cur.x[i].value(j);
                if (a.residual) v[i][j] = rounded_to<T>(v[i][j] + cur.residual[i].value(j));
            }
            if (a.h && live && n > 0) store_upto8(a.h + r * a.ldh + c, n, v[i]);
            ss += squares8<T>(v[i]);
        }
        ss = row_sum64<TPR>(ss, red[buf]);
        buf ^= 1;
        const double scale = rsqrt64(__builtin_fma(ss, a.inv_cols, a.eps));
        const float rstd = (float)scale, rstd_lo = (float)(scale - (double)rstd);
        if (a.rstd && live && t == 0) a.rstd[r] = rstd;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = 8 * ((int64_t)i * TPR + t), n = a.cols - c;
            if (n <= 0) continue;
            float w[8], y[8];
            load_weight(a.weight, a.w_bf16, c, n, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = scaled(v[i][j], rstd, rstd_lo, w[j]);
            if (a.y && live) store_upto8(a.y + r * a.ldy + c, n, y);
            if (a.codes) {  // cols % 32 == 0: the four lanes of a block agree on n > 0
                // Halfway between two codes, or at a power of two, which sets a
                // block's scale, a binary32 number ends in 19 zeros, and which
                // side y lies on is lost: about one wave in a thousand.
                uint32_t ends = ~0u;
#pragma unroll
                for (int j = 0; j < 8; ++j) ends = min(ends, __float_as_uint(y[j]) << 13);
                if (__builtin_expect(ends == 0, 0)) scaled_odd(v[i], rstd, rstd_lo, w, y);
                uint32_t cw[2];
                const uint32_t sb = a.mx_e2m1 ? mx_block_rne8<kMxE2M1>(y, cw) : mx_block_rne8<kMxE4M3>(y, cw);
                if (live) {
                    if (a.mx_e2m1)
                        *reinterpret_cast<uint32_t*>(a.codes + r * (a.cols / 2) + c / 2) = cw[0];
                    else
                        *reinterpret_cast<uint2*>(a.codes + r * a.cols + c) = make_uint2(cw[0], cw[1]);
                    if ((t & 3) == 0) a.scales[r * (a.cols / 32) + c / 32] = (uint8_t)sb;
                }
            }
        }
        if constexpr (AHEAD) cur = next;
    }
}

template <typename T>
struct NormBwd {
    const T* dy;
    const T* h;
    const T* dh;  // nullable
    const float* rstd;
    const void* weight;
    T* dx;
    float* parts;  // groups x cols
    int64_t rows, cols, lddy, ldh, lddh, lddx, groups;
    bool w_bf16;
};

// What a row's thread reads: its elements of dy, h and dh, and the row's rstd.
template <typename T, int NC>
struct BwdRow {
    Raw<T> dy[NC], h[NC], dh[NC];
    float rstd;
};

template <typename T, int TPR, int NC>
__device__ __forceinline__ void load_row(const NormBwd<T>& a, int64_t r, int t, BwdRow<T, NC>& b) {
    b.rstd = a.rstd[r];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t c = 8 * ((int64_t)i * TPR + t), n = a.cols - c;
        b.dy[i].clear();
        b.h[i].clear();
        b.dh[i].clear();
        if (n > 0) {
            b.dy[i].load(a.dy + r * a.lddy + c, n);
            b.h[i].load(a.h + r * a.ldh + c, n);
            if (a.dh) b.dh[i].load(a.dh + r * a.lddh + c, n);
        }
    }
}

// Whether a row's and the next row's elements fit in registers (a workgroup of
// 1024 threads has 128 a thread).
constexpr bool reads_ahead(int tpr, int nc) { return tpr < 1024 || nc == 1; }

// A chunk's terms: adds to dw and returns the chunk's part of sum g xhat.
template <typename T>
__device__ __forceinline__ float bwd_terms(const Raw<T>& dy, const Raw<T>& h, const float w[8], float rstd, float dw[8]) {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float d = dy.value(j), xh = h.value(j) * rstd;
        dw[j] = __builtin_fmaf(d, xh, dw[j]);
        s = __builtin_fmaf(d * w[j], xh, s);
    }
    return s;
}

template <typename T>
__device__ __forceinline__ void bwd_store(const Raw<T>& dy, const Raw<T>& h, const Raw<T>& dh, const float w[8], float rstd,
                                          float s, T* dx, int64_t n) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float gx = __builtin_fmaf(-(h.value(j) * rstd), s, dy.value(j) * w[j]);
        q[j] = __builtin_fmaf(rstd, gx, dh.value(j));
    }
    store_upto8(dx, n, q);
}

// Row group g takes rows g, g + groups, ...; a workgroup's groups leave their
// sum of dy * xhat in parts[blockIdx.x].  The next row's elements are under way
// while the current row's sum goes round, so that the loads never wait for a
// reduction; rows too wide for that are read once for the sum and, from the
// cache, once more for the outputs.
template <typename T, int TPR, int NC>
__global__ void __launch_bounds__(block_of(TPR)) k_rmsnorm_backward(const NormBwd<T> a) {
    constexpr int per = block_of(TPR) / TPR;
    __shared__ float red[2][TPR > 64 ? TPR / 64 : 1];
    const int t = threadIdx.x % TPR;
    const int64_t g = (int64_t)blockIdx.x * per + threadIdx.x / TPR;
    float dw[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    // every group of a workgroup makes the same number of turns (row_sum needs
    // all lanes); turns past the last row read it again and add nothing
    const int64_t turns = (a.rows + a.groups - 1) / a.groups, last = a.rows - 1;
    const float inv_n = 1.0f / (float)a.cols;
    int buf = 0;
    if constexpr (reads_ahead(TPR, NC)) {
        float w[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = 8 * ((int64_t)i * TPR + t), n = a.cols - c;
#pragma unroll
            for (int j = 0; j < 8; ++j) w[i][j] = 0.0f;
            if (n > 0) load_weight(a.weight, a.w_bf16, c, n, w[i]);
        }
        BwdRow<T, NC> cur, next;
        load_row<T, TPR, NC>(a, min(g, last), t, cur);
        for (int64_t k = 0; k < turns; ++k) {
            const int64_t row = g + k * a.groups;
            if (k + 1 < turns) load_row<T, TPR, NC>(a, min(row + a.groups, last), t, next);
            const bool live = row <= last;
            if (!live) {
                cur.rstd = 0.0f;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    cur.dy[i].clear();
                    cur.h[i].clear();
                }
            }
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NC; ++i) s += bwd_terms(cur.dy[i], cur.h[i], w[i], cur.rstd, dw[i]);
            s = row_sum<TPR>(s, red[buf]) * inv_n;
            buf ^= 1;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int64_t c = 8 * ((int64_t)i * TPR + t), n = a.cols - c;
                if (n > 0 && live)
                    bwd_store(cur.dy[i], cur.h[i], cur.dh[i], w[i], cur.rstd, s, a.dx + row * a.lddx + c, n);
            }
            cur = next;
        }
    } else {  // (a group is a workgroup: each of its rows exists)
        for (int64_t row = g; row <= last; row += a.groups) {
            const float rstd = a.rstd[row];
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int64_t c = 8 * ((int64_t)i * TPR + t), n = a.cols - c;
                if (n <= 0) continue;
                Raw<T> dy, h;
                float w[8];
                dy.load(a.dy + row * a.lddy + c, n);
                h.load(a.h + row * a.ldh + c, n);
                load_weight(a.weight, a.w_bf16, c, n, w);
                s += bwd_terms(dy, h, w, rstd, dw[i]);
            }
            s = row_sum<TPR>(s, red[buf]) * inv_n;
            buf ^= 1;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int64_t c = 8 * ((int64_t)i * TPR + t), n = a.cols - c;
                if (n <= 0) continue;
                Raw<T> dy, h, dh;
                float w[8];
                dy.load(a.dy + row * a.lddy + c, n);
                h.load(a.h + row * a.ldh + c, n);
                dh.clear();
                if (a.dh) dh.load(a.dh + row * a.lddh + c, n);
                load_weight(a.weight, a.w_bf16, c, n, w);
                bwd_store(dy, h, dh, w, rstd, s, a.dx + row * a.lddx + c, n);
            }
        }
    }
    float* part = a.parts + (int64_t)blockIdx.x * a.cols;
    if constexpr (per == 1) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int64_t c = 8 * ((int64_t)i * TPR + t), n = a.cols - c;
            if (n > 0) store_upto8(part + c, n, dw[i]);
        }
    } else {
        __shared__ float of[per][TPR * NC * 8];
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) of[threadIdx.x / TPR][8 * (i * TPR + t) + j] = dw[i][j];
        __syncthreads();
        for (int c = threadIdx.x; c < (int)a.cols; c += block_of(TPR)) {
            float v = of[0][c];
#pragma unroll
            for (int k = 1; k < per; ++k) v += of[k][c];
            part[c] = v;
        }
    }
}

// dweight[c] = sum over g of parts[g][c] in a fixed order: 32 columns a
// workgroup, 32 threads a column (few groups: all their loads at once).
__global__ void __launch_bounds__(1024) k_sum_parts(const float* __restrict__ parts, int64_t groups, int64_t cols,
                                                    float* __restrict__ out) {
    __shared__ float s[32][33];
    const int cx = threadIdx.x & 31, gy = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + cx;
    float v = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t g = gy; g < groups; g += 32) v += parts[g * cols + c];
    }
    s[gy][cx] = v;
    __syncthreads();
    // column gy of the 32, its parts over the lanes of a half wave
    v = s[cx][gy];
    float a, b;
    row_pair(reduce16(v, AddOp()), a, b);
    if (cx == 0 && (int64_t)blockIdx.x * 32 + gy < cols) out[(int64_t)blockIdx.x * 32 + gy] = a + b;
}

inline int64_t n_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads per row: the fewest that hold the row in kNC chunks each; more
// where there are too few rows to give every SIMD a wave (the row's latency
// then counts).
int threads_per_row(int64_t rows, int64_t cols) {
    const int64_t chunks = n_cdiv(cols, 8);
    const auto more = [](int tpr) { return tpr == 256 || tpr == 512 ? 2 * tpr : 4 * tpr; };
    int tpr = 16;
    while (tpr < 1024 && chunks > (int64_t)tpr * kNC) tpr = more(tpr);
    while (tpr < 1024 && tpr < chunks && rows * tpr < 64 * 1024) tpr = more(tpr);
    return tpr;
}

struct BwdPlan {
    int tpr;
    int64_t blocks, groups;
};

// Row groups of the backward pass: two workgroups a compute unit at most, and
// at least two rows a group where there are that many (each workgroup costs a
// row of binary32 partial sums, written and read again).
BwdPlan bwd_plan(int64_t rows, int64_t cols) {
    BwdPlan p;
    p.tpr = threads_per_row(rows, cols);
    const int64_t per = block_of(p.tpr) / p.tpr;
    p.blocks = std::min<int64_t>(512, n_cdiv(n_cdiv(rows, 2), per));
    p.groups = p.blocks * per;
    return p;
}

#define NVFP4_NORM_NC(K, T, TPR, ...)                                                                       \
    do {                                                                                                    \
        const int64_t nc = n_cdiv(n_cdiv(a.cols, 8), TPR);                                                  \
        if (nc <= 1) hipLaunchKernelGGL((K<T, TPR, 1>), __VA_ARGS__, a);                                    \
        else if (nc <= 2 || TPR < 1024) hipLaunchKernelGGL((K<T, TPR, 2>), __VA_ARGS__, a);                 \
        else hipLaunchKernelGGL((K<T, TPR, (TPR < 1024 ? kNC : kMaxNC)>), __VA_ARGS__, a);                  \
    } while (0)

// The rows of a from r on.
template <typename T>
NormFwd<T> rows_from(NormFwd<T> a, int64_t r) {
    a.x += r * a.ldx;
    if (a.residual) a.residual += r * a.ldr;
    if (a.h) a.h += r * a.ldh;
    if (a.y) a.y += r * a.ldy;
    if (a.codes) {
        a.codes += r * (a.mx_e2m1 ? a.cols / 2 : a.cols);
        a.scales += r * (a.cols / 32);
    }
    if (a.rstd) a.rstd += r;
    a.rows -= r;
    return a;
}

// More rows than fill the chip with 1024 threads a compute unit: that many
// workgroups take the rows in turn, reading ahead (8192 x 5120, with binary32
// sums: one workgroup a row 82.8 us, reading ahead 76.9 with 1024 threads a
// unit and 78.0 with 2048).
template <typename T, int TPR, int NC>
void norm_launch(NormFwd<T> a, hipStream_t s) {
    // (rows that one grid cannot hold: over 4 million of over 8192 columns)
    const int64_t most_rows = max_blocks(block_of(TPR)) * (block_of(TPR) / TPR);
    for (; TPR == 1024 && a.rows > most_rows; a = rows_from(a, most_rows)) {
        NormFwd<T> part = a;
        part.rows = most_rows;
        norm_launch<T, TPR, NC>(part, s);
    }
    constexpr int per = block_of(TPR) / TPR;
    constexpr bool ahead = TPR < 1024;
    int64_t blocks = n_cdiv(a.rows, per);
    const int64_t most = 256 * (1024 / block_of(TPR));
    if (ahead && blocks > most) {
        blocks = most;
        a.groups = blocks * per;
        a.turns = n_cdiv(a.rows, a.groups);
        hipLaunchKernelGGL((k_rmsnorm<T, TPR, NC, ahead>), dim3((unsigned)blocks), dim3(block_of(TPR)), 0, s, a);
    } else {
        a.groups = blocks * per;
        a.turns = 1;
        hipLaunchKernelGGL((k_rmsnorm<T, TPR, NC, false>), dim3((unsigned)blocks), dim3(block_of(TPR)), 0, s, a);
    }
}

template <typename T>
hipError_t norm_typed(const NormFwd<T>& a, hipStream_t s) {
    const int tpr = threads_per_row(a.rows, a.cols);
    const int64_t nc = n_cdiv(n_cdiv(a.cols, 8), tpr);
#define NVFP4_NORM_FWD(TPR)                                       \
    if (nc <= 1) norm_launch<T, TPR, 1>(a, s);                    \
    else if (nc <= 2 || TPR < 1024) norm_launch<T, TPR, 2>(a, s); \
    else norm_launch<T, TPR, (TPR < 1024 ? kNC : kMaxNC)>(a, s)
    switch (tpr) {
        case 16: NVFP4_NORM_FWD(16); break;
        case 64: NVFP4_NORM_FWD(64); break;
        case 256: NVFP4_NORM_FWD(256); break;
        case 512: NVFP4_NORM_FWD(512); break;
        default: NVFP4_NORM_FWD(1024);
    }
#undef NVFP4_NORM_FWD
    return hipGetLastError();
}

template <typename T>
hipError_t norm_bwd_typed(NormBwd<T> a, float* dweight, hipStream_t s) {
    const BwdPlan p = bwd_plan(a.rows, a.cols);
    a.groups = p.groups;
    const dim3 g((unsigned)p.blocks), b(block_of(p.tpr));
    switch (p.tpr) {
        case 16: NVFP4_NORM_NC(k_rmsnorm_backward, T, 16, g, b, 0, s); break;
        case 64: NVFP4_NORM_NC(k_rmsnorm_backward, T, 64, g, b, 0, s); break;
        case 256: NVFP4_NORM_NC(k_rmsnorm_backward, T, 256, g, b, 0, s); break;
        case 512: NVFP4_NORM_NC(k_rmsnorm_backward, T, 512, g, b, 0, s); break;
        default: NVFP4_NORM_NC(k_rmsnorm_backward, T, 1024, g, b, 0, s);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_sum_parts, dim3((unsigned)n_cdiv(a.cols, 32)), dim3(1024), 0, s, a.parts, p.blocks, a.cols,
                       dweight);
    return hipGetLastError();
}
#undef NVFP4_NORM_NC

template <typename T>
hipError_t norm_any(const RmsNorm& n, hipStream_t s) {
    NormFwd<T> a;
    a.x = static_cast<const T*>(n.x);
    a.residual = static_cast<const T*>(n.residual);
    a.weight = n.weight;
    a.h = static_cast<T*>(n.h);
    a.y = static_cast<T*>(n.y);
    a.codes = n.codes;
    a.scales = n.scales;
    a.rstd = n.rstd;
    a.rows = n.rows;
    a.cols = n.cols;
    a.ldx = n.ldx;
    a.ldr = n.ldr;
    a.ldh = n.ldh;
    a.ldy = n.ldy;
    a.eps = n.eps;
    a.inv_cols = 1.0 / (double)n.cols;
    a.w_bf16 = n.w_bf16;
    a.mx_e2m1 = n.elem == kMxE2M1;
    return norm_typed(a, s);
}

template <typename T>
hipError_t norm_bwd_any(const RmsNormBackward& n, hipStream_t s) {
    NormBwd<T> a;
    a.dy = static_cast<const T*>(n.dy);
    a.h = static_cast<const T*>(n.h);
    a.dh = static_cast<const T*>(n.dh);
    a.rstd = n.rstd;
    a.weight = n.weight;
    a.dx = static_cast<T*>(n.dx);
    a.parts = n.ws;
    a.rows = n.rows;
    a.cols = n.cols;
    a.lddy = n.lddy;
    a.ldh = n.ldh;
    a.lddh = n.lddh;
    a.lddx = n.lddx;
    a.w_bf16 = n.w_bf16;
    return norm_bwd_typed(a, n.dweight, s);
}

}  // namespace

int64_t rmsnorm_backward_workspace_floats(int64_t rows, int64_t cols) {
    return rows == 0 ? 0 : bwd_plan(rows, cols).blocks * cols;
}

hipError_t launch_rmsnorm(const RmsNorm& n, hipStream_t s) {
    if (n.rows == 0) return hipSuccess;
    return n.bf16 ? norm_any<uint16_t>(n, s) : norm_any<float>(n, s);
}

hipError_t launch_rmsnorm_backward(const RmsNormBackward& n, hipStream_t s) {
    if (n.rows == 0) {
        // no rows: the weight's gradient is zero (the sum over no parts)
        hipLaunchKernelGGL(k_sum_parts, dim3((unsigned)n_cdiv(n.cols, 32)), dim3(1024), 0, s, n.ws, (int64_t)0,
                           n.cols, n.dweight);
        return hipGetLastError();
    }
    return n.bf16 ? norm_bwd_any<uint16_t>(n, s) : norm_bwd_any<float>(n, s);
}

}  // namespace nvfp4
