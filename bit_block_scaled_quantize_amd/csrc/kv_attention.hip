// Attention over the paged 4-bit key/value cache, for gfx950:
//   o = softmax(scale q K^T) V,   row at position p sees keys (p - window, p].
//
// The G = q_heads / kv_heads heads of q that share a kv head, and the rows of a
// sequence, are the columns of one product, so that a key is read and converted
// once for up to 16 of them.  E2M1 times E4M3 is an FP16 value exactly (6
// significant bits, 2^-10 to 2688) and E2M1 times a power of two a BF16 value,
// so the products of the matrix cores are exact; their sums, the running
// maximum and the sum of the softmax are binary32.
//
// A wave takes 16 KT keys at a time: S^T = K Q^T by 16x16x32 MFMA with a key's
// codes converted in registers (lane l: key l % 16, the D / 4 elements from
// (l / 16) D / 4; the order of k is the same for q and otherwise free).  The
// sums lie with 4 keys of one column to a lane, which is the B operand of the
// second product, O^T = V^T P^T, as it is; V goes through LDS, converted, and
// comes back transposed (ds_read_b64_tr_b16).
//
// Work is split by keys: the 64-key tiles of all (sequence, kv head, 16
// columns) form one list, of which every workgroup takes an equal share, its 4
// waves in turn.  Where a share begins or ends inside a segment its sums go to
// the workspace and a second kernel joins them, in order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv_device.hpp"
#include "launch.hpp"
#include "nvfp4_device.hpp"
#include "row_device.hpp"

namespace nvfp4 {

namespace {

typedef _Float16 v8h_t __attribute__((ext_vector_type(8)));
typedef _Float16 v4h_t __attribute__((ext_vector_type(4)));
typedef _Float16 v2h_t __attribute__((ext_vector_type(2)));
typedef __bf16 v8b_t __attribute__((ext_vector_type(8)));
typedef __bf16 v4b_t __attribute__((ext_vector_type(4)));
typedef __bf16 v2b_t __attribute__((ext_vector_type(2)));
typedef float v4f_t __attribute__((ext_vector_type(4)));
typedef float v2f_t __attribute__((ext_vector_type(2)));
typedef short v4s_t __attribute__((ext_vector_type(4)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef uint16_t h_align1 __attribute__((aligned(1)));
typedef uint32_t w_align1 __attribute__((aligned(1)));

constexpr int kThreads = 256, kWaves = 4;
constexpr int kCols = 16;     // columns (rows of q x heads of a group) of a segment
constexpr int kTile = 64;     // keys of a unit of work
constexpr int kShares = 512;  // workgroups: two on each of 256 compute units
constexpr float kLowest = -3.402823466e38f;
// weights are taken times 2^kBias, near FP16's largest: half a step of its
// subnormal numbers is then 2^-40 of the largest weight
constexpr float kBias = 15.0f;
constexpr float kLog2e = 1.4426950408889634f;

// One format's operand type: FP16 for NVFP4, BF16 (whose exponents hold every
// E8M0 scale) for MXFP4; a value in binary32 is the sum of kParts<F32> of them.
template <bool MX>
struct Form;
template <>
struct Form<false> {
    typedef v8h_t v8;
    typedef v2h_t v2;
    typedef _Float16 one;
    static __device__ __forceinline__ v4f_t mfma(v8 a, v8 b, v4f_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    // 8 codes times the block scale of their byte
    static __device__ __forceinline__ v8 values(uint32_t w, uint32_t byte) {
        const _Float16 s = (_Float16)e4m3_value(byte);
        const v2h_t ss = {s, s};
        u4_t r;
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * ss);
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * ss);
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * ss);
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * ss);
        return __builtin_bit_cast(v8, r);
    }
};
template <>
struct Form<true> {
    typedef v8b_t v8;
    typedef v2b_t v2;
    typedef __bf16 one;
    static __device__ __forceinline__ v4f_t mfma(v8 a, v8 b, v4f_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ v8 values(uint32_t w, uint32_t byte) {
        const float s = e8m0_value(byte);
        u4_t r;
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
        return __builtin_bit_cast(v8, r);
    }
};

// Parts of q: a BF16 value fits FP16 once its row is scaled to [2^14, 2^15) (an
// element below 2^-29 of the row's largest keeps 2^-25 of 2^14, past the
// products' binary32 sums), a binary32 one two FP16 or three BF16 parts.  Parts
// of a weight in [0, 2^kBias]: one FP16 part is off by 2^-12, two BF16 parts by
// 2^-17, of binary32 results two FP16 parts by 2^-23, three BF16 parts by 2^-25.
template <bool MX, bool F32>
constexpr int kQParts = F32 ? (MX ? 3 : 2) : 1;
template <bool MX, bool F32>
constexpr int kPParts = F32 ? (MX ? 3 : 2) : (MX ? 2 : 1);

// v as PARTS values of the form, each nearest to what is left.
template <bool MX, int PARTS>
__device__ __forceinline__ void split8(const float v[8], typename Form<MX>::v8 out[PARTS]) {
    float left[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) left[j] = v[j];
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        u4_t r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const v2f_t f = {left[2 * j], left[2 * j + 1]};
            const auto h = __builtin_convertvector(f, typename Form<MX>::v2);
            r[j] = __builtin_bit_cast(uint32_t, h);
            if (i + 1 < PARTS) {
                left[2 * j] -= (float)h[0];
                left[2 * j + 1] -= (float)h[1];
            }
        }
        out[i] = __builtin_bit_cast(typename Form<MX>::v8, r);
    }
}

// ---------------------------------------------------------------- the list of work
// Sequence s has `columns` blocks of 16 columns and `tiles` tiles of keys from
// first_tile (one at least, so that rows that see no key have a place where
// they are written).
struct Seq {
    int row, rows, length, columns, first_tile, tiles;
};

__device__ __forceinline__ Seq seq_of(const KvAttention& p, int s) {
    Seq q;
    kv_rows(p.plan, s, q.row, q.rows);
    q.length = kv_length(p.plan, s);
    q.columns = (int)(((int64_t)q.rows * p.group + kCols - 1) / kCols);
    const int64_t low = p.window ? (int64_t)q.length - q.rows - p.window + 1 : 0;
    q.first_tile = low > 0 ? (int)(low / kTile) : 0;
    q.tiles = max(1, (q.length + kTile - 1) / kTile - q.first_tile);
    return q;
}

__device__ __forceinline__ int64_t units_of(const KvAttention& p, const Seq& q) {
    return (int64_t)q.columns * q.tiles * p.cache.heads;
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int from) {
    return (int64_t)((uint64_t)(uint32_t)__shfl((int)(v >> 32), from) << 32 | (uint32_t)__shfl((int)v, from));
}

// Inclusive sum over the lanes.
__device__ __forceinline__ int64_t scan64(int64_t v) {
    const int lane = threadIdx.x & 63;
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = shfl64(v, lane >= d ? lane - d : lane);
        if (lane >= d) v += o;
    }
    return v;
}

// Units of sequences 64 b and on, by lane.
__device__ __forceinline__ int64_t lane_units(const KvAttention& p, int b) {
    const int s = b + (threadIdx.x & 63);
    return s < p.plan.seqs ? units_of(p, seq_of(p, s)) : 0;
}

__device__ __forceinline__ int64_t all_units(const KvAttention& p) {
    int64_t sum = 0;
    for (int b = 0; b < p.plan.seqs; b += 64) sum += shfl64(scan64(lane_units(p, b)), 63);
    return sum;
}

// Sequence of unit u (< all_units) and the first unit of that sequence.
__device__ __forceinline__ int find_seq(const KvAttention& p, int64_t u, int64_t& first) {
    int64_t before = 0;
    for (int b = 0;; b += 64) {
        const int64_t own = lane_units(p, b), upto = scan64(own), all = shfl64(upto, 63);
        if (u < before + all) {
            const int l = __builtin_ctzll(__ballot(u < before + upto));
            first = before + shfl64(upto - own, l);
            return b + l;
        }
        before += all;
    }
}

// Workgroups that take a share: one for 4 tiles (its waves) at least.
__device__ __forceinline__ int64_t shares_of(int64_t units) { return max((int64_t)1, min((int64_t)kShares, units / kWaves)); }

__device__ __forceinline__ int64_t share_begin(int64_t w, int64_t shares, int64_t units) {
    const int64_t each = units / shares, rest = units % shares;
    return w * each + min(w, rest);
}

// Columns [first, first + count) of a segment are rows and heads of q: column c
// is row c / group, head c % group of the kv head's.
struct Segment {
    int head, first, count;
    int64_t begin, end;  // units
};

__device__ __forceinline__ Segment segment_at(const KvAttention& p, const Seq& q, int64_t seq_first, int64_t u) {
    const int64_t at = (u - seq_first) / q.tiles;
    Segment g;
    g.head = (int)(at / q.columns);
    g.first = (int)(at % q.columns) * kCols;
    g.count = (int)min((int64_t)kCols, (int64_t)q.rows * p.group - g.first);
    g.begin = seq_first + at * q.tiles;
    g.end = g.begin + q.tiles;
    return g;
}

// ---------------------------------------------------------------- sums of a share
// A share's sums of a segment in the workspace: [16][D] of O, then the columns'
// maxima and sums.
template <int D>
constexpr int kSlotFloats = kCols * D + 2 * kCols;

// The two slots of share w: of a segment that an earlier share began (0), and
// of one that it begins and does not end (1).
template <int D>
__device__ __forceinline__ float* slot_of(const KvAttention& p, int64_t w, int which) {
    return p.ws + (2 * w + which) * kSlotFloats<D>;
}

template <bool F32>
__device__ __forceinline__ void store_out(const KvAttention& p, const Seq& q, const Segment& g, int c, int d, v4f_t o) {
    const int row = q.row + (g.first + c) / p.group, head = g.head * p.group + (g.first + c) % p.group;
    const int64_t at = row * p.out.row + head * p.out.head + d;
    if constexpr (F32) {
        f4_align4 v = {o[0], o[1], o[2], o[3]};
        *reinterpret_cast<f4_align4*>(static_cast<float*>(p.out.data) + at) = v;
    } else {
        typedef uint32_t u2_align2 __attribute__((ext_vector_type(2), aligned(2)));
        u2_align2 v = {pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
        *reinterpret_cast<u2_align2*>(static_cast<uint16_t*>(p.out.data) + at) = v;
    }
}

__device__ __forceinline__ void store_lse(const KvAttention& p, const Seq& q, const Segment& g, int c, float m, float l) {
    const int64_t row = q.row + (g.first + c) / p.group;
    const int head = g.head * p.group + (g.first + c) % p.group;
    p.lse[row * p.q_heads + head] = l > 0.0f ? (m - kBias + __builtin_log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// Keys of a sub-tile of 16 in a lane: codes and scale bytes.
template <int D>
struct Codes {
    uint32_t w[D / 32];
    uint32_t s;
};

extern __shared__ __attribute__((aligned(16))) char kv_lds[];

// V rows in LDS: 32 bytes after each row put 8 rows' 32-byte pieces, which a
// transposed read takes at once, into different banks.
template <int D>
constexpr int kRowBytes = 2 * D + 32;
template <int D>
constexpr int kWaveBytes = 32 * kRowBytes<D>;
// floats between the columns of a wave's O in LDS
template <int D>
constexpr int kMergeStride = D + 4;

template <int D, bool MX>
__device__ __forceinline__ void load_codes(const uint8_t* codes, const uint8_t* scales, Codes<D>& c) {
    if constexpr (D == 64) {
        const uint2 q = *reinterpret_cast<const uint2*>(codes);
        c.w[0] = q.x;
        c.w[1] = q.y;
    } else {
#pragma unroll
        for (int i = 0; i < D / 128; ++i) {
            const u4_t q = *reinterpret_cast<const u4_t*>(codes + 16 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) c.w[4 * i + j] = q[j];
        }
    }
    constexpr int n = MX ? D / 128 : D / 64;  // scale bytes of D / 4 elements (0: half a block)
    if constexpr (n <= 1) c.s = *scales;
    else if constexpr (n == 2) c.s = *reinterpret_cast<const h_align1*>(scales);
    else c.s = *reinterpret_cast<const w_align1*>(scales);
}

// The j-th 8 of the lane's elements.
template <int D, bool MX>
__device__ __forceinline__ typename Form<MX>::v8 values8(const Codes<D>& c, int j) {
    return Form<MX>::values(c.w[j], (c.s >> (8 * (8 * j / (MX ? 32 : 16)))) & 0xFFu);
}

template <bool MX, bool F32, int D>
__global__ void __launch_bounds__(kThreads, 2) k_kv_attention(const KvAttention p) {
    typedef Form<MX> F;
    typedef typename F::v8 v8;
    constexpr int QP = kQParts<MX, F32>, PP = kPParts<MX, F32>, KD = D / 32;
    constexpr int per = MX ? 32 : 16;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g4 = lane >> 4;
    char* lds = kv_lds + wave * kWaveBytes<D>;
    __shared__ float stats[2][kWaves][kCols];

    const int64_t units = all_units(p);
    const int64_t shares = shares_of(units), me = blockIdx.x;
    if (units == 0 || me >= shares) return;
    int64_t u = share_begin(me, shares, units);
    const int64_t u_end = share_begin(me + 1, shares, units);
    int64_t seq_first;
    int s = find_seq(p, u, seq_first);
    Seq q = seq_of(p, s);
    const int slot_mask = (1 << p.plan.page_shift) - 1;

    while (u < u_end) {
        while (u >= seq_first + units_of(p, q)) {
            seq_first += units_of(p, q);
            q = seq_of(p, ++s);
        }
        const Segment g = segment_at(p, q, seq_first, u);
        const int64_t stop = min(g.end, u_end);
        // the lane's column
        const int c = g.first + min(col, g.count - 1);
        const int qrow = c / p.group, qhead = g.head * p.group + c % p.group;
        const int pos = q.length - q.rows + qrow;  // sees keys low .. pos
        const int low = p.window ? max(0, pos - p.window + 1) : 0;
        // of the segment's first and last column
        const int pos_first = q.length - q.rows + g.first / p.group;
        const int pos_last = q.length - q.rows + (g.first + g.count - 1) / p.group;
        const int seg_low = p.window ? max(0, pos_first - p.window + 1) : 0;

        // q, its row scaled into FP16's range
        v8 qf[KD][QP];
        float factor = p.scale * kLog2e;
        if constexpr (!MX) factor *= p.cache.k_scale[g.head];
        {
            float v[KD][8];
            const int64_t at = (q.row + qrow) * p.q.row + qhead * p.q.head + g4 * (D / 4);
#pragma unroll
            for (int j = 0; j < KD; ++j) {
                if constexpr (F32) load_upto8(static_cast<const float*>(p.q.data) + at + 8 * j, 8, v[j]);
                else load_upto8(static_cast<const uint16_t*>(p.q.data) + at + 8 * j, 8, v[j]);
            }
            if constexpr (!MX) {
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < KD; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[j][i]));
                float a, b;
                row_pair(top, a, b);
                half_pair(fmaxf(a, b), a, b);
                const int e = __builtin_amdgcn_frexp_expf(fmaxf(a, b));  // 0 for 0
#pragma unroll
                for (int j = 0; j < KD; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] = ldexpf(v[j][i], 15 - e);
                factor = ldexpf(factor, e - 15);
            }
#pragma unroll
            for (int j = 0; j < KD; ++j) split8<MX, QP>(v[j], qf[j]);
        }

        float m = kLowest, l = 0.0f;
        v4f_t o[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i] = v4f_t{0.0f, 0.0f, 0.0f, 0.0f};

        const int j0 = q.first_tile + (int)(u - g.begin), j1 = q.first_tile + (int)(stop - g.begin);
        for (int j = j0 + wave; j < j1; j += kWaves) {
            const int key0 = j * kTile;
            if (key0 > pos_last || key0 + kTile <= seg_low) continue;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                const int k32 = key0 + 32 * half;
                if (k32 > pos_last) break;
                // pages of the two sub-tiles of 16 keys (-1: none)
                int page[2];
                Codes<D> kc[2], vc[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int k16 = k32 + 16 * t;
                    page[t] = -1;
                    if (k16 < q.length)
                        page[t] = __builtin_amdgcn_readfirstlane(kv_page(p.plan, p.cache.pages, s, k16));
                    if (page[t] >= 0) {
                        const int64_t slot = (((int64_t)page[t] * p.cache.heads + g.head) << p.plan.page_shift) + (k16 & slot_mask) + col;
                        const int64_t sc = slot * (D / per) + g4 * (D / 4) / per;
                        load_codes<D, MX>(p.cache.k_codes + slot * (D / 2) + g4 * (D / 8), p.cache.k_scales + sc, kc[t]);
                        load_codes<D, MX>(p.cache.v_codes + slot * (D / 2) + g4 * (D / 8), p.cache.v_scales + sc, vc[t]);
                        if (k16 + col >= q.length) kc[t].s = vc[t].s = 0;  // what lies behind the end is no number
                    } else {
#pragma unroll
                        for (int i = 0; i < KD; ++i) kc[t].w[i] = vc[t].w[i] = 0;
                        kc[t].s = vc[t].s = 0;
                    }
                }
                // scores: register r of sub-tile t is key 16 t + 4 g4 + r of the column
                v4f_t sc[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    sc[t] = v4f_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < KD; ++i) {
                        const v8 a = values8<D, MX>(kc[t], i);
#pragma unroll
                        for (int x = QP - 1; x >= 0; --x) sc[t] = F::mfma(a, qf[i][x], sc[t]);
                    }
                }
                float top = kLowest;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int key = k32 + 16 * t + 4 * g4 + r;
                        const bool seen = page[t] >= 0 && key <= pos && key >= low && key < q.length;
                        sc[t][r] = seen ? sc[t][r] * factor : -INFINITY;
                        top = fmaxf(top, sc[t][r]);
                    }
                {
                    float a, b;
                    row_pair(top, a, b);
                    half_pair(fmaxf(a, b), a, b);
                    top = fmaxf(a, b);
                }
                if (__any(top > m)) {
                    const float next = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - next);
                    m = next;
                    l *= f;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[i][r] *= f;
                }
                float w[8];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        w[4 * t + r] = __builtin_amdgcn_exp2f(sc[t][r] - m + kBias);
                        l += w[4 * t + r];
                    }
                v8 pf[PP];
                split8<MX, PP>(w, pf);
                // V through LDS
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < KD; ++i)
                        *reinterpret_cast<v8*>(lds + (16 * t + col) * kRowBytes<D> + g4 * (D / 2) + 16 * i) = values8<D, MX>(vc[t], i);
                asm volatile("" ::: "memory");
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    typedef __attribute__((address_space(3))) v4s_t lds_v4s;
                    char* at = lds + (4 * g4 + (col >> 2)) * kRowBytes<D> + 32 * i + 8 * (col & 3);
                    const v4s_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)at);
                    const v4s_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + 16 * kRowBytes<D>));
                    typedef short v8s_t __attribute__((ext_vector_type(8)));
                    const v8s_t z = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
                    for (int k = PP - 1; k >= 0; --k) o[i] = F::mfma(__builtin_bit_cast(v8, z), pf[k], o[i]);
                }
                asm volatile("" ::: "memory");
            }
        }

        // the waves' sums, joined in order
        {
            float a, b;
            row_pair(l, a, b);
            half_pair(a + b, a, b);
            l = a + b;
        }
        float* mine = reinterpret_cast<float*>(lds);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            *reinterpret_cast<v4f_t*>(mine + col * kMergeStride<D> + 16 * i + 4 * g4) = o[i];
        if (g4 == 0) {
            stats[0][wave][col] = m;
            stats[1][wave][col] = l;
        }
        __syncthreads();
        const bool whole = u == g.begin && stop == g.end;
        float* slot = slot_of<D>(p, me, u == g.begin ? 1 : 0);
        const float v_scale = MX ? 1.0f : p.cache.v_scale[g.head];
        for (int i = threadIdx.x; i < g.count * (D / 4); i += kThreads) {
            const int cc = i / (D / 4), d = 4 * (i % (D / 4));
            float top = kLowest;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stats[0][w][cc]);
            float total = 0.0f;
            v4f_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float f = __builtin_amdgcn_exp2f(stats[0][w][cc] - top);
                const v4f_t x = *reinterpret_cast<const v4f_t*>(reinterpret_cast<const float*>(kv_lds + w * kWaveBytes<D>) +
                                                                cc * kMergeStride<D> + d);
                total += f * stats[1][w][cc];
#pragma unroll
                for (int r = 0; r < 4; ++r) sum[r] += f * x[r];
            }
            if (whole) {
                const float f = total > 0.0f ? v_scale / total : 0.0f;
#pragma unroll
                for (int r = 0; r < 4; ++r) sum[r] *= f;
                store_out<F32>(p, q, g, cc, d, sum);
                if (p.lse && d == 0) store_lse(p, q, g, cc, top, total);
            } else {
                *reinterpret_cast<v4f_t*>(slot + cc * D + d) = sum;
                if (d == 0) {
                    slot[kCols * D + cc] = top;
                    slot[kCols * D + kCols + cc] = total;
                }
            }
        }
        __syncthreads();
        u = stop;
    }
}

// Share w joins the segment that its first unit lies inside of, where it is the
// first share that does.
template <bool MX, bool F32, int D>
__global__ void __launch_bounds__(kThreads) k_kv_join(const KvAttention p) {
    const int64_t units = all_units(p);
    const int64_t shares = shares_of(units), w = blockIdx.x + 1;
    if (units == 0 || w >= shares) return;
    const int64_t u = share_begin(w, shares, units);
    int64_t seq_first;
    const int s = find_seq(p, u, seq_first);
    const Seq q = seq_of(p, s);
    const Segment g = segment_at(p, q, seq_first, u);
    if (u == g.begin || share_begin(w - 1, shares, units) > g.begin) return;
    const float v_scale = MX ? 1.0f : p.cache.v_scale[g.head];
    for (int i = threadIdx.x; i < g.count * (D / 4); i += kThreads) {
        const int cc = i / (D / 4), d = 4 * (i % (D / 4));
        float top = kLowest, total = 0.0f;
        v4f_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int64_t k = w - 1; k < shares && share_begin(k, shares, units) < g.end; ++k) {
            const float* slot = slot_of<D>(p, k, k == w - 1 ? 1 : 0);
            const float m = slot[kCols * D + cc], next = fmaxf(top, m);
            const float f = __builtin_amdgcn_exp2f(top - next), h = __builtin_amdgcn_exp2f(m - next);
            const v4f_t x = *reinterpret_cast<const v4f_t*>(slot + cc * D + d);
            total = total * f + slot[kCols * D + kCols + cc] * h;
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[r] = sum[r] * f + x[r] * h;
            top = next;
        }
        const float f = total > 0.0f ? v_scale / total : 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] *= f;
        store_out<F32>(p, q, g, cc, d, sum);
        if (p.lse && d == 0) store_lse(p, q, g, cc, top, total);
    }
}

template <bool MX, bool F32, int D>
hipError_t run(const KvAttention& p, hipStream_t s) {
    constexpr int bytes = kWaves * kWaveBytes<D>;
    static_assert(kCols * kMergeStride<D> * 4 <= kWaveBytes<D>);
    if constexpr (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_kv_attention<MX, F32, D>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((k_kv_attention<MX, F32, D>), dim3(kShares), dim3(kThreads), bytes, s, p);
    hipLaunchKernelGGL((k_kv_join<MX, F32, D>), dim3(kShares - 1), dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t rows, int q_heads, int kv_heads, int dim, bool bf16) {
    (void)q_heads;
    (void)kv_heads;
    (void)bf16;
    return rows > 0 ? (size_t)2 * kShares * (kCols * dim + 2 * kCols) * sizeof(float) : 0;
}

hipError_t launch_kv_attention(const KvAttention& p, hipStream_t s) {
    if (p.plan.rows == 0) return hipSuccess;
    const auto pick = [&](auto mx, auto f32) {
        constexpr bool MX = decltype(mx)::value, F32 = decltype(f32)::value;
        if (p.cache.dim == 64) return run<MX, F32, 64>(p, s);
        if (p.cache.dim == 128) return run<MX, F32, 128>(p, s);
        return run<MX, F32, 256>(p, s);
    };
    const std::true_type yes;
    const std::false_type no;
    if (p.cache.mx) return p.bf16 ? pick(yes, no) : pick(yes, yes);
    return p.bf16 ? pick(no, no) : pick(no, yes);
}

}  // namespace nvfp4
