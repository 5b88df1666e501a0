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
// Few columns (k_kv_attention; bounded by the cache's bytes when sequences are many
// or long, by one workgroup's latency else): a wave takes 32 keys at a time,
// S^T = K Q^T by 16x16x32 MFMA with a key's codes converted in registers (lane l:
// key l % 16, the D / 4 elements from (l / 16) D / 4; the order of k is the same for
// q and otherwise free).  The sums lie with 4 keys of one column to a lane, which is
// the B operand of the second product, O^T = V^T P^T, as it is; V goes through LDS,
// converted, and comes back transposed (ds_read_b64_tr_b16).  The steps of 32 keys of
// all (sequence, kv head, 16 columns) form one list that is divided by its sizes on
// the device (Division), so the host needs no length and a captured call serves
// changing ones; what several workgroups share of a segment is joined by a second
// kernel, in order.  Time, of 8 kv heads of 128, BF16, without offsets: one token of 40
// heads over 8192 positions 14.6 us; 256 of 40 over up to 501 30.2 us; 64 of 56 over up
// to 20480 158 us, 4.7 TB/s of codes and scales, where a large copy, read and written,
// reaches 5.04.  (The D 256 instance of binary32 over MXFP4, with three parts of both
// operands, keeps 24 bytes a lane in scratch memory.)
//
// Many columns of BF16 (k_kv_prefill; bounded by the alternation of matrix and vector
// instructions, neither of which fills its pipe): 256 columns, 64 keys at a time, in
// two phases; 8192 rows of 40 heads with causal masks in 731 to 766 us on several cards,
// 900 to 940 TFLOP/s of the 1220 that a product of 8192^3 reaches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

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
constexpr int kStep = 32;     // keys of a unit of work
constexpr int kTile = 64;     // keys of a tile of k_kv_prefill
constexpr float kLowest = -3.402823466e38f;
// Weights are taken over a maximum that may lie up to kSlack (in powers of two)
// below the true one, so that the sums are rescaled seldom.
constexpr float kSlack = 4.0f;
// exp2(score - maximum + bias) is one multiply-add before the exponential while the
// maxima are no further than this from 0: what m - bias and the product round is then
// below 2^-3 in the exponent, and the weight below 2^15.2.  Further away that rounding
// would pass FP16's largest (or all bounds), so scores are rounded to binary32 first
// and the maximum, the true one of all keys so far, taken off exactly.
constexpr float kFar = 1048576.0f;
// Sequences of more columns than this for a kv head are k_kv_prefill's (BF16 q).  (Over
// 4096 positions, by k_kv_attention and k_kv_prefill: 64 sequences of 35 columns 181 and
// 203 us, of 60 204 and 205, of 80 266 and 212; 16 sequences of 60 67 and 80, of 80 81 and
// 82, of 100 102 and 85.  For fewer sequences it could be more: 4 of 80 39 and 46, of 125
// 42 and 49; one of 80 25 and 43.)
constexpr int kFewColumns = 64;
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
// of a weight: one FP16 part is off by 2^-11, two BF16 parts by 2^-17, of binary32
// results two FP16 parts by 2^-23, three BF16 parts by 2^-25.
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

// Weights are taken times 2^bias.  FP16: so that they reach its largest; half a step
// of its subnormal numbers is then 2^-36 of the largest weight.  BF16 has no such
// limit, but MXFP4's values go up to binary32's own: the weights of all keys that a
// row sees add up to at most one (and some 9% that rounding far scores may add), so
// that no sum of products passes 1.1 x 6 x 2^125.  (The matrix cores keep subnormal
// numbers: results of small values lose bits below 2^-126 / 2^bias, but not at once.)
template <bool MX>
__device__ __forceinline__ float weight_bias(const KvAttention& p, int length) {
    if constexpr (!MX) return 11.0f;
    const int keys = p.window ? min(length, p.window) : length;
    return -kSlack - (float)(keys > 1 ? 32 - __clz(keys - 1) : 0);
}

// Scores in powers of two for a product of q, times 2^(15 - e), with a head's keys:
// |scale| log2(e) (NVFP4: times k_scale, 2^(e - 15)).  The significands are multiplied
// and the exponents added, since scale x k_scale alone may leave the normal numbers where
// the scores do not.  (At least the least normal number: 0 times a hidden score's -inf is
// no number.)
template <bool MX>
__device__ __forceinline__ float score_factor(const KvAttention& p, int head, int e) {
    const float scale = fabsf(p.scale);
    int exponent = __builtin_amdgcn_frexp_expf(scale);
    float f = __builtin_amdgcn_frexp_mantf(scale) * kLog2e;
    if constexpr (!MX) {
        const float k = p.cache.k_scale[head];
        exponent += __builtin_amdgcn_frexp_expf(k) + e - 15;
        f *= __builtin_amdgcn_frexp_mantf(k);
    }
    return fmaxf(ldexpf(f, exponent), 1.1754944e-38f);
}

// The sum of 8 values, in pairs (a sum one by one waits for each addition).
__device__ __forceinline__ float sum8(const float v[8]) {
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// ---------------------------------------------------------------- the list of work
// Sequence s has `columns` blocks of 16 columns for each kv head: segments of
// `real` steps of keys from first_step (one at least, so that rows that see no
// key have a place where they are written).
struct Seq {
    int row, rows, length, columns, first_step, real;
};

__device__ __forceinline__ Seq seq_of(const KvAttention& p, int s) {
    Seq q;
    kv_rows(p.plan, s, q.row, q.rows);
    q.length = kv_length(p.plan, s);
    const int64_t cols = (int64_t)q.rows * p.group;
    q.columns = p.bf16 && cols > kFewColumns ? 0 : (int)((cols + kCols - 1) / kCols);
    const int64_t low = p.window ? (int64_t)q.length - q.rows - p.window + 1 : 0;
    q.first_step = low > 0 ? (int)(low / kStep) : 0;
    q.real = max(1, (q.length + kStep - 1) / kStep - q.first_step);
    return q;
}

// a / b of numbers that are not negative (a 64-bit division takes some hundred
// instructions).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// A lane's value in every lane.
__device__ __forceinline__ int64_t from_lane(int64_t v, int lane) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
                     (uint32_t)__builtin_amdgcn_readlane((int)v, lane));
}

// v of the lane SHIFT places below within its row of 16, 0 where there is none.
template <int SHIFT>
__device__ __forceinline__ int64_t row_below(int64_t v) {
    const int lo = __builtin_amdgcn_update_dpp(0, (int)v, 0x110 + SHIFT, 0xF, 0xF, true);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), 0x110 + SHIFT, 0xF, 0xF, true);
    return (int64_t)((uint64_t)(uint32_t)hi << 32 | (uint32_t)lo);
}

// Inclusive sum over the lanes (all active): rows of 16, then the rows below.
__device__ __forceinline__ int64_t scan64(int64_t v) {
    v += row_below<1>(v);
    v += row_below<2>(v);
    v += row_below<4>(v);
    v += row_below<8>(v);
    const int row = (threadIdx.x & 63) >> 4;
    const int64_t a = from_lane(v, 15), b = a + from_lane(v, 31), c = b + from_lane(v, 47);
    return v + (row == 0 ? 0 : row == 1 ? a : row == 2 ? b : c);
}

// Sum over the lanes.
__device__ __forceinline__ int64_t sum64(int64_t v) {
    v += row_below<1>(v);
    v += row_below<2>(v);
    v += row_below<4>(v);
    v += row_below<8>(v);
    return from_lane(v, 15) + from_lane(v, 31) + from_lane(v, 47) + from_lane(v, 63);
}

// Steps and segments of 256 sequences, 4 consecutive ones to a lane, whose loads
// are under way together; where there are 64 in all or fewer, one to a lane.
struct Quad {
    int real[4], segs[4];
    static __device__ __forceinline__ int each(const KvAttention& p) { return p.plan.seqs <= 64 ? 1 : 4; }
    __device__ __forceinline__ Quad(const KvAttention& p, int b) {
        const int s = b + each(p) * (threadIdx.x & 63);
#pragma unroll
        for (int i = 0; i < 4; ++i) real[i] = segs[i] = 0;
        count(p, s, 0);
        if (each(p) == 4) {
#pragma unroll
            for (int i = 1; i < 4; ++i) count(p, s + i, i);
        }
    }
    __device__ __forceinline__ void count(const KvAttention& p, int s, int i) {
        const Seq q = seq_of(p, min(s, p.plan.seqs - 1));  // (past the end the last one's again, without a branch)
        real[i] = q.real;
        segs[i] = s < p.plan.seqs ? q.columns * p.cache.heads : 0;
    }
};

// The list of entries by sequence, count(real, segs) of each: the sum of all, and
// the sequence of entry u (< sum) with the first entry of that sequence.  The first
// 256 sequences are loaded once.
template <typename Count>
struct List {
    const KvAttention& p;
    const Quad& first256;
    Count count;
    int64_t upto0, sum;
    __device__ __forceinline__ List(const KvAttention& p_, const Quad& q, Count c) : p(p_), first256(q), count(c) {
        upto0 = scan64(all_of(q));
        sum = from_lane(upto0, 63);
        for (int b = 256; b < p.plan.seqs; b += 256) sum += from_lane(scan64(all_of(Quad(p, b))), 63);
    }
    __device__ __forceinline__ int64_t all_of(const Quad& q) const {
        int64_t n = count(q.real[0], q.segs[0]);
        if (Quad::each(p) == 4) n += count(q.real[1], q.segs[1]) + count(q.real[2], q.segs[2]) + count(q.real[3], q.segs[3]);
        return n;
    }
    __device__ __forceinline__ int find(int64_t u, int64_t& first) const {
        int64_t before = 0, upto = upto0;
        Quad q = first256;
        for (int b = 0;;) {
            const int64_t all = from_lane(upto, 63);
            if (u < before + all) {
                const int l = __builtin_ctzll(__ballot(u < before + upto));
                int s = b + Quad::each(p) * l;
                first = before + from_lane(upto - all_of(q), l);
                if (Quad::each(p) == 4) {
#pragma unroll
                    for (int i = 0; i < 3; ++i) {
                        const int64_t n = from_lane(count(q.real[i], q.segs[i]), l);
                        if (s == b + 4 * l + i && u >= first + n) {
                            first += n;
                            ++s;
                        }
                    }
                }
                return __builtin_amdgcn_readfirstlane(s);
            }
            before += all;
            b += 256;
            q = Quad(p, b);
            upto = scan64(all_of(q));
        }
    }
};
template <typename Count>
__device__ __forceinline__ List<Count> list_of(const KvAttention& p, const Quad& q, Count c) {
    return List<Count>(p, q, c);
}

// Workgroups (as many as 256 compute units hold at once by their registers and
// LDS).
template <bool F32, int D>
constexpr int kShares = D == 256 ? 512 : F32 && D == 128 ? 768 : 1024;

// How the segments are divided, by what they are on the device:
//   by team    no segment has more than kShort steps, and there are kManySegments
//              at least and no more than all waves: teams of 4, 2 or 1 waves, as many
//              as there are segments or nearly, have one each;
//   in parts   of `part` steps (kLeast at least), as many as there are workgroups
//              or fewer, if that takes no more than kMostPart steps: a workgroup
//              has one part;
//   in shares  else: every workgroup has an equal share of the list of all steps,
//              whose first and last may lie inside segments.  A segment counts
//              kExtra steps more than it has, about what its beginning and end
//              cost.
// (Parts end with their segment where shares would have a second one to begin,
// which costs some 5 us; many steps are better divided evenly.  40 heads, 8 kv heads of
// 128, by team and in shares: 256 sequences of up to 500 positions 28.4 and 43.5 us, 512
// of them 51.8 and 76, up to 1000 positions 45.7 and 59.8, 91 and 109; one of 1000 among
// 256 of up to 500 29.8 and 44.0, one of 2000 (kShort 64) 46.1 and 44.2, among 512 96 and
// 79.  Past all waves, where teams would go round again, 520 sequences 166 and 79, 4096
// 1897 and 460.  In parts and in shares: one token over 2048 11.9 and 11.3, over 8192 14.9
// and 15.3, 16 over up to 8000 27.6 and 28.7; with parts of 8 steps and more one over 2048
// 13.0, over 8192 14.0, 16 over up to 2000 18.2 instead of 20.2.  kExtra: 33 sequences of
// up to 10000 46 us, without it 92.)
constexpr int kShort = 32, kManySegments = 512, kLeast = kWaves, kMostPart = 32, kExtra = 4;
struct Division {
    int team;           // waves of a team; 0: not by team
    int part;           // 0: in shares
    int64_t sum;        // segments, parts or units of the list
    int64_t each, rest; // shares: the first `rest` have a unit more
    int64_t shares;
    __device__ __forceinline__ int64_t begin(int64_t w) const { return w * each + min(w, rest); }
    __device__ __forceinline__ int64_t share_of(int64_t u) const {
        const int64_t split = rest * (each + 1);
        return u < split ? quotient(u, each + 1) : rest + quotient(u - split, each);
    }
    // entries of a sequence
    __device__ __forceinline__ int64_t operator()(int real, int segs) const {
        return team ? segs : part ? (int64_t)segs * ((uint32_t)(real + part - 1) / (uint32_t)part)
                                     : segs * ((int64_t)real + kExtra);
    }
};

__device__ __forceinline__ Division divide(const KvAttention& p, const Quad& first256, int most) {
    bool longer = false;
    int64_t steps = 0, segments = 0;
    for (int b = 0; b < p.plan.seqs; b += 256) {
        const Quad q = b ? Quad(p, b) : first256;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            longer |= q.segs[i] > 0 && q.real[i] > kShort;
            steps += (int64_t)q.real[i] * q.segs[i];
            segments += q.segs[i];
        }
    }
    steps = sum64(steps);
    segments = sum64(segments);
    Division d = {};
    if (!__any(longer) && segments >= kManySegments) d.team = segments <= most ? 4 : segments <= 2 * most ? 2 : segments <= 4 * most ? 1 : 0;
    if (d.team || segments == 0) {
        d.sum = segments;
        return d;
    }
    if (segments <= most) {
        int64_t part = max((int64_t)kLeast, quotient(steps + most - 1, most));
        for (; part <= kMostPart; part += part / 4) {
            d.part = (int)part;
            d.sum = list_of(p, first256, d).sum;
            if (d.sum <= most) return d;
        }
        d.part = 0;
    }
    d.sum = steps + kExtra * segments;
    d.shares = max((int64_t)1, min((int64_t)most, quotient(d.sum, kLeast)));
    d.each = quotient(d.sum, d.shares);
    d.rest = d.sum - d.each * d.shares;
    return d;
}

// Columns [first, first + count) of a segment are rows and heads of q: column c
// is row c / group, head c % group of the kv head's.  Its entries of the list are
// `begin` and on.
struct Segment {
    int head, first, count;
    int64_t begin, entries;
};

__device__ __forceinline__ Segment segment_at(const KvAttention& p, const Division& d, const Seq& q, int64_t seq_first,
                                              int64_t u) {
    Segment g;
    g.entries = d(q.real, 1);
    const int64_t at = quotient(u - seq_first, g.entries);
    g.begin = seq_first + at * g.entries;
    g.head = (int)quotient(at, q.columns);
    g.first = (int)(at - (int64_t)g.head * q.columns) * kCols;
    g.count = (int)min((int64_t)kCols, (int64_t)q.rows * p.group - g.first);
    return g;
}

// ---------------------------------------------------------------- sums of a share
// A share's sums of a segment in the workspace: [16][D] of O, then the columns'
// maxima and sums.
template <int D>
constexpr int kSlotFloats = kCols * D + 2 * kCols;

// Two slots for a workgroup: of a segment that an earlier one began (0), and of one
// that it begins and does not end (1).
template <int D>
__device__ __forceinline__ float* slot_of(const KvAttention& p, int64_t w, int which) {
    return p.ws + (2 * w + which) * kSlotFloats<D>;
}

// What the second kernel's workgroup w - 1 joins: an equal part (the rank-th of n - 1)
// of the segment that workgroup w's share begins inside of, whose n parts are those of
// workgroups first_share and on.  n 0: nothing.  (With that found again there, one token
// over 8192 positions took 15.4 us instead of 14.3.)
struct Join {
    int n, rank, first_share, row, head, first, count;
    float bias;
};
template <int D>
constexpr int64_t kShareFloats = 2 * kSlotFloats<D> + sizeof(Join) / sizeof(float);
template <int D, int SHARES>
__device__ __forceinline__ Join* join_of(const KvAttention& p, int w) {
    return reinterpret_cast<Join*>(p.ws + (int64_t)2 * SHARES * kSlotFloats<D>) + w;
}

// What a sum of weighted values is multiplied by for the result: 2^-exponent, then
// v_scale over l's significand, since v_scale / l may lie below the normal numbers where
// the result does not.  The significand is in [1, 2) over NVFP4, whose values are at most
// 2688 until v_scale comes in, and in [1/2, 1) over MXFP4, where the first product may
// then not pass the result.  Without weights: 0.
template <bool MX>
struct Mean {
    float factor;
    int exponent;
    __device__ __forceinline__ Mean(float l, float v_scale) {
        exponent = __builtin_amdgcn_frexp_expf(l) - (MX ? 0 : 1);
        factor = l > 0.0f ? v_scale / ldexpf(l, -exponent) : 0.0f;
    }
    __device__ __forceinline__ float operator()(float x) const { return ldexpf(x, -exponent) * factor; }
    __device__ __forceinline__ v4f_t operator()(float a, float b, float c, float d) const {
        return v4f_t{(*this)(a), (*this)(b), (*this)(c), (*this)(d)};
    }
};

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

__device__ __forceinline__ void store_lse(const KvAttention& p, const Seq& q, const Segment& g, int c, float m, float bias,
                                          float l) {
    const int64_t row = q.row + (g.first + c) / p.group;
    const int head = g.head * p.group + (g.first + c) % p.group;
    p.lse[row * p.q_heads + head] = l > 0.0f ? (m - bias + __builtin_log2f(l)) * 0.6931471805599453f : -INFINITY;
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
__device__ __forceinline__ Codes<D> load_codes(const uint8_t* codes, const uint8_t* scales) {
    Codes<D> c;
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
    return c;
}

// The j-th 8 of the lane's elements.
template <int D, bool MX>
__device__ __forceinline__ typename Form<MX>::v8 values8(const Codes<D>& c, int j) {
    return Form<MX>::values(c.w[j], (c.s >> (8 * (8 * j / (MX ? 32 : 16)))) & 0xFFu);
}

// What a lane holds of 32 keys: of sub-tile t key 16 t + lane % 16.
template <int D>
struct Step {
    Codes<D> k[2], v[2];
};

template <bool MX, bool F32, int D>
__global__ void __launch_bounds__(kThreads, (kShares<F32, D> / 256)) k_kv_attention(const KvAttention p) {
    typedef Form<MX> F;
    typedef typename F::v8 v8;
    constexpr int QP = kQParts<MX, F32>, PP = kPParts<MX, F32>, KD = D / 32;
    constexpr int per = MX ? 32 : 16;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g4 = lane >> 4;
    char* lds = kv_lds + wave * kWaveBytes<D>;
    __shared__ float stats[2][kWaves][kCols];

    if (threadIdx.x == 0) join_of<D, kShares<F32, D>>(p, blockIdx.x)->n = 0;
    const Quad first256(p, 0);
    const Division d = divide(p, first256, kShares<F32, D>);
    const int team = d.team ? d.team : kWaves, teams = kWaves / team, member = wave & (team - 1), mine0 = wave - member;
    // the workgroup's first entry; its team's is `team_u` further on
    const int team_u = d.team ? wave / team : 0;
    int64_t u = d.team ? (int64_t)blockIdx.x * teams : blockIdx.x, u_end = d.sum;
    if (!d.team && !d.part) {
        if (u >= d.shares) return;
        u_end = d.begin(u + 1);
        u = d.begin(u);
    }
    if (u >= u_end) return;
    int64_t seq_first;
    int s = list_of(p, first256, d).find(min(u + team_u, u_end - 1), seq_first);
    Seq q = seq_of(p, s);
    const int slot_mask = (1 << p.plan.page_shift) - 1;

    while (u < u_end) {
        const bool idle = u + team_u >= u_end;  // (a team past the last segment has its barriers alone)
        const int64_t own = min(u + team_u, u_end - 1);
        for (;;) {
            const int64_t n = d(q.real, q.columns * p.cache.heads);
            if (own < seq_first + n) break;
            seq_first += n;
            q = seq_of(p, ++s);
        }
        const Segment g = segment_at(p, d, q, seq_first, own);
        // steps [from, to) of the segment's
        int from = 0, to = idle ? 0 : q.real;
        if (d.team || d.part) u_end = 0;  // (a team or a workgroup has one entry)
        if (d.part) {
            from = (int)(u - g.begin) * d.part;
            to = min(q.real, from + d.part);
        } else if (!d.team) {
            from = (int)min(u - g.begin, (int64_t)q.real);
            to = (int)min(u_end - g.begin, (int64_t)q.real);
            if (from > 0 && from >= to) {  // (an end that counts but has no steps)
                u = g.begin + g.entries;
                continue;
            }
        }
        // the lane's column
        const int c = g.first + min(col, g.count - 1);
        const int qrow = c / p.group, qhead = g.head * p.group + c % p.group;
        const int pos = q.length - q.rows + qrow;  // sees keys low .. pos
        const int low = p.window ? max(0, pos - p.window + 1) : 0;
        // of the segment's first and last column
        const int pos_first = q.length - q.rows + g.first / p.group;
        const int pos_last = q.length - q.rows + (g.first + g.count - 1) / p.group;
        const int low_first = p.window ? max(0, pos_first - p.window + 1) : 0;
        const int low_last = p.window ? max(0, pos_last - p.window + 1) : 0;

        const float bias = weight_bias<MX>(p, q.length);

        // steps of 32 keys that some column sees
        const int j1 = min(q.first_step + to, pos_last < 0 ? 0 : pos_last / kStep + 1);
        int j = max(q.first_step + from, low_first / kStep) + member;

        // (the table's entries are looked at a step later)
        const auto find_entry = [&](int at, int t) {
            const int k16 = at * kStep + 16 * t;
            return at < j1 && k16 < q.length ? kv_entry(p.plan, s, k16) : -1;
        };
        const auto page_of = [&](int entry) { return kv_page_of(__builtin_amdgcn_readfirstlane(entry), p.cache.pages); };
        const auto load = [&](int at, int t, int page, const uint8_t* codes, const uint8_t* scales) {
            Codes<D> c = {};
            if (page >= 0) {
                const int64_t first = (((int64_t)page * p.cache.heads + g.head) << p.plan.page_shift) + ((at * kStep + 16 * t) & slot_mask);
                c = load_codes<D, MX>(codes + first * (D / 2) + (col * (D / 2) + g4 * (D / 8)),
                                      scales + first * (D / per) + (col * (D / per) + g4 * (D / 4) / per));
            }
            return c;
        };
        Step<D> st;  // the step at j
        int page[2], next[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            page[t] = page_of(find_entry(j, t));
            st.k[t] = load(j, t, page[t], p.cache.k_codes, p.cache.k_scales);
            st.v[t] = load(j, t, page[t], p.cache.v_codes, p.cache.v_scales);
            next[t] = find_entry(j + team, t);
        }

        if (!d.team && from > 0 && threadIdx.x == 0) {
            const int64_t first = d.part ? g.begin : d.share_of(g.begin);
            const int n = d.part ? (int)g.entries : (int)(d.share_of(g.begin + q.real - 1) - first) + 1;
            *join_of<D, kShares<F32, D>>(p, blockIdx.x) =
                Join{n, (int)(blockIdx.x - first) - 1, (int)first, q.row, g.head, g.first, g.count, bias};
        }

        // q, its row scaled into FP16's range
        v8 qf[KD][QP];
        float factor;
        {
            float v[KD][8];
            const int64_t at = (q.row + qrow) * p.q.row + qhead * p.q.head + g4 * (D / 4);
#pragma unroll
            for (int i = 0; i < KD; ++i) {
                if constexpr (F32) load_upto8(static_cast<const float*>(p.q.data) + at + 8 * i, 8, v[i]);
                else load_upto8(static_cast<const uint16_t*>(p.q.data) + at + 8 * i, 8, v[i]);
            }
            int e = 15;
            if constexpr (!MX) {
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < KD; ++i)
#pragma unroll
                    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[i][k]));
                float a, b;
                row_pair(top, a, b);
                half_pair(fmaxf(a, b), a, b);
                e = __builtin_amdgcn_frexp_expf(fmaxf(a, b));  // 0 for 0
            }
            factor = score_factor<MX>(p, g.head, e);
            // (the scale's sign goes with q, so that larger sums are larger scores)
#pragma unroll
            for (int i = 0; i < KD; ++i) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if constexpr (!MX) v[i][k] = ldexpf(v[i][k], 15 - e);
                    if (p.scale < 0.0f) v[i][k] = -v[i][k];
                }
                split8<MX, QP>(v[i], qf[i]);
            }
        }

        float m = kLowest, l = 0.0f;
        // weights are exp2(score x times - base) of scores up to `limit`
        float limit = m, times = factor, base = m - bias;
        v4f_t o[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i] = v4f_t{0.0f, 0.0f, 0.0f, 0.0f};

        // Codes are loaded again as soon as they are converted: the next step's
        // are under way while one is multiplied, and the pages of the one after.
        for (; j < j1; j += team) {
            const int k32 = j * kStep;
            const bool holes[2] = {page[0] < 0, page[1] < 0};
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t there = k32 + 16 * t + col < q.length ? ~0u : 0u;  // (behind the end is no number)
                st.k[t].s &= there;
                st.v[t].s &= there;
                page[t] = page_of(next[t]);
            }
            // scores: register r of sub-tile t is key 16 t + 4 g4 + r of the column
            v4f_t sc[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                sc[t] = v4f_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < KD; ++i) {
                    const v8 a = values8<D, MX>(st.k[t], i);
#pragma unroll
                    for (int x = QP - 1; x >= 0; --x) sc[t] = F::mfma(a, qf[i][x], sc[t]);
                }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) st.k[t] = load(j + team, t, page[t], p.cache.k_codes, p.cache.k_scales);
            // V to LDS
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < KD; ++i)
                    *reinterpret_cast<v8*>(lds + (16 * t + col) * kRowBytes<D> + g4 * (D / 2) + 16 * i) = values8<D, MX>(st.v[t], i);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                st.v[t] = load(j + team, t, page[t], p.cache.v_codes, p.cache.v_scales);
                next[t] = find_entry(j + 2 * team, t);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (k32 + kStep - 1 > pos_first || k32 < low_last || holes[0] || holes[1]) {
                int first = k32;
                asm volatile("" : "+v"(first));  // (so that the compiler keeps the branch, and compares in few steps)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int key = first + 16 * t + 4 * g4 + r;
                        sc[t][r] = key <= pos && key >= low && !holes[t] ? sc[t][r] : -INFINITY;
                    }
            }
            float top = -INFINITY;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) top = fmaxf(top, sc[t][r]);
            {
                float a, b;
                row_pair(top, a, b);
                half_pair(fmaxf(a, b), a, b);
                top = fmaxf(a, b) * factor;
            }
            if (__any(top > limit)) {
                const float next = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - next);
                m = next;
                l *= f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[i][r] *= f;
                limit = m + kSlack;
                times = factor;
                base = m - bias;
                if (__any(fabsf(m) > kFar && m > kLowest)) {
                    limit = -INFINITY;
                    times = 1.0f;
                    base = -bias;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r) sc[t][r] = sc[t][r] * factor - m;
                }
            }
            float w[8];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) w[4 * t + r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][r], times, -base));
            v8 pf[PP];
            split8<MX, PP>(w, pf);
            l += sum8(w);
            asm volatile("" ::: "memory");
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                typedef __attribute__((address_space(3))) v4s_t lds_v4s;
                typedef short v8s_t __attribute__((ext_vector_type(8)));
                char* from = lds + (4 * g4 + (col >> 2)) * kRowBytes<D> + 32 * i + 8 * (col & 3);
                const v4s_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)from);
                const v4s_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(from + 16 * kRowBytes<D>));
                const v8s_t z = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
                for (int k = PP - 1; k >= 0; --k) o[i] = F::mfma(__builtin_bit_cast(v8, z), pf[k], o[i]);
            }
            asm volatile("" ::: "memory");
        }

        {
            float a, b;
            row_pair(l, a, b);
            half_pair(a + b, a, b);
            l = a + b;
        }
        const float v_scale = MX ? 1.0f : p.cache.v_scale[g.head];
        if (d.team == 1) {
            if (col < g.count && !idle) {
                const Mean<MX> mean(l, v_scale);
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    store_out<F32>(p, q, g, col, 16 * i + 4 * g4, mean(o[i][0], o[i][1], o[i][2], o[i][3]));
                if (p.lse && g4 == 0) store_lse(p, q, g, col, m, bias, l);
            }
            continue;
        }
        // the waves' sums, joined in order
        float* mine = reinterpret_cast<float*>(lds);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            *reinterpret_cast<v4f_t*>(mine + col * kMergeStride<D> + 16 * i + 4 * g4) = o[i];
        if (g4 == 0) {
            stats[0][wave][col] = m;
            stats[1][wave][col] = l;
        }
        __syncthreads();
        const bool whole = d.team || (from == 0 && to == q.real);
        float* slot = slot_of<D>(p, blockIdx.x, from == 0 ? 1 : 0);
        for (int i = 64 * member + lane; i < (idle ? 0 : g.count * (D / 4)); i += 64 * team) {
            const int cc = i / (D / 4), d4 = 4 * (i % (D / 4));
            float top = kLowest;
            for (int w = mine0; w < mine0 + team; ++w) top = fmaxf(top, stats[0][w][cc]);
            float total = 0.0f;
            v4f_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int w = mine0; w < mine0 + team; ++w) {
                const float f = __builtin_amdgcn_exp2f(stats[0][w][cc] - top);
                const v4f_t x = *reinterpret_cast<const v4f_t*>(reinterpret_cast<const float*>(kv_lds + w * kWaveBytes<D>) +
                                                                cc * kMergeStride<D> + d4);
                total += f * stats[1][w][cc];
#pragma unroll
                for (int r = 0; r < 4; ++r) sum[r] += f * x[r];
            }
            if (whole) {
                store_out<F32>(p, q, g, cc, d4, Mean<MX>(total, v_scale)(sum[0], sum[1], sum[2], sum[3]));
                if (p.lse && d4 == 0) store_lse(p, q, g, cc, top, bias, total);
            } else {
                *reinterpret_cast<v4f_t*>(slot + cc * D + d4) = sum;
                if (d4 == 0) {
                    slot[kCols * D + cc] = top;
                    slot[kCols * D + kCols + cc] = total;
                }
            }
        }
        __syncthreads();
        u = g.begin + g.entries;
    }
}

// LANES lanes add four elements of the n parts, a part in turn to a lane; items
// [i0, i1) of a segment's count x D / 4.
template <int LANES, typename Op>
__device__ __forceinline__ float reduce_lanes(float x, Op op) {
    if constexpr (LANES == 64) return reduce64(x, op);
    if constexpr (LANES == 16) return reduce16(x, op);
    if constexpr (LANES >= 2) x = op(x, lane_xor1(x));
    if constexpr (LANES == 4) x = op(x, lane_xor2(x));
    return x;
}

template <bool MX, bool F32, int D, int LANES, typename Part>
__device__ __forceinline__ void join_items(const KvAttention& p, const Seq& q, const Segment& g, float bias, float v_scale, int i0,
                                           int i1, int n, Part part) {
    const int at = threadIdx.x / LANES, k0 = threadIdx.x % LANES;
    for (int b = i0; b < i1; b += kThreads / LANES) {  // (the same in all lanes)
        const int i = min(b + at, i1 - 1), c = i / (D / 4), d = 4 * (i % (D / 4));
        float top = kLowest, total = 0.0f;
        v4f_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
        for (int k = k0; k < n; k += LANES) {
            const float* x = part(k);
            const float m = x[kCols * D + c], l = x[kCols * D + kCols + c];
            const v4f_t y = *reinterpret_cast<const v4f_t*>(x + c * D + d);
            const float next = fmaxf(top, m), f = __builtin_amdgcn_exp2f(top - next), e = __builtin_amdgcn_exp2f(m - next);
            total = total * f + l * e;
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[r] = sum[r] * f + y[r] * e;
            top = next;
        }
        const float most = reduce_lanes<LANES>(top, MaxOp()), e = __builtin_amdgcn_exp2f(top - most);
        total = reduce_lanes<LANES>(total * e, AddOp());
        const Mean<MX> mean(total, v_scale);
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[r] = mean(reduce_lanes<LANES>(sum[r] * e, AddOp()));
        if (k0 == 0 && b + at < i1) {
            store_out<F32>(p, q, g, c, d, sum);
            if (p.lse && d == 0) store_lse(p, q, g, c, most, bias, total);
        }
    }
}

template <bool MX, bool F32, int D>
__global__ void __launch_bounds__(kThreads) k_kv_join(const KvAttention p) {
    const Join j = *join_of<D, kShares<F32, D>>(p, blockIdx.x + 1);
    const int n = j.n;
    if (n == 0) return;
    Seq q = {};
    q.row = j.row;
    Segment g = {};
    g.head = j.head;
    g.first = j.first;
    g.count = j.count;
    const auto part = [&](int k) { return slot_of<D>(p, j.first_share + k, k == 0 ? 1 : 0); };
    const float v_scale = MX ? 1.0f : p.cache.v_scale[g.head];
    const int items = g.count * (D / 4), rank = j.rank;
    const int i0 = (int)((int64_t)items * rank / (n - 1)), i1 = (int)((int64_t)items * (rank + 1) / (n - 1));
    // (lanes for all items at once, but no more than have a part)
    if (n < 4 || i1 - i0 > 128) join_items<MX, F32, D, 1>(p, q, g, j.bias, v_scale, i0, i1, n, part);
    else if (n < 16 || i1 - i0 > 32) join_items<MX, F32, D, 4>(p, q, g, j.bias, v_scale, i0, i1, n, part);
    else if (n < 64 || i1 - i0 > 8) join_items<MX, F32, D, 16>(p, q, g, j.bias, v_scale, i0, i1, n, part);
    else join_items<MX, F32, D, 64>(p, q, g, j.bias, v_scale, i0, i1, n, part);
}

// ---------------------------------------------------------------- many rows
// k_kv_prefill: a workgroup has 32 columns to a wave and goes over 64 keys at a
// time, converted once for all of them into LDS.  S^T = K Q^T and O^T = V^T P^T by
// 32x32x16 MFMA; as in k_kv_attention the first product's sums are the second's
// operand as they lie.
//
// A wave alternates between two phases, with a barrier after each: the products of
// the tile before with V and of this one with K (matrix instructions), and this
// one's softmax and the conversion of a later tile (vector instructions).  The two
// waves of a SIMD are a phase apart, so that one's matrix instructions go with the
// other's vector instructions.  Keys are then converted two tiles ahead, values one,
// into three buffers each (D 256 has one wave to a SIMD: one tile ahead, one buffer).
// 8192 rows of 40 heads behind nothing, a causal half: D 128 731 to 766 us (with the
// waves' phases together 804 instead of 723): the matrix cores are busy in 39% of the
// cycles, vector instructions issue in 44%, both in 24%; the rest are the phases' ends and
// what their first instructions wait for.  Over MXFP4, whose weights have two parts, 875
// (52, 48 and 31%); D 64 532, where the softmax is twice as much beside a product (26, 49
// and 17%); D 256 2155, one wave to a SIMD (25, 36 and 2%, and LDS busy in 39% of the
// cycles, half of them conflicts).
template <int D>
constexpr int kPreWaves = D == 256 ? 4 : 8;
template <int D>
constexpr int kPreCols = 32 * kPreWaves<D>;
// K rows: 16 bytes after each put 16 rows' pieces of a 16-byte read in
// different banks; V rows: 64 bytes put 4 rows' 64-byte pieces there.
template <int D>
constexpr int kPreK = 2 * D + 16;
template <int D>
constexpr int kPreV = 2 * D + 64;
// Of a buffer; K's ends with 16 bytes, whether its keys 16 i and on have no page.
template <int D>
constexpr int kPreKBytes = kTile * kPreK<D> + 16;
template <int D>
constexpr int kPreVBytes = kTile * kPreV<D>;
template <int D>
constexpr int kPreBuffers = D == 256 ? 1 : 3;

typedef float v16f_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ v16f_t mfma32(v8h_t a, v8h_t b, v16f_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v16f_t mfma32(v8b_t a, v8b_t b, v16f_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// f(0) .. f(N - 1), each with its number as a constant.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void in_order(F f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        in_order<N, I + 1>(f);
    }
}

// Blocks of kPreCols columns of sequence s for a kv head.
template <int D>
__device__ __forceinline__ int pre_blocks(const KvAttention& p, int s) {
    int row, rows;
    kv_rows(p.plan, s, row, rows);
    const int64_t cols = (int64_t)rows * p.group;
    return cols > kFewColumns ? (int)((cols + kPreCols<D> - 1) / kPreCols<D>) : 0;
}

// Block `index` of all, the last ones first (they see the most keys): its
// sequence and number there; false past the end.
template <int D>
__device__ __forceinline__ bool pre_find(const KvAttention& p, int64_t index, int& s, int& block) {
    const int lane = threadIdx.x & 63;
    const auto blocks = [&](int b) { return b + lane < p.plan.seqs ? (int64_t)pre_blocks<D>(p, b + lane) : 0; };
    int64_t all = 0;
    for (int b = 0; b < p.plan.seqs; b += 64) all += from_lane(scan64(blocks(b)), 63);
    if (index >= all) return false;
    index = all - 1 - index;
    for (int b = 0;; b += 64) {
        const int64_t own = blocks(b), upto = scan64(own), sum = from_lane(upto, 63);
        if (index < sum) {
            const int l = __builtin_ctzll(__ballot(index < upto));
            s = __builtin_amdgcn_readfirstlane(b + l);
            block = __builtin_amdgcn_readfirstlane((int)(index - from_lane(upto - own, l)));
            return true;
        }
        index -= sum;
    }
}

// What a workgroup of k_kv_prefill does: columns `id` of a kv head (neighbouring
// workgroups have different heads, so that with 8 of them one head's keys stay
// in one XCD's L2) and the split-th of `parts` equal parts of its tiles, of which
// there are as many as leave each kLeastTiles; a workgroup past them has none.
// (40 heads of 128, 8 kv heads: 2048 rows take 91 us, 130 with parts of any size,
// which cost a slot's bytes each; 512 rows behind 3584 74 and 131; 64 behind 8128 56
// and 75.  Least parts of 8 or 24 tiles: 112 and 91, 105 and 89, 48 and 71.  A block's
// parts beside each other: 1024 rows 61 instead of 57, 512 behind 3584 105, three
// chunks behind up to 16384 402 instead of 408.)
constexpr int kLeastTiles = 16, kMostParts = 16;
static_assert(kLeastTiles >= kMostParts);  // so that parts of ceil(tiles / parts) tiles leave none without any
struct PreWork {
    Seq q;
    Segment g;
    int s, parts, from, to;  // tiles of keys
    int64_t slot;  // of the workspace
};

template <int D>
__device__ __forceinline__ bool pre_work(const KvAttention& p, int64_t id, int split, PreWork& w) {
    w.slot = id + split * p.blocks;
    w.g.head = (int)(id % p.cache.heads);
    int block;
    if (!pre_find<D>(p, id / p.cache.heads, w.s, block)) return false;
    kv_rows(p.plan, w.s, w.q.row, w.q.rows);
    w.q.length = kv_length(p.plan, w.s);
    w.g.first = block * kPreCols<D>;
    w.g.count = (int)min((int64_t)kPreCols<D>, (int64_t)w.q.rows * p.group - w.g.first);
    const int pos0 = w.q.length - w.q.rows;
    const int first = pos0 + w.g.first / p.group, last = pos0 + (w.g.first + w.g.count - 1) / p.group;
    const int low = p.window ? max(0, first - p.window + 1) / kTile : 0;
    const int tiles = last >= 0 && p.cache.pages > 0 ? last / kTile + 1 - low : 0;  // (without a page nothing is seen)
    w.parts = max(1, min(p.splits, tiles / kLeastTiles));
    if (split >= w.parts) return false;
    const int each = (tiles + w.parts - 1) / w.parts;
    w.from = low + min(tiles, split * each);
    w.to = low + min(tiles, (split + 1) * each);
    return true;
}

// A slot: [columns][D] of O, then the columns' maxima and sums.
template <int D>
constexpr int64_t kPreSlotFloats = (int64_t)kPreCols<D> * (D + 2);

template <bool MX, int D>
__global__ void __launch_bounds__(64 * kPreWaves<D>, kPreWaves<D> / 4) k_kv_prefill(const KvAttention p) {
    typedef Form<MX> F;
    typedef typename F::v8 v8;
    constexpr int W = kPreWaves<D>, PP = kPParts<MX, false>, EPT = D / W, KS = D / 16, DB = D / 32;
    constexpr int per = MX ? 32 : 16;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, h = lane >> 5;
    PreWork work;
    // (the last parts first: the first ones, which every block has, fill up behind them)
    const int split = p.splits - 1 - (int)(blockIdx.x / p.blocks);
    const int64_t id = blockIdx.x % p.blocks;
    if (!pre_work<D>(p, id, split, work)) return;
    const Seq& q = work.q;
    const Segment& g = work.g;
    const int pos0 = q.length - q.rows;
    // the lane's column, and the positions of its wave's
    const int wfirst = g.first + 32 * wave, wlast = min(wfirst + 31, g.first + g.count - 1);
    const bool idle = wfirst > wlast;
    const int c = min(wfirst + col, g.first + g.count - 1);
    const int qrow = c / p.group, qhead = g.head * p.group + c % p.group;
    const int pos = pos0 + qrow, low = p.window ? max(0, pos - p.window + 1) : 0;
    const int wpos_first = pos0 + wfirst / p.group, wpos_last = idle ? -1 : pos0 + wlast / p.group;
    const int wlow_first = p.window ? max(0, wpos_first - p.window + 1) : 0;
    const int wlow_last = p.window ? max(0, wpos_last - p.window + 1) : 0;

    const float bias = weight_bias<MX>(p, q.length);

    v8 qf[KS];
    float factor;
    {
        float v[KS][8];
        const uint16_t* src = static_cast<const uint16_t*>(p.q.data) + (q.row + qrow) * p.q.row + qhead * p.q.head + 8 * h;
#pragma unroll
        for (int i = 0; i < KS; ++i) load_upto8(src + 16 * i, 8, v[i]);
        int e = 15;
        if constexpr (!MX) {
            float top = 0.0f, a, b;
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[i][k]));
            half_pair(top, a, b);
            e = __builtin_amdgcn_frexp_expf(fmaxf(a, b));
        }
        factor = score_factor<MX>(p, g.head, e);
        // (the scale's sign goes with q, so that larger sums are larger scores)
#pragma unroll
        for (int i = 0; i < KS; ++i) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if constexpr (!MX) v[i][k] = ldexpf(v[i][k], 15 - e);
                if (p.scale < 0.0f) v[i][k] = -v[i][k];
            }
            split8<MX, 1>(v[i], &qf[i]);
        }
    }

    // what a thread loads of a tile: EPT elements of a key
    const int lkey = threadIdx.x / W, part = threadIdx.x % W;
    struct Raw {
        uint32_t w[EPT / 8], s;
    };
    const int slot_mask = (1 << p.plan.page_shift) - 1;
    const int j0 = work.from, j1 = work.to;
    // the table's entry for the thread's key of tile j, as it is loaded (past the end
    // the last key's), and where that key lies: some slot, and whether it is its own
    const auto find_entry = [&](int j) { return kv_entry(p.plan, work.s, min(j * kTile + lkey, q.length - 1)); };
    struct Place {
        int64_t slot;
        bool there;
    };
    const auto place_of = [&](int j, int entry) {
        const int key = j * kTile + lkey, page = kv_page_of(entry, p.cache.pages);
        return Place{(((int64_t)max(page, 0) * p.cache.heads + g.head) << p.plan.page_shift) + (key & slot_mask),
                     page >= 0 && key < q.length};
    };
    // (without a branch: scales of a key that is not there become zero when it is converted)
    const auto load = [&](int64_t slot, const uint8_t* codes, const uint8_t* scales) {
        Raw r;
        const uint8_t* c = codes + slot * (D / 2) + part * (EPT / 2);
        if constexpr (EPT == 8) {
            r.w[0] = *reinterpret_cast<const uint32_t*>(c);
        } else if constexpr (EPT == 16) {
            const uint2 x = *reinterpret_cast<const uint2*>(c);
            r.w[0] = x.x;
            r.w[1] = x.y;
        } else {
#pragma unroll
            for (int i = 0; i < EPT / 32; ++i) {
                const u4_t x = *reinterpret_cast<const u4_t*>(c + 16 * i);
#pragma unroll
                for (int k = 0; k < 4; ++k) r.w[4 * i + k] = x[k];
            }
        }
        const uint8_t* at = scales + slot * (D / per) + part * EPT / per;
        constexpr int n = EPT / per;
        if constexpr (n <= 1) r.s = *at;
        else if constexpr (n == 2) r.s = *reinterpret_cast<const h_align1*>(at);
        else r.s = *reinterpret_cast<const w_align1*>(at);
        return r;
    };
    char* const k_lds = kv_lds;
    char* const v_lds = kv_lds + kPreBuffers<D> * kPreKBytes<D>;
    const auto stage = [&](Raw r, bool there, char* to) {
        r.s = there ? r.s : 0u;
#pragma unroll
        for (int i = 0; i < EPT / 8; ++i)
            *reinterpret_cast<v8*>(to + part * (2 * EPT) + 16 * i) = F::values(r.w[i], (r.s >> (8 * (8 * i / per))) & 0xFFu);
    };
    const auto stage_k = [&](const Raw& r, bool there, int j, int b) {
        char* to = k_lds + b * kPreKBytes<D>;
        stage(r, there, to + lkey * kPreK<D>);
        if (part == 0 && (lkey & 15) == 0)
            *reinterpret_cast<int*>(to + kTile * kPreK<D> + lkey / 4) = !there && j * kTile + lkey < q.length;
    };
    const auto stage_v = [&](const Raw& r, bool there, int b) { stage(r, there, v_lds + b * kPreVBytes<D> + lkey * kPreV<D>); };

    float m, l;
    v16f_t o[DB], sc[2];
    v8 pf[4][PP];
    uint32_t holes = 0;  // bit i: keys 16 i and on of the tile have no page

    // The operands of the products are read from LDS kDepth products ahead, in the
    // order that is written here: left to itself the compiler reads each right before
    // its product, which then waits for it.
    constexpr int kDepth = 4;
    const auto pipelined = [&](auto count, auto read, auto product) {
        constexpr int N = decltype(count)::value;
        v8 a[N];
        in_order<kDepth>([&](auto n) { a[n] = read(n); });
        in_order<N>([&](auto n) {
            if constexpr (n + kDepth < N) a[n + kDepth] = read(std::integral_constant<int, n + kDepth>());
            __builtin_amdgcn_sched_barrier(0);
            product(n, a[n]);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    const auto times_k = [&](int b) {
        const char* kt = k_lds + b * kPreKBytes<D> + col * kPreK<D> + 16 * h;
        const u4_t flags = *reinterpret_cast<const u4_t*>(k_lds + b * kPreKBytes<D> + kTile * kPreK<D>);
        holes = __builtin_amdgcn_readfirstlane(flags[0] | flags[1] << 1 | flags[2] << 2 | flags[3] << 3);
        // product n: keys 32 (n % 2) and on, elements 16 (n / 2) and on
        pipelined(
            std::integral_constant<int, 2 * KS>(),
            [&](auto n) { return *reinterpret_cast<const v8*>(kt + 32 * (n % 2) * kPreK<D> + 32 * (n / 2)); },
            [&](auto n, v8 x) {
                const v16f_t zero = {};
                sc[n % 2] = mfma32(x, qf[n / 2], n / 2 == 0 ? zero : sc[n % 2]);
            });
    };
    const auto times_v = [&](int b) {
        const char* vt = v_lds + b * kPreVBytes<D> + (4 * h + ((lane & 15) >> 2)) * kPreV<D> + 32 * ((lane >> 4) & 1) + 8 * (lane & 3);
        // product n: keys 16 (n / DB) and on, elements 32 (n % DB) and on
        pipelined(
            std::integral_constant<int, 4 * DB>(),
            [&](auto n) {
                typedef __attribute__((address_space(3))) v4s_t lds_v4s;
                typedef short v8s_t __attribute__((ext_vector_type(8)));
                const char* at = vt + 16 * (n / DB) * kPreV<D> + 64 * (n % DB);
                const v4s_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)at);
                const v4s_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + 8 * kPreV<D>));
                const v8s_t z = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
                return __builtin_bit_cast(v8, z);
            },
            [&](auto n, v8 x) {
#pragma unroll
                for (int k = PP - 1; k >= 0; --k) o[n % DB] = mfma32(x, pf[n / DB][k], o[n % DB]);
            });
    };
    // (`also`: the rest of the phase, where the compiler mixes its instructions in: 704
    // us instead of 730 after it, 766 before the exponentials; prefill of 8192 rows)
    const auto softmax = [&](int j, auto exact, auto also) {
        constexpr bool kExact = decltype(exact)::value;
        const int key0 = j * kTile;
        if (holes || key0 + kTile - 1 > wpos_first || key0 < wlow_last) {
            int first = key0;
            asm volatile("" : "+v"(first));  // (so that the compiler keeps the branch, and compares in few tiles)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int key = first + 32 * t + 8 * (r >> 2) + 4 * h + (r & 3);
                    const bool seen = key <= pos && key >= low && !(holes >> (2 * t + (r >> 3)) & 1);
                    sc[t][r] = seen ? sc[t][r] : -INFINITY;
                }
        }
        float tops[4], a0, a1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            tops[i] = sc[i >> 1][8 * (i & 1)];
#pragma unroll
            for (int r = 1; r < 8; ++r) tops[i] = fmaxf(tops[i], sc[i >> 1][8 * (i & 1) + r]);
        }
        float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        half_pair(top, a0, a1);
        top = fmaxf(a0, a1) * factor;
        if (__any(top > (kExact ? m : m + kSlack))) {
            const float next = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - next);
            m = next;
            l *= f;
#pragma unroll
            for (int i = 0; i < DB; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[i][r] *= f;
        }
        const float base = m - bias;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float w[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float x = sc[u >> 1][8 * (u & 1) + r];
                w[r] = __builtin_amdgcn_exp2f(kExact ? (x * factor - m) + bias : __builtin_fmaf(x, factor, -base));
            }
            split8<MX, PP>(w, pf[u]);
            l += sum8(w);
        }
        also();
    };
    // (nothing is moved over a phase's end)
    const auto phase_end = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        lds_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };

    constexpr int NB = kPreBuffers<D>, KA = NB == 3 ? 2 : 1;  // tiles that keys are ahead (values: one less)
    const auto all_tiles = [&](auto exact) {
        m = kLowest;
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
        if (j0 >= j1) return;
        int entry[4];  // of the key in tiles j0 .. j0 + 3
#pragma unroll
        for (int i = 0; i < KA + 2; ++i) entry[i] = find_entry(j0 + i);
        Place at[3];
#pragma unroll
        for (int i = 0; i < KA + 1; ++i) at[i] = place_of(j0 + i, entry[i]);
        Raw rk[KA], rv;
#pragma unroll
        for (int i = 0; i < KA; ++i) rk[i] = load(at[i].slot, p.cache.k_codes, p.cache.k_scales);
        rv = load(at[0].slot, p.cache.v_codes, p.cache.v_scales);
        bool v_there = at[0].there;
#pragma unroll
        for (int i = 0; i < KA; ++i) stage_k(rk[i], at[i].there, j0 + i, i);
        // what is under way: keys of tile j + KA (at `k_at`), values of j + KA - 1; the
        // next keys' entry of the table
        Place k_at = at[KA];
        rk[0] = load(k_at.slot, p.cache.k_codes, p.cache.k_scales);
        if constexpr (KA == 2) {
            stage_v(rv, v_there, 0);
            rv = load(at[1].slot, p.cache.v_codes, p.cache.v_scales);
            v_there = at[1].there;
        }
        int next = entry[KA + 1];
        phase_end();
        if (NB == 3 && wave >= 4) phase_end();
        bool weights = false;  // of the tile before
        int b = 0;             // tile j's buffer
        for (int j = j0; j <= j1; ++j) {
            const bool active = j < j1 && j * kTile <= wpos_last && j * kTile + kTile > wlow_first;
            const int before = NB == 3 ? (b == 0 ? 2 : b - 1) : 0, after = NB == 3 ? (b == 2 ? 0 : b + 1) : 0;
            __builtin_amdgcn_s_setprio(1);
            if (weights) times_v(before);
            if (active) times_k(b);
            __builtin_amdgcn_s_setprio(0);
            phase_end();
            weights = active;
            if (j < j1) {
                const auto convert = [&]() {
                    stage_k(rk[0], k_at.there, j + KA, before);  // (of three, the buffer after the next is the one before)
                    stage_v(rv, v_there, after);
                    rv = load(k_at.slot, p.cache.v_codes, p.cache.v_scales);
                    v_there = k_at.there;
                    k_at = place_of(j + KA + 1, next);
                    rk[0] = load(k_at.slot, p.cache.k_codes, p.cache.k_scales);
                    next = find_entry(j + KA + 2);
                };
                if (active) softmax(j, exact, convert);
                else convert();
            }
            phase_end();
            b = after;
        }
        if (NB == 3 && wave < 4) phase_end();
    };
    // Where some score was far the tiles are gone over again, with exact differences: the
    // maximum is still far, or a weight that passed its type's largest has left what is no
    // number, which no later rescaling takes away.  (A choice between the two in every tile
    // cost 1 to 13% of the time, by where it stood.)
    __shared__ int some_far;
    if (threadIdx.x == 0) some_far = 0;
    all_tiles(std::false_type());
    const float seen_of_all = fabsf(l) + fabsf(o[0][0]);
    if ((fabsf(m) > kFar && m > kLowest) || !(seen_of_all < INFINITY)) some_far = 1;
    __syncthreads();
    if (some_far) all_tiles(std::true_type());
    {
        float a, b;
        half_pair(l, a, b);
        l = a + b;
    }
    const int lc = 32 * wave + col;  // column of the block
    if (lc >= g.count) return;
    if (work.parts > 1) {
        float* slot = p.pre_ws + work.slot * kPreSlotFloats<D>;
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *reinterpret_cast<v4f_t*>(slot + lc * D + 32 * i + 8 * r + 4 * h) =
                    v4f_t{o[i][4 * r], o[i][4 * r + 1], o[i][4 * r + 2], o[i][4 * r + 3]};
        if (h == 0) {
            slot[kPreCols<D> * D + lc] = m;
            slot[kPreCols<D> * (D + 1) + lc] = l;
        }
        return;
    }
    const Mean<MX> mean(l, MX ? 1.0f : p.cache.v_scale[g.head]);
#pragma unroll
    for (int i = 0; i < DB; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            store_out<false>(p, q, g, lc, 32 * i + 8 * r + 4 * h,
                             mean(o[i][4 * r], o[i][4 * r + 1], o[i][4 * r + 2], o[i][4 * r + 3]));
    if (p.lse && h == 0) store_lse(p, q, g, lc, m, bias, l);
}

// The parts of a block, joined in order: kJoinCols of its columns.
constexpr int kJoinCols = 32;
template <bool MX, int D>
__global__ void __launch_bounds__(kThreads) k_kv_prefill_join(const KvAttention p) {
    constexpr int pieces = kPreCols<D> / kJoinCols;
    PreWork work;
    const int64_t id = blockIdx.x / pieces;
    if (!pre_work<D>(p, id, 0, work) || work.parts == 1) return;
    const float v_scale = MX ? 1.0f : p.cache.v_scale[work.g.head], bias = weight_bias<MX>(p, work.q.length);
    const int c0 = (int)(blockIdx.x % pieces) * kJoinCols;
    for (int i = threadIdx.x; i < kJoinCols * (D / 4); i += kThreads) {
        const int cc = c0 + i / (D / 4), d = 4 * (i % (D / 4));
        if (cc >= work.g.count) return;
        float top = kLowest, total = 0.0f;
        v4f_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int k = 0; k < work.parts; ++k) {
            const float* slot = p.pre_ws + (id + k * p.blocks) * kPreSlotFloats<D>;
            const float l = slot[kPreCols<D> * (D + 1) + cc];
            const float m = slot[kPreCols<D> * D + cc], next = fmaxf(top, m);
            const float f = __builtin_amdgcn_exp2f(top - next), e = __builtin_amdgcn_exp2f(m - next);
            const v4f_t x = *reinterpret_cast<const v4f_t*>(slot + cc * D + d);
            total = total * f + l * e;
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[r] = sum[r] * f + x[r] * e;
            top = next;
        }
        store_out<false>(p, work.q, work.g, cc, d, Mean<MX>(total, v_scale)(sum[0], sum[1], sum[2], sum[3]));
        if (p.lse && d == 0) store_lse(p, work.q, work.g, cc, top, bias, total);
    }
}

// Blocks of one kv head at most, and the most parts of each: with fewer than 1024
// workgroups (four for each compute unit) a block's keys may be split.  (With up to 512
// three chunks behind up to 16384 positions took 408 us, with 1024 399, with 1280 419;
// with 1536, which splits the blocks of 4096 rows, these took 270 instead of 229.)
int64_t pre_blocks_most(int64_t rows, int64_t seqs, int group, int dim) {
    const int64_t cols = dim == 256 ? kPreCols<256> : kPreCols<128>;
    return rows * group / cols + std::min(seqs, rows * group / (kFewColumns + 1));
}

int pre_splits(int64_t rows, int64_t seqs, int group, int heads, int dim) {
    const int64_t blocks = pre_blocks_most(rows, seqs, group, dim) * heads;
    return (int)std::max<int64_t>(1, std::min<int64_t>(kMostParts, 1024 / std::max<int64_t>(1, blocks)));
}

template <bool MX, int D>
hipError_t run_prefill(KvAttention p, hipStream_t s) {
    constexpr int bytes = kPreBuffers<D> * (kPreKBytes<D> + kPreVBytes<D>);
    const int64_t blocks = pre_blocks_most(p.plan.rows, p.plan.seqs, p.group, D) * p.cache.heads;
    p.blocks = blocks;
    p.splits = pre_splits(p.plan.rows, p.plan.seqs, p.group, p.cache.heads, D);
    p.pre_ws = p.ws + kShares<false, D> * kShareFloats<D>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_kv_prefill<MX, D>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_kv_prefill<MX, D>), dim3((uint32_t)(blocks * p.splits)), dim3(64 * kPreWaves<D>), bytes, s, p);
    if (p.splits > 1)
        hipLaunchKernelGGL((k_kv_prefill_join<MX, D>), dim3((uint32_t)(blocks * (kPreCols<D> / kJoinCols))), dim3(kThreads), 0, s, p);
    return hipGetLastError();
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
    hipLaunchKernelGGL((k_kv_attention<MX, F32, D>), dim3(kShares<F32, D>), dim3(kThreads), bytes, s, p);
    hipLaunchKernelGGL((k_kv_join<MX, F32, D>), dim3(kShares<F32, D> - 1), dim3(kThreads), 0, s, p);
    if constexpr (!F32) {
        // (offsets may give all rows to one sequence)
        const int64_t most = p.plan.offsets ? (int64_t)p.plan.rows * p.group : p.group;
        if (most > kFewColumns) return run_prefill<MX, D>(p, s);
    }
    return hipGetLastError();
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t rows, int64_t seqs, int q_heads, int kv_heads, int dim, bool bf16) {
    if (rows == 0) return 0;
    int64_t floats = (dim == 256  ? kShares<false, 256> * kShareFloats<256>
                      : dim == 64 ? kShares<false, 64> * kShareFloats<64>
                      : bf16      ? kShares<false, 128> * kShareFloats<128>
                                  : kShares<true, 128> * kShareFloats<128>);
    const int group = q_heads / kv_heads;
    if (bf16 && rows * group > kFewColumns) {
        const int64_t cols = dim == 256 ? kPreCols<256> : kPreCols<128>;
        const int splits = pre_splits(rows, seqs, group, kv_heads, dim);
        if (splits > 1) floats += pre_blocks_most(rows, seqs, group, dim) * kv_heads * splits * cols * (dim + 2);
    }
    return (size_t)floats * sizeof(float);
}

hipError_t launch_kv_attention(const KvAttention& p, hipStream_t s) {
    if (p.plan.rows == 0 || p.plan.seqs == 0) return hipSuccess;
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
