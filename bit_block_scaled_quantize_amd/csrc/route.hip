// Routing of tokens to experts and its backward pass, for gfx950.
//
// Per token: scores p of its logits l (softmax over all experts, or the
// sigmoid of each), selection scores s = p + bias; with groups, the top_groups
// groups of the largest group score (the largest s, or the sum of the two
// largest) stay; the top_k experts of the largest s among them are chosen
// (ties to the lower index) and weighted by p, divided by the chosen ones' sum
// with renorm.  Without a bias experts, and groups by their largest, go by the
// logits themselves, in whose order their scores are.  The dispatch plan sorts the T * k assignments (token-major) by
// expert, stably: order (assignment at each sorted place), its inverse
// position, and offsets (the first place of each expert).
//
// Backward, with w the renormalised weights of the chosen i, D = sum_i dw_i w_i
// and ds the gradient of all scores:
//   softmax: dl_e = p_e (ds_e - sum_f p_f ds_f) + [e chosen] w_e (dw_e - D)
//   sigmoid: dl_e = (1 - p_e) (p_e ds_e + [e chosen] w_e (dw_e - D))
// (the division by the chosen sum cancels, so nothing is divided by a small
// number).
//
// The bytes are few (16384 tokens of 256 experts: 19 MB with the plan, 4 us);
// what bounds the choice is the instructions and the latency of top_k rounds
// of selection.  A token is shared by 16 lanes (4 tokens a wave) where they
// hold its scores, so a round's reduction is four register exchanges; a lane
// sorts its keys once, and a round takes the largest head.  Measured: 16384
// tokens, top 8 of 256 in 8 groups, sigmoid with bias, 27 to 29 us (choice 20 to
// 25, plan 7); top 4 of 32, softmax, 12.7 us (7 and 5); one token 8.7 us; 4096
// tokens of 512, 1024 and 2048 experts 18, 31 and 86; backward with score
// gradients, 16384 x 256 BF16, 10.3 us (3.3 TB/s), sigmoid 12.1.
//
// The kernels of 16 values on 16 lanes and of 32 on 64 keep some of them in
// scratch memory (15 and 64 registers).  Tokens that binary64 has to settle whole go
// one by one through a wave (choose_exactly): more near scores than candidates
// (binary32 logits all alike, 16384 x 256: 62 us, in groups 82; fewer live experts
// than top_k: 62), and sums of two scores that all lie below the binary32 scores'
// error (sigmoids of logits around -16 in groups without a bias: 79).  Experts and
// groups masked by a bias do not: 25 to 29.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch.hpp"
#include "nvfp4_device.hpp"
#include "row_device.hpp"

namespace nvfp4 {

namespace {

constexpr float kLowest = -3.402823466e38f;

// A logit as the operators read it: NaN and -inf count as the lowest finite
// value, +inf as the largest (their scores are then those of a masked and of
// a certain expert, and no row gives NaN).
__device__ __forceinline__ float logit(float l) { return __builtin_fminf(__builtin_fmaxf(l, kLowest), -kLowest); }

// Element i of a BF16 or binary32 array.
__device__ __forceinline__ float load1(const void* p, bool bf16, int64_t i) {
    return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16) : static_cast<const float*>(p)[i];
}

// From e^-|l|, which neither overflows nor leaves a small sigmoid's last bits out.
__device__ __forceinline__ float sigmoid32(float l) {
    const float e = expf(-fabsf(l));
    return (l < 0.0f ? e : 1.0f) / (1.0f + e);
}

// Scores for the choice alone, by the hardware's exponential and reciprocal (a
// unit in the last place each).  With U = 2^-24, an exponential e^-x of a
// difference is off by (2.2 x + 2) U of itself, under 2.1 U of 1 for every
// x >= 0, and the sigmoid, whose slope in log e is p (1 - p), by under 3.3 U.
__device__ __forceinline__ float quick_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }
__device__ __forceinline__ float quick_sigmoid(float l) { return __builtin_amdgcn_rcpf(1.0f + quick_exp(-l)); }

// exp(l - m) with the rounding error of the difference put back (the error of
// a binary32 difference is itself a binary32 value): a few ulp for any l <= m.
__device__ __forceinline__ float exp_diff(float l, float m) {
    const float d = l - m, z = d - l;
    const float err = (l - (d - z)) - (m + z);
    const float e = expf(d);
    return __builtin_isfinite(err) ? __builtin_fmaf(e, err, e) : e;
}

// The score of l by e^m, m the largest of the logits that share a sum: of
// sigmoids of negative logits, which are to be normalised and of which binary32
// may hold the quotients alone.
__device__ __forceinline__ float share(float l, float m, bool softmax) {
    const float e = exp_diff(l, m);
    return softmax ? e : e / (1.0f + expf(l));
}

// Reductions over the LPT (16, 32 or 64) lanes of a token, result in every lane.
template <int LPT, typename Op>
__device__ __forceinline__ float lanes_reduce(float x, Op op) {
    if constexpr (LPT == 16) return reduce16(x, op);
    if constexpr (LPT == 64) return reduce64(x, op);
    float a, b;
    row_pair(reduce16(x, op), a, b);
    return op(a, b);
}
template <int LPT>
__device__ __forceinline__ float lanes_max(float x) { return lanes_reduce<LPT>(x, MaxOp()); }
template <int LPT>
__device__ __forceinline__ int lanes_max(int x) {
    x = max(x, (int)lane_xor1((uint32_t)x));
    x = max(x, (int)lane_xor2((uint32_t)x));
    x = max(x, (int)quad_perm<0x141>((uint32_t)x));  // (mirrors, as reduce16)
    x = max(x, (int)quad_perm<0x140>((uint32_t)x));
    if constexpr (LPT >= 32) {
        const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        x = max((int)a[0], (int)a[1]);
    }
    if constexpr (LPT == 64) {
        const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        x = max((int)b[0], (int)b[1]);
    }
    return x;
}

// The bits of a ballot that belong to the caller's token, from bit 0.
template <int LPT>
__device__ __forceinline__ uint64_t own_bits(uint64_t mask) {
    if constexpr (LPT == 64) return mask;
    else return (mask >> (threadIdx.x & 63 & ~(LPT - 1))) & ((1ull << LPT) - 1);
}

// Elements p[0 .. min(n, V) - 1] as binary32 (what lies beyond stays as it was).
template <int V>
__device__ __forceinline__ void load_values(const void* p, bool bf16, int n, float v[V]) {
    if constexpr (V >= 8) {
#pragma unroll
        for (int c = 0; c < V; c += 8)
            if (c < n) {
                if (bf16) load_upto8(static_cast<const uint16_t*>(p) + c, n - c, v + c);
                else load_upto8(static_cast<const float*>(p) + c, n - c, v + c);
            }
    } else {
        typedef float fv_t __attribute__((ext_vector_type(V), aligned(4)));
        typedef uint16_t hv_t __attribute__((ext_vector_type(V), aligned(2)));
        if (n >= V && bf16) {
            const hv_t q = *static_cast<const hv_t*>(p);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = bf16_to_f32(q[j]);
        } else if (n >= V) {
            const fv_t q = *static_cast<const fv_t*>(p);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = q[j];
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < n) v[j] = load1(p, bf16, j);
        }
    }
}

// A selection score that compares: NaN and infinities as `logit` takes them.
template <typename F>
__device__ __forceinline__ F comparable(F s) {
    return fmin(fmax(s, (F)kLowest), (F)-kLowest);
}

// How far binary32 scores are off, counted twice (two are compared): a score
// of size x by tol(x).  Sigmoid: 3.3 U, and U x of the sum with the bias.
// Exponentials that are not divided by their sum: 2.1 U.  Softmax, p <= 1 /
// total: 2.1 U of that and the sum's relative error, 38 U of its additions and
// (2.2 x + 2) U of its terms, x = m - l, whose mean under p is at most log E < 8.
struct Tolerance {
    float absolute, relative;
    __device__ __forceinline__ float operator()(float x) const { return absolute + relative * x; }
};

// The error of a group's score x (+ y, unless -inf): those of x and y, each of
// its own size however much of it cancels in the sum, and a rounding of the sum
// and one of adding the error to it: absolute + 3 U (|x| + |y|), at most what
// the tolerance's two counts of 2 U give, 1.5 times.  A score that stands for an infinity is
// exact, and so is its sum with any under 2^70, which binary64 rounds away too.
__device__ __forceinline__ float sum_error(float x, float y, Tolerance tol) {
    const bool two = y > -__builtin_inff();
    const float ax = fabsf(x), ay = two ? fabsf(y) : 0.0f, most = fmaxf(ax, ay), least = fminf(ax, ay);
    if (most == -kLowest && (least < 0x1p70f || least == -kLowest)) return 0.0f;
    return tol.absolute + 1.5f * tol.relative * (ax + ay);
}

// Which groups stay, from a and b, the best and second best key of the
// caller's lane (-inf where there is none): `kept` tells whether the lane
// belongs to one of the top_groups groups of the largest group score (ties to
// the lower index).  score(a, b): the group score of a group's best two;
// error(a, b): how far it may be off.  Returns false where a group that stays
// and one that does not are nearer than their errors and not alike (`exact`:
// equal keys are equal scores; else equal ones without an error are).
template <int LPT, typename Score, typename Error>
__device__ __forceinline__ bool keep_groups(float a, float b, const RouteShape& g, Score score, Error error, bool exact,
                                            bool& kept) {
    const int lane = threadIdx.x & (LPT - 1), mine = lane >> g.lane_shift;
    const int first = threadIdx.x & 63 & ~(LPT - 1);  // the token's first lane of the wave
    for (int d = 1; d < 1 << g.lane_shift; d <<= 1) {
        const float a2 = __shfl_xor(a, d), b2 = __shfl_xor(b, d);
        b = fmaxf(fminf(a, a2), fmaxf(b, b2));
        a = fmaxf(a, a2);
    }
    const float gs = score(a, b), err = error(a, b);
    const bool is = mine < g.groups;
    int ahead = 0;  // groups before the own one
    for (int o = 0; o < g.groups; ++o) {
        const float q = __shfl(gs, first + (o << g.lane_shift));
        ahead += (q > gs || (q == gs && o < mine)) ? 1 : 0;
    }
    kept = is && ahead < g.top_groups;
    const float none = -__builtin_inff();
    const float least = -lanes_max<LPT>(kept ? err - gs : none), most = lanes_max<LPT>(is && !kept ? gs + err : none);
    // (a sum past binary32 has an infinite error: it may be any score)
    if (!__any(least <= most || (is && err == -none))) return true;
    bool certain = true;
    for (int o = 0; o < g.groups; ++o) {
        const int at = first + (o << g.lane_shift);
        const float qa = __shfl(a, at), qb = __shfl(b, at);
        const float mine_of = score(a, b), q = score(qa, qb), off = error(a, b) + error(qa, qb);
        const bool other = __shfl((int)kept, at) != (int)kept;
        const bool alike = exact ? qa == a && qb == b : q == mine_of && off == 0.0f;
        if (is && other && !(fabsf(q - mine_of) > off) && !alike) certain = false;
    }
    return certain;
}

// Integers in the order of binary32 values, and back (to the value of a key
// whose low bits are cleared).
__device__ __forceinline__ int ordered(float s) {
    const int b = (int)__float_as_uint(s + 0.0f);  // (-0 as 0)
    return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float value_of(int key) { return __uint_as_float((uint32_t)(key ^ ((key >> 31) & 0x7FFFFFFF))); }

constexpr int kNone = (int)0x80000000;  // below every key

constexpr int low_bits(int v) { return v <= 2 ? 1 : v <= 4 ? 2 : v <= 8 ? 3 : v <= 16 ? 4 : 5; }

// Exchanges of Batcher's odd-even merge sort of V values.
template <int V>
struct Exchanges {
    int n = 0;
    uint8_t lo[V * 8] = {}, hi[V * 8] = {};
    constexpr Exchanges() {
        for (int p = 1; p < V; p *= 2)
            for (int q = p; q >= 1; q /= 2)
                for (int j = q % p; j + q < V; j += 2 * q)
                    for (int i = 0; i < q && i + j + q < V; ++i)
                        if ((i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                            lo[n] = (uint8_t)(i + j);
                            hi[n++] = (uint8_t)(i + j + q);
                        }
    }
};

// The lane's keys, largest first.
template <int V>
__device__ __forceinline__ void sort_keys(int key[V]) {
    constexpr Exchanges<V> net;
#pragma unroll
    for (int c = 0; c < net.n; ++c) {
        const int a = key[net.lo[c]], b = key[net.hi[c]];
        key[net.lo[c]] = max(a, b);
        key[net.hi[c]] = min(a, b);
    }
}

// The next largest of the keys (sorted in each lane; it is taken out): goes to
// lane `it`, its expert to out[it].  WHOLE: a key's low 16 bits are the
// expert's index, from the end; else its low bits are the value's place in the
// lane, from the end, and of lanes with the same key the first is taken.
template <int LPT, int V, bool WHOLE>
__device__ __forceinline__ void take(int key[V], int it, int base, int* out, int& mine) {
    const int lane = threadIdx.x & (LPT - 1);
    const int M = lanes_max<LPT>(key[0]);
    if (lane == it) mine = M;
    bool win = key[0] == M;
    if constexpr (!WHOLE) {
        win = win && (own_bits<LPT>(__ballot(win)) & ((1ull << lane) - 1)) == 0;
        if (win) out[it] = base + V - 1 - (M & ((1 << low_bits(V)) - 1));
    }
    // (by bits: a choice between neighbours is compiled to indexing)
    const int up = win ? -1 : 0;
#pragma unroll
    for (int j = 0; j + 1 < V; ++j) key[j] = (key[j + 1] & up) | (key[j] & ~up);
    key[V - 1] = win ? kNone : key[V - 1];
}

// The largest of the wave's binary64 values, in every lane.
__device__ __forceinline__ double wave_max(double x) {
    x = fmax(x, quad_perm64<0xB1>(x));
    x = fmax(x, quad_perm64<0x4E>(x));
    x = fmax(x, quad_perm64<0x141>(x));
    x = fmax(x, quad_perm64<0x140>(x));
    x = fmax(x, __shfl_xor(x, 16));
    return fmax(x, __shfl_xor(x, 32));
}

// The selection score of expert c in binary64 (without a bias its logit, which
// orders alike): row, m, base and have as route_token has them.
template <int LPT>
__device__ __forceinline__ double exact_score(const RouteArgs& a, int64_t row, float m, int base, int have, int c) {
    const double x = (double)logit(load1(a.logits, a.bf16, row + c));
    if (!a.bias) return x;
    double sum = 1.0;
    if (!a.sigmoid) {
        sum = 0.0;
#pragma unroll 1
        for (int j = 0; j < have; ++j)
            sum += exp((double)logit(load1(a.logits, a.bf16, row + base + j)) - (double)m);
#pragma unroll
        for (int d = 1; d < LPT; d <<= 1) sum += __shfl_xor(sum, d);
    }
    const double e = exp(a.sigmoid ? -x : x - (double)m);
    return comparable((a.sigmoid ? 1.0 / (1.0 + e) : e / sum) + (double)a.bias[c]);
}

// The choice of one token by binary64 scores, by a whole wave: lane
// `to` + j gets the j-th chosen expert in place of id.  score: a row of LDS
// (experts doubles).
__device__ __forceinline__ int choose_exactly(const RouteArgs& a, int64_t t, double* score, int to, int id) {
    const RouteShape& g = a.shape;
    const int lane = threadIdx.x & 63, E = g.experts;
    const double none = -__builtin_inf();
    const int64_t row = t * a.ld;
    float m = kLowest;
    double total = 1.0;
    if (!a.sigmoid) {
#pragma unroll 1
        for (int e = lane; e < E; e += 64) m = fmaxf(m, logit(load1(a.logits, a.bf16, row + e)));
        m = lanes_max<64>(m);
        total = 0.0;
    }
#pragma unroll 1
    for (int e = lane; e < E; e += 64) {
        const double x = (double)logit(load1(a.logits, a.bf16, row + e));
        const double v = exp(a.sigmoid ? -x : x - (double)m);
        score[e] = a.sigmoid ? 1.0 / (1.0 + v) : v;
        if (!a.sigmoid) total += v;
    }
    if (!a.sigmoid) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
    }
#pragma unroll 1
    for (int e = lane; e < E; e += 64) {
        const double p = score[e] / total;
        score[e] = a.bias ? comparable(p + (double)a.bias[e]) : p;
        // (as on the quick path: without a bias only sums of two compare scores)
        if (!a.bias && !g.group_top2) score[e] = (double)logit(load1(a.logits, a.bf16, row + e));
    }
    __builtin_amdgcn_wave_barrier();
    if (g.top_groups < g.groups) {
        double best = none, second = none;
        if (lane < g.groups)
#pragma unroll 1
            for (int e = lane * g.group_size; e < (lane + 1) * g.group_size; ++e) {
                second = fmax(second, fmin(best, score[e]));
                best = fmax(best, score[e]);
            }
        const double gs = g.group_top2 && second > none ? best + second : best;
        int ahead = 0;
#pragma unroll 1
        for (int o = 0; o < g.groups; ++o) {
            const double q = __shfl(gs, o);
            ahead += (q > gs || (q == gs && o < lane)) ? 1 : 0;
        }
        const uint64_t kept = __ballot(lane < g.groups && ahead < g.top_groups);
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int e = lane; e < E; e += 64)
            if (!(kept >> (e / g.group_size) & 1)) score[e] = none;
    }
    // without a bias, the kept experts by their logits
    if (!a.bias)
#pragma unroll 1
        for (int e = lane; e < E; e += 64)
            if (score[e] > none) score[e] = (double)logit(load1(a.logits, a.bf16, row + e));
#pragma unroll 1
    for (int it = 0; it < g.top_k; ++it) {
        double best = none;
        int at = E;
#pragma unroll 1
        for (int e = lane; e < E; e += 64)
            if (const double v = score[e]; v > best) {
                best = v;
                at = e;
            }
        const double most = wave_max(best);
        at = -lanes_max<64>(best == most ? -at : -E);
        if (lane == to + it) id = at;
        if ((at & 63) == lane) score[at] = none;
    }
    __builtin_amdgcn_wave_barrier();
    return id;
}

// One wave's tokens, 64 / LPT of them: the caller's lane group has token t.
// Returns lane j < top_k's chosen expert and weight.  out: a row of LDS for
// the token; exact: one for the wave.
template <int LPT, int V>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, int* out, double* exact, int& id,
                                            float& weight) {
    const RouteShape& g = a.shape;
    const int lane = threadIdx.x & (LPT - 1);
    const int grp = lane >> g.lane_shift, li = lane & ((1 << g.lane_shift) - 1);
    const int base = grp * g.group_size + li * V;
    int have = grp < g.groups ? max(0, min(V, g.group_size - li * V)) : 0;
    // (opaque, or V comparisons of it are kept in scalar registers throughout)
    asm volatile("" : "+v"(have));
    const int64_t row = t * a.ld;
    const float none = -__builtin_inff();
    float s[V];
    load_values<V>(static_cast<const char*>(a.logits) + (row + base) * (a.bf16 ? 2 : 4), a.bf16, have, s);
    float m = kLowest;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s[j] = j < have ? logit(s[j]) : none;
        m = fmaxf(m, s[j]);
    }
    const bool softmax = !a.sigmoid, by_group = g.top_groups < g.groups;
    float total = 1.0f;
    if (softmax) {
        m = lanes_max<LPT>(m);
        if (!a.renorm) {  // the sum is part of the weights
            total = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) total += exp_diff(s[j], m);
            total = lanes_reduce<LPT>(total, AddOp());
        } else if (a.bias) {
            total = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) total += quick_exp(s[j] - m);
            total = lanes_reduce<LPT>(total, AddOp());
        }
    }
    // Without a bias the scores grow with the logits, which are compared
    // instead.  With one, binary32 scores decide wherever they are further
    // apart than their error; nearer ones are settled in binary64 (16384
    // tokens of 256 experts: some tens).
    const float inv_total = 1.0f / total;
    const Tolerance tol = {softmax && a.bias ? 0x1p-17f * inv_total : 0x1p-21f, 0x1p-23f};
    if (a.bias) {
        if (softmax) {
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = quick_exp(s[j] - m) * inv_total;
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = quick_sigmoid(s[j]);
        }
        float b[V];
#pragma unroll
        for (int j = 0; j < V; ++j) b[j] = 0.0f;
        load_values<V>(a.bias + base, false, have, b);
        asm volatile("" : "+v"(have));
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = j < have ? comparable(s[j] + b[j]) : none;
    }
    bool certain = true;
    if (by_group) {
        float best = none, second = none;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            second = fmaxf(second, fminf(best, s[j]));
            best = fmaxf(best, s[j]);
        }
        bool kept;
        if (!g.group_top2 && !a.bias) {
            keep_groups<LPT>(best, second, g, [](float x, float) { return x; }, [](float, float) { return -1.0f; }, true, kept);
        } else if (a.bias) {
            const bool two = g.group_top2;
            certain = keep_groups<LPT>(best, second, g, [=](float x, float y) { return two && y > none ? x + y : x; },
                                       [=](float x, float y) { return sum_error(x, two ? y : none, tol); }, false, kept);
        } else {
            const auto p = [=](float l) { return softmax ? quick_exp(l - m) : quick_sigmoid(l); };
            certain = keep_groups<LPT>(best, second, g, [=](float x, float y) { return y > none ? p(x) + p(y) : p(x); },
                                       [=](float x, float y) { return sum_error(p(x), y > none ? p(y) : none, tol); }, true, kept);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = kept ? s[j] : none;
    }
    // The keys: without a bias of BF16 logits, the logit's 16 bits over the
    // expert's index, exact and distinct (less 1, which keeps the binary32 limits
    // that stand for infinities apart from BF16's largest); else the upper bits of the binary32
    // score over its place in the lane, 2^-19 of the score with 16 a lane.
    const int k = g.top_k;
    int key[V], last = kNone;
    if (a.bf16 && !a.bias) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            key[j] = s[j] == none ? kNone : ((ordered(s[j]) - 1) & ~0xFFFF) | (0xFFFF - (base + j));
        sort_keys<V>(key);
        for (int it = 0; it < k; ++it) take<LPT, V, true>(key, it, base, out, last);
        id = lane < k ? 0xFFFF - (last & 0xFFFF) : 0;
    } else {
        constexpr int low = (1 << low_bits(V)) - 1;
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = s[j] == none ? kNone : (ordered(s[j]) & ~low) | (V - 1 - j);
        sort_keys<V>(key);
        // one more than top_k, to see how far the next one is behind
        for (int it = 0; it <= k; ++it) take<LPT, V, false>(key, it, base, out, last);
        // the steps of the keys, and the scores' own error where they are not exact
        const Tolerance step = {a.bias ? tol.absolute + 0x1p-120f : 0x1p-120f, (float)(low + 2) * 0x1p-23f};
        const float at = value_of(last & ~low);
        const float before = __shfl_up(at, 1, LPT);
        const bool near = lane > 0 && lane <= k && last != kNone && before - at <= step(fmaxf(fabsf(before), fabsf(at)));
        __builtin_amdgcn_wave_barrier();
        if (__any(near)) {
            // near ones change places by their scores in binary64; candidates
            // are added until the next one is out of the k-th's reach
            int n = k + 1;
            const float kth = __shfl(at, k - 1, LPT);
            bool open = own_bits<LPT>(__ballot(near && lane == k)) != 0;
            while (n < min(LPT, kMaxTopK + 1) && __any(open)) {
                take<LPT, V, false>(key, n, base, out, last);
                const float next = value_of(__shfl(last, n, LPT) & ~low);
                open = open && __shfl(last, n, LPT) != kNone && kth - next <= step(fmaxf(fabsf(kth), fabsf(next)));
                ++n;
            }
            certain &= !open;
            __builtin_amdgcn_wave_barrier();
            const bool in = lane < n && last != kNone;
            const int c = in ? out[lane] : 0;
            const double score = exact_score<LPT>(a, row, m, base, have, c);
            int ahead = 0;
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const double o = __shfl(score, i, LPT);
                const int oc = __shfl(c, i, LPT), there = __shfl((int)in, i, LPT);
                ahead += (there && (o > score || (o == score && oc < c))) ? 1 : 0;
            }
            __builtin_amdgcn_wave_barrier();
            if (in && ahead <= k) out[ahead] = c;
            __builtin_amdgcn_wave_barrier();
        }
        id = lane < k ? out[lane] : 0;
    }
    // a token whose lanes are not all certain
    uint64_t open = __ballot(!certain);
#pragma clang loop unroll(disable)
    while (open) {
        const int u = (__ffsll((unsigned long long)open) - 1) & ~(LPT - 1);  // its first lane
        id = choose_exactly(a, __shfl(t, u), exact, u, id);
        open = LPT == 64 ? 0 : open & ~(((1ull << (LPT & 63)) - 1) << u);
    }
    // the chosen scores from their logits
    const bool mine = lane < g.top_k;
    const float lc = mine ? logit(load1(a.logits, a.bf16, row + id)) : none;
    if (a.renorm) {
        const float mc = lanes_max<LPT>(lc);
        float p = 0.0f;
        if (!softmax && mine) p = sigmoid32(lc);
        const bool by_exp = softmax || mc < 0.0f;
        if (__any(by_exp) && mine && by_exp) p = share(lc, mc, softmax);
        weight = p / lanes_reduce<LPT>(p, AddOp());
    } else {
        weight = !mine ? 0.0f : softmax ? exp_diff(lc, m) / total : sigmoid32(lc);
    }
}

// Exclusive prefix sum of v[0 .. n) in LDS by the workgroup, in place; returns
// the total.  tmp: an int for each wave.
__device__ __forceinline__ int exclusive_scan(int* v, int n, int* tmp) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int per = (n + blockDim.x - 1) / blockDim.x, b = threadIdx.x * per;
    int sum = 0;
    for (int j = 0; j < per; ++j)
        if (b + j < n) sum += v[b + j];
    int upto = sum;  // over the wave's lanes up to the own one
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int x = __shfl_up(upto, d);
        if (lane >= d) upto += x;
    }
    if (lane == 63) tmp[wv] = upto;
    __syncthreads();
    int run = upto - sum, total = 0;
    for (int w = 0; w < waves; ++w) {
        const int x = tmp[w];
        if (w < wv) run += x;
        total += x;
    }
    for (int j = 0; j < per; ++j)
        if (b + j < n) {
            const int x = v[b + j];
            v[b + j] = run;
            run += x;
        }
    __syncthreads();
    return total;
}

// Experts of a row of counts (bytes), rounded up so that rows are 16-byte aligned.
__host__ __device__ __forceinline__ int count_row(int experts) { return (experts + 15) / 16 * 16; }

// LDS of k_route, in 4-byte words: a row of choices for each token, a row of
// binary64 scores for each wave; with the plan a count and a mask of 64 tokens
// for each expert and a word for each wave.
__host__ __device__ __forceinline__ int route_lds_words(int experts, int waves, int lpt, bool plan) {
    return waves * (64 / lpt * (kMaxTopK + 1) + 2 * (experts + 1)) + (plan ? 3 * experts + waves : 0);
}

extern __shared__ __attribute__((aligned(16))) int route_lds[];

// Threads of a workgroup at most: with 1024, a thread has 128 registers.
__host__ __device__ constexpr int most_threads(int lpt, int v) { return lpt == 32 && v == 16 ? 512 : 1024; }

// The choice over the tokens of span blockIdx.x, 64 / LPT for each wave at a
// time.  With the plan, position gets the rank of each assignment among those
// of its expert in the span (the experts of a token are distinct: the bits of
// the tokens before it in the expert's mask, and the count of earlier rounds),
// and counts[span][expert] their number; a lone workgroup (a round of tokens: a
// second launch would cost more than its work) goes on to the sorted places.
template <int LPT, int V>
__global__ void __launch_bounds__(most_threads(LPT, V)) k_route(const RouteArgs a) {
    const int E = a.shape.experts, k = a.shape.top_k;
    const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6, lane = threadIdx.x & (LPT - 1);
    const int u = threadIdx.x / LPT, round = blockDim.x / LPT;
    double* exact = reinterpret_cast<double*>(route_lds) + wave * (E + 1);
    int* out = route_lds + 2 * waves * (E + 1) + u * (kMaxTopK + 1);
    int* count = route_lds + 2 * waves * (E + 1) + round * (kMaxTopK + 1);
    uint32_t* mask = reinterpret_cast<uint32_t*>(count + E);  // low and high words
    int* tmp = count + 3 * E;
    const bool plan = a.offsets != nullptr;
    const int64_t t0 = (int64_t)blockIdx.x * a.span, t1 = min(t0 + a.span, a.tokens);
    if (plan) {
        for (int e = threadIdx.x; e < 3 * E; e += blockDim.x) count[e] = 0;
        __syncthreads();
    }
#pragma unroll 1
    for (int64_t r = t0; r < t1; r += round) {
        const int64_t t = r + u;
        int id = 0;
        float w;
        // (tokens past the end repeat the last one)
        route_token<LPT, V>(a, min(t, t1 - 1), out, exact, id, w);
        const bool mine = t < t1 && lane < k;
        if (mine) {
            a.ids[t * k + lane] = id;
            a.weights[t * k + lane] = w;
            if (plan) atomicOr(mask + 2 * id + (u >> 5), 1u << (u & 31));  // (the order does not matter)
        }
        if (!plan) continue;
        __syncthreads();
        int rank = 0;
        if (mine) {
            const uint32_t lo = mask[2 * id], hi = mask[2 * id + 1], below = (1u << (u & 31)) - 1;
            rank = count[id] + (u < 32 ? __popc(lo & below) : __popc(lo) + __popc(hi & below));
            if (gridDim.x > 1) a.position[t * k + lane] = rank;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += blockDim.x) {
            count[e] += __popc(mask[2 * e]) + __popc(mask[2 * e + 1]);
            mask[2 * e] = mask[2 * e + 1] = 0;
        }
        __syncthreads();
        if (gridDim.x == 1) {  // (one round: all assignments are ranked)
            const int sum = exclusive_scan(count, E, tmp);
            if (mine) {
                const int i = (int)t * k + lane, p = count[id] + rank;
                a.position[i] = p;
                a.order[p] = i;
            }
            for (int e = threadIdx.x; e < E; e += blockDim.x) a.offsets[e] = count[e];
            if (threadIdx.x == 0) a.offsets[E] = sum;
        }
    }
    if (!plan || gridDim.x == 1) return;
    const int row = count_row(E);
    uint8_t* counts = a.counts + (int64_t)blockIdx.x * row;
    for (int e = threadIdx.x; e < row; e += blockDim.x) counts[e] = e < E ? (uint8_t)count[e] : (uint8_t)0;
}

// Parts of the spans that k_route_places sums side by side.
__host__ __device__ __forceinline__ int route_parts(int row) { return min(1024 / (row / 4), 32); }

// Sorted places of the assignments of spans [blockIdx.x * a.group, + a.group):
// every workgroup sums the spans' counts itself (all of them for the experts'
// offsets, those before its own for its places) instead of waiting for a scan
// in a launch between.  A thread sums 4 experts (a word of bytes, as two pairs
// of 16 bits) over one part of the spans; the parts are added through LDS.
__global__ void __launch_bounds__(1024) k_route_places(const RouteArgs a, int spans) {
    const int E = a.shape.experts, k = a.shape.top_k, row = count_row(E), words = row / 4, parts = route_parts(row);
    int* total = route_lds;     // assignments of each expert, then its first place
    int* before = total + row;  // those of earlier spans, then the next place
    int* tmp = before + row;    // 16
    int* all_of = tmp + 16;     // parts x row
    int* pre_of = all_of + parts * row;
    const int first = blockIdx.x * a.group, c = threadIdx.x % words, part = threadIdx.x / words;
    if (part < parts) {
        const uint32_t* counts = reinterpret_cast<const uint32_t*>(a.counts) + c;
        const int per = (spans + parts - 1) / parts, b0 = part * per, b1 = min(b0 + per, spans);
        int sum[4] = {}, pre[4] = {};
        const auto add = [&](int b, int end) {
            while (b < end) {
                uint32_t even = 0, odd = 0;
                const int stop = min(end, b + 256);
#pragma unroll 8
                for (; b < stop; ++b) {
                    const uint32_t w = counts[(int64_t)b * words];
                    even += w & 0x00FF00FFu;
                    odd += (w >> 8) & 0x00FF00FFu;
                }
                sum[0] += even & 0xFFFFu;
                sum[1] += odd & 0xFFFFu;
                sum[2] += even >> 16;
                sum[3] += odd >> 16;
            }
        };
        const int mid = max(b0, min(b1, first));
        add(b0, mid);
#pragma unroll
        for (int j = 0; j < 4; ++j) pre[j] = sum[j];
        add(mid, b1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            all_of[part * row + 4 * c + j] = sum[j];
            pre_of[part * row + 4 * c + j] = pre[j];
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < row; e += blockDim.x) {
        int sum = 0, pre = 0;
#pragma unroll 8
        for (int q = 0; q < parts; ++q) {
            sum += all_of[q * row + e];
            pre += pre_of[q * row + e];
        }
        total[e] = sum;
        before[e] = pre;
    }
    __syncthreads();
    const int sum = exclusive_scan(total, E, tmp);
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        before[e] += total[e];
        if (blockIdx.x == 0) a.offsets[e] = total[e];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[E] = sum;
    for (int b = first; b < min(first + a.group, spans); ++b) {
        __syncthreads();
        const int64_t i1 = min((b + 1) * a.span, a.tokens) * k;
        for (int64_t i = b * a.span * k + threadIdx.x; i < i1; i += blockDim.x) {
            const int p = before[a.ids[i]] + a.position[i];
            a.position[i] = p;
            a.order[p] = (int)i;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += blockDim.x) before[e] += a.counts[(int64_t)b * row + e];
    }
}

// ---------------------------------------------------------------- backward
// LPT lanes a token, NC chunks of 8 consecutive experts a lane (chunk c of lane
// i starts at 8 (c LPT + i)); the chosen experts' logits are read from, and
// their terms added through, a row of LDS per token.
template <typename T, int LPT, int NC>
__global__ void __launch_bounds__(64) k_route_backward(const RouteBackward a) {
    constexpr int W = LPT * NC * 8;  // row of LDS: covers the experts
    __shared__ __attribute__((aligned(16))) float chosen[64 / LPT][W];
    const int lane = threadIdx.x & (LPT - 1), u = threadIdx.x / LPT;
    const int64_t tt = (int64_t)blockIdx.x * (64 / LPT) + u;
    const bool live = tt < a.tokens;
    const int64_t t = live ? tt : a.tokens - 1;
    const int E = a.experts;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    float l[NC][8], ds[NC][8];
    float m = kLowest;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int e = 8 * (c * LPT + lane), n = E - e;
#pragma unroll
        for (int j = 0; j < 8; ++j) l[c][j] = ds[c][j] = 0.0f;
        if (n > 0) {
            load_upto8(row + e, n, l[c]);
            if (a.dscores) load_upto8(a.dscores + t * a.ldds + e, n, ds[c]);
        }
    }
    // the chosen experts: lane i < k holds one (an index out of range has none)
    int id = -1;
    float dw = 0.0f;
    if (lane < a.top_k) {
        id = a.ids[t * a.top_k + lane];
        dw = a.dweights[t * a.top_k + lane];
    }
    const bool mine = id >= 0 && id < E;
    dw = mine ? dw : 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int e = 8 * (c * LPT + lane), n = E - e;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            l[c][j] = j < n ? logit(l[c][j]) : -__builtin_inff();
            m = fmaxf(m, l[c][j]);
            chosen[u][e + j] = l[c][j];
        }
    }
    __syncthreads();  // (one wave)
    const float lc = mine ? chosen[u][id] : -__builtin_inff();
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) chosen[u][8 * (c * LPT + lane) + j] = 0.0f;
    float total = 1.0f;
    const bool softmax = !a.sigmoid;
    if (softmax) {
        m = lanes_max<LPT>(m);
        total = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                l[c][j] = exp_diff(l[c][j], m);
                total += l[c][j];
            }
        total = lanes_reduce<LPT>(total, AddOp());
    }
    // q = 1 - p of the sigmoid, without cancellation
    const float pc = !mine ? 0.0f : softmax ? exp_diff(lc, m) / total : sigmoid32(lc);
    const float qc = softmax ? 1.0f : sigmoid32(-lc);
    float S = 0.0f, term;
    if (a.renorm) {
        const float mc = fmaxf(lanes_max<LPT>(lc), kLowest);
        const bool by_exp = softmax || mc < 0.0f;
        float w = !mine ? 0.0f : by_exp ? share(lc, mc, softmax) : pc;
        const float sum = lanes_reduce<LPT>(w, AddOp());
        w = mine ? w / sum : 0.0f;
        const float D = lanes_reduce<LPT>(dw * w, AddOp());
        term = w * (dw - D) * qc;
    } else {
        term = pc * dw * qc;
        if (softmax) S = lanes_reduce<LPT>(pc * dw, AddOp());
    }
    __syncthreads();  // (one wave; the rows are cleared)
    if (mine) chosen[u][id] = term;
    __syncthreads();
    if (softmax) {
        const float inv = 1.0f / total;
        float acc = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                l[c][j] *= inv;
                acc = __builtin_fmaf(l[c][j], ds[c][j], acc);
            }
        S += lanes_reduce<LPT>(acc, AddOp());
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int e = 8 * (c * LPT + lane), n = E - e;
        if (n <= 0 || !live) continue;
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float extra = chosen[u][e + j];
            if (softmax) d[j] = __builtin_fmaf(l[c][j], ds[c][j] - S, extra);
            else d[j] = __builtin_fmaf(sigmoid32(l[c][j]) * sigmoid32(-l[c][j]), ds[c][j], extra);
        }
        store_upto8(static_cast<T*>(a.dlogits) + t * a.lddl + e, n, d);
    }
}

inline int64_t r_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Lanes per token and values per lane for a routing shape; {0, 0} when the
// groups do not fit.  A group's experts lie on LPT / (groups rounded up to a
// power of two) lanes, in index order, so that the lowest lane and the lowest
// value among equal ones is the lowest expert.  Fewer lanes do less work a
// token (12616 of 304 experts in 8 groups: 41.6 us with 32, 63 with 64), 64 come to its end sooner: those where the tokens are few.
struct LaneShape {
    int lpt, v, per_group;
};
LaneShape lane_shape(int experts, int groups, int top_k, int64_t tokens) {
    int slots = 1;
    while (slots < groups) slots *= 2;
    for (int lpt : {16, 32, 64}) {
        if (slots > lpt || (lpt < 64 && tokens <= 256) || (lpt == 16 && top_k >= 16)) continue;
        const int per = lpt / slots, need = (int)r_cdiv(experts / groups, per);
        for (int v : {2, 4, 8, 16, 32}) {
            // (32 lanes: what 16 of them cannot hold)
            if (lpt == 16 ? v > 16 : lpt == 32 ? v < 8 || v > 16 : v < 4) continue;
            if (need <= v) return {lpt, v, per};
        }
    }
    return {0, 0, 0};
}

// Threads of a workgroup: as many as have their waves' rows of binary64 scores
// in 32 KiB of LDS.
int route_threads(int experts) { return experts <= 256 ? 1024 : experts <= 512 ? 512 : experts <= 1024 ? 256 : 128; }

// Tokens of a span: a round of its workgroup, or as many rounds as leave at
// most 256 spans, but no more than a byte counts.
int64_t route_span_tokens(int64_t tokens, int round) {
    return std::min<int64_t>(r_cdiv(r_cdiv(tokens, 256), round) * round, 192);
}

template <int LPT, int V>
hipError_t route_shaped(RouteArgs a, hipStream_t s) {
    const int E = a.shape.experts;
    int threads = std::min(route_threads(E), most_threads(LPT, V));
    if (a.tokens * LPT < threads) threads = std::max<int>((int)r_cdiv(a.tokens * LPT, 64) * 64, std::min(threads, 256));
    const int round = threads / LPT;
    a.span = route_span_tokens(a.tokens, round);
    const int spans = (int)r_cdiv(a.tokens, a.span);
    const size_t lds = route_lds_words(E, threads / 64, LPT, a.offsets != nullptr) * sizeof(int);
    // (spans that one grid cannot hold, over 4 million, go in equal parts: none
    // of them is a lone workgroup, which would make the plan by itself)
    const int64_t parts = r_cdiv(spans, max_blocks(threads)), per = r_cdiv(spans, parts);
    for (int64_t first = 0; first < spans; first += per) {
        const int64_t n = std::min(per, spans - first), t = first * a.span;
        RouteArgs part = a;
        part.logits = static_cast<const char*>(a.logits) + t * a.ld * (a.bf16 ? 2 : 4);
        part.ids += t * a.shape.top_k;
        part.weights += t * a.shape.top_k;
        if (a.offsets) {
            part.position += t * a.shape.top_k;
            part.counts += first * count_row(E);
        }
        part.tokens = std::min(n * a.span, a.tokens - t);
        hipLaunchKernelGGL((k_route<LPT, V>), dim3((unsigned)n), dim3(threads), lds, s, part);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!a.offsets || spans == 1) return hipSuccess;
    a.group = (int)r_cdiv(spans, 256);
    hipLaunchKernelGGL(k_route_places, dim3((unsigned)r_cdiv(spans, a.group)), dim3(1024),
                       (2 * count_row(E) * (1 + route_parts(count_row(E))) + 16) * sizeof(int), s, a, spans);
    return hipGetLastError();
}

hipError_t route_lanes(const RouteArgs& a, LaneShape ls, hipStream_t s) {
    if (ls.lpt == 16) {
        switch (ls.v) {
            case 2: return route_shaped<16, 2>(a, s);
            case 4: return route_shaped<16, 4>(a, s);
            case 8: return route_shaped<16, 8>(a, s);
            default: return route_shaped<16, 16>(a, s);
        }
    }
    if (ls.lpt == 32) return ls.v == 8 ? route_shaped<32, 8>(a, s) : route_shaped<32, 16>(a, s);
    switch (ls.v) {
        case 4: return route_shaped<64, 4>(a, s);
        case 8: return route_shaped<64, 8>(a, s);
        case 16: return route_shaped<64, 16>(a, s);
        default: return route_shaped<64, 32>(a, s);
    }
}

template <typename T>
hipError_t route_backward_typed(RouteBackward a, hipStream_t s) {
    const int lpt = a.experts <= 512 ? 16 : 64, nc = (int)r_cdiv(a.experts, 8 * lpt);
    // (tokens that one grid cannot hold: over 2^28, of more than 512 experts 2^26)
    const int64_t most = max_blocks(64) * (64 / lpt);
    if (a.tokens > most) {
        RouteBackward rest = a;
        a.tokens = most;
        rest.tokens -= most;
        rest.dweights += most * a.top_k;
        rest.ids += most * a.top_k;
        rest.logits = static_cast<const T*>(a.logits) + most * a.ld;
        rest.dlogits = static_cast<T*>(a.dlogits) + most * a.lddl;
        if (a.dscores) rest.dscores += most * a.ldds;
        const hipError_t e = route_backward_typed<T>(rest, s);
        if (e != hipSuccess) return e;
    }
    const dim3 g((unsigned)r_cdiv(a.tokens, 64 / lpt));
    if (lpt == 16) {
        if (nc <= 1) hipLaunchKernelGGL((k_route_backward<T, 16, 1>), g, dim3(64), 0, s, a);
        else if (nc <= 2) hipLaunchKernelGGL((k_route_backward<T, 16, 2>), g, dim3(64), 0, s, a);
        else hipLaunchKernelGGL((k_route_backward<T, 16, 4>), g, dim3(64), 0, s, a);
    } else {
        if (nc <= 2) hipLaunchKernelGGL((k_route_backward<T, 64, 2>), g, dim3(64), 0, s, a);
        else hipLaunchKernelGGL((k_route_backward<T, 64, 4>), g, dim3(64), 0, s, a);
    }
    return hipGetLastError();
}

__global__ void k_zero_offsets(int64_t* offsets, int n) {
    for (int i = threadIdx.x; i < n; i += 64) offsets[i] = 0;
}

}  // namespace

bool route_shape_fits(int experts, int groups) { return lane_shape(experts, groups, kMaxTopK, 1).lpt != 0; }

size_t route_workspace_bytes(int64_t tokens, int experts) {
    // (a workgroup's round is least with 64 lanes a token)
    const int round = route_threads(experts) / 64;
    return tokens <= round ? 0 : (size_t)(r_cdiv(tokens, route_span_tokens(tokens, round)) * count_row(experts));
}

hipError_t launch_route(RouteArgs a, hipStream_t s) {
    if (a.tokens == 0) {
        if (!a.offsets) return hipSuccess;
        hipLaunchKernelGGL(k_zero_offsets, dim3(1), dim3(64), 0, s, a.offsets, a.shape.experts + 1);
        return hipGetLastError();
    }
    const LaneShape ls = lane_shape(a.shape.experts, a.shape.groups, a.shape.top_k, a.tokens);
    a.shape.lane_shift = __builtin_ctz((unsigned)ls.per_group);
    return route_lanes(a, ls, s);
}

hipError_t launch_route_backward(const RouteBackward& a, bool bf16, hipStream_t s) {
    if (a.tokens == 0) return hipSuccess;
    return bf16 ? route_backward_typed<uint16_t>(a, s) : route_backward_typed<float>(a, s);
}

}  // namespace nvfp4
