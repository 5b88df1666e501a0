// Routing of tokens to experts and its backward pass, for gfx950.
//
// Per token: scores p of its logits l (softmax over all experts, or the
// sigmoid of each), selection scores s = p + bias; with groups, the top_groups
// groups of the largest group score (the largest s, or the sum of the two
// largest) stay; the top_k experts of the largest s among them are chosen
// (ties to the lower index) and weighted by p, divided by the chosen ones' sum
// with renorm.  The dispatch plan sorts the T * k assignments (token-major) by
// expert, stably: order (assignment at each sorted place), its inverse
// position, and offsets (the first place of each expert).
//
// Backward, with w the renormalised weights of the chosen i, D = sum_i dw_i w_i
// and ds the gradient of all scores:
//   softmax: dl_e = p_e (ds_e - sum_f p_f ds_f) + [e chosen] w_e (dw_e - D)
//   sigmoid: dl_e = (1 - p_e) (p_e ds_e + [e chosen] w_e (dw_e - D))
// (the division by the chosen sum cancels, so nothing is divided by a small
// number).
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

__device__ __forceinline__ float sigmoid32(float l) { return 1.0f / (1.0f + expf(-l)); }

// exp(l - m) with the rounding error of the difference put back (the error of
// a binary32 difference is itself a binary32 value): a few ulp for any l <= m.
__device__ __forceinline__ float exp_diff(float l, float m) {
    const float d = l - m, z = d - l;
    const float err = (l - (d - z)) - (m + z);
    const float e = expf(d);
    return __builtin_isfinite(err) ? __builtin_fmaf(e, err, e) : e;
}

// Reductions over the LPT (16 or 64) lanes of a token, result in every lane.
template <int LPT, typename Op>
__device__ __forceinline__ float lanes_reduce(float x, Op op) {
    return LPT == 16 ? reduce16(x, op) : reduce64(x, op);
}
template <int LPT>
__device__ __forceinline__ float lanes_max(float x) { return lanes_reduce<LPT>(x, MaxOp()); }
template <int LPT>
__device__ __forceinline__ double lanes_max(double x) {
#pragma unroll
    for (int d = 1; d < LPT; d <<= 1) x = fmax(x, __shfl_xor(x, d));
    return x;
}
template <int LPT>
__device__ __forceinline__ double lanes_sum(double x) {
#pragma unroll
    for (int d = 1; d < LPT; d <<= 1) x += __shfl_xor(x, d);
    return x;
}

// The bits of a ballot that belong to the caller's token, from bit 0.
template <int LPT>
__device__ __forceinline__ uint64_t own_bits(uint64_t mask) {
    if constexpr (LPT == 64) return mask;
    else return (mask >> (threadIdx.x & 48)) & 0xFFFFull;
}

// Which groups stay: `kept` tells whether the caller's lane belongs to one of
// the top_groups groups of the largest group score (ties to the lower index).
// s: the selection scores, V a lane, -inf where there is none.  Returns false
// where two group scores are nearer than tol(x) of a score of size x, twice
// what they may be off by (negative: exact).
template <typename F, int LPT, int V, typename Tol>
__device__ __forceinline__ bool keep_groups(const F s[V], const RouteShape& g, Tol tol, bool& kept) {
    const F none = -(F)__builtin_inf();
    const int lane = threadIdx.x & (LPT - 1), mine = lane / g.lanes_per_group;
    // the group's best two scores
    F a = none, b = none;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        b = fmax(b, fmin(a, s[j]));
        a = fmax(a, s[j]);
    }
    for (int d = 1; d < g.lanes_per_group; d <<= 1) {
        const F a2 = __shfl_xor(a, d), b2 = __shfl_xor(b, d);
        b = fmax(fmin(a, a2), fmax(b, b2));
        a = fmax(a, a2);
    }
    const F gs = (g.group_top2 && b > none) ? a + b : a;
    int ahead = 0;  // groups before the own one
    bool certain = true;
    for (int o = 0; o < g.groups; ++o) {
        const F q = __shfl(gs, (threadIdx.x & 63 & ~(LPT - 1)) + o * g.lanes_per_group);
        ahead += (q > gs || (q == gs && o < mine)) ? 1 : 0;
        if (mine < g.groups && o != mine && fabs(q - gs) <= tol(fmax(fabs(q), fabs(gs)))) certain = false;
    }
    kept = mine < g.groups && ahead < g.top_groups;
    return certain;
}

// The top_k largest of the keys s (V a lane, -inf where there is none; used
// up), ties to the lower index: lane j < top_k gets the j-th one's expert in
// id.  Returns as keep_groups does.
template <typename F, int LPT, int V, typename Tol>
__device__ __forceinline__ bool choose(F s[V], const RouteShape& g, int base, Tol tol, int& id) {
    const F none = -(F)__builtin_inf();
    const int lane = threadIdx.x & (LPT - 1);
    bool certain = true;
    F last = 0;
    id = 0;
    for (int it = 0; it <= g.top_k; ++it) {
        F m = s[0];
#pragma unroll
        for (int j = 1; j < V; ++j) m = fmax(m, s[j]);
        const F M = lanes_max<LPT>(m);
        if (it > 0 && M > none && last - M <= tol(fmax(fabs(last), fabs(M)))) certain = false;
        if (it == g.top_k) break;
        last = M;
        const uint64_t has = own_bits<LPT>(__ballot(m == M));
        const int win = __ffsll((unsigned long long)has) - 1;
        int at = 0;
        if (lane == win) {
            bool done = false;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (!done && s[j] == M) {
                    done = true;
                    at = base + j;
                    s[j] = none;
                }
        }
        at = __shfl(at, (threadIdx.x & 63 & ~(LPT - 1)) + win);
        if (lane == it) id = at;
    }
    return certain;
}

// A selection score that compares: NaN and infinities as `logit` takes them.
template <typename F>
__device__ __forceinline__ F comparable(F s) {
    return fmin(fmax(s, (F)kLowest), (F)-kLowest);
}

// One wave's tokens (64 / LPT of them from t0): lane group u's token is t0 + u;
// tokens past the end repeat the last one.  Returns lane j < top_k's chosen
// expert and weight.
template <int LPT, int V>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, int& id, float& weight) {
    const RouteShape& g = a.shape;
    const int lane = threadIdx.x & (LPT - 1);
    const int grp = lane / g.lanes_per_group, li = lane % g.lanes_per_group;
    const int base = grp * g.group_size + li * V;
    const int have = grp < g.groups ? max(0, min(V, g.group_size - li * V)) : 0;
    const int64_t row = t * a.ld;
    float l[V];
    if constexpr (V >= 8) {
#pragma unroll
        for (int c = 0; c < V / 8; ++c) {
            const int64_t at = row + base + 8 * c;
            if (8 * c >= have)
#pragma unroll
                for (int j = 0; j < 8; ++j) l[8 * c + j] = 0.0f;
            else if (a.bf16) load_upto8(static_cast<const uint16_t*>(a.logits) + at, have - 8 * c, l + 8 * c);
            else load_upto8(static_cast<const float*>(a.logits) + at, have - 8 * c, l + 8 * c);
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] = j < have ? load1(a.logits, a.bf16, row + base + j) : 0.0f;
    }
    float m = kLowest;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        l[j] = j < have ? logit(l[j]) : -__builtin_inff();
        m = fmaxf(m, l[j]);
    }
    const bool softmax = !a.sigmoid;
    float total = 1.0f;
    if (softmax) {
        m = lanes_max<LPT>(m);
        if (a.bias || !a.renorm) {
            total = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) total += exp_diff(l[j], m);
            total = lanes_reduce<LPT>(total, AddOp());
        }
    }
    // Without a bias the scores grow with the logits, so single experts (and
    // groups judged by their best one) are compared by the logits themselves,
    // exactly.  Elsewhere binary32 scores decide wherever they are further
    // apart than twice their error, and a wave with a nearer pair takes them
    // in binary64 (16384 tokens of 256 experts with a bias: a few waves).
    const bool by_group = g.top_groups < g.groups;
    const bool need_scores = a.bias || (by_group && g.group_top2);
    const float none = -__builtin_inff();
    bool kept = true, certain = true;
    float s[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s[j] = l[j];
        if (need_scores && j < have) {
            const float p = softmax ? exp_diff(l[j], m) / total : sigmoid32(l[j]);
            s[j] = a.bias ? comparable(p + a.bias[base + j]) : p;
        }
    }
    // sigmoid: p <= 1 within 2^-22; softmax: p = e / total, the sum's relative
    // error (at most 2^-19) common to all p <= 1 / total
    const float abs_tol = softmax ? 0x1p-18f / total : 0x1p-20f;
    const auto tol = [=](float x) { return need_scores ? abs_tol + 0x1p-20f * x : -1.0f; };
    if (by_group) {
        certain = keep_groups<float, LPT, V>(s, g, [=](float x) { return 2.0f * tol(x); }, kept);
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] = !kept ? none : a.bias ? s[j] : l[j];
    }
    if (a.bias) certain &= choose<float, LPT, V>(s, g, base, tol, id);
    if (__any(!certain)) {
        const double nothing = -__builtin_inf();
        double sd[V];
        double tot = 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const double x = (double)l[j];
            sd[j] = j >= have ? 0.0 : softmax ? exp(x - (double)m) : 1.0 / (1.0 + exp(-x));
            tot += sd[j];
        }
        tot = lanes_sum<LPT>(tot);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const double p = softmax ? sd[j] / tot : sd[j];
            sd[j] = j >= have ? nothing : a.bias ? comparable(p + (double)a.bias[base + j]) : p;
        }
        const auto exact = [](double) { return -1.0; };
        if (by_group) keep_groups<double, LPT, V>(sd, g, exact, kept);
        if (a.bias) {
#pragma unroll
            for (int j = 0; j < V; ++j) sd[j] = kept ? sd[j] : nothing;
            choose<double, LPT, V>(sd, g, base, exact, id);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] = kept ? l[j] : none;
        }
    }
    if (!a.bias) choose<float, LPT, V>(s, g, base, [](float) { return -1.0f; }, id);
    // the chosen scores from their logits
    const bool mine = lane < g.top_k;
    const float lc = mine ? logit(load1(a.logits, a.bf16, row + id)) : -__builtin_inff();
    float p;
    if (a.renorm) {
        const float mc = lanes_max<LPT>(lc);
        // sigmoids so small that their logits' exponentials are the same to
        // 2^-64 are normalised as those (binary32 would underflow)
        const bool by_exp = softmax || mc < -64.0f;
        p = !mine ? 0.0f : by_exp ? exp_diff(lc, mc) : sigmoid32(lc);
        p = p / lanes_reduce<LPT>(p, AddOp());
    } else {
        p = !mine ? 0.0f : softmax ? exp_diff(lc, m) / total : sigmoid32(lc);
    }
    weight = p;
}

// Chosen experts and weights of tokens [t0, t1) by one workgroup of 256
// threads, counted by expert into count[] (LDS, cleared here) when given.
template <int LPT, int V>
__device__ __forceinline__ void route_span(const RouteArgs& a, int64_t t0, int64_t t1, int* count) {
    constexpr int TPB = 256 / LPT;
    const RouteShape& g = a.shape;
    if (count) {
        for (int e = threadIdx.x; e < g.experts; e += 256) count[e] = 0;
        __syncthreads();
    }
    const int lane = threadIdx.x & (LPT - 1);
    for (int64_t t = t0 + threadIdx.x / LPT; t - threadIdx.x / LPT < t1; t += TPB) {
        int id;
        float w;
        route_token<LPT, V>(a, t < t1 ? t : t1 - 1, id, w);
        if (t < t1 && lane < g.top_k) {
            a.ids[t * g.top_k + lane] = id;
            a.weights[t * g.top_k + lane] = w;
            if (count) atomicAdd(count + id, 1);  // (integer: the order does not matter)
        }
    }
}

// Exclusive prefix sum of v[0 .. n) in LDS by 256 threads, in place; returns
// the total.  tmp: 256 ints.
__device__ __forceinline__ int exclusive_scan(int* v, int n, int* tmp) {
    const int per = (n + 255) / 256, b = threadIdx.x * per;
    int sum = 0;
    for (int j = 0; j < per; ++j)
        if (b + j < n) sum += v[b + j];
    tmp[threadIdx.x] = sum;
    __syncthreads();
    for (int d = 1; d < 256; d <<= 1) {
        const int x = threadIdx.x >= d ? tmp[threadIdx.x - d] : 0;
        __syncthreads();
        tmp[threadIdx.x] += x;
        __syncthreads();
    }
    int run = tmp[threadIdx.x] - sum;
    const int total = tmp[255];
    for (int j = 0; j < per; ++j)
        if (b + j < n) {
            const int x = v[b + j];
            v[b + j] = run;
            run += x;
        }
    __syncthreads();
    return total;
}

// Sorted places of assignments [a0, a1), next[e] (LDS) the place of the next
// assignment of expert e.  Each wave finds, for its 64 assignments, the lanes
// of the same expert by one ballot per bit of the expert's index; a table of
// the four waves' counts puts the waves in order.  wave_count: 4 * experts
// ints, zero.
__device__ __forceinline__ void place_span(const RouteArgs& a, int64_t a0, int64_t a1, int* next, int* wave_count) {
    const int E = a.shape.experts, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    for (int64_t c = a0; c < a1; c += 256) {
        const int64_t i = c + threadIdx.x;
        const bool in = i < a1;
        const int id = in ? a.ids[i] : 0;
        uint64_t same = __ballot(in);
        for (int b = 1; b < E; b <<= 1) {
            const uint64_t m = __ballot((id & b) != 0);
            same &= (id & b) ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1)), n = __popcll(same);
        const bool leader = in && rank == 0;
        if (leader) wave_count[wv * E + id] = n;
        __syncthreads();
        if (in) {
            int p = next[id] + rank;
            for (int w = 0; w < wv; ++w) p += wave_count[w * E + id];
            a.position[i] = p;
            a.order[p] = (int)i;
        }
        __syncthreads();
        if (leader) {
            atomicAdd(next + id, n);
            wave_count[wv * E + id] = 0;
        }
        __syncthreads();
    }
}

extern __shared__ int route_lds[];

// Choice over the tokens of span blockIdx.x, and counts[span][expert] for the
// plan.  A lone workgroup (few tokens: a second launch would cost more than
// its work) goes on to the sorted places itself.
template <int LPT, int V>
__global__ void __launch_bounds__(256) k_route(const RouteArgs a) {
    const int E = a.shape.experts;
    const int64_t t0 = (int64_t)blockIdx.x * a.span, t1 = min(t0 + a.span, a.tokens);
    int* count = a.offsets ? route_lds : nullptr;
    route_span<LPT, V>(a, t0, t1, count);
    if (!count) return;
    __syncthreads();  // (and the chosen ids, written by this workgroup, are read back below)
    if (gridDim.x > 1) {
        for (int e = threadIdx.x; e < E; e += 256) a.counts[(int64_t)blockIdx.x * E + e] = count[e];
        return;
    }
    int* waves = count + E;
    int* tmp = waves + 4 * E;
    for (int e = threadIdx.x; e < 4 * E; e += 256) waves[e] = 0;
    const int sum = exclusive_scan(count, E, tmp);
    for (int e = threadIdx.x; e < E; e += 256) a.offsets[e] = count[e];
    if (threadIdx.x == 0) a.offsets[E] = sum;
    place_span(a, 0, a.tokens * a.shape.top_k, count, waves);
}

// Sorted places of span blockIdx.x's assignments: every workgroup sums the
// spans' counts itself (all of them for the experts' offsets, those before it
// for its own places) instead of waiting for a scan in a launch between.
__global__ void __launch_bounds__(256) k_route_places(const RouteArgs a, int spans) {
    const int E = a.shape.experts;
    int* total = route_lds;       // E: assignments of each expert, then its first place
    int* before = total + E;      // E: those of earlier spans, then the next place
    int* waves = before + E;      // 4 E
    int* tmp = waves + 4 * E;     // 256
    for (int e = threadIdx.x; e < E; e += 256) {
        int all = 0, pre = 0;
#pragma unroll 8
        for (int b = 0; b < spans; ++b) {
            const int n = a.counts[(int64_t)b * E + e];
            all += n;
            pre += b < (int)blockIdx.x ? n : 0;
        }
        total[e] = all;
        before[e] = pre;
    }
    for (int e = threadIdx.x; e < 4 * E; e += 256) waves[e] = 0;
    __syncthreads();
    const int sum = exclusive_scan(total, E, tmp);
    for (int e = threadIdx.x; e < E; e += 256) {
        before[e] += total[e];
        if (blockIdx.x == 0) a.offsets[e] = total[e];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[E] = sum;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * a.span, t1 = min(t0 + a.span, a.tokens);
    place_span(a, t0 * a.shape.top_k, t1 * a.shape.top_k, before, waves);
}

// ---------------------------------------------------------------- backward
// LPT lanes a token, NC chunks of 8 consecutive experts a lane (chunk c of lane
// i starts at 8 (c LPT + i)); the chosen experts' terms are added through a row
// of LDS per token.
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
        for (int j = 0; j < 8; ++j) {
            l[c][j] = ds[c][j] = 0.0f;
            chosen[u][e + j] = 0.0f;
        }
        if (n > 0) {
            load_upto8(row + e, n, l[c]);
            if (a.dscores) load_upto8(a.dscores + t * a.ldds + e, n, ds[c]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            l[c][j] = j < n ? logit(l[c][j]) : -__builtin_inff();
            m = fmaxf(m, l[c][j]);
        }
    }
    // the chosen experts: lane i < k holds one (an index out of range has none)
    const int id = lane < a.top_k ? a.ids[t * a.top_k + lane] : -1;
    const bool mine = id >= 0 && id < E;
    const float lc = mine ? logit(load1(row, sizeof(T) == 2, id)) : -__builtin_inff();
    const float dw = mine ? a.dweights[t * a.top_k + lane] : 0.0f;
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
        const bool by_exp = softmax || mc < -64.0f;
        float w = !mine ? 0.0f : by_exp ? exp_diff(lc, mc) : pc;
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
// value among equal ones is the lowest expert.
struct LaneShape {
    int lpt, v, per_group;
};
LaneShape lane_shape(int experts, int groups) {
    int slots = 1;
    while (slots < groups) slots *= 2;
    for (int lpt : {16, 64}) {
        if (slots > lpt) continue;
        const int per = lpt / slots, need = (int)r_cdiv(experts / groups, per);
        for (int v : {2, 4, 8, 16, 32})
            if (need <= v) return {lpt, lpt == 64 ? std::max(v, 8) : v, per};
    }
    return {0, 0, 0};
}

// Tokens of one workgroup's span: a multiple of 16, at most 256 spans.
int64_t route_span_tokens(int64_t tokens) { return r_cdiv(r_cdiv(tokens, 256), 16) * 16; }

constexpr int64_t kSmallTokens = 32;  // one workgroup takes both steps up to here

template <int LPT, int V>
hipError_t route_shaped(RouteArgs a, hipStream_t s) {
    const size_t E = (size_t)a.shape.experts;
    a.span = a.tokens <= kSmallTokens ? a.tokens : route_span_tokens(a.tokens);
    const int spans = (int)r_cdiv(a.tokens, a.span);
    hipLaunchKernelGGL((k_route<LPT, V>), dim3((unsigned)spans), dim3(256), (5 * E + 256) * sizeof(int), s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.offsets || spans == 1) return e;
    hipLaunchKernelGGL(k_route_places, dim3((unsigned)spans), dim3(256), (6 * E + 256) * sizeof(int), s, a, spans);
    return hipGetLastError();
}

hipError_t route_lanes(const RouteArgs& a, LaneShape ls, hipStream_t s) {
    if (ls.lpt == 16) {
        switch (ls.v) {
            case 2: return route_shaped<16, 2>(a, s);
            case 4: return route_shaped<16, 4>(a, s);
            case 8: return route_shaped<16, 8>(a, s);
            case 16: return route_shaped<16, 16>(a, s);
            default: return route_shaped<16, 32>(a, s);
        }
    }
    switch (ls.v) {
        case 8: return route_shaped<64, 8>(a, s);
        case 16: return route_shaped<64, 16>(a, s);
        default: return route_shaped<64, 32>(a, s);
    }
}

template <typename T>
hipError_t route_backward_typed(const RouteBackward& a, hipStream_t s) {
    const int lpt = a.experts <= 512 ? 16 : 64, nc = (int)r_cdiv(a.experts, 8 * lpt);
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

bool route_shape_fits(int experts, int groups) { return lane_shape(experts, groups).lpt != 0; }

int64_t route_workspace_ints(int64_t tokens, int experts) {
    if (tokens <= kSmallTokens) return 0;
    return r_cdiv(tokens, route_span_tokens(tokens)) * experts;
}

hipError_t launch_route(RouteArgs a, hipStream_t s) {
    if (a.tokens == 0) {
        if (!a.offsets) return hipSuccess;
        hipLaunchKernelGGL(k_zero_offsets, dim3(1), dim3(64), 0, s, a.offsets, a.shape.experts + 1);
        return hipGetLastError();
    }
    const LaneShape ls = lane_shape(a.shape.experts, a.shape.groups);
    a.shape.lanes_per_group = ls.per_group;
    return route_lanes(a, ls, s);
}

hipError_t launch_route_backward(const RouteBackward& a, bool bf16, hipStream_t s) {
    if (a.tokens == 0) return hipSuccess;
    return bf16 ? route_backward_typed<uint16_t>(a, s) : route_backward_typed<float>(a, s);
}

}  // namespace nvfp4
