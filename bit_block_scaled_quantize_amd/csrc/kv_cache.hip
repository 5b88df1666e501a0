// Appending keys and values to the paged 4-bit cache, with the rotation of their
// positions, and reading them back, for gfx950.
//
// Both go over (row, head) pairs: a head of D elements takes D / 16 lanes of 16
// elements each, so that a wave has 16, 8 or 4 heads of one row (D 64, 128,
// 256) at a time, and its position and page are the same in all its lanes.  A
// wave has some rows (whose places it finds together, one to a lane) and some of
// their heads, the loads of the next heads under way while some are converted.
// Bound by HBM: 16384 BF16 rows of 40 heads of q and 8 of k and v, D 128, NVFP4, are
// appended with rotation in 94 us, 4.5 TB/s read and written, and read back in 18;
// binary32 ones in 162, 5.1 TB/s, and 43 (a large copy: 5.04).  A few rows are bound by
// launch and latency: kernels of 3.3 and 2.5 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "kv_device.hpp"
#include "launch.hpp"
#include "nvfp4_device.hpp"
#include "row_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

// Byte offset of slot `slot` of head h of a page, in units of `width` bytes a slot.
__device__ __forceinline__ int64_t slot_at(const KvCache& c, int page_shift, int page, int h, int slot, int width) {
    return ((((int64_t)page * c.heads + h) << page_shift) + slot) * width;
}

// The block's scale byte and the multiplier of its elements (rules of
// include/nvfp4.h; NVFP4 with the head's float as tensor scale).  A block that is not
// finite gets the largest scale that a finite one may have, so that its elements are
// numbers (6 x 2^126 is none) for the rows that attend to others beside them.
template <bool MX>
__device__ __forceinline__ BlockScale kv_block_scale(float amax, float head_scale) {
    BlockScale bs;
    if constexpr (MX) {
        const int s = max(min((int)(__float_as_uint(amax) >> 23), 254) - 127 - 2, -127);
        bs.byte = (uint32_t)(s + 127);
        bs.R = __uint_as_float((uint32_t)(127 - s) << 23);
    } else {
        bs.byte = e4m3_encode(amax / (6.0f * head_scale));
        bs.R = block_multiplier(bs.byte, head_scale);
    }
    return bs;
}

__device__ __forceinline__ float absmax8(const float v[8]) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
    return m;
}

// (a, b) turned by the angle of cosine c and sine s: each product and each sum
// rounded once.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float x = a * c - b * s;
    b = b * c + a * s;
    a = x;
}

// 16 elements of a head as they are loaded: 8 from each of two places.
template <typename T>
struct Raw {
    u4_align2 w[sizeof(T)];  // BF16: two of 16 bytes; binary32: four
};

template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* a, const T* b) {
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
        r.w[i] = *reinterpret_cast<const u4_align2*>(a + 4 * i);
        r.w[sizeof(T) / 2 + i] = *reinterpret_cast<const u4_align2*>(b + 4 * i);
    }
    return r;
}

// The 8 elements of place i.
template <typename T>
__device__ __forceinline__ void unpack_raw(const Raw<T>& r, int i, float v[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 2) {
            v[2 * j] = __uint_as_float(r.w[i][j] << 16);
            v[2 * j + 1] = __uint_as_float(r.w[i][j] & 0xFFFF0000u);
        } else {
            v[j] = __uint_as_float(r.w[2 * i][j]);
            v[4 + j] = __uint_as_float(r.w[2 * i + 1][j]);
        }
    }
}

// What a wave has: rows [t0, t0 + n) and chunks [c0, c1) of their heads.
struct Share {
    int t0, n, c0, c1;
};
__device__ __forceinline__ bool share_of_wave(int rows, int chunks, int rows_each, int chunks_each, Share& w) {
    const int64_t wave = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int parts = (chunks + chunks_each - 1) / chunks_each;
    const int64_t group = wave / parts;
    if (group * rows_each >= rows) return false;
    w.t0 = (int)group * rows_each;
    w.n = min(rows_each, rows - w.t0);
    w.c0 = (int)(wave - group * parts) * chunks_each;
    w.c1 = min(chunks, w.c0 + chunks_each);
    return true;
}

// A row and a chunk of a wave's share, in order.
struct Cursor {
    int r, c;
    __device__ __forceinline__ void next(const Share& w) {
        if (++c == w.c1) {
            c = w.c0;
            ++r;
        }
    }
};

// A lane has the 8 elements from a and the 8 from b of its head: consecutive
// ones, but in the part of a head that is rotated in halves, pairs that lie
// rot / 2 apart.  A block's largest magnitude is then that of the lane's own
// 16, or of the first (second) eight of 2 or 4 neighbours.
template <typename T, int D, bool MX>
__global__ void __launch_bounds__(kThreads) k_kv_append(const KvAppend p) {
    constexpr int kLanes = D / 16, kHeads = 64 / kLanes;
    const int lane = threadIdx.x & 63, li = lane % kLanes;
    const int heads = p.q_heads + 2 * p.cache.heads, chunks = (heads + kHeads - 1) / kHeads;
    Share w;
    if (!share_of_wave(p.plan.rows, chunks, p.rows_each, p.chunks_each, w)) return;
    const KvPlaces places = kv_places(p.plan, p.cache.pages, w.t0, w.n);
    if (places.owned == 0) return;
    const int rot = p.rot, half = rot / 2;
    const bool turned = li < rot / 16, halves = turned && !p.interleaved;
    const int a = halves ? 8 * li : 16 * li, b = halves ? a + half : a + 8;

    const auto load = [&](int r, int c) {
        const int hd = min(c * kHeads + lane / kLanes, heads - 1);  // (past the last head: it again)
        const bool is_q = hd < p.q_heads, is_k = !is_q && hd < p.q_heads + p.cache.heads;
        const int h = is_q ? hd : is_k ? hd - p.q_heads : hd - p.q_heads - p.cache.heads;
        const void* data = is_q ? p.q.data : is_k ? p.k.data : p.v.data;
        const int64_t row = is_q ? p.q.row : is_k ? p.k.row : p.v.row, head = is_q ? p.q.head : is_k ? p.k.head : p.v.head;
        // (for a row of no sequence one that is: without a branch around loads under way)
        const int own = places.owned >> r & 1 ? r : __builtin_ctzll(places.owned);
        const T* src = static_cast<const T*>(data) + (w.t0 + own) * row + h * head;
        return load_raw(src + a, src + b);
    };
    Raw<T> now = load(0, w.c0);
    for (int r = 0; r < w.n; ++r) {
        const int t = w.t0 + r;
        const int pos = __builtin_amdgcn_readlane(places.pos, r), page = __builtin_amdgcn_readlane(places.page, r);
        const bool angle = pos >= 0 && pos < p.rope_rows;
        float cosine[8] = {}, sine[8] = {};
        if (angle && turned) {
            const float* row = p.rope + (int64_t)pos * p.rope_ld + 8 * li;
            load_upto8(row, 8, cosine);
            load_upto8(row + half, 8, sine);
        }
        for (int c = w.c0; c < w.c1; ++c) {
            const int hd = c * kHeads + lane / kLanes;
            const bool is_q = hd < p.q_heads, is_k = !is_q && hd < p.q_heads + p.cache.heads;
            const int h = is_q ? hd : is_k ? hd - p.q_heads : hd - p.q_heads - p.cache.heads;
            float x[8], y[8];
            unpack_raw(now, 0, x);
            unpack_raw(now, 1, y);
            // (two ahead, 15047 rows of 72 heads took 119 us instead of 114)
            if (c + 1 < w.c1) now = load(r, c + 1);
            else if (r + 1 < w.n) now = load(r + 1, w.c0);
            if (!(places.owned >> r & 1)) continue;
            if (turned && (is_q || is_k)) {
                if (halves) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) turn(x[j], y[j], cosine[j], sine[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        turn(x[2 * j], x[2 * j + 1], cosine[j], sine[j]);
                        turn(y[2 * j], y[2 * j + 1], cosine[4 + j], sine[4 + j]);
                    }
                }
            }
            // the block maxima, in all lanes (exchanges between lanes)
            float mx = absmax8(x), my = absmax8(y);
            const float own = fmaxf(mx, my), own2 = fmaxf(own, lane_xor1(own));
            mx = fmaxf(mx, lane_xor1(mx));
            my = fmaxf(my, lane_xor1(my));
            if constexpr (MX) {
                const float x4 = fmaxf(mx, lane_xor2(mx)), y4 = fmaxf(my, lane_xor2(my));
                mx = halves && half >= 32 ? x4 : own2;  // (half 16: one block of 32, on two lanes)
                my = halves && half >= 32 ? y4 : own2;
            } else {
                mx = halves ? mx : own;
                my = halves ? my : own;
            }
            if (hd >= heads) continue;
            if (is_q) {
                T* dst = static_cast<T*>(p.q_out.data) + t * p.q_out.row + h * p.q_out.head;
                if (!angle)
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = y[j] = 0.0f;
                store_upto8(dst + a, 8, x);
                store_upto8(dst + b, 8, y);
                continue;
            }
            if (page < 0 || !angle) continue;
            const float head_scale = MX ? 1.0f : (is_k ? p.cache.k_scale : p.cache.v_scale)[h];
            const BlockScale bx = kv_block_scale<MX>(mx, head_scale), by = kv_block_scale<MX>(my, head_scale);
            uint32_t cx, cy;
            encode<false, 8>(x, bx, mx, nullptr, &cx);
            encode<false, 8>(y, by, my, nullptr, &cy);
            const int slot = pos & ((1 << p.plan.page_shift) - 1);
            uint8_t* codes = (is_k ? p.cache.k_codes : p.cache.v_codes) + slot_at(p.cache, p.plan.page_shift, page, h, slot, D / 2);
            *reinterpret_cast<uint32_t*>(codes + a / 2) = cx;
            *reinterpret_cast<uint32_t*>(codes + b / 2) = cy;
            constexpr int per = MX ? 32 : 16;
            uint8_t* scales = (is_k ? p.cache.k_scales : p.cache.v_scales) + slot_at(p.cache, p.plan.page_shift, page, h, slot, D / per);
            // (the lane whose part begins a block writes its byte)
            if (a % per == 0) scales[a / per] = (uint8_t)bx.byte;
            if (halves && b % per == 0) scales[b / per] = (uint8_t)by.byte;
        }
    }
}

template <typename T, int D, bool MX>
__global__ void __launch_bounds__(kThreads) k_kv_gather(const KvGather p) {
    constexpr int kLanes = D / 16, kHeads = 64 / kLanes;
    const int lane = threadIdx.x & 63, li = lane % kLanes;
    const int heads = 2 * p.cache.heads, chunks = (heads + kHeads - 1) / kHeads;
    Share w;
    if (!share_of_wave(p.plan.rows, chunks, p.rows_each, p.chunks_each, w)) return;
    const KvPlaces places = kv_places(p.plan, p.cache.pages, w.t0, w.n);
    if (places.owned == 0) return;
    const int slot_mask = (1 << p.plan.page_shift) - 1;

    struct Held {
        uint2 w;
        uint32_t byte;
    };
    Cursor ahead = {0, w.c0};
    const auto load = [&]() {
        Held v = {{0u, 0u}, 0u};
        const int r = min(ahead.r, 63), c = ahead.c;  // (lanes past the last row have no page)
        const int pos = __builtin_amdgcn_readlane(places.pos, r), page = __builtin_amdgcn_readlane(places.page, r);
        ahead.next(w);
        if (page >= 0) {
            const int hd = min(c * kHeads + lane / kLanes, heads - 1);
            const bool is_k = hd < p.cache.heads;
            const int h = is_k ? hd : hd - p.cache.heads;
            v.w = *reinterpret_cast<const uint2*>((is_k ? p.cache.k_codes : p.cache.v_codes) +
                                                  slot_at(p.cache, p.plan.page_shift, page, h, pos & slot_mask, D / 2) + 8 * li);
            v.byte = ((is_k ? p.cache.k_scales : p.cache.v_scales) +
                      slot_at(p.cache, p.plan.page_shift, page, h, pos & slot_mask, D / (MX ? 32 : 16)))[MX ? li / 2 : li];
        }
        return v;
    };
    constexpr int kAhead = 4;
    Held held[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) held[i] = load();
    for (Cursor at = {0, w.c0}; at.r < w.n;) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const Held now = held[i];
            held[i] = load();
            const int r = min(at.r, 63), c = at.c, t = w.t0 + r;
            const int pos = __builtin_amdgcn_readlane(places.pos, r), page = __builtin_amdgcn_readlane(places.page, r);
            at.next(w);
            const int hd = c * kHeads + lane / kLanes;
            if (!(places.owned >> r & 1) || hd >= heads) continue;
            const bool is_k = hd < p.cache.heads;
            const int h = is_k ? hd : hd - p.cache.heads;
            float v[16] = {};
            if (page >= 0) {
                const float f = MX ? e8m0_value(now.byte) : e4m3_value(now.byte);
                const float hs = MX ? 1.0f : (is_k ? p.cache.k_scale : p.cache.v_scale)[h];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 u = e2m1x2_unpack(j < 4 ? now.w.x : now.w.y, j & 3);
                    v[2 * j] = u.x * f * hs;
                    v[2 * j + 1] = u.y * f * hs;
                }
            }
            void* data = const_cast<void*>(is_k ? p.k.data : p.v.data);
            T* dst = static_cast<T*>(data) + t * (is_k ? p.k.row : p.v.row) + h * (is_k ? p.k.head : p.v.head) + 16 * li;
            store_upto8(dst, 8, v);
            store_upto8(dst + 8, 8, v + 8);
        }
    }
}

// Chunks of heads and rows for a wave: more chunks than one where there are over 8192
// waves to have them (32 on each of 256 compute units), and then more rows, up to
// 8, where there are over 32768 (64 rows of over 2^26, so that a grid holds them).
// 15047 rows of 72 heads to append, 16 to gather: from 4096 on 127 and 21.9 us, from
// 8192 119 and 21.6, from 32768 141 and 27.8; 79926 rows to gather, more rows from
// 8192 on 134 us, from 32768 109.
template <typename P>
int divide_rows(P& p, int heads) {
    const int per = 64 / (p.cache.dim / 16), chunks = (heads + per - 1) / per;
    const int64_t items = (int64_t)p.plan.rows * chunks;
    p.chunks_each = (int)std::max<int64_t>(1, std::min<int64_t>(chunks, items / 8192));
    p.rows_each = (int)std::max<int64_t>(1, std::min<int64_t>(p.plan.rows > (1 << 26) ? 64 : 8, items / chunks / 32768));
    const int64_t waves = (int64_t)((p.plan.rows + p.rows_each - 1) / p.rows_each) * ((chunks + p.chunks_each - 1) / p.chunks_each);
    return (int)((waves + kWaves - 1) / kWaves);
}

}  // namespace

hipError_t launch_kv_append(KvAppend p, hipStream_t s) {
    if (p.plan.rows == 0 || p.plan.seqs == 0) return hipSuccess;
    const dim3 grid(divide_rows(p, p.q_heads + 2 * p.cache.heads));
    const auto run = [&](auto t, auto d) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value;
        if (p.cache.mx) hipLaunchKernelGGL((k_kv_append<T, D, true>), grid, dim3(kThreads), 0, s, p);
        else hipLaunchKernelGGL((k_kv_append<T, D, false>), grid, dim3(kThreads), 0, s, p);
    };
    const auto pick = [&](auto t) {
        if (p.cache.dim == 64) run(t, std::integral_constant<int, 64>());
        else if (p.cache.dim == 128) run(t, std::integral_constant<int, 128>());
        else run(t, std::integral_constant<int, 256>());
    };
    if (p.bf16) pick(uint16_t());
    else pick(float());
    return hipGetLastError();
}

hipError_t launch_kv_gather(KvGather p, hipStream_t s) {
    if (p.plan.rows == 0 || p.plan.seqs == 0) return hipSuccess;
    const dim3 grid(divide_rows(p, 2 * p.cache.heads));
    const auto run = [&](auto t, auto d) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value;
        if (p.cache.mx) hipLaunchKernelGGL((k_kv_gather<T, D, true>), grid, dim3(kThreads), 0, s, p);
        else hipLaunchKernelGGL((k_kv_gather<T, D, false>), grid, dim3(kThreads), 0, s, p);
    };
    const auto pick = [&](auto t) {
        if (p.cache.dim == 64) run(t, std::integral_constant<int, 64>());
        else if (p.cache.dim == 128) run(t, std::integral_constant<int, 128>());
        else run(t, std::integral_constant<int, 256>());
    };
    if (p.bf16) pick(uint16_t());
    else pick(float());
    return hipGetLastError();
}

}  // namespace nvfp4
