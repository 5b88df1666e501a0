// Appending keys and values to the paged 4-bit cache, with the rotation of their
// positions, and reading them back, for gfx950.
//
// Both go over (row, head) pairs: a head of D elements takes D / 16 lanes of 16
// elements each, so that a wave has 16, 8 or 4 heads of one row (D 64, 128,
// 256) and its sequence, position and page are the same in all its lanes.
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
// include/nvfp4.h; NVFP4 with the head's float as tensor scale).
template <bool MX>
__device__ __forceinline__ BlockScale kv_block_scale(float amax, float head_scale) {
    BlockScale bs;
    if constexpr (MX) {
        const int s = max((int)(__float_as_uint(amax) >> 23) - 127 - 2, -127);
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

// A lane has the 8 elements from a and the 8 from b of its head: consecutive
// ones, but in the part of a head that is rotated in halves, pairs that lie
// rot / 2 apart.  A block's largest magnitude is then that of the lane's own
// 16, or of the first (second) eight of 2 or 4 neighbours.
template <typename T, int D, bool MX>
__global__ void __launch_bounds__(kThreads) k_kv_append(const KvAppend p) {
    constexpr int kLanes = D / 16, kHeads = 64 / kLanes;
    const int lane = threadIdx.x & 63, li = lane % kLanes;
    const int heads = p.q_heads + 2 * p.cache.heads, chunks = (heads + kHeads - 1) / kHeads;
    const int rot = p.rot, half = rot / 2;
    const bool halves = !p.interleaved && li < rot / 16;
    const int a = halves ? 8 * li : 16 * li, b = halves ? a + half : a + 8;
    const int64_t items = (int64_t)p.plan.rows * chunks;
    for (int64_t it = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); it < items;
         it += (int64_t)gridDim.x * kWaves) {
        const int t = (int)(it / chunks), hd = (int)(it % chunks) * kHeads + lane / kLanes;
        int s, pos;
        if (!kv_place(p.plan, t, s, pos)) continue;
        const bool angle = pos >= 0 && pos < p.rope_rows;
        int page = -1;
        if (angle) page = kv_page(p.plan, p.cache.pages, s, pos);
        const bool is_q = hd < p.q_heads, is_k = !is_q && hd < p.q_heads + p.cache.heads;
        const int h = is_q ? hd : is_k ? hd - p.q_heads : hd - p.q_heads - p.cache.heads;
        float x[8] = {}, y[8] = {};
        if (hd < heads && angle) {
            const KvRows& r = is_q ? p.q : is_k ? p.k : p.v;
            const T* src = static_cast<const T*>(r.data) + t * r.row + h * r.head;
            load_upto8(src + a, 8, x);
            load_upto8(src + b, 8, y);
        }
        const bool rotated = (is_q || is_k) && li < rot / 16 && angle;
        if (rotated) {
            float c[8], sn[8];
            const float* row = p.rope + (int64_t)pos * p.rope_ld + 8 * li;
            load_upto8(row, 8, c);
            load_upto8(row + half, 8, sn);
            if (halves) {
#pragma unroll
                for (int j = 0; j < 8; ++j) turn(x[j], y[j], c[j], sn[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    turn(x[2 * j], x[2 * j + 1], c[j], sn[j]);
                    turn(y[2 * j], y[2 * j + 1], c[4 + j], sn[4 + j]);
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
            store_upto8(dst + a, 8, x);
            store_upto8(dst + b, 8, y);
            continue;
        }
        if (page < 0) continue;
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

template <typename T, int D, bool MX>
__global__ void __launch_bounds__(kThreads) k_kv_gather(const KvGather p) {
    constexpr int kLanes = D / 16, kHeads = 64 / kLanes;
    const int lane = threadIdx.x & 63, li = lane % kLanes;
    const int heads = 2 * p.cache.heads, chunks = (heads + kHeads - 1) / kHeads;
    const int64_t items = (int64_t)p.plan.rows * chunks;
    for (int64_t it = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); it < items;
         it += (int64_t)gridDim.x * kWaves) {
        const int t = (int)(it / chunks), hd = (int)(it % chunks) * kHeads + lane / kLanes;
        int s, pos;
        if (!kv_place(p.plan, t, s, pos) || hd >= heads) continue;
        const int page = pos >= 0 ? kv_page(p.plan, p.cache.pages, s, pos) : -1;
        const bool is_k = hd < p.cache.heads;
        const int h = is_k ? hd : hd - p.cache.heads;
        float v[16] = {};
        if (page >= 0) {
            const int slot = pos & ((1 << p.plan.page_shift) - 1);
            const uint2 w = *reinterpret_cast<const uint2*>(
                (is_k ? p.cache.k_codes : p.cache.v_codes) + slot_at(p.cache, p.plan.page_shift, page, h, slot, D / 2) + 8 * li);
            const uint32_t byte = ((is_k ? p.cache.k_scales : p.cache.v_scales) +
                                   slot_at(p.cache, p.plan.page_shift, page, h, slot, D / (MX ? 32 : 16)))[MX ? li / 2 : li];
            const float f = MX ? e8m0_value(byte) : e4m3_value(byte);
            const float hs = MX ? 1.0f : (is_k ? p.cache.k_scale : p.cache.v_scale)[h];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 u = e2m1x2_unpack(j < 4 ? w.x : w.y, j & 3);
                v[2 * j] = u.x * f * hs;
                v[2 * j + 1] = u.y * f * hs;
            }
        }
        const KvRows& r = is_k ? p.k : p.v;
        T* dst = static_cast<T*>(const_cast<void*>(r.data)) + t * r.row + h * r.head + 16 * li;
        store_upto8(dst, 8, v);
        store_upto8(dst + 8, 8, v + 8);
    }
}

int grid_of(int64_t rows, int heads, int dim) {
    const int per = 64 / (dim / 16);
    const int64_t items = rows * ((heads + per - 1) / per);
    return (int)std::min<int64_t>((items + kWaves - 1) / kWaves, max_blocks(kThreads));
}

}  // namespace

hipError_t launch_kv_append(const KvAppend& p, hipStream_t s) {
    if (p.plan.rows == 0) return hipSuccess;
    const dim3 grid(grid_of(p.plan.rows, p.q_heads + 2 * p.cache.heads, p.cache.dim));
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

hipError_t launch_kv_gather(const KvGather& p, hipStream_t s) {
    if (p.plan.rows == 0) return hipSuccess;
    const dim3 grid(grid_of(p.plan.rows, 2 * p.cache.heads, p.cache.dim));
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
