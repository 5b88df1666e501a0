// Device helpers of the paged 4-bit key/value cache (append, gather,
// attention): where a row of the plan lies, and the cache's values.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"
#include "nvfp4_device.hpp"
#include "row_device.hpp"

namespace nvfp4 {

// Keys of sequence s: a length beyond what its row of the table can hold counts
// as that, a negative one as 0.
__device__ __forceinline__ int kv_length(const KvPlan& p, int s) {
    return max(0, min(p.lengths[s], p.width << p.page_shift));
}

// Rows [first, first + n) of sequence s; offsets outside [0, rows] or out of
// order are clamped.
__device__ __forceinline__ void kv_rows(const KvPlan& p, int s, int& first, int& n) {
    if (!p.offsets) {
        first = s;
        n = 1;
        return;
    }
    first = max(0, min(p.offsets[s], p.rows));
    n = max(first, min(p.offsets[s + 1], p.rows)) - first;
}

// Page of position pos of sequence s, -1 where the table names none.
__device__ __forceinline__ int kv_page(const KvPlan& p, int pages, int s, int pos) {
    const int page = p.table[s * p.ld_table + (pos >> p.page_shift)];
    return (uint32_t)page < (uint32_t)pages ? page : -1;
}

// Sequence and position of row t (the same in every lane of the wave); false for
// a row that belongs to no sequence.  64 offsets are compared at a time: the
// sequence is the number of offsets[1 ...] that are <= t.
__device__ __forceinline__ bool kv_place(const KvPlan& p, int t, int& s, int& pos) {
    if (!p.offsets) {
        s = t;
    } else {
        if (t < p.offsets[0]) return false;
        const int lane = threadIdx.x & 63;
        s = 0;
        for (int b = 0; b < p.seqs; b += 64) {
            const int c = __popcll(__ballot(b + lane < p.seqs && p.offsets[b + lane + 1] <= t));
            s += c;
            if (c < 64) break;
        }
        s = __builtin_amdgcn_readfirstlane(s);
        if (s >= p.seqs) return false;
    }
    int first, n;
    kv_rows(p, s, first, n);
    if (t < first || t - first >= n) return false;  // (offsets out of order)
    pos = kv_length(p, s) - n + (t - first);
    return true;
}

// E8M0 byte as binary32: 2^(b - 127) (b = 0: a subnormal number).
__device__ __forceinline__ float e8m0_value(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x00400000u); }

}  // namespace nvfp4
