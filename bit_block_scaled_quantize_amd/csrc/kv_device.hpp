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

// What the table says for position pos of sequence s, and the page that names: -1
// for none.  (Looking at the entry waits for its load and for all loads before it.)
__device__ __forceinline__ int kv_entry(const KvPlan& p, int s, int pos) {
    return p.table[s * p.ld_table + (pos >> p.page_shift)];
}
__device__ __forceinline__ int kv_page_of(int entry, int pages) { return (uint32_t)entry < (uint32_t)pages ? entry : -1; }

// Where rows t0 .. t0 + n - 1 (n <= 64) lie: lane r has row t0 + r's position and
// page.
struct KvPlaces {
    int pos;
    int page;        // -1: none
    uint64_t owned;  // bit r: row t0 + r belongs to a sequence (known before the rest)
};

// A row's sequence is the number of offsets[1 ...] that are <= it; 64 offsets are
// compared at a time.
__device__ __forceinline__ KvPlaces kv_places(const KvPlan& p, int pages, int t0, int n) {
    const int lane = threadIdx.x & 63, t = t0 + lane;
    KvPlaces w = {-1, -1, 0};
    int s = t;
    if (p.offsets) {
        s = 0;
        for (int b = 0; b < p.seqs; b += 64) {
            const int end = b + lane < p.seqs ? p.offsets[b + lane + 1] : 0x7FFFFFFF;
            int more = 0;
            for (int r = 0; r < n; ++r) {
                const int c = __popcll(__ballot(end <= t0 + r));
                if (lane == r) s += c;
                more = c;  // (of the last row)
            }
            if (more < 64) break;
        }
    }
    int first = 0, count = 0;
    if (lane < n && s < p.seqs && (!p.offsets || t >= p.offsets[0])) kv_rows(p, s, first, count);
    const bool own = t >= first && t - first < count;  // (else also where offsets are out of order)
    w.owned = __ballot(own);
    if (own) {
        w.pos = kv_length(p, s) - count + (t - first);
        if (w.pos >= 0) w.page = kv_page_of(kv_entry(p, s, w.pos), pages);
    }
    return w;
}

// E8M0 byte as binary32: 2^(b - 127) (b = 0: a subnormal number).
__device__ __forceinline__ float e8m0_value(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x00400000u); }

}  // namespace nvfp4
