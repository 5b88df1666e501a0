/* The exact status of the key/value cache's entry points for each size at the
 * ends of its type, under AddressSanitizer and UndefinedBehaviorSanitizer (test
 * infrastructure only; built and run by tests/test_abi_sanitize_kv_status.py).
 * Attention is given a workspace that is large enough and lies 8 bytes off its
 * alignment, gather a v and append a q_out 1 byte off theirs, which is what they
 * look at last: sizes in order end with NVFP4_ERR_ALIGN and nothing is ever
 * launched.  Pointers are plain integers that are never dereferenced.  Prints
 * "ok" at the end; a wrong status or a sanitizer report fails.
 */
#include <stdint.h>
#include <stdio.h>

#include "nvfp4.h"

static int failures = 0;

#define CHECK(expr, want)                                                                     \
    do {                                                                                      \
        const long long got_ = (long long)(expr);                                             \
        if (got_ != (long long)(want)) {                                                      \
            fprintf(stderr, "line %d, %lld: %s returned %lld, expected %lld\n", __LINE__,     \
                    (long long)n, #expr, got_, (long long)(want));                            \
            ++failures;                                                                       \
        }                                                                                     \
    } while (0)

#define P ((void*)(uintptr_t)65536)
#define OFF ((void*)(uintptr_t)65537)
#define OFF8 ((void*)(uintptr_t)65544)
static const int64_t kEnds[] = {INT64_MIN, INT64_MIN + 1, -1, 0, 1, 4, 15, 16, 48, 64, 127, 128, 129, 255, 256, 640, 1152, 65536,
                                65537, ((int64_t)1 << 25), ((int64_t)1 << 25) + 1, (int64_t)1 << 27, ((int64_t)1 << 27) + 1,
                                (int64_t)1 << 28, ((int64_t)1 << 28) + 1, (int64_t)1 << 29, (int64_t)1 << 30,
                                ((int64_t)1 << 30) + 1, INT32_MAX, (int64_t)1 << 31, (int64_t)1 << 40, (int64_t)1 << 62,
                                INT64_MAX - 31, INT64_MAX};
enum { kN = sizeof(kEnds) / sizeof(kEnds[0]) };

static nvfp4_status attention(const nvfp4_kv_cache* c, const nvfp4_kv_plan* p, nvfp4_kv_rows q, nvfp4_kv_rows out, int32_t heads,
                              int64_t window) {
    return nvfp4_kv_attention(&q, 1, heads, c, p, 1.0f, window, &out, P, OFF8, SIZE_MAX, NULL);
}
static nvfp4_status gather(const nvfp4_kv_cache* c, const nvfp4_kv_plan* p, nvfp4_kv_rows k) {
    nvfp4_kv_rows v = {OFF, k.row_stride, k.head_stride};
    return nvfp4_kv_gather(c, p, &k, &v, 1, NULL);
}
static nvfp4_status append(const nvfp4_kv_cache* c, const nvfp4_kv_plan* p, nvfp4_kv_rows in, nvfp4_kv_rows q_out) {
    q_out.data = OFF;
    return nvfp4_kv_append(&in, &in, 1, c, p, NULL, &in, 2, &q_out, NULL);
}

static void cache_and_plan(int64_t n, const nvfp4_kv_cache* c, const nvfp4_kv_plan* p, nvfp4_status want, nvfp4_status attend) {
    const nvfp4_kv_rows r = {P, 256, 128};
    CHECK(attention(c, p, r, r, 2, 0), attend);
    CHECK(gather(c, p, r), want);
    CHECK(append(c, p, r, r), want);
}

int main(void) {
    const nvfp4_kv_cache good = {P, P, P, P, P, P, 8, 32, 2, 128, NVFP4_KV_NVFP4};
    const nvfp4_kv_plan plan = {P, 4, 4, P, P, 3, 5};
    const nvfp4_kv_rows r = {P, 256, 128};
    for (int i = 0; i < kN; ++i) {
        const int64_t n = kEnds[i];
        nvfp4_kv_cache c = good;
        nvfp4_kv_plan p = plan;
        nvfp4_status want = n < 0 ? NVFP4_ERR_SHAPE : n > INT32_MAX ? NVFP4_ERR_UNSUPPORTED : NVFP4_ERR_ALIGN;
        c.pages = n;
        cache_and_plan(n, &c, &plan, want, want);
        c = good;
        c.page_size = n;
        want = n < 1 ? NVFP4_ERR_SHAPE
                     : n < 16 || (n & (n - 1)) || n > ((int64_t)1 << 28) ? NVFP4_ERR_UNSUPPORTED : NVFP4_ERR_ALIGN;
        cache_and_plan(n, &c, &plan, want, want);
        p.rows = n;
        want = n < 0 ? NVFP4_ERR_SHAPE : n > ((int64_t)1 << 30) ? NVFP4_ERR_UNSUPPORTED : NVFP4_ERR_ALIGN;
        cache_and_plan(n, &good, &p, want, n > ((int64_t)1 << 27) ? NVFP4_ERR_UNSUPPORTED : n == 0 ? NVFP4_OK : want);
        p = plan;
        p.seqs = n;
        want = n < 0 ? NVFP4_ERR_SHAPE : n > 65536 ? NVFP4_ERR_UNSUPPORTED : NVFP4_ERR_ALIGN;
        cache_and_plan(n, &good, &p, want, want);
        p = plan;
        p.width = n;
        p.ld_table = INT64_MAX;
        want = n < 0 ? NVFP4_ERR_SHAPE : n > ((int64_t)1 << 25) ? NVFP4_ERR_UNSUPPORTED : NVFP4_ERR_ALIGN;
        cache_and_plan(n, &good, &p, want, want);
        p = plan;
        p.ld_table = n;
        want = n < 4 ? NVFP4_ERR_SHAPE : NVFP4_ERR_ALIGN;
        cache_and_plan(n, &good, &p, want, want);
        /* strides of what is read, then of what is written: 5 rows of 2 heads of 128 */
        const nvfp4_kv_rows by_row = {P, n, 128}, by_head = {P, 256, n};
        want = n < 0 ? NVFP4_ERR_SHAPE : NVFP4_ERR_ALIGN;
        CHECK(attention(&good, &plan, by_row, r, 2, 0), want);
        CHECK(attention(&good, &plan, by_head, r, 2, 0), want);
        CHECK(append(&good, &plan, by_row, r), want);
        CHECK(append(&good, &plan, by_head, r), want);
        want = n < 256 ? NVFP4_ERR_SHAPE : NVFP4_ERR_ALIGN;
        CHECK(attention(&good, &plan, r, by_row, 2, 0), want);
        CHECK(gather(&good, &plan, by_row), want);
        CHECK(append(&good, &plan, r, by_row), want);
        want = n != 128 && n < 4 * 256 + 128 ? NVFP4_ERR_SHAPE : NVFP4_ERR_ALIGN;
        CHECK(attention(&good, &plan, r, by_head, 2, 0), want);
        CHECK(gather(&good, &plan, by_head), want);
        CHECK(append(&good, &plan, r, by_head), want);
        CHECK(attention(&good, &plan, r, r, 2, n), n < 0 ? NVFP4_ERR_SHAPE : NVFP4_ERR_ALIGN);
        if (n >= INT32_MIN && n <= INT32_MAX) {
            const nvfp4_kv_rows wide = {P, INT64_MAX, 128};
            want = n < 1 || n % 2 ? NVFP4_ERR_SHAPE : 5 * n > ((int64_t)1 << 28) ? NVFP4_ERR_UNSUPPORTED : NVFP4_ERR_ALIGN;
            CHECK(attention(&good, &plan, r, wide, (int32_t)n, 0), want);
            c = good;
            c.head_dim = (int32_t)n;
            const nvfp4_kv_rows apart = {P, (int64_t)1 << 33, (int64_t)1 << 32};
            want = n < 1 ? NVFP4_ERR_SHAPE : n != 64 && n != 128 && n != 256 ? NVFP4_ERR_UNSUPPORTED : NVFP4_ERR_ALIGN;
            CHECK(attention(&c, &plan, r, apart, 2, 0), want);
            CHECK(gather(&c, &plan, apart), want);
        }
    }
    if (failures) return 1;
    puts("ok");
    return 0;
}
