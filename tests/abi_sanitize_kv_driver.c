/* Host-side argument validation of the key/value cache's entry points under
 * AddressSanitizer and UndefinedBehaviorSanitizer (test infrastructure only;
 * built and run by tests/test_abi_sanitize_kv.py).  Every call passes an
 * argument that validation must refuse, or sizes that leave nothing to do, so
 * nothing is ever launched; pointers are plain integers that are never
 * dereferenced.  Sizes go up to the ends of their types.  Prints "ok" at the
 * end; a wrong status or a sanitizer report fails.
 */
#include <stdint.h>
#include <stdio.h>

#include "nvfp4.h"

static int failures = 0;

#define CHECK(expr, want)                                                                     \
    do {                                                                                      \
        const long long got_ = (long long)(expr);                                             \
        if (got_ != (long long)(want)) {                                                      \
            fprintf(stderr, "line %d: %s returned %lld, expected %lld\n", __LINE__, #expr,    \
                    got_, (long long)(want));                                                 \
            ++failures;                                                                       \
        }                                                                                     \
    } while (0)

#define P ((void*)(uintptr_t)65536)
static const int64_t kEnds[] = {INT64_MIN, INT64_MIN + 1, -1, 0, 1, 16, 64, 128, (int64_t)1 << 28, (int64_t)1 << 30,
                                ((int64_t)1 << 30) + 1, (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX - 31, INT64_MAX};
enum { kN = sizeof(kEnds) / sizeof(kEnds[0]) };
static const int32_t kSmall[] = {INT32_MIN, -1, 0, 1, 2, 64, 128, 256, INT32_MAX - 1, INT32_MAX};
enum { kM = sizeof(kSmall) / sizeof(kSmall[0]) };

/* Every call on c and p; rows of zero stride, which no output may have where
 * there is more than one row. */
static int all_refused(const nvfp4_kv_cache* c, const nvfp4_kv_plan* p, int64_t row, int64_t head, int32_t q_heads,
                       int64_t window) {
    nvfp4_kv_rows r = {P, row, head};
    const nvfp4_kv_rope rope = {P, row, row, (int32_t)(head & 0xFF), 0};
    return nvfp4_kv_append(&r, &r, 1, c, p, &rope, &r, q_heads, &r, NULL) != NVFP4_OK &&
           nvfp4_kv_gather(c, p, &r, &r, 0, NULL) != NVFP4_OK &&
           nvfp4_kv_attention(&r, 1, q_heads, c, p, 1.0f, window, &r, P, NULL, 0, NULL) != NVFP4_OK;
}

int main(void) {
    const nvfp4_kv_cache good = {P, P, P, P, P, P, 8, 32, 2, 128, NVFP4_KV_NVFP4};
    const nvfp4_kv_plan plan = {P, 4, 4, P, P, 3, 5};
    nvfp4_kv_rows r = {P, 256, 128};
    CHECK(nvfp4_kv_append(NULL, &r, 1, &good, &plan, NULL, NULL, 0, NULL, NULL), NVFP4_ERR_NULL);
    CHECK(nvfp4_kv_append(&r, &r, 1, NULL, &plan, NULL, NULL, 0, NULL, NULL), NVFP4_ERR_NULL);
    CHECK(nvfp4_kv_append(&r, &r, 1, &good, NULL, NULL, NULL, 0, NULL, NULL), NVFP4_ERR_NULL);
    CHECK(nvfp4_kv_append(&r, &r, INT32_MAX, &good, &plan, NULL, NULL, 0, NULL, NULL), NVFP4_ERR_ENUM);
    CHECK(nvfp4_kv_gather(&good, &plan, NULL, &r, 1, NULL), NVFP4_ERR_NULL);
    CHECK(nvfp4_kv_gather(&good, &plan, &r, &r, INT32_MIN, NULL), NVFP4_ERR_ENUM);
    CHECK(nvfp4_kv_attention(&r, 1, 2, &good, &plan, 1.0f, 0, &r, NULL, NULL, 0, NULL), NVFP4_ERR_WORKSPACE);
    for (int i = 0; i < kN; ++i) {
        const int64_t n = kEnds[i];
        /* sizes that are refused, in each field */
        nvfp4_kv_cache c = good;
        nvfp4_kv_plan p = plan;
        c.pages = n;
        if (n < 0 || n > INT32_MAX) CHECK(all_refused(&c, &plan, 256, 128, 2, 0), 1);
        c = good;
        c.page_size = n;
        if (n < 16 || n > ((int64_t)1 << 28)) CHECK(all_refused(&c, &plan, 256, 128, 2, 0), 1);
        p.rows = n;
        if (n < 0 || n > ((int64_t)1 << 30)) CHECK(all_refused(&good, &p, 256, 128, 2, 0), 1);
        p = plan;
        p.seqs = n;
        if (n < 0 || n > 65536) CHECK(all_refused(&good, &p, 256, 128, 2, 0), 1);
        p = plan;
        p.width = n;
        p.ld_table = INT64_MAX;
        if (n < 0 || n > ((int64_t)1 << 25)) CHECK(all_refused(&good, &p, 256, 128, 2, 0), 1);
        p = plan;
        p.ld_table = n;
        if (n < 4) CHECK(all_refused(&good, &p, 256, 128, 2, 0), 1);
        if (n < 0) CHECK(all_refused(&good, &plan, n, 128, 2, 0), 1);
        if (n < 128) CHECK(all_refused(&good, &plan, 1, n, 2, 0), 1);
        /* strides at the ends of their type that leave outputs apart or not: a cache
         * without its arrays is refused after them */
        for (int j = 0; j < kN; ++j) {
            c = good;
            c.k_codes = NULL;
            CHECK(all_refused(&c, &plan, n, kEnds[j], 2, n), 1);
            c = good;
            c.head_dim = 96;
            CHECK(all_refused(&c, &plan, n, kEnds[j], 2, kEnds[j]), 1);
            nvfp4_kv_rows o = {P, n, kEnds[j]};
            nvfp4_kv_rows off = {(void*)(uintptr_t)65537, n, kEnds[j]};
            CHECK(nvfp4_kv_gather(&good, &plan, &o, &off, 1, NULL) != NVFP4_OK, 1);
            CHECK(nvfp4_kv_attention(&r, 1, 2, &good, &plan, 1.0f, kEnds[j], &o, NULL, NULL, 0, NULL) != NVFP4_OK, 1);
        }
        for (int j = 0; j < kN; ++j)
            for (int k = 0; k < kM; ++k)
                for (int l = 0; l < kM; ++l)
                    for (int m = 0; m < kM; ++m)
                        (void)nvfp4_kv_attention_workspace_size(n, kEnds[j], kSmall[k], kSmall[l], kSmall[m], j & 1);
    }
    for (int i = 0; i < kM; ++i) {
        nvfp4_kv_cache c = good;
        c.kv_heads = kSmall[i];
        if (kSmall[i] < 1) CHECK(all_refused(&c, &plan, 256, 128, 2, 0), 1);
        nvfp4_kv_plan none = {P, 4, 4, P, P, 3, 0};
        /* (no rows: refused for the heads, or nothing to do) */
        (void)nvfp4_kv_attention(&r, 1, kSmall[i], &c, &none, 1.0f, INT64_MAX, &r, P, NULL, 0, NULL);
        (void)nvfp4_kv_gather(&c, &none, &r, &r, 1, NULL);
        (void)nvfp4_kv_append(&r, &r, 1, &c, &none, NULL, &r, kSmall[i], &r, NULL);
        c = good;
        c.head_dim = kSmall[i];
        if (kSmall[i] != 64 && kSmall[i] != 128 && kSmall[i] != 256) CHECK(all_refused(&c, &plan, 256, 128, 2, 0), 1);
        c = good;
        c.format = kSmall[i];
        if (kSmall[i] != 0 && kSmall[i] != 1) CHECK(all_refused(&c, &plan, 256, 128, 2, 0), 1);
        nvfp4_kv_rope rope = {P, INT64_MAX, INT64_MAX, kSmall[i], 1};
        if (kSmall[i] != 64 && kSmall[i] != 128)
            CHECK(nvfp4_kv_append(&r, &r, 1, &good, &plan, &rope, NULL, 0, NULL, NULL) != NVFP4_OK, 1);
    }
    if (failures) return 1;
    puts("ok");
    return 0;
}
