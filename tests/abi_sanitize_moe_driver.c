/* Host-side argument validation of the MoE-block entry points under
 * AddressSanitizer and UndefinedBehaviorSanitizer (test infrastructure only;
 * built and run by tests/test_abi_sanitize_moe.py).  Every call passes an
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
#define ODD ((void*)(uintptr_t)65537)
static const int64_t kEnds[] = {INT64_MIN, INT64_MIN + 1, -1, 0, 1, 16, 32, 64, (int64_t)1 << 31, (int64_t)1 << 40,
                                INT64_MAX - 31, INT64_MAX};
enum { kN = sizeof(kEnds) / sizeof(kEnds[0]) };

static void norm_cases(void) {
    nvfp4_mx_tensor mx = {P, P, 4, 64, NVFP4_MX_E4M3}, bad = {P, P, 4, 64, 7};
#define NORM(x, ldx, r, w, wdt, dt, rows, cols, eps, y, m, rstd) \
    nvfp4_rmsnorm(x, ldx, r, 64, w, wdt, dt, rows, cols, eps, P, 64, y, 64, m, rstd, NULL)
    CHECK(NORM(NULL, 64, P, P, 1, 1, 4, 64, 1e-6f, P, &mx, P), NVFP4_ERR_NULL);
    CHECK(NORM(P, 64, P, NULL, 1, 1, 4, 64, 1e-6f, P, &mx, P), NVFP4_ERR_NULL);
    CHECK(NORM(P, 64, P, P, 1, 1, 4, 64, 1e-6f, NULL, NULL, P), NVFP4_ERR_NULL);
    CHECK(NORM(P, 64, P, P, INT32_MAX, 1, 4, 64, 1e-6f, P, &mx, P), NVFP4_ERR_ENUM);
    CHECK(NORM(P, 64, P, P, 1, INT32_MIN, 4, 64, 1e-6f, P, &mx, P), NVFP4_ERR_ENUM);
    CHECK(NORM(P, 64, P, P, 1, 1, 4, 64, 1e-6f, P, &bad, P), NVFP4_ERR_ENUM);
    CHECK(NORM(ODD, 64, P, P, 1, 1, 4, 64, 1e-6f, P, &mx, P), NVFP4_ERR_ALIGN);
    CHECK(NORM(P, 64, P, P, 1, 1, 4, 64, -0.0f, P, &mx, P), NVFP4_ERR_UNSUPPORTED);
    CHECK(NORM(P, 64, P, P, 1, 1, 5, 64, 1e-6f, P, &mx, P), NVFP4_ERR_SHAPE);
    for (int i = 0; i < kN; ++i) {
        /* (ld 64, h 64: wider rows are inconsistent) */
        const int64_t n = kEnds[i];
        if (n < 1 || n > 64) CHECK(NORM(P, n, P, P, 1, 1, 4, n, 1e-6f, P, NULL, P), NVFP4_ERR_SHAPE);
        if (n < 0) CHECK(NORM(P, 64, P, P, 1, 1, n, 64, 1e-6f, P, NULL, P), NVFP4_ERR_SHAPE);
        if (n > INT32_MAX) CHECK(NORM(P, 64, P, P, 1, 1, n, 64, 1e-6f, P, NULL, P), NVFP4_ERR_UNSUPPORTED);
        if (n < 0 || n > 32768) {
            CHECK(nvfp4_rmsnorm_backward_workspace_size(4, n), 0);
            CHECK(nvfp4_rmsnorm_backward(P, n, P, n, P, P, 1, P, n, 1, 4, n, P, n, P, P, SIZE_MAX, NULL),
                  n < 0 ? NVFP4_ERR_SHAPE : NVFP4_ERR_UNSUPPORTED);
        }
        for (int j = 0; j < kN; ++j) (void)nvfp4_rmsnorm_backward_workspace_size(n, kEnds[j]);
    }
    CHECK(nvfp4_rmsnorm_backward(P, 64, P, 64, NULL, P, 1, P, 64, 1, 4, 64, P, 64, P, P, SIZE_MAX, NULL), NVFP4_ERR_NULL);
    CHECK(nvfp4_rmsnorm_backward(P, 64, P, 64, P, P, 9, P, 64, 1, 4, 64, P, 64, P, P, SIZE_MAX, NULL), NVFP4_ERR_ENUM);
    CHECK(nvfp4_rmsnorm_backward(P, 64, P, 64, P, P, 1, ODD, 64, 1, 4, 64, P, 64, P, P, SIZE_MAX, NULL), NVFP4_ERR_ALIGN);
    CHECK(nvfp4_rmsnorm_backward(P, 64, P, 64, P, P, 1, P, 64, 1, 4, 64, P, 64, P, P, 0, NULL), NVFP4_ERR_WORKSPACE);
}

static void route_cases(void) {
    nvfp4_route_opts o = {4, NVFP4_ROUTE_SOFTMAX, 1, 1, NVFP4_GROUP_TOP2, 1, NULL}, b;
#define ROUTE(l, dt, T, n, op, ids) nvfp4_route(l, dt, T, n, 64, op, ids, P, P, P, P, P, SIZE_MAX, NULL)
    CHECK(ROUTE(P, 1, 8, 64, NULL, P), NVFP4_ERR_NULL);
    CHECK(ROUTE(NULL, 1, 8, 64, &o, P), NVFP4_ERR_NULL);
    CHECK(ROUTE(P, 1, 8, 64, &o, NULL), NVFP4_ERR_NULL);
    CHECK(ROUTE(P, 3, 8, 64, &o, P), NVFP4_ERR_ENUM);
    CHECK(ROUTE(P, 1, 8, 64, &o, ODD), NVFP4_ERR_ALIGN);
    b = o, b.score = -1;
    CHECK(ROUTE(P, 1, 8, 64, &b, P), NVFP4_ERR_ENUM);
    b = o, b.group_score = INT32_MAX;
    CHECK(ROUTE(P, 1, 8, 64, &b, P), NVFP4_ERR_ENUM);
    const int32_t ends[] = {INT32_MIN, -1, 0, 65, INT32_MAX};
    for (int i = 0; i < 5; ++i) {
        b = o, b.top_k = ends[i];
        CHECK(ROUTE(P, 1, 8, 64, &b, P), NVFP4_ERR_SHAPE);
        b = o, b.groups = ends[i];
        CHECK(ROUTE(P, 1, 8, 64, &b, P), NVFP4_ERR_SHAPE);
        b = o, b.top_groups = ends[i];
        CHECK(ROUTE(P, 1, 8, 64, &b, P), NVFP4_ERR_SHAPE);
        CHECK(nvfp4_route_backward(P, P, 1, 8, 64, 64, P, ends[i], 0, 1, P, 64, P, 64, NULL), NVFP4_ERR_SHAPE);
        CHECK(nvfp4_route_backward(P, P, 1, 8, 64, 64, P, 4, ends[i] ? ends[i] : 2, 1, P, 64, P, 64, NULL), NVFP4_ERR_ENUM);
    }
    for (int i = 0; i < kN; ++i) {
        const int64_t n = kEnds[i];
        if (n < 1 || n > 64) CHECK(ROUTE(P, 1, 8, n, &o, P), NVFP4_ERR_SHAPE);
        if (n < 0) CHECK(ROUTE(P, 1, n, 64, &o, P), NVFP4_ERR_SHAPE);
        if (n >= (int64_t)1 << 31 && n <= (int64_t)1 << 40) CHECK(ROUTE(P, 1, n, 64, &o, P), NVFP4_ERR_UNSUPPORTED);
        /* (tokens * top_k past 64 bits) */
        if (n > (int64_t)1 << 40) CHECK(ROUTE(P, 1, n, 64, &o, P), NVFP4_ERR_UNSUPPORTED);
        if (n > INT32_MAX)
            CHECK(nvfp4_route_backward(P, P, 1, n, 64, 64, P, 4, 0, 1, P, 64, P, 64, NULL), NVFP4_ERR_UNSUPPORTED);
        for (int j = 0; j < kN; ++j) (void)nvfp4_route_workspace_size(n, kEnds[j]);
    }
    CHECK(nvfp4_route_backward(NULL, P, 1, 8, 64, 64, P, 4, 0, 1, P, 64, P, 64, NULL), NVFP4_ERR_NULL);
    CHECK(nvfp4_route_backward(P, P, 1, 8, 64, 64, P, 4, 0, 1, P, 63, P, 64, NULL), NVFP4_ERR_SHAPE);
    CHECK(nvfp4_route_backward(P, P, 1, 8, 64, 64, ODD, 4, 0, 1, P, 64, P, 64, NULL), NVFP4_ERR_ALIGN);
    CHECK(nvfp4_route_backward(NULL, NULL, 1, 0, 64, 64, NULL, 4, 0, 1, NULL, 64, NULL, 64, NULL), NVFP4_OK);
}

static void gemv_cases(void) {
    nvfp4_tensor w = {P, P, P, 32, 64, NVFP4_SCALE_1D}, v;
    nvfp4_mx_tensor m = {P, P, 32, 64, NVFP4_MX_E2M1}, q;
#define GEMV(x, rows, ldx, t, y, ldy, ep) nvfp4_gemv(x, 1, rows, ldx, t, y, 1, ldy, ep, NULL)
#define MXV(x, rows, ldx, t, y, ldy) nvfp4_mx_gemv(x, 1, rows, ldx, t, y, 1, ldy, NULL)
#define EXPERT(xr, T, k, t, e, ldy, ep, ws) \
    nvfp4_expert_gemv(P, 1, xr, INT64_MAX, P, T, k, t, e, P, P, 1, ldy, ep, P, ws, NULL)
    CHECK(GEMV(P, 4, 64, NULL, P, 32, 0), NVFP4_ERR_NULL);
    CHECK(GEMV(NULL, 4, 64, &w, P, 32, 0), NVFP4_ERR_NULL);
    CHECK(GEMV(P, 4, 64, &w, NULL, 32, 0), NVFP4_ERR_NULL);
    CHECK(GEMV(ODD, 4, 64, &w, P, 32, 0), NVFP4_ERR_ALIGN);
    CHECK(GEMV(P, 4, 64, &w, P, 32, INT32_MIN), NVFP4_ERR_ENUM);
    CHECK(MXV(P, 4, 64, NULL, P, 32), NVFP4_ERR_NULL);
    CHECK(MXV(P, 4, 64, &m, ODD, 32), NVFP4_ERR_ALIGN);
    CHECK(EXPERT(4, 4, 2, NULL, 2, 16, 0, SIZE_MAX), NVFP4_ERR_NULL);
    CHECK(EXPERT(4, 4, 2, &w, 2, 16, 0, 0), NVFP4_ERR_WORKSPACE);
    CHECK(EXPERT(4, 4, 2, &w, 3, 16, 0, SIZE_MAX), NVFP4_ERR_SHAPE);
    CHECK(EXPERT(5, 4, 2, &w, 2, 16, 0, SIZE_MAX), NVFP4_ERR_SHAPE);
    CHECK(EXPERT(4, 4, 2, &w, 2, 16, 3, SIZE_MAX), NVFP4_ERR_ENUM);
    CHECK(EXPERT(4, 4, INT32_MIN, &w, 2, 16, 0, SIZE_MAX), NVFP4_ERR_SHAPE);
    CHECK(EXPERT(4, 4, INT32_MAX, &w, 2, 16, 0, SIZE_MAX), NVFP4_ERR_UNSUPPORTED);
    CHECK(EXPERT(4, 4, 2, &w, INT32_MIN, 16, 0, SIZE_MAX), NVFP4_ERR_SHAPE);
    for (int i = 0; i < kN; ++i) {
        const int64_t n = kEnds[i];
        if (n < 0) {
            CHECK(GEMV(P, n, 64, &w, P, 32, 0), NVFP4_ERR_SHAPE);
            CHECK(MXV(P, n, 64, &m, P, 32), NVFP4_ERR_SHAPE);
            CHECK(EXPERT(n, n, 1, &w, 2, 16, 0, SIZE_MAX), NVFP4_ERR_SHAPE);
        }
        if (n > 1024) {
            CHECK(GEMV(P, n, 64, &w, P, 32, 0), NVFP4_ERR_UNSUPPORTED);
            CHECK(MXV(P, n, 64, &m, P, 32), NVFP4_ERR_UNSUPPORTED);
            CHECK(EXPERT(n, n, 1, &w, 2, 16, 0, SIZE_MAX), NVFP4_ERR_UNSUPPORTED);
        }
        if (n < 64) CHECK(GEMV(P, 4, n, &w, P, 32, 0), NVFP4_ERR_SHAPE);
        if (n < 32) CHECK(GEMV(P, 4, 64, &w, P, n, 0), NVFP4_ERR_SHAPE);
        v = w, v.rows = n;
        q = m, q.rows = n;
        if (n < 0 || n > INT32_MAX) {
            CHECK(GEMV(P, 4, 64, &v, P, INT64_MAX, 0), n < 0 ? NVFP4_ERR_SHAPE : NVFP4_ERR_UNSUPPORTED);
            CHECK(MXV(P, 4, 64, &q, P, INT64_MAX), n < 0 ? NVFP4_ERR_SHAPE : NVFP4_ERR_UNSUPPORTED);
            CHECK(EXPERT(4, 4, 1, &v, 1, INT64_MAX, 0, SIZE_MAX), n < 0 ? NVFP4_ERR_SHAPE : NVFP4_ERR_UNSUPPORTED);
        }
        v = w, v.cols = n;
        q = m, q.cols = n;
        if (n < 0 || n % 16) CHECK(GEMV(P, 4, INT64_MAX, &v, P, 32, 0), NVFP4_ERR_SHAPE);
        if (n < 0 || n % 32) CHECK(MXV(P, 4, INT64_MAX, &q, P, 32), NVFP4_ERR_SHAPE);
        for (int j = 0; j < kN; ++j) (void)nvfp4_expert_gemv_workspace_size(n, 4, kEnds[j]);
        (void)nvfp4_expert_gemv_workspace_size(4, INT32_MAX, n);
    }
    v = w, v.scale_mode = 2;
    CHECK(GEMV(P, 4, 64, &v, P, 32, 0), NVFP4_ERR_ENUM);
    v = w, v.tensor_scale = NULL;
    CHECK(GEMV(P, 4, 64, &v, P, 32, 0), NVFP4_ERR_NULL);
    q = m, q.elem = NVFP4_MX_E4M3;
    CHECK(MXV(P, 4, 64, &q, P, 32), NVFP4_ERR_UNSUPPORTED);
    q = m, q.elem = -5;
    CHECK(MXV(P, 4, 64, &q, P, 32), NVFP4_ERR_ENUM);
}

int main(void) {
    norm_cases();
    route_cases();
    gemv_cases();
    if (failures) {
        fprintf(stderr, "%d mismatches\n", failures);
        return 1;
    }
    printf("ok\n");
    return 0;
}
