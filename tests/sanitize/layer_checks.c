/* Host-side validation of gdn_norm, gdn_linear_act and gdn_logprob, for a build of the library's host code under
 * AddressSanitizer and UndefinedBehaviorSanitizer: nothing here reaches a launch.  Each call passes a bad argument and
 * must return its documented code; the fake pointers below are never dereferenced.  Exit status 0 = all checks passed. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "gdn.h"

static int failures = 0;
#define CHECK(call, want)                                                                              \
    do {                                                                                               \
        long long got_ = (long long)(call);                                                            \
        if (got_ != (long long)(want)) {                                                               \
            fprintf(stderr, "%s:%d: %s returned %lld, expected %lld (%s)\n", __FILE__, __LINE__, #call, got_, \
                    (long long)(want), gdn_last_error());                                              \
            ++failures;                                                                                \
        }                                                                                              \
    } while (0)

int main(void)
{
    void *F = (void *)(uintptr_t)0x10000, *G = (void *)(uintptr_t)0x20000, *H = (void *)(uintptr_t)0x30000;
    float *S = (float *)(uintptr_t)0x40000;
    const int32_t big = 2147483647;

    gdn_rows x = {F, 512, 128, 4, GDN_BF16}, o = {G, 512, 128, 4, GDN_BF16}, r = {H, 512, 128, 4, GDN_F32}, bad;
    CHECK(gdn_norm(&x, &r, &r, S, &o, NULL, 128, 0, 1e-6f, 0, NULL), GDN_OK); /* nothing to do */
    CHECK(gdn_norm(&x, NULL, NULL, S, &o, NULL, 128, big, 1e-6f, 0, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_norm(&x, NULL, NULL, S, &o, NULL, big, 3, 1e-6f, 0, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_norm(&x, NULL, NULL, S, &o, NULL, 128, -big - 1, 1e-6f, 0, NULL), GDN_ERR_RANGE);
    CHECK(gdn_norm(&x, NULL, NULL, S, &o, NULL, 128, 3, NAN, 0, NULL), GDN_ERR_ARG);
    bad = o; bad.ld = INT64_MIN; bad.hd = INT64_MAX;
    CHECK(gdn_norm(&x, NULL, NULL, S, &bad, NULL, 128, 3, 1e-6f, 7, NULL), GDN_ERR_ARG);
    bad = o; bad.ld = 0;
    CHECK(gdn_norm(&x, NULL, NULL, S, &bad, NULL, 128, 3, 1e-6f, 0, NULL), GDN_ERR_ARG);
    bad = o; bad.dtype = big;
    CHECK(gdn_norm(&x, NULL, NULL, S, &bad, NULL, 128, 3, 1e-6f, 0, NULL), GDN_ERR_DTYPE);
    bad = x; bad.n_heads = big;
    CHECK(gdn_norm(&bad, NULL, NULL, S, &o, NULL, 128, 3, 1e-6f, 0, NULL), GDN_ERR_SHAPE);

    gdn_mat a = {F, NULL, 256, GDN_BF16}, w = {G, NULL, 256, GDN_BF16}, y = {H, NULL, 64, GDN_F32}, m;
    CHECK(gdn_linear_act(&a, &w, 0, 64, 256, NULL, 0, 0, NULL, &y, NULL, 0, NULL), GDN_OK);
    CHECK(gdn_linear_act(&a, &w, big, 64, 256, NULL, 0, 0, NULL, &y, NULL, 0, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_linear_act(&a, &w, 4, big, 256, NULL, 0, 0, NULL, &y, NULL, 0, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_linear_act(&a, &w, 4, 64, big, NULL, 0, 0, NULL, &y, NULL, 0, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_linear_act(&a, &w, 4, 64, 256, NULL, big, 0, NULL, &y, NULL, 0, NULL), GDN_ERR_ARG);
    m = y; m.ld = INT64_MIN;
    CHECK(gdn_linear_act(&a, &w, 4, 64, 256, NULL, 0, 0, &m, &m, NULL, 0, NULL) != GDN_ERR_DTYPE, 1);
    m = a; m.dtype = GDN_E4M3;
    CHECK(gdn_linear_act(&m, &w, 4, 64, 256, NULL, 0, 0, NULL, &y, NULL, 0, NULL), GDN_ERR_DTYPE);
    /* sizes at their ends: a number of bytes, or 0, and no overflow on the way */
    for (int t = -1; t <= 4; ++t)
        for (int g = 0; g < 2; ++g) {
            const int32_t s[] = {0, 1, 16, 17, 64, 65, 4096, (1 << 26) - 16, 1 << 26, big, -1};
            for (unsigned i = 0; i < sizeof s / sizeof *s; ++i)
                for (unsigned j = 0; j < sizeof s / sizeof *s; ++j)
                    for (unsigned k = 0; k < sizeof s / sizeof *s; ++k) (void)gdn_linear_act_workspace_bytes(s[i], s[j], s[k], t, g);
        }
    CHECK(gdn_linear_act_workspace_bytes(4, 64, 256, GDN_F32, 0), 0);
    CHECK(gdn_linear_act_workspace_bytes(1, 5120, 4096, GDN_BF16, 0) > 0, 1);

    gdn_mat l = {F, NULL, 1000, GDN_BF16};
    int32_t *ids = (int32_t *)G;
    CHECK(gdn_logprob(&l, 0, 1000, 1.0f, ids, 1, S, NULL, S, S, NULL, NULL, 0, NULL, 0, NULL), GDN_OK);
    CHECK(gdn_logprob(&l, big, 1000, 1.0f, ids, 1, S, NULL, S, S, NULL, NULL, 0, NULL, 0, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_logprob(&l, 3, big, 1.0f, ids, 1, S, NULL, S, S, NULL, NULL, 0, NULL, 0, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_logprob(&l, 3, 1000, 1.0f, ids, big, S, NULL, S, S, NULL, NULL, 0, NULL, 0, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_logprob(&l, 3, 1000, 1.0f, ids, 1, S, NULL, S, S, ids, S, big, NULL, 0, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_logprob(&l, 3, 1000, INFINITY, ids, 1, S, NULL, S, S, NULL, NULL, 0, NULL, 0, NULL), GDN_ERR_ARG);
    CHECK(gdn_logprob_workspace_bytes(big, 1000, GDN_BF16, 0, 0), 0);
    CHECK(gdn_logprob_workspace_bytes(1, 1 << 24, GDN_F32, 64, 64) > 0, 1);
    CHECK(gdn_logprob_workspace_bytes(1 << 26, 1 << 24, GDN_F32, 64, 64), 0); /* a slice for each row needs none */

    printf("%d failures\n", failures);
    return failures != 0;
}
