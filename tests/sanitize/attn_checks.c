/* Host-side validation of the rotary, KV-cache and attention entry points of gdn.h, for a build of the
 * library's host code under AddressSanitizer and UndefinedBehaviorSanitizer: nothing here reaches a launch.
 * Each call passes a bad argument and must return its documented code; the fake pointers below are never
 * dereferenced.  Exit status 0 = all checks passed. */
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
    void *F = (void *)(uintptr_t)0x1000, *G = (void *)(uintptr_t)0x2000; /* aligned, never dereferenced */

    /* tables: every scaling, the extremes of the sizes, and what is refused */
    gdn_rope_params p;
    memset(&p, 0, sizeof p);
    p.rot_dim = 64; p.theta = 1e6; p.factor = 8.0; p.orig_ctx = 32768;
    gdn_rope_table t, big;
    for (int s = GDN_ROPE_PLAIN; s <= GDN_ROPE_YARN; ++s) {
        p.scaling = s;
        CHECK(gdn_rope_init(&p, &t), GDN_OK);
        for (int i = 0; i < 32; ++i) CHECK(isfinite(t.turns[i]) && t.turns[i] > 0, 1);
    }
    gdn_rope_params q = p;
    q.orig_ctx = 1; q.theta = 1.0000001;
    CHECK(gdn_rope_init(&q, &big), GDN_OK);
    q = p; q.scaling = GDN_ROPE_PLAIN; q.rot_dim = 256;
    CHECK(gdn_rope_init(&q, &big), GDN_OK);
    q.sections[0] = 2147483647; q.sections[1] = 2147483647;
    CHECK(gdn_rope_init(&q, &big), GDN_ERR_SHAPE);
    q.sections[1] = -1;
    CHECK(gdn_rope_init(&q, &big), GDN_ERR_SHAPE);
    q = p; q.rot_dim = 258;
    CHECK(gdn_rope_init(&q, &t), GDN_ERR_SHAPE);
    q = p; q.theta = NAN;
    CHECK(gdn_rope_init(&q, &t), GDN_ERR_ARG);
    CHECK(gdn_rope_init(NULL, &t), GDN_ERR_ARG);

    gdn_rows r = {F, 512, 128, 4, GDN_BF16}, o = {G, 512, 128, 4, GDN_BF16}, bad = o;
    CHECK(gdn_rope(&t, &r, &o, 1, 128, F, 0, 0, NULL), GDN_OK); /* nothing to do */
    CHECK(gdn_rope(&t, &r, &o, 5, 128, F, 3, 0, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_rope(&t, &r, &o, 1, 62, F, 3, 0, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_rope(&t, &r, &o, 1, 128, NULL, 3, 0, NULL), GDN_ERR_ARG);
    bad.ld = 0;
    CHECK(gdn_rope(&t, &r, &bad, 1, 128, F, 3, 0, NULL), GDN_ERR_ARG);
    gdn_rope_table forged = t;
    forged.axis_end[0] = 2147483647;
    CHECK(gdn_rope(&forged, &r, &o, 1, 128, F, 3, 0, NULL), GDN_ERR_ARG);

    /* the cache */
    gdn_kv kv = {4, 128, 64, 100, GDN_KV_E4M3, 0, F, F, F, F};
    size_t sb = 0;
    CHECK(gdn_kv_bytes(&kv, &sb), 4 * 128 * 64 * 100);
    CHECK(sb, 4 * 4 * 64 * 100);
    gdn_kv wrong = kv;
    wrong.n_pages = 2147483647; wrong.n_kv = 1024; wrong.page_size = 4096; wrong.d = 256;
    CHECK(gdn_kv_bytes(&wrong, NULL) > 0, 1);
    wrong.page_size = 8192;
    CHECK(gdn_kv_bytes(&wrong, NULL), 0);
    CHECK(gdn_kv_bytes(NULL, &sb), 0);
    gdn_kv_batch b = {F, F, NULL, 4, 2, 3}, huge = {F, F, NULL, 2147483647, 65535, 2147483647};
    gdn_rows k = {F, 512, 128, 4, GDN_BF16};
    CHECK(gdn_kv_write(&kv, &huge, &k, &k, NULL, NULL, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_kv_read(&kv, &huge, &k, &k, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_kv_write(&kv, &b, &k, NULL, NULL, NULL, NULL), GDN_ERR_ARG);
    CHECK(gdn_kv_write(&kv, &b, &k, &k, &big, F, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_kv_write(&kv, &b, &k, &k, &t, NULL, NULL), GDN_ERR_ARG);
    bad = k; bad.hd = -64;
    CHECK(gdn_kv_read(&kv, &b, &bad, &k, NULL), GDN_ERR_ARG);
    wrong = kv; wrong.k_scale = NULL;
    CHECK(gdn_kv_write(&wrong, &b, &k, &k, NULL, NULL, NULL), GDN_ERR_ARG);
    CHECK(gdn_kv_commit(&kv, &b, F, F, 4, NULL), GDN_ERR_RANGE);
    CHECK(gdn_kv_commit(&kv, NULL, F, F, 2, NULL), GDN_ERR_ARG);

    /* attention */
    gdn_rows qr = {F, 1024, 128, 8, GDN_BF16}, out = {G, 1024, 128, 8, GDN_BF16};
    size_t ws = gdn_attn_workspace_bytes(&kv, 8, 2, 3, 1);
    CHECK(ws > 0, 1);
    CHECK(gdn_attn_workspace_bytes(&kv, 6, 2, 3, 1), 0);
    CHECK(gdn_attn_workspace_bytes(&kv, 8, 65535, 2147483647, 1), 0);
    CHECK(gdn_attn_verify(&kv, &b, NULL, NULL, 0, NULL, &qr, &out, 0.1f, F, 16, NULL), GDN_ERR_ARG);
    CHECK(gdn_attn_verify(&kv, &b, NULL, F, 4, F, &qr, &out, 0.1f, F, ws - 1, NULL), GDN_ERR_ARG);
    CHECK(gdn_attn_verify(&kv, &b, NULL, F, 2147483647, F, &qr, &out, 0.1f, F, (size_t)-1, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_attn_verify(&kv, &huge, NULL, NULL, 0, NULL, &qr, &out, 0.1f, F, (size_t)-1, NULL), GDN_ERR_SHAPE);
    CHECK(gdn_attn_verify(&kv, &b, NULL, NULL, 0, NULL, &qr, &out, 3e38f, F, ws, NULL), GDN_ERR_ARG);
    CHECK(gdn_attn_verify(&kv, &b, NULL, NULL, 0, F, &qr, &out, 0.1f, F, ws, NULL), GDN_ERR_ARG);
    gdn_kv_batch wide = b;
    wide.n_tok = 1025; wide.n_batch = 1;
    CHECK(gdn_attn_verify(&kv, &wide, F, NULL, 0, NULL, &qr, &out, 0.1f, F, (size_t)-1, NULL), GDN_ERR_SHAPE);

    printf("%d failures\n", failures);
    return failures != 0;
}
