// gdn_layer_abi.cpp - C ABI of the norms, the products with an epilogue and the log probabilities: validation and dispatch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/gdn.h"
#include "gdn_internal.h"

#define GDN_API extern "C" __attribute__((visibility("default")))

static_assert((int)gdn::kF32 == GDN_F32 && (int)gdn::kBf16 == GDN_BF16 && (int)gdn::kE4m3 == GDN_E4M3 && (int)gdn::kI8 == GDN_I8,
              "types");

namespace gdn {
namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool plain(int t) { return t == GDN_F32 || t == GDN_BF16; }
bool codes(int t) { return t == GDN_E4M3 || t == GDN_I8; }
int64_t elem_bytes(int t) { return t == GDN_F32 ? 4 : t == GDN_BF16 ? 2 : 1; }

constexpr int64_t kMaxSide = (int64_t)1 << 26;  // rows, columns and depth of a product, rows of logits

// What is written on the memory of what is read: only the same rows, where that is allowed.
int check_shared(const char *fn, const char *what, const gdn_rows *w, const char *other, const gdn_rows *r, bool may)
{
    if (!w || !r || w->ptr != r->ptr) return GDN_OK;
    if (!may || w->ld != r->ld || w->hd != r->hd || w->dtype != r->dtype)
        return abi_fail(GDN_ERR_ARG, "%s: %s on %s's memory%s", fn, what, other, may ? " with other strides or another type" : "");
    return GDN_OK;
}

int check_norm_rows(const char *fn, const char *what, const gdn_rows *r, int n_heads, bool may_codes)
{
    if (!r->ptr) return abi_fail(GDN_ERR_ARG, "%s: %s: ptr is NULL", fn, what);
    if (!plain(r->dtype) && !(may_codes && codes(r->dtype)))
        return abi_fail(GDN_ERR_DTYPE, "%s: %s: dtype must be GDN_F32 or GDN_BF16%s", fn, what,
                        may_codes ? ", GDN_E4M3 or GDN_I8" : "");
    if (r->n_heads != n_heads) return abi_fail(GDN_ERR_SHAPE, "%s: %s has %d heads, x has %d", fn, what, r->n_heads, n_heads);
    if (!aligned(r->ptr, elem_bytes(r->dtype))) return abi_fail(GDN_ERR_ARG, "%s: %s is not aligned to its elements", fn, what);
    return GDN_OK;
}

MatView mat_view(const gdn_mat &m) { return MatView{m.ptr, m.scale, m.ld, m.dtype}; }

// A workspace as the entry points take it.
int check_workspace(const char *fn, const void *ws, size_t got, size_t need)
{
    if (!need) return GDN_OK;
    if (!ws || !aligned(ws, 16)) return abi_fail(GDN_ERR_ARG, "%s: workspace must not be NULL and 16-byte aligned", fn);
    if (got < need) return abi_fail(GDN_ERR_ARG, "%s: workspace of %zu bytes, needs %zu", fn, got, need);
    return GDN_OK;
}

bool linear_sizes(int64_t M, int64_t N, int64_t K, int dtype)
{
    return M >= 0 && M < kMaxSide && N >= 1 && N < kMaxSide && K >= 1 && K < kMaxSide && K * elem_bytes(dtype) % 16 == 0 &&
           (dtype != GDN_I8 || K < 1 << 17);
}

// out [M][N] or residual: rows to read or write as they are.
int check_result(const char *fn, const char *what, const gdn_mat *m, int64_t rows, int64_t cols, bool written)
{
    if (!m->ptr) return abi_fail(GDN_ERR_ARG, "%s: %s: ptr is NULL", fn, what);
    if (!plain(m->dtype)) return abi_fail(GDN_ERR_DTYPE, "%s: %s: dtype must be GDN_F32 or GDN_BF16", fn, what);
    if (m->scale) return abi_fail(GDN_ERR_ARG, "%s: %s takes no scale", fn, what);
    if (!aligned(m->ptr, elem_bytes(m->dtype))) return abi_fail(GDN_ERR_ARG, "%s: %s is not aligned to its elements", fn, what);
    if (written && rows > 1 && (m->ld < 0 ? -(__int128)m->ld : m->ld) < cols)
        return abi_fail(GDN_ERR_ARG, "%s: %s: rows that are written lie on top of each other", fn, what);
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

GDN_API int gdn_norm(const gdn_rows *x, const gdn_rows *residual, const gdn_rows *total, const float *weight,
                     const gdn_rows *out, float *scale, int32_t d, int32_t n_tok, float eps, int32_t mode, void *stream)
{
    const char *fn = "gdn_norm";
    if (!x || !out) return abi_fail(GDN_ERR_ARG, "%s: x and out must not be NULL", fn);
    if (mode != GDN_NORM_RMS && mode != GDN_NORM_NONE) return abi_fail(GDN_ERR_ARG, "%s: unknown mode %d", fn, mode);
    if (n_tok < 0) return abi_fail(GDN_ERR_RANGE, "%s: n_tok %d is negative", fn, n_tok);
    const int most = mode == GDN_NORM_NONE ? kNormMaxLong : kNormMaxD;
    if (d < 1 || d > most) return abi_fail(GDN_ERR_SHAPE, "%s: d must be 1 .. %d in this mode (got %d)", fn, most, d);
    if (x->n_heads < 1 || x->n_heads > 8192) return abi_fail(GDN_ERR_SHAPE, "%s: n_heads must be 1 .. 8192", fn);
    if ((int64_t)n_tok * x->n_heads > kMaxTokenRows) return abi_fail(GDN_ERR_SHAPE, "%s: more than 2^26 rows", fn);
    if (mode == GDN_NORM_RMS && (!(eps >= 0x1p-126f) || !std::isfinite(eps)))
        return abi_fail(GDN_ERR_ARG, "%s: eps must be finite and at least 2^-126", fn);
    if (codes(out->dtype) != (scale != nullptr))
        return abi_fail(GDN_ERR_ARG, "%s: scale is given for an out of 8 bits, and only then", fn);
    if (!aligned(scale, 4) || !aligned(weight, 4))
        return abi_fail(GDN_ERR_ARG, "%s: scale and weight must be 4-byte aligned", fn);
    if (!n_tok) return abi_ok();
    if (int r = check_norm_rows(fn, "x", x, x->n_heads, false)) return r;
    if (int r = residual ? check_norm_rows(fn, "residual", residual, x->n_heads, false) : GDN_OK) return r;
    if (int r = total ? check_norm_rows(fn, "total", total, x->n_heads, false) : GDN_OK) return r;
    if (int r = check_norm_rows(fn, "out", out, x->n_heads, true)) return r;
    if (int r = abi_check_apart(fn, "out", out, n_tok, d)) return r;
    if (int r = total ? abi_check_apart(fn, "total", total, n_tok, d) : GDN_OK) return r;
    if (int r = check_shared(fn, "total", total, "x", x, true)) return r;
    if (int r = check_shared(fn, "total", total, "residual", residual, true)) return r;
    if (int r = check_shared(fn, "out", out, "x", x, true)) return r;
    if (int r = check_shared(fn, "out", out, "residual", residual, true)) return r;
    if (int r = check_shared(fn, "out", out, "total", total, false)) return r;
    NormArgs a{};
    a.x = rows_view(*x);
    if (residual) a.residual = rows_view(*residual);
    if (total) a.total = rows_view(*total);
    a.out = rows_view(*out);
    a.weight = weight;
    a.scale = scale;
    a.out_type = out->dtype;
    a.d = d;
    a.n_heads = x->n_heads;
    a.n_tok = n_tok;
    a.rms = mode == GDN_NORM_RMS;
    a.eps = eps;
    if (hipError_t e = launch_norm(a, static_cast<hipStream_t>(stream)))
        return abi_fail(GDN_ERR_HIP, "%s launch: %s", fn, hipGetErrorString(e));
    return abi_ok();
}

GDN_API size_t gdn_linear_act_workspace_bytes(int32_t M, int32_t N, int32_t K, int32_t dtype, int32_t gated)
{
    if ((dtype != GDN_BF16 && !codes(dtype)) || !linear_sizes(M, N, K, dtype)) return 0;
    return linear_act_workspace_bytes(M, N, K, dtype, gated != 0);
}

GDN_API int gdn_linear_act(const gdn_mat *x, const gdn_mat *w, int32_t M, int32_t N, int32_t K, const float *bias, int32_t act,
                           int32_t gated, const gdn_mat *residual, const gdn_mat *out, void *workspace, size_t ws_bytes,
                           void *stream)
{
    const char *fn = "gdn_linear_act";
    if (!x || !w || !out) return abi_fail(GDN_ERR_ARG, "%s: x, w and out must not be NULL", fn);
    if (x->dtype != GDN_BF16 && !codes(x->dtype))
        return abi_fail(GDN_ERR_DTYPE, "%s: x and w must be GDN_BF16, GDN_E4M3 or GDN_I8", fn);
    if (w->dtype != x->dtype) return abi_fail(GDN_ERR_DTYPE, "%s: x and w must have the same type", fn);
    if (act < GDN_ACT_NONE || act > GDN_ACT_SIGMOID) return abi_fail(GDN_ERR_ARG, "%s: unknown act %d", fn, act);
    if (M < 0) return abi_fail(GDN_ERR_RANGE, "%s: M %d is negative", fn, M);
    if (!linear_sizes(M, N, K, x->dtype))
        return abi_fail(GDN_ERR_SHAPE, "%s: M = %d, N = %d, K = %d: below 2^26, K in whole runs of 16 bytes (GDN_I8: below 2^17)",
                        fn, M, N, K);
    if (!M) return abi_ok();
    const int64_t per = 16 / elem_bytes(x->dtype);
    for (const gdn_mat *m : {x, w}) {
        const char *what = m == x ? "x" : "w";
        if (!m->ptr) return abi_fail(GDN_ERR_ARG, "%s: %s: ptr is NULL", fn, what);
        if (!aligned(m->ptr, 16) || m->ld % per) return abi_fail(GDN_ERR_ARG, "%s: %s: rows must be 16-byte aligned", fn, what);
        if ((m->scale != nullptr) != codes(m->dtype))
            return abi_fail(GDN_ERR_ARG, "%s: %s: the 8-bit types take a scale, GDN_BF16 none", fn, what);
        if (!aligned(m->scale, 4)) return abi_fail(GDN_ERR_ARG, "%s: %s: scale must be 4-byte aligned", fn, what);
    }
    if (!aligned(bias, 4)) return abi_fail(GDN_ERR_ARG, "%s: bias must be 4-byte aligned", fn);
    if (int r = check_result(fn, "out", out, M, N, true)) return r;
    if (int r = residual ? check_result(fn, "residual", residual, M, N, false) : GDN_OK) return r;
    if (residual && residual->ptr == out->ptr && (residual->dtype != out->dtype || (residual->ld != out->ld && M > 1)))
        return abi_fail(GDN_ERR_ARG, "%s: out on residual's memory with another stride or type", fn);
    if (out->ptr == x->ptr || out->ptr == w->ptr) return abi_fail(GDN_ERR_ARG, "%s: out on x's or w's memory", fn);
    if (int r = check_workspace(fn, workspace, ws_bytes, linear_act_workspace_bytes(M, N, K, x->dtype, gated != 0))) return r;
    LinearActArgs a{};
    a.x = mat_view(*x);
    a.w = mat_view(*w);
    if (residual) a.residual = mat_view(*residual);
    a.out = mat_view(*out);
    a.bias = bias;
    a.M = M;
    a.N = N;
    a.K = K;
    a.act = act;
    a.gated = gated != 0;
    a.ws = static_cast<unsigned char *>(workspace);
    if (hipError_t e = launch_linear_act(a, static_cast<hipStream_t>(stream)))
        return abi_fail(GDN_ERR_HIP, "%s launch: %s", fn, hipGetErrorString(e));
    return abi_ok();
}

static bool logprob_sizes(int64_t n_rows, int V, int dtype, int n_ids, int top_k)
{
    return n_rows >= 0 && n_rows <= kMaxSide && V >= 1 && V <= 1 << 24 && plain(dtype) && n_ids >= 0 && n_ids <= kMaxIds &&
           top_k >= 0 && top_k <= kMaxTop && top_k <= V;
}

GDN_API size_t gdn_logprob_workspace_bytes(int32_t n_rows, int32_t n_vocab, int32_t dtype, int32_t n_ids, int32_t top_k)
{
    if (!logprob_sizes(n_rows, n_vocab, dtype, n_ids, top_k)) return 0;
    return logprob_workspace_bytes(n_rows, n_vocab, dtype == GDN_BF16, n_ids, top_k);
}

GDN_API int gdn_logprob(const gdn_mat *logits, int32_t n_rows, int32_t n_vocab, float temperature, const int32_t *ids,
                        int32_t n_ids, float *logprob, int32_t *rank, float *lse, float *entropy, int32_t *top_ids,
                        float *top_logprob, int32_t top_k, void *workspace, size_t ws_bytes, void *stream)
{
    const char *fn = "gdn_logprob";
    if (!logits) return abi_fail(GDN_ERR_ARG, "%s: logits must not be NULL", fn);
    if (!plain(logits->dtype)) return abi_fail(GDN_ERR_DTYPE, "%s: logits must be GDN_F32 or GDN_BF16", fn);
    if (logits->scale) return abi_fail(GDN_ERR_ARG, "%s: logits take no scale", fn);
    if (n_rows < 0) return abi_fail(GDN_ERR_RANGE, "%s: n_rows %d is negative", fn, n_rows);
    if (!logprob_sizes(n_rows, n_vocab, logits->dtype, n_ids, top_k))
        return abi_fail(GDN_ERR_SHAPE, "%s: n_rows %d (at most 2^26), n_vocab %d (1 .. 2^24), n_ids %d (0 .. %d) or top_k %d (0 .. %d, n_vocab)",
                        fn, n_rows, n_vocab, n_ids, kMaxIds, top_k, kMaxTop);
    if (!(temperature >= 0x1p-20f && temperature <= 0x1p20f))
        return abi_fail(GDN_ERR_ARG, "%s: temperature must be 2^-20 .. 2^20", fn);
    if ((n_ids > 0) != (ids && (logprob || rank)) || (n_ids == 0 && (logprob || rank)))
        return abi_fail(GDN_ERR_ARG, "%s: n_ids, ids and logprob or rank come together", fn);
    if ((top_k > 0) != (top_ids && top_logprob) || (top_k == 0 && (top_ids || top_logprob)))
        return abi_fail(GDN_ERR_ARG, "%s: top_k, top_ids and top_logprob come together", fn);
    if (!n_ids && !top_k && !lse && !entropy) return abi_fail(GDN_ERR_ARG, "%s: no output is asked for", fn);
    for (const void *p : {(const void *)ids, (const void *)logprob, (const void *)rank, (const void *)lse, (const void *)entropy,
                          (const void *)top_ids, (const void *)top_logprob})
        if (!aligned(p, 4)) return abi_fail(GDN_ERR_ARG, "%s: ids and outputs must be 4-byte aligned", fn);
    if (!n_rows) return abi_ok();
    if (!logits->ptr || !aligned(logits->ptr, elem_bytes(logits->dtype)))
        return abi_fail(GDN_ERR_ARG, "%s: logits: ptr must not be NULL and aligned to its elements", fn);
    if (int r = check_workspace(fn, workspace, ws_bytes,
                                logprob_workspace_bytes(n_rows, n_vocab, logits->dtype == GDN_BF16, n_ids, top_k)))
        return r;
    LogprobArgs a{};
    a.logits = logits->ptr;
    a.ld = logits->ld;
    a.bf16 = logits->dtype == GDN_BF16;
    a.n_rows = n_rows;
    a.V = n_vocab;
    a.n_ids = n_ids;
    a.top_k = top_k;
    a.inv_t = 1.0f / temperature;
    a.ids = ids;
    a.logprob = logprob;
    a.rank = rank;
    a.lse = lse;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprob = top_logprob;
    a.ws = static_cast<unsigned char *>(workspace);
    if (hipError_t e = launch_logprob(a, static_cast<hipStream_t>(stream)))
        return abi_fail(GDN_ERR_HIP, "%s launch: %s", fn, hipGetErrorString(e));
    return abi_ok();
}
