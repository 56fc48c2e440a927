// gdn_attn_abi.cpp - C ABI of the drafted tokens' attention: validation and dispatch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <memory>
#include <new>

#include "../../include/gdn.h"
#include "gdn_internal.h"

#define GDN_API extern "C" __attribute__((visibility("default")))

using gdn::abi_fail;

namespace {

constexpr int kMaxTreeNodes = 1024;

int check_heads(const char *fn, const gdn_kv *kv, int n_q)
{
    if (n_q < kv->n_kv || n_q % kv->n_kv || n_q > 65536)
        return abi_fail(GDN_ERR_SHAPE, "%s: %d query heads must be a multiple of the %d KV heads, at most 65536", fn, n_q, kv->n_kv);
    return GDN_OK;
}

int check_tree(const char *fn, const gdn_kv_batch *b, const int32_t *parent, hipStream_t st)
{
    const size_t n = (size_t)b->n_batch * b->n_tok;
    std::unique_ptr<int32_t[]> h(new (std::nothrow) int32_t[n]);
    if (!h) return abi_fail(GDN_ERR_HIP, "%s: no host memory for the index check", fn);
    if (int r = gdn::abi_fetch_i32(parent, n, st, h.get())) return r;
    for (size_t i = 0; i < n; ++i) {
        const int32_t node = (int32_t)(i % b->n_tok), p = h[i];
        if (p < -1 || p >= node || (node == 0 && p != -1))
            return abi_fail(GDN_ERR_RANGE, "%s: parent[%zu][%d] = %d", fn, i / b->n_tok, node, p);
    }
    return GDN_OK;
}

int check_prefix(const char *fn, const gdn_kv *kv, const int32_t *pages, int32_t n, const int32_t *len, hipStream_t st)
{
    std::unique_ptr<int32_t[]> h(new (std::nothrow) int32_t[(size_t)n + 1]);
    if (!h) return abi_fail(GDN_ERR_HIP, "%s: no host memory for the index check", fn);
    if (int r = gdn::abi_fetch_i32(pages, n, st, h.get())) return r;
    if (int r = gdn::abi_fetch_i32(len, 1, st, h.get() + n)) return r;
    const int64_t have = h[n];
    if (have < 0 || have > (int64_t)n * kv->page_size)
        return abi_fail(GDN_ERR_RANGE, "%s: prefix_len = %d outside [0, %d pages]", fn, h[n], n);
    for (int64_t p = 0; p * kv->page_size < have; ++p)
        if (h[p] < 0 || h[p] >= kv->n_pages)
            return abi_fail(GDN_ERR_RANGE, "%s: prefix_pages[%lld] = %d outside [0, %d)", fn, (long long)p, h[p], kv->n_pages);
    return GDN_OK;
}

}  // namespace

GDN_API size_t gdn_attn_workspace_bytes(const gdn_kv *kv, int32_t n_q, int32_t n_batch, int32_t n_tok, int32_t prefix)
{
    const char *fn = "gdn_attn_workspace_bytes";
    if (gdn::abi_check_kv(fn, kv, false) || check_heads(fn, kv, n_q)) return 0;
    if (n_batch < 1 || n_batch > 65535 || n_tok < 1 || (int64_t)n_batch * n_tok > gdn::kMaxTokenRows) {
        abi_fail(GDN_ERR_SHAPE, "%s: n_batch or n_tok out of range", fn);
        return 0;
    }
    gdn::AttnPlan p;
    if (!gdn::attn_plan(kv->d, kv->format, kv->page_size, kv->n_kv, n_q / kv->n_kv, n_batch, n_tok, 1, prefix != 0, 1, p)) {
        abi_fail(GDN_ERR_SHAPE, "%s: 2^26 rows of a KV head or more", fn);
        return 0;
    }
    return p.bytes;
}

GDN_API int gdn_attn_verify(const gdn_kv *kv, const gdn_kv_batch *batch, const int32_t *parent, const int32_t *prefix_pages,
                            int32_t max_prefix_pages, const int32_t *prefix_len, const gdn_rows *q, const gdn_rows *out,
                            float scale, void *workspace, size_t ws_bytes, void *stream)
{
    const char *fn = "gdn_attn_verify";
    if (int r = gdn::abi_check_kv(fn, kv, true)) return r;
    if (int r = gdn::abi_check_batch(fn, batch)) return r;
    if (!q || !out) return abi_fail(GDN_ERR_ARG, "%s: q and out must not be NULL", fn);
    if (int r = check_heads(fn, kv, q->n_heads)) return r;
    if (int r = gdn::abi_check_rows(fn, "q", q, q->n_heads)) return r;
    if (int r = gdn::abi_check_rows(fn, "out", out, q->n_heads)) return r;
    if (int r = gdn::abi_check_apart(fn, "out", out, (int64_t)batch->n_batch * batch->n_tok, kv->d)) return r;
    if (q->dtype != GDN_BF16 || out->dtype != GDN_BF16) return abi_fail(GDN_ERR_DTYPE, "%s: q and out must be GDN_BF16", fn);
    // Workgroups read rows of q that others have not reached yet: out may only lie where the same row of q does.
    const int64_t rows = (int64_t)batch->n_batch * batch->n_tok;
    if (q->ptr == out->ptr && ((rows > 1 && q->ld != out->ld) || (q->n_heads > 1 && q->hd != out->hd)))
        return abi_fail(GDN_ERR_ARG, "%s: out is q's memory with other strides", fn);
    if (!(scale > 0.0f) || !std::isfinite(scale * gdn::kLog2E)) return abi_fail(GDN_ERR_ARG, "%s: scale must be finite and > 0", fn);
    if (parent && batch->n_tok > kMaxTreeNodes)
        return abi_fail(GDN_ERR_SHAPE, "%s: a tree of %d nodes, at most %d", fn, batch->n_tok, kMaxTreeNodes);
    if ((prefix_pages != nullptr) != (prefix_len != nullptr))
        return abi_fail(GDN_ERR_ARG, "%s: prefix_pages and prefix_len go together", fn);
    if (prefix_pages && max_prefix_pages < 1) return abi_fail(GDN_ERR_SHAPE, "%s: max_prefix_pages must be >= 1", fn);
    gdn::AttnArgs a{};
    a.grp = q->n_heads / kv->n_kv;
    if (!gdn::attn_plan(kv->d, kv->format, kv->page_size, kv->n_kv, a.grp, batch->n_batch, batch->n_tok, batch->max_pages,
                        prefix_pages != nullptr, max_prefix_pages, a.plan))
        return abi_fail(GDN_ERR_SHAPE, "%s: the call's tiles or its tables' positions pass 2^31", fn);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u))
        return abi_fail(GDN_ERR_ARG, "%s: workspace must be 16-byte aligned device memory", fn);
    if (ws_bytes < a.plan.bytes)
        return abi_fail(GDN_ERR_ARG, "%s: workspace smaller than gdn_attn_workspace_bytes()", fn);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (kv->flags & GDN_F_CHECK_INDICES) {
        if (int r = gdn::abi_check_places(fn, kv, batch, true, st)) return r;
        if (parent) {
            if (int r = check_tree(fn, batch, parent, st)) return r;
        }
        if (prefix_pages) {
            if (int r = check_prefix(fn, kv, prefix_pages, max_prefix_pages, prefix_len, st)) return r;
        }
    }
    a.kv = gdn::kv_view(*kv);
    a.b = gdn::kv_batch_view(*batch);
    a.q = gdn::rows_view(*q);
    a.out = gdn::rows_view(*out);
    a.scale = scale * gdn::kLog2E;
    a.parent = parent;
    a.prefix_pages = prefix_pages;
    a.prefix_len = prefix_len;
    a.max_prefix_pages = max_prefix_pages;
    a.ws = static_cast<unsigned char *>(workspace);
    if (hipError_t e = gdn::launch_attn(a, st)) return abi_fail(GDN_ERR_HIP, "%s launch: %s", fn, hipGetErrorString(e));
    return gdn::abi_ok();
}
