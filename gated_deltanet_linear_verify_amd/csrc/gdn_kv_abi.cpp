// gdn_kv_abi.cpp - C ABI of the rotary positions and the paged KV cache: validation and dispatch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <memory>
#include <new>

#include "../../include/gdn.h"
#include "gdn_internal.h"

#define GDN_API extern "C" __attribute__((visibility("default")))

static_assert(gdn::kMaxRopePairs == GDN_ROPE_MAX_PAIRS, "rope table size");
static_assert((int)gdn::kKvBf16 == GDN_KV_BF16 && (int)gdn::kKvE4m3 == GDN_KV_E4M3 && (int)gdn::kKvI8 == GDN_KV_I8,
              "cache formats");

static constexpr double kPi = 3.14159265358979323846;

namespace gdn {
namespace {

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t elem_bytes(int dtype) { return dtype == GDN_BF16 ? 2 : 4; }

int check_table(const char *fn, const gdn_rope_table *t, int d)
{
    bool good = t->rot_dim >= 2 && t->rot_dim <= 2 * GDN_ROPE_MAX_PAIRS && t->rot_dim % 2 == 0 &&
                (t->layout == GDN_ROPE_HALF || t->layout == GDN_ROPE_INTERLEAVED) && (t->n_axes == 1 || t->n_axes == 4);
    for (int a = 0; good && a < 4; ++a) good = t->axis_end[a] >= (a ? t->axis_end[a - 1] : 0);
    good = good && t->axis_end[t->n_axes - 1] == t->rot_dim / 2;
    if (!good) return abi_fail(GDN_ERR_ARG, "%s: the rope table was not made by gdn_rope_init", fn);
    if (t->rot_dim > d) return abi_fail(GDN_ERR_SHAPE, "%s: rot_dim %d exceeds the head's %d channels", fn, t->rot_dim, d);
    return GDN_OK;
}

RopeTab tab_view(const gdn_rope_table &t)
{
    RopeTab v{};
    v.rot = t.rot_dim;
    v.pairs = t.rot_dim / 2;
    v.interleaved = t.layout == GDN_ROPE_INTERLEAVED;
    v.n_axes = t.n_axes;
    for (int a = 0; a < 4; ++a) v.axis_end[a] = t.axis_end[a];
    v.mscale = t.mscale;
    std::memcpy(v.turns, t.turns, sizeof v.turns);
    return v;
}

}  // namespace

KvView kv_view(const gdn_kv &kv)
{
    int shift = 0;
    while ((1 << shift) < kv.page_size) ++shift;
    return KvView{static_cast<unsigned char *>(kv.k), static_cast<unsigned char *>(kv.v), kv.k_scale, kv.v_scale, kv.n_kv,
                  kv.d, shift, kv.n_pages, kv.format};
}
KvBatchView kv_batch_view(const gdn_kv_batch &b)
{
    return KvBatchView{b.block_table, b.start, b.n_new, b.max_pages, b.n_batch, b.n_tok};
}
RowsView rows_view(const gdn_rows &r) { return RowsView{r.ptr, r.ld, r.hd, r.dtype == GDN_BF16}; }

int abi_check_kv(const char *fn, const gdn_kv *kv, bool pointers)
{
    if (!kv) return abi_fail(GDN_ERR_ARG, "%s: kv is NULL", fn);
    if (kv->format != GDN_KV_BF16 && kv->format != GDN_KV_E4M3 && kv->format != GDN_KV_I8)
        return abi_fail(GDN_ERR_DTYPE, "%s: unknown cache format %d", fn, kv->format);
    if (kv->d != 64 && kv->d != 128 && kv->d != 256)
        return abi_fail(GDN_ERR_SHAPE, "%s: head dim must be 64, 128 or 256 (got %d)", fn, kv->d);
    if (kv->n_kv < 1 || kv->n_kv > 1024 || kv->n_pages < 1)
        return abi_fail(GDN_ERR_SHAPE, "%s: n_kv must be 1 .. 1024 and n_pages positive", fn);
    if (kv->page_size < 16 || kv->page_size > 4096 || (kv->page_size & (kv->page_size - 1)))
        return abi_fail(GDN_ERR_SHAPE, "%s: page_size must be a power of two, 16 .. 4096 (got %d)", fn, kv->page_size);
    if (kv->flags & ~GDN_F_CHECK_INDICES) return abi_fail(GDN_ERR_ARG, "%s: unknown kv flag bits 0x%x", fn, kv->flags);
    if (!pointers) return GDN_OK;
    if (!kv->k || !kv->v) return abi_fail(GDN_ERR_ARG, "%s: kv->k and kv->v must not be NULL", fn);
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16))
        return abi_fail(GDN_ERR_ARG, "%s: kv->k and kv->v must be 16-byte aligned", fn);
    const bool scaled = kv->format != GDN_KV_BF16;
    if ((kv->k_scale != nullptr) != scaled || (kv->v_scale != nullptr) != scaled)
        return abi_fail(GDN_ERR_ARG, "%s: the 8-bit formats take k_scale and v_scale, the bf16 format neither", fn);
    if (!aligned(kv->k_scale, 4) || !aligned(kv->v_scale, 4))
        return abi_fail(GDN_ERR_ARG, "%s: scales must be 4-byte aligned", fn);
    return GDN_OK;
}

int abi_check_rows(const char *fn, const char *what, const gdn_rows *r, int n_heads)
{
    if (!r || !r->ptr) return abi_fail(GDN_ERR_ARG, "%s: %s is NULL", fn, what);
    if (r->dtype != GDN_F32 && r->dtype != GDN_BF16)
        return abi_fail(GDN_ERR_DTYPE, "%s: %s: dtype must be GDN_F32 or GDN_BF16", fn, what);
    if (r->n_heads != n_heads)
        return abi_fail(GDN_ERR_SHAPE, "%s: %s has %d heads, expected %d", fn, what, r->n_heads, n_heads);
    const int64_t per = 16 / (int64_t)elem_bytes(r->dtype);
    if (!aligned(r->ptr, 16) || r->ld % per || r->hd % per)
        return abi_fail(GDN_ERR_ARG, "%s: %s: rows and heads must be 16-byte aligned", fn, what);
    return GDN_OK;
}

// Runs of d elements at a ld + b hd, 0 <= a < n_rows, 0 <= b < n_heads, apart from each other?  Two of them overlap
// where |a ld + b hd| < d for differences a, b that are not both 0.
static bool rows_apart(const gdn_rows *r, int64_t n_rows, int d)
{
    __int128 ld = r->ld, hd = r->hd;
    if (ld < 0) ld = -ld;
    if (hd < 0) hd = -hd;  // the mirrored case has the same differences, with the other sign of a
    const __int128 a_max = n_rows - 1, b_max = r->n_heads - 1;
    if ((a_max > 0 && ld < d) || (b_max > 0 && hd < d)) return false;
    if (a_max == 0 || b_max == 0 || ld >= b_max * hd + d || hd >= a_max * ld + d) return true;  // one inside the other
    for (__int128 b = 1; b <= b_max; ++b) {
        const __int128 a = b * hd / ld;  // the difference in rows that comes nearest from below, and the next one
        if ((a <= a_max && b * hd - a * ld < d) || (a < a_max && (a + 1) * ld - b * hd < d)) return false;
    }
    return true;
}

int abi_check_apart(const char *fn, const char *what, const gdn_rows *r, int64_t n_rows, int d)
{
    if (!rows_apart(r, n_rows, d))
        return abi_fail(GDN_ERR_ARG, "%s: %s: rows or heads that are written lie on top of each other", fn, what);
    return GDN_OK;
}

int abi_check_batch(const char *fn, const gdn_kv_batch *b)
{
    if (!b || !b->block_table || !b->start)
        return abi_fail(GDN_ERR_ARG, "%s: batch, its block_table and its start must not be NULL", fn);
    if (b->n_batch < 1 || b->n_batch > 65535) return abi_fail(GDN_ERR_RANGE, "%s: n_batch %d outside [1, 65535]", fn, b->n_batch);
    if (b->n_tok < 1) return abi_fail(GDN_ERR_RANGE, "%s: n_tok must be >= 1", fn);
    if (b->max_pages < 1) return abi_fail(GDN_ERR_SHAPE, "%s: max_pages must be >= 1", fn);
    if ((int64_t)b->n_batch * b->n_tok > kMaxTokenRows)
        return abi_fail(GDN_ERR_SHAPE, "%s: more than 2^26 token rows", fn);
    return GDN_OK;
}

int abi_check_places(const char *fn, const gdn_kv *kv, const gdn_kv_batch *b, bool from_zero, hipStream_t st)
{
    if (!(kv->flags & GDN_F_CHECK_INDICES)) return GDN_OK;
    const size_t B = b->n_batch, np = B * b->max_pages;
    std::unique_ptr<int32_t[]> h(new (std::nothrow) int32_t[np + 2 * B]);
    if (!h) return abi_fail(GDN_ERR_HIP, "%s: no host memory for the index check", fn);
    int32_t *start = h.get() + np, *n_new = start + B;
    if (int r = abi_fetch_i32(b->block_table, np, st, h.get())) return r;
    if (int r = abi_fetch_i32(b->start, B, st, start)) return r;
    if (b->n_new) {
        if (int r = abi_fetch_i32(b->n_new, B, st, n_new)) return r;
    }
    for (size_t e = 0; e < B; ++e) {
        const int64_t n = b->n_new ? n_new[e] : b->n_tok;
        if (n < 0 || n > b->n_tok) return abi_fail(GDN_ERR_RANGE, "%s: n_new[%zu] = %d outside [0, n_tok]", fn, e, n_new[e]);
        if (start[e] < 0) return abi_fail(GDN_ERR_RANGE, "%s: start[%zu] = %d is negative", fn, e, start[e]);
        const int64_t end = start[e] + n;
        if (end > (int64_t)b->max_pages * kv->page_size)
            return abi_fail(GDN_ERR_RANGE, "%s: entry %zu ends at position %lld, past its %d pages", fn, e, (long long)end,
                            b->max_pages);
        if (!n) continue;
        for (int64_t p = (from_zero ? 0 : start[e]) / kv->page_size; p * kv->page_size < end; ++p) {
            const int32_t page = h[e * b->max_pages + p];
            if (page < 0 || page >= kv->n_pages)
                return abi_fail(GDN_ERR_RANGE, "%s: block_table[%zu][%lld] = %d outside [0, %d)", fn, e, (long long)p, page,
                                kv->n_pages);
        }
    }
    return GDN_OK;
}

}  // namespace gdn

using gdn::abi_fail;

GDN_API int gdn_rope_init(const gdn_rope_params *p, gdn_rope_table *t)
{
    const char *fn = "gdn_rope_init";
    if (!p || !t) return abi_fail(GDN_ERR_ARG, "%s: params and table must not be NULL", fn);
    if (p->rot_dim < 2 || p->rot_dim > 2 * GDN_ROPE_MAX_PAIRS || p->rot_dim % 2)
        return abi_fail(GDN_ERR_SHAPE, "%s: rot_dim must be even, 2 .. %d (got %d)", fn, 2 * GDN_ROPE_MAX_PAIRS, p->rot_dim);
    if (p->layout != GDN_ROPE_HALF && p->layout != GDN_ROPE_INTERLEAVED)
        return abi_fail(GDN_ERR_ARG, "%s: unknown layout %d", fn, p->layout);
    if (p->scaling < GDN_ROPE_PLAIN || p->scaling > GDN_ROPE_YARN)
        return abi_fail(GDN_ERR_ARG, "%s: unknown scaling %d", fn, p->scaling);
    if (!(p->theta > 1.0) || !std::isfinite(p->theta)) return abi_fail(GDN_ERR_ARG, "%s: theta must be finite and > 1", fn);
    if (!(p->mscale >= 0.0) || !std::isfinite(p->mscale))
        return abi_fail(GDN_ERR_ARG, "%s: mscale must be finite and >= 0", fn);
    const bool scaled = p->scaling != GDN_ROPE_PLAIN;
    if (scaled && (!(p->factor >= 1.0) || !std::isfinite(p->factor)))
        return abi_fail(GDN_ERR_ARG, "%s: factor must be finite and >= 1", fn);
    if (p->scaling == GDN_ROPE_NTK && p->rot_dim == 2)
        return abi_fail(GDN_ERR_ARG, "%s: NTK scaling needs more than one pair", fn);
    double fast = p->beta_fast, slow = p->beta_slow;
    if (fast == 0.0 && slow == 0.0) {
        fast = 32.0;
        slow = 1.0;
    }
    if (p->scaling == GDN_ROPE_YARN &&
        (p->orig_ctx < 1 || !(slow > 0.0) || !(fast >= slow) || !std::isfinite(fast)))
        return abi_fail(GDN_ERR_ARG, "%s: YARN needs orig_ctx >= 1 and beta_fast >= beta_slow > 0", fn);
    const int pairs = p->rot_dim / 2;
    int64_t sum = 0;
    for (int a = 0; a < 4; ++a) {
        if (p->sections[a] < 0) return abi_fail(GDN_ERR_SHAPE, "%s: negative section", fn);
        sum += p->sections[a];
    }
    if (sum != 0 && sum != pairs)
        return abi_fail(GDN_ERR_SHAPE, "%s: sections sum to %lld, not rot_dim / 2 = %d", fn, (long long)sum, pairs);

    gdn_rope_table r{};
    r.rot_dim = p->rot_dim;
    r.layout = p->layout;
    r.n_axes = sum ? 4 : 1;
    for (int a = 0, end = 0; a < 4; ++a) r.axis_end[a] = sum ? (end += p->sections[a]) : pairs;
    const double rot = p->rot_dim;
    const double theta = p->scaling == GDN_ROPE_NTK ? p->theta * std::pow(p->factor, rot / (rot - 2.0)) : p->theta;
    // YARN: the index (not whole) of the pair that turns over n times within orig_ctx tokens
    const auto index_of = [&](double n) { return rot * std::log(p->orig_ctx / (n * 2.0 * kPi)) / (2.0 * std::log(theta)); };
    double lo = 0.0, hi = 0.0;
    if (p->scaling == GDN_ROPE_YARN) {
        lo = std::fmax(std::floor(index_of(fast)), 0.0);
        hi = std::fmin(std::ceil(index_of(slow)), rot - 1.0);
    }
    const double wide = hi > lo ? hi - lo : 0.001;
    for (int i = 0; i < pairs; ++i) {
        double f = std::pow(theta, -2.0 * i / rot);
        if (p->scaling == GDN_ROPE_LINEAR) f /= p->factor;
        if (p->scaling == GDN_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax((i - lo) / wide, 0.0), 1.0);
            f = f / p->factor * ramp + f * (1.0 - ramp);
        }
        r.turns[i] = f / (2.0 * kPi);
    }
    r.mscale = (float)(p->mscale > 0.0                  ? p->mscale
                       : p->scaling == GDN_ROPE_YARN ? 0.1 * std::log(p->factor) + 1.0
                                                        : 1.0);
    *t = r;
    return gdn::abi_ok();
}

GDN_API int gdn_rope(const gdn_rope_table *table, const gdn_rows *x, const gdn_rows *out, int32_t n_segs, int32_t d,
                     const int32_t *positions, int32_t n_tok, int32_t inverse, void *stream)
{
    const char *fn = "gdn_rope";
    if (!table || !x || !out || (!positions && n_tok != 0))
        return abi_fail(GDN_ERR_ARG, "%s: table, x, out and positions must not be NULL", fn);
    if (n_segs < 1 || n_segs > gdn::kMaxRopeSegs)
        return abi_fail(GDN_ERR_SHAPE, "%s: n_segs = %d outside [1, %d]", fn, n_segs, gdn::kMaxRopeSegs);
    if (d < 2 || d > 256) return abi_fail(GDN_ERR_SHAPE, "%s: d = %d outside [2, 256]", fn, d);
    if (int r = gdn::check_table(fn, table, d)) return r;
    if (n_tok < 0) return abi_fail(GDN_ERR_RANGE, "%s: n_tok must be >= 0", fn);
    gdn::RopeArgs a{};
    a.tab = gdn::tab_view(*table);
    a.n_segs = n_segs;
    a.d = d;
    a.inverse = inverse != 0;
    a.n_tok = n_tok;
    a.positions = positions;
    for (int s = 0; s < n_segs; ++s) {
        if (n_tok && (!x[s].ptr || !out[s].ptr)) return abi_fail(GDN_ERR_ARG, "%s: segment %d has a NULL pointer", fn, s);
        for (const gdn_rows *r : {&x[s], &out[s]}) {
            if (r->dtype != GDN_F32 && r->dtype != GDN_BF16)
                return abi_fail(GDN_ERR_DTYPE, "%s: segment %d: dtype must be GDN_F32 or GDN_BF16", fn, s);
            if (!gdn::aligned(r->ptr, gdn::elem_bytes(r->dtype)))
                return abi_fail(GDN_ERR_ARG, "%s: segment %d is not aligned to its elements", fn, s);
        }
        if (x[s].n_heads < 1 || x[s].n_heads > 8192 || out[s].n_heads != x[s].n_heads)
            return abi_fail(GDN_ERR_SHAPE, "%s: segment %d: %d heads in, %d out", fn, s, x[s].n_heads, out[s].n_heads);
        if (int r = gdn::abi_check_apart(fn, "out", &out[s], n_tok, d)) return r;
        const bool same = x[s].ptr == out[s].ptr;
        if (same && (x[s].ld != out[s].ld || x[s].hd != out[s].hd || x[s].dtype != out[s].dtype))
            return abi_fail(GDN_ERR_ARG, "%s: segment %d is in place with other strides or another dtype", fn, s);
        a.seg[s] = gdn::RopeSeg{gdn::rows_view(x[s]), gdn::rows_view(out[s]), x[s].n_heads, same};
        a.heads += x[s].n_heads;
    }
    if (n_tok == 0) return gdn::abi_ok();
    if (hipError_t e = gdn::launch_rope(a, static_cast<hipStream_t>(stream)))
        return abi_fail(GDN_ERR_HIP, "%s launch: %s", fn, hipGetErrorString(e));
    return gdn::abi_ok();
}

GDN_API size_t gdn_kv_bytes(const gdn_kv *kv, size_t *scale_bytes)
{
    if (scale_bytes) *scale_bytes = 0;
    if (gdn::abi_check_kv("gdn_kv_bytes", kv, false)) return 0;
    const size_t rows = (size_t)kv->n_pages * kv->n_kv * kv->page_size;
    if (scale_bytes && kv->format != GDN_KV_BF16) *scale_bytes = rows * sizeof(float);
    return rows * kv->d * (kv->format == GDN_KV_BF16 ? 2 : 1);
}

static int kv_rows(const char *fn, bool write, const gdn_kv *kv, const gdn_kv_batch *batch, const gdn_rows *k,
                   const gdn_rows *v, const gdn_rope_table *rope, const int32_t *positions, void *stream)
{
    if (int r = gdn::abi_check_kv(fn, kv, true)) return r;
    if (int r = gdn::abi_check_batch(fn, batch)) return r;
    if (int r = gdn::abi_check_rows(fn, "k", k, kv->n_kv)) return r;
    if (int r = gdn::abi_check_rows(fn, "v", v, kv->n_kv)) return r;
    if (write && k->dtype != v->dtype) return abi_fail(GDN_ERR_DTYPE, "%s: k and v must have one dtype", fn);
    if (!write) {
        const int64_t rows = (int64_t)batch->n_batch * batch->n_tok;
        if (int r = gdn::abi_check_apart(fn, "k", k, rows, kv->d)) return r;
        if (int r = gdn::abi_check_apart(fn, "v", v, rows, kv->d)) return r;
    }
    gdn::KvRowsArgs a{};
    if (rope) {
        if (!positions) return abi_fail(GDN_ERR_ARG, "%s: a rope table without positions", fn);
        if (int r = gdn::check_table(fn, rope, kv->d)) return r;
        a.rope = 1;
        a.tab = gdn::tab_view(*rope);
        a.positions = positions;
    }
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (int r = gdn::abi_check_places(fn, kv, batch, false, st)) return r;
    a.kv = gdn::kv_view(*kv);
    a.b = gdn::kv_batch_view(*batch);
    a.k = gdn::rows_view(*k);
    a.v = gdn::rows_view(*v);
    if (hipError_t e = write ? gdn::launch_kv_write(a, st) : gdn::launch_kv_read(a, st))
        return abi_fail(GDN_ERR_HIP, "%s launch: %s", fn, hipGetErrorString(e));
    return gdn::abi_ok();
}

GDN_API int gdn_kv_write(const gdn_kv *kv, const gdn_kv_batch *batch, const gdn_rows *k, const gdn_rows *v,
                         const gdn_rope_table *rope, const int32_t *positions, void *stream)
{
    return kv_rows("gdn_kv_write", true, kv, batch, k, v, rope, positions, stream);
}

GDN_API int gdn_kv_read(const gdn_kv *kv, const gdn_kv_batch *batch, const gdn_rows *k, const gdn_rows *v, void *stream)
{
    return kv_rows("gdn_kv_read", false, kv, batch, k, v, nullptr, nullptr, stream);
}

GDN_API int gdn_kv_commit(const gdn_kv *kv, const gdn_kv_batch *batch, const int32_t *path, const int32_t *n_path,
                          int32_t max_path, void *stream)
{
    const char *fn = "gdn_kv_commit";
    if (int r = gdn::abi_check_kv(fn, kv, true)) return r;
    if (int r = gdn::abi_check_batch(fn, batch)) return r;
    if (!path || !n_path) return abi_fail(GDN_ERR_ARG, "%s: path and n_path must not be NULL", fn);
    if (max_path < 1 || max_path > batch->n_tok)
        return abi_fail(GDN_ERR_RANGE, "%s: max_path %d outside [1, n_tok]", fn, max_path);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (int r = gdn::abi_check_places(fn, kv, batch, false, st)) return r;
    if (kv->flags & GDN_F_CHECK_INDICES) {
        const size_t B = batch->n_batch, n = B * max_path;
        std::unique_ptr<int32_t[]> h(new (std::nothrow) int32_t[n + 2 * B]);
        if (!h) return abi_fail(GDN_ERR_HIP, "%s: no host memory for the index check", fn);
        if (int r = gdn::abi_fetch_i32(path, n, st, h.get())) return r;
        if (int r = gdn::abi_fetch_i32(n_path, B, st, h.get() + n)) return r;
        if (batch->n_new) {
            if (int r = gdn::abi_fetch_i32(batch->n_new, B, st, h.get() + n + B)) return r;
        }
        for (size_t b = 0; b < B; ++b) {
            const int32_t m = h[n + b], nodes = batch->n_new ? h[n + B + b] : batch->n_tok;
            if (m < 0 || m > max_path) return abi_fail(GDN_ERR_RANGE, "%s: n_path[%zu] = %d outside [0, max_path]", fn, b, m);
            for (int32_t j = 0; j < m; ++j) {
                const int32_t node = h[b * max_path + j];
                if (node < (j ? h[b * max_path + j - 1] + 1 : 0) || node >= nodes)
                    return abi_fail(GDN_ERR_RANGE, "%s: path[%zu][%d] = %d is no increasing node index", fn, b, j, node);
            }
        }
    }
    gdn::KvCommitArgs a{};
    a.kv = gdn::kv_view(*kv);
    a.b = gdn::kv_batch_view(*batch);
    a.path = path;
    a.n_path = n_path;
    a.max_path = max_path;
    if (hipError_t e = gdn::launch_kv_commit(a, st)) return abi_fail(GDN_ERR_HIP, "%s launch: %s", fn, hipGetErrorString(e));
    return gdn::abi_ok();
}
