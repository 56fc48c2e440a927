// gdn_internal.h - launch interface between the C ABI (gdn_abi.cpp) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

struct gdn_dims;  // include/gdn.h
struct gdn_kv;
struct gdn_kv_batch;
struct gdn_rope_table;
struct gdn_rows;

namespace gdn {

constexpr int kTokenTile = 16;  // tokens per LDS tile in the verify kernels

struct VerifyArgs {
    int32_t n_kh, n_vh, d, n_pool, T, t_cap, C;
    int32_t t0, nt;  // chain verify: first token and token count of one launch (set by the launcher)
    float eps;
    float *state;
    float *conv_state;
    const void *qkv, *z, *alpha, *beta;
    const float *A_log, *dt_bias, *conv_w, *norm_w;
    float *cap_ssm;   // NULL: no capture
    float *cap_conv;
    void *out;
    const int32_t *slot_ids;
    const int32_t *resume;  // chain verify with capture: per batch entry, the capture position whose
                            // state and conv window the first token starts from (< 0: the slot's
                            // state); NULL: every entry starts from the slot's state
    const int32_t *parent;  // tree only
    int32_t n_batch;
    int32_t defer;  // chain verify with capture: leave state and conv_state untouched (the state
                    // after the last token stays at its capture position)
    int32_t hpw;    // chain verify: value heads per workgroup, set by the launcher (H_v/H_k, or 1)
    float *oscr;    // chain verify, row split: the launch's readout [n_batch][16][H_v][d] (set by the launcher)
};

// The row-split verify's readout scratch for stream st on the current device: the buffer kept for
// the stream (while st is capturing, only one reserved for capture), else (allocate, and st not
// capturing) a new one of kSplitScratchBytes, else NULL.
constexpr size_t kSplitScratchBytes = size_t(4) << 20;
void *split_scratch(hipStream_t st, bool allocate);
// Keep a buffer for st that launches under a capture on st may use (allocated now if st has none
// and is not capturing); false if there is none.
bool split_scratch_reserve(hipStream_t st);
// Remove the buffer kept for st and hand it to the caller (who frees it), or NULL.
void *split_scratch_take(hipStream_t st);

struct LaunchCfg {
    bool act_bf16, out_bf16, qk_norm;
};

// Chain verify: grid B * H_k workgroups of (H_v/H_k) * waves_per_head(d) waves.
hipError_t launch_verify_chain(const VerifyArgs &a, const LaunchCfg &c, hipStream_t stream);
// Tree verify: grid B * H_v workgroups of 2 * waves_per_head(d) waves; at most 64 nodes.
hipError_t launch_verify_tree(const VerifyArgs &a, const LaunchCfg &c, hipStream_t stream);

int verify_waves_per_head(int d);
size_t verify_chain_lds_bytes(int d, int ratio, bool act_bf16);
size_t verify_tree_lds_bytes(int d, int T, bool act_bf16);  // (size_t)-1 above the node limit

struct RollbackArgs {
    float *state, *conv_state;
    const float *cap_ssm, *cap_conv;
    int32_t n_pool, t_cap, mode;
    size_t ssm_elems;   // H_v * d_v * d_k floats per slot and position
    size_t conv_elems;  // 3 * C floats
    size_t C;
    const int32_t *slots;  // device array, or NULL: use slot0 / idx0
    const int32_t *idx;
    int32_t slot0, idx0, n;
};
hipError_t launch_rollback(const RollbackArgs &a, hipStream_t stream);

// Rollback of several layers' captures in one launch: the shapes, slots and indices are shared
// (geo; its buffer pointers are unused), each layer brings its own four buffers.
constexpr int kMaxLayersPerLaunch = 64;
struct LayerBuffers {
    float *state, *conv_state;
    const float *cap_ssm, *cap_conv;
};
struct RollbackLayersArgs {
    RollbackArgs geo;
    int32_t n_layers;  // 1 .. kMaxLayersPerLaunch
    LayerBuffers layer[kMaxLayersPerLaunch];
};
hipError_t launch_rollback_layers(const RollbackLayersArgs &a, hipStream_t stream);

hipError_t launch_fill_zero(float *p, size_t n, hipStream_t stream);

// Snapshot / restore: for each listed slot, copy its state and conv state from one pool-shaped
// pair of buffers to another.
struct SlotCopyArgs {
    float *dst_state, *dst_conv;
    const float *src_state, *src_conv;
    const int32_t *slots;  // device array of n slots; entries outside [0, n_pool) are skipped
    int32_t n, n_pool;
    size_t ssm_elems;   // H_v * d_v * d_k floats per slot
    size_t conv_elems;  // 3 * C floats per slot
};
hipError_t launch_slot_copy(const SlotCopyArgs &a, hipStream_t stream);

// Projections y = x W^T (bf16 in, fp32 accumulate): product columns [n0, n1) of segment s go to
// seg[s].ptr[m * ld + n - n0], as bf16 or fp32, optionally through a sigmoid.
constexpr int kMaxLinearSegs = 4;
struct LinearSeg {
    int32_t n0, ld, bf16, sigmoid;
    void *ptr;
};
struct LinearArgs {
    const uint16_t *x;  // [M][K] bf16
    const uint16_t *w;  // [N][K] bf16
    int32_t M, N, K;    // K a multiple of 64
    int32_t n_segs;     // 1 .. kMaxLinearSegs, ascending n0, seg[0].n0 == 0
    LinearSeg seg[kMaxLinearSegs];
};
hipError_t launch_linear(const LinearArgs &a, hipStream_t stream);

// ---- full-attention layers: rotary positions, paged KV cache, attention ----

// gdn_rope_table as the kernels take it (by value).
constexpr float kLog2E = 1.44269504088896341f;
constexpr int kMaxRopePairs = 128;
struct RopeTab {
    int32_t rot, pairs, interleaved, n_axes;
    int32_t axis_end[4];
    float mscale;
    double turns[kMaxRopePairs];
};
struct RowsView {
    void *p;
    int64_t ld, hd;
    int32_t bf16;
};
constexpr int kMaxRopeSegs = 4;
struct RopeSeg {
    RowsView x, out;
    int32_t n_heads, in_place;
};
struct RopeArgs {
    RopeTab tab;
    RopeSeg seg[kMaxRopeSegs];
    int32_t n_segs, d, heads, inverse;  // heads: of all segments together
    int32_t n_tok, t0, nt;              // tokens of the call (the positions' axis stride) and of one launch
    const int32_t *positions;
};
hipError_t launch_rope(const RopeArgs &a, hipStream_t stream);

enum { kKvBf16 = 0, kKvE4m3 = 1, kKvI8 = 2 };  // gdn_kv_format
struct KvView {
    unsigned char *k, *v;
    float *ks, *vs;
    int32_t n_kv, d, shift, n_pages, format;  // page_size = 1 << shift
};
struct KvBatchView {
    const int32_t *table, *start, *n_new;
    int32_t max_pages, n_batch, n_tok;
};
struct KvRowsArgs {
    KvView kv;
    KvBatchView b;
    RowsView k, v;
    const int32_t *positions;  // [n_axes][n_batch * n_tok]; used when rope is set
    int32_t rope;
    RopeTab tab;
};
hipError_t launch_kv_write(const KvRowsArgs &a, hipStream_t stream);
hipError_t launch_kv_read(const KvRowsArgs &a, hipStream_t stream);
struct KvCommitArgs {
    KvView kv;
    KvBatchView b;
    const int32_t *path, *n_path;
    int32_t max_path;
};
hipError_t launch_kv_commit(const KvCommitArgs &a, hipStream_t stream);
// Attention of drafted tokens (gdn_attn.hip).  A launch's work is a list of items, each a tile of query
// rows of one KV head with the keys they see; AttnPhase describes one launch's items.
// Token rows of a call: 2^26 rows of 32 lanes stay below the 2^32 threads of a launch's x axis.  For attention,
// token rows times the query heads of a group: fewer than 2^26, as the join takes 64 lanes for each.
constexpr int64_t kMaxTokenRows = (int64_t)1 << 26;

struct AttnPhase {
    int32_t cfg;        // tile shape, by rows (attn_config)
    int32_t bm, bn;     // rows and keys of a tile
    int32_t row_tiles;  // row tiles per entry (the prefix: of the whole batch)
    int32_t items;      // items per KV head
    int32_t wgs;        // workgroups launched
    size_t po, pml, first, per;  // workspace offsets: partial outputs, their (max, sum), first units, units per workgroup
};
struct AttnPlan {
    AttnPhase suffix, prefix;
    size_t live, rank, anc, bytes;  // workspace offsets: token rows that count, their places, ancestor words
    int32_t words;                  // ancestor words per node
};
struct AttnArgs {
    KvView kv;
    KvBatchView b;
    RowsView q, out;
    int32_t grp;                    // query heads per KV head
    float scale;                    // of the scores, times log2(e)
    const int32_t *parent;          // tree, else NULL
    const int32_t *prefix_pages, *prefix_len;
    int32_t max_prefix_pages;
    unsigned char *ws;
    AttnPlan plan;
};
// Sizes only; false where a launch's rows, tiles or positions would pass what the kernels count in.
bool attn_plan(int d, int format, int page_size, int n_kv, int grp, int n_batch, int n_tok, int max_pages, bool prefix,
               int max_prefix_pages, AttnPlan &p);
hipError_t launch_attn(const AttnArgs &a, hipStream_t stream);

// Checks shared by the cache's entry points (gdn_kv_abi.cpp); each sets the last error.
int abi_check_kv(const char *fn, const gdn_kv *kv, bool pointers);
int abi_check_rows(const char *fn, const char *what, const gdn_rows *r, int n_heads);  // aligned rows
int abi_check_apart(const char *fn, const char *what, const gdn_rows *r, int64_t n_rows, int d);  // rows to write do not overlap
int abi_check_batch(const char *fn, const gdn_kv_batch *b);
// Under GDN_F_CHECK_INDICES: the batch's arrays, copied to the host, name places that exist, for
// positions [0, start + n) (from_zero) or [start, start + n).
int abi_check_places(const char *fn, const gdn_kv *kv, const gdn_kv_batch *b, bool from_zero, hipStream_t st);
KvView kv_view(const gdn_kv &kv);
KvBatchView kv_batch_view(const gdn_kv_batch &b);
RowsView rows_view(const gdn_rows &r);

// Host copy of n device int32 for GDN_F_CHECK_INDICES (synchronises with st; a capturing stream is
// refused untouched).  Sets the last error; GDN_OK if the copy was made.
int abi_fetch_i32(const int32_t *dev, size_t n, hipStream_t st, int32_t *out);

// The C ABI's thread-local last error (gdn_last_error): set it and return code, or clear it and
// return GDN_OK.
int abi_fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int abi_ok();
// Validation of gdn_dims as every entry point does it (sets the last error; GDN_OK if valid).
int abi_check_dims(const gdn_dims *d);

struct PrefillArgs {
    int32_t n_kh, n_vh, d, T, C, slot;
    float eps;
    float *state, *conv_state;
    const void *qkv, *z, *alpha, *beta;
    const float *A_log, *dt_bias, *conv_w, *norm_w;
    void *out;
    float *ws;  // workspace of prefill_workspace_bytes(): per-chunk operands and the fp32 readout
};
// Chunked prefill: a chunk-parallel prep kernel (conv, gates, T = (I + A)^-1 and P per chunk and
// value head), a sequential scan over H_v * (d / 16) workgroups, then the norm epilogue.
hipError_t launch_prefill(const PrefillArgs &a, const LaunchCfg &c, hipStream_t stream);
size_t prefill_workspace_bytes(int d, int n_kh, int n_vh, int T);
size_t prefill_lds_bytes(int d, bool act_bf16);  // the larger of the two kernels' LDS
// Every check of a prefill call except the workspace's (sets the last error); on GDN_OK, a holds
// the launch arguments with ws unset and c the kernel configuration.
int prefill_prepare(const char *fn, const gdn_dims *dims, float *state, float *conv_state, const void *qkv,
                    const void *z, const void *alpha, const void *beta, const float *A_log, const float *dt_bias,
                    const float *conv_w, const float *norm_w, void *out, int32_t n_tok, int32_t slot, PrefillArgs &a,
                    LaunchCfg &c);

}  // namespace gdn
