// gdn_kv.hip - the paged KV cache: rows written (rotated and quantised on the way), read back, and
// the accepted path of a tree moved into place (gfx950).
//
// Cache [n_pages][n_kv][page_size][d] (lucebox-hub internal.h, struct TargetCache keeps attn_k and
// attn_v in 8 bits).  An 8-bit row has one fp32 scale s = max |x| / Q, Q = 448 (e4m3) or 127 (i8), and
// codes rne(x (1 / s)).  A row of d channels is d / 8 lanes of 8 channels, so the maximum is a
// few shuffles inside the row's lanes and every value is read once and written once: HBM-bound.
#include "gdn_rows.h"

namespace gdn {

// max over the d / 8 lanes of a row (LPR = 8, 16 or 32 neighbouring lanes), without LDS: within quads,
// then mirrored halves of 8 and 16 lanes, then the two rows of 16.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v)
{
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false));
}
template <int LPR>
__device__ __forceinline__ uint32_t row_umax(uint32_t v)
{
    v = dpp_umax<0xB1>(v);                       // quad_perm [1,0,3,2]
    v = dpp_umax<0x4E>(v);                       // quad_perm [2,3,0,1]
    v = dpp_umax<0x141>(v);                      // row_half_mirror
    if constexpr (LPR >= 16) v = dpp_umax<0x140>(v);  // row_mirror
    if constexpr (LPR == 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16));
    return v;
}

// One row's 8 channels of this lane into the cache; STREAM: past the caches (a prefill's rows, which
// nothing reads soon: 46 us against 50 for 4 x 8191 tokens of 8 heads into i8).
template <int FMT, int LPR, bool STREAM>
__device__ __forceinline__ void write_codes(unsigned char *dst, float *scales, int64_t row, int li, bool live, const float (&x)[8])
{
#pragma clang fp contract(off)  // a code is the rounded product's, not the exact product's
    constexpr int d = 8 * LPR;
    if constexpr (FMT == kKvBf16) {
        if (live) store_row<8>(dst, row * d + 8 * li, true, x);
        return;
    }
    // |x| as its bits: ordered like the values, with infinity and the NaNs above all of them
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
    top = row_umax<LPR>(top);
    const bool finite = top < 0x7f800000u;
    const float most = __uint_as_float(top), full = FMT == kKvE4m3 ? 448.0f : 127.0f;
    float scale = most / full, inv = 1.0f / scale;
    if (!(inv < __builtin_inff())) scale = inv = 0.0f;  // a row of zeros, or of values whose 1 / s overflows
    if (!finite) {
        scale = __builtin_nanf("");
        inv = 0.0f;
    }
    uint32_t w[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = finite ? x[4 * q + j] * inv : 0.0f;
        if constexpr (FMT == kKvE4m3) {
            uint32_t c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
            w[q] = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c, true);
        } else {
            // |x (1 / s)| <= 127 (1 + 2^-22): adding 1.5 2^23 rounds to nearest, ties to even, and leaves
            // the whole number in the low byte
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = __float_as_uint(y[j] + 12582912.0f);
            w[q] = (u[0] & 0xff) | (u[1] & 0xff) << 8 | (u[2] & 0xff) << 16 | u[3] << 24;
        }
    }
    if (!live) return;
    const uint64_t codes = w[0] | (uint64_t)w[1] << 32;
    uint64_t *to = reinterpret_cast<uint64_t *>(dst + row * d + 8 * li);
    if constexpr (STREAM)
        __builtin_nontemporal_store(codes, to);
    else
        *to = codes;
    if (li == 0) scales[row] = scale;
}

// blockIdx.y: k rows of a group of heads, then v rows.  A thread keeps its 8 channels over the
// group's heads, so a token's factors are formed once per group.
template <int FMT, int LPR, int HB>
__global__ __launch_bounds__(256) void kv_write_kernel(KvRowsArgs a, int hpt, int groups)
{
    const int li = threadIdx.x % LPR;
    const int64_t r = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;  // token row b * n_tok + t
    const int64_t rows = (int64_t)a.b.n_batch * a.b.n_tok;
    const bool is_v = (int)blockIdx.y >= groups;
    const int h0 = (blockIdx.y - (is_v ? groups : 0)) * hpt;
    const int64_t rr = r < rows ? r : rows - 1;  // lanes past the end follow the last row and store nothing
    const int b = (int)(rr / a.b.n_tok), t = (int)(rr % a.b.n_tok);
    const int start = a.b.start[b];
    const bool counts = r < rows && start >= 0 && t < kv_new(a.b, b);
    const int64_t row0 = counts ? kv_row(a.kv, a.b, b, (int64_t)start + t, 0) : -1;
    const bool live = row0 >= 0;
    const RowsView &src = is_v ? a.v : a.k;
    const int ch = 8 * li;
    const bool turn = a.rope && !is_v && ch < a.tab.rot;
    // Channel ch + j's pair, its factors and where its partner is.  Halves: the partner is half of
    // rot away, in one aligned run of 8 when that is a multiple of 8.
    float c[8], s[8];
    int mate[8];
    if (turn) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int x = ch + j, half = a.tab.pairs;
            const bool in = x < a.tab.rot;
            const int i = a.tab.interleaved ? x / 2 : x < half ? x : x - half;
            const bool first = a.tab.interleaved ? (x & 1) == 0 : x < half;
            c[j] = 1.0f;
            s[j] = 0.0f;
            mate[j] = x;
            if (in && live) {
                float cc, ss;
                if (a.tab.interleaved && (j & 1)) {
                    cc = c[j - 1];
                    ss = -s[j - 1];  // the pair's second channel: + sin, below
                } else {
                    rope_factors(a.tab, a.positions, rows, rr, i, cc, ss);
                }
                c[j] = cc;
                s[j] = first ? -ss : ss;  // out = x cos + mate * s
                mate[j] = a.tab.interleaved ? x ^ 1 : first ? x + half : x - half;
            }
        }
    }
    const bool run8 = turn && !a.tab.interleaved && a.tab.pairs % 8 == 0;
    unsigned char *dst = is_v ? a.kv.v : a.kv.k;
    float *scales = is_v ? a.kv.vs : a.kv.ks;
    // HB heads at a time, every load before the first store
    for (int hb = h0; hb < min(h0 + hpt, a.kv.n_kv); hb += HB) {
        float x[HB][8], y[HB][8];
#pragma unroll
        for (int k = 0; k < HB; ++k) {
            const int h = min(hb + k, a.kv.n_kv - 1);
            const int64_t at = rr * src.ld + h * src.hd;
            load_row<8>(src.p, at + ch, src.bf16, x[k]);
            if (turn) {
                if (run8) {
                    load_row<8>(src.p, at + mate[0], src.bf16, y[k]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float one[1];
                        load_row<1>(src.p, at + mate[j], src.bf16, one);
                        y[k][j] = one[0];
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < HB; ++k) {
            const int h = hb + k;
            if (turn) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (ch + j < a.tab.rot) x[k][j] = x[k][j] * c[j] + y[k][j] * s[j];
            }
            write_codes<FMT, LPR, (HB > 1)>(dst, scales, row0 + ((int64_t)h << a.kv.shift), li, live && h < min(h0 + hpt, a.kv.n_kv), x[k]);
        }
    }
}

// blockIdx.y: a group of HB heads, whose k and v rows a thread reads before it stores any.
template <int FMT, int LPR, int HB>
__global__ __launch_bounds__(256) void kv_read_kernel(KvRowsArgs a)
{
    constexpr int d = 8 * LPR;
    const int li = threadIdx.x % LPR;
    const int64_t r = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    if (r >= (int64_t)a.b.n_batch * a.b.n_tok) return;
    const int b = (int)(r / a.b.n_tok), t = (int)(r % a.b.n_tok);
    const int start = a.b.start[b];
    if (start < 0 || t >= kv_new(a.b, b)) return;
    const int64_t row0 = kv_row(a.kv, a.b, b, (int64_t)start + t, 0);
    if (row0 < 0) return;
    const int h0 = blockIdx.y * HB;
    uint4 code[2][HB];  // bf16: 8 values; 8 bits: 8 codes in x and y, the scale in z
#pragma unroll
    for (int k = 0; k < HB; ++k) {
        const int64_t row = row0 + ((int64_t)min(h0 + k, a.kv.n_kv - 1) << a.kv.shift);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const unsigned char *src = w ? a.kv.v : a.kv.k;
            if constexpr (FMT == kKvBf16) {
                code[w][k] = *reinterpret_cast<const uint4 *>(src + (row * d + 8 * li) * 2);
            } else {
                const uint2 q = *reinterpret_cast<const uint2 *>(src + row * d + 8 * li);
                code[w][k] = make_uint4(q.x, q.y, __float_as_uint((w ? a.kv.vs : a.kv.ks)[row]), 0);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < HB; ++k) {
        if (h0 + k >= a.kv.n_kv) break;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const RowsView &out = w ? a.v : a.k;
            const uint32_t q[4] = {code[w][k].x, code[w][k].y, code[w][k].z, code[w][k].w};
            float x[8];
            if constexpr (FMT == kKvBf16) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = bf16_to_f32((uint16_t)(q[j / 2] >> (16 * (j % 2))));
            } else {
                const float scale = __uint_as_float(q[2]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float v;
                    if constexpr (FMT == kKvE4m3) {
                        // byte j % 4 of the word; the builtin takes its index as a literal
                        switch (j % 4) {
                        case 0: v = __builtin_amdgcn_cvt_f32_fp8(q[j / 4], 0); break;
                        case 1: v = __builtin_amdgcn_cvt_f32_fp8(q[j / 4], 1); break;
                        case 2: v = __builtin_amdgcn_cvt_f32_fp8(q[j / 4], 2); break;
                        default: v = __builtin_amdgcn_cvt_f32_fp8(q[j / 4], 3); break;
                        }
                    } else {
                        v = (float)(int8_t)(q[j / 4] >> (8 * (j % 4)));
                    }
                    x[j] = v * scale;
                }
            }
            store_row<8>(out.p, r * out.ld + (h0 + k) * out.hd + 8 * li, out.bf16, x);
        }
    }
}

// One wave per (entry, head, k or v): lanes below the row's 16-byte chunks carry a chunk column
// each, lane 63 the scale, over the path's rows in order.  Row j goes to place j and comes from
// place path[j] >= j, so a row already written is never a later source (the path increases), and
// rows may be read eight at a time before they are written.
__global__ __launch_bounds__(64) void kv_commit_kernel(KvCommitArgs a)
{
    const int b = blockIdx.x, head = blockIdx.y >> 1, lane = threadIdx.x;
    const bool is_v = blockIdx.y & 1;
    const int start = a.b.start[b];
    if (start < 0) return;
    const int n = min(a.n_path[b], a.max_path), nodes = kv_new(a.b, b);
    const int row_bytes = a.kv.d * (a.kv.format == kKvBf16 ? 2 : 1);
    unsigned char *base = is_v ? a.kv.v : a.kv.k;
    float *scales = is_v ? a.kv.vs : a.kv.ks;
    for (int j0 = 0; j0 < n; j0 += 8) {
        int64_t to[8];
        uint4 v[8];
        float s[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            to[q] = -1;
            const int j = j0 + q;
            if (j >= n) continue;
            const int node = a.path[(int64_t)b * a.max_path + j];
            if (node <= j || node >= nodes) continue;  // already in place, or no node of the tree
            const int64_t from = kv_row(a.kv, a.b, b, (int64_t)start + node, head);
            to[q] = kv_row(a.kv, a.b, b, (int64_t)start + j, head);
            if (from < 0) to[q] = -1;
            if (to[q] < 0) continue;
            if (16 * lane < row_bytes) v[q] = *reinterpret_cast<const uint4 *>(base + from * row_bytes + 16 * lane);
            if (lane == 63 && scales) s[q] = scales[from];
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (to[q] < 0) continue;
            if (16 * lane < row_bytes) *reinterpret_cast<uint4 *>(base + to[q] * row_bytes + 16 * lane) = v[q];
            if (lane == 63 && scales) scales[to[q]] = s[q];
        }
    }
}

template <int FMT, int LPR>
static hipError_t launch_rows(const KvRowsArgs &a, bool write, hipStream_t stream)
{
    const int64_t rows = (int64_t)a.b.n_batch * a.b.n_tok;
    const unsigned blocks = (unsigned)((rows + 256 / LPR - 1) / (256 / LPR));
    // Four heads of a token per thread (a write: in batches of two, up to all heads, which share the rotary
    // factors) once that leaves two waves per SIMD, else a thread per head: few tokens are latency.
    // Writing 4 x 8191 tokens of 8 heads into i8: 86 us with a head per thread, 54 with four, 50 with all.
    const int64_t threads = rows * LPR, two_waves = 256 * 4 * 2 * 64;
    const bool four = threads * a.kv.n_kv / 4 >= two_waves && a.kv.n_kv > 1;
    if (write) {
        const int hpt = !four ? 1 : 2 * threads >= two_waves ? (a.kv.n_kv + 3) / 4 * 4 : 4;
        const int groups = (a.kv.n_kv + hpt - 1) / hpt;
        const dim3 grid(blocks, 2 * groups);
        if (four)
            hipLaunchKernelGGL((kv_write_kernel<FMT, LPR, 2>), grid, dim3(256), 0, stream, a, hpt, groups);
        else
            hipLaunchKernelGGL((kv_write_kernel<FMT, LPR, 1>), grid, dim3(256), 0, stream, a, hpt, groups);
    } else if (four) {
        hipLaunchKernelGGL((kv_read_kernel<FMT, LPR, 4>), dim3(blocks, (a.kv.n_kv + 3) / 4), dim3(256), 0, stream, a);
    } else {
        hipLaunchKernelGGL((kv_read_kernel<FMT, LPR, 1>), dim3(blocks, a.kv.n_kv), dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

template <int FMT>
static hipError_t launch_rows_d(const KvRowsArgs &a, bool write, hipStream_t stream)
{
    return a.kv.d == 64    ? launch_rows<FMT, 8>(a, write, stream)
           : a.kv.d == 128 ? launch_rows<FMT, 16>(a, write, stream)
                           : launch_rows<FMT, 32>(a, write, stream);
}

static hipError_t launch_rows_fmt(const KvRowsArgs &a, bool write, hipStream_t stream)
{
    return a.kv.format == kKvBf16   ? launch_rows_d<kKvBf16>(a, write, stream)
           : a.kv.format == kKvE4m3 ? launch_rows_d<kKvE4m3>(a, write, stream)
                                    : launch_rows_d<kKvI8>(a, write, stream);
}

hipError_t launch_kv_write(const KvRowsArgs &a, hipStream_t stream) { return launch_rows_fmt(a, true, stream); }
hipError_t launch_kv_read(const KvRowsArgs &a, hipStream_t stream) { return launch_rows_fmt(a, false, stream); }

hipError_t launch_kv_commit(const KvCommitArgs &a, hipStream_t stream)
{
    hipLaunchKernelGGL(kv_commit_kernel, dim3(a.b.n_batch, 2 * a.kv.n_kv), dim3(64), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdn
