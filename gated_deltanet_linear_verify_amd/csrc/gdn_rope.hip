// gdn_rope.hip - rotary positions of rows of heads (gfx950).
//
// Pair i of a head, channels (a, b) = (i, i + rot / 2) or (2 i, 2 i + 1), turns by position * f_i:
// out_a = m (x_a cos - x_b sin), out_b = m (x_a sin + x_b cos) (lucebox-hub internal.h, struct
// TargetWeights: rope sections over the first 64 of 256 channels).  Every value is read and written
// once, so the kernel is HBM-bound, and the factors, ~60 vector instructions per pair of which
// three are fp64, are shared by HPT heads of a token: a thread takes P neighbouring pairs of HPT
// heads, all loads first.
#include "gdn_rows.h"

namespace gdn {

// Units of a (token, head): pairs / P groups of P pairs, then the channels past rot in groups of P
// where out is another buffer.
template <int P, int HPT, bool STREAM>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, int units)
{
    const uint32_t id = blockIdx.x * 256u + threadIdx.x;
    if (id >= (uint32_t)a.nt * (uint32_t)units) return;
    const int u = (int)(id % (uint32_t)units);
    const int64_t t = a.t0 + (int)(id / (uint32_t)units);
    const int gp = a.tab.pairs / P;
    const bool turn = u < gp;
    float c[P], s[P];
    if (turn) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            rope_factors(a.tab, a.positions, a.n_tok, t, u * P + j, c[j], s[j]);
            if (a.inverse) s[j] = -s[j];
        }
    }
    // the unit's channels: two runs of P (halves), one run of 2 P (interleaved) or P copied ones
    const int ca = turn ? (a.tab.interleaved ? 2 * P * u : P * u) : a.tab.rot + P * (u - gp);
    const int cb = a.tab.interleaved ? ca + P : ca + a.tab.pairs;
    float xa[HPT][P], xb[HPT][P];
    int seg[HPT], head[HPT];
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
        int h = blockIdx.y * HPT + k, q = 0;
        while (q < a.n_segs && h >= a.seg[q].n_heads) h -= a.seg[q++].n_heads;
        seg[k] = q;
        head[k] = h;
        if (q >= a.n_segs) continue;
        const RowsView &x = a.seg[q].x;
        const int64_t at = t * x.ld + h * x.hd;
        load_row<P>(x.p, at + ca, x.bf16, xa[k]);
        if (turn) load_row<P>(x.p, at + cb, x.bf16, xb[k]);
    }
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
        if (seg[k] >= a.n_segs) continue;
        const RopeSeg &sg = a.seg[seg[k]];
        const int64_t at = t * sg.out.ld + head[k] * sg.out.hd;
        if (!turn) {
            if (!sg.in_place) store_row<P, STREAM>(sg.out.p, at + ca, sg.out.bf16, xa[k]);
            continue;
        }
        float ya[P], yb[P];
        if (a.tab.interleaved) {
            // element e of the run of 2 P: pair e / 2
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float p = 2 * j < P ? xa[k][(2 * j) % P] : xb[k][(2 * j) % P];
                const float q = 2 * j + 1 < P ? xa[k][(2 * j + 1) % P] : xb[k][(2 * j + 1) % P];
                const float y0 = p * c[j] - q * s[j], y1 = p * s[j] + q * c[j];
                if (2 * j < P) ya[(2 * j) % P] = y0; else yb[(2 * j) % P] = y0;
                if (2 * j + 1 < P) ya[(2 * j + 1) % P] = y1; else yb[(2 * j + 1) % P] = y1;
            }
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                ya[j] = xa[k][j] * c[j] - xb[k][j] * s[j];
                yb[j] = xa[k][j] * s[j] + xb[k][j] * c[j];
            }
        }
        store_row<P, STREAM>(sg.out.p, at + ca, sg.out.bf16, ya);
        store_row<P, STREAM>(sg.out.p, at + cb, sg.out.bf16, yb);
    }
}

template <int P, int HPT, bool STREAM>
static hipError_t launch_rope_as(RopeArgs a, hipStream_t stream)
{
    bool copies = false;
    for (int s = 0; s < a.n_segs; ++s) copies |= !a.seg[s].in_place;
    const int units = a.tab.pairs / P + (copies ? (a.d - a.tab.rot) / P : 0);
    constexpr int kTokensPerLaunch = 1 << 22;  // 2^22 tokens x at most 256 units stay below 2^31 threads
    for (int t0 = 0; t0 < a.n_tok;) {
        a.t0 = t0;
        a.nt = a.n_tok - t0 < kTokensPerLaunch ? a.n_tok - t0 : kTokensPerLaunch;
        const dim3 grid((unsigned)(((int64_t)a.nt * units + 255) / 256), (unsigned)((a.heads + HPT - 1) / HPT));
        hipLaunchKernelGGL((rope_kernel<P, HPT, STREAM>), grid, dim3(256), 0, stream, a, units);
        if (hipError_t e = hipGetLastError()) return e;
        t0 += a.nt;
    }
    return hipSuccess;
}

// Four pairs at a time where every run of four starts aligned (pairs and copied channels in whole
// fours, strides multiples of four elements, and for interleaved runs of eight likewise: they are
// read as two runs of four); single pairs otherwise.  Four heads per thread once that still leaves
// two waves per SIMD (256 CUs x 4 x 2 x 64 threads); a few tokens get a thread per head (1024 tokens of
// 40 heads, interleaved bf16 with YaRN: 7.4 us in a graph; 8191 tokens of 40 heads in fp32: 67 us with
// four heads, 72 with eight).  Results past 64 MiB, twice the L2s, are stored past the caches (67 us
// against 75, 336 MB at 5.0 TB/s).
hipError_t launch_rope(const RopeArgs &a, hipStream_t stream)
{
    bool four = a.tab.pairs % 4 == 0 && (a.d - a.tab.rot) % 4 == 0;
    for (int s = 0; s < a.n_segs; ++s)
        for (const RowsView *r : {&a.seg[s].x, &a.seg[s].out})
            four = four && r->ld % 4 == 0 && r->hd % 4 == 0 && (uintptr_t)r->p % (r->bf16 ? 8 : 16) == 0;
    const int64_t threads = (int64_t)a.n_tok * a.heads * (a.d / (four ? 8 : 2));
    const bool share = threads / 4 >= 256 * 4 * 2 * 64;
    if (four) {
        if (!share) return launch_rope_as<4, 1, false>(a, stream);
        const int64_t values = (int64_t)a.n_tok * a.heads * a.d;
        return values * (a.seg[0].out.bf16 ? 2 : 4) > (64 << 20) ? launch_rope_as<4, 4, true>(a, stream)
                                                                : launch_rope_as<4, 4, false>(a, stream);
    }
    return share ? launch_rope_as<1, 4, false>(a, stream) : launch_rope_as<1, 1, false>(a, stream);
}

}  // namespace gdn
