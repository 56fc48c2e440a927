// gdn_linear_act.hip - products with bias, activation and residual in their epilogue, operands in 16 or 8 bits, on MFMA
// (gfx950): an FFN's gate, up and down products, an output projection with its residual, a vocabulary's logits.
//
//   out[m][n] = act(p[m][n]) (p[m][N + n]) + residual[m][n],   p[m][n] = sx[m] sw[n] sum_k x[m][k] w[n][k] + bias[n]
//
// Tiling: a workgroup computes BM rows of x by BN rows of w with a grid of waves, each a grid of 16 x 16 MFMA tiles.  A tile
// row is 128 bytes of K whatever the type (64 bf16 or 128 codes: 8 chunks of 16 bytes), so the tiles' way through LDS is the
// same for all: global_load_lds, chunk c of row r at position c ^ (r & 7).  The product is taken transposed (w's rows are
// MFMA's rows), so that a lane ends with four neighbouring columns of one row of out.  Of a gated product a tile holds 16
// gate rows beside the 16 up rows of the same columns, so that both are in the same lane.
#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i8v __attribute__((ext_vector_type(8)));

constexpr int kRowBytes = 128, kChunks = kRowBytes / 16;

__device__ __attribute__((aligned(16))) unsigned char kZeros[16];  // what a tile reads past the end of K

template <int T>
struct Acc {
    typedef f4 type;
};
template <>
struct Acc<kI8> {
    typedef i4 type;
};

// Two chunks of 16 bytes per lane of each operand: the tile row's chunks lg and lg + 4.
template <int T>
__device__ __forceinline__ typename Acc<T>::type mma(i4 a0, i4 a1, i4 b0, i4 b1, typename Acc<T>::type c)
{
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (T == kBf16) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a0), __builtin_bit_cast(bf16x8_t, b0), c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a1), __builtin_bit_cast(bf16x8_t, b1), c, 0, 0, 0);
    } else if constexpr (T == kI8) {
        c = __builtin_amdgcn_mfma_i32_16x16x64_i8(a0, b0, c, 0, 0, 0);
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(a1, b1, c, 0, 0, 0);
    } else {
        const i8v a = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
        const i8v b = {b0[0], b0[1], b0[2], b0[3], b1[0], b1[1], b1[2], b1[3]};
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
    }
#else
    (void)a0, (void)a1, (void)b0, (void)b1;
    return c;
#endif
}

__device__ __forceinline__ float activate(int act, float v)
{
    switch (act) {
    case 1: return v / (1.0f + expf(-v));
    case 2: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    case 3: return v / (1.0f + expf(-1.5957691216057308f * (v + 0.044715f * v * v * v)));
    case 4: return v < 0.0f ? 0.0f : v;
    case 5: return 1.0f / (1.0f + expf(-v));
    default: return v;
    }
}

// Columns n .. n + 3 (those below N) of row m of out, from the sums p (and q of the up rows).
__device__ __forceinline__ void finish(const LinearActArgs &a, int m, int n, f4 p, f4 q)
{
    const float sx = a.x.scale ? a.x.scale[m] : 1.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (n + r >= a.N) return;
        float v = a.x.scale ? p[r] * (sx * a.w.scale[n + r]) : p[r];
        if (a.bias) v += a.bias[n + r];
        v = activate(a.act, v);
        if (a.gated) {
            float u = a.x.scale ? q[r] * (sx * a.w.scale[a.N + n + r]) : q[r];
            if (a.bias) u += a.bias[a.N + n + r];
            v *= u;
        }
        if (a.residual.p) v += a.residual.type == kBf16 ? load_act<true>(a.residual.p, m * a.residual.ld + n + r)
                                                        : load_act<false>(a.residual.p, m * a.residual.ld + n + r);
        const int64_t at = m * a.out.ld + n + r;
        if (a.out.type == kBf16)
            static_cast<uint16_t *>(a.out.p)[at] = f32_to_bf16(v);
        else
            static_cast<float *>(a.out.p)[at] = v;
    }
}

__device__ __forceinline__ int chunk_at(int r, int c) { return (r * kChunks + (c ^ (r & 7))) * 16; }

// GM x GN waves, each WM x WN MFMA tiles (rows of x by rows of w).
template <int T, bool GATED, int GM, int GN, int WM, int WN>
__global__ __launch_bounds__(64 * GM * GN) void linear_act_kernel(LinearActArgs a)
{
    constexpr int BM = 16 * WM * GM, BN = 16 * WN * GN, TH = 64 * GM * GN;
    constexpr int XT = BM * kChunks / TH, WT = BN * kChunks / TH;
    static_assert(BM * kChunks % TH == 0 && BN * kChunks % TH == 0, "whole rounds of transfers");
    static_assert(!GATED || WN % 2 == 0, "gate and up rows in one wave");
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];  // two buffers of [x tile | w tile]
    constexpr int XB = BM * kRowBytes, BUF = (BM + BN) * kRowBytes;
    constexpr int CB = GATED ? BN / 2 : BN;  // columns of out
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, li = lane & 15, lg = lane >> 4;
    const int wm = wave / GN, wn = wave % GN;
    const int mt = (a.M + BM - 1) / BM;
    const int m0 = (blockIdx.x % mt) * BM, n0 = (blockIdx.x / mt) * CB;
    constexpr int kElem = T == kBf16 ? 2 : 1;
    const int64_t kbytes = (int64_t)a.K * kElem;
    const int nk = (int)((kbytes + kRowBytes - 1) / kRowBytes);

    // rows past M or N re-read the last row; their results are not stored
    const unsigned char *xsrc[XT], *wsrc[WT];
    int xc[XT], wc[WT];
#pragma unroll
    for (int i = 0; i < XT; ++i) {
        const int p = tid + TH * i, r = p / kChunks, c = (p % kChunks) ^ (r & 7);
        xc[i] = c;
        xsrc[i] = static_cast<const unsigned char *>(a.x.p) + (int64_t)min(m0 + r, a.M - 1) * a.x.ld * kElem + 16 * c;
    }
#pragma unroll
    for (int i = 0; i < WT; ++i) {
        const int p = tid + TH * i, r = p / kChunks, c = (p % kChunks) ^ (r & 7);
        int64_t row;
        if (GATED)
            row = (int64_t)((r >> 4) & 1) * a.N + min(n0 + (r >> 5) * 16 + (r & 15), a.N - 1);
        else
            row = min(n0 + r, a.N - 1);
        wc[i] = c;
        wsrc[i] = static_cast<const unsigned char *>(a.w.p) + row * a.w.ld * kElem + 16 * c;
    }
    auto issue = [&](int kt, int buf) {
        unsigned char *base = lds + buf * BUF;
        const int64_t k0 = (int64_t)kt * kRowBytes;
#pragma unroll
        for (int i = 0; i < XT; ++i)
            lds_dma16(k0 + 16 * xc[i] < kbytes ? xsrc[i] + k0 : kZeros, base + (tid + TH * i) * 16);
#pragma unroll
        for (int i = 0; i < WT; ++i)
            lds_dma16(k0 + 16 * wc[i] < kbytes ? wsrc[i] + k0 : kZeros, base + XB + (tid + TH * i) * 16);
    };

    typename Acc<T>::type acc[WN][WM];
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
        for (int i = 0; i < WM; ++i) acc[j][i] = typename Acc<T>::type{0, 0, 0, 0};
    issue(0, 0);
#pragma unroll 1
    for (int kt = 0; kt < nk; ++kt) {
        __builtin_amdgcn_s_waitcnt(0x0F70);  // this thread's transfers have landed
        lds_barrier();                       // and every wave's, and every wave is done with the other buffer
        if (kt + 1 < nk) issue(kt + 1, (kt + 1) & 1);
        const unsigned char *xs = lds + (kt & 1) * BUF, *ws = xs + XB;
        i4 xf[2][WM], wf[2][WN];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < WM; ++i) xf[h][i] = *reinterpret_cast<const i4 *>(xs + chunk_at(16 * (WM * wm + i) + li, lg + 4 * h));
#pragma unroll
            for (int j = 0; j < WN; ++j) wf[h][j] = *reinterpret_cast<const i4 *>(ws + chunk_at(16 * (WN * wn + j) + li, lg + 4 * h));
        }
#pragma unroll
        for (int j = 0; j < WN; ++j)
#pragma unroll
            for (int i = 0; i < WM; ++i) acc[j][i] = mma<T>(wf[0][j], wf[1][j], xf[0][i], xf[1][i], acc[j][i]);
    }

    // lane (li, lg) of an MFMA tile holds row li of x and the tile's w rows 4 lg .. 4 lg + 3
    constexpr int STEP = GATED ? 2 : 1;
#pragma unroll
    for (int i = 0; i < WM; ++i) {
        const int m = m0 + 16 * (WM * wm + i) + li;
        if (m >= a.M) continue;
#pragma unroll
        for (int j = 0; j < WN; j += STEP) {
            const int n = n0 + 16 * ((WN * wn + j) / STEP) + 4 * lg;
            f4 p, q;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                p[r] = (float)acc[j][i][r];
                q[r] = (float)acc[j + STEP - 1][i][r];
            }
            finish(a, m, n, p, q);
        }
    }
}

template <int T, bool GATED, int GM, int GN, int WM, int WN>
hipError_t launch_tile(const LinearActArgs &a, hipStream_t stream)
{
    constexpr int BM = 16 * WM * GM, BN = 16 * WN * GN, CB = GATED ? BN / 2 : BN;
    const int64_t tiles = (int64_t)((a.M + BM - 1) / BM) * ((a.N + CB - 1) / CB);
    if (tiles > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL((linear_act_kernel<T, GATED, GM, GN, WM, WN>), dim3((unsigned)tiles), dim3(64 * GM * GN),
                       2 * (BM + BN) * kRowBytes, stream, a);
    return hipGetLastError();
}

template <int T, bool GATED>
hipError_t launch_of(const LinearActArgs &a, hipStream_t stream)
{
    if (a.M <= 32) return launch_tile<T, GATED, 1, 2, 2, 2>(a, stream);
    return launch_tile<T, GATED, 2, 2, 4, 4>(a, stream);
}

}  // namespace

size_t linear_act_workspace_bytes(int64_t, int64_t, int64_t, int, bool) { return 0; }

hipError_t launch_linear_act(const LinearActArgs &a, hipStream_t stream)
{
    if (a.x.type == kBf16) return a.gated ? launch_of<kBf16, true>(a, stream) : launch_of<kBf16, false>(a, stream);
    if (a.x.type == kE4m3) return a.gated ? launch_of<kE4m3, true>(a, stream) : launch_of<kE4m3, false>(a, stream);
    return a.gated ? launch_of<kI8, true>(a, stream) : launch_of<kI8, false>(a, stream);
}

}  // namespace gdn
