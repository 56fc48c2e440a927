// gdn_linear_act.hip - products with bias, activation and residual in their epilogue, operands in 16 or 8 bits, on MFMA
// (gfx950): an FFN's gate, up and down products, an output projection with its residual, a vocabulary's logits.
//
//   out[m][n] = act(p[m][n]) (p[m][N + n]) + residual[m][n],   p[m][n] = sx[m] sw[n] sum_k x[m][k] w[n][k] + bias[n]
//
// K advances 128 bytes of every row at a time whatever the type (64 bf16 or 128 codes: 8 chunks of 16 bytes), so all types
// share the operands' way.  A lane of a 32 x 32 MFMA holds two chunks of each half of a row: one MFMA of depth 64 in e4m3, two
// otherwise (the sum over k does not depend on which k a lane holds, as long as x and w agree).  The product is taken
// transposed (w's rows are MFMA's rows), so that a lane ends with quads of neighbouring columns of one row of out.  Of a gated
// product a tile holds 16 gate rows beside the 16 up rows of the same columns, so that both are in the same lane.
//
// Few rows are bound by w's bytes (16 x 5120 -> 2 x 13824 e4m3: 29.5 us, 4.8 TB/s), many by the tiles' way from L2 beside the
// matrix unit (1024 rows of the same 151 us, 1.92 PFLOP/s; 8191 x 5120 -> 12352 bf16 1.05 ms, 0.99; the library's products of
// these sizes take 131 and 829 us).
#include <type_traits>

#include "gdn_device.h"
#include "gdn_internal.h"
#include "gdn_tiles.h"

namespace gdn {

namespace {

typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i8v __attribute__((ext_vector_type(8)));

constexpr int kRowBytes = kStepBytes, kChunks = kRowBytes / 16;

__device__ __attribute__((aligned(16))) unsigned char kZeros[16];  // what a tile reads past the end of K

typedef float f16v __attribute__((ext_vector_type(16)));
typedef int i16v __attribute__((ext_vector_type(16)));

// e4m3 operands whose result is kept in fp32.  The 8-bit matrix instructions add eight neighbouring k at a time, each product cut
// toward zero at 2^-13 of the largest one's power of two (beside 448 x 448 a product of 15 counts as 8, one of 7 as 0), and
// these sums in fp32.  A result is off by less than 7 2^-13 of the sum of its products' sizes: 1.6e-4 of it at K = 64 for codes
// spread over eight binades, 1.4e-5 of the result's norm for normal values at any K, in the forms of depth 16 and 64 alike.  Half
// a step of bf16, 2^-9 of a result of that size, hides it; fp32's does not.  Widened to bf16, which is exact, the products and
// their sums are fp32's (2e-7), at half the matrix rate (1024 x 13824 -> 5120: 148 us against 96).
constexpr int kE4m3Wide = 4;

template <int T>
struct Acc {
    typedef f16v type;
};
template <>
struct Acc<kI8> {
    typedef i16v type;
};
template <int T>
constexpr int kElem = T == kBf16 ? 2 : 1;

// 16 codes of e4m3 as bf16: the lower and the upper half.
[[maybe_unused]] __device__ __forceinline__ void widen(i4 c, bf16x8_t &lo, bf16x8_t &hi)
{
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[q], 1.0f, false);
        const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[q], 1.0f, true);
        bf16x8_t &to = q < 2 ? lo : hi;
        const int at = 4 * (q & 1);
        to[at] = a[0], to[at + 1] = a[1], to[at + 2] = b[0], to[at + 3] = b[1];
    }
#else
    (void)c, (void)lo, (void)hi;
#endif
}

// One 32 x 32 tile by 64 bytes of K: two chunks of 16 bytes of each operand's row.
template <int T>
__device__ __forceinline__ typename Acc<T>::type mma(i4 a0, i4 a1, i4 b0, i4 b1, typename Acc<T>::type c)
{
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (T == kBf16) {
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a0), __builtin_bit_cast(bf16x8_t, b0), c, 0, 0, 0);
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a1), __builtin_bit_cast(bf16x8_t, b1), c, 0, 0, 0);
    } else if constexpr (T == kI8) {
        c = __builtin_amdgcn_mfma_i32_32x32x32_i8(a0, b0, c, 0, 0, 0);
        return __builtin_amdgcn_mfma_i32_32x32x32_i8(a1, b1, c, 0, 0, 0);
    } else if constexpr (T == kE4m3Wide) {
        const i4 as[2] = {a0, a1}, bs[2] = {b0, b1};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            bf16x8_t a[2], b[2];
            widen(as[q], a[0], a[1]);
            widen(bs[q], b[0], b[1]);
            c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[0], b[0], c, 0, 0, 0);
            c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[1], b[1], c, 0, 0, 0);
        }
        return c;
    } else {
        // e4m3 by e4m3 without block scales: scales of 0 select the form that has none
        const i8v a = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
        const i8v b = {b0[0], b0[1], b0[2], b0[3], b1[0], b1[1], b1[2], b1[3]};
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
    }
#else
    (void)a0, (void)a1, (void)b0, (void)b1;
    return c;
#endif
}

// ------------------------------------------------------------------------------------------------ epilogue
// 1 / (1 + e^-v): v's factor log2(e) rounds once, the power and the quotient about once each.
__device__ __forceinline__ float logistic(float v) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2E * v)); }

__device__ __forceinline__ float activate(int act, float v)
{
    switch (act) {
    case 1: return v * logistic(v);
    case 2: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    case 3: return v * logistic(1.5957691216057308f * (v + 0.044715f * v * v * v));  // (1 + tanh(z)) / 2 = logistic(2 z)
    case 4: return v < 0.0f ? 0.0f : v;
    case 5: return logistic(v);
    default: return v;
    }
}

// One column: what belongs to it is loaded once for many rows.
struct Column {
    float s = 1.0f, s2 = 1.0f, b = 0.0f, b2 = 0.0f;
    int n;
    __device__ Column(const LinearActArgs &a, int n_) : n(n_)
    {
        if (a.x.scale) s = a.w.scale[n];
        if (a.bias) b = a.bias[n];
        if (!a.gated) return;
        if (a.x.scale) s2 = a.w.scale[a.N + n];
        if (a.bias) b2 = a.bias[a.N + n];
    }
    // of row m, from the sums p (and q of the up row)
    __device__ float value(const LinearActArgs &a, int64_t m, float p, float q) const
    {
        const float sx = a.x.scale ? a.x.scale[m] : 1.0f;
        float v = activate(a.act, (a.x.scale ? p * (sx * s) : p) + b);
        if (a.gated) v *= (a.x.scale ? q * (sx * s2) : q) + b2;
        const int64_t at = m * a.residual.ld + n;
        if (a.residual.p) v += a.residual.type == kBf16 ? load_act<true>(a.residual.p, at) : load_act<false>(a.residual.p, at);
        return v;
    }
    __device__ void store(const LinearActArgs &a, int64_t m, float v) const
    {
        const int64_t at = m * a.out.ld + n;
        if (a.out.type == kBf16)
            static_cast<__bf16 *>(a.out.p)[at] = (__bf16)v;
        else
            static_cast<float *>(a.out.p)[at] = v;
    }
};

// Four columns from n on (all below N) at once: what belongs to the columns is loaded once for many rows.
struct Columns {
    f4 s, s2, b, b2;
    int n;
    __device__ Columns(const LinearActArgs &a, int n_) : s{1, 1, 1, 1}, s2{1, 1, 1, 1}, b{0, 0, 0, 0}, b2{0, 0, 0, 0}, n(n_)
    {
        if (a.x.scale) s = *reinterpret_cast<const f4 *>(a.w.scale + n);
        if (a.bias) b = *reinterpret_cast<const f4 *>(a.bias + n);
        if (!a.gated) return;
        if (a.x.scale) s2 = *reinterpret_cast<const f4 *>(a.w.scale + a.N + n);
        if (a.bias) b2 = *reinterpret_cast<const f4 *>(a.bias + a.N + n);
    }
    __device__ f4 residual(const LinearActArgs &a, int64_t m) const
    {
        f4 v = {0, 0, 0, 0};
        if (!a.residual.p) return v;
        const int64_t at = m * a.residual.ld + n;
        if (a.residual.type == kF32) return *reinterpret_cast<const f4 *>(static_cast<const float *>(a.residual.p) + at);
        const bf16x4_t h = *reinterpret_cast<const bf16x4_t *>(static_cast<const uint16_t *>(a.residual.p) + at);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = (float)h[r];
        return v;
    }
    template <bool GATED>
    __device__ f4 value(const LinearActArgs &a, float sx, f4 p, f4 q, f4 residual) const
    {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (a.x.scale) p[r] *= sx * s[r];
            p[r] = activate(a.act, p[r] + b[r]);
            if (GATED) {
                if (a.x.scale) q[r] *= sx * s2[r];
                p[r] *= q[r] + b2[r];
            }
            p[r] += residual[r];
        }
        return p;
    }
    __device__ void store(const LinearActArgs &a, int64_t m, f4 p) const
    {
        const int64_t at = m * a.out.ld + n;
        if (a.out.type == kF32) {
            *reinterpret_cast<f4 *>(static_cast<float *>(a.out.p) + at) = p;
            return;
        }
        bf16x4_t v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = (__bf16)p[r];
        *reinterpret_cast<bf16x4_t *>(static_cast<uint16_t *>(a.out.p) + at) = v;
    }
};

// Row of w that tile row r of the tile from column n0 on holds (the last one again past the end).
template <bool GATED>
__device__ __forceinline__ int64_t weight_row(const LinearActArgs &a, int n0, int r)
{
    if constexpr (GATED) return (int64_t)((r >> 4) & 1) * a.N + min(n0 + (r >> 5) * 16 + (r & 15), a.N - 1);
    return min(n0 + r, a.N - 1);
}

// ------------------------------------------------------------------------------------------------ tiles
__device__ __forceinline__ int chunk_at(int r, int c) { return (r * kChunks + (c ^ (r >> 1 & 7))) * 16; }

// Four sums as they are staged: in fp32, or as they are where parts of K are still to be added (int32 stays exact).
template <int T, class V>
__device__ __forceinline__ f4 staged(V a, V b, V c, V d, bool raw)
{
    if (T == kI8 && raw) return __builtin_bit_cast(f4, i4{(int)a, (int)b, (int)c, (int)d});
    return f4{(float)a, (float)b, (float)c, (float)d};
}
__host__ __device__ constexpr int64_t quads(int64_t n) { return (n + 3) / 4; }

// GM x GN waves, each WM x WN MFMA tiles of 32 x 32 (rows of x by rows of w); NBUF tiles in LDS.
//
// A k tile's first 64 bytes and its last are two sets of registers.  While the products of the first set run, the second one
// is read; then every wave has what it needs of the tile, and after the one barrier of the step the tile's buffer takes the
// transfers of tile kt + NBUF and the first set those of tile kt + 1, while the products of the second set run.
template <int T, bool GATED, int GM, int GN, int WM, int WN, int NBUF, bool PIPE = true, bool SHORT = false>
__global__ __launch_bounds__(64 * GM * GN, WM * WN <= 8 ? 2 : 1) void linear_act_kernel(LinearActArgs a, int wide)
{
    constexpr int BM = 32 * WM * GM, BN = 32 * WN * GN, TH = 64 * GM * GN;
    constexpr int XROWS = SHORT ? 16 : BM;  // rows of x that are loaded: SHORT has no more
    static_assert(!SHORT || BM == 32, "16 of 32 rows");
    constexpr int XT = XROWS * kChunks / TH, WT = BN * kChunks / TH, TPT = XT + WT;
    static_assert(XROWS * kChunks % TH == 0 && BN * kChunks % TH == 0, "whole rounds of transfers");
    static_assert((NBUF - 1) * TPT < 64, "transfers in flight");
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];  // buffers of [x tile | w tile]
    constexpr int XB = XROWS * kRowBytes, BUF = (XROWS + BN) * kRowBytes;
    constexpr int CB = GATED ? BN / 2 : BN;  // columns of out
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, li = lane & 31, lg = lane >> 5;
    const int wm = wave / GN, wn = wave % GN;
    // Workgroups are dealt to the 8 XCDs in turn; an XCD takes a contiguous range of tiles (the first T mod 8 one more), and
    // the tiles go in groups of 8 rows of tiles, down a group's column first: those that run at a time on an XCD share
    // their x and w rows through its L2.
    const int mt = (a.M + BM - 1) / BM, ntiles = gridDim.x;
    const int xcd = blockIdx.x % 8, q8 = ntiles / 8, r8 = ntiles % 8;
    const int t = xcd * q8 + min(xcd, r8) + blockIdx.x / 8;
    const int nt = ntiles / mt, group = t / (8 * nt), rows = min(8, mt - 8 * group), in = t - group * 8 * nt;
    const int m0 = (8 * group + in % rows) * BM, n0 = in / rows * CB;
    // this part's share of K: whole tiles, the last part with K's end
    const int all = (a.K * kElem<T> + kRowBytes - 1) / kRowBytes, part = blockIdx.y;
    const int k0 = (int)((int64_t)all * part / a.splits), nk = (int)((int64_t)all * (part + 1) / a.splits) - k0;
    const int tail = part == a.splits - 1 ? a.K * kElem<T> % kRowBytes : 0;

    // rows past M or N re-read the last row; their results are not stored
    const unsigned char *xsrc[XT], *wsrc[WT];
#pragma unroll
    for (int i = 0; i < XT; ++i) {
        const int p = tid + TH * i, r = p / kChunks, c = (p % kChunks) ^ (r >> 1 & 7);
        xsrc[i] = static_cast<const unsigned char *>(a.x.p) + (int64_t)min(m0 + r, a.M - 1) * a.x.ld * kElem<T> + (int64_t)k0 * kRowBytes + 16 * c;
    }
#pragma unroll
    for (int i = 0; i < WT; ++i) {
        const int p = tid + TH * i, r = p / kChunks, c = (p % kChunks) ^ (r >> 1 & 7);
        wsrc[i] = static_cast<const unsigned char *>(a.w.p) + weight_row<GATED>(a, n0, r) * a.w.ld * kElem<T> + (int64_t)k0 * kRowBytes + 16 * c;
    }
    const int thread0 = __builtin_amdgcn_readfirstlane(tid & ~63);  // of the wave
    // this thread's transfers of the next whole tile into buffer buf, transfer i of TPT
    auto transfer = [&](int i, int buf) {
        unsigned char *base = lds + buf * BUF;
        if (i < XT) {
            lds_dma16(xsrc[i], base + (thread0 + TH * i) * 16);
            xsrc[i] += kRowBytes;
        } else {
            lds_dma16(wsrc[i - XT], base + XB + (thread0 + TH * (i - XT)) * 16);
            wsrc[i - XT] += kRowBytes;
        }
    };
    auto issue = [&](int kt, int buf) {
        if (kt < nk - 1 || !tail) {
#pragma unroll
            for (int i = 0; i < TPT; ++i) transfer(i, buf);
        } else {  // the last tile ends inside its rows: zeros for what is behind
            unsigned char *base = lds + buf * BUF;
#pragma unroll
            for (int i = 0; i < XT; ++i) {
                const int p = tid + TH * i, c = (p % kChunks) ^ (p / kChunks >> 1 & 7);
                lds_dma16(16 * c < tail ? xsrc[i] : kZeros, base + (thread0 + TH * i) * 16);
            }
#pragma unroll
            for (int i = 0; i < WT; ++i) {
                const int p = tid + TH * i, c = (p % kChunks) ^ (p / kChunks >> 1 & 7);
                lds_dma16(16 * c < tail ? wsrc[i] : kZeros, base + XB + (thread0 + TH * i) * 16);
            }
        }
    };

    typename Acc<T>::type acc[WN][WM];
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0;
    i4 xf[2][2][WM], wf[2][2][WN];  // [half of the tile row][its chunks lg and lg + 2]
    auto read = [&](auto half, int buf) {
        constexpr int H = decltype(half)::value;
        const unsigned char *xs = lds + buf * BUF, *ws = xs + XB;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int c = 4 * H + 2 * q + lg;
#pragma unroll
            for (int j = 0; j < WN; ++j) wf[H][q][j] = *reinterpret_cast<const i4 *>(ws + chunk_at(32 * (WN * wn + j) + li, c));
#pragma unroll
            for (int i = 0; i < WM; ++i) xf[H][q][i] = *reinterpret_cast<const i4 *>(xs + chunk_at(SHORT ? li & 15 : 32 * (WM * wm + i) + li, c));
        }
    };
    auto multiply = [&](auto half) {
        constexpr int H = decltype(half)::value;
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
            for (int j = 0; j < WN; ++j) acc[j][i] = mma<T>(wf[H][0][j], wf[H][1][j], xf[H][0][i], xf[H][1][i], acc[j][i]);
    };
    constexpr std::integral_constant<int, 0> H0{};
    constexpr std::integral_constant<int, 1> H1{};
    // this thread's transfers of the tile in question have landed; those of `later` tiles behind it may travel
    auto landed = [&](int kt) {
        if (NBUF > 2 && kt + NBUF - 2 < nk)
            __builtin_amdgcn_s_waitcnt(vmcnt_imm((NBUF - 2) * TPT));
        else
            __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    };
    if constexpr (PIPE) {
#pragma unroll
    for (int p = 0; p < NBUF; ++p)
        if (p < nk) issue(p, p);
    if (NBUF <= nk)
        __builtin_amdgcn_s_waitcnt(vmcnt_imm((NBUF - 1) * TPT));
    else
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    lds_barrier();
    read(H0, 0);
    int buf = 0;
    constexpr int NM = WM * WN * (T == kE4m3 ? 1 : T == kE4m3Wide ? 4 : 2), NR = 2 * (WM + WN);
    // While whole tiles are to come: their transfers and the reads of the next set lie between the products, one of each to
    // a product, as a wave that issued them in a row would keep its SIMD's matrix unit waiting.
    int kt = 0;
#pragma unroll 1
    for (; kt + NBUF < nk - 1; ++kt) {
        read(H1, buf);
        multiply(H0);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            if (i < NM) sched_group(kSchedMfma, 1);
            sched_group(kSchedDsRead, 1);
        }
        if (NM > NR) sched_group(kSchedMfma, NM - NR);
        __builtin_amdgcn_s_waitcnt(vmcnt_imm((NBUF - 2) * TPT));
        lds_barrier();
        const int next = buf == NBUF - 1 ? 0 : buf + 1;
        read(H0, next);
#pragma unroll
        for (int i = 0; i < TPT; ++i) transfer(i, buf);
        multiply(H1);
        constexpr int AHEAD = NR / 2 < NM ? NR / 2 : NM, REST = NM - AHEAD;  // products beside two reads each, and the others
        constexpr int EACH = (TPT + REST - 1) / (REST > 0 ? REST : 1);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            sched_group(kSchedMfma, 1);
            sched_group(kSchedDsRead, 2);
        }
#pragma unroll
        for (int i = 0; i < REST; ++i) {
            sched_group(kSchedVmem, EACH);
            sched_group(kSchedMfma, 1);
        }
        buf = next;
    }
#pragma unroll 1
    for (; kt < nk - 1; ++kt) {
        read(H1, buf);
        multiply(H0);
        landed(kt + 1);
        lds_barrier();
        const int next = buf == NBUF - 1 ? 0 : buf + 1;
        if (kt + NBUF < nk) issue(kt + NBUF, buf);
        read(H0, next);
        multiply(H1);
        buf = next;
    }
    read(H1, buf);
    multiply(H0);
    multiply(H1);
    } else {
        // Sixteen waves, four to a SIMD, hide each other's reads and have no registers for a second set.
        int buf = 0;
#pragma unroll
        for (int p = 0; p < NBUF - 1; ++p)
            if (p < nk) issue(p, p);
#pragma unroll 1
        for (int kt = 0; kt < nk; ++kt) {
            if (NBUF > 2 && kt + NBUF - 2 < nk)
                __builtin_amdgcn_s_waitcnt(vmcnt_imm((NBUF - 2) * TPT));
            else
                __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
            lds_barrier();  // every wave is done with the buffer that is filled next
            if (kt + NBUF - 1 < nk) issue(kt + NBUF - 1, buf == 0 ? NBUF - 1 : buf - 1);
            read(H0, buf);
            read(H1, buf);
            multiply(H0);
            multiply(H1);
            buf = buf == NBUF - 1 ? 0 : buf + 1;
        }
    }

    // Lane (li, lg) of an MFMA tile holds row li of x and the tile's w rows 8 b + 4 lg .. + 3, b = 0 .. 3.  Through LDS, a wave
    // by itself, it goes out by rows: quads of columns, quad c of row r at place c ^ (r & 7).
    constexpr int STEP = GATED ? 2 : 1, QUADS = 8 * WN, OUT = QUADS / STEP;
    constexpr int PASSES = (BM * BN * 4 + NBUF * BUF - 1) / (NBUF * BUF), ROWS = 32 * WM / PASSES;  // rows of a pass
    static_assert(WM % PASSES == 0, "passes of whole tiles");
    constexpr int STRIDE = 64 / OUT, AT = ROWS / STRIDE < 4 ? ROWS / STRIDE : GM * GN > 8 ? 2 : 4;  // rows of a store, and stores at a time
    static_assert(64 % OUT == 0 && ROWS % STRIDE == 0 && ROWS / STRIDE % AT == 0, "whole rows");
    const int c = lane % OUT, r0 = lane / OUT, first = GATED ? (c >> 2) * 8 + (c & 3) : c;
    const int n = n0 + 32 * WN / STEP * wn + 4 * c;
    lds_barrier();  // every wave is done with the last tile
    f4 *mine = reinterpret_cast<f4 *>(lds) + wave * (ROWS * QUADS);
#pragma unroll
    for (int pass = 0; pass < PASSES; ++pass) {
#pragma unroll
        for (int i = 0; i < WM / PASSES; ++i)
#pragma unroll
            for (int j = 0; j < WN; ++j) {
                const typename Acc<T>::type v = acc[j][pass * (WM / PASSES) + i];
                const int r = 32 * i + li;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    mine[r * QUADS + ((8 * j + 2 * b + lg) ^ (r & 7))] = staged<T>(v[4 * b], v[4 * b + 1], v[4 * b + 2], v[4 * b + 3], a.splits > 1);
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const int mp = m0 + 32 * WM * wm + ROWS * pass;
        auto sums = [&](int r, int at) { return mine[r * QUADS + (at ^ (r & 7))]; };
        if (a.splits > 1) {
#pragma unroll 4
            for (int it = 0; it < ROWS / STRIDE; ++it) {
                const int r = it * STRIDE + r0, m = mp + r;
                if (m >= a.M || n >= a.N) continue;
                f4 *to = reinterpret_cast<f4 *>(a.ws) + (((int64_t)part * a.M + m) * STEP) * quads(a.N) + n / 4;
                *to = sums(r, first);
                if constexpr (GATED) to[quads(a.N)] = sums(r, first + 4);
            }
        } else if (wide) {  // N is a multiple of 4: a quad is inside or past the end
            if (n >= a.N) continue;
            const Columns cols(a, n);
#pragma unroll 1
            for (int it = 0; it < ROWS / STRIDE; it += AT) {  // AT rows' loads before the first is used
                f4 p[AT], q[AT], res[AT];
                float sx[AT];
#pragma unroll
                for (int k = 0; k < AT; ++k) {
                    const int r = (it + k) * STRIDE + r0, m = min(mp + r, a.M - 1);
                    p[k] = sums(r, first);
                    q[k] = GATED ? sums(r, first + 4) : p[k];
                    sx[k] = a.x.scale ? a.x.scale[m] : 1.0f;
                    res[k] = cols.residual(a, m);
                }
#pragma unroll
                for (int k = 0; k < AT; ++k) {
                    const int m = mp + (it + k) * STRIDE + r0;
                    const f4 v = cols.value<GATED>(a, sx[k], p[k], q[k], res[k]);
                    if (m < a.M) cols.store(a, m, v);
                }
            }
        } else {
            // any alignment: a column per lane, a row (or a few) at a time
            constexpr int COLS = 4 * OUT < 64 ? 4 * OUT : 64, DOWN = 64 / COLS, UP = GM * GN > 8 ? 1 : 4;
            static_assert(4 * OUT <= 64 && ROWS % (DOWN * UP) == 0, "columns of a wave");
            const int col = lane % COLS, quad = GATED ? (col >> 4) * 8 + (col >> 2 & 3) : col >> 2;
            const int nc = n0 + 32 * WN / STEP * wn + col;
            const Column one(a, min(nc, a.N - 1));
#pragma unroll 1
            for (int it = 0; it < ROWS / DOWN; it += UP) {
                float v[UP];
#pragma unroll
                for (int k = 0; k < UP; ++k) {
                    const int r = (it + k) * DOWN + lane / COLS;
                    const float *p = reinterpret_cast<const float *>(&mine[r * QUADS + (quad ^ (r & 7))]);
                    const float *q = reinterpret_cast<const float *>(&mine[r * QUADS + ((GATED ? quad + 4 : quad) ^ (r & 7))]);
                    v[k] = one.value(a, min(mp + r, a.M - 1), p[col & 3], q[col & 3]);
                }
#pragma unroll
                for (int k = 0; k < UP; ++k) {
                    const int m = mp + (it + k) * DOWN + lane / COLS;
                    if (m < a.M && nc < a.N) one.store(a, m, v[k]);
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// The parts' sums [part][M][gate, up][quads of N] added in order, and the epilogue: a thread per quad of a row.
template <bool I8>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearActArgs a, int wide)
{
    const int64_t nq = quads(a.N), e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= a.M * nq) return;
    const int64_t m = e / nq;
    const int n = (int)(e % nq) * 4, step = a.gated ? 2 : 1;
    f4 s[2] = {};
    for (int g = 0; g < step; ++g) {
        const f4 *from = reinterpret_cast<const f4 *>(a.ws) + (m * step + g) * nq + n / 4;
        i4 whole = {0, 0, 0, 0};
#pragma unroll 4
        for (int p = 0; p < a.splits; ++p) {
            const f4 v = from[p * a.M * step * nq];
            if (I8)
                whole += __builtin_bit_cast(i4, v);
            else
                s[g] += v;
        }
        if (I8)
#pragma unroll
            for (int r = 0; r < 4; ++r) s[g][r] = (float)whole[r];
    }
    if (wide) {
        const Columns cols(a, n);
        const float sx = a.x.scale ? a.x.scale[m] : 1.0f;
        const f4 res = cols.residual(a, m);
        cols.store(a, m, a.gated ? cols.value<true>(a, sx, s[0], s[1], res) : cols.value<false>(a, sx, s[0], s[0], res));
        return;
    }
    for (int r = 0; r < 4 && n + r < a.N; ++r) {
        const Column one(a, n + r);
        one.store(a, m, one.value(a, m, s[0][r], s[1][r]));
    }
}

template <int T, bool GATED, int GM, int GN, int WM, int WN, int NBUF, bool PIPE = true, bool SHORT = false>
hipError_t launch_tile(const LinearActArgs &a, int wide, hipStream_t stream)
{
    constexpr int BM = 32 * WM * GM, BN = 32 * WN * GN, CB = GATED ? BN / 2 : BN;
    const int64_t tiles = (int64_t)((a.M + BM - 1) / BM) * ((a.N + CB - 1) / CB);
    if (tiles * 64 * GM * GN > 0xffffffffll) return hipErrorInvalidValue;  // a launch's x axis holds fewer than 2^32 threads
    hipLaunchKernelGGL((linear_act_kernel<T, GATED, GM, GN, WM, WN, NBUF, PIPE, SHORT>), dim3((unsigned)tiles, a.splits), dim3(64 * GM * GN),
                       NBUF * ((SHORT ? 16 : BM) + BN) * kRowBytes, stream, a, wide);
    if (hipError_t e = hipGetLastError()) return e;
    if (a.splits == 1) return hipSuccess;
    hipLaunchKernelGGL((linear_join_kernel<T == kI8>), dim3((unsigned)((a.M * quads(a.N) + 255) / 256)), dim3(256), 0, stream, a, wide);
    return hipGetLastError();
}

template <int T, bool GATED>
hipError_t launch_of(const LinearActArgs &a, int tile, int wide, hipStream_t stream)
{
    switch (tile) {
    case kShort6: return launch_tile<T, GATED, 1, 2, 1, 1, 6, true, true>(a, wide, stream);
    case kShort4: return launch_tile<T, GATED, 1, 2, 1, 1, 4, true, true>(a, wide, stream);
    case k32x64: return launch_tile<T, GATED, 1, 2, 1, 1, 6>(a, wide, stream);
    case k64x64: return launch_tile<T, GATED, 2, 2, 1, 1, 4>(a, wide, stream);
    case k64x128: return launch_tile<T, GATED, 2, 2, 1, 2, 3>(a, wide, stream);
    case k128x128Deep: return launch_tile<T, GATED, 2, 2, 2, 2, 3>(a, wide, stream);
    case k128x128: return launch_tile<T, GATED, 2, 2, 2, 2, 2>(a, wide, stream);
    default: return launch_tile<T, GATED, 4, 4, 2, 2, 2, false>(a, wide, stream);
    }
}

}  // namespace

size_t linear_act_workspace_bytes(int64_t M, int64_t N, int64_t K, int type, bool gated)
{
    const int splits = M ? choose_tile(M, N, K, type == kBf16 ? 2 : 1, gated).splits : 1;
    return splits > 1 ? 16 * (size_t)splits * M * quads(N) * (gated ? 2 : 1) : 0;
}

hipError_t launch_linear_act(const LinearActArgs &args, hipStream_t stream)
{
    LinearActArgs a = args;
    const Choice c = choose_tile(a.M, a.N, a.K, a.x.type == kBf16 ? 2 : 1, a.gated);
    a.splits = c.splits;
    const auto fits = [](const void *p, int64_t ld, int type) {
        return !p || ((uintptr_t)p % (type == kF32 ? 16 : 8) == 0 && ld % 4 == 0);
    };
    const int wide = a.N % 4 == 0 && fits(a.out.p, a.out.ld, a.out.type) && fits(a.residual.p, a.residual.ld, a.residual.type) &&
                     (uintptr_t)a.bias % 16 == 0 && (uintptr_t)a.w.scale % 16 == 0;
    if (a.x.type == kBf16) return a.gated ? launch_of<kBf16, true>(a, c.tile, wide, stream) : launch_of<kBf16, false>(a, c.tile, wide, stream);
    if (a.x.type == kE4m3 && a.out.type == kF32)
        return a.gated ? launch_of<kE4m3Wide, true>(a, c.tile, wide, stream) : launch_of<kE4m3Wide, false>(a, c.tile, wide, stream);
    if (a.x.type == kE4m3) return a.gated ? launch_of<kE4m3, true>(a, c.tile, wide, stream) : launch_of<kE4m3, false>(a, c.tile, wide, stream);
    return a.gated ? launch_of<kI8, true>(a, c.tile, wide, stream) : launch_of<kI8, false>(a, c.tile, wide, stream);
}

}  // namespace gdn
