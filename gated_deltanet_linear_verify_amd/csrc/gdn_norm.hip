// gdn_norm.hip - the norm between a layer's mixers (gfx950): s = x + residual, y = s / sqrt(mean(s^2) + eps) * w, in
// 32 or 16 bits, or in 8 with one scale per row (lucebox-hub internal.h, struct TargetLayer: a layer's norms, q_norm
// and k_norm; struct TargetWeights: rms_eps).
//
// A row stays in registers between its one read and its one write.  The row's scale needs max |y|, which is
// max |s w| times the row's factor r = 1 / sqrt(mean(s^2) + eps): y is formed as (s w) r, and the rounding of a product with
// one factor keeps the order, so max |y| is the rounded max |s w| r exactly.  The two reductions, sum s^2 and max |s w|, are
// therefore one round between the lanes, and one exchange through LDS for rows of several waves.  Every value is read and
// written once: HBM-bound (8191 x 5120 bf16 with an fp32 stream into e4m3: 461 MB in 87 us, 5.3 TB/s, a copy's rate here;
// one token 3.5 us).
#include "gdn_rows.h"

namespace gdn {

namespace {

// The sum of a and the maximum of the bits b over the TPR neighbouring lanes that share a row (8 .. 64): within quads, then
// mirrored halves of 8 and 16 lanes by DPP, then rows of 16.
template <int CTRL>
__device__ __forceinline__ void dpp_reduce(float &a, uint32_t &b)
{
    a += dpp_mov<CTRL>(a);
    b = max(b, (uint32_t)__builtin_amdgcn_mov_dpp((int)b, CTRL, 0xF, 0xF, false));
}
template <int TPR>
__device__ __forceinline__ void lanes_reduce(float &a, uint32_t &b)
{
    dpp_reduce<0xB1>(a, b);                          // quad_perm [1,0,3,2]
    dpp_reduce<0x4E>(a, b);                          // quad_perm [2,3,0,1]
    dpp_reduce<0x141>(a, b);                         // row_half_mirror
    if constexpr (TPR >= 16) dpp_reduce<0x140>(a, b);  // row_mirror
#pragma unroll
    for (int o = 16; o < TPR; o *= 2) {
        a += __shfl_xor(a, o);
        b = max(b, (uint32_t)__shfl_xor((int)b, o));
    }
}

// What brings a row to 8 bits, from its largest size.
struct Scale {
    float scale, inv;
    bool finite;  // neither infinite nor NaN
    __device__ Scale(float most, int type) : scale(most / (type == kE4m3 ? 448.0f : 127.0f)), inv(1.0f / scale), finite(most < __builtin_inff())
    {
        if (!(inv < __builtin_inff())) scale = inv = 0.0f;  // a row of zeros, or of values whose 1 / scale overflows
        if (!finite) {
            scale = __builtin_nanf("");
            inv = 0.0f;
        }
    }
};

// The codes of W neighbouring values y.
template <int W, bool STREAM>
__device__ __forceinline__ void store_codes(unsigned char *to, int type, const Scale &q, const float (&y)[W])
{
#pragma clang fp contract(off)  // a code is the rounded y (1 / scale)
    uint32_t code[W];
#pragma unroll
    for (int j = 0; j < W; ++j) {
        const float z = q.finite ? y[j] * q.inv : 0.0f;
        if (type == kE4m3)
            code[j] = __builtin_amdgcn_cvt_pk_fp8_f32(z, 0.0f, 0, false) & 0xff;
        else  // |z| <= 127 (1 + 2^-22): adding 1.5 2^23 rounds to nearest, ties to even
            code[j] = __float_as_uint(z + 12582912.0f) & 0xff;
    }
    if constexpr (W == 8) {
        const uint32_t lo = code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24;
        const uint32_t hi = code[4] | code[5] << 8 | code[6] << 16 | code[7] << 24;
        put_row<STREAM>(reinterpret_cast<uint64_t *>(to), lo | (uint64_t)hi << 32);
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) to[j] = (unsigned char)code[j];
    }
}

// W channels per chunk (8 where every row is aligned for it, else 1), PER chunks per thread.  TPR > 0: a row is TPR
// neighbouring lanes of a wave, 256 / TPR rows to a workgroup; TPR == 0: a row is a workgroup.  STREAM: results of 8 and
// 16 bits past the caches.
template <int W, int PER, int TPR, bool STREAM>
__global__ __launch_bounds__(TPR ? 256 : 1024) void norm_kernel(NormArgs a)
{
#pragma clang fp contract(off)  // y is the rounded product (s w) r
    __shared__ float sums[16];
    __shared__ uint32_t tops[16];
    const int rpw = TPR ? 256 / (TPR ? TPR : 1) : 1;
    const int tpr = TPR ? TPR : (int)blockDim.x;
    const int li = TPR ? threadIdx.x % (TPR ? TPR : 1) : threadIdx.x;
    const int64_t n_rows = (int64_t)a.n_tok * a.n_heads;
    int64_t row = a.row0 + (int64_t)blockIdx.x * rpw + (TPR ? threadIdx.x / (TPR ? TPR : 1) : 0);
    const bool live = row < n_rows;
    if (!live) row = n_rows - 1;  // lanes past the end follow the last row and store nothing
    const int64_t t = row / a.n_heads, h = row % a.n_heads;
    const int64_t xat = t * a.x.ld + h * a.x.hd;

    float v[PER][W], w[PER][W];
    const int d = a.d;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = (li + i * tpr) * W;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            v[i][j] = 0.0f;
            w[i][j] = 1.0f;
        }
        if (c < d) {
            load_row<W>(a.x.p, xat + c, a.x.bf16, v[i]);
            if (a.weight) load_row<W>(a.weight, c, false, w[i]);
        }
    }
    if (a.residual.p) {
        const int64_t at = t * a.residual.ld + h * a.residual.hd;
        float u[PER][W];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = (li + i * tpr) * W;
            if (c < d) {
                load_row<W>(a.residual.p, at + c, a.residual.bf16, u[i]);
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) u[i][j] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) v[i][j] += u[i][j];
    }
    if (a.total.p && live) {
        const int64_t at = t * a.total.ld + h * a.total.hd;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = (li + i * tpr) * W;
            if (c < d) store_row<W, STREAM>(a.total.p, at + c, a.total.bf16, v[i]);
        }
    }

    // one round between the lanes of a row: the sum of q, and the largest of the bits
    auto round = [&](float &q, uint32_t &top) {
        if constexpr (TPR > 0) {
            lanes_reduce<TPR>(q, top);
        } else {
            lanes_reduce<64>(q, top);
            const int wave = threadIdx.x >> 6, n_waves = blockDim.x >> 6, o = threadIdx.x & 15;
            __syncthreads();  // the last round's values have been read
            if ((threadIdx.x & 63) == 0) {
                sums[wave] = q;
                tops[wave] = top;
            }
            __syncthreads();
            q = o < n_waves ? sums[o] : 0.0f;
            top = o < n_waves ? tops[o] : 0u;
            lanes_reduce<16>(q, top);
        }
    };
    // sum s^2, and max |s w| by its bits (ordered like the values, infinity and the NaNs above all)
    auto measure = [&](float &q, uint32_t &top, bool weighed) {
        q = 0.0f;
        top = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) {
                q = __builtin_fmaf(v[i][j], v[i][j], q);
                top = max(top, __float_as_uint(weighed ? v[i][j] * w[i][j] : v[i][j]) & 0x7fffffffu);
            }
        round(q, top);
    };
    float r = 1.0f, ssq = 0.0f;
    uint32_t top = 0;
    const bool codes = a.out_type == kE4m3 || a.out_type == kI8;
    if (a.rms || codes) measure(ssq, top, true);
    if (a.rms) {
        const float n = (float)d;
        r = 1.0f / sqrtf(ssq / n + a.eps);
        if (!(ssq < __builtin_inff()) || top >= 0x7f800000u) {  // the same for all lanes of a row
            uint32_t big;
            measure(ssq, big, false);
            // finite values, some of them above 1: scaled by the power of two that puts the largest in [1/2, 1), where neither
            // their squares nor their products with any weight pass fp32's range
            if (big < 0x7f800000u && big >= 0x3f800000u) {
                const int e = (int)(big >> 23) - 126;
#pragma unroll
                for (int i = 0; i < PER; ++i)
#pragma unroll
                    for (int j = 0; j < W; ++j) v[i][j] = ldexpf(v[i][j], -e);
                measure(ssq, top, true);
                r = 1.0f / sqrtf(ssq / n + ldexpf(a.eps, -2 * e));
            }
        }
    }
    const int64_t oat = t * a.out.ld + h * a.out.hd;
    if (a.out_type == kF32 || a.out_type == kBf16) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = (li + i * tpr) * W;
#pragma unroll
            for (int j = 0; j < W; ++j) v[i][j] = v[i][j] * w[i][j] * r;
            if (c < d && live) store_row<W, STREAM>(a.out.p, oat + c, a.out.bf16, v[i]);
        }
        return;
    }
    const Scale q(__uint_as_float(top) * r, a.out_type);
    unsigned char *to = static_cast<unsigned char *>(a.out.p) + oat;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int c = (li + i * tpr) * W;
        if (c >= d || !live) continue;
#pragma unroll
        for (int j = 0; j < W; ++j) v[i][j] = v[i][j] * w[i][j] * r;
        store_codes<W, STREAM>(to + c, a.out_type, q, v[i]);
    }
    if (li == 0 && live) a.scale[row] = q.scale;
}

// Rows past kNormMaxD, without the division: a workgroup reads its row for the largest |s w| where codes ask for it, and
// again, out of the caches, for the results.  A thread reads what it writes, so both may be in place.  (8-bit operands as wide as
// an FFN's inner rows: 1024 x 25600 bf16 into e4m3 34 us, 79 MB read and written, and 52 MB of it read again; 16 x 17408 9 us.)
constexpr int kLongThreads = 1024;
template <int W>
__global__ __launch_bounds__(kLongThreads) void long_rows_kernel(NormArgs a)
{
    __shared__ uint32_t tops[kLongThreads / 64];
    const int tid = threadIdx.x;
    const int64_t row = a.row0 + blockIdx.x, t = row / a.n_heads, h = row % a.n_heads;
    const int64_t xat = t * a.x.ld + h * a.x.hd, rat = t * a.residual.ld + h * a.residual.hd;
    auto read = [&](int c, float (&s)[W], float (&y)[W]) {
        float u[W], w[W];
        load_row<W>(a.x.p, xat + c, a.x.bf16, s);
        if (a.residual.p) load_row<W>(a.residual.p, rat + c, a.residual.bf16, u);
        if (a.weight) load_row<W>(a.weight, c, false, w);
#pragma unroll
        for (int j = 0; j < W; ++j) {
            if (a.residual.p) s[j] += u[j];
            y[j] = a.weight ? s[j] * w[j] : s[j];
        }
    };
    const bool codes = a.out_type == kE4m3 || a.out_type == kI8;
    uint32_t top = 0;
    if (codes) {
        for (int c = tid * W; c < a.d; c += kLongThreads * W) {
            float s[W], y[W];
            read(c, s, y);
#pragma unroll
            for (int j = 0; j < W; ++j) top = max(top, __float_as_uint(y[j]) & 0x7fffffffu);
        }
        float none = 0.0f;
        lanes_reduce<64>(none, top);
        if ((tid & 63) == 0) tops[tid >> 6] = top;
        __syncthreads();
        top = tops[tid & 15];
        lanes_reduce<16>(none, top);
    }
    const Scale q(__uint_as_float(top), a.out_type);
    const int64_t tat = t * a.total.ld + h * a.total.hd, oat = t * a.out.ld + h * a.out.hd;
    for (int c = tid * W; c < a.d; c += kLongThreads * W) {
        float s[W], y[W];
        read(c, s, y);
        if (a.total.p) store_row<W>(a.total.p, tat + c, a.total.bf16, s);
        if (codes)
            store_codes<W, false>(static_cast<unsigned char *>(a.out.p) + oat + c, a.out_type, q, y);
        else
            store_row<W>(a.out.p, oat + c, a.out.bf16, y);
    }
    if (codes && tid == 0) a.scale[row] = q.scale;
}

// launch(n, a) for runs of n rows from a.row0 on: a launch's x axis holds fewer than 2^32 threads.
template <class F>
hipError_t in_runs(NormArgs a, int64_t run, F launch)
{
    const int64_t rows = (int64_t)a.n_tok * a.n_heads;
    for (a.row0 = 0; a.row0 < rows; a.row0 += run) {
        launch(rows - a.row0 < run ? rows - a.row0 : run, a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    return hipSuccess;
}

template <int W, int PER, int TPR, bool STREAM = false>
hipError_t launch_as(const NormArgs &args, int threads, hipStream_t stream)
{
    const int64_t rpw = TPR ? 256 / (TPR ? TPR : 1) : 1;
    return in_runs(args, (int64_t)0xffffffff / threads * rpw, [&](int64_t n, const NormArgs &a) {
        hipLaunchKernelGGL((norm_kernel<W, PER, TPR, STREAM>), dim3((unsigned)((n + rpw - 1) / rpw)), dim3(threads), 0, stream, a);
    });
}

// A row's threads: neighbouring lanes of a wave up to 64 chunks (single channels: up to 512, eight to a lane, as a load
// of one channel is an instruction: 8191 x 24 heads of 129 channels 162 us with a thread each, 86 so), else a workgroup with
// as few chunks to a thread as its 1024 threads allow (5120 channels of one token: one chunk each; single channels: 8 or 16,
// 8191 x 5121 215 us against 286 with 16 in whole workgroups).
template <int W>
hipError_t launch_wide(const NormArgs &a, hipStream_t stream)
{
    if (a.d > kNormMaxD)
        return in_runs(a, 0xffffffff / kLongThreads, [&](int64_t n, const NormArgs &b) {
            hipLaunchKernelGGL((long_rows_kernel<W>), dim3((unsigned)n), dim3(kLongThreads), 0, stream, b);
        });
    const int chunks = (a.d + W - 1) / W;
    const auto threads = [&](int per) { return ((chunks + per - 1) / per + 63) / 64 * 64; };
    if (chunks <= 8) return launch_as<W, 1, 8>(a, 256, stream);
    if (chunks <= 16) return launch_as<W, 1, 16>(a, 256, stream);
    if (chunks <= 32) return launch_as<W, 1, 32>(a, 256, stream);
    if (chunks <= 64) return launch_as<W, 1, 64>(a, 256, stream);
    if constexpr (W == 8) {
        // Many rows: two chunks to a thread, so that half the waves wait at the exchange (8191 x 5120, bf16 onto bf16 into
        // e4m3, 294 MB: 63 us against 72), and results of 8 and 16 bits past the caches (58); fp32 results that way are
        // slower (sum in fp32, 461 MB: 93 against 87).
        const bool many = (int64_t)a.n_tok * a.n_heads * a.d > (16 << 20);
        if (many && chunks > 128 && chunks <= 1024) {
            const bool f32 = (a.total.p && !a.total.bf16) || a.out_type == kF32;
            return f32 ? launch_as<W, 2, 0>(a, threads(2), stream) : launch_as<W, 2, 0, true>(a, threads(2), stream);
        }
        if (chunks <= 1024) return launch_as<W, 1, 0>(a, threads(1), stream);
        return launch_as<W, 2, 0>(a, threads(2), stream);  // d <= kNormMaxD = 2048 chunks of 8
    } else {
        if (chunks <= 128) return launch_as<W, 2, 64>(a, 256, stream);
        if (chunks <= 256) return launch_as<W, 4, 64>(a, 256, stream);
        if (chunks <= 512) return launch_as<W, 8, 64>(a, 256, stream);
        if (chunks <= 8192) return launch_as<W, 8, 0>(a, threads(8), stream);
        return launch_as<W, 16, 0>(a, threads(16), stream);
    }
}

}  // namespace

hipError_t launch_norm(const NormArgs &a, hipStream_t stream)
{
    bool wide = a.d % 8 == 0 && (uintptr_t)a.weight % 16 == 0;
    for (const RowsView *r : {&a.x, &a.residual, &a.total, &a.out}) {
        const bool codes = r == &a.out && a.out_type >= kE4m3;
        wide = wide && r->ld % 8 == 0 && r->hd % 8 == 0 && (uintptr_t)r->p % (codes ? 8 : 16) == 0;
    }
    return wide ? launch_wide<8>(a, stream) : launch_wide<1>(a, stream);
}

}  // namespace gdn
