// gdn_rows.h - device helpers of the full-attention layers' kernels: rows of heads in either type,
// rotary factors, and places in the paged cache.
#pragma once

#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {

typedef float f8 __attribute__((ext_vector_type(8)));

// N consecutive elements at element offset i, in fp32 (N = 1, 4 or 8; the address is aligned to
// min(16, N elements) bytes, which the launchers check).
template <int N>
__device__ __forceinline__ void load_row(const void *p, int64_t i, bool bf16, float (&x)[N])
{
    if (bf16) {
        const __bf16 *s = static_cast<const __bf16 *>(p) + i;
        if constexpr (N == 8) {
            const bf16x8_t v = *reinterpret_cast<const bf16x8_t *>(s);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (float)v[j];
        } else if constexpr (N == 4) {
            const bf16x4_t v = *reinterpret_cast<const bf16x4_t *>(s);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = (float)v[j];
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = (float)s[j];
        }
    } else {
        const float *s = static_cast<const float *>(p) + i;
        if constexpr (N % 4 == 0) {
#pragma unroll
            for (int q = 0; q < N / 4; ++q) {
                const f4 v = *reinterpret_cast<const f4 *>(s + 4 * q);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[4 * q + j] = v[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = s[j];
        }
    }
}

template <bool STREAM, class T, class V>
__device__ __forceinline__ void put_row(T *p, V v)
{
    if constexpr (STREAM)
        __builtin_nontemporal_store(v, reinterpret_cast<V *>(p));
    else
        *reinterpret_cast<V *>(p) = v;
}

// STREAM: vector stores past the caches, for rows that do not fit them.
template <int N, bool STREAM = false>
__device__ __forceinline__ void store_row(void *p, int64_t i, bool bf16, const float (&x)[N])
{
    if (bf16) {
        __bf16 *s = static_cast<__bf16 *>(p) + i;
        if constexpr (N == 8) {
            bf16x8_t v;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (__bf16)x[j];
            put_row<STREAM>(s, v);
        } else if constexpr (N == 4) {
            bf16x4_t v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = (__bf16)x[j];
            put_row<STREAM>(s, v);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) s[j] = (__bf16)x[j];
        }
    } else {
        float *s = static_cast<float *>(p) + i;
        if constexpr (N % 4 == 0) {
#pragma unroll
            for (int q = 0; q < N / 4; ++q) {
                f4 v;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = x[4 * q + j];
                put_row<STREAM>(s + 4 * q, v);
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) s[j] = x[j];
        }
    }
}

// m cos and m sin of pair i for a token at column t of the positions ([n_axes] rows of `ld`).  The
// angle is formed in turns in fp64 and its whole turns are dropped there: position times frequency
// in fp32 would be off by up to 0.06 radians at a million tokens.  What is left, in [-1/2, 1/2]
// turns, is rounded to fp32 once (2^-25 turns) and goes through sincospi.
__device__ __forceinline__ void rope_factors(const RopeTab &tab, const int32_t *positions, int64_t ld, int64_t t, int i,
                                             float &c, float &s)
{
    int axis = 0;
#pragma unroll
    for (int a = 0; a < 3; ++a) axis += i >= tab.axis_end[a] ? 1 : 0;
    const double x = (double)positions[axis * ld + t] * tab.turns[i];
    sincospif(2.0f * (float)(x - rint(x)), &s, &c);
    c *= tab.mscale;
    s *= tab.mscale;
}

// Row (page, head, place) of position p of entry b as an index into [n_pages][n_kv][page_size], or -1
// where the entry has no such place.
__device__ __forceinline__ int64_t kv_row(const KvView &kv, const KvBatchView &b, int entry, int64_t p, int head)
{
    const int64_t pg = p >> kv.shift;
    if (p < 0 || pg >= b.max_pages) return -1;
    const int page = b.table[(int64_t)entry * b.max_pages + pg];
    if (page < 0 || page >= kv.n_pages) return -1;
    return (((int64_t)page * kv.n_kv + head) << kv.shift) + (p & ((1 << kv.shift) - 1));
}

// Tokens of entry b that count.
__device__ __forceinline__ int kv_new(const KvBatchView &b, int entry)
{
    return b.n_new ? min(b.n_new[entry], b.n_tok) : b.n_tok;
}

}  // namespace gdn
