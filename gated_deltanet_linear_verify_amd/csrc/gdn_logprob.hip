// gdn_logprob.hip - log probabilities of given tokens, their ranks, the rows' log sum exp and entropy, and their top
// alternatives (gfx950): what a verify step answers with (hf2q qwen35_target.rs, forward_decode_verify_batched: the
// logits of every position and their argmax).
//
// In powers of two, with c = log2(e) / T and a whole number K next to c max x:  a = c x - K (one rounding),
// s = sum 2^a, u = sum 2^a a, and then lse = ln 2 (K + log2 s), entropy = ln 2 (log2 s - u / s) and the log probability of x
// is ln 2 (a - log2 s).  c's own rounding is that of T, the same in all of them.  K is a whole number, but c max x was rounded
// to fp32 on the way to it: the largest a is up to half a step of c max x from 0, 32 below 2^30, where kFar ends it.
//
// A workgroup runs over its slice of a row (the whole row where there are many) in batches of up to 32 KiB that it holds in
// registers: every logit is read once, and a batch's maxima, sums, ranks and candidates come from there.  Each thread sums
// against an exponent of its own, which rises with its maximum.  The k alternatives of the first batch are at least the
// k-th largest of its threads' maxima, which one wave finds by halving; chunks that reach this bar go to a list in LDS, and
// whenever that has grown its logits are ordered by counting, which leaves k of them and a higher bar.  Where too many reach the
// bar because they equal it (a finite mask over most of the row, a row of few values), only larger ones are listed, and the
// places that those leave go to the equal ones by their index, in a pass behind the loop that ends with the last place (8 tokens of
// 131072 allowed beside -1e10, top 20: 1024 rows 58 us, and 53 beside -infinity; one row 11 and 8, and 11 and 5 for the join; one
// alternative at a time took 50 times as long).  Slices of one row meet in the workspace, where a second kernel joins them.
//
// 1024 x 131071 bf16 with a token and 20 alternatives each: 68 us, 3.9 TB/s (a plain read 5.65); the vector unit issues for 78%
// of the time: 8.5 instructions a logit (unpacking 1, the chunks' maxima 1.5, the exponent 1, the power 2, the sums 3).
// One row of 131072: 6.8 us and 6.1 for the join.
#include <algorithm>

#include "gdn_rows.h"

namespace gdn {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int64_t kMaxGrid = (int64_t)0xffffffff / kThreads;  // a launch's x axis holds fewer than 2^32 threads
constexpr int kMaxSlices = 64, kMaxKeys = 1024;  // of a row, and the keys of its slices, which the join orders by counting
constexpr int kList = 1024; // candidates that a workgroup orders by counting
constexpr int kHits = 256;  // chunks that it lists to look through for them,
constexpr int kMany = 40;   // and from how many on it does so before the slice's end
template <bool BF16>
constexpr uint32_t kNone = BF16 ? 0xff80ff80u : 0xff800000u;  // -infinity
constexpr float kInf = __builtin_inff();

// The order of the logits as whole numbers that are never 0: larger logits first, -0 as 0, a NaN as -infinity.
__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t b = __float_as_uint(fmaxf(x, -kInf) + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o); }
// and of equal ones the lower index first: a key is more the earlier
__device__ __forceinline__ uint64_t key_of(float x, int i) { return (uint64_t)order_of(x) << 32 | (uint32_t)~i; }
__device__ __forceinline__ int index_of(uint64_t key) { return (int)~(uint32_t)key; }

template <bool BF16>
__device__ __forceinline__ float logit(const LogprobArgs &a, int64_t row, int i)
{
    return load_act<BF16>(a.logits, row * a.ld + i);
}

// A slice's part of a row in the workspace: its maximum, exponent and sums, the counts of n_ids, the keys of top_k (0: none)
struct Part {
    float top, k, s, u;
};
__host__ __device__ constexpr size_t part_bytes(int n_ids, int top_k)
{
    return sizeof(Part) + ((size_t)n_ids * 4 + 15) / 16 * 16 + ((size_t)top_k * 8 + 15) / 16 * 16;
}
struct PartView {
    Part *stat;
    int32_t *before;
    uint64_t *keys;
};
__device__ __forceinline__ PartView part_at(const LogprobArgs &a, int64_t i)
{
    unsigned char *p = a.ws + i * part_bytes(a.n_ids, a.top_k);
    return {reinterpret_cast<Part *>(p), reinterpret_cast<int32_t *>(p + sizeof(Part)),
            reinterpret_cast<uint64_t *>(p + sizeof(Part) + ((size_t)a.n_ids * 4 + 15) / 16 * 16)};
}

// Sums s and u against the exponent k.  A row (or slice) whose maximum is `far` has none: from 2^30 on logits are equal or at
// least 2^30 2^-24 = 64 powers of two apart, of which 2^24 together are 2^-40 of the largest, so s counts those that are
// equal to the top.  Below, 2^a of the largest logit is within 2^33 of 1.  A thread whose logits are all below
// kNoExponent keeps that exponent, and has nothing beside a row that is not far.
constexpr float kFar = 0x1p30f, kNoExponent = -0x1p31f;
__device__ __forceinline__ bool is_far(float top, float c) { return !(fabsf(top * c) < kFar); }
struct Sums {
    float k, s, u;
    // takes the exponent to `to`, which is at least k
    __device__ void raise(float to)
    {
        const float d = k - to, f = __builtin_amdgcn_exp2f(d);
        u = f * __builtin_fmaf(s, d, u);
        s *= f;
        k = to;
    }
};

// The row's answers from its maximum and sums.
constexpr float kLn2 = 0.693147180559945309f;
struct Row {
    float top, c, k, logs, lse, entropy;
    bool empty, bad, far;
    __device__ Row(float top_, float c_, Sums a) : top(top_), c(c_), k(a.k)
    {
        empty = a.s == 0.0f;  // -infinity everywhere
        bad = !(a.s < kInf);  // a NaN or +infinity among the logits
        far = is_far(top, c);
        logs = log2f(a.s);
        lse = far ? top * (c * kLn2) + logs * kLn2 : (k + logs) * kLn2;
        entropy = far ? logs * kLn2 : fmaxf(logs - a.u / a.s, 0.0f) * kLn2;  // of a row that is sure, both are a top's a
        if (empty) lse = -kInf, entropy = 0.0f;
        if (bad) lse = entropy = __builtin_nanf("");
    }
    __device__ float lp(float x) const
    {
        if (bad) return __builtin_nanf("");
        if (empty) return -kInf;
        const float d = __builtin_fmaf(x, c, -k);  // c x may pass fp32's range where ln 2 times it does not
        // and x - top may where its halves, times 2 c, do not
        if (far || (!(d > -kInf) && x > -kInf)) return (0.5f * x - 0.5f * top) * (2.0f * kLn2 * c) - logs * kLn2;
        return (d - logs) * kLn2;
    }
};

// 16 bytes of a row: 8 or 4 logits, in fp32.  bf16's are unpacked by instructions that the compiler does not know, so that
// each phase unpacks anew: kept from one to the next they would take twice the registers, and spill.
template <bool BF16>
__device__ __forceinline__ void unpack(const uint32_t (&w)[4], float (&x)[BF16 ? 8 : 4])
{
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (BF16) {
#if defined(__HIP_DEVICE_COMPILE__)
            asm volatile("v_lshlrev_b32 %0, 16, %1" : "=v"(x[2 * q]) : "v"(w[q]));
            asm volatile("v_and_b32 %0, 0xffff0000, %1" : "=v"(x[2 * q + 1]) : "v"(w[q]));
#endif
        } else {
            x[q] = __uint_as_float(w[q]);
        }
    }
}

// What all threads read alike from LDS, in a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ float uniform(float x) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x))); }

// The thread's index as a value of its own: what a rare phase makes of it is computed there, not ahead of the loop around it,
// where it would take registers all along.
__device__ __forceinline__ int own_index()
{
    int t = threadIdx.x;
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(t));
#endif
    return t;
}

__device__ __forceinline__ float wave_max(float x)
{
    x = fmaxf(x, dpp_mov<0xB1>(x));
    x = fmaxf(x, dpp_mov<0x4E>(x));
    x = fmaxf(x, dpp_mov<0x141>(x));
    x = fmaxf(x, dpp_mov<0x140>(x));
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
#if defined(__HIP_DEVICE_COMPILE__)
    float r;  // fmaxf would first quiet each operand, an instruction of its own
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
#else
    return fmaxf(a, fmaxf(b, c));
#endif
}

// The largest logit of a chunk (of one with a NaN it may be NaN: such a slice takes its alternatives another way).
template <bool BF16>
__device__ __forceinline__ float chunk_max(const uint32_t (&w)[4])
{
    float r = -kInf;
    if constexpr (BF16) {
#pragma unroll
        for (int q = 0; q < 4; ++q) r = max3(r, __uint_as_float(w[q] & 0xffff0000u), __uint_as_float(w[q] << 16));
    } else {
        r = max3(r, __uint_as_float(w[0]), __uint_as_float(w[1]));
        r = max3(r, __uint_as_float(w[2]), __uint_as_float(w[3]));
    }
    return r;
}

// The largest number below x in fp32 (of -infinity: a NaN), so that v >= x where not v <= below(x).
__device__ __forceinline__ float below(float x)
{
    const uint32_t b = __float_as_uint(x);
    return __uint_as_float(x == 0.0f ? 0x80000001u : b & 0x80000000u ? b + 1 : b - 1);
}
// The smallest one above x, so that v > x where v >= above(x).
__device__ __forceinline__ float above(float x)
{
    const uint32_t b = __float_as_uint(x);
    return __uint_as_float(x == 0.0f ? 1u : b & 0x80000000u ? b - 1 : b + 1);
}

// How many of the n keys are above `mine`, two to a read.
__device__ __forceinline__ int count_above(const uint64_t *keys, int n, uint64_t mine)
{
    const ulonglong2 *pairs = reinterpret_cast<const ulonglong2 *>(keys);
    int c = (n & 1) && keys[n - 1] > mine;
#pragma unroll 4
    for (int j = 0; j < n / 2; ++j) {
        const ulonglong2 q = pairs[j];
        c += (q.x > mine) + (q.y > mine);
    }
    return c;
}

// Places k .. top_k of a row's alternatives, where only -infinity (and NaN) is left: by their index, 64 at a time (one wave).
template <bool BF16>
__device__ void fill_masked(const LogprobArgs &a, int64_t row, const Row &r, int k)
{
    const int lane = own_index() & 63;
    for (int i0 = 0; i0 < a.V && k < a.top_k; i0 += 64) {
        const int i = i0 + lane;
        const bool gone = i < a.V && fmaxf(logit<BF16>(a, row, i), -kInf) == -kInf;
        const uint64_t which = __ballot(gone);
        const int place = k + __popcll(which & ((1ull << lane) - 1));
        if (gone && place < a.top_k) {
            a.top_ids[row * a.top_k + place] = i;
            a.top_logprob[row * a.top_k + place] = r.lp(-kInf);
        }
        k += __popcll(which);
    }
}

// CH: chunks of 16 bytes per thread and batch.  Slice blockIdx.x % slices of row blockIdx.x / slices.
template <bool BF16, int CH>
__global__ __launch_bounds__(kThreads, 5) void logprob_slice_kernel(LogprobArgs a, int slices)
{
    constexpr int E = BF16 ? 8 : 4, kSize = BF16 ? 2 : 4, kBatch = kThreads * CH;
    __shared__ float tops[kThreads], singles[16], sum_k[kWaves], sum_s[kWaves], sum_u[kWaves], given[kMaxIds], bar_lds;
    __shared__ __attribute__((aligned(16))) uint4 hit[kHits];
    __shared__ __attribute__((aligned(16))) uint64_t list[2][kList];
    __shared__ uint64_t best[kWaves];
    __shared__ int hit_at[kHits], hits, listed, ids[kMaxIds], before[kMaxIds];
    int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int64_t row = a.row0 + blockIdx.x / slices;
    const int slice = blockIdx.x % slices;
    // A row is `head` logits up to the first 16-byte boundary, chunks of 16 bytes, and a tail.  Head and tail go as single
    // values to threads of the first and the last slice.
    const unsigned char *p = static_cast<const unsigned char *>(a.logits) + row * a.ld * kSize;
    const int head = min(a.V, (int)((16 - ((uintptr_t)p & 15)) & 15) / kSize), chunks = (a.V - head) / E;
    const int tail = (a.V - head) % E, per = (chunks + slices - 1) / slices;
    const int c0 = min(slice * per, chunks), c1 = min(c0 + per, chunks);
    const int first_i = c0 * E + head, end_i = c1 * E + head;  // the logits of the slice's chunks
    const unsigned char *body = p + head * kSize;
    const float c2 = a.inv_t * kLog2E;

    // The single values wait in LDS: kept in registers through the loop they would make others spill.
    const bool in_head = slice == 0 && tid < head, in_tail = slice == slices - 1 && tid >= 64 && tid < 64 + tail;
    auto extra_of = [&](int t) { return in_head ? t : in_tail ? a.V - tail + t - 64 : -1; };
    auto single_of = [&](int t) -> float & { return singles[in_head ? t : 8 + (t & 7)]; };
    const int extra = extra_of(tid);
    const float single = extra >= 0 ? logit<BF16>(a, row, extra) : -kInf;
    if (extra >= 0) single_of(tid) = single;
    if (tid < a.n_ids) {
        int id = a.ids[row * a.n_ids + tid], n = 0;
        if (id < 0 || id >= a.V) id = -1;
        const float x = id >= 0 ? logit<BF16>(a, row, id) : 0.0f;
        // how many equal logits are before a given token in its own chunk
        if (id >= first_i && id < end_i)
            for (int i = id - (id - head) % E; i < id; ++i) n += logit<BF16>(a, row, i) == x;
        ids[tid] = id;
        given[tid] = x;
        before[tid] = n;
    }
    if (tid == 0) hits = listed = 0;

    Sums sum{kNoExponent, 0.0f, 0.0f};
    float top = fmaxf(single, -kInf), bar = -kInf;
    int kept = 0;        // ordered entries at the front of list[side]
    int side = 0;
    bool first = true;   // nothing has been ordered yet
    bool slow = false;   // alternatives one at a time, behind the loop
    // Where very many logits are equal to the bar (a finite mask, a row of few values) only larger ones are listed: `equal` is
    // that bar, which at least top_k logits of the slice reach, and the places that larger ones leave are filled behind the loop.
    bool wide = false;   // at least top_k logits reach the bar, and those equal to it are listed
    bool closed = false; // there is an `equal`
    float equal = 0.0f;
    auto close = [&] {
        equal = bar;
        bar = above(bar);
        closed = true;
        wide = false;
    };
    // A batch is summed by itself (up to 64 logits a thread) before it joins the sums: one chain of additions over a long row of
    // equal logits would round the same way at each (2^22 of them: off by 2e-4).
    float bs = 0.0f, bu = 0.0f;
    auto add = [&](float x) {
        const float d = __builtin_fmaf(x, c2, -sum.k), e = __builtin_amdgcn_exp2f(d);
        bs += e;
        bu = __builtin_fmaf(e, fmaxf(d, -1e30f), bu);  // a masked logit's e is 0, but not its d
    };
    auto join = [&] {
        sum.s += bs;
        sum.u += bu;
        bs = bu = 0.0f;
    };
    // The logits of the listed chunks that reach the bar, and what was kept, ordered: all threads, between barriers.
    // Those of -infinity are not listed.  The head's come first, as its indexes do, and the tail's last.
    auto order = [&](int n_hits, bool last) {
        const int tid = own_index();
        auto offer = [&](float x, int i) {
            if (x >= bar && x > -kInf) {
                const int at = kept + atomicAdd(&listed, 1);
                if (at < kList) list[side][at] = key_of(x, i);
            }
        };
        int n;
        for (;;) {
            for (int i = tid; i < n_hits * E; i += kThreads) {
                const int c = i / E, j = i % E;
                const uint32_t v = reinterpret_cast<const uint32_t *>(hit)[4 * c + (BF16 ? j / 2 : j)];
                offer(__uint_as_float(BF16 ? (j % 2 ? v & 0xffff0000u : v << 16) : v), hit_at[c] * E + j + head);
            }
            if ((in_head && first) || (in_tail && last)) offer(single_of(tid), extra_of(tid));
            __syncthreads();
            n = kept + uniform(listed);
            if (n <= kList || !wide) break;
            close();
            __syncthreads();
            if (tid == 0) listed = 0;
            __syncthreads();
        }
        first = false;
        if (n > kList) {
            slow = true;
        } else {
            for (int i = tid; i < n; i += kThreads) {
                const uint64_t mine = list[side][i];
                const int place = count_above(list[side], n, mine);
                if (place < a.top_k) list[side ^ 1][place] = mine;
                if (place == a.top_k - 1) bar_lds = value_of((uint32_t)(mine >> 32));
            }
            kept = min(n, a.top_k);
            side ^= 1;
        }
        __syncthreads();
        // those that come behind and equal the last one kept are after it
        const float last_kept = uniform(bar_lds);
        if (kept == a.top_k && !slow && last_kept >= bar) {
            bar = above(last_kept);
            wide = false;
        }
        if (tid == 0) hits = listed = 0;
        __syncthreads();
    };

    uint32_t w[CH][4];
    auto load_at = [&](int c, uint32_t (&to)[4]) {  // chunk c, of -infinities past the slice's end
        uint4 v = make_uint4(kNone<BF16>, kNone<BF16>, kNone<BF16>, kNone<BF16>);
        if (c < c1) v = *reinterpret_cast<const uint4 *>(body + (uint32_t)c * 16u);
        to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
    };
    auto load = [&](int b, int i) { load_at(b + tid + i * kThreads, w[i]); };  // chunk i of the batch from b on
#pragma unroll
    for (int i = 0; i < CH; ++i) load(c0, i);
    sum.k = fmaxf(sum.k, rintf(single * c2));
    add(single);
    join();
    __syncthreads();
    if (extra >= 0)
        for (int k = 0; k < a.n_ids; ++k) {
            const float mine = fmaxf(given[k], -kInf);
            if (!(single <= (extra < ids[k] ? below(mine) : mine))) atomicAdd(&before[k], 1);
        }
#pragma unroll 1
    for (int b0 = c0; b0 < c1 || b0 == c0; b0 += kBatch) {
        float cm[CH], batch_top = b0 == c0 ? top : -kInf;  // the largest of each chunk, and of the thread's
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            cm[i] = chunk_max<BF16>(w[i]);
            batch_top = max3(batch_top, cm[i], cm[i]);
        }
        top = fmaxf(top, batch_top);
        const float to = fmaxf(sum.k, rintf(batch_top * c2));
        if (__ballot(to > sum.k)) sum.raise(to);
        for (int k = 0; k < a.n_ids; ++k) {
            const int id = ids[k];
            const float mine = fmaxf(given[k], -kInf);
            if (id < 0 || !__ballot(batch_top >= mine)) continue;
            const float or_equal = below(mine);
            int n = 0;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                if (!__ballot(cm[i] >= mine)) continue;
                float x[E];
                unpack<BF16>(w[i], x);
                // equal ones count in the chunks that end before id's own (whose equal ones were counted above)
                const int c = b0 + tid + i * kThreads;
                const float than = c < c1 && (c + 1) * E + head <= id ? or_equal : mine;
#pragma unroll
                for (int j = 0; j < E; ++j) n += __popcll(__ballot(!(x[j] <= than)));
            }
            if (lane == 0) atomicAdd(&before[k], n);
        }
        float raised = -kInf;
        // stage 1 raises the bar by this batch's maxima, stage 2 leaves what equals it for later
        for (int stage = b0 == c0; a.top_k && !slow; ++stage) {
            if (stage == 1) {
                // a bar that at least top_k of the threads' maxima reach, and few more: by halving the range that they span
                tops[tid] = batch_top;
                __syncthreads();
                if (wave == 0) {
                    uint32_t o[kWaves], lo = ~0u, hi = 0;
#pragma unroll
                    for (int i = 0; i < kWaves; ++i) {
                        o[i] = order_of(tops[lane + 64 * i]);
                        lo = min(lo, o[i]);
                        hi = max(hi, o[i]);
                    }
#pragma unroll
                    for (int x = 1; x < 64; x *= 2) {
                        lo = min(lo, (uint32_t)__shfl_xor((int)lo, x));
                        hi = max(hi, (uint32_t)__shfl_xor((int)hi, x));
                    }
                    uint32_t found = __builtin_amdgcn_readfirstlane(lo);
                    hi = __builtin_amdgcn_readfirstlane(hi);
                    while (found < hi) {
                        const uint32_t at = found + (hi - found + 1) / 2;
                        int n = 0;
#pragma unroll
                        for (int i = 0; i < kWaves; ++i) n += __popcll(__ballot(o[i] >= at));
                        if (n >= a.top_k)
                            found = at;
                        else
                            hi = at - 1;
                        if (n >= a.top_k && n <= a.top_k + 4) break;
                    }
                    if (lane == 0) bar_lds = value_of(found);
                }
                __syncthreads();
                const float most = uniform(bar_lds);
                if (most >= bar) {
                    bar = most;
                    wide = bar > -kInf;
                }
                raised = bar;
            } else if (stage > 1) {
                if (stage > 2 || (bar == raised && !wide)) slow = true;
                if (slow) break;
                if (bar == raised) close();
            }
            const int had = uniform(hits);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                if (cm[i] >= bar && cm[i] > -kInf) {
                    const int at = atomicAdd(&hits, 1);
                    if (at < kHits) {
                        hit[at] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
                        hit_at[at] = b0 + tid + i * kThreads;
                    }
                }
            }
            __syncthreads();
            const int have = uniform(hits);
            // too many: logits that rise from batch to batch, the first that are not masked, or very many equal ones; what was there
            // before is ordered, and the bar raised
            const bool fit = have <= kHits && (stage || have - had <= kMany);
            if (!fit || have > kMany) order(fit ? have : had, false);
            if (fit) break;
        }
        // the sums, each chunk's registers taking the next batch's at once
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            if (b0 + i * kThreads >= c1) continue;
            float x[E];
            unpack<BF16>(w[i], x);
#pragma unroll
            for (int j = 0; j < E; ++j) add(x[j]);
            load(b0 + kBatch, i);
        }
        join();
    }

    tid = own_index();
    wave = tid >> 6;
    lane = tid & 63;
    // the workgroup's maximum and sums
    {
        float k = wave_max(sum.k), t = wave_max(fmaxf(top, -kInf));
        sum.raise(k);
        sum.s = wave_sum(sum.s);
        sum.u = wave_sum(sum.u);
        __syncthreads();
        if (lane == 0) {
            tops[wave] = t;
            sum_k[wave] = k;
            sum_s[wave] = sum.s;
            sum_u[wave] = sum.u;
        }
        __syncthreads();
        float s = 0.0f, u = 0.0f;
        k = sum_k[0];
        top = tops[0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) k = fmaxf(k, sum_k[i]), top = fmaxf(top, tops[i]);
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            Sums q{sum_k[i], sum_s[i], sum_u[i]};
            q.raise(k);
            s += q.s;
            u += q.u;
        }
        sum = Sums{k, s, u};
    }
    if (is_far(top, c2) && top != -kInf) {  // rare: the sum is a count
        float n = 0.0f;
        auto count = [&](float x) { n += !(x < kInf) ? __builtin_nanf("") : x == top ? 1.0f : 0.0f; };
        for (int i = first_i + tid; i < end_i; i += kThreads) count(logit<BF16>(a, row, i));
        if (extra_of(tid) >= 0) count(single_of(tid));
        n = wave_sum(n);
        __syncthreads();
        if (lane == 0) sum_s[wave] = n;
        __syncthreads();
        sum = Sums{kNoExponent, 0.0f, 0.0f};
        for (int i = 0; i < kWaves; ++i) sum.s += sum_s[i];
    }
    const Row r(top, c2, sum);
    const bool whole = slices == 1;
    const PartView part = part_at(a, row * slices + slice);
    if (r.bad && a.n_ids) {  // a NaN or +infinity was passed over: count again, by the order's keys
        __syncthreads();
        if (tid < a.n_ids) before[tid] = 0;
        __syncthreads();
        for (int k = 0; k < a.n_ids; ++k) {
            if (ids[k] < 0) continue;
            const uint64_t key = key_of(given[k], ids[k]);
            int n = extra_of(tid) >= 0 && key_of(single_of(tid), extra_of(tid)) > key;
            for (int i = first_i + tid; i < end_i; i += kThreads) n += key_of(logit<BF16>(a, row, i), i) > key;
            if (n) atomicAdd(&before[k], n);
        }
        __syncthreads();
    }
    if (whole) {
        if (tid == 0 && a.lse) a.lse[row] = r.lse;
        if (tid == 0 && a.entropy) a.entropy[row] = r.entropy;
        if (tid < a.n_ids) {
            const int64_t at = row * a.n_ids + tid;
            if (a.rank) a.rank[at] = ids[tid] >= 0 ? before[tid] : -1;
            if (a.logprob) a.logprob[at] = ids[tid] >= 0 ? r.lp(given[tid]) : -kInf;
        }
    } else {
        if (tid == 0) *part.stat = Part{top, sum.k, sum.s, sum.u};
        if (tid < a.n_ids) part.before[tid] = before[tid];
    }
    if (!a.top_k) return;
    auto put = [&](int k, uint64_t key) {
        if (!whole) {
            part.keys[k] = key;
            return;
        }
        a.top_ids[row * a.top_k + k] = index_of(key);
        a.top_logprob[row * a.top_k + k] = r.lp(value_of((uint32_t)(key >> 32)));
    };
    if (!slow && !r.bad) order(hits, true);
    if (!slow && !r.bad) {
        int n = kept;
        if (closed) n = __popcll(__ballot(lane < kept && (uint32_t)(list[side][lane] >> 32) > order_of(equal)));
        for (int i = tid; i < (whole || closed ? n : a.top_k); i += kThreads) put(i, i < n ? list[side][i] : 0);
        if (!closed) {
            if (whole && n < a.top_k && wave == 0) fill_masked<BF16>(a, row, r, n);
            return;
        }
        // places n .. top_k: those equal to `equal` by their index, up to a chunk per thread at a time (bit j: base + j is one)
        auto fill = [&](uint32_t which, int base) {
            int upto = __popc(which);
#pragma unroll
            for (int o = 1; o < 64; o *= 2) {
                const int u = __shfl_up(upto, o);
                upto += lane >= o ? u : 0;
            }
            __syncthreads();  // the last round's counts have been read
            if (lane == 63) hit_at[wave] = upto;
            __syncthreads();
            int at = n + upto - __popc(which);
#pragma unroll
            for (int i = 0; i < kWaves; ++i) {
                at += i < wave ? hit_at[i] : 0;
                n += hit_at[i];
            }
            for (; which && at < a.top_k; which &= which - 1) put(at++, key_of(equal, base + __ffs(which) - 1));
        };
        if (n < a.top_k) fill(in_head && single_of(tid) == equal, tid);
        for (int b = c0; b < c1 && n < a.top_k; b += kThreads) {
            load_at(b + tid, w[0]);
            float x[E];
            unpack<BF16>(w[0], x);
            uint32_t which = 0;
#pragma unroll
            for (int j = 0; j < E; ++j) which |= (uint32_t)(x[j] == equal) << j;
            fill(which, (b + tid) * E + head);
        }
        if (n < a.top_k) fill(in_tail && single_of(tid) == equal, extra_of(tid));
        return;
    }
    // A NaN or +infinity among the logits, or candidates past the lists, as where few threads hold them all: one alternative at a
    // time, the largest key below the last.
    uint64_t last = ~0ull;
    for (int k = 0; k < a.top_k; ++k) {
        uint64_t mine = extra_of(tid) >= 0 ? key_of(single_of(tid), extra_of(tid)) : 0;
        if (mine >= last) mine = 0;
        for (int i = first_i + tid; i < end_i; i += kThreads) {
            const uint64_t key = key_of(logit<BF16>(a, row, i), i);
            if (key < last) mine = max(mine, key);
        }
#pragma unroll
        for (int o = 1; o < 64; o *= 2) mine = max(mine, (uint64_t)__shfl_xor((unsigned long long)mine, o));
        __syncthreads();
        if (lane == 0) best[wave] = mine;
        __syncthreads();
        last = 0;
        for (int i = 0; i < kWaves; ++i) last = max(last, best[i]);
        if (tid == 0) put(k, last);
        if (!last) last = 1;  // a slice of fewer logits than top_k has no more
    }
}

// One workgroup joins the slices of a row.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void logprob_join_kernel(LogprobArgs a, int slices)
{
    extern __shared__ __attribute__((aligned(16))) uint64_t keys[];  // [slices][top_k], and as many again
    __shared__ uint64_t bar;
    __shared__ int listed, found, before[kMaxIds];
    const int tid = threadIdx.x, lane = tid & 63;
    const int64_t row = a.row0 + blockIdx.x, part0 = row * slices;
    int id = -1;
    float given = 0.0f;
    if (tid < a.n_ids) {
        id = a.ids[row * a.n_ids + tid];
        if (id < 0 || id >= a.V) id = -1;
        if (id >= 0) given = logit<BF16>(a, row, id);
        before[tid] = 0;
    }
    if (tid == 0) {
        found = listed = 0;
        bar = 0;
    }
    for (int i = tid; i < slices * a.top_k; i += kThreads) keys[i] = part_at(a, part0 + i / a.top_k).keys[i % a.top_k];
    // every wave takes the slices' sums, a slice per lane
    const float c2 = a.inv_t * kLog2E;
    float top = -kInf, k = kNoExponent;
    for (int i = lane; i < slices; i += 64) {
        const Part q = *part_at(a, part0 + i).stat;
        top = fmaxf(top, q.top);
        k = fmaxf(k, q.k);
    }
    top = wave_max(top);
    k = wave_max(k);
    Sums sum{k, 0.0f, 0.0f};
    for (int i = lane; i < slices; i += 64) {
        const Part p = *part_at(a, part0 + i).stat;
        Sums q{p.k, p.s, p.u};
        // a slice whose own maximum is far counts where the row's is the same, and has nothing beside a larger one
        if (is_far(top, c2))
            q = Sums{k, p.top == top || !(p.s < kInf) ? p.s : 0.0f, 0.0f};
        else if (is_far(p.top, c2) && p.s < kInf)
            q = Sums{k, 0.0f, 0.0f};
        else
            q.raise(k);
        sum.s += q.s;
        sum.u += q.u;
    }
    // the lanes add in orders of their own, and have to go on with one result
    sum.s = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(wave_sum(sum.s))));
    sum.u = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(wave_sum(sum.u))));
    const Row r(top, c2, sum);
    if (tid == 0 && a.lse) a.lse[row] = r.lse;
    if (tid == 0 && a.entropy) a.entropy[row] = r.entropy;
    __syncthreads();
    if (a.n_ids) {
        for (int i = tid; i < slices * a.n_ids; i += kThreads) {
            const int n = part_at(a, part0 + i / a.n_ids).before[i % a.n_ids];
            if (n) atomicAdd(&before[i % a.n_ids], n);
        }
        __syncthreads();
        if (tid < a.n_ids) {
            const int64_t at = row * a.n_ids + tid;
            if (a.rank) a.rank[at] = id >= 0 ? before[tid] : -1;
            if (a.logprob) a.logprob[at] = id >= 0 ? r.lp(given) : -kInf;
        }
    }
    if (!a.top_k) return;
    auto put = [&](int k, int i, float x) {
        a.top_ids[row * a.top_k + k] = i;
        a.top_logprob[row * a.top_k + k] = r.lp(x);
    };
    // The slices' keys are in order: the top_k-th of the first few of each is a bar that at least top_k keys reach, and not
    // many more (counting among all of them took 30 us for 32 slices of 20, this 4).  Where many logits are equal, the first
    // slices have all the keys, and a bar from as many of each as there are threads leaves fewer of them.
    const int n = slices * a.top_k;
    uint64_t *some = keys + (n + 1) / 2 * 2;
    for (int each = (a.top_k + slices - 1) / slices, last = 0;; each = min(a.top_k, kThreads / slices), last = 1) {
        const int m = each * slices;
        if (tid < m) some[tid] = keys[tid / each * a.top_k + tid % each];
        __syncthreads();
        if (tid < m && some[tid] && count_above(some, m, some[tid]) == a.top_k - 1) bar = some[tid];
        __syncthreads();
        int mine = 0;
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t key = keys[i];
            if (!key || value_of((uint32_t)(key >> 32)) == -kInf) continue;
            ++mine;
            if (key >= bar) some[atomicAdd(&listed, 1)] = key;
        }
        if (mine && !last) atomicAdd(&found, mine);
        __syncthreads();
        if (last || listed <= kThreads / 2) break;
        __syncthreads();
        if (tid == 0) listed = 0;
    }
    for (int i = tid; i < listed; i += kThreads) {
        const uint64_t key = some[i];
        const int place = count_above(some, listed, key);
        if (place < a.top_k) put(place, index_of(key), value_of((uint32_t)(key >> 32)));
    }
    if (found < a.top_k && tid < 64) fill_masked<BF16>(a, row, r, found);
}

// Chunks per thread and batch, and slices of a row.
struct Shape {
    int ch, slices;
};
Shape shape_of(int64_t n_rows, int V, bool bf16, int top_k)
{
    const int chunks = V / (bf16 ? 8 : 4);
    auto batches = [&](int ch) { return std::max(1, (chunks + kThreads * ch - 1) / (kThreads * ch)); };
    const int ch = n_rows * batches(8) >= 512 ? 8 : 2;
    const int64_t most = std::min<int64_t>(std::min(kMaxSlices, kMaxKeys / std::max(1, top_k)), 1024 / n_rows);
    return {ch, (int)std::min<int64_t>(batches(ch), std::max<int64_t>(1, most))};
}

template <bool BF16, int CH>
hipError_t launch_as(LogprobArgs a, int slices, hipStream_t stream)
{
    const int64_t run = kMaxGrid / slices;  // rows of one launch
    for (a.row0 = 0; a.row0 < a.n_rows; a.row0 += run) {
        const unsigned rows = (unsigned)std::min(run, a.n_rows - a.row0);
        hipLaunchKernelGGL((logprob_slice_kernel<BF16, CH>), dim3(rows * slices), dim3(kThreads), 0, stream, a, slices);
        if (hipError_t e = hipGetLastError()) return e;
        if (slices == 1) continue;
        hipLaunchKernelGGL((logprob_join_kernel<BF16>), dim3(rows), dim3(kThreads),
                           ((size_t)slices * a.top_k + 1) / 2 * 32, stream, a, slices);
        if (hipError_t e = hipGetLastError()) return e;
    }
    return hipSuccess;
}

}  // namespace

size_t logprob_workspace_bytes(int64_t n_rows, int V, bool bf16, int n_ids, int top_k)
{
    const int slices = n_rows ? shape_of(n_rows, V, bf16, top_k).slices : 1;
    return slices == 1 ? 0 : n_rows * slices * part_bytes(n_ids, top_k);
}

hipError_t launch_logprob(const LogprobArgs &a, hipStream_t stream)
{
    const Shape s = shape_of(a.n_rows, a.V, a.bf16, a.top_k);
    if (a.bf16) return s.ch == 8 ? launch_as<true, 8>(a, s.slices, stream) : launch_as<true, 2>(a, s.slices, stream);
    return s.ch == 8 ? launch_as<false, 8>(a, s.slices, stream) : launch_as<false, 2>(a, s.slices, stream);
}

}  // namespace gdn
