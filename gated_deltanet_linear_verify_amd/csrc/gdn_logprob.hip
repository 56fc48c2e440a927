// gdn_logprob.hip - log probabilities of given tokens, their ranks, the rows' log sum exp and entropy, and their top
// alternatives (gfx950): what a verify step answers with (hf2q qwen35_target.rs, forward_decode_verify_batched: the
// logits of every position and their argmax).
//
// l = logits / T, m = max l, s = sum e^(l - m), u = sum e^(l - m) (l - m):  lse = m + log s,  entropy = log s - u / s.
#include "gdn_rows.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;

// The order of the logits: larger first, of equal ones the lower index, a NaN as -infinity, -0 as 0.  A key is more the earlier.
__device__ __forceinline__ uint64_t key_of(float x, int i)
{
    uint32_t b = __float_as_uint(fmaxf(x, -__builtin_inff()) + 0.0f);
    b = b & 0x80000000u ? ~b : b | 0x80000000u;
    return (uint64_t)b << 32 | (uint32_t)~i;
}

__device__ __forceinline__ float logit(const LogprobArgs &a, int64_t row, int i)
{
    const int64_t at = row * a.ld + i;
    return a.bf16 ? bf16_to_f32(static_cast<const uint16_t *>(a.logits)[at]) : static_cast<const float *>(a.logits)[at];
}

__global__ __launch_bounds__(kThreads) void logprob_kernel(LogprobArgs a)
{
    __shared__ float fs[kThreads];
    __shared__ uint64_t ks[kThreads];
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const float inf = __builtin_inff(), t = a.inv_t;
    auto sum = [&](float v) {
        __syncthreads();
        fs[tid] = v;
        __syncthreads();
        for (int o = kThreads / 2; o; o /= 2) {
            if (tid < o) fs[tid] += fs[tid + o];
            __syncthreads();
        }
        return fs[0];
    };
    auto most = [&](uint64_t v) {
        __syncthreads();
        ks[tid] = v;
        __syncthreads();
        for (int o = kThreads / 2; o; o /= 2) {
            if (tid < o) ks[tid] = max(ks[tid], ks[tid + o]);
            __syncthreads();
        }
        return ks[0];
    };
    uint64_t top = 0;
    for (int i = tid; i < a.V; i += kThreads) top = max(top, key_of(logit(a, row, i), i));
    const float m = logit(a, row, (int)~(uint32_t)most(top)), base = fmaxf(m, -3.40282347e38f);
    float s = 0.0f, u = 0.0f;
    for (int i = tid; i < a.V; i += kThreads) {
        const float d = (logit(a, row, i) - base) * t, e = expf(d);
        s += e;
        u += e > 0.0f ? e * d : e;
    }
    s = sum(s);
    u = sum(u);
    const float logs = logf(s), lse = m > -inf ? m * t + logs : s == 0.0f ? -inf : s;
    if (tid == 0 && a.lse) a.lse[row] = lse;
    if (tid == 0 && a.entropy) a.entropy[row] = s == 0.0f ? 0.0f : logs - u / s;
    auto lp = [&](float x) { return s == 0.0f ? -inf : (x - base) * t - logs; };
    for (int k = 0; k < a.n_ids; ++k) {
        const int id = a.ids[row * a.n_ids + k];
        const bool valid = id >= 0 && id < a.V;
        const uint64_t mine = valid ? key_of(logit(a, row, id), id) : 0;
        int before = 0;
        for (int i = tid; i < a.V; i += kThreads) before += key_of(logit(a, row, i), i) > mine;
        before = (int)sum((float)before);
        if (tid == 0) {
            if (a.rank) a.rank[row * a.n_ids + k] = valid ? before : -1;
            if (a.logprob) a.logprob[row * a.n_ids + k] = valid ? lp(logit(a, row, id)) : -inf;
        }
    }
    uint64_t last = ~0ull;
    for (int k = 0; k < a.top_k; ++k) {
        uint64_t best = 0;
        for (int i = tid; i < a.V; i += kThreads) {
            const uint64_t key = key_of(logit(a, row, i), i);
            if (key < last) best = max(best, key);
        }
        last = most(best);
        const int id = (int)~(uint32_t)last;
        if (tid == 0) {
            a.top_ids[row * a.top_k + k] = id;
            a.top_logprob[row * a.top_k + k] = lp(logit(a, row, id));
        }
    }
}

}  // namespace

size_t logprob_workspace_bytes(int64_t, int, bool, int, int) { return 0; }

hipError_t launch_logprob(const LogprobArgs &a, hipStream_t stream)
{
    hipLaunchKernelGGL(logprob_kernel, dim3(a.n_rows), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdn
