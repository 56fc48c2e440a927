// gdn_attn.hip - attention of drafted tokens over the paged KV cache (gfx950).
//
//   o_r = sum_j w_rj v_j / sum_j w_rj,   w_rj = 2^(s_rj - m_r),   s_rj = log2(e) scale q_r . k_j
//
// over the keys j that row r sees, with the running maximum m_r and sum kept per row while the keys
// pass by once (lucebox-hub internal.h, struct QwenGraphInputs: full attention over the cache for the
// tokens of a chain or tree).  A row is a (token, query head of the group) pair: the group's query
// heads share a KV head, so all rows of an entry share the keys, and the rows of all entries share
// those of a prefix.
//
// Work: items are (KV head, tile of rows) with their key tiles in sequence.  A launch's key tiles, all
// items one after another, are cut into equal runs, one per workgroup, whatever the lengths in the
// cache are; a workgroup scans the entries' lengths at its start to find its run.  An item cut by a
// run's end leaves partial results (o, m, l) in the workspace, joined by attn_join_kernel.
//
// Tile: a workgroup's NR x NK waves hold 16 RT NR rows; each wave takes BN / NK of the tile's keys.
// S^T = K Q^T and O^T = V^T P^T on 16x16x32 MFMA: with the keys along the result's rows, a lane's
// scores, its row's maximum, sum and outputs all belong to query row lane % 16, so the softmax needs
// two cross-lane steps per tile and P goes from the first product's result registers to the second's
// operand registers without leaving the lane (the key order inside a 32-deep step is permuted alike
// on both operands).
//
// Formats.  A bf16 cache goes into LDS as it is (global_load_lds), and the second product takes its
// weights in bf16: in two parts (at most 2^-15 of a weight is lost) in tiles of up to 64 rows, which the cache's
// bytes bound (32 entries of 1000 .. 4000 keys, 16 to 64 rows: d 128 + 0 .. 1%, d 256 + 2 .. 4%), in one
// beyond, where the second part's products would cost 5 .. 22% (128 and 256 rows) for an error of 2^-9 of a
// weight, rms, beside the 2^-9 of the stored result.  8-bit codes travel through registers and are widened on
// the way into LDS, k to bf16 and v to fp16, both exactly.  The k scale multiplies the scores; the v scale is
// folded into the exponent, w_j = 2^(s_j + log2 vs_j - m) with m 7 to 15 below the maximum of that sum, so the
// largest weight lies in 2^7 .. 2^15 whatever the scales are and rounding to fp16 costs at most 2^-11 of a weight
// down to 2^-21 of the largest, and 2^-32 of the largest below that (where one key draws nearly all of a row, the
// others are that small, and they alone make the channels in which its v is 0); the softmax's own sum takes
// w_j / vs_j in fp32.  (That holds while the v scales of the keys a workgroup meets lie within
// 2^100 of each other.  One below 2^-64, 0 among them, counts as 2^-64, which moves an output by at most 448 2^-64.)
//
// What bounds it.  Few rows per key: the cache's bytes (64 tokens over 50 .. 20000 keys each, 8 heads, e4m3:
// 1.35 GB in 245 us, 5.5 TB/s, as fast as a large copy).  Many rows per key: a tile's LDS reads (32 KB per wave
// and tile), its softmax (240 vector instructions beside 64 MFMA at d 128 and 32 rows per wave) and its MFMA
// follow one another in a wave, and two waves per SIMD, which is what the registers hold, overlap them only in
// part: 8.1k shared keys under 64 x 16 rows (half of them there) of 32 heads in e4m3, 72 GFLOP, 120 us under the
// profiler, 0.60 PFLOP/s of 1.40; the vector unit issues in 50% of the time, the matrix unit is busy in 37%.  A wave
// of 32 rows at d <= 128 reads half the LDS bytes per row of one of 16 (the same call: 174 -> 164 us).  One token:
// latency (11 us): a chain of three dependent loads (lengths, page, rows), two barriers of the scan before it, and the
// joins between the key waves.  A long chain (8191 tokens at start 0): 1.2 ms, 0.46 PFLOP/s; from the first drafted
// key on every tile is taken as one that some row may not see, though only the last of a row tile's are.
#include <algorithm>
#include <type_traits>

#include "gdn_rows.h"

namespace gdn {

typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 bf16x4_lds;
typedef unsigned long long u64x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr float kNegInf = -__builtin_inff();
constexpr float kSlack = 8.0f;  // how far the maximum may grow before the sums are rescaled
constexpr float kLift = 7.0f;   // 8-bit caches: the largest weight starts at 2^7 and reaches 2^15 where fp16 ends at 2^16

__device__ __forceinline__ f4 mfma_kq(bf16x8_t a, bf16x8_t b, f4 c)
{
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
#else
    (void)a;
    (void)b;
    return c;
#endif
}

// Transposing LDS load: within 16 lanes, lane i receives element i % 4 of the 4-element chunks that
// lanes i / 4, i / 4 + 4, i / 4 + 8 and i / 4 + 12 address.
__device__ __forceinline__ unsigned long long lds_tr4(const unsigned char *p)
{
#if defined(__HIP_DEVICE_COMPILE__)
    const auto lp = (__attribute__((address_space(3))) bf16x4_lds *)(const_cast<unsigned char *>(p));
    return __builtin_bit_cast(unsigned long long, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(lp));
#else
    (void)p;
    return 0;
#endif
}

// Over the four lanes that share lane % 16 (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float quad_max(float x)
{
#if defined(__HIP_DEVICE_COMPILE__)
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
#endif
    return x;
}
__device__ __forceinline__ float quad_sum(float x)
{
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    return x;
}

// 2^(x - m) with 2^(-inf - -inf) = 0: m is the finite stand-in of soft_max below.
__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float finite_max(float m) { return m == kNegInf ? 0.0f : m; }

// The bf16 value next below w > 0 (below, where w is one itself); 0 for 0, a NaN for a NaN.  What is left of w is
// positive, so an infinity of v times either part keeps its sign (a rest of 0 or less would make it a NaN).
__device__ __forceinline__ float bf16_below(float w)
{
    return __uint_as_float(__builtin_elementwise_sub_sat(__float_as_uint(w), 1u) & 0xffff0000u);
}

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f4 mfma_vp(bf16x8_t a, bf16x8_t b, f4 c) { return mfma_kq(a, b, c); }
__device__ __forceinline__ f4 mfma_vp(f16x8_t a, f16x8_t b, f4 c)
{
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
#else
    (void)a;
    (void)b;
    return c;
#endif
}

// Eight 8-bit codes as bf16 (k) or fp16 (v), exactly.
template <int FMT>
__device__ __forceinline__ u32x4_t widen_k(uint32_t lo, uint32_t hi)
{
    u32x4_t r{};
    const uint32_t w[2] = {lo, hi};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#if defined(__HIP_DEVICE_COMPILE__)
        if constexpr (FMT == kKvE4m3) {
            r[2 * q] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[q], 1.0f, false));
            r[2 * q + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[q], 1.0f, true));
        } else
#endif
        {
            // a whole number of 7 bits and sign: its fp32 ends in 16 zero bits
#pragma unroll
            for (int j = 0; j < 2; ++j)
                r[2 * q + j] = __builtin_amdgcn_perm(__float_as_uint((float)(int8_t)(w[q] >> (16 * j + 8))),
                                                     __float_as_uint((float)(int8_t)(w[q] >> (16 * j))), 0x07060302u);
        }
    }
    return r;
}
template <int FMT>
__device__ __forceinline__ u32x4_t widen_v(uint32_t lo, uint32_t hi)
{
    u32x4_t r{};
    const uint32_t w[2] = {lo, hi};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#if defined(__HIP_DEVICE_COMPILE__)
        if constexpr (FMT == kKvE4m3) {
            r[2 * q] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[q], 1.0f, false));
            r[2 * q + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[q], 1.0f, true));
        } else
#endif
        {
            // code + 128 in the low byte of 0x6400 is 1024 + 128 + code; one subtraction leaves the code
            const uint32_t u = w[q] ^ 0x80808080u;
            const f16x2_t bias = {(_Float16)1152.0f, (_Float16)1152.0f};
            r[2 * q] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - bias);
            r[2 * q + 1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - bias);
        }
    }
    return r;
}

// What is not finite in 16 bytes of v becomes 0; whether there was any.
template <int FMT>
__device__ __forceinline__ bool strip(u32x4_t &v)
{
    uint32_t any = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t off = 0;
        if constexpr (FMT == kKvBf16) {
            off |= (v[q] & 0x7f80u) == 0x7f80u ? 0xffffu : 0u;
            off |= (v[q] & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u;
        } else if constexpr (FMT == kKvE4m3) {
#pragma unroll
            for (int j = 0; j < 4; ++j) off |= ((v[q] >> (8 * j)) & 0x7fu) == 0x7fu ? 0xffu << (8 * j) : 0u;
        }
        v[q] &= ~off;
        any |= off;
    }
    return any != 0;
}

// ---------------------------------------------------------------------------------- items and runs

struct Item {
    int entry;         // batch entry (prefix: unused)
    int row0, rows;    // the tile's first row and the rows there are, among the entry's (prefix: the batch's)
    int ctx;           // keys below it are seen by every row
    int limit;         // keys that exist for this item
    int tiles;
};

// BM_, BN_: the tile's rows and keys where they are known, 0 to take them from the phase.
template <bool PREFIX, int BM_ = 0, int BN_ = 0>
__device__ __forceinline__ Item attn_item(const AttnArgs &a, const AttnPhase &ph, int item)
{
    const int bm = BM_ ? BM_ : ph.bm, bn = BN_ ? BN_ : ph.bn;
    Item it{};
    if constexpr (PREFIX) {
        const int *live = reinterpret_cast<const int *>(a.ws + a.plan.live);
        it.row0 = item * bm;
        it.rows = (a.b.n_new ? live[0] : a.b.n_batch * a.b.n_tok) * a.grp;
        const int64_t cap = (int64_t)a.max_prefix_pages << a.kv.shift;
        it.limit = it.ctx = (int)min((int64_t)max(a.prefix_len[0], 0), cap);
        it.tiles = it.row0 < it.rows ? (it.limit + bn - 1) / bn : 0;
    } else {
        it.entry = ph.row_tiles == 1 ? item : item / ph.row_tiles;
        it.row0 = (item - it.entry * ph.row_tiles) * bm;
        const int start = a.b.start[it.entry], n = kv_new(a.b, it.entry);
        it.rows = n * a.grp;
        // a chain's last row of the tile sees no key after its own token
        const int last = a.parent ? n - 1 : (max(min(it.row0 + bm, it.rows), 1) - 1) / a.grp;
        const int64_t cap = (int64_t)a.b.max_pages << a.kv.shift;
        it.ctx = (int)min((int64_t)max(start, 0), cap);
        it.limit = (int)min((int64_t)max(start, 0) + last + 1, cap);
        it.tiles = start >= 0 && it.row0 < it.rows ? (it.limit + bn - 1) / bn : 0;
    }
    return it;
}

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ uint32_t scalar(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }

// ------------------------------------------------------------------------------------ the tile kernel

template <int D, int FMT, int NR, int NK, int RT, int BN_, int NB_>
struct AttnTile {
    static constexpr int THREADS = 64 * NR * NK, BM = 16 * RT * NR, BN = BN_, KW = BN / NK, KB = KW / 16;
    static constexpr int NB = NB_;                               // buffered tiles
    static constexpr bool DMA = FMT == kKvBf16;                  // straight into LDS
    static constexpr bool TWO = DMA && BM <= 64;                 // weights in two bf16 parts
    static constexpr int ROWB = D * 2;                           // bytes of a row in LDS
    static constexpr int ES = DMA ? 2 : 1, CPR = D * ES / 16;    // 16-byte chunks of a cache row
    static constexpr int NCH = BN * CPR / THREADS;               // chunks of K (and of V) per thread
    // Chunk c of K's row r lies at c ^ (r & SWZ): an operand load takes one chunk of 16 rows.  V's lies at
    // c ^ 2 (r & VSWZ): a transposing load takes two neighbouring chunks of 4 rows per 16 lanes.
    static constexpr int SWZ = (D / 8 < 16 ? D / 8 : 16) - 1, VSWZ = SWZ / 2;
    static constexpr int buf_bytes = 2 * BN * ROWB, merge_bytes = NK > 1 ? BM * D * 4 : 0;
    static constexpr int tile_bytes = NB * buf_bytes > merge_bytes ? NB * buf_bytes : merge_bytes;
    static constexpr int sc_bytes = DMA ? 0 : 3 * BN * 4;        // k scale | log2 v scale | 1 / v scale
    // K and V buffers (reused to join the waves' outputs) | scales | bad | scan | m, l
    static constexpr int o_sc = tile_bytes, o_bad = o_sc + NB * sc_bytes, o_scan = o_bad + 16,
                         o_ml = o_scan + (THREADS + 8) * 4, lds = o_ml + NK * BM * 4;
    static constexpr int waves = NR * NK;
    // workgroups per CU: by LDS, and eight waves (two per SIMD) where the registers allow that
    static constexpr int by_lds = 160 * 1024 / lds, occ = D == 256 ? (waves == 2 ? 1 : 2) : waves == 2 || RT == 2 ? 2 : waves == 4 && D == 128 ? 3 : 4;
    static constexpr int by_waves = 4 * occ / waves, per_cu = by_lds < by_waves ? by_lds : by_waves;
    static_assert(KW % 32 == 0 && NCH >= 1 && BN * CPR % THREADS == 0 && BN <= 128, "tile");
    static_assert(DMA ? NB == 2 : 2 * BN <= THREADS, "staging");
    static_assert(64 / CPR <= 16, "a wave's chunks of one pass lie in one 16-row block");
    static_assert(per_cu >= 1, "one workgroup fits");
};

template <int D, int FMT, int NR, int NK, int RT, int BN, int NB, bool PREFIX>
__global__ __launch_bounds__(64 * NR * NK, (AttnTile<D, FMT, NR, NK, RT, BN, NB>::occ)) void attn_kernel(AttnArgs a)
{
    using TL = AttnTile<D, FMT, NR, NK, RT, BN, NB>;
    constexpr int THREADS = TL::THREADS, BM = TL::BM, KW = TL::KW, KB = TL::KB, NCH = TL::NCH, CPR = TL::CPR;
    constexpr bool DMA = TL::DMA, TWO = TL::TWO;
    constexpr float LIFT = DMA ? 0.0f : kLift;  // bf16 weights have fp32's range
    using P8 = std::conditional_t<DMA, bf16x8_t, f16x8_t>;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    int *bad = reinterpret_cast<int *>(lds + TL::o_bad);  // v of the item's tiles held something not finite
    int *scan = reinterpret_cast<int *>(lds + TL::o_scan);
    float *ml = reinterpret_cast<float *>(lds + TL::o_ml);
    const AttnPhase &ph = PREFIX ? a.plan.prefix : a.plan.suffix;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, lg = lane >> 4, wr = wave / NK, wk = wave % NK;
    // Workgroups are dealt to the 8 XCDs in turn; neighbouring runs, which may share keys, go to one XCD.
    const int W = gridDim.x;
    const int wg = W % 8 ? (int)blockIdx.x : (int)(blockIdx.x % 8) * (W / 8) + (int)(blockIdx.x / 8);

    // ---- this workgroup's run of key tiles.  Every loop below runs alike in all lanes and what steers
    // the kernel is held in scalar registers: values kept in vector registers across lane-dependent
    // branches have come back wrong from spills that the compiler restored with no lane active.
    const int chunk = (ph.items + THREADS - 1) / THREADS;
    int mine = 0, t_last = 0;
    for (int j = 0; j < chunk; ++j) {
        const int i = tid * chunk + j;
        t_last = attn_item<PREFIX, BM, BN>(a, ph, min(i, ph.items - 1)).tiles;
        mine += i < ph.items ? t_last : 0;
    }
    int upto = mine;  // inclusive scan: waves, then across them
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        const int v = __shfl_up(upto, m);
        upto += lane >= m ? v : 0;
    }
    if (lane == 63) scan[wave] = upto;
    __syncthreads();
    int before = upto - mine, total_head = 0;
#pragma unroll
    for (int w = 0; w < NR * NK; ++w) {
        const int v = __builtin_amdgcn_readfirstlane(scan[w]);
        if (w < wave) before += v;
        total_head += v;
    }
    const uint32_t total = (uint32_t)total_head * (uint32_t)a.kv.n_kv;
    const uint32_t per = max(1u, (total + W - 1) / W);
    if (wg == 0 && tid == 0) *reinterpret_cast<uint32_t *>(a.ws + ph.per) = per;
    uint32_t unit = scalar(per * (uint32_t)wg);
    const uint32_t end = scalar(min(unit + per, total));
    if (unit >= end) return;
    int head = scalar(unit / (uint32_t)total_head);
    {
        const int rem = (int)(unit - (uint32_t)head * (uint32_t)total_head);
        for (int j = 0; j < chunk; ++j) {
            const int i = tid * chunk + j;
            const int t = chunk == 1 ? t_last : attn_item<PREFIX, BM, BN>(a, ph, min(i, ph.items - 1)).tiles;
            if (i < ph.items && rem >= before && rem < before + t) {  // one lane of the workgroup, once
                scan[THREADS] = i;
                scan[THREADS + 1] = rem - before;
            }
            before += t;
        }
        __syncthreads();
    }
    int item = scalar(scan[THREADS]), off = scalar(scan[THREADS + 1]);

    while (unit < end) {
        Item it = attn_item<PREFIX, BM, BN>(a, ph, item);
        it.entry = scalar(it.entry);
        it.row0 = scalar(it.row0);
        it.rows = scalar(it.rows);
        it.ctx = scalar(it.ctx);
        it.limit = scalar(it.limit);
        it.tiles = scalar(it.tiles);
        const int kt0 = off, kt1 = max(kt0, min(it.tiles, off + (int)(end - unit)));
        if (it.tiles > 0) {
            if (kt0 == 0 && tid == 0)
                reinterpret_cast<uint32_t *>(a.ws + ph.first)[head * ph.items + item] = unit;
            const int *table = PREFIX ? a.prefix_pages : a.b.table + (int64_t)it.entry * a.b.max_pages;

            // ---- staging.  A tile's rows are read one tile ahead
            // (bf16: into the other LDS buffer; 8 bits: into registers).  A wave's rows of one pass lie
            // in one aligned run of at most 16, so on one page: its address is uniform but for the
            // lane's fixed offset.  Every load is made: a page that is not in the pool becomes page 0, rows
            // past the limit come from the page that holds its last one, and no query row sees either.
            u32x4_t kreg[DMA ? 1 : NCH], vreg[DMA ? 1 : NCH];
            uint32_t gone = 0, gone_next = 0;  // bit i: rows 16 i .. of the tile (of the next one) have no page in the pool
            float sreg = 0.0f;
            const int in_page = (1 << a.kv.shift) - 1;
            // Table entries p0 .. p0 + 63 of the item's run of pages, one per lane: a page is then a lane
            // read away (a load per tile would be waited for, 1.2k - 3.8k clocks of a tile's ~6k).
            const int last_page = (it.limit - 1) >> a.kv.shift;
            int p0 = (kt0 * BN) >> a.kv.shift, pages = table[min(p0 + lane, last_page)];
            uint64_t absent = __ballot((uint32_t)pages >= (uint32_t)a.kv.n_pages);  // lanes whose page is not in the pool
            const auto page_of_run = [&](int pos) {
                return __builtin_amdgcn_readlane(pages, (min(pos, it.limit - 1) >> a.kv.shift) - p0);
            };
            const auto pass_row = [&](int i) { return (64 * wave + THREADS * i) / CPR; };
            const int srow = tid % BN;  // 8 bits: thread's row of the k (tid < BN) or v scales
            const auto row_of = [&](int page, int pos) {
                return (((int64_t)page * a.kv.n_kv + head) << a.kv.shift) + (pos & in_page);
            };
            const auto issue = [&](int kt, int buf) {
                const int end_page = min(kt * BN + BN - 1, it.limit - 1) >> a.kv.shift;
                if (end_page >= p0 + 64) {
                    p0 = (kt * BN) >> a.kv.shift;
                    pages = table[min(p0 + lane, last_page)];
                    absent = __ballot((uint32_t)pages >= (uint32_t)a.kv.n_pages);
                }
                // pass i's rows start `at` bytes into k and v
                const auto load = [&](int i, int64_t at) {
                    if constexpr (DMA) {
                        // LDS is written linearly: the swizzle is in the chunk each lane fetches
                        const int r = pass_row(i) + lane / CPR, c = lane % CPR;
                        unsigned char *to = lds + buf * TL::buf_bytes + pass_row(i) * TL::ROWB;
                        const int64_t from = at + (lane / CPR) * TL::ROWB;
                        lds_dma16(a.kv.k + from + 16 * (c ^ (r & TL::SWZ)), to + 16 * lane);
                        lds_dma16(a.kv.v + from + 16 * (c ^ (2 * (r & TL::VSWZ))), to + BN * TL::ROWB + 16 * lane);
                    } else {
                        kreg[i] = *reinterpret_cast<const u32x4_t *>(a.kv.k + at + 16 * lane);
                        vreg[i] = *reinterpret_cast<const u32x4_t *>(a.kv.v + at + 16 * lane);
                    }
                };
                if ((1 << a.kv.shift) >= BN) {
                    // the whole tile on one page: one address
                    const int pg = page_of_run(kt * BN);
                    const bool in_pool = (uint32_t)pg < (uint32_t)a.kv.n_pages;
                    gone_next = in_pool ? 0 : 0xffffffffu;
                    const int64_t at = row_of(in_pool ? pg : 0, kt * BN) * (D * TL::ES);
#pragma unroll
                    for (int i = 0; i < NCH; ++i) load(i, at + pass_row(i) * (D * TL::ES));
                } else {
                    gone_next = 0;
#pragma unroll
                    for (int i = 0; i < BN / 16; ++i)
                        gone_next |= (uint32_t)((absent >> ((min(kt * BN + 16 * i, it.limit - 1) >> a.kv.shift) - p0)) & 1) << i;
#pragma unroll
                    for (int i = 0; i < NCH; ++i) {
                        const int pg = page_of_run(kt * BN + pass_row(i));
                        const bool in_pool = (uint32_t)pg < (uint32_t)a.kv.n_pages;
                        load(i, row_of(in_pool ? pg : 0, kt * BN + pass_row(i)) * (D * TL::ES));
                    }
                }
                if constexpr (!DMA) {
                    int pg;
                    if ((1 << a.kv.shift) >= BN)
                        pg = page_of_run(kt * BN);
                    else
                        pg = __shfl(pages, (min(kt * BN + srow, it.limit - 1) >> a.kv.shift) - p0);  // in all lanes
                    const bool in_pool = (uint32_t)pg < (uint32_t)a.kv.n_pages;
                    if (tid < 2 * BN) {
                        sreg = (tid < BN ? a.kv.ks : a.kv.vs)[row_of(in_pool ? pg : 0, kt * BN + srow)];
                        sreg = in_pool ? sreg : 0.0f;
                    }
                }
            };
            // 8 bits: registers to LDS.  tail: the tile holds keys from ctx on, which some row may not see.
            // What is not finite in their v must not meet a zero weight: it becomes 0 here, and the
            // item's end adds it for the rows that do see it.
            const auto put = [&](int kt, int buf, bool tail) {
                unsigned char *kl = lds + buf * TL::buf_bytes, *vl = kl + BN * TL::ROWB;
                if (gone) {
#pragma unroll
                    for (int i = 0; i < NCH; ++i)
                        if ((gone >> (pass_row(i) >> 4)) & 1) vreg[DMA ? 0 : i] = u32x4_t{0, 0, 0, 0};
                }
                if (FMT == kKvE4m3 && tail) {
#pragma unroll
                    for (int i = 0; i < NCH; ++i)
                        if (kt * BN + pass_row(i) + lane / CPR >= it.ctx && strip<FMT>(vreg[DMA ? 0 : i])) *bad = 1;
                }
#pragma unroll
                for (int i = 0; i < NCH; ++i) {
                    const int row = pass_row(i) + lane / CPR, c = lane % CPR;
                    const int zk = row & TL::SWZ, zv = 2 * (row & TL::VSWZ);
                    const u32x4_t k = kreg[DMA ? 0 : i], v = vreg[DMA ? 0 : i];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int at = row * TL::ROWB, cc = 2 * c + e;
                        *reinterpret_cast<u32x4_t *>(kl + at + 16 * (cc ^ zk)) = widen_k<FMT>(k[2 * e], k[2 * e + 1]);
                        *reinterpret_cast<u32x4_t *>(vl + at + 16 * (cc ^ zv)) = widen_v<FMT>(v[2 * e], v[2 * e + 1]);
                    }
                }
                if (tid < 2 * BN) {
                    float *sc = reinterpret_cast<float *>(lds + TL::o_sc + buf * TL::sc_bytes);
                    if (tid < BN) {
                        sc[srow] = sreg * a.scale;
                    } else {
                        if (tail && kt * BN + srow >= it.ctx && !(__builtin_fabsf(sreg) < __builtin_inff())) {
                            sreg = 0.0f;
                            *bad = 1;
                        }
                        // 2^-64 at least: 1 / vs and the sums of w / vs stay finite (a NaN stays one), and a row of
                        // zeros (scale 0) adds its weight to the sum without lifting the maximum of s + log2 vs
                        const float vs = sreg < 0x1p-64f ? 0x1p-64f : sreg;
                        sc[BN + srow] = __builtin_amdgcn_logf(vs);  // base 2
                        sc[2 * BN + srow] = 1.0f / vs;
                    }
                }
            };
            // bf16: the same for a tile that lies in LDS already; between two barriers.
            const auto strip_tile = [&](int kt, int buf) {
                unsigned char *vl = lds + buf * TL::buf_bytes + BN * TL::ROWB;
#pragma unroll 1
                for (int x = tid; x < BN * CPR; x += THREADS) {
                    const int row = x / CPR;
                    if (kt * BN + row < it.ctx && !((gone >> (row >> 4)) & 1)) continue;
                    u32x4_t *at = reinterpret_cast<u32x4_t *>(vl + 16 * x);
                    u32x4_t v = *at;
                    if (!strip<FMT>(v)) continue;
                    *at = v;
                    *bad = 1;
                }
            };

            // ---- the tile's query rows: B operand, lane li holds row li of each 16-row block
            bf16x8_t qf[RT][D / 32];
            int tok[RT];  // token of the row within its entry; -1 past the last row
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const int r = it.row0 + 16 * (RT * wr + rt) + li;
                tok[rt] = -1;
#pragma unroll
                for (int ks = 0; ks < D / 32; ++ks) qf[rt][ks] = bf16x8_t{};
                if (r < it.rows) {
                    const int t = r / a.grp, g = r - t * a.grp;
                    tok[rt] = t;
                    int64_t row = PREFIX ? t : (int64_t)it.entry * a.b.n_tok + t;
                    if (PREFIX && a.b.n_new) row = reinterpret_cast<const int *>(a.ws + a.plan.live)[1 + t];
                    const __bf16 *q = static_cast<const __bf16 *>(a.q.p) + row * a.q.ld + (int64_t)(head * a.grp + g) * a.q.hd;
#pragma unroll
                    for (int ks = 0; ks < D / 32; ++ks)
                        qf[rt][ks] = *reinterpret_cast<const bf16x8_t *>(q + 32 * ks + 8 * lg);
                }
            }
            f4 o[RT][D / 16];
            float m[RT], l[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                m[rt] = kNegInf;
                l[rt] = 0.0f;
#pragma unroll
                for (int cb = 0; cb < D / 16; ++cb) o[rt][cb] = f4{0.f, 0.f, 0.f, 0.f};
            }

            // A row sees the positions below seen[rt]: the context and, in a chain, itself and what was
            // drafted before it; the rest of a tree's row is in its ancestor words.
            int seen[RT];
            const uint32_t *anc[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                seen[rt] = PREFIX ? it.limit : min(it.limit, it.ctx + (a.parent ? 0 : tok[rt] + 1));
                anc[rt] = reinterpret_cast<const uint32_t *>(a.ws + a.plan.anc) +
                          ((int64_t)it.entry * a.b.n_tok + max(tok[rt], 0)) * a.plan.words;
            }
            const auto in_tree = [&](const uint32_t *words, int pos) {  // ctx <= pos < limit
                const int rel = pos - it.ctx;
                return ((words[rel >> 5] >> (rel & 31)) & 1) != 0;
            };
            const auto compute = [&](int kt, int buf, bool masked) {
                const unsigned char *kl = lds + buf * TL::buf_bytes, *vl = kl + BN * TL::ROWB;
                const float *sc = reinterpret_cast<const float *>(lds + TL::o_sc + buf * TL::sc_bytes);
                f4 s[RT][KB];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) s[rt][kb] = f4{0.f, 0.f, 0.f, 0.f};
                // the depth outermost: consecutive products go to different sums
#pragma unroll
                for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        // row 16 kb + li of the wave's keys: its swizzle is li's alone
                        const bf16x8_t kf = *reinterpret_cast<const bf16x8_t *>(
                            kl + (wk * KW + 16 * kb + li) * TL::ROWB + (((4 * ks + lg) ^ (li & TL::SWZ)) * 16));
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) s[rt][kb] = mfma_kq(kf, qf[rt][ks], s[rt][kb]);
                    }
                float top[RT];
                const auto maxima = [&](int kb) {
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        if (kb == 0) top[rt] = fmaxf(s[rt][0][0], s[rt][0][1]);
                        if (kb > 0) top[rt] = fmaxf(fmaxf(top[rt], s[rt][kb][0]), s[rt][kb][1]);
                        top[rt] = fmaxf(fmaxf(top[rt], s[rt][kb][2]), s[rt][kb][3]);
                    }
                };
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    const int k0 = wk * KW + 16 * kb + 4 * lg;  // the lane's four keys of the block
                    if constexpr (!DMA) {  // bf16: the scale is applied on the way into the exponent
                        const f4 c = *reinterpret_cast<const f4 *>(sc + k0), lv = *reinterpret_cast<const f4 *>(sc + BN + k0);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) s[rt][kb][i] = __builtin_fmaf(s[rt][kb][i], c[i], lv[i]);
                    }
                    maxima(kb);
                }
                if (masked) {
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb) {
                        const bool here = !((gone >> ((wk * KW >> 4) + kb)) & 1);
                        const int p0 = kt * BN + wk * KW + 16 * kb + 4 * lg;
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                bool on = p0 + i < seen[rt];
                                if (!PREFIX && a.parent && !on && p0 + i < it.limit) on = in_tree(anc[rt], p0 + i);
                                s[rt][kb][i] = on && here ? s[rt][kb][i] : kNegInf;
                            }
                        maxima(kb);
                    }
                }
                // The maximum is let grow by kSlack before it is taken over and the sums are rescaled (64 to 128
                // multiplications): any stand-in serves that keeps the weights in range.  With scores in no
                // order the true one grows in every second tile of a hundred for some row of a wave's 32 (8.1k
                // shared keys as above 158 -> 150 us, trees 79 -> 75 us).
                bool grew = false;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    if constexpr (DMA) top[rt] *= a.scale;
                    grew |= top[rt] - m[rt] > kSlack + LIFT;  // from -inf as well
                }
                if (__any(grew)) {
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const float mn = fmaxf(m[rt], quad_max(top[rt]) - LIFT), f = exp2_f(m[rt] - finite_max(mn));
                        m[rt] = mn;
                        l[rt] *= f;
#pragma unroll
                        for (int cb = 0; cb < D / 16; ++cb)
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[rt][cb][i] *= f;
                    }
                }
                P8 pf[RT][KB / 2], pl[TWO ? RT : 1][TWO ? KB / 2 : 1];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    f4 iv = f4{1.f, 1.f, 1.f, 1.f};
                    if constexpr (!DMA) iv = *reinterpret_cast<const f4 *>(sc + 2 * BN + wk * KW + 16 * kb + 4 * lg);
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt) {
                        const float mf = finite_max(m[rt]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float w = exp2_f(DMA ? __builtin_fmaf(s[rt][kb][i], a.scale, -mf) : s[rt][kb][i] - mf);
                            if constexpr (DMA)
                                l[rt] += w;
                            else
                                l[rt] = __builtin_fmaf(w, iv[i], l[rt]);
                            if constexpr (TWO) {
                                const float hi = bf16_below(w);
                                pf[rt][kb / 2][4 * (kb % 2) + i] = __builtin_bit_cast(__bf16, (uint16_t)(__float_as_uint(hi) >> 16));
                                pl[rt][kb / 2][4 * (kb % 2) + i] = (__bf16)(w - hi);
                            } else {
                                pf[rt][kb / 2][4 * (kb % 2) + i] = w;
                            }
                        }
                    }
                }
#pragma unroll
                for (int kp = 0; kp < KB / 2; ++kp) {
                    const int r = 4 * lg + (li >> 2), z = 2 * (r & TL::VSWZ);  // row 32 kp + r, then 16 rows on
                    const unsigned char *base = vl + (wk * KW + 32 * kp + r) * TL::ROWB + (li & 1) * 8;
#pragma unroll
                    for (int cb = 0; cb < D / 16; ++cb) {
                        const int c = ((2 * cb + ((li & 3) >> 1)) ^ z) * 16;
                        const P8 vf = __builtin_bit_cast(P8, u64x2_t{lds_tr4(base + c), lds_tr4(base + c + 16 * TL::ROWB)});
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            o[rt][cb] = mfma_vp(vf, pf[rt][kp], o[rt][cb]);
                            if constexpr (TWO) o[rt][cb] = mfma_vp(vf, pl[rt][kp], o[rt][cb]);
                        }
                    }
                }
            };

            // A barrier lies between this and the first store of 1: with one buffer or a bf16 cache the loop's
            // first one, else the one here, under which the first tile's loads are on their way.
            if (tid == 0) *bad = 0;
            issue(kt0, 0);
            if constexpr (!DMA && NB > 1) __syncthreads();
#pragma unroll 1
            for (int kt = kt0; kt < kt1; ++kt) {
                const int buf = NB > 1 ? (kt - kt0) & 1 : 0;
                const bool tail = (kt + 1) * BN > it.ctx;  // keys that some row may not see
                // One barrier per tile with two buffers: what this tile's copy overwrites was last read two
                // tiles ago, before the barrier between.
                gone = gone_next;
                if constexpr (NB == 1) __syncthreads();
                if constexpr (!DMA) put(kt, buf, tail);
                if constexpr (DMA) __builtin_amdgcn_s_waitcnt(0x0F70);  // this wave's part of the tile is in LDS
                __syncthreads();
                if (kt + 1 < kt1) issue(kt + 1, buf ^ 1);
                const bool masked = tail || gone != 0;
                if (DMA && masked) {
                    strip_tile(kt, buf);
                    __syncthreads();
                }
                compute(kt, buf, masked);
            }

            // ---- join the key waves: the last one ends with the item's sums
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) l[rt] = quad_sum(l[rt]);
            if constexpr (NK > 1) {
                __syncthreads();  // tile reads done: its LDS is free
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    if (lg == 0) ml[wk * BM + 16 * (RT * wr + rt) + li] = m[rt];
                __syncthreads();
                float *ob = reinterpret_cast<float *>(lds);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const int r = 16 * (RT * wr + rt) + li;
                    float mn = kNegInf;
#pragma unroll
                    for (int w = 0; w < NK; ++w) mn = fmaxf(mn, ml[w * BM + r]);
                    const float f = exp2_f(m[rt] - finite_max(mn));
                    m[rt] = mn;
                    l[rt] *= f;
#pragma unroll
                    for (int cb = 0; cb < D / 16; ++cb)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[rt][cb][i] *= f;
                }
                __syncthreads();  // maxima read: ml now carries the sums
                for (int w = 0; w < NK; ++w) {
                    if (wk == w) {
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            const int r = 16 * (RT * wr + rt) + li;
                            if (w > 0) l[rt] += ml[r];
#pragma unroll
                            for (int cb = 0; cb < D / 16; ++cb) {
                                f4 *at = reinterpret_cast<f4 *>(ob + r * D + ((4 * cb + lg) ^ (r & 15)) * 4);
                                if (w > 0) o[rt][cb] += *at;
                                if (w + 1 < NK) *at = o[rt][cb];
                            }
                        }
                        if (w + 1 < NK)
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt)
                                if (lg == 0) ml[16 * (RT * wr + rt) + li] = l[rt];
                    }
                    __syncthreads();
                }
            }
            if (wk == NK - 1) {
                // What put() took out of v, for the rows that see it: infinities and NaNs add up to what
                // they are whatever their weight.
                if (__builtin_amdgcn_readfirstlane(*bad)) {
#pragma unroll 1
                    for (int pos = max(it.ctx, kt0 * BN); pos < min(it.limit, kt1 * BN); ++pos) {
                        const int page = scalar(table[pos >> a.kv.shift]);
                        if ((uint32_t)page >= (uint32_t)a.kv.n_pages) continue;
                        const int64_t at = row_of(page, pos);
                        const bool none = FMT != kKvBf16 && !(__builtin_fabsf(a.kv.vs[at]) < __builtin_inff());
#pragma unroll
                        for (int cb = 0; cb < D / 16; ++cb) {
                            const int64_t ch = at * D + 16 * cb + 4 * lg;
                            float x[4];
                            if constexpr (FMT == kKvBf16) {
                                load_row<4>(a.kv.v, ch, true, x);
                            } else {
                                const uint32_t w = *reinterpret_cast<const uint32_t *>(a.kv.v + ch);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    x[e] = none || (FMT == kKvE4m3 && ((w >> (8 * e)) & 0x7f) == 0x7f) ? __builtin_nanf("") : 0.0f;
                            }
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt) {
                                bool on = pos < seen[rt];
                                if (!PREFIX && a.parent && !on) on = in_tree(anc[rt], pos);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (on && !(__builtin_fabsf(x[e]) < __builtin_inff())) o[rt][cb][e] += x[e];
                            }
                        }
                    }
                }
                const bool final = !PREFIX && !a.prefix_pages && kt0 == 0 && kt1 == it.tiles;
                const int64_t slot = (int64_t)head * ph.items + item + wg;  // its own: item and wg never both go back
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    const int lr = 16 * (RT * wr + rt) + li, r = it.row0 + lr;
                    if (r >= it.rows) continue;
                    if (final) {
                        const int t = r / a.grp, g = r - t * a.grp;
                        const float inv = l[rt] == 0.0f ? 0.0f : 1.0f / l[rt];
                        __bf16 *out = static_cast<__bf16 *>(a.out.p) + ((int64_t)it.entry * a.b.n_tok + t) * a.out.ld +
                                      (int64_t)(head * a.grp + g) * a.out.hd;
#pragma unroll
                        for (int cb = 0; cb < D / 16; ++cb) {
                            bf16x4_t y;
#pragma unroll
                            for (int i = 0; i < 4; ++i) y[i] = (__bf16)(o[rt][cb][i] * inv);
                            *reinterpret_cast<bf16x4_t *>(out + 16 * cb + 4 * lg) = y;
                        }
                    } else {
                        float *po = reinterpret_cast<float *>(a.ws + ph.po) + (slot * BM + lr) * D;
#pragma unroll
                        for (int cb = 0; cb < D / 16; ++cb) *reinterpret_cast<f4 *>(po + 16 * cb + 4 * lg) = o[rt][cb];
                        if (lg == 0) reinterpret_cast<float2 *>(a.ws + ph.pml)[slot * BM + lr] = make_float2(m[rt], l[rt]);
                    }
                }
            }
            __syncthreads();  // LDS is free for the next item
        }
        unit += kt1 - kt0;
        off = 0;
        if (++item == ph.items) {
            item = 0;
            ++head;
        }
    }
}

// ---------------------------------------------------------------------------- before and after

// Bit j of node t's words: node t sees drafted node j, its ancestor or itself.  A block per entry, whose
// parents lie in LDS: a walk up is a chain of dependent reads.
__global__ __launch_bounds__(256) void attn_ancestors_kernel(AttnArgs a)
{
    __shared__ int up[1024];
    const int64_t first = (int64_t)blockIdx.x * a.b.n_tok;
    for (int t = threadIdx.x; t < a.b.n_tok; t += 256) {
        const int p = a.parent[first + t];
        up[t] = p >= 0 && p < t ? p : -1;
    }
    __syncthreads();
    for (int t = threadIdx.x; t < a.b.n_tok; t += 256) {
        uint32_t *w = reinterpret_cast<uint32_t *>(a.ws + a.plan.anc) + (first + t) * a.plan.words;
        int node = t;
        for (int word = a.plan.words - 1; word >= 0; --word) {
            uint32_t bits = 0;
            for (; node >= 32 * word; node = up[node]) bits |= 1u << (node & 31);  // a parent comes before its child
            w[word] = bits;
        }
    }
}

// The token rows that count, in order, and each one's place among them: live[0] is their number.
__global__ __launch_bounds__(1024) void attn_live_kernel(AttnArgs a)
{
    __shared__ int part[16];
    __shared__ int base;
    int *live = reinterpret_cast<int *>(a.ws + a.plan.live), *rank = reinterpret_cast<int *>(a.ws + a.plan.rank);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = a.b.n_batch * a.b.n_tok;
    if (tid == 0) base = 0;
    for (int i0 = 0; i0 < n; i0 += 1024) {
        const int i = i0 + tid, b = i / a.b.n_tok;
        const bool on = i < n && a.b.start[b] >= 0 && i - b * a.b.n_tok < kv_new(a.b, b);
        const uint64_t vote = __ballot(on);
        if (lane == 0) part[wave] = __popcll(vote);
        __syncthreads();
        int at = base;
        for (int w = 0; w < wave; ++w) at += part[w];
        at += __popcll(vote & ((1ull << lane) - 1));
        if (on) {
            live[1 + at] = i;
            rank[i] = at;
        }
        __syncthreads();
        if (tid == 1023) base = at + on;
    }
    __syncthreads();
    if (tid == 0) live[0] = base;
}

// The parts of one item: slots [slot, slot + n).
struct Parts {
    int64_t slot;
    int n, row;
};
__device__ __forceinline__ Parts attn_parts(const AttnPhase &ph, const Item &it, uint32_t per, uint32_t first, int item, int row,
                                            int head)
{
    const uint32_t w0 = first / per, w1 = (first + it.tiles - 1) / per;
    return Parts{(int64_t)head * ph.items + item + w0, it.tiles > 0 ? (int)(w1 - w0 + 1) : 0, row - it.row0};
}

// Rows of the result from their parts.  D / 4 threads take a row, four channels each; with SPLIT the
// block's groups of that many threads share one row (few rows can have many parts: long contexts),
// otherwise each has its own.  What a row has to look up (its lengths, its place in the prefix's rows,
// its items' first units) is read before any of it is used: one wait instead of a chain of them (37 -> 20 us
// beside the shared prefix of 8.1k; eight rows per wave that looked them up once were no faster, and slower
// by 25 us where a row has eight parts).
template <int D, bool SPLIT>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int rows)
{
    constexpr int LANES = D / 4, GROUPS = 256 / LANES;
    __shared__ f4 so[SPLIT ? GROUPS : 1][LANES];
    __shared__ float2 sml[SPLIT ? GROUPS : 1];
    const int c = threadIdx.x % LANES, group = threadIdx.x / LANES, sub = SPLIT ? group : 0;
    const int id = SPLIT ? (int)blockIdx.x : (int)blockIdx.x * GROUPS + group;  // row of the head: token row, query head of the group
    const int head = blockIdx.y, rr = min(id, rows - 1);
    const int tokrow = rr / a.grp, g = rr - tokrow * a.grp, b = tokrow / a.b.n_tok, t = tokrow - b * a.b.n_tok;
    const AttnPhase &sp = a.plan.suffix, &pp = a.plan.prefix;
    const int r = t * a.grp + g, item = b * sp.row_tiles + r / sp.bm;
    const uint32_t sfirst = reinterpret_cast<const uint32_t *>(a.ws + sp.first)[head * sp.items + item];
    const uint32_t sper = *reinterpret_cast<const uint32_t *>(a.ws + sp.per);
    const Item it = attn_item<false>(a, sp, item);
    const bool live = id < rows && a.b.start[b] >= 0 && t < kv_new(a.b, b);
    Parts own = attn_parts(sp, it, max(sper, 1u), sfirst, item, r, head), pre{0, 0, 0};
    if (a.prefix_pages) {
        const int at = a.b.n_new ? reinterpret_cast<const int *>(a.ws + a.plan.rank)[tokrow] : tokrow;
        const int pr = (live ? at : 0) * a.grp + g, pitem = pr / pp.bm;
        const uint32_t pfirst = reinterpret_cast<const uint32_t *>(a.ws + pp.first)[head * pp.items + pitem];
        const uint32_t pper = *reinterpret_cast<const uint32_t *>(a.ws + pp.per);
        pre = attn_parts(pp, attn_item<true>(a, pp, pitem), max(pper, 1u), pfirst, pitem, pr, head);
    }
    const bool work = live && (a.prefix_pages || own.n > 1);  // else written whole, or not at all
    const int n_pre = work ? pre.n : 0, n = work ? n_pre + own.n : 0;
    const float *spo = reinterpret_cast<const float *>(a.ws + sp.po), *ppo = reinterpret_cast<const float *>(a.ws + pp.po);
    const float2 *spml = reinterpret_cast<const float2 *>(a.ws + sp.pml), *ppml = reinterpret_cast<const float2 *>(a.ws + pp.pml);
    float m = kNegInf, l = 0.0f;
    f4 o = f4{0.f, 0.f, 0.f, 0.f};
    constexpr int U = 4;  // parts in flight
    for (int j0 = sub; j0 < n; j0 += (SPLIT ? GROUPS : 1) * U) {
        f4 x[U];
        float2 y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + (SPLIT ? GROUPS : 1) * u;
            x[u] = f4{0.f, 0.f, 0.f, 0.f};
            y[u] = make_float2(kNegInf, 0.0f);
            if (j >= n) continue;
            const bool p = j < n_pre;
            const int64_t at = p ? (pre.slot + j) * pp.bm + pre.row : (own.slot + j - n_pre) * sp.bm + own.row;
            y[u] = (p ? ppml : spml)[at];
            x[u] = *reinterpret_cast<const f4 *>((p ? ppo : spo) + at * D + 4 * c);
        }
        float mn = m;
#pragma unroll
        for (int u = 0; u < U; ++u) mn = fmaxf(mn, y[u].x);
        const float f = exp2_f(m - finite_max(mn));
        l *= f;
        o *= f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float w = exp2_f(y[u].x - finite_max(mn));
            l += w * y[u].y;
            o += w * x[u];
        }
        m = mn;
    }
    if constexpr (SPLIT) {
        so[group][c] = o;
        if (c == 0) sml[group] = make_float2(m, l);
        __syncthreads();
        float mn = kNegInf;
        for (int w = 0; w < GROUPS; ++w) mn = fmaxf(mn, sml[w].x);
        l = 0.0f;
        o = f4{0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < GROUPS; ++w) {
            const float f = exp2_f(sml[w].x - finite_max(mn));
            l += f * sml[w].y;
            o += f * so[w][c];
        }
    }
    if (work && sub == 0) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        bf16x4_t y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = (__bf16)(o[e] * inv);
        __bf16 *out = static_cast<__bf16 *>(a.out.p) + tokrow * a.out.ld + (int64_t)(head * a.grp + g) * a.out.hd + 4 * c;
        *reinterpret_cast<bf16x4_t *>(out) = y;
    }
}

// -------------------------------------------------------------------------------------- launches

// Tile shapes by the rows that share keys (attn_config): the smallest of 16, 32, 64, 128 and, at d 128, 256 rows
// that holds them.  32 entries of 1000 .. 4000 keys, 8 heads, us with that shape (with the next smaller, the next
// larger one):
//    rows             16             32             64              128              256
//    e4m3, d 128   50 (-, 53)   57 (69, 62)    69 (85, 90)    103 (111, 150)    169 (177, -)
//    bf16, d 128   75 (-, 76)   83 (111, 82)   92 (118, 93)   107 (132, 130)    151 (164, -)
//    bf16, d 256  149 (-, 146) 160 (272, 168) 181 (287, 185)  204 (332, -)
// Eight waves of 32 rows halve what 128-row tiles stage per row.  At d 256 a wave's registers hold 16 rows (32 in
// four waves of 512 registers: 32.7k shared keys 128 -> 180 us), and at d 64 a tile's 8-bit codes are less than
// 16 bytes per thread.  with_shape calls f with the shape's type.
static int attn_config(int64_t rows, int d) { return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : rows <= 128 || d != 128 ? 3 : 4; }
constexpr int kAttnBm[5] = {16, 32, 64, 128, 256};

template <int NR_, int NK_, int RT_, int BN_, int NB_>
struct Shape {
    static constexpr int NR = NR_, NK = NK_, RT = RT_, BN = BN_, NB = NB_;
};
template <int D, int FMT, class F>
static auto with_shape(int cfg, F f)
{
    constexpr bool bf16 = FMT == kKvBf16;
    switch (cfg) {
    case 0: return f(Shape<1, 2, 1, 64, bf16 ? 2 : 1>{});
    case 1: return f(Shape<2, 2, 1, 64, bf16 ? 2 : 1>{});
    case 2: return f(Shape<4, 1, 1, 64, bf16 ? 2 : 1>{});
    case 3: return f(Shape<D == 256 ? 8 : 4, 1, D == 256 ? 1 : 2, 64, 2>{});
    default: return f(Shape<D == 64 ? 4 : 8, 1, D == 256 ? 1 : 2, 64, 2>{});  // d 128 alone; else the type above
    }
}
template <int D, int FMT>
static void tile_sizes(int cfg, int &bn, int &per_cu)
{
    with_shape<D, FMT>(cfg, [&](auto s) {
        using S = decltype(s);
        bn = S::BN;
        per_cu = AttnTile<D, FMT, S::NR, S::NK, S::RT, S::BN, S::NB>::per_cu;
    });
}
template <int D>
static void tile_sizes_f(int format, int cfg, int &bn, int &per_cu)
{
    format == kKvBf16   ? tile_sizes<D, kKvBf16>(cfg, bn, per_cu)
    : format == kKvE4m3 ? tile_sizes<D, kKvE4m3>(cfg, bn, per_cu)
                        : tile_sizes<D, kKvI8>(cfg, bn, per_cu);
}

bool attn_plan(int d, int format, int page_size, int n_kv, int grp, int n_batch, int n_tok, int max_pages, bool prefix,
               int max_prefix_pages, AttnPlan &p)
{
    p = AttnPlan{};
    constexpr int kCus = 256;
    size_t at = 0;
    const auto room = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    bool fits = true;
    const auto phase = [&](AttnPhase &ph, int64_t rows, int entries, int64_t pages) {
        ph.cfg = attn_config(rows, d);
        ph.bm = kAttnBm[ph.cfg];
        int per_cu = 1;
        d == 64 ? tile_sizes_f<64>(format, ph.cfg, ph.bn, per_cu)
        : d == 128 ? tile_sizes_f<128>(format, ph.cfg, ph.bn, per_cu)
                   : tile_sizes_f<256>(format, ph.cfg, ph.bn, per_cu);
        const int64_t row_tiles = (rows + ph.bm - 1) / ph.bm, items = row_tiles * entries;
        const int64_t tiles = (pages * page_size + ph.bn - 1) / ph.bn;
        // The kernels count positions in 32 bits, up to a table's end and a call's tokens or a tile beyond it.
        if (rows * entries >= kMaxTokenRows || items * n_kv >= (int64_t)1 << 30 ||
            pages * page_size + std::max(n_tok, ph.bn) >= (int64_t)1 << 31 ||
            (double)items * n_kv * (double)tiles >= 2147483648.0) {
            fits = false;
            return;
        }
        ph.row_tiles = (int)row_tiles;
        ph.items = (int)items;
        ph.wgs = (int)std::min<int64_t>(kCus * per_cu, items * n_kv * tiles);
        const size_t slots = (size_t)(items * n_kv) + kCus * per_cu;
        ph.per = room(4);
        ph.first = room((size_t)(items * n_kv) * 4);
        ph.pml = room(slots * ph.bm * 8);
        ph.po = room(slots * ph.bm * d * 4);
    };
    phase(p.suffix, (int64_t)n_tok * grp, n_batch, max_pages);
    if (prefix && fits) {
        phase(p.prefix, (int64_t)n_batch * n_tok * grp, 1, max_prefix_pages);
        p.live = room(((size_t)n_batch * n_tok + 1) * 4);
        p.rank = room((size_t)n_batch * n_tok * 4);
    }
    p.words = (n_tok + 31) / 32;
    if (n_tok <= 1024) p.anc = room((size_t)n_batch * n_tok * p.words * 4);  // the longest tree
    p.bytes = at;
    return fits;
}

template <int D, int FMT, bool PREFIX>
static hipError_t launch_cfg(const AttnArgs &a, hipStream_t stream)
{
    const AttnPhase &ph = PREFIX ? a.plan.prefix : a.plan.suffix;
    return with_shape<D, FMT>(ph.cfg, [&](auto s) {
        using S = decltype(s);
        using TL = AttnTile<D, FMT, S::NR, S::NK, S::RT, S::BN, S::NB>;
        hipLaunchKernelGGL((attn_kernel<D, FMT, S::NR, S::NK, S::RT, S::BN, S::NB, PREFIX>), dim3(ph.wgs), dim3(TL::THREADS),
                           TL::lds, stream, a);
        return hipGetLastError();
    });
}

template <int D>
static hipError_t launch_join(const AttnArgs &a, hipStream_t stream)
{
    const int rows = a.b.n_batch * a.b.n_tok * a.grp, groups = 1024 / D;
    // Few rows can have many parts each: a block per row while that is at most four blocks per CU.
    if ((int64_t)rows * a.kv.n_kv <= 1024)
        hipLaunchKernelGGL((attn_join_kernel<D, true>), dim3((unsigned)rows, (unsigned)a.kv.n_kv), dim3(256), 0, stream, a, rows);
    else
        hipLaunchKernelGGL((attn_join_kernel<D, false>), dim3((unsigned)((rows + groups - 1) / groups), (unsigned)a.kv.n_kv), dim3(256),
                           0, stream, a, rows);
    return hipGetLastError();
}

template <int D>
static hipError_t launch_attn_d(const AttnArgs &a, hipStream_t stream)
{
    const auto tiles = [&](auto prefix) {
        constexpr bool P = decltype(prefix)::value;
        return a.kv.format == kKvBf16   ? launch_cfg<D, kKvBf16, P>(a, stream)
               : a.kv.format == kKvE4m3 ? launch_cfg<D, kKvE4m3, P>(a, stream)
                                        : launch_cfg<D, kKvI8, P>(a, stream);
    };
    if (a.parent) {
        hipLaunchKernelGGL(attn_ancestors_kernel, dim3((unsigned)a.b.n_batch), dim3(256), 0, stream, a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    if (a.prefix_pages) {
        if (a.b.n_new) {
            hipLaunchKernelGGL(attn_live_kernel, dim3(1), dim3(1024), 0, stream, a);
            if (hipError_t e = hipGetLastError()) return e;
        }
        if (hipError_t e = tiles(std::true_type{})) return e;
    }
    if (hipError_t e = tiles(std::false_type{})) return e;
    // where no item can have a second tile and there is no prefix, every row was written whole
    if (!a.prefix_pages && ((int64_t)a.b.max_pages << a.kv.shift) <= a.plan.suffix.bn) return hipSuccess;
    return launch_join<D>(a, stream);
}

hipError_t launch_attn(const AttnArgs &a, hipStream_t stream)
{
    return a.kv.d == 64 ? launch_attn_d<64>(a, stream) : a.kv.d == 128 ? launch_attn_d<128>(a, stream) : launch_attn_d<256>(a, stream);
}

}  // namespace gdn
