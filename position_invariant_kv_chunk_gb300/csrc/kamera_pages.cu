// kamera_pages.cu -- which pages of a long context a query needs.
//
// A page's keys lie in a box: per channel their minimum and maximum.  For one
// query head the largest q . k a key of the box can reach is
// sum_i max(q_i min_i, q_i max_i), which takes max_i where q_i > 0 and min_i
// where q_i < 0.  Summed over the G query heads of a KV head it is one dot
// product of length 2 d,
//     score = q+ . max + q- . min,   q+ = sum_g max(q_g, 0),  q- = sum_g min(q_g, 0)
// so a page costs 4 d bytes read and 2 d multiplies per KV head, whatever G is.
//
// The choice of pages is a whole-number result, and fp32 sums of 2 d terms in
// one order or another would flip it where two scores lie close.  So it is made
// in two steps:
//   - every page's score in fp32 on the tensor cores (m16n8k16: 16 pages by the
//     weights), read-bound.  The box is bf16 and exact; the weights q+, q- enter
//     as three bf16 parts in three columns of the B operand.  The sum of the
//     weights' magnitudes times the largest entry of the boxes bounds the sum of
//     the terms' magnitudes, and with it the score's error.
//   - the n-th largest of these scores, t, and the largest error bound, E, split
//     the pages into those surely in (above t + 2 E), surely out (below t - 2 E)
//     and a few between, which are scored again, exactly to about 2^-40 of their
//     terms: the weights as a 16-bit part, whose products with the box are exact
//     in fp32, and a remainder, the products added with the error of every
//     addition kept (the two-sum of Knuth, The Art of Computer Programming
//     vol. 2, 4.2.2).
// Scoring every page the second way took 127 us where the boxes (32 sequences x 4
// heads of up to 8192 pages, 0.47 GB) take 67 us to read: two-sums cost 100
// instructions a page and head.
#include <algorithm>
#include <cooperative_groups.h>
#include <cstdint>
#include <cstring>

#include "kamera_common.cuh"
#include "kamera_hostcheck.h"
#include "kamera_internal.h"
#include "kamera_ptx.cuh"
#include "kamera_warpmma.cuh"

namespace kamera {

namespace {

// ---------------------------------------------------------------- summaries --
struct SummaryParams {
    const __nv_bfloat16* k;
    __nv_bfloat16* out;
    const int32_t* ids;
    const int32_t* tokens;
    int64_t slot_stride, num_pages, items;   // items: 16-byte vectors over all pages of the call
    int32_t H, d, P, vecs;                   // vecs: 16-byte vectors of a row
    int32_t* err;
};

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b)
{
    asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return a;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return a;
}
// The same of the numbers alone: a NaN gives way to the other operand.
__device__ __forceinline__ uint32_t min_num_bf16x2(uint32_t a, uint32_t b)
{
    asm("min.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return a;
}
__device__ __forceinline__ uint32_t max_num_bf16x2(uint32_t a, uint32_t b)
{
    asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return a;
}

// A thread takes one 16-byte vector of a page's rows, 16 tokens in flight at a
// time (a warp reads 512 contiguous bytes of each).  Read-bound: each key once,
// min and max exact in bf16, no exchange between threads.  8192 pages of 16 tokens
// of four heads of 128 (151 MB): 27 us, 5.6 TB/s; CTAs that stay for several pages
// took 34.
__global__ void __launch_bounds__(128) summary_kernel(const SummaryParams p)
{
    const int64_t item = (int64_t)blockIdx.x * 128 + threadIdx.x;
    ptx::grid_wait();
    ptx::grid_launch_next();
    if (item >= p.items)
        return;
    const int64_t e = item / p.vecs;
    const int vec = (int)(item - e * p.vecs);
    const int64_t page = p.ids[e];
    const int c = p.tokens[e];
    int32_t bits = 0;
    if (page < 0 || page >= p.num_pages)
        bits |= KAMERA_DEVERR_SLOT;
    if (c < 0 || c > p.P)
        bits |= KAMERA_DEVERR_LEN;
    if (bits && vec == 0)
        raise_err(p.err, bits);
    if (bits || c == 0)
        return;
    const __nv_bfloat16* src = p.k + page * p.P * p.slot_stride + 8 * vec;
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo[i] = 0x7F807F80u;   // +infinity
        hi[i] = 0xFF80FF80u;   // -infinity
    }
    for (int t0 = 0; t0 < c; t0 += 16, src += 16 * p.slot_stride) {
        uint4 v[16];
#pragma unroll
        for (int t = 0; t < 16; ++t)   // past the count: the first token again
            v[t] = *reinterpret_cast<const uint4*>(src + (t0 + t < c ? t : 0) * p.slot_stride);
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            const uint32_t w[4] = {v[t].x, v[t].y, v[t].z, v[t].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] = min_bf16x2(lo[i], w[i]);
                hi[i] = max_bf16x2(hi[i], w[i]);
            }
        }
    }
    const int vh = p.d / 8, h = vec / vh;
    __nv_bfloat16* o = p.out + (page * p.H + h) * 2 * p.d + 8 * (vec - h * vh);
    *reinterpret_cast<uint4*>(o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(o + p.d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
}

// ------------------------------------------------------------------- scores --
struct SelectParams {
    const __nv_bfloat16* q;
    const __nv_bfloat16* summary;
    const int32_t* pages;
    const int32_t* lens;
    int32_t* selected;
    uint64_t* keys;              // [n_seqs * H][width]: (score, error bound) as float2, then refined keys
    int64_t num_pages;
    int32_t n_seqs, H, G, P;
    int32_t max_pages, max_len, width;
    int32_t k, n_first, n_last;
    int32_t sweeps;              // score kernel: batches of a warp
    int32_t scored;              // the score kernel runs before the choice
    int32_t* err;
};

// Pages of sequence s; the scored ones are [lo, hi) (none when every page is taken).
__device__ __forceinline__ int page_range(const SelectParams& p, int s, int& lo, int& hi)
{
    const int len = p.lens[s];
    const int n = len > 0 && len <= p.max_len ? (len - 1) / p.P + 1 : 0;
    lo = p.n_first;
    hi = n > p.k ? n - p.n_last : lo;
    return n;
}

__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e)
{
    s = __fadd_rn(a, b);
    const float z = __fadd_rn(s, -a);
    e = __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -z)), __fadd_rn(b, -z));
}

// (s, e) += (s2, e2)
__device__ __forceinline__ void pair_add(float& s, float& e, float s2, float e2)
{
    float t, r;
    two_sum(s, s2, t, r);
    s = t;
    e = __fadd_rn(__fadd_rn(e, e2), r);
}

// Larger float, larger word.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t u = __float_as_uint(__fadd_rn(x, 0.f));   // -0 -> +0
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// q- (i < D) or q+ of channel i mod D as a pair of floats; q: the G query rows.
template <int D>
__device__ __forceinline__ void signed_sum(const __nv_bfloat16* q, int G, int i, float& a, float& e)
{
    const int ch = i < D ? i : i - D;
    a = e = 0.f;
#pragma unroll 4
    for (int g = 0; g < G; ++g) {
        const float x = __bfloat162float(q[g * D + ch]);
        pair_add(a, e, i < D ? fminf(x, 0.f) : fmaxf(x, 0.f), 0.f);
        if (x != x)
            a = x;   // fminf and fmaxf drop a NaN
    }
}

// Six warps with two batches each: two CTAs an SM, whose start (weights, table) the
// other covers.  Of 32 x 4 x 8192 pages, with the attention: 114.4 us; three CTAs of
// four warps 117.2; one of thirteen 115.9; two of four warps with three batches 119.0.
constexpr int kScoreWarps = 6;
constexpr int kScoreStages = 2;  // batches in a warp's ring
constexpr int kScorePages = 16;  // pages of a warp's MMA
// A score's error: 2 d / 16 MMAs, each a sum of 17 terms no better than truncated
// fp32, is at most 2 d / 16 x 17 x 2^-23 < 2^-14.9 of the sum of the terms'
// magnitudes (d = 128).
constexpr float kScoreErr = 3.4e-5f;

// Scores and error bounds of the pages of (sequence, KV head) rows.  Each warp
// keeps a ring of batches of 16 boxes, filled by 16-byte async copies (a box of d =
// 128 is 512 bytes, one copy of a warp), so copies stay in flight while it
// multiplies.  75 us, 6.3 TB/s, for 32 sequences x 4 heads of up to 8192 pages (0.47
// GB); with a bulk copy a box it took 86 us, as the copy engine takes about 28
// cycles for each.  The sum over channels may run in any order, so a lane feeds the A operand with whole
// 16-byte pieces: lane (page gq, t4) reads pieces t4 + 4 j of its page's box, and
// the B operand holds the weights of the same pieces.  Column gq of B: 0-2 the
// weights' bf16 parts.  (m16n8k16 takes about 32 cycles of a sub-partition here:
// 16 of them a batch leave room for the copies, 32 would not.)
template <int D, int WARPS>
struct ScoreLayout {
    static constexpr int NC = 2 * D / 32;                     // 16-byte pieces of a box that a lane reads
    static constexpr uint32_t kBox = 4 * D;                   // bytes
    static constexpr uint32_t kStage = kScorePages * kBox;    // piece c of row r at c ^ 4 (r & 1): no bank conflicts
    static constexpr uint32_t kBytes = WARPS * kScoreStages * kStage;
};

template <int D, int WARPS>
struct ScoreSmem {
    alignas(16) __nv_bfloat16 wt[3][2 * D];
    alignas(16) __nv_bfloat16 qs[16 * D];
    float norm[WARPS];
};

// A batch with an infinite bound among its boxes, which spoils the tensor cores' sums
// where its weight is zero (the bound on the side that no query asks for): each page
// by fp32 sums that leave such entries out, with the sum of its own terms' magnitudes
// for the error.  Lane r: page r's score and error bound; a score that is not finite
// has none, as it ranks first whatever its error.  A call, so that the loop around
// it keeps its registers.
template <int D, int WARPS>
__device__ __noinline__ float2 score_infinite(uint32_t stage, const ScoreSmem<D, WARPS>& sm)
{
    using Y = ScoreLayout<D, WARPS>;
    const int lane = threadIdx.x & 31;
    float2 mine = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int r = 0; r < kScorePages; ++r) {
        float v = 0.f, mag = 0.f;
        if (lane < D / 4) {   // a lane, a 16-byte piece
            uint32_t x[4];
            ptx::lds128(stage + r * Y::kBox + 16 * (lane ^ ((r & 1) << 2)), x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int ch = 8 * lane + i;
                const float w = __bfloat162float(sm.wt[0][ch]) +
                                (__bfloat162float(sm.wt[1][ch]) + __bfloat162float(sm.wt[2][ch]));
                const float y = i & 1 ? bf16hi(x[i >> 1]) : bf16lo(x[i >> 1]);
                if (!(w == 0.f && fabsf(y) == INFINITY)) {
                    v = fmaf(w, y, v);
                    mag = fmaf(fabsf(w), fabsf(y), mag);
                }
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o /= 2) {
            v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            mag += __shfl_xor_sync(0xFFFFFFFFu, mag, o);
        }
        if (lane == r)
            mine = fabsf(v) <= 3.402823466e38f ? make_float2(v, __fmul_ru(kScoreErr, mag)) : make_float2(INFINITY, 0.f);
    }
    return mine;
}

// The CTA's share (`part`) of the pages of one (sequence, KV head): put(j, score and
// error bound) for page j of the sequence, weight(i, a, e) for each of the weights
// q- | q+ (the sum a + e), by one thread each; ready() before the first put.
template <int D, int WARPS, typename Put, typename Weight, typename Ready>
__device__ __forceinline__ void score_pages(const SelectParams& p, int s, int h, int part, unsigned char* ring_raw,
                                            ScoreSmem<D, WARPS>& sm, Put put, Weight weight, Ready ready)
{
    using Y = ScoreLayout<D, WARPS>;
    constexpr int NC = Y::NC, NS = kScoreStages;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, t4 = lane & 3;
    // The queries, the first entries of the page table and the sequence's length at
    // once: one after another they took longer than a batch.
    const __nv_bfloat16* q = p.q + ((int64_t)s * p.H + h) * p.G * D;
    for (int i = threadIdx.x; i < p.G * (D / 8); i += 32 * WARPS)
        ptx::cp_async16(ptx::smem_addr(sm.qs + 8 * i), q + 8 * i);
    ptx::cp_async_commit();
    constexpr int step = WARPS * kScorePages;
    // the warp's batches: pages first + step k .. + 15
    const int chunk = step * p.sweeps, c0 = p.n_first + part * chunk, first = c0 + warp * kScorePages;
    const int32_t* table = p.pages + (int64_t)s * p.max_pages;
    int start[NS];
#pragma unroll
    for (int k = 0; k < NS; ++k) {
        const int j = first + k * step + lane;
        start[k] = lane < kScorePages && j < p.max_pages ? table[j] : -1;
    }
    int lo, hi;
    page_range(p, s, lo, hi);
    const int c1 = min(c0 + chunk, hi);
    if (c0 >= hi) {
        ptx::cp_async_wait<0>();
        return;
    }
    const int count = first < c1 ? (c1 - first + step - 1) / step : 0;
    const uint32_t ring = ptx::smem_addr(ring_raw) + warp * NS * Y::kStage;
    auto entry = [&](int k) {   // this lane's page of batch k as the table has it; -1 past the range
        const int j = first + k * step + lane;
        return k < count && lane < kScorePages && j < c1 ? table[j] : -1;
    };
#pragma unroll
    for (int k = 0; k < NS; ++k)
        if (first + k * step + lane >= c1)
            start[k] = -1;
    uint32_t known_of[NS];   // the pages of a stage inside the pool
#pragma unroll
    for (int b = 0; b < NS; ++b)
        known_of[b] = 0;
    constexpr int LB = Y::kBox / 16, PI = 32 / LB;   // lanes of a box, boxes of one copy of the warp
    const __nv_bfloat16* src = p.summary + (int64_t)h * (2 * D) + 8 * (lane % LB);
    const uint32_t row_bytes = (uint32_t)p.H * Y::kBox;
    // A row without a page repeats one of the batch's boxes, which changes nothing.
    auto load = [&](int k, int page, uint32_t& known_b) {   // one group of copies a batch, empty past the last
        const bool in = k < count && lane < kScorePages && first + k * step + lane < c1;
        const bool good = in && page >= 0 && page < p.num_pages;
        if (in && !good && h == 0)
            raise_err(p.err, KAMERA_DEVERR_SLOT);
        known_b = __ballot_sync(0xFFFFFFFFu, good);
        if (known_b) {
            const int some = __shfl_sync(0xFFFFFFFFu, page, __ffs((int)known_b) - 1);
            const uint32_t safe = (uint32_t)(good ? page : some);
            // rows alternate in parity (one box a copy) or share it by halves of the warp (two)
            const uint32_t dst = ring + (k % NS) * Y::kStage + (lane / LB) * Y::kBox;
            const uint32_t even = dst + 16 * ((lane % LB) ^ (PI == 2 ? (lane / LB) << 2 : 0));
            const uint32_t odd = dst + 16 * ((lane % LB) ^ 4);
#pragma unroll
            for (int i = 0; i < kScorePages / PI; ++i) {
                const uint32_t from = __shfl_sync(0xFFFFFFFFu, safe, i * PI + lane / LB);
                ptx::cp_async16((PI == 1 && (i & 1) ? odd : even) + i * PI * Y::kBox,
                                reinterpret_cast<const unsigned char*>(src) + (uint64_t)from * row_bytes);
            }
        }
        ptx::cp_async_commit();
    };
    int ahead = start[NS - 1];
#pragma unroll
    for (int k = 0; k < NS - 1; ++k)
        load(k, start[k], known_of[k]);
    ptx::cp_async_wait<NS - 1>();   // the queries
    __syncthreads();

    float norm = 0.f;   // the sum of the weights' magnitudes, rounded up
    for (int i = threadIdx.x; i < 2 * D; i += 32 * WARPS) {
        float a, e;
        signed_sum<D>(sm.qs, p.G, i, a, e);
        weight(i, a, e);
        a = __fadd_rn(a, e);
        norm = __fadd_ru(norm, fabsf(a));
        sm.wt[0][i] = __float2bfloat16_rn(a);
        a = __fadd_rn(a, -__bfloat162float(sm.wt[0][i]));
        sm.wt[1][i] = __float2bfloat16_rn(a);
        a = __fadd_rn(a, -__bfloat162float(sm.wt[1][i]));
        sm.wt[2][i] = __float2bfloat16_rn(a);
    }
#pragma unroll
    for (int o = 16; o >= 1; o /= 2)
        norm = __fadd_ru(norm, __shfl_xor_sync(0xFFFFFFFFu, norm, o));
    if (lane == 0)
        sm.norm[warp] = norm;
    __syncthreads();
    norm = 0.f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i)
        norm = __fadd_ru(norm, sm.norm[i]);
    uint4 w[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j)
        w[j] = gq < 3 ? *reinterpret_cast<const uint4*>(&sm.wt[gq < 3 ? gq : 0][8 * (t4 + 4 * j)])
                      : make_uint4(0u, 0u, 0u, 0u);
    ready();
    for (int k0 = 0; k0 < count; k0 += NS) {
#pragma unroll
        for (int u = 0; u < NS; ++u) {   // batch k in stage u
            const int k = k0 + u;
            if (k >= count)
                break;
            const int page = ahead;
            ahead = entry(k + NS);
            load(k + NS - 1, page, known_of[(u + NS - 1) % NS]);
            ptx::cp_async_wait<NS - 1>();   // batch k has landed, for this lane's copies and
            __syncwarp();                   // then for every lane's
            const uint32_t ra = ring + u * Y::kStage + gq * Y::kBox + 16 * t4, rb = ra + 8 * Y::kBox;
            const uint32_t odd = (uint32_t)(gq & 1) << 6;
            float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};   // two chains
            // the least and the largest entry of the batch's boxes: among the minima (the
            // first half of a box), among the maxima (every other entry lies between).  A NaN
            // makes its own page's score NaN, and does not bound the others'
            uint32_t least = 0u, most = 0u;
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                uint32_t a[4], b[4];
                ptx::lds128(ra + ((64 * j) ^ odd), a);
                ptx::lds128(rb + ((64 * j) ^ odd), b);
                const uint32_t f0[4] = {a[0], b[0], a[1], b[1]}, f1[4] = {a[2], b[2], a[3], b[3]};
                wmma16::mma_bf16(sc[0], f0, w[j].x, w[j].y);
                wmma16::mma_bf16(sc[1], f1, w[j].z, w[j].w);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (j < NC / 2)
                        least = min_num_bf16x2(least, min_num_bf16x2(a[i], b[i]));
                    else
                        most = max_num_bf16x2(most, max_num_bf16x2(a[i], b[i]));
            }
            most = max_num_bf16x2(most, least ^ 0x80008000u);
#pragma unroll
            for (int o = 16; o >= 1; o /= 2)
                most = max_num_bf16x2(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
            const float top = fmaxf(bf16lo(most), bf16hi(most));
            if (top == INFINITY) {   // (the warp) an infinite bound: the batch page by page
                const float2 x = score_infinite<D, WARPS>(ring + u * Y::kStage, sm);
                const int j = first + k * step + lane;
                if (lane < kScorePages && j < c1)
                    put(j, (known_of[u] >> lane) & 1u ? x : make_float2(0.f, -1.f));
                __syncwarp();
                continue;
            }
            const float e = __fmul_ru(kScoreErr, __fmul_ru(norm, top));
            // columns 0, 1 of pages gq, gq + 8 sit in lanes t4 = 0, column 2 in t4 = 1
            const float la = __shfl_down_sync(0xFFFFFFFFu, sc[0][0] + sc[1][0], 1);
            const float lb = __shfl_down_sync(0xFFFFFFFFu, sc[0][2] + sc[1][2], 1);
            if (t4 == 0) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int j = first + k * step + gq + 8 * r;
                    if (j < c1) {
                        const float v = (sc[0][2 * r] + sc[1][2 * r]) + ((sc[0][2 * r + 1] + sc[1][2 * r + 1]) + (r == 0 ? la : lb));
                        const bool finite = fabsf(v) <= 3.402823466e38f;   // else it ranks first
                        put(j, (known_of[u] >> (gq + 8 * r)) & 1u ? make_float2(finite ? v : INFINITY, e)
                                                                  : make_float2(0.f, -1.f));
                    }
                }
            }
            __syncwarp();   // the stage's rows are read before it is filled again
        }
    }
    ptx::cp_async_wait<0>();
}

template <int D>
__global__ void __launch_bounds__(32 * kScoreWarps) score_kernel(const SelectParams p)
{
    extern __shared__ __align__(16) unsigned char ring_raw[];
    __shared__ ScoreSmem<D, kScoreWarps> sm;
    ptx::grid_wait();
    ptx::grid_launch_next();
    const int s = blockIdx.y, part = blockIdx.x / p.H, h = blockIdx.x - part * p.H;   // a page's heads side by side
    float2* keys = reinterpret_cast<float2*>(p.keys + ((int64_t)s * p.H + h) * p.width);
    score_pages<D, kScoreWarps>(
        p, s, h, part, ring_raw, sm, [&](int j, float2 x) { keys[j] = x; }, [](int, float, float) {}, [] {});
}

// ------------------------------------------------------------------- choice --
constexpr int kBins = 2048;              // digits of 11 bits
constexpr int kGather = 1024;            // keys that are ranked by comparison
constexpr int kMaxWidth = 49152;         // pages of a sequence: 48 scores a thread, in registers

// NTH: threads of the CTA.
template <int D, int NTH>
struct SelSmem {
    static constexpr int kWarps = NTH / 32;
    uint32_t hist[kBins];
    uint64_t cand[kGather];
    int32_t cand_j[kGather];
    float qa[2 * D], qb[2 * D];          // q- | q+: the 16-bit part and the rest
    uint32_t warp_sum[kWarps], bin_sum[kWarps], counts[kWarps];
    uint64_t warp_min[kWarps], warp_max[kWarps];
    float lo[kWarps], hi[kWarps], err[kWarps];
    int32_t bin, above, n_cand, n_in, n_band;
};

// Least and largest of a warp's floats (no NaN among them).
__device__ __forceinline__ float warp_min(float x)
{
    float y;
    asm("redux.sync.min.f32 %0, %1, 0xFFFFFFFF;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float warp_max(float x)
{
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(y) : "f"(x));
    return y;
}

// Exclusive sum over the block of one value a thread; `total` for everybody.
// FRESH: nothing has used `warp_sum` before.
template <int NTH, bool FRESH = false>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sum, uint32_t& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o)
            x += y;
    }
    if (!FRESH)
        __syncthreads();
    if (lane == 31)
        warp_sum[warp] = x;
    __syncthreads();
    const uint32_t sum = lane < NTH / 32 ? warp_sum[lane] : 0u;
    total = __reduce_add_sync(0xFFFFFFFFu, sum);
    return __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sum : 0u) + x - v;
}

// The `need`-th largest key of a set (1 <= need <= its size), by radix steps of 11
// bits from the first bit in which the keys differ (kmin .. kmax over the set):
// on return the keys whose (>> shift) exceeds `prefix` are more than it, and
// `need` is what is left to take of those whose (>> shift) equals it; shift is 0,
// or `count` of them are at most kGather, or all of them are to be taken.
// each(f) calls f(key) for the thread's share of the set.
template <int NTH, typename SM, typename Each>
__device__ __forceinline__ void radix_find(SM& sm, uint64_t kmin, uint64_t kmax, Each each, int& need, int& shift,
                                           uint64_t& prefix, int& count)
{
    const int tid = threadIdx.x;
    constexpr int PT = kBins / NTH;
    const int top = 63 - __clzll((long long)(kmin ^ kmax));   // the highest bit that differs
    shift = max(0, top - 10);
    uint64_t fixed = top == 63 ? 0ull : kmin >> (top + 1);    // bits above the digit, shared so far
    int width = top + 1 - shift;                              // bits of the digit
    for (;;) {
        __syncthreads();
        for (int b = tid; b < kBins; b += NTH)
            sm.hist[b] = 0u;
        __syncthreads();
        const int up = shift + width;                         // 64: no bits above
        each([&](uint64_t key) {
            if ((up >= 64 ? 0ull : key >> up) == fixed)
                atomicAdd(&sm.hist[(key >> shift) & ((1u << width) - 1u)], 1u);
        });
        __syncthreads();
        // thread t's bins, from the top: kBins - 1 - PT t downwards
        uint32_t c[PT], mine = 0, total;
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            c[i] = sm.hist[kBins - 1 - PT * tid - i];
            mine += c[i];
        }
        uint32_t above = block_scan<NTH>(mine, sm.warp_sum, total);
#pragma unroll
        for (int i = 0; i < PT; ++i) {
            if ((int)above < need && need <= (int)(above + c[i])) {
                sm.bin = kBins - 1 - PT * tid - i;
                sm.above = (int)above;
            }
            above += c[i];
        }
        __syncthreads();
        count = (int)sm.hist[sm.bin];
        need -= sm.above;
        prefix = (fixed << width) | (uint64_t)sm.bin;         // width <= 11 < 64
        if (shift == 0 || count <= kGather || count == need)
            return;
        fixed = prefix;
        width = min(11, shift);
        shift -= width;
    }
}

// A lane's weights for the exact scores: 8 entries' 16-bit parts and remainders, and
// 0xFFFF for those that are zero.
template <int D>
struct ExactWeights {
    uint64_t a[4], b[4];
    uint32_t zero[4];
    __device__ __forceinline__ ExactWeights(const float* qa, const float* qb, int lane)
    {
        const bool on = lane < D / 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = on ? *reinterpret_cast<const uint64_t*>(qa + 8 * lane + 2 * i) : 0ull;
            b[i] = on ? *reinterpret_cast<const uint64_t*>(qb + 8 * lane + 2 * i) : 0ull;
            const uint64_t any = (a[i] | b[i]) & 0x7FFFFFFF7FFFFFFFull;
            zero[i] = ((uint32_t)any ? 0u : 0xFFFFu) | ((uint32_t)(any >> 32) ? 0u : 0xFFFF0000u);
        }
    }
};

// The exact score of a page (16 bytes of its box to a lane), as an ordered key.
// Infinite entries of zero weight count as 0.
template <int D>
__device__ __forceinline__ uint64_t exact_key(const SelectParams& p, int page, int h, const ExactWeights<D>& q, int lane)
{
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (lane < D / 4)
        v = reinterpret_cast<const uint4*>(p.summary + ((int64_t)page * p.H + h) * (2 * D))[lane];
    const uint64_t neg1 = ptx::f2_make(0xBF800000u, 0xBF800000u);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] &= ~(__vcmpeq2(w[i] & 0x7FFF7FFFu, 0x7F807F80u) & q.zero[i]);
    uint64_t x = ptx::f2_from_bf16x2(w[0]);
    uint64_t sum = ptx::f2_mul(q.a[0], x), err = ptx::f2_mul(q.b[0], x);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        x = ptx::f2_from_bf16x2(w[i]);
        const uint64_t pr = ptx::f2_mul(q.a[i], x);          // exact
        const uint64_t t = ptx::f2_add(sum, pr);
        const uint64_t z = ptx::f2_fma(sum, neg1, t);        // t - sum
        const uint64_t tz = ptx::f2_fma(z, neg1, t);         // t - z
        const uint64_t r = ptx::f2_add(ptx::f2_fma(tz, neg1, sum), ptx::f2_fma(z, neg1, pr));
        err = ptx::f2_add(ptx::f2_fma(q.b[i], x, err), r);
        sum = t;
    }
    uint32_t s0, s1, e0, e1;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(s0), "=r"(s1) : "l"(sum));
    asm("mov.b64 {%0, %1}, %2;" : "=r"(e0), "=r"(e1) : "l"(err));
    float S = __uint_as_float(s0), E = __uint_as_float(e0);
    pair_add(S, E, __uint_as_float(s1), __uint_as_float(e1));
#pragma unroll
    for (int dist = 16; dist >= 1; dist /= 2)
        pair_add(S, E, __shfl_xor_sync(0xFFFFFFFFu, S, dist), __shfl_xor_sync(0xFFFFFFFFu, E, dist));
    float t, r;
    two_sum(S, E, t, r);   // t + r, t the sum rounded: (t, r) orders as the sum does
    if (!(fabsf(t) <= 3.402823466e38f && r == r)) {
        t = INFINITY;
        r = 0.f;
    }
    return ((uint64_t)ordered(t) << 32) | ordered(r);
}

// What every thread does before the scores are needed: an empty histogram.
template <int D, int NTH>
__device__ __forceinline__ void clear_choice(SelSmem<D, NTH>& sm)
{
    for (int i = threadIdx.x; i < kBins; i += NTH)
        sm.hist[i] = 0u;
    if (threadIdx.x == 0)
        sm.n_cand = sm.n_in = sm.n_band = 0;
}

// The exact weights: a 16-bit part and the rest.
template <int D, int NTH>
__device__ __forceinline__ void keep_weight(SelSmem<D, NTH>& sm, int i, float a, float e)
{
    const float top = __uint_as_float(__float_as_uint(a) & 0xFFFFFF00u);
    sm.qa[i] = top;
    sm.qb[i] = __fadd_rn(__fadd_rn(a, -top), e);
}

// A sequence that has no more pages than are selected: all of them.
template <int NTH>
__device__ __forceinline__ void take_all(const SelectParams& p, int s, int h, int n)
{
    int32_t* out = p.selected + ((int64_t)s * p.H + h) * p.k;
    for (int i = threadIdx.x; i < p.k; i += NTH)
        out[i] = i < n ? i : -1;
}

// The choice for one (sequence, KV head) by one CTA: the pages surely in by their
// fp32 scores, the exact order of those near the border, and the pages in order from
// a bitmap.  All latency (a chain of barriers and dependent loads, and fetching code
// that a CTA runs once): 5 us for 2048 pages, 10 us for 8192.  So each thread keeps
// its NK scores in registers, and one histogram of them is enough: the border lies in
// the bin that holds the n-th largest score, and whatever is within the errors of that
// bin counts as near it.  keys64: the scores, overwritten; maps: two bitmaps.
template <int D, int NTH, int NK>
__device__ __forceinline__ void choose(const SelectParams& p, int s, int h, int n, int lo, int hi, uint64_t* keys64,
                                       uint32_t* maps, SelSmem<D, NTH>& sm)
{
    constexpr int NW = NTH / 32;
    const int words = (p.width + 31) >> 5, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t* bm = maps;              // pages taken
    uint32_t* band = maps + words;    // pages near the border
    int32_t* out = p.selected + ((int64_t)s * p.H + h) * p.k;
    const float2* scores = reinterpret_cast<const float2*>(keys64);
    int need = p.k - p.n_first - p.n_last;
    // ---- the scores, page i NTH + tid a thread: finite, +infinity (not finite: first),
    // NaN (no such page: last)
    float v[NK], smin = INFINITY, smax = -INFINITY, err = 0.f;
    int n_inf = 0, n_fin = 0;
    if (need > 0) {
        uint32_t count = 0;   // finite ones, and 2^16 times the others: a row has at most kMaxWidth < 2^16
#pragma unroll
        for (int i0 = 0; i0 < NK; i0 += 8) {
            float2 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = (i0 + i) * NTH + tid;
                x[i] = make_float2(0.f, -2.f);
                if (j >= lo && j < hi)
                    x[i] = scores[j];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool known = x[i].y >= 0.f || x[i].y != x[i].y;   // (a NaN bound comes of a NaN query)
                const bool fin = known && fabsf(x[i].x) <= 3.402823466e38f;
                v[i0 + i] = fin ? x[i].x : known ? INFINITY : __int_as_float(0x7FC00000);
                if (known)
                    err = fmaxf(err, x[i].y == x[i].y ? x[i].y : INFINITY);
                if (fin) {
                    smin = fminf(smin, x[i].x);
                    smax = fmaxf(smax, x[i].x);
                }
                count += fin ? 1u : known ? 0x10000u : 0u;
            }
        }
        smin = warp_min(smin);
        smax = warp_max(smax);
        err = warp_max(err);
        count = __reduce_add_sync(0xFFFFFFFFu, count);
        if (lane == 0) {
            sm.lo[warp] = smin;
            sm.hi[warp] = smax;
            sm.err[warp] = err;
            sm.counts[warp] = count;
        }
        __syncthreads();
        smin = warp_min(lane < NW ? sm.lo[lane] : INFINITY);
        smax = warp_max(lane < NW ? sm.hi[lane] : -INFINITY);
        err = warp_max(lane < NW ? sm.err[lane] : 0.f);
        count = __reduce_add_sync(0xFFFFFFFFu, lane < NW ? sm.counts[lane] : 0u);
        n_fin = (int)(count & 0xFFFFu);
        n_inf = (int)(count >> 16);
    }
    // ---- in: above `in_above`; near: from `near_from` on; ties: the near ones are equal
    enum { kInf, kFinite, kUnknown } border = kFinite;
    float in_above = INFINITY, near_from = INFINITY;
    if (need > 0) {
        if (need <= n_inf) {
            border = kInf;
        } else if (need - n_inf > n_fin) {
            border = kUnknown;
        } else {
            // bins of equal width between the least and the largest score.  The quotient is
            // good to 2^-20, so a score's bin is off by less than 2^-8 of a bin: the edges are
            // taken a whole bin wide of it
            const float range = __fadd_ru(smax, -smin);
            float inv = __fdividef((float)kBins, range);
            if (!(inv <= 3.402823466e38f))
                inv = 0.f;   // one value, or as good as one (or a range past 2^126): a single bin
#pragma unroll
            for (int i = 0; i < NK; ++i)
                if (fabsf(v[i]) <= 3.402823466e38f)
                    atomicAdd(&sm.hist[min(kBins - 1, (int)((v[i] - smin) * inv))], 1u);
            __syncthreads();
            // thread t's bins, from the top: kBins - 1 - PT t downwards
            constexpr int PT = kBins / NTH;
            const int want = need - n_inf;
            uint32_t c[PT], mine = 0, total;
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                c[i] = sm.hist[kBins - 1 - PT * tid - i];
                mine += c[i];
            }
            uint32_t above = block_scan<NTH, true>(mine, sm.bin_sum, total);
#pragma unroll
            for (int i = 0; i < PT; ++i) {
                if ((int)above < want && want <= (int)(above + c[i]))
                    sm.bin = kBins - 1 - PT * tid - i;
                above += c[i];
            }
            __syncthreads();
            const float b = (float)sm.bin, e2 = __fmul_ru(2.f, err);
            const float w = range * (1.f / (float)kBins);
            const float edge_hi = inv > 0.f ? __fadd_ru(smin, __fmul_ru(b + 2.f, w)) : smax;
            const float edge_lo = inv > 0.f ? __fadd_rd(smin, __fmul_rd(b - 1.f, w)) : smin;
            in_above = __fadd_ru(edge_hi, e2);
            near_from = __fadd_rd(edge_lo, -e2);
        }
    }
    // ---- the bitmaps, a word a warp: pages taken whatever their scores, pages surely in,
    // pages near the border, which are listed too (the first kGather of them)
    int n_in = 0;
    uint64_t near_of = 0;
    static_assert(NK <= 64, "a bit a page of the thread");
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const int word = i * NW + warp, j = 32 * word + lane;
        if (word >= words)
            break;
        const bool inside = j >= lo && j < hi;
        bool take = false, near = false;
        if (need > 0 && inside) {
            const bool inf = v[i] == INFINITY, unknown = v[i] != v[i];
            if (border == kInf) {
                near = inf;
            } else if (border == kUnknown) {
                take = !unknown;
                near = unknown;
            } else if (!unknown) {
                take = inf || v[i] > in_above;
                near = !take && v[i] >= near_from;
            }
        }
        const uint32_t a = __ballot_sync(0xFFFFFFFFu, take), c = __ballot_sync(0xFFFFFFFFu, near);
        const uint32_t always = __ballot_sync(0xFFFFFFFFu, j < n && !inside);
        n_in += __popc(a);
        if (lane == 0) {
            bm[word] = a | always;
            band[word] = c;
        }
        near_of |= (uint64_t)near << i;
    }
    for (; near_of; near_of &= near_of - 1ull) {   // outside the unrolled loop: one copy of the code to fetch
        const int at = atomicAdd(&sm.n_band, 1);
        if (at < kGather)
            sm.cand_j[at] = (__ffsll((long long)near_of) - 1) * NTH + tid;
    }
    if (lane == 0 && n_in)
        atomicAdd(&sm.n_in, n_in);
    __syncthreads();
    const uint32_t total_band = (uint32_t)sm.n_band;
    int left = need - sm.n_in;                  // of the near ones
    bool lowest = border != kFinite;            // take the lowest pages of the (remaining) band
    if (left > 0 && !lowest && left < (int)total_band) {
        const ExactWeights<D> weights(sm.qa, sm.qb, lane);
        const int32_t* table = p.pages + (int64_t)s * p.max_pages;
        if (total_band <= (uint32_t)kGather) {
            for (int i = warp; i < (int)total_band; i += NW) {
                const uint64_t key = exact_key<D>(p, table[sm.cand_j[i]], h, weights, lane);
                if (lane == 0)
                    sm.cand[i] = key;
            }
            __syncthreads();
            for (int i = tid; i < (int)total_band; i += NTH) {
                const uint64_t key = sm.cand[i];
                const int j = sm.cand_j[i];
                int rank = 0;
                for (int o = 0; o < (int)total_band; ++o)
                    rank += sm.cand[o] > key || (sm.cand[o] == key && sm.cand_j[o] < j);
                if (rank < left)
                    atomicOr(&bm[j >> 5], 1u << (j & 31));
            }
            left = 0;
        } else {   // many equal or nearly equal scores: exact keys over the scores, then a search by digits
            uint64_t kmin = ~0ull, kmax = 0ull;
            for (int w = warp; w < words; w += NW)
                for (uint32_t e = band[w]; e; e &= e - 1u) {
                    const int j = 32 * w + __ffs((int)e) - 1;
                    const uint64_t key = exact_key<D>(p, table[j], h, weights, lane);
                    if (lane == 0)
                        keys64[j] = key;
                    kmin = min(kmin, key);
                    kmax = max(kmax, key);
                }
            if (lane == 0) {
                sm.warp_min[warp] = kmin;
                sm.warp_max[warp] = kmax;
            }
            __syncthreads();
            for (int w = 0; w < NW; ++w) {
                kmin = min(kmin, sm.warp_min[w]);
                kmax = max(kmax, sm.warp_max[w]);
            }
            uint64_t prefix = kmin;
            int shift = 0, count = 0;
            auto each = [&](auto f) {
                for (int j = tid; j < words * 32; j += NTH)
                    if ((band[j >> 5] >> (j & 31)) & 1u)
                        f(keys64[j]);
            };
            if (kmin != kmax)
                radix_find<NTH>(sm, kmin, kmax, each, left, shift, prefix, count);
            // what is above the digit is in; what shares it is the new band
            __syncthreads();
            const bool rank_them = kmin != kmax && shift > 0 && count != left;
            for (int j = tid; j < words * 32; j += NTH) {
                bool take = false, near = false;
                if ((band[j >> 5] >> (j & 31)) & 1u) {
                    const uint64_t key = keys64[j];
                    take = (key >> shift) > prefix;
                    near = (key >> shift) == prefix;
                    if (near && rank_them) {
                        const int i = atomicAdd(&sm.n_cand, 1);
                        sm.cand[i] = key;
                        sm.cand_j[i] = j;
                    }
                }
                const uint32_t a = __ballot_sync(0xFFFFFFFFu, take), c = __ballot_sync(0xFFFFFFFFu, near);
                if (lane == 0) {
                    bm[j >> 5] |= a;
                    band[j >> 5] = c;
                }
            }
            __syncthreads();
            if (rank_them) {
                for (int i = tid; i < count; i += NTH) {
                    const uint64_t key = sm.cand[i];
                    const int j = sm.cand_j[i];
                    int rank = 0;
                    for (int o = 0; o < count; ++o)
                        rank += sm.cand[o] > key || (sm.cand[o] == key && sm.cand_j[o] < j);
                    if (rank < left)
                        atomicOr(&bm[j >> 5], 1u << (j & 31));
                }
                left = 0;
            } else {
                lowest = true;
            }
        }
    } else if (left > 0) {
        lowest = true;   // all of them, or equal ones
    }
    __syncthreads();
    if (left > 0 && lowest) {   // the lowest `left` pages of the band
        uint32_t run = 0;
        for (int w0 = 0; w0 < words; w0 += NTH) {
            const int w = w0 + tid;
            uint32_t e = w < words ? band[w] : 0u, total, take = 0;
            int room = left - (int)(run + block_scan<NTH>((uint32_t)__popc(e), sm.warp_sum, total));
            for (; room > 0 && e; --room, e &= e - 1u)
                take |= e & (0u - e);
            if (take)
                bm[w] |= take;
            run += total;
        }
        __syncthreads();
    }
    uint32_t run = 0;
    for (int w0 = 0; w0 < words; w0 += NTH) {
        const int w = w0 + tid;
        uint32_t e = w < words ? bm[w] : 0u, total;
        uint32_t at = run + block_scan<NTH>((uint32_t)__popc(e), sm.warp_sum, total);
        while (e) {
            if (at < (uint32_t)p.k)
                out[at] = 32 * w + __ffs((int)e) - 1;
            ++at;
            e &= e - 1u;
        }
        run += total;
    }
}

template <int D, int NTH, int NK>
__global__ void __launch_bounds__(NTH) select_kernel(const SelectParams p)
{
    extern __shared__ __align__(16) unsigned char sel_raw[];
    __shared__ SelSmem<D, NTH> sm;
    const int s = blockIdx.x / p.H, h = blockIdx.x - s * p.H;
    if (!p.scored)   // the call's first kernel
        ptx::grid_wait();
    ptx::grid_launch_next();
    int lo, hi;
    const int n = page_range(p, s, lo, hi);
    if (h == 0 && threadIdx.x == 0 && (p.lens[s] < 0 || p.lens[s] > p.max_len))
        raise_err(p.err, KAMERA_DEVERR_LEN);
    if (n <= p.k) {
        ptx::grid_wait();
        take_all<NTH>(p, s, h, n);
        return;
    }
    for (int i = threadIdx.x; i < 2 * D; i += NTH) {
        float a, e;
        signed_sum<D>(p.q + ((int64_t)s * p.H + h) * p.G * D, p.G, i, a, e);
        keep_weight(sm, i, a, e);
    }
    clear_choice(sm);
    __syncthreads();
    ptx::grid_wait();   // the scores
    choose<D, NTH, NK>(p, s, h, n, lo, hi, p.keys + (int64_t)blockIdx.x * p.width, reinterpret_cast<uint32_t*>(sel_raw),
                       sm);
}

// Scores and choice in one launch, for rows of at most 2048 pages that leave every
// row an SM: the CTAs of a cluster score a row's pages into the first one's shared
// memory, which chooses.  With the attention, against two launches: 32 sequences x 4
// heads of 2048 pages 43.4 us for 49.0, 8 x 4 19.0 for 20.7, 48 x 2 of 334 pages of
// 64-wide heads 15.8 for 16.6; 1 x 4 15.0 for 14.2 (eight CTAs a row where the other
// form has 22), but 3 us less of host time.
constexpr int kFusedThreads = 256;
constexpr int kFusedWidth = 8 * kFusedThreads;

template <int D>
__global__ void __launch_bounds__(kFusedThreads) score_select_kernel(const SelectParams p)
{
    constexpr int WARPS = kFusedThreads / 32;
    using Y = ScoreLayout<D, WARPS>;
    extern __shared__ __align__(16) unsigned char ring_raw[];
    __shared__ ScoreSmem<D, WARPS> score;
    __shared__ SelSmem<D, kFusedThreads> sm;
    __shared__ uint64_t keys[kFusedWidth];
    __shared__ uint32_t maps[2 * kFusedWidth / 32];
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int s = blockIdx.y / p.H, h = blockIdx.y - s * p.H, rank = blockIdx.x;
    cluster.barrier_arrive();
    clear_choice(sm);
    ptx::grid_wait();
    ptx::grid_launch_next();
    bool peers = false;   // known: every CTA of the cluster runs, and its shared memory may be written
    float2* at = reinterpret_cast<float2*>(cluster.map_shared_rank(keys, 0));
    score_pages<D, WARPS>(
        p, s, h, rank, ring_raw, score, [&](int j, float2 x) { at[j] = x; },
        [&](int i, float a, float e) {
            if (rank == 0)
                keep_weight(sm, i, a, e);
        },
        [&] {
            cluster.barrier_wait();
            peers = true;
        });
    if (!peers)   // a share without pages
        cluster.barrier_wait();
    int lo, hi;
    const int n = page_range(p, s, lo, hi);
    if (h == 0 && rank == 0 && threadIdx.x == 0 && (p.lens[s] < 0 || p.lens[s] > p.max_len))
        raise_err(p.err, KAMERA_DEVERR_LEN);
    if (n <= p.k) {   // (the whole cluster)
        if (rank == 0)
            take_all<kFusedThreads>(p, s, h, n);
        return;
    }
    cluster.sync();
    if (rank == 0)
        choose<D, kFusedThreads, 8>(p, s, h, n, lo, hi, keys, maps, sm);
}

// Clusters of the grid's x extent.
template <typename K, typename... A>
cudaError_t launch_cluster(K kernel, dim3 grid, int block, size_t smem, cudaStream_t stream, const A&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = grid.x;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D>
cudaError_t launch_score(SelectParams& p, int scored, cudaStream_t stream)
{
    // CTAs that run at once: two an SM (four for boxes half the size).  Where a warp has
    // at most four batches that way, one round of CTAs (32 sequences of 512 pages with
    // the attention: 42.0 us, 46.4 in three rounds); else three, so that ragged lengths
    // even out (32 x 8192 pages: 114.4 us, 115.1 in two rounds, 115.5 in four; 125.7 against
    // 119.5 in one, both with CTAs of four warps)
    const int64_t units = (int64_t)p.n_seqs * p.H, step = kScoreWarps * kScorePages;
    const int64_t batches = (scored + step - 1) / step, slots = device_sms() * (D == 128 ? 2ll : 4ll);
    const int64_t each = (units * batches + slots - 1) / slots;
    p.sweeps = (int)std::max<int64_t>(1, each <= 4 ? each : (each + 2) / 3);
    const int64_t gx = (batches + p.sweeps - 1) / p.sweeps;
    const cudaError_t a = cudaFuncSetAttribute(score_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)ScoreLayout<D, kScoreWarps>::kBytes);
    if (a != cudaSuccess)
        return a;
    return launch_after(score_kernel<D>, dim3((unsigned)(gx * p.H), (unsigned)p.n_seqs), 32 * kScoreWarps, ScoreLayout<D, kScoreWarps>::kBytes,
                        stream, true, p);
}

template <int D>
cudaError_t launch_select(SelectParams& p, cudaStream_t stream)
{
    const int64_t units = (int64_t)p.n_seqs * p.H;
    const int scored = p.width - p.n_first - p.n_last;   // at most, of one sequence
    const bool score = p.width > p.k && scored > 0 && p.k > p.n_first + p.n_last;
    const int64_t each = units > 0 ? std::min<int64_t>(8, device_sms() / units) : 0;   // CTAs of a row
    if (score && p.width <= kFusedWidth && each > 0) {
        constexpr int WARPS = kFusedThreads / 32;
        using Y = ScoreLayout<D, WARPS>;
        const int64_t batches = (scored + WARPS * kScorePages - 1) / (WARPS * kScorePages);
        const int64_t ctas = std::min(each, batches);
        p.sweeps = (int)((batches + ctas - 1) / ctas);
        const cudaError_t e = cudaFuncSetAttribute(score_select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)Y::kBytes);
        if (e != cudaSuccess)
            return e;
        return launch_cluster(score_select_kernel<D>, dim3((unsigned)ctas, (unsigned)units), kFusedThreads, Y::kBytes,
                              stream, p);
    }
    if (score) {
        const cudaError_t e = launch_score<D>(p, scored, stream);
        if (e != cudaSuccess)
            return e;
        p.scored = 1;
    }
    const size_t smem = (size_t)((p.width + 31) / 32) * 8;
    // set at every launch: the attribute belongs to the current device's context
    // few pages: few threads, whose barriers are cheaper (32 rows x 4 of 512 pages and
    // one of 2048, with the attention: 40.1 and 14.2 us, with 1024 threads 42.0 and 15.2;
    // with 128 the latter took 2.6 us more).  Past 8192 pages a thread holds 48 scores,
    // some of them spilled: one context of 8192 pages 20.7 us with the attention over 128
    // pages, of 8193 26.1, of 16384 31.5, of 49152 57.1; eight contexts 46.5, 52.2, 71.1 and 152.8
    auto launch = [&](auto kernel, int threads) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        return e != cudaSuccess ? e : launch_after(kernel, dim3((unsigned)units), threads, smem, stream, true, p);
    };
    return p.width <= 2048   ? launch(select_kernel<D, 256, 8>, 256)
           : p.width <= 8192 ? launch(select_kernel<D, 1024, 8>, 1024)
                             : launch(select_kernel<D, 1024, 48>, 1024);
}

int check_select(const KameraPageSelect* x, const KameraPageTable* t)
{
    if (!x || !t)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (x->n_seqs < 0 || x->num_kv_heads < 1 || x->num_q_heads < 1 || x->num_q_heads % x->num_kv_heads ||
        x->num_pages < 0 || x->n_select < 0 || x->n_first < 0 || x->n_last < 0 ||
        (int64_t)x->n_first + x->n_last > x->n_select || t->max_len < 0 || t->max_pages < 0 || x->page_size < 1)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if ((x->head_dim != 64 && x->head_dim != 128) || x->num_q_heads / x->num_kv_heads > 16 || (x->page_size % 16) ||
        x->num_pages > 0x7FFFFFFF || (int64_t)x->n_seqs * x->num_kv_heads > 65535 ||
        ((int64_t)t->max_len + x->page_size - 1) / x->page_size > kMaxWidth)
        return KAMERA_ERR_UNSUPPORTED;
    if ((int64_t)t->max_pages * x->page_size < t->max_len)
        return KAMERA_ERR_INVALID_ARGUMENT;
    return KAMERA_OK;
}

int64_t select_width(const KameraPageSelect* x, const KameraPageTable* t)
{
    return ((int64_t)t->max_len + x->page_size - 1) / x->page_size;
}

}  // namespace

}  // namespace kamera

using namespace kamera;

extern "C" {

int kamera_summarize_pages(const KameraPagedKV* kv, const int32_t* d_page_ids, const int32_t* d_page_tokens, int32_t n,
                           void* summary, int32_t* d_err, struct CUstream_st* stream)
{
    if (!kv || kv->reserved != 0 || n < 0 || kv->num_kv_heads < 1 || kv->head_dim < 8 || kv->page_size < 1)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if ((kv->head_dim % 8) || kv->head_dim > KAMERA_MAX_ROW_ELEMS || (kv->page_size % 16) ||
        kv->num_slots > 0x7FFFFFFF || kv->num_kv_heads > 65535)
        return KAMERA_ERR_UNSUPPORTED;
    const int64_t W = (int64_t)kv->num_kv_heads * kv->head_dim;
    int rc;
    if ((rc = check_strided(kv->k, 1, 0, kv->num_slots, kv->slot_stride, W, false)))
        return rc;
    if (n == 0)
        return KAMERA_OK;
    if (!d_page_ids || !d_page_tokens || !summary)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (!aligned16(summary) || ((reinterpret_cast<uintptr_t>(d_page_ids) | reinterpret_cast<uintptr_t>(d_page_tokens)) & 3))
        return KAMERA_ERR_MISALIGNED;
    const int64_t pages = kv->num_slots / kv->page_size;
    if (overlap(span(kv->k, 1, 0, kv->num_slots, kv->slot_stride, W), span(summary, 1, 0, pages, 2 * W, 2 * W)))
        return KAMERA_ERR_INVALID_ARGUMENT;
    SummaryParams p;
    std::memset(&p, 0, sizeof(p));
    p.k = static_cast<const __nv_bfloat16*>(kv->k);
    p.out = static_cast<__nv_bfloat16*>(summary);
    p.ids = d_page_ids;
    p.tokens = d_page_tokens;
    p.slot_stride = kv->slot_stride;
    p.num_pages = pages;
    p.H = kv->num_kv_heads;
    p.d = kv->head_dim;
    p.P = kv->page_size;
    p.vecs = (int32_t)(W / 8);
    p.items = (int64_t)n * p.vecs;
    p.err = d_err;
    const int64_t ctas = (p.items + 127) / 128;
    if (ctas > 0x7FFFFFFF)
        return KAMERA_ERR_UNSUPPORTED;
    return launch_after(summary_kernel, dim3((unsigned)ctas), 128, 0, reinterpret_cast<cudaStream_t>(stream), true, p) ==
                   cudaSuccess
               ? KAMERA_OK
               : KAMERA_ERR_CUDA;
}

size_t kamera_select_pages_workspace_bytes(const KameraPageSelect* select, const KameraPageTable* table)
{
    if (check_select(select, table))
        return 0;
    return (size_t)select->n_seqs * select->num_kv_heads * (size_t)select_width(select, table) * 8u;
}

int kamera_select_pages(const KameraPageSelect* select, const KameraPageTable* table, void* d_workspace,
                        size_t workspace_bytes, int32_t* d_err, struct CUstream_st* stream)
{
    int rc = check_select(select, table);
    if (rc)
        return rc;
    const KameraPageSelect& x = *select;
    if (x.n_seqs == 0 || x.n_select == 0)
        return KAMERA_OK;
    const int64_t width = select_width(select, table);
    if (!x.q || !x.selected || !table->lens || (width > 0 && (!table->pages || (x.num_pages > 0 && !x.summary))))
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (!aligned16(x.q) || !aligned16(x.summary) ||
        ((reinterpret_cast<uintptr_t>(x.selected) | reinterpret_cast<uintptr_t>(table->lens) |
          reinterpret_cast<uintptr_t>(table->pages)) & 3))
        return KAMERA_ERR_MISALIGNED;
    const size_t need = kamera_select_pages_workspace_bytes(select, table);
    if (need > 0) {
        if (!d_workspace || workspace_bytes < need)
            return KAMERA_ERR_INVALID_ARGUMENT;
        if (!aligned16(d_workspace))
            return KAMERA_ERR_MISALIGNED;
    }
    const auto ws = std::pair<uintptr_t, uintptr_t>{reinterpret_cast<uintptr_t>(d_workspace),
                                                    reinterpret_cast<uintptr_t>(d_workspace) + need};
    const auto qs = span(x.q, 1, 0, x.n_seqs, (int64_t)x.num_q_heads * x.head_dim, (int64_t)x.num_q_heads * x.head_dim);
    const int64_t row = 2ll * x.num_kv_heads * x.head_dim;
    const auto ss = span(x.summary, 1, 0, x.num_pages, row, row);
    const int64_t sel = 2ll * x.num_kv_heads * x.n_select;   // int32: two bf16 widths each
    const auto os = span(x.selected, 1, 0, x.n_seqs, sel, sel);
    const auto ts = span(table->pages, 1, 0, x.n_seqs, 2ll * table->max_pages, 2ll * table->max_pages);
    const auto ls = span(table->lens, 1, 0, x.n_seqs, 2, 2);
    for (const auto& a : {qs, ss, ts, ls})
        if (overlap(os, a) || overlap(ws, a))
            return KAMERA_ERR_INVALID_ARGUMENT;
    if (overlap(ws, os))
        return KAMERA_ERR_INVALID_ARGUMENT;
    SelectParams p;
    std::memset(&p, 0, sizeof(p));
    p.q = static_cast<const __nv_bfloat16*>(x.q);
    p.summary = static_cast<const __nv_bfloat16*>(x.summary);
    p.pages = table->pages;
    p.lens = table->lens;
    p.selected = x.selected;
    p.keys = static_cast<uint64_t*>(d_workspace);
    p.num_pages = x.num_pages;
    p.n_seqs = x.n_seqs;
    p.H = x.num_kv_heads;
    p.G = x.num_q_heads / x.num_kv_heads;
    p.P = x.page_size;
    p.max_pages = table->max_pages;
    p.max_len = table->max_len;
    p.width = (int32_t)width;
    p.k = x.n_select;
    p.n_first = x.n_first;
    p.n_last = x.n_last;
    p.err = d_err;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return (x.head_dim == 128 ? launch_select<128>(p, st) : launch_select<64>(p, st)) == cudaSuccess ? KAMERA_OK
                                                                                                     : KAMERA_ERR_CUDA;
}

}  // extern "C"
