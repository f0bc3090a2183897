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
// one order or another would flip it where two scores lie close.  The scores
// are therefore held as pairs of floats: q+ and q- are split into a 16-bit part,
// whose products with the bf16 box are exact in fp32, and a remainder; the
// exact products are added with the error of every addition kept (the two-sum
// of Knuth, The Art of Computer Programming vol. 2, 4.2.2), which leaves about
// 2^-40 of the sum of the terms' magnitudes.  Two channels go through each
// packed fp32 instruction, and the sums of eight pages are reduced across the
// warp together (each step halves the pages a lane holds), so the arithmetic
// stays below the time the boxes take to arrive.
#include <algorithm>
#include <cstdint>
#include <cstring>

#include "kamera_common.cuh"
#include "kamera_hostcheck.h"
#include "kamera_internal.h"
#include "kamera_ptx.cuh"

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

// Four lanes share a 16-byte vector of a page's rows, each taking every fourth
// token (lanes 8 apart, so eight neighbouring vectors of a token are read
// together), and join by shuffles.  Read-bound: each key once, min and max
// exact in bf16.
__global__ void __launch_bounds__(256) summary_kernel(const SummaryParams p)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = lane >> 3;
    const int64_t item = ((int64_t)blockIdx.x * 8 + warp) * 8 + (lane & 7);
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo[i] = 0x7F807F80u;   // +infinity
        hi[i] = 0xFF80FF80u;   // -infinity
    }
    bool write = false;
    int64_t page = 0;
    int vec = 0;
    if (item < p.items) {
        const int64_t e = item / p.vecs;
        vec = (int)(item - e * p.vecs);
        page = p.ids[e];
        const int c = p.tokens[e];
        int32_t bits = 0;
        if (page < 0 || page >= p.num_pages)
            bits |= KAMERA_DEVERR_SLOT;
        if (c < 0 || c > p.P)
            bits |= KAMERA_DEVERR_LEN;
        if (bits && vec == 0 && part == 0)
            raise_err(p.err, bits);
        if (!bits && c > 0) {
            write = true;
            const __nv_bfloat16* src = p.k + page * p.P * p.slot_stride + 8 * vec;
#pragma unroll 4
            for (int t = part; t < c; t += 4) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + (int64_t)t * p.slot_stride));
                lo[0] = min_bf16x2(lo[0], v.x);
                lo[1] = min_bf16x2(lo[1], v.y);
                lo[2] = min_bf16x2(lo[2], v.z);
                lo[3] = min_bf16x2(lo[3], v.w);
                hi[0] = max_bf16x2(hi[0], v.x);
                hi[1] = max_bf16x2(hi[1], v.y);
                hi[2] = max_bf16x2(hi[2], v.z);
                hi[3] = max_bf16x2(hi[3], v.w);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int s = 8; s <= 16; s *= 2) {
            lo[i] = min_bf16x2(lo[i], __shfl_xor_sync(0xFFFFFFFFu, lo[i], s));
            hi[i] = max_bf16x2(hi[i], __shfl_xor_sync(0xFFFFFFFFu, hi[i], s));
        }
    if (write && part < 2) {   // lanes of part 0 write the minima, of part 1 the maxima
        const int vh = p.d / 8, h = vec / vh;
        __nv_bfloat16* o = p.out + ((page * p.H + h) * 2 + part) * p.d + 8 * (vec - h * vh);
        *reinterpret_cast<uint4*>(o) =
            part == 0 ? make_uint4(lo[0], lo[1], lo[2], lo[3]) : make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
}

// ------------------------------------------------------------------- scores --
struct SelectParams {
    const __nv_bfloat16* q;
    const __nv_bfloat16* summary;
    const int32_t* pages;
    const int32_t* lens;
    int32_t* selected;
    uint64_t* keys;              // [n_seqs * H][width]
    int64_t num_pages;
    int32_t n_seqs, H, G, P;
    int32_t max_pages, max_len, width;
    int32_t k, n_first, n_last;
    int32_t sweeps;              // score kernel: batches of a warp
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

constexpr int kScoreWarps = 8;
constexpr int kBatch = 8;        // loads a lane keeps in flight: kBatch * (32 / LP) pages a warp

template <int D>
__global__ void __launch_bounds__(32 * kScoreWarps) score_kernel(const SelectParams p)
{
    constexpr int LP = D / 4;                    // lanes of a page: 16 bytes of [min | max] each
    constexpr int PL = 32 / LP;                  // pages a warp loads at once
    constexpr int PB = kBatch * PL;              // pages of a warp's batch
    __shared__ __align__(16) float qa[2 * D], qb[2 * D];   // q- | q+ : the 16-bit part and the rest
    const int s = blockIdx.y / p.H, h = blockIdx.y - s * p.H;
    int lo, hi;
    page_range(p, s, lo, hi);
    const int chunk = kScoreWarps * PB * p.sweeps;
    const int c0 = lo + (int)blockIdx.x * chunk;
    if (c0 >= hi)
        return;
    for (int i = threadIdx.x; i < 2 * D; i += 32 * kScoreWarps) {
        const int ch = i < D ? i : i - D;
        float a = 0.f, e = 0.f;
        for (int g = 0; g < p.G; ++g) {
            const float x = __bfloat162float(p.q[((int64_t)s * p.H * p.G + h * p.G + g) * D + ch]);
            pair_add(a, e, i < D ? fminf(x, 0.f) : fmaxf(x, 0.f), 0.f);
            if (x != x)
                a = x;   // fminf and fmaxf drop a NaN
        }
        const float top = __uint_as_float(__float_as_uint(a) & 0xFFFFFF00u);   // 16 significant bits
        qa[i] = top;
        qb[i] = __fadd_rn(__fadd_rn(a, -top), e);
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & (LP - 1), which = lane / LP;
    uint64_t wa[4], wb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        wa[i] = *reinterpret_cast<const uint64_t*>(&qa[8 * sub + 2 * i]);
        wb[i] = *reinterpret_cast<const uint64_t*>(&qb[8 * sub + 2 * i]);
    }
    const uint64_t neg1 = ptx::f2_make(0xBF800000u, 0xBF800000u);
    const int32_t* table = p.pages + (int64_t)s * p.max_pages;
    uint64_t* keys = p.keys + (int64_t)blockIdx.y * p.width;
    const int c1 = min(c0 + chunk, hi);
    for (int j0 = c0 + warp * PB; j0 < c1; j0 += kScoreWarps * PB) {
        // the batch's pages, one to a lane (-1: past the range or outside the pool)
        int mine = -1;
        if (lane < PB && j0 + lane < c1) {
            mine = table[j0 + lane];
            if (mine < 0 || mine >= p.num_pages) {
                mine = -1;
                if (h == 0)
                    raise_err(p.err, KAMERA_DEVERR_SLOT);
            }
        }
        uint4 v[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int page = __shfl_sync(0xFFFFFFFFu, mine, b * PL + which);
            v[b] = make_uint4(0u, 0u, 0u, 0u);
            if (page >= 0)
                v[b] = __ldg(reinterpret_cast<const uint4*>(p.summary + ((int64_t)page * p.H + h) * (2 * D)) + sub);
        }
        float S[kBatch], E[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
            uint64_t x = ptx::f2_from_bf16x2(w[0]);
            uint64_t sum = ptx::f2_mul(wa[0], x), err = ptx::f2_mul(wb[0], x);
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                x = ptx::f2_from_bf16x2(w[i]);
                const uint64_t pr = ptx::f2_mul(wa[i], x);           // exact
                const uint64_t t = ptx::f2_add(sum, pr);
                const uint64_t z = ptx::f2_fma(sum, neg1, t);        // t - sum
                const uint64_t tz = ptx::f2_fma(z, neg1, t);         // t - z
                const uint64_t r = ptx::f2_add(ptx::f2_fma(tz, neg1, sum), ptx::f2_fma(z, neg1, pr));
                err = ptx::f2_add(ptx::f2_fma(wb[i], x, err), r);
                sum = t;
            }
            uint32_t s0, s1, e0, e1;
            asm("mov.b64 {%0, %1}, %2;" : "=r"(s0), "=r"(s1) : "l"(sum));
            asm("mov.b64 {%0, %1}, %2;" : "=r"(e0), "=r"(e1) : "l"(err));
            S[b] = __uint_as_float(s0);
            E[b] = __uint_as_float(e0);
            pair_add(S[b], E[b], __uint_as_float(s1), __uint_as_float(e1));
        }
        // reduce over a page's LP lanes: each of three steps halves the batch a lane holds
#pragma unroll
        for (int step = 0; step < 3; ++step) {
            const int dist = LP >> (step + 1), keep = kBatch >> (step + 1);
            const bool up = (sub & dist) != 0;
#pragma unroll
            for (int i = 0; i < keep; ++i) {
                const float ss = up ? S[i] : S[i + keep], ee = up ? E[i] : E[i + keep];
                float ks = up ? S[i + keep] : S[i], ke = up ? E[i + keep] : E[i];
                pair_add(ks, ke, __shfl_xor_sync(0xFFFFFFFFu, ss, dist), __shfl_xor_sync(0xFFFFFFFFu, ee, dist));
                S[i] = ks;
                E[i] = ke;
            }
        }
#pragma unroll
        for (int dist = LP / 16; dist >= 1; dist /= 2)
            pair_add(S[0], E[0], __shfl_xor_sync(0xFFFFFFFFu, S[0], dist), __shfl_xor_sync(0xFFFFFFFFu, E[0], dist));
        // lane `sub` holds batch entry sub / (LP / 8)
        const int at = (sub / (LP / 8)) * PL + which;
        const bool known = __shfl_sync(0xFFFFFFFFu, mine, at) >= 0;
        if ((sub & (LP / 8 - 1)) == 0 && j0 + at < c1) {
            float t, r;
            two_sum(S[0], E[0], t, r);   // t + r, t the sum rounded: (t, r) orders as the sum does
            uint64_t key = 0;
            if (known) {
                if (!(fabsf(t) <= 3.402823466e38f && r == r)) {   // not finite: ranks first
                    t = INFINITY;
                    r = 0.f;
                }
                key = ((uint64_t)ordered(t) << 32) | ordered(r);
            }
            keys[j0 + at] = key;
        }
    }
}

// ------------------------------------------------------------------- choice --
constexpr int kSelThreads = 512;
constexpr int kBins = 2048;              // digits of 11 bits
constexpr int kGather = 1024;            // keys of one digit that are ranked by comparison
constexpr int kMaxWidth = 1 << 17;       // pages of a sequence
constexpr int kStage = 12288;            // keys kept in shared memory (96 KB)

struct SelSmem {
    uint32_t hist[kBins];
    uint64_t cand[kGather];
    int32_t cand_j[kGather];
    uint32_t warp_sum[kSelThreads / 32];
    uint64_t warp_min[kSelThreads / 32], warp_max[kSelThreads / 32];
    int32_t bin, above, n_cand;
};

// Exclusive sum over the block of one value a thread; `total` for everybody.
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
    __syncthreads();
    if (lane == 31)
        warp_sum[warp] = x;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kSelThreads / 32; ++w) {
        if (w < warp)
            before += warp_sum[w];
        total += warp_sum[w];
    }
    return before + x - v;
}

// One CTA per (sequence, KV head): the k-th largest key by radix steps of 11
// bits from the first bit in which the keys differ, then the pages above it in
// order from a bitmap.  A step ends the search when a digit's keys are all
// taken, all equal (the lowest pages win), or few enough to rank by comparison,
// which random scores reach after one or two steps.  Latency-bound: a handful of
// passes over the keys, which stay in shared memory up to 12288 pages.
template <bool STAGE>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p)
{
    extern __shared__ __align__(16) unsigned char sel_raw[];
    __shared__ SelSmem sm;
    const int words = (p.width + 31) >> 5;
    uint32_t* bm = reinterpret_cast<uint32_t*>(sel_raw);        // pages taken
    uint32_t* beq = bm + words;                                 // pages whose key equals the last one taken
    uint64_t* stage = reinterpret_cast<uint64_t*>(sel_raw + ((size_t)words * 8 + 15) / 16 * 16);
    const int s = blockIdx.x / p.H, h = blockIdx.x - s * p.H, tid = threadIdx.x, lane = tid & 31;
    int lo, hi;
    const int n = page_range(p, s, lo, hi);
    int32_t* out = p.selected + (int64_t)blockIdx.x * p.k;
    if (h == 0 && tid == 0 && (p.lens[s] < 0 || p.lens[s] > p.max_len))
        raise_err(p.err, KAMERA_DEVERR_LEN);
    if (n <= p.k) {   // every page
        for (int i = tid; i < p.k; i += kSelThreads)
            out[i] = i < n ? i : -1;
        return;
    }
    const uint64_t* keys = p.keys + (int64_t)blockIdx.x * p.width;
    int need = p.k - p.n_first - p.n_last;
    uint64_t kmin = ~0ull, kmax = 0ull;
    if (need > 0) {
        for (int j = lo + tid; j < hi; j += kSelThreads) {
            const uint64_t key = keys[j];
            if (STAGE)
                stage[j] = key;
            kmin = min(kmin, key);
            kmax = max(kmax, key);
        }
#pragma unroll
        for (int o = 16; o >= 1; o /= 2) {
            kmin = min(kmin, __shfl_xor_sync(0xFFFFFFFFu, kmin, o));
            kmax = max(kmax, __shfl_xor_sync(0xFFFFFFFFu, kmax, o));
        }
        if (lane == 0) {
            sm.warp_min[tid >> 5] = kmin;
            sm.warp_max[tid >> 5] = kmax;
        }
    }
    for (int w = tid; w < words; w += kSelThreads)
        bm[w] = beq[w] = 0u;
    if (tid == 0)
        sm.n_cand = 0;
    __syncthreads();
    const uint64_t* src = STAGE ? stage : keys;
    // taken: keys whose top bits (>> shift) exceed `prefix`, and of those that
    // equal it: all (mode 0), the listed ones (mode 1) or the lowest `need` pages (mode 2)
    int mode = 0, shift = 0;
    uint64_t prefix = ~0ull;
    if (need > 0) {
        for (int w = 0; w < kSelThreads / 32; ++w) {
            kmin = min(kmin, sm.warp_min[w]);
            kmax = max(kmax, sm.warp_max[w]);
        }
        if (kmin == kmax) {
            prefix = kmin;
            mode = 2;
        } else {
            const int top = 63 - __clzll((long long)(kmin ^ kmax));   // the highest bit that differs
            shift = max(0, top - 10);
            uint64_t fixed = top == 63 ? 0ull : kmin >> (top + 1);    // bits above the digit, shared so far
            int width = top + 1 - shift;                              // bits of the digit
            for (;;) {
                for (int b = tid; b < kBins; b += kSelThreads)
                    sm.hist[b] = 0u;
                __syncthreads();
                const int up = shift + width;                         // 64: no bits above
                for (int j = lo + tid; j < hi; j += kSelThreads) {
                    const uint64_t key = src[j];
                    if ((up >= 64 ? 0ull : key >> up) == fixed)
                        atomicAdd(&sm.hist[(key >> shift) & ((1u << width) - 1u)], 1u);
                }
                __syncthreads();
                // thread t's bins, from the top: kBins - 1 - 4 t downwards
                uint32_t c[kBins / kSelThreads], mine = 0;
#pragma unroll
                for (int i = 0; i < kBins / kSelThreads; ++i) {
                    c[i] = sm.hist[kBins - 1 - (kBins / kSelThreads) * tid - i];
                    mine += c[i];
                }
                uint32_t total;
                uint32_t above = block_scan(mine, sm.warp_sum, total);
#pragma unroll
                for (int i = 0; i < kBins / kSelThreads; ++i) {
                    if ((int)above < need && need <= (int)(above + c[i])) {
                        sm.bin = kBins - 1 - (kBins / kSelThreads) * tid - i;
                        sm.above = (int)above;
                    }
                    above += c[i];
                }
                __syncthreads();
                const int bin = sm.bin, count = (int)sm.hist[bin];
                need -= sm.above;
                prefix = (fixed << width) | (uint64_t)bin;            // width <= 11 < 64
                if (count == need) {
                    mode = 0;
                    break;
                }
                if (shift == 0) {
                    mode = 2;
                    break;
                }
                if (count <= kGather) {
                    mode = 1;
                    break;
                }
                fixed = prefix;
                width = min(11, shift);
                shift -= width;
                __syncthreads();   // the histogram is cleared next
            }
        }
    }
    // the bitmaps: whole words, so every thread of a warp takes part
    for (int j = tid; j < words * 32; j += kSelThreads) {
        bool take = j < n && (j < p.n_first || j >= n - p.n_last), eq = false;
        uint64_t key = 0;
        if (need > 0 && j >= lo && j < hi) {
            key = src[j];
            const uint64_t t = key >> shift;
            take = t > prefix || (mode == 0 && t == prefix);
            eq = mode != 0 && t == prefix;
        }
        if (mode == 1 && eq) {
            const int i = atomicAdd(&sm.n_cand, 1);
            sm.cand[i] = key;
            sm.cand_j[i] = j;
        }
        const uint32_t a = __ballot_sync(0xFFFFFFFFu, take), b = __ballot_sync(0xFFFFFFFFu, eq);
        if (lane == 0) {
            bm[j >> 5] = a;
            beq[j >> 5] = b;
        }
    }
    __syncthreads();
    if (mode == 1) {
        const int m = sm.n_cand;
        for (int i = tid; i < m; i += kSelThreads) {
            const uint64_t key = sm.cand[i];
            const int j = sm.cand_j[i];
            int rank = 0;
            for (int o = 0; o < m; ++o)
                rank += sm.cand[o] > key || (sm.cand[o] == key && sm.cand_j[o] < j);
            if (rank < need)
                atomicOr(&bm[j >> 5], 1u << (j & 31));
        }
    } else if (mode == 2) {   // the lowest `need` of the equal ones
        uint32_t run = 0;
        for (int w0 = 0; w0 < words; w0 += kSelThreads) {
            const int w = w0 + tid;
            uint32_t e = w < words ? beq[w] : 0u, total;
            const uint32_t before = run + block_scan((uint32_t)__popc(e), sm.warp_sum, total);
            int left = need - (int)before;
            uint32_t take = 0;
            while (left > 0 && e) {
                take |= e & (0u - e);
                e &= e - 1u;
                --left;
            }
            if (take)
                bm[w] |= take;
            run += total;
        }
    }
    __syncthreads();
    uint32_t run = 0;
    for (int w0 = 0; w0 < words; w0 += kSelThreads) {
        const int w = w0 + tid;
        uint32_t e = w < words ? bm[w] : 0u, total;
        uint32_t at = run + block_scan((uint32_t)__popc(e), sm.warp_sum, total);
        while (e) {
            if (at < (uint32_t)p.k)
                out[at] = 32 * w + __ffs((int)e) - 1;
            ++at;
            e &= e - 1u;
        }
        run += total;
    }
}

template <int D>
cudaError_t launch_select(SelectParams& p, cudaStream_t stream)
{
    constexpr int PB = kBatch * (32 / (D / 4));
    const int64_t units = (int64_t)p.n_seqs * p.H;
    const int scored = p.width - p.n_first - p.n_last;   // at most, of one sequence
    if (p.width > p.k && scored > 0 && p.k > p.n_first + p.n_last) {
        // enough CTAs for every SM's slots several times over before a warp takes
        // a second batch
        const int64_t batches = (scored + kScoreWarps * PB - 1) / (kScoreWarps * PB);
        p.sweeps = (int)std::max<int64_t>(1, std::min<int64_t>(8, units * batches / (152 * 16)));
        const int64_t gx = (batches + p.sweeps - 1) / p.sweeps;
        score_kernel<D><<<dim3((unsigned)gx, (unsigned)units), 32 * kScoreWarps, 0, stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
    }
    const size_t bits = ((size_t)((p.width + 31) / 32) * 8 + 15) / 16 * 16;
    const bool stage = p.width <= kStage;
    const size_t smem = bits + (stage ? (size_t)p.width * 8 : 0);
    // set at every launch: the attribute belongs to the current device's context
    const cudaError_t e = stage ? cudaFuncSetAttribute(select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       (int)smem)
                                : cudaFuncSetAttribute(select_kernel<false>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess)
        return e;
    if (stage)
        select_kernel<true><<<(unsigned)units, kSelThreads, smem, stream>>>(p);
    else
        select_kernel<false><<<(unsigned)units, kSelThreads, smem, stream>>>(p);
    return cudaGetLastError();
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
    const int64_t ctas = (p.items + 63) / 64;
    if (ctas > 0x7FFFFFFF)
        return KAMERA_ERR_UNSUPPORTED;
    summary_kernel<<<(unsigned)ctas, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? KAMERA_OK : KAMERA_ERR_CUDA;
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
