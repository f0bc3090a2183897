// kamera_packed.cu -- decode attention over pages in 4 bits (kamera_pack.cu has their
// layout), joined with a tail of bf16 pages.
//
// A packed token costs 9 d / 8 bytes a KV head (144 for d = 128) where bf16 costs 4 d,
// for the same 4 d G flops: warp-level MMAs, which just keep up with bf16 pages, would
// bound it.  So the products run on the 5th-generation tensor cores, and what the
// threads do is decode: one conversion (two e2m1 codes to fp16) and one multiplication
// (the scale) for two numbers, straight into TMEM as the A operands:
//   S^T [128 tokens x N]    = K [128 x d] q^T      thread = token: its row of K
//   O^T [d channels x N]   += V^T [d x 128] P^T    thread = channel: its 128 tokens
// with the query heads of a KV head (8 or 16) as N.  Everything is exact in fp16: e2m1
// times e4m3 has 6 significant bits, and the queries enter as q 2^(10 - e), e the
// exponent of the row's largest (a bf16 number keeps its 8 bits down to 2^-24 of it).
// The weights are rounded to fp16 (2^-11), as 2^7 times the usual ones, so that small
// ones stay normal down to 2^-21.
//   warps 0-3   softmax (warp w: tokens 32 w .. 32 w + 31) and output
//   warps 4-7   keys, two tiles of them in TMEM
//   warps 8-11  values
//   warp 12     producer: one bulk copy for 16 tokens of a head, a ring of tiles
//   warp 13     MMA; it owns TMEM (256 columns, so that two CTAs share an SM: one
//               decodes while the other waits for its products)
// Work: the batch's tiles of 128 tokens, all (sequence, KV head) behind one another, in
// equal ranges, one a CTA; each leaves a partial state for every (sequence, KV head)
// that it touches, and a last launch joins them with the tail's.
// Measured, calls back to back on data in turn: 32 contexts of up to 32768 tokens, 4 KV
// heads of 128 with 7 query heads, in 105 us (4.9 TB/s), 32 KV heads with one each 56: a
// tile takes an SM 865 cycles where HBM alone would need 785 (the issue slots are 70%
// full), but CTAs with equal work end up to 20% apart.  One context of 32768 takes 14.9:
// start, four tiles, the join.  Steps of two tiles for the softmax (8 query heads) took 5%
// more: a step's products then wait for the keys of two more tiles.
#include <algorithm>
#include <cstdint>
#include <cstring>

#include "kamera_common.cuh"
#include "kamera_hostcheck.h"
#include "kamera_internal.h"
#include "kamera_packed.h"
#include "kamera_paged.h"
#include "kamera_ptx.cuh"
#include "kamera_tc.cuh"
#include "kamera_warpmma.cuh"

namespace kamera {

namespace {

using namespace tc;

constexpr int kP4Tok = 128, kP4Pieces = kP4Tok / 16;
constexpr int kP4Threads = 448, kP4Keys = 4, kP4Values = 8, kP4Prod = 12, kP4Mma = 13;   // first warps of the roles
constexpr int kP4Masks = 16;              // tiles whose masks are kept: the ring's and those behind it
// TMEM columns: two tiles' keys, a tile's values, two tiles' scores, the output
constexpr uint32_t kP4TmK = 0, kP4TmV = 128, kP4TmS = 192, kP4TmO = 224, kP4TmCols = 256;
constexpr float kP4Lazy = 8.0f;
constexpr float kP4Up = 7.0f;             // weights are 2^7 times the usual ones: at most 2^15 with the lazy growth
constexpr float kP4Log2e = 1.4426950408889634f, kP4Ln2 = 0.6931471805599453f;

template <int D, int N>
struct P4Layout {
    static constexpr uint32_t kTile = kP4Pieces * kPackedPiece<D>;
    static constexpr int NS = D == 128 ? 5 : 8;               // tiles in the ring
    static constexpr uint32_t kQ = 0;                         // [2 segments][d / 64 blocks][N rows][128 bytes]
    static constexpr uint32_t kQSeg = (D / 64) * N * 128;
    static constexpr uint32_t kP = kQ + 2 * kQSeg;            // [2 tiles][2 blocks of 64 tokens][N rows][128 bytes]
    static constexpr uint32_t kPTile = 2 * N * 128;
    static constexpr uint32_t kRing = kP + 2 * kPTile;
    static constexpr uint32_t kBar = kRing + NS * kTile;
    static constexpr uint32_t kBytes = kBar + 512 + 7 * N * 4 + 1024;   // + alignment slack
    static_assert(2 * (kBytes + 1024) <= 228 * 1024, "two CTAs an SM");
    static_assert(kRing % 128 == 0 && kTile % 128 == 0, "copies");
};

struct P4Params {
    const __nv_bfloat16* q;
    __nv_bfloat16* out;
    float* lse;                    // or null
    const unsigned char* data;     // packed pages
    const int32_t* pages;
    const int32_t* lens;           // null: max_len is 0
    float* o;                      // [2 ranges][G][d]: partial outputs
    float2* ml;                    // [2 ranges][G]
    int4* span;                    // [n_seqs * H]: first and last range, first slot
    int64_t num_pages;
    int32_t n_seqs, H, G, P, max_pages, max_len, ranges;
    float scale, k_unit, v_unit;
    // the tail's partial states: [rows][tail_slots]
    const float* tail_o;
    const float2* tail_ml;
    const int32_t* tail_lens;      // or null
    int32_t max_tail, tail_split, tail_slots;   // 16-token pieces of a split; splits (0: no tail)
    int32_t first;                 // the call's first kernel
    int32_t* err;
    uint64_t half_wait;
    int32_t withhold;
};

struct P4Bars {
    uint64_t full[8], empty[8], q_full[2], k_full[2], v_full, s_full[2], p_full[2], pv_done[2], drained;
    uint32_t mask[kP4Masks];       // tile t (mod kP4Masks): 16-token pieces that are there
    int64_t total, lo, hi;         // the batch's tiles and the range's
    int32_t first_seq, first_len, first_n, first_h, first_t;   // where the range starts
    uint32_t tiles;                // whose loads were issued
    uint32_t tmem;
    int32_t abort;
};
static_assert(sizeof(P4Bars) <= 512, "barrier block");

__device__ __forceinline__ int p4_len(const P4Params& p, int s)
{
    const int len = p.lens[s];
    return len >= 0 && len <= p.max_len ? len : 0;
}
__device__ __forceinline__ int p4_tiles(int len) { return (len + kP4Tok - 1) / kP4Tok; }
// The ranges in use.  Where each has a few tiles, as few as leave the longest as it is:
// fewer states to join (one context of 32768 tokens 16.5 -> 15.1 us a call); with many
// tiles in each all of them (32 MHA heads 56.3 us, 57.5 with fewer).
__device__ __forceinline__ int64_t p4_ranges(const P4Params& p, int64_t T)
{
    if (T <= p.ranges || T > 8ll * p.ranges)
        return min((int64_t)p.ranges, T);
    const int64_t each = wmma16::quotient(T + p.ranges - 1, p.ranges);
    return wmma16::quotient(T + each - 1, each);
}
__device__ __forceinline__ int64_t p4_start(int64_t r, int64_t T, int64_t R) { return wmma16::quotient(r * T, R); }
__device__ __forceinline__ int64_t p4_range_of(int64_t tile, int64_t T, int64_t R) { return wmma16::quotient((tile + 1) * R - 1, T); }

// A range's tiles, walked alike by every role: sequence, KV head, tile.
struct P4Walk {
    int64_t left;
    int s, h, len, n, t;
    bool fresh;
    __device__ __forceinline__ void start(const P4Bars& b)
    {
        left = b.hi - b.lo;
        s = b.first_seq;
        len = b.first_len;
        n = b.first_n;
        h = b.first_h;
        t = b.first_t;
        fresh = true;
    }
    __device__ __forceinline__ bool last() const { return t + 1 == n || left == 1; }
    // to the next segment's first tile (left 0: there is none)
    __device__ __forceinline__ void skip(const P4Params& p)
    {
        const int rest = n - 1 - t;
        if (left <= rest + 1) {
            left = 0;
            return;
        }
        left -= rest;
        t = n - 1;
        next(p);
    }
    __device__ __forceinline__ void next(const P4Params& p)
    {
        --left;
        fresh = false;
        if (++t == n && left > 0) {
            t = 0;
            fresh = true;
            if (++h == p.H) {
                h = 0;
                do {               // (a tile is left, so a sequence has one)
                    ++s;
                    len = p4_len(p, s);
                } while (len == 0);
                n = p4_tiles(len);
            }
        }
    }
};

// Total tiles and where the range starts, by one warp: one look at the lengths of up to
// 32 sequences, two at those of more.
__device__ void p4_locate(const P4Params& p, P4Bars& b, int r, int lane)
{
    auto length = [&](int s) { return s < p.n_seqs ? p4_len(p, s) : 0; };
    const int first = length(lane);
    if (p.n_seqs <= 32 && p.H <= 32) {   // one scan in 32 bits where the counts fit (one context 15.1 -> 14.9 us)
        const int n = p4_tiles(first);
        const uint64_t all = (uint64_t)n * (uint32_t)p.H;
        if (!__any_sync(0xFFFFFFFFu, all >> 26)) {
            const uint32_t mine = (uint32_t)all;
            uint32_t x = mine;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
                if (lane >= d)
                    x += y;
            }
            const uint32_t T = __shfl_sync(0xFFFFFFFFu, x, 31);
            if (lane == 0)
                b.total = T;
            const int64_t R = p4_ranges(p, T);
            if (r >= R)
                return;
            const uint32_t lo = (uint32_t)p4_start(r, T, R), before = x - mine;
            if (before <= lo && lo < x) {
                const int h = (int)((lo - before) / (uint32_t)n);
                b.first_seq = lane;
                b.first_len = first;
                b.first_n = n;
                b.first_h = h;
                b.first_t = (int)(lo - before) - h * n;
                b.lo = lo;
                b.hi = p4_start(r + 1, T, R);
            }
            return;
        }
    }
    int64_t sum = (int64_t)p4_tiles(first) * p.H;
    for (int s = lane + 32; s < p.n_seqs; s += 32)
        sum += (int64_t)p4_tiles(length(s)) * p.H;
#pragma unroll
    for (int d = 16; d >= 1; d /= 2)
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    const int64_t T = sum;
    if (lane == 0)
        b.total = T;
    const int64_t R = p4_ranges(p, T);
    if (r >= R)   // fewer tiles than ranges
        return;
    const int64_t lo = p4_start(r, T, R);
    int64_t at = 0;
    for (int s0 = 0; s0 < p.n_seqs; s0 += 32) {
        const int len = s0 == 0 ? first : length(s0 + lane), n = p4_tiles(len);
        const int64_t mine = (int64_t)n * p.H;
        int64_t x = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
            if (lane >= d)
                x += y;
        }
        const int64_t before = at + x - mine;
        if (mine > 0 && before <= lo && lo < before + mine) {
            const int h = (int)wmma16::quotient(lo - before, n);
            b.first_seq = s0 + lane;
            b.first_len = len;
            b.first_n = n;
            b.first_h = h;
            b.first_t = (int)(lo - before - (int64_t)h * n);
            b.lo = lo;
            b.hi = p4_start(r + 1, T, R);
        }
        at += __shfl_sync(0xFFFFFFFFu, x, 31);
        if (at > lo)
            break;
    }
}

// ---------------------------------------------------------------- producer --
template <int D, int N>
__device__ void p4_producer(const P4Params& p, P4Bars& b, uint32_t sbase, int lane, int64_t lo, int64_t hi)
{
    using Y = P4Layout<D, N>;
    const int ppp = p.P / 16;      // pieces of a page
    // Lane l is at piece l % 8 of tile l / 8 of four tiles, and of the four after them:
    // pages are looked up, and addresses worked out, for 32 pieces at once and four tiles
    // ahead.  (Under load a look-up takes 2000 cycles, and a tile's divisions and
    // look-ups as it came 1900: more than its decoding.)
    constexpr int kAhead = 32 / kP4Pieces;
    P4Walk mine;
    mine.start(b);
    auto advance = [&](int n) {
        if (mine.left > n && mine.t + n < mine.n) {
            mine.left -= n;
            mine.t += n;
        } else {
            for (int i = 0; i < n && mine.left > 0; ++i)
                mine.next(p);
        }
    };
    auto look_up = [&](int& page, int64_t& at) {   // page -1: no piece; at: its place in pieces, beside the page's
        page = -1;
        at = 0;
        const int piece = mine.t * kP4Pieces + lane % kP4Pieces;
        if (mine.left <= 0 || 16 * (int64_t)piece >= mine.len)
            return;
        const int slot = piece / ppp;
        at = ((int64_t)mine.h * ppp + (piece - slot * ppp)) * 2 + (mine.h == 0 ? 1 : 0);
        page = p.pages[(int64_t)mine.s * p.max_pages + slot];
        page = page < 0 ? -2 : page;
    };
    advance(lane / kP4Pieces);
    int page, page_next = -1;
    int64_t place, place_next = 0;
    look_up(page, place);
    const int64_t page_bytes = (int64_t)p.H * ppp * kPackedPiece<D>;
    const unsigned char* src = nullptr;
    bool good = false;
    uint32_t there = 0;            // the four tiles' pieces that are there
    const uint32_t n = (uint32_t)(hi - lo);
    uint32_t k = 0, at = 0, lap = 0;
    for (; k < n; ++k) {
        if (k % kAhead == 0) {
            if (k > 0) {
                page = page_next;
                place = place_next;
            }
            good = page >= 0 && page < p.num_pages;
            if (page != -1 && !good && (place & 1))   // (once, with the first head)
                raise_err(p.err, KAMERA_DEVERR_SLOT);
            src = p.data + page * page_bytes + (place >> 1) * kPackedPiece<D>;
            there = __ballot_sync(0xFFFFFFFFu, good);
        }
        const int mine_now = (int)(k % kAhead);
        const uint32_t mask = (there >> (kP4Pieces * mine_now)) & 0xFFu;
        if (lap > 0) {
            bool got = true;
            if (lane == 0)
                got = wmma16::cycle_wait(ptx::smem_addr(&b.empty[at]), (lap & 1u) ^ 1u, &b.abort, p.err, p.half_wait);
            if (!__shfl_sync(0xFFFFFFFFu, got ? 1 : 0, 0))
                break;
        }
        const uint32_t full = ptx::smem_addr(&b.full[at]);
        if (lane == 0) {
            b.mask[k % kP4Masks] = mask;
            if (!p.withhold) {
                if (mask)
                    ptx::mbar_arrive_expect_tx(full, __popc(mask) * (uint32_t)kPackedPiece<D>);
                else
                    ptx::mbar_arrive(full);
            }
        }
        __syncwarp();
        if (mask == 0xFFu && !p.withhold) {   // by one thread, its addresses at hand: eight lanes, each by itself, take 1400 cycles
            const unsigned char* from[kP4Pieces];
#pragma unroll
            for (int i = 0; i < kP4Pieces; ++i)
                from[i] = reinterpret_cast<const unsigned char*>(
                    __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(src), kP4Pieces * mine_now + i));
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < kP4Pieces; ++i)
                    ptx::bulk_g2s(sbase + Y::kRing + at * Y::kTile + i * kPackedPiece<D>, from[i], kPackedPiece<D>, full);
            }
            __syncwarp();
        } else if (lane / kP4Pieces == mine_now && good && !p.withhold)
            ptx::bulk_g2s(sbase + Y::kRing + at * Y::kTile + (lane % kP4Pieces) * kPackedPiece<D>, src, kPackedPiece<D>, full);
        if (k % kAhead == 0) {     // the four tiles after these
            advance(kAhead);
            look_up(page_next, place_next);
        }
        if (++at == (uint32_t)Y::NS) {
            at = 0;
            ++lap;
        }
    }
    if (lane == 0 && !p.withhold)
        b.tiles = k;
    __syncwarp();
}

// --------------------------------------------------------------------- MMA --
template <int D, int N>
__device__ void p4_mma(const P4Params& p, P4Bars& b, uint32_t sbase, uint32_t tm)
{
    using Y = P4Layout<D, N>;
    constexpr uint32_t id = (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24);   // fp16 x fp16 -> fp32, M 128
    const uint32_t q_lo = ((sbase + Y::kQ) >> 4) | (1u << 16), p_lo = ((sbase + Y::kP) >> 4) | (1u << 16);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return wmma16::cycle_wait(ptx::smem_addr(bar), parity & 1u, &b.abort, p.err, p.half_wait);
    };
    uint32_t seg = 0;
    auto scores = [&](uint32_t t, const P4Walk& v) -> bool {   // of tile t, whose keys are there
        if ((v.fresh && !wait(&b.q_full[seg & 1u], seg >> 1)) || !wait(&b.k_full[t & 1u], t >> 1))
            return false;
        ptx::tc_fence_after();
        const uint32_t d = tm + kP4TmS + (t & 1u) * 16, k = tm + kP4TmK + (t & 1u) * 64;
        const uint32_t q = q_lo + (seg & 1u) * (Y::kQSeg >> 4);
        mma_ts<false>(d, k, q, id);
#pragma unroll
        for (int ks = 1; ks < D / 16; ++ks)
            mma_ts<true>(d, k + 8 * ks, q + (ks >> 2) * (N * 128 >> 4) + 2 * (ks & 3), id);
        ptx::umma_commit(ptx::smem_addr(&b.s_full[t & 1u]));
        seg += v.last() ? 1u : 0u;
        return true;
    };
    P4Walk w;
    w.start(b);
    bool ok = w.left <= 0 || scores(0, w);
    for (uint32_t t = 0; ok && w.left > 0; ++t) {
        const bool fresh = w.fresh;
        w.next(p);
        if (!(ok = w.left <= 0 || scores(t + 1, w)) || !(ok = wait(&b.v_full, t) && wait(&b.p_full[t & 1u], t >> 1)))
            break;
        ptx::tc_fence_after();
        const uint32_t pt = p_lo + (t & 1u) * (Y::kPTile >> 4);
        if (fresh)
            mma_ts<false>(tm + kP4TmO, tm + kP4TmV, pt, id);
        else
            mma_ts<true>(tm + kP4TmO, tm + kP4TmV, pt, id);
#pragma unroll
        for (int ks = 1; ks < kP4Tok / 16; ++ks)
            mma_ts<true>(tm + kP4TmO, tm + kP4TmV + 8 * ks, pt + (ks >> 2) * (N * 128 >> 4) + 2 * (ks & 3), id);
        ptx::umma_commit(ptx::smem_addr(&b.pv_done[t & 1u]));
    }
    // every MMA issued here completes before TMEM is freed
    ptx::umma_commit(ptx::smem_addr(&b.drained));
    pf_drain_wait(ptx::smem_addr(&b.drained), 0u);
}

// ------------------------------------------------------------------ values --
__device__ __forceinline__ void decode_word(uint32_t codes, uint32_t scale2, uint32_t* out)
{
    out[0] = mul_f16x2(e2m1_pair<0>(codes), scale2);
    out[1] = mul_f16x2(e2m1_pair<1>(codes), scale2);
    out[2] = mul_f16x2(e2m1_pair<2>(codes), scale2);
    out[3] = mul_f16x2(e2m1_pair<3>(codes), scale2);
}

// Thread = channel c: the tile's 128 tokens into the columns of its TMEM lane.
template <int D, int N>
__device__ void p4_values(const P4Params& p, P4Bars& b, const unsigned char* ring, uint32_t tm, int warp, int lane, int64_t n)
{
    using Y = P4Layout<D, N>;
    const int c = 32 * warp + lane;
    const uint32_t tV = tm + ((uint32_t)warp << 21) + kP4TmV;
    bool ok = true;
    for (uint32_t t = 0; t < n; ++t) {
        const uint32_t at = t % Y::NS;
        ok = wmma16::cycle_wait(ptx::smem_addr(&b.full[at]), (t / Y::NS) & 1u, &b.abort, p.err, p.half_wait);
        if (!__all_sync(0xFFFFFFFFu, ok))
            return;
        const unsigned char* tile = ring + at * Y::kTile;
        const uint32_t mask = *reinterpret_cast<volatile uint32_t*>(&b.mask[t % kP4Masks]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {   // four pieces, 32 columns
            uint32_t v[32];
            if (c < D) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int piece = 4 * half + i;
                    const unsigned char* rec = tile + piece * kPackedPiece<D>;
                    const uint2 codes = *reinterpret_cast<const uint2*>(rec + kPackedV<D> + 8 * c);
                    uint32_t s = rec[kPackedVS<D> + c] * 0x00800080u;
                    if (mask != 0xFFu && !((mask >> piece) & 1u))
                        s = 0u;   // a piece that is not there: zero, so that zero weights add nothing
                    decode_word(codes.x, s, v + 8 * i);
                    decode_word(codes.y, s, v + 8 * i + 4);
                }
            }
            if (half == 0 && t > 0) {   // the product before has read the last tile's values
                ok = wmma16::cycle_wait(ptx::smem_addr(&b.pv_done[(t - 1) & 1u]), ((t - 1) >> 1) & 1u, &b.abort, p.err, p.half_wait);
                if (!__all_sync(0xFFFFFFFFu, ok))
                    return;
                ptx::tc_fence_after();
            }
            if (32 * warp < D)
                tmem_st32(tV + 32 * half, v);
        }
        ptx::mbar_arrive(ptx::smem_addr(&b.empty[at]));
        tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_addr(&b.v_full));
    }
}

// -------------------------------------------------------- keys, softmax --
__device__ __forceinline__ void p4_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The four warps meet; whether any thread said yes.
__device__ __forceinline__ bool p4_any(bool x)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 2, 128, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(x ? 1u : 0u)
                 : "memory");
    return r != 0;
}

// 16 lanes of a warp's quarter, N columns: register 4 j + 2 r + c is lane l / 4 + 8 r,
// column 8 j + 2 (l % 4) + c.  Issue only.
template <int N>
__device__ __forceinline__ void p4_ld_scores(uint32_t ta, uint32_t* r)
{
    if constexpr (N == 8)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(ta)
                     : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(ta)
                     : "memory");
}

template <int N>
__device__ __forceinline__ void p4_ld_out(uint32_t ta, uint32_t (&r)[N])
{
    if constexpr (N == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(ta)
                     : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
                     "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                       "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                       "=r"(r[15])
                     : "r"(ta)
                     : "memory");
}
template <int N>
__device__ __forceinline__ void p4_st_out(uint32_t ta, const uint32_t (&r)[N])
{
    if constexpr (N == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(ta), "r"(r[0]),
                     "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    else
        tmem_st16(ta, r);
}

__device__ __forceinline__ void p4_stsm_x4_t(uint32_t a, const uint32_t (&x)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x[0]), "r"(x[1]),
                 "r"(x[2]), "r"(x[3])
                 : "memory");
}

// The query heads of (sequence, KV head) as the B operand: fp16, each row times a power
// of two that takes its largest entry to [2^10, 2^11); what a score is to be multiplied
// with (log2 units) into fs.  Rows past the heads are zero.
template <int D, int N>
__device__ __forceinline__ void p4_stage_q(const P4Params& p, uint32_t q_smem, float* fs, int s, int h, int warp, int lane)
{
    constexpr int V = D / 32;      // channels of a lane
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const int r = 4 * i + warp;
        float x[V];
        float amax = 0.f;
        const __nv_bfloat16* src = p.q + (((int64_t)s * p.H + h) * p.G + r) * D + V * lane;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            x[j] = r < p.G ? __bfloat162float(src[j]) : 0.f;
            amax = fmaxf(amax, fabsf(x[j]));
        }
#pragma unroll
        for (int d = 16; d >= 1; d /= 2)
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
        // exponent of the largest entry; not below -100 (a row that small has few bits left), not above 127
        const int e = max((int)(__float_as_uint(amax) >> 23) - 127, -100), ec = min(e, 127);
        const float up = __uint_as_float((uint32_t)(127 + 10 - ec) << 23);   // 2^(10 - e), e in -100 .. 127
        if (lane == 0)   // K is held at 2^-8 of its value
            fs[r] = p.scale * kP4Log2e * p.k_unit * (__uint_as_float((uint32_t)(127 + ec) << 23) * 0.25f);
        const int ch = V * lane;
        const uint32_t dst = q_smem + (ch >> 6) * (N * 128) + (r >> 3) * 1024 + sw128(r & 7, (ch & 63) >> 3) +
                             (ch & 7) * 2;
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const __half2 y = __floats2half2_rn(x[j] * up, x[j + 1] * up);
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + 2 * j), "r"(*reinterpret_cast<const uint32_t*>(&y)) : "memory");
        }
    }
}

// Thread = token of the tile: its keys into the columns of its TMEM lane.
template <int D, int N>
__device__ void p4_keys(const P4Params& p, P4Bars& b, const unsigned char* ring, uint32_t tm, int warp, int lane, int64_t n)
{
    using Y = P4Layout<D, N>;
    const int tok = 32 * warp + lane;
    const uint32_t tK = tm + ((uint32_t)warp << 21) + kP4TmK;
    for (uint32_t t = 0; t < n; ++t) {
        const uint32_t at = t % Y::NS;
        bool ok = wmma16::cycle_wait(ptx::smem_addr(&b.full[at]), (t / Y::NS) & 1u, &b.abort, p.err, p.half_wait);
        if (t >= 2)   // the keys of two tiles before have been scored
            ok = ok && wmma16::cycle_wait(ptx::smem_addr(&b.s_full[t & 1u]), ((t >> 1) - 1) & 1u, &b.abort, p.err, p.half_wait);
        if (!__all_sync(0xFFFFFFFFu, ok))
            return;
        ptx::tc_fence_after();
        const unsigned char* rec = ring + at * Y::kTile + (tok >> 4) * kPackedPiece<D>;
        uint32_t sc[D / 64];
        const unsigned char* ss = rec + kPackedKS<D> + (tok & 15) * (D / 16);
        if constexpr (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(ss);
            sc[0] = x.x, sc[1] = x.y;
        } else {
            sc[0] = *reinterpret_cast<const uint32_t*>(ss);
        }
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {   // 64 channels, 32 columns
            uint32_t x[32];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint4 c = *reinterpret_cast<const uint4*>(rec + (2 * half + j) * 256 + (tok & 15) * 16);
                const uint32_t s0 = ((sc[half] >> (16 * j)) & 0xFFu) * 0x00800080u;
                const uint32_t s1 = ((sc[half] >> (16 * j + 8)) & 0xFFu) * 0x00800080u;
                decode_word(c.x, s0, x + 16 * j);
                decode_word(c.y, s0, x + 16 * j + 4);
                decode_word(c.z, s1, x + 16 * j + 8);
                decode_word(c.w, s1, x + 16 * j + 12);
            }
            tmem_st32(tK + (t & 1u) * 64 + 32 * half, x);
        }
        ptx::mbar_arrive(ptx::smem_addr(&b.empty[at]));
        tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_addr(&b.k_full[t & 1u]));
    }
}

template <int D, int N>
__device__ void p4_softmax(const P4Params& p, P4Bars& b, uint32_t sbase, float* ex, uint32_t tm, int warp, int lane,
                           int range, int64_t lo, int64_t hi)
{
    using Y = P4Layout<D, N>;
    constexpr int J = N / 8;
    const int gq = lane >> 2, t4 = lane & 3, tok = 32 * warp + lane;
    const uint32_t lanes = tm + ((uint32_t)warp << 21);
    const int64_t T = b.total, R = p4_ranges(p, T);
    float* wmax = ex;              // [4 warps][N]
    float* fac = ex + 4 * N;       // [N]
    float* fs = ex + 5 * N;        // [2 segments][N]: scores' factors
    float m[J][2], l[J][2], f2[J][2];
    const uint32_t st = sbase + Y::kP + (warp >> 1) * (N * 128) + sw128(lane & 7, 4 * (warp & 1) + (lane >> 3));
    bool ok = true;
    uint32_t seg = 0;              // segments whose queries are staged
    // Segment i's queries, staged as segment i - 1 starts: what stood there, of segment
    // i - 2, has been scored.
    auto stage = [&](const P4Walk& v) {
        p4_stage_q<D, N>(p, sbase + Y::kQ + (seg & 1u) * Y::kQSeg, fs + (seg & 1u) * N, v.s, v.h, warp, lane);
        ptx::fence_proxy_async();
        ptx::mbar_arrive(ptx::smem_addr(&b.q_full[seg & 1u]));
        ++seg;
    };
    P4Walk w;
    w.start(b);
    if (w.left > 0)
        stage(w);
    p4_sync();
    int64_t at_tile = lo;
    for (uint32_t t = 0; w.left > 0; ++t, ++at_tile) {
        if (w.fresh) {
            const float* from = fs + ((seg - 1) & 1u) * N;   // (a barrier lies behind their staging)
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    m[j][c] = -INFINITY;
                    l[j][c] = 0.f;
                    f2[j][c] = from[8 * j + 2 * t4 + c];
                }
            P4Walk next = w;
            next.skip(p);
            if (next.left > 0)
                stage(next);
        }
        ok = ok && wmma16::cycle_wait(ptx::smem_addr(&b.s_full[t & 1u]), (t >> 1) & 1u, &b.abort, p.err, p.half_wait);
        ok = __all_sync(0xFFFFFFFFu, ok);
        const uint32_t mask = *reinterpret_cast<volatile uint32_t*>(&b.mask[t % kP4Masks]);
        const int ntok = min(kP4Tok, w.len - w.t * kP4Tok);
        bool grew = false;
        float x[2][J][4];   // half of the warp's tokens; [j][2 r + c]
        if (ok) {
            ptx::tc_fence_after();
            uint32_t s[2][4 * J];
            p4_ld_scores<N>(lanes + kP4TmS + (t & 1u) * 16, s[0]);
            p4_ld_scores<N>(lanes + kP4TmS + (t & 1u) * 16 + (16u << 16), s[1]);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4 * J; ++j)
                    asm volatile("" : "+r"(s[i][j]));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool here = (mask >> (2 * warp + i)) & 1u;
                const int t0 = 32 * warp + 16 * i + gq;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const bool in = here && t0 + 8 * r < ntok;
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            x[i][j][2 * r + c] = in ? __uint_as_float(s[i][4 * j + 2 * r + c]) * f2[j][c] : -INFINITY;
                            grew |= x[i][j][2 * r + c] > m[j][c] + kP4Lazy;
                        }
                }
            }
        }
        if (p4_any(grew || !ok)) {   // rare but for a segment's first tile
            if (p4_any(!ok))
                return;              // all four warps
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v = fmaxf(fmaxf(x[0][j][c], x[0][j][2 + c]), fmaxf(x[1][j][c], x[1][j][2 + c]));
                    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
                    if (gq == 0)
                        wmax[warp * N + 8 * j + 2 * t4 + c] = v;
                }
            p4_sync();
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int h = 8 * j + 2 * t4 + c;
                    float v = m[j][c];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v = fmaxf(v, wmax[k * N + h]);
                    const float f = v == -INFINITY ? 1.f : pf_ex2(m[j][c] - v);
                    l[j][c] *= f;
                    m[j][c] = v;
                    if (warp == 0 && gq == 0)
                        fac[h] = f;
                }
            if (!w.fresh) {          // the running output, once the products before are in it
                ok = wmma16::cycle_wait(ptx::smem_addr(&b.pv_done[(t - 1) & 1u]), ((t - 1) >> 1) & 1u, &b.abort, p.err, p.half_wait);
                ok = __all_sync(0xFFFFFFFFu, ok);
                ptx::tc_fence_after();
                p4_sync();
                uint32_t o[N];
                p4_ld_out<N>(lanes + kP4TmO, o);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    o[i] = __float_as_uint(__uint_as_float(o[i]) * fac[i]);
                p4_st_out<N>(lanes + kP4TmO, o);
                tmem_wait_st();
            }
            p4_sync();               // the exchange's arrays are free again
        }
        // weights, transposed into the operand rows (heads) of the second product
        uint32_t pk[J][4];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const float m0 = m[j][0] == -INFINITY ? 0.f : m[j][0] - kP4Up, m1 = m[j][1] == -INFINITY ? 0.f : m[j][1] - kP4Up;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float a = pf_ex2(x[k >> 1][j][2 * (k & 1)] - m0), c = pf_ex2(x[k >> 1][j][2 * (k & 1) + 1] - m1);
                l[j][0] += a;
                l[j][1] += c;
                const __half2 y = __floats2half2_rn(a, c);
                pk[j][k] = *reinterpret_cast<const uint32_t*>(&y);
            }
        }
        if (t > 1) {                 // the weights of two tiles before have been read
            ok = ok && wmma16::cycle_wait(ptx::smem_addr(&b.pv_done[t & 1u]), ((t >> 1) - 1) & 1u, &b.abort, p.err, p.half_wait);
            ok = __all_sync(0xFFFFFFFFu, ok);
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
            p4_stsm_x4_t(st + (t & 1u) * Y::kPTile + j * 1024, pk[j]);
        ptx::fence_proxy_async();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0)
            ptx::mbar_arrive(ptx::smem_addr(&b.p_full[t & 1u]));
        if (!w.last()) {
            w.next(p);
            continue;
        }
        // ---- the segment's end: its partial state
        const int64_t a0 = at_tile - w.t, r0 = p4_range_of(a0, T, R), r1 = p4_range_of(a0 + w.n - 1, T, R);
        const int first_slot = (int)(2 * r0 + (p4_start(r0, T, R) == a0 ? 0 : 1));
        const int unit = w.s * p.H + w.h;
        // a unit inside one range leaves its state at the unit's own place
        const int64_t part = r0 == r1 ? 2 * (int64_t)p.ranges + unit : range == r0 ? first_slot : 2 * range;
        if (range == r0 && threadIdx.x == 0)
            p.span[unit] = make_int4((int)r0, (int)r1, first_slot, 0);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                l[j][c] += __shfl_xor_sync(0xFFFFFFFFu, l[j][c], 4);
                l[j][c] += __shfl_xor_sync(0xFFFFFFFFu, l[j][c], 8);
                l[j][c] += __shfl_xor_sync(0xFFFFFFFFu, l[j][c], 16);
                if (gq == 0)
                    wmax[warp * N + 8 * j + 2 * t4 + c] = l[j][c];
            }
        p4_sync();
        if (warp == 0 && gq == 0) {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int h = 8 * j + 2 * t4 + c;
                    if (h < p.G)
                        p.ml[part * p.G + h] = make_float2(m[j][c] - kP4Up, (wmax[h] + wmax[N + h]) +
                                                                                (wmax[2 * N + h] + wmax[3 * N + h]));
                }
        }
        ok = ok && wmma16::cycle_wait(ptx::smem_addr(&b.pv_done[t & 1u]), (t >> 1) & 1u, &b.abort, p.err, p.half_wait);
        ok = __all_sync(0xFFFFFFFFu, ok);
        ptx::tc_fence_after();
        uint32_t o[N];
        p4_ld_out<N>(lanes + kP4TmO, o);
        const float up = p.v_unit * 256.f;   // V is held at 2^-8 of its value
        if (ok && tok < D) {
#pragma unroll
            for (int h = 0; h < N; ++h)
                if (h < p.G)
                    p.o[(part * p.G + h) * D + tok] = __uint_as_float(o[h]) * up;
        }
        ptx::tc_fence_before();
        p4_sync();   // the exchange's arrays are free for the next segment
        w.next(p);
    }
}

template <int D, int N>
__global__ void __launch_bounds__(kP4Threads, 2) packed_kernel(const P4Params p)
{
    using Y = P4Layout<D, N>;
    extern __shared__ __align__(16) unsigned char raw[];
    const uint32_t addr = ptx::smem_addr(raw), pad = (1024u - (addr & 1023u)) & 1023u, sbase = addr + pad;
    P4Bars& b = *reinterpret_cast<P4Bars*>(raw + pad + Y::kBar);
    float* ex = reinterpret_cast<float*>(raw + pad + Y::kBar + 512);
    const unsigned char* ring = raw + pad + Y::kRing;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, range = blockIdx.x;
    if (threadIdx.x == 0) {
        for (int i = 0; i < Y::NS; ++i) {
            ptx::mbar_init(ptx::smem_addr(&b.full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.empty[i]), 256);
        }
        ptx::mbar_init(ptx::smem_addr(&b.v_full), 128);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_addr(&b.q_full[i]), 128);
            ptx::mbar_init(ptx::smem_addr(&b.k_full[i]), 128);
            ptx::mbar_init(ptx::smem_addr(&b.s_full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.p_full[i]), 4);
            ptx::mbar_init(ptx::smem_addr(&b.pv_done[i]), 1);
        }
        ptx::mbar_init(ptx::smem_addr(&b.drained), 1);
        b.abort = 0;
        b.tiles = 0;
        ptx::fence_barrier_init();
    }
    if (warp == kP4Mma) {
        ptx::tmem_alloc(ptx::smem_addr(&b.tmem), kP4TmCols);
        ptx::tmem_relinquish();
    }
    if (p.first)   // behind the tail's kernel the call's inputs are there already
        ptx::grid_wait();
    if (warp == 0)
        p4_locate(p, b, range, lane);
    if (blockIdx.x == 0 && warp > 0)
        for (int s = threadIdx.x - 32; s < p.n_seqs; s += kP4Threads - 32)
            if (p.lens[s] < 0 || p.lens[s] > p.max_len)
                raise_err(p.err, KAMERA_DEVERR_LEN);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    ptx::grid_launch_next();   // (this CTA has its TMEM: none that starts early can take it)
    const uint32_t tm = b.tmem;
    const int64_t T = b.total, R = p4_ranges(p, T);
    if (range < R) {   // (else: fewer tiles than ranges)
        const int64_t lo = b.lo, hi = b.hi;
        if (warp < kP4Keys)
            p4_softmax<D, N>(p, b, sbase, ex, tm, warp, lane, range, lo, hi);
        else if (warp < kP4Values)
            p4_keys<D, N>(p, b, ring, tm, warp - kP4Keys, lane, hi - lo);
        else if (warp < kP4Prod)
            p4_values<D, N>(p, b, ring, tm, warp - kP4Values, lane, hi - lo);
        else if (warp == kP4Prod)
            p4_producer<D, N>(p, b, sbase, lane, lo, hi);
        else if (elect_one())
            p4_mma<D, N>(p, b, sbase, tm);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kP4Mma) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tm, kP4TmCols);
    }
    // After a timeout the copies that the CTA started land before it leaves.  (Without one
    // every fill has been waited for.)
    if (threadIdx.x == 32 * kP4Prod && b.abort)
        pf_drain_ring(b.full, b.tiles, Y::NS);
    // The merge that follows waits for this grid alone, which ends after the tail's.
    if (!p.first && blockIdx.x == gridDim.x - 1)
        ptx::grid_wait();
}

// ------------------------------------------------------------------- merge --
// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over a row's packed and tail
// states.  All latency: a CTA a row, warp w takes every NW-th state; a warp's outputs
// are asked for eight at a time before their weights are known, and the lanes work out
// the weights of 32 states at once; the warps' sums join in order.  16 warps where a row
// may have many states (77 of 28 rows: 6 us less than with four), four where the rows
// are many.
template <int D, int NW>
__global__ void __launch_bounds__(32 * NW) packed_merge_kernel(const P4Params p)
{
    constexpr int V = D / 32, PW = 8, SW = NW / 4;   // a round: eight states a warp, SW a lane
    __shared__ float part[NW][D];
    __shared__ float sum;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x, unit = row / p.G, g = row - unit * p.G, s = unit / p.H;
    // what the call was given, while the kernels before may still run
    int n_tail = 0;
    if (p.tail_slots > 0) {
        const int len = p.tail_lens[s];
        n_tail = len > 0 && len <= p.max_tail ? ((len + 15) / 16 + p.tail_split - 1) / p.tail_split : 0;
    }
    const bool some = p.max_len > 0 && p4_len(p, s) > 0;
    ptx::grid_wait();
    ptx::grid_launch_next();
    if (threadIdx.x == 0 && g == 0 && unit == s * p.H &&   // a bound of no tokens: no other kernel looks at the lengths
        ((p.max_len == 0 && p.lens && p.lens[s] != 0) || (p.tail_slots == 0 && p.tail_lens && p.tail_lens[s] != 0)))
        raise_err(p.err, KAMERA_DEVERR_LEN);
    int n_packed = 0;
    int4 sp = make_int4(0, 0, 0, 0);
    if (some) {
        sp = p.span[unit];
        // (after a timeout it may never have been written)
        if (sp.x >= 0 && sp.y >= sp.x && sp.y < p.ranges && (sp.z >> 1) == sp.x)
            n_packed = sp.y - sp.x + 1;
    }
    const int n = n_packed + n_tail;
    auto at = [&](int i) -> int64_t {
        if (i >= n_packed)
            return (int64_t)row * p.tail_slots + i - n_packed;
        return (sp.x == sp.y ? 2 * (int64_t)p.ranges + unit : i == 0 ? sp.z : 2 * (sp.x + i)) * p.G + g;
    };
    float x[PW][V];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < PW; ++k) {
            const int i = i0 + NW * k + warp;
            if (i >= n)
                continue;
            const float* src = (i < n_packed ? p.o : p.tail_o) + at(i) * D + V * lane;
            if constexpr (V == 4) {
                const float4 y = *reinterpret_cast<const float4*>(src);
                x[k][0] = y.x, x[k][1] = y.y, x[k][2] = y.z, x[k][3] = y.w;
            } else {
                const float2 y = *reinterpret_cast<const float2*>(src);
                x[k][0] = y.x, x[k][1] = y.y;
            }
        }
    };
    load(0);
    float m = -INFINITY;
    for (int i = lane; i < n; i += 32)
        m = fmaxf(m, (i < n_packed ? p.ml : p.tail_ml)[at(i)].x);
#pragma unroll
    for (int d = 16; d >= 1; d /= 2)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    float l = 0.f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        acc[v] = 0.f;
    for (int i0 = 0; i0 < n; i0 += PW * NW) {
        if (i0 > 0)
            load(i0);
        float f[SW];   // lane's states i0 + 32 c + lane; one without weight adds nothing (and has no maximum to scale by)
        uint32_t any[SW];
#pragma unroll
        for (int c = 0; c < SW; ++c) {
            const int i = i0 + 32 * c + lane;
            f[c] = 0.f;
            bool live = false;
            if (i < n) {
                const float2 y = (i < n_packed ? p.ml : p.tail_ml)[at(i)];
                live = y.y != 0.f;
                if (live) {
                    f[c] = pf_ex2(y.x - m);
                    l = fmaf(y.y, f[c], l);
                }
            }
            any[c] = __ballot_sync(0xFFFFFFFFu, live);
        }
#pragma unroll
        for (int k = 0; k < PW; ++k) {
            const int j = NW * k + warp;   // of the round's states
            const int c = (NW * k) / 32;
            const float y = __shfl_sync(0xFFFFFFFFu, f[c], j & 31);
            if ((any[c] >> (j & 31)) & 1u)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    acc[v] = fmaf(x[k][v], y, acc[v]);
        }
    }
    if (warp == 0) {
#pragma unroll
        for (int d = 16; d >= 1; d /= 2)
            l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
        if (lane == 0)
            sum = l;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        part[warp][V * lane + v] = acc[v];
    __syncthreads();
    l = sum;
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    for (int i = 2 * threadIdx.x; i < D; i += 64 * NW) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            a += part[w][i];
            b += part[w][i + 1];
        }
        *reinterpret_cast<uint32_t*>(p.out + (int64_t)row * D + i) = pack_bf16x2(a * inv, b * inv);
    }
    if (threadIdx.x == 0 && p.lse)
        p.lse[row] = l > 0.f ? (m + log2f(l)) * kP4Ln2 : (l == l ? -INFINITY : l);
}

// -------------------------------------------------------------------- host --
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct P4Plan {
    P4Params p;
    PagedParams tail;
    bool has_tail;
    size_t o, ml, span, tail_o, tail_ml;
    size_t bytes() const { return o + ml + span + tail_o + tail_ml; }
};

int p4_plan(const KameraPackedPool* pk, const KameraPagedQuery* q, const KameraPageTable* t, const KameraPagedKV* kv,
            const KameraPageTable* tail, P4Plan* x)
{
    const int rc = check_packed(pk);
    if (rc == KAMERA_ERR_INVALID_ARGUMENT)
        return rc;
    if (!q || !t || q->reserved != 0 || q->n_seqs < 0 || q->num_q_heads < 1 || q->num_q_heads % pk->num_kv_heads ||
        !(q->scale == q->scale) || t->max_len < 0 || t->max_pages < 0 || (kv == nullptr) != (tail == nullptr))
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (kv && (kv->num_kv_heads != pk->num_kv_heads || kv->head_dim != pk->head_dim))
        return KAMERA_ERR_INVALID_ARGUMENT;
    const int G = q->num_q_heads / pk->num_kv_heads;
    if (rc || G > 16 || (int64_t)q->n_seqs * pk->num_kv_heads > 65535 ||
        (int64_t)q->n_seqs * q->num_q_heads > 0x3FFFFFF || t->max_len > 0x7FFFFF00)
        return KAMERA_ERR_UNSUPPORTED;
    if ((int64_t)t->max_pages * pk->page_size < t->max_len)
        return KAMERA_ERR_INVALID_ARGUMENT;
    std::memset(x, 0, sizeof(*x));
    P4Params& p = x->p;
    p.n_seqs = q->n_seqs;
    p.H = pk->num_kv_heads;
    p.G = G;
    p.P = pk->page_size;
    p.num_pages = pk->num_pages;
    p.max_pages = t->max_pages;
    p.max_len = t->max_len;
    p.scale = q->scale;
    p.k_unit = pk->k_unit;
    p.v_unit = pk->v_unit;
    if (kv) {
        const int e = plan_own_pages(kv, q, tail, &x->tail);
        if (e)
            return e;
        x->has_tail = q->n_seqs > 0 && x->tail.own_slots > 0;
    }
    if (q->n_seqs == 0)
        return KAMERA_OK;
    const int64_t units = (int64_t)p.n_seqs * p.H, rows = units * G;
    const int64_t most = units * (((int64_t)p.max_len + kP4Tok - 1) / kP4Tok);
    p.ranges = (int32_t)std::min<int64_t>(2ll * device_sms(), most);
    if (p.ranges > 0) {
        const size_t slots = (size_t)(2 * p.ranges + units) * G;
        x->o = up256(slots * pk->head_dim * 4);
        x->ml = up256(slots * 8);
        x->span = up256((size_t)units * 16);
    }
    if (x->has_tail) {
        p.tail_split = x->tail.own_split;
        p.tail_slots = x->tail.own_slots;
        p.max_tail = tail->max_len;
        x->tail_o = up256((size_t)rows * p.tail_slots * pk->head_dim * 4);
        x->tail_ml = up256((size_t)rows * p.tail_slots * 8);
    }
    return KAMERA_OK;
}

template <int D, int N>
cudaError_t p4_launch(const P4Params& p, cudaStream_t stream)
{
    using Y = P4Layout<D, N>;
    // set at every launch: the attribute belongs to the current device's context
    const cudaError_t e = cudaFuncSetAttribute(packed_kernel<D, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Y::kBytes);
    if (e != cudaSuccess)
        return e;
    return launch_after(packed_kernel<D, N>, dim3((unsigned)p.ranges), kP4Threads, Y::kBytes, stream, true, p);
}

}  // namespace

}  // namespace kamera

using namespace kamera;

extern "C" {

size_t kamera_attend_packed_workspace_bytes(const KameraPackedPool* packed, const KameraPagedQuery* query,
                                            const KameraPageTable* table, const KameraPagedKV* tail_kv,
                                            const KameraPageTable* tail)
{
    P4Plan x;
    return p4_plan(packed, query, table, tail_kv, tail, &x) == KAMERA_OK && x.p.n_seqs > 0 ? x.bytes() : 0;
}

int kamera_attend_packed(const KameraPackedPool* packed, const KameraPagedQuery* query, const KameraPageTable* table,
                         const KameraPagedKV* tail_kv, const KameraPageTable* tail, void* d_workspace,
                         size_t workspace_bytes, int32_t* d_err, struct CUstream_st* stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    P4Plan x;
    const int rc = p4_plan(packed, query, table, tail_kv, tail, &x);
    if (rc || x.p.n_seqs == 0)
        return rc;
    P4Params& p = x.p;
    const int d = packed->head_dim;
    const int64_t rows = (int64_t)p.n_seqs * p.H * p.G, W = (int64_t)p.H * d;
    if (!query->q || !query->out || (p.ranges > 0 && (!packed->data || !table->pages || !table->lens)) ||
        (x.has_tail && (!tail->pages || !tail->lens)) || (x.bytes() > 0 && !d_workspace))
        return KAMERA_ERR_INVALID_ARGUMENT;
    int e;
    if (x.has_tail && ((e = check_strided(tail_kv->k, 1, 0, tail_kv->num_slots, tail_kv->slot_stride, W, false)) ||
                       (e = check_strided(tail_kv->v, 1, 0, tail_kv->num_slots, tail_kv->slot_stride, W, false))))
        return e;
    const int32_t* tail_lens = tail ? tail->lens : nullptr;
    const uintptr_t ints = (p.ranges > 0 ? reinterpret_cast<uintptr_t>(table->pages) : 0) | reinterpret_cast<uintptr_t>(table->lens) |
                           (x.has_tail ? reinterpret_cast<uintptr_t>(tail->pages) : 0) | reinterpret_cast<uintptr_t>(tail_lens);
    if (!aligned16(query->q) || !aligned16(query->out) || !aligned16(packed->data) || !aligned16(d_workspace) ||
        ((reinterpret_cast<uintptr_t>(query->lse) | ints) & 3))
        return KAMERA_ERR_MISALIGNED;
    if (workspace_bytes < x.bytes())
        return KAMERA_ERR_INVALID_ARGUMENT;
    using Span = std::pair<uintptr_t, uintptr_t>;
    auto bytes = [](const void* a, int64_t n) -> Span {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(a);
        return {lo, a && n > 0 ? lo + (uintptr_t)n : lo};
    };
    const Span in[] = {bytes(query->q, rows * d * 2),
                       bytes(packed->data, p.ranges > 0 ? packed_bytes(packed) : 0),
                       bytes(table->pages, p.ranges > 0 ? (int64_t)p.n_seqs * p.max_pages * 4 : 0),
                       bytes(table->lens, (int64_t)p.n_seqs * 4),
                       x.has_tail ? span(tail_kv->k, 1, 0, tail_kv->num_slots, tail_kv->slot_stride, W) : Span{0, 0},
                       x.has_tail ? span(tail_kv->v, 1, 0, tail_kv->num_slots, tail_kv->slot_stride, W) : Span{0, 0},
                       x.has_tail ? bytes(tail->pages, (int64_t)p.n_seqs * tail->max_pages * 4) : Span{0, 0},
                       bytes(tail_lens, (int64_t)p.n_seqs * 4)};
    const Span outs[] = {bytes(query->out, rows * d * 2), bytes(query->lse, rows * 4),
                         bytes(d_workspace, (int64_t)x.bytes())};
    for (int i = 0; i < 3; ++i) {
        for (const Span& a : in)
            if (overlap(a, outs[i]))
                return KAMERA_ERR_INVALID_ARGUMENT;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j]))
                return KAMERA_ERR_INVALID_ARGUMENT;
    }
    p.q = static_cast<const __nv_bfloat16*>(query->q);
    p.out = static_cast<__nv_bfloat16*>(query->out);
    p.lse = query->lse;
    p.data = static_cast<const unsigned char*>(packed->data);
    p.pages = table->pages;
    p.lens = table->lens;
    p.tail_lens = tail_lens;
    unsigned char* ws = static_cast<unsigned char*>(d_workspace);
    p.o = reinterpret_cast<float*>(ws);
    p.ml = reinterpret_cast<float2*>(ws + x.o);
    p.span = reinterpret_cast<int4*>(ws + x.o + x.ml);
    p.err = d_err;
    p.half_wait = half_wait(wait_limit_ns());
    p.withhold = test_withhold_loads() ? 1 : 0;
    p.first = x.has_tail ? 0 : 1;
    // The tail's kernel first: short, and the packed one's CTAs start beside it.
    if (x.has_tail) {
        PagedParams& t = x.tail;
        t.q = p.q;
        t.out = p.out;
        t.pages = tail->pages;
        t.lens = tail->lens;
        t.o = reinterpret_cast<float*>(ws + x.o + x.ml + x.span);
        t.ml = reinterpret_cast<float2*>(ws + x.o + x.ml + x.span + x.tail_o);
        t.err = d_err;
        t.wait_ns = wait_limit_ns();
        t.withhold = p.withhold;
        p.tail_o = t.o;
        p.tail_ml = t.ml;
        if (launch_own_pages(t, tail_kv, stream) != cudaSuccess)
            return KAMERA_ERR_CUDA;
    }
    cudaError_t ce = cudaSuccess;
    if (p.ranges > 0) {
        const bool few = p.G <= 8;
        if (d == 128)
            ce = few ? p4_launch<128, 8>(p, stream) : p4_launch<128, 16>(p, stream);
        else
            ce = few ? p4_launch<64, 8>(p, stream) : p4_launch<64, 16>(p, stream);
        if (ce != cudaSuccess)
            return KAMERA_ERR_CUDA;
    }
    const dim3 grid((unsigned)rows);
    const bool many = p.ranges >= 8ll * p.n_seqs * p.H;   // states of a row on average: a range ends in each but the last
    if (d == 128)
        ce = many ? launch_after(packed_merge_kernel<128, 16>, grid, 512, 0, stream, true, p)
                  : launch_after(packed_merge_kernel<128, 4>, grid, 128, 0, stream, true, p);
    else
        ce = many ? launch_after(packed_merge_kernel<64, 16>, grid, 512, 0, stream, true, p)
                  : launch_after(packed_merge_kernel<64, 4>, grid, 128, 0, stream, true, p);
    return ce == cudaSuccess ? KAMERA_OK : KAMERA_ERR_CUDA;
}

}  // extern "C"
