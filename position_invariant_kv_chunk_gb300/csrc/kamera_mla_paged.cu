// kamera_mla_paged.cu -- MLA decode attention over the paged pool (absorbed form), on
// the tensor cores.
//
// All query heads share one latent row a token, so a step reads 1152 bytes a token for
// 2 H (576 + 512) flops: 30 flops a byte with 16 heads, 242 with 128.  Warp-level MMAs
// (about 256 multiplies a cycle and SM) cannot do the first at the speed of HBM; the
// 5th-generation ones can if few heads do not cost what 128 would:
//   S^T [64 tokens x N]    = rows [64 x 576] q^T      (A: the rows as they lie, K-major; the heads are N)
//   O [64 x 512 columns]  += P [64 x 64 tokens] c     (B: the same rows, MN-major; the heads are M)
// The queries stay N x 1152 bytes of shared memory (as the M of an MMA 64 rows of them
// would take 72 KB), and both products read the one copy of the rows: a tile of 64
// tokens is four units of 128 columns, [8 groups of 8 rows][2 blocks of 64
// columns][8][128 bytes] as a TMA box lands them.  A tile's MMAs take 36 x 26 (N = 16)
// or 34 (N = 64) and 16 x 66 cycles.  An M = 64 accumulator sits in 16 lanes of each
// warp's quarter of TMEM: columns 0-255 of O in the lower 16, 256-511 in the upper 16.
//   N = 16, 32 (up to as many heads)   weights as bf16 hi + lo pairs, the lo parts eight
//                more rows behind eight heads: free, as M is 64 anyway
//   N = 64       weights rounded to bf16; 65 to 128 heads are two CTAs that walk the
//                same rows at the same time, so that the second reads them from L2
// Work: one CTA an SM; the batch's tiles, all sequences behind one another, are cut into
// as many equal ranges as there are SMs, whatever the lengths.  A sequence that lies in
// one range is finished there; the pieces of one that is cut leave partial states, two a
// range at most (its first sequence and its last), and a second launch joins them.
//   four warps  softmax (N = 64: eight, four for each half of the heads): warp w has
//              tokens 16 w .. 16 w + 15 of a tile (an M = 64 accumulator sits in 16
//              lanes of each warp's quarter of TMEM), so a score fragment is that of a
//              warp-level MMA; the maxima of the four warps meet only when one grew by
//              more than 2^8 (a reduced barrier says so)
//   one warp   producer: TMA boxes of as many rows as lie together in a page
//   two warps  MMA, the scores' and the products': what a lane issues next waits behind
//              its MMAs, barriers too, and with one lane for both (300 cycles for every
//              barrier between MMAs) neither kept the tensor pipe busy
// Measured, calls back to back on data in turn: 32 contexts of up to 16384 tokens with 16
// heads in 90 us (5.7 TB/s of the rows; HBM, 84% of a copy's rate), 48 of up to 8192 with
// 128 heads in 140 (674 TFLOP/s).  There the ring holds two tiles, beside 72 KB of queries,
// and a tile stays from its load (1700 cycles) over its scores and their softmax to its
// product: the tensor pipe works 62% of the time, in M = 64 MMAs that run at half rate.
// One context of 4096 tokens takes 11.9: one tile a CTA and the join.
// Every wait is bounded in time.
#include <algorithm>
#include <cstdint>
#include <cstring>

#include "kamera_common.cuh"
#include "kamera_hostcheck.h"
#include "kamera_internal.h"
#include "kamera_paged.h"
#include "kamera_ptx.cuh"
#include "kamera_tc.cuh"
#include "kamera_warpmma.cuh"

namespace kamera {

namespace {

using namespace tc;

constexpr int kMpTok = 64;              // tokens of a tile
constexpr int kMpUnits = 4;             // units of 128 value columns
constexpr int kMpDim = 512, kMpRow = 576;
constexpr uint32_t kMpUnit = 16384;     // 64 rows x 128 columns
constexpr uint32_t kMpRope = 8192;      // 64 rows x 64 columns
constexpr uint32_t kMpAtom = 1024;
constexpr int kMpMasks = 8;
constexpr float kMpLazy = 8.0f;
constexpr float kMpLog2e = 1.4426950408889634f, kMpLn2 = 0.6931471805599453f;

template <int N>
struct MpLayout {
    static constexpr bool kPair = N <= 32;           // weights as hi + lo
    static constexpr int NW = kPair ? 2 * N : N;     // rows of the second product: heads, or eight hi, eight lo, ...
    static constexpr int HG = kPair ? N : 32;        // heads of a softmax warpgroup
    static constexpr int kProd = 4 * (N / HG), kScores = kProd + 1, kProducts = kProd + 2;   // warps
    static constexpr int kThreads = 32 * (kProducts + 1);
    static constexpr int NU = N == 16 ? 11 : N == 32 ? 9 : 8;   // units in the ring: two tiles at least, the one whose
                                                                // scores are issued and the one still to be weighed
    static constexpr int NR = N == 32 ? 3 : 2;                  // rope blocks in theirs
    static constexpr int NP = N == 64 ? 1 : 2;                  // buffers of weights
    static constexpr uint32_t kQ = 0;                           // [9 blocks][N rows][128 bytes]
    static constexpr uint32_t kQBlock = N * 128;
    static constexpr uint32_t kP = kQ + 9 * kQBlock;            // [NP][NW rows][128 bytes]
    static constexpr uint32_t kPTile = NW * 128;
    static constexpr uint32_t kRing = kP + NP * kPTile;
    static constexpr uint32_t kRopes = kRing + NU * kMpUnit;
    static constexpr uint32_t kBar = kRopes + NR * kMpRope;
    static constexpr uint32_t kBytes = kBar + 512 + 5 * N * 4 + 1024;   // + alignment slack
    static constexpr uint32_t kTmS = 0, kTmO = 2 * N;           // TMEM columns
    static constexpr uint32_t kTmCols = 512;
    static_assert(kTmO + kMpDim / 2 <= kTmCols, "TMEM columns");
    static_assert(kBytes <= 227 * 1024, "shared memory");
    static_assert(NU >= 2 * kMpUnits && NR >= 2, "a tile's scores while the one before is weighed");
    static_assert(kP % 1024 == 0 && kRing % 1024 == 0, "swizzle atoms");
};

struct MpParams {
    __nv_bfloat16* out;            // [n_seqs][Hq][512]
    float* lse;                    // or null
    const int32_t* pages;          // [n_seqs][max_pages]
    const int32_t* lens;
    float* o;                      // [2 ranges][Hq][512] partial outputs
    float2* ml;                    // [2 ranges][Hq]
    int4* span;                    // [n_seqs]: first and last range, first slot
    int64_t num_pages;
    int32_t n_seqs, Hq, P, max_pages, max_len;
    int32_t blocks, ranges;        // head blocks of N; ranges of tiles
    int32_t box_rows;
    float scale;
    int32_t* err;
    uint64_t half_wait;
    int32_t withhold;
};

struct MpLaunch {
    MpParams p;
    CUtensorMap map_c, map_r, map_q;
};

struct MpBars {
    uint64_t full[11], empty[11], rfull[3], rempty[3];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], pv_done[2], drained[2];
    uint32_t mask[kMpMasks];
    int64_t total, lo, hi;     // the batch's tiles and the range's
    int32_t first_seq, first_len, first_n, first_t;   // where the range starts
    uint32_t units, ropes, segs;   // fills whose loads were issued
    uint32_t tmem;
    int32_t abort;
};
static_assert(sizeof(MpBars) <= 512, "barrier block");

__device__ __forceinline__ int mp_len(const MpParams& p, int s)
{
    const int len = p.lens[s];
    return len >= 0 && len <= p.max_len ? len : 0;
}
// Tiles of a sequence; an empty one has one, which writes its zeros.
__device__ __forceinline__ int mp_tiles(int len) { return len > 0 ? (len - 1) / kMpTok + 1 : 1; }

// The ranges in use, of T tiles.  Where one sequence gives each a few tiles, as few as
// leave the longest as it is: fewer states to join (12000 tokens 21.0 -> 16.8 us, 40000
// 26.6 -> 24.5); ranges that hold the end of one sequence and the start of another are
// better short (four of 8000 tokens 16.8, 18.9 with fewer).  A batch of more rows has all
// ranges, one that is a single sequence and empty rows too.
__device__ __forceinline__ int64_t mp_ranges(const MpParams& p, int64_t T)
{
    if (p.n_seqs > 1 || T <= p.ranges || T > 8ll * p.ranges)
        return min((int64_t)p.ranges, T);
    const int64_t each = wmma16::quotient(T + p.ranges - 1, p.ranges);
    return wmma16::quotient(T + each - 1, each);
}
__device__ __forceinline__ int64_t mp_start(int64_t r, int64_t T, int64_t R) { return wmma16::quotient(r * T, R); }
__device__ __forceinline__ int64_t mp_range_of(int64_t tile, int64_t T, int64_t R) { return wmma16::quotient((tile + 1) * R - 1, T); }

// A range's tiles, walked alike by every role.
struct MpWalk {
    int64_t left;        // tiles of the range from this one on
    int s, len, n, t;    // sequence, its tokens and tiles, the tile
    bool fresh;          // the first tile of a segment
    __device__ __forceinline__ void start(const MpBars& b)
    {
        left = b.hi - b.lo;
        s = b.first_seq;
        len = b.first_len;
        n = b.first_n;
        t = b.first_t;
        fresh = true;
    }
    __device__ __forceinline__ bool last() const { return t + 1 == n || left == 1; }
    __device__ __forceinline__ void next(const MpParams& p)
    {
        --left;
        fresh = false;
        if (++t == n && left > 0) {
            ++s;
            len = mp_len(p, s);
            n = mp_tiles(len);
            t = 0;
            fresh = true;
        }
    }
};

// Total tiles and where the range starts, by one warp: one look at the lengths of up to
// 32 sequences, two at those of more.
__device__ void mp_locate(const MpParams& p, MpBars& b, int r, int lane)
{
    auto length = [&](int s) { return s < p.n_seqs ? mp_len(p, s) : 0; };
    const int first = length(lane);
    if (p.n_seqs <= 32) {   // one scan in 32 bits, as a sequence has at most 2^25 tiles (one context: 12.3 -> 12.0 us)
        const uint32_t n = lane < p.n_seqs ? (uint32_t)mp_tiles(first) : 0u;
        uint32_t x = n;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
            if (lane >= d)
                x += y;
        }
        const uint32_t T = __shfl_sync(0xFFFFFFFFu, x, 31);
        const int64_t R = mp_ranges(p, T);
        if (lane == 0)
            b.total = T;
        if (r >= R)
            return;
        const uint32_t lo = (uint32_t)mp_start(r, T, R), before = x - n;
        if (before <= lo && lo < x) {
            b.first_seq = lane;
            b.first_len = first;
            b.first_n = (int)n;
            b.first_t = (int)(lo - before);
            b.lo = lo;
            b.hi = mp_start(r + 1, T, R);
        }
        return;
    }
    int64_t sum = lane < p.n_seqs ? mp_tiles(first) : 0;
    for (int s = lane + 32; s < p.n_seqs; s += 32)
        sum += mp_tiles(length(s));
#pragma unroll
    for (int d = 16; d >= 1; d /= 2)
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    const int64_t T = sum, R = mp_ranges(p, T);
    int64_t at = 0;
    if (lane == 0)
        b.total = T;
    if (r >= R)   // fewer tiles than ranges
        return;
    const int64_t lo = mp_start(r, T, R);
    for (int s0 = 0; s0 < p.n_seqs; s0 += 32) {
        const int len = s0 == 0 ? first : length(s0 + lane);
        const int64_t mine = s0 + lane < p.n_seqs ? mp_tiles(len) : 0;
        int64_t x = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
            if (lane >= d)
                x += y;
        }
        const int64_t before = at + x - mine;
        if (mine > 0 && before <= lo && lo < before + mine) {
            b.first_seq = s0 + lane;
            b.first_len = len;
            b.first_n = (int)mine;
            b.first_t = (int)(lo - before);
            b.lo = lo;
            b.hi = mp_start(r + 1, T, R);
        }
        at += __shfl_sync(0xFFFFFFFFu, x, 31);
        if (at > lo)
            break;
    }
}

// ---------------------------------------------------------------- producer --
// The rows that a load of the same place would bring, into L2.
__device__ __forceinline__ void mp_prefetch(const CUtensorMap* map, int col, int group)
{
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %1, %2, %3}];" ::"l"(map), "r"(0), "r"(col),
                 "r"(group)
                 : "memory");
}

template <int N>
__device__ void mp_producer(const MpLaunch& L, MpBars& b, uint32_t sbase, int lane, int block)
{
    using Y = MpLayout<N>;
    const MpParams& p = L.p;
    // Lane l is at 16-token piece l % 4 of tile l / 4 of eight tiles, and of the eight
    // after them: pages are looked up, and rows worked out, for 32 pieces at once and
    // eight tiles ahead (under load a look-up takes 2000 cycles).
    constexpr int kPieces = kMpTok / 16, kAhead = 32 / kPieces;
    constexpr bool kPrefetch = N == 64;
    const int R = p.box_rows, off = 16 * (lane % kPieces);   // a box of R rows is issued by its first piece's lane
    MpWalk w, mine;
    w.start(b);
    mine = w;
    auto advance = [&](int n) {
        if (mine.left > n && mine.t + n < mine.n) {
            mine.left -= n;
            mine.t += n;
        } else {
            for (int i = 0; i < n && mine.left > 0; ++i)
                mine.next(p);
        }
    };
    auto look_up = [&](int& page, int& row) {   // page -1: no piece; row: its first one in the page
        page = -1;
        row = 0;
        const int tok = mine.t * kMpTok + off;
        if (mine.left <= 0 || tok >= mine.len)
            return;
        const int slot = tok / p.P;
        row = tok - slot * p.P;
        page = p.pages[(int64_t)mine.s * p.max_pages + slot];
        page = page < 0 ? -2 : page;
    };
    advance(lane / kPieces);
    int page, row, page_next = -1, row_next = 0, group = 0;
    look_up(page, row);
    const uint32_t starts = R == 16 ? 0xFu : R == 32 ? 0x5u : 0x1u;   // the pieces at which a box of R rows starts
    // The lane that waits and issues has these to itself.
    uint32_t unit = 0, rope = 0, seg = 0, at = 0, lap = 0, ra = 0, rl = 0;   // issued so far; places in the rings
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return wmma16::cycle_wait(ptx::smem_addr(bar), parity & 1u, &b.abort, p.err, p.half_wait);
    };
    uint32_t tile = 0, there = 0, there_next = 0;   // (the _next ones: once two tiles on are of the eight after)
    int group_next = 0;
    bool ok = true;
    while (w.left > 0 && ok) {
        if (tile % kAhead == 0) {
            if (tile > 0) {
                page = page_next;
                row = row_next;
            }
            const bool good = page >= 0 && page < p.num_pages;
            if (page != -1 && !good && block == 0)
                raise_err(p.err, KAMERA_DEVERR_SLOT);
            group = (int)(((int64_t)page * p.P + row) >> 3);
            there = __ballot_sync(0xFFFFFFFFu, good);
        }
        const uint32_t mask = (there >> (kPieces * (tile % kAhead))) & 0xFu, boxes = mask & starts;
        const int n = __popc(boxes);
        int groups[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            groups[i] = __shfl_sync(0xFFFFFFFFu, group, kPieces * (int)(tile % kAhead) + i);
        // The rows of two tiles on are asked into L2 where the ring is short, by each head
        // block its share of the units: 150 -> 146 us for 128 heads (16 heads, whose ring
        // is longer: 93.4 -> 94.4, so not there).
        uint32_t far_boxes = 0;
        int far[kPieces] = {};
        if constexpr (kPrefetch) {
            const int to = (int)(tile % kAhead) + 2;
            if (to == kAhead) {
                group_next = (int)(((int64_t)page_next * p.P + row_next) >> 3);
                there_next = __ballot_sync(0xFFFFFFFFu, page_next >= 0 && page_next < p.num_pages);
            }
            far_boxes = ((to < kAhead ? there : there_next) >> (kPieces * (to % kAhead))) & starts;
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                far[i] = __shfl_sync(0xFFFFFFFFu, to < kAhead ? group : group_next, kPieces * (to % kAhead) + i);
        }
        // One lane for all of a tile: a step that the warp takes together, or that lanes
        // take each by itself, costs this warp 150 cycles and more, and 580 a unit made it
        // what the whole CTA waited for.
        if (elect_one()) {
            auto load = [&](uint32_t dst, uint32_t full, const CUtensorMap* map, int col, uint32_t row_group) {
                if (p.withhold)
                    return;
                if (n > 0)
                    ptx::mbar_arrive_expect_tx(full, (uint32_t)(n * (R >> 3)) * row_group);
                else
                    ptx::mbar_arrive(full);
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
                    if ((boxes >> i) & 1u)
                        ptx::tma_load_4d(dst + 2 * i * row_group, map, 0, 0, col, groups[i], full);
            };
            if (w.fresh && (seg == 0 || (ok = wait(&b.q_empty, seg - 1)))) {
                if (!p.withhold) {
                    ptx::mbar_arrive_expect_tx(ptx::smem_addr(&b.q_full), 9 * Y::kQBlock);
                    for (int i = 0; i < 9; ++i)
                        ptx::tma_load_2d(sbase + Y::kQ + i * Y::kQBlock, &L.map_q, 64 * i, w.s * p.Hq + block * N,
                                         ptx::smem_addr(&b.q_full));
                }
                ++seg;
            }
            b.mask[tile % kMpMasks] = mask;
            for (int u = 0; u < kMpUnits && ok; ++u) {
                if (lap > 0 && !(ok = wait(&b.empty[at], lap - 1)))
                    break;
                load(sbase + Y::kRing + at * kMpUnit, ptx::smem_addr(&b.full[at]), &L.map_c, 2 * u, 2 * kMpAtom);
                ++unit;
                if (++at == (uint32_t)Y::NU) {
                    at = 0;
                    ++lap;
                }
            }
            if (ok && (rl == 0 || (ok = wait(&b.rempty[ra], rl - 1)))) {
                load(sbase + Y::kRopes + ra * kMpRope, ptx::smem_addr(&b.rfull[ra]), &L.map_r, kMpDim / 64, kMpAtom);
                ++rope;
                if (++ra == (uint32_t)Y::NR) {
                    ra = 0;
                    ++rl;
                }
            }
            if (kPrefetch && ok && !p.withhold)
#pragma unroll 1
                for (int i = 0; i < kPieces; ++i)
                    if ((far_boxes >> i) & 1u) {
                        const int g = i == 0 ? far[0] : i == 1 ? far[1] : i == 2 ? far[2] : far[3];
#pragma unroll 1
                        for (int u = block; u < kMpUnits; u += p.blocks)
                            mp_prefetch(&L.map_c, 2 * u, g);
                        if (block == 0)
                            mp_prefetch(&L.map_r, kMpDim / 64, g);
                    }
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (tile % kAhead == 0) {  // the eight tiles after these
            advance(kAhead);
            look_up(page_next, row_next);
        }
        w.next(p);
        ++tile;
    }
    if (elect_one() && !p.withhold) {
        b.units = unit;
        b.ropes = rope;
        b.segs = seg;
    }
    __syncwarp();
}

// After a timeout, once every role has left its loop: the copies that the CTA started land
// before it leaves.  (Without one the MMA lanes have waited for every fill.)
template <int N>
__device__ __forceinline__ void mp_drain(const MpBars& b)
{
    using Y = MpLayout<N>;
    pf_drain_ring(&b.q_full, b.segs, 1);
    pf_drain_ring(b.full, b.units, Y::NU);
    pf_drain_ring(b.rfull, b.ropes, Y::NR);
}

// --------------------------------------------------------------------- MMA --
// MMAs whose A (mma_ds) or B (mma_sd) is a unit, groups of eight rows 2 KB apart; the
// other operand has them 1 KB apart.  The accumulate flag and the descriptors' high
// words are constants: with them in registers an issue took 58 cycles, where the tensor
// pipe needs 26 to 66.
constexpr uint32_t kMpHiU = (2 * kMpAtom >> 4) | (1u << 14) | (2u << 29);

template <bool ACC>
__device__ __forceinline__ void mma_ds(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc)
{
    mma_ss2<ACC, kMpHiU, kDescHi>(d, a_lo, b_lo, idesc);
}
template <bool ACC>
__device__ __forceinline__ void mma_sd(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc)
{
    mma_ss2<ACC, kDescHi, kMpHiU>(d, a_lo, b_lo, idesc);
}

// The scores' lane: tile by tile as the rows come.
template <int N>
__device__ void mp_scores(const MpLaunch& L, MpBars& b, uint32_t sbase, uint32_t tm)
{
    using Y = MpLayout<N>;
    const MpParams& p = L.p;
    constexpr uint32_t idS = ptx::idesc_bf16_f32(kMpTok, N);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return wmma16::cycle_wait(ptx::smem_addr(bar), parity & 1u, &b.abort, p.err, p.half_wait);
    };
    const uint32_t q_lo = ((sbase + Y::kQ) >> 4) | (1u << 16), u_lo = ((sbase + Y::kRing) >> 4) | (1u << 16);
    const uint32_t r_lo = ((sbase + Y::kRopes) >> 4) | (1u << 16);
    MpWalk w;
    w.start(b);
    uint32_t seg = 0, at = 0, lap = 0;   // place in the ring
    for (uint32_t t = 0; w.left > 0; ++t, w.next(p)) {
        if (w.fresh && !wait(&b.q_full, seg))
            break;
        if (t >= 2 && !wait(&b.p_full[t & 1u], (t >> 1) - 1))   // the scores that stood there have been read
            break;
        const uint32_t d = tm + Y::kTmS + (t & 1u) * N;
        bool ok = true;
#pragma unroll
        for (uint32_t u = 0; u < kMpUnits; ++u) {
            if (!(ok = ok && wait(&b.full[at], lap)))
                break;
            ptx::tc_fence_after();
            const uint32_t a = u_lo + at * (kMpUnit >> 4), q = q_lo + 2 * u * (Y::kQBlock >> 4);
            if (u == 0)
                mma_ds<false>(d, a, q, idS);
            else
                mma_ds<true>(d, a, q, idS);
#pragma unroll
            for (int i = 1; i < 8; ++i)   // two blocks of 64 columns
                mma_ds<true>(d, a + (i >> 2) * (kMpAtom >> 4) + 2 * (i & 3),
                             q + (i >> 2) * (Y::kQBlock >> 4) + 2 * (i & 3), idS);
            if (++at == (uint32_t)Y::NU) {
                at = 0;
                ++lap;
            }
        }
        const uint32_t ra = t % Y::NR;
        if (!ok || !wait(&b.rfull[ra], t / Y::NR))
            break;
        ptx::tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
            mma_ss<true>(d, r_lo + ra * (kMpRope >> 4) + 2 * ks, q_lo + 8 * (Y::kQBlock >> 4) + 2 * ks, idS);
        ptx::umma_commit(ptx::smem_addr(&b.rempty[ra]));
        ptx::umma_commit(ptx::smem_addr(&b.s_full[t & 1u]));
        if (w.last()) {
            ptx::umma_commit(ptx::smem_addr(&b.q_empty));
            ++seg;
        }
    }
    // every MMA issued here completes before TMEM is freed
    ptx::umma_commit(ptx::smem_addr(&b.drained[0]));
    pf_drain_wait(ptx::smem_addr(&b.drained[0]), 0u);
}

// The products' lane: tile by tile as the weights come; a tile's units are free behind it.
template <int N>
__device__ void mp_products(const MpLaunch& L, MpBars& b, uint32_t sbase, uint32_t tm)
{
    using Y = MpLayout<N>;
    const MpParams& p = L.p;
    constexpr uint32_t idO = ptx::idesc_bf16_f32(64, 128) | (1u << 16);   // B: MN-major
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return wmma16::cycle_wait(ptx::smem_addr(bar), parity & 1u, &b.abort, p.err, p.half_wait);
    };
    const uint32_t p_lo = ((sbase + Y::kP) >> 4) | (1u << 16);
    const uint32_t u_lo = ((sbase + Y::kRing) >> 4) | ((kMpAtom >> 4) << 16);
    MpWalk w;
    w.start(b);
    uint32_t at = 0, lap = 0;
    for (uint32_t t = 0; w.left > 0; ++t, w.next(p)) {
        uint32_t x = at, xl = lap;
        bool ok = true;
        for (uint32_t u = 0; u < kMpUnits && ok; ++u) {   // there long since: the weights come behind their scores
            ok = wait(&b.full[x], xl);
            if (++x == (uint32_t)Y::NU) {
                x = 0;
                ++xl;
            }
        }
        if (!ok || !wait(&b.p_full[t & 1u], t >> 1))
            break;
        ptx::tc_fence_after();
        const uint32_t pb = p_lo + t % Y::NP * (Y::kPTile >> 4);
#pragma unroll
        for (uint32_t u = 0; u < kMpUnits; ++u) {
            const uint32_t v = u_lo + at * (kMpUnit >> 4);
            const uint32_t d = tm + Y::kTmO + (u & 1u) * 128 + ((u >> 1) << 20);   // columns 256 on: 16 lanes further
            if (w.fresh)
                mma_sd<false>(d, pb, v, idO);
            else
                mma_sd<true>(d, pb, v, idO);
#pragma unroll
            for (int ks = 1; ks < 4; ++ks)
                mma_sd<true>(d, pb + 2 * ks, v + ks * (4 * kMpAtom >> 4), idO);
            ptx::umma_commit(ptx::smem_addr(&b.empty[at]));
            if (++at == (uint32_t)Y::NU) {
                at = 0;
                ++lap;
            }
        }
        ptx::umma_commit(ptx::smem_addr(&b.pv_done[t & 1u]));
    }
    ptx::umma_commit(ptx::smem_addr(&b.drained[1]));
    pf_drain_wait(ptx::smem_addr(&b.drained[1]), 0u);
}

// ----------------------------------------------------------------- softmax --
// A warp's 16 tokens x N heads: register 4 j + 2 r + c is token lane / 4 + 8 r, head
// 8 j + 2 (lane % 4) + c.
template <int N>
__device__ __forceinline__ void mp_ld_scores(uint32_t ta, uint32_t (&r)[N / 2])
{
    if constexpr (N == 16) {
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
                     "tcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(ta)
                     : "memory");
    } else {
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
                     "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                       "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                       "=r"(r[15])
                     : "r"(ta)
                     : "memory");
    }
}

// Four 8 x 8 blocks of bf16 pairs, each stored transposed: row i of block k at the
// address of lane 8 k + i.
__device__ __forceinline__ void stsm_x4_t(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y),
                 "r"(z), "r"(w)
                 : "memory");
}

// The four warps of a softmax group meet.
__device__ __forceinline__ void mp_sync(int grp) { asm volatile("bar.sync %0, 128;" ::"r"(1 + 2 * grp) : "memory"); }
// The same; whether any thread said yes.
__device__ __forceinline__ bool mp_any(int grp, bool x)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(x ? 1u : 0u), "r"(2 + 2 * grp)
                 : "memory");
    return r != 0;
}

// Softmax group grp: heads grp HG .. of the block.  One code for all groups: with two
// copies of it the roles' loops do not fit the instruction cache together (128 heads: 173
// us instead of 150, a quarter of the stalls for want of instructions).
template <int N>
__device__ void mp_softmax(const MpLaunch& L, MpBars& b, uint32_t sbase, float* ex, uint32_t tm, int grp, int warp, int lane,
                           int block, int range, int64_t lo, int64_t hi)
{
    using Y = MpLayout<N>;
    constexpr int HG = Y::HG, J = HG / 8;
    const int G0 = grp * HG;
    const MpParams& p = L.p;
    const int gq = lane >> 2, t4 = lane & 3;
    const uint32_t lanes = tm + ((uint32_t)warp << 21);
    const float sl2 = p.scale * kMpLog2e;
    const int head0 = block * N + G0, heads = min(HG, p.Hq - head0);   // (none at all for a last group: 0 or less)
    const int64_t T = b.total, R = mp_ranges(p, T);
    float* wmax = ex + 5 * G0;     // [4 warps][HG]: the warps' maxima; their sums
    float* fac = wmax + 4 * HG;    // [HG]: factors of the running output
    // the output's rows of this group: whether this warp's lanes hold some, and the lane's head
    const int Q0 = Y::kPair ? 0 : G0 / 16, Q1 = Q0 + (Y::kPair ? 2 : 1) * HG / 16;
    const bool out_warp = warp >= Q0 && warp < Q1;
    const int out_head = out_warp ? (Y::kPair ? 8 * warp + (lane & 7) : 16 * (warp - Q0) + (lane & 15)) : 0;
    float m[J][2], l[J][2];        // heads 8 j + 2 t4, + 1: the agreed maximum (log2 units), this thread's sum
    // where this lane's row of a stored block goes: block k = (j, half of the tokens) in pairs of j
    const uint32_t st_row = lane & 7, st_half = (lane >> 3) & 1, st_j = lane >> 4;
    const uint32_t st = sbase + Y::kP + (G0 / 8 + st_j) * (Y::kPair ? 2 : 1) * kMpAtom + sw128(st_row, 2 * warp + st_half);
    MpWalk w;
    w.start(b);
    int64_t at = lo;               // the tile's place among all
    bool ok = true;
    for (uint32_t t = 0; w.left > 0; ++t, ++at) {
        if (w.fresh) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                m[j][0] = m[j][1] = -INFINITY, l[j][0] = l[j][1] = 0.f;
        }
        const int ntok = min(kMpTok, w.len - w.t * kMpTok);
        ok = ok && wmma16::cycle_wait(ptx::smem_addr(&b.s_full[t & 1u]), (t >> 1) & 1u, &b.abort, p.err, p.half_wait);
        ok = __all_sync(0xFFFFFFFFu, ok);
        uint32_t s[HG / 2];
        bool grew = false;
        const uint32_t mask = *reinterpret_cast<volatile uint32_t*>(&b.mask[t % kMpMasks]);
        float x[J][4];
        if (ok) {
            ptx::tc_fence_after();
            mp_ld_scores<HG>(lanes + Y::kTmS + (t & 1u) * N + G0, s);
            const bool here = (mask >> warp) & 1u;
            const bool in0 = here && 16 * warp + gq < ntok, in1 = here && 16 * warp + gq + 8 < ntok;
#pragma unroll
            for (int j = 0; j < J; ++j) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    x[j][c] = in0 ? __uint_as_float(s[4 * j + c]) * sl2 : -INFINITY;
                    x[j][2 + c] = in1 ? __uint_as_float(s[4 * j + 2 + c]) * sl2 : -INFINITY;
                    grew |= fmaxf(x[j][c], x[j][2 + c]) > m[j][c] + kMpLazy;
                }
            }
        }
        if (mp_any(grp, grew || !ok)) {   // rare but for a segment's first tile
            if (mp_any(grp, !ok))
                break;               // all four warps
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v = fmaxf(x[j][c], x[j][2 + c]);
                    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
                    if (gq == 0)
                        wmax[warp * HG + 8 * j + 2 * t4 + c] = v;
                }
            mp_sync(grp);
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int h = 8 * j + 2 * t4 + c;
                    float v = m[j][c];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v = fmaxf(v, wmax[k * HG + h]);
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
                mp_sync(grp);
                if (out_warp) {
                    const float f = fac[out_head];
#pragma unroll 1
                    for (int c = 0; c < kMpDim / 2 / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(lanes + Y::kTmO + 32 * c, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st32(lanes + Y::kTmO + 32 * c, o);
                    }
                    tmem_wait_st();
                }
            }
            mp_sync(grp);               // the exchange's arrays are free again
        }
        // weights, transposed into the operand rows (heads) of the second product
        const uint32_t dst = st + t % Y::NP * Y::kPTile;
        if (t >= Y::NP) {            // the product that read the buffer's last weights
            const uint32_t k = t - Y::NP;
            ok = wmma16::cycle_wait(ptx::smem_addr(&b.pv_done[k & 1u]), (k >> 1) & 1u, &b.abort, p.err, p.half_wait);
            ok = __all_sync(0xFFFFFFFFu, ok);
        }
#pragma unroll
        for (int j = 0; j < J; j += 2) {
            uint32_t h[4], lo4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {   // block k: heads of j + k / 2, tokens of half k & 1
                const int jj = j + (k >> 1), r = k & 1;
                const float m0 = m[jj][0] == -INFINITY ? 0.f : m[jj][0], m1 = m[jj][1] == -INFINITY ? 0.f : m[jj][1];
                const float a = pf_ex2(x[jj][2 * r] - m0), c = pf_ex2(x[jj][2 * r + 1] - m1);
                l[jj][0] += a;
                l[jj][1] += c;
                if constexpr (Y::kPair) {
                    h[k] = weight_hi(a, c);
                    lo4[k] = pack_bf16x2(fmaf(bf16lo(h[k]), kLessHi, a), fmaf(bf16hi(h[k]), kLessHi, c));
                } else {
                    h[k] = pack_bf16x2(a, c);
                }
            }
            stsm_x4_t(dst + j * (Y::kPair ? 2 : 1) * kMpAtom, h[0], h[1], h[2], h[3]);
            if constexpr (Y::kPair)
                stsm_x4_t(dst + (2 * j + 1) * kMpAtom, lo4[0], lo4[1], lo4[2], lo4[3]);
        }
        if (ntok < kMpTok || mask != 0xFu) {   // value rows without a token: zero, so that zero weights add nothing
            for (int e = threadIdx.x; e < kMpTok * 64; e += 4 * 32 * (N / HG)) {
                const int r = e >> 6, piece = e & 63, u = piece >> 4, blk = (piece >> 3) & 1;
                if (r >= ntok || !((mask >> (r >> 4)) & 1u))
                    ptx::st_shared_zero16(sbase + Y::kRing + (kMpUnits * t + u) % Y::NU * kMpUnit +
                                          (uint32_t)(r >> 3) * 2 * kMpAtom + blk * kMpAtom + sw128(r & 7, piece & 7));
            }
        }
        ptx::fence_proxy_async();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0)
            ptx::mbar_arrive(ptx::smem_addr(&b.p_full[t & 1u]));
        if (!w.last()) {
            w.next(p);
            continue;
        }
        // ---- the segment's end: its state
        const int s_seq = w.s;
        const int64_t a0 = at - w.t, r0 = mp_range_of(a0, T, R), r1 = mp_range_of(a0 + w.n - 1, T, R);
        const int first_slot = (int)(2 * r0 + (mp_start(r0, T, R) == a0 ? 0 : 1));
        const bool whole = r0 == r1;
        const int slot = range == r0 ? first_slot : 2 * range;
        if (range == r0 && block == 0 && grp == 0 && warp == 0 && lane == 0)
            p.span[s_seq] = make_int4((int)r0, (int)r1, first_slot, 0);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                l[j][c] += __shfl_xor_sync(0xFFFFFFFFu, l[j][c], 4);
                l[j][c] += __shfl_xor_sync(0xFFFFFFFFu, l[j][c], 8);
                l[j][c] += __shfl_xor_sync(0xFFFFFFFFu, l[j][c], 16);
                if (gq == 0)
                    wmax[warp * HG + 8 * j + 2 * t4 + c] = l[j][c];
            }
        mp_sync(grp);
        const int64_t row0 = (int64_t)s_seq * p.Hq + head0, part0 = (int64_t)slot * p.Hq + head0;
        if (warp == 0 && gq == 0) {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int h = 8 * j + 2 * t4 + c;
                    const float sum = (wmax[h] + wmax[HG + h]) + (wmax[2 * HG + h] + wmax[3 * HG + h]);
                    fac[h] = sum > 0.f ? 1.f / sum : (sum == sum ? 0.f : sum);
                    if (h < heads) {
                        if (!whole)
                            p.ml[part0 + h] = make_float2(m[j][c], sum);
                        else if (p.lse)
                            p.lse[row0 + h] = sum > 0.f ? (m[j][c] + log2f(sum)) * kMpLn2 : (sum == sum ? -INFINITY : sum);
                    }
                }
        }
        ok = wmma16::cycle_wait(ptx::smem_addr(&b.pv_done[t & 1u]), (t >> 1) & 1u, &b.abort, p.err, p.half_wait);
        ok = __all_sync(0xFFFFFFFFu, ok);
        ptx::tc_fence_after();
        mp_sync(grp);
        if (out_warp) {
            const bool mine = ok && out_head < heads;
            const float inv = fac[out_head];
            const int dim0 = (lane >> 4) * (kMpDim / 2);
            auto put = [&](int c, uint32_t (&o)[32]) {   // 32 of the columns
                if constexpr (Y::kPair) {   // a lane with hi sums and one with lo sums: each writes half of the columns
                    const bool lo_row = lane & 8;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float give = __uint_as_float(lo_row ? o[i] : o[16 + i]);
                        const float keep = __uint_as_float(lo_row ? o[16 + i] : o[i]);
                        o[i] = __float_as_uint(keep + __shfl_xor_sync(0xFFFFFFFFu, give, 8));
                    }
                }
                constexpr int C = Y::kPair ? 16 : 32;
                const int dim = dim0 + 32 * c + (Y::kPair ? (lane & 8) * 2 : 0);
                if (mine && whole) {
                    __nv_bfloat16* dst = p.out + (row0 + out_head) * kMpDim + dim;
#pragma unroll
                    for (int i = 0; i < C; i += 8)
                        *reinterpret_cast<uint4*>(dst + i) =
                            make_uint4(pack_bf16x2(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv),
                                       pack_bf16x2(__uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv),
                                       pack_bf16x2(__uint_as_float(o[i + 4]) * inv, __uint_as_float(o[i + 5]) * inv),
                                       pack_bf16x2(__uint_as_float(o[i + 6]) * inv, __uint_as_float(o[i + 7]) * inv));
                } else if (mine) {
                    float* dst = p.o + (part0 + out_head) * kMpDim + dim;
#pragma unroll
                    for (int i = 0; i < C; i += 4)
                        *reinterpret_cast<uint4*>(dst + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
                __syncwarp();
            };
#pragma unroll 1
            for (int c = 0; c < kMpDim / 2 / 32; c += 2) {   // (one at a time takes 3400 cycles in all)
                uint32_t o[2][32];
                tmem_ld32_issue(lanes + Y::kTmO + 32 * c, o[0]);
                tmem_ld32(lanes + Y::kTmO + 32 * c + 32, o[1]);   // waits for both
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    asm volatile("" : "+r"(o[0][i]));
                put(c, o[0]);
                put(c + 1, o[1]);
            }
        }
        ptx::tc_fence_before();
        mp_sync(grp);   // the exchange's arrays, and TMEM, are free for the next segment
        w.next(p);
    }
}

template <int N>
__global__ void __launch_bounds__(MpLayout<N>::kThreads, 1) mla_paged_kernel(const __grid_constant__ MpLaunch L)
{
    using Y = MpLayout<N>;
    const MpParams& p = L.p;
    extern __shared__ __align__(16) unsigned char raw[];
    const uint32_t addr = ptx::smem_addr(raw), pad = (1024u - (addr & 1023u)) & 1023u, sbase = addr + pad;
    MpBars& b = *reinterpret_cast<MpBars*>(raw + pad + Y::kBar);
    float* ex = reinterpret_cast<float*>(raw + pad + Y::kBar + 512);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int block = blockIdx.x % p.blocks, range = blockIdx.x / p.blocks;
    if (threadIdx.x == 0) {
        for (int i = 0; i < Y::NU; ++i) {
            ptx::mbar_init(ptx::smem_addr(&b.full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.empty[i]), 1);
        }
        for (int i = 0; i < Y::NR; ++i) {
            ptx::mbar_init(ptx::smem_addr(&b.rfull[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.rempty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_addr(&b.s_full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.p_full[i]), Y::kProd);   // softmax warps
            ptx::mbar_init(ptx::smem_addr(&b.pv_done[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.drained[i]), 1);
        }
        ptx::mbar_init(ptx::smem_addr(&b.q_full), 1);
        ptx::mbar_init(ptx::smem_addr(&b.q_empty), 1);
        b.abort = 0;
        b.units = b.ropes = b.segs = 0;
        ptx::fence_barrier_init();
    }
    if (warp == Y::kProd && lane == 0) {
        ptx::prefetch_tmap(&L.map_c);
        ptx::prefetch_tmap(&L.map_r);
        ptx::prefetch_tmap(&L.map_q);
    }
    if (warp == Y::kScores) {
        ptx::tmem_alloc(ptx::smem_addr(&b.tmem), Y::kTmCols);
        ptx::tmem_relinquish();
    }
    ptx::grid_wait();
    if (warp == 0)
        mp_locate(p, b, range, lane);
    if (blockIdx.x == 0 && warp > 0)
        for (int s = threadIdx.x - 32; s < p.n_seqs; s += Y::kThreads - 32)
            if (p.lens[s] < 0 || p.lens[s] > p.max_len)
                raise_err(p.err, KAMERA_DEVERR_LEN);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    ptx::grid_launch_next();   // (this CTA has its TMEM: none that starts early can take it)
    const uint32_t tm = b.tmem;
    const int64_t T = b.total, R = mp_ranges(p, T);
    if (range < R) {   // (else: fewer tiles than ranges)
        const int64_t lo = b.lo, hi = b.hi;
        if (warp < Y::kProd)
            mp_softmax<N>(L, b, sbase, ex, tm, Y::kProd > 4 ? warp >> 2 : 0, warp & 3, lane, block, range, lo, hi);
        else if (warp == Y::kProd)
            mp_producer<N>(L, b, sbase, lane, block);
        else if (warp == Y::kScores) {
            if (elect_one())
                mp_scores<N>(L, b, sbase, tm);
        } else if (elect_one())
            mp_products<N>(L, b, sbase, tm);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == Y::kScores) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tm, Y::kTmCols);
    }
    if (threadIdx.x == 32 * Y::kProd && b.abort)
        mp_drain<N>(b);
}

// ------------------------------------------------------------------- merge --
// The rows whose sequence was cut: out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i
// over the partial states of its ranges.  CQ CTAs a row, a thread four columns of every
// GR-th state, whose outputs it asks for eight at a time before their weights are known;
// the GR sums join in order.  Where a sequence may have many states it is all latency: a
// warp a state and a quarter of the columns, 16 of them (for one sequence cut 64 times 2 us
// less than four groups of whole rows, which took 9 less than one); where the rows are
// many and have two or three states, a thread for all of them (four groups: 30 us more
// for 6144 rows).
template <int GR, int CQ>
__global__ void __launch_bounds__(128 / CQ * GR) mla_merge_kernel(const MpParams p)
{
    constexpr int TG = 128 / CQ;   // threads of a group
    __shared__ float4 part[GR > 1 ? GR - 1 : 1][TG];
    const int64_t row = blockIdx.x / CQ;
    const int s = (int)(row / p.Hq), h = (int)(row - (int64_t)s * p.Hq);
    const int lane = threadIdx.x & 31, group = threadIdx.x / TG, mine = threadIdx.x % TG;
    const int col = (int)(blockIdx.x % CQ) * TG + mine;
    ptx::grid_wait();
    ptx::grid_launch_next();
    const int4 sp = p.span[s];
    // finished where it was read; or, after a timeout, never written
    if (sp.x == sp.y || sp.x < 0 || sp.y < sp.x || sp.y >= p.ranges || (sp.z >> 1) != sp.x)
        return;
    const int n = sp.y - sp.x + 1;
    auto slot = [&](int i) { return (int64_t)(i == 0 ? sp.z : 2 * (sp.x + i)) * p.Hq + h; };
    constexpr int U = 8, SW = U * GR > 32 ? U * GR / 32 : 1;   // a round: eight states a group, SW a lane
    float4 v[U];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int i = i0 + GR * k + group;
            if (i < n)
                v[k] = *reinterpret_cast<const float4*>(p.o + slot(i) * kMpDim + 4 * col);
        }
    };
    load(0);
    float m = -INFINITY;
    for (int i = lane; i < n; i += 32)
        m = fmaxf(m, p.ml[slot(i)].x);
#pragma unroll
    for (int d = 16; d >= 1; d /= 2)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += U * GR) {
        if (i0 > 0)
            load(i0);
        float f[SW];   // a state without weight adds nothing (and has no maximum to scale by)
        uint32_t live[SW];
#pragma unroll
        for (int c = 0; c < SW; ++c) {
            const int j = 32 * c + lane;
            f[c] = 0.f;
            bool some = false;
            if (j < U * GR && i0 + j < n) {
                const float2 y = p.ml[slot(i0 + j)];
                some = y.y != 0.f;
                if (some) {
                    f[c] = pf_ex2(y.x - m);
                    l = fmaf(y.y, f[c], l);
                }
            }
            live[c] = __ballot_sync(0xFFFFFFFFu, some);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int j = GR * k + group, c = GR * k / 32;   // (a round's state j: lane j % 32 has its weight)
            const float x = __shfl_sync(0xFFFFFFFFu, f[c], j & 31);
            if ((live[c] >> (j & 31)) & 1u) {
                acc.x = fmaf(v[k].x, x, acc.x);
                acc.y = fmaf(v[k].y, x, acc.y);
                acc.z = fmaf(v[k].z, x, acc.z);
                acc.w = fmaf(v[k].w, x, acc.w);
            }
        }
    }
    if constexpr (GR > 1) {
        if (group > 0)
            part[group - 1][mine] = acc;
        __syncthreads();
        if (group > 0)
            return;
    }
#pragma unroll
    for (int d = 16; d >= 1; d /= 2)
        l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
#pragma unroll
    for (int g = 0; g < GR - 1; ++g) {
        const float4 y = part[g][mine];
        acc.x += y.x, acc.y += y.y, acc.z += y.z, acc.w += y.w;
    }
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    *reinterpret_cast<uint2*>(p.out + row * kMpDim + 4 * col) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (col == 0 && p.lse)
        p.lse[row] = l > 0.f ? (m + log2f(l)) * kMpLn2 : (l == l ? -INFINITY : l);
}

// -------------------------------------------------------------------- host --
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int mp_heads(int Hq) { return Hq <= 16 ? 16 : Hq <= 32 ? 32 : 64; }

struct MpNeed {
    size_t o, ml, span;
    size_t bytes() const { return o + ml + span; }
};
MpNeed mp_need(const MpParams& p)
{
    const size_t rows = (size_t)2 * p.ranges * p.Hq;
    return {up256(rows * kMpDim * 4), up256(rows * 8), up256((size_t)p.n_seqs * 16)};
}

int mp_plan(const KameraPagedMlaKV* kv, const KameraPagedQuery* q, const KameraPageTable* t, MpParams* p)
{
    if (!kv || !q || !t || kv->reserved != 0 || q->reserved != 0 || kv->kv_lora_rank < 1 || kv->rope_dim < 0 ||
        kv->page_size < 1 || kv->num_slots < 0 || q->n_seqs < 0 || q->num_q_heads < 1 || !(q->scale == q->scale) ||
        t->max_len < 0 || t->max_pages < 0)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (kv->kv_lora_rank != kMpDim || kv->rope_dim != kMpRow - kMpDim || q->num_q_heads > 128 || kv->page_size % 16 ||
        kv->num_slots > 0x7FFFFFFF || q->n_seqs > 65535 || t->max_len > 0x7FFFFF00)
        return KAMERA_ERR_UNSUPPORTED;
    if ((int64_t)t->max_pages * kv->page_size < t->max_len)
        return KAMERA_ERR_INVALID_ARGUMENT;
    std::memset(p, 0, sizeof(*p));
    p->n_seqs = q->n_seqs;
    p->Hq = q->num_q_heads;
    p->P = kv->page_size;
    p->num_pages = kv->num_slots / kv->page_size;
    p->max_pages = t->max_pages;
    p->max_len = t->max_len;
    p->scale = q->scale;
    if (q->n_seqs == 0)
        return KAMERA_OK;
    const int N = mp_heads(p->Hq);
    p->blocks = (p->Hq + N - 1) / N;
    const int64_t most = (int64_t)p->n_seqs * std::max<int64_t>(1, ((int64_t)p->max_len + kMpTok - 1) / kMpTok);
    p->ranges = (int32_t)std::min<int64_t>(std::max(1, device_sms() / p->blocks), most);
    return KAMERA_OK;
}

template <int N>
cudaError_t mp_launch(const MpLaunch& L, cudaStream_t stream)
{
    using Y = MpLayout<N>;
    // set at every launch: the attribute belongs to the current device's context
    const cudaError_t e =
        cudaFuncSetAttribute(mla_paged_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Y::kBytes);
    if (e != cudaSuccess)
        return e;
    return launch_after(mla_paged_kernel<N>, dim3((unsigned)(L.p.ranges * L.p.blocks)), Y::kThreads, Y::kBytes, stream,
                        true, L);
}

}  // namespace

}  // namespace kamera

using namespace kamera;

extern "C" {

size_t kamera_mla_attend_paged_workspace_bytes(const KameraPagedMlaKV* kv, const KameraPagedQuery* query,
                                               const KameraPageTable* table)
{
    MpParams p;
    return mp_plan(kv, query, table, &p) == KAMERA_OK && p.n_seqs > 0 ? mp_need(p).bytes() : 0;
}

int kamera_mla_attend_paged(const KameraPagedMlaKV* kv, const KameraPagedQuery* query, const KameraPageTable* table,
                            void* d_workspace, size_t workspace_bytes, int32_t* d_err, struct CUstream_st* stream_)
{
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    MpLaunch L;
    std::memset(&L, 0, sizeof(L));
    MpParams& p = L.p;
    const int rc = mp_plan(kv, query, table, &p);
    if (rc || p.n_seqs == 0)
        return rc;
    if (!query->q || !query->out || !table->lens || (!table->pages && table->max_len > 0) || !d_workspace)
        return KAMERA_ERR_INVALID_ARGUMENT;
    int e;
    if ((e = check_strided(kv->kv, 1, 0, kv->num_slots, kv->slot_stride, kMpRow, false)))
        return e;
    if (!aligned16(query->q) || !aligned16(query->out) || !aligned16(d_workspace) ||
        ((reinterpret_cast<uintptr_t>(query->lse) | reinterpret_cast<uintptr_t>(table->pages) |
          reinterpret_cast<uintptr_t>(table->lens)) & 3))
        return KAMERA_ERR_MISALIGNED;
    const MpNeed need = mp_need(p);
    if (workspace_bytes < need.bytes())
        return KAMERA_ERR_INVALID_ARGUMENT;
    using Span = std::pair<uintptr_t, uintptr_t>;
    auto bytes = [](const void* a, int64_t n) -> Span {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(a);
        return {lo, a ? lo + (uintptr_t)n : lo};
    };
    const int64_t rows = (int64_t)p.n_seqs * p.Hq;
    const Span in[] = {span(kv->kv, 1, 0, kv->num_slots, kv->slot_stride, kMpRow), bytes(query->q, rows * kMpRow * 2),
                       bytes(table->pages, (int64_t)p.n_seqs * p.max_pages * 4), bytes(table->lens, (int64_t)p.n_seqs * 4)};
    const Span outs[] = {bytes(query->out, rows * kMpDim * 2), bytes(query->lse, rows * 4),
                         bytes(d_workspace, (int64_t)need.bytes())};
    for (int i = 0; i < 3; ++i) {
        for (const Span& a : in)
            if (overlap(a, outs[i]))
                return KAMERA_ERR_INVALID_ARGUMENT;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j]))
                return KAMERA_ERR_INVALID_ARGUMENT;
    }
    p.out = static_cast<__nv_bfloat16*>(query->out);
    p.lse = query->lse;
    p.pages = table->pages;
    p.lens = table->lens;
    unsigned char* ws = static_cast<unsigned char*>(d_workspace);
    p.o = reinterpret_cast<float*>(ws);
    p.ml = reinterpret_cast<float2*>(ws + need.o);
    p.span = reinterpret_cast<int4*>(ws + need.o + need.ml);
    p.err = d_err;
    p.half_wait = half_wait(wait_limit_ns());
    p.withhold = test_withhold_loads() ? 1 : 0;
    p.box_rows = 16;
    while (p.box_rows < kMpTok && p.P % (2 * p.box_rows) == 0)
        p.box_rows *= 2;
    const int N = mp_heads(p.Hq);
    const int64_t map_rows = std::max<int64_t>(kv->num_slots, 8);   // a pool without a whole page has none to read
    if (!make_groups_map(&L.map_c, kv->kv, map_rows, kMpRow, kv->slot_stride, 2, p.box_rows / 8) ||
        !make_groups_map(&L.map_r, kv->kv, map_rows, kMpRow, kv->slot_stride, 1, p.box_rows / 8) ||
        !make_rows_map(&L.map_q, query->q, rows, kMpRow, kMpRow, 64, N))
        return KAMERA_ERR_CUDA;
    const cudaError_t ce = N == 16 ? mp_launch<16>(L, stream) : N == 32 ? mp_launch<32>(L, stream) : mp_launch<64>(L, stream);
    if (ce != cudaSuccess)
        return KAMERA_ERR_CUDA;
    if (p.ranges > 1) {
        // states of a row on average: a range ends in each but the last
        const bool many = p.ranges >= 8ll * p.n_seqs;
        if ((many ? launch_after(mla_merge_kernel<16, 4>, dim3(4 * (unsigned)rows), 512, 0, stream, true, p)
                  : launch_after(mla_merge_kernel<1, 1>, dim3((unsigned)rows), 128, 0, stream, true, p)) != cudaSuccess)
            return KAMERA_ERR_CUDA;
    }
    return KAMERA_OK;
}

}  // extern "C"
