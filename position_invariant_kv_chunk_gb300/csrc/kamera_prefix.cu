// kamera_prefix.cu -- decode attention over a prefix that a batch shares, on the
// tensor cores.
//
// The sequences of a group attend over the same prefix, so per KV head the query
// heads of all of them are rows of one matrix: (sequences x G) x d against the
// prefix's keys, and the prefix is read once for the group where per-sequence
// decode reads it once each.  That turns a read-bound step (4 d G flops per 4 d
// bytes) into a matrix product: with 448 rows, 448 flops a byte, the tensor pipe
// is the bound.
//
// A CTA owns a share of the prefix's 128-token tiles (a split; there are as many
// as fill the SMs in the fewest rounds) for 256 rows, or for 128 when the groups
// are small.  It runs two sides, A and B, each a 128-row attention with its own
// scores, weights and output in TMEM and its own softmax warpgroup:
//   two tiles of rows   both sides see every tile of the split, so a tile is
//                       loaded once for 256 rows
//   one tile of rows    the sides take alternate tiles of the split, and leave
//                       two partial states (few tiles: side A takes them all)
// The MMA lane alternates between the sides -- P v of tile n and the scores of
// tile n + 1 of A while B's softmax runs, and the other way round -- so the
// tensor pipe works through either side's softmax.  Per side and tile:
//   S [128 x 128]  = Q K^T                  (both from shared memory)
//   O [128 x d]   += [P_hi | P_lo] V        (P from TMEM, over S's columns)
// The weights are not bf16 values and enter as a hi + lo pair (about 16
// significant bits), as in the library's other attention kernels: half of P V's
// MMAs, for an output whose error is its rounding to bf16 alone.
//   warps 0-3, 4-7  softmax of side A, B: thread = row = TMEM lane; running
//                   maximum with lazy rescaling (only when it grows by more than
//                   2^8), at the end the partial state into the workspace
//   warps 8, 9      producers of keys and of values: 128B-swizzled TMA boxes of
//                   whole rows, as many as a page holds in one piece, one box a
//                   lane, into a ring of five buffers (a tile of keys or of
//                   values each).  A value tile that the prefix ends in, or with
//                   a page outside the pool, comes by async copies, zero where no
//                   token is: a zero weight times what lies there must add nothing.
//   warp 10         MMA; the warp owns TMEM (warp 11 idles: registers are moved
//                   between whole warpgroups)
// 448 rows over 98304 tokens of four heads of 128 (90.9 GFLOP, 136 with the pairs):
// 98 us, tensor- and power-bound (the clock falls to about 1.6 GHz); an MMA's issue is
// 3217 of the 3870 cycles of a pair of tiles.  The pairs are a third
// of the MMAs; weights rounded to bf16 once would cost the output a sqrt(2) larger
// error.  Four prefixes of 4099 tokens of 32 MHA heads, 16 rows each (268 MB): 50 us,
// 5.4 TB/s.  One tile of keys: 8 us, all latency (entry, table, first keys, scores,
// weights, values, the state's way out).
// Every wait is bounded in time: on expiry KAMERA_DEVERR_TIMEOUT is raised, the
// roles leave their loops, the producers drain the copies they started and the
// MMA lane what it issued, and TMEM is freed.
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "kamera_common.cuh"
#include "kamera_internal.h"
#include "kamera_paged.h"
#include "kamera_ptx.cuh"
#include "kamera_tc.cuh"
#include "kamera_warpmma.cuh"

namespace kamera {

namespace {

using namespace tc;

constexpr int kPxRows = 128;           // rows of a side = MMA M = TMEM lanes
constexpr int kPxTok = 128;            // tokens of a tile = MMA N of the scores
constexpr int kPxThreads = 384;
constexpr int kPxProdK = 8, kPxProdV = 9, kPxMma = 10;
constexpr int kPxBuf = 5;              // ring buffers
constexpr int kPxMasks = 8;            // tiles whose masks are kept (the ring holds at most three)
constexpr float kPxLazy = 8.0f;        // log2 growth of the running maximum that forces a rescale
constexpr uint32_t kAtom = 1024;       // 8 rows x 128 bytes, 128B-swizzled

template <int D>
struct PxLayout {
    static constexpr int NB = D / 64;
    // A tile (of Q, K or V): [16 groups of 8 rows][NB blocks of 64 columns][8][128 bytes]
    static constexpr uint32_t kGroup = NB * kAtom;
    static constexpr uint32_t kTile = 16 * kGroup;
    // descriptor high word: groups kGroup apart, version 1, 128-byte swizzle
    static constexpr uint32_t kHi = (kGroup >> 4) | (1u << 14) | (2u << 29);
    static constexpr uint32_t kOutRow = D * 4 + 16;           // a staged output row (padded)
    static constexpr uint32_t kQ = 0;                         // [2 sides][NB atoms]
    static constexpr uint32_t kRing = 2 * kTile;
    static constexpr uint32_t kBar = kRing + kPxBuf * kTile;
    static constexpr uint32_t kBytes = kBar + 512 + 1024;     // + alignment slack
    // TMEM columns: scores (and weights) of A and B, outputs of A and B
    static constexpr uint32_t kTmS = 0, kTmO = 2 * kPxTok;
    static constexpr uint32_t kTmCols = 512;
    static_assert(kTmO + 2 * D <= kTmCols, "TMEM columns");
    static_assert(kBytes <= 227 * 1024, "shared memory");
    static_assert(2 * kPxRows * kOutRow <= kRing + kPxBuf * kTile, "staged outputs");
    // 16-byte piece c (of D / 8) of row r of a tile
    static __device__ __forceinline__ uint32_t at(int r, int c)
    {
        return (uint32_t)(r >> 3) * kGroup + (uint32_t)(c >> 3) * kAtom + sw128(r & 7, c & 7);
    }
};

struct PxBars {
    uint64_t full[kPxBuf], empty[kPxBuf];
    uint64_t q_full;           // the query rows are in shared memory
    uint64_t s_full[2], p_full[2][2], pv_done[2];   // p_full: tokens 0-63, 64-127 of the tile
    uint64_t drained;
    uint32_t mask[kPxMasks];   // tile t (mod kPxMasks): 16-token pieces with tokens that count
    uint32_t tmem;
    int32_t abort;
};
static_assert(sizeof(PxBars) <= 512, "barrier block");

// What a CTA does, worked out alike by every role.
struct PxWork {
    int group, h, split, blk;
    int s0, rows;            // the group's first sequence; where the CTA's rows (sequences x G) end
    int len;                 // prefix tokens
    int t0, tiles;           // the split's tiles
    int tiles_a, tiles_b;    // tiles of side A, B (0: the side is idle)
    int row_a, row_b;        // first row of side A, B
    __device__ __forceinline__ int n_side(int a) const { return a ? tiles_b : tiles_a; }
    __device__ __forceinline__ int row0(int a) const { return a ? row_b : row_a; }
};

__device__ __forceinline__ void px_work(const PagedParams& p, PxWork& w)
{
    int id = blockIdx.x;
    w.blk = id % p.row_blocks;
    id /= p.row_blocks;
    w.split = id % p.prefix_splits;
    id /= p.prefix_splits;
    w.h = id % p.H;
    w.group = id / p.H;
    int s1;
    const bool good = group_range(p, w.group, w.s0, s1, w.len);
    w.rows = good ? (s1 - w.s0) * p.G : 0;
    const int all = w.len > 0 ? (w.len - 1) / kPxTok + 1 : 0;
    w.t0 = w.split * p.prefix_split;
    w.tiles = max(0, min(p.prefix_split, all - w.t0));
    w.row_a = w.blk * p.block_rows;   // one tile of rows: a single block
    w.rows = min(w.rows, w.row_a + p.block_rows);
    w.row_b = p.two_tile ? w.row_a + kPxRows : 0;
    if (p.two_tile) {
        w.tiles_a = w.row_a < w.rows ? w.tiles : 0;
        w.tiles_b = w.row_b < w.rows ? w.tiles : 0;
    } else {
        w.tiles_a = w.rows > 0 ? (w.tiles + 1) / 2 : 0;
        w.tiles_b = w.rows > 0 ? w.tiles / 2 : 0;
    }
}

// Place of tile t's keys and values in the ring's fill order.  Both sides on
// every tile: K0 V0 K1 V1 ...; alternate tiles: K0 K1 V0 K2 V1 K3 V2 ..., the
// order in which the MMA lane needs them.
__device__ __forceinline__ uint32_t px_k_at(bool two, int t) { return two ? 2u * t : (t < 2 ? t : 2u * t - 1); }
__device__ __forceinline__ uint32_t px_v_at(bool two, int t, int tiles)
{
    return two ? 2u * t + 1 : (t == tiles - 1 ? 2u * tiles - 1 : 2u * t + 2);
}

// The page of tile t's 16-token piece `lane` (0..7); -1 past the prefix.
__device__ __forceinline__ int px_page(const PagedParams& p, const PxWork& w, int t, int lane)
{
    const int tok = (w.t0 + t) * kPxTok + 16 * lane;
    return lane < kPxTok / 16 && t < w.tiles && tok < w.len
               ? p.prefix_pages[(int64_t)w.group * p.max_prefix_pages + tok / p.P]
               : -1;
}

// The producer of the keys (VALUES false) or the values: every tile of the split,
// in order, into its places in the ring.  A page lies in one box of `box_rows`
// rows or in several; lane l looks up and issues box l.  The next tile's pages
// are looked up before the wait for a free buffer, and the two producers work
// side by side: a fill is all latency (table, barrier, issue), and one warp
// doing both had the tensor pipe wait for it.
template <int D, bool VALUES>
__device__ void px_producer(const PagedLaunch& L, const PxWork& w, PxBars& b, uint32_t ring, int lane, int first_page)
{
    using Y = PxLayout<D>;
    const PagedParams& p = L.p;
    const bool two = p.two_tile != 0;
    const int32_t* table = p.prefix_pages + (int64_t)w.group * p.max_prefix_pages;
    const int R = L.box_rows, boxes = kPxTok / R;
    int next = first_page;
    int t = 0;
    bool ok = true;
    for (; t < w.tiles; ++t) {
        const int tok0 = (w.t0 + t) * kPxTok, ntok = min(kPxTok, w.len - tok0), page = next;
        next = px_page(p, w, t + 1, lane);
        const bool in = lane < kPxTok / 16 && 16 * lane < ntok, good = in && page >= 0 && page < p.num_pages;
        if (in && !good)
            raise_err(p.err, KAMERA_DEVERR_SLOT);
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, good);
        const uint32_t at = VALUES ? px_v_at(two, t, w.tiles) : px_k_at(two, t), buf = at % kPxBuf, lap = at / kPxBuf;
        const uint32_t dst = ring + buf * Y::kTile, full = ptx::smem_addr(&b.full[buf]);
        if (lap > 0) {
            bool got = true;
            if (lane == 0)
                got = wmma16::tile_wait(ptx::smem_addr(&b.empty[buf]), (lap & 1u) ^ 1u, &b.abort, p.err, p.wait_ns);
            ok = __shfl_sync(0xFFFFFFFFu, got ? 1 : 0, 0) != 0;
            if (!ok)
                break;
        }
        if (VALUES && (ntok < kPxTok || mask != 0xFFu)) {
            // the prefix ends in this tile, or a page is missing: zero where no token is
            for (int e = lane; e < kPxTok * 8 * Y::NB; e += 32) {
                const int r = e / (8 * Y::NB), c = e % (8 * Y::NB);
                if (r < ntok && ((mask >> (r >> 4)) & 1u)) {
                    const int64_t row = (int64_t)table[(tok0 + r) / p.P] * p.P + (tok0 + r) % p.P;
                    ptx::cp_async16(dst + Y::at(r, c), L.v + row * L.slot_stride + (int64_t)w.h * D + 8 * c);
                } else {
                    ptx::st_shared_zero16(dst + Y::at(r, c));
                }
            }
            ptx::cp_async_commit();
            ptx::cp_async_wait<0>();
            ptx::fence_proxy_async();
            __syncwarp();
            if (lane == 0 && !p.withhold)
                ptx::mbar_arrive(full);
            continue;
        }
        // box l covers rows l R .. l R + R - 1, whose page piece l R / 16 looked up
        const int off = lane * R, from = __shfl_sync(0xFFFFFFFFu, page, (off / 16) & 31);
        const bool mine = lane < boxes && off < ntok && ((mask >> (off / 16)) & 1u);
        const uint32_t total = __popc(__ballot_sync(0xFFFFFFFFu, mine)) * (uint32_t)(R / 8) * Y::kGroup;
        if (lane == 0) {
            if (!VALUES)
                b.mask[t % kPxMasks] = mask;
            if (!p.withhold) {
                if (total > 0)
                    ptx::mbar_arrive_expect_tx(full, total);
                else
                    ptx::mbar_arrive(full);
            }
        }
        __syncwarp();
        if (mine && !p.withhold)
            ptx::tma_load_4d(dst + (uint32_t)(off / 8) * Y::kGroup, VALUES ? &L.map_v : &L.map_k, 0, 0, w.h * Y::NB,
                             (from * p.P + (tok0 + off) % p.P) >> 3, full);
    }
    // Without a timeout the MMA lane has waited for every fill.  After one, the
    // copies this warp started land before the CTA leaves.
    if (lane == 0 && !p.withhold && *static_cast<volatile int32_t*>(&b.abort))
        for (int k = max(0, t - kPxBuf); k < t; ++k) {
            const uint32_t at = VALUES ? px_v_at(two, k, w.tiles) : px_k_at(two, k);
            pf_drain_wait(ptx::smem_addr(&b.full[at % kPxBuf]), (at / kPxBuf) & 1u, p.wait_ns);
        }
    __syncwarp();
}

// One lane of the (converged) warp: the compiler knows that a branch on it holds
// a single thread, and hands the MMA its operands without a loop over the lanes
// that might differ (which cost 35 of 100 cycles an MMA in a branch on lane 0).
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// The MMA lane.  TMEM addresses are offsets: the CTA holds all 512 columns, so
// its allocation starts at address 0.
template <int D>
__device__ void px_mma(const PagedLaunch& L, const PxWork& w, PxBars& b, uint32_t sbase)
{
    using Y = PxLayout<D>;
    const PagedParams& p = L.p;
    const bool two = p.two_tile != 0;
    constexpr uint32_t idS = ptx::idesc_bf16_f32(kPxRows, kPxTok);
    constexpr uint32_t idV = ptx::idesc_bf16_f32(kPxRows, D) | (1u << 16);   // value rows: MN-major
    const uint32_t q_lo = ((sbase + Y::kQ) >> 4) | (1u << 16);
    const uint32_t r_lo = (sbase + Y::kRing) >> 4;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return wmma16::tile_wait(ptx::smem_addr(bar), parity & 1u, &b.abort, p.err, p.wait_ns);
    };
    // scores of side a's tile n; the tile's keys are free after its last side
    auto scores = [&](auto side, int n) -> bool {
        constexpr int a = decltype(side)::value;
        const int t = two ? n : 2 * n + a;
        const uint32_t at = px_k_at(two, t), buf = at % kPxBuf;
        if (!wait(&b.full[buf], at / kPxBuf))
            return false;
        ptx::tc_fence_after();
        constexpr uint32_t dS = Y::kTmS + a * kPxTok;
        const uint32_t aq = q_lo + (two ? a : 0) * (Y::kTile >> 4), bk = (r_lo + buf * (Y::kTile >> 4)) | (1u << 16);
        mma_ss<false, Y::kHi>(dS, aq, bk, idS);
#pragma unroll
        for (int ks = 1; ks < D / 16; ++ks)
            mma_ss<true, Y::kHi>(dS, aq + (ks >> 2) * (kAtom >> 4) + 2 * (ks & 3),
                                    bk + (ks >> 2) * (kAtom >> 4) + 2 * (ks & 3), idS);
        ptx::umma_commit(ptx::smem_addr(&b.s_full[a]));
        if (!two || a == 1 || w.tiles_b == 0)
            ptx::umma_commit(ptx::smem_addr(&b.empty[buf]));
        return true;
    };
    auto weigh = [&](auto side, int n) -> bool {
        constexpr int a = decltype(side)::value;
        const int t = two ? n : 2 * n + a;
        const uint32_t at = px_v_at(two, t, w.tiles), buf = at % kPxBuf;
        if (!wait(&b.full[buf], at / kPxBuf))
            return false;
        constexpr uint32_t dO = Y::kTmO + a * D, aP = Y::kTmS + a * kPxTok;
        const uint32_t bv = (r_lo + buf * (Y::kTile >> 4)) | ((kAtom >> 4) << 16);
#pragma unroll
        for (int half = 0; half < 2; ++half) {   // the first 64 tokens while the others' weights are computed
            if (!wait(&b.p_full[a][half], n))
                return false;
            ptx::tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int ks = 4 * half + k;
                const uint32_t v = bv + (2 * Y::kGroup >> 4) * ks;
                if (ks == 0 && n == 0)
                    mma_ts<false, Y::kHi>(dO, aP, v, idV);
                else
                    mma_ts<true, Y::kHi>(dO, aP + 8 * ks, v, idV);
                mma_ts<true, Y::kHi>(dO, aP + kPxTok / 2 + 8 * ks, v, idV);
            }
        }
        ptx::umma_commit(ptx::smem_addr(&b.pv_done[a]));
        if (!two || a == 1 || w.tiles_b == 0)
            ptx::umma_commit(ptx::smem_addr(&b.empty[buf]));
        return true;
    };
    constexpr auto A = std::integral_constant<int, 0>{};
    constexpr auto B = std::integral_constant<int, 1>{};
    bool ok = wait(&b.q_full, 0) && scores(A, 0) && (w.tiles_b == 0 || scores(B, 0));
    for (int n = 0; n < w.tiles_a && ok; ++n) {
        ok = weigh(A, n) && (n + 1 >= w.tiles_a || scores(A, n + 1));
        if (ok && n < w.tiles_b)
            ok = weigh(B, n) && (n + 1 >= w.tiles_b || scores(B, n + 1));
    }
    // every MMA issued here completes before TMEM is freed
    ptx::umma_commit(ptx::smem_addr(&b.drained));
    pf_drain_wait(ptx::smem_addr(&b.drained), 0u, p.wait_ns);
}

__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return d;
}
__device__ __forceinline__ float min3(float a, uint32_t b, uint32_t c)
{
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return d;
}

// Row `row` of a group counted over the batch, n_seqs x H x G rows: sequence row / G
// of the group, head h G + row mod G.  The quotient by one multiplication (a group
// has fewer than 2^24 rows: its blocks of 256 are at most 65535).
struct RowOf {
    int64_t first, step;
    uint32_t inv;   // 2^32 / G, rounded up; 0: G is 1
    __device__ __forceinline__ RowOf(const PagedParams& p, const PxWork& w)
        : first(((int64_t)w.s0 * p.H + w.h) * p.G), step((int64_t)(p.H - 1) * p.G),
          inv(p.G > 1 ? 0xFFFFFFFFu / (uint32_t)p.G + 1u : 0u)
    {
    }
    __device__ __forceinline__ int64_t operator()(int row) const
    {
        return first + row + (int64_t)(inv ? __umulhi((uint32_t)row, inv) : (uint32_t)row) * step;
    }
};

// The query rows of side a into shared memory (K-major, zero past the group's
// rows) by the side's 128 threads, a row's pieces on neighbouring lanes; all of
// a thread's loads are in flight before the first store.
template <int D>
__device__ __forceinline__ void px_stage_q(const PagedParams& p, const PxWork& w, PxBars& b, uint32_t sbase, int a, int r)
{
    using Y = PxLayout<D>;
    constexpr int PC = D / 8, RS = kPxRows / PC, N = kPxRows / RS;   // pieces of a row, rows a step, steps
    uint4 x[N];
    const int c = r % PC;
    const RowOf row_of(p, w);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int row = w.row0(a) + i * RS + r / PC;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row < w.rows)
            x[i] = *reinterpret_cast<const uint4*>(p.q + row_of(row) * D + 8 * c);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        ptx::sts128(sbase + Y::kQ + a * Y::kTile + Y::at(i * RS + r / PC, c), x[i].x, x[i].y, x[i].z, x[i].w);
    ptx::fence_proxy_async();
    ptx::mbar_arrive(ptx::smem_addr(&b.q_full));
}

// Side a's softmax, thread r = row r of the side = TMEM lane r.
template <int D>
__device__ void px_softmax(const PagedLaunch& L, const PxWork& w, PxBars& b, uint32_t sbase, uint32_t tm, int a, int r)
{
    using Y = PxLayout<D>;
    const PagedParams& p = L.p;
    const int nt = w.n_side(a), row = w.row0(a) + r;
    const bool valid = row < w.rows;
    const bool idle = !__any_sync(0xFFFFFFFFu, valid);   // no row of this warp counts
    const uint32_t lanes = tm + ((uint32_t)(r & ~31) << 16);
    const uint32_t tS = lanes + Y::kTmS + a * kPxTok, tO = lanes + Y::kTmO + a * D;
    // scores in log2 units; a scale of zero becomes the smallest normal float, so that
    // a masked score stays infinite under it (a score of 2^100 still rounds to 0)
    const float sl2 = p.scale == 0.f ? 1.17549435e-38f : p.scale * 1.4426950408889634f;
    const bool neg = sl2 < 0.f;
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int n = 0; n < nt; ++n) {
        if (!wmma16::tile_wait(ptx::smem_addr(&b.s_full[a]), (uint32_t)n & 1u, &b.abort, p.err, p.wait_ns))
            ok = false;
        if (!__all_sync(0xFFFFFFFFu, ok)) {
            ok = false;
            break;
        }
        ptx::tc_fence_after();
        if (!idle) {
            const int t = p.two_tile ? n : 2 * n + a;
            const int ntok = min(kPxTok, w.len - (w.t0 + t) * kPxTok);
            const uint32_t mask = *reinterpret_cast<volatile uint32_t*>(&b.mask[t % kPxMasks]);
            uint32_t s[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                tmem_ld32_issue(tS + 32 * c, s[c]);
            tmem_ld_wait128(s);
            if (ntok < kPxTok || mask != 0xFFu) {   // tokens that do not count: weight 0
                const uint32_t out = neg ? 0x7F800000u : 0xFF800000u;
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int col = 32 * c + j;
                        if (col >= ntok || !((mask >> (col >> 4)) & 1u))
                            s[c][j] = out;
                    }
            }
            // the row's extreme score: three inputs an instruction, eight chains
            float e[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t* v = &s[k >> 1][16 * (k & 1)];
                e[k] = neg ? fminf(__uint_as_float(v[0]), __uint_as_float(v[1]))
                           : fmaxf(__uint_as_float(v[0]), __uint_as_float(v[1]));
            }
            if (neg) {
#pragma unroll
                for (int j = 2; j < 16; j += 2)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        e[k] = min3(e[k], s[k >> 1][16 * (k & 1) + j], s[k >> 1][16 * (k & 1) + j + 1]);
            } else {
#pragma unroll
                for (int j = 2; j < 16; j += 2)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        e[k] = max3(e[k], s[k >> 1][16 * (k & 1) + j], s[k >> 1][16 * (k & 1) + j + 1]);
            }
#pragma unroll
            for (int d = 4; d >= 1; d /= 2)
#pragma unroll
                for (int k = 0; k < d; ++k)
                    e[k] = neg ? fminf(e[k], e[k + d]) : fmaxf(e[k], e[k + d]);
            const float e0 = e[0];
            const float m_new = fmaxf(m_run, sl2 * e0);
            if (n == 0) {
                m_run = m_new;   // O is still empty
            } else if (__any_sync(0xFFFFFFFFu, m_new > m_run + kPxLazy)) {
                const float f = m_new == -INFINITY ? 1.f : pf_ex2(m_run - m_new);
                l_run *= f;
                m_run = m_new;
                if (!wmma16::tile_wait(ptx::smem_addr(&b.pv_done[a]), (uint32_t)(n - 1) & 1u, &b.abort, p.err, p.wait_ns))
                    ok = false;
                ok = __all_sync(0xFFFFFFFFu, ok);
                ptx::tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(tO + 32 * c, o);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                    tmem_st32(tO + 32 * c, o);
                }
            }
            // weights 2^(sl2 s - m) as hi + lo pairs over the scores' columns
            const float ref = m_run == -INFINITY ? 0.f : m_run;
            const uint64_t sl2x2 = ptx::f2_make(__float_as_uint(sl2), __float_as_uint(sl2));
            const uint64_t nmx2 = ptx::f2_make(__float_as_uint(-ref), __float_as_uint(-ref));
            const uint64_t less = ptx::f2_make(__float_as_uint(kLessHi), __float_as_uint(kLessHi));
            uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
            for (int c = 0; c < 4; ++c) {   // 32 tokens: 16 columns of hi, 16 of lo
                uint32_t ph[16], pl[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    uint32_t a0, a1;
                    asm("mov.b64 {%0, %1}, %2;"
                        : "=r"(a0), "=r"(a1)
                        : "l"(ptx::f2_fma(ptx::f2_make(s[c][2 * j], s[c][2 * j + 1]), sl2x2, nmx2)));
                    const float p0 = pf_ex2(__uint_as_float(a0)), p1 = pf_ex2(__uint_as_float(a1));
                    const uint64_t pp = ptx::f2_make(__float_as_uint(p0), __float_as_uint(p1));
                    sum2[j & 1] = ptx::f2_add(sum2[j & 1], pp);
                    ph[j] = weight_hi(p0, p1);
                    pl[j] = ptx::f2_to_bf16x2(ptx::f2_fma(ptx::f2_from_bf16x2(ph[j]), less, pp));
                }
                tmem_st16(tS + 16 * c, ph);
                tmem_st16(tS + kPxTok / 2 + 16 * c, pl);
                if (c == 1) {
                    tmem_wait_st();
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(ptx::smem_addr(&b.p_full[a][0]));
                }
            }
            uint32_t x0, x1;
            asm("mov.b64 {%0, %1}, %2;" : "=r"(x0), "=r"(x1) : "l"(ptx::f2_add(sum2[0], sum2[1])));
            l_run += __uint_as_float(x0) + __uint_as_float(x1);
            tmem_wait_st();
        } else {
            ptx::tc_fence_before();
            ptx::mbar_arrive(ptx::smem_addr(&b.p_full[a][0]));
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_addr(&b.p_full[a][1]));
    }
    // ---- the partial state: a row through shared memory (Q and the ring are free once
    // both sides are done), copied out in one piece: rows written from the registers,
    // 16 bytes of 32 rows at a time, cost the long prefix above 24 us
    if (nt > 0 && ok) {
        if (!wmma16::tile_wait(ptx::smem_addr(&b.pv_done[a]), (uint32_t)(nt - 1) & 1u, &b.abort, p.err, p.wait_ns))
            ok = false;
        ok = __all_sync(0xFFFFFFFFu, ok);
        ptx::tc_fence_after();
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (idle)
        return;
    const uint32_t mine = sbase + (uint32_t)(a * kPxRows + r) * Y::kOutRow;
    if (nt > 0 && ok) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                ptx::sts128(mine + 128 * c + 16 * j, o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
    }
    if (!valid)
        return;
    const int64_t slot = RowOf(p, w)(row) * p.slots + (p.two_tile ? w.split : 2 * w.split + a);
    const bool some = nt > 0 && ok;   // a side without tiles leaves the empty state
    p.ml[slot] = some ? make_float2(m_run, l_run) : make_float2(-INFINITY, 0.f);
    if (!some)
        return;
    ptx::fence_proxy_async();
    ptx::bulk_s2g(p.o + slot * D, mine, D * 4);
    ptx::bulk_commit();
    ptx::bulk_wait_all();
}

template <int D>
__global__ void __launch_bounds__(kPxThreads, 1) prefix_kernel(const __grid_constant__ PagedLaunch L)
{
    using Y = PxLayout<D>;
    const PagedParams& p = L.p;
    extern __shared__ __align__(16) unsigned char raw[];
    const uint32_t at = ptx::smem_addr(raw), pad = (1024u - (at & 1023u)) & 1023u, sbase = at + pad;
    PxBars& b = *reinterpret_cast<PxBars*>(raw + pad + Y::kBar);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ptx::grid_wait();
    ptx::grid_launch_next();
    PxWork w;
    px_work(p, w);
    if (threadIdx.x == 0 && w.h == 0 && w.split == 0 && w.blk == 0) {
        int s0, s1, len;
        if (!group_range(p, w.group, s0, s1, len))
            raise_err(p.err, KAMERA_DEVERR_DESCRIPTOR);
        if (p.prefix_lens[w.group] != len)
            raise_err(p.err, KAMERA_DEVERR_LEN);
    }
    if (w.tiles_a == 0)   // no rows, or no tokens: nothing for either side
        return;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPxBuf; ++i) {
            ptx::mbar_init(ptx::smem_addr(&b.full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.empty[i]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(ptx::smem_addr(&b.s_full[a]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.p_full[a][0]), kPxRows);
            ptx::mbar_init(ptx::smem_addr(&b.p_full[a][1]), kPxRows);
            ptx::mbar_init(ptx::smem_addr(&b.pv_done[a]), 1);
        }
        ptx::mbar_init(ptx::smem_addr(&b.q_full), (p.two_tile ? 2 : 1) * kPxRows);
        ptx::mbar_init(ptx::smem_addr(&b.drained), 1);
        b.abort = 0;
        ptx::fence_barrier_init();
    }
    if (warp == kPxProdK && lane == 0) {
        ptx::prefetch_tmap(&L.map_k);
        ptx::prefetch_tmap(&L.map_v);
    }
    int first_page = -1;   // the producers' first look-up, in flight over the barrier below
    if (warp == kPxProdK || warp == kPxProdV)
        first_page = px_page(p, w, 0, lane);
    if (warp == kPxMma) {
        ptx::tmem_alloc(ptx::smem_addr(&b.tmem), Y::kTmCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tm = b.tmem;

    // Registers: the softmax warps hold a row of 128 scores, the others next to
    // nothing (256 x 208 + 128 x 56 of the launch's 384 x 168).
    if (warp < 8) {
        ptx::setmaxnreg_inc<208>();
        const int a = warp >> 2, r = threadIdx.x & (kPxRows - 1);
        if (p.two_tile || a == 0)
            px_stage_q<D>(p, w, b, sbase, a, r);
        px_softmax<D>(L, w, b, sbase, tm, a, r);
    } else {
        ptx::setmaxnreg_dec<56>();
        if (warp == kPxProdK)
            px_producer<D, false>(L, w, b, sbase + Y::kRing, lane, first_page);
        else if (warp == kPxProdV)
            px_producer<D, true>(L, w, b, sbase + Y::kRing, lane, first_page);
        else if (warp == kPxMma && elect_one())
            px_mma<D>(L, w, b, sbase);
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kPxMma) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tm, Y::kTmCols);
    }
}

template <int D>
cudaError_t launch_prefix_d(const PagedLaunch& L, cudaStream_t stream)
{
    using Y = PxLayout<D>;
    // set at every launch: the attribute belongs to the current device's context
    const cudaError_t e =
        cudaFuncSetAttribute(prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Y::kBytes);
    if (e != cudaSuccess)
        return e;
    const unsigned ctas = (unsigned)L.p.n_groups * L.p.H * L.p.row_blocks * L.p.prefix_splits;
    return launch_after(prefix_kernel<D>, dim3(ctas), kPxThreads, Y::kBytes, stream, true, L);
}

}  // namespace

cudaError_t launch_prefix(const PagedLaunch& L, cudaStream_t stream)
{
    return L.p.d == 128 ? launch_prefix_d<128>(L, stream) : launch_prefix_d<64>(L, stream);
}

}  // namespace kamera
