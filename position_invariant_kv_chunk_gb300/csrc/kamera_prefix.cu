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
//                       two partial states
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
//   warp 8          producer: key and value tiles as 128B-swizzled TMA boxes of
//                   as many rows as a page holds in one piece, one box a lane,
//                   into a ring of five buffers (a tile of keys or of values
//                   each).  A value tile that the prefix ends in, or with a page
//                   outside the pool, comes by async copies, zero where no token
//                   is: a zero weight times what lies there must add nothing.
//   warp 9          MMA: one lane; the warp owns TMEM
// Every wait is bounded in time: on expiry KAMERA_DEVERR_TIMEOUT is raised, the
// roles leave their loops, the producer drains the copies it started and the
// MMA lane what it issued, and TMEM is freed.
#include <cstdint>
#include <cstring>

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
constexpr int kPxThreads = 320;
constexpr int kPxProd = 8, kPxMma = 9;
constexpr int kPxBuf = 5;              // ring buffers
constexpr int kPxMasks = 8;            // tiles whose masks are kept (the ring holds at most three)
constexpr float kPxLazy = 8.0f;        // log2 growth of the running maximum that forces a rescale
constexpr uint32_t kAtom = 16384;      // 128 rows x 128 bytes: 64 columns of a tile

template <int D>
struct PxLayout {
    static constexpr int NB = D / 64;
    static constexpr uint32_t kTile = NB * kAtom;
    static constexpr uint32_t kQ = 0;                         // [2 sides][NB atoms]
    static constexpr uint32_t kRing = 2 * kTile;
    static constexpr uint32_t kBar = kRing + kPxBuf * kTile;
    static constexpr uint32_t kBytes = kBar + 512 + 1024;     // + alignment slack
    // TMEM columns: scores (and weights) of A and B, outputs of A and B
    static constexpr uint32_t kTmS = 0, kTmO = 2 * kPxTok;
    static constexpr uint32_t kTmCols = 512;
    static_assert(kTmO + 2 * D <= kTmCols, "TMEM columns");
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct PxBars {
    uint64_t full[kPxBuf], empty[kPxBuf];
    uint64_t s_full[2], p_full[2], pv_done[2];
    uint64_t drained;
    uint32_t mask[kPxMasks];   // tile t (mod kPxMasks): 16-token pieces with tokens that count
    uint32_t tmem;
    int32_t abort;
};
static_assert(sizeof(PxBars) <= 512, "barrier block");

// What a CTA does, worked out alike by every role.
struct PxWork {
    int group, h, split, blk;
    int s0, rows;            // the group's first sequence, its rows (sequences x G)
    int len;                 // prefix tokens
    int t0, tiles;           // the split's tiles
    int n_side[2];           // tiles of side A, B (0: the side is idle)
    int row0[2];             // first row of side A, B
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
    if (p.two_tile) {
        w.row0[0] = w.blk * 2 * kPxRows;
        w.row0[1] = w.row0[0] + kPxRows;
        w.n_side[0] = w.row0[0] < w.rows ? w.tiles : 0;
        w.n_side[1] = w.row0[1] < w.rows ? w.tiles : 0;
    } else {
        w.row0[0] = w.row0[1] = 0;
        w.n_side[0] = w.rows > 0 ? (w.tiles + 1) / 2 : 0;
        w.n_side[1] = w.rows > 0 ? w.tiles / 2 : 0;
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

// One tile of keys (V = false) or values into buffer `dst`.
template <int D>
__device__ void px_load(const PagedLaunch& L, const PxWork& w, PxBars& b, uint32_t dst, uint32_t full, int t, bool values,
                        int lane)
{
    using Y = PxLayout<D>;
    const PagedParams& p = L.p;
    const int tok0 = (w.t0 + t) * kPxTok, ntok = min(kPxTok, w.len - tok0);
    const int32_t* table = p.prefix_pages + (int64_t)w.group * p.max_prefix_pages;
    // the pieces that hold tokens of pages inside the pool
    bool good = false;
    if (lane < kPxTok / 16 && 16 * lane < ntok) {
        const int page = __ldg(table + (tok0 + 16 * lane) / p.P);
        good = page >= 0 && page < p.num_pages;
        if (!good)
            raise_err(p.err, KAMERA_DEVERR_SLOT);
    }
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, good);
    const bool plain = ntok == kPxTok && mask == 0xFFu;
    if (values && !plain) {
        for (int e = lane; e < kPxTok * 8 * Y::NB; e += 32) {
            const int r = e / (8 * Y::NB), c = e % (8 * Y::NB);
            const uint32_t at = dst + (c >> 3) * kAtom + sw128(r, c & 7);
            if (r < ntok && ((mask >> (r >> 4)) & 1u)) {
                const int page = __ldg(table + (tok0 + r) / p.P);
                const int64_t row = (int64_t)page * p.P + (tok0 + r) % p.P;
                ptx::cp_async16(at, L.v + row * L.slot_stride + (int64_t)w.h * D + 8 * c);
            } else {
                ptx::st_shared_zero16(at);
            }
        }
        ptx::cp_async_commit();
        ptx::cp_async_wait<0>();
        ptx::fence_proxy_async();
        __syncwarp();
        if (lane == 0 && !p.withhold)
            ptx::mbar_arrive(full);
        return;
    }
    const int R = L.box_rows, boxes = (kPxTok / R) * Y::NB;
    // lane e's box: rows rp R .. of column block x (a box lies in one page)
    uint32_t bytes = 0;
    int row = 0;
    const int rp = lane / Y::NB, x = lane - rp * Y::NB;
    if (lane < boxes && rp * R < ntok && ((mask >> (rp * R / 16)) & 1u)) {
        const int tok = tok0 + rp * R;
        row = __ldg(table + tok / p.P) * p.P + tok % p.P;
        bytes = (uint32_t)R * 128u;
    }
    const uint32_t total = __reduce_add_sync(0xFFFFFFFFu, bytes);
    if (lane == 0) {
        if (!values)
            b.mask[t % kPxMasks] = mask;
        if (!p.withhold) {
            if (total > 0)
                ptx::mbar_arrive_expect_tx(full, total);
            else
                ptx::mbar_arrive(full);
        }
    }
    __syncwarp();
    if (bytes && !p.withhold)
        ptx::tma_load_2d(dst + x * kAtom + rp * R * 128, values ? &L.map_v : &L.map_k, w.h * D + 64 * x, row, full);
}

template <int D>
__device__ void px_producer(const PagedLaunch& L, const PxWork& w, PxBars& b, uint32_t ring, int lane)
{
    using Y = PxLayout<D>;
    const PagedParams& p = L.p;
    const bool two = p.two_tile != 0;
    const int n = 2 * w.tiles;
    int kt = 0, vt = 0;   // next tile of keys, of values
    int i = 0;
    for (; i < n; ++i) {
        const int buf = i % kPxBuf;
        if (i >= kPxBuf) {
            bool got = true;
            if (lane == 0)
                got = wmma16::tile_wait(ptx::smem_addr(&b.empty[buf]), ((uint32_t)(i / kPxBuf) & 1u) ^ 1u, &b.abort,
                                        p.err, p.wait_ns);
            if (!__shfl_sync(0xFFFFFFFFu, got ? 1 : 0, 0))
                break;
        }
        const bool values = !(kt < w.tiles && px_k_at(two, kt) == (uint32_t)i);
        px_load<D>(L, w, b, ring + buf * Y::kTile, ptx::smem_addr(&b.full[buf]), values ? vt++ : kt++, values, lane);
    }
    // the copies this warp started land before the CTA leaves
    if (lane == 0 && !p.withhold)
        for (int k = i > kPxBuf ? i - kPxBuf : 0; k < i; ++k)
            pf_drain_wait(ptx::smem_addr(&b.full[k % kPxBuf]), (uint32_t)(k / kPxBuf) & 1u, p.wait_ns);
    __syncwarp();
}

template <int D>
__device__ void px_mma(const PagedLaunch& L, const PxWork& w, PxBars& b, uint32_t sbase, uint32_t tm)
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
    auto scores = [&](int a, int n) -> bool {
        const int t = two ? n : 2 * n + a;
        const uint32_t at = px_k_at(two, t), buf = at % kPxBuf;
        if (!wait(&b.full[buf], at / kPxBuf))
            return false;
        ptx::tc_fence_after();
        const uint32_t dS = tm + Y::kTmS + a * kPxTok;
        const uint32_t aq = q_lo + (two ? a : 0) * (Y::kTile >> 4), bk = (r_lo + buf * (Y::kTile >> 4)) | (1u << 16);
        mma_ss<false>(dS, aq, bk, idS);
#pragma unroll
        for (int ks = 1; ks < D / 16; ++ks)
            mma_ss<true>(dS, aq + (ks >> 2) * (kAtom >> 4) + 2 * (ks & 3), bk + (ks >> 2) * (kAtom >> 4) + 2 * (ks & 3),
                         idS);
        ptx::umma_commit(ptx::smem_addr(&b.s_full[a]));
        if (!two || a == 1 || w.n_side[1] == 0)
            ptx::umma_commit(ptx::smem_addr(&b.empty[buf]));
        return true;
    };
    auto weigh = [&](int a, int n) -> bool {
        const int t = two ? n : 2 * n + a;
        const uint32_t at = px_v_at(two, t, w.tiles), buf = at % kPxBuf;
        if (!wait(&b.p_full[a], n) || !wait(&b.full[buf], at / kPxBuf))
            return false;
        ptx::tc_fence_after();
        const uint32_t dO = tm + Y::kTmO + a * D, aP = tm + Y::kTmS + a * kPxTok;
        const uint32_t bv = (r_lo + buf * (Y::kTile >> 4)) | ((kAtom >> 4) << 16);
        if (n == 0)
            mma_ts<false>(dO, aP, bv, idV);
        else
            mma_ts<true>(dO, aP, bv, idV);
#pragma unroll
        for (int ks = 1; ks < kPxTok / 16; ++ks)
            mma_ts<true>(dO, aP + 8 * ks, bv + (2048 >> 4) * ks, idV);
#pragma unroll
        for (int ks = 0; ks < kPxTok / 16; ++ks)
            mma_ts<true>(dO, aP + kPxTok / 2 + 8 * ks, bv + (2048 >> 4) * ks, idV);
        ptx::umma_commit(ptx::smem_addr(&b.pv_done[a]));
        if (!two || a == 1 || w.n_side[1] == 0)
            ptx::umma_commit(ptx::smem_addr(&b.empty[buf]));
        return true;
    };
    bool ok = true;
    for (int a = 0; a < 2 && ok; ++a)
        if (w.n_side[a] > 0)
            ok = scores(a, 0);
    for (int n = 0; n < w.n_side[0] && ok; ++n)
        for (int a = 0; a < 2 && ok; ++a)
            if (n < w.n_side[a]) {
                ok = weigh(a, n);
                if (ok && n + 1 < w.n_side[a])
                    ok = scores(a, n + 1);
            }
    // every MMA issued here completes before TMEM is freed
    ptx::umma_commit(ptx::smem_addr(&b.drained));
    pf_drain_wait(ptx::smem_addr(&b.drained), 0u, p.wait_ns);
}

// Side a's softmax, thread r = row r of the side = TMEM lane r.
template <int D>
__device__ void px_softmax(const PagedLaunch& L, const PxWork& w, PxBars& b, uint32_t tm, int a, int r)
{
    using Y = PxLayout<D>;
    const PagedParams& p = L.p;
    const int nt = w.n_side[a], row = w.row0[a] + r;
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
            float e0 = neg ? INFINITY : -INFINITY, e1 = e0, e2 = e0, e3 = e0;
            if (neg) {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    e0 = fminf(e0, __uint_as_float(s[0][j]));
                    e1 = fminf(e1, __uint_as_float(s[1][j]));
                    e2 = fminf(e2, __uint_as_float(s[2][j]));
                    e3 = fminf(e3, __uint_as_float(s[3][j]));
                }
                e0 = fminf(fminf(e0, e1), fminf(e2, e3));
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    e0 = fmaxf(e0, __uint_as_float(s[0][j]));
                    e1 = fmaxf(e1, __uint_as_float(s[1][j]));
                    e2 = fmaxf(e2, __uint_as_float(s[2][j]));
                    e3 = fmaxf(e3, __uint_as_float(s[3][j]));
                }
                e0 = fmaxf(fmaxf(e0, e1), fmaxf(e2, e3));
            }
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
            const uint64_t neg1 = ptx::f2_make(0xBF800000u, 0xBF800000u);
            uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t ph[32], pl[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const uint32_t* src = s[2 * half + (j >> 4)];
                    const int jj = 2 * (j & 15);
                    uint32_t a0, a1;
                    asm("mov.b64 {%0, %1}, %2;"
                        : "=r"(a0), "=r"(a1)
                        : "l"(ptx::f2_fma(ptx::f2_make(src[jj], src[jj + 1]), sl2x2, nmx2)));
                    const float p0 = pf_ex2(__uint_as_float(a0)), p1 = pf_ex2(__uint_as_float(a1));
                    const uint64_t pp = ptx::f2_make(__float_as_uint(p0), __float_as_uint(p1));
                    sum2[j & 1] = ptx::f2_add(sum2[j & 1], pp);
                    ph[j] = pack_bf16x2(p0, p1);
                    pl[j] = ptx::f2_to_bf16x2(ptx::f2_fma(ptx::f2_from_bf16x2(ph[j]), neg1, pp));
                }
                tmem_st32(tS + 32 * half, ph);
                tmem_st32(tS + kPxTok / 2 + 32 * half, pl);
            }
            uint32_t x0, x1;
            asm("mov.b64 {%0, %1}, %2;" : "=r"(x0), "=r"(x1) : "l"(ptx::f2_add(sum2[0], sum2[1])));
            l_run += __uint_as_float(x0) + __uint_as_float(x1);
            tmem_wait_st();
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_addr(&b.p_full[a]));
    }
    // ---- the partial state
    if (nt > 0 && ok) {
        if (!wmma16::tile_wait(ptx::smem_addr(&b.pv_done[a]), (uint32_t)(nt - 1) & 1u, &b.abort, p.err, p.wait_ns))
            ok = false;
        ok = __all_sync(0xFFFFFFFFu, ok);
        ptx::tc_fence_after();
    }
    if (idle)
        return;
    const int seq = w.s0 + row / p.G;
    const int64_t slot = ((int64_t)seq * p.H * p.G + w.h * p.G + row % p.G) * p.slots +
                         (p.two_tile ? w.split : 2 * w.split + a);
    if (nt > 0 && ok) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
            if (valid) {
                float* dst = p.o + slot * D + 32 * c;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4*>(dst + 4 * j) =
                        make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
        }
    }
    if (valid)   // a side without tiles leaves the empty state
        p.ml[slot] = nt > 0 && ok ? make_float2(m_run, l_run) : make_float2(-INFINITY, 0.f);
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
    PxWork w;
    px_work(p, w);
    if (threadIdx.x == 0 && w.h == 0 && w.split == 0 && w.blk == 0) {
        int s0, s1, len;
        if (!group_range(p, w.group, s0, s1, len))
            raise_err(p.err, KAMERA_DEVERR_DESCRIPTOR);
        if (p.prefix_lens[w.group] != len)
            raise_err(p.err, KAMERA_DEVERR_LEN);
    }
    if (w.n_side[0] == 0)   // no rows, or no tokens: nothing for either side
        return;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPxBuf; ++i) {
            ptx::mbar_init(ptx::smem_addr(&b.full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.empty[i]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(ptx::smem_addr(&b.s_full[a]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.p_full[a]), kPxRows);
            ptx::mbar_init(ptx::smem_addr(&b.pv_done[a]), 1);
        }
        ptx::mbar_init(ptx::smem_addr(&b.drained), 1);
        b.abort = 0;
        ptx::fence_barrier_init();
    }
    if (warp == kPxProd && lane == 0) {
        ptx::prefetch_tmap(&L.map_k);
        ptx::prefetch_tmap(&L.map_v);
    }
    if (warp == kPxMma) {
        ptx::tmem_alloc(ptx::smem_addr(&b.tmem), Y::kTmCols);
        ptx::tmem_relinquish();
    }
    // the query rows, K-major and 128B-swizzled; zero past the group's rows
    const int sides = p.two_tile ? 2 : 1;
    for (int e = threadIdx.x; e < sides * kPxRows * (D / 8); e += kPxThreads) {
        const int c = e % (D / 8), rr = e / (D / 8), a = rr >> 7, r = rr & (kPxRows - 1), row = w.row0[a] + r;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (row < w.rows)
            x = __ldg(reinterpret_cast<const uint4*>(
                p.q + (((int64_t)(w.s0 + row / p.G) * p.H + w.h) * p.G + row % p.G) * D + 8 * c));
        ptx::sts128(sbase + Y::kQ + a * Y::kTile + (c >> 3) * kAtom + sw128(r, c & 7), x.x, x.y, x.z, x.w);
    }
    ptx::fence_proxy_async();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tm = b.tmem;

    if (warp < 8)
        px_softmax<D>(L, w, b, tm, warp >> 2, threadIdx.x & (kPxRows - 1));
    else if (warp == kPxProd)
        px_producer<D>(L, w, b, sbase + Y::kRing, lane);
    else if (lane == 0)
        px_mma<D>(L, w, b, sbase, tm);

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
    prefix_kernel<D><<<ctas, kPxThreads, Y::kBytes, stream>>>(L);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefix(const PagedLaunch& L, cudaStream_t stream)
{
    return L.p.d == 128 ? launch_prefix_d<128>(L, stream) : launch_prefix_d<64>(L, stream);
}

}  // namespace kamera
