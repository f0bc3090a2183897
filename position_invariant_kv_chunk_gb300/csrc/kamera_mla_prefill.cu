// kamera_mla_prefill.cu -- MLA prefill attention over expanded rows, on the tensor
// cores: heads of 128 + 64 key columns (the rope part shared by the heads) and 128
// value columns, ragged sequences, causal mask.
//
// A pair of a query and a row costs 2 (192 + 128) flops, the exponential one MUFU
// operation: for a 128 x 128 tile 1280 cycles of the tensor pipe against 1024 (half
// that on this chip) of the MUFU, so the tensor pipe is the bound as long as it never
// waits for a softmax.  A CTA therefore has two sides of 128 queries each, A and B,
// with their own scores, weights and output in TMEM (2 x 128 + 2 x 128 columns: all of
// it) and their own softmax warpgroup; the MMA lane alternates between them:
//   S [128 x 128]  = Q [128 x 192] K^T      (both from shared memory)
//   O [128 x 128] += P V                    (P from TMEM, over S's columns, bf16)
// Both sides see the same rows, so a row is read once for 256 queries; or, where there
// are too few queries to fill the GPU that way, the sides have the same 128 queries and
// every second tile of rows each (SPLIT), and join their states at the end.  The weights are
// rounded to bf16 (2^-8 of each at the most): a hi + lo pair, as the library's decode
// kernels take, would be 40% more MMAs here, where they are the bound.
//   warps 0-3, 4-7  softmax of side A, B: thread = query = TMEM lane; running maximum
//                   with lazy rescaling (only when it grows by more than 2^8)
//   warp 8          producer: 128B-swizzled TMA boxes of 64 columns into a ring of eight
//                   (SPLIT: eleven) 16 KB units: a tile is three of keys (64 columns x 128 rows) and two
//                   of values (128 columns x 64 rows, so that an MMA takes N = 128 from
//                   one unit: 67 cycles, where two of N = 64 take 100)
//   warp 10         MMA; it owns TMEM (warps 9, 11 idle: registers are moved between
//                   whole warpgroups)
// Blocks of queries with the most rows to see start first.  Every wait is bounded.
// Measured, calls back to back on data in turn: 4 prompts of up to 4096 tokens, 16 heads,
// in 209 us (1275 TFLOP/s; over one prompt's rows again and again, which L2 holds in part,
// 189), 777 queries behind 1296 rows in 22.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <cuda.h>
#include <type_traits>

#include "kamera_common.cuh"
#include "kamera_hostcheck.h"
#include "kamera_internal.h"
#include "kamera_ptx.cuh"
#include "kamera_tc.cuh"
#include "kamera_warpmma.cuh"

namespace kamera {

namespace {

using namespace tc;

constexpr int kPrRows = 128, kPrTok = 128;
constexpr int kPrQk = 192, kPrNope = 128, kPrV = 128;
constexpr int kPrThreads = 384;
constexpr int kPrProd = 8, kPrMma = 10;
constexpr int kPrTile = 5;              // units of a tile: three of keys, two of values
constexpr uint32_t kPrUnit = 16384;     // 128 rows x 128 bytes
constexpr float kPrLazy = 8.0f;
// Queries ([1 or 2 sides][3 blocks of 64 columns][128 rows][128 bytes]) and the ring share
// 14 units: one block of queries leaves the ring eleven, two leave it eight.
template <bool SPLIT>
struct PrLayout {
    static constexpr int kQUnits = SPLIT ? 3 : 6, kUnits = 14 - kQUnits;
    static constexpr int kQueries = SPLIT ? kPrRows : 2 * kPrRows;   // of a CTA
};
constexpr uint32_t kPrBar = 14 * kPrUnit;
constexpr uint32_t kPrOdd = kPrBar + 512;   // [NaN, +inf, -inf][128 value columns]: the first masked row that holds one
constexpr uint32_t kPrBytes = kPrOdd + 3 * kPrV * 4 + 1024;
static_assert(3 * kPrV == kPrThreads, "a thread an entry");
constexpr uint32_t kPrTmS = 0, kPrTmO = 2 * kPrTok;
static_assert(kPrBytes <= 227 * 1024, "shared memory");

struct PrParams {
    __nv_bfloat16* out;            // [n_q][H][128]
    float* lse;                    // or null
    const int32_t* q_start;
    const int32_t* kv_start;
    int32_t n_q, n_kv, n_seqs, H, max_q, blocks;   // blocks: of a CTA's queries, of a sequence
    int32_t causal, wide;          // wide: out is 32-byte aligned
    float scale;
    int32_t* err;
    uint64_t half_wait;
    int32_t withhold;
};

struct PrLaunch {
    PrParams p;
    CUtensorMap map_q, map_k, map_v, map_r;
};

struct PrBars {
    uint64_t full[11], empty[11];
    uint64_t q_full, s_full[2], p_full[2][2], pv_done[2], drained;   // p_full: tokens 0-63, 64-127 of the tile
    uint32_t units, queries;   // fills whose loads were issued: of the ring, of the queries (0 or 1)
    uint32_t tmem;
    int32_t abort, odd;      // odd: some masked value is not finite
};
static_assert(sizeof(PrBars) <= 512, "barrier block");

// What a CTA does, worked out alike by every role.
template <bool SPLIT>
struct PrWork {
    int h, q0, k0;           // head, the block's first query and the sequence's first row (of all)
    int rows;                // queries of the block
    int nk, shift;           // rows of the sequence; query i of the block sees rows j <= i + shift (causal)
    int tiles_a, tiles_b;
    __device__ __forceinline__ int tiles(int a) const { return a ? tiles_b : tiles_a; }
    __device__ __forceinline__ int most() const { return max(tiles_a, tiles_b); }
    __device__ __forceinline__ int all() const { return SPLIT ? tiles_a + tiles_b : most(); }
    // side a's i-th tile; its first query (of the CTA's)
    __device__ __forceinline__ static int tile(int a, int i) { return SPLIT ? 2 * i + a : i; }
    __device__ __forceinline__ static int query0(int a) { return SPLIT ? 0 : a * kPrRows; }
    __device__ __forceinline__ int side_rows(int a) const { return min(kPrRows, rows - a * kPrRows); }
};

template <bool SPLIT>
__device__ __forceinline__ int pr_tiles(const PrParams& p, const PrWork<SPLIT>& w, int a)
{
    const int r = w.side_rows(a);
    if (r <= 0)
        return 0;
    const int see = p.causal ? min(w.nk, a * kPrRows + r + w.shift) : w.nk;   // rows that the side's last query sees
    return see > 0 ? (see - 1) / kPrTok + 1 : 0;
}

// False: nothing to do (no queries, or a malformed sequence).
template <bool SPLIT>
__device__ __forceinline__ bool pr_work(const PrParams& p, PrWork<SPLIT>& w)
{
    constexpr int kQueries = PrLayout<SPLIT>::kQueries;
    int id = blockIdx.x;
    w.h = id % p.H;
    id /= p.H;
    const int s = id % p.n_seqs, blk = p.blocks - 1 - id / p.n_seqs;   // later queries see more: first
    const int a = p.q_start[s], b = p.q_start[s + 1], c = p.kv_start[s], d = p.kv_start[s + 1];
    int32_t bits = 0;
    if (a < 0 || b < a || b > p.n_q || c < 0 || d < c || d > p.n_kv)
        bits = KAMERA_DEVERR_DESCRIPTOR;
    else if (b - a > p.max_q)
        bits = KAMERA_DEVERR_LEN;
    if (bits) {
        if (blk == 0 && w.h == 0 && threadIdx.x == 0)
            raise_err(p.err, bits);
        return false;
    }
    const int nq = b - a, first = kQueries * blk;
    w.rows = min(kQueries, nq - first);
    if (w.rows <= 0)
        return false;
    w.q0 = a + first;
    w.k0 = c;
    w.nk = d - c;
    w.shift = w.nk - nq + first;
    const int n = pr_tiles(p, w, 0);
    w.tiles_a = SPLIT ? (n + 1) / 2 : n;
    w.tiles_b = SPLIT ? n / 2 : pr_tiles(p, w, 1);
    return true;
}

template <bool SPLIT>
__device__ void pr_producer(const PrLaunch& L, const PrWork<SPLIT>& w, PrBars& b, uint32_t sbase)
{
    const PrParams& p = L.p;
    const uint32_t q_full = ptx::smem_addr(&b.q_full);
    constexpr int kPrUnits = PrLayout<SPLIT>::kUnits;
    constexpr uint32_t kPrRing = PrLayout<SPLIT>::kQUnits * kPrUnit;
    const int sides = w.rows > kPrRows ? 2 : 1, n = w.all();
    if (p.withhold)
        return;
    ptx::mbar_arrive_expect_tx(q_full, (uint32_t)sides * 3 * kPrUnit);
    for (int i = 0; i < 3 * sides; ++i)
        ptx::tma_load_3d(sbase + i * kPrUnit, &L.map_q, 64 * (i % 3), w.h, w.q0 + kPrRows * (i / 3), q_full);
    uint32_t k = 0;
    bool ok = true;
    for (int t = 0; t < n && ok; ++t)
        for (int u = 0; u < kPrTile; ++u, ++k) {
            const uint32_t at = k % kPrUnits, lap = k / kPrUnits, full = ptx::smem_addr(&b.full[at]);
            if (lap > 0 && !wmma16::cycle_wait(ptx::smem_addr(&b.empty[at]), (lap & 1u) ^ 1u, &b.abort, p.err, p.half_wait)) {
                ok = false;
                break;
            }
            ptx::mbar_arrive_expect_tx(full, kPrUnit);
            const uint32_t dst = sbase + kPrRing + at * kPrUnit;
            const int row = w.k0 + t * kPrTok;
            const int col = w.h * (kPrNope + kPrV);
            if (u < 2) {
                ptx::tma_load_2d(dst, &L.map_k, col + 64 * u, row, full);
            } else if (u == 2) {
                ptx::tma_load_2d(dst, &L.map_r, 0, row, full);
            } else {
                ptx::tma_load_2d(dst, &L.map_v, col + kPrNope, row + 64 * (u - 3), full);
                ptx::tma_load_2d(dst + kPrUnit / 2, &L.map_v, col + kPrNope + 64, row + 64 * (u - 3), full);
            }
        }
    b.queries = 1;
    b.units = k;
}

// After a timeout, once every role has left its loop: the copies that the CTA started land
// before it leaves.  (Without one the MMA lane has waited for every fill.  Out of line, and
// called with a softmax warp's registers: in line it costs a short prompt's call 0.2 us.)
template <bool SPLIT>
__device__ __noinline__ void pr_drain(const PrBars& b)
{
    pf_drain_ring(&b.q_full, b.queries, 1);
    pf_drain_ring(b.full, b.units, PrLayout<SPLIT>::kUnits);
}

// The MMA lane.  What it does next waits behind the dispatch of its MMAs, looks at
// barriers too, which leaves the tensor pipe idle for about 500 of 3350 cycles a pair of
// tiles (2680 of MMAs).  Tried for 4 x 4096 tokens, at 195 us: a lane a side 230 (both sides
// then weigh at the same time), with turns 214; one barrier for a tile's keys, its values
// and its weights 200 (the first half of the weights starts the product early).  TMEM
// addresses are offsets: the CTA holds all 512 columns, so its allocation starts at
// address 0.
template <bool SPLIT>
__device__ void pr_mma(const PrLaunch& L, const PrWork<SPLIT>& w, PrBars& b, uint32_t sbase)
{
    const PrParams& p = L.p;
    constexpr uint32_t idS = ptx::idesc_bf16_f32(kPrRows, kPrTok);
    constexpr uint32_t idV = ptx::idesc_bf16_f32(kPrRows, kPrV) | (1u << 16);   // value rows: MN-major
    constexpr int kPrUnits = PrLayout<SPLIT>::kUnits;
    const uint32_t q_lo = (sbase >> 4) | (1u << 16), r_lo = (sbase + PrLayout<SPLIT>::kQUnits * kPrUnit) >> 4;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return wmma16::cycle_wait(ptx::smem_addr(bar), parity & 1u, &b.abort, p.err, p.half_wait);
    };
    // scores of side a's t-th tile; its keys are free after the last side that sees it
    auto scores = [&](auto side, int t) -> bool {
        constexpr int a = decltype(side)::value;
        constexpr uint32_t dS = kPrTmS + a * kPrTok;
        const bool free = SPLIT || a == 1 || t >= w.tiles_b;
#pragma unroll
        for (int u = 0; u < 3; ++u) {
            const uint32_t k = (uint32_t)(kPrTile * w.tile(a, t) + u), at = k % kPrUnits;
            if (!wait(&b.full[at], k / kPrUnits))
                return false;
            ptx::tc_fence_after();
            const uint32_t aq = q_lo + ((SPLIT ? 0 : 3 * a) + u) * (kPrUnit >> 4), bk = (r_lo + at * (kPrUnit >> 4)) | (1u << 16);
            if (u == 0)
                mma_ss<false>(dS, aq, bk, idS);
            else
                mma_ss<true>(dS, aq, bk, idS);
#pragma unroll
            for (int ks = 1; ks < 4; ++ks)
                mma_ss<true>(dS, aq + 2 * ks, bk + 2 * ks, idS);
            if (free)
                ptx::umma_commit(ptx::smem_addr(&b.empty[at]));
        }
        ptx::umma_commit(ptx::smem_addr(&b.s_full[a]));
        return true;
    };
    auto weigh = [&](auto side, int t) -> bool {
        constexpr int a = decltype(side)::value;
        constexpr uint32_t dO = kPrTmO + a * kPrV, aP = kPrTmS + a * kPrTok;
        const uint32_t k = (uint32_t)(kPrTile * w.tile(a, t) + 3), at0 = k % kPrUnits, at1 = (k + 1) % kPrUnits;
        if (!wait(&b.full[at0], k / kPrUnits) || !wait(&b.full[at1], (k + 1) / kPrUnits))
            return false;
#pragma unroll
        for (int half = 0; half < 2; ++half) {   // the first 64 tokens while the others' weights are computed
            if (!wait(&b.p_full[a][half], t))
                return false;
            ptx::tc_fence_after();
            // 64 columns are 8 KB from the next 64, 16 tokens 2 KB from the next 16
            const uint32_t v = (r_lo + (half ? at1 : at0) * (kPrUnit >> 4)) | ((kPrUnit / 2 >> 4) << 16);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (half == 0 && i == 0 && t == 0)
                    mma_ts<false>(dO, aP, v, idV);
                else
                    mma_ts<true>(dO, aP + 8 * (4 * half + i), v + 128 * i, idV);
        }
        ptx::umma_commit(ptx::smem_addr(&b.pv_done[a]));
        if (SPLIT || a == 1 || t >= w.tiles_b) {
            ptx::umma_commit(ptx::smem_addr(&b.empty[at0]));
            ptx::umma_commit(ptx::smem_addr(&b.empty[at1]));
        }
        return true;
    };
    constexpr auto A = std::integral_constant<int, 0>{};
    constexpr auto B = std::integral_constant<int, 1>{};
    bool ok = wait(&b.q_full, 0) && (w.tiles_a == 0 || scores(A, 0)) && (w.tiles_b == 0 || scores(B, 0));
    for (int t = 0; t < w.most() && ok; ++t) {
        if (t < w.tiles_a)
            ok = weigh(A, t) && (t + 1 >= w.tiles_a || scores(A, t + 1));
        if (ok && t < w.tiles_b)
            ok = weigh(B, t) && (t + 1 >= w.tiles_b || scores(B, t + 1));
    }
    // every MMA issued here completes before TMEM is freed
    ptx::umma_commit(ptx::smem_addr(&b.drained));
    pf_drain_wait(ptx::smem_addr(&b.drained), 0u);
}

__device__ __forceinline__ float pr_max3(float a, uint32_t b, uint32_t c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return d;
}

// 16 bf16 pairs of a row: two 32-byte stores where the row allows them.
__device__ __forceinline__ void pr_store(__nv_bfloat16* dst, const uint32_t (&w)[16], bool wide)
{
    if (wide) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 16 * i), "r"(w[8 * i]),
                         "r"(w[8 * i + 1]), "r"(w[8 * i + 2]), "r"(w[8 * i + 3]), "r"(w[8 * i + 4]), "r"(w[8 * i + 5]),
                         "r"(w[8 * i + 6]), "r"(w[8 * i + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(dst + 8 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
}

// A barrier of both sides: whether all of their threads said yes.
__device__ __forceinline__ bool pr_all(bool ok)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, 256, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(ok ? 1u : 0u)
                 : "memory");
    return r != 0;
}

// A masked weight is zero, and zero times a value that is not finite is not zero.  So a
// value row that some query of a side does not see is looked through, a value that is not
// finite becomes 0, and its row is noted for its column; what queries that do see it get
// is added at the end (out of line, both: the code that never runs costs a short prompt's
// call 2 us in line).
__device__ __noinline__ void pr_clean(uint32_t at, int in_unit, int row, int32_t* first, int32_t* odd)
{
#pragma unroll 1
    for (int c = 0; c < kPrV; ++c) {
        const uint32_t a = at + (c >> 6) * (kPrUnit / 2) + sw128(in_unit & 7, (c & 63) >> 3) + (c & 7) * 2;
        uint16_t x;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(a) : "memory");
        if ((x & 0x7F80) != 0x7F80)
            continue;
        atomicMin(first + ((x & 0x7F) ? 0 : (x >> 15) ? 2 : 1) * kPrV + c, row);
        *static_cast<volatile int32_t*>(odd) = 1;
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"((uint16_t)0) : "memory");
    }
}

// Thread r: row r of the tile; `unit` holds it, `in_unit` is its place there.
__device__ __forceinline__ void pr_clean_row(uint32_t unit, int in_unit, int row, int32_t* first, int32_t* odd)
{
    const uint32_t at = unit + (uint32_t)(in_unit >> 3) * 1024u;
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        uint32_t x[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                     : "r"(at + (i >> 3) * (kPrUnit / 2) + sw128(in_unit & 7, i & 7))
                     : "memory");
#pragma unroll
        for (int j = 0; j < 4; ++j)
            most = __vmaxu2(most, x[j] & 0x7FFF7FFFu);
    }
    if (max(most & 0xFFFFu, most >> 16) >= 0x7F80u)
        pr_clean(at, in_unit, row, first, odd);
}

// A query that sees the rows below `limit`: what is noted for columns c0 .. c1 - 1, added
// to its output.
__device__ __noinline__ void pr_add_odd(const int32_t* first, __nv_bfloat16* out, int c0, int c1, int limit)
{
    for (int c = c0; c < c1; ++c) {
        const volatile int32_t* f = first + c;
        float x = f[0] < limit ? __uint_as_float(0x7FC00000u) : 0.f;
        x += f[kPrV] < limit ? INFINITY : 0.f;
        x -= f[2 * kPrV] < limit ? INFINITY : 0.f;
        if (x != 0.f)
            out[c] = __float2bfloat16(__bfloat162float(out[c]) + x);
    }
}

// Side a's softmax, thread r = query r of the side = TMEM lane r.
template <bool SPLIT>
__device__ void pr_softmax(const PrLaunch& L, const PrWork<SPLIT>& w, PrBars& b, uint32_t sbase, uint32_t tm, int a, int r,
                           int32_t* first)
{
    const PrParams& p = L.p;
    constexpr int kPrUnits = PrLayout<SPLIT>::kUnits;
    constexpr uint32_t kPrRing = PrLayout<SPLIT>::kQUnits * kPrUnit;
    const int nt = w.tiles(a), query = w.query0(a) + r;
    const bool valid = query < w.rows;
    const uint32_t lanes = tm + ((uint32_t)(r & ~31) << 16);
    const uint32_t tS = lanes + kPrTmS + a * kPrTok, tO = lanes + kPrTmO + a * kPrV;
    // scores in log2 units; a scale of zero becomes the smallest float, 2^-149, so that a
    // masked score stays infinite under it (the largest finite one becomes 2^-21)
    const float sl2 = p.scale == 0.f ? 1.40129846e-45f : p.scale * 1.4426950408889634f;
    const int limit = p.causal ? min(w.nk, query + w.shift + 1) : w.nk;   // rows that the query sees
    const int least = p.causal ? min(w.nk, w.query0(a) + w.shift + 1) : w.nk;   // ... that the side's first one sees
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int t = 0; t < nt; ++t) {
        const int base = w.tile(a, t) * kPrTok;
        if (base + kPrTok > least) {   // value rows that not every query of the side sees; while the scores come
            const uint32_t k = (uint32_t)(kPrTile * w.tile(a, t) + 3);
            auto unit = [&](int row) { return sbase + kPrRing + (k + (row >> 6)) % kPrUnits * kPrUnit; };
            bool in = true;
            for (int u = 0; u < 2; ++u)
                in = in && wmma16::cycle_wait(ptx::smem_addr(&b.full[(k + u) % kPrUnits]), ((k + u) / kPrUnits) & 1u, &b.abort,
                                             p.err, p.half_wait);
            ok = __all_sync(0xFFFFFFFFu, ok && in);
            if (base + r >= least && base + r < w.nk)
                pr_clean_row(unit(r), r & 63, base + r, first, &b.odd);
            // past the sequence: zero, so that zero weights add nothing
            for (int i = r; i < (base + kPrTok - w.nk) * 16; i += kPrRows) {
                const int row = w.nk - base + (i >> 4), in_unit = row & 63;
                ptx::st_shared_zero16(unit(row) + ((i >> 3) & 1) * (kPrUnit / 2) + (uint32_t)(in_unit >> 3) * 1024u +
                                      sw128(in_unit & 7, i & 7));
            }
            ptx::fence_proxy_async();   // (the product waits for every thread's weights, which follow)
        }
        if (!wmma16::cycle_wait(ptx::smem_addr(&b.s_full[a]), (uint32_t)t & 1u, &b.abort, p.err, p.half_wait))
            ok = false;
        if (!__all_sync(0xFFFFFFFFu, ok)) {
            ok = false;
            break;
        }
        ptx::tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            tmem_ld32_issue(tS + 32 * c, s[c]);
        tmem_ld_wait128(s);
        if (base + kPrTok > least) {
            const int mine = limit - base;   // columns of the tile that this query sees
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (32 * c + j >= mine)
                        s[c][j] = sl2 < 0.f ? 0x7F800000u : 0xFF800000u;
        }
        // the row's largest score: three inputs an instruction, eight chains
        float e[8];
        if (sl2 >= 0.f) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                e[k] = fmaxf(__uint_as_float(s[k >> 1][16 * (k & 1)]), __uint_as_float(s[k >> 1][16 * (k & 1) + 1]));
#pragma unroll
            for (int j = 2; j < 16; j += 2)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    e[k] = pr_max3(e[k], s[k >> 1][16 * (k & 1) + j], s[k >> 1][16 * (k & 1) + j + 1]);
        } else {   // (a negative scale: the largest of the negated ones)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                e[k] = -INFINITY;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    e[k] = fmaxf(e[k], -__uint_as_float(s[k >> 1][16 * (k & 1) + j]));
            }
        }
#pragma unroll
        for (int d = 4; d >= 1; d /= 2)
#pragma unroll
            for (int k = 0; k < d; ++k)
                e[k] = fmaxf(e[k], e[k + d]);
        const float m_new = fmaxf(m_run, fabsf(sl2) * e[0]);
        if (t == 0) {
            m_run = m_new;   // O is still empty
        } else if (__any_sync(0xFFFFFFFFu, m_new > m_run + kPrLazy)) {
            const float f = m_new == -INFINITY ? 1.f : pf_ex2(m_run - m_new);
            l_run *= f;
            m_run = m_new;
            if (!wmma16::cycle_wait(ptx::smem_addr(&b.pv_done[a]), (uint32_t)(t - 1) & 1u, &b.abort, p.err, p.half_wait))
                ok = false;
            ok = __all_sync(0xFFFFFFFFu, ok);
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kPrV / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tO + 32 * c, o);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                tmem_st32(tO + 32 * c, o);
            }
        }
        // weights 2^(sl2 s - m), bf16, over the scores' columns
        const float ref = m_run == -INFINITY ? 0.f : m_run;
        const uint64_t sl2x2 = ptx::f2_make(__float_as_uint(sl2), __float_as_uint(sl2));
        const uint64_t nmx2 = ptx::f2_make(__float_as_uint(-ref), __float_as_uint(-ref));
        uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int c = 2 * half; c < 2 * half + 2; ++c) {
                uint32_t ph[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    uint32_t a0, a1;
                    asm("mov.b64 {%0, %1}, %2;"
                        : "=r"(a0), "=r"(a1)
                        : "l"(ptx::f2_fma(ptx::f2_make(s[c][2 * j], s[c][2 * j + 1]), sl2x2, nmx2)));
                    const float p0 = pf_ex2(__uint_as_float(a0)), p1 = pf_ex2(__uint_as_float(a1));
                    const uint64_t pp = ptx::f2_make(__float_as_uint(p0), __float_as_uint(p1));
                    sum2[j & 1] = ptx::f2_add(sum2[j & 1], pp);
                    ph[j] = ptx::f2_to_bf16x2(pp);
                }
                tmem_st16(tS + 16 * c, ph);
            }
            if (half == 1) {
                uint32_t x0, x1;
                asm("mov.b64 {%0, %1}, %2;" : "=r"(x0), "=r"(x1) : "l"(ptx::f2_add(sum2[0], sum2[1])));
                l_run += __uint_as_float(x0) + __uint_as_float(x1);
            }
            tmem_wait_st();
            ptx::tc_fence_before();
            ptx::mbar_arrive(ptx::smem_addr(&b.p_full[a][half]));
        }
    }
    if (nt > 0 && ok) {
        if (!wmma16::cycle_wait(ptx::smem_addr(&b.pv_done[a]), (uint32_t)(nt - 1) & 1u, &b.abort, p.err, p.half_wait))
            ok = false;
        ok = __all_sync(0xFFFFFFFFu, ok);
        ptx::tc_fence_after();
    }
    if constexpr (SPLIT) {
        // The sides have seen every second tile each: they exchange their state and half
        // of their output's columns through the ring, which nobody reads any more, and
        // either finishes the other half, 2^(m_a - m) O_a + 2^(m_b - m) O_b.
        if (!pr_all(ok))
            return;              // both sides
        auto theirs = [&](int side, int c) { return sbase + kPrRing + (uint32_t)((side * 66 + c) * kPrRows + r) * 4; };
        auto put = [&](uint32_t at, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory"); };
        auto get = [&](uint32_t at) {
            float v;
            asm volatile("ld.shared.b32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
            return v;
        };
        put(theirs(a ^ 1, 64), __float_as_uint(m_run));
        put(theirs(a ^ 1, 65), __float_as_uint(l_run));
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
            uint32_t o[32];
            if (nt > 0)
                tmem_ld32(tO + 64 * (a ^ 1) + 32 * c, o);
#pragma unroll
            for (int j = 0; j < 32; ++j)
                put(theirs(a ^ 1, 32 * c + j), nt > 0 ? o[j] : 0u);
        }
        pr_all(true);
        const float m_other = get(theirs(a, 64)), l_other = get(theirs(a, 65)), m = fmaxf(m_run, m_other);
        const float f = m_run == -INFINITY ? 0.f : pf_ex2(m_run - m), f_other = m_other == -INFINITY ? 0.f : pf_ex2(m_other - m);
        const float l = l_run * f + l_other * f_other;
        const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
        const int64_t row = (int64_t)(w.q0 + query) * p.H + w.h;
        if (valid && p.lse && a == 0)
            p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : (l == l ? -INFINITY : l);
        const float g = f * inv, g_other = f_other * inv;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
            uint32_t o[32], x[16];
            if (nt > 0)
                tmem_ld32(tO + 64 * a + 32 * c, o);
            float y[32];
#pragma unroll
            for (int j = 0; j < 32; ++j)
                y[j] = fmaf(get(theirs(a, 32 * c + j)), g_other, nt > 0 ? __uint_as_float(o[j]) * g : 0.f);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                x[j] = pack_bf16x2(y[2 * j], y[2 * j + 1]);
            if (valid)
                pr_store(p.out + row * kPrV + 64 * a + 32 * c, x, p.wide != 0);
        }
        if (valid && *static_cast<volatile int32_t*>(&b.odd))
            pr_add_odd(first, p.out + row * kPrV, 64 * a, 64 * a + 64, limit);
        return;
    }
    if (!ok)
        return;
    const float inv = l_run > 0.f ? 1.f / l_run : (l_run == l_run ? 0.f : l_run);
    const int64_t row = (int64_t)(w.q0 + query) * p.H + w.h;
    if (valid && p.lse)
        p.lse[row] = l_run > 0.f ? (m_run + log2f(l_run)) * 0.6931471805599453f : (l_run == l_run ? -INFINITY : l_run);
#pragma unroll 1
    for (int c = 0; c < kPrV / 32; ++c) {
        uint32_t o[32], x[16];
        if (nt > 0)
            tmem_ld32(tO + 32 * c, o);
#pragma unroll
        for (int j = 0; j < 16; ++j)   // no row seen by any of the side's queries: O was never written
            x[j] = nt > 0 ? pack_bf16x2(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv) : 0u;
        if (valid)
            pr_store(p.out + row * kPrV + 32 * c, x, p.wide != 0);
    }
    if (valid && *static_cast<volatile int32_t*>(&b.odd))
        pr_add_odd(first, p.out + row * kPrV, 0, kPrV, limit);
}

template <bool SPLIT>
__global__ void __launch_bounds__(kPrThreads, 1) mla_prefill_kernel(const __grid_constant__ PrLaunch L)
{
    const PrParams& p = L.p;
    extern __shared__ __align__(16) unsigned char raw[];
    const uint32_t at = ptx::smem_addr(raw), pad = (1024u - (at & 1023u)) & 1023u, sbase = at + pad;
    PrBars& b = *reinterpret_cast<PrBars*>(raw + pad + kPrBar);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < PrLayout<SPLIT>::kUnits; ++i) {
            ptx::mbar_init(ptx::smem_addr(&b.full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.empty[i]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(ptx::smem_addr(&b.s_full[a]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.p_full[a][0]), kPrRows);
            ptx::mbar_init(ptx::smem_addr(&b.p_full[a][1]), kPrRows);
            ptx::mbar_init(ptx::smem_addr(&b.pv_done[a]), 1);
        }
        ptx::mbar_init(ptx::smem_addr(&b.q_full), 1);
        ptx::mbar_init(ptx::smem_addr(&b.drained), 1);
        b.abort = 0;
        b.odd = 0;
        b.units = b.queries = 0;
        ptx::fence_barrier_init();
    }
    int32_t* first = reinterpret_cast<int32_t*>(raw + pad + kPrOdd);
    first[threadIdx.x] = 0x7FFFFFFF;
    ptx::grid_wait();
    PrWork<SPLIT> w;
    if (!pr_work(p, w))   // (the CTA)
        return;
    if (warp == kPrMma) {
        ptx::tmem_alloc(ptx::smem_addr(&b.tmem), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    ptx::grid_launch_next();   // (this CTA has its TMEM: none that starts early can take it)
    const uint32_t tm = b.tmem;
    // Registers: the softmax warps hold a row of 128 scores, the others next to nothing
    // (256 x 208 + 128 x 56 of the launch's 384 x 168).
    if (warp < 8) {
        ptx::setmaxnreg_inc<208>();
        pr_softmax(L, w, b, sbase, tm, warp >> 2, threadIdx.x & (kPrRows - 1), first);
    } else {
        ptx::setmaxnreg_dec<56>();
        if (w.most() > 0) {
            if (warp == kPrProd && elect_one())
                pr_producer(L, w, b, sbase);
            else if (warp == kPrMma && elect_one())
                pr_mma(L, w, b, sbase);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kPrMma) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tm, 512);
    }
    if (threadIdx.x == 0 && b.abort)
        pr_drain<SPLIT>(b);
}

}  // namespace

}  // namespace kamera

using namespace kamera;

extern "C" {

int kamera_mla_prefill_attend(const KameraMlaPrefill* x, int32_t* d_err, struct CUstream_st* stream)
{
    if (!x || x->n_q < 0 || x->n_kv < 0 || x->n_seqs < 0 || x->num_heads < 1 || x->nope_dim < 0 || x->rope_dim < 0 ||
        x->v_dim < 0 || x->max_q < 0 || !(x->scale == x->scale))
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (x->nope_dim != kPrNope || x->rope_dim != kPrQk - kPrNope || x->v_dim != kPrV || x->num_heads > 128 ||
        x->n_kv > (1 << 30) || x->n_q > (1 << 30))
        return KAMERA_ERR_UNSUPPORTED;
    // (a bound of no queries still has a block a sequence, which reports those that have some)
    auto blocks_of = [&](int rows) { return std::max<int64_t>(1, ((int64_t)x->max_q + rows - 1) / rows); };
    const int64_t pairs = (int64_t)x->n_seqs * x->num_heads;
    // One block of queries a CTA, its tiles split between the sides, while that makes no
    // more than two CTAs an SM: then blocks of 256 would leave SMs idle or half of a CTA's
    // sides (16 heads; 777 queries behind 1296 rows, 112 such CTAs: 21 us against 35; 2000
    // behind 4000, 256: 78 against 87; 2432, 304: 29 against 37).  With more, rows are
    // better read once for 256 queries (4 x 1200, 640: 39 against 30).
    const bool split = blocks_of(kPrRows) * pairs <= 2 * (int64_t)device_sms();
    const int64_t blocks = blocks_of(split ? kPrRows : 2 * kPrRows), ctas = blocks * pairs;
    if (ctas > 0x7FFFFFFF)
        return KAMERA_ERR_UNSUPPORTED;
    if (x->n_seqs == 0 || x->n_q == 0 || (x->max_q == 0 && !d_err))   // nothing to write, or to report
        return KAMERA_OK;
    if (!x->q || !x->out || !x->q_start || !x->kv_start || (x->n_kv > 0 && (!x->kv || !x->k_rope)))
        return KAMERA_ERR_INVALID_ARGUMENT;
    const int H = x->num_heads, kvw = H * (kPrNope + kPrV);
    // strides of dimensions with one element are not looked at
    const int64_t qh = H > 1 ? x->q_head_stride : kPrQk, qt = x->n_q > 1 ? x->q_stride : qh * H;
    const int64_t kt = x->n_kv > 1 ? x->kv_stride : kvw, rt = x->n_kv > 1 ? x->k_rope_stride : kPrQk - kPrNope;
    if (qh < kPrQk || qt < kPrQk || kt < kvw || rt < kPrQk - kPrNope)
        return KAMERA_ERR_INVALID_ARGUMENT;
    const void* ptrs[] = {x->q, x->kv, x->k_rope, x->out};
    for (const void* a : ptrs)
        if (!aligned16(a))
            return KAMERA_ERR_MISALIGNED;
    if ((qh & 7) || (qt & 7) || (kt & 7) || (rt & 7) ||
        ((reinterpret_cast<uintptr_t>(x->lse) | reinterpret_cast<uintptr_t>(x->q_start) |
          reinterpret_cast<uintptr_t>(x->kv_start)) & 3))
        return KAMERA_ERR_MISALIGNED;
    using Span = std::pair<uintptr_t, uintptr_t>;
    auto bytes = [](const void* a, int64_t n) -> Span {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(a);
        return {lo, a ? lo + (uintptr_t)n : lo};
    };
    const Span in[] = {bytes(x->q, ((x->n_q - 1) * qt + (H - 1) * qh + kPrQk) * 2),
                       span(x->kv, 1, 0, x->n_kv, kt, kvw), span(x->k_rope, 1, 0, x->n_kv, rt, kPrQk - kPrNope),
                       bytes(x->q_start, ((int64_t)x->n_seqs + 1) * 4), bytes(x->kv_start, ((int64_t)x->n_seqs + 1) * 4)};
    const Span os = bytes(x->out, (int64_t)x->n_q * H * kPrV * 2), ls = bytes(x->lse, (int64_t)x->n_q * H * 4);
    for (const Span& a : in)
        if (overlap(a, os) || overlap(a, ls))
            return KAMERA_ERR_INVALID_ARGUMENT;
    if (overlap(os, ls))
        return KAMERA_ERR_INVALID_ARGUMENT;
    PrLaunch L;
    std::memset(&L, 0, sizeof(L));
    PrParams& p = L.p;
    p.out = static_cast<__nv_bfloat16*>(x->out);
    p.lse = x->lse;
    p.q_start = x->q_start;
    p.kv_start = x->kv_start;
    p.n_q = x->n_q;
    p.n_kv = x->n_kv;
    p.n_seqs = x->n_seqs;
    p.H = H;
    p.max_q = x->max_q;
    p.blocks = (int32_t)blocks;
    p.causal = x->causal ? 1 : 0;
    p.wide = (reinterpret_cast<uintptr_t>(x->out) & 31) == 0;
    p.scale = x->scale;
    p.err = d_err;
    p.half_wait = half_wait(wait_limit_ns());
    p.withhold = test_withhold_loads() ? 1 : 0;
    // (without a row no tile is read: the maps take the queries' memory)
    const void* kv = x->n_kv > 0 ? x->kv : x->q;
    const void* kr = x->n_kv > 0 ? x->k_rope : x->q;
    const int64_t rows = std::max(x->n_kv, 1);
    if (!make_heads_map(&L.map_q, x->q, x->n_q, H, kPrQk, qt, qh, 64, kPrRows) ||
        !make_rows_map(&L.map_k, kv, rows, kvw, kt, 64, kPrTok) || !make_rows_map(&L.map_v, kv, rows, kvw, kt, 64, 64) ||
        !make_rows_map(&L.map_r, kr, rows, kPrQk - kPrNope, rt, 64, kPrTok))
        return KAMERA_ERR_CUDA;
    auto launch = [&](auto kernel) {
        // set at every launch: the attribute belongs to the current device's context
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPrBytes) == cudaSuccess &&
               launch_after(kernel, dim3((unsigned)ctas), kPrThreads, kPrBytes, reinterpret_cast<cudaStream_t>(stream), true,
                            L) == cudaSuccess;
    };
    if (!(split ? launch(mla_prefill_kernel<true>) : launch(mla_prefill_kernel<false>)))
        return KAMERA_ERR_CUDA;
    return KAMERA_OK;
}

}  // extern "C"
