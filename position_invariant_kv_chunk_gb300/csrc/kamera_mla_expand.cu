// kamera_mla_expand.cu -- latent rows of the pool expanded into every head's keys and
// values: kv[t][h] = W_h c_t, the rope part gathered beside it.
//
// A matrix product, [tokens x 512] [512 x heads 256], whose left rows lie at pool slots.
// 2 x 512 flops a value written (2 bytes): bound by the tensor cores from some hundred
// tokens on.  Two CTAs form a pair (cta_group::2) of 256 tokens: each holds the latent
// parts of its 128 in shared memory (128 KB, gathered once), and the pair runs heads past
// them, one MMA (M 256, N 256) taking each CTA's tokens and half of the head's weights
// from either CTA's shared memory.  So an SM loads half of the weights -- they come in
// eight chunks of 64 columns, 16 KB to a CTA, through a ring of four -- and reads 8 KB of
// shared memory an MMA.  (A CTA alone: 70 us for 16381 tokens of 16 heads, its ring of
// 96 KB too short for L2's latency; with the weights by multicast to both, 65.)  A head's
// 128 x 256 sums stand in one of two TMEM halves while two epilogue groups empty the other,
// each 64 columns at a time through shared memory and a TMA store (one group took 6200
// cycles a head, rows stored from the registers 6000, its MMAs 4200).  16381 tokens of 16
// heads take 58 us on data in turn (1180 TFLOP/s, floor 35): a head now takes 6100 cycles,
// in which an SM reads 128 KB of weights from L2 and writes 64 KB.
//   warps 0-3, 4-7  epilogue of a head's first and last 128 columns: thread = token = TMEM lane
//   warp 8     producer of the CTA's half of the weights (TMA, counted on the first CTA's
//              barriers)
//   warp 9     MMA (the first CTA's for both); it owns TMEM
//   warps 10-13  gather of the tokens' rows: 16-byte async copies, a warp a row, and
//              k_rope's copy
// Work: (2 x 128 tokens, head) items, tokens outermost, cut into equal ranges, one a
// cluster.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <cuda.h>

#include "kamera_common.cuh"
#include "kamera_hostcheck.h"
#include "kamera_internal.h"
#include "kamera_ptx.cuh"
#include "kamera_tc.cuh"
#include "kamera_warpmma.cuh"

namespace kamera {

namespace {

using namespace tc;

constexpr int kExTok = 128, kExK = 512, kExRope = 64, kExN = 256;
constexpr int kExChunks = kExK / 64;
constexpr int kExStages = 4;
constexpr int kExThreads = 448, kExProd = 8, kExMma = 9, kExGather = 10;
constexpr uint32_t kExBlock = kExTok * 128;           // 64 columns of the tokens: 16 KB
constexpr uint32_t kExStage = kExN / 2 * 128;         // 64 columns of half of a head's weights: 16 KB
constexpr uint32_t kExRing = kExK / 64 * kExBlock;
constexpr uint32_t kExOut = kExRing + kExStages * kExStage;   // two groups' 64 columns of the output: 16 KB each
constexpr uint32_t kExBar = kExOut + 2 * kExTok * 128;
constexpr uint32_t kExBytes = kExBar + 256 + 1024;
static_assert(kExBytes <= 227 * 1024, "shared memory");

struct ExParams {
    const __nv_bfloat16* pool;
    const int64_t* slots;
    __nv_bfloat16* rope;
    int64_t num_slots, slot_stride, items;
    int32_t T, H;
    int32_t* err;
    uint64_t half_wait;
    int32_t withhold;
};

struct ExLaunch {
    ExParams p;
    CUtensorMap map_w, map_o;
};

struct ExBars {
    uint64_t full[kExStages], empty[kExStages], acc_full[2], acc_empty[2], a_full, a_empty[kExChunks], drained;
    uint32_t issued;       // fills whose loads this CTA issued
    uint32_t gave_up[2];   // either CTA of the pair: 0, or 1 + its fills where a wait ran out
    uint32_t tmem;
    int32_t abort;
};
static_assert(sizeof(ExBars) <= 256, "barrier block");

// A cluster's items [lo, hi), walked alike by every role of both CTAs: tile of tokens
// (each its own of the pair), head.
struct ExWalk {
    int64_t i, hi;
    int tile, head, H;
    __device__ __forceinline__ ExWalk(const ExParams& p) : H(p.H)
    {
        const int64_t c = blockIdx.x >> 1, n = gridDim.x >> 1;
        i = c * p.items / n;
        hi = (c + 1) * p.items / n;
        const int pair = (int)(i / H);
        tile = 2 * pair + (int)(blockIdx.x & 1);
        head = (int)(i - (int64_t)pair * H);
    }
    __device__ __forceinline__ bool more() const { return i < hi; }
    __device__ __forceinline__ bool last_of_tile() const { return head + 1 == H || i + 1 == hi; }
    __device__ __forceinline__ void next()
    {
        ++i;
        if (++head == H) {
            head = 0;
            tile += 2;
        }
    }
};

__device__ __forceinline__ void ex_cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A shared-memory address of this CTA as a CTA of the pair has it.
__device__ __forceinline__ uint32_t ex_at(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t ex_first(uint32_t addr) { return ex_at(addr, 0); }
__device__ __forceinline__ void ex_arrive_first(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(ex_first(bar)) : "memory");
}

// A box into this CTA's shared memory, counted on a barrier of the pair's first CTA.
__device__ __forceinline__ void ex_load(uint32_t dst, const void* tmap, int x, int y, uint32_t first_bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                 "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(tmap), "r"(x), "r"(y), "r"(first_bar)
                 : "memory");
}

// D (+)= A B^T over the pair: M 256 (each CTA its 128 rows and accumulator), N 256 (half
// of B's rows in each CTA).
template <bool ACC>
__device__ __forceinline__ void ex_mma2(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc)
{
    if constexpr (ACC)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, 1, 1;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                     "l"(pf_desc(a_lo)), "l"(pf_desc(b_lo)), "r"(idesc)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, 1, 1;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                     "l"(pf_desc(a_lo)), "l"(pf_desc(b_lo)), "r"(idesc)
                     : "memory");
}

// Arrives on both CTAs' barrier once every MMA this thread issued so far has completed.
__device__ __forceinline__ void ex_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}

// This CTA's half of fill k, of a head's weights.
__device__ __forceinline__ void ex_fill(const ExLaunch& L, ExBars& b, uint32_t sbase, uint32_t k, int head)
{
    const int half = blockIdx.x & 1, c = (int)(k % kExChunks);
    const uint32_t at = k % kExStages, full = ptx::smem_addr(&b.full[at]);
    if (half == 0)
        ptx::mbar_arrive_expect_tx(full, 2 * kExStage);
    ex_load(sbase + kExRing + at * kExStage, &L.map_w, 64 * c, head * kExN + half * (kExN / 2), ex_first(full));
}

__device__ void ex_producer(const ExLaunch& L, ExBars& b, uint32_t sbase)
{
    const ExParams& p = L.p;
    if (p.withhold)
        return;
    uint32_t k = 0;
    bool ok = true;
    for (ExWalk w(p); w.more() && ok; w.next())
        for (int c = 0; c < kExChunks; ++c, ++k) {
            const uint32_t at = k % kExStages, lap = k / kExStages;
            if (lap > 0 && !wmma16::cycle_wait(ptx::smem_addr(&b.empty[at]), (lap & 1u) ^ 1u, &b.abort, p.err, p.half_wait)) {
                ok = false;
                break;
            }
            ex_fill(L, b, sbase, k, w.head);
        }
    b.issued = k;
}

// After a timeout, once every role of both CTAs has left its loop and either knows the
// other's fills: the copies that the pair started land before its CTAs leave.  (Without one
// the MMA lane has waited for every fill.)  A fill counts both halves, so the CTA that is
// behind issues its own of those that the other issued -- no more than the ring holds: the
// other had waited for the use of what stood there before -- and the first CTA, whose
// barriers count them, waits.
__device__ __forceinline__ void ex_drain(const ExLaunch& L, ExBars& b, uint32_t sbase)
{
    const ExWalk w(L.p);
    const uint32_t all = (uint32_t)(w.hi - w.i) * kExChunks;
    auto fills = [&](int r) {
        const uint32_t x = *static_cast<volatile uint32_t*>(&b.gave_up[r]);
        return x ? x - 1 : all;   // one whose waits were all met has issued every fill
    };
    const int half = blockIdx.x & 1;
    const uint32_t most = max(fills(0), fills(1));
    for (uint32_t k = fills(half); k < most; ++k)
        ex_fill(L, b, sbase, k, (int)((w.head + k / kExChunks) % w.H));
    if (half == 0)
        pf_drain_ring(b.full, most, kExStages);
}

__device__ void ex_mma(const ExLaunch& L, ExBars& b, uint32_t sbase, uint32_t tm)
{
    const ExParams& p = L.p;
    constexpr uint32_t id = ptx::idesc_bf16_f32(2 * kExTok, kExN);
    const uint32_t a_lo = (sbase >> 4) | (1u << 16), r_lo = ((sbase + kExRing) >> 4) | (1u << 16);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return wmma16::cycle_wait(ptx::smem_addr(bar), parity & 1u, &b.abort, p.err, p.half_wait);
    };
    uint32_t k = 0, n = 0, tiles = 0;
    bool ok = true, fresh = true;
    for (ExWalk w(p); w.more() && ok; ++n) {
        const bool last = w.last_of_tile();
        if (fresh && !(ok = wait(&b.a_full, tiles)))
            break;
        if (n >= 2 && !(ok = wait(&b.acc_empty[n & 1u], (n >> 1) - 1)))
            break;
        const uint32_t d = tm + (n & 1u) * kExN;
#pragma unroll 1
        for (int c = 0; c < kExChunks; ++c, ++k) {
            const uint32_t at = k % kExStages;
            if (!(ok = wait(&b.full[at], k / kExStages)))
                break;
            ptx::tc_fence_after();
            const uint32_t x = a_lo + c * (kExBlock >> 4), w_lo = r_lo + at * (kExStage >> 4);
            if (c == 0)
                ex_mma2<false>(d, x, w_lo, id);
            else
                ex_mma2<true>(d, x, w_lo, id);
#pragma unroll
            for (int ks = 1; ks < 4; ++ks)
                ex_mma2<true>(d, x + 2 * ks, w_lo + 2 * ks, id);
            ex_commit(ptx::smem_addr(&b.empty[at]));
            if (last)
                ex_commit(ptx::smem_addr(&b.a_empty[c]));
        }
        if (!ok)
            break;
        ex_commit(ptx::smem_addr(&b.acc_full[n & 1u]));
        fresh = last;
        tiles += last ? 1u : 0u;
        w.next();
    }
    // every MMA issued here completes before TMEM is freed
    ex_commit(ptx::smem_addr(&b.drained));
    pf_drain_wait(ptx::smem_addr(&b.drained), 0u);
}

// The tokens' rows into shared memory (K-major, 128B-swizzled blocks of 64 columns),
// zero where there is none, a block as soon as the tile before has no MMA left that reads
// it; k_rope's rows by the CTA that has the tile's first head.  The rows of the pair's
// next tile are asked into L2 meanwhile.
__device__ void ex_gather(const ExLaunch& L, ExBars& b, uint32_t sbase, int warp, int lane)
{
    const ExParams& p = L.p;
    uint32_t tiles = 0;
    bool fresh = true, ok = true;
    auto piece = [&](int r, int c, int64_t slot) {   // 16-byte piece c of row r's latent part
        const uint32_t dst = sbase + (uint32_t)(c >> 3) * kExBlock + (uint32_t)(r >> 3) * 1024u + sw128(r & 7, c & 7);
        if (slot >= 0)
            ptx::cp_async16(dst, p.pool + slot * p.slot_stride + 8 * c);
        else
            ptx::st_shared_zero16(dst);
    };
    auto slot_of = [&](int t) -> int64_t { return t < p.T ? p.slots[t] : -1; };
    int64_t mine = -1;
    for (ExWalk w(p); w.more(); w.next()) {
        if (fresh) {
            const int t0 = w.tile * kExTok + 32 * warp;
            if (tiles == 0)
                mine = slot_of(t0 + lane);   // lane l: row l of the warp's 32
            if (mine < 0 || mine >= p.num_slots) {
                if (mine != -1 && w.head == 0)
                    raise_err(p.err, KAMERA_DEVERR_SLOT);
                mine = -1;
            }
            int64_t slot[8];   // the rows of this lane's pieces of a block: 4 i + lane / 8
#pragma unroll
            for (int i = 0; i < 8; ++i)
                slot[i] = __shfl_sync(0xFFFFFFFFu, mine, 4 * i + (lane >> 3));
            if (tiles == 0) {   // nothing to wait for: row after row (block after block, 1296 tokens 18.4 us, not 16.7)
#pragma unroll 8
                for (int i = 0; i < 32; ++i) {
                    const int64_t s = __shfl_sync(0xFFFFFFFFu, mine, i);
                    piece(32 * warp + i, lane, s);
                    piece(32 * warp + i, 32 + lane, s);
                }
            } else {
#pragma unroll
                for (int c = 0; c < kExChunks; ++c) {
                    ok = wmma16::cycle_wait(ptx::smem_addr(&b.a_empty[c]), (tiles - 1) & 1u, &b.abort, p.err, p.half_wait);
                    if (!__all_sync(0xFFFFFFFFu, ok)) {
                        ptx::cp_async_commit();
                        ptx::cp_async_wait<0>();
                        return;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        piece(32 * warp + 4 * i + (lane >> 3), 8 * c + (lane & 7), slot[i]);
                }
            }
            ptx::cp_async_commit();
            uint4 v[8];   // k_rope
            const bool rope = w.head == 0;
            if (rope) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (slot[i] >= 0)
                        v[i] = *reinterpret_cast<const uint4*>(p.pool + slot[i] * p.slot_stride + kExK + 8 * (lane & 7));
                }
            }
            ptx::cp_async_wait<0>();
            ptx::fence_proxy_async();
            if (!p.withhold)
                ex_arrive_first(ptx::smem_addr(&b.a_full));
            if (rope) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int t = t0 + 4 * i + (lane >> 3);
                    if (t < p.T)
                        *reinterpret_cast<uint4*>(p.rope + (int64_t)t * kExRope + 8 * (lane & 7)) = v[i];
                }
            }
            ++tiles;
            if (w.hi - w.i > w.H - w.head) {   // the pair has a tile after this one
                mine = slot_of(t0 + 2 * kExTok + lane);
                if (mine >= 0 && mine < p.num_slots) {
                    const char* row = reinterpret_cast<const char*>(p.pool + mine * p.slot_stride);
#pragma unroll
                    for (int i = 0; i < (kExK + kExRope) * 2 / 128; ++i)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(row + 128 * i));
                }
            }
        }
        fresh = w.last_of_tile();
    }
}

template <int GRP>
__device__ void ex_epilogue(const ExLaunch& L, ExBars& b, uint32_t sbase, uint32_t tm, int warp, int lane)
{
    const ExParams& p = L.p;
    const uint32_t lanes = tm + ((uint32_t)warp << 21);
    const int r = 32 * warp + lane;
    const uint32_t out = sbase + kExOut + GRP * kExTok * 128, row = out + (uint32_t)(r >> 3) * 1024u;
    uint32_t n = 0, ok_word;
    bool ok = true;
    for (ExWalk w(p); w.more() && ok; w.next(), ++n) {
        ok = wmma16::cycle_wait(ptx::smem_addr(&b.acc_full[n & 1u]), (n >> 1) & 1u, &b.abort, p.err, p.half_wait);
        ptx::tc_fence_after();
        const bool some = w.tile * kExTok < p.T;
#pragma unroll 1
        for (int c = GRP * (kExN / 128); c < (GRP + 1) * (kExN / 128); ++c) {
            uint32_t o[32], q[32];
            tmem_ld32_issue(lanes + (n & 1u) * kExN + 64 * c, o);
            tmem_ld32(lanes + (n & 1u) * kExN + 64 * c + 32, q);   // waits for both
#pragma unroll
            for (int j = 0; j < 32; ++j)
                asm volatile("" : "+r"(o[j]));
            if (r == 0)
                ptx::bulk_wait_read_all();   // the store before has read the buffer
            asm volatile("bar.sync %0, 128;" ::"n"(1 + 2 * GRP) : "memory");
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t* x = j < 4 ? o + 8 * j : q + 8 * (j - 4);
                ptx::sts128(row + sw128(r & 7, j), pack_bf16x2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                            pack_bf16x2(__uint_as_float(x[2]), __uint_as_float(x[3])),
                            pack_bf16x2(__uint_as_float(x[4]), __uint_as_float(x[5])),
                            pack_bf16x2(__uint_as_float(x[6]), __uint_as_float(x[7])));
            }
            ptx::fence_proxy_async();
            asm volatile("bar.sync %0, 128;" ::"n"(1 + 2 * GRP) : "memory");
            if (r == 0 && some && ok) {      // rows past the last token are not written
                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(&L.map_o),
                             "r"(w.head * kExN + 64 * c), "r"(w.tile * kExTok), "r"(out)
                             : "memory");
                ptx::bulk_commit();
            }
        }
        ptx::tc_fence_before();
        ex_arrive_first(ptx::smem_addr(&b.acc_empty[n & 1u]));
        // a thread whose wait ran out leaves with the others
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, %2, 128, p;\n\t"
                     "selp.u32 %0, 1, 0, q;\n\t}"
                     : "=r"(ok_word)
                     : "r"(ok ? 1u : 0u), "n"(2 + 2 * GRP)
                     : "memory");
        ok = ok_word != 0;
    }
    if (r == 0)
        ptx::bulk_wait_all();
}

__global__ void __launch_bounds__(kExThreads, 1) mla_expand_kernel(const __grid_constant__ ExLaunch L)
{
    extern __shared__ __align__(16) unsigned char raw[];
    const uint32_t at = ptx::smem_addr(raw), pad = (1024u - (at & 1023u)) & 1023u, sbase = at + pad;
    ExBars& b = *reinterpret_cast<ExBars*>(raw + pad + kExBar);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kExStages; ++i) {
            ptx::mbar_init(ptx::smem_addr(&b.full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_addr(&b.acc_full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.acc_empty[i]), 512);   // both CTAs' epilogues
        }
        ptx::mbar_init(ptx::smem_addr(&b.a_full), 256);
        for (int i = 0; i < kExChunks; ++i)
            ptx::mbar_init(ptx::smem_addr(&b.a_empty[i]), 1);
        ptx::mbar_init(ptx::smem_addr(&b.drained), 1);
        b.abort = 0;
        b.issued = b.gave_up[0] = b.gave_up[1] = 0;
        ptx::fence_barrier_init();
    }
    if (warp == kExProd && lane == 0)
        ptx::prefetch_tmap(&L.map_w);
    if (warp == kExMma) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_addr(&b.tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    ptx::tc_fence_before();
    ex_cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tm = b.tmem;
    ptx::grid_wait();
    ptx::grid_launch_next();
    if (warp < 4)
        ex_epilogue<0>(L, b, sbase, tm, warp, lane);
    else if (warp < kExProd)
        ex_epilogue<1>(L, b, sbase, tm, warp - 4, lane);
    else if (warp == kExProd) {
        if (elect_one())
            ex_producer(L, b, sbase);
    } else if (warp == kExMma) {
        if ((blockIdx.x & 1) == 0 && elect_one())
            ex_mma(L, b, sbase, tm);
    } else
        ex_gather(L, b, sbase, warp - kExGather, lane);
    ptx::tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 32 * kExMma && (blockIdx.x & 1))   // the first CTA's MMA lane has waited for its own
        pf_drain_wait(ptx::smem_addr(&b.drained), 0u);
    if (threadIdx.x == 0 && b.abort)
        for (uint32_t r = 0; r < 2; ++r)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(ex_at(ptx::smem_addr(&b.gave_up[blockIdx.x & 1]), r)),
                         "r"(b.issued + 1)
                         : "memory");
    __syncwarp();
    ex_cluster_sync();   // neither CTA leaves while the other may write to it
    const volatile uint32_t* gave_up = b.gave_up;
    const bool late = (gave_up[0] | gave_up[1]) != 0 && !L.p.withhold;
    if (warp == kExMma) {
        ptx::tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512) : "memory");
    }
    if (late) {   // (both CTAs alike)
        if (threadIdx.x == 32 * kExProd)
            ex_drain(L, b, sbase);
        __syncwarp();
        ex_cluster_sync();
    }
}

}  // namespace

}  // namespace kamera

using namespace kamera;

extern "C" {

int kamera_mla_expand(const KameraPagedMlaKV* kv, const KameraMlaExpand* x, int32_t* d_err, struct CUstream_st* stream)
{
    if (!kv || !x || kv->reserved != 0 || x->reserved != 0 || kv->num_slots < 0 || kv->kv_lora_rank < 1 ||
        kv->rope_dim < 0 || x->n_tokens < 0 || x->num_heads < 1 || x->head_width < 1)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (kv->kv_lora_rank != kExK || kv->rope_dim != kExRope || x->head_width != kExN || x->num_heads > 128)
        return KAMERA_ERR_UNSUPPORTED;
    if (x->n_tokens == 0)
        return KAMERA_OK;
    if (!x->weight || !x->slots || !x->kv_out || !x->k_rope_out)
        return KAMERA_ERR_INVALID_ARGUMENT;
    constexpr int W = kExK + kExRope;
    int e;
    if ((e = check_strided(kv->kv, 1, 0, kv->num_slots, kv->slot_stride, W, false)))
        return e;
    if (!aligned16(x->weight) || !aligned16(x->kv_out) || !aligned16(x->k_rope_out) ||
        (reinterpret_cast<uintptr_t>(x->slots) & 7))
        return KAMERA_ERR_MISALIGNED;
    using Span = std::pair<uintptr_t, uintptr_t>;
    auto bytes = [](const void* a, int64_t n) -> Span {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(a);
        return {lo, lo + (uintptr_t)n};
    };
    const int64_t T = x->n_tokens, H = x->num_heads;
    const Span in[] = {span(kv->kv, 1, 0, kv->num_slots, kv->slot_stride, W), bytes(x->weight, H * kExN * kExK * 2),
                       bytes(x->slots, T * 8)};
    const Span a = bytes(x->kv_out, T * H * kExN * 2), c = bytes(x->k_rope_out, T * kExRope * 2);
    for (const Span& s : in)
        if (overlap(s, a) || overlap(s, c))
            return KAMERA_ERR_INVALID_ARGUMENT;
    if (overlap(a, c))
        return KAMERA_ERR_INVALID_ARGUMENT;
    ExLaunch L;
    std::memset(&L, 0, sizeof(L));
    ExParams& p = L.p;
    p.pool = static_cast<const __nv_bfloat16*>(kv->kv);
    p.slots = x->slots;
    p.rope = static_cast<__nv_bfloat16*>(x->k_rope_out);
    p.num_slots = kv->num_slots;
    p.slot_stride = kv->slot_stride;
    p.T = x->n_tokens;
    p.H = x->num_heads;
    p.items = (T + 2 * kExTok - 1) / (2 * kExTok) * H;
    p.err = d_err;
    p.half_wait = half_wait(wait_limit_ns());
    p.withhold = test_withhold_loads() ? 1 : 0;
    if (!make_rows_map(&L.map_w, x->weight, H * kExN, kExK, kExK, 64, kExN / 2) ||
        !make_rows_map(&L.map_o, x->kv_out, T, H * kExN, H * kExN, 64, kExTok))
        return KAMERA_ERR_CUDA;
    // set at every launch: the attribute belongs to the current device's context
    if (cudaFuncSetAttribute(mla_expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kExBytes) != cudaSuccess)
        return KAMERA_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    const int fit = cluster_fit(reinterpret_cast<const void*>(mla_expand_kernel), kExThreads, (int)kExBytes, 2);
    cfg.gridDim = dim3(2u * (unsigned)std::min<int64_t>(fit > 0 ? fit : std::max(1, device_sms() / 2), p.items));
    cfg.blockDim = dim3(kExThreads);
    cfg.dynamicSmemBytes = kExBytes;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, mla_expand_kernel, L) != cudaSuccess)
        return KAMERA_ERR_CUDA;
    return KAMERA_OK;
}

}  // extern "C"
