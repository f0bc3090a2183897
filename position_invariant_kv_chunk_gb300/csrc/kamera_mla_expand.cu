// kamera_mla_expand.cu -- latent rows of the pool expanded into every head's keys and
// values: kv[t][h] = W_h c_t, the rope part gathered beside it.
//
// A matrix product, [tokens x 512] [512 x heads 256], whose left rows lie at pool slots.
// 2 x 512 flops a value written (2 bytes): bound by the tensor cores from some hundred
// tokens on.  A CTA holds the latent parts of 128 tokens in shared memory (128 KB,
// gathered once) and runs heads past them: a head's weights come in sixteen 16 KB chunks
// of 32 columns through a ring of five, and its 128 x 256 sums stand in one of two TMEM
// halves while the epilogue empties the other, 64 columns at a time through shared memory
// and a TMA store (rows stored from the registers, 32 bytes a lane, took 6000 cycles a
// head, half more than its MMAs).
//   warps 0-3  epilogue: thread = token = TMEM lane
//   warp 4     producer of the weights (TMA)
//   warp 5     MMA (M 128, N 256); it owns TMEM
//   warps 6-9  gather of the tokens' rows: 16-byte async copies, a warp a row, and
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
constexpr int kExChunks = kExK / 32;
constexpr int kExStages = 5;
constexpr int kExThreads = 320, kExProd = 4, kExMma = 5, kExGather = 6;
constexpr uint32_t kExBlock = kExTok * 128;           // 64 columns of the tokens: 16 KB
constexpr uint32_t kExStage = kExN * 64;              // 32 columns of a head's weights: 16 KB
constexpr uint32_t kExRing = kExK / 64 * kExBlock;
constexpr uint32_t kExOut = kExRing + kExStages * kExStage;   // 64 columns of the output: 16 KB
constexpr uint32_t kExBar = kExOut + kExTok * 128;
constexpr uint32_t kExHi64 = (512u >> 4) | (1u << 14) | (4u << 29);   // descriptors of the weights: 64-byte swizzle
constexpr uint32_t kExBytes = kExBar + 256 + 1024;
static_assert(kExBytes <= 227 * 1024, "shared memory");

struct ExParams {
    const __nv_bfloat16* pool;
    const int64_t* slots;
    __nv_bfloat16* kv;
    __nv_bfloat16* rope;
    int64_t num_slots, slot_stride, items;
    int32_t T, H;
    int32_t* err;
    uint64_t wait_ns;
    int32_t withhold;
};

struct ExLaunch {
    ExParams p;
    CUtensorMap map_w, map_o;
};

struct ExBars {
    uint64_t full[kExStages], empty[kExStages], acc_full[2], acc_empty[2], a_full, a_empty, drained;
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

// A box into the same place of both CTAs' shared memory, counted on both CTAs' barriers.
__device__ __forceinline__ void ex_load_both(uint32_t dst, const void* tmap, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.multicast::cluster "
                 "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
                 "l"(tmap), "r"(x), "r"(y), "r"(bar), "h"((uint16_t)3)
                 : "memory");
}

// Arrives on both CTAs' barrier once every MMA this thread issued so far has completed.
__device__ __forceinline__ void ex_commit_both(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}

__device__ __forceinline__ bool ex_elect()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
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
            const uint32_t at = k % kExStages, lap = k / kExStages, full = ptx::smem_addr(&b.full[at]);
            if (lap > 0 && !wmma16::cycle_wait(ptx::smem_addr(&b.empty[at]), (lap & 1u) ^ 1u, &b.abort, p.err, p.wait_ns)) {
                ok = false;
                break;
            }
            // this CTA's half of the chunk's rows for both, the other's half from the other
            ptx::mbar_arrive_expect_tx(full, kExStage);
            const int half = blockIdx.x & 1;
            ex_load_both(sbase + kExRing + at * kExStage + half * (kExStage / 2), &L.map_w, 32 * c,
                         w.head * kExN + half * (kExN / 2), full);
        }
    // Without a timeout the MMA lane has waited for every fill.  After one, the copies
    // started here land before the CTA leaves.
    if (*static_cast<volatile int32_t*>(&b.abort))
        for (uint32_t i = k > (uint32_t)kExStages ? k - kExStages : 0u; i < k; ++i)
            pf_drain_wait(ptx::smem_addr(&b.full[i % kExStages]), (i / kExStages) & 1u, p.wait_ns);
}

__device__ void ex_mma(const ExLaunch& L, ExBars& b, uint32_t sbase, uint32_t tm)
{
    const ExParams& p = L.p;
    constexpr uint32_t id = ptx::idesc_bf16_f32(kExTok, kExN);
    const uint32_t a_lo = (sbase >> 4) | (1u << 16), r_lo = ((sbase + kExRing) >> 4) | (1u << 16);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return wmma16::cycle_wait(ptx::smem_addr(bar), parity & 1u, &b.abort, p.err, p.wait_ns);
    };
    uint32_t k = 0, n = 0, tiles = 0;
    bool ok = true, fresh = true;
    for (ExWalk w(p); w.more() && ok; ++n) {
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
            const uint32_t a = a_lo + (c >> 1) * (kExBlock >> 4) + 4 * (c & 1), w_lo = r_lo + at * (kExStage >> 4);
            if (c == 0)
                mma_ss2<false, kDescHi, kExHi64>(d, a, w_lo, id);
            else
                mma_ss2<true, kDescHi, kExHi64>(d, a, w_lo, id);
            mma_ss2<true, kDescHi, kExHi64>(d, a + 2, w_lo + 2, id);
            ex_commit_both(ptx::smem_addr(&b.empty[at]));
        }
        if (!ok)
            break;
        ptx::umma_commit(ptx::smem_addr(&b.acc_full[n & 1u]));
        fresh = w.last_of_tile();
        if (fresh) {
            ptx::umma_commit(ptx::smem_addr(&b.a_empty));
            ++tiles;
        }
        w.next();
    }
    // every MMA issued here completes before TMEM is freed
    ptx::umma_commit(ptx::smem_addr(&b.drained));
    pf_drain_wait(ptx::smem_addr(&b.drained), 0u, p.wait_ns);
}

// The tokens' rows into shared memory (K-major, 128B-swizzled blocks of 64 columns),
// zero where there is none; k_rope's rows by the CTA that has the tile's first head.
__device__ void ex_gather(const ExLaunch& L, ExBars& b, uint32_t sbase, int warp, int lane)
{
    const ExParams& p = L.p;
    uint32_t tiles = 0;
    bool fresh = true, ok = true;
    for (ExWalk w(p); w.more(); w.next()) {
        if (fresh) {
            if (tiles > 0)
                ok = wmma16::cycle_wait(ptx::smem_addr(&b.a_empty), (tiles - 1) & 1u, &b.abort, p.err, p.wait_ns);
            if (!__all_sync(0xFFFFFFFFu, ok))
                return;
            const int t0 = w.tile * kExTok + 32 * warp;
            int64_t mine = t0 + lane < p.T ? p.slots[t0 + lane] : -1;   // lane l: row l of the warp's 32
            if (mine < 0 || mine >= p.num_slots) {
                if (mine != -1 && w.head == 0)
                    raise_err(p.err, KAMERA_DEVERR_SLOT);
                mine = -1;
            }
#pragma unroll 8
            for (int i = 0; i < 32; ++i) {
                const int64_t slot = __shfl_sync(0xFFFFFFFFu, mine, i);
                const int r = 32 * warp + i;
                const __nv_bfloat16* src = p.pool + slot * p.slot_stride;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int c = 32 * x + lane;   // 16-byte piece of the latent part
                    const uint32_t dst = sbase + (uint32_t)(c >> 3) * kExBlock + (uint32_t)(r >> 3) * 1024u + sw128(r & 7, c & 7);
                    if (slot >= 0)
                        ptx::cp_async16(dst, src + 8 * c);
                    else
                        ptx::st_shared_zero16(dst);
                }
            }
            ptx::cp_async_commit();
            uint4 v[8];   // k_rope: four rows of eight pieces at a time
            const bool rope = w.head == 0;
            if (rope) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t slot = __shfl_sync(0xFFFFFFFFu, mine, 4 * i + (lane >> 3));
                    v[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (slot >= 0)
                        v[i] = *reinterpret_cast<const uint4*>(p.pool + slot * p.slot_stride + kExK + 8 * (lane & 7));
                }
            }
            ptx::cp_async_wait<0>();
            ptx::fence_proxy_async();
            if (!p.withhold)
                ptx::mbar_arrive(ptx::smem_addr(&b.a_full));
            if (rope) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int t = t0 + 4 * i + (lane >> 3);
                    if (t < p.T)
                        *reinterpret_cast<uint4*>(p.rope + (int64_t)t * kExRope + 8 * (lane & 7)) = v[i];
                }
            }
            ++tiles;
        }
        fresh = w.last_of_tile();
    }
}

__device__ void ex_epilogue(const ExLaunch& L, ExBars& b, uint32_t sbase, uint32_t tm, int warp, int lane)
{
    const ExParams& p = L.p;
    const uint32_t lanes = tm + ((uint32_t)warp << 21);
    const int r = 32 * warp + lane;
    const uint32_t row = sbase + kExOut + (uint32_t)(r >> 3) * 1024u;
    uint32_t n = 0, ok_word;
    bool ok = true;
    for (ExWalk w(p); w.more() && ok; w.next(), ++n) {
        ok = wmma16::cycle_wait(ptx::smem_addr(&b.acc_full[n & 1u]), (n >> 1) & 1u, &b.abort, p.err, p.wait_ns);
        ptx::tc_fence_after();
        const bool some = w.tile * kExTok < p.T;
#pragma unroll 1
        for (int c = 0; c < kExN / 64; ++c) {
            uint32_t o[32], q[32];
            tmem_ld32_issue(lanes + (n & 1u) * kExN + 64 * c, o);
            tmem_ld32(lanes + (n & 1u) * kExN + 64 * c + 32, q);   // waits for both
#pragma unroll
            for (int j = 0; j < 32; ++j)
                asm volatile("" : "+r"(o[j]));
            if (r == 0)
                ptx::bulk_wait_read_all();   // the store before has read the buffer
            asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t* x = j < 4 ? o + 8 * j : q + 8 * (j - 4);
                ptx::sts128(row + sw128(r & 7, j), pack_bf16x2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                            pack_bf16x2(__uint_as_float(x[2]), __uint_as_float(x[3])),
                            pack_bf16x2(__uint_as_float(x[4]), __uint_as_float(x[5])),
                            pack_bf16x2(__uint_as_float(x[6]), __uint_as_float(x[7])));
            }
            ptx::fence_proxy_async();
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (r == 0 && some && ok) {      // rows past the last token are not written
                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(&L.map_o),
                             "r"(w.head * kExN + 64 * c), "r"(w.tile * kExTok), "r"(sbase + kExOut)
                             : "memory");
                ptx::bulk_commit();
            }
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_addr(&b.acc_empty[n & 1u]));
        // a thread whose wait ran out leaves with the others
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 2, 128, p;\n\t"
                     "selp.u32 %0, 1, 0, q;\n\t}"
                     : "=r"(ok_word)
                     : "r"(ok ? 1u : 0u)
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
            ptx::mbar_init(ptx::smem_addr(&b.empty[i]), 2);   // both CTAs' MMAs
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_addr(&b.acc_full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&b.acc_empty[i]), 128);
        }
        ptx::mbar_init(ptx::smem_addr(&b.a_full), 128);
        ptx::mbar_init(ptx::smem_addr(&b.a_empty), 1);
        ptx::mbar_init(ptx::smem_addr(&b.drained), 1);
        b.abort = 0;
        ptx::fence_barrier_init();
    }
    if (warp == kExProd && lane == 0)
        ptx::prefetch_tmap(&L.map_w);
    if (warp == kExMma) {
        ptx::tmem_alloc(ptx::smem_addr(&b.tmem), 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    ex_cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tm = b.tmem;
    ptx::grid_wait();
    ptx::grid_launch_next();
    if (warp < 4)
        ex_epilogue(L, b, sbase, tm, warp, lane);
    else if (warp == kExProd) {
        if (ex_elect())
            ex_producer(L, b, sbase);
    } else if (warp == kExMma) {
        if (ex_elect())
            ex_mma(L, b, sbase, tm);
    } else
        ex_gather(L, b, sbase, warp - kExGather, lane);
    ptx::tc_fence_before();
    __syncwarp();
    ex_cluster_sync();   // neither CTA leaves while the other may write to it
    if (warp == kExMma) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tm, 512);
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
    p.kv = static_cast<__nv_bfloat16*>(x->kv_out);
    p.rope = static_cast<__nv_bfloat16*>(x->k_rope_out);
    p.num_slots = kv->num_slots;
    p.slot_stride = kv->slot_stride;
    p.T = x->n_tokens;
    p.H = x->num_heads;
    p.items = (T + 2 * kExTok - 1) / (2 * kExTok) * H;
    p.err = d_err;
    p.wait_ns = wait_limit_ns();
    p.withhold = test_withhold_loads() ? 1 : 0;
    if (!make_rows_map64(&L.map_w, x->weight, H * kExN, kExK, kExK, kExN / 2) ||
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
