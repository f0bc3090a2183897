// kamera_paged.cu -- decode attention over the paged pool: the sequences' own
// (or selected) pages, the merge of partial softmax states, and the C entry
// points kamera_attend_shared and kamera_attend_selected.
//
// A decode step has at most 16 query rows per (sequence, KV head), so its own
// pages are read-bound: 4 d bytes a token against 4 d G flops.  The kernel
// keeps HBM busy and everything else out of its way:
//   - A page holds whole 16-token pieces (page sizes are multiples of 16), and a
//     piece is one 128B-swizzled TMA box per 64 columns.  Each warp owns a ring of
//     pieces of its own, loads them itself NS - 1 ahead and runs attention over
//     them alone; warps of a CTA meet only at the end.
//   - The tokens are the M of the warp-level MMA (m16n8k16) and the query heads
//     its N: S^T[16 x 8] = K Q^T, O^T[d x 8] += V^T P^T.  Eight heads fill an N
//     tile, where heads as M would leave half of 16 rows empty, and O^T takes
//     d / 8 registers a thread per eight heads.  P^T passes from the score
//     fragments to the B operand through 8 x 8 transposes in registers.
//   - Softmax weights are not bf16 values: they enter as hi + lo pairs (about 16
//     significant bits, both parts positive), which costs MMAs the tensor pipe has spare.
//   - Two buffers a warp and three CTAs an SM: with three buffers and two CTAs 32
//     sequences of 2048 selected tokens took 48.5 us with the selection, where this
//     took 40.1 (38 since the selection got shorter).  Their 134 MB take 20 us of HBM;
//     the kernel's 25 add the start (three dependent loads) and the join.
//   - Few rows: the tokens of a (sequence, KV head) are split over CTAs.  Without a
//     shared prefix up to eight of them form a cluster and join their states in
//     shared memory; else each leaves a partial state in the workspace, and the
//     merge joins them with the prefix's.
#include <algorithm>
#include <cooperative_groups.h>
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

using namespace wmma16;

constexpr int kPgWarps = 4;
constexpr int kPgThreads = 32 * kPgWarps;
constexpr int kPgTok = 16;             // tokens of a piece
constexpr int kMaxCluster = 8;         // splits that a cluster joins
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Shared memory: per warp NS buffers of a piece's key and value boxes (16 rows x
// 128 bytes each, NB of them), reused at the end for the warps' outputs.
template <int D, int NT>
struct PgLayout {
    static constexpr int NB = D / 64;
    static constexpr uint32_t kBox = kPgTok * 128;
    static constexpr uint32_t kPiece = 2 * NB * kBox;          // keys, then values
    static constexpr int NS = D == 128 ? 2 : 4;
    static constexpr uint32_t kWarp = NS * kPiece;
    static constexpr uint32_t kRing = kPgWarps * kWarp;
    static constexpr uint32_t kOut = kPgWarps * 8 * NT * (D + 4) * 4;   // warps' outputs (rows padded)
    static constexpr uint32_t kState = kRing > kOut ? kRing : kOut;
    static constexpr uint32_t kBytes = kState + 2 * (kPgWarps + 1) * 8 * NT * 4 + kPgWarps * NS * 8 + 64 + 1024;
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;   // relative error near 2^-22
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One CTA per (sequence, KV head, split).  NT: 8-head tiles of the KV head's
// query heads.  `final`: the only partial state, written as the output.
template <int D, int NT>
__global__ void __launch_bounds__(kPgThreads) paged_kernel(const __grid_constant__ PagedLaunch L)
{
    using Y = PgLayout<D, NT>;
    constexpr int NS = Y::NS, NB = Y::NB, MT = D / 16;
    const PagedParams& p = L.p;
    extern __shared__ __align__(16) unsigned char raw[];
    unsigned char* base = raw + ((1024u - (ptx::smem_addr(raw) & 1023u)) & 1023u);   // swizzled boxes
    float* outs = reinterpret_cast<float*>(base);                              // [warp][head][D + 4] at the end
    float* wm = reinterpret_cast<float*>(base + Y::kState);                    // [warp][8 NT]
    float* wl = wm + kPgWarps * 8 * NT;
    float* cm = wl + kPgWarps * 8 * NT;                                        // [8 NT]: the CTA's state
    float* cl = cm + 8 * NT;
    uint64_t* full = reinterpret_cast<uint64_t*>(cl + 8 * NT);                 // [warp][NS]
    volatile int32_t* abort = reinterpret_cast<volatile int32_t*>(full + kPgWarps * NS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, t4 = lane & 3;
    const int seq = blockIdx.y / p.H, h = blockIdx.y - seq * p.H, split = blockIdx.x;
    const int HQ = p.H * p.G, ppp = p.P / kPgTok;   // pieces per page
    if (threadIdx.x < kPgWarps * NS)
        ptx::mbar_init(ptx::smem_addr(full + threadIdx.x), 1);
    if (threadIdx.x == 0) {
        *abort = 0;
        ptx::prefetch_tmap(&L.map_k);
        ptx::prefetch_tmap(&L.map_v);
    }
    ptx::fence_barrier_init();
    if (p.n_groups == 0)   // the call's first kernel
        ptx::grid_wait();
    ptx::grid_launch_next();

    // the queries as the B operand: heads 8 nt + gq, channels 16 ks + 2 t4 (+ 8)
    uint32_t qb[NT][MT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int g = 8 * nt + gq;
        const uint32_t* qp =
            reinterpret_cast<const uint32_t*>(p.q + ((int64_t)seq * HQ + h * p.G + min(g, p.G - 1)) * D);
#pragma unroll
        for (int ks = 0; ks < MT; ++ks) {
            qb[nt][ks][0] = g < p.G ? qp[8 * ks + t4] : 0u;
            qb[nt][ks][1] = g < p.G ? qp[8 * ks + t4 + 4] : 0u;
        }
    }

    // The warp's pieces are i0 + warp, i0 + warp + 4, ...; lane l looks up the
    // (32 r + l)-th of them: its page (read ahead of the sequence's length, which
    // says later whether it counts), its first token's place in the sequence.
    const int32_t* table = p.pages + (int64_t)seq * p.max_pages;
    const int32_t* sel = p.selected ? p.selected + ((int64_t)seq * p.H + h) * p.n_select : nullptr;
    const int i0 = split * p.own_split;
    const int most = sel ? p.n_select * ppp : (p.max_len + kPgTok - 1) / kPgTok;   // pieces at most
    auto look_up = [&](int k, int& page, int& token) {
        const int i = i0 + warp + kPgWarps * k;
        page = -1;
        token = -1;
        if (k >= (p.own_split + kPgWarps - 1) / kPgWarps || i >= most)
            return;
        int slot = i / ppp;                      // place in the page table row
        const int off = (i - slot * ppp) * kPgTok;
        if (sel)
            slot = sel[slot];
        if (slot < 0)
            return;                              // not selected
        token = (int)min((int64_t)slot * p.P + off, (int64_t)0x7FFFFFFF);
        if (slot < p.max_pages)
            page = table[slot];
    };
    int page_c, token_c, page_n, token_n;        // this round's 32 pieces and the next round's
    look_up(lane, page_c, token_c);
    look_up(32 + lane, page_n, token_n);
    const int len = own_len(p, seq);
    if (threadIdx.x == 0 && split == 0 && h == 0 && p.max_len > 0 && (p.lens[seq] < 0 || p.lens[seq] > p.max_len))
        raise_err(p.err, KAMERA_DEVERR_LEN);
    const int n_pieces = p.selected ? p.n_select * ppp : (len + kPgTok - 1) / kPgTok;
    const int i1 = min(n_pieces, i0 + p.own_split);
    // The prefix kernel may still run beside this one, and the merge that follows
    // waits for this grid alone: its last CTA leaves when the prefix is done.
    auto leave = [&]() {
        if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1)
            ptx::grid_wait();
    };
    if (i0 >= i1 && p.o) {   // the merge knows that this slot is empty
        leave();
        return;
    }
    __syncthreads();

    float o[NT][MT][4];                 // O^T: channels 16 mt + gq (+ 8), heads 8 nt + 2 t4, + 1
    float m_run[NT][2], l_run[NT][2];   // heads 8 nt + 2 t4, + 1 (log2 units; the sum of this lane's tokens)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m_run[nt][0] = m_run[nt][1] = -INFINITY;
        l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
    }
    const float sl2 = p.scale * kLog2e;
    const uint32_t ring = ptx::smem_addr(base) + warp * Y::kWarp;
    const uint32_t bar = ptx::smem_addr(full + warp * NS);
    const int count = i1 > i0 + warp ? (i1 - i0 - warp + kPgWarps - 1) / kPgWarps : 0;
    // The pool row and the tokens (0: left out) of a piece that was looked up.
    auto settle = [&](int k, int page, int token, int& row, int& tok) {
        row = 0;
        tok = 0;
        if (k >= count || token < 0)
            return;
        if (sel && token >= ((int64_t)len + p.P - 1) / p.P * p.P) {   // past the sequence's last page
            raise_err(p.err, KAMERA_DEVERR_SLOT);
            return;
        }
        if (token >= len)
            return;
        if (page < 0 || page >= p.num_pages) {
            raise_err(p.err, KAMERA_DEVERR_SLOT);
            return;
        }
        row = page * p.P + token % p.P;          // < num_slots < 2^31
        tok = min(len - token, kPgTok);
    };
    int row_c, tok_c, row_n, tok_n;
    settle(lane, page_c, token_c, row_c, tok_c);
    settle(32 + lane, page_n, token_n, row_n, tok_n);
    look_up(64 + lane, page_n, token_n);         // two rounds ahead
    int base_k = 0;                              // piece of lane 0 of row_c
    auto piece = [&](int k, int& row, int& tok) {   // k in [base_k, base_k + 64)
        const int at = k - base_k;
        row = at < 32 ? __shfl_sync(0xFFFFFFFFu, row_c, at) : __shfl_sync(0xFFFFFFFFu, row_n, at - 32);
        tok = at < 32 ? __shfl_sync(0xFFFFFFFFu, tok_c, at) : __shfl_sync(0xFFFFFFFFu, tok_n, at - 32);
    };
    auto load = [&](int k) {   // piece k into buffer k % NS
        if (k >= count)
            return;
        int row, tok;
        piece(k, row, tok);
        if (tok > 0 && lane == 0 && !p.withhold) {
            const int b = k % NS;
            const uint32_t dst = ring + b * Y::kPiece;
            ptx::mbar_arrive_expect_tx(bar + 8 * b, Y::kPiece);
#pragma unroll
            for (int x = 0; x < NB; ++x) {
                ptx::tma_load_2d(dst + x * Y::kBox, &L.map_k, h * D + 64 * x, row, bar + 8 * b);
                ptx::tma_load_2d(dst + (NB + x) * Y::kBox, &L.map_v, h * D + 64 * x, row, bar + 8 * b);
            }
        }
    };
    uint32_t parity = 0;    // phase of each buffer's barrier
    uint32_t flying = 0;    // buffers with copies not yet waited for
    bool ok = true;
    auto mark = [&](int k) {
        if (k < count) {
            int row, tok;
            piece(k, row, tok);
            if (tok > 0 && !p.withhold)
                flying |= 1u << (k % NS);
        }
    };
#pragma unroll 1
    for (int k = 0; k < NS - 1; ++k) {
        load(k);
        mark(k);
    }
    // K as the A operand: matrices (tokens 0-7 | 8-15) x (channels 0-7 | 8-15);
    // V^T as the A operand (transposing loads): (channels 0-7 | 8-15) x (tokens 0-7 | 8-15)
    const uint32_t kr = (uint32_t)((lane & 7) + ((lane >> 3) & 1) * 8) * 128u, kc = (uint32_t)(lane >> 4);
    const uint32_t vr = (uint32_t)((lane & 7) + (lane >> 4) * 8) * 128u, vc = (uint32_t)((lane >> 3) & 1);
    const uint32_t sw = (uint32_t)(lane & 7);

#pragma unroll 1
    for (int k = 0; k < count && ok; ++k) {
        if (k - base_k >= 32) {
            base_k += 32;
            row_c = row_n;
            tok_c = tok_n;
            settle(base_k + 32 + lane, page_n, token_n, row_n, tok_n);
            look_up(base_k + 64 + lane, page_n, token_n);
        }
        load(k + NS - 1);
        mark(k + NS - 1);
        int row, tok;
        piece(k, row, tok);
        if (tok == 0)
            continue;
        const int b = k % NS;
        if (!tile_wait(bar + 8 * b, (parity >> b) & 1u, abort, p.err, p.wait_ns)) {
            ok = false;
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok)
            break;
        parity ^= 1u << b;
        flying &= ~(1u << b);
        const uint32_t kb = ring + b * Y::kPiece, vb = kb + NB * Y::kBox;
        if (tok < kPgTok) {   // value rows past the sequence: zero, so that zero weights add nothing
            for (int e = lane; e < (kPgTok - tok) * 8 * NB; e += 32) {
                const int r = tok + e / (8 * NB), c = e % (8 * NB);
                ptx::st_shared_zero16(vb + (c >> 3) * Y::kBox + r * 128 + (c & 7) * 16);
            }
            __syncwarp();
        }
        float sc[NT][2][4];   // S^T in two chains: tokens gq (+ 8), heads 2 t4, + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                sc[nt][c][0] = sc[nt][c][1] = sc[nt][c][2] = sc[nt][c][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < MT; ++ks) {
            uint32_t a[4];
            const uint32_t c = 2 * ks + kc;
            ldsm_x4(kb + (c >> 3) * Y::kBox + kr + (((c & 7) ^ sw) << 4), a);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma_bf16(sc[nt][ks & 1], a, qb[nt][ks][0], qb[nt][ks][1]);
        }
        uint32_t pb[NT][2][2];   // P^T as the B operand: [hi | lo][tokens 0-7 | 8-15]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x[4], mx[2], alpha[2];
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const float v = sc[nt][0][f] + sc[nt][1][f];
                x[f] = gq + 8 * (f >> 1) < tok ? v * sl2 : -INFINITY;
            }
            bool grew = false;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                mx[c] = fmaxf(x[c], x[c + 2]);
                mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xFFFFFFFFu, mx[c], 4));
                mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xFFFFFFFFu, mx[c], 8));
                mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xFFFFFFFFu, mx[c], 16));
                const float m_new = fmaxf(m_run[nt][c], mx[c]);
                const float ref = m_new == -INFINITY ? 0.f : m_new;   // scores of -infinity only: weights 0
                alpha[c] = ex2(m_run[nt][c] - ref);
                grew |= m_new != m_run[nt][c];
                m_run[nt][c] = m_new;
                x[c] = ex2(x[c] - ref);
                x[c + 2] = ex2(x[c + 2] - ref);
                l_run[nt][c] = fmaf(l_run[nt][c], alpha[c], x[c] + x[c + 2]);
            }
            if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    o[nt][mt][0] *= alpha[0];
                    o[nt][mt][1] *= alpha[1];
                    o[nt][mt][2] *= alpha[0];
                    o[nt][mt][3] *= alpha[1];
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t hi = weight_hi(x[2 * i], x[2 * i + 1]);
                const uint32_t lo =
                    pack_bf16x2(fmaf(bf16lo(hi), kLessHi, x[2 * i]), fmaf(bf16hi(hi), kLessHi, x[2 * i + 1]));
                pb[nt][0][i] = transpose8x8(hi);
                pb[nt][1][i] = transpose8x8(lo);
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            uint32_t a[4];
            const uint32_t c = 2 * mt + vc;
            ldsm_x4_t(vb + (c >> 3) * Y::kBox + vr + (((c & 7) ^ sw) << 4), a);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_bf16(o[nt][mt], a, pb[nt][0][0], pb[nt][0][1]);
                mma_bf16(o[nt][mt], a, pb[nt][1][0], pb[nt][1][1]);
            }
        }
        if (tok < kPgTok)
            ptx::fence_proxy_async();   // the zeroed rows precede a later TMA refill of the buffer
        __syncwarp();
    }
    if (!ok) {   // a wait ran out: the copies in flight land before the CTA leaves
        for (int b = 0; b < NS; ++b)
            if ((flying >> b) & 1u)
                tc::pf_drain_wait(bar + 8 * b, (parity >> b) & 1u);
    }
    // ---- the warps' states through shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {   // the sums of the eight token lanes
            l_run[nt][c] += __shfl_xor_sync(0xFFFFFFFFu, l_run[nt][c], 4);
            l_run[nt][c] += __shfl_xor_sync(0xFFFFFFFFu, l_run[nt][c], 8);
            l_run[nt][c] += __shfl_xor_sync(0xFFFFFFFFu, l_run[nt][c], 16);
        }
    __syncthreads();   // every warp is done with the ring
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int g = 8 * nt + 2 * t4 + c;
            float* dst = outs + (warp * 8 * NT + g) * (D + 4);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                dst[16 * mt + gq] = o[nt][mt][c];
                dst[16 * mt + gq + 8] = o[nt][mt][c + 2];
            }
            if (gq == 0) {
                wm[warp * 8 * NT + g] = m_run[nt][c];
                wl[warp * 8 * NT + g] = l_run[nt][c];
            }
        }
    __syncthreads();
    const int row0 = seq * HQ + h * p.G;
    for (int e = threadIdx.x; e < p.G * (D / 4); e += kPgThreads) {
        const int g = e / (D / 4), i = 4 * (e - g * (D / 4));
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kPgWarps; ++w)
            m = fmaxf(m, wm[w * 8 * NT + g]);
        float l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kPgWarps; ++w) {
            // no weight: nothing to add (and no maximum to scale by)
            const float f = wl[w * 8 * NT + g] == 0.f ? 0.f : ex2(wm[w * 8 * NT + g] - m);
            const float4 v = *reinterpret_cast<const float4*>(outs + (w * 8 * NT + g) * (D + 4) + i);
            l = fmaf(wl[w * 8 * NT + g], f, l);
            acc.x = fmaf(v.x, f, acc.x);
            acc.y = fmaf(v.y, f, acc.y);
            acc.z = fmaf(v.z, f, acc.z);
            acc.w = fmaf(v.w, f, acc.w);
        }
        if (p.o) {
            const int64_t at = (int64_t)(row0 + g) * p.slots + p.prefix_slots + split;
            *reinterpret_cast<float4*>(p.o + at * D + i) = acc;
            if (i == 0)
                p.ml[at] = make_float2(m, l);
        } else {   // over warp 0's output: this thread alone reads and writes it
            *reinterpret_cast<float4*>(outs + g * (D + 4) + i) = acc;
            if (i == 0) {
                cm[g] = m;
                cl[g] = l;
            }
        }
    }
    if (p.o) {
        leave();
        return;
    }
    // ---- no workspace: the splits of these rows are this cluster's CTAs; each
    // joins its share of the outputs through distributed shared memory
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const int n = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    for (int e = threadIdx.x + rank * kPgThreads; e < p.G * (D / 4); e += n * kPgThreads) {
        const int g = e / (D / 4), i = 4 * (e - g * (D / 4));
        float ms[kMaxCluster], ls[kMaxCluster], m = -INFINITY;   // of every CTA before the first is used
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
            ms[r] = r < n ? *cluster.map_shared_rank(cm + g, r) : -INFINITY;
            ls[r] = r < n ? *cluster.map_shared_rank(cl + g, r) : 0.f;
        }
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            m = fmaxf(m, ms[r]);
        float l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
            if (ls[r] == 0.f)
                continue;
            const float f = ex2(ms[r] - m);
            const float4 v = *reinterpret_cast<const float4*>(cluster.map_shared_rank(outs + g * (D + 4) + i, r));
            l = fmaf(ls[r], f, l);
            acc.x = fmaf(v.x, f, acc.x);
            acc.y = fmaf(v.y, f, acc.y);
            acc.z = fmaf(v.z, f, acc.z);
            acc.w = fmaf(v.w, f, acc.w);
        }
        const int64_t r = row0 + g;
        const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
        uint2 w;
        w.x = pack_bf16x2(acc.x * inv, acc.y * inv);
        w.y = pack_bf16x2(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(p.out + r * D + i) = w;
        if (i == 0 && p.lse)
            p.lse[r] = l > 0.f ? (m + log2f(l)) * kLn2 : (l == l ? -INFINITY : l);
    }
    cluster.sync();   // peers stay until their shares are read
}

// ----------------------------------------------------------------- merge --
// One CTA per row: out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over the
// row's partial states.  The row's sequence and lengths say which slots were
// written.  All latency (1.6 us; 3.5 us for 896 rows of 29 states): every warp works
// out the weights of 32 states at a time in its lanes and takes every fourth
// state's output; the four warps' sums join in warp order.  With the outputs asked
// for only when the weights were known the calls took 0.6 to 0.8 us more; with eight
// warps a row 1.8 us more for the 896 rows (fewer of them at a time).
constexpr int kMergeWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_kernel(const PagedParams p)
{
    constexpr int V = D / 32;   // floats of a lane
    __shared__ float part[kMergeWarps][D];
    __shared__ float sum;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;
    const int HQ = p.H * p.G;
    const int s = (int)(row / HQ);
    const float2* ml = p.ml + row * p.slots;
    const float* o = p.o + row * p.slots * D + V * lane;
    // what the call was given, while the kernels before may still run
    const int own = p.own_slots > 0 ? own_len(p, s) : 0;
    int tiles = -1;   // of the prefix of the (last) group that holds the sequence; -1: none
    for (int g0 = 0; g0 < p.n_groups; g0 += 32) {
        int s0, s1, len;
        const bool mine = g0 + lane < p.n_groups && group_range(p, g0 + lane, s0, s1, len) && s >= s0 && s < s1;
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, mine);
        if (who)
            tiles = __shfl_sync(0xFFFFFFFFu, len > 0 ? (len - 1) / 128 + 1 : 0, 31 - __clz((int)who));
    }
    if (p.n_groups > 0 && tiles < 0 && threadIdx.x == 0 && row % HQ == 0)
        raise_err(p.err, KAMERA_DEVERR_DESCRIPTOR);
    const int n_prefix = tiles > 0 ? (tiles + p.prefix_split - 1) / p.prefix_split * (p.two_tile ? 1 : 2) : 0;
    const int pieces = p.selected ? p.n_select * (p.P / kPgTok) : (own + kPgTok - 1) / kPgTok;
    const int n_own = p.own_slots > 0 ? (pieces + p.own_split - 1) / p.own_split : 0;
    const int n = n_prefix + n_own, gap = p.prefix_slots - n_prefix;   // unused prefix slots between
    ptx::grid_wait();
    ptx::grid_launch_next();
    // The first 32 states' outputs are asked for before their weights are known.  A
    // slot without weight may never have been written: what it holds is not used.
    constexpr int PW = 32 / kMergeWarps;
    float x[PW][V];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < PW; ++k) {
            const int i = i0 + kMergeWarps * k + warp;
            if (i >= n)
                continue;
            const float* src = o + (int64_t)(i < n_prefix ? i : i + gap) * D;
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
        m = fmaxf(m, ml[i < n_prefix ? i : i + gap].x);
#pragma unroll
    for (int d = 16; d >= 1; d /= 2)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    float l = 0.f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        acc[v] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        if (i0 > 0)
            load(i0);
        float f = 0.f;   // a state without weight adds nothing: its output was not written or is zero
        bool some = false;
        if (i < n) {
            const float2 y = ml[i < n_prefix ? i : i + gap];
            some = y.y != 0.f;
            if (some) {
                f = ex2(y.x - m);
                if (warp == 0)
                    l = fmaf(y.y, f, l);
            }
        }
        const uint32_t live = __ballot_sync(0xFFFFFFFFu, some);
#pragma unroll
        for (int k = 0; k < PW; ++k) {
            const int j = kMergeWarps * k + warp;
            const float w = __shfl_sync(0xFFFFFFFFu, f, j);
            if ((live >> j) & 1u)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    acc[v] = fmaf(x[k][v], w, acc[v]);
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
    for (int i = 2 * threadIdx.x; i < D; i += 64 * kMergeWarps) {
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
            x += part[w][i];
            y += part[w][i + 1];
        }
        *reinterpret_cast<uint32_t*>(p.out + row * D + i) = pack_bf16x2(x * inv, y * inv);
    }
    if (threadIdx.x == 0 && p.lse)
        p.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : (l == l ? -INFINITY : l);
}

// ------------------------------------------------------------------- host --
int box_rows(int P, int most)   // the largest power of two that divides a page, at most `most`
{
    int r = 16;
    while (r < most && P % (2 * r) == 0)
        r *= 2;
    return r;
}

// Splits of the own tokens: `pieces` 16-token pieces of each of `units`; three
// CTAs share an SM.
//   - Beyond 1536 tokens a slot, about six rounds of CTAs of at least 512 tokens, so
//     that ragged lengths even out (64 sequences of up to 8192 tokens: 131 us, 148 in
//     one round).
//   - Without a prefix as many splits as fill one round of CTAs, each of at least 64
//     tokens.  Up to eight are a cluster, whose CTAs join their states in shared
//     memory: no workspace and no merge launch (one context, 1024 tokens selected:
//     14.2 us with the selection, 19.9 in splits of 512 tokens), so 9 to 16 become
//     eight.
//   - Beside a prefix, the number with the least estimate of the time: the prefix
//     kernel's, or the start, 2 us a CTA and 0.75 us a round of its warps' pieces
//     (the sum of both where the prefix leaves no SM free), and after it the merge's
//     share a split.  Against as many splits as fill one round: 64 sequences of 1024
//     tokens 22.8 us where those take 24.4, one sequence of 2048 10.8 and 12.0.
void split_own(PagedParams& p, int64_t pieces, int sms)
{
    const int64_t units = (int64_t)p.n_seqs * p.H, slots = 3ll * sms;
    if (pieces <= 0) {
        p.own_split = 1;
        p.own_slots = 0;
        return;
    }
    int64_t n = 1;
    if (units * pieces > 96 * slots) {
        n = pieces / std::min(pieces, std::max<int64_t>(32, units * pieces / (6 * slots)));
    } else if (p.n_groups == 0) {
        n = std::min(std::max<int64_t>(1, slots / units), (pieces + 3) / 4);
        if (n > kMaxCluster && n <= 2 * kMaxCluster)
            n = kMaxCluster;
    } else {
        const int64_t ctas = (int64_t)p.n_groups * p.H * p.row_blocks * p.prefix_splits;
        const double prefix = (double)((ctas + sms - 1) / sms) * (6.0 + (p.two_tile ? 2.3 : 1.3) * p.prefix_split);
        const double state = 0.06 + 1.3e-6 * (double)units * p.G * p.d;   // us
        double best = 1e300;
        for (int64_t k = 1; k <= std::min<int64_t>(256, (pieces + 3) / 4); ++k) {
            const double rounds = (double)((pieces + 4 * k - 1) / (4 * k));
            const double own = 2.3 + std::max(1.0, (double)(units * k) / (double)slots) * (2.0 + 0.75 * rounds);
            const double t = (ctas % sms ? std::max(prefix, own) : prefix + own) + state * (double)k;
            if (t < best) {
                best = t;
                n = k;
            }
        }
    }
    n = std::min<int64_t>(n, 256);
    int64_t per = (pieces + n - 1) / n;
    per = (per + 3) / 4 * 4;   // whole rounds of the four warps
    p.own_split = (int32_t)std::min(per, pieces);
    p.own_slots = (int32_t)((pieces + p.own_split - 1) / p.own_split);
}

// Splits of the prefixes: the number that ends first, by waves of CTAs (one to an
// SM) times the tiles of each and about three tiles of fixed cost (between 0.3 and
// 12 the choice is the same in every case measured: one wave wherever that is
// possible).  Up to 128 rows are one tile, whose two sides take a split's tiles in
// turn; with fewer than eight tiles one side takes them all, and leaves one state
// where two would leave two (16 readers of 8192 tokens: two tiles a split, 17.2 us
// instead of 19.7; of 32768, seven tiles, 27.8 and 27.9; of 65536, fourteen, 45.5 and
// 43.7).
void split_prefix(PagedParams& p, int sms)
{
    const int64_t rows = (int64_t)p.max_group * p.G;
    p.two_tile = rows > 128 ? 1 : 0;
    p.row_blocks = (int32_t)((rows + 255) / 256);
    p.block_rows = (int32_t)(((rows + p.row_blocks - 1) / p.row_blocks + 31) / 32 * 32);   // whole warps
    const int64_t units = (int64_t)p.n_groups * p.H * p.row_blocks;
    const int64_t tiles = ((int64_t)p.max_prefix + 127) / 128;
    int64_t best = 1;
    double best_t = 1e300;
    for (int64_t ns = 1; ns <= std::min<int64_t>(tiles, 64); ++ns) {
        const int64_t per = (tiles + ns - 1) / ns;
        if ((tiles + per - 1) / per != ns)
            continue;   // the same split length as a smaller count
        const double t = (double)((units * ns + sms - 1) / sms) * (3.0 + (p.two_tile ? per : 0.5 * per));
        if (t < best_t * 0.999) {
            best_t = t;
            best = ns;
        }
    }
    p.prefix_split = (int32_t)((tiles + best - 1) / best);
    p.prefix_splits = (int32_t)best;
    if (p.prefix_split < 8)
        p.two_tile = 1;
    p.prefix_slots = p.prefix_splits * (p.two_tile ? 1 : 2);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

size_t state_bytes(const PagedParams& p)
{
    if (p.prefix_slots == 0 && p.own_slots <= kMaxCluster)
        return 0;   // a cluster
    const size_t n = (size_t)p.n_seqs * p.H * p.G * p.slots;
    return align256(n * p.d * 4) + align256(n * 8);
}

// Everything both entry points check before any pointer is looked at, and the
// plan of the call.
int plan(const KameraPagedKV* kv, const KameraPagedQuery* q, const KameraPrefixGroups* pre, const KameraPageTable* own,
         bool selected, int32_t n_select, PagedParams* p)
{
    if (!kv || !q || !own || kv->reserved != 0 || q->reserved != 0)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (kv->num_kv_heads < 1 || kv->head_dim < 8 || kv->page_size < 1 || kv->num_slots < 0 || q->n_seqs < 0 ||
        q->num_q_heads < 1 || q->num_q_heads % kv->num_kv_heads || !(q->scale == q->scale) || own->max_len < 0 ||
        own->max_pages < 0 || n_select < 0)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (pre && (pre->n_groups < 0 || pre->max_pages < 0 || pre->max_len < 0 || pre->max_group < 0))
        return KAMERA_ERR_INVALID_ARGUMENT;
    const int G = q->num_q_heads / kv->num_kv_heads;
    if ((kv->head_dim != 64 && kv->head_dim != 128) || G > 16 || (kv->page_size % 16) || kv->num_slots > 0x7FFFFFFF ||
        (int64_t)q->n_seqs * kv->num_kv_heads > 65535 || (int64_t)q->n_seqs * q->num_q_heads > 0x3FFFFFF ||
        own->max_len > 0x7FFFFF00)
        return KAMERA_ERR_UNSUPPORTED;
    if ((int64_t)own->max_pages * kv->page_size < own->max_len)
        return KAMERA_ERR_INVALID_ARGUMENT;
    std::memset(p, 0, sizeof(*p));
    p->n_seqs = q->n_seqs;
    p->H = kv->num_kv_heads;
    p->G = G;
    p->d = kv->head_dim;
    p->P = kv->page_size;
    p->num_pages = kv->num_slots / kv->page_size;
    p->scale = q->scale;
    p->max_pages = own->max_pages;
    p->max_len = own->max_len;
    p->n_select = selected ? n_select : 0;
    if (q->n_seqs == 0)
        return KAMERA_OK;
    const int s = device_sms();
    const int64_t ppp = kv->page_size / 16;
    if (selected && n_select * ppp > 0x7FFFFFF)
        return KAMERA_ERR_UNSUPPORTED;
    if (pre && pre->n_groups > 0 && pre->max_len > 0) {
        if ((int64_t)pre->max_pages * kv->page_size < pre->max_len || pre->max_group < 1 || pre->max_group > q->n_seqs)
            return KAMERA_ERR_INVALID_ARGUMENT;
        if (pre->max_len > 0x7FFFFF00)
            return KAMERA_ERR_UNSUPPORTED;
        p->n_groups = pre->n_groups;
        p->max_prefix_pages = pre->max_pages;
        p->max_prefix = pre->max_len;
        p->max_group = pre->max_group;
        split_prefix(*p, s);
        if ((int64_t)p->n_groups * p->H * p->row_blocks > 65535)
            return KAMERA_ERR_UNSUPPORTED;
    }
    split_own(*p, selected ? (own->max_len > 0 ? n_select * ppp : 0) : ((int64_t)own->max_len + 15) / 16, s);
    p->slots = p->prefix_slots + p->own_slots;
    return KAMERA_OK;
}

template <int D, int NT>
cudaError_t launch_own(const PagedLaunch& L, cudaStream_t stream)
{
    using Y = PgLayout<D, NT>;
    static_assert(Y::kBytes <= 227 * 1024, "shared memory");
    // set at every launch: the attribute belongs to the current device's context
    const cudaError_t e = cudaFuncSetAttribute(paged_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)Y::kBytes);
    if (e != cudaSuccess)
        return e;
    const dim3 grid((unsigned)std::max(L.p.own_slots, 1), (unsigned)(L.p.n_seqs * L.p.H));
    if (L.p.o || grid.x == 1)
        return launch_after(paged_kernel<D, NT>, grid, kPgThreads, Y::kBytes, stream, true, L);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kPgThreads);
    cfg.dynamicSmemBytes = Y::kBytes;
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
    return cudaLaunchKernelEx(&cfg, paged_kernel<D, NT>, L);
}

// The pointers both entry points share, then the launches.
int attend(PagedParams& p, const KameraPagedKV* kv, const KameraPagedQuery* q, const KameraPrefixGroups* pre,
           const KameraPageTable* own, const int32_t* selected, void* ws, size_t ws_bytes, int32_t* d_err,
           cudaStream_t stream)
{
    if (p.n_seqs == 0)
        return KAMERA_OK;
    if (!q->q || !q->out || (p.own_slots > 0 && (!own->pages || !own->lens || (p.n_select > 0 && !selected))) ||
        (p.n_groups > 0 && (!pre->group_start || !pre->pages || !pre->lens)))
        return KAMERA_ERR_INVALID_ARGUMENT;
    const int64_t W = (int64_t)p.H * p.d;
    int rc;
    if ((rc = check_strided(kv->k, 1, 0, kv->num_slots, kv->slot_stride, W, false)) ||
        (rc = check_strided(kv->v, 1, 0, kv->num_slots, kv->slot_stride, W, false)))
        return rc;
    if (!aligned16(q->q) || !aligned16(q->out) || (reinterpret_cast<uintptr_t>(q->lse) & 3))
        return KAMERA_ERR_MISALIGNED;
    const uintptr_t ints = reinterpret_cast<uintptr_t>(own->pages) | reinterpret_cast<uintptr_t>(own->lens) |
                           reinterpret_cast<uintptr_t>(selected) |
                           (p.n_groups > 0 ? reinterpret_cast<uintptr_t>(pre->group_start) |
                                                 reinterpret_cast<uintptr_t>(pre->pages) |
                                                 reinterpret_cast<uintptr_t>(pre->lens)
                                           : 0);
    if (ints & 3)
        return KAMERA_ERR_MISALIGNED;
    const size_t need = state_bytes(p);
    if (need > 0) {
        if (!ws || ws_bytes < need)
            return KAMERA_ERR_INVALID_ARGUMENT;
        if (!aligned16(ws))
            return KAMERA_ERR_MISALIGNED;
    }
    using Span = std::pair<uintptr_t, uintptr_t>;
    auto words = [](const int32_t* a, int64_t n) -> Span {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(a);
        return a && n > 0 ? Span{lo, lo + (uintptr_t)n * 4} : Span{lo, lo};
    };
    const int64_t rows = (int64_t)p.n_seqs * p.H * p.G;
    const Span os = span(q->out, 1, 0, rows, p.d, p.d);
    const Span ls = words(reinterpret_cast<const int32_t*>(q->lse), rows);
    const Span wss{reinterpret_cast<uintptr_t>(ws), reinterpret_cast<uintptr_t>(ws) + need};
    const Span in[] = {span(kv->k, 1, 0, kv->num_slots, kv->slot_stride, W),
                       span(kv->v, 1, 0, kv->num_slots, kv->slot_stride, W),
                       span(q->q, 1, 0, rows, p.d, p.d),
                       words(p.own_slots > 0 ? own->pages : nullptr, (int64_t)p.n_seqs * p.max_pages),
                       words(p.own_slots > 0 ? own->lens : nullptr, p.n_seqs),
                       words(selected, (int64_t)p.n_seqs * p.H * p.n_select),
                       words(p.n_groups > 0 ? pre->group_start : nullptr, (int64_t)p.n_groups + 1),
                       words(p.n_groups > 0 ? pre->pages : nullptr, (int64_t)p.n_groups * p.max_prefix_pages),
                       words(p.n_groups > 0 ? pre->lens : nullptr, p.n_groups)};
    for (const Span& a : in)
        if (overlap(a, os) || overlap(a, ls) || (need > 0 && overlap(a, wss)))
            return KAMERA_ERR_INVALID_ARGUMENT;
    if (overlap(os, ls) || (need > 0 && (overlap(wss, os) || overlap(wss, ls))))
        return KAMERA_ERR_INVALID_ARGUMENT;

    p.q = static_cast<const __nv_bfloat16*>(q->q);
    p.out = static_cast<__nv_bfloat16*>(q->out);
    p.lse = q->lse;
    p.pages = own->pages;
    p.lens = own->lens;
    if (p.own_slots == 0)
        p.n_select = p.max_len = 0;   // nothing to read: no length and no selection is looked at
    p.selected = p.n_select > 0 ? selected : nullptr;
    if (p.n_groups > 0) {
        p.group_start = pre->group_start;
        p.prefix_pages = pre->pages;
        p.prefix_lens = pre->lens;
    }
    if (need > 0) {
        p.o = static_cast<float*>(ws);
        p.ml = reinterpret_cast<float2*>(static_cast<unsigned char*>(ws) + align256((size_t)rows * p.slots * p.d * 4));
    }
    p.err = d_err;
    p.wait_ns = wait_limit_ns();
    p.withhold = test_withhold_loads() ? 1 : 0;
    // an empty pool gets one-row maps that no tile reads
    const int64_t map_rows = kv->num_slots > 0 ? kv->num_slots : 1;
    PagedLaunch L;
    std::memset(&L, 0, sizeof(L));
    // The prefix kernel first, a CTA to an SM; the own pages' kernel needs nothing
    // of it and starts at once, on the SMs that it leaves free and as they fall
    // free; the merge's CTAs read the call's inputs and wait for both.
    if (p.n_groups > 0) {
        const int r = box_rows(p.P, 128);
        L.p = p;
        L.v = static_cast<const __nv_bfloat16*>(kv->v);
        L.slot_stride = kv->slot_stride;
        L.box_rows = r;
        const int64_t groups = std::max<int64_t>(map_rows, 8);   // a pool without a whole page has none to read
        if (!make_groups_map(&L.map_k, kv->k, groups, W, kv->slot_stride, p.d / 64, r / 8) ||
            !make_groups_map(&L.map_v, kv->v, groups, W, kv->slot_stride, p.d / 64, r / 8) ||
            launch_prefix(L, stream) != cudaSuccess)
            return KAMERA_ERR_CUDA;
    }
    if (p.own_slots > 0 || p.slots == 0) {   // without any token to read the one CTA of a unit writes the empty output
        if (p.slots == 0)
            p.slots = 1;
        L.p = p;
        cudaError_t e = cudaErrorInvalidValue;
        if (make_rows_map(&L.map_k, kv->k, map_rows, W, kv->slot_stride, 64, kPgTok) &&
            make_rows_map(&L.map_v, kv->v, map_rows, W, kv->slot_stride, 64, kPgTok)) {
            if (p.d == 128)
                e = p.G <= 8 ? launch_own<128, 1>(L, stream) : launch_own<128, 2>(L, stream);
            else
                e = p.G <= 8 ? launch_own<64, 1>(L, stream) : launch_own<64, 2>(L, stream);
        }
        if (e != cudaSuccess)
            return KAMERA_ERR_CUDA;
    }
    if (need > 0) {
        const cudaError_t e =
            p.d == 128 ? launch_after(merge_kernel<128>, dim3((unsigned)rows), 32 * kMergeWarps, 0, stream, true, p)
                       : launch_after(merge_kernel<64>, dim3((unsigned)rows), 32 * kMergeWarps, 0, stream, true, p);
        if (e != cudaSuccess)
            return KAMERA_ERR_CUDA;
    }
    return KAMERA_OK;
}

}  // namespace

int plan_own_pages(const KameraPagedKV* kv, const KameraPagedQuery* q, const KameraPageTable* own, PagedParams* p)
{
    return plan(kv, q, nullptr, own, false, 0, p);
}

cudaError_t launch_own_pages(const PagedParams& p, const KameraPagedKV* kv, cudaStream_t stream)
{
    const int64_t W = (int64_t)p.H * p.d, map_rows = kv->num_slots > 0 ? kv->num_slots : 1;
    PagedLaunch L;
    std::memset(&L, 0, sizeof(L));
    L.p = p;
    if (!make_rows_map(&L.map_k, kv->k, map_rows, W, kv->slot_stride, 64, kPgTok) ||
        !make_rows_map(&L.map_v, kv->v, map_rows, W, kv->slot_stride, 64, kPgTok))
        return cudaErrorInvalidValue;
    if (p.d == 128)
        return p.G <= 8 ? launch_own<128, 1>(L, stream) : launch_own<128, 2>(L, stream);
    return p.G <= 8 ? launch_own<64, 1>(L, stream) : launch_own<64, 2>(L, stream);
}

}  // namespace kamera

using namespace kamera;

extern "C" {

size_t kamera_attend_shared_workspace_bytes(const KameraPagedKV* kv, const KameraPagedQuery* query,
                                            const KameraPrefixGroups* prefix, const KameraPageTable* own)
{
    PagedParams p;
    return plan(kv, query, prefix, own, false, 0, &p) == KAMERA_OK && p.n_seqs > 0 ? state_bytes(p) : 0;
}

int kamera_attend_shared(const KameraPagedKV* kv, const KameraPagedQuery* query, const KameraPrefixGroups* prefix,
                         const KameraPageTable* own, void* d_workspace, size_t workspace_bytes, int32_t* d_err,
                         struct CUstream_st* stream)
{
    PagedParams p;
    const int rc = plan(kv, query, prefix, own, false, 0, &p);
    return rc ? rc
              : attend(p, kv, query, prefix, own, nullptr, d_workspace, workspace_bytes, d_err,
                       reinterpret_cast<cudaStream_t>(stream));
}

size_t kamera_attend_selected_workspace_bytes(const KameraPagedKV* kv, const KameraPagedQuery* query,
                                              const KameraPageTable* table, int32_t n_select)
{
    PagedParams p;
    return plan(kv, query, nullptr, table, true, n_select, &p) == KAMERA_OK && p.n_seqs > 0 ? state_bytes(p) : 0;
}

int kamera_attend_selected(const KameraPagedKV* kv, const KameraPagedQuery* query, const KameraPageTable* table,
                           const int32_t* d_selected, int32_t n_select, void* d_workspace, size_t workspace_bytes,
                           int32_t* d_err, struct CUstream_st* stream)
{
    PagedParams p;
    const int rc = plan(kv, query, nullptr, table, true, n_select, &p);
    return rc ? rc
              : attend(p, kv, query, nullptr, table, d_selected, d_workspace, workspace_bytes, d_err,
                       reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
