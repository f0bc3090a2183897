// kamera_append.cu -- new tokens' rows into the paged pool, rotated on the way.
//
//     K[slot_t] = bf16(R(p_t) k_t),   V[slot_t] = v_t,   q'_t = bf16(R(p_t) q_t)
// (MLA: row = c_KV copied | R(p) k_rope, and the queries' rope part.)
//
// The call moves each row once in and once out, so HBM bandwidth bounds a
// prompt and launch latency a decode step; the arithmetic has to stay out of
// the way.  What costs arithmetic is the angle p theta: it is formed in fixed
// point, theta / 2 pi as a 64-bit fraction of a turn (made on the host in
// double-double) times the position modulo 2^64, which reduces the angle to
// one turn exactly by dropping the carries: three integer multiply-adds in
// place of fp64, whose rate here is 1/64 of fp32's.  The error, 2^-65 |p| turns
// from the fraction's last bit, is below 2^-34 turns for every int32 position; the
// reduced phase then goes to sine and cosine as fp32, rounded by up to 2^-26 turns.
// Each (token, frequency) is formed once per CTA, into shared memory, and
// serves every head of K and q.
//
// A row is cut into passes of 16-byte units (a rotate-half unit is the vector
// and its partner half a range on, so both are read and written by one
// thread).  A CTA owns TT tokens; a thread keeps its unit (pass, head, place)
// and walks the tokens, so the unit is decoded once and the tokens' loads
// overlap.  10368 tokens of 28 + 4 heads of 128 (191 MB): 30.6 us, 6.2 TB/s; 16381
// latent rows with 16 rope queries (105 MB): 21.3 us, 4.9 TB/s, out of HBM (17 us with
// the pool in L2); a step of 64 tokens 2.4 us in a graph, its launch and two dependent
// loads.
#include <cstdint>
#include <cstring>

#include "kamera_common.cuh"
#include "kamera_hostcheck.h"
#include "kamera_internal.h"
#include "kamera_ptx.cuh"

namespace kamera {

namespace {

constexpr int kMaxPass = 7;       // K: before / rotated / after, V (or c_KV), q: before / rotated / after

enum UnitKind { UNIT_COPY = 0, UNIT_HALF = 1, UNIT_IL = 2 };

struct AppendPass {
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;
    int64_t src_ts, src_hs, dst_ts, dst_hs;   // token and head strides (elements)
    int32_t kind, heads, units;               // units of a head
    int32_t off;                              // first element of a head's unit 0
    int32_t half;                             // UNIT_HALF: elements to the partner vector
    int32_t to_pool;                          // dst_ts counts slots, not tokens
};

struct AppendParams {
    AppendPass pass[kMaxPass];
    int32_t n_pass, items;                    // items: units of a token over all passes
    int32_t n_tokens, tokens_per_cta;
    int64_t num_slots;
    const int64_t* positions;
    const int64_t* slots;
    const int64_t* axis_pos;                  // [n_tokens][n_axes], or null
    int32_t n_axes, n_freq;
    int32_t unit_log;                         // frequencies of a unit: 2^3 (halves) or 2^2 (pairs)
    int32_t* err;
    uint64_t turn[KAMERA_MAX_ROT_DIM / 2];    // theta / 2 pi, in 2^-64 turns
    uint8_t axis[KAMERA_MAX_ROT_DIM / 2];
};

__device__ __forceinline__ uint4 ldg_row(const __nv_bfloat16* p)
{
    uint4 v;   // read once: keep it out of L1
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// q may be rotated in place: a unit is read and written by one thread alone, its
// loads before its stores, so the loads need no order beyond the data's.
template <bool INPLACE>
__device__ __forceinline__ uint4 unit_load(const __nv_bfloat16* p)
{
    if constexpr (INPLACE)
        return *reinterpret_cast<const uint4*>(p);
    else
        return ldg_row(p);
}

// A thread's unit: pass, source of the CTA's first token and destination of slot
// (or token) 0.
struct Unit {
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;
    int64_t src_ts, dst_ts;
    int32_t kind, half, to_pool, unit;   // unit: its place among the head's rotated ones
};

__device__ __forceinline__ Unit find_unit(const AppendParams& p, int it, int t0)
{
    int k = 0, u = it;
    while (u >= p.pass[k].heads * p.pass[k].units) {
        u -= p.pass[k].heads * p.pass[k].units;
        ++k;
    }
    const AppendPass& ps = p.pass[k];
    const int head = u / ps.units, unit = u - head * ps.units;
    Unit x;
    x.src = ps.src + (int64_t)t0 * ps.src_ts + (int64_t)head * ps.src_hs + ps.off + 8 * unit;
    x.dst = ps.dst + (int64_t)head * ps.dst_hs + ps.off + 8 * unit;
    x.src_ts = ps.src_ts;
    x.dst_ts = ps.dst_ts;
    x.kind = ps.kind;
    x.half = ps.half;
    x.to_pool = ps.to_pool;
    x.unit = unit;
    return x;
}

// HALVES: some pass rotates halves (else b is not used).
template <int TT, bool INPLACE, bool HALVES>
__device__ __forceinline__ void load_unit(const Unit& u, int nt, uint4 (&a)[TT], uint4 (&b)[TT])
{
#pragma unroll
    for (int t = 0; t < TT; ++t)
        if (t < nt) {   // a padding row is read too: its rows exist
            a[t] = unit_load<INPLACE>(u.src + t * u.src_ts);
            if (HALVES && u.kind == UNIT_HALF)
                b[t] = unit_load<INPLACE>(u.src + t * u.src_ts + u.half);
        }
}

template <int TT, bool HALVES>
__device__ __forceinline__ void store_unit(const AppendParams& p, const Unit& u, int t0, const float2* cs,
                                           const int64_t* slot_s, uint4 (&a)[TT], uint4 (&b)[TT])
{
#pragma unroll
    for (int t = 0; t < TT; ++t) {
        const int64_t slot = slot_s[t];
        if (slot < 0)
            continue;
        __nv_bfloat16* o = u.dst + (u.to_pool ? slot : (int64_t)(t0 + t)) * u.dst_ts;
        // pairs of frequencies: pair j of unit u at j * units + u, so that neighbouring units' reads
        // fall into neighbouring banks
        const float4* c4 = reinterpret_cast<const float4*>(cs + t * p.n_freq) + u.unit;
        if (HALVES && u.kind == UNIT_HALF) {
            float x[8], y[8];
            unpack8(a[t], x);
            unpack8(b[t], y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {   // (cos, sin) of two frequencies
                const float4 w = c4[j * (p.n_freq >> 3)];
                const float x0 = x[2 * j], x1 = x[2 * j + 1];
                x[2 * j] = fmaf(x0, w.x, -(y[2 * j] * w.y));
                y[2 * j] = fmaf(y[2 * j], w.x, x0 * w.y);
                x[2 * j + 1] = fmaf(x1, w.z, -(y[2 * j + 1] * w.w));
                y[2 * j + 1] = fmaf(y[2 * j + 1], w.z, x1 * w.w);
            }
            a[t] = pack8(x);
            *reinterpret_cast<uint4*>(o + u.half) = pack8(y);
        } else if (!HALVES && u.kind == UNIT_IL) {   // pairs (2i, 2i + 1) inside the vector
            float x[8];
            unpack8(a[t], x);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float4 w = c4[j * (p.n_freq >> 2)];
                const float a0 = x[4 * j], b0 = x[4 * j + 1], a1 = x[4 * j + 2], b1 = x[4 * j + 3];
                x[4 * j] = fmaf(a0, w.x, -(b0 * w.y));
                x[4 * j + 1] = fmaf(b0, w.x, a0 * w.y);
                x[4 * j + 2] = fmaf(a1, w.z, -(b1 * w.w));
                x[4 * j + 3] = fmaf(b1, w.z, a1 * w.w);
            }
            a[t] = pack8(x);
        }
        *reinterpret_cast<uint4*>(o) = a[t];
    }
}

// The rows of a thread's first unit are loaded before anything else: their
// latency covers the slots', the positions' and the angles'.  Four tokens and two
// vectors of each are 32 registers of loads: held to 64 in all three CTAs fit an SM
// instead of two (10368 tokens of 28 + 4 heads of 128: 30.6 us, 33.1 with 87).
template <int TT, bool INPLACE, bool HALVES>
__global__ void __launch_bounds__(512, HALVES && TT > 1 ? 2 : 0) append_kernel(const __grid_constant__ AppendParams p)
{
    extern __shared__ __align__(16) float2 cs[];   // [TT][n_freq] cos, sin
    __shared__ int64_t slot_s[TT];                 // -1: this token is not written
    const int t0 = blockIdx.x * TT;
    const int nt = min(TT, p.n_tokens - t0);
    ptx::grid_wait();
    ptx::grid_launch_next();
    uint4 a[TT], b[TT];
    Unit u;
    const bool has = (int)threadIdx.x < p.items;
    if (has) {
        u = find_unit(p, threadIdx.x, t0);
        load_unit<TT, INPLACE, HALVES>(u, nt, a, b);
    }
    if (threadIdx.x < TT) {
        int64_t slot = -1;
        if ((int)threadIdx.x < nt) {
            const int t = t0 + threadIdx.x;
            slot = p.slots[t];
            int32_t bits = 0;
            if (slot < -1 || slot >= p.num_slots)
                bits |= KAMERA_DEVERR_SLOT;
            if (slot != -1) {
                if (p.n_axes == 0) {
                    const int64_t x = p.positions[t];
                    if (x > KAMERA_MAX_ABS_DELTA || x < -KAMERA_MAX_ABS_DELTA)
                        bits |= KAMERA_DEVERR_DESCRIPTOR;
                }
                for (int c = 0; c < p.n_axes; ++c) {
                    const int64_t x = p.axis_pos[(int64_t)t * p.n_axes + c];
                    if (x > KAMERA_MAX_ABS_DELTA || x < -KAMERA_MAX_ABS_DELTA)
                        bits |= KAMERA_DEVERR_DESCRIPTOR;
                }
            }
            if (bits) {
                raise_err(p.err, bits);
                slot = -1;
            }
        }
        slot_s[threadIdx.x] = slot;
    }
    for (int e = threadIdx.x; e < nt * p.n_freq; e += blockDim.x) {
        const int t = e / p.n_freq, f = e - t * p.n_freq;
        const int64_t pos = p.n_axes == 0 ? p.positions[t0 + t]
                                          : p.axis_pos[(int64_t)(t0 + t) * p.n_axes + p.axis[f]];
        // the phase modulo a turn, signed: [-1/2, 1/2) turns = [-1, 1) half-turns
        const int64_t ph = (int64_t)((uint64_t)pos * p.turn[f]);
        float s, c;
        sincospif((float)ph * 1.08420217248550443e-19f, &s, &c);   // 2^-63
        const int unit = f >> p.unit_log, pair = (f & ((1 << p.unit_log) - 1)) >> 1;
        cs[t * p.n_freq + 2 * (pair * (p.n_freq >> p.unit_log) + unit) + (f & 1)] = make_float2(c, s);
    }
    __syncthreads();
    if (has)
        store_unit<TT, HALVES>(p, u, t0, cs, slot_s, a, b);
    for (int it = threadIdx.x + blockDim.x; it < p.items; it += blockDim.x) {   // rows of more than 512 units
        u = find_unit(p, it, t0);
        load_unit<TT, INPLACE, HALVES>(u, nt, a, b);
        store_unit<TT, HALVES>(p, u, t0, cs, slot_s, a, b);
    }
}

template <int TT>
cudaError_t launch_append_t(const AppendParams& p, bool inplace, cudaStream_t stream)
{
    const int rounds = (p.items + 511) / 512;
    const int threads = ((p.items + rounds - 1) / rounds + 31) / 32 * 32;
    const unsigned grid = (unsigned)((p.n_tokens + TT - 1) / TT);
    const size_t smem = sizeof(float2) * (size_t)TT * (size_t)p.n_freq;   // at most 8 KB
    const auto kernel = p.unit_log == 3 ? (inplace ? append_kernel<TT, true, true> : append_kernel<TT, false, true>)
                                        : (inplace ? append_kernel<TT, true, false> : append_kernel<TT, false, false>);
    return launch_after(kernel, dim3(grid), threads, smem, stream, true, p);
}

// The passes of one source row kind: the rotary range [ro, ro + rr) rotated
// (rr = 0: none), the rest copied.
void add_passes(AppendParams& p, const RopeParams* r, const void* src, void* dst, int64_t src_ts, int64_t src_hs,
                int64_t dst_ts, int64_t dst_hs, int heads, int width, int dst_off, int to_pool)
{
    auto add = [&](int kind, int off, int units, int half) {
        if (units <= 0 || heads <= 0)
            return;
        AppendPass& a = p.pass[p.n_pass++];
        a.src = static_cast<const __nv_bfloat16*>(src);
        a.dst = static_cast<__nv_bfloat16*>(dst) + dst_off;
        a.src_ts = src_ts;
        a.src_hs = src_hs;
        a.dst_ts = dst_ts;
        a.dst_hs = dst_hs;
        a.kind = kind;
        a.heads = heads;
        a.units = units;
        a.off = off;
        a.half = half;
        a.to_pool = to_pool;
        p.items += heads * units;
    };
    if (!r || r->rot_dim == 0) {
        add(UNIT_COPY, 0, width / 8, 0);
        return;
    }
    const int ro = r->rot_offset, rr = r->rot_dim;
    add(UNIT_COPY, 0, ro / 8, 0);
    if (r->pairing == KAMERA_ROPE_ROTATE_HALF)
        add(UNIT_HALF, ro, rr / 16, rr / 2);
    else
        add(UNIT_IL, ro, rr / 8, 0);
    add(UNIT_COPY, ro + rr, (width - ro - rr) / 8, 0);
}

cudaError_t launch_append(AppendParams& p, const RopeParams& r, bool inplace, cudaStream_t stream)
{
    p.n_freq = r.n_freq;
    p.unit_log = r.pairing == KAMERA_ROPE_ROTATE_HALF ? 3 : 2;
    p.n_axes = r.n_axes;
    p.axis_pos = r.axis_delta;
    for (int f = 0; f < r.n_freq; ++f) {
        p.turn[f] = turn_fraction(r.inv_freq[f]);
        p.axis[f] = r.axis[f];
    }
    // One token a CTA while that leaves SMs idle or barely filled (a decode step is
    // latency); four from eight tokens an SM on, so that the set-up (slots, angles) is
    // shared and 64 bytes a thread are in flight.  28 + 4 heads of 128: 5.5 us either way
    // for 912 and 1216 tokens, 6.1 with four and 8.2 with one for 1824, 29.1 and 38.4 for
    // 9728.  Narrow rows fill an SM later and lose nothing by four before: one 64-wide head
    // 5.0 and 4.8 us (launches) for 1824, 7.6 and 10.5 for 9728; latent rows of 576 without
    // queries 5.1 and 4.7, 6.7 and 11.3.  (10368 tokens of the first: 30.6 with four, 34.0
    // with two; before the registers were held down 47.7 with one, 34.9 with two, 33.8
    // with four, 42.3 with eight.)
    if (p.n_tokens >= 8 * device_sms())
        return launch_append_t<4>(p, inplace, stream);
    return launch_append_t<1>(p, inplace, stream);
}

// Whether rows of `wa` and `wb` elements (token strides sa, sb) from a and b may
// touch: with one stride the rows interleave, and only the columns decide.
bool rows_touch(const void* a, int64_t sa, int64_t wa, const void* b, int64_t sb, int64_t wb, int64_t n)
{
    if (!overlap(span(a, 1, 0, n, sa, wa), span(b, 1, 0, n, sb, wb)))
        return false;
    if (sa != sb || sa < 1)
        return true;
    const int64_t d = ((int64_t)(reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a))) / 2;
    const int64_t r = ((d % sa) + sa) % sa;
    return r < wa || r + wb > sa;
}

// What both entry points check of the rows: k [n][wk], v [n][wv], q [n][Hq][wq].
int check_rows(const KameraAppendRows* x, const KameraRope* rope, int64_t wk, int64_t wv, int64_t wq, int num_layers)
{
    if (x->reserved != 0 || x->n_tokens < 0 || x->num_q_heads < 0 || x->layer < 0 || x->layer >= num_layers)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if ((x->q == nullptr) != (x->q_out == nullptr) || (x->q && x->num_q_heads < 1))
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (x->n_tokens == 0)
        return KAMERA_OK;
    if (!x->slots || (rope->n_axes == 0 && !x->positions) || (wk > 0 && !x->k) || (wv > 0 && !x->v))
        return KAMERA_ERR_INVALID_ARGUMENT;
    if ((reinterpret_cast<uintptr_t>(x->slots) & 7) || (reinterpret_cast<uintptr_t>(x->positions) & 7))
        return KAMERA_ERR_MISALIGNED;
    const int64_t n = x->n_tokens, heads = x->num_q_heads > 1 ? x->num_q_heads - 1 : 0;
    struct Rows {
        const void* p;
        int64_t stride, width;
    };
    const Rows in[3] = {{wk > 0 ? x->k : nullptr, x->k_stride, wk},
                        {wv > 0 ? x->v : nullptr, x->v_stride, wv},
                        {x->q, x->q_stride, heads * x->q_head_stride + wq}};
    for (const Rows& r : in) {
        if (!r.p)
            continue;
        if (!aligned16(r.p) || (n > 1 && (r.stride & 7)))
            return KAMERA_ERR_MISALIGNED;
        if (n > 1 && r.stride < r.width)
            return KAMERA_ERR_INVALID_ARGUMENT;
    }
    if (x->q) {
        const int64_t wo = heads * x->q_out_head_stride + wq;
        if (!aligned16(x->q_out) || (n > 1 && (x->q_out_stride & 7)) ||
            (x->num_q_heads > 1 && ((x->q_head_stride | x->q_out_head_stride) & 7)))
            return KAMERA_ERR_MISALIGNED;
        if (x->num_q_heads > 1 && (x->q_head_stride < wq || x->q_out_head_stride < wq))
            return KAMERA_ERR_INVALID_ARGUMENT;
        if (n > 1 && x->q_out_stride < wo)
            return KAMERA_ERR_INVALID_ARGUMENT;
        const bool same = x->q == x->q_out && (n == 1 || x->q_stride == x->q_out_stride) &&
                          (x->num_q_heads == 1 || x->q_head_stride == x->q_out_head_stride);
        for (int i = 0; i < 3; ++i)
            if (in[i].p && !(i == 2 && same) &&
                rows_touch(x->q_out, x->q_out_stride, wo, in[i].p, in[i].stride, in[i].width, n))
                return KAMERA_ERR_INVALID_ARGUMENT;
    }
    return KAMERA_OK;
}

std::pair<uintptr_t, uintptr_t> rows_span(const void* p, int64_t n, int64_t stride, int64_t width)
{
    return p ? span(p, 1, 0, n, stride, width) : std::pair<uintptr_t, uintptr_t>{0, 0};
}

}  // namespace

}  // namespace kamera

using namespace kamera;

extern "C" {

int kamera_append_kv(const KameraGqaPool* pool, const KameraAppendRows* rows, const KameraRope* rope, int32_t* d_err,
                     struct CUstream_st* stream)
{
    if (!pool || !rows || !rope)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (pool->num_layers < 1 || pool->num_kv_heads < 1 || pool->head_dim < 8 || pool->reserved != 0)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if ((pool->head_dim % 8) || pool->head_dim > KAMERA_MAX_ROW_ELEMS || pool->num_kv_heads > 65535 ||
        rows->num_q_heads > 65535)
        return KAMERA_ERR_UNSUPPORTED;
    const int64_t L = pool->num_layers, d = pool->head_dim, W = pool->num_kv_heads * d;
    int rc;
    if ((rc = check_strided(pool->k, L, pool->layer_stride, pool->num_slots, pool->slot_stride, W, true)))
        return rc;
    if ((rc = check_strided(pool->v, L, pool->layer_stride, pool->num_slots, pool->slot_stride, W, true)))
        return rc;
    const auto pk = span(pool->k, L, pool->layer_stride, pool->num_slots, pool->slot_stride, W);
    const auto pv = span(pool->v, L, pool->layer_stride, pool->num_slots, pool->slot_stride, W);
    if (overlap(pk, pv))
        return KAMERA_ERR_INVALID_ARGUMENT;
    RopeParams r;
    if ((rc = fill_rope(rope, pool->head_dim, &r)))
        return rc;
    if ((rc = check_rows(rows, rope, W, W, d, pool->num_layers)) || rows->n_tokens == 0)
        return rc;
    const int64_t n = rows->n_tokens;
    const auto ks = rows_span(rows->k, n, rows->k_stride, W), vs = rows_span(rows->v, n, rows->v_stride, W);
    const auto qs = rows_span(rows->q, n, rows->q_stride, (rows->num_q_heads - 1) * rows->q_head_stride + d);
    const auto os = rows_span(rows->q_out, n, rows->q_out_stride, (rows->num_q_heads - 1) * rows->q_out_head_stride + d);
    for (const auto& s : {ks, vs, qs, os})
        if (overlap(s, pk) || overlap(s, pv))
            return KAMERA_ERR_INVALID_ARGUMENT;
    AppendParams p;
    std::memset(&p, 0, sizeof(p));
    __nv_bfloat16* dk = static_cast<__nv_bfloat16*>(pool->k) + rows->layer * pool->layer_stride;
    __nv_bfloat16* dv = static_cast<__nv_bfloat16*>(pool->v) + rows->layer * pool->layer_stride;
    add_passes(p, &r, rows->k, dk, rows->k_stride, d, pool->slot_stride, d, pool->num_kv_heads, (int)d, 0, 1);
    add_passes(p, nullptr, rows->v, dv, rows->v_stride, d, pool->slot_stride, d, pool->num_kv_heads, (int)d, 0, 1);
    if (rows->q)
        add_passes(p, &r, rows->q, rows->q_out, rows->q_stride, rows->q_head_stride, rows->q_out_stride,
                   rows->q_out_head_stride, rows->num_q_heads, (int)d, 0, 0);
    p.n_tokens = rows->n_tokens;
    p.num_slots = pool->num_slots;
    p.positions = rows->positions;
    p.slots = rows->slots;
    p.err = d_err;
    return launch_append(p, r, rows->q && rows->q == rows->q_out, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? KAMERA_OK
               : KAMERA_ERR_CUDA;
}

int kamera_mla_append_kv(const KameraMlaPool* pool, const KameraAppendRows* rows, const KameraRope* rope,
                         int32_t* d_err, struct CUstream_st* stream)
{
    if (!pool || !rows || !rope)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (pool->num_layers < 1 || pool->kv_lora_rank < 0 || pool->rope_dim < 0 || pool->reserved != 0 ||
        pool->kv_lora_rank + pool->rope_dim < 16)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if ((pool->kv_lora_rank % 16) || (pool->rope_dim % 16) ||
        pool->kv_lora_rank + pool->rope_dim > KAMERA_MAX_ROW_ELEMS || pool->rope_dim > KAMERA_MAX_ROT_DIM ||
        rows->num_q_heads > 65535)
        return KAMERA_ERR_UNSUPPORTED;
    const int64_t L = pool->num_layers, lora = pool->kv_lora_rank, rd = pool->rope_dim, W = lora + rd;
    int rc;
    if ((rc = check_strided(pool->kv, L, pool->layer_stride, pool->num_slots, pool->slot_stride, W, true)))
        return rc;
    RopeParams r;
    if ((rc = fill_rope(rope, pool->rope_dim, &r)))
        return rc;
    if (rows->q && rd == 0)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if ((rc = check_rows(rows, rope, rd, lora, rd, pool->num_layers)) || rows->n_tokens == 0)
        return rc;
    const int64_t n = rows->n_tokens;
    const auto ps = span(pool->kv, L, pool->layer_stride, pool->num_slots, pool->slot_stride, W);
    const auto ks = rows_span(rd > 0 ? rows->k : nullptr, n, rows->k_stride, rd);
    const auto vs = rows_span(lora > 0 ? rows->v : nullptr, n, rows->v_stride, lora);
    const auto qs = rows_span(rows->q, n, rows->q_stride, (rows->num_q_heads - 1) * rows->q_head_stride + rd);
    const auto os =
        rows_span(rows->q_out, n, rows->q_out_stride, (rows->num_q_heads - 1) * rows->q_out_head_stride + rd);
    for (const auto& s : {ks, vs, qs, os})
        if (overlap(s, ps))
            return KAMERA_ERR_INVALID_ARGUMENT;
    AppendParams p;
    std::memset(&p, 0, sizeof(p));
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(pool->kv) + rows->layer * pool->layer_stride;
    add_passes(p, nullptr, rows->v, dst, rows->v_stride, 0, pool->slot_stride, 0, 1, (int)lora, 0, 1);
    if (rd > 0)
        add_passes(p, &r, rows->k, dst, rows->k_stride, 0, pool->slot_stride, 0, 1, (int)rd, (int)lora, 1);
    if (rows->q)
        add_passes(p, &r, rows->q, rows->q_out, rows->q_stride, rows->q_head_stride, rows->q_out_stride,
                   rows->q_out_head_stride, rows->num_q_heads, (int)rd, 0, 0);
    p.n_tokens = rows->n_tokens;
    p.num_slots = pool->num_slots;
    p.positions = rows->positions;
    p.slots = rows->slots;
    p.err = d_err;
    return launch_append(p, r, rows->q && rows->q == rows->q_out, reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? KAMERA_OK
               : KAMERA_ERR_CUDA;
}

}  // extern "C"
