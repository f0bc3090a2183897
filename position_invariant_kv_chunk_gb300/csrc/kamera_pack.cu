// kamera_pack.cu -- pages of the pool in 4 bits: packing and unpacking.
//
// 16 numbers share a scale s (e4m3) and are each a level of e2m1 (0, 0.5, 1, 1.5, 2,
// 3, 4, 6) times s.  s = rn(max |x| / (6 unit)); a number's code is rn(x / (s unit)).
// Both roundings are decided exactly:
//   - a bf16 maximum over 6 lies at least 2^-11 of itself from a tie of e4m3 or on it, so
//     the product with fp32's 1/6 (2^-23 off at most) is rounded to 14 bits first, which
//     puts ties (five bits) back where they belong;
//   - x / s (8 bits over 4) lies on a tie of e2m1 or at least 2^-10 from it, so the
//     product with the reciprocal (2^-22 off at most) is likewise rounded to a multiple
//     of 2^-13 first.
// What attention reads (kamera_packed.cu) sets the layout: 16 tokens of a head are one
// run of 18 d bytes,
//   keys     [d / 32][16 tokens][16 bytes]   32 channels of a token in 16 bytes
//   values   [d][8 bytes]                    16 tokens of a channel in 8 bytes
//   scales   keys [16 tokens][d / 16], values [d]
// so that a thread per token (keys) or per channel (values) reads its numbers in whole
// vectors without bank conflicts.
// A warp takes 16 tokens of a head: 8 d values, all its loads in flight at once.
// Bound by memory: 65536 tokens of four heads of 128, 172 MB either way, take 30 us to
// pack and 25.5 to unpack (5.7 and 6.7 TB/s).  Packing has most of its instructions in the
// rounding: divisions in it, instead of products rounded once more, cost 5 us.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>
#include <utility>

#include "kamera_common.cuh"
#include "kamera_hostcheck.h"
#include "kamera_internal.h"
#include "kamera_packed.h"
#include "kamera_ptx.cuh"
#include "kamera_warpmma.cuh"

namespace kamera {

namespace {

constexpr int kPkWarps = 4;

struct PackParams {
    __nv_bfloat16* k;              // one layer of the pool
    __nv_bfloat16* v;
    unsigned char* data;           // packed pages
    const int32_t* kv_pages;
    const int32_t* packed_pages;
    const int32_t* tokens;
    int64_t slot_stride, kv_pages_n, packed_pages_n, items;   // items: (entry, piece, head)
    int32_t H, P, pieces;
    float k_unit, v_unit;
    int32_t* err;
};

// One item of the call: false when there is nothing to do.
struct PackItem {
    int64_t row;             // the first of its 16 rows
    unsigned char* rec;      // its 18 d bytes
    int count;               // rows that count, 1..16
    int h;
};

template <int D>
__device__ __forceinline__ bool pack_item(const PackParams& p, PackItem& it)
{
    const int64_t item = (int64_t)blockIdx.x * kPkWarps + (threadIdx.x >> 5);
    if (item >= p.items)
        return false;
    const int64_t at = wmma16::quotient(item, p.H);
    it.h = (int)(item - at * p.H);
    const int64_t e = wmma16::quotient(at, p.pieces);
    const int piece = (int)(at - e * p.pieces);
    const int64_t a = p.kv_pages[e], b = p.packed_pages[e];
    const int n = p.tokens[e];
    int32_t bits = 0;
    if (a < 0 || a >= p.kv_pages_n || b < 0 || b >= p.packed_pages_n)
        bits |= KAMERA_DEVERR_SLOT;
    if (n < 0 || n > p.P)
        bits |= KAMERA_DEVERR_LEN;
    if (bits && piece == 0 && it.h == 0 && (threadIdx.x & 31) == 0)
        raise_err(p.err, bits);
    it.count = min(n - 16 * piece, 16);
    if (bits || it.count <= 0)
        return false;
    it.row = a * p.P + 16 * piece;
    it.rec = p.data + ((b * p.H + it.h) * p.pieces + piece) * (int64_t)kPackedPiece<D>;
    return true;
}

// The largest magnitude of a group of bf16 numbers, as bf16 bits without the sign, and
// NaN (above 0x7F80) among them.
__device__ __forceinline__ uint32_t mag2(uint32_t w) { return w & 0x7FFF7FFFu; }

// NaN halves of a bf16 pair become 0.
__device__ __forceinline__ uint32_t drop_nan(uint32_t w)
{
    return w & ~__vcmpgtu2(mag2(w), 0x7F807F80u);
}

// A group's scale byte and the factor that takes a number to its code's level, from
// the largest magnitude (bf16 bits, no NaN).
__device__ __forceinline__ uint32_t group_scale(uint32_t amax, float unit, float& factor)
{
    // (an infinity saturates to 448; the unit is a power of two)
    const float sixth = __uint_as_float(amax << 16) * (1.f / unit) * (1.f / 6.f);
    const float want = __uint_as_float((__float_as_uint(sixth) + 0x200u) & ~0x3FFu);
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(want));
    const uint32_t byte = two & 0xFFu;
    const float s = e4m3_to_float(byte);
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));   // (2^-23 off at most; s is 2^-9 to 448)
    factor = byte ? inv * (1.f / unit) : 0.f;
    return byte;
}

// Two numbers to their codes: a byte, the first in its low half.
__device__ __forceinline__ uint32_t codes2(float a, float b, float factor)
{
    constexpr float kRound = 1536.f;   // the sum's last place is 2^-13
    uint16_t r;
    const uint64_t f2 = ptx::f2_make(__float_as_uint(factor), __float_as_uint(factor));
    const uint64_t up = ptx::f2_make(__float_as_uint(kRound), __float_as_uint(kRound));
    const uint64_t down = ptx::f2_make(__float_as_uint(-kRound), __float_as_uint(-kRound));
    float x, y;
    asm("mov.b64 {%0, %1}, %2;"
        : "=f"(x), "=f"(y)
        : "l"(ptx::f2_add(ptx::f2_fma(ptx::f2_make(__float_as_uint(a), __float_as_uint(b)), f2, up), down)));
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u16.u8 %0, t;\n\t}" : "=h"(r) : "f"(y), "f"(x));
    return r;
}

// Packing.  Keys: a lane takes whole groups (16 channels of a token).  Values: a lane
// takes eight channels of 8 (d = 64: 4) tokens, and the lanes that share channels
// exchange maxima and codes.
template <int D>
__global__ void __launch_bounds__(32 * kPkWarps) pack_kernel(const PackParams p)
{
    constexpr int GR = D / 16;            // key groups of a token
    constexpr int KI = 16 * GR / 32;      // groups of a lane
    constexpr int VC = D / 8;             // 16-byte vectors of a value row
    constexpr int TS = 32 / VC;           // lanes that share eight channels (2 or 4)
    constexpr int VT = 16 / TS;           // tokens of a lane (8 or 4)
    const int lane = threadIdx.x & 31;
    ptx::grid_wait();
    ptx::grid_launch_next();
    PackItem it;
    if (!pack_item<D>(p, it))
        return;
    const int64_t head = (int64_t)it.h * D;
    const __nv_bfloat16* ks = p.k + it.row * p.slot_stride + head;
    const __nv_bfloat16* vs = p.v + it.row * p.slot_stride + head;
    uint4 x[KI][2], y[VT];
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < KI; ++i) {
        const int t = (32 * i + lane) / GR, g = lane % GR;
        const uint4* src = reinterpret_cast<const uint4*>(ks + t * p.slot_stride + 16 * g);
        x[i][0] = t < it.count ? src[0] : none;
        x[i][1] = t < it.count ? src[1] : none;
    }
    const int vc = lane % VC, part = lane / VC;
#pragma unroll
    for (int i = 0; i < VT; ++i) {
        const int t = VT * part + i;
        y[i] = t < it.count ? *reinterpret_cast<const uint4*>(vs + t * p.slot_stride + 8 * vc) : none;
    }
    bool nan = false;
#pragma unroll
    for (int i = 0; i < KI; ++i) {
        const int t = (32 * i + lane) / GR, g = lane % GR;
        uint32_t w[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            m = __vmaxu2(m, mag2(w[j]));
        uint32_t amax = max(m & 0xFFFFu, m >> 16);
        if (amax > 0x7F80u) {
            nan = true;
            m = 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                w[j] = drop_nan(w[j]);
                m = __vmaxu2(m, mag2(w[j]));
            }
            amax = max(m & 0xFFFFu, m >> 16);
        }
        float f;
        const uint32_t s = group_scale(amax, p.k_unit, f);
        uint32_t c[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            c[j >> 2] |= codes2(bf16lo(w[j]), bf16hi(w[j]), f) << (8 * (j & 3));
        *reinterpret_cast<uint2*>(it.rec + (g >> 1) * 256 + t * 16 + (g & 1) * 8) = make_uint2(c[0], c[1]);
        it.rec[kPackedKS<D> + t * GR + g] = (unsigned char)s;
    }
    // values: channels 8 vc .. 8 vc + 7, two to a word
    uint32_t m[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < VT; ++i) {
        const uint32_t w[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            m[j] = __vmaxu2(m[j], mag2(w[j]));
    }
    const uint32_t big = __vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3]));
    if (max(big & 0xFFFFu, big >> 16) > 0x7F80u) {
        nan = true;
        m[0] = m[1] = m[2] = m[3] = 0u;
#pragma unroll
        for (int i = 0; i < VT; ++i) {
            y[i] = make_uint4(drop_nan(y[i].x), drop_nan(y[i].y), drop_nan(y[i].z), drop_nan(y[i].w));
            const uint32_t w[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                m[j] = __vmaxu2(m[j], mag2(w[j]));
        }
    }
#pragma unroll
    for (int o = VC; o < 32; o *= 2)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            m[j] = __vmaxu2(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], o));
    uint32_t sc[2] = {0u, 0u}, code[8];   // channel i: VT / 2 bytes
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f;
        const uint32_t s = group_scale((i & 1) ? m[i >> 1] >> 16 : m[i >> 1] & 0xFFFFu, p.v_unit, f);
        sc[i >> 2] |= s << (8 * (i & 3));
        code[i] = 0u;
#pragma unroll
        for (int t = 0; t < VT; t += 2) {
            const uint32_t wa = (i >> 1) == 0 ? y[t].x : (i >> 1) == 1 ? y[t].y : (i >> 1) == 2 ? y[t].z : y[t].w;
            const uint32_t wb =
                (i >> 1) == 0 ? y[t + 1].x : (i >> 1) == 1 ? y[t + 1].y : (i >> 1) == 2 ? y[t + 1].z : y[t + 1].w;
            const float a = (i & 1) ? bf16hi(wa) : bf16lo(wa), b = (i & 1) ? bf16hi(wb) : bf16lo(wb);
            code[i] |= codes2(a, b, f) << (4 * t);
        }
    }
    unsigned char* out = it.rec + kPackedV<D> + 64 * vc;
    if constexpr (D == 128) {
        // the two lanes of eight channels swap halves: each writes four channels whole
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, part ? code[i] : code[4 + i], VC);
            w[2 * i] = part ? other : code[i];
            w[2 * i + 1] = part ? code[4 + i] : other;
        }
        *reinterpret_cast<uint4*>(out + 32 * part) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(out + 32 * part + 16) = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
        // four lanes with four tokens each: lane `part` gathers channels 2 part, 2 part + 1
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int r = 0; r < 4; ++r) {   // from the lane with tokens 4 r .. 4 r + 3
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t a = __shfl_sync(0xFFFFFFFFu, code[2 * q], vc + VC * r);
                const uint32_t b = __shfl_sync(0xFFFFFFFFu, code[2 * q + 1], vc + VC * r);
                if (q == part) {
                    w[r >> 1] |= a << (16 * (r & 1));
                    w[2 + (r >> 1)] |= b << (16 * (r & 1));
                }
            }
        }
        *reinterpret_cast<uint4*>(out + 16 * part) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (part == 0)
        *reinterpret_cast<uint2*>(it.rec + kPackedVS<D> + 8 * vc) = make_uint2(sc[0], sc[1]);
    if (__any_sync(0xFFFFFFFFu, nan) && lane == 0)
        raise_err(p.err, KAMERA_DEVERR_VALUE);
}

// A group's scale as a pair of fp16 numbers, 2^-8 of its value (exact), and a pair of
// codes times it, in fp32 (2^8 folded into `unit`).
__device__ __forceinline__ float2 stored_pair(uint32_t codes, uint32_t scale2, float unit)
{
    const uint32_t w = mul_f16x2(codes, scale2);   // 6 significant bits: exact
    const __half2 h = *reinterpret_cast<const __half2*>(&w);
    return make_float2(__low2float(h) * unit, __high2float(h) * unit);
}

// Unpacking: a lane takes eight channels (16 bytes of a row) of every second (fourth)
// token, so that a warp writes whole rows.
template <int D>
__global__ void __launch_bounds__(32 * kPkWarps) unpack_kernel(const PackParams p)
{
    constexpr int GR = D / 16, VC = D / 8, TS = 32 / VC, VT = 16 / TS;
    const int lane = threadIdx.x & 31;
    ptx::grid_wait();
    ptx::grid_launch_next();
    PackItem it;
    if (!pack_item<D>(p, it))
        return;
    const int vc = lane % VC, part = lane / VC;
    __nv_bfloat16* kd = p.k + it.row * p.slot_stride + (int64_t)it.h * D + 8 * vc;
    __nv_bfloat16* vd = p.v + it.row * p.slot_stride + (int64_t)it.h * D + 8 * vc;
    uint32_t kc[VT], ksc[VT], vcode[8];
#pragma unroll
    for (int i = 0; i < VT; ++i) {   // tokens TS i + part
        const int t = TS * i + part;
        kc[i] = *reinterpret_cast<const uint32_t*>(it.rec + (vc >> 2) * 256 + t * 16 + (vc & 3) * 4);
        ksc[i] = it.rec[kPackedKS<D> + t * GR + (vc >> 1)];
    }
    // values: tokens VT part .. VT part + VT - 1 of the lane's eight channels
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const unsigned char* src = it.rec + kPackedV<D> + 64 * vc + 8 * i + VT / 2 * part;
        if constexpr (VT == 8)
            vcode[i] = *reinterpret_cast<const uint32_t*>(src);
        else
            vcode[i] = *reinterpret_cast<const uint16_t*>(src);
    }
    const uint2 vsc = *reinterpret_cast<const uint2*>(it.rec + kPackedVS<D> + 8 * vc);
    const float ku = p.k_unit * 256.f, vu = p.v_unit * 256.f;
#pragma unroll
    for (int i = 0; i < VT; ++i) {
        const int t = TS * i + part;
        const uint32_t s2 = ksc[i] * 0x00800080u;
        const float2 a = stored_pair(e2m1_pair<0>(kc[i]), s2, ku), b = stored_pair(e2m1_pair<1>(kc[i]), s2, ku);
        const float2 c = stored_pair(e2m1_pair<2>(kc[i]), s2, ku), d = stored_pair(e2m1_pair<3>(kc[i]), s2, ku);
        if (t < it.count)
            *reinterpret_cast<uint4*>(kd + t * p.slot_stride) =
                make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y), pack_bf16x2(c.x, c.y), pack_bf16x2(d.x, d.y));
    }
    auto tokens2 = [&](auto pair) {   // tokens 2 B, 2 B + 1 of the lane's VT
        constexpr int B = decltype(pair)::value;
        float2 f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t s = ((i < 4 ? vsc.x : vsc.y) >> (8 * (i & 3))) & 0xFFu;
            f[i] = stored_pair(e2m1_pair<B>(vcode[i]), s * 0x00800080u, vu);
        }
        const int t = VT * part + 2 * B;
        if (t < it.count)
            *reinterpret_cast<uint4*>(vd + t * p.slot_stride) =
                make_uint4(pack_bf16x2(f[0].x, f[1].x), pack_bf16x2(f[2].x, f[3].x), pack_bf16x2(f[4].x, f[5].x),
                           pack_bf16x2(f[6].x, f[7].x));
        if (t + 1 < it.count)
            *reinterpret_cast<uint4*>(vd + (t + 1) * p.slot_stride) =
                make_uint4(pack_bf16x2(f[0].y, f[1].y), pack_bf16x2(f[2].y, f[3].y), pack_bf16x2(f[4].y, f[5].y),
                           pack_bf16x2(f[6].y, f[7].y));
    };
    tokens2(std::integral_constant<int, 0>{});
    tokens2(std::integral_constant<int, 1>{});
    if constexpr (VT == 8) {
        tokens2(std::integral_constant<int, 2>{});
        tokens2(std::integral_constant<int, 3>{});
    }
}

int convert(const KameraGqaPool* pool, int32_t layer, const KameraPackedPool* packed, const int32_t* kv_pages,
            const int32_t* packed_pages, const int32_t* tokens, int32_t n, int32_t* d_err, cudaStream_t stream, bool pack)
{
    if (!pool || pool->reserved != 0 || pool->num_layers < 1 || layer < 0 || layer >= pool->num_layers || n < 0 ||
        pool->num_kv_heads < 1 || pool->head_dim < 1 || pool->num_slots < 0)
        return KAMERA_ERR_INVALID_ARGUMENT;
    const int rc = check_packed(packed);
    if (rc)
        return rc;
    if (pool->num_kv_heads != packed->num_kv_heads || pool->head_dim != packed->head_dim)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (pool->num_slots > 0x7FFFFFFF)
        return KAMERA_ERR_UNSUPPORTED;
    if (n == 0)
        return KAMERA_OK;
    if (!kv_pages || !packed_pages || !tokens || !packed->data)
        return KAMERA_ERR_INVALID_ARGUMENT;
    const int H = pool->num_kv_heads, d = pool->head_dim;
    int e;
    if ((e = check_strided(pool->k, pool->num_layers, pool->layer_stride, pool->num_slots, pool->slot_stride,
                           (int64_t)H * d, false)) ||
        (e = check_strided(pool->v, pool->num_layers, pool->layer_stride, pool->num_slots, pool->slot_stride,
                           (int64_t)H * d, false)))
        return e;
    if (!aligned16(packed->data) ||
        ((reinterpret_cast<uintptr_t>(kv_pages) | reinterpret_cast<uintptr_t>(packed_pages) |
          reinterpret_cast<uintptr_t>(tokens)) & 3))
        return KAMERA_ERR_MISALIGNED;
    const auto ks = span(pool->k, pool->num_layers, pool->layer_stride, pool->num_slots, pool->slot_stride, (int64_t)H * d);
    const auto vs = span(pool->v, pool->num_layers, pool->layer_stride, pool->num_slots, pool->slot_stride, (int64_t)H * d);
    const uintptr_t at = reinterpret_cast<uintptr_t>(packed->data);
    const std::pair<uintptr_t, uintptr_t> ps{at, at + (uintptr_t)packed_bytes(packed)};
    auto ints = [n](const int32_t* a) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(a);
        return std::pair<uintptr_t, uintptr_t>{lo, lo + (uintptr_t)n * 4};
    };
    if (overlap(ks, ps) || overlap(vs, ps) || overlap(ks, vs))
        return KAMERA_ERR_INVALID_ARGUMENT;
    for (const int32_t* a : {kv_pages, packed_pages, tokens})
        if (pack ? overlap(ints(a), ps) : overlap(ints(a), ks) || overlap(ints(a), vs))
            return KAMERA_ERR_INVALID_ARGUMENT;
    PackParams p;
    std::memset(&p, 0, sizeof(p));
    p.k = static_cast<__nv_bfloat16*>(pool->k) + layer * (pool->num_layers > 1 ? pool->layer_stride : 0);
    p.v = static_cast<__nv_bfloat16*>(pool->v) + layer * (pool->num_layers > 1 ? pool->layer_stride : 0);
    p.data = static_cast<unsigned char*>(packed->data);
    p.kv_pages = kv_pages;
    p.packed_pages = packed_pages;
    p.tokens = tokens;
    p.slot_stride = pool->slot_stride;
    p.P = packed->page_size;
    p.kv_pages_n = pool->num_slots / p.P;
    p.packed_pages_n = packed->num_pages;
    p.H = H;
    p.pieces = p.P / 16;
    p.items = (int64_t)n * p.pieces * H;
    p.k_unit = packed->k_unit;
    p.v_unit = packed->v_unit;
    p.err = d_err;
    const int64_t blocks = (p.items + kPkWarps - 1) / kPkWarps;
    if (blocks > 0x7FFFFFFF)
        return KAMERA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks);
    cudaError_t err;
    if (pack)
        err = d == 128 ? launch_after(pack_kernel<128>, grid, 32 * kPkWarps, 0, stream, true, p)
                       : launch_after(pack_kernel<64>, grid, 32 * kPkWarps, 0, stream, true, p);
    else
        err = d == 128 ? launch_after(unpack_kernel<128>, grid, 32 * kPkWarps, 0, stream, true, p)
                       : launch_after(unpack_kernel<64>, grid, 32 * kPkWarps, 0, stream, true, p);
    return err == cudaSuccess ? KAMERA_OK : KAMERA_ERR_CUDA;
}

}  // namespace

}  // namespace kamera

using namespace kamera;

extern "C" {

int kamera_pack_pages(const KameraGqaPool* pool, int32_t layer, const KameraPackedPool* packed, const int32_t* d_kv_pages,
                      const int32_t* d_packed_pages, const int32_t* d_tokens, int32_t n, int32_t* d_err,
                      struct CUstream_st* stream)
{
    return convert(pool, layer, packed, d_kv_pages, d_packed_pages, d_tokens, n, d_err,
                   reinterpret_cast<cudaStream_t>(stream), true);
}

int kamera_unpack_pages(const KameraGqaPool* pool, int32_t layer, const KameraPackedPool* packed,
                        const int32_t* d_kv_pages, const int32_t* d_packed_pages, const int32_t* d_tokens, int32_t n,
                        int32_t* d_err, struct CUstream_st* stream)
{
    return convert(pool, layer, packed, d_kv_pages, d_packed_pages, d_tokens, n, d_err,
                   reinterpret_cast<cudaStream_t>(stream), false);
}

}  // extern "C"
