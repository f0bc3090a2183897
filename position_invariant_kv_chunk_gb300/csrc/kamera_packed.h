// kamera_packed.h -- the 4-bit pages' layout, shared by the kernels that write them
// (kamera_pack.cu) and the one that attends over them (kamera_packed.cu).
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kamera.h"

namespace kamera {

// 16 tokens of a head: bytes, and where its parts start.
template <int D>
constexpr int kPackedPiece = 18 * D;
template <int D>
constexpr int kPackedV = 8 * D;        // value codes (key codes at 0)
template <int D>
constexpr int kPackedKS = 16 * D;      // key scales
template <int D>
constexpr int kPackedVS = 17 * D;      // value scales

// The value of an e4m3 byte without a sign (0x7F, its NaN, does not occur): its
// exponent and fraction are those of an fp16 number 2^8 smaller.
__device__ __forceinline__ float e4m3_to_float(uint32_t byte)
{
    return __half2float(__ushort_as_half((unsigned short)(byte << 7))) * 256.f;
}

// A byte of two e2m1 codes to its fp16 values, byte B of w.
template <int B>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t w)
{
    uint32_t r;
    if constexpr (B == 0)
        asm("{\n\t.reg .b8 a,b,c,d;\n\tmov.b32 {a,b,c,d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (B == 1)
        asm("{\n\t.reg .b8 a,b,c,d;\n\tmov.b32 {a,b,c,d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (B == 2)
        asm("{\n\t.reg .b8 a,b,c,d;\n\tmov.b32 {a,b,c,d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b8 a,b,c,d;\n\tmov.b32 {a,b,c,d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// What both sides check of a packed pool (host).
inline int check_packed(const KameraPackedPool* p)
{
    if (!p || p->reserved != 0 || p->num_pages < 0 || p->num_kv_heads < 1 || p->head_dim < 1 || p->page_size < 1)
        return KAMERA_ERR_INVALID_ARGUMENT;
    for (float u : {p->k_unit, p->v_unit}) {
        int e;
        if (!(u > 0.f) || std::frexp(u, &e) != 0.5f || e < -63 || e > 65)
            return KAMERA_ERR_INVALID_ARGUMENT;
    }
    if ((p->head_dim != 64 && p->head_dim != 128) || p->page_size % 16 || p->page_size > (1 << 20) ||
        p->num_pages > 0x7FFFFFFF || p->num_kv_heads > 65535)
        return KAMERA_ERR_UNSUPPORTED;
    return KAMERA_OK;
}

inline int64_t packed_bytes(const KameraPackedPool* p)
{
    return p->num_pages * p->num_kv_heads * (int64_t)p->page_size * (p->head_dim + p->head_dim / 8);
}

}  // namespace kamera
