// kamera_tc.cuh -- helpers shared by the attention kernels on the 5th-generation
// tensor cores (sm_103a): TMEM loads and stores of a warp's rows, MMA issue with
// descriptors whose low word is computed by one add, and the drain wait.
#pragma once

#include <cstdint>

#include "kamera_ptx.cuh"

namespace kamera {
namespace tc {

__device__ __forceinline__ void tmem_ld32(uint32_t ta, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(ta)
        : "memory");
}

// The same without the wait: the registers hold the values after tmem_ld_wait128.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t ta, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(ta)
        : "memory");
}

// Waits for every TMEM load this thread issued; the four blocks pass through so
// the compiler reads none of them before.
__device__ __forceinline__ void tmem_ld_wait128(uint32_t (&s)[4][32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 32; j += 8)
            asm volatile("" : "+r"(s[c][j]), "+r"(s[c][j + 1]), "+r"(s[c][j + 2]), "+r"(s[c][j + 3]), "+r"(s[c][j + 4]),
                         "+r"(s[c][j + 5]), "+r"(s[c][j + 6]), "+r"(s[c][j + 7]));
}

__device__ __forceinline__ void tmem_st32(uint32_t ta, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(ta),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
        "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
        "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t ta, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(ta),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st4(uint32_t ta, const uint32_t (&r)[4])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(ta), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16-byte piece c of row r of a 128B-swizzled tile of 128-byte rows (the TMA
// and MMA layout): piece c ^ (r & 7).
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// One lane of the (converged) warp: the compiler knows that a branch on it holds a single
// thread, and hands an MMA its operands without a loop over the lanes that might differ
// (which cost 35 of 100 cycles an MMA in a branch on lane 0).
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// Waits for a phase whatever the abort flag says: the drain of copies and MMAs that a CTA
// started, before it leaves.  Up to 1 s, whatever bound the call's other waits have: one
// that is shorter than a load would let the CTA go with copies on their way into shared
// memory that its successor owns.  False: given up.
__device__ __forceinline__ bool pf_drain_wait(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(bar, parity))
        if (ptx::globaltimer() - t0 > 1000000000ull)
            return false;
    return true;
}

// The last `ring` of `n` fills of a ring of barriers (fill k: barrier k % ring), waited for.
__device__ __forceinline__ void pf_drain_ring(const uint64_t* bars, uint32_t n, uint32_t ring)
{
    for (uint32_t k = n > ring ? n - ring : 0u; k < n; ++k)
        if (!pf_drain_wait(ptx::smem_addr(&bars[k % ring]), (k / ring) & 1u))
            return;
}

// Shared-memory matrix descriptors as (low word, high word): the low word holds
// the start address (bytes >> 4) and the leading byte offset, so a step inside
// an operand is one 32-bit add.  High word: stride byte offset 1024 (8-row
// groups), descriptor version 1, 128-byte swizzle.  A K-major operand (the key
// and U rows) ignores the leading offset; for an MN-major one (the value and U'
// rows: the rows of a TMA box are K, the N dimension is contiguous) it is the
// distance between 64-element atoms along N.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
template <uint32_t HI = kDescHi>
__device__ __forceinline__ uint64_t pf_desc(uint32_t lo)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(HI));
    return d;
}

// D[tmem] (+)= A[tmem] * B[smem]^T (kind::f16: bf16 in, fp32 accumulate), the
// accumulate flag a compile-time constant.  A's row r sits in TMEM lane r,
// elements 2c and 2c + 1 in the low and high half of column c.
template <bool ACC, uint32_t HI = kDescHi>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc)
{
    if constexpr (ACC)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, 1, 1;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
                     "r"(a_tmem), "l"(pf_desc<HI>(b_lo)), "r"(idesc)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, 1, 1;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
                     "r"(a_tmem), "l"(pf_desc<HI>(b_lo)), "r"(idesc)
                     : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T (kind::f16), accumulate flag constant.
template <bool ACC, uint32_t HI = kDescHi>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc)
{
    if constexpr (ACC)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, 1, 1;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                     "l"(pf_desc<HI>(a_lo)), "l"(pf_desc<HI>(b_lo)), "r"(idesc)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, 1, 1;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                     "l"(pf_desc<HI>(a_lo)), "l"(pf_desc<HI>(b_lo)), "r"(idesc)
                     : "memory");
}

// The same with a descriptor high word for each operand.
template <bool ACC, uint32_t HA, uint32_t HB>
__device__ __forceinline__ void mma_ss2(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc)
{
    if constexpr (ACC)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, 1, 1;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                     "l"(pf_desc<HA>(a_lo)), "l"(pf_desc<HB>(b_lo)), "r"(idesc)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, 1, 1;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                     "l"(pf_desc<HA>(a_lo)), "l"(pf_desc<HB>(b_lo)), "r"(idesc)
                     : "memory");
}

// 2^x (the MUFU approximation: relative error near 2^-22, subnormal results
// flushed to zero).
__device__ __forceinline__ float pf_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace tc
}  // namespace kamera
