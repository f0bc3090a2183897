// kamera_hostcheck.h -- argument checks shared by the C entry points (host side).
#pragma once

#include <cmath>
#include <cstdint>
#include <utility>

#include "kamera.h"

namespace kamera {

struct RopeParams;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Byte range [lo, hi) spanned by a strided [L][rows][width] bf16 array.
inline std::pair<uintptr_t, uintptr_t> span(const void* base, int64_t L, int64_t ls, int64_t rows, int64_t rs,
                                     int64_t width)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(base);
    if (L <= 0 || rows <= 0)
        return {lo, lo};
    const int64_t last = (L - 1) * ls + (rows - 1) * rs + width;
    return {lo, lo + static_cast<uintptr_t>(last) * 2u};
}

inline bool overlap(std::pair<uintptr_t, uintptr_t> a, std::pair<uintptr_t, uintptr_t> b)
{
    return a.first < b.second && b.first < a.second;
}

inline int check_strided(const void* base, int64_t L, int64_t ls, int64_t rows, int64_t rs, int64_t width,
                  bool need_rows)
{
    if (!base)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (!aligned16(base) || (ls & 7) || (rs & 7))
        return KAMERA_ERR_MISALIGNED;
    if (rows < 0 || (need_rows && rows < 1) || rs < width || ls < 0)
        return KAMERA_ERR_INVALID_ARGUMENT;
    if (L > 1 && ls < rows * rs)
        return KAMERA_ERR_INVALID_ARGUMENT;
    return KAMERA_OK;
}

// theta / (2 pi) modulo 1, in units of 2^-64 (theta finite): the quotient as a
// double-double, whose integer part drops out of a phase.  The fraction is taken
// of |theta|, where it is exact (x - floor(x) is not for x in (-1, 0)), and negated
// modulo a turn.
inline uint64_t turn_fraction(double theta)
{
    const double inv_hi = 0.15915494309189535, inv_lo = -9.839338337591243e-18;   // 1 / (2 pi)
    const double t = std::fabs(theta), hi = t * inv_hi;
    const double lo = std::fma(t, inv_hi, -hi) + t * inv_lo;
    const double f = (hi - std::floor(hi)) * 18446744073709551616.0;   // in [0, 2^64): exact
    const double whole = std::floor(f);
    const double rest = (f - whole) + lo * 18446744073709551616.0;
    // (a quotient past 2^51 has no fraction worth the name)
    const uint64_t r = std::fabs(rest) < 4.0e18 ? (uint64_t)(int64_t)std::llrint(rest) : 0;
    const uint64_t x = (uint64_t)whole + r;
    return theta < 0.0 ? 0ull - x : x;
}

// KameraRope -> RopeParams (defined with the relocation entry points): the
// frequency table and axis map of a call; `width` is the extent the rotary
// range must fit in.
int fill_rope(const KameraRope* r, int width, RopeParams* out);

}  // namespace kamera
