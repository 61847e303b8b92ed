// The int8 rule, of rows and of weight columns: a scale for all of a row (column) and the nearest codes.
#pragma once

#include "common.hpp"

namespace moe {
namespace {

// Bits of the largest |v| as an unsigned number: ordered as the values are, with infinity and NaN above them all.
constexpr uint32_t kInfBits = 0x7F800000u;
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
// scale = amax / 127, at least the smallest normal number (a row that is all zeros, or smaller still, has no use for
// its digits, and 1 / scale stays finite).  A row with an infinity or NaN has the scale NaN and zeros for codes, so
// that its products are NaN.
__device__ __forceinline__ float int8_scale(uint32_t most) {
    return most >= kInfBits ? __uint_as_float(0x7FC00000u) : fmaxf(__uint_as_float(most) / 127.0f, 0x1p-126f);
}

// The integer nearest to v / scale, ties to even.  r from the rounded product v * inv is off by one at most, next to
// a half only; the remainder v - r scale decides there.  It is exact where it is compared: |r| >= 1 makes v at
// least scale / 2, so v and r scale are multiples of 2^-24 times the remainder's binade (below scale / 2 a remainder
// may round onto -scale / 2, whose tie goes to the even 0, as it must).
__device__ __forceinline__ float int8_nearest(float v, float scale, float inv) {
    float r = __builtin_rintf(v * inv);
    const float rest = fmaf(-r, scale, v), half = 0.5f * scale;
    const bool odd = (static_cast<int>(r) & 1) != 0;
    if (rest > half || (rest == half && odd)) r += 1.0f;
    else if (rest < -half || (rest == -half && odd)) r -= 1.0f;
    return r;
}

__device__ __forceinline__ int int8_code(float v, float scale, float inv) {
    return static_cast<int>(fminf(fmaxf(int8_nearest(v, scale, inv), -127.0f), 127.0f));
}

}  // namespace
}  // namespace moe
