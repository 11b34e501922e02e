// lm_q8.h -- 8 bits with scales, shared by rms_norm.hip, q8.hip and norm_q8.hip.
//
// With a the largest magnitude of a group: q = rint(x r), r = 127 / a, each
// rounded to fp32, so a host with fp32 finds the same whole numbers.  |x r| is
// at most 127 (1 + 2^-23): nothing has to be clamped.
#pragma once

#include "lm_common.h"

namespace sgc {

// Magnitudes are compared as unsigned integers: NaN above infinity above all else.
__device__ inline uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ inline uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
constexpr uint32_t kInfinity = 0x7f800000u;

struct Quant {
    float pre;      // 2^100 where 127 / a would pass fp32's range, else 1
    float factor;   // 127 / a
    uint32_t keep;  // 0 where the group's q are 0
    float scale;    // a / 127; NaN where something is not finite
};
__device__ inline Quant quant_of(uint32_t top)
{
    const float a = __uint_as_float(top);
    Quant k;
    k.pre = a < 0x1p-100f ? 0x1p100f : 1.f;
    const bool fine = top < kInfinity;
    k.keep = fine && top ? 0xffffffffu : 0u;
    k.factor = k.keep ? 127.f / (a * k.pre) : 0.f;
    k.scale = fine ? a / 127.f : __uint_as_float(0x7fc00000u);
    return k;
}
// The whole number in the low byte: adding 1.5 x 2^23 rounds x r to the nearest
// whole number, ties to even, as rint does.
__device__ inline uint32_t quantized(float x, const Quant& k)
{
    return __float_as_uint((x * k.pre) * k.factor + 12582912.f);
}
__device__ inline uint32_t four_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), hi = __builtin_amdgcn_perm(d, c, 0x0c0c0400u);
    return lo | (hi << 16);
}

inline bool q8_group_ok(int32_t g) { return g == 0 || g == 32 || g == 64 || g == 128 || g == 256; }
inline int64_t q8_groups(int64_t cols, int32_t g) { return g ? cdiv(cols, g) : 1; }
// c >> q8_shift(g) is the group of column c < 2^20.
inline int q8_shift(int32_t g) { return g ? __builtin_ctz((unsigned)g) : 30; }
inline bool q8_rows_ok(const void* p, int64_t stride, int64_t rows, int64_t len, bool out)
{
    return p && stride >= 0 && (rows <= 1 || stride >= len || (!out && stride == 0));
}

}  // namespace sgc
