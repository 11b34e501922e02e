// lm_q8.h -- 8 bits with scales, shared by rms_norm.hip, q8.hip and norm_q8.hip.
//
// With a the largest magnitude of a group: q = rint(x r), r = 127 / a, each
// rounded to fp32, so a host with fp32 finds the same whole numbers.  |x r| is
// at most 127 (1 + 2^-23): nothing has to be clamped.
#pragma once

#include "lm_norm.h"

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

// ---------------------------------------------------- reductions of magnitudes
template <int CTRL, int ROWS>
__device__ inline uint32_t dpp_own(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, CTRL, ROWS, 0xf, false);
}
// Over a wave; every lane must be active.
__device__ inline uint32_t wave_umax(uint32_t x)
{
    x = umax(x, dpp_own<0x111, 0xf>(x));
    x = umax(x, dpp_own<0x112, 0xf>(x));
    x = umax(x, dpp_own<0x114, 0xf>(x));
    x = umax(x, dpp_own<0x118, 0xf>(x));
    x = umax(x, dpp_own<0x142, 0xa>(x));
    x = umax(x, dpp_own<0x143, 0xc>(x));
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}
// Over the N lanes (a power of two up to 16) that hold lane mod N alike.
template <int N>
__device__ inline uint32_t lanes_umax(uint32_t x)
{
    if (N > 8) x = umax(x, dpp_own<0x128, 0xf>(x));
    if (N > 4) x = umax(x, dpp_own<0x124, 0xf>(x));
    if (N > 2) x = umax(x, dpp_own<0x122, 0xf>(x));
    if (N > 1) x = umax(x, dpp_own<0x121, 0xf>(x));
    return x;
}

// ------------------------------------------------------------ rows of bytes
// V bytes, loaded and stored in one access at any address.
template <int V>
struct __attribute__((packed, aligned(1))) Bytes {
    uint32_t w[V / 4];
};
template <int V, bool RAG>
__device__ inline void store_bytes(int8_t* p, int v, int cols, const Bytes<V>& b)
{
    if ((v + 1) * V <= cols) {
        *(Bytes<V>*)(p + v * V) = b;
    } else if (RAG && v * V < cols) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (v * V + e < cols) p[v * V + e] = (int8_t)(b.w[e / 4] >> (e % 4 * 8));
    }
}
// Past the end of the row 0.
template <int V, bool RAG>
__device__ inline Bytes<V> load_bytes(const int8_t* p, int v, int cols)
{
    if ((v + 1) * V <= cols) return *(const Bytes<V>*)(p + v * V);
    Bytes<V> b = {};
    if (RAG && v * V < cols) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (v * V + e < cols) b.w[e / 4] |= (uint32_t)(uint8_t)p[v * V + e] << (e % 4 * 8);
    }
    return b;
}
__device__ inline float byte_of(uint32_t w, int e) { return (float)(int8_t)(w >> (e * 8)); }

// load_raw with the choice of cache at run time.
template <typename T, bool RAG>
__device__ inline Raw load_vec(const T* p, int v, int cols, bool once)
{
    return once ? load_raw<T, RAG, true>(p, v, cols) : load_raw<T, RAG, false>(p, v, cols);
}
template <typename T, bool RAG>
__device__ inline void store_vec(T* p, int v, int cols, const float* x, bool once)
{
    if (once) store_raw<T, RAG, true>(p, v, cols, x);
    else store_raw<T, RAG, false>(p, v, cols, x);
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
