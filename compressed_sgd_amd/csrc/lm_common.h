// lm_common.h -- internals shared by the language-model operators
// (layer_norm.hip, token_logprobs.hip, distill.hip).
#pragma once

#include <cmath>

#include "sgc_common.h"

namespace sgc {

inline bool lm_dtype(int32_t t) { return t == SGC_F32 || t == SGC_BF16 || t == SGC_F16; }
inline int64_t lm_size(int32_t t) { return t == SGC_F32 ? 4 : 2; }
inline bool lm_aligned(const void* p, int64_t a) { return ((uintptr_t)p & (uintptr_t)(a - 1)) == 0; }

// rows x len elements at `stride`: an input may repeat one row (stride 0),
// an output's rows lie apart.
inline bool lm_rows_ok(const void* p, int64_t stride, int64_t rows, int64_t len, int32_t dtype, bool out)
{
    if (!p || !lm_aligned(p, lm_size(dtype)) || stride < 0) return false;
    return rows <= 1 || stride >= len || (!out && stride == 0);
}

// ------------------------------------------------------------ element types
typedef __bf16 bf16_t;
typedef _Float16 f16_t;

// V consecutive elements, loaded and stored in one access at the element's
// own alignment: rows of an odd length start at any element, and the
// hardware takes a 16-byte access at any 2-byte address.
template <typename T, int V>
struct __attribute__((packed, aligned(sizeof(T)))) Pack {
    T v[V];
};

template <typename T>
__device__ inline float to_f(T x) { return (float)x; }
// one rounding, to nearest even
template <typename T>
__device__ inline T from_f(float x) { return (T)x; }

template <typename T>
struct VecLen {
    static constexpr int value = 16 / (int)sizeof(T);
};

// 16 bytes of a row as four words, which stay packed in registers, and their
// elements as fp32.
struct __attribute__((packed, aligned(2))) Raw {
    uint32_t w[4];
};
// Accesses of data that passes once (ONCE) go past the caches: a bare copy of 1
// GiB in rows of 256 KB runs at 5.9 TB/s with both of them so, 4.6 with
// neither.  A call takes them where what it reads and writes is more than the
// last-level cache holds; below that the next call finds its input there (a
// layer norm backward of 156 MB: 40.1 us without, 40.9 with; the gradients of
// 2048 x 50000 logits, 410 MB: 66 without, 47 with).
constexpr int64_t kCacheBytes = (int64_t)256 << 20;
typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));
template <bool ONCE>
__device__ inline Raw load_row(const Raw* p)
{
    if (!ONCE) return *p;
    const Words w = __builtin_nontemporal_load((const Words*)p);
    return {{w.x, w.y, w.z, w.w}};
}
template <bool ONCE>
__device__ inline void store_row(Raw* p, const Raw& q)
{
    const Words w = {q.w[0], q.w[1], q.w[2], q.w[3]};
    if (ONCE)
        __builtin_nontemporal_store(w, (Words*)p);
    else
        *p = q;
}
template <typename T>
__device__ inline void unpack(const Raw& q, float* x)
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(q.w[i]);
    } else if constexpr (__is_same(T, bf16_t)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(q.w[i] << 16);
            x[2 * i + 1] = __uint_as_float(q.w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = (float)__builtin_bit_cast(f16_t, (uint16_t)q.w[i]);
            x[2 * i + 1] = (float)__builtin_bit_cast(f16_t, (uint16_t)(q.w[i] >> 16));
        }
    }
}
template <typename T>
__device__ inline Raw pack(const float* x)
{
    Raw q;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q.w[i] = __float_as_uint(x[i]);
    } else {
        typedef T Two __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            Two t = {from_f<T>(x[2 * i]), from_f<T>(x[2 * i + 1])};
            q.w[i] = __builtin_bit_cast(uint32_t, t);
        }
    }
    return q;
}
// -inf in every element.
template <typename T>
__device__ inline Raw raw_low()
{
    const uint32_t w = sizeof(T) == 4 ? 0xff800000u : __is_same(T, bf16_t) ? 0xff80ff80u : 0xfc00fc00u;
    return {{w, w, w, w}};
}

// One workgroup for each of n < 2^31 rows: a grid of at most 2^20 x 2^11
// (a launch holds fewer than 2^32 threads in x); the last ones past n.
inline dim3 row_grid(int64_t n)
{
    const int64_t gx = n < ((int64_t)1 << 20) ? n : (int64_t)1 << 20;
    return dim3((unsigned)gx, (unsigned)cdiv(n, gx));
}
__device__ inline int64_t row_of_block() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// ------------------------------------------------------- block reductions
// Over a wave by data-parallel moves inside the vector unit (shifts in rows of
// 16 lanes, then rows 0 and 2 into 1 and 3, then the lower half into the
// upper): lane 63 has seen every lane.  No trip through shared memory, which
// a shuffle makes.  The steps' lanes without a source add 0, or keep their own.
template <int CTRL, int ROWS>
__device__ inline float dpp_or(float old, float x)
{
    return __int_as_float(
        __builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(x), CTRL, ROWS, 0xf, false));
}
__device__ inline float last_lane(float x) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63)); }

// A value that is the same in all lanes, in a scalar register.
__device__ inline float in_scalar(float x)
{
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
}

// Every lane of the wave must be active.
__device__ inline float wave_sum(float x)
{
    x += dpp_or<0x111, 0xf>(0.f, x);
    x += dpp_or<0x112, 0xf>(0.f, x);
    x += dpp_or<0x114, 0xf>(0.f, x);
    x += dpp_or<0x118, 0xf>(0.f, x);
    x += dpp_or<0x142, 0xa>(0.f, x);
    x += dpp_or<0x143, 0xc>(0.f, x);
    return last_lane(x);
}
__device__ inline float wave_max(float x)
{
    x = fmaxf(x, dpp_or<0x111, 0xf>(x, x));
    x = fmaxf(x, dpp_or<0x112, 0xf>(x, x));
    x = fmaxf(x, dpp_or<0x114, 0xf>(x, x));
    x = fmaxf(x, dpp_or<0x118, 0xf>(x, x));
    x = fmaxf(x, dpp_or<0x142, 0xa>(x, x));
    x = fmaxf(x, dpp_or<0x143, 0xc>(x, x));
    return last_lane(x);
}

// The sum of N values (a power of two up to 16) of which lane l holds number
// l mod N: rotations in rows of 16 lanes.
template <int N>
__device__ inline float sum_of_lanes(float x)
{
    if (N > 8) x += dpp_or<0x128, 0xf>(0.f, x);
    if (N > 4) x += dpp_or<0x124, 0xf>(0.f, x);
    if (N > 2) x += dpp_or<0x122, 0xf>(0.f, x);
    if (N > 1) x += dpp_or<0x121, 0xf>(0.f, x);
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
}

// The sum over each row of 16 lanes, the same bits in all of them.
__device__ inline float row16_sum(float x)
{
    x += dpp_or<0x128, 0xf>(0.f, x);
    x += dpp_or<0x124, 0xf>(0.f, x);
    x += dpp_or<0x122, 0xf>(0.f, x);
    x += dpp_or<0x121, 0xf>(0.f, x);
    return x;
}
template <int N>
__device__ inline float max_of_lanes(float x)
{
    if (N > 8) x = fmaxf(x, dpp_or<0x128, 0xf>(x, x));
    if (N > 4) x = fmaxf(x, dpp_or<0x124, 0xf>(x, x));
    if (N > 2) x = fmaxf(x, dpp_or<0x122, 0xf>(x, x));
    if (N > 1) x = fmaxf(x, dpp_or<0x121, 0xf>(x, x));
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
}

// Sum over a workgroup of NW waves, the same value in every thread; tmp
// holds NW floats and is free again after the call.
template <int NW>
__device__ inline float block_sum(float x, float* tmp)
{
    x = wave_sum(x);
    if (NW == 1) return x;
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = x;
    __syncthreads();
    const float r = sum_of_lanes<NW>(tmp[threadIdx.x % NW]);
    __syncthreads();
    return r;
}
template <int NW>
__device__ inline float block_max(float x, float* tmp)
{
    x = wave_max(x);
    if (NW == 1) return x;
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = x;
    __syncthreads();
    const float r = max_of_lanes<NW>(tmp[threadIdx.x % NW]);
    __syncthreads();
    return r;
}
// Two at once; tmp holds 2 NW floats.
template <int NW>
__device__ inline void block_sums(float& x, float& y, float* tmp)
{
    x = wave_sum(x);
    y = wave_sum(y);
    if (NW == 1) return;
    if ((threadIdx.x & 63) == 0) {
        tmp[threadIdx.x >> 6] = x;
        tmp[NW + (threadIdx.x >> 6)] = y;
    }
    __syncthreads();
    x = sum_of_lanes<NW>(tmp[threadIdx.x % NW]);
    y = sum_of_lanes<NW>(tmp[NW + threadIdx.x % NW]);
    __syncthreads();
}
template <int NW>
__device__ inline void block_maxima(float& x, float& y, float* tmp)
{
    x = wave_max(x);
    y = wave_max(y);
    if (NW == 1) return;
    if ((threadIdx.x & 63) == 0) {
        tmp[threadIdx.x >> 6] = x;
        tmp[NW + (threadIdx.x >> 6)] = y;
    }
    __syncthreads();
    x = max_of_lanes<NW>(tmp[threadIdx.x % NW]);
    y = max_of_lanes<NW>(tmp[NW + threadIdx.x % NW]);
    __syncthreads();
}

// Order of values as unsigned integers: -inf lowest, both zeros alike, NaN
// (either sign) above +inf.
__device__ inline uint32_t order_key(float x)
{
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
// The same with the place as second key: among equals the lower one is
// larger.  Unique within a row.
__device__ inline uint64_t order_key(float x, uint32_t at) { return ((uint64_t)order_key(x) << 32) | (uint32_t)~at; }

}  // namespace sgc
