// lm_q8.h -- 8 bits with scales, ends of ragged rows, rows in registers: shared by
// rms_norm.hip, q8.hip, norm_q8.hip and int8_linear.hip.
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

// The largest magnitude over a workgroup of NW waves, in every thread.
template <int NW>
__device__ inline uint32_t block_umax(uint32_t x, uint32_t* tmp)
{
    x = wave_umax(x);
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = x;
    __syncthreads();
    x = (uint32_t)__builtin_amdgcn_readfirstlane((int)lanes_umax<NW>(tmp[threadIdx.x % NW]));
    __syncthreads();
    return x;
}

// ------------------------------------------------------ ends of ragged rows
// Four words (or two, or one) without their first `drop` bytes, zeros behind.
__device__ inline void drop_bytes(uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d, int drop)
{
    if (drop & 8) a = c, b = d, c = 0, d = 0;
    if (drop & 4) a = b, b = c, c = d, d = 0;
    a = __builtin_amdgcn_alignbyte(b, a, drop & 3);
    b = __builtin_amdgcn_alignbyte(c, b, drop & 3);
    c = __builtin_amdgcn_alignbyte(d, c, drop & 3);
    d = __builtin_amdgcn_alignbyte(0u, d, drop & 3);
}
__device__ inline void drop_bytes(uint32_t& a, uint32_t& b, int drop)
{
    if (drop & 4) a = b, b = 0;
    a = __builtin_amdgcn_alignbyte(b, a, drop & 3);
    b = __builtin_amdgcn_alignbyte(0u, b, drop & 3);
}
__device__ inline void drop_bytes(uint32_t& a, int drop) { a = __builtin_amdgcn_alignbyte(0u, a, drop & 3); }

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
        const int rest = cols - v * V;
        int8_t* at = p + v * V;
        uint32_t w = b.w[0];
        if (V > 4 && (rest & 4)) {
            *(Bytes<4>*)at = {{w}};
            at += 4;
            w = b.w[V / 4 - 1];
        }
        if (rest & 2) {
            typedef uint16_t Two __attribute__((aligned(1)));
            *(Two*)at = (uint16_t)w;
            at += 2;
            w >>= 16;
        }
        if (rest & 1) *at = (int8_t)w;
    }
}
// The end of a ragged row is read with what lies before it, in one access (rows
// shorter than that byte by byte), and `settled` where the values are used: the
// load is waited for there, not where it was issued.  Past the end 0.
template <int V, bool RAG>
__device__ inline Bytes<V> load_bytes(const int8_t* p, int v, int cols)
{
    if (!RAG) return (v + 1) * V <= cols ? *(const Bytes<V>*)(p + v * V) : Bytes<V>{};
    Bytes<V> b = {};
    if (cols >= V) {
        if (v * V < cols) {
            const int over = (v + 1) * V - cols;
            b = *(const Bytes<V>*)(p + v * V - (over > 0 ? over : 0));
        }
        return b;
    }
    if (v == 0) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < cols) b.w[e / 4] |= (uint32_t)(uint8_t)p[e] << (e % 4 * 8);
    }
    return b;
}
template <int V, bool RAG>
__device__ inline void settle(Bytes<V>& b, int v, int cols)
{
    const int over = (v + 1) * V - cols;
    if (!RAG || over <= 0 || over >= V || cols < V) return;
    if constexpr (V == 4) {
        uint32_t w0 = b.w[0];
        drop_bytes(w0, over);
        b = {{w0}};
    } else {
        uint32_t w0 = b.w[0], w1 = b.w[1];
        drop_bytes(w0, w1, over);
        b = {{w0, w1}};
    }
}
__device__ inline float byte_of(uint32_t w, int e) { return (float)(int8_t)(w >> (e * 8)); }

// A row's vectors of elements the same way; `once` as ONCE of load_row.
template <typename T, bool RAG>
__device__ inline Raw load_vec(const T* p, int v, int cols, bool once)
{
    constexpr int VL = VecLen<T>::value;
    Raw q = {};
    if (RAG && cols < VL) {
        if (v == 0) {
#pragma unroll
            for (int e = 0; e < VL; ++e)
                if (e < cols) {
                    if constexpr (sizeof(T) == 4) q.w[e] = __builtin_bit_cast(uint32_t, p[e]);
                    else q.w[e / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[e]) << (e % 2 * 16);
                }
        }
    } else if (v * VL < cols) {
        const int over = RAG ? (v + 1) * VL - cols : 0;
        const Raw* at = (const Raw*)(p + v * VL - (RAG && over > 0 ? over : 0));
        q = once ? load_row<true>(at) : load_row<false>(at);
    }
    return q;
}
template <typename T, bool RAG>
__device__ inline void settle(Raw& q, int v, int cols)
{
    constexpr int VL = VecLen<T>::value;
    const int over = (v + 1) * VL - cols;
    if (!RAG || over <= 0 || over >= VL || cols < VL) return;
    uint32_t w0 = q.w[0], w1 = q.w[1], w2 = q.w[2], w3 = q.w[3];
    drop_bytes(w0, w1, w2, w3, over * (int)sizeof(T));
    q = {{w0, w1, w2, w3}};
}
template <typename T, bool RAG>
__device__ inline void store_vec(T* p, int v, int cols, const float* x, bool once)
{
    constexpr int VL = VecLen<T>::value;
    if ((v + 1) * VL <= cols) {
        if (once) store_row<true>((Raw*)p + v, pack<T>(x));
        else store_row<false>((Raw*)p + v, pack<T>(x));
    } else if (RAG && v * VL < cols) {
        // the end of the row in pieces of 8, 4 and 2 bytes
        Raw q = pack<T>(x);
        const int rest = (cols - v * VL) * (int)sizeof(T);
        char* at = (char*)(p + v * VL);
        uint32_t w0 = q.w[0], w1 = q.w[1];
        if (rest & 8) {
            *(Bytes<8>*)at = {{w0, w1}};
            at += 8;
            w0 = q.w[2];
            w1 = q.w[3];
        }
        if (rest & 4) {
            *(Bytes<4>*)at = {{w0}};
            at += 4;
            w0 = w1;
        }
        if (sizeof(T) == 2 && (rest & 2)) *(uint16_t*)at = (uint16_t)w0;
    }
}

// ----------------------------------------------------- rows in registers
// How a workgroup's threads share rows: 16 or 32 lanes a row (LANES), or
// `waves` whole ones (LANES 64), `rows` rows side by side.
struct RowShape {
    int lanes, ept, waves, rows;
    int threads() const { return lanes < 64 ? 512 : 64 * waves * rows; }
};
// Workgroups that share out the rows: `waves` waves a compute unit to the nearest
// whole workgroup, the same number on each.  That may be one more than a kernel's
// registers leave room for, which then runs after the others; which number is best
// differs.  As here, and rounded down (forward from 28 waves where rows are ragged,
// what their registers allow in 16 bits): forward 10922 x 6144 bf16 92.5 and 91.6
// us, 16384 x 4099 140 and 144, 46153 x 1300 105 and 106, into 8 bits 16384 x 4099
// 131 and 111, 46153 x 1300 93 and 96; backward 10922 x 6144 91 and 91, 16384 x 4099
// 137 and 132, 46153 x 1300 114 and 90, 13000 x 5120 fp32 182 and 175, layer norm
// from 8 bits 16384 x 4099 bf16 175 and 171.
inline int64_t row_groups(const RowShape& sh, int64_t rows, int waves)
{
    const int each = (waves * 64 + sh.threads() / 2) / sh.threads();
    const int64_t need = cdiv(rows, sh.rows), most = kCus * (each > 1 ? each : 1);
    return need < most ? need : most;
}
template <int LANES>
struct RowPlace {
    int sub, t, across;  // the row among the workgroup's, the thread within it, threads of a row
    __device__ RowPlace(int waves)
    {
        if (LANES < 64) {
            sub = threadIdx.x / LANES;
            t = threadIdx.x % LANES;
            across = LANES;
        } else {
            const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            sub = wave / waves;
            t = threadIdx.x - sub * waves * 64;
            across = waves * 64;
        }
    }
};
// Sums of two values over the threads of a row, or of one and the largest of
// the other as a magnitude; one barrier where a row has several waves, whose
// values meet in another half of tmp at every other call (`turn`), so that the
// next call may write while this one reads.  tmp holds zeros at first.
typedef float RowJoin[2][8][16][2];
template <bool MAX, int LANES>
__device__ inline void row_join(float& a, float& b, RowJoin& tmp, int turn, int waves, int sub)
{
    if constexpr (LANES < 64) {
        a = row16_sum(a);
        b = MAX ? __uint_as_float(lanes_umax<16>(__float_as_uint(b))) : row16_sum(b);
        if (LANES == 32) {
            const float a2 = __shfl_xor(a, 16, 64), b2 = __shfl_xor(b, 16, 64);
            a += a2;
            b = MAX ? __uint_as_float(umax(__float_as_uint(b), __float_as_uint(b2))) : b + b2;
        }
    } else {
        a = wave_sum(a);
        b = MAX ? __uint_as_float(wave_umax(__float_as_uint(b))) : wave_sum(b);
        if (waves == 1) return;
        if ((threadIdx.x & 63) == 0) {
            const int w = (threadIdx.x >> 6) - sub * waves;
            tmp[turn][sub][w][0] = a;
            tmp[turn][sub][w][1] = b;
        }
        __syncthreads();
        a = sum_of_lanes<16>(tmp[turn][sub][threadIdx.x & 15][0]);
        b = tmp[turn][sub][threadIdx.x & 15][1];
        b = MAX ? __int_as_float(__builtin_amdgcn_readfirstlane((int)lanes_umax<16>(__float_as_uint(b))))
                : sum_of_lanes<16>(b);
    }
}
__device__ inline void clear_join(RowJoin& tmp)
{
    for (int i = threadIdx.x; i < 2 * 8 * 16 * 2; i += blockDim.x) ((float*)tmp)[i] = 0.f;
    __syncthreads();
}
// EPT columns of a thread's weights as fp32; `none` where there are none.
template <typename T, int NV>
__device__ inline void row_weights(const void* w, bool w32, int across, int t, int cols, float none, float* out)
{
    constexpr int VL = VecLen<T>::value;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int v = n * across + t;
        float* x = out + n * VL;
        if (w && (v + 1) * VL <= cols && w32) {
            const Pack<float, VL> q = ((const Pack<float, VL>*)w)[v];
#pragma unroll
            for (int e = 0; e < VL; ++e) x[e] = q.v[e];
        } else if (w && (v + 1) * VL <= cols) {
            unpack<T>(((const Raw*)w)[v], x);
        } else {
#pragma unroll
            for (int e = 0; e < VL; ++e) {
                const int c = v * VL + e;
                x[e] = !w || c >= cols ? none : w32 ? ((const float*)w)[c] : to_f(((const T*)w)[c]);
            }
        }
    }
}

// 8 elements a thread, in 16 or 32 lanes, or in as many waves as that takes; 4
// (a vector of fp32) where 8 waves hold a row so (8000 x 4001 fp32 backward 98 ->
// 91 us with them, 20001 x 650 from 8 bits 40.5 -> 35.8, but by 16 waves the
// layer norm's 88 -> 97), 16 in rows that are longer than 16 waves hold with 8.
inline RowShape row_shape(int64_t cols, int32_t dtype)
{
    if (cols <= 128) return {16, 8, 1, 32};
    if (cols <= 256) return {32, 8, 1, 16};
    const int ept = cols <= 2048 && dtype == SGC_F32 ? 4 : cols <= 8192 ? 8 : 16, waves = (int)cdiv(cols, 64 * ept);
    return {64, ept, waves, waves < 8 ? 8 / waves : 1};
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
