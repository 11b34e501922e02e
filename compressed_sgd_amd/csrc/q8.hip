// q8.hip -- rows kept in 8 bits with a scale a group, and read back.
#include "lm_q8.h"

namespace sgc {

// Vectors of 16 bytes of all rows in one line, kAtOnce a thread and trip; `each`
// vectors a row, with what pads a row to whole groups, and 1 / each.
constexpr int kThreads = 256, kAtOnce = 4;
struct Line {
    int64_t rows;
    int cols, each;
    float inverse;
};
// Row and vector of number `at` past vector `first` of row r.
__device__ inline void line_place(const Line& l, int64_t r, int first, int at, int64_t& row, int& v)
{
    const int n = first + at;
    int k = (int)((float)n * l.inverse);  // off by one at most: n < 2^18 + 2^10
    k -= k * l.each > n;
    k += (k + 1) * l.each <= n;
    row = r + k;
    v = n - k * l.each;
}
// The largest over each L neighbouring lanes, a power of two from 4.
__device__ inline uint32_t neighbours_umax(uint32_t x, int lanes)
{
    x = umax(x, dpp_own<0xb1, 0xf>(x));
    x = umax(x, dpp_own<0x4e, 0xf>(x));
    if (lanes >= 8) x = umax(x, dpp_own<0x141, 0xf>(x));   // mirrored in eights: fours are alike by now
    if (lanes >= 16) x = umax(x, dpp_own<0x140, 0xf>(x));  // in sixteens
    if (lanes >= 32) x = umax(x, (uint32_t)__shfl_xor((int)x, 16, 64));
    if (lanes >= 64) x = umax(x, (uint32_t)__shfl_xor((int)x, 32, 64));
    return x;
}
template <int VL>
__device__ inline Bytes<VL> quantized_vec(const float* f, const Quant& k)
{
    uint32_t q[VL];
#pragma unroll
    for (int e = 0; e < VL; ++e) q[e] = quantized(f[e], k);
    Bytes<VL> b;
#pragma unroll
    for (int e = 0; e < VL; e += 4) b.w[e / 4] = four_bytes(q[e], q[e + 1], q[e + 2], q[e + 3]) & k.keep;
    return b;
}

// A group is 4 to 64 neighbouring lanes.  Bound by memory: 16384 x 4096 bf16 34 us
// from the cache (5.9 TB/s).
template <typename T, bool RAG>
__global__ __launch_bounds__(kThreads) void k_quantize(const T* x, int64_t xs, int8_t* q, int64_t qs, float* scale,
                                                       Line l, int shift, int lanes, int64_t groups, bool once)
{
    constexpr int VL = VecLen<T>::value;
    const int64_t total = l.rows * l.each;
    for (int64_t base = (int64_t)blockIdx.x * kThreads * kAtOnce; base < total;
         base += (int64_t)gridDim.x * kThreads * kAtOnce) {
        const int64_t r0 = base / l.each;
        const int first = (int)(base - r0 * l.each);
        int64_t r[kAtOnce];
        int v[kAtOnce];
        Raw raw[kAtOnce] = {};
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            line_place(l, r0, first, u * kThreads + threadIdx.x, r[u], v[u]);
            if (r[u] < l.rows) raw[u] = load_vec<T, RAG>(x + r[u] * xs, v[u], l.cols, once);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            float f[VL];
            settle<T, RAG>(raw[u], v[u], l.cols);
            unpack<T>(raw[u], f);
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < VL; ++e) top = umax(top, magnitude(f[e]));
            const Quant k = quant_of(neighbours_umax(top, lanes));
            if (r[u] >= l.rows) continue;
            store_bytes<VL, RAG>(q + r[u] * qs, v[u], l.cols, quantized_vec<VL>(f, k));
            if ((v[u] & (lanes - 1)) == 0) scale[r[u] * groups + (v[u] * VL >> shift)] = k.scale;
        }
    }
}

// One scale a row, the row in registers.  50000 x 1024 fp32: 58 us (4.4 TB/s; two
// vectors a thread gain nothing).
template <typename T, int LANES, int EPT, bool RAG>
__global__ __launch_bounds__(LANES < 64 ? 512 : 1024) void k_quantize_rows(const T* x, int64_t xs, int8_t* q,
                                                                           int64_t qs, float* scale, int64_t rows,
                                                                           int cols, int waves, int side, bool once)
{
    constexpr int VL = VecLen<T>::value, NV = EPT / VL;
    __shared__ RowJoin tmp;
    if (LANES == 64 && waves > 1) clear_join(tmp);
    const RowPlace<LANES> place(waves);
    int64_t r = (int64_t)blockIdx.x * side + place.sub;
    const int64_t step = (int64_t)gridDim.x * side;
    Raw next[NV] = {};
    const auto fetch = [&](int64_t at) {
#pragma unroll
        for (int n = 0; n < NV; ++n)
            next[n] = load_vec<T, RAG>(x + at * xs, n * place.across + place.t, cols, once);
    };
    if (r < rows) fetch(r);
    int turn = 0;
    for (; r - place.sub < rows; r += step, turn ^= 1) {
        float f[EPT], none = 0.f;
        uint32_t top = 0;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            settle<T, RAG>(next[n], n * place.across + place.t, cols);
            unpack<T>(next[n], f + n * VL);
        }
        if (r + step < rows) fetch(r + step);
#pragma unroll
        for (int i = 0; i < EPT; ++i) top = umax(top, magnitude(f[i]));
        float most = __uint_as_float(top);
        row_join<true, LANES>(none, most, tmp, turn, waves, place.sub);
        if (r >= rows) continue;
        const Quant k = quant_of(__float_as_uint(most));
#pragma unroll
        for (int n = 0; n < NV; ++n)
            store_bytes<VL, RAG>(q + r * qs, n * place.across + place.t, cols, quantized_vec<VL>(f + n * VL, k));
        if (place.t == 0) scale[r] = k.scale;
    }
}

// One scale a row, read twice.
template <typename T>
__global__ __launch_bounds__(kLongThreads) void k_quantize_long(const T* x, int64_t xs, int8_t* q, int64_t qs,
                                                                float* scale, int64_t rows, int cols)
{
    constexpr int VL = VecLen<T>::value;
    __shared__ uint32_t tmp[kLongWaves];
    const int64_t r = row_of_block();
    if (r >= rows) return;
    const T* xr = x + r * xs;
    uint32_t top = 0;
    const auto values = [&](int v, float* f) {
        Raw raw = load_vec<T, true>(xr, v, cols, false);
        settle<T, true>(raw, v, cols);
        unpack<T>(raw, f);
    };
    for (int v = threadIdx.x; v * VL < cols; v += kLongThreads) {
        float f[VL];
        values(v, f);
#pragma unroll
        for (int e = 0; e < VL; ++e) top = umax(top, magnitude(f[e]));
    }
    const Quant k = quant_of(block_umax<kLongWaves>(top, tmp));
    for (int v = threadIdx.x; v * VL < cols; v += kLongThreads) {
        float f[VL];
        values(v, f);
        store_bytes<VL, true>(q + r * qs, v, cols, quantized_vec<VL>(f, k));
    }
    if (threadIdx.x == 0) scale[r] = k.scale;
}

// 16384 x 4096 bf16: 31 us, 6.4 TB/s.
template <typename T, bool RAG>
__global__ __launch_bounds__(kThreads) void k_dequantize(const int8_t* q, int64_t qs, const float* scale, T* x,
                                                         int64_t xs, Line l, int shift, int64_t groups, bool once)
{
    constexpr int VL = VecLen<T>::value;
    const int64_t total = l.rows * l.each;
    for (int64_t base = (int64_t)blockIdx.x * kThreads * kAtOnce; base < total;
         base += (int64_t)gridDim.x * kThreads * kAtOnce) {
        const int64_t r0 = base / l.each;
        const int first = (int)(base - r0 * l.each);
        int64_t r[kAtOnce];
        int v[kAtOnce];
        Bytes<VL> b[kAtOnce] = {};
        float s[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            line_place(l, r0, first, u * kThreads + threadIdx.x, r[u], v[u]);
            s[u] = 0.f;
            if (r[u] < l.rows) {
                b[u] = load_bytes<VL, RAG>(q + r[u] * qs, v[u], l.cols);
                s[u] = scale[r[u] * groups + (v[u] * VL >> shift)];
            }
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            if (r[u] >= l.rows) continue;
            float f[VL];
            settle<VL, RAG>(b[u], v[u], l.cols);
#pragma unroll
            for (int e = 0; e < VL; ++e) f[e] = byte_of(b[u].w[e / 4], e % 4) * s[u];
            store_vec<T, RAG>(x + r[u] * xs, v[u], l.cols, f, once);
        }
    }
}

static bool q8_ok(const sgc_q8_opts* o)
{
    return o && o->rows >= 0 && o->rows < ((int64_t)1 << 31) && o->cols >= 1 && o->cols <= kNormMaxCols &&
           lm_dtype(o->dtype) && q8_group_ok(o->group);
}

static Line line_of(const sgc_q8_opts* o, int vl, int whole)
{
    const int each = (int)cdiv(o->cols, whole) * (whole / vl);
    return {o->rows, (int)o->cols, each, 1.f / (float)each};
}
// 8 workgroups of 256 threads a compute unit, twice over.
static unsigned line_groups(const Line& l)
{
    const int64_t need = cdiv(l.rows * l.each, kThreads * kAtOnce), most = kCus * 16;
    return (unsigned)(need < most ? need : most);
}

template <typename T, int LANES, int EPT>
static void quantize_rows(const sgc_q8_opts* o, const RowShape& sh, const T* x, int64_t xs, int8_t* q, int64_t qs,
                          float* scale, bool once, hipStream_t s)
{
    const int cols = (int)o->cols;
    const unsigned g = (unsigned)row_groups(sh, o->rows, kForwardWaves);
    if (cols % VecLen<T>::value)
        k_quantize_rows<T, LANES, EPT, true><<<g, sh.threads(), 0, s>>>(x, xs, q, qs, scale, o->rows, cols, sh.waves,
                                                                       sh.rows, once);
    else
        k_quantize_rows<T, LANES, EPT, false><<<g, sh.threads(), 0, s>>>(x, xs, q, qs, scale, o->rows, cols, sh.waves,
                                                                        sh.rows, once);
}

template <typename T>
static int quantize(const sgc_q8_opts* o, const void* xv, int64_t xs, int8_t* q, int64_t qs, float* scale,
                    hipStream_t s)
{
    constexpr int VL = VecLen<T>::value;
    const T* x = (const T*)xv;
    const int cols = (int)o->cols;
    // x is not read again, what becomes of it may be: x past the caches from half of
    // them on, so that the 8 bits stay there.  Quantised from memory and read back at
    // once, from half and from all: 16384 x 4096 bf16 67.8 and 73.0 us, 65536 x 1024
    // one scale a row 67.7 and 73.0, 20000 x 2048 fp32 68.6 and 79.1, 12000 x 4096
    // bf16 50.9 and 50.3, 6000 x 8192 fp32 97.0 and 96.3; quantised alone 0 to 2% more
    const bool once = o->rows * cols * (int64_t)(sizeof(T) + 1) >= kCacheBytes / 2;
    if (o->group) {
        const Line l = line_of(o, VL, o->group);
        const unsigned g = line_groups(l);
        const int shift = q8_shift(o->group), lanes = o->group / VL;
        const int64_t groups = q8_groups(cols, o->group);
        if (cols % VL) k_quantize<T, true><<<g, kThreads, 0, s>>>(x, xs, q, qs, scale, l, shift, lanes, groups, once);
        else k_quantize<T, false><<<g, kThreads, 0, s>>>(x, xs, q, qs, scale, l, shift, lanes, groups, once);
    } else if (cols > kNormHeld) {
        k_quantize_long<T><<<row_grid(o->rows), kLongThreads, 0, s>>>(x, xs, q, qs, scale, o->rows, cols);
    } else {
        const RowShape sh = row_shape(cols, o->dtype);
        if (sh.lanes == 16) quantize_rows<T, 16, 8>(o, sh, x, xs, q, qs, scale, once, s);
        else if (sh.lanes == 32) quantize_rows<T, 32, 8>(o, sh, x, xs, q, qs, scale, once, s);
        else if (sh.ept == 8) quantize_rows<T, 64, 8>(o, sh, x, xs, q, qs, scale, once, s);
        else if (sh.ept == 16) quantize_rows<T, 64, 16>(o, sh, x, xs, q, qs, scale, once, s);
        else if constexpr (sizeof(T) == 4) quantize_rows<T, 64, 4>(o, sh, x, xs, q, qs, scale, once, s);
    }
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}
template <typename T>
static int dequantize(const sgc_q8_opts* o, const int8_t* q, int64_t qs, const float* scale, void* xv, int64_t xs,
                      hipStream_t s)
{
    constexpr int VL = VecLen<T>::value;
    T* x = (T*)xv;
    const bool once = o->rows * o->cols * (int64_t)(sizeof(T) + 1) >= kCacheBytes;
    const Line l = line_of(o, VL, VL);
    const unsigned g = line_groups(l);
    const int shift = q8_shift(o->group);
    const int64_t groups = q8_groups(o->cols, o->group);
    if (o->cols % VL) k_dequantize<T, true><<<g, kThreads, 0, s>>>(q, qs, scale, x, xs, l, shift, groups, once);
    else k_dequantize<T, false><<<g, kThreads, 0, s>>>(q, qs, scale, x, xs, l, shift, groups, once);
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}

}  // namespace sgc

using namespace sgc;

extern "C" int sgc_quantize_q8(const sgc_q8_opts* o, const void* x, int64_t x_stride, int8_t* q, int64_t q_stride,
                               float* scale, sgc_stream_t stream)
{
    if (!q8_ok(o)) return SGC_EINVAL;
    if (o->rows == 0) return SGC_OK;
    if (!lm_rows_ok(x, x_stride, o->rows, o->cols, o->dtype, false)) return SGC_EINVAL;
    if (!q8_rows_ok(q, q_stride, o->rows, o->cols, true) || !scale || !lm_aligned(scale, 4)) return SGC_EINVAL;
    const hipStream_t s = (hipStream_t)stream;
    return o->dtype == SGC_F32    ? quantize<float>(o, x, x_stride, q, q_stride, scale, s)
           : o->dtype == SGC_BF16 ? quantize<bf16_t>(o, x, x_stride, q, q_stride, scale, s)
                                  : quantize<f16_t>(o, x, x_stride, q, q_stride, scale, s);
}

extern "C" int sgc_dequantize_q8(const sgc_q8_opts* o, const int8_t* q, int64_t q_stride, const float* scale, void* x,
                                 int64_t x_stride, sgc_stream_t stream)
{
    if (!q8_ok(o)) return SGC_EINVAL;
    if (o->rows == 0) return SGC_OK;
    if (!lm_rows_ok(x, x_stride, o->rows, o->cols, o->dtype, true)) return SGC_EINVAL;
    if (!q8_rows_ok(q, q_stride, o->rows, o->cols, false) || !scale || !lm_aligned(scale, 4)) return SGC_EINVAL;
    const hipStream_t s = (hipStream_t)stream;
    return o->dtype == SGC_F32    ? dequantize<float>(o, q, q_stride, scale, x, x_stride, s)
           : o->dtype == SGC_BF16 ? dequantize<bf16_t>(o, q, q_stride, scale, x, x_stride, s)
                                  : dequantize<f16_t>(o, q, q_stride, scale, x, x_stride, s);
}
