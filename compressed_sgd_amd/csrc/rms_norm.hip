// rms_norm.hip -- RMS norm of a residual stream with the addition before it,
// its output in the stream's type or in 8 bits, and its backward pass.
//
//   s = x + residual,  rstd = (mean(s^2) + eps)^(-1/2),  y = s rstd w
//   8 bits: p = s w, a = max |p|, q = rint(p (127 / a)), scale = (a / 127) rstd
#include "norm_back.h"

namespace sgc {

struct Rms {
    const void* x;
    int64_t xs;
    const void* res;
    int64_t ress;
    const void* w;
    bool w32;
    void* sum;
    int64_t ss;
    void* y;
    int64_t ys;
    int8_t* q;
    int64_t qs;
    float *qscale, *rstd;
    int64_t rows;
    int cols;
    float eps;
};

// Rows in registers between their sums and their output, the next rows on their
// way; the weights stay in registers across a workgroup's rows.  E8: 8 bits out;
// the largest magnitude comes with the sum of squares, through the same barrier.
// Bound by memory: 16384 x 4096 bf16 with the residual 94 us, 5.7 TB/s; 10007 x
// 1024 fp16 into 8 bits 15 us; 8 x 1024 3.2 us.  Ragged rows start at any 2 bytes
// (16384 x 4094 bf16: 109 us); one whose last vector takes a wave of its own has
// nine where eight would do (16384 x 4099: 140).
template <typename T, int LANES, int EPT, bool RAG, bool E8>
__global__ __launch_bounds__(LANES < 64 ? 512 : 1024) void k_rms(Rms k, int waves, int side, bool once)
{
    constexpr int VL = VecLen<T>::value, NV = EPT / VL;
    __shared__ RowJoin tmp;
    if (LANES == 64 && waves > 1) clear_join(tmp);
    const RowPlace<LANES> place(waves);
    const int sub = place.sub, t = place.t, across = place.across, cols = k.cols;
    float wf[EPT];
    row_weights<T, NV>(k.w, k.w32, across, t, cols, 1.f, wf);
    Raw nx[NV] = {}, nr[NV] = {};
    int64_t r = (int64_t)blockIdx.x * side + sub;
    const int64_t step = (int64_t)gridDim.x * side;
    const auto fetch = [&](int64_t at) {
#pragma unroll
        for (int n = 0; n < NV; ++n) nx[n] = load_vec<T, RAG>((const T*)k.x + at * k.xs, n * across + t, cols, once);
        if (k.res) {
#pragma unroll
            for (int n = 0; n < NV; ++n)
                nr[n] = load_vec<T, RAG>((const T*)k.res + at * k.ress, n * across + t, cols, once);
        }
    };
    if (r < k.rows) fetch(r);
    int turn = 0;
    for (; r - sub < k.rows; r += step, turn ^= 1) {
        float f[EPT];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            settle<T, RAG>(nx[n], n * across + t, cols);
            unpack<T>(nx[n], f + n * VL);
        }
        if (k.res) {
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                float g[VL];
                settle<T, RAG>(nr[n], n * across + t, cols);
                unpack<T>(nr[n], g);
#pragma unroll
                for (int e = 0; e < VL; ++e) f[n * VL + e] += g[e];
                unpack<T>(pack<T>(f + n * VL), f + n * VL);
            }
        }
        if (r + step < k.rows) fetch(r + step);
        const bool live = r < k.rows;
        if (k.sum && live) {
#pragma unroll
            for (int n = 0; n < NV; ++n)
                store_vec<T, RAG>((T*)k.sum + r * k.ss, n * across + t, cols, f + n * VL, once);
        }
        float ss = 0.f, most = 0.f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            ss = fmaf(f[i], f[i], ss);
            if (E8) {
                f[i] *= wf[i];
                // past the end 0 times the 1 that stands for a weight there
                most = __uint_as_float(umax(__float_as_uint(most), magnitude(f[i])));
            }
        }
        row_join<E8, LANES>(ss, most, tmp, turn, waves, sub);
        const float rs = 1.f / sqrtf(ss / (float)cols + k.eps);
        if (!live) continue;
        if (E8) {
            const Quant u = quant_of(__float_as_uint(most));
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                uint32_t q[VL];
#pragma unroll
                for (int e = 0; e < VL; ++e) q[e] = quantized(f[n * VL + e], u);
                Bytes<VL> b;
#pragma unroll
                for (int e = 0; e < VL; e += 4) b.w[e / 4] = four_bytes(q[e], q[e + 1], q[e + 2], q[e + 3]) & u.keep;
                store_bytes<VL, RAG>(k.q + r * k.qs, n * across + t, cols, b);
            }
            if (t == 0) k.qscale[r] = u.scale == 0.f ? 0.f : u.scale * rs;  // rs is infinite for zeros and eps 0
        } else {
#pragma unroll
            for (int i = 0; i < EPT; ++i) f[i] = f[i] * rs * wf[i];
#pragma unroll
            for (int n = 0; n < NV; ++n)
                store_vec<T, RAG>((T*)k.y + r * k.ys, n * across + t, cols, f + n * VL, once);
        }
        if (t == 0 && k.rstd) k.rstd[r] = rs;
    }
}

// Rows that registers do not hold: one workgroup a row, element by element, the
// row read again for every pass.  Every element is
// read and written by one thread alone, so the sum and y may take the inputs'
// places; once the sum is written it is read instead of them.
template <typename T>
__global__ __launch_bounds__(kLongThreads) void k_rms_long(Rms k)
{
    __shared__ float tmp[kLongWaves];
    __shared__ uint32_t utmp[kLongWaves];
    const int64_t r = row_of_block();
    if (r >= k.rows) return;
    const T* x = (const T*)k.x + r * k.xs;
    const T* res = k.res ? (const T*)k.res + r * k.ress : nullptr;
    T* sum = k.sum ? (T*)k.sum + r * k.ss : nullptr;
    float ss = 0.f;
    uint32_t top = 0;
    for (int c = threadIdx.x; c < k.cols; c += kLongThreads) {
        const T t = res ? from_f<T>(to_f(x[c]) + to_f(res[c])) : x[c];
        if (sum) sum[c] = t;
        const float f = to_f(t);
        ss = fmaf(f, f, ss);
        if (k.q) top = umax(top, magnitude(f * weight_at<T>(k.w, k.w32, c, 1.f)));
    }
    const float rs = 1.f / sqrtf(block_sum<kLongWaves>(ss, tmp) / (float)k.cols + k.eps);
    Quant u = {};
    if (k.q) {
        u = quant_of(block_umax<kLongWaves>(top, utmp));
        if (threadIdx.x == 0) k.qscale[r] = u.scale == 0.f ? 0.f : u.scale * rs;  // rs is infinite for zeros and eps 0
    }
    if (threadIdx.x == 0 && k.rstd) k.rstd[r] = rs;
    for (int c = threadIdx.x; c < k.cols; c += kLongThreads) {
        const T t = sum ? sum[c] : res ? from_f<T>(to_f(x[c]) + to_f(res[c])) : x[c];
        const float w = weight_at<T>(k.w, k.w32, c, 1.f), f = to_f(t);
        if (k.q) k.q[r * k.qs + c] = (int8_t)(quantized(f * w, u) & u.keep);
        else ((T*)k.y)[r * k.ys + c] = from_f<T>(f * rs * w);
    }
}

template <typename T, int LANES, int EPT>
static void rms_held(const Rms& k, const RowShape& sh, unsigned g, bool once, hipStream_t s)
{
    const bool rag = k.cols % VecLen<T>::value;
    if (k.q) {
        if (rag) k_rms<T, LANES, EPT, true, true><<<g, sh.threads(), 0, s>>>(k, sh.waves, sh.rows, once);
        else k_rms<T, LANES, EPT, false, true><<<g, sh.threads(), 0, s>>>(k, sh.waves, sh.rows, once);
    } else {
        if (rag) k_rms<T, LANES, EPT, true, false><<<g, sh.threads(), 0, s>>>(k, sh.waves, sh.rows, once);
        else k_rms<T, LANES, EPT, false, false><<<g, sh.threads(), 0, s>>>(k, sh.waves, sh.rows, once);
    }
}

template <typename T>
static int rms_forward(const Rms& k, int32_t dtype, hipStream_t s)
{
    if (k.cols > kNormHeld) {
        k_rms_long<T><<<row_grid(k.rows), kLongThreads, 0, s>>>(k);
        SGC_LAUNCH_CHECK();
        return SGC_OK;
    }
    const RowShape sh = row_shape(k.cols, dtype);
    const unsigned g = (unsigned)row_groups(sh, k.rows, kForwardWaves);
    const int64_t moved = (1 + (k.res != nullptr) + (k.sum != nullptr)) * (int64_t)sizeof(T) + (k.q ? 1 : sizeof(T));
    const bool once = k.rows * k.cols * moved >= kCacheBytes;
    if (sh.lanes == 16) rms_held<T, 16, 8>(k, sh, g, once, s);
    else if (sh.lanes == 32) rms_held<T, 32, 8>(k, sh, g, once, s);
    else if (sh.ept == 8) rms_held<T, 64, 8>(k, sh, g, once, s);
    else if (sh.ept == 4) {
        if constexpr (sizeof(T) == 4) rms_held<T, 64, 4>(k, sh, g, once, s);
    }
    else rms_held<T, 64, 16>(k, sh, g, once, s);
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}

}  // namespace sgc

using namespace sgc;

extern "C" int sgc_rms_norm(const sgc_norm_opts* o, const void* x, int64_t x_stride, const void* residual,
                            int64_t r_stride, const void* weight, void* sum, int64_t s_stride, void* y,
                            int64_t y_stride, int8_t* q, int64_t q_stride, float* qscale, float* rstd,
                            sgc_stream_t stream)
{
    if (!norm_opts_ok(o) || o->flags) return SGC_EINVAL;
    if (o->rows == 0) return SGC_OK;
    if (!y == !q || !q != !qscale) return SGC_EINVAL;
    const int64_t n = o->rows, c = o->cols;
    if (!lm_rows_ok(x, x_stride, n, c, o->dtype, false)) return SGC_EINVAL;
    if (residual && !lm_rows_ok(residual, r_stride, n, c, o->dtype, false)) return SGC_EINVAL;
    if (sum && !lm_rows_ok(sum, s_stride, n, c, o->dtype, true)) return SGC_EINVAL;
    if (y && (!lm_rows_ok(y, y_stride, n, c, o->dtype, true) || y == sum)) return SGC_EINVAL;
    if (q && !q8_rows_ok(q, q_stride, n, c, true)) return SGC_EINVAL;
    if (!lm_aligned(weight, lm_size(o->wdtype)) || !lm_aligned(qscale, 4) || !lm_aligned(rstd, 4)) return SGC_EINVAL;
    const Rms k = {x,        x_stride, residual, r_stride, weight, o->wdtype == SGC_F32, sum, s_stride, y, y_stride, q,
                   q_stride, qscale,   rstd,     n,        (int)c, o->eps};
    const hipStream_t s = (hipStream_t)stream;
    return o->dtype == SGC_F32    ? rms_forward<float>(k, o->dtype, s)
           : o->dtype == SGC_BF16 ? rms_forward<bf16_t>(k, o->dtype, s)
                                  : rms_forward<f16_t>(k, o->dtype, s);
}

extern "C" size_t sgc_rms_norm_backward_workspace(const sgc_norm_opts* o)
{
    if (!norm_opts_ok(o)) return 0;
    Carver c(nullptr);
    c.take<float>(back_parts(o->rows, o->cols, o->dtype) * o->cols);
    return c.off;
}

extern "C" int sgc_rms_norm_backward(const sgc_norm_opts* o, const void* dy, int64_t dy_stride, const void* x,
                                     int64_t s_stride, const void* weight, const float* rstd, const void* dsum,
                                     int64_t dsum_stride, void* dx, int64_t dx_stride, float* dweight, void* ws,
                                     size_t ws_bytes, sgc_stream_t stream)
{
    if (!norm_opts_ok(o)) return SGC_EINVAL;
    if (!lm_aligned(dweight, 4) || !lm_aligned(weight, lm_size(o->wdtype))) return SGC_EINVAL;
    if (o->rows) {
        if (!lm_rows_ok(dy, dy_stride, o->rows, o->cols, o->dtype, false)) return SGC_EINVAL;
        if (!lm_rows_ok(x, s_stride, o->rows, o->cols, o->dtype, false)) return SGC_EINVAL;
        if (dsum && !lm_rows_ok(dsum, dsum_stride, o->rows, o->cols, o->dtype, false)) return SGC_EINVAL;
        if (dx && !lm_rows_ok(dx, dx_stride, o->rows, o->cols, o->dtype, true)) return SGC_EINVAL;
        if (!rstd || !lm_aligned(rstd, 4)) return SGC_EINVAL;
    }
    float* part = nullptr;
    if (dweight) {
        if (!ws || ws_bytes < sgc_rms_norm_backward_workspace(o)) return SGC_ENOSPC;
        if (!aligned16(ws)) return SGC_EINVAL;
        part = Carver(ws).take<float>(1);
    }
    const Back k = {dy, dy_stride, weight,  nullptr, o->wdtype == SGC_F32, nullptr, rstd, dsum, dsum_stride,
                    dx, dx_stride, nullptr, 0,       part,                 o->rows, (int)o->cols,
                    dweight, nullptr, (o->flags & SGC_NORM_ADD_GRADS) != 0};
    const hipStream_t s = (hipStream_t)stream;
    switch (o->dtype) {
    case SGC_F32:
        return norm_back<float, AsIs<float>, false>({(const float*)x, s_stride}, k, o->dtype, s);
    case SGC_BF16:
        return norm_back<bf16_t, AsIs<bf16_t>, false>({(const bf16_t*)x, s_stride}, k, o->dtype, s);
    default:
        return norm_back<f16_t, AsIs<f16_t>, false>({(const f16_t*)x, s_stride}, k, o->dtype, s);
    }
}
