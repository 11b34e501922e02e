// layer_norm.hip -- layer norm over the last dimension, forward and backward,
// with the sums over the rows that are the gradients of weight and bias.
//
//   y  = (x - mean) rstd w + b
//   dx = rstd (v - mean(v) - xh mean(v xh)),  v = dy w,  xh = (x - mean) rstd
//   dw = sum_rows dy xh,  db = sum_rows dy
#include "lm_common.h"

namespace sgc {

constexpr int kNormThreads = 256;
constexpr int kNormWaves = kNormThreads / 64;

template <typename T, typename W>
__global__ __launch_bounds__(kNormThreads) void k_norm(const T* x, int64_t xs, const W* w, const W* b, T* y,
                                                       int64_t ys, float* mean, float* rstd, int64_t rows, int64_t cols, float eps)
{
    __shared__ float tmp[kNormWaves];
    const int64_t r = row_of_block();
    if (r >= rows) return;
    const T* xr = x + r * xs;
    T* yr = y + r * ys;
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < cols; c += kNormThreads) s += to_f(xr[c]);
    const float m = block_sum<kNormWaves>(s, tmp) / (float)cols;
    float q = 0.f;
    for (int64_t c = threadIdx.x; c < cols; c += kNormThreads) {
        const float d = to_f(xr[c]) - m;
        q = fmaf(d, d, q);
    }
    const float rs = 1.0f / sqrtf(block_sum<kNormWaves>(q, tmp) / (float)cols + eps);
    for (int64_t c = threadIdx.x; c < cols; c += kNormThreads) {
        const float h = (to_f(xr[c]) - m) * rs;
        yr[c] = from_f<T>(fmaf(h, w ? to_f(w[c]) : 1.f, b ? to_f(b[c]) : 0.f));
    }
    if (threadIdx.x == 0) {
        if (mean) mean[r] = m;
        if (rstd) rstd[r] = rs;
    }
}

template <typename T, typename W>
__global__ __launch_bounds__(kNormThreads) void k_norm_dx(const T* dy, int64_t dys, const T* x, int64_t xs, const W* w,
                                                          const float* mean, const float* rstd, T* dx, int64_t dxs,
                                                          int64_t rows, int64_t cols)
{
    __shared__ float tmp[kNormWaves];
    const int64_t r = row_of_block();
    if (r >= rows) return;
    const float m = mean[r], rs = rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t c = threadIdx.x; c < cols; c += kNormThreads) {
        const float v = to_f(dy[r * dys + c]) * (w ? to_f(w[c]) : 1.f);
        s1 += v;
        s2 = fmaf(v, (to_f(x[r * xs + c]) - m) * rs, s2);
    }
    const float c1 = block_sum<kNormWaves>(s1, tmp) / (float)cols;
    const float c2 = block_sum<kNormWaves>(s2, tmp) / (float)cols;
    for (int64_t c = threadIdx.x; c < cols; c += kNormThreads) {
        const float v = to_f(dy[r * dys + c]) * (w ? to_f(w[c]) : 1.f);
        const float h = (to_f(x[r * xs + c]) - m) * rs;
        dx[r * dxs + c] = from_f<T>(rs * (v - fmaf(h, c2, c1)));
    }
}

// Partial sums over the rows part, part + parts, ...
template <typename T>
__global__ __launch_bounds__(kNormThreads) void k_norm_dw(const T* dy, int64_t dys, const T* x, int64_t xs,
                                                          const float* mean, const float* rstd, float* part,
                                                          int64_t rows, int64_t cols)
{
    const int64_t c = (int64_t)blockIdx.x * kNormThreads + threadIdx.x;
    if (c >= cols) return;
    float aw = 0.f, ab = 0.f;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const float g = to_f(dy[r * dys + c]);
        aw = fmaf(g, (to_f(x[r * xs + c]) - mean[r]) * rstd[r], aw);
        ab += g;
    }
    part[(2 * (int64_t)blockIdx.y + 0) * cols + c] = aw;
    part[(2 * (int64_t)blockIdx.y + 1) * cols + c] = ab;
}

__global__ __launch_bounds__(kNormThreads) void k_norm_join(const float* part, int64_t parts, int64_t cols, float* dw,
                                                            float* db, int add)
{
    const int64_t c = (int64_t)blockIdx.x * kNormThreads + threadIdx.x;
    if (c >= cols) return;
    float aw = 0.f, ab = 0.f;
    for (int64_t p = 0; p < parts; ++p) {
        aw += part[(2 * p + 0) * cols + c];
        ab += part[(2 * p + 1) * cols + c];
    }
    if (dw) dw[c] = add ? dw[c] + aw : aw;
    if (db) db[c] = add ? db[c] + ab : ab;
}

constexpr int64_t kNormMaxCols = (int64_t)1 << 20;

static bool norm_opts_ok(const sgc_norm_opts* o)
{
    return o && o->rows >= 0 && o->rows < ((int64_t)1 << 31) && o->cols >= 1 && o->cols <= kNormMaxCols &&
           lm_dtype(o->dtype) && (o->wdtype == SGC_F32 || o->wdtype == o->dtype) && o->eps >= 0.f &&
           std::isfinite(o->eps) && (o->flags & ~SGC_NORM_ADD_GRADS) == 0;
}

static int64_t norm_parts(const sgc_norm_opts* o) { return o->rows < 256 ? o->rows : 256; }

template <typename T, typename W>
static int norm_forward(const sgc_norm_opts* o, const void* x, int64_t xs, const void* w, const void* b, void* y,
                        int64_t ys, float* mean, float* rstd, hipStream_t s)
{
    k_norm<T, W><<<row_grid(o->rows), kNormThreads, 0, s>>>((const T*)x, xs, (const W*)w, (const W*)b, (T*)y, ys, mean,
                                                            rstd, o->rows, o->cols, o->eps);
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}

template <typename T, typename W>
static int norm_backward(const sgc_norm_opts* o, const void* dy, int64_t dys, const void* x, int64_t xs, const void* w,
                         const float* mean, const float* rstd, void* dx, int64_t dxs, float* dw, float* db, float* part,
                         hipStream_t s)
{
    const int64_t parts = norm_parts(o);
    const unsigned cb = (unsigned)cdiv(o->cols, kNormThreads);
    if ((dw || db) && parts) {
        k_norm_dw<T><<<dim3(cb, (unsigned)parts), kNormThreads, 0, s>>>((const T*)dy, dys, (const T*)x, xs, mean, rstd,
                                                                       part, o->rows, o->cols);
        SGC_LAUNCH_CHECK();
    }
    if (dx && o->rows) {
        k_norm_dx<T, W><<<row_grid(o->rows), kNormThreads, 0, s>>>((const T*)dy, dys, (const T*)x, xs, (const W*)w,
                                                                   mean, rstd, (T*)dx, dxs, o->rows, o->cols);
        SGC_LAUNCH_CHECK();
    }
    if (dw || db) {
        k_norm_join<<<cb, kNormThreads, 0, s>>>(part, parts, o->cols, dw, db, o->flags & SGC_NORM_ADD_GRADS);
        SGC_LAUNCH_CHECK();
    }
    return SGC_OK;
}

#define SGC_NORM_DISPATCH(call, ...)                                                                       \
    (o->dtype == SGC_F32                                                                                   \
         ? call<float, float>(__VA_ARGS__)                                                                 \
         : o->dtype == SGC_BF16                                                                            \
               ? (o->wdtype == SGC_F32 ? call<bf16_t, float>(__VA_ARGS__) : call<bf16_t, bf16_t>(__VA_ARGS__)) \
               : (o->wdtype == SGC_F32 ? call<f16_t, float>(__VA_ARGS__) : call<f16_t, f16_t>(__VA_ARGS__)))

}  // namespace sgc

using namespace sgc;

extern "C" int sgc_layer_norm(const sgc_norm_opts* o, const void* x, int64_t x_stride, const void* weight,
                              const void* bias, void* y, int64_t y_stride, float* mean, float* rstd,
                              sgc_stream_t stream)
{
    if (!norm_opts_ok(o) || o->flags) return SGC_EINVAL;
    if (o->rows == 0) return SGC_OK;
    if (!lm_rows_ok(x, x_stride, o->rows, o->cols, o->dtype, false)) return SGC_EINVAL;
    if (!lm_rows_ok(y, y_stride, o->rows, o->cols, o->dtype, true)) return SGC_EINVAL;
    const int64_t wa = lm_size(o->wdtype);
    if (!lm_aligned(weight, wa) || !lm_aligned(bias, wa) || !lm_aligned(mean, 4) || !lm_aligned(rstd, 4))
        return SGC_EINVAL;
    return SGC_NORM_DISPATCH(norm_forward, o, x, x_stride, weight, bias, y, y_stride, mean, rstd, (hipStream_t)stream);
}

extern "C" size_t sgc_layer_norm_backward_workspace(const sgc_norm_opts* o)
{
    if (!norm_opts_ok(o)) return 0;
    Carver c(nullptr);
    c.take<float>(2 * norm_parts(o) * o->cols);
    return c.off;
}

extern "C" int sgc_layer_norm_backward(const sgc_norm_opts* o, const void* dy, int64_t dy_stride, const void* x,
                                       int64_t x_stride, const void* weight, const float* mean, const float* rstd,
                                       void* dx, int64_t dx_stride, float* dweight, float* dbias, void* ws,
                                       size_t ws_bytes, sgc_stream_t stream)
{
    if (!norm_opts_ok(o)) return SGC_EINVAL;
    if (!lm_aligned(dweight, 4) || !lm_aligned(dbias, 4) || !lm_aligned(weight, lm_size(o->wdtype))) return SGC_EINVAL;
    if (o->rows) {
        if (!lm_rows_ok(dy, dy_stride, o->rows, o->cols, o->dtype, false)) return SGC_EINVAL;
        if (!lm_rows_ok(x, x_stride, o->rows, o->cols, o->dtype, false)) return SGC_EINVAL;
        if (dx && !lm_rows_ok(dx, dx_stride, o->rows, o->cols, o->dtype, true)) return SGC_EINVAL;
        if (!mean || !rstd || !lm_aligned(mean, 4) || !lm_aligned(rstd, 4)) return SGC_EINVAL;
    }
    float* part = nullptr;
    if (dweight || dbias) {
        if (!ws || ws_bytes < sgc_layer_norm_backward_workspace(o)) return SGC_ENOSPC;
        if (!aligned16(ws)) return SGC_EINVAL;
        Carver c(ws);
        part = c.take<float>(2 * norm_parts(o) * o->cols);
    }
    return SGC_NORM_DISPATCH(norm_backward, o, dy, dy_stride, x, x_stride, weight, mean, rstd, dx, dx_stride, dweight,
                             dbias, part, (hipStream_t)stream);
}
