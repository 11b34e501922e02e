// norm_q8.hip -- the backward pass of a norm whose input was kept in 8 bits
// (norm_back.h), and the norm's output once more.
#include "norm_back.h"

namespace sgc {

static bool norm_q8_ok(const sgc_norm_q8_opts* o)
{
    return o && o->rows >= 0 && o->rows < ((int64_t)1 << 31) && o->cols >= 1 && o->cols <= kNormMaxCols &&
           lm_dtype(o->dtype) && (o->wdtype == SGC_F32 || o->wdtype == o->dtype) && q8_group_ok(o->group) &&
           (o->kind == SGC_NORM_LAYER || o->kind == SGC_NORM_RMS) && (o->flags & ~SGC_NORM_ADD_GRADS) == 0 &&
           o->reserved == 0;
}

template <typename T>
static int norm_back_8(const sgc_norm_q8_opts* o, const int8_t* q, int64_t qs, const float* scale, const Back& k,
                       hipStream_t s)
{
    const As8Bits<T> x = {q, qs, scale, q8_groups(o->cols, o->group), q8_shift(o->group)};
    return o->kind == SGC_NORM_LAYER ? norm_back<T, As8Bits<T>, true>(x, k, o->dtype, s)
                                     : norm_back<T, As8Bits<T>, false>(x, k, o->dtype, s);
}

}  // namespace sgc

using namespace sgc;

extern "C" size_t sgc_norm_backward_q8_workspace(const sgc_norm_q8_opts* o)
{
    if (!norm_q8_ok(o)) return 0;
    Carver c(nullptr);
    c.take<float>(back_parts(o->rows, o->cols, o->dtype) * o->cols * (o->kind == SGC_NORM_LAYER ? 2 : 1));
    return c.off;
}

extern "C" int sgc_norm_backward_q8(const sgc_norm_q8_opts* o, const void* dy, int64_t dy_stride, const int8_t* q,
                                    int64_t q_stride, const float* scale, const void* weight, const void* bias,
                                    const float* mean, const float* rstd, const void* dsum, int64_t dsum_stride,
                                    void* dx, int64_t dx_stride, void* y, int64_t y_stride, float* dweight,
                                    float* dbias, void* ws, size_t ws_bytes, sgc_stream_t stream)
{
    if (!norm_q8_ok(o)) return SGC_EINVAL;
    const bool layer = o->kind == SGC_NORM_LAYER;
    const int64_t wa = lm_size(o->wdtype);
    if (!lm_aligned(dweight, 4) || !lm_aligned(dbias, 4) || !lm_aligned(weight, wa) || !lm_aligned(bias, wa))
        return SGC_EINVAL;
    if (!layer && (mean || bias || dbias)) return SGC_EINVAL;
    if (o->rows) {
        const int64_t n = o->rows, c = o->cols;
        if (!lm_rows_ok(dy, dy_stride, n, c, o->dtype, false) || !q8_rows_ok(q, q_stride, n, c, false))
            return SGC_EINVAL;
        if (dsum && !lm_rows_ok(dsum, dsum_stride, n, c, o->dtype, false)) return SGC_EINVAL;
        if (dx && !lm_rows_ok(dx, dx_stride, n, c, o->dtype, true)) return SGC_EINVAL;
        if (y && !lm_rows_ok(y, y_stride, n, c, o->dtype, true)) return SGC_EINVAL;
        if (!scale || !rstd || (layer && !mean)) return SGC_EINVAL;
        if (!lm_aligned(scale, 4) || !lm_aligned(rstd, 4) || !lm_aligned(mean, 4)) return SGC_EINVAL;
        if (y && (y == dx || y == dy || y == dsum)) return SGC_EINVAL;
    }
    float* part = nullptr;
    if (dweight || dbias) {
        if (!ws || ws_bytes < sgc_norm_backward_q8_workspace(o)) return SGC_ENOSPC;
        if (!aligned16(ws)) return SGC_EINVAL;
        part = Carver(ws).take<float>(1);
    }
    const Back k = {dy, dy_stride, weight, bias,     o->wdtype == SGC_F32, mean,    rstd, dsum, dsum_stride,
                    dx, dx_stride, y,      y_stride, part,                 o->rows, (int)o->cols,
                    dweight, dbias, (o->flags & SGC_NORM_ADD_GRADS) != 0};
    const hipStream_t s = (hipStream_t)stream;
    return o->dtype == SGC_F32    ? norm_back_8<float>(o, q, q_stride, scale, k, s)
           : o->dtype == SGC_BF16 ? norm_back_8<bf16_t>(o, q, q_stride, scale, k, s)
                                  : norm_back_8<f16_t>(o, q, q_stride, scale, k, s);
}
