// q8.hip -- rows kept in 8 bits with a scale a group, and read back.
#include "lm_norm.h"
#include "lm_q8.h"

namespace sgc {

// A wave takes group after group of a row.
template <typename T>
__global__ __launch_bounds__(256) void k_quantize(const T* x, int64_t xs, int8_t* q, int64_t qs, float* scale,
                                                  int64_t rows, int cols, int group, int64_t groups)
{
    const int64_t r = row_of_block();
    if (r >= rows) return;
    const int lane = threadIdx.x & 63;
    for (int64_t g = threadIdx.x >> 6; g < groups; g += 4) {
        const int a = (int)g * group, b = a + group < cols ? a + group : cols;
        uint32_t top = 0;
        for (int c = a + lane; c < b; c += 64) top = umax(top, magnitude(to_f(x[r * xs + c])));
        for (int d = 1; d < 64; d <<= 1) top = umax(top, (uint32_t)__shfl_xor((int)top, d, 64));
        const Quant k = quant_of(top);
        if (lane == 0) scale[r * groups + g] = k.scale;
        for (int c = a + lane; c < b; c += 64) q[r * qs + c] = (int8_t)(quantized(to_f(x[r * xs + c]), k) & k.keep);
    }
}

template <typename T>
__global__ __launch_bounds__(256) void k_dequantize(const int8_t* q, int64_t qs, const float* scale, T* x, int64_t xs,
                                                    int64_t rows, int cols, int shift, int64_t groups)
{
    const int64_t r = row_of_block();
    if (r >= rows) return;
    for (int c = threadIdx.x; c < cols; c += 256)
        x[r * xs + c] = from_f<T>((float)q[r * qs + c] * scale[r * groups + (c >> shift)]);
}

static bool q8_ok(const sgc_q8_opts* o)
{
    return o && o->rows >= 0 && o->rows < ((int64_t)1 << 31) && o->cols >= 1 && o->cols <= kNormMaxCols &&
           lm_dtype(o->dtype) && q8_group_ok(o->group);
}

template <typename T>
static int quantize(const sgc_q8_opts* o, const void* x, int64_t xs, int8_t* q, int64_t qs, float* scale,
                    hipStream_t s)
{
    const int cols = (int)o->cols;
    k_quantize<T><<<row_grid(o->rows), 256, 0, s>>>((const T*)x, xs, q, qs, scale, o->rows, cols,
                                                    o->group ? o->group : cols, q8_groups(cols, o->group));
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}
template <typename T>
static int dequantize(const sgc_q8_opts* o, const int8_t* q, int64_t qs, const float* scale, void* x, int64_t xs,
                      hipStream_t s)
{
    const int cols = (int)o->cols;
    k_dequantize<T><<<row_grid(o->rows), 256, 0, s>>>(q, qs, scale, (T*)x, xs, o->rows, cols, q8_shift(o->group),
                                                      q8_groups(cols, o->group));
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
