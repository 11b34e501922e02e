// int8_linear.hip -- product of 8-bit rows with a scale for each token and each
// channel: y = (sum xq wq) xscale wscale + bias.
#include "lm_q8.h"

namespace sgc {

struct Product {
    const int8_t* x;
    int64_t xs;
    const float* xscale;
    const int8_t* w;
    int64_t ws;
    const float *wscale, *bias;
    void* y;
    int64_t ys;
    int64_t rows, out;
    int width;
};

// The sum is a whole number below 2^31; one fp32 rounding of it, one for each
// scale, one for the bias, one to the output's type.
template <typename T>
__device__ inline T product_out(int32_t sum, float xscale, float wscale, float bias)
{
    return from_f<T>((float)sum * xscale * wscale + bias);
}

template <typename T>
__global__ __launch_bounds__(256) void k_product(Product k)
{
    const int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (o >= k.out) return;
    for (int64_t r = blockIdx.y; r < k.rows; r += gridDim.y) {
        int32_t sum = 0;
        for (int i = 0; i < k.width; ++i) sum += (int)k.x[r * k.xs + i] * (int)k.w[o * k.ws + i];
        ((T*)k.y)[r * k.ys + o] = product_out<T>(sum, k.xscale[r], k.wscale[o], k.bias ? k.bias[o] : 0.f);
    }
}

template <typename T>
static int product(const Product& k, hipStream_t s)
{
    const dim3 grid((unsigned)cdiv(k.out, 256), (unsigned)(k.rows < 65535 ? k.rows : 65535));
    k_product<T><<<grid, 256, 0, s>>>(k);
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}

}  // namespace sgc

using namespace sgc;

extern "C" int sgc_int8_linear(const sgc_int8_opts* o, const int8_t* xq, int64_t xq_stride, const float* xscale,
                               const int8_t* wq, int64_t wq_stride, const float* wscale, const float* bias, void* y,
                               int64_t y_stride, sgc_stream_t stream)
{
    if (!o || o->rows < 0 || o->rows >= ((int64_t)1 << 31) || o->width < 1 || o->width >= (1 << 17) || o->out < 1 ||
        o->out >= ((int64_t)1 << 31) || !lm_dtype(o->dtype) || o->reserved)
        return SGC_EINVAL;
    if (o->rows == 0) return SGC_OK;
    if (!q8_rows_ok(xq, xq_stride, o->rows, o->width, false) || !q8_rows_ok(wq, wq_stride, o->out, o->width, false))
        return SGC_EINVAL;
    if (!lm_rows_ok(y, y_stride, o->rows, o->out, o->dtype, true) || !xscale || !wscale) return SGC_EINVAL;
    if (!lm_aligned(xscale, 4) || !lm_aligned(wscale, 4) || !lm_aligned(bias, 4)) return SGC_EINVAL;
    const Product k = {xq, xq_stride, xscale, wq, wq_stride, wscale, bias, y, y_stride, o->rows, o->out,
                       (int)o->width};
    const hipStream_t s = (hipStream_t)stream;
    return o->dtype == SGC_F32    ? product<float>(k, s)
           : o->dtype == SGC_BF16 ? product<bf16_t>(k, s)
                                  : product<f16_t>(k, s);
}
