// norm_back.h -- the backward pass of an RMS norm or a layer norm, from the
// norm's input as it was (rms_norm.hip) or as 8 bits hold it (norm_q8.hip).
//
//   xh = (x - mean) rstd (no mean in an RMS norm),  v = dy w
//   dx = rstd (v - mean(v) - xh mean(v xh)) + dsum  (no mean(v) in an RMS norm)
//   dw = sum_rows dy xh,  db = sum_rows dy,  y = xh w + b
#pragma once

#include "lm_norm.h"
#include "lm_q8.h"

namespace sgc {

// Where the norm's input comes from.
template <typename T>
struct AsIs {
    const T* p;
    int64_t stride;
    __device__ float at(int64_t r, int c) const { return to_f(p[r * stride + c]); }
};
struct As8Bits {
    const int8_t* q;
    int64_t stride;
    const float* scale;
    int64_t groups;
    int shift;
    __device__ float at(int64_t r, int c) const
    {
        return (float)q[r * stride + c] * scale[r * groups + (c >> shift)];
    }
};

// What a backward call reads and writes beside the norm's input.
struct Back {
    const void* dy;
    int64_t dys;
    const void *w, *b;
    bool w32;
    const float *mean, *rstd;
    const void* dsum;
    int64_t dss;
    void* dx;
    int64_t dxs;
    void* y;
    int64_t ys;
    float* part;
    int64_t rows;
    int cols;
};

template <typename T>
__device__ inline float weight_at(const void* w, bool w32, int c, float none)
{
    return !w ? none : w32 ? ((const float*)w)[c] : to_f(((const T*)w)[c]);
}

// ------------------------------------------------- rows that are not held
template <typename T, typename X, bool LAYER>
__global__ __launch_bounds__(kLongThreads) void k_back_long(X x, Back k)
{
    __shared__ float tmp[kLongWaves];
    const int64_t r = row_of_block();
    if (r >= k.rows) return;
    const T* dy = (const T*)k.dy + r * k.dys;
    const T* dsum = k.dsum ? (const T*)k.dsum + r * k.dss : nullptr;
    T* dx = k.dx ? (T*)k.dx + r * k.dxs : nullptr;
    T* y = k.y ? (T*)k.y + r * k.ys : nullptr;
    const float m = LAYER ? k.mean[r] : 0.f, rs = k.rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < k.cols; c += kLongThreads) {
        const float w = weight_at<T>(k.w, k.w32, c, 1.f), h = (x.at(r, c) - m) * rs;
        const float v = to_f(dy[c]) * w;
        s1 += v;
        s2 = fmaf(v, h, s2);
        if (y) y[c] = from_f<T>(LAYER ? fmaf(h, w, weight_at<T>(k.b, k.w32, c, 0.f)) : h * w);
    }
    if (!dx) return;
    const float c1 = LAYER ? block_sum<kLongWaves>(s1, tmp) / (float)k.cols : 0.f;
    const float c2 = block_sum<kLongWaves>(s2, tmp) / (float)k.cols;
    for (int c = threadIdx.x; c < k.cols; c += kLongThreads) {
        const float v = to_f(dy[c]) * weight_at<T>(k.w, k.w32, c, 1.f);
        const float h = (x.at(r, c) - m) * rs;
        const float d = rs * (v - fmaf(h, c2, c1));
        dx[c] = from_f<T>(dsum ? d + to_f(dsum[c]) : d);
    }
}

// Sums over the rows part, part + parts, ... of 256 columns.
template <typename T, typename X, bool LAYER>
__global__ __launch_bounds__(256) void k_back_long_dw(X x, Back k)
{
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= k.cols) return;
    float aw = 0.f, ab = 0.f;
    for (int64_t r = blockIdx.y; r < k.rows; r += gridDim.y) {
        const float g = to_f(((const T*)k.dy)[r * k.dys + c]);
        aw = fmaf(g, (x.at(r, (int)c) - (LAYER ? k.mean[r] : 0.f)) * k.rstd[r], aw);
        ab += g;
    }
    constexpr int kSums = LAYER ? 2 : 1;
    float* p = k.part + kSums * (int64_t)blockIdx.y * k.cols + c;
    p[0] = aw;
    if (LAYER) p[k.cols] = ab;
}

inline int64_t back_parts(int64_t rows, int64_t cols, int32_t dtype)
{
    return rows < 64 ? rows : 64;
}

template <typename T, typename X, bool LAYER>
static int norm_back(const X& x, const Back& k, int32_t dtype, float* dw, float* db, bool add, hipStream_t s)
{
    const int64_t parts = back_parts(k.rows, k.cols, dtype);
    if (k.rows) {
        if (k.part) {  // before dx, which may take dy's or the input's place
            k_back_long_dw<T, X, LAYER><<<dim3((unsigned)cdiv(k.cols, 256), (unsigned)parts), 256, 0, s>>>(x, k);
            SGC_LAUNCH_CHECK();
        }
        if (k.dx || k.y) {
            k_back_long<T, X, LAYER><<<row_grid(k.rows), kLongThreads, 0, s>>>(x, k);
            SGC_LAUNCH_CHECK();
        }
    }
    if (k.part) {
        const int64_t width = (LAYER ? 2 : 1) * (int64_t)k.cols;
        k_norm_join<<<(unsigned)cdiv(width, kJoinCols), kJoinCols * kJoinDeep, 0, s>>>(k.part, parts, width, k.cols,
                                                                                        dw, db, add);
        SGC_LAUNCH_CHECK();
    }
    return SGC_OK;
}

}  // namespace sgc
