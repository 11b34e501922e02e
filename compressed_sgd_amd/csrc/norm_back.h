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
    // a vector of a row on its way, and its values
    struct Held {
        Raw v;
    };
    template <bool RAG>
    __device__ Held load(int64_t r, int v, int cols, bool once) const
    {
        return {load_vec<T, RAG>(p + r * stride, v, cols, once)};
    }
    template <bool RAG>
    __device__ static void values(Held& h, int v, int cols, float* x)
    {
        settle<T, RAG>(h.v, v, cols);
        unpack<T>(h.v, x);
    }
};
template <typename T>
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
    // groups are of 32 or more: a vector has one scale
    static constexpr int VL = VecLen<T>::value;
    struct Held {
        Bytes<VL> b;
        float scale;
    };
    template <bool RAG>
    __device__ Held load(int64_t r, int v, int cols, bool once) const
    {
        return {load_bytes<VL, RAG>(q + r * stride, v, cols), v * VL < cols ? scale[r * groups + (v * VL >> shift)] : 0.f};
    }
    template <bool RAG>
    __device__ static void values(Held& h, int v, int cols, float* x)
    {
        settle<VL, RAG>(h.b, v, cols);
#pragma unroll
        for (int e = 0; e < VL; ++e) x[e] = byte_of(h.b.w[e / 4], e % 4) * h.scale;
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
    // where the sums over the rows go: by way of part and k_norm_join, or from one
    // workgroup straight
    float *dw, *db;
    bool add;
};

template <typename T>
__device__ inline float weight_at(const void* w, bool w32, int c, float none)
{
    return !w ? none : w32 ? ((const float*)w)[c] : to_f(((const T*)w)[c]);
}

// ------------------------------------------------------- rows in registers
// A workgroup takes row after row, its columns' weights and their gradients' sums
// in registers; part [workgroups, sums, cols].  Bound by memory: 16384 x 4096 bf16
// with dsum 91 us (5.9 TB/s), from 8 bits and with y 98 us (6.2 TB/s); 20001 x 650
// fp32, layer norm from 8 bits with y, 33 us (5.1 TB/s).
// MOST: threads of a workgroup at most.  16 waves a compute unit have 128
// registers each.  Where a row has more than 8 waves a layer norm's bias, and at 16
// elements a thread the weights, lie in shared memory, each thread's own, and are
// read again in every row (volatile: else they move back into registers); even so
// a layer norm's rows of 16 elements a thread spill, and an RMS norm's in fp32 or
// where they are ragged (4000 x 16384 from 8 bits: RMS norm bf16 102 us, layer norm
// bf16 156, fp32 396).
typedef float Four __attribute__((ext_vector_type(4)));
template <typename T, typename X, bool LAYER, int LANES, int EPT, bool RAG, int MOST>
__global__ __launch_bounds__(MOST, 4) void k_back(X x, Back k, int waves, int side,
                                                                             bool once)
{
    constexpr int VL = VecLen<T>::value, NV = EPT / VL;
    __shared__ RowJoin tmp;
    if (LANES == 64 && waves > 1) clear_join(tmp);
    const RowPlace<LANES> place(waves);
    const int sub = place.sub, t = place.t, across = place.across, cols = k.cols;
    constexpr bool kW = EPT == 16, kB = LAYER && MOST == 1024;
    __shared__ Four ws[kW ? EPT / 4 : 1][kW ? MOST : 1], bs[kB ? EPT / 4 : 1][kB ? MOST : 1];
    float wh[EPT], bh[EPT], aw[EPT], ab[EPT];
    row_weights<T, NV>(k.w, k.w32, across, t, cols, 1.f, wh);
    if (LAYER) row_weights<T, NV>(k.b, k.w32, across, t, cols, 0.f, bh);
#pragma unroll
    for (int i = 0; i < EPT; i += 4) {
        if constexpr (kW) ws[i / 4][threadIdx.x] = Four{wh[i], wh[i + 1], wh[i + 2], wh[i + 3]};
        if constexpr (kB) bs[i / 4][threadIdx.x] = Four{bh[i], bh[i + 1], bh[i + 2], bh[i + 3]};
    }
    const auto weights = [&](int i) {
        if constexpr (kW) return *(volatile Four*)&ws[i / 4][threadIdx.x];
        else return Four{wh[i], wh[i + 1], wh[i + 2], wh[i + 3]};
    };
    const auto biases = [&](int i) {
        if constexpr (kB) return *(volatile Four*)&bs[i / 4][threadIdx.x];
        else return Four{bh[i], bh[i + 1], bh[i + 2], bh[i + 3]};
    };
#pragma unroll
    for (int i = 0; i < EPT; ++i) aw[i] = ab[i] = 0.f;
    typename X::Held nx[NV] = {};
    Raw ny[NV] = {}, ns[NV] = {};
    float nm = 0.f, nr = 0.f;
    int64_t r = (int64_t)blockIdx.x * side + sub;
    const int64_t step = (int64_t)gridDim.x * side;
    // at 16 elements a thread there are no registers for the next row's
    constexpr bool kAhead = EPT < 16;
    const auto fetch = [&](int64_t at) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            nx[n] = x.template load<RAG>(at, n * across + t, cols, once);
            ny[n] = load_vec<T, RAG>((const T*)k.dy + at * k.dys, n * across + t, cols, once);
        }
        if (kAhead && k.dsum) {
#pragma unroll
            for (int n = 0; n < NV; ++n)
                ns[n] = load_vec<T, RAG>((const T*)k.dsum + at * k.dss, n * across + t, cols, once);
        }
        if (LAYER) nm = k.mean[at];
        nr = k.rstd[at];
    };
    if (kAhead && r < k.rows) fetch(r);
    int turn = 0;
    for (; r - sub < k.rows; r += step, turn ^= 1) {
        const bool live = r < k.rows;
        if (!kAhead && live) fetch(r);
        float h[EPT], g[EPT];
        Raw ds[NV] = {};
        const float m = live && LAYER ? nm : 0.f, rs = live ? nr : 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            X::template values<RAG>(nx[n], n * across + t, cols, h + n * VL);
            settle<T, RAG>(ny[n], n * across + t, cols);
            unpack<T>(ny[n], g + n * VL);
            if (kAhead) ds[n] = ns[n];
        }
        if (!live) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) h[i] = g[i] = 0.f;
        }
        if (kAhead && r + step < k.rows) fetch(r + step);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {  // past cols dy is 0
            float y[VL];
#pragma unroll
            for (int i = n * VL; i < (n + 1) * VL; i += 4) {
                const Four w = weights(i);
                Four b = {0.f, 0.f, 0.f, 0.f};
                if (LAYER && k.y) b = biases(i);
#pragma unroll
                for (int e = i; e < i + 4; ++e) {
                    h[e] = (LAYER ? h[e] - m : h[e]) * rs;
                    y[e - n * VL] = LAYER ? fmaf(h[e], w[e - i], b[e - i]) : h[e] * w[e - i];
                    aw[e] = fmaf(g[e], h[e], aw[e]);
                    if (LAYER) ab[e] += g[e];
                    g[e] *= w[e - i];
                    if (LAYER) s1 += g[e];
                    s2 = fmaf(g[e], h[e], s2);
                }
            }
            if (k.y && live) store_vec<T, RAG>((T*)k.y + r * k.ys, n * across + t, cols, y, once);
        }
        if (!kAhead && live && k.dsum) {
#pragma unroll
            for (int n = 0; n < NV; ++n)
                ds[n] = load_vec<T, RAG>((const T*)k.dsum + r * k.dss, n * across + t, cols, once);
        }
        if (k.dx) {
            row_join<false, LANES>(s1, s2, tmp, turn, waves, sub);
            const float c1 = LAYER ? s1 / (float)cols : 0.f, c2 = s2 / (float)cols;
            if (live) {
#pragma unroll
                for (int i = 0; i < EPT; ++i) g[i] = rs * (g[i] - fmaf(h[i], c2, c1));
                if (k.dsum) {
#pragma unroll
                    for (int n = 0; n < NV; ++n) {
                        float d[VL];
                        settle<T, RAG>(ds[n], n * across + t, cols);
                        unpack<T>(ds[n], d);
#pragma unroll
                        for (int e = 0; e < VL; ++e) g[n * VL + e] += d[e];
                    }
                }
#pragma unroll
                for (int n = 0; n < NV; ++n)
                    store_vec<T, RAG>((T*)k.dx + r * k.dxs, n * across + t, cols, g + n * VL, once);
            }
        }
    }
    if (!k.part) return;
    // the rows side by side in a wave, then those (or the waves) side by side in
    // the workgroup, one after the other
    constexpr bool kFold = LANES < 64;
    constexpr int kSums = LAYER ? 2 : 1;
    if (kFold) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
#pragma unroll
            for (int d = LANES; d < 64; d <<= 1) {
                aw[i] += __shfl_xor(aw[i], d, 64);
                if (LAYER) ab[i] += __shfl_xor(ab[i], d, 64);
            }
        }
    }
    const int at = kFold ? threadIdx.x >> 6 : sub, beside = kFold ? 8 : side;
    const bool mine = !kFold || (threadIdx.x & 63) < LANES;
    // rows side by side have 4 waves at most
    __shared__ float sw[kSums][EPT * (kFold ? LANES : EPT <= 8 ? 256 : 1)];
    if (beside > 1) {
        for (int o = beside - 1; o > 0; --o) {
            __syncthreads();
            if (at == o && mine) {
#pragma unroll
                for (int i = 0; i < EPT; ++i) {
                    if (o < beside - 1) {
                        aw[i] += sw[0][i * across + t];
                        if (LAYER) ab[i] += sw[kSums - 1][i * across + t];
                    }
                    sw[0][i * across + t] = aw[i];
                    if (LAYER) sw[kSums - 1][i * across + t] = ab[i];
                }
            }
        }
        __syncthreads();
        if (at || !mine) return;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            aw[i] += sw[0][i * across + t];
            if (LAYER) ab[i] += sw[kSums - 1][i * across + t];
        }
    }
    if (gridDim.x == 1) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const int c = (i / VL * across + t) * VL + i % VL;
            if (c >= cols) continue;
            if (k.dw) k.dw[c] = k.add ? k.dw[c] + aw[i] : aw[i];
            if (LAYER && k.db) k.db[c] = k.add ? k.db[c] + ab[i] : ab[i];
        }
        return;
    }
    float* p = k.part + kSums * (int64_t)blockIdx.x * cols;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int e = 0; e < VL; e += 4) {
            const int v = (n * across + t) * (VL / 4) + e / 4;
            store_raw<float, RAG, false>(p, v, cols, aw + n * VL + e);
            if (LAYER) store_raw<float, RAG, false>(p + cols, v, cols, ab + n * VL + e);
        }
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
    if (cols > kNormHeld) return rows < 64 ? rows : 64;
    const RowShape sh = row_shape(cols, dtype);
    return row_groups(sh, rows, kBackwardWaves);
}

template <typename T, typename X, bool LAYER, int LANES, int EPT>
static void back_held(const X& x, const Back& k, const RowShape& sh, unsigned g, bool once, hipStream_t s)
{
    const bool rag = k.cols % VecLen<T>::value;
    if constexpr (EPT <= 8) {
        if (sh.threads() <= 512) {
            if (rag) k_back<T, X, LAYER, LANES, EPT, true, 512><<<g, sh.threads(), 0, s>>>(x, k, sh.waves, sh.rows, once);
            else k_back<T, X, LAYER, LANES, EPT, false, 512><<<g, sh.threads(), 0, s>>>(x, k, sh.waves, sh.rows, once);
            return;
        }
    }
    if constexpr (LANES == 64 && EPT >= 8) {
        if (rag) k_back<T, X, LAYER, LANES, EPT, true, 1024><<<g, sh.threads(), 0, s>>>(x, k, sh.waves, sh.rows, once);
        else k_back<T, X, LAYER, LANES, EPT, false, 1024><<<g, sh.threads(), 0, s>>>(x, k, sh.waves, sh.rows, once);
    }
}

template <typename T, typename X, bool LAYER>
static int norm_back(const X& x, const Back& k, int32_t dtype, hipStream_t s)
{
    const int64_t parts = back_parts(k.rows, k.cols, dtype);
    const bool straight = k.cols <= kNormHeld && parts == 1;
    if (k.rows && k.cols > kNormHeld) {
        if (k.part) {  // before dx, which may take dy's or the input's place
            k_back_long_dw<T, X, LAYER><<<dim3((unsigned)cdiv(k.cols, 256), (unsigned)parts), 256, 0, s>>>(x, k);
            SGC_LAUNCH_CHECK();
        }
        if (k.dx || k.y) {
            k_back_long<T, X, LAYER><<<row_grid(k.rows), kLongThreads, 0, s>>>(x, k);
            SGC_LAUNCH_CHECK();
        }
    } else if (k.rows && (k.part || k.dx || k.y)) {
        const unsigned g = (unsigned)parts;
        const int64_t moved = 2 + (k.dsum != nullptr) + (k.dx != nullptr) + (k.y != nullptr);
        const bool once = k.rows * k.cols * moved * (int64_t)sizeof(T) >= kCacheBytes;
        const RowShape sh = row_shape(k.cols, dtype);
        if (sh.lanes == 16) back_held<T, X, LAYER, 16, 8>(x, k, sh, g, once, s);
        else if (sh.lanes == 32) back_held<T, X, LAYER, 32, 8>(x, k, sh, g, once, s);
        else if (sh.ept == 8) back_held<T, X, LAYER, 64, 8>(x, k, sh, g, once, s);
        else if (sh.ept == 4) {
            if constexpr (sizeof(T) == 4) back_held<T, X, LAYER, 64, 4>(x, k, sh, g, once, s);
        }
        else back_held<T, X, LAYER, 64, 16>(x, k, sh, g, once, s);
        SGC_LAUNCH_CHECK();
    }
    if (k.part && !straight) {
        const int64_t width = (LAYER ? 2 : 1) * (int64_t)k.cols;
        k_norm_join<<<(unsigned)cdiv(width, kJoinCols), kJoinCols * kJoinDeep, 0, s>>>(k.part, parts, width, k.cols,
                                                                                        k.dw, k.db, k.add);
        SGC_LAUNCH_CHECK();
    }
    return SGC_OK;
}

}  // namespace sgc
