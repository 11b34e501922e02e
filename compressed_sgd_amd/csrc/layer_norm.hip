// layer_norm.hip -- layer norm over the last dimension, forward and backward,
// with the sums over the rows that are the gradients of weight and bias.
//
//   y  = (x - mean) rstd w + b
//   dx = rstd (v - mean(v) - xh mean(v xh)),  v = dy w,  xh = (x - mean) rstd
//   dw = sum_rows dy xh,  db = sum_rows dy
//
// A row stays in registers between its sums and its output: it is read once.
// NTR threads share a row, EPT elements each; RPB rows go through a
// workgroup side by side, and a workgroup takes row after row, so that its
// columns' weights are loaded once and their gradients' sums stay in its
// registers; the next rows are on their way while one is worked on.  Rows too
// long for that (over kNormHeld elements) are read again for every pass.
#include "lm_common.h"

namespace sgc {

constexpr int64_t kNormHeld = 16384;
constexpr int64_t kCus = 256;
// Waves that a compute unit holds of the forward and the backward kernel.
constexpr int kForwardWaves = 32, kBackwardWaves = 16;

// Elements [v VL, v VL + VL) of a row that ends at cols; past it 0.  RAG: cols
// may be no multiple of VL.
template <typename T, bool RAG, bool ONCE>
__device__ inline Raw load_raw(const T* p, int v, int cols)
{
    constexpr int VL = VecLen<T>::value;
    if ((v + 1) * VL <= cols) return load_row<ONCE>((const Raw*)p + v);
    Raw q = {{0, 0, 0, 0}};
    if (RAG && v * VL < cols) {
        float x[VL];
#pragma unroll
        for (int e = 0; e < VL; ++e) x[e] = v * VL + e < cols ? to_f(p[v * VL + e]) : 0.f;
        q = pack<T>(x);
    }
    return q;
}
template <typename T, bool RAG, bool ONCE>
__device__ inline void store_raw(T* p, int v, int cols, const float* x)
{
    constexpr int VL = VecLen<T>::value;
    if ((v + 1) * VL <= cols) {
        store_row<ONCE>((Raw*)p + v, pack<T>(x));
    } else if (RAG && v * VL < cols) {
#pragma unroll
        for (int e = 0; e < VL; ++e)
            if (v * VL + e < cols) p[v * VL + e] = from_f<T>(x[e]);
    }
}
// EPT columns of a thread's weights as fp32; `none` where there are none.
template <typename T, int NV, int NTR>
__device__ inline void load_weights(const void* w, bool w32, int t, int cols, float none, float* out)
{
    constexpr int VL = VecLen<T>::value;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int v = n * NTR + t;
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

// A row's place among the RPB of its workgroup.
template <int NTR>
__device__ inline int row_place()
{
    const int sub = threadIdx.x / NTR;
    return NTR < 64 ? sub : __builtin_amdgcn_readfirstlane(sub);
}

// Two sums over the NTR threads of a row: 16 lanes, or whole waves with one
// barrier; tmp is another half at every other call (`turn`), so the next call
// may write while this one reads.
template <int NTR, int RPB>
using RowTmp = float[2][RPB][NTR < 64 ? 1 : NTR / 64][2];
template <int NTR, int RPB>
__device__ inline void row_sums(float& a, float& b, RowTmp<NTR, RPB>& tmp, int turn)
{
    if constexpr (NTR == 16) {
        a = row16_sum(a);
        b = row16_sum(b);
    } else {
        constexpr int NWR = NTR / 64;
        a = wave_sum(a);
        b = wave_sum(b);
        if (NWR == 1) return;
        const int wave = threadIdx.x >> 6, sub = wave / NWR, w = wave % NWR;
        if ((threadIdx.x & 63) == 0) {
            tmp[turn][sub][w][0] = a;
            tmp[turn][sub][w][1] = b;
        }
        __syncthreads();
        a = sum_of_lanes<NWR>(tmp[turn][sub][threadIdx.x % NWR][0]);
        b = sum_of_lanes<NWR>(tmp[turn][sub][threadIdx.x % NWR][1]);
    }
}

// The variance is summed from the differences to the mean, which costs nothing
// where the row is held.  Bound by memory: 16384 x 4096 bf16 51 us, 5.2 TB/s; 8
// x 1024 2.8 us.
template <typename T, int NTR, int EPT, int RPB, bool RAG, bool ONCE>
__global__ __launch_bounds__(NTR* RPB) void k_norm(const T* x, int64_t xs, const void* w, const void* b,
                                                   bool w32, T* y, int64_t ys, float* mean, float* rstd, int64_t rows,
                                                   int cols, float eps)
{
    constexpr int VL = VecLen<T>::value, NV = EPT / VL;
    __shared__ RowTmp<NTR, RPB> tmp;
    const int sub = row_place<NTR>(), t = threadIdx.x % NTR;
    float wf[EPT], bf[EPT];
    load_weights<T, NV, NTR>(w, w32, t, cols, 1.f, wf);
    load_weights<T, NV, NTR>(b, w32, t, cols, 0.f, bf);
    Raw next[NV] = {};
    int64_t r = (int64_t)blockIdx.x * RPB + sub;
    const int64_t step = (int64_t)gridDim.x * RPB;
    if (r < rows) {
#pragma unroll
        for (int n = 0; n < NV; ++n) next[n] = load_raw<T, RAG, ONCE>(x + r * xs, n * NTR + t, cols);
    }
    for (; r - sub < rows; r += step) {
        float f[EPT];
#pragma unroll
        for (int n = 0; n < NV; ++n) unpack<T>(next[n], f + n * VL);
        if (r + step < rows) {
#pragma unroll
            for (int n = 0; n < NV; ++n) next[n] = load_raw<T, RAG, ONCE>(x + (r + step) * xs, n * NTR + t, cols);
        }
        float s = 0.f, q = 0.f, none = 0.f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) s += f[i];
        row_sums<NTR, RPB>(s, none, tmp, 0);
        const float m = s / (float)cols;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const float d = f[i] - m;
            f[i] = d;
            if ((i / VL * NTR + t) * VL + i % VL < cols) q = fmaf(d, d, q);
        }
        none = 0.f;
        row_sums<NTR, RPB>(q, none, tmp, 1);
        const float rs = 1.f / sqrtf(q / (float)cols + eps);
        if (r < rows) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) f[i] = fmaf(f[i] * rs, wf[i], bf[i]);
#pragma unroll
            for (int n = 0; n < NV; ++n) store_raw<T, RAG, ONCE>(y + r * ys, n * NTR + t, cols, f + n * VL);
            if (t == 0) {
                if (mean) mean[r] = m;
                if (rstd) rstd[r] = rs;
            }
        }
    }
}

// dx, and the workgroup's sums of dy xh and dy over its rows: part
// [workgroups, 2, cols], 16 MB for 4096 columns.  Bound by memory: 16384 x 4096
// bf16 70.7 us, 5.7 TB/s; 20001 x 650 fp32 32.9 us.  16 waves a compute unit:
// at 24 or 32 the registers spill (85 -> 91, 124 us).
template <typename T, int NTR, int EPT, int RPB, bool RAG, bool ONCE>
__global__ __launch_bounds__(NTR* RPB, kBackwardWaves / 4) void k_norm_back(const T* dy, int64_t dys, const T* x,
                                                                            int64_t xs, const void* w, bool w32,
                                                                            const float* mean, const float* rstd,
                                                                            T* dx, int64_t dxs, float* part,
                                                                            int64_t rows, int cols)
{
    constexpr int VL = VecLen<T>::value, NV = EPT / VL;
    __shared__ RowTmp<NTR, RPB> tmp;
    const int sub = row_place<NTR>(), t = threadIdx.x % NTR;
    float wf[EPT], aw[EPT], ab[EPT];
    load_weights<T, NV, NTR>(w, w32, t, cols, 1.f, wf);
#pragma unroll
    for (int i = 0; i < EPT; ++i) aw[i] = ab[i] = 0.f;
    Raw nx[NV] = {}, ny[NV] = {};
    float nm = 0.f, nr = 0.f;
    int64_t r = (int64_t)blockIdx.x * RPB + sub;
    const int64_t step = (int64_t)gridDim.x * RPB;
    const auto fetch = [&](int64_t at) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            nx[n] = load_raw<T, RAG, ONCE>(x + at * xs, n * NTR + t, cols);
            ny[n] = load_raw<T, RAG, ONCE>(dy + at * dys, n * NTR + t, cols);
        }
        nm = mean[at];
        nr = rstd[at];
    };
    // 16 elements a thread leave no registers for the next row's (128 of them at
    // 16 waves: fetched ahead they spill 108, as it is up to 43 in rows by one, two
    // or eight waves, 16384 x 4099 bf16 140 us)
    constexpr bool kAhead = EPT < 16;
    if (kAhead && r < rows) fetch(r);
    int turn = 0;
    for (; r - sub < rows; r += step, turn ^= 1) {
        const bool live = r < rows;
        if (!kAhead && live) fetch(r);
        float h[EPT], g[EPT];
        const float m = live ? nm : 0.f, rs = live ? nr : 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            unpack<T>(nx[n], h + n * VL);
            unpack<T>(ny[n], g + n * VL);
        }
        if (!live) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) h[i] = g[i] = 0.f;
        }
        if (kAhead && r + step < rows) fetch(r + step);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {  // past cols dy is 0
            h[i] = (h[i] - m) * rs;
            aw[i] = fmaf(g[i], h[i], aw[i]);
            ab[i] += g[i];
            g[i] *= wf[i];
            s1 += g[i];
            s2 = fmaf(g[i], h[i], s2);
        }
        if (dx) {
            row_sums<NTR, RPB>(s1, s2, tmp, turn);
            const float c1 = s1 / (float)cols, c2 = s2 / (float)cols;
            if (live) {
#pragma unroll
                for (int i = 0; i < EPT; ++i) g[i] = rs * (g[i] - fmaf(h[i], c2, c1));
#pragma unroll
                for (int n = 0; n < NV; ++n) store_raw<T, RAG, ONCE>(dx + r * dxs, n * NTR + t, cols, g + n * VL);
            }
        }
    }
    if (!part) return;
    // the rows side by side in a wave, then those (or the waves) side by side in
    // the workgroup, one after the other
    constexpr bool kFold = NTR < 64;
    constexpr int kSums = kFold ? NTR * RPB / 64 : RPB;
    if (kFold) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
#pragma unroll
            for (int d = NTR; d < 64; d <<= 1) {
                aw[i] += __shfl_xor(aw[i], d, 64);
                ab[i] += __shfl_xor(ab[i], d, 64);
            }
        }
    }
    const int at = kFold ? threadIdx.x >> 6 : sub;
    const bool mine = !kFold || (threadIdx.x & 63) < NTR;
    __shared__ float sw[2][kSums > 1 ? NTR * EPT : 1];
    if (kSums > 1) {
        for (int k = kSums - 1; k > 0; --k) {
            __syncthreads();
            if (at == k && mine) {
#pragma unroll
                for (int i = 0; i < EPT; ++i) {
                    if (k < kSums - 1) {
                        aw[i] += sw[0][i * NTR + t];
                        ab[i] += sw[1][i * NTR + t];
                    }
                    sw[0][i * NTR + t] = aw[i];
                    sw[1][i * NTR + t] = ab[i];
                }
            }
        }
        __syncthreads();
        if (at || !mine) return;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            aw[i] += sw[0][i * NTR + t];
            ab[i] += sw[1][i * NTR + t];
        }
    }
    float* p = part + 2 * (int64_t)blockIdx.x * cols;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int e = 0; e < VL; e += 4) {
            const int v = (n * NTR + t) * (VL / 4) + e / 4;
            store_raw<float, RAG, false>(p, v, cols, aw + n * VL + e);
            store_raw<float, RAG, false>(p + cols, v, cols, ab + n * VL + e);
        }
}

// The parts' sums: a workgroup takes 32 of the 2 cols columns, 32 threads each,
// eight parts in flight a thread.  512 parts of 4096 columns: 4.8 us.
constexpr int kJoinCols = 32, kJoinDeep = 32;
__global__ __launch_bounds__(kJoinCols* kJoinDeep) void k_norm_join(const float* part, int64_t parts, int64_t cols,
                                                                    float* dw, float* db, int add)
{
    __shared__ float tmp[kJoinDeep][kJoinCols];
    const int tc = threadIdx.x % kJoinCols, td = threadIdx.x / kJoinCols;
    const int64_t c = (int64_t)blockIdx.x * kJoinCols + tc;
    float s = 0.f;
    if (c < 2 * cols) {
#pragma unroll 8
        for (int64_t p = td; p < parts; p += kJoinDeep) s += part[2 * p * cols + c];
    }
    tmp[td][tc] = s;
    __syncthreads();
    if (td || c >= 2 * cols) return;
#pragma unroll
    for (int d = 1; d < kJoinDeep; ++d) s += tmp[d][tc];
    float* out = c < cols ? dw : db;
    const int64_t at = c < cols ? c : c - cols;
    if (out) out[at] = add ? out[at] + s : s;
}

// ------------------------------------------------- rows that are not held
// One workgroup of 16 waves a row, the row read again for every pass (from the
// cache); the sums over the rows in a kernel of their own.
constexpr int kLongThreads = 1024, kLongWaves = kLongThreads / 64;

template <typename T, typename W>
__global__ __launch_bounds__(kLongThreads) void k_norm_long(const T* x, int64_t xs, const W* w, const W* b, T* y,
                                                            int64_t ys, float* mean, float* rstd, int64_t rows,
                                                            int cols, float eps)
{
    __shared__ float tmp[kLongWaves];
    const int64_t r = row_of_block();
    if (r >= rows) return;
    const T* xr = x + r * xs;
    T* yr = y + r * ys;
    float s = 0.f;
    for (int c = threadIdx.x; c < cols; c += kLongThreads) s += to_f(xr[c]);
    const float m = block_sum<kLongWaves>(s, tmp) / (float)cols;
    float q = 0.f;
    for (int c = threadIdx.x; c < cols; c += kLongThreads) {
        const float d = to_f(xr[c]) - m;
        q = fmaf(d, d, q);
    }
    const float rs = 1.f / sqrtf(block_sum<kLongWaves>(q, tmp) / (float)cols + eps);
    for (int c = threadIdx.x; c < cols; c += kLongThreads) {
        const float h = (to_f(xr[c]) - m) * rs;
        yr[c] = from_f<T>(fmaf(h, w ? to_f(w[c]) : 1.f, b ? to_f(b[c]) : 0.f));
    }
    if (threadIdx.x == 0) {
        if (mean) mean[r] = m;
        if (rstd) rstd[r] = rs;
    }
}

template <typename T, typename W>
__global__ __launch_bounds__(kLongThreads) void k_norm_long_dx(const T* dy, int64_t dys, const T* x, int64_t xs,
                                                               const W* w, const float* mean, const float* rstd,
                                                               T* dx, int64_t dxs, int64_t rows, int cols)
{
    __shared__ float tmp[kLongWaves];
    const int64_t r = row_of_block();
    if (r >= rows) return;
    const float m = mean[r], rs = rstd[r];
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < cols; c += kLongThreads) {
        const float v = to_f(dy[r * dys + c]) * (w ? to_f(w[c]) : 1.f);
        s1 += v;
        s2 = fmaf(v, (to_f(x[r * xs + c]) - m) * rs, s2);
    }
    const float c1 = block_sum<kLongWaves>(s1, tmp) / (float)cols;
    const float c2 = block_sum<kLongWaves>(s2, tmp) / (float)cols;
    for (int c = threadIdx.x; c < cols; c += kLongThreads) {
        const float v = to_f(dy[r * dys + c]) * (w ? to_f(w[c]) : 1.f);
        const float h = (to_f(x[r * xs + c]) - m) * rs;
        dx[r * dxs + c] = from_f<T>(rs * (v - fmaf(h, c2, c1)));
    }
}

// Sums over the rows part, part + parts, ... of 256 columns.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_long_dw(const T* dy, int64_t dys, const T* x, int64_t xs,
                                                      const float* mean, const float* rstd, float* part, int64_t rows,
                                                      int64_t cols)
{
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= cols) return;
    float aw = 0.f, ab = 0.f;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const float g = to_f(dy[r * dys + c]);
        aw = fmaf(g, (to_f(x[r * xs + c]) - mean[r]) * rstd[r], aw);
        ab += g;
    }
    part[2 * (int64_t)blockIdx.y * cols + c] = aw;
    part[(2 * (int64_t)blockIdx.y + 1) * cols + c] = ab;
}

constexpr int64_t kNormMaxCols = (int64_t)1 << 20;

static bool norm_opts_ok(const sgc_norm_opts* o)
{
    return o && o->rows >= 0 && o->rows < ((int64_t)1 << 31) && o->cols >= 1 && o->cols <= kNormMaxCols &&
           lm_dtype(o->dtype) && (o->wdtype == SGC_F32 || o->wdtype == o->dtype) && o->eps >= 0.f &&
           std::isfinite(o->eps) && (o->flags & ~SGC_NORM_ADD_GRADS) == 0;
}

// The shape of a workgroup for rows of `cols` held elements: 8 elements a
// thread, in 16 lanes up to 128 columns and else in as few waves as that takes
// (a power of two); 16 in the longest rows.  Where that would leave a quarter
// of the waves idle, 16-bit rows take half the waves and 16 elements a thread
// (46153 x 1300 bf16 backward: 151 -> 106 us; in fp32 16 elements spill), and
// fp32 rows of 513 to 768 one wave and 12, backward only where a row is no
// whole number of vectors (about 13 M elements: forward 577 23.3 -> 21.9 us,
// 600 19.2 -> 18.5, 768 19.8; backward 515 43.2 -> 39.7, 650 39.9 -> 39.0, but
// 600 34.2 -> 36.1 and 768 33.7 -> 36.5).  At least 8 waves.
struct NormShape {
    int ntr, ept, rpb;
};
static NormShape norm_shape(int64_t cols, int32_t dtype, bool back)
{
    if (cols <= 128) return {16, 8, 32};
    if (dtype == SGC_F32 && cols > 512 && cols <= 768 && (!back || cols % 4)) return {64, 12, 8};
    int ntr = 64, ept = 8;
    while (ntr < 1024 && ntr * 8 < cols) ntr *= 2;
    if (ntr * 8 < cols) ept = 16;
    if (dtype != SGC_F32 && ntr > 64 && cols <= ntr * 6) ntr /= 2, ept = 16;
    return {ntr, ept, ntr < 512 ? 512 / ntr : 1};
}

// Workgroups that share out the rows.
static int64_t norm_groups(const sgc_norm_opts* o, bool back)
{
    const NormShape sh = norm_shape(o->cols, o->dtype, back);
    const int64_t most = kCus * (back ? kBackwardWaves : kForwardWaves) * 64 / (sh.ntr * sh.rpb), need = cdiv(o->rows, sh.rpb);
    return need < most ? need : most;
}

static int64_t norm_parts(const sgc_norm_opts* o)
{
    if (o->cols <= kNormHeld) return norm_groups(o, true);
    return o->rows < 64 ? o->rows : 64;
}

template <typename T, typename W>
static int norm_forward(const sgc_norm_opts* o, const void* xv, int64_t xs, const void* wv, const void* bv, void* yv,
                        int64_t ys, float* mean, float* rstd, hipStream_t s)
{
    const T* x = (const T*)xv;
    const W *w = (const W*)wv, *b = (const W*)bv;
    T* y = (T*)yv;
    const int cols = (int)o->cols;
    const bool w32 = o->wdtype == SGC_F32;
    if (cols > kNormHeld) {
        k_norm_long<T, W><<<row_grid(o->rows), kLongThreads, 0, s>>>(x, xs, w, b, y, ys, mean, rstd, o->rows, cols,
                                                                     o->eps);
    } else {
        const unsigned g = (unsigned)norm_groups(o, false);
        const bool once = 2 * o->rows * cols * (int64_t)sizeof(T) >= kCacheBytes;
#define SGC_NORM_RUN(NTR, EPT, RPB, RAG, ONCE)                                                                      \
    k_norm<T, NTR, EPT, RPB, RAG, ONCE><<<g, NTR * RPB, 0, s>>>(x, xs, wv, bv, w32, y, ys, mean, rstd, o->rows, cols, \
                                                                o->eps)
// rows of whole vectors or not, past the caches or not
#define SGC_NORM(NTR, EPT, RPB)                                   \
    do {                                                          \
        if (cols % VecLen<T>::value) {                            \
            if (once) SGC_NORM_RUN(NTR, EPT, RPB, true, true);    \
            else SGC_NORM_RUN(NTR, EPT, RPB, true, false);        \
        } else {                                                  \
            if (once) SGC_NORM_RUN(NTR, EPT, RPB, false, true);   \
            else SGC_NORM_RUN(NTR, EPT, RPB, false, false);       \
        }                                                         \
    } while (0)
        const NormShape sh = norm_shape(cols, o->dtype, false);
        if (sh.ept == 12) { if constexpr (sizeof(T) == 4) { SGC_NORM(64, 12, 8); } }
        else if (sh.ept == 16 && sh.ntr == 1024) SGC_NORM(1024, 16, 1);
        else if (sh.ept == 16) {
            if constexpr (sizeof(T) == 2) {
                if (sh.ntr == 512) SGC_NORM(512, 16, 1);
                else if (sh.ntr == 256) SGC_NORM(256, 16, 2);
                else if (sh.ntr == 128) SGC_NORM(128, 16, 4);
                else SGC_NORM(64, 16, 8);
            }
        }
        else if (sh.ntr == 1024) SGC_NORM(1024, 8, 1);
        else if (sh.ntr == 512) SGC_NORM(512, 8, 1);
        else if (sh.ntr == 256) SGC_NORM(256, 8, 2);
        else if (sh.ntr == 128) SGC_NORM(128, 8, 4);
        else if (sh.ntr == 64) SGC_NORM(64, 8, 8);
        else SGC_NORM(16, 8, 32);
#undef SGC_NORM_RUN
    }
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}

template <typename T, typename W>
static int norm_backward(const sgc_norm_opts* o, const void* dyv, int64_t dys, const void* xv, int64_t xs,
                         const void* wv, const float* mean, const float* rstd, void* dxv, int64_t dxs, float* dw,
                         float* db, float* part, hipStream_t s)
{
    const T *dy = (const T*)dyv, *x = (const T*)xv;
    const W* w = (const W*)wv;
    T* dx = (T*)dxv;
    const int cols = (int)o->cols;
    const bool w32 = o->wdtype == SGC_F32;
    const int64_t parts = norm_parts(o);
    if (!o->rows) {
        // nothing to read
    } else if (cols > kNormHeld) {
        if (part) {  // before dx, which may take dy's or x's place
            k_norm_long_dw<T><<<dim3((unsigned)cdiv(cols, 256), (unsigned)parts), 256, 0, s>>>(
                dy, dys, x, xs, mean, rstd, part, o->rows, cols);
            SGC_LAUNCH_CHECK();
        }
        if (dx) {
            k_norm_long_dx<T, W><<<row_grid(o->rows), kLongThreads, 0, s>>>(dy, dys, x, xs, w, mean, rstd, dx, dxs,
                                                                            o->rows, cols);
            SGC_LAUNCH_CHECK();
        }
    } else if (dx || part) {
        const unsigned g = (unsigned)parts;
        const bool once = (dx ? 3 : 2) * o->rows * cols * (int64_t)sizeof(T) >= kCacheBytes;
#define SGC_NORM_RUN(NTR, EPT, RPB, RAG, ONCE)                                                                     \
    k_norm_back<T, NTR, EPT, RPB, RAG, ONCE><<<g, NTR * RPB, 0, s>>>(dy, dys, x, xs, wv, w32, mean, rstd, dx, dxs, \
                                                                     part, o->rows, cols)
        const NormShape sh = norm_shape(cols, o->dtype, true);
        if (sh.ept == 12) {
            if constexpr (sizeof(T) == 4) {
                if (once) SGC_NORM_RUN(64, 12, 8, true, true);
                else SGC_NORM_RUN(64, 12, 8, true, false);
            }
        }
        else if (sh.ept == 16 && sh.ntr == 1024) SGC_NORM(1024, 16, 1);
        else if (sh.ept == 16) {
            if constexpr (sizeof(T) == 2) {
                if (sh.ntr == 512) SGC_NORM(512, 16, 1);
                else if (sh.ntr == 256) SGC_NORM(256, 16, 2);
                else if (sh.ntr == 128) SGC_NORM(128, 16, 4);
                else SGC_NORM(64, 16, 8);
            }
        }
        else if (sh.ntr == 1024) SGC_NORM(1024, 8, 1);
        else if (sh.ntr == 512) SGC_NORM(512, 8, 1);
        else if (sh.ntr == 256) SGC_NORM(256, 8, 2);
        else if (sh.ntr == 128) SGC_NORM(128, 8, 4);
        else if (sh.ntr == 64) SGC_NORM(64, 8, 8);
        else SGC_NORM(16, 8, 32);
#undef SGC_NORM
#undef SGC_NORM_RUN
        SGC_LAUNCH_CHECK();
    }
    if (part) {
        k_norm_join<<<(unsigned)cdiv(2 * o->cols, kJoinCols), kJoinCols * kJoinDeep, 0, s>>>(
            part, parts, o->cols, dw, db, o->flags & SGC_NORM_ADD_GRADS);
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
