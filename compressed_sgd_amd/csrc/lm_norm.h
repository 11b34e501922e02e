// lm_norm.h -- shared by the norms (layer_norm.hip, rms_norm.hip, norm_q8.hip):
// the join of the parts' sums over the rows, options; the layer norm's rows in
// registers and the shape of its workgroups (the others': lm_q8.h).
#pragma once

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

// The parts' sums: a workgroup takes 32 of the `width` columns (the weight's cols,
// then the bias'), 32 threads each, eight parts in flight a thread.  512 parts of 4096 columns: 4.8 us.
constexpr int kJoinCols = 32, kJoinDeep = 32;
static __global__ __launch_bounds__(kJoinCols* kJoinDeep) void k_norm_join(const float* part, int64_t parts,
                                                                           int64_t width, int64_t cols, float* dw,
                                                                           float* db, int add)
{
    __shared__ float tmp[kJoinDeep][kJoinCols];
    const int tc = threadIdx.x % kJoinCols, td = threadIdx.x / kJoinCols;
    const int64_t c = (int64_t)blockIdx.x * kJoinCols + tc;
    float s = 0.f;
    if (c < width) {
#pragma unroll 8
        for (int64_t p = td; p < parts; p += kJoinDeep) s += part[p * width + c];
    }
    tmp[td][tc] = s;
    __syncthreads();
    if (td || c >= width) return;
#pragma unroll
    for (int d = 1; d < kJoinDeep; ++d) s += tmp[d][tc];
    float* out = c < cols ? dw : db;
    const int64_t at = c < cols ? c : c - cols;
    if (out) out[at] = add ? out[at] + s : s;
}

// Rows that are not held: one workgroup of 16 waves a row.
constexpr int kLongThreads = 1024, kLongWaves = kLongThreads / 64;

constexpr int64_t kNormMaxCols = (int64_t)1 << 20;

inline bool norm_opts_ok(const sgc_norm_opts* o)
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
inline NormShape norm_shape(int64_t cols, int32_t dtype, bool back)
{
    if (cols <= 128) return {16, 8, 32};
    if (dtype == SGC_F32 && cols > 512 && cols <= 768 && (!back || cols % 4)) return {64, 12, 8};
    int ntr = 64, ept = 8;
    while (ntr < 1024 && ntr * 8 < cols) ntr *= 2;
    if (ntr * 8 < cols) ept = 16;
    if (dtype != SGC_F32 && ntr > 64 && cols <= ntr * 6) ntr /= 2, ept = 16;
    return {ntr, ept, ntr < 512 ? 512 / ntr : 1};
}

}  // namespace sgc
