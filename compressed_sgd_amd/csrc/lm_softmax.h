// lm_softmax.h -- one pass over a row of logits with the running maximum and
// sums of its softmax, shared by token_logprobs.hip and distill.hip.
//
// A thread keeps m = max z, s = sum e and, for the entropy, t = sum e d, with
// d = (z - m) c, e = 2^d and c = scale / ln 2; when a group of its elements
// raises m, s and t are carried over to the new one.  Two threads' (or two
// workgroups') triples join the same way.  z - m is taken before the factor:
// masks at the type's lowest value then stay finite next to any maximum, and
// rows of that value alone are uniform as they should be.
#pragma once

#include "lm_common.h"

namespace sgc {

// 2^x in one instruction, 1 ulp; results below the normal range are 0.
__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// d below this has e = 0; keeps e * d and d * s away from 0 * inf.
constexpr float kLowD = -1000.f;

__device__ inline float finite_base(float m) { return m == -INFINITY ? 0.f : m; }

struct SoftSum {
    float m = -INFINITY, s = 0.f, t = 0.f;

    // Carry the sums over to a larger maximum.
    template <bool ENT>
    __device__ void raise(float to, float c)
    {
        const float d = fmaxf((m - to) * c, kLowD);
        const float f = exp2_fast(d);
        if (ENT) t = fmaf(d, s, t) * f;
        s *= f;
        m = to;
    }

    // N elements; those with a bit in `skip` count for the maximum alone.
    template <int N, bool ENT, bool SKIP>
    __device__ void add(float* x, float c, uint32_t skip)
    {
        float g = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) g = fmaxf(g, x[i]);
        if (g > m) raise<ENT>(g, c);
        if (SKIP && skip) {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = (skip >> i) & 1u ? -INFINITY : x[i];
        }
        const float base = finite_base(m);
        float s2 = 0.f, t2 = 0.f;  // two chains of additions
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float d = (x[i] - base) * c;
            const float e = exp2_fast(d);
            (i & 1 ? s2 : s) += e;
            if (ENT) (i & 1 ? t2 : t) = fmaf(e, fmaxf(d, kLowD), i & 1 ? t2 : t);
        }
        s += s2;
        if (ENT) t += t2;
    }
};

// Bits of the vector v of VL elements in a row's bitmap.
template <int VL>
__device__ inline uint32_t vec_bits(const uint32_t* bm, int v)
{
    if (VL == 8) return ((const uint8_t*)bm)[v];
    return (((const uint8_t*)bm)[v >> 1] >> ((v & 1) * 4)) & 0xfu;
}

// The elements [0, len) of z, by the NT threads of a workgroup.  U vectors of
// 16 bytes are in flight for each thread.
template <typename T, int NT, int U, bool ENT, bool SKIP>
__device__ inline void stream_sums(const T* z, int len, float c, const uint32_t* bm, SoftSum& a)
{
    constexpr int VL = VecLen<T>::value;
    using P = Pack<T, VL>;
    const P* p = (const P*)z;
    const int nv = len / VL;
    int v = threadIdx.x;
    for (; v + (U - 1) * NT < nv; v += U * NT) {
        P q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) q[u] = p[v + u * NT];
        uint32_t skip = 0;
        float x[U * VL];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (SKIP) skip |= vec_bits<VL>(bm, v + u * NT) << (u * VL);
#pragma unroll
            for (int e = 0; e < VL; ++e) x[u * VL + e] = to_f(q[u].v[e]);
        }
        a.template add<U * VL, ENT, SKIP>(x, c, skip);
    }
    for (; v < nv; v += NT) {
        const P q = p[v];
        float x[VL];
#pragma unroll
        for (int e = 0; e < VL; ++e) x[e] = to_f(q.v[e]);
        a.template add<VL, ENT, SKIP>(x, c, SKIP ? vec_bits<VL>(bm, v) : 0u);
    }
    const int i = nv * VL + threadIdx.x;
    if (i < len) {
        float x[1] = {to_f(z[i])};
        a.template add<1, ENT, SKIP>(x, c, SKIP ? (bm[i >> 5] >> (i & 31)) & 1u : 0u);
    }
}

// The threads' sums joined: the same values in every thread.  Each wave joins
// its own, then all threads the waves': one barrier, and one after, so that
// tmp may be used again.
template <int NW, bool ENT>
__device__ inline void block_join(SoftSum& a, float c, float (*tmp)[3])
{
    const float wm = wave_max(a.m);
    const float d = fmaxf((a.m - finite_base(wm)) * c, kLowD);
    const float f = exp2_fast(d);
    float t = ENT ? wave_sum(fmaf(d, a.s, a.t) * f) : 0.f;
    float s = wave_sum(a.s * f);
    float m = wm;
    if (NW > 1) {
        const int w = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            tmp[w][0] = wm;
            tmp[w][1] = s;
            tmp[w][2] = t;
        }
        __syncthreads();
        m = tmp[0][0];
#pragma unroll
        for (int i = 1; i < NW; ++i) m = fmaxf(m, tmp[i][0]);
        s = t = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const float di = fmaxf((tmp[i][0] - finite_base(m)) * c, kLowD), fi = exp2_fast(di);
            s += tmp[i][1] * fi;
            if (ENT) t += fmaf(di, tmp[i][1], tmp[i][2]) * fi;
        }
        __syncthreads();
    }
    a.m = m;
    a.s = s;
    a.t = t;
}

}  // namespace sgc
