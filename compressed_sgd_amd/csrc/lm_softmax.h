// lm_softmax.h -- one pass over a row of logits with the running maximum and
// sums of its softmax, shared by token_logprobs.hip and distill.hip.
//
// A thread keeps m = max z, s = sum e and, for the entropy, t = sum e d, with
// e = 2^d, d = (z - m) c and c = scale / ln 2; when a group of its elements
// raises m, s and t are carried over to the new one.  Two threads' sums join
// the same way.
//
// The pass is bound by the vector unit as much as by memory, so d is one fma:
// z c - b with b = m c rounded to fp32.  All e are then too large by the same
// 2^r, r = m c - b, which the sums are freed from once a row.  That needs a
// small r: b is at least -1e8 (|r| <= 4), and a row whose |m c| is more than
// 1e8 is done again with z - m before the factor (FAR).  Such is the row that a
// mask at the type's lowest value leaves nothing but itself; it is uniform.
#pragma once

#include "lm_common.h"

namespace sgc {

// 2^x in one instruction, 1 ulp; results below the normal range are 0.
__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// d below this has e = 0; keeps e * d and d * s away from 0 * inf.
constexpr float kLowD = -1000.f;
constexpr float kLn2 = 0.693147180559945309f;

__device__ inline float finite_base(float m) { return m == -INFINITY ? 0.f : m; }

// c of a scale that a call may have: positive and finite as fp32.
inline float exponent_factor(float scale) { return (float)((double)scale * M_LOG2E); }
inline bool scale_ok(float scale) { return scale > 0.f && std::isfinite(exponent_factor(scale)); }

constexpr float kFar = 1e8f;
__device__ inline bool is_far(float m, float c) { return fabsf(m * c) > kFar && fabsf(m) != INFINITY; }

template <bool FAR>
struct SoftSum {
    float m = -INFINITY, s = 0.f, t = 0.f;

    // What z is measured from: m itself (FAR), or m c.
    __device__ static float base_of(float m, float c) { return FAR ? finite_base(m) : fmaxf(m * c, -kFar); }
    __device__ static float power(float x, float base, float c) { return FAR ? (x - base) * c : fmaf(x, c, -base); }
    // log2 of the factor from sums at one maximum to sums at a larger one
    __device__ static float step(float from, float to, float c)
    {
        return fmaxf(FAR ? (from - finite_base(to)) * c : base_of(from, c) - base_of(to, c), kLowD);
    }

    // N elements.
    template <int N, bool ENT>
    __device__ void add(float* x, float c)
    {
        float g = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) g = fmaxf(g, x[i]);
        if (g > m) {
            const float d = step(m, g, c), f = exp2_fast(d);
            if (ENT) t = fmaf(d, s, t) * f;
            s *= f;
            m = g;
        }
        const float base = base_of(m, c), was = t;
        float s2 = 0.f, t2 = 0.f;  // two chains of additions
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = power(x[i], base, c);
            const float e = exp2_fast(x[i]);
            (i & 1 ? s2 : s) += e;
            if (ENT) (i & 1 ? t2 : t) = fmaf(e, x[i], i & 1 ? t2 : t);
        }
        s += s2;
        if (ENT) {
            t += t2;
            if (t != t) {  // 0 * -inf: only groups with masked elements pay for the clamp
                t = was;
#pragma unroll
                for (int i = 0; i < N; ++i) t = fmaf(exp2_fast(x[i]), fmaxf(x[i], kLowD), t);
            }
        }
    }
};

// Bits of the vector v of VL elements in a row's bitmap.
template <int VL>
__device__ inline uint32_t vec_bits(const uint32_t* bm, int v)
{
    if (VL == 8) return ((const uint8_t*)bm)[v];
    return (((const uint8_t*)bm)[v >> 1] >> ((v & 1) * 4)) & 0xfu;
}

// -inf in the elements of q with a bit in `skip`.
template <typename T>
__device__ inline void remove(Raw& q, uint32_t skip)
{
    const Raw low = raw_low<T>();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t gone;
        if (sizeof(T) == 4)
            gone = (skip >> i) & 1u ? 0xffffffffu : 0u;
        else
            gone = ((skip >> (2 * i)) & 1u ? 0xffffu : 0u) | ((skip >> (2 * i + 1)) & 1u ? 0xffff0000u : 0u);
        q.w[i] = (q.w[i] & ~gone) | (low.w[i] & gone);
    }
}

// The elements [0, len) of z, by the NT threads of a workgroup: thread i takes
// the vectors i, i + NT, ... and one element past the last whole vector.  U
// vectors of 16 bytes are in flight for each thread.  (The next U fetched
// ahead, with the last group padded: 195 -> 199 us for 4096 x 131072 bf16.)
template <typename T, int NT, int U, bool ENT, bool SKIP, bool ONCE, bool FAR>
__device__ inline void stream_sums(const T* z, int len, float c, const uint32_t* bm, SoftSum<FAR>& a)
{
    constexpr int VL = VecLen<T>::value;
    const Raw* p = (const Raw*)z;
    const int nv = len / VL;
    int v0 = 0;  // the group's first vector
    for (; v0 + U * NT <= nv; v0 += U * NT) {
        const int v = v0 + threadIdx.x;
        Raw q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) q[u] = load_row<ONCE>(p + v + u * NT);
        __builtin_amdgcn_sched_barrier(0);  // all on their way before the first is waited for
#pragma unroll
        for (int u = 0; u < U; u += 2) {  // two vectors at a time: four take registers that cost a workgroup
            float x[2 * VL];
            if (SKIP) {
                const uint32_t s0 = vec_bits<VL>(bm, v + u * NT), s1 = vec_bits<VL>(bm, v + (u + 1) * NT);
                if (s0) remove<T>(q[u], s0);
                if (s1) remove<T>(q[u + 1], s1);
            }
            unpack<T>(q[u], x);
            unpack<T>(q[u + 1], x + VL);
            a.template add<2 * VL, ENT>(x, c);
        }
    }
    if (v0 < nv) {  // fewer than U vectors a thread: one trip to memory for them too
        const int v = v0 + threadIdx.x;
        Raw q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) q[u] = v + u * NT < nv ? load_row<ONCE>(p + v + u * NT) : raw_low<T>();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (v0 + u * NT < nv) {  // the same for all
                if (SKIP) {
                    const uint32_t s0 = v + u * NT < nv ? vec_bits<VL>(bm, v + u * NT) : 0u;
                    if (s0) remove<T>(q[u], s0);
                }
                float x[VL];
                unpack<T>(q[u], x);
                a.template add<VL, ENT>(x, c);
            }
        }
    }
    const int i = nv * VL + threadIdx.x;
    if (i < len) {
        float x[1] = {SKIP && (bm[i >> 5] >> (i & 31)) & 1u ? -INFINITY : to_f(z[i])};
        a.template add<1, ENT>(x, c);
    }
}

// The threads' sums joined, the same values in every thread, s and t at m
// itself.  Each wave joins its own, then all threads the waves': one barrier,
// and one after, so that tmp may be used again.
template <int NW, bool ENT, bool FAR>
__device__ inline void block_join(SoftSum<FAR>& a, float c, float (*tmp)[3])
{
    float m = wave_max(a.m);
    const float d = SoftSum<FAR>::step(a.m, m, c), f = exp2_fast(d);
    float t = ENT ? wave_sum(fmaf(d, a.s, a.t) * f) : 0.f;
    float s = wave_sum(a.s * f);
    if (NW > 1) {
        const int w = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            tmp[w][0] = m;
            tmp[w][1] = s;
            tmp[w][2] = t;
        }
        __syncthreads();
        const int i = threadIdx.x % NW;  // a wave's sums a lane
        m = max_of_lanes<NW>(tmp[i][0]);
        const float di = SoftSum<FAR>::step(tmp[i][0], m, c), fi = exp2_fast(di);
        s = sum_of_lanes<NW>(tmp[i][1] * fi);
        if (ENT) t = sum_of_lanes<NW>(fmaf(di, tmp[i][1], tmp[i][2]) * fi);
        __syncthreads();
    }
    if (!FAR) {
        const float r = m == -INFINITY ? 0.f : fmaf(m, c, -SoftSum<FAR>::base_of(m, c)), f1 = exp2_fast(-r);
        if (ENT) t = fmaf(-r, s, t) * f1;
        s *= f1;
    }
    a.m = m;
    a.s = s;
    a.t = t;
}

// A row's (or chunk's) m, s, t in every thread; *own: the thread's maximum.
struct Sums {
    float m, s, t;
};
template <typename T, int NW, bool ENT, bool SKIP, bool ONCE>
__device__ inline Sums row_softmax(const T* z, int len, float c, const uint32_t* bm, float (*tmp)[3], float* own)
{
    SoftSum<false> a;
    stream_sums<T, NW * 64, 4, ENT, SKIP, ONCE>(z, len, c, bm, a);
    *own = a.m;
    block_join<NW, ENT>(a, c, tmp);
    if (!is_far(a.m, c)) return {a.m, a.s, a.t};
    SoftSum<true> b;
    stream_sums<T, NW * 64, 2, ENT, SKIP, ONCE>(z, len, c, bm, b);
    block_join<NW, ENT>(b, c, tmp);
    return {b.m, b.s, b.t};
}

// The sums of the parts k, k + NT, ... of n, four floats each, joined.
template <int NW, bool ENT>
__device__ inline Sums join_parts(const float* p, int n, float c, float (*tmp)[3])
{
    SoftSum<true> a;
    for (int k = threadIdx.x; k < n; k += NW * 64) {
        const float m = p[4 * k], s = p[4 * k + 1], t = p[4 * k + 2];
        const float to = fmaxf(m, a.m);
        const float d0 = a.step(a.m, to, c), f0 = exp2_fast(d0), d1 = a.step(m, to, c), f1 = exp2_fast(d1);
        if (ENT) a.t = fmaf(d0, a.s, a.t) * f0 + fmaf(d1, s, t) * f1;
        a.s = a.s * f0 + s * f1;
        a.m = to;
    }
    block_join<NW, ENT>(a, c, tmp);
    return {a.m, a.s, a.t};
}

}  // namespace sgc
