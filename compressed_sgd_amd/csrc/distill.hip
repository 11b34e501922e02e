// distill.hip -- divergence of a student's distribution from a teacher's top
// entries, loss and gradient.
//
//   e_i = exp(scale (z_i - m)),  s = sum e,  o = sum of e outside the entries
//   loss = sum_j t_j (log t_j - log q_j) + u (log u - log(o / s)),  q = e / s
//   dz_i = scale g ((T + u) q_i - t_i)          entries,  T = sum_j t_j
//   dz_i = scale g ((T + u) q_i - u e_i / o)    else
// The entries of a row are bits in shared memory: one look tells the vectors
// that hold one, so that o is summed without them and not found by
// subtraction, which loses it where the student has learnt its teacher.  There
// o is small besides: with the tail the outside is measured from its own
// maximum mo, so that its sum is at least 1 however far below m it lies, and
// joins the entries' as o 2^-D, D = (m - mo) c.
#include "lm_softmax.h"

namespace sgc {

// The most vectors a row may have to be held in a workgroup's registers.
constexpr int kMostHeld = 16384;
// Rows are shared out in chunks of at most kChunkMax elements a workgroup
// (its bitmap is 16 KB).
constexpr int kChunkMax = 131072;

struct DistillArgs {
    int64_t rows, zs, dzs;
    int32_t vocab, top, mode;
    float scale, c, teacher_scale;
    const int32_t* idx;
    const float* val;
    float* loss;
    float* stats;
    const float* dloss;
    uint32_t* dstatus;
};

// A row's entries, in shared memory; entry j belongs to thread j mod NT.
struct Entries {
    float lt[SGC_TOP_MAX];  // log of the teacher's probability
    float z[SGC_TOP_MAX];   // the student's logit
    int32_t idx[SGC_TOP_MAX];
};

// Loads a row's entries and gives T and u.  An entry that is absent or out of
// range has log t = -inf.  z0, z1: the part of the row that the workgroup
// reads the logits of.
template <typename T, int NW>
__device__ inline void load_entries(Entries& en, const DistillArgs& a, int64_t r, const T* zr, int z0, int z1,
                                    float* tmp, float* total, float* u)
{
    constexpr int NT = NW * 64;
    float m = -INFINITY;
    for (int j = threadIdx.x; j < a.top; j += NT) {
        const int32_t at = a.idx[r * a.top + j];
        const float v = at >= 0 && at < a.vocab ? a.val[r * a.top + j] * a.teacher_scale : -INFINITY;
        en.idx[j] = at;
        en.lt[j] = v;
        en.z[j] = at >= z0 && at < z1 ? to_f(zr[at]) : -INFINITY;
        m = fmaxf(m, v);
    }
    float sum = 0.f;
    if (a.mode == SGC_DISTILL_RENORM) {
        const float base = finite_base(block_max<NW>(m, tmp));
        for (int j = threadIdx.x; j < a.top; j += NT) sum += expf(en.lt[j] - base);
        sum = block_sum<NW>(sum, tmp);
        const float ln = sum == 0.f ? 0.f : logf(sum) ;
        for (int j = threadIdx.x; j < a.top; j += NT) en.lt[j] = (en.lt[j] - base) - ln;
        *total = sum == 0.f ? 0.f : sum != sum ? sum : 1.f;
        *u = 0.f;
    } else {
        for (int j = threadIdx.x; j < a.top; j += NT) sum += expf(en.lt[j]);
        *total = block_sum<NW>(sum, tmp);
        *u = fmaxf(0.f, 1.f - *total);
    }
}

// An outside this many powers of two below the row's maximum is one that a mask
// has removed (2^-1074 is the smallest number of 64 bits): q = 0 there.
constexpr float kGone = 1074.f;
// Up to here the sum outside is kept at the row's maximum.
constexpr float kNear = 32.f;

// What a row's elements add up to: s = sum e at the maximum m, and the sum
// outside the entries at m, times 2^k (k a whole number, 0 where it is near).
struct Mass {
    float m, s, o, k;
};
__device__ inline float log_outside(const Mass& w) { return logf(w.o) - w.k * kLn2; }

// o: the sum outside at its own maximum, D powers of two below the row's.
__device__ inline void place_outside(float o, float D, Mass* w)
{
    w->k = D < kNear ? 0.f : floorf(D);
    w->o = o * exp2_fast(w->k - D);
    if (o == 0.f || D > kGone) w->o = w->k = 0.f;
}

// The outside's maximum mo and sum o there (without the tail, the whole row's)
// joined with the entries.
template <int NW, bool TAIL>
__device__ inline Mass row_mass(const Entries& en, const DistillArgs& a, float mo, float o, float* tmp)
{
    if (!TAIL) return {mo, o, o, 0.f};
    constexpr int NT = NW * 64;
    float mi = -INFINITY, in = 0.f;
    for (int j = threadIdx.x; j < a.top; j += NT) mi = fmaxf(mi, en.z[j]);
    Mass w;
    w.m = fmaxf(mo, block_max<NW>(mi, tmp));
    const float base = finite_base(w.m), D = (base - mo) * a.c;  // inf if nothing is outside
    for (int j = threadIdx.x; j < a.top; j += NT) in += exp2_fast((en.z[j] - base) * a.c);
    w.s = o * exp2_fast(-D) + block_sum<NW>(in, tmp);
    place_outside(o, D, &w);
    return w;
}

// Marks the entries inside [z0, z1) in the bitmap; whether one of the row's is
// out of range or one of these repeated.  bm holds (z1 - z0 + 31) / 32 words.
template <int NW>
__device__ inline bool mark_entries(const Entries& en, const DistillArgs& a, int z0, int z1, uint32_t* bm)
{
    constexpr int NT = NW * 64;
    for (int w = threadIdx.x; w < (z1 - z0 + 31) / 32; w += NT) bm[w] = 0;
    __syncthreads();
    int bad = 0;
    for (int j = threadIdx.x; j < a.top; j += NT) {
        const int32_t at = en.idx[j];
        if (at < -1 || at >= a.vocab) bad = 1;
        if (at >= z0 && at < z1) {
            const uint32_t bit = 1u << ((at - z0) & 31);
            if (atomicOr(&bm[(at - z0) >> 5], bit) & bit) bad = 1;
        }
    }
    return __syncthreads_or(bad) != 0;
}

// Factors of the gradient: of e_i 2^up outside the entries, of e_i inside, of t.
// u / o is at most 2 u: a smaller o is taken at a larger power of two.
struct Factors {
    float out, up, in, t;
};
__device__ inline Factors factors(const DistillArgs& a, float g, const Mass& w, float total, float u)
{
    const float k = a.scale * g, q = (total + u) / w.s;
    Factors f = {k * q, 0.f, k * q, k};
    if (u > 0.f && w.o > 0.f) {
        const int e = w.o < 1.f ? -ilogbf(w.o) : 0;
        f.up = w.k + (float)e;
        f.out = k * (q * exp2_fast(-f.up) - u / ldexpf(w.o, e));
    }
    return f;
}

// The gradient of the chunk [z0, z1): the outside's everywhere, then the entries'
// own values over it (every thread's stores are done at the barrier).
template <typename T, int NW, int U, bool ONCE>
__device__ inline void write_gradient(const Entries& en, const DistillArgs& a, const T* zr, T* out, int z0, int z1,
                                      float m, const Factors& f)
{
    constexpr int NT = NW * 64, VL = VecLen<T>::value;
    const Raw* p = (const Raw*)(zr + z0);
    Raw* o = (Raw*)(out + z0);
    const int nv = (z1 - z0) / VL;
    const auto one = [&](const Raw& q, int v) {
        float x[VL];
        unpack<T>(q, x);
#pragma unroll
        for (int e = 0; e < VL; ++e) x[e] = exp2_fast(fmaf(x[e] - m, a.c, f.up)) * f.out;
        store_row<ONCE>(o + v, pack<T>(x));
    };
    int v = threadIdx.x;
    for (; v + (U - 1) * NT < nv; v += U * NT) {
        Raw q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) q[u] = load_row<ONCE>(p + v + u * NT);
#pragma unroll
        for (int u = 0; u < U; ++u) one(q[u], v + u * NT);
    }
    for (; v < nv; v += NT) one(load_row<ONCE>(p + v), v);
    const int64_t i = (int64_t)z0 + nv * VL + threadIdx.x;  // may pass 2^31
    if (i < z1) out[i] = from_f<T>(exp2_fast(fmaf(to_f(zr[i]) - m, a.c, f.up)) * f.out);
    __syncthreads();
    for (int j = threadIdx.x; j < a.top; j += NT) {
        const int32_t at = en.idx[j];
        if (at >= z0 && at < z1)
            out[at] = from_f<T>(exp2_fast((en.z[j] - m) * a.c) * f.in - expf(en.lt[j]) * f.t);
    }
}

template <typename T, int NW, bool ONCE>
__device__ inline void write_zeros(T* out, int z0, int z1)
{
    constexpr int NT = NW * 64, VL = VecLen<T>::value;
    const int nv = (z1 - z0) / VL;
    for (int v = threadIdx.x; v < nv; v += NT) store_row<ONCE>((Raw*)(out + z0) + v, Raw{{0, 0, 0, 0}});
    const int64_t i = (int64_t)z0 + nv * VL + threadIdx.x;
    if (i < z1) out[i] = (T)0.f;
}

__device__ inline void write_stats(const DistillArgs& a, int64_t r, const Mass& w, bool skip)
{
    if (!a.stats) return;
    a.stats[4 * r] = w.m;
    a.stats[4 * r + 1] = w.s;
    a.stats[4 * r + 2] = w.o;
    a.stats[4 * r + 3] = skip ? 0.f : 1.f + w.k;
}

// Loss and stats of a row from its sums; whether its gradient is zero.
template <int NW>
__device__ inline bool finish_row(const Entries& en, const DistillArgs& a, int64_t r, const Mass& w, float total,
                                  float u, bool bad, float* tmp)
{
    constexpr int NT = NW * 64;
    const float ln_s = logf(w.s), base = finite_base(w.m);
    float l = 0.f;
    for (int j = threadIdx.x; j < a.top; j += NT) {
        const float lt = en.lt[j], t = expf(lt);
        if (t != 0.f) l += t * (lt - ((en.z[j] - base) * a.scale - ln_s));
    }
    l = block_sum<NW>(l, tmp);
    if (u > 0.f && w.o != 0.f) l += u * (logf(u) - (log_outside(w) - ln_s));
    const bool skip = bad || w.s == 0.f || (a.mode == SGC_DISTILL_RENORM && total == 0.f);
    if (threadIdx.x == 0) {
        a.loss[r] = bad ? NAN : skip ? 0.f : l;
        write_stats(a, r, w, skip);
        if (bad && a.dstatus) atomicOr(a.dstatus, SGC_STATUS_CORRUPT);
    }
    return skip;
}

// A row a workgroup, vocab <= kChunkMax: loss, and with dz the gradient; the
// row's second reading comes from the cache.  For the loss alone, and rows too
// long to be held.  2000 x 10001 fp16 with the tail 13.5 us, one row's chain of
// trips and barriers; 4096 x 50000 bf16 80 us, 5.1 TB/s.
template <typename T, int NW, bool TAIL>
__global__ __launch_bounds__(NW * 64) void k_distill_row(DistillArgs a, const T* z, T* dz)
{
    extern __shared__ uint32_t bm[];
    __shared__ Entries en;
    __shared__ float tmp[NW];
    __shared__ float tmj[NW][3];
    const int64_t r = row_of_block();
    if (r >= a.rows) return;
    const T* zr = z + r * a.zs;
    float total, u;
    load_entries<T, NW>(en, a, r, zr, 0, a.vocab, tmp, &total, &u);
    const bool bad = mark_entries<NW>(en, a, 0, a.vocab, bm);
    float own;
    const Sums sum = row_softmax<T, NW, false, TAIL, false>(zr, a.vocab, a.c, bm, tmj, &own);
    const Mass w = row_mass<NW, TAIL>(en, a, sum.m, sum.s, tmp);
    const bool skip = finish_row<NW>(en, a, r, w, total, u, bad, tmp);
    if (!dz) return;
    const float g = a.dloss ? a.dloss[r] : 1.f;
    T* out = dz + r * a.dzs;
    if (skip || g == 0.f) {
        write_zeros<T, NW, false>(out, 0, a.vocab);
        return;
    }
    write_gradient<T, NW, 4, false>(en, a, zr, out, 0, a.vocab, finite_base(w.m), factors(a, g, w, total, u));
}

// The held vectors are the same 16 bytes after this, but the compiler does not
// know it: else it keeps the elements that it unpacked to fp32 for the next
// pass, in twice the registers.
template <int NV>
__device__ inline void keep_packed(Raw (&q)[NV])
{
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(q[n].w[i]));
}

// A row a workgroup with loss and gradient in one reading: NV vectors of the
// row stay in each thread's registers from the sums to the gradient (a vector
// past the row is -inf, and with the tail so is an entry, once marked).  One
// entry a thread.  The exponent is one fma, z c - M c with M c rounded to b (M
// the largest held): every e is then too large by 2^(M c - b), which the sums
// are freed from once a row (lm_softmax.h); a maximum far from zero takes z - M
// first.  Bound by memory: 4096 x 50000 bf16 with the tail 154
// us, 5.3 TB/s, by three workgroups a compute unit (by two 160, by one of 16
// waves 232); 4096 x 131072 455 us, 4.7 TB/s, where a row takes half the unit's
// registers.
template <typename T, int NW, int NV, bool TAIL, bool ONCE, bool HEAD>
__global__ __launch_bounds__(NW * 64, NV > 8 ? 4 : 1) void k_distill_held(DistillArgs a, const T* z, T* dz)
{
    constexpr int NT = NW * 64, VL = VecLen<T>::value;
    static_assert(NT >= SGC_TOP_MAX, "one entry a thread");
    extern __shared__ uint32_t bm[];
    __shared__ float tmp[2 * NW];
    const int64_t r = row_of_block();
    if (r >= a.rows) return;
    const T* zr = z + r * a.zs;
    // HEAD: vectors are counted from a 128-byte line of the output (where its
    // row starts at a vector of one), so that the waves write whole lines.
    T* out = dz + r * a.dzs;
    const int tid = threadIdx.x, nv = a.vocab / VL;
    const int head = HEAD && !((uintptr_t)out & 15) ? (int)(((uintptr_t)out & 127) >> 4) : 0;
    const int first = tid - head;
    const auto vec = [&](int n) { return first + n * NT; };
    const auto held = [&](int n) { return (!HEAD || n > 0 || first >= 0) && n * NT < nv - first; };
    const float g = a.dloss ? a.dloss[r] : 1.f;
    int32_t at = -1;
    float v = -INFINITY;
    if (tid < a.top) {
        at = a.idx[r * a.top + tid];
        v = a.val[r * a.top + tid] * a.teacher_scale;
    }
    Raw q[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) q[n] = held(n) ? load_row<ONCE>((const Raw*)zr + vec(n)) : raw_low<T>();
    const int last = nv * VL + tid;
    float z_last = last < a.vocab ? to_f(zr[last]) : -INFINITY;
    // the entries: marks, T and u
    const bool in_row = at >= 0 && at < a.vocab;
    const float z_in = in_row ? to_f(zr[at]) : -INFINITY;
    if (!in_row) v = -INFINITY;
    for (int w = tid; w < (a.vocab + 31) / 32; w += NT) bm[w] = 0;
    __syncthreads();
    int bad = at < -1 || at >= a.vocab;
    if (in_row) bad |= (atomicOr(&bm[at >> 5], 1u << (at & 31)) >> (at & 31)) & 1u;
    bad = __syncthreads_or(bad);
    float lt = v, total, u = 0.f;
    if (TAIL) {
        total = block_sum<NW>(expf(lt), tmp);
        u = in_scalar(fmaxf(0.f, 1.f - total));
    } else {
        const float base = finite_base(block_max<NW>(v, tmp));
        const float sum = block_sum<NW>(expf(v - base), tmp);
        lt = (v - base) - (sum == 0.f ? 0.f : logf(sum));
        total = sum == 0.f ? 0.f : sum != sum ? sum : 1.f;
    }
    // the held elements' maximum and sum
    if (TAIL) {
        if (last < a.vocab && (bm[last >> 5] >> (last & 31)) & 1u) z_last = -INFINITY;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const uint32_t skip = held(n) ? vec_bits<VL>(bm, vec(n)) : 0u;
            if (skip) remove<T>(q[n], skip);
        }
        keep_packed(q);
    }
    float mo = z_last, m = z_in;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        float x[VL];
        unpack<T>(q[n], x);
#pragma unroll
        for (int e = 0; e < VL; ++e) mo = fmaxf(mo, x[e]);
    }
    if (TAIL) {
        block_maxima<NW>(mo, m, tmp);
        m = fmaxf(mo, m);
    } else {
        m = mo = block_max<NW>(mo, tmp);
    }
    keep_packed(q);
    m = in_scalar(m);
    const float base = in_scalar(finite_base(mo)), b = in_scalar(base * a.c);
    const bool far = is_far(mo, a.c);
    float o = 0.f, o2 = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        float x[VL];
        unpack<T>(q[n], x);
        if (far) {
#pragma unroll
            for (int e = 0; e < VL; ++e) (e & 1 ? o2 : o) += exp2_fast((x[e] - base) * a.c);
        } else {
#pragma unroll
            for (int e = 0; e < VL; ++e) (e & 1 ? o2 : o) += exp2_fast(fmaf(x[e], a.c, -b));
        }
    }
    const float e_last = exp2_fast(far ? (z_last - base) * a.c : fmaf(z_last, a.c, -b));
    keep_packed(q);
    o += o2 + e_last;
    // joined with the entries
    asm volatile("" : "+v"(lt));  // t is taken here, not kept in a register through the loops
    const float t = expf(lt);
    const float e_in = exp2_fast((z_in - finite_base(m)) * a.c);
    const float free = far ? 1.f : exp2_fast(-fmaf(base, a.c, -b));
    const float D = TAIL ? (finite_base(m) - mo) * a.c : 0.f, down = exp2_fast(-D);
    float in = e_in;
    if (TAIL)
        block_sums<NW>(o, in, tmp);
    else
        o = block_sum<NW>(o, tmp);
    o *= free;
    Mass w = {m, TAIL ? fmaf(o, down, in) : o, o, 0.f};
    if (TAIL) place_outside(o, D, &w);
    const float ln_s = logf(w.s);
    float l = block_sum<NW>(t != 0.f ? t * (lt - ((z_in - finite_base(m)) * a.scale - ln_s)) : 0.f, tmp);
    if (u > 0.f && w.o != 0.f) l += u * (logf(u) - (log_outside(w) - ln_s));
    const bool skip = bad || w.s == 0.f || (!TAIL && total == 0.f);
    if (tid == 0) {
        a.loss[r] = bad ? NAN : skip ? 0.f : l;
        write_stats(a, r, w, skip);
        if (bad && a.dstatus) atomicOr(a.dstatus, SGC_STATUS_CORRUPT);
    }
    if (skip || g == 0.f) {
        write_zeros<T, NW, ONCE>(out, 0, a.vocab);
        return;
    }
    // as factors(), for elements measured from the largest held
    const float k = a.scale * g, k_in = k * ((total + u) / w.s);
    const float k_out = free * (k_in * down - (u > 0.f && w.o > 0.f ? k * (u / o) : 0.f));
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        if (held(n)) {
            float x[VL];
            unpack<T>(q[n], x);
            if (far) {
#pragma unroll
                for (int e = 0; e < VL; ++e) x[e] = exp2_fast((x[e] - base) * a.c) * k_out;
            } else {
#pragma unroll
                for (int e = 0; e < VL; ++e) x[e] = exp2_fast(fmaf(x[e], a.c, -b)) * k_out;
            }
            store_row<ONCE>((Raw*)out + vec(n), pack<T>(x));
        }
    }
    if (last < a.vocab) out[last] = from_f<T>(e_last * k_out);
    __syncthreads();
    if (in_row) out[at] = from_f<T>(e_in * k_in - t * k);
}

// A chunk of a row: maximum and sum outside the entries (without the tail, of
// all), and whether an entry is bad.  part [rows, chunks, 3].
template <typename T, int NW, bool TAIL>
__global__ __launch_bounds__(NW * 64) void k_distill_part(DistillArgs a, const T* z, int chunk, int chunks,
                                                          float* part)
{
    extern __shared__ uint32_t bm[];
    __shared__ Entries en;
    __shared__ float tmj[NW][3];
    const int64_t b = row_of_block(), r = b / chunks;
    if (r >= a.rows) return;
    const int z0 = (int)(b - r * chunks) * chunk, z1 = a.vocab - z0 < chunk ? a.vocab : z0 + chunk;
    const T* zr = z + r * a.zs;
    for (int j = threadIdx.x; j < a.top; j += NW * 64) en.idx[j] = a.idx[r * a.top + j];
    const bool bad = mark_entries<NW>(en, a, z0, z1, bm);
    float own;
    const Sums sum = row_softmax<T, NW, false, TAIL, false>(zr + z0, z1 - z0, a.c, bm, tmj, &own);
    if (threadIdx.x == 0) {
        float* p = part + 3 * b;
        p[0] = sum.m;
        p[1] = sum.s;
        p[2] = bad ? 1.f : 0.f;
    }
}

// The chunks of a row joined, then its loss.
template <typename T, int NW, bool TAIL>
__global__ __launch_bounds__(NW * 64) void k_distill_join(DistillArgs a, const T* z, int chunks, const float* part)
{
    __shared__ Entries en;
    __shared__ float tmp[NW];
    const int64_t r = row_of_block();
    if (r >= a.rows) return;
    float total, u;
    load_entries<T, NW>(en, a, r, z + r * a.zs, 0, a.vocab, tmp, &total, &u);
    const float* p = part + 3 * r * chunks;
    float m = -INFINITY;
    int bad = 0;
    for (int k = threadIdx.x; k < chunks; k += NW * 64) {
        m = fmaxf(m, p[3 * k]);
        bad |= p[3 * k + 2] != 0.f;
    }
    m = block_max<NW>(m, tmp);
    bad = __syncthreads_or(bad);
    float o = 0.f;
    for (int k = threadIdx.x; k < chunks; k += NW * 64)
        o += p[3 * k + 1] * exp2_fast(fmaxf((p[3 * k] - finite_base(m)) * a.c, kLowD));
    o = block_sum<NW>(o, tmp);
    finish_row<NW>(en, a, r, row_mass<NW, TAIL>(en, a, m, o, tmp), total, u, bad != 0, tmp);
}

// The gradient of a chunk of a row from the row's stats.  Bound by memory: 4096 x
// 50000 bf16 141 us, 5.8 TB/s.
template <typename T, int NW, bool ONCE>
__global__ __launch_bounds__(NW * 64) void k_distill_grad(DistillArgs a, const float* stats, const T* z, T* dz,
                                                          int chunk, int chunks)
{
    __shared__ Entries en;
    __shared__ float tmp[NW];
    const int64_t b = row_of_block(), r = b / chunks;
    if (r >= a.rows) return;
    const int z0 = (int)(b - r * chunks) * chunk, z1 = a.vocab - z0 < chunk ? a.vocab : z0 + chunk;
    const T* zr = z + r * a.zs;
    T* out = dz + r * a.dzs;
    const float g = a.dloss ? a.dloss[r] : 1.f;
    if (stats[4 * r + 3] == 0.f || g == 0.f) {
        write_zeros<T, NW, ONCE>(out, z0, z1);
        return;
    }
    float total, u;
    load_entries<T, NW>(en, a, r, zr, z0, z1, tmp, &total, &u);
    __syncthreads();  // the entries' logits are read before any of the chunk's gradient is written
    const Mass w = {stats[4 * r], stats[4 * r + 1], stats[4 * r + 2], stats[4 * r + 3] - 1.f};
    write_gradient<T, NW, 4, ONCE>(en, a, zr, out, z0, z1, finite_base(w.m), factors(a, g, w, total, u));
}

static bool distill_opts_ok(const sgc_distill_opts* o)
{
    return o && o->rows >= 0 && o->rows < ((int64_t)1 << 31) && o->vocab >= 1 && o->vocab < ((int64_t)1 << 31) &&
           lm_dtype(o->dtype) && o->top >= 1 && o->top <= SGC_TOP_MAX &&
           (o->mode == SGC_DISTILL_RENORM || o->mode == SGC_DISTILL_TAIL) && scale_ok(o->scale) &&
           o->teacher_scale > 0.f && std::isfinite(o->teacher_scale) &&
           (o->mode != SGC_DISTILL_TAIL || o->teacher_scale == 1.f) && o->reserved == 0;
}

static bool entries_ok(const int32_t* idx, const float* val)
{
    return idx && val && lm_aligned(idx, 4) && lm_aligned(val, 4);
}

// How the rows are shared out.  With the gradient a row that can be held is: one
// launch, one reading (1 x 50000 bf16: 15 us, in chunks 23; 300 x 131072 57 and
// 56, 500 x 131072 69 and 87).  Else one
// workgroup a row from kManyRows rows on, which fill the card, and for rows up
// to kShort (twice that where every row has a compute unit of its own), which
// take no longer than a second launch; and chunks for the rest, about
// kWantBlocks workgroups of at least kChunkMin elements each (the loss of 150
// x 131072: 15 us so, 17.7 in chunks; of 300 x 131072 24.3 and 22).
constexpr int64_t kWantBlocks = 1024, kManyRows = 512, kShort = 65536;
constexpr int kChunkMin = 4096;

static int chunks_of(const sgc_distill_opts* o)
{
    int64_t n = cdiv(kWantBlocks, o->rows > 0 ? o->rows : 1);
    if (n > cdiv(o->vocab, kChunkMin)) n = cdiv(o->vocab, kChunkMin);
    if (o->rows >= kManyRows || o->vocab <= kShort * (o->rows <= 256 ? 2 : 1)) n = 1;
    if (n < cdiv(o->vocab, kChunkMax)) n = cdiv(o->vocab, kChunkMax);
    return (int)n;
}

// Chunks start at a multiple of 64 elements.
static int chunk_size(int64_t vocab, int chunks) { return (int)((cdiv(vocab, chunks) + 63) & ~(int64_t)63); }

static DistillArgs distill_args(const sgc_distill_opts* o, int64_t zs, const int32_t* idx, const float* val,
                                const float* dloss, int64_t dzs)
{
    DistillArgs a = {};
    a.rows = o->rows;
    a.zs = zs;
    a.dzs = dzs;
    a.vocab = (int32_t)o->vocab;
    a.top = o->top;
    a.mode = o->mode;
    a.scale = o->scale;
    a.c = exponent_factor(o->scale);
    a.teacher_scale = o->teacher_scale;
    a.idx = idx;
    a.val = val;
    a.dloss = dloss;
    return a;
}

template <typename T>
static int distill_grad(const DistillArgs& a, const float* stats, const T* z, T* dz, hipStream_t s)
{
    const bool once = 2 * a.rows * a.vocab * (int64_t)sizeof(T) >= kCacheBytes;
    const int chunk = a.vocab <= 2048 ? 2048 : 8192, chunks = (int)cdiv(a.vocab, chunk);
    const dim3 grid = row_grid(a.rows * chunks);
    if (a.vocab <= 2048)
        once ? k_distill_grad<T, 1, true><<<grid, 64, 0, s>>>(a, stats, z, dz, chunk, chunks)
             : k_distill_grad<T, 1, false><<<grid, 64, 0, s>>>(a, stats, z, dz, chunk, chunks);
    else
        once ? k_distill_grad<T, 4, true><<<grid, 256, 0, s>>>(a, stats, z, dz, chunk, chunks)
             : k_distill_grad<T, 4, false><<<grid, 256, 0, s>>>(a, stats, z, dz, chunk, chunks);
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}

template <typename T, int NW, int NV, bool TAIL>
static void distill_held(const DistillArgs& a, const T* z, T* dz, bool head, size_t lds, hipStream_t s)
{
    const bool once = 2 * a.rows * a.vocab * (int64_t)sizeof(T) >= kCacheBytes;
    const dim3 rows = row_grid(a.rows);
    if (once && head)
        k_distill_held<T, NW, NV, TAIL, true, true><<<rows, NW * 64, lds, s>>>(a, z, dz);
    else if (once)
        k_distill_held<T, NW, NV, TAIL, true, false><<<rows, NW * 64, lds, s>>>(a, z, dz);
    else
        k_distill_held<T, NW, NV, TAIL, false, false><<<rows, NW * 64, lds, s>>>(a, z, dz);
}

// Whether the gradient's rows start inside a 128-byte line: then held rows have
// up to 7 vectors less room.
template <typename T>
static bool has_head(const DistillArgs& a, const T* dz)
{
    return dz && ((a.rows > 1 && a.dzs * sizeof(T) % 128) || (uintptr_t)dz % 128);
}
template <typename T>
static int64_t held_vectors(const DistillArgs& a, const T* dz)
{
    return a.vocab / VecLen<T>::value + (has_head(a, dz) ? 7 : 0);
}

template <typename T, bool TAIL>
static int distill_mode(const DistillArgs& a, int chunks, const T* z, T* dz, float* part, float* stats,
                        hipStream_t s)
{
    const dim3 rows = row_grid(a.rows);
    if (chunks == 1) {
        const size_t lds = (size_t)(a.vocab + 31) / 32 * 4;
        const bool head = has_head(a, dz);
        const int64_t nv = held_vectors(a, dz);
        if (a.vocab <= 2048)
            k_distill_row<T, 1, TAIL><<<rows, 64, lds, s>>>(a, z, dz);
        else if (dz && nv <= 1024)
            distill_held<T, 4, 4, TAIL>(a, z, dz, head, lds, s);
        else if (dz && nv <= 2048)
            distill_held<T, 4, 8, TAIL>(a, z, dz, head, lds, s);
        else if (dz && nv <= 4096)
            distill_held<T, 8, 8, TAIL>(a, z, dz, head, lds, s);
        else if (dz && nv <= 6656)  // 80 registers (bf16), three workgroups a unit: 154 us; two at 16: 160
            distill_held<T, 8, 13, TAIL>(a, z, dz, head, lds, s);
        else if (dz && nv <= 8192)
            distill_held<T, 8, 16, TAIL>(a, z, dz, head, lds, s);
        else if (dz && nv <= kMostHeld)
            distill_held<T, 16, 16, TAIL>(a, z, dz, head, lds, s);
        else if (a.rows >= kManyRows && nv <= 1536)  // the loss of 8000 x 10000 bf16: 40 us, by four waves 45
            k_distill_row<T, 2, TAIL><<<rows, 128, lds, s>>>(a, z, dz);
        else if (a.vocab <= 16384)
            k_distill_row<T, 4, TAIL><<<rows, 256, lds, s>>>(a, z, dz);
        else if (a.rows >= kManyRows)
            k_distill_row<T, 8, TAIL><<<rows, 512, lds, s>>>(a, z, dz);
        else
            k_distill_row<T, 16, TAIL><<<rows, 1024, lds, s>>>(a, z, dz);
        SGC_LAUNCH_CHECK();
        return SGC_OK;
    }
    const int chunk = chunk_size(a.vocab, chunks);
    const int used = (int)cdiv(a.vocab, chunk);
    k_distill_part<T, 4, TAIL><<<row_grid(a.rows * used), 256, (size_t)chunk / 8, s>>>(a, z, chunk, used, part);
    SGC_LAUNCH_CHECK();
    DistillArgs j = a;
    j.stats = stats;
    k_distill_join<T, 4, TAIL><<<rows, 256, 0, s>>>(j, z, used, part);
    SGC_LAUNCH_CHECK();
    return dz ? distill_grad<T>(a, stats, z, dz, s) : SGC_OK;
}

template <typename T>
static int distill(const sgc_distill_opts* o, const void* z, int64_t zs, const int32_t* idx, const float* val,
                   float* loss, float* stats, const float* dloss, void* dz, int64_t dzs, uint32_t* dstatus, void* ws,
                   hipStream_t s)
{
    DistillArgs a = distill_args(o, zs, idx, val, dloss, dzs);
    a.loss = loss;
    a.stats = stats;
    a.dstatus = dstatus;
    int chunks = chunks_of(o);
    if (dz && held_vectors(a, (const T*)dz) <= kMostHeld) chunks = 1;
    float* part = nullptr;
    if (chunks > 1) {
        Carver c(ws);
        part = c.take<float>(3 * o->rows * chunks);
        float* own = c.take<float>(4 * o->rows);
        if (!stats) stats = own;
    }
    return o->mode == SGC_DISTILL_TAIL ? distill_mode<T, true>(a, chunks, (const T*)z, (T*)dz, part, stats, s)
                                       : distill_mode<T, false>(a, chunks, (const T*)z, (T*)dz, part, stats, s);
}

template <typename T>
static int distill_back(const sgc_distill_opts* o, const void* z, int64_t zs, const int32_t* idx, const float* val,
                        const float* stats, const float* dloss, void* dz, int64_t dzs, hipStream_t s)
{
    return distill_grad<T>(distill_args(o, zs, idx, val, dloss, dzs), stats, (const T*)z, (T*)dz, s);
}

}  // namespace sgc

using namespace sgc;

extern "C" size_t sgc_distill_workspace(const sgc_distill_opts* o)
{
    if (!distill_opts_ok(o)) return 0;
    const int chunks = chunks_of(o);
    if (chunks == 1) return SGC_LM_WS_NONE;
    Carver c(nullptr);
    c.take<float>(3 * o->rows * chunks);
    c.take<float>(4 * o->rows);
    return c.off;
}

extern "C" int sgc_distill(const sgc_distill_opts* o, const void* logits, int64_t stride, const int32_t* t_idx,
                           const float* t_val, float* loss, float* stats, const float* dloss, void* dlogits,
                           int64_t dstride, uint32_t* dstatus, void* ws, size_t ws_bytes, sgc_stream_t stream)
{
    if (!distill_opts_ok(o)) return SGC_EINVAL;
    if (o->rows == 0) return SGC_OK;
    if (!lm_rows_ok(logits, stride, o->rows, o->vocab, o->dtype, false)) return SGC_EINVAL;
    if (!entries_ok(t_idx, t_val) || !loss) return SGC_EINVAL;
    if (dlogits && !lm_rows_ok(dlogits, dstride, o->rows, o->vocab, o->dtype, true)) return SGC_EINVAL;
    if (!lm_aligned(loss, 4) || !lm_aligned(stats, 4) || !lm_aligned(dloss, 4) || !lm_aligned(dstatus, 4))
        return SGC_EINVAL;
    const size_t need = sgc_distill_workspace(o);
    if (need != SGC_LM_WS_NONE) {
        if (!ws || ws_bytes < need) return SGC_ENOSPC;
        if (!aligned16(ws)) return SGC_EINVAL;
    }
    const hipStream_t s = (hipStream_t)stream;
    return o->dtype == SGC_F32
               ? distill<float>(o, logits, stride, t_idx, t_val, loss, stats, dloss, dlogits, dstride, dstatus, ws, s)
           : o->dtype == SGC_BF16
               ? distill<bf16_t>(o, logits, stride, t_idx, t_val, loss, stats, dloss, dlogits, dstride, dstatus, ws, s)
               : distill<f16_t>(o, logits, stride, t_idx, t_val, loss, stats, dloss, dlogits, dstride, dstatus, ws, s);
}

extern "C" int sgc_distill_backward(const sgc_distill_opts* o, const void* logits, int64_t stride,
                                    const int32_t* t_idx, const float* t_val, const float* stats, const float* dloss,
                                    void* dlogits, int64_t dstride, sgc_stream_t stream)
{
    if (!distill_opts_ok(o)) return SGC_EINVAL;
    if (o->rows == 0) return SGC_OK;
    if (!lm_rows_ok(logits, stride, o->rows, o->vocab, o->dtype, false)) return SGC_EINVAL;
    if (!lm_rows_ok(dlogits, dstride, o->rows, o->vocab, o->dtype, true)) return SGC_EINVAL;
    if (!entries_ok(t_idx, t_val) || !stats || !lm_aligned(stats, 4) || !lm_aligned(dloss, 4)) return SGC_EINVAL;
    const hipStream_t s = (hipStream_t)stream;
    return o->dtype == SGC_F32
               ? distill_back<float>(o, logits, stride, t_idx, t_val, stats, dloss, dlogits, dstride, s)
           : o->dtype == SGC_BF16
               ? distill_back<bf16_t>(o, logits, stride, t_idx, t_val, stats, dloss, dlogits, dstride, s)
               : distill_back<f16_t>(o, logits, stride, t_idx, t_val, stats, dloss, dlogits, dstride, s);
}
