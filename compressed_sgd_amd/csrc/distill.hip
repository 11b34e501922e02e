// distill.hip -- divergence of a student's distribution from a teacher's top
// entries, loss and gradient.
//
//   e_i = exp(scale (z_i - m)),  s = sum e,  o = sum of e outside the entries
//   loss = sum_j t_j (log t_j - log q_j) + u (log u - log(o / s)),  q = e / s
//   dz_i = scale g ((T + u) q_i - t_i)          entries,  T = sum_j t_j
//   dz_i = scale g ((T + u) q_i - u e_i / o)    else
// where q_i o / s ... the derivative of the last term of the loss by an outer
// logit is u (q_i - e_i / o): the rest's share that the logit has of it.
#include "lm_common.h"

namespace sgc {

constexpr int kDiThreads = 256;
constexpr int kDiWaves = kDiThreads / 64;
static_assert(SGC_TOP_MAX <= kDiThreads, "one thread an entry");

// The row's entries in shared memory, and the teacher's side of them.
struct Entries {
    int32_t idx[SGC_TOP_MAX];
    float t[SGC_TOP_MAX];
    int bad;
};

// Loads the entries of a row (bounds and repeats checked: en.bad) and gives
// T and u; log t_j of the thread's own entry in *log_t.
__device__ inline void load_entries(Entries& en, const int32_t* idx, const float* val, int top, int64_t vocab, int mode,
                                    float teacher_scale, float* tmp, float* T, float* u, float* log_t)
{
    const int j = threadIdx.x;
    if (j == 0) en.bad = 0;
    __syncthreads();
    const int32_t at = j < top ? idx[j] : -1;
    float v = -INFINITY;
    if (j < top) {
        en.idx[j] = at;
        if (at < -1 || at >= vocab) en.bad = 1;
        if (at >= 0) v = val[j] * teacher_scale;
    }
    __syncthreads();
    if (at >= 0)
        for (int i = 0; i < j; ++i)
            if (en.idx[i] == at) en.bad = 1;
    float lt = v;
    if (mode == SGC_DISTILL_RENORM) {
        const float m = block_max<kDiWaves>(v, tmp);
        const float d = v - (m == -INFINITY ? 0.f : m);
        const float sum = block_sum<kDiWaves>(expf(d), tmp);
        lt = sum == 0.f ? -INFINITY : d - logf(sum);
    }
    const float t = expf(lt);
    if (j < top) en.t[j] = t;
    *log_t = lt;
    const float total = block_sum<kDiWaves>(t, tmp);  // its barriers make t and bad visible
    *T = mode == SGC_DISTILL_RENORM ? (total > 0.f ? 1.f : total) : total;
    *u = mode == SGC_DISTILL_RENORM ? 0.f : fmaxf(0.f, 1.f - total);
}

__device__ inline int find_entry(const Entries& en, int top, int64_t i)
{
    int at = -1;
    for (int j = 0; j < top; ++j)
        if (en.idx[j] == i) at = j;
    return at;
}

template <typename T>
__device__ inline void write_gradient(const Entries& en, int top, const T* zr, T* out, int64_t vocab, float scale,
                                      float g, float m, float s, float o, float mass, float u, bool skip)
{
    const float a = mass / s, b = o > 0.f ? u / o : 0.f;
    for (int64_t i = threadIdx.x; i < vocab; i += kDiThreads) {
        float d = 0.f;
        if (!skip) {
            const float e = expf((to_f(zr[i]) - m) * scale);
            const int at = find_entry(en, top, i);
            d = at >= 0 ? e * a - en.t[at] : e * (a - b);
            d *= scale * g;
        }
        out[i] = from_f<T>(d);
    }
}

template <typename T>
__global__ __launch_bounds__(kDiThreads) void k_distill(const T* z, int64_t zs, const int32_t* idx, const float* val,
                                                        int64_t rows, int64_t vocab, int top, int mode, float scale,
                                                        float teacher_scale, float* loss, float* stats,
                                                        const float* dloss, T* dz, int64_t dzs, uint32_t* dstatus)
{
    __shared__ float tmp[kDiWaves];
    __shared__ Entries en;
    const int64_t r = row_of_block();
    if (r >= rows) return;
    const T* zr = z + r * zs;
    float mass, u, log_t;
    load_entries(en, idx + r * top, val + r * top, top, vocab, mode, teacher_scale, tmp, &mass, &u, &log_t);
    const bool bad = en.bad != 0;
    float m = -INFINITY;
    for (int64_t i = threadIdx.x; i < vocab; i += kDiThreads) m = fmaxf(m, to_f(zr[i]));
    m = block_max<kDiWaves>(m, tmp);
    const float base = m == -INFINITY ? 0.f : m;
    float o = 0.f;
    for (int64_t i = threadIdx.x; i < vocab; i += kDiThreads)
        if (find_entry(en, top, i) < 0) o += expf((to_f(zr[i]) - base) * scale);
    o = block_sum<kDiWaves>(o, tmp);
    const int j = threadIdx.x;
    const bool has = j < top && !bad && en.idx[j] >= 0;
    const float y = has ? (to_f(zr[en.idx[j]]) - base) * scale : -INFINITY;
    const float s = o + block_sum<kDiWaves>(has ? expf(y) : 0.f, tmp);
    const float ln_s = logf(s);
    const float t = has ? en.t[j] : 0.f;
    float l = block_sum<kDiWaves>(has && t != 0.f ? t * (log_t - (y - ln_s)) : 0.f, tmp);
    if (u > 0.f && o != 0.f) l += u * (logf(u) - (logf(o) - ln_s));
    const bool skip = bad || s == 0.f || (mode == SGC_DISTILL_RENORM && mass == 0.f);
    if (threadIdx.x == 0) {
        loss[r] = bad ? NAN : skip ? 0.f : l;
        if (stats) {
            stats[4 * r] = m;
            stats[4 * r + 1] = s;
            stats[4 * r + 2] = o;
            stats[4 * r + 3] = skip ? 0.f : 1.f;
        }
        if (bad && dstatus) atomicOr(dstatus, SGC_STATUS_CORRUPT);
    }
    if (dz) {
        const float g = dloss ? dloss[r] : 1.f;
        __syncthreads();
        write_gradient<T>(en, top, zr, dz + r * dzs, vocab, scale, g, base, s, o, mass + u, u, skip || g == 0.f);
    }
}

template <typename T>
__global__ __launch_bounds__(kDiThreads) void k_distill_back(const T* z, int64_t zs, const int32_t* idx,
                                                             const float* val, int64_t rows, int64_t vocab, int top,
                                                             int mode, float scale, float teacher_scale,
                                                             const float* stats, const float* dloss, T* dz,
                                                             int64_t dzs)
{
    __shared__ float tmp[kDiWaves];
    __shared__ Entries en;
    const int64_t r = row_of_block();
    if (r >= rows) return;
    float mass, u, log_t;
    load_entries(en, idx + r * top, val + r * top, top, vocab, mode, teacher_scale, tmp, &mass, &u, &log_t);
    const float g = dloss ? dloss[r] : 1.f;
    write_gradient<T>(en, top, z + r * zs, dz + r * dzs, vocab, scale, g, stats[4 * r], stats[4 * r + 1],
                      stats[4 * r + 2], mass + u, u, stats[4 * r + 3] == 0.f || en.bad || g == 0.f);
}

static bool distill_opts_ok(const sgc_distill_opts* o)
{
    return o && o->rows >= 0 && o->rows < ((int64_t)1 << 31) && o->vocab >= 1 && o->vocab < ((int64_t)1 << 31) &&
           lm_dtype(o->dtype) && o->top >= 1 && o->top <= SGC_TOP_MAX &&
           (o->mode == SGC_DISTILL_RENORM || o->mode == SGC_DISTILL_TAIL) && o->scale > 0.f &&
           std::isfinite(o->scale) && o->teacher_scale > 0.f && std::isfinite(o->teacher_scale) &&
           (o->mode != SGC_DISTILL_TAIL || o->teacher_scale == 1.f) && o->reserved == 0;
}

static bool entries_ok(const int32_t* idx, const float* val)
{
    return idx && val && lm_aligned(idx, 4) && lm_aligned(val, 4);
}

template <typename T>
static int distill(const sgc_distill_opts* o, const void* z, int64_t zs, const int32_t* idx, const float* val,
                   float* loss, float* stats, const float* dloss, void* dz, int64_t dzs, uint32_t* dstatus,
                   hipStream_t s)
{
    k_distill<T><<<row_grid(o->rows), kDiThreads, 0, s>>>((const T*)z, zs, idx, val, o->rows, o->vocab, o->top,
                                                          o->mode, o->scale, o->teacher_scale, loss, stats, dloss,
                                                          (T*)dz, dzs, dstatus);
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}

template <typename T>
static int distill_back(const sgc_distill_opts* o, const void* z, int64_t zs, const int32_t* idx, const float* val,
                        const float* stats, const float* dloss, void* dz, int64_t dzs, hipStream_t s)
{
    k_distill_back<T><<<row_grid(o->rows), kDiThreads, 0, s>>>((const T*)z, zs, idx, val, o->rows, o->vocab, o->top,
                                                               o->mode, o->scale, o->teacher_scale, stats, dloss,
                                                               (T*)dz, dzs);
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}

}  // namespace sgc

using namespace sgc;

extern "C" size_t sgc_distill_workspace(const sgc_distill_opts* o)
{
    if (!distill_opts_ok(o)) return 0;
    return SGC_LM_WS_NONE;
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
               ? distill<float>(o, logits, stride, t_idx, t_val, loss, stats, dloss, dlogits, dstride, dstatus, s)
           : o->dtype == SGC_BF16
               ? distill<bf16_t>(o, logits, stride, t_idx, t_val, loss, stats, dloss, dlogits, dstride, dstatus, s)
               : distill<f16_t>(o, logits, stride, t_idx, t_val, loss, stats, dloss, dlogits, dstride, dstatus, s);
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
