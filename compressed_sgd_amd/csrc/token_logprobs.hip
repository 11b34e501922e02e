// token_logprobs.hip -- log probabilities of given tokens with entropy and
// the top alternatives of every row, and their gradient.
//
//   y_i = scale (z_i - m),  m = max z,  s = sum exp(y)
//   log p_i = y_i - ln s,   H = ln s - sum(exp(y) y) / s
//   dz_i = scale (g ([i = token] - p_i) - h p_i (log p_i + H))
#include "lm_common.h"

namespace sgc {

constexpr int kLpThreads = 256;
constexpr int kLpWaves = kLpThreads / 64;

__device__ inline int64_t token_at(const void* tokens, int type, int64_t r)
{
    return type == SGC_TOKEN_I64 ? ((const int64_t*)tokens)[r] : (int64_t)((const int32_t*)tokens)[r];
}

template <typename T>
__global__ __launch_bounds__(kLpThreads) void k_logprobs(const T* z, int64_t zs, const void* tokens, int token_type,
                                                         int64_t rows, int64_t vocab, float scale, int top,
                                                         float* logp, float* entropy, float* stats, int32_t* top_idx,
                                                         float* top_logp, uint32_t* dstatus)
{
    __shared__ float tmp[kLpWaves];
    __shared__ unsigned long long best;
    const int64_t r = row_of_block();
    if (r >= rows) return;
    const T* zr = z + r * zs;
    float m = -INFINITY;
    for (int64_t i = threadIdx.x; i < vocab; i += kLpThreads) m = fmaxf(m, to_f(zr[i]));
    m = block_max<kLpWaves>(m, tmp);
    const float base = m == -INFINITY ? 0.f : m;
    float s = 0.f, t = 0.f;
    for (int64_t i = threadIdx.x; i < vocab; i += kLpThreads) {
        const float y = (to_f(zr[i]) - base) * scale;
        const float e = expf(y);
        s += e;
        t = fmaf(e, fmaxf(y, -1e4f), t);
    }
    s = block_sum<kLpWaves>(s, tmp);
    t = block_sum<kLpWaves>(t, tmp);
    const float ln_s = logf(s);
    const bool none = s == 0.f;
    if (threadIdx.x == 0) {
        if (stats) {
            stats[2 * r] = m;
            stats[2 * r + 1] = s;
        }
        if (entropy) entropy[r] = none ? 0.f : ln_s - t / s;
        if (logp) {
            const int64_t tok = token_at(tokens, token_type, r);
            float lp = 0.f;
            if (tok >= vocab) {
                lp = NAN;
                if (dstatus) atomicOr(dstatus, SGC_STATUS_BAD_INPUT);
            } else if (tok >= 0) {
                lp = none ? -INFINITY : (to_f(zr[tok]) - base) * scale - ln_s;
            }
            logp[r] = lp;
        }
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < top; ++k) {
        if (threadIdx.x == 0) best = 0;
        __syncthreads();
        unsigned long long mine = 0;
        for (int64_t i = threadIdx.x; i < vocab; i += kLpThreads) {
            const unsigned long long key = order_key(to_f(zr[i]), (uint32_t)i);
            if ((key < last || k == 0) && key > mine) mine = key;
        }
        atomicMax(&best, mine);
        __syncthreads();
        last = best;
        if (threadIdx.x == 0) {
            const uint32_t at = ~(uint32_t)last;
            top_idx[r * top + k] = (int32_t)at;
            top_logp[r * top + k] = none ? -INFINITY : (to_f(zr[at]) - base) * scale - ln_s;
        }
        __syncthreads();
    }
}

template <typename T>
__global__ __launch_bounds__(kLpThreads) void k_logprobs_back(const T* z, int64_t zs, const void* tokens,
                                                              int token_type, int64_t rows, int64_t vocab, float scale,
                                                              const float* stats, const float* entropy,
                                                              const float* dlogp, const float* dentropy, T* dz,
                                                              int64_t dzs)
{
    const int64_t r = row_of_block();
    if (r >= rows) return;
    const T* zr = z + r * zs;
    T* out = dz + r * dzs;
    const float m = stats[2 * r], s = stats[2 * r + 1];
    const int64_t tok = tokens ? token_at(tokens, token_type, r) : -1;
    const float g = dlogp && tok >= 0 && tok < vocab ? dlogp[r] : 0.f;
    const float h = dentropy ? dentropy[r] : 0.f;
    const float H = dentropy ? entropy[r] : 0.f;
    const bool zero = (g == 0.f && h == 0.f) || s == 0.f;
    const float ln_s = logf(s);
    for (int64_t i = threadIdx.x; i < vocab; i += kLpThreads) {
        float d = 0.f;
        if (!zero) {
            const float y = (to_f(zr[i]) - m) * scale;
            const float p = expf(y) / s;
            d = -p * (g + h * (fmaxf(y, -1e4f) - ln_s + H));
            if (i == tok) d += g;
            d *= scale;
        }
        out[i] = from_f<T>(d);
    }
}

static bool logprob_opts_ok(const sgc_logprob_opts* o)
{
    return o && o->rows >= 0 && o->rows < ((int64_t)1 << 31) && o->vocab >= 1 && o->vocab < ((int64_t)1 << 31) &&
           lm_dtype(o->dtype) && (o->token_type == SGC_TOKEN_I32 || o->token_type == SGC_TOKEN_I64) && o->top >= 0 &&
           o->top <= SGC_TOP_MAX && o->top <= o->vocab && o->scale > 0.f && std::isfinite(o->scale);
}

static bool tokens_ok(const sgc_logprob_opts* o, const void* tokens)
{
    return tokens && lm_aligned(tokens, o->token_type == SGC_TOKEN_I64 ? 8 : 4);
}

template <typename T>
static int logprobs(const sgc_logprob_opts* o, const void* z, int64_t zs, const void* tokens, float* logp,
                    float* entropy, float* stats, int32_t* top_idx, float* top_logp, uint32_t* dstatus, hipStream_t s)
{
    k_logprobs<T><<<row_grid(o->rows), kLpThreads, 0, s>>>((const T*)z, zs, tokens, o->token_type, o->rows, o->vocab,
                                                           o->scale, o->top, logp, entropy, stats, top_idx, top_logp,
                                                           dstatus);
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}

template <typename T>
static int logprobs_back(const sgc_logprob_opts* o, const void* z, int64_t zs, const void* tokens, const float* stats,
                         const float* entropy, const float* dlogp, const float* dentropy, void* dz, int64_t dzs,
                         hipStream_t s)
{
    k_logprobs_back<T><<<row_grid(o->rows), kLpThreads, 0, s>>>((const T*)z, zs, tokens, o->token_type, o->rows,
                                                                o->vocab, o->scale, stats, entropy, dlogp, dentropy,
                                                                (T*)dz, dzs);
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}

}  // namespace sgc

using namespace sgc;

extern "C" size_t sgc_token_logprobs_workspace(const sgc_logprob_opts* o)
{
    if (!logprob_opts_ok(o)) return 0;
    return SGC_LM_WS_NONE;
}

extern "C" int sgc_token_logprobs(const sgc_logprob_opts* o, const void* logits, int64_t stride, const void* tokens,
                                  float* logp, float* entropy, float* stats, int32_t* top_idx, float* top_logp,
                                  uint32_t* dstatus, void* ws, size_t ws_bytes, sgc_stream_t stream)
{
    if (!logprob_opts_ok(o)) return SGC_EINVAL;
    if (o->rows == 0) return SGC_OK;
    if (!lm_rows_ok(logits, stride, o->rows, o->vocab, o->dtype, false)) return SGC_EINVAL;
    if ((tokens == nullptr) != (logp == nullptr) || (tokens && !tokens_ok(o, tokens))) return SGC_EINVAL;
    if (o->top && (!top_idx || !top_logp)) return SGC_EINVAL;
    if (!lm_aligned(logp, 4) || !lm_aligned(entropy, 4) || !lm_aligned(stats, 4) || !lm_aligned(top_idx, 4) ||
        !lm_aligned(top_logp, 4) || !lm_aligned(dstatus, 4))
        return SGC_EINVAL;
    const size_t need = sgc_token_logprobs_workspace(o);
    if (need != SGC_LM_WS_NONE) {
        if (!ws || ws_bytes < need) return SGC_ENOSPC;
        if (!aligned16(ws)) return SGC_EINVAL;
    }
    const hipStream_t s = (hipStream_t)stream;
    return o->dtype == SGC_F32
               ? logprobs<float>(o, logits, stride, tokens, logp, entropy, stats, top_idx, top_logp, dstatus, s)
           : o->dtype == SGC_BF16
               ? logprobs<bf16_t>(o, logits, stride, tokens, logp, entropy, stats, top_idx, top_logp, dstatus, s)
               : logprobs<f16_t>(o, logits, stride, tokens, logp, entropy, stats, top_idx, top_logp, dstatus, s);
}

extern "C" int sgc_token_logprobs_backward(const sgc_logprob_opts* o, const void* logits, int64_t stride,
                                           const void* tokens, const float* stats, const float* entropy,
                                           const float* dlogp, const float* dentropy, void* dlogits, int64_t dstride,
                                           sgc_stream_t stream)
{
    if (!logprob_opts_ok(o)) return SGC_EINVAL;
    if (o->rows == 0) return SGC_OK;
    if (!lm_rows_ok(logits, stride, o->rows, o->vocab, o->dtype, false)) return SGC_EINVAL;
    if (!lm_rows_ok(dlogits, dstride, o->rows, o->vocab, o->dtype, true)) return SGC_EINVAL;
    if (!stats || (dlogp && !tokens_ok(o, tokens)) || (dentropy && !entropy)) return SGC_EINVAL;
    if (!lm_aligned(stats, 4) || !lm_aligned(entropy, 4) || !lm_aligned(dlogp, 4) || !lm_aligned(dentropy, 4))
        return SGC_EINVAL;
    if (!dlogp) tokens = nullptr;
    const hipStream_t s = (hipStream_t)stream;
    return o->dtype == SGC_F32
               ? logprobs_back<float>(o, logits, stride, tokens, stats, entropy, dlogp, dentropy, dlogits, dstride, s)
           : o->dtype == SGC_BF16
               ? logprobs_back<bf16_t>(o, logits, stride, tokens, stats, entropy, dlogp, dentropy, dlogits, dstride, s)
               : logprobs_back<f16_t>(o, logits, stride, tokens, stats, entropy, dlogp, dentropy, dlogits, dstride, s);
}
