// token_logprobs.hip -- log probabilities of given tokens with entropy and
// the top alternatives of every row, and their gradient.
//
//   y_i = scale (z_i - m),  m = max z,  s = sum exp(y)
//   log p_i = y_i - ln s,   H = ln s - sum(exp(y) y) / s
//   dz_i = scale (g ([i = token] - p_i) - h p_i (log p_i + H))
//
// The alternatives cost the pass over the row nothing: each thread's running
// maximum, which the softmax needs anyway, is a filter.  At least `top`
// elements reach the top-th largest of the threads' maxima, few others do,
// and only the threads whose own maximum reaches it hold any: their elements
// are read again (from the cache), the ones that reach it are ranked by
// counting.
#include "lm_softmax.h"

namespace sgc {

struct LogprobArgs {
    int64_t rows, zs;
    int32_t vocab, top, token_type;
    float scale, c;
    const void* tokens;
    float* logp;
    float* entropy;
    float* stats;
    int32_t* top_idx;
    float* top_logp;
    uint32_t* dstatus;
};

__device__ inline int64_t token_at(const void* tokens, int type, int64_t r)
{
    return type == SGC_TOKEN_I64 ? ((const int64_t*)tokens)[r] : (int64_t)((const int32_t*)tokens)[r];
}

// The value an order key was made of (the two zeros as +0, any NaN as one).
__device__ inline float key_value(uint32_t k)
{
    if (k == 0xffffffffu) return NAN;
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// Candidates in shared memory: the fallback adds two a thread to a kept list.
template <int NW>
struct Candidates {
    static constexpr int NT = NW * 64;
    static constexpr int kCap = 2 * NT + SGC_TOP_MAX;
    uint64_t key[kCap];
    uint64_t sorted[SGC_TOP_MAX];
    uint32_t peak[NT];  // the threads' maxima as order keys, then the threads that hold candidates
    int n, threads;
    uint32_t bar;
};

// sorted[0 .. min(n, top)) = the largest of key[0 .. n), largest first: each
// key's place is the number of larger ones (keys are unique).
template <int NW>
__device__ inline void rank_keys(Candidates<NW>& cd, int n, int top)
{
    for (int i = threadIdx.x; i < n; i += NW * 64) {
        const uint64_t k = cd.key[i];
        int place = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) place += cd.key[j] > k;
        if (place < top) cd.sorted[place] = k;
    }
    __syncthreads();
}

// The `top` best of any row, one pass in order of the places: a full list is
// cut to its best, whose last key later elements have to pass.  For rows with
// NaN or +inf, or with so many equal values that the filter lets too many
// through.  Returns how many there are (less than top in a short row).
template <int NW, typename K>
__device__ inline int top_in_order(Candidates<NW>& cd, const K& key_at, int len, int top)
{
    constexpr int NT = NW * 64;
    uint64_t bar = 0;
    if (threadIdx.x == 0) cd.n = 0;
    __syncthreads();
    int n = 0;
    for (int i0 = 0; i0 < len; i0 += 2 * NT) {
        if (n > SGC_TOP_MAX) {
            rank_keys<NW>(cd, n, top);
            bar = cd.sorted[top - 1];  // n > top
            for (int j = threadIdx.x; j < top; j += NT) cd.key[j] = cd.sorted[j];
            if (threadIdx.x == 0) cd.n = top;
            __syncthreads();
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = i0 + e * NT + threadIdx.x;
            const uint64_t k = i < len ? key_at(i) : 0;
            if (k > bar) cd.key[atomicAdd(&cd.n, 1)] = k;
        }
        __syncthreads();
        n = cd.n;
        __syncthreads();
    }
    rank_keys<NW>(cd, n, top);
    return n < top ? n : top;
}

// The largest value of 16 leading bits that `top` of the threads' keys reach (0
// if there are fewer threads); clears the candidates.
template <int NW>
__device__ inline uint32_t bar_of(Candidates<NW>& cd, uint32_t key, int top)
{
    cd.peak[threadIdx.x] = key;
    if (threadIdx.x == 0) cd.n = cd.threads = 0;
    __syncthreads();
    if (threadIdx.x < 64) {
        uint32_t k[NW], bar = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) k[w] = cd.peak[w * 64 + threadIdx.x];
        if (top <= NW * 64)
            for (int b = 31; b >= 16; --b) {
                const uint32_t to = bar | (1u << b);
                int reach = 0;
#pragma unroll
                for (int w = 0; w < NW; ++w) reach += __popcll(__ballot(k[w] >= to));
                if (reach >= top) bar = to;
            }
        if (threadIdx.x == 0) cd.bar = bar;
    }
    __syncthreads();
    return cd.bar;
}

// The `top` best elements of z[0, len) into cd.sorted as order keys with their
// places from `first` on.  m: the thread's maximum over its elements, those of
// stream_sums.  Returns how many.
template <typename T, int NW>
__device__ inline int top_of(Candidates<NW>& cd, const T* z, int len, int first, int top, float m, bool broken)
{
    constexpr int NT = NW * 64, VL = VecLen<T>::value;
    const int nv = len / VL;
    if (!broken) {
        // A short row's vectors are too few for a filter: its elements then go
        // to the threads one by one (4756 x 440 fp16 top 64: 21 us, without 113).
        const bool single = nv < NT && nv < 4 * top;
        if (single) {
            m = -INFINITY;
            for (int i = threadIdx.x; i < len; i += NT) m = fmaxf(m, to_f(z[i]));
        }
        const uint32_t bar = bar_of<NW>(cd, order_key(m), top);
        const float low = bar < 0x00800000u ? -INFINITY : key_value(bar);
        const bool holds = m >= low;
        const auto offer = [&](float x, int i) {
            if (x >= low) {
                const int at = atomicAdd(&cd.n, 1);
                if (at < cd.kCap) cd.key[at] = order_key(x, (uint32_t)(first + i));
            }
        };
        if (single) {
            if (holds)
                for (int i = threadIdx.x; i < len; i += NT) offer(to_f(z[i]), i);
        } else {
            if (holds) cd.peak[atomicAdd(&cd.threads, 1)] = threadIdx.x;
            __syncthreads();
            // 2^g threads take a holding thread's vectors, and its element past them
            const int per = (nv + NT - 1) / NT;
            int g = 0;
            while (g < 6 && (1 << g) <= per) ++g;
            for (int f = threadIdx.x >> g; f < cd.threads; f += NT >> g) {
                const int th = (int)cd.peak[f];
                for (int k = threadIdx.x & ((1 << g) - 1); k <= per; k += 1 << g) {
                    const int at = th + k * NT;
                    if (k < per && at < nv) {
                        float x[VL];
                        unpack<T>(((const Raw*)z)[at], x);
#pragma unroll
                        for (int e = 0; e < VL; ++e) offer(x[e], at * VL + e);
                    }
                    if (k == per && nv * VL + th < len) offer(to_f(z[nv * VL + th]), nv * VL + th);
                }
            }
        }
        __syncthreads();
        const int n = cd.n;
        if (n <= cd.kCap) {
            rank_keys<NW>(cd, n, top);
            return n < top ? n : top;
        }
        __syncthreads();
    }
    return top_in_order<NW>(
        cd, [&](int i) { return order_key(to_f(z[i]), (uint32_t)(first + i)); }, len, top);
}

// What a row's sums give: logp, entropy, stats; ln s and the base of y.
__device__ inline void finish_row(const LogprobArgs& a, int64_t r, float z_tok, int64_t tok, const Sums& sum,
                                  float ln_s)
{
    const bool none = sum.s == 0.f;
    if (a.stats) {
        a.stats[2 * r] = sum.m;
        a.stats[2 * r + 1] = sum.s;
    }
    if (a.entropy) a.entropy[r] = none ? 0.f : ln_s - kLn2 * (sum.t / sum.s);
    if (a.logp) {
        float lp = 0.f;
        if (tok >= a.vocab) {
            lp = NAN;
            if (a.dstatus) atomicOr(a.dstatus, SGC_STATUS_BAD_INPUT);
        } else if (tok >= 0) {
            lp = none ? -INFINITY : (z_tok - finite_base(sum.m)) * a.scale - ln_s;
        }
        a.logp[r] = lp;
    }
}

__device__ inline void write_top(const LogprobArgs& a, int64_t r, int k, uint64_t key, const Sums& sum, float ln_s)
{
    const float v = key_value((uint32_t)(key >> 32));
    a.top_idx[r * a.top + k] = (int32_t)~(uint32_t)key;
    a.top_logp[r * a.top + k] = sum.s == 0.f ? -INFINITY : (v - finite_base(sum.m)) * a.scale - ln_s;
}

// A row a workgroup.  Bound by memory for long rows (4096 x 131072 bf16 top 8:
// 184 us, 5.8 of the 6.25 TB/s of a bare read, the vector unit 82% busy), by
// one row's chain of trips and barriers for few (4 x 50000 top 20: 11.6 us).
template <typename T, int NW, bool ONCE>
__global__ __launch_bounds__(NW * 64) void k_lp_row(LogprobArgs a, const T* z)
{
    __shared__ Candidates<NW> cd;
    __shared__ float tmp[NW][3];
    const int64_t r = row_of_block();
    if (r >= a.rows) return;
    const T* zr = z + r * a.zs;
    int64_t tok = -1;
    float z_tok = 0.f;
    if (threadIdx.x == 0 && a.logp) {
        tok = token_at(a.tokens, a.token_type, r);
        if (tok >= 0 && tok < a.vocab) z_tok = to_f(zr[tok]);
    }
    float m;
    const Sums sum = row_softmax<T, NW, true, false, ONCE>(zr, a.vocab, a.c, nullptr, tmp, &m);
    const float ln_s = logf(sum.s);
    if (threadIdx.x == 0) finish_row(a, r, z_tok, tok, sum, ln_s);
    if (a.top) {
        const int n = top_of<T, NW>(cd, zr, a.vocab, 0, a.top, m, !(sum.s < INFINITY));
        for (int k = threadIdx.x; k < n; k += NW * 64) write_top(a, r, k, cd.sorted[k], sum, ln_s);
    }
}

// A chunk of a row: its sums in part [rows, chunks, 4], its best elements in
// keys [rows, chunks, top] (0: none).  300 x 131072 bf16 top 20: 24 us, join 6.
template <typename T, int NW>
__global__ __launch_bounds__(NW * 64) void k_lp_part(LogprobArgs a, const T* z, int chunk, int chunks, float* part,
                                                     uint64_t* keys)
{
    __shared__ Candidates<NW> cd;
    __shared__ float tmp[NW][3];
    const int64_t b = row_of_block(), r = b / chunks;
    if (r >= a.rows) return;
    const int z0 = (int)(b - r * chunks) * chunk, len = a.vocab - z0 < chunk ? a.vocab - z0 : chunk;
    const T* zr = z + r * a.zs + z0;
    float m;
    const Sums sum = row_softmax<T, NW, true, false, false>(zr, len, a.c, nullptr, tmp, &m);
    if (threadIdx.x == 0) {
        part[4 * b] = sum.m;
        part[4 * b + 1] = sum.s;
        part[4 * b + 2] = sum.t;
    }
    if (a.top) {
        const int n = top_of<T, NW>(cd, zr, len, z0, a.top, m, !(sum.s < INFINITY));
        for (int k = threadIdx.x; k < a.top; k += NW * 64) keys[b * a.top + k] = k < n ? cd.sorted[k] : 0;
    }
}

// The chunks of a row joined.  A call of few rows is a chain of trips to
// memory: everything it may need of the first trip is asked for at once.
template <typename T, int NW>
__global__ __launch_bounds__(NW * 64) void k_lp_join(LogprobArgs a, const T* z, int chunks, const float* part,
                                                     const uint64_t* keys)
{
    constexpr int NT = NW * 64, kFirst = 2;
    __shared__ Candidates<NW> cd;
    __shared__ float tmp[NW][3];
    const int64_t r = row_of_block();
    if (r >= a.rows) return;
    const uint64_t* kr = keys + r * chunks * a.top;
    const int len = chunks * a.top;
    uint64_t mine[kFirst];
#pragma unroll
    for (int e = 0; e < kFirst; ++e) mine[e] = e * NT + (int)threadIdx.x < len ? kr[e * NT + threadIdx.x] : 0;
    int64_t tok = -1;
    float z_tok = 0.f;
    if (threadIdx.x == 0 && a.logp) {
        tok = token_at(a.tokens, a.token_type, r);
        if (tok >= 0 && tok < a.vocab) z_tok = to_f(z[r * a.zs + tok]);
    }
    const Sums sum = join_parts<NW, true>(part + 4 * r * chunks, chunks, a.c, tmp);
    const float ln_s = logf(sum.s);
    if (a.top) {
        // the chunks' keys are cut as a row's elements are
        uint64_t most = 0;
#pragma unroll
        for (int e = 0; e < kFirst; ++e) most = mine[e] > most ? mine[e] : most;
        for (int i = kFirst * NT + threadIdx.x; i < len; i += NT) {
            const uint64_t k = kr[i];
            most = k > most ? k : most;
        }
        const uint32_t bar = bar_of<NW>(cd, (uint32_t)(most >> 32), a.top);
        const auto offer = [&](uint64_t k) {
            if (k && (uint32_t)(k >> 32) >= bar) {
                const int at = atomicAdd(&cd.n, 1);
                if (at < cd.kCap) cd.key[at] = k;
            }
        };
#pragma unroll
        for (int e = 0; e < kFirst; ++e) offer(mine[e]);
        if ((uint32_t)(most >> 32) >= bar)
            for (int i = kFirst * NT + threadIdx.x; i < len; i += NT) offer(kr[i]);
        __syncthreads();
        int n = cd.n;
        if (n <= cd.kCap) {
            rank_keys<NW>(cd, n, a.top);
            n = n < a.top ? n : a.top;
        } else {
            __syncthreads();
            n = top_in_order<NW>(cd, [&](int i) { return kr[i]; }, len, a.top);
        }
        for (int k = threadIdx.x; k < n; k += NT) write_top(a, r, k, cd.sorted[k], sum, ln_s);
    }
    if (threadIdx.x == 0) finish_row(a, r, z_tok, tok, sum, ln_s);
}

// The gradient of a chunk of a row: e (A + B d) with d and e of the softmax's
// pass, and the token's own part where it falls.  Bound by memory: one reading
// and one writing, 2048 x 50000 bf16 with entropy 62 us, 6.6 TB/s (a part of the
// logits comes from the cache).
template <typename T, int NW, bool ENT, bool ONCE>
__global__ __launch_bounds__(NW * 64) void k_lp_back(LogprobArgs a, const float* stats, const float* entropy,
                                                     const float* dlogp, const float* dentropy, const T* z, T* dz,
                                                     int64_t dzs, int chunk, int chunks)
{
    constexpr int NT = NW * 64, VL = VecLen<T>::value, U = 4;
    const int64_t b = row_of_block(), r = b / chunks;
    if (r >= a.rows) return;
    const int z0 = (int)(b - r * chunks) * chunk, len = a.vocab - z0 < chunk ? a.vocab - z0 : chunk;
    const int nv = len / VL;
    const T* zr = z + r * a.zs + z0;
    T* out = dz + r * dzs + z0;
    const Raw* p = (const Raw*)zr;
    Raw* o = (Raw*)out;
    const int64_t tok = dlogp ? token_at(a.tokens, a.token_type, r) : -1;
    const float g = tok >= 0 && tok < a.vocab ? dlogp[r] : 0.f;
    const float h = ENT ? dentropy[r] : 0.f;
    const float s = stats[2 * r + 1];
    if ((g == 0.f && h == 0.f) || s == 0.f) {
        for (int v = threadIdx.x; v < nv; v += NT) store_row<ONCE>(o + v, Raw{{0, 0, 0, 0}});
        if (nv * VL + (int)threadIdx.x < len) out[nv * VL + threadIdx.x] = (T)0.f;
        return;
    }
    const float m = finite_base(stats[2 * r]);
    const float A = -a.scale / s * (ENT ? fmaf(h, entropy[r] - logf(s), g) : g), B = ENT ? -a.scale * h * kLn2 / s : 0.f;
    const int at = tok >= z0 && tok < z0 + len ? (int)(tok - z0) : -1;  // the token's place in the chunk
    const float add = a.scale * g;
    const auto grad = [&](float x, int i) {
        const float d = (x - m) * a.c;
        const float v = exp2_fast(d) * (ENT ? fmaf(B, fmaxf(d, kLowD), A) : A);
        return i == at ? v + add : v;
    };
    int v = threadIdx.x;
    const auto one = [&](const Raw& q, int at_v) {
        float x[VL];
        unpack<T>(q, x);
#pragma unroll
        for (int e = 0; e < VL; ++e) x[e] = grad(x[e], at_v * VL + e);
        store_row<ONCE>(o + at_v, pack<T>(x));
    };
    for (; v + (U - 1) * NT < nv; v += U * NT) {
        Raw q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) q[u] = load_row<ONCE>(p + v + u * NT);
#pragma unroll
        for (int u = 0; u < U; ++u) one(q[u], v + u * NT);
    }
    for (; v < nv; v += NT) one(load_row<ONCE>(p + v), v);
    const int i = nv * VL + threadIdx.x;
    if (i < len) out[i] = from_f<T>(grad(to_f(zr[i]), i));
}

static bool logprob_opts_ok(const sgc_logprob_opts* o)
{
    return o && o->rows >= 0 && o->rows < ((int64_t)1 << 31) && o->vocab >= 1 && o->vocab < ((int64_t)1 << 31) &&
           lm_dtype(o->dtype) && (o->token_type == SGC_TOKEN_I32 || o->token_type == SGC_TOKEN_I64) && o->top >= 0 &&
           o->top <= SGC_TOP_MAX && o->top <= o->vocab && scale_ok(o->scale);
}

static bool tokens_ok(const sgc_logprob_opts* o, const void* tokens)
{
    return tokens && lm_aligned(tokens, o->token_type == SGC_TOKEN_I64 ? 8 : 4);
}

// How the rows are shared out: one workgroup a row from kManyRows rows on, which
// fill the card, and for rows up to kShort (twice that where every row has a
// compute unit of its own), which take no longer than a second launch; else
// chunks, about kWantBlocks workgroups of at least kChunkMin elements each.
// 1 x 131072 top 20: 16 us so, 20 in chunks; 300 x 131072: 30.7 and 30.3.  No
// workgroup takes more than kMostElements (but for a chunk's rounding): places
// inside its part, and those its threads step to past the end, are 32 bits.
constexpr int64_t kWantBlocks = 1024, kManyRows = 512, kShort = 65536, kMostElements = (int64_t)1 << 30;
constexpr int kChunkMin = 4096;

static int chunks_of(const sgc_logprob_opts* o)
{
    int64_t n = cdiv(kWantBlocks, o->rows > 0 ? o->rows : 1);
    if (n > cdiv(o->vocab, kChunkMin)) n = cdiv(o->vocab, kChunkMin);
    if (o->rows >= kManyRows || o->vocab <= kShort * (o->rows <= 256 ? 2 : 1)) n = 1;
    if (n < cdiv(o->vocab, kMostElements)) n = cdiv(o->vocab, kMostElements);
    return (int)n;
}

// Chunks start at a multiple of 64 elements.
static int chunk_size(int64_t vocab, int chunks) { return (int)((cdiv(vocab, chunks) + 63) & ~(int64_t)63); }

static LogprobArgs logprob_args(const sgc_logprob_opts* o, int64_t zs, const void* tokens)
{
    LogprobArgs a = {};
    a.rows = o->rows;
    a.zs = zs;
    a.vocab = (int32_t)o->vocab;
    a.top = o->top;
    a.token_type = o->token_type;
    a.scale = o->scale;
    a.c = exponent_factor(o->scale);
    a.tokens = tokens;
    return a;
}

template <typename T>
static int logprobs(const sgc_logprob_opts* o, const void* zv, int64_t zs, const void* tokens, float* logp,
                    float* entropy, float* stats, int32_t* top_idx, float* top_logp, uint32_t* dstatus, void* ws,
                    hipStream_t s)
{
    LogprobArgs a = logprob_args(o, zs, tokens);
    a.logp = logp;
    a.entropy = entropy;
    a.stats = stats;
    a.top_idx = top_idx;
    a.top_logp = top_logp;
    a.dstatus = dstatus;
    const T* z = (const T*)zv;
    const int chunks = chunks_of(o);
    const dim3 rows = row_grid(o->rows);
    if (chunks == 1) {
        const bool once = a.rows * a.vocab * (int64_t)sizeof(T) >= kCacheBytes;
        // As few waves a row as keep its chain of trips short: each has its share
        // of the joins (8192 x 10000 bf16 top 5: 44 us by two, 49 by four, 71 by
        // eight; 4096 x 50000 90 by eight, 107 by four).  A thread for four of
        // the alternatives at least, so that the maxima are a filter.
        if (a.vocab <= 2048 && a.top <= 32)
            once ? k_lp_row<T, 1, true><<<rows, 64, 0, s>>>(a, z) : k_lp_row<T, 1, false><<<rows, 64, 0, s>>>(a, z);
        else if (a.rows >= kManyRows && a.vocab / VecLen<T>::value <= 1536 && a.top <= 32)
            once ? k_lp_row<T, 2, true><<<rows, 128, 0, s>>>(a, z) : k_lp_row<T, 2, false><<<rows, 128, 0, s>>>(a, z);
        else if (a.vocab <= 16384 && a.top <= (a.vocab <= 2048 ? 128 : 64))
            once ? k_lp_row<T, 4, true><<<rows, 256, 0, s>>>(a, z) : k_lp_row<T, 4, false><<<rows, 256, 0, s>>>(a, z);
        else if (a.rows < kManyRows)
            k_lp_row<T, 16, false><<<rows, 1024, 0, s>>>(a, z);
        else
            once ? k_lp_row<T, 8, true><<<rows, 512, 0, s>>>(a, z) : k_lp_row<T, 8, false><<<rows, 512, 0, s>>>(a, z);
        SGC_LAUNCH_CHECK();
        return SGC_OK;
    }
    const int chunk = chunk_size(a.vocab, chunks), used = (int)cdiv(a.vocab, chunk);
    Carver c(ws);
    float* part = c.take<float>(4 * o->rows * chunks);
    uint64_t* keys = c.take<uint64_t>((int64_t)o->top * o->rows * chunks);
    const dim3 parts = row_grid(o->rows * used);
    if (a.top <= 64)
        k_lp_part<T, 4><<<parts, 256, 0, s>>>(a, z, chunk, used, part, keys);
    else
        k_lp_part<T, 8><<<parts, 512, 0, s>>>(a, z, chunk, used, part, keys);
    SGC_LAUNCH_CHECK();
    k_lp_join<T, 8><<<rows, 512, 0, s>>>(a, z, used, part, keys);
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}

template <typename T, int NW, bool ENT>
static int logprobs_back(const LogprobArgs& a, const T* z, const float* stats, const float* entropy,
                         const float* dlogp, const float* dentropy, T* dz, int64_t dzs, int chunk, hipStream_t s)
{
    const int chunks = (int)cdiv(a.vocab, chunk);
    const dim3 grid = row_grid(a.rows * chunks);
    if (2 * a.rows * a.vocab * (int64_t)sizeof(T) >= kCacheBytes)
        k_lp_back<T, NW, ENT, true><<<grid, NW * 64, 0, s>>>(a, stats, entropy, dlogp, dentropy, z, dz, dzs, chunk,
                                                             chunks);
    else
        k_lp_back<T, NW, ENT, false><<<grid, NW * 64, 0, s>>>(a, stats, entropy, dlogp, dentropy, z, dz, dzs, chunk,
                                                              chunks);
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}

template <typename T>
static int logprobs_back(const sgc_logprob_opts* o, const void* zv, int64_t zs, const void* tokens,
                         const float* stats, const float* entropy, const float* dlogp, const float* dentropy,
                         void* dzv, int64_t dzs, hipStream_t s)
{
    const LogprobArgs a = logprob_args(o, zs, tokens);
    const T* z = (const T*)zv;
    T* dz = (T*)dzv;
    if (a.vocab <= 2048)
        return dentropy ? logprobs_back<T, 1, true>(a, z, stats, entropy, dlogp, dentropy, dz, dzs, 2048, s)
                        : logprobs_back<T, 1, false>(a, z, stats, entropy, dlogp, dentropy, dz, dzs, 2048, s);
    return dentropy ? logprobs_back<T, 4, true>(a, z, stats, entropy, dlogp, dentropy, dz, dzs, 8192, s)
                    : logprobs_back<T, 4, false>(a, z, stats, entropy, dlogp, dentropy, dz, dzs, 8192, s);
}

}  // namespace sgc

using namespace sgc;

extern "C" size_t sgc_token_logprobs_workspace(const sgc_logprob_opts* o)
{
    if (!logprob_opts_ok(o)) return 0;
    const int chunks = chunks_of(o);
    if (chunks == 1) return SGC_LM_WS_NONE;
    Carver c(nullptr);
    c.take<float>(4 * o->rows * chunks);
    c.take<uint64_t>((int64_t)o->top * o->rows * chunks);
    return c.off;
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
               ? logprobs<float>(o, logits, stride, tokens, logp, entropy, stats, top_idx, top_logp, dstatus, ws, s)
           : o->dtype == SGC_BF16
               ? logprobs<bf16_t>(o, logits, stride, tokens, logp, entropy, stats, top_idx, top_logp, dstatus, ws, s)
               : logprobs<f16_t>(o, logits, stride, tokens, logp, entropy, stats, top_idx, top_logp, dstatus, ws, s);
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
