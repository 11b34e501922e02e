// int8_linear.hip -- product of 8-bit rows with a scale for each token and each
// channel: y = (sum xq wq) xscale wscale + bias.
//
// Both operands lie along the sum, 16 of a row's bytes in a lane are one
// operand of a matrix instruction, and the order within the sum is free as long
// as both sides take the same.  The weights' rows are the instruction's first
// operand: a lane then holds four neighbouring channels of one token, which it
// stores together.
#include "lm_q8.h"

namespace sgc {

struct Product {
    const int8_t* x;
    int64_t xs;
    const float* xscale;
    const int8_t* w;
    int64_t ws;
    const float *wscale, *bias;
    void* y;
    int64_t ys;
    int64_t rows, out;
    int width;
};

typedef int Int4 __attribute__((ext_vector_type(4)));
// 16 bytes of a row, at any address.
typedef int Bytes16 __attribute__((ext_vector_type(4), aligned(1)));

// Bytes [at, at + 16) of a row of `width`; past it 0.  The row's end is read with
// what lies before it, in one access; rows shorter than that byte by byte.
__device__ inline Int4 load16(const int8_t* row, int at, int width)
{
    Int4 v = {0, 0, 0, 0};
    if (at >= width) return v;
    if (width >= 16) {
        const int over = at + 16 - width;
        v = *(const Bytes16*)(row + at - (over > 0 ? over : 0));
        if (over > 0) {
            uint32_t w0 = v.x, w1 = v.y, w2 = v.z, w3 = v.w;
            drop_bytes(w0, w1, w2, w3, over);
            v = {(int)w0, (int)w1, (int)w2, (int)w3};
        }
        return v;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < width) v[i / 4] |= (int)(uint8_t)row[i] << (i % 4 * 8);
    return v;
}

// The sum is a whole number below 2^31: one fp32 rounding of it, one for each
// scale, one for the bias, one to the output's type.
__device__ inline float product_out(int32_t sum, float xscale, float wscale, float bias)
{
    return (float)sum * xscale * wscale + bias;
}
// Four neighbouring channels of one token.
template <typename T>
__device__ inline void store4(const Product& k, int64_t r, int64_t o, const float* v)
{
    T* y = (T*)k.y + r * k.ys + o;
    if (o + 4 <= k.out) {
        Pack<T, 4> p;
#pragma unroll
        for (int i = 0; i < 4; ++i) p.v[i] = from_f<T>(v[i]);
        *(Pack<T, 4>*)y = p;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (o + i < k.out) y[i] = from_f<T>(v[i]);
    }
}
__device__ inline void channel4(const Product& k, int64_t o, float* scale, float* bias)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t at = o + i < k.out ? o + i : k.out - 1;
        scale[i] = k.wscale[at];
        bias[i] = k.bias ? k.bias[at] : 0.f;
    }
}

// --------------------------------------------------------------- tiles
// A workgroup takes TM tokens x TN channels, its WM x WN waves a part each; 128
// bytes of every row (a step) go through shared memory at a time.  A row's
// 16-byte pieces lie there at piece ^ (row mod 8): eight rows' same piece, which
// lanes read together, and one row's eight pieces, which they write together,
// both lie in all banks once.  Rows that begin at multiples of 16 bytes come
// straight from memory (DIRECT), others through registers.
//
// 4096 x 4096 x 50000: 757 to 776 us, 2.16 to 2.21 PFLOP/s; 8192 cubed 423 us, 2.60;
// the matrix units are 53% busy, and the clock follows the power that the values
// take.  A step is 64 matrix instructions a wave for 24 reads of shared memory,
// all of which are on their way while the products before them run.  256 x 256 by
// eight waves of 64 x 128: four waves of 128 x 128 would read a third less, but
// spill.  A round's beginning and end, 6 us of 60 here, are not overlapped.
// With rows through registers 256 x 256 spill (88 bytes a lane, 104 with fp32
// results): 4096 x 4096 x 50000 with rows 4099 bytes apart 1967 us, 1500 x 650 x
// 10000 fp32 45 (26 straight), 512 x 4096 x 4096 27 (15).
constexpr int kStep = 128;
constexpr int kBand = 8, kChips = 8;
// Workgroups go to the chips in turn; each chip takes consecutive tiles.
__device__ inline int64_t tile_of_block(int64_t tiles)
{
    const int64_t id = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (id >= tiles) return -1;
    const int64_t chip = id % kChips, each = tiles / kChips, more = tiles % kChips;
    return chip * each + (chip < more ? chip : more) + id / kChips;
}
// 16 bytes for every lane of a wave from memory into shared memory, without
// registers between: lane l's go to `to` + l.  p at multiples of 16 bytes.
__device__ inline void into_shared(const int8_t* p, Int4* to)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p,
                                     (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}
template <typename T, int TM, int TN, int WM, int WN, int STAGES, bool DIRECT>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_tile(Product k, int tiles_m, int tiles_n)
{
    constexpr int kThreads = 64 * WM * WN, PM = TM / WM / 16, PN = TN / WN / 16;
    constexpr int CX = TM * 8 / kThreads, CW = TN * 8 / kThreads, kRows = kThreads / 8;
    // Each step's rows in an array of its own: the compiler then knows that rows on
    // their way into one are not what is read from another.  Later 32 tokens of
    // each wave's results, a row's pitch 16 bytes past its length.
    constexpr int kPitch = PN * 16 * (int)sizeof(T) + 16, kOut = WM * WN / 4 * 2 * kPitch;
    constexpr int kX = TM * 8 > kOut ? TM * 8 : kOut, kW = TN * 8 > kOut ? TN * 8 : kOut;
    __shared__ Int4 x0[kX], x1[kX], w0[kW], w1[kW];
    constexpr int kX4 = STAGES > 2 ? TM * 8 : 1, kW4 = STAGES > 2 ? TN * 8 : 1;
    constexpr int kX8 = STAGES > 4 ? TM * 8 : 1, kW8 = STAGES > 4 ? TN * 8 : 1;
    __shared__ Int4 x2[kX4], x3[kX4], w2[kW4], w3[kW4];
    __shared__ Int4 x4[kX8], x5[kX8], x6[kX8], x7[kX8], w4[kW8], w5[kW8], w6[kW8], w7[kW8];
    __shared__ alignas(16) float channels[2][TN];  // their scales and biases
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6), wm = wave % WM, wn = wave / WM;
    const int64_t at_tile = tile_of_block((int64_t)tiles_m * tiles_n);
    if (at_tile < 0) return;
    // kBand tiles of tokens side by side: the workgroups that run together on a chip
    // share rows of both operands in its L2
    const int64_t band = at_tile / ((int64_t)kBand * tiles_n), in_band = at_tile - band * kBand * tiles_n;
    const int high = tiles_m - band * kBand < kBand ? (int)(tiles_m - band * kBand) : kBand;
    const int64_t m0 = (band * kBand + in_band % high) * TM, n0 = in_band / high * TN;
    for (int c = t; c < TN; c += kThreads) {
        const int64_t o = n0 + c < k.out ? n0 + c : k.out - 1;
        channels[0][c] = k.wscale[o];
        channels[1][c] = k.bias ? k.bias[o] : 0.f;
    }
    // rows past the last one read the last one; what they give is not written.  Thread
    // t fills piece t of shared memory's kThreads, which is piece (t ^ row) mod 8 of its row.
    const int row = t >> 3, piece = (t ^ row) & 7;
    const int8_t *px[CX], *pw[CW];
#pragma unroll
    for (int i = 0; i < CX; ++i) {
        const int64_t r = m0 + row + i * kRows;
        px[i] = k.x + (r < k.rows ? r : k.rows - 1) * k.xs + piece * 16;
    }
#pragma unroll
    for (int i = 0; i < CW; ++i) {
        const int64_t r = n0 + row + i * kRows;
        pw[i] = k.w + (r < k.out ? r : k.out - 1) * k.ws + piece * 16;
    }
    // where the width is no multiple of 128 its end is step 0 (the order within the sum
    // is free), which is cheapest there: nothing else is in registers yet
    const int steps = (k.width + kStep - 1) / kStep, part = k.width % kStep ? 1 : 0;
    Int4 rx[CX], rw[CW];
    const auto fetch = [&](int s) __attribute__((always_inline)) {
        if (DIRECT || s < part || s >= steps) return;
        const int at = (s - part) * kStep;
#pragma unroll
        for (int i = 0; i < CX; ++i) rx[i] = *(const Bytes16*)(px[i] + at);
#pragma unroll
        for (int i = 0; i < CW; ++i) rw[i] = *(const Bytes16*)(pw[i] + at);
    };
    // Step s, whole, into shared memory.
    const auto put = [&](Int4* x, Int4* w, int s) __attribute__((always_inline)) {
        if (s >= steps) return;
        const int at = (s - part) * kStep;
#pragma unroll
        for (int i = 0; i < CX; ++i) {
            if constexpr (DIRECT)
                into_shared(px[i] + at, x + wave * 64 + i * kThreads);
            else
                x[t + i * kThreads] = rx[i];
        }
#pragma unroll
        for (int i = 0; i < CW; ++i) {
            if constexpr (DIRECT)
                into_shared(pw[i] + at, w + wave * 64 + i * kThreads);
            else
                w[t + i * kThreads] = rw[i];
        }
    };
    const auto put_end = [&](Int4* x, Int4* w) __attribute__((always_inline)) {
        const int at = (steps - 1) * kStep + piece * 16;
#pragma unroll
        for (int i = 0; i < CX; ++i) rx[i] = load16(px[i] - piece * 16, at, k.width);
#pragma unroll
        for (int i = 0; i < CW; ++i) rw[i] = load16(pw[i] - piece * 16, at, k.width);
#pragma unroll
        for (int i = 0; i < CX; ++i) x[t + i * kThreads] = rx[i];
#pragma unroll
        for (int i = 0; i < CW; ++i) w[t + i * kThreads] = rw[i];
    };
    // 16 x 16 results an instruction (32 x 32: 4096 x 4096 x 50000 834 us, with 16 754)
    Int4 acc[PN][PM];
#pragma unroll
    for (int i = 0; i < PN; ++i)
#pragma unroll
        for (int j = 0; j < PM; ++j) acc[i][j] = Int4{0, 0, 0, 0};
    const int lr = lane & 15, quarter = lane >> 4;
    const int ax = (wm * PM * 16 + lr) * 8, aw = (wn * PN * 16 + lr) * 8;
    // A step is four phases: 64 bytes of the sum with one half of the channels, with
    // the other, and the same for the other 64 bytes.
    constexpr int kPhases = 4, kHalf = PN / 2;
    Int4 fx[2][PM], fw[2][kHalf];
    const auto read = [&](const Int4* x, const Int4* w, int ph) __attribute__((always_inline)) {
        const int p = ((ph >> 1) * 4 + quarter) ^ (lr & 7);
        if ((ph & 1) == 0) {
#pragma unroll
            for (int j = 0; j < PM; ++j) fx[ph >> 1][j] = x[ax + j * 128 + p];
        }
#pragma unroll
        for (int i = 0; i < kHalf; ++i) fw[ph & 1][i] = w[aw + ((ph & 1) * kHalf + i) * 128 + p];
    };
    const auto multiply = [&](int ph) __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kHalf; ++i)
#pragma unroll
            for (int j = 0; j < PM; ++j) {
                Int4& a = acc[(ph & 1) * kHalf + i][j];
                a = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[ph & 1][i], fx[ph >> 1][j], a, 0, 0, 0);
            }
        __builtin_amdgcn_sched_barrier(0);
    };
    // Waits until this wave's part of step s lies in shared memory; of the later ones
    // up to `ahead` may be on their way (a barrier alone does not wait for them).
    const auto arrived = [&](int s, int ahead) __attribute__((always_inline)) {
        if constexpr (DIRECT) {
            constexpr int kEach = CX + CW;
            static_assert((STAGES - 1) * kEach < 64, "");
            constexpr auto code = [](int n) constexpr { return 0x0f70 | (n & 15) | (n >> 4) << 14; };  // vmcnt(n)
            if (ahead == STAGES - 1 && s + ahead < steps) __builtin_amdgcn_s_waitcnt(code((STAGES - 1) * kEach));
            else if (ahead == STAGES - 2 && s + ahead < steps) __builtin_amdgcn_s_waitcnt(code((STAGES - 2) * kEach));
            else __builtin_amdgcn_s_waitcnt(code(0));
        }
    };
    // with more than two stages later rows stay on their way across the barrier: only
    // what this wave reads and writes in shared memory is waited for (lgkmcnt(0))
    const auto meet = [] {
        if constexpr (STAGES == 2) {
            __syncthreads();
        } else {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0xc07f);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        }
    };
    // Small tiles: a wave's few products do not cover its reads' way, so the whole next
    // step's operands are read while one step's products run.
    constexpr bool kWhole = PM * PN <= 4;
    struct Operands {
        Int4 x[kWhole ? 2 : 1][PM], w[kWhole ? 2 : 1][PN];
    } even, odd;
    const auto read_whole = [&](const Int4* x, const Int4* w, Operands& f) __attribute__((always_inline)) {
        if constexpr (kWhole) {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const int p = (kk * 4 + quarter) ^ (lr & 7);
#pragma unroll
                for (int j = 0; j < PM; ++j) f.x[kk][j] = x[ax + j * 128 + p];
#pragma unroll
                for (int i = 0; i < PN; ++i) f.w[kk][i] = w[aw + i * 128 + p];
            }
        }
    };
    // The operands of the next products are read while one step's run.  One barrier a
    // step, before its last products (or, whole steps at a time, all of them): what
    // is read of this step's rows has been read, and rows STAGES steps on take their
    // place; the next step's lie ready.
    const auto step = [&](int s, Int4* x, Int4* w, const Int4* next_x, const Int4* next_w, Operands& now,
                          Operands& next) __attribute__((always_inline)) {
        if constexpr (!kWhole) {
#pragma unroll
            for (int ph = 0; ph + 1 < kPhases; ++ph) {
                read(x, w, ph + 1);
                multiply(ph);
            }
        }
        arrived(s + 1, STAGES - 2);
        meet();
        put(x, w, s + STAGES);
        fetch(s + STAGES + 1);
        if constexpr (kWhole) {
            read_whole(next_x, next_w, next);  // past the last step what lies there, unused
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int i = 0; i < PN; ++i)
#pragma unroll
                    for (int j = 0; j < PM; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(now.w[kk][i], now.x[kk][j], acc[i][j], 0, 0, 0);
            // a read beside each product
#pragma unroll
            for (int i = 0; i < 2 * (PM + PN); ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        } else {
            if (s + 1 < steps) read(next_x, next_w, 0);
            multiply(kPhases - 1);
        }
    };
    if (part) {
        put_end(x0, w0);
    } else {
        fetch(0);
        put(x0, w0, 0);
    }
    fetch(1);
    put(x1, w1, 1);
    fetch(2);
    static_assert(STAGES == 2 || DIRECT, "");  // rows through registers are fetched one step ahead
    if constexpr (STAGES > 2) {
        put(x2, w2, 2);
        put(x3, w3, 3);
    }
    if constexpr (STAGES > 4) {
        put(x4, w4, 4);
        put(x5, w5, 5);
        put(x6, w6, 6);
        put(x7, w7, 7);
    }
    arrived(0, STAGES - 1);
    meet();
    if constexpr (kWhole) read_whole(x0, w0, even);
    else read(x0, w0, 0);
    for (int s = 0; s < steps; s += STAGES) {
        step(s, x0, w0, x1, w1, even, odd);
        if constexpr (STAGES == 2) {
            if (s + 1 < steps) step(s + 1, x1, w1, x0, w0, odd, even);
        } else {
            if (s + 1 < steps) step(s + 1, x1, w1, x2, w2, odd, even);
            if (s + 2 < steps) step(s + 2, x2, w2, x3, w3, even, odd);
            if constexpr (STAGES == 4) {
                if (s + 3 < steps) step(s + 3, x3, w3, x0, w0, odd, even);
            } else {
                if (s + 3 < steps) step(s + 3, x3, w3, x4, w4, odd, even);
                if (s + 4 < steps) step(s + 4, x4, w4, x5, w5, even, odd);
                if (s + 5 < steps) step(s + 5, x5, w5, x6, w6, odd, even);
                if (s + 6 < steps) step(s + 6, x6, w6, x7, w7, even, odd);
                if (s + 7 < steps) step(s + 7, x7, w7, x0, w0, odd, even);
            }
        }
    }
    __syncthreads();
    // 32 tokens of a wave at a time through its own part of shared memory, so that
    // rows are written in long pieces
    constexpr int kPiece = 16 / (int)sizeof(T);
    char* mine = (char*)((wave & 2) ? (wave & 1) ? w1 : w0 : (wave & 1) ? x1 : x0) + (wave >> 2) * 32 * kPitch;
    const int64_t on = n0 + wn * PN * 16;
#pragma unroll
    for (int j = 0; j < PM / 2; ++j) {
        const int64_t rm = m0 + (wm * PM + j * 2) * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t r = rm + h * 16 + lr;
            const float xscale = k.xscale[r < k.rows ? r : k.rows - 1];
#pragma unroll
            for (int i = 0; i < PN; ++i) {
                const int c0 = i * 16 + quarter * 4;
                const float4 ws = *(const float4*)&channels[0][wn * PN * 16 + c0];
                const float4 bias = *(const float4*)&channels[1][wn * PN * 16 + c0];
                const Int4 a = acc[i][j * 2 + h];
                Pack<T, 4> p;
                p.v[0] = from_f<T>(product_out(a.x, xscale, ws.x, bias.x));
                p.v[1] = from_f<T>(product_out(a.y, xscale, ws.y, bias.y));
                p.v[2] = from_f<T>(product_out(a.z, xscale, ws.z, bias.z));
                p.v[3] = from_f<T>(product_out(a.w, xscale, ws.w, bias.w));
                *(Pack<T, 4>*)(mine + (h * 16 + lr) * kPitch + c0 * (int)sizeof(T)) = p;
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        constexpr int kPieces = PN * 16 / kPiece, kAtOnce = 64 / kPieces;
#pragma unroll
        for (int a = 0; a < 32; a += kAtOnce) {
            const int rr = a + lane / kPieces, c0 = lane % kPieces * kPiece;
            const Raw q = *(const Raw*)(mine + rr * kPitch + c0 * (int)sizeof(T));
            if (rm + rr >= k.rows) continue;
            T* y = (T*)k.y + (rm + rr) * k.ys + on + c0;
            if (on + c0 + kPiece <= k.out) {
                *(Raw*)y = q;
            } else {
                const T* v = (const T*)(mine + rr * kPitch) + c0;
#pragma unroll
                for (int c = 0; c < kPiece; ++c)
                    if (on + c0 + c < k.out) y[c] = v[c];
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// ------------------------------------------------------------- few tokens
// A workgroup takes 16 channels x 16 B tokens, each wave a share of the sum,
// straight from memory into the matrix instruction; the waves join their sums in
// shared memory.  Bound by memory: 1 x 1024 x 50000 10.6 us a pass (4.9 TB/s; rows
// 1027 bytes apart 21), 2 x 4096 x 50000 34 us (6.1 TB/s).  Fetching a trip ahead takes twice the registers
// and gains nothing.
constexpr int kFewWaves = 8, kFewDeep = 8;
template <typename T, int B>
__global__ __launch_bounds__(64 * kFewWaves) void k_few(Product k, int split)
{
    __shared__ Int4 part[kFewWaves][B][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int share = wave;
    const int64_t n0 = row_of_block() * 16;
    const int lr = lane & 15, quarter = lane >> 4;
    Int4 acc[B];
#pragma unroll
    for (int j = 0; j < B; ++j) acc[j] = Int4{0, 0, 0, 0};
    if (n0 < k.out) {
        const int64_t o = n0 + lr < k.out ? n0 + lr : k.out - 1;
        const int8_t* pw = k.w + o * k.ws;
        const int8_t* px[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int64_t r = j * 16 + lr;
            px[j] = k.x + (r < k.rows ? r : k.rows - 1) * k.xs;
        }
        const int steps = (k.width + 63) / 64, each = (steps + split - 1) / split;
        const int from = share * each, to = from + each < steps ? from + each : steps;
        for (int s = from; s < to; s += kFewDeep) {
            Int4 fw[kFewDeep], fx[kFewDeep][B];
            if (s + kFewDeep <= to && (s + kFewDeep) * 64 <= k.width) {
#pragma unroll
                for (int d = 0; d < kFewDeep; ++d) {
                    const int at = (s + d) * 64 + quarter * 16;
                    fw[d] = *(const Bytes16*)(pw + at);
#pragma unroll
                    for (int j = 0; j < B; ++j) fx[d][j] = *(const Bytes16*)(px[j] + at);
                }
            } else {
#pragma unroll
                for (int d = 0; d < kFewDeep; ++d) {
                    const int at = s + d < to ? (s + d) * 64 + quarter * 16 : k.width;
                    fw[d] = load16(pw, at, k.width);
#pragma unroll
                    for (int j = 0; j < B; ++j) fx[d][j] = load16(px[j], at, k.width);
                }
            }
#pragma unroll
            for (int d = 0; d < kFewDeep; ++d)
#pragma unroll
                for (int j = 0; j < B; ++j)
                    acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[d], fx[d][j], acc[j], 0, 0, 0);
        }
    }
    if (split > 1) {
#pragma unroll
        for (int j = 0; j < B; ++j) part[wave][j][lane] = acc[j];
        __syncthreads();
        if (share) return;
        for (int d = 1; d < split; ++d)
#pragma unroll
            for (int j = 0; j < B; ++j) acc[j] += part[wave + d][j][lane];
    }
    const int64_t o = n0 + quarter * 4;
    if (o >= k.out) return;
    float ws[4], bias[4], v[4];
    channel4(k, o, ws, bias);
#pragma unroll
    for (int j = 0; j < B; ++j) {
        const int64_t r = j * 16 + lr;
        if (r >= k.rows) continue;
        const float xscale = k.xscale[r];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = product_out(acc[j][c], xscale, ws[c], bias[c]);
        store4<T>(k, r, o, v);
    }
}

// The sum is split until eight waves a compute unit have work or each has one
// trip's loads (32 x 4096 x 4096: 9.1 us a pass, 10.0 traced).
template <typename T, int B>
static int few(const Product& k, hipStream_t s)
{
    const int64_t units = cdiv(k.out, 16);
    int split = 1;
    while (split < kFewWaves && units * split < 256 * 8 && k.width > split * 64 * kFewDeep) split *= 2;
    k_few<T, B><<<row_grid(units), 64 * split, 0, s>>>(k, split);
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}

template <typename T, int TM, int TN, int WM, int WN, int STAGES, bool DIRECT>
static int tiles(const Product& k, hipStream_t s)
{
    const int64_t tm = cdiv(k.rows, TM), tn = cdiv(k.out, TN);
    k_tile<T, TM, TN, WM, WN, STAGES, DIRECT><<<row_grid(tm * tn), 64 * WM * WN, 0, s>>>(k, (int)tm, (int)tn);
    SGC_LAUNCH_CHECK();
    return SGC_OK;
}

template <typename T, int TM, int TN, int WM, int WN, int STAGES>
static int tiles_of(const Product& k, hipStream_t s)
{
    const bool direct = aligned16(k.x) && aligned16(k.w) && k.xs % 16 == 0 && k.ws % 16 == 0;
    return direct ? tiles<T, TM, TN, WM, WN, STAGES, true>(k, s) : tiles<T, TM, TN, WM, WN, 2, false>(k, s);
}

// Few tokens: straight from memory up to 8192 channels (past that most of what is
// read are the tokens' rows: every workgroup reads them, a tile once), for one or two
// tokens always.  bf16, straight and in tiles, us a pass: 32 x 4096 x 4096 9.1 and
// 10.0, 32 x 14336 x 4096 22.5 and 25.7, 3 x 14336 x 4096 13 and 25; 24 x 4096 x 16384
// 22 and 14.3, 32 x 14336 x 16384 92 and 47.  The bound looks neither at the number of
// tokens nor at the width: 32 x 4096 x 8192 14.2 and 10.5, 32 x 14336 x 8192 49 and 40,
// 3 x 14336 x 16384 43.2 and 45.4 lie on its other side; at a width of 1024 both take
// 8.3.
// Else tiles of the size whose rounds over the chip take least, by what a round
// takes there in microseconds, a part and a part a step, the latter less where
// a compute unit has one tile (and about 2 more a call): 2048 x 1024 x 10000 in
// tiles of 64, 128, 256: 53, 35, 44; 512 x 4096 x 4096: 15, 23, 54; 1500 x 656 x
// 10000: 41, 25, 22; 800 x 2048 x 6000: 25, 21, 34; 1024 x 4096 x 4096: 31, 26, 54.
// Tiles of 64 that have a compute unit each keep eight steps in shared memory, not
// four (40 x 16384 x 4096: 37.7 -> 33.1 us, 28.6 with reads beside products).
template <typename T>
static int product(const Product& k, hipStream_t s)
{
    if (k.rows <= 2 || (k.rows <= 32 && k.out <= 8192)) return k.rows <= 16 ? few<T, 1>(k, s) : few<T, 2>(k, s);
    const double steps = (double)cdiv(k.width, kStep);
    const auto count = [&](int64_t tile) { return cdiv(k.rows, tile) * cdiv(k.out, tile); };
    const auto cost = [&](int64_t tile, int64_t at_once, double round, double alone, double step) {
        const int64_t n = count(tile);
        return n <= 256 ? round + alone * steps : (double)cdiv(n, at_once) * (round + step * steps);
    };
    const double c64 = cost(64, 512, 2.3, 0.2, 0.33), c128 = cost(128, 512, 4.0, 0.65, 1.0),
                 c256 = cost(256, 256, 6.0, 1.5, 1.65);
    if (c64 <= c128 && c64 <= c256)
        return count(64) <= 256 ? tiles_of<T, 64, 64, 2, 2, 8>(k, s) : tiles_of<T, 64, 64, 2, 2, 4>(k, s);
    return c128 <= c256 ? tiles_of<T, 128, 128, 2, 2, 2>(k, s) : tiles_of<T, 256, 256, 4, 2, 2>(k, s);
}

}  // namespace sgc

using namespace sgc;

extern "C" int sgc_int8_linear(const sgc_int8_opts* o, const int8_t* xq, int64_t xq_stride, const float* xscale,
                               const int8_t* wq, int64_t wq_stride, const float* wscale, const float* bias, void* y,
                               int64_t y_stride, sgc_stream_t stream)
{
    if (!o || o->rows < 0 || o->rows >= ((int64_t)1 << 31) || o->width < 1 || o->width >= (1 << 17) || o->out < 1 ||
        o->out >= ((int64_t)1 << 31) || !lm_dtype(o->dtype) || o->reserved)
        return SGC_EINVAL;
    if (o->rows == 0) return SGC_OK;
    if (!q8_rows_ok(xq, xq_stride, o->rows, o->width, false) || !q8_rows_ok(wq, wq_stride, o->out, o->width, false))
        return SGC_EINVAL;
    if (!lm_rows_ok(y, y_stride, o->rows, o->out, o->dtype, true) || !xscale || !wscale) return SGC_EINVAL;
    if (!lm_aligned(xscale, 4) || !lm_aligned(wscale, 4) || !lm_aligned(bias, 4)) return SGC_EINVAL;
    const Product k = {xq, xq_stride, xscale, wq, wq_stride, wscale, bias, y, y_stride, o->rows, o->out,
                       (int)o->width};
    const hipStream_t s = (hipStream_t)stream;
    return o->dtype == SGC_F32    ? product<float>(k, s)
           : o->dtype == SGC_BF16 ? product<bf16_t>(k, s)
                                  : product<f16_t>(k, s);
}
