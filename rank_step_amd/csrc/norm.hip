// Layer norm and root-mean-square norm, forward and backward (gfx950 /
// MI355X).  The arithmetic of each call is stated in include/fsdp_norm.h.
//
// Both are bound by memory: the forward pass reads and writes each element
// once, the backward pass reads two or three matrices and writes one, with about
// ten operations an element.  So a row is read once, into registers, where its
// sums are taken about its mean; rows too long for that are read again.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fsdp_norm.h"
#include "internal.h"
#include "linear_plan.h"
#include "stream_device.h"

using fsdp::fail;

namespace {

using namespace fsdp::linear;

// ---------------------------------------------------------------- sums over a row

// The sum over the wave, in every lane: within quads, eights and 16s by DPP
// moves, then over the four 16s by the lane swaps; both lanes of a pair add the
// same two values, so all lanes hold the same bits.
__device__ __forceinline__ float wave_sum(float v) {
    auto dpp = [](float x, auto ctrl) {
        return __uint_as_float(static_cast<uint32_t>(
            __builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(x)), decltype(ctrl)::value, 0xf, 0xf, true)));
    };
    v += dpp(v, std::integral_constant<int, 0xB1>());   // quad_perm 1 0 3 2
    v += dpp(v, std::integral_constant<int, 0x4E>());   // quad_perm 2 3 0 1
    v += dpp(v, std::integral_constant<int, 0x141>());  // row_half_mirror
    v += dpp(v, std::integral_constant<int, 0x140>());  // row_mirror
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// The sums of N values over a row's waves, in the waves' order.  `s` is not
// written again before every wave has read it: two uses of one `s` have a
// barrier of another between them.
template <int WAVES, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*s)[WAVES]) {
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] = wave_sum(v[q]);
    if constexpr (WAVES > 1) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        if (lane == 0)
#pragma unroll
            for (int q = 0; q < N; ++q) s[q][wave] = v[q];
        __syncthreads();
#pragma unroll
        for (int q = 0; q < N; ++q) {
            v[q] = s[q][0];
#pragma unroll
            for (int p = 1; p < WAVES; ++p) v[q] += s[q][p];
        }
    }
}

// N parameters from element j on in fp32, `none` where there is no vector.  Of a
// row's last, shorter chunk (back > 0) the N that end with the row are read and
// moved down, as stream_load does; of rows shorter than a chunk (back < 0) each.
template <int N>
__device__ __forceinline__ void load_params(const void* p, int f32, int64_t j, int cnt, int back, float none, float (&v)[N]) {
#pragma unroll
    for (int q = 0; q < N; ++q) v[q] = none;
    if (!p || cnt <= 0) return;
    if (back < 0) {
#pragma unroll
        for (int q = 0; q < N; ++q)
            if (q < cnt) v[q] = f32 ? static_cast<const float*>(p)[j + q] : widen(static_cast<const uint16_t*>(p)[j + q]);
        return;
    }
    struct __attribute__((packed, aligned(4))) Floats { float v[N]; };
    struct __attribute__((packed, aligned(2))) Halves { uint16_t v[N]; };
    if (f32) {
        const Floats w = *reinterpret_cast<const Floats*>(static_cast<const float*>(p) + j - back);
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = w.v[q];
    } else {
        const Halves w = *reinterpret_cast<const Halves*>(static_cast<const uint16_t*>(p) + j - back);
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = widen(w.v[q]);
    }
    if (back > 0) {
#pragma unroll
        for (int d = N / 2; d > 0; d /= 2)
            if (back & d)
#pragma unroll
                for (int q = 0; q + d < N; ++q) v[q] = v[q + d];
    }
}

// A thread's chunks of a row: chunk c starts at element (c * 64 WAVES + t) * E.
// TAIL: the row's last chunk may be shorter.
template <typename T, int WAVES, int C, bool TAIL>
struct Row {
    static constexpr int kEach = 16 / sizeof(T);
    int first;  // of the thread's first chunk
    int n;

    __device__ __forceinline__ void init(int t, int64_t len) {
        first = t * kEach;
        n = static_cast<int>(len);
    }
    __device__ __forceinline__ int at(int c) const { return first + c * (64 * WAVES * kEach); }
    __device__ __forceinline__ bool has(int c) const { return at(c) < n; }
    // elements of a chunk that the row has
    __device__ __forceinline__ int cnt(int c) const { return TAIL ? min(n - at(c), kEach) : kEach; }
    __device__ __forceinline__ int back(int c) const { return TAIL ? chunk_back<T>(cnt(c), n) : 0; }
    __device__ __forceinline__ void load(const T* row, u32x4 (&w)[C]) const {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            w[c] = u32x4{0, 0, 0, 0};
            if (has(c)) w[c] = stream_load(row + at(c), cnt(c), back(c));
        }
    }
    // Chunk c's values, zeros behind the row's end.
    __device__ __forceinline__ void values(const u32x4 (&w)[C], int c, float (&v)[kEach]) const {
        arrange(w[c], TAIL && has(c) ? back(c) : 0, v);
    }
    __device__ __forceinline__ bool inside(int c, int q) const { return TAIL ? at(c) + q < n : has(c); }
};

// Packed chunks whose widened values are not kept from here on: the compiler
// would rather hold them, at twice the registers of bf16, than widen again.
template <int C>
__device__ __forceinline__ void widen_again(u32x4 (&w)[C]) {
#pragma unroll
    for (int c = 0; c < C; ++c) asm volatile("" : "+v"(w[c])::"memory");
}

// ---------------------------------------------------------------- forward

struct ForwardArgs {
    void* y;
    const void* x;
    const void* w;
    const void* b;
    float* mean;
    float* rstd;
    int64_t ldy, ldx, m, n;
    float eps;
    int32_t w_f32, rms, wt;
};

// A row by WAVES waves of C chunks of 16 bytes a lane, which stay packed in
// registers and are widened for each pass over them.  Bound by memory: 8192 x
// 4096 bf16 with one wave a row, whose 8 KB need no barrier, XXX us; by four waves
// 42, as a workgroup then has little on its way while it waits for its sums.
template <typename T, int WAVES, int C, bool TAIL>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void norm_forward_kernel(ForwardArgs a) {
    constexpr int kEach = 16 / sizeof(T), kRows = WAVES == 1 ? 4 : 1;
    __shared__ float s0[1][WAVES], s1[2][WAVES];
    const int t = threadIdx.x % (64 * WAVES);
    Row<T, WAVES, C, TAIL> row;
    row.init(t, a.n);
    const float n = static_cast<float>(a.n);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / (64 * WAVES); i < a.m;
         i += static_cast<int64_t>(gridDim.x) * kRows) {
        u32x4 raw[C];
        row.load(static_cast<const T*>(a.x) + i * a.ldx, raw);
        float mean = 0.0f;
        if (!a.rms) {
            float sum[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float v[kEach];
                row.values(raw, c, v);
#pragma unroll
                for (int q = 0; q < kEach; ++q) sum[0] += v[q];
            }
            row_sum<WAVES>(sum, s0);
            mean = sum[0] / n;
            widen_again(raw);
        }
        // About that mean, whose own rounding and sum the first moment corrects.
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float v[kEach];
            row.values(raw, c, v);
#pragma unroll
            for (int q = 0; q < kEach; ++q) {
                const float d = row.inside(c, q) ? v[q] - mean : 0.0f;
                sum[0] += d;
                sum[1] = fmaf(d, d, sum[1]);
            }
        }
        row_sum<WAVES>(sum, s1);
        float var = sum[1] / n;
        if (!a.rms) {
            const float off = sum[0] / n;
            mean += off;
            var = fmaf(-off, off, var);
            var = var < 0.0f ? 0.0f : var;  // NaN stays
        }
        const float rstd = 1.0f / sqrtf(var + a.eps);
        if (t == 0) {
            if (a.mean) a.mean[i] = mean;
            if (a.rstd) a.rstd[i] = rstd;
        }
        widen_again(raw);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!row.has(c)) continue;
            float v[kEach], w[kEach], b[kEach];
            load_params(a.w, a.w_f32, row.at(c), row.cnt(c), row.back(c), 1.0f, w);
            load_params(a.b, a.w_f32, row.at(c), row.cnt(c), row.back(c), 0.0f, b);
            row.values(raw, c, v);
#pragma unroll
            for (int q = 0; q < kEach; ++q) v[q] = fmaf((v[q] - mean) * rstd, w[q], b[q]);
            stream_store(static_cast<T*>(a.y) + i * a.ldy + row.at(c), row.cnt(c), a.wt, v);
        }
        // s0's and s1's next writes come behind a barrier of the other; alone, behind this one.
        if (WAVES > 1 && a.rms) __syncthreads();
    }
}

// A row that registers do not hold, read once for each sum and once for y.
constexpr int kLongBlock = 1024, kLongWaves = kLongBlock / 64;
template <typename T>
__global__ __launch_bounds__(kLongBlock) void norm_forward_long_kernel(ForwardArgs a) {
    __shared__ float s0[1][kLongWaves], s1[2][kLongWaves];
    const float n = static_cast<float>(a.n);
    for (int64_t i = blockIdx.x; i < a.m; i += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + i * a.ldx;
        T* y = static_cast<T*>(a.y) + i * a.ldy;
        auto value = [&](int64_t j) {
            if constexpr (sizeof(T) == 2) return widen(x[j]);
            else return x[j];
        };
        float mean = 0.0f;
        if (!a.rms) {
            float sum[1] = {0.0f};
            for (int64_t j = threadIdx.x; j < a.n; j += kLongBlock) sum[0] += value(j);
            row_sum<kLongWaves>(sum, s0);
            mean = sum[0] / n;
        }
        float sum[2] = {0.0f, 0.0f};
        for (int64_t j = threadIdx.x; j < a.n; j += kLongBlock) {
            const float d = value(j) - mean;
            sum[0] += d;
            sum[1] = fmaf(d, d, sum[1]);
        }
        row_sum<kLongWaves>(sum, s1);
        float var = sum[1] / n;
        if (!a.rms) {
            const float off = sum[0] / n;
            mean += off;
            var = fmaf(-off, off, var);
            var = var < 0.0f ? 0.0f : var;  // NaN stays
        }
        const float rstd = 1.0f / sqrtf(var + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[i] = mean;
            if (a.rstd) a.rstd[i] = rstd;
        }
        for (int64_t j = threadIdx.x; j < a.n; j += kLongBlock) {
            float w[1], b[1];
            load_params(a.w, a.w_f32, j, 1, 0, 1.0f, w);
            load_params(a.b, a.w_f32, j, 1, 0, 0.0f, b);
            const float v = fmaf((value(j) - mean) * rstd, w[0], b[0]);
            if constexpr (sizeof(T) == 2) y[j] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
            else y[j] = v;
        }
        if (a.rms) __syncthreads();
    }
}

// ---------------------------------------------------------------- backward

struct BackwardArgs {
    void* dx;
    const void* dy;
    const void* x;
    const void* res;
    const void* w;
    const float* mean;
    const float* rstd;
    float* part;  // [rows of sums][2][n], or null: no column sums
    int64_t lddx, lddy, ldx, ldr, m, n;
    int32_t w_f32, rms, wt;
};

// dx, and the column sums of the rows that a thread passes, which it holds for
// the columns of its chunks.  Rows stay packed in registers, and the next one is
// on its way while one is summed.
template <typename T, int WAVES, int C, bool TAIL>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void norm_backward_kernel(BackwardArgs a) {
    constexpr int kEach = 16 / sizeof(T), kRows = WAVES == 1 ? 4 : 1;
    __shared__ float s[2][2][WAVES];
    const int t = threadIdx.x % (64 * WAVES);
    Row<T, WAVES, C, TAIL> row;
    row.init(t, a.n);
    float w[C][kEach], dw[C][kEach], db[C][kEach];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        load_params(a.w, a.w_f32, row.at(c), row.has(c) ? row.cnt(c) : 0, row.back(c), 1.0f, w[c]);
#pragma unroll
        for (int q = 0; q < kEach; ++q) dw[c][q] = db[c][q] = 0.0f;
    }
    const float n = static_cast<float>(a.n);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / (64 * WAVES);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    struct Rows {
        u32x4 x[C], dy[C], res[C];
        float mean, rstd;
    };
    auto load = [&](int64_t i, Rows& r) {
        row.load(static_cast<const T*>(a.dy) + i * a.lddy, r.dy);
        row.load(static_cast<const T*>(a.x) + i * a.ldx, r.x);
        if (a.res) row.load(static_cast<const T*>(a.res) + i * a.ldr, r.res);
        r.mean = a.rms ? 0.0f : a.mean[i];
        r.rstd = a.rstd[i];
    };
    int turn = 0;
    Rows r;
    if (first < a.m) load(first, r);
    for (int64_t i = first; i < a.m; i += step, turn ^= 1) {
        Rows next;
        const bool more = i + step < a.m;
        if (more) load(i + step, next);
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float x[kEach], g[kEach];
            row.values(r.x, c, x);
            row.values(r.dy, c, g);
#pragma unroll
            for (int q = 0; q < kEach; ++q) {
                const float xhat = row.inside(c, q) ? (x[q] - r.mean) * r.rstd : 0.0f;
                dw[c][q] = fmaf(g[q], xhat, dw[c][q]);
                db[c][q] += g[q];
                const float gw = g[q] * w[c][q];
                sum[0] += gw;
                sum[1] = fmaf(gw, xhat, sum[1]);
            }
        }
        if (a.dx) {
            row_sum<WAVES>(sum, s[turn]);
            const float m1 = a.rms ? 0.0f : sum[0] / n, m2 = sum[1] / n;
            widen_again(r.x);
            widen_again(r.dy);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (!row.has(c)) continue;
                float x[kEach], g[kEach], res[kEach];
                row.values(r.x, c, x);
                row.values(r.dy, c, g);
                if (a.res) row.values(r.res, c, res);
#pragma unroll
                for (int q = 0; q < kEach; ++q) {
                    const float xhat = (x[q] - r.mean) * r.rstd, v = r.rstd * (g[q] * w[c][q] - m1 - xhat * m2);
                    g[q] = a.res ? v + res[q] : v;
                }
                stream_store(static_cast<T*>(a.dx) + i * a.lddx + row.at(c), row.cnt(c), a.wt, g);
            }
        }
        if (more) r = next;
    }
    if (!a.part) return;
    float* p = a.part + first * 2 * a.n;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int q = 0; q < kEach; ++q)
            if (row.inside(c, q)) {
                p[row.at(c) + q] = dw[c][q];
                p[a.n + row.at(c) + q] = db[c][q];
            }
}

// dx of a row that registers do not hold.
template <typename T>
__global__ __launch_bounds__(kLongBlock) void norm_backward_long_kernel(BackwardArgs a) {
    __shared__ float s[2][2][kLongWaves];
    const float n = static_cast<float>(a.n);
    int turn = 0;
    for (int64_t i = blockIdx.x; i < a.m; i += gridDim.x, turn ^= 1) {
        const float mean = a.rms ? 0.0f : a.mean[i], rstd = a.rstd[i];
        auto value = [](const void* p, int64_t at) {
            if constexpr (sizeof(T) == 2) return widen(static_cast<const T*>(p)[at]);
            else return static_cast<const T*>(p)[at];
        };
        auto terms = [&](int64_t j, float& xhat) {
            float w[1];
            load_params(a.w, a.w_f32, j, 1, 0, 1.0f, w);
            xhat = (value(a.x, i * a.ldx + j) - mean) * rstd;
            return value(a.dy, i * a.lddy + j) * w[0];
        };
        float sum[2] = {0.0f, 0.0f}, xhat;
        for (int64_t j = threadIdx.x; j < a.n; j += kLongBlock) {
            const float g = terms(j, xhat);
            sum[0] += g;
            sum[1] = fmaf(g, xhat, sum[1]);
        }
        row_sum<kLongWaves>(sum, s[turn]);
        const float m1 = a.rms ? 0.0f : sum[0] / n, m2 = sum[1] / n;
        for (int64_t j = threadIdx.x; j < a.n; j += kLongBlock) {
            const float g = terms(j, xhat);
            float v = rstd * (g - m1 - xhat * m2);
            if (a.res) v += value(a.res, i * a.ldr + j);
            T* const p = static_cast<T*>(a.dx) + i * a.lddx + j;
            if constexpr (sizeof(T) == 2) *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
            else *p = v;
        }
    }
}

// The column sums alone: 64 chunks of columns by 4 rows at a time, `rows` rows a
// block, into a row of `part` each; with one row block, into the results.
struct Sums {
    void* dw;
    void* db;
    int32_t f32, accumulate;
};
template <typename T>
__global__ __launch_bounds__(256) void norm_columns_kernel(BackwardArgs a, Sums out, int32_t cblocks, int64_t rows) {
    constexpr int kEach = 16 / sizeof(T);
    __shared__ float sums[2][4][64][kEach + 1];
    const int lane = threadIdx.x & 63, place = threadIdx.x >> 6;
    const int64_t rb = blockIdx.x / cblocks;
    const int64_t j0 = static_cast<int64_t>(blockIdx.x % cblocks) * (64 * kEach), j = j0 + lane * kEach;
    const int cnt = static_cast<int>(max(static_cast<int64_t>(0), min(a.n - j, static_cast<int64_t>(kEach))));
    const int back = chunk_back<T>(cnt, a.n);
    float dw[kEach], db[kEach];
#pragma unroll
    for (int q = 0; q < kEach; ++q) dw[q] = db[q] = 0.0f;
    const int64_t end = cnt > 0 ? min(a.m, (rb + 1) * rows) : 0;
    for (int64_t i = rb * rows + place; i < end; i += 4) {
        float x[kEach], g[kEach];
        const u32x4 wx = stream_load(static_cast<const T*>(a.x) + i * a.ldx + j, cnt, back);
        const u32x4 wg = stream_load(static_cast<const T*>(a.dy) + i * a.lddy + j, cnt, back);
        const float mean = a.rms ? 0.0f : a.mean[i], rstd = a.rstd[i];
        arrange(wx, back, x);
        arrange(wg, back, g);
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
            dw[q] = fmaf(g[q], (x[q] - mean) * rstd, dw[q]);
            db[q] += g[q];
        }
    }
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
        sums[0][place][lane][q] = dw[q];
        sums[1][place][lane][q] = db[q];
    }
    __syncthreads();
    for (int t = threadIdx.x; t < 2 * 64 * kEach; t += 256) {
        const int which = t / (64 * kEach), at = t % (64 * kEach);
        if (j0 + at >= a.n) continue;
        float v = sums[which][0][at / kEach][at % kEach];
#pragma unroll
        for (int p = 1; p < 4; ++p) v += sums[which][p][at / kEach][at % kEach];
        void* const to = which ? out.db : out.dw;
        if (a.part) a.part[(rb * 2 + which) * a.n + j0 + at] = v;
        else if (to) put_sum(to, out.f32, out.accumulate, j0 + at, v);
    }
}

// dw and db from `rows` rows of sums: 64 columns a block, 16 threads a column,
// their sums added in order.
constexpr int kSumBlock = 1024;
__global__ __launch_bounds__(kSumBlock) void norm_sum_kernel(const float* part, int64_t n, int64_t rows, Sums out) {
    __shared__ float sums[16][64];
    const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + c;
    float s = 0;
    if (col < 2 * n) {
#pragma unroll 8
        for (int64_t r = q; r < rows; r += 16) s += part[r * 2 * n + col];
    }
    sums[q][c] = s;
    __syncthreads();
    if (q != 0 || col >= 2 * n) return;
#pragma unroll
    for (int r = 1; r < 16; ++r) s += sums[r][c];
    void* const to = col < n ? out.dw : out.db;
    if (to) put_sum(to, out.f32, out.accumulate, col < n ? col : col - n, s);
}

// ---------------------------------------------------------------- host

int32_t check_kind(int32_t kind, const char* who) {
    if (kind != FSDP_NORM_LAYER && kind != FSDP_NORM_RMS) return fail(FSDP_E_ARG, "%s: unknown norm", who);
    return FSDP_OK;
}

int elem_of(int32_t dtype) { return dtype == FSDP_DT_BF16 ? 2 : 4; }

// How a row is divided: waves and chunks a lane; 0 waves: too long for registers.
struct Division {
    int waves, chunks;
};

// By its length alone, so that a row's result is the same among any others.
Division forward_division(int64_t n, int elem) {
    const int64_t chunks = ceil_div(n, 16 / elem);
    for (const Division d : {Division{1, 1}, {1, 2}, {1, 4}, {1, 8}, {4, 4}, {16, 2}, {16, 4}})
        if (chunks <= int64_t(64) * d.waves * d.chunks) return d;
    return {0, 0};
}

// The backward pass holds the column sums and two rows as well.
Division backward_division(int64_t n, int elem) {
    const int64_t chunks = ceil_div(n, 16 / elem);
    for (const Division d : {Division{1, 1}, {1, 2}, {4, 1}, {4, 2}, {4, 4}})
        if (chunks <= int64_t(64) * d.waves * d.chunks) return d;
    return {0, 0};
}

// f(waves, chunks) with constants
template <int W, int C, typename F>
bool with(const Division& d, F&& f) {
    if (d.waves != W || d.chunks != C) return false;
    f(std::integral_constant<int, W>(), std::integral_constant<int, C>());
    return true;
}

template <typename T>
void launch_forward(const ForwardArgs& a, hipStream_t stream) {
    const Division d = forward_division(a.n, sizeof(T));
    auto run = [&](auto waves, auto chunks) {
        constexpr int W = decltype(waves)::value, C = decltype(chunks)::value;
        const int64_t blocks = std::min<int64_t>(W == 1 ? ceil_div(a.m, 4) : a.m, kMaxBlocks);
        const dim3 grid(static_cast<uint32_t>(blocks)), block(W == 1 ? 256 : W * 64);
        if (a.n % (16 / sizeof(T)) == 0) norm_forward_kernel<T, W, C, false><<<grid, block, 0, stream>>>(a);
        else norm_forward_kernel<T, W, C, true><<<grid, block, 0, stream>>>(a);
    };
    if (with<1, 1>(d, run) || with<1, 2>(d, run) || with<1, 4>(d, run) || with<1, 8>(d, run) || with<4, 4>(d, run) ||
        with<16, 2>(d, run) || with<16, 4>(d, run))
        return;
    const uint32_t blocks = static_cast<uint32_t>(std::min<int64_t>(a.m, 2 * kCus));
    norm_forward_long_kernel<T><<<dim3(blocks), dim3(kLongBlock), 0, stream>>>(a);
}

int32_t forward_impl(void* y, int64_t ldy, float* mean, float* rstd, const void* x, int64_t ldx, int32_t dtype,
                     int32_t kind, const void* weight, const void* bias, int32_t w_dtype, double eps, int64_t m,
                     int64_t n, hipStream_t stream) {
    const char* who = "fsdp_norm_forward";
    TRY(check_sizes(m, n, 0, who));
    TRY(check_float_dtype(dtype, "dtype", who));
    TRY(check_float_dtype(w_dtype, "w_dtype", who));
    TRY(check_kind(kind, who));
    if (!(eps >= 0.0 && std::isfinite(static_cast<float>(eps))))
        return fail(FSDP_E_ARG, "%s: eps must be at least 0, and finite in fp32", who);
    if (kind == FSDP_NORM_RMS && mean) return fail(FSDP_E_ARG, "%s: the RMS norm has no mean", who);
    const int e = elem_of(dtype), we = elem_of(w_dtype);
    const Matrix my{y, m, n, ldy, e, "y", true}, mx{x, m, n, ldx, e, "x", false};
    const Matrix mm = vector(mean, m, 4, "mean", true), mr = vector(rstd, m, 4, "rstd", true);
    const Matrix mw = vector(weight, n, we, "weight"), mb = vector(bias, n, we, "bias");
    TRY(check_matrix(my, false, who));
    TRY(check_matrix(mx, false, who));
    for (const Matrix& v : {mm, mr, mw, mb}) TRY(check_matrix(v, true, who));
    TRY(check_overlaps({my, mm, mr, mx, mw, mb}, who,
                       [&](const Matrix& p, const Matrix& q) { return p.what == my.what && q.what == mx.what; }));
    if (m == 0 || n == 0) return FSDP_OK;
    ForwardArgs a{};
    a.y = y;
    a.x = x;
    a.w = weight;
    a.b = bias;
    a.mean = mean;
    a.rstd = rstd;
    a.ldy = ldy;
    a.ldx = ldx;
    a.m = m;
    a.n = n;
    a.eps = static_cast<float>(eps);
    a.w_f32 = we == 4;
    a.rms = kind == FSDP_NORM_RMS;
    a.wt = stream_ok(y, ldy, e);
    if (e == 2) launch_forward<uint16_t>(a, stream);
    else launch_forward<float>(a, stream);
    return launched(who);
}

template <typename T>
int32_t launch_backward(BackwardArgs a, const Sums& out, float* workspace, int64_t bytes, hipStream_t stream,
                        const char* who) {
    const bool sums = out.dw || out.db;
    const Division d = backward_division(a.n, sizeof(T));
    const int64_t room = std::min(bytes, FSDP_NORM_WORKSPACE_BYTES) / (8 * a.n);  // rows of sums
    int64_t blocks = std::min<int64_t>(d.waves == 1 ? ceil_div(a.m, 4) : a.m, 2 * kCus);
    const int64_t each = d.waves == 1 ? 4 : 1;  // rows of sums that a block writes
    if (d.waves > 0 && (a.dx || sums)) {
        // with fewer parts than a quarter of the chip the sums are taken apart
        const bool together = sums && room >= std::min<int64_t>(a.m, each * kCus / 4);
        if (together) {
            blocks = std::min(blocks, room / each);
            a.part = workspace;
        }
        if (together || a.dx) {
            auto run = [&](auto waves, auto chunks) {
                constexpr int W = decltype(waves)::value, C = decltype(chunks)::value;
                const dim3 grid(static_cast<uint32_t>(blocks)), block(W == 1 ? 256 : W * 64);
                if (a.n % (16 / sizeof(T)) == 0) norm_backward_kernel<T, W, C, false><<<grid, block, 0, stream>>>(a);
                else norm_backward_kernel<T, W, C, true><<<grid, block, 0, stream>>>(a);
            };
            with<1, 1>(d, run) || with<1, 2>(d, run) || with<4, 1>(d, run) || with<4, 2>(d, run) || with<4, 4>(d, run);
            TRY(launched(who));
        }
        if (together) {
            norm_sum_kernel<<<dim3(static_cast<uint32_t>(ceil_div(2 * a.n, 64))), dim3(kSumBlock), 0, stream>>>(
                workspace, a.n, blocks * each, out);
            return launched(who);
        }
    } else if (a.dx) {
        const uint32_t long_blocks = static_cast<uint32_t>(std::min<int64_t>(a.m, 2 * kCus));
        norm_backward_long_kernel<T><<<dim3(long_blocks), dim3(kLongBlock), 0, stream>>>(a);
        TRY(launched(who));
    }
    if (!sums) return FSDP_OK;
    const int64_t cblocks = ceil_div(a.n, 64 * (16 / static_cast<int64_t>(sizeof(T))));
    const int64_t want = std::max<int64_t>(1, std::min(8 * kCus / cblocks, room));
    const int64_t rows = ceil_div(ceil_div(a.m, 4), want) * 4, rblocks = ceil_div(a.m, rows);
    a.part = rblocks > 1 ? workspace : nullptr;
    norm_columns_kernel<T><<<dim3(static_cast<uint32_t>(cblocks * rblocks)), dim3(256), 0, stream>>>(
        a, out, static_cast<int32_t>(cblocks), rows);
    TRY(launched(who));
    if (rblocks == 1) return FSDP_OK;
    norm_sum_kernel<<<dim3(static_cast<uint32_t>(ceil_div(2 * a.n, 64))), dim3(kSumBlock), 0, stream>>>(workspace, a.n,
                                                                                                       rblocks, out);
    return launched(who);
}

// dw and db of no rows.
__global__ __launch_bounds__(256) void norm_zero_kernel(int64_t n, Sums out) {
    for (int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; j < n; j += static_cast<int64_t>(gridDim.x) * 256) {
        if (out.dw) put_sum(out.dw, out.f32, 0, j, 0.0f);
        if (out.db) put_sum(out.db, out.f32, 0, j, 0.0f);
    }
}

int32_t backward_impl(void* dx, int64_t lddx, void* dw, void* db, int32_t dw_dtype, int32_t accumulate, const void* dy,
                      int64_t lddy, const void* x, int64_t ldx, int32_t dtype, int32_t kind, const void* weight,
                      int32_t w_dtype, const float* mean, const float* rstd, const void* residual, int64_t ldr,
                      int64_t m, int64_t n, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    const char* who = "fsdp_norm_backward";
    TRY(check_sizes(m, n, 0, who));
    TRY(check_float_dtype(dtype, "dtype", who));
    TRY(check_float_dtype(w_dtype, "w_dtype", who));
    TRY(check_float_dtype(dw_dtype, "dw_dtype", who));
    TRY(check_flag(accumulate, "accumulate", who));
    TRY(check_kind(kind, who));
    TRY(check_workspace(workspace, workspace_bytes, who));
    if (kind == FSDP_NORM_RMS && mean) return fail(FSDP_E_ARG, "%s: the RMS norm has no mean", who);
    const int e = elem_of(dtype), we = elem_of(w_dtype), de = elem_of(dw_dtype);
    const Matrix mdx{dx, m, n, lddx, e, "dx", true}, mdy{dy, m, n, lddy, e, "dy", false};
    const Matrix mx{x, m, n, ldx, e, "x", false}, mr{residual, m, n, ldr, e, "residual", false};
    const Matrix mdw = vector(dw, n, de, "dw", true), mdb = vector(db, n, de, "db", true);
    const Matrix mw = vector(weight, n, we, "weight"), mm = vector(mean, m, 4, "mean"), ms = vector(rstd, m, 4, "rstd");
    TRY(check_matrix(mdx, true, who));
    TRY(check_matrix(mdy, false, who));
    TRY(check_matrix(mx, false, who));
    TRY(check_matrix(ms, n == 0, who));
    TRY(check_matrix(mm, n == 0 || kind == FSDP_NORM_RMS, who));
    for (const Matrix& v : {mr, mdw, mdb, mw}) TRY(check_matrix(v, true, who));
    TRY(check_overlaps({mdx, mdw, mdb, bytes_of(workspace, std::min(workspace_bytes, FSDP_NORM_WORKSPACE_BYTES), "workspace", true),
                        mdy, mx, mr, mw, mm, ms},
                       who, [&](const Matrix& p, const Matrix& q) { return p.what == mdx.what && q.what == mr.what; }));
    if (n == 0 || (!dx && !dw && !db)) return FSDP_OK;
    const Sums out{dw, db, de == 4, accumulate};
    if (m == 0) {
        if (accumulate || (!dw && !db)) return FSDP_OK;
        norm_zero_kernel<<<dim3(static_cast<uint32_t>(std::min<int64_t>(ceil_div(n, 256), kCus))), dim3(256), 0, stream>>>(n, out);
        return launched(who);
    }
    BackwardArgs a{};
    a.dx = dx;
    a.dy = dy;
    a.x = x;
    a.res = residual;
    a.w = weight;
    a.mean = mean;
    a.rstd = rstd;
    a.lddx = lddx;
    a.lddy = lddy;
    a.ldx = ldx;
    a.ldr = ldr;
    a.m = m;
    a.n = n;
    a.w_f32 = we == 4;
    a.rms = kind == FSDP_NORM_RMS;
    a.wt = stream_ok(dx, lddx, e);
    float* const ws = static_cast<float*>(workspace);
    if (e == 2) return launch_backward<uint16_t>(a, out, ws, workspace_bytes, stream, who);
    return launch_backward<float>(a, out, ws, workspace_bytes, stream, who);
}

}  // namespace

// ---------------------------------------------------------------- entry points

extern "C" int32_t fsdp_norm_forward(void* y, int64_t ldy, float* mean, float* rstd, const void* x, int64_t ldx,
                                     int32_t dtype, int32_t kind, const void* weight, const void* bias,
                                     int32_t w_dtype, double eps, int64_t m, int64_t n, hipStream_t stream) {
    return fsdp::guarded("fsdp_norm_forward", [&] {
        return forward_impl(y, ldy, mean, rstd, x, ldx, dtype, kind, weight, bias, w_dtype, eps, m, n, stream);
    });
}

extern "C" int32_t fsdp_norm_backward(void* dx, int64_t lddx, void* dw, void* db, int32_t dw_dtype, int32_t accumulate,
                                      const void* dy, int64_t lddy, const void* x, int64_t ldx, int32_t dtype,
                                      int32_t kind, const void* weight, int32_t w_dtype, const float* mean,
                                      const float* rstd, const void* residual, int64_t ldr, int64_t m, int64_t n,
                                      void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    return fsdp::guarded("fsdp_norm_backward", [&] {
        return backward_impl(dx, lddx, dw, db, dw_dtype, accumulate, dy, lddy, x, ldx, dtype, kind, weight, w_dtype,
                             mean, rstd, residual, ldr, m, n, workspace, workspace_bytes, stream);
    });
}
