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

// The sum of N values, a power of two, by halves: a shorter chain of roundings
// and of waits than one after the other.
template <int N>
__device__ __forceinline__ float sum_halves(float (&v)[N]) {
#pragma unroll
    for (int h = N / 2; h > 0; h /= 2)
#pragma unroll
        for (int i = 0; i < h; ++i) v[i] += v[i + h];
    return v[0];
}

// N parameters from element j on in fp32, `none` where there is no vector.
template <int N>
__device__ __forceinline__ void load_params(const void* p, int f32, int64_t j, float none, float (&v)[N]) {
    struct __attribute__((packed, aligned(4))) Floats { float v[N]; };
    struct __attribute__((packed, aligned(2))) Halves { uint16_t v[N]; };
    if (!p) {
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = none;
    } else if (f32) {
        const Floats w = *reinterpret_cast<const Floats*>(static_cast<const float*>(p) + j);
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = w.v[q];
    } else {
        const Halves w = *reinterpret_cast<const Halves*>(static_cast<const uint16_t*>(p) + j);
#pragma unroll
        for (int q = 0; q < N; ++q) v[q] = widen(w.v[q]);
    }
}
__device__ __forceinline__ float load_param(const void* p, int f32, int64_t j, float none) {
    float v[1];
    load_params(p, f32, j, none, v);
    return v[0];
}

// A thread's part of a row: of the whole chunks of 16 bytes, chunk c from element
// (c * 64 WAVES + t) * E on; and with TAIL one of the fewer than E elements
// behind them, or none.  (A last chunk read as the E elements that end with the
// row, and moved, cost twice the registers for all chunks.)
template <typename T, int WAVES, int C, bool TAIL>
struct Row {
    static constexpr int kEach = 16 / sizeof(T);
    int first;  // element of the thread's first chunk
    int whole;  // elements in whole chunks
    int last;   // the element behind them, or -1

    __device__ __forceinline__ void init(int t, int64_t n) {
        first = t * kEach;
        whole = static_cast<int>(n) / kEach * kEach;
        last = TAIL && whole + t < n ? whole + t : -1;
    }
    __device__ __forceinline__ int at(int c) const { return first + c * (64 * WAVES * kEach); }
    __device__ __forceinline__ bool has(int c) const { return at(c) < whole; }
    __device__ __forceinline__ bool tail() const { return TAIL && last >= 0; }
    __device__ __forceinline__ void load(const T* row, u32x4 (&w)[C], float& end) const {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            w[c] = u32x4{0, 0, 0, 0};
            if (has(c)) w[c] = stream_load(row + at(c), kEach, 0);
        }
        end = 0.0f;
        if (tail()) end = element(row);
    }
    __device__ __forceinline__ float element(const T* row) const {
        if constexpr (sizeof(T) == 2) return widen(row[last]);
        else return row[last];
    }
    __device__ __forceinline__ void store_element(T* row, float v) const {
        if constexpr (sizeof(T) == 2) row[last] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
        else row[last] = v;
    }
};

// Packed chunks whose widened values are not kept from here on: the compiler
// would rather hold them, at twice the registers of bf16, than widen again.
template <int C>
__device__ __forceinline__ void widen_again(u32x4 (&w)[C]) {
#pragma unroll
    for (int c = 0; c < C; ++c) asm volatile("" : "+v"(w[c])::"memory");
}

// The variance about the true mean, which lies `off` from the first estimate
// by the sum of the differences; and the mean itself where it is large against the
// spread.  Elsewhere the first estimate is the better one: of bf16 values a sum is
// nearly exact, where the differences' roundings are alike for all values of a
// binade and do not cancel (3e-8 of the spread).
__device__ __forceinline__ void correct(float off, float& mean, float& var) {
    if (mean * mean > 16.0f * var) mean += off;
    var = fmaf(-off, off, var);
    var = var < 0.0f ? 0.0f : var;  // NaN stays
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
    double eps;  // rounded to fp32 but in forward_row_wide
    int32_t w_f32, rms, wt;
};

// Whether fp32 held the sum of squares: not where it, or the row's sum, has passed
// 2^128, nor where squares may have been lost below 2^-126.  The same in all the
// row's lanes; false for NaN.
__device__ __forceinline__ bool in_range(float var_eps) { return var_eps >= 0x1p-100f && var_eps < INFINITY; }

__device__ __forceinline__ double wide(uint16_t v) { return widen(v); }
__device__ __forceinline__ double wide(float v) { return v; }

// Thread t's sum over the row's waves, as row_sum, with a shared `s` of its own for
// each of a row's sums.
template <int WAVES>
__device__ __forceinline__ double row_sum(double v, double* s, int t) {
#pragma unroll 1
    for (int d = 1; d < 64; d <<= 1) {
        const u32x2 w = __builtin_bit_cast(u32x2, v);
        const int from = ((t ^ d) & 63) * 4;
        v += __builtin_bit_cast(double, u32x2{static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(from, static_cast<int>(w[0]))),
                                              static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(from, static_cast<int>(w[1])))});
    }
    if constexpr (WAVES > 1) {
        if ((t & 63) == 0) s[t >> 6] = v;
        __syncthreads();
        v = s[0];
#pragma unroll 1
        for (int p = 1; p < WAVES; ++p) v += s[p];
    }
    return v;
}

// The thread's number among a row's threads, which the compiler takes for another
// one each time: what depends on it is made where it is used, and holds no
// registers across forward_row_wide.
template <int WAVES>
__device__ __forceinline__ int opaque_thread() {
    int t = threadIdx.x % (64 * WAVES);
    asm volatile("" : "+v"(t));
    return t;
}

// Row i in 64 bits, read again for each sum: the few rows that fp32's range does
// not hold, and those with an infinity or a NaN.  A thread reads and writes the
// same elements, so y may be x.  8192 such rows of 4096 bf16: 131 us.
template <typename T, int WAVES>
__device__ __forceinline__ void forward_row_wide(const ForwardArgs& a, int64_t i, int t) {
    __shared__ double s[2][WAVES];
    int64_t cols = a.n;
    asm volatile("" : "+s"(cols));  // as in opaque_thread
    const T* const x = static_cast<const T*>(a.x) + i * a.ldx;
    T* const y = static_cast<T*>(a.y) + i * a.ldy;
    const double n = static_cast<double>(cols);
    double mean = 0.0, var = 0.0;
    if (!a.rms) {
#pragma unroll 1
        for (int64_t j = t; j < cols; j += 64 * WAVES) mean += wide(x[j]);
        mean = row_sum<WAVES>(mean, s[0], t) / n;
    }
#pragma unroll 1
    for (int64_t j = t; j < cols; j += 64 * WAVES) {
        const double d = wide(x[j]) - mean;
        var = fma(d, d, var);
    }
    const double rstd = 1.0 / sqrt(row_sum<WAVES>(var, s[1], t) / n + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[i] = static_cast<float>(mean);
        if (a.rstd) a.rstd[i] = static_cast<float>(rstd);
    }
#pragma unroll 1
    for (int64_t j = t; j < cols; j += 64 * WAVES) {
        const float w = load_param(a.w, a.w_f32, j, 1.0f), b = load_param(a.b, a.w_f32, j, 0.0f);
        const float v = static_cast<float>(fma((wide(x[j]) - mean) * rstd, static_cast<double>(w), static_cast<double>(b)));
        if constexpr (sizeof(T) == 2) y[j] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
        else y[j] = v;
    }
    if (WAVES > 1) __syncthreads();  // before the next row's sums
}

// A row by WAVES waves of C chunks of 16 bytes a lane, which stay packed in
// registers and are widened for each pass over them.  Bound by memory, a
// workgroup a row (four where a wave takes one), so that some rows load while
// others store: 8192 x 4096 bf16 26.8 us (5.0 TB/s; a copy's 20.7).  With rows held
// widened and workgroups that stay for several 42, one wave a row 30, eight 32.
// The addresses and conditions of a lane's chunks are made for each row, which
// takes up to half of the registers less than before the loop (8192 x 2048 bf16
// 14.5 us for 17.5, 8192 x 11008 75.5 for 97, 8192 x 11007 fp32 140 for 171); but
// before it (kAhead) where that was the faster way: 8192 x 4096 bf16 28.7 for 30.2,
// fp32 48.6 for 51.7, 8192 x 4095 fp32 52.9 for 55.6.  With more than 80 scalar
// registers a SIMD has not eight waves: 8192 x 1024 fp32 13.5 us, with 87 15.0.
template <typename T, int WAVES, int C, bool TAIL>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) __attribute__((amdgpu_num_sgpr(80)))
void norm_forward_kernel(ForwardArgs a) {
    constexpr int kEach = 16 / sizeof(T), kRows = WAVES == 1 ? 4 : 1;
    constexpr bool kAhead = WAVES == 4 && (sizeof(T) == 4 ? C == 4 : C == 2 && !TAIL);
    __shared__ float s0[1][WAVES], s1[2][WAVES];
    const float n = static_cast<float>(a.n), eps = static_cast<float>(a.eps);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / (64 * WAVES); i < a.m;
         i += static_cast<int64_t>(gridDim.x) * kRows) {
        const int t = kAhead ? threadIdx.x % (64 * WAVES) : opaque_thread<WAVES>();
        Row<T, WAVES, C, TAIL> row;
        row.init(t, a.n);
        u32x4 raw[C];
        float end;
        row.load(static_cast<const T*>(a.x) + i * a.ldx, raw, end);
        float mean = 0.0f;
        if (!a.rms) {
            float sum[1] = {end};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float v[kEach];
                arrange(raw[c], 0, v);
#pragma unroll
                for (int q = 0; q < kEach; ++q) sum[0] += v[q];
            }
            row_sum<WAVES>(sum, s0);
            mean = sum[0] / n;
            widen_again(raw);
        }
        // About that mean.
        float sum[2] = {0.0f, 0.0f};
        if (row.tail()) {
            sum[0] = end - mean;
            sum[1] = sum[0] * sum[0];
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float v[kEach];
            arrange(raw[c], 0, v);
#pragma unroll
            for (int q = 0; q < kEach; ++q) {
                const float d = row.has(c) ? v[q] - mean : 0.0f;
                sum[0] += d;
                sum[1] = fmaf(d, d, sum[1]);
            }
        }
        row_sum<WAVES>(sum, s1);
        float var = sum[1] / n;
        if (!a.rms) correct(sum[0] / n, mean, var);
        if (__builtin_expect(!in_range(var + eps), 0)) {
            forward_row_wide<T, WAVES>(a, i, opaque_thread<WAVES>());
            continue;
        }
        const float rstd = 1.0f / sqrtf(var + eps);
        if (t == 0) {
            if (a.mean) a.mean[i] = mean;
            if (a.rstd) a.rstd[i] = rstd;
        }
        widen_again(raw);
        T* const y = static_cast<T*>(a.y) + i * a.ldy;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!row.has(c)) continue;
            float v[kEach], w[kEach], b[kEach];
            load_params(a.w, a.w_f32, row.at(c), 1.0f, w);
            load_params(a.b, a.w_f32, row.at(c), 0.0f, b);
            arrange(raw[c], 0, v);
#pragma unroll
            for (int q = 0; q < kEach; ++q) v[q] = fmaf((v[q] - mean) * rstd, w[q], b[q]);
            stream_store(y + row.at(c), kEach, a.wt, v);
        }
        if (row.tail())
            row.store_element(y, fmaf((end - mean) * rstd, load_param(a.w, a.w_f32, row.last, 1.0f),
                                      load_param(a.b, a.w_f32, row.last, 0.0f)));
        // s0's and s1's next writes come behind a barrier of the other; alone, behind this one.
        if (WAVES > 1 && a.rms) __syncthreads();
    }
}

// f(j, v) with the values from element j on of what a thread takes of a row of any
// length: of the whole chunks of 16 bytes every kLongBlock-th, then one of the
// elements behind them or none.  Each of `rows` gives as many values.
constexpr int kLongBlock = 1024, kLongWaves = kLongBlock / 64;
template <int N>
struct Values {
    float v[N];
};
template <typename T, int ROWS, typename F>
__device__ __forceinline__ void over_row(const T* const (&rows)[ROWS], int64_t n, F&& f) {
    constexpr int kEach = 16 / sizeof(T);
    const int64_t whole = n / kEach * kEach, last = whole + threadIdx.x;
#pragma unroll 2
    for (int64_t j = static_cast<int64_t>(threadIdx.x) * kEach; j < whole; j += kLongBlock * kEach) {
        Values<kEach> v[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            if (rows[r]) arrange(reinterpret_cast<const Bytes16*>(rows[r] + j)->v, 0, v[r].v);
        }
        f(j, v);
    }
    if (last >= n) return;
    Values<1> v[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (!rows[r]) continue;
        if constexpr (sizeof(T) == 2) v[r].v[0] = widen(rows[r][last]);
        else v[r].v[0] = rows[r][last];
    }
    f(last, v);
}
template <int N>
__device__ __forceinline__ void store_values(uint16_t* p, const Values<N>& x) {
    if constexpr (N == 1) *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x.v[0]));
    else store8(p, N, x.v);
}
template <int N>
__device__ __forceinline__ void store_values(float* p, const Values<N>& x) {
    if constexpr (N == 1) *p = x.v[0];
    else stream_store(p, N, false, x.v);
}

// A row that registers do not hold, read once for each sum and once for y.  Its
// length has no bound, so a thread joins its chunks' sums in 64 bits.
// 1024 x 65536 bf16 with weight, bias and statistics 95 us (a copy's 41): a row's
// second and third read come from L2.
template <typename T>
__global__ __launch_bounds__(kLongBlock) void norm_forward_long_kernel(ForwardArgs a) {
    __shared__ float s0[1][kLongWaves], s1[2][kLongWaves];
    const float n = static_cast<float>(a.n), eps = static_cast<float>(a.eps);
    for (int64_t i = blockIdx.x; i < a.m; i += gridDim.x) {
        const T* const x[1] = {static_cast<const T*>(a.x) + i * a.ldx};
        T* const y = static_cast<T*>(a.y) + i * a.ldy;
        float mean = 0.0f;
        if (!a.rms) {
            double all = 0.0;
            over_row(x, a.n, [&](int64_t, const auto(&v)[1]) {
                float part = 0.0f;
                for (float e : v[0].v) part += e;
                all += part;
            });
            float sum[1] = {static_cast<float>(all)};
            row_sum<kLongWaves>(sum, s0);
            mean = sum[0] / n;
        }
        double all[2] = {0.0, 0.0};
        over_row(x, a.n, [&](int64_t, const auto(&v)[1]) {
            float part[2] = {0.0f, 0.0f};
            for (float e : v[0].v) {
                const float d = e - mean;
                part[0] += d;
                part[1] = fmaf(d, d, part[1]);
            }
            all[0] += part[0];
            all[1] += part[1];
        });
        float sum[2] = {static_cast<float>(all[0]), static_cast<float>(all[1])};
        row_sum<kLongWaves>(sum, s1);
        float var = sum[1] / n;
        if (!a.rms) correct(sum[0] / n, mean, var);
        if (__builtin_expect(!in_range(var + eps), 0)) {
            forward_row_wide<T, kLongWaves>(a, i, opaque_thread<kLongWaves>());
            continue;
        }
        const float rstd = 1.0f / sqrtf(var + eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[i] = mean;
            if (a.rstd) a.rstd[i] = rstd;
        }
        over_row(x, a.n, [&](int64_t j, const auto(&v)[1]) {
            auto out = v[0];
            constexpr int N = sizeof(out.v) / sizeof(float);
            float w[N], b[N];
            load_params(a.w, a.w_f32, j, 1.0f, w);
            load_params(a.b, a.w_f32, j, 0.0f, b);
#pragma unroll
            for (int q = 0; q < N; ++q) out.v[q] = fmaf((out.v[q] - mean) * rstd, w[q], b[q]);
            store_values(y + j, out);
        });
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
    float* part;  // [rows of sums][2][n]; norm_columns_kernel: null with one row of them
    int64_t lddx, lddy, ldx, ldr, m, n;
    int32_t w_f32, rms, wt;
};

// dx of row i by WAVES waves, which read it once.
template <typename T, int WAVES, int C, bool TAIL>
__device__ __forceinline__ void dx_row(const BackwardArgs& a, int64_t i, int t, float (*s)[WAVES]) {
    constexpr int kEach = 16 / sizeof(T);
    Row<T, WAVES, C, TAIL> row;
    row.init(t, a.n);
    u32x4 rx[C], rdy[C];
    float ex, edy;
    row.load(static_cast<const T*>(a.dy) + i * a.lddy, rdy, edy);
    row.load(static_cast<const T*>(a.x) + i * a.ldx, rx, ex);
    const float mean = a.rms ? 0.0f : a.mean[i], rstd = a.rstd[i], n = static_cast<float>(a.n);
    float sum[2] = {0.0f, 0.0f};
    if (row.tail()) {
        sum[0] = edy *= load_param(a.w, a.w_f32, row.last, 1.0f);
        sum[1] = edy * (ex = (ex - mean) * rstd);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (!row.has(c)) continue;
        float x[kEach], g[kEach], w[kEach];
        load_params(a.w, a.w_f32, row.at(c), 1.0f, w);
        arrange(rx[c], 0, x);
        arrange(rdy[c], 0, g);
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
            const float gw = g[q] * w[q];
            sum[0] += gw;
            sum[1] = fmaf(gw, (x[q] - mean) * rstd, sum[1]);
        }
    }
    row_sum<WAVES>(sum, s);
    const float m1 = a.rms ? 0.0f : sum[0] / n, m2 = sum[1] / n;
    widen_again(rx);
    widen_again(rdy);
    const T* const res = static_cast<const T*>(a.res) + (a.res ? i * a.ldr : 0);
    T* const dx = static_cast<T*>(a.dx) + i * a.lddx;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (!row.has(c)) continue;
        float x[kEach], g[kEach], w[kEach], r[kEach];
        if (a.res) arrange(stream_load(res + row.at(c), kEach, 0), 0, r);
        load_params(a.w, a.w_f32, row.at(c), 1.0f, w);
        arrange(rx[c], 0, x);
        arrange(rdy[c], 0, g);
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
            const float xhat = (x[q] - mean) * rstd, v = rstd * (g[q] * w[q] - m1 - xhat * m2);
            g[q] = a.res ? v + r[q] : v;
        }
        stream_store(dx + row.at(c), kEach, a.wt, g);
    }
    if (row.tail()) {
        const float v = rstd * (edy - m1 - ex * m2);
        row.store_element(dx, a.res ? v + row.element(res) : v);
    }
}

// dx alone: without column sums, or beside norm_columns_kernel for rows whose
// sums registers do not hold.  Bound by memory: 8192 x 4096 bf16 35 us (5.8 TB/s).
template <typename T, int WAVES, int C, bool TAIL>
__global__ __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) void norm_dx_kernel(BackwardArgs a) {
    constexpr int kRows = WAVES == 1 ? 4 : 1;
    __shared__ float s[2][2][WAVES];
    int turn = 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / (64 * WAVES); i < a.m;
         i += static_cast<int64_t>(gridDim.x) * kRows, turn ^= 1)
        dx_row<T, WAVES, C, TAIL>(a, i, threadIdx.x % (64 * WAVES), s[turn]);
}

// Rows of a workgroup of the backward pass at a time.
constexpr int backward_rows(int waves) { return waves == 1 ? 8 : 1; }

// Rows that a thread adds in fp32, one after the other; the sums of as many are
// joined in 64 bits.  In one chain the roundings of terms that are alike go one
// way, and a sum stops growing at 2^24 times them: over 2^17 equal rows chains of
// 2^11 were off by 3e-5, of 2^15 by 4e-4, for at most 9e-6 this way.
constexpr int kChain = 64;

// dx, and the column sums of the rows that a thread passes, which it holds for
// the columns of its chunks.  Rows stay packed in registers, and the next one is
// on its way while one is summed (two ahead: 20 % slower).  Bound by memory: 8192
// x 4096 bf16 with a residual and both sums 58 us, of which 5 for joining the
// workgroups' sums (floor 41).  A workgroup leaves one row of sums, and two a CU
// stay for all rows: three a CU 69 us, four 73, for more sums to write and read;
// one 69, for fewer loads on their way.  The registers allow two a CU with one
// chunk a lane only (8192 x 1000: two of which one waits 24 us, one 18), and there
// they are held to it (8192 x 4095: 113 us without, this way 84).  LONG: a wave
// passes more than kChain rows; their sums wait in LDS, 16 bytes a column, which
// leaves room for as many workgroups.
template <typename T, int WAVES, int C, bool TAIL, bool LONG>
__global__ __launch_bounds__(backward_rows(WAVES) * WAVES * 64, C == 1 ? 4 : 2) void norm_backward_kernel(BackwardArgs a) {
    constexpr int kEach = 16 / sizeof(T), kRows = backward_rows(WAVES);
    __shared__ float s[2][2][WAVES];
    __shared__ float joined[kRows > 1 ? 2 : 1][kRows > 1 ? C * kEach + TAIL : 1][64];
    __shared__ double2 chains[LONG ? C * kEach + TAIL : 1][LONG ? kRows * WAVES * 64 : 1];  // each thread's own
    const int t = threadIdx.x % (64 * WAVES);
    Row<T, WAVES, C, TAIL> row;
    row.init(t, a.n);
    float w[C][kEach], dw[C][kEach], db[C][kEach];
    float ew = 0.0f, edw = 0.0f, edb = 0.0f;  // the tail's
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int q = 0; q < kEach; ++q) w[c][q] = dw[c][q] = db[c][q] = 0.0f;
        if (row.has(c)) load_params(a.w, a.w_f32, row.at(c), 1.0f, w[c]);
    }
    if (row.tail()) ew = load_param(a.w, a.w_f32, row.last, 1.0f);
    const float n = static_cast<float>(a.n);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / (64 * WAVES);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    struct Rows {
        u32x4 x[C], dy[C], res[C];
        float ex, edy, eres, mean, rstd;
    };
    auto load = [&](int64_t i, Rows& r) {
        row.load(static_cast<const T*>(a.dy) + i * a.lddy, r.dy, r.edy);
        row.load(static_cast<const T*>(a.x) + i * a.ldx, r.x, r.ex);
        if (a.res) row.load(static_cast<const T*>(a.res) + i * a.ldr, r.res, r.eres);
        r.mean = a.rms ? 0.0f : a.mean[i];
        r.rstd = a.rstd[i];
    };
    // f(number, dw, db) of each pair of the thread's sums
    auto each_sum = [&](auto&& f) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int q = 0; q < kEach; ++q) f(c * kEach + q, dw[c][q], db[c][q]);
        if (TAIL) f(C * kEach, edw, edb);
    };
    int turn = 0, added = 0;
    Rows r;
    if (first < a.m) load(first, r);
    for (int64_t i = first; i < a.m; i += step, turn ^= 1) {
        Rows next;
        const bool more = i + step < a.m;
        if (more) load(i + step, next);
        float sum[2] = {0.0f, 0.0f};
        if (row.tail()) {
            r.ex = (r.ex - r.mean) * r.rstd;
            edw = fmaf(r.edy, r.ex, edw);
            edb += r.edy;
            sum[0] = r.edy *= ew;
            sum[1] = r.edy * r.ex;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float x[kEach], g[kEach];
            arrange(r.x[c], 0, x);
            arrange(r.dy[c], 0, g);
#pragma unroll
            for (int q = 0; q < kEach; ++q) {
                const float xhat = row.has(c) ? (x[q] - r.mean) * r.rstd : 0.0f;
                dw[c][q] = fmaf(g[q], xhat, dw[c][q]);
                db[c][q] += g[q];
                const float gw = g[q] * w[c][q];
                sum[0] += gw;
                sum[1] = fmaf(gw, xhat, sum[1]);
            }
        }
        row_sum<WAVES>(sum, s[turn]);
        const float m1 = a.rms ? 0.0f : sum[0] / n, m2 = sum[1] / n;
        widen_again(r.x);
        widen_again(r.dy);
        T* const dx = static_cast<T*>(a.dx) + i * a.lddx;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!row.has(c)) continue;
            float x[kEach], g[kEach], res[kEach];
            arrange(r.x[c], 0, x);
            arrange(r.dy[c], 0, g);
            if (a.res) arrange(r.res[c], 0, res);
#pragma unroll
            for (int q = 0; q < kEach; ++q) {
                const float xhat = (x[q] - r.mean) * r.rstd, v = r.rstd * (g[q] * w[c][q] - m1 - xhat * m2);
                g[q] = a.res ? v + res[q] : v;
            }
            stream_store(dx + row.at(c), kEach, a.wt, g);
        }
        if (row.tail()) {
            const float v = r.rstd * (r.edy - m1 - r.ex * m2);
            row.store_element(dx, a.res ? v + r.eres : v);
        }
        if (more) r = next;
        if constexpr (LONG) {
            if (++added % kChain == 0)
                each_sum([&](int at, float& x, float& y) {
                    double2& sum = chains[at][threadIdx.x];
                    sum = added > kChain ? double2{sum.x + x, sum.y + y} : double2{x, y};
                    x = y = 0.0f;
                });
        }
    }
    if (LONG && added >= kChain)
        each_sum([&](int at, float& x, float& y) {
            x = static_cast<float>(chains[at][threadIdx.x].x + x);
            y = static_cast<float>(chains[at][threadIdx.x].y + y);
        });
    if constexpr (kRows > 1) {
        // the waves' sums one after the other, into the last one's registers
        const int wave = threadIdx.x >> 6;
        for (int turn = 0; turn < kRows; ++turn) {
            if (wave == turn)
                each_sum([&](int at, float& x, float& y) {
                    x = joined[0][at][t] = turn ? joined[0][at][t] + x : x;
                    y = joined[1][at][t] = turn ? joined[1][at][t] + y : y;
                });
            __syncthreads();
        }
        if (wave != kRows - 1) return;
    }
    float* p = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.n;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int q = 0; q < kEach; ++q)
            if (row.has(c)) {
                p[row.at(c) + q] = dw[c][q];
                p[a.n + row.at(c) + q] = db[c][q];
            }
    if (row.tail()) {
        p[row.last] = edw;
        p[a.n + row.last] = edb;
    }
}

// dx of a row that registers do not hold; as norm_forward_long_kernel.
template <typename T>
__global__ __launch_bounds__(kLongBlock) void norm_backward_long_kernel(BackwardArgs a) {
    __shared__ float s[2][2][kLongWaves];
    const float n = static_cast<float>(a.n);
    int turn = 0;
    for (int64_t i = blockIdx.x; i < a.m; i += gridDim.x, turn ^= 1) {
        const float mean = a.rms ? 0.0f : a.mean[i], rstd = a.rstd[i];
        const T* const rows[3] = {static_cast<const T*>(a.x) + i * a.ldx, static_cast<const T*>(a.dy) + i * a.lddy,
                                  a.res ? static_cast<const T*>(a.res) + i * a.ldr : nullptr};
        const T* const both[2] = {rows[0], rows[1]};
        T* const dx = static_cast<T*>(a.dx) + i * a.lddx;
        double all[2] = {0.0, 0.0};
        over_row(both, a.n, [&](int64_t j, const auto(&v)[2]) {
            constexpr int N = sizeof(v[0].v) / sizeof(float);
            float w[N], part[2] = {0.0f, 0.0f};
            load_params(a.w, a.w_f32, j, 1.0f, w);
#pragma unroll
            for (int q = 0; q < N; ++q) {
                const float g = v[1].v[q] * w[q];
                part[0] += g;
                part[1] = fmaf(g, (v[0].v[q] - mean) * rstd, part[1]);
            }
            all[0] += part[0];
            all[1] += part[1];
        });
        float sum[2] = {static_cast<float>(all[0]), static_cast<float>(all[1])};
        row_sum<kLongWaves>(sum, s[turn]);
        const float m1 = a.rms ? 0.0f : sum[0] / n, m2 = sum[1] / n;
        over_row(rows, a.n, [&](int64_t j, const auto(&v)[3]) {
            auto out = v[0];
            constexpr int N = sizeof(out.v) / sizeof(float);
            float w[N];
            load_params(a.w, a.w_f32, j, 1.0f, w);
#pragma unroll
            for (int q = 0; q < N; ++q) {
                const float xhat = (v[0].v[q] - mean) * rstd, d = rstd * (v[1].v[q] * w[q] - m1 - xhat * m2);
                out.v[q] = a.res ? d + v[2].v[q] : d;
            }
            store_values(dx + j, out);
        });
    }
}

// The column sums alone: 64 chunks of columns by 4 rows at a time, `rows` rows a
// block, into a row of `part` each; with one row block, into the results.  The
// second read of dy and x makes 8192 x 11008 bf16 208 us in all, of which dx 108.
// LONG: a place passes more than kChain rows.
struct Sums {
    void* dw;
    void* db;
    int32_t f32, accumulate;
};
template <typename T, bool LONG>
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
    double chains[LONG ? 2 : 1][LONG ? kEach : 1] = {};
    int added = 0;
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
        if constexpr (LONG) {
            if (++added % kChain != 0) continue;
#pragma unroll
            for (int q = 0; q < kEach; ++q) {
                chains[0][q] += dw[q];
                chains[1][q] += db[q];
                dw[q] = db[q] = 0.0f;
            }
        }
    }
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
        sums[0][place][lane][q] = LONG ? static_cast<float>(chains[0][q] + dw[q]) : dw[q];
        sums[1][place][lane][q] = LONG ? static_cast<float>(chains[1][q] + db[q]) : db[q];
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

// Few rows, everything in one launch: the first workgroups take 8 chunks of
// columns each over all rows, 32 at a time, for the column sums; each of the
// others one row, for dx.  Both read dy and x, which are small.
constexpr int kFewChunks = 4;  // a lane
template <typename T>
__global__ __launch_bounds__(256) void norm_backward_few_kernel(BackwardArgs a, Sums out, int32_t cblocks) {
    constexpr int kEach = 16 / sizeof(T);
    __shared__ float sums[2][32][8 * kEach + 1], row_sums[2][4];
    const int tid = threadIdx.x;
    if (static_cast<int>(blockIdx.x) < cblocks) {
        const int lane = tid & 7, place = tid >> 3;
        const int64_t j0 = static_cast<int64_t>(blockIdx.x) * (8 * kEach), j = j0 + lane * kEach;
        const int cnt = static_cast<int>(max(static_cast<int64_t>(0), min(a.n - j, static_cast<int64_t>(kEach))));
        const int back = chunk_back<T>(cnt, a.n);
        float dw[kEach], db[kEach];
#pragma unroll
        for (int q = 0; q < kEach; ++q) dw[q] = db[q] = 0.0f;
        const int64_t end = cnt > 0 ? a.m : 0;
#pragma unroll 4
        for (int64_t i = place; i < end; i += 32) {
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
            sums[0][place][lane * kEach + q] = dw[q];
            sums[1][place][lane * kEach + q] = db[q];
        }
        __syncthreads();
        const int which = tid / (8 * kEach), at = tid % (8 * kEach);
        void* const to = which == 0 ? out.dw : which == 1 ? out.db : nullptr;
        if (!to || j0 + at >= a.n) return;
        float v[32];
#pragma unroll
        for (int p = 0; p < 32; ++p) v[p] = sums[which][p][at];
        put_sum(to, out.f32, out.accumulate, j0 + at, sum_halves(v));
        return;
    }
    dx_row<T, 4, kFewChunks, true>(a, static_cast<int64_t>(blockIdx.x) - cblocks, tid, row_sums);
}

// dw and db from `rows` rows of sums: 32 columns a block, 32 threads a column.
// 512 rows of 8192 columns: 4.8 us.
constexpr int kSumBlock = 1024, kSumColumns = 32;
__global__ __launch_bounds__(kSumBlock) void norm_sum_kernel(const float* part, int64_t n, int64_t rows, Sums out) {
    __shared__ float sums[kSumBlock / kSumColumns][kSumColumns + 1];
    const int c = threadIdx.x % kSumColumns, q = threadIdx.x / kSumColumns;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * kSumColumns + c;
    float s = 0;
    if (col < 2 * n) {
#pragma unroll 8
        for (int64_t r = q; r < rows; r += kSumBlock / kSumColumns) s += part[r * 2 * n + col];
    }
    sums[q][c] = s;
    __syncthreads();
    if (q != 0 || col >= 2 * n) return;
    float v[kSumBlock / kSumColumns];
#pragma unroll
    for (int r = 0; r < kSumBlock / kSumColumns; ++r) v[r] = sums[r][c];
    void* const to = col < n ? out.dw : out.db;
    if (to) put_sum(to, out.f32, out.accumulate, col < n ? col : col - n, sum_halves(v));
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

// A row by itself: by its length alone, so that its result is the same among any
// other rows.  8192 bf16 rows of 2048 13.5 to 14.5 us by one wave, by four 19.8;
// fp32 rows of 11007 140 by 16 waves of 4 chunks, as by 8 of 8.
Division row_division(int64_t n, int elem) {
    const int64_t chunks = ceil_div(n, 16 / elem);
    for (const Division d : {Division{1, 1}, {1, 2}, {1, 4}, {4, 2}, {4, 4}, {8, 4}, {16, 4}})
        if (chunks <= int64_t(64) * d.waves * d.chunks) return d;
    return {0, 0};
}

// With column sums, which are held as well, and the next row.  8192 x 8192 bf16
// with a residual: 110 us by 16 waves of one chunk, by 4 of 4 151.
Division sums_division(int64_t n, int elem) {
    const int64_t chunks = ceil_div(n, 16 / elem);
    for (const Division d : {Division{1, 1}, {1, 2}, {4, 1}, {8, 1}, {16, 1}})
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
    const Division d = row_division(a.n, sizeof(T));
    auto run = [&](auto waves, auto chunks) {
        constexpr int W = decltype(waves)::value, C = decltype(chunks)::value;
        const int64_t blocks = std::min<int64_t>(W == 1 ? ceil_div(a.m, 4) : a.m, kMaxBlocks);
        const dim3 grid(static_cast<uint32_t>(blocks)), block(W == 1 ? 256 : W * 64);
        if (a.n % (16 / sizeof(T)) == 0) norm_forward_kernel<T, W, C, false><<<grid, block, 0, stream>>>(a);
        else norm_forward_kernel<T, W, C, true><<<grid, block, 0, stream>>>(a);
    };
    if (with<1, 1>(d, run) || with<1, 2>(d, run) || with<1, 4>(d, run) || with<4, 2>(d, run) || with<4, 4>(d, run) ||
        with<8, 4>(d, run) || with<16, 4>(d, run))
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
    a.eps = eps;
    a.w_f32 = we == 4;
    a.rms = kind == FSDP_NORM_RMS;
    a.wt = stream_ok(y, ldy, e);
    if (e == 2) launch_forward<uint16_t>(a, stream);
    else launch_forward<float>(a, stream);
    return launched(who);
}

// Rows up to which the column sums are taken beside dx in one launch.  In one
// launch and in two, with a residual, us:
//   rows              400          600          820         1024
//   bf16, 1024      9, 12.7     14, 12.7   20.3, 12.8   25.3, 12.6
//   bf16, 2048   11.3, 15.1   17.3, 15.9   22.6, 16.3   26.8, 16.9
//   bf16, 4096   13.0, 22.4   18.6, 26.1   25.0, 28.0   30.0, 28.5
//   bf16, 8192   15.0, 24.6   21.0, 27.9   27.5, 30.8   32.2, 32.2
//   fp32, 1024   10.6, 11.9   15.9, 12.3   21.0, 12.2   25.1, 12.4
//   fp32, 2048   12.2, 13.0   17.5, 14.5   23.4, 16.0   28.2, 16.3
//   fp32, 4096   14.2, 15.3   19.5, 18.3   26.2, 21.4   32.2, 22.3
// so the bound is right for wide bf16 rows; others cross between 400 and 600 rows.
// 333 x 1365 fp32: 10.2 and 11.4.
constexpr int64_t kFewRows = 1024;

template <typename T>
int32_t launch_backward(BackwardArgs a, const Sums& out, float* workspace, int64_t bytes, hipStream_t stream,
                        const char* who) {
    constexpr int64_t kEach = 16 / sizeof(T);
    const bool sums = out.dw || out.db, whole = a.n % kEach == 0;
    if (sums && a.m <= kFewRows && a.n <= 256 * kFewChunks * kEach) {
        const int64_t cblocks = ceil_div(a.n, 8 * kEach);
        norm_backward_few_kernel<T><<<dim3(static_cast<uint32_t>(cblocks + (a.dx ? a.m : 0))), dim3(256), 0, stream>>>(
            a, out, static_cast<int32_t>(cblocks));
        return launched(who);
    }
    const int64_t room = std::min(bytes, FSDP_NORM_WORKSPACE_BYTES) / (8 * a.n);  // rows of sums
    auto join = [&](int64_t rows) {
        norm_sum_kernel<<<dim3(static_cast<uint32_t>(ceil_div(2 * a.n, kSumColumns))), dim3(kSumBlock), 0, stream>>>(
            workspace, a.n, rows, out);
        return launched(who);
    };
    const Division d = sums_division(a.n, sizeof(T));
    // with room for fewer parts than a quarter of the chip the sums are taken apart
    if (sums && a.dx && d.waves > 0 && room >= kCus / 4) {
        // as many as a CU holds at a time; of four waves, two, or three for many rows
        // (30000 x 2048 bf16 101 us by two, 91 by three; 8192 x 2001 59 and 52; 2000 x 2048
        // 18 and 22)
        const int64_t per_cu = d.waves > 8 || d.chunks > 1 ? 1 : d.waves == 4 && a.m >= 32 * kCus ? 3 : 2;
        const int64_t blocks = std::min(std::min<int64_t>(ceil_div(a.m, backward_rows(d.waves)), per_cu * kCus), room);
        a.part = workspace;
        auto run = [&](auto waves, auto chunks) {
            constexpr int W = decltype(waves)::value, C = decltype(chunks)::value;
            const dim3 grid(static_cast<uint32_t>(blocks)), block(backward_rows(W) * W * 64);
            const bool chains = a.m > kChain * backward_rows(W) * blocks;
            if (whole && !chains) norm_backward_kernel<T, W, C, false, false><<<grid, block, 0, stream>>>(a);
            else if (whole) norm_backward_kernel<T, W, C, false, true><<<grid, block, 0, stream>>>(a);
            else if (!chains) norm_backward_kernel<T, W, C, true, false><<<grid, block, 0, stream>>>(a);
            else norm_backward_kernel<T, W, C, true, true><<<grid, block, 0, stream>>>(a);
        };
        with<1, 1>(d, run) || with<1, 2>(d, run) || with<4, 1>(d, run) || with<8, 1>(d, run) || with<16, 1>(d, run);
        TRY(launched(who));
        return join(blocks);
    }
    if (a.dx) {
        const Division r = row_division(a.n, sizeof(T));
        auto run = [&](auto waves, auto chunks) {
            constexpr int W = decltype(waves)::value, C = decltype(chunks)::value;
            const int64_t blocks = std::min<int64_t>(W == 1 ? ceil_div(a.m, 4) : a.m, kMaxBlocks);
            const dim3 grid(static_cast<uint32_t>(blocks)), block(W == 1 ? 256 : W * 64);
            if (whole) norm_dx_kernel<T, W, C, false><<<grid, block, 0, stream>>>(a);
            else norm_dx_kernel<T, W, C, true><<<grid, block, 0, stream>>>(a);
        };
        if (!(with<1, 1>(r, run) || with<1, 2>(r, run) || with<1, 4>(r, run) || with<4, 2>(r, run) || with<4, 4>(r, run) ||
              with<8, 4>(r, run) || with<16, 4>(r, run))) {
            const uint32_t blocks = static_cast<uint32_t>(std::min<int64_t>(a.m, 2 * kCus));
            norm_backward_long_kernel<T><<<dim3(blocks), dim3(kLongBlock), 0, stream>>>(a);
        }
        TRY(launched(who));
    }
    if (!sums) return FSDP_OK;
    const int64_t cblocks = ceil_div(a.n, 64 * kEach);
    const int64_t want = std::max<int64_t>(1, std::min(8 * kCus / cblocks, room));
    const int64_t rows = ceil_div(ceil_div(a.m, 4), want) * 4, rblocks = ceil_div(a.m, rows);
    a.part = rblocks > 1 ? workspace : nullptr;
    const dim3 grid(static_cast<uint32_t>(cblocks * rblocks));
    if (rows > 4 * kChain) norm_columns_kernel<T, true><<<grid, dim3(256), 0, stream>>>(a, out, static_cast<int32_t>(cblocks), rows);
    else norm_columns_kernel<T, false><<<grid, dim3(256), 0, stream>>>(a, out, static_cast<int32_t>(cblocks), rows);
    TRY(launched(who));
    return rblocks == 1 ? FSDP_OK : join(rblocks);
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
