// Microscaled 4-bit copies of matrices (gfx950 / MI355X): quantisation, of a
// matrix and of its transpose, and the values read back.  The format and the
// rounding are stated in include/fsdp_mx4.h.
//
// The scale of a block is a power of two, so the hardware's conversion, which
// takes the scale from a float's exponent bits alone (0 for 2^-127), divides
// exactly and rounds once, to nearest, ties to the even code, and saturates.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "fsdp_mx4.h"
#include "internal.h"
#include "linear_plan.h"
#include "mx4_plan.h"
#include "stream_device.h"

using fsdp::fail;

namespace {

using namespace fsdp::linear;

constexpr uint32_t kInfBits = 0x7f800000u;

// The scale byte of a block from the bits of its largest magnitude (of an
// infinity or a NaN, the largest bits there are).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    if (amax_bits >= kInfBits) return 255;
    const int e = static_cast<int>(amax_bits >> 23) - 2;
    return static_cast<uint32_t>(max(e, 0));
}

// Eight elements' codes; of a block of scale 255, zeros.
__device__ __forceinline__ uint32_t encode8(const float (&v)[8], uint32_t scale) {
    if (scale == 255) return 0;
    const float s = __uint_as_float(scale << 23);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
}

// ---------------------------------------------------------------- blocks along rows

struct RowsArgs {
    uint8_t* codes;
    uint8_t* scales;
    const void* x;
    int64_t ldc, lds, ldx, rows, cols;
    Grid g;
};

// Eight elements a lane, four lanes a block.
template <typename T>
__global__ __launch_bounds__(kElemBlock) void quantize_rows_kernel(RowsArgs a) {
    const int tid = threadIdx.x, per = kElemBlock >> a.g.tx;
    const int64_t rb = blockIdx.x / a.g.cblocks;
    const int64_t c = (static_cast<int64_t>(blockIdx.x % a.g.cblocks) << a.g.tx) + (tid & ((1 << a.g.tx) - 1));
    const int64_t block = c >> 2, blocks = (a.cols + 31) / 32, padded = (blocks + 15) / 16 * 16;
    if (block >= padded) return;
    const int64_t end = min(a.rows, (rb + 1) * a.g.rows);
    const int cnt = static_cast<int>(max(static_cast<int64_t>(0), min(a.cols - c * 8, static_cast<int64_t>(8))));
    for (int64_t i = rb * a.g.rows + (tid >> a.g.tx); i < end; i += per) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = 0.0f;
        if (cnt > 0) load8(static_cast<const T*>(a.x) + i * a.ldx + c * 8, cnt, v);
        uint32_t top = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) top = max(top, __float_as_uint(v[q]) & 0x7fffffffu);
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 1)));
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 2)));
        const uint32_t scale = scale_byte(top);
        if (block < blocks) *reinterpret_cast<uint32_t*>(a.codes + i * a.ldc + c * 4) = encode8(v, scale);
        if ((c & 3) == 0) a.scales[i * a.lds + block] = static_cast<uint8_t>(scale);
    }
}

// ---------------------------------------------------------------- blocks along columns

// One column's 32 rows a thread.
template <typename T>
__global__ __launch_bounds__(kElemBlock) void quantize_columns_kernel(RowsArgs a, int64_t cblocks) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t blocks = (a.rows + 31) / 32, padded = (blocks + 15) / 16 * 16;
    const int64_t j = static_cast<int64_t>(blockIdx.x % cblocks) * 64 + lane;
    const int64_t block = static_cast<int64_t>(blockIdx.x / cblocks) * 4 + wave;
    if (j >= a.cols || block >= padded) return;
    if (block >= blocks) {
        a.scales[j * a.lds + block] = 0;
        return;
    }
    float v[4][8];
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
        const int64_t i = block * 32 + r;
        float x = 0.0f;
        if (i < a.rows) {
            if constexpr (sizeof(T) == 2) x = widen(static_cast<const T*>(a.x)[i * a.ldx + j]);
            else x = static_cast<const T*>(a.x)[i * a.ldx + j];
        }
        v[r / 8][r % 8] = x;
        top = max(top, __float_as_uint(x) & 0x7fffffffu);
    }
    const uint32_t scale = scale_byte(top);
    *reinterpret_cast<u32x4*>(a.codes + j * a.ldc + block * 16) =
        u32x4{encode8(v[0], scale), encode8(v[1], scale), encode8(v[2], scale), encode8(v[3], scale)};
    a.scales[j * a.lds + block] = static_cast<uint8_t>(scale);
}

// ---------------------------------------------------------------- values

struct ValuesArgs {
    void* y;
    const uint8_t* codes;
    const uint8_t* scales;
    int64_t ldy, ldc, lds, rows, cols;
    Grid g;
    int32_t wt;
};

// 16 bytes of values a lane.
template <typename T>
__global__ __launch_bounds__(kElemBlock) void dequantize_kernel(ValuesArgs a) {
    constexpr int kEach = 16 / sizeof(T);
    const int tid = threadIdx.x, per = kElemBlock >> a.g.tx;
    const int64_t rb = blockIdx.x / a.g.cblocks;
    const int64_t j = ((static_cast<int64_t>(blockIdx.x % a.g.cblocks) << a.g.tx) + (tid & ((1 << a.g.tx) - 1))) * kEach;
    if (j >= a.cols) return;
    const int cnt = static_cast<int>(min(a.cols - j, static_cast<int64_t>(kEach)));
    const int64_t end = min(a.rows, (rb + 1) * a.g.rows);
    for (int64_t i = rb * a.g.rows + (tid >> a.g.tx); i < end; i += per) {
        const uint8_t* const p = a.codes + i * a.ldc + j / 2;
        const float s = __uint_as_float(static_cast<uint32_t>(a.scales[i * a.lds + j / 32]) << 23);
        const uint32_t c = kEach == 8 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
        float v[kEach];
        auto pair = [&](int q, auto which) {
            typedef float f32x2 __attribute__((ext_vector_type(2)));
            const f32x2 f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, decltype(which)::value);
            v[2 * q] = f[0];
            v[2 * q + 1] = f[1];
        };
        pair(0, std::integral_constant<int, 0>());
        pair(1, std::integral_constant<int, 1>());
        if constexpr (kEach == 8) {
            pair(2, std::integral_constant<int, 2>());
            pair(3, std::integral_constant<int, 3>());
        }
        stream_store(static_cast<T*>(a.y) + i * a.ldy + j, cnt, a.wt, v);
    }
}

// ---------------------------------------------------------------- host

int32_t quantize_impl(uint8_t* codes, int64_t ldc, uint8_t* scales, int64_t lds, uint8_t* codes_t, int64_t ldct,
                      uint8_t* scales_t, int64_t ldst, const void* x, int64_t ldx, int32_t x_dtype, int64_t rows,
                      int64_t cols, hipStream_t stream) {
    const char* who = "fsdp_mx4_quantize";
    TRY(check_sizes(rows, cols, 0, who));
    TRY(check_float_dtype(x_dtype, "x", who));
    const int e = x_dtype == FSDP_DT_BF16 ? 2 : 4;
    const Matrix mx{x, rows, cols, ldx, e, "x", false};
    const Mx4Matrix q = mx4_matrix(codes, ldc, "codes", scales, lds, "scales", rows, cols, true);
    const Mx4Matrix t = mx4_matrix(codes_t, ldct, "codes_t", scales_t, ldst, "scales_t", cols, rows, true);
    TRY(check_matrix(mx, false, who));
    if (!codes != !scales || !codes_t != !scales_t) return fail(FSDP_E_ARG, "%s: codes without scales, or scales without codes", who);
    if (codes) TRY(check_mx4(q, who));
    if (codes_t) TRY(check_mx4(t, who));
    TRY(check_overlaps({q.codes, q.scales, t.codes, t.scales, mx}, who, [](const Matrix&, const Matrix&) { return false; }));
    if (rows == 0 || cols == 0) return FSDP_OK;
    if (!codes && !codes_t) return fail(FSDP_E_ARG, "%s: null codes and codes_t", who);
    RowsArgs r{codes, scales, x, ldc, lds, ldx, rows, cols, {}};
    int64_t blocks;
    r.g = elementwise_grid(rows, FSDP_MX4_SCALE_BYTES(cols) * 4, 16 * kCus / ceil_div(FSDP_MX4_SCALE_BYTES(cols) * 4, 64), &blocks);
    blocks *= r.g.cblocks;
    RowsArgs c{codes_t, scales_t, x, ldct, ldst, ldx, rows, cols, {}};
    const int64_t cblocks = ceil_div(cols, 64), columns = cblocks * (FSDP_MX4_SCALE_BYTES(rows) / 4);
    if ((codes && blocks > kMaxBlocks) || (codes_t && columns > kMaxBlocks))
        return fail(FSDP_E_CAPACITY, "%s: more blocks than one launch holds", who);
    if (codes) {
        const dim3 grid(static_cast<uint32_t>(blocks));
        if (e == 2) quantize_rows_kernel<uint16_t><<<grid, dim3(kElemBlock), 0, stream>>>(r);
        else quantize_rows_kernel<float><<<grid, dim3(kElemBlock), 0, stream>>>(r);
        TRY(launched(who));
    }
    if (codes_t) {
        const dim3 grid(static_cast<uint32_t>(columns));
        if (e == 2) quantize_columns_kernel<uint16_t><<<grid, dim3(kElemBlock), 0, stream>>>(c, cblocks);
        else quantize_columns_kernel<float><<<grid, dim3(kElemBlock), 0, stream>>>(c, cblocks);
        TRY(launched(who));
    }
    return FSDP_OK;
}

int32_t dequantize_impl(void* y, int64_t ldy, int32_t y_dtype, const uint8_t* codes, int64_t ldc, const uint8_t* scales,
                        int64_t lds, int64_t rows, int64_t cols, hipStream_t stream) {
    const char* who = "fsdp_mx4_dequantize";
    TRY(check_sizes(rows, cols, 0, who));
    TRY(check_float_dtype(y_dtype, "y", who));
    const int e = y_dtype == FSDP_DT_BF16 ? 2 : 4;
    const Matrix my{y, rows, cols, ldy, e, "y", true};
    const Mx4Matrix q = mx4_matrix(codes, ldc, "codes", scales, lds, "scales", rows, cols, false);
    TRY(check_matrix(my, false, who));
    TRY(check_mx4(q, who));
    TRY(check_overlaps({my, q.codes, q.scales}, who, [](const Matrix&, const Matrix&) { return false; }));
    if (rows == 0 || cols == 0) return FSDP_OK;
    ValuesArgs a{y, codes, scales, ldy, ldc, lds, rows, cols, {}, stream_ok(y, ldy, e)};
    const int64_t chunks = ceil_div(cols, 16 / e);
    int64_t blocks;
    a.g = elementwise_grid(rows, chunks, 16 * kCus / ceil_div(chunks, 64), &blocks);
    if (blocks * a.g.cblocks > kMaxBlocks) return fail(FSDP_E_CAPACITY, "%s: more blocks than one launch holds", who);
    const dim3 grid(static_cast<uint32_t>(blocks * a.g.cblocks));
    if (e == 2) dequantize_kernel<uint16_t><<<grid, dim3(kElemBlock), 0, stream>>>(a);
    else dequantize_kernel<float><<<grid, dim3(kElemBlock), 0, stream>>>(a);
    return launched(who);
}

}  // namespace

// ---------------------------------------------------------------- entry points

extern "C" int32_t fsdp_mx4_quantize(uint8_t* codes, int64_t ldc, uint8_t* scales, int64_t lds, uint8_t* codes_t,
                                     int64_t ldct, uint8_t* scales_t, int64_t ldst, const void* x, int64_t ldx,
                                     int32_t x_dtype, int64_t rows, int64_t cols, hipStream_t stream) {
    return fsdp::guarded("fsdp_mx4_quantize", [&] {
        return quantize_impl(codes, ldc, scales, lds, codes_t, ldct, scales_t, ldst, x, ldx, x_dtype, rows, cols, stream);
    });
}

extern "C" int32_t fsdp_mx4_dequantize(void* y, int64_t ldy, int32_t y_dtype, const uint8_t* codes, int64_t ldc,
                                       const uint8_t* scales, int64_t lds, int64_t rows, int64_t cols,
                                       hipStream_t stream) {
    return fsdp::guarded("fsdp_mx4_dequantize",
                         [&] { return dequantize_impl(y, ldy, y_dtype, codes, ldc, scales, lds, rows, cols, stream); });
}
