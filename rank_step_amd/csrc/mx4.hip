// Microscaled 4-bit copies of matrices (gfx950 / MI355X): quantisation, of a
// matrix and of its transpose, and the values read back.  The format and the
// rounding are stated in include/fsdp_mx4.h.
//
// The scale of a block is a power of two, so the hardware's conversion, which
// takes the scale from a float's exponent bits alone (0 for 2^-127), divides
// exactly and rounds once, to nearest, ties to the even code, and saturates.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

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

// Eight elements a lane, four lanes a block.  Bound by memory: 8192 x 4096 bf16 13.9
// us (6.1 TB/s), fp32 23.
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

// ---------------------------------------------------------------- blocks along columns, and both

// Eight waves take 256 rows of 128 columns, each wave 32 rows, a lane two
// columns of them: 32 loads on their way, 256 bytes of a row (bf16) each.  A
// column's block is a lane's own; a row's block is 16 lanes', whose largest
// magnitude four DPP steps find.  So x is read once for both copies, from registers.
// The codes of a column's eight blocks are a line, which goes through LDS to be
// stored as one; a row's go out as words, after the four lanes of a quad have
// exchanged bytes of four rows.  8192 x 4096 bf16 26 us (3.9 TB/s; floor 16);
// with 16 bytes of a column stored by each lane 30, by a launch for each copy 48.
// What is left is the vector unit beside memory: about 12 operations an element.
// Workgroups that stay and fetch their next tile meanwhile: 6 to 15 % slower; four
// waves: 2 to 5 %; ordinary loads: 13 %.
struct TileArgs {
    uint8_t* codes;    // blocks along rows, or null
    uint8_t* scales;
    uint8_t* codes_t;  // along columns
    uint8_t* scales_t;
    const void* x;
    int64_t ldc, lds, ldct, ldst, ldx, rows, cols;
    int64_t ctiles, tiles;
};

// Two columns of a row: their bits, and their codes as byte WHICH of w.
template <typename T>
struct Two;
template <>
struct Two<uint16_t> {
    uint32_t v;  // bf16 in each half
    __device__ __forceinline__ void load(const uint16_t* p, int cnt) {
        typedef uint32_t word __attribute__((aligned(2)));
        v = cnt >= 2 ? __builtin_nontemporal_load(reinterpret_cast<const word*>(p)) : static_cast<uint32_t>(*p);
    }
    __device__ __forceinline__ uint32_t low() const { return v << 16; }
    __device__ __forceinline__ uint32_t high() const { return v & 0xffff0000u; }
    template <int WHICH>
    __device__ __forceinline__ uint32_t encode(uint32_t w, float s) const {
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, v), s, WHICH);
    }
    // column c of this row and the next one
    template <int WHICH>
    __device__ __forceinline__ uint32_t encode_down(const Two& next, int c, uint32_t w, float s) const {
        const uint32_t p = c ? __builtin_amdgcn_perm(next.v, v, 0x07060302) : __builtin_amdgcn_perm(next.v, v, 0x05040100);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, p), s, WHICH);
    }
};
template <>
struct Two<float> {
    float v[2];
    __device__ __forceinline__ void load(const float* p, int cnt) {
        typedef u32x2 pair __attribute__((aligned(4)));
        const u32x2 w = cnt >= 2 ? __builtin_nontemporal_load(reinterpret_cast<const pair*>(p)) : u32x2{__float_as_uint(*p), 0};
        v[0] = __uint_as_float(w[0]);
        v[1] = __uint_as_float(w[1]);
    }
    __device__ __forceinline__ uint32_t low() const { return __float_as_uint(v[0]); }
    __device__ __forceinline__ uint32_t high() const { return __float_as_uint(v[1]); }
    template <int WHICH>
    __device__ __forceinline__ uint32_t encode(uint32_t w, float s) const {
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, WHICH);
    }
    template <int WHICH>
    __device__ __forceinline__ uint32_t encode_down(const Two& next, int c, uint32_t w, float s) const {
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[c], next.v[c], s, WHICH);
    }
};

__device__ __forceinline__ uint32_t magnitude(uint32_t bits) { return bits & 0x7fffffffu; }

// The largest over the 16 lanes of a row's block, in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    auto step = [](uint32_t x, auto ctrl) {
        return max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), decltype(ctrl)::value, 0xf, 0xf, true)));
    };
    v = step(v, std::integral_constant<int, 0xB1>());   // quad_perm 1 0 3 2
    v = step(v, std::integral_constant<int, 0x4E>());   // quad_perm 2 3 0 1
    v = step(v, std::integral_constant<int, 0x141>());  // row_half_mirror
    return step(v, std::integral_constant<int, 0x140>());  // row_mirror
}

// Lane l of a quad gets byte l of each of its four lanes' words, in their order.
__device__ __forceinline__ uint32_t transpose_quad(uint32_t w, uint32_t pick) {
    auto from = [&](auto ctrl) {
        return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(w), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    const uint32_t w0 = from(std::integral_constant<int, 0x00>()), w1 = from(std::integral_constant<int, 0x55>());
    const uint32_t w2 = from(std::integral_constant<int, 0xAA>()), w3 = from(std::integral_constant<int, 0xFF>());
    // pick: byte l of the first operand (7..4) and of the second (3..0)
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(w3, w2, pick), __builtin_amdgcn_perm(w1, w0, pick), 0x05040100);
}

constexpr int kTileBlock = 512;
template <typename T, bool ROWS>
__global__ __launch_bounds__(kTileBlock) void quantize_tile_kernel(TileArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // neighbouring tiles of a row of tiles on one XCD, whose L2 joins their halves of lines
    const int64_t per = (a.tiles + kXcds - 1) / kXcds;
    const int64_t tile = static_cast<int64_t>(blockIdx.x % kXcds) * per + blockIdx.x / kXcds;
    if (tile >= a.tiles) return;
    const int64_t ct = tile % a.ctiles, block = tile / a.ctiles * 8 + wave, r0 = block * 32, j = ct * 128 + lane * 2;
    const int64_t blocks = (a.cols + 31) / 32, blocks_t = (a.rows + 31) / 32;
    __shared__ u32x4 line[128][8];  // a column's codes of the eight waves' blocks
    __shared__ __attribute__((aligned(8))) uint8_t bytes[128][8];
    const T* const x = static_cast<const T*>(a.x) + r0 * a.ldx + j;
    Two<T> v[32];
    if (r0 + 32 <= a.rows && ct * 128 + 128 <= a.cols) {
#pragma unroll
        for (int r = 0; r < 32; ++r) v[r].load(x + r * a.ldx, 2);
    } else {
        const int cnt = static_cast<int>(max(static_cast<int64_t>(0), min(a.cols - j, static_cast<int64_t>(2))));
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            v[r] = Two<T>{};
            if (r0 + r < a.rows && cnt > 0) v[r].load(x + r * a.ldx, cnt);
        }
    }
    {
        uint32_t top[2] = {0, 0};
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            top[0] = max(top[0], magnitude(v[r].low()));
            top[1] = max(top[1], magnitude(v[r].high()));
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t scale = scale_byte(top[c]);
            const float s = __uint_as_float(scale << 23);
            u32x4 w = {0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                w[q] = v[q * 8].template encode_down<0>(v[q * 8 + 1], c, w[q], s);
                w[q] = v[q * 8 + 2].template encode_down<1>(v[q * 8 + 3], c, w[q], s);
                w[q] = v[q * 8 + 4].template encode_down<2>(v[q * 8 + 5], c, w[q], s);
                w[q] = v[q * 8 + 6].template encode_down<3>(v[q * 8 + 7], c, w[q], s);
            }
            if (scale == 255) w = u32x4{0, 0, 0, 0};
            line[lane * 2 + c][wave ^ (lane & 7)] = w;
            bytes[lane * 2 + c][wave] = static_cast<uint8_t>(scale);
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int id = k * kTileBlock + threadIdx.x, col = id >> 3, at = id & 7;
        const int64_t to = tile / a.ctiles * 8 + at;
        if (ct * 128 + col < a.cols && to < blocks_t)
            *reinterpret_cast<u32x4*>(a.codes_t + (ct * 128 + col) * a.ldct + to * 16) = line[col][at ^ (col >> 1 & 7)];
    }
    if (threadIdx.x < 128 && ct * 128 + threadIdx.x < a.cols)
        *reinterpret_cast<u32x2*>(a.scales_t + (ct * 128 + threadIdx.x) * a.ldst + tile / a.ctiles * 8) =
            *reinterpret_cast<const u32x2*>(bytes[threadIdx.x]);
    if constexpr (ROWS) {
        const int in = lane & 15;
        const int64_t row_block = ct * 4 + (lane >> 4);
        const uint32_t pick = 0x01010101u * (lane & 3) + 0x00000400u;  // bytes l and 4 + l
        uint32_t kept[2] = {0, 0};                                     // the scales of rows `in` and 16 + in
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            uint32_t w = 0;
            auto encode = [&](auto which) {
                constexpr int k = decltype(which)::value;
                const int r = g * 4 + k;
                const uint32_t scale = scale_byte(max16(max(magnitude(v[r].low()), magnitude(v[r].high()))));
                const bool finite = scale != 255;
                w = (finite ? v[r] : Two<T>{}).template encode<k>(w, __uint_as_float(finite ? scale << 23 : 0x3f800000u));
                if (in == (r & 15)) kept[r >> 4] = scale;
            };
            encode(std::integral_constant<int, 0>());
            encode(std::integral_constant<int, 1>());
            encode(std::integral_constant<int, 2>());
            encode(std::integral_constant<int, 3>());
            const uint32_t t = transpose_quad(w, pick);
            const int64_t row = r0 + g * 4 + (lane & 3);
            if (row < a.rows && row_block < blocks)
                *reinterpret_cast<uint32_t*>(a.codes + row * a.ldc + ct * 64 + (lane >> 2) * 4) = t;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = r0 + h * 16 + in;
            if (row < a.rows && row_block < (blocks + 15) / 16 * 16)
                a.scales[row * a.lds + row_block] = static_cast<uint8_t>(kept[h]);
        }
    }
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

// 16 bytes of values a lane, of four rows whose codes are on their way together
// (of one at a time 18.5 us for 8192 x 4096 as bf16, this way 16.2, 5.2 TB/s; of
// eight no faster).  Bound by the stores.
template <typename T>
__global__ __launch_bounds__(kElemBlock) void dequantize_kernel(ValuesArgs a) {
    constexpr int kEach = 16 / sizeof(T), kRows = 4;
    const int tid = threadIdx.x, per = kElemBlock >> a.g.tx;
    const int64_t rb = blockIdx.x / a.g.cblocks;
    const int64_t j = ((static_cast<int64_t>(blockIdx.x % a.g.cblocks) << a.g.tx) + (tid & ((1 << a.g.tx) - 1))) * kEach;
    if (j >= a.cols) return;
    const int cnt = static_cast<int>(min(a.cols - j, static_cast<int64_t>(kEach)));
    const int64_t end = min(a.rows, (rb + 1) * a.g.rows);
    for (int64_t i = rb * a.g.rows + (tid >> a.g.tx); i < end; i += kRows * per) {
        uint32_t c[kRows], s[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            c[r] = s[r] = 0;
            if (i + r * per >= end) continue;
            const uint8_t* const p = a.codes + (i + r * per) * a.ldc + j / 2;
            c[r] = kEach == 8 ? __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p))
                              : static_cast<uint32_t>(__builtin_nontemporal_load(reinterpret_cast<const uint16_t*>(p)));
            s[r] = a.scales[(i + r * per) * a.lds + j / 32];
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (i + r * per >= end) continue;
            const float scale = __uint_as_float(s[r] << 23);
            float v[kEach];
            auto pair = [&](auto which) {
                typedef float f32x2 __attribute__((ext_vector_type(2)));
                constexpr int q = decltype(which)::value;
                const f32x2 f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[r], scale, q);
                v[2 * q] = f[0];
                v[2 * q + 1] = f[1];
            };
            pair(std::integral_constant<int, 0>());
            pair(std::integral_constant<int, 1>());
            if constexpr (kEach == 8) {
                pair(std::integral_constant<int, 2>());
                pair(std::integral_constant<int, 3>());
            }
            stream_store(static_cast<T*>(a.y) + (i + r * per) * a.ldy + j, cnt, a.wt, v);
        }
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
    if (!codes_t) {
        RowsArgs r{codes, scales, x, ldc, lds, ldx, rows, cols, {}};
        const int64_t chunks = FSDP_MX4_SCALE_BYTES(cols) * 4;
        int64_t blocks;
        r.g = elementwise_grid(rows, chunks, 16 * kCus / ceil_div(chunks, 64), &blocks);
        blocks *= r.g.cblocks;
        if (blocks > kMaxBlocks) return fail(FSDP_E_CAPACITY, "%s: more blocks than one launch holds", who);
        const dim3 grid(static_cast<uint32_t>(blocks));
        if (e == 2) quantize_rows_kernel<uint16_t><<<grid, dim3(kElemBlock), 0, stream>>>(r);
        else quantize_rows_kernel<float><<<grid, dim3(kElemBlock), 0, stream>>>(r);
        return launched(who);
    }
    // tiles to the end of the scale rows' padding
    TileArgs a{codes, scales, codes_t, scales_t, x, ldc, lds, ldct, ldst, ldx, rows, cols, 0, 0};
    a.ctiles = codes ? FSDP_MX4_SCALE_BYTES(cols) / 4 : ceil_div(cols, 128);
    a.tiles = a.ctiles * (FSDP_MX4_SCALE_BYTES(rows) / 8);
    const int64_t blocks = round_up(a.tiles, kXcds);
    if (blocks > kMaxBlocks) return fail(FSDP_E_CAPACITY, "%s: more blocks than one launch holds", who);
    const dim3 grid(static_cast<uint32_t>(blocks)), block(kTileBlock);
    if (e == 2 && codes) quantize_tile_kernel<uint16_t, true><<<grid, block, 0, stream>>>(a);
    else if (e == 2) quantize_tile_kernel<uint16_t, false><<<grid, block, 0, stream>>>(a);
    else if (codes) quantize_tile_kernel<float, true><<<grid, block, 0, stream>>>(a);
    else quantize_tile_kernel<float, false><<<grid, block, 0, stream>>>(a);
    return launched(who);
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
