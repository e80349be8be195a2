// What the passes over rows of a matrix share (gfx950): 16-byte accesses of
// rows that may start at any element, streaming loads and written-through
// stores, and the launch check.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"
#include "linear_plan.h"

namespace fsdp {
namespace linear {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

// Vectors that may start at any element: gfx950's global accesses take any
// alignment, so these are still single instructions.
struct __attribute__((packed, aligned(2))) Bytes16 { u32x4 v; };
struct __attribute__((packed, aligned(1))) Bytes8 { uint32_t v[2]; };
typedef u32x4 u32x4_any __attribute__((aligned(2)));  // for non-temporal accesses

// ---------------------------------------------------------------- 8 elements of a row

__device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

__device__ __forceinline__ void unpack8(const u32x4& w, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x2 p = {static_cast<__bf16>(v[2 * i]), static_cast<__bf16>(v[2 * i + 1])};
        w[i] = __builtin_bit_cast(uint32_t, p);
    }
    return w;
}

// The `cnt` (1 to 8) elements at p, zeros in the places behind them.
__device__ __forceinline__ void load8(const uint16_t* p, int cnt, float (&v)[8]) {
    if (cnt >= 8) {
        unpack8(reinterpret_cast<const Bytes16*>(p)->v, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < cnt ? widen(p[i]) : 0.0f;
    }
}

__device__ __forceinline__ void load8(const float* p, int cnt, float (&v)[8]) {
    if (cnt >= 8) {
        const u32x4 a = reinterpret_cast<const Bytes16*>(p)->v, b = reinterpret_cast<const Bytes16*>(p + 4)->v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(a[i]);
            v[4 + i] = __uint_as_float(b[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < cnt ? p[i] : 0.0f;
    }
}

__device__ __forceinline__ void store8(uint16_t* p, int cnt, const float (&v)[8]) {
    if (cnt >= 8) {
        reinterpret_cast<Bytes16*>(p)->v = pack8(v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < cnt) p[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[i]));
    }
}

__device__ __forceinline__ void store8(float* p, int cnt, const float (&v)[8]) {
    if (cnt >= 8) {
        reinterpret_cast<Bytes16*>(p)->v = __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
        reinterpret_cast<Bytes16*>(p + 4)->v = __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]});
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < cnt) p[i] = v[i];
    }
}

// ---------------------------------------------------------------- elementwise passes

// Every value passes once, so loads are non-temporal and stores are written
// through to memory (sc1): a launch then does not end with dirty lines in the
// eight L2s for its release to write back.  8192 x 4096 bf16 with a residual:
// 32.1 us (6.3 TB/s), with ordinary accesses 38.8, with non-temporal ones both
// ways 35.4.
//
// A row's last, shorter chunk is read from as many elements earlier as it lacks
// (`back`) and then moved down, so that it costs one load, as the others: one
// lane that loads its elements one by one holds up its wave, and that wave the
// launch (8192 x 4095 bf16 with a residual 79.5 us, this way 41.6).  Every load
// of a row is issued before the first is moved.  Rows shorter than a chunk
// (back < 0) are loaded element by element.
template <typename T>
__device__ __forceinline__ int chunk_back(int cnt, int64_t n) {
    constexpr int kEach = 16 / sizeof(T);
    return n < kEach ? -1 : kEach - min(cnt, kEach);
}

template <typename T>
__device__ __forceinline__ u32x4 stream_load(const T* p, int cnt, int back) {
    if (back >= 0) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p - back));
    u32x4 w = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) {
        if (i >= cnt) continue;
        if constexpr (sizeof(T) == 2) w[i / 2] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
        else w[i] = __float_as_uint(p[i]);
    }
    return w;
}

// Zeros take the places behind.
__device__ __forceinline__ void arrange(u32x4 w, int back, float (&v)[8]) {
    if (back > 0) {
        if (back & 4) w = u32x4{w[2], w[3], 0, 0};
        if (back & 2) w = u32x4{w[1], w[2], w[3], 0};
        if (back & 1) w = u32x4{w[0] >> 16 | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | w[3] << 16, w[3] >> 16};
    }
    unpack8(w, v);
}

__device__ __forceinline__ void arrange(u32x4 w, int back, float (&v)[4]) {
    if (back > 0) {
        if (back & 2) w = u32x4{w[2], w[3], 0, 0};
        if (back & 1) w = u32x4{w[1], w[2], w[3], 0};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
}

// A written-through 16-byte store.  It is a buffer store (their cache policy
// is an immediate) from a base that the wave shares, its first active lane's
// address: the lanes of a wave go up along a row and then from row to row, so
// that is the lowest, and the others lie within the range when 64 rows do
// (stream_ok).
__device__ __forceinline__ void write_through(void* p, const u32x4& w) {
    constexpr int kSc1 = 16;
    const uintptr_t u = reinterpret_cast<uintptr_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u >> 32));
    const uintptr_t base = (static_cast<uintptr_t>(hi) << 32) | lo;
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), 0, 0x7fffffff, 0x00020000);
    __builtin_amdgcn_raw_buffer_store_b128(w, r, static_cast<int>(u - base), 0, kSc1);
}

// wt: stream_ok for the matrix (the same for the whole launch).
__device__ __forceinline__ void stream_store(uint16_t* p, int cnt, bool wt, const float (&v)[8]) {
    if (wt && cnt >= 8) write_through(p, pack8(v));
    else store8(p, cnt, v);
}

__device__ __forceinline__ void stream_store(float* p, int cnt, bool wt, const float (&v)[4]) {
    const u32x4 w = __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]});
    if (wt && cnt >= 4) {
        write_through(p, w);
    } else if (cnt >= 4) {
        reinterpret_cast<Bytes16*>(p)->v = w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < cnt) p[i] = v[i];
    }
}

// Column j of a vector of sums: s stored, or added to what is there.
__device__ __forceinline__ void put_sum(void* out, int f32, int accumulate, int64_t j, float s) {
    if (f32) {
        float* p = static_cast<float*>(out) + j;
        *p = accumulate ? *p + s : s;
    } else {
        uint16_t* p = static_cast<uint16_t*>(out) + j;
        *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(accumulate ? widen(*p) + s : s));
    }
}

// 2^tx lanes take one row's chunks of 16 bytes (as many as the row has, up
// to a wave), the block's 256 >> tx other places take rows, one at a time: two
// at a time, with twice the loads on their way, were 8 % slower.
constexpr int kElemBlock = 256;
struct Grid {
    int32_t tx, cblocks;  // lanes a row (log2), column blocks
    int64_t rows;         // rows a block takes in all (a multiple of 256 >> tx)
};

// ---------------------------------------------------------------- host

// Whether rows take written-through stores: 16-byte boundaries, and 64 rows
// within the 31 bits of a buffer offset.
inline bool stream_ok(const void* p, int64_t ld, int elem) {
    return aligned(p, 16) && ld * elem % 16 == 0 && ld <= (int64_t(1) << 22);
}

// chunks: 16-byte ones of a row; rows_max: the most row blocks wanted.
inline Grid elementwise_grid(int64_t m, int64_t chunks, int64_t rows_max, int64_t* blocks) {
    Grid g{};
    while (g.tx < 6 && (int64_t(1) << g.tx) < chunks) ++g.tx;
    g.cblocks = static_cast<int32_t>(ceil_div(chunks, int64_t(1) << g.tx));
    const int64_t per = kElemBlock >> g.tx;
    g.rows = std::max<int64_t>(1, ceil_div(ceil_div(m, per), std::max<int64_t>(1, rows_max))) * per;
    *blocks = ceil_div(m, g.rows);
    return g;
}

inline int32_t launched(const char* who) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(FSDP_E_HIP, "%s: launch failed: %s", who, hipGetErrorString(e));
    return FSDP_OK;
}

}  // namespace linear
}  // namespace fsdp
