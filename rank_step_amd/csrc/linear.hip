// The linear layer's kernels and entry points (gfx950 / MI355X): the product
// that reads the all-gathered weight copy, with bias, activation, dropout and
// residual in its epilogue, the gradients of both, and dropout alone.  The
// arithmetic of each call is stated in include/fsdp_linear.h.
//
// Every product is C(i, j) = sum_l A(i, l) B(j, l) for output row i, output
// column j and contraction index l:
//   forward       i = token,  j = output feature, l = input feature: A = x,    B = W
//   input grad    i = token,  j = input feature,  l = output feature: A = dz,  B = W
//   weight grad   i = output feature, j = input feature, l = token:  A = dz,   B = x
// An operand whose rows run along l ("l-major": x, W of the forward product,
// dz of the input gradient) has the 8 consecutive l that one lane of a matrix
// instruction takes in one 16-byte LDS read; one whose rows run along i or j
// (W of the input gradient, both operands of the weight gradient) is read
// through the LDS transpose read (ds_read_b64_tr_b16), so no operand is ever
// transposed in memory.
//
// Floating point: bf16 matrix instructions accumulating in fp32, the epilogue
// in fp32, FMA only where written (built with -ffp-contract=off).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fsdp_linear.h"
#include "internal.h"
#include "linear_plan.h"

using fsdp::fail;

namespace {

using namespace fsdp::linear;

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

// ---------------------------------------------------------------- dropout

struct Mask {
    uint64_t seed, offset;
    const int64_t* offset_dev;
    uint32_t t;      // keep where the 16 bits are at least t; 0: no dropout
    uint32_t above;  // t * 65536 - 1: the same of bits in a word's high half
    float scale;     // 65536 / (65536 - t)
};

// The counter's high half: which mask of the seed's sequence.
__device__ __forceinline__ uint64_t mask_offset(const Mask& m) {
    return m.offset + (m.offset_dev ? static_cast<uint64_t>(*m.offset_dev) : 0);
}

// Philox-4x32-10 (Salmon et al. 2011): ten rounds of two 32x32 -> 64 bit
// products.  One block serves the 8 elements of one 16-byte store: at 16 bits
// an element the generator costs about half of what 32 would, which is what
// lets the elementwise kernels stay on memory's side of the balance.
__device__ __forceinline__ u32x4 philox(uint64_t block, uint64_t offset, uint64_t seed) {
    uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32);
    uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
        const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(p1);
        c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// D with the block's bits.  A dropped element is +0 whatever it held, so this
// selects.
template <int N>
__device__ __forceinline__ void select(float (&v)[N], const Mask& m, const u32x4& w) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        // bits >= t, with the 16 bits in the high half: what is below them cannot
        // lift a word past t * 65536 - 1 unless they are at least t.
        const uint32_t bits = (i & 1) ? w[i / 2] : w[i / 2] << 16;
        v[i] = bits > m.above ? v[i] * m.scale : 0.0f;
    }
}

__device__ __forceinline__ void drop8(float (&v)[8], const Mask& m, uint64_t off, uint64_t block) {
    select(v, m, philox(block, off, m.seed));
}

// ---------------------------------------------------------------- activations

constexpr float kLog2e = 1.44269504f;

// exp through the hardware's base-2 exponential: off by about (|x| + 1) 2^-23
// relative, from the rounding of x log2(e).
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
// 1 / x within 1 ulp, without the division's refinement steps.
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }

__device__ __forceinline__ float sigmoid(float z) { return rcp_fast(1.0f + exp_fast(-z)); }

// The normal distribution function and exp(-z^2/2).  With u = |z| / sqrt(2),
// erfc(u) = exp(-u^2) g(u) and g(u) = t P(t), t = 1 / (1 + 0.4 u): g is smooth
// and falls like 1/u, so a polynomial of degree 8 in t holds its relative
// error under 2.1e-7 for every u >= 0 (coefficients fitted to erfc by weighted
// least squares); evaluated in fp32 it is 4.6e-7, and 6.3e-7 with a reciprocal
// a whole unit off.  erfc itself, and not 1 + erf, so that the lower tail keeps
// a relative precision: g's, and up to z^2 2^-24 by the rounding of the exponent
// (1.4e-6 at z = -5).  It shares its exponential with the density that the
// gradient needs, and costs about a third of separate erf and exp calls.
__device__ __forceinline__ void normal(float z, float* phi, float* gauss) {
    const float t = rcp_fast(fmaf(0.28284271f, fabsf(z), 1.0f));  // 0.4 / sqrt(2)
    float p = 0.0251327585f;  // the coefficients halved
    p = fmaf(p, t, -0.0914575756f);
    p = fmaf(p, t, 0.0845539942f);
    p = fmaf(p, t, -0.00281356019f);
    p = fmaf(p, t, 0.0707205161f);
    p = fmaf(p, t, 0.0842696726f);
    p = fmaf(p, t, 0.10392154f);
    p = fmaf(p, t, 0.112834789f);
    p = fmaf(p, t, 0.112837933f);
    const float e = __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2e));
    const float tail = p * t * e;
    *phi = z > 0.0f ? 1.0f - tail : tail;
    *gauss = e;
}

// act is the same for the whole launch: one uniform branch for 8 elements.
__device__ __forceinline__ void activate8(float (&v)[8], int act) {
    if (act == FSDP_ACT_RELU) {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = v[q] <= 0.0f ? 0.0f : v[q];  // NaN stays
    } else if (act == FSDP_ACT_GELU) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float phi, e;
            normal(v[q], &phi, &e);
            v[q] *= phi;
        }
    } else if (act == FSDP_ACT_SILU) {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] *= sigmoid(v[q]);
    }
}

// d *= act'(z)
__device__ __forceinline__ void activation_grad8(float (&d)[8], const float (&z)[8], int act) {
    if (act == FSDP_ACT_RELU) {
#pragma unroll
        for (int q = 0; q < 8; ++q) d[q] = z[q] <= 0.0f ? 0.0f : z[q] != z[q] ? z[q] : d[q];  // NaN stays
    } else if (act == FSDP_ACT_GELU) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float phi, e;
            normal(z[q], &phi, &e);
            d[q] *= fmaf(z[q] * 0.39894228f, e, phi);  // 1 / sqrt(2 pi)
        }
    } else if (act == FSDP_ACT_SILU) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float s = sigmoid(z[q]);
            d[q] *= s * fmaf(z[q], 1.0f - s, 1.0f);
        }
    }
}

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

// Two of the four E4M3 codes in c (its low or high half) as bf16, exactly.
template <bool HIGH>
__device__ __forceinline__ uint32_t widen2_e4m3(uint32_t c) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, HIGH));
}

__device__ __forceinline__ u32x4 widen_e4m3(uint32_t c0, uint32_t c1) {
    return u32x4{widen2_e4m3<false>(c0), widen2_e4m3<true>(c0), widen2_e4m3<false>(c1), widen2_e4m3<true>(c1)};
}

// ---------------------------------------------------------------- epilogue

// A product's outputs are not read again by its launch: stored non-temporally
// they leave L2 to the operands (8192 x 4096 x 11008 581 -> 553 us, 8192 x 8192 x
// 8192 770 -> 750; written through, 572 and 765).
__device__ __forceinline__ void output8(uint16_t* p, int cnt, const float (&v)[8]) {
    if (cnt >= 8) __builtin_nontemporal_store(pack8(v), reinterpret_cast<u32x4_any*>(p));
    else store8(p, cnt, v);
}

__device__ __forceinline__ void output8(float* p, int cnt, const float (&v)[8]) {
    if (cnt >= 8) {
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}), reinterpret_cast<u32x4_any*>(p));
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]}), reinterpret_cast<u32x4_any*>(p + 4));
    } else {
        store8(p, cnt, v);
    }
}

struct Epilogue {
    void* out;
    const void* res;  // of out's type: the residual, or out itself to accumulate
    uint16_t* z;
    const uint16_t* bias;
    const float* scale;  // the product is divided by it; null: 1
    int64_t ldo, ldr, ldz;
    Mask mask;
    int64_t n, i0, j0;  // the whole matrix's columns; the first row and column of this product in it (j0 a multiple of 8)
    int32_t out_f32, act;
};

// Elements (i, j .. j + cnt) of the output for the NB rows i = row, row + step,
// ... below m, j a multiple of 8: the forward call's bias, activation, dropout
// and residual; the gradients use the division, the accumulation and the
// store.  Every row's residual is read before the first row is stored, so that
// the reads wait once (the output may be the residual, element for element).
template <int NB>
__device__ __forceinline__ void epilogue8(const Epilogue& e, int64_t row, int step, int64_t m, int64_t j, int cnt,
                                          float recip, uint64_t off, float (&v)[NB][8]) {
    float r[NB][8];
    if (e.res) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int64_t i = row + b * step;
            if (i < m) {
                if (e.out_f32) load8(static_cast<const float*>(e.res) + i * e.ldr + j, cnt, r[b]);
                else load8(static_cast<const uint16_t*>(e.res) + i * e.ldr + j, cnt, r[b]);
            }
        }
    }
    if (e.scale) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int q = 0; q < 8; ++q) v[b][q] *= recip;
    }
    if (e.bias) {
        float c[8];
        load8(e.bias + j, cnt, c);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int q = 0; q < 8; ++q) v[b][q] += c[q];
    }
    if (e.z) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
            if (row + b * step < m) output8(e.z + (row + b * step) * e.ldz + j, cnt, v[b]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) activate8(v[b], e.act);
    if (e.mask.t) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
            drop8(v[b], e.mask, off, static_cast<uint64_t>(e.i0 + row + b * step) * ((e.n + 7) >> 3) + ((e.j0 + j) >> 3));
    }
    if (e.res) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int q = 0; q < 8; ++q) v[b][q] += r[b][q];
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int64_t i = row + b * step;
        if (i < m) {
            if (e.out_f32) output8(static_cast<float*>(e.out) + i * e.ldo + j, cnt, v[b]);
            else output8(static_cast<uint16_t*>(e.out) + i * e.ldo + j, cnt, v[b]);
        }
    }
}

// ---------------------------------------------------------------- tiled product

// In this order: with the sizes before the pointers 16 tokens of [11008, 4096]
// codes took 12.45 us for 12.2, the odd gradients 1 % more.
struct Product {
    const void* a;
    const void* b;
    int64_t lda, ldb;
    int32_t m, n, k;        // output rows and columns, contraction length
    int32_t splits, kper;   // the contraction in `splits` parts of kper (a multiple of kBK)
    int32_t tm, tn;         // output tiles
    float* part;            // splits > 1: [splits][m][pitch] partial sums
    int32_t pitch;          // n rounded up to 8
    Epilogue e;

    Extent extent() const { return {m, n, k, pitch}; }
};

// Workgroup b runs on XCD b mod 8, and each XCD has its own L2: consecutive
// ids go to one XCD, so that the tiles it works on at a time are neighbours
// and share operand rows in its L2.
__device__ __forceinline__ int tile_id(int b, int total) {
    const int x = b % kXcds, q = total / kXcds, r = total % kXcds;
    return x * q + min(x, r) + b / kXcds;
}

// Tile `id` in bands of `kBand` tile rows walked column by column: any run of
// consecutive ids covers a nearly square patch of the output.
constexpr int kBand = 4;
__device__ __forceinline__ void tile_at(int id, int tm, int tn, int* ti, int* tj) {
    const int band = id / (kBand * tn), first = band * kBand, rows = min(kBand, tm - first);
    const int in = id - band * (kBand * tn);
    *ti = first + in % rows;
    *tj = in / rows;
}

// LDS images of one operand's tile of kBK contraction elements, in 16-byte
// slots of E = 8 bf16 or 16 E4M3 codes.  l-major: slot = row * (kBK / E) +
// place, and a row's chunks are permuted among its places by the row, so that
// the 8 rows which 8 lanes read at one chunk lie on different banks: by row mod
// 8 where a row is 128 bytes, by row / 2 mod 4 where two are.
template <int E>
__device__ __forceinline__ int lmajor_swizzle(int row) {
    return E == 8 ? row & 7 : (row >> 1) & 3;
}
template <int E>
__device__ __forceinline__ int lmajor_chunk(int slot) {
    return (slot & (kBK / E - 1)) ^ lmajor_swizzle<E>(slot / (kBK / E));
}
// Row-of-outputs ("o-major"): slot = l * (width / E) + place.  A transpose
// read takes 16 outputs of several consecutive l in each 16 lanes: 32 bytes of
// 4 l (bf16), so pairs of chunks are moved, by l mod 4 and bit 3 of l; or 16
// bytes of 8 l (E4M3), moved by l mod 16.  The rows that half a wave reads then
// lie on different banks.
template <int W, int E>
__device__ __forceinline__ int omajor_swizzle(int l) {
    return E == 8 ? (((l & 3) | ((l >> 1) & 4)) & (W / 16 - 1)) << 1 : l & (W / 16 - 1);
}
template <int W, int E>
__device__ __forceinline__ int omajor_chunk(int slot) {
    return slot % (W / E) ^ omajor_swizzle<W, E>(slot / (W / E));
}

using Lds = __attribute__((address_space(3))) uint8_t;

constexpr uint32_t kOutside = 0x80000000u;  // a buffer offset past every range used here

// Copies one operand's tile from memory to LDS without passing through
// registers.  What lies outside the matrix comes as zeros: buffer loads are
// checked against a range, and such lanes' offsets lie beyond it.  Needs
// 16-byte aligned rows and lengths that are multiples of E, so that no 16-byte
// chunk is partly outside.
template <int W, int THREADS, bool LMAJOR, int E>
struct DirectTile {
    static constexpr int kBytes = 16 / E;  // of an element
    static constexpr int kLoads = W * (kBK / E) / THREADS;
    const uint8_t* base;  // the tile's first row and column at this contraction index
    int64_t step;         // bytes per kBK contraction elements
    int left;             // contraction elements from here to the end, may be negative
    int row;              // bytes of a row
    int chunk;            // l-major: this thread's first element in a row (the same in all its loads)
    uint32_t off[kLoads];

    __device__ __forceinline__ void init(const void* p, int64_t ld, int o0, int no, int l0, int lend, int tid) {
        row = static_cast<int>(ld * kBytes);
        left = lend - l0;
        if (LMAJOR) {
            base = static_cast<const uint8_t*>(p) + o0 * (ld * kBytes) + static_cast<int64_t>(l0) * kBytes;
            step = kBK * kBytes;
            chunk = lmajor_chunk<E>(tid) * E;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int r = (i * THREADS + tid) / (kBK / E);
                off[i] = o0 + r < no ? static_cast<uint32_t>(r * row + chunk * kBytes) : kOutside;
            }
        } else {
            base = static_cast<const uint8_t*>(p) + l0 * (ld * kBytes) + static_cast<int64_t>(o0) * kBytes;
            step = kBK * (ld * kBytes);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int slot = i * THREADS + tid, c = omajor_chunk<W, E>(slot);
                off[i] = o0 + c * E < no ? static_cast<uint32_t>(slot / (W / E) * row + c * 16) : kOutside;
            }
        }
    }

    // Load q of the tile.  Behind the contraction's end no load touches
    // memory.  l-major: the lanes whose chunk lies there are sent out of
    // range; else the range ends with the last row.
    __device__ __forceinline__ void load(Lds* dst, int wave, int q) {
        const int range = LMAJOR ? 0x7fffffff : __builtin_amdgcn_readfirstlane(max(0, min(left, kBK)) * row);
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, range, 0x00020000);
        const uint32_t o = LMAJOR && chunk >= left ? kOutside : off[q];
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void*)(dst + (q * THREADS + wave * 64) * 16), 16, o, 0, 0, 0);
    }

    __device__ __forceinline__ void advance() {
        base += step;
        left -= kBK;
    }
};

// The same through registers, for rows that start anywhere, lengths that are
// no multiple of 8, and E4M3 codes, which become bf16 on the way.
template <int W, int THREADS, bool LMAJOR, bool FP8>
struct StagedTile {
    static constexpr int kLoads = W * (kBK / 8) / THREADS;
    const uint8_t* p;
    int64_t ld;
    int o0, no, nl, tid;
    u32x4 reg[kLoads];

    __device__ __forceinline__ void init(const void* ptr, int64_t ld_, int o0_, int no_, int tid_, int nl_) {
        p = static_cast<const uint8_t*>(ptr);
        ld = ld_;
        o0 = o0_;
        no = no_;
        nl = nl_;
        tid = tid_;
    }

    // l0: the tile's first contraction index; nl: the end of this part's.
    __device__ __forceinline__ void load(int l0) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int slot = i * THREADS + tid;
            int64_t row, col;
            int cnt;  // elements of this chunk inside the matrix
            if (LMAJOR) {
                row = o0 + (slot >> 3);
                col = l0 + lmajor_chunk<8>(slot) * 8;
                cnt = row < no ? static_cast<int>(min(static_cast<int64_t>(8), nl - col)) : 0;
            } else {
                row = l0 + slot / (W / 8);
                col = o0 + omajor_chunk<W, 8>(slot) * 8;
                cnt = row < nl ? static_cast<int>(min(static_cast<int64_t>(8), no - col)) : 0;
            }
            if (FP8) {
                const uint8_t* q = p + row * ld + col;
                uint32_t w0 = 0, w1 = 0;
                if (cnt >= 8) {
                    const Bytes8 b = *reinterpret_cast<const Bytes8*>(q);
                    w0 = b.v[0];
                    w1 = b.v[1];
                } else {
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const uint32_t c = s < cnt ? q[s] : 0u;
                        if (s < 4) w0 |= c << (8 * s);
                        else w1 |= c << (8 * (s - 4));
                    }
                }
                reg[i][0] = w0;
                reg[i][1] = w1;
            } else {
                const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + row * ld + col;
                if (cnt >= 8) {
                    reg[i] = reinterpret_cast<const Bytes16*>(q)->v;
                } else {
                    u32x4 w = {0, 0, 0, 0};
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const uint32_t c = s < cnt ? q[s] : 0u;
                        w[s / 2] |= c << (16 * (s & 1));
                    }
                    reg[i] = w;
                }
            }
        }
    }

    __device__ __forceinline__ void store(Lds* dst) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            u32x4 w = reg[i];
            if (FP8) w = widen_e4m3(w[0], w[1]);
            *(__attribute__((address_space(3))) u32x4*)(dst + (i * THREADS + tid) * 16) = w;
        }
    }
};

// One lane's operand of a 16x16x32 matrix instruction from a tile's LDS image:
// lane l holds output o0 + l mod 16 and contraction elements 8 (l / 16) + 0..7
// of the 32 that start at 32 * kk.
template <int W, bool LMAJOR, int NF, int E>
struct Fragments {
    using Raw = std::conditional_t<E == 8, bf16x8, u32x2>;  // 8 bf16 or 8 codes
    static constexpr int kRow = LMAJOR ? kBK * (16 / E) : W * (16 / E);  // bytes of an LDS row
    int at[LMAJOR ? (E == 8 ? 1 : 2) : NF];

    __device__ __forceinline__ void init(int o0, int lane) {
        const int lo = lane & 15, g = lane >> 4;
        if (LMAJOR) {
            at[0] = (o0 + lo) * kRow + ((E == 8 ? g : g >> 1) ^ lmajor_swizzle<E>(lo)) * 16;
            if (E == 16) {
                at[0] += (g & 1) * 8;
                at[E == 16] = at[0] ^ 32;
            }
        } else {
            const int l = E == 8 ? g * 8 + (lo >> 2) : g * 8 + (lo >> 1);
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const int chunk = (o0 / 16 + f) * (16 / E) ^ omajor_swizzle<W, E>(l);
                at[f] = l * kRow + chunk * 16 + (E == 8 ? lo & 3 : lo & 1) * 8;
            }
        }
    }

    __device__ __forceinline__ Raw get(const Lds* tile, int f, int kk) const {
        if constexpr (LMAJOR && E == 8) {
            // chunk 4 kk + g: kk flips bit 2 of the place
            return *(const __attribute__((address_space(3))) bf16x8*)(tile + (at[0] ^ (kk << 6)) + f * (16 * kRow));
        } else if constexpr (LMAJOR) {
            // chunk 2 kk + g / 2: kk flips bit 1
            return *(const __attribute__((address_space(3))) u32x2*)(tile + at[kk] + f * (16 * kRow));
        } else if constexpr (E == 8) {
            using P = __attribute__((address_space(3))) s16x4*;
            const Lds* q = tile + at[f] + kk * 32 * kRow;
            const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)q);
            const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(q + 4 * kRow));
            const struct { s16x4 x, y; } xy = {x, y};
            return __builtin_bit_cast(bf16x8, xy);
        } else {
            using P = __attribute__((address_space(3))) i32x2*;
            return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((P)(tile + at[f] + kk * 32 * kRow)));
        }
    }
};

// acc += the 16x16 product of two fragments.  Written as assembly for its
// register classes: accumulators in AGPRs, operands in VGPRs.  Left to choose,
// the compiler mixes the two for 256 accumulators a lane and moves them about
// between the products.  What it then cannot see is the wait of a few cycles
// between a product and another unit's read or write of its accumulator:
// settle() stands where accumulators change hands, before the first product
// and after the last, and names them all, so that neither their zeros nor
// their uses can move across it.
__device__ __forceinline__ void mfma(f32x4& acc, const bf16x8& b, const bf16x8& a) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
}
template <int FI, int FJ>
__device__ __forceinline__ void settle(f32x4 (&acc)[FI][FJ]) {
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) asm volatile("" : "+a"(acc[i][j]));
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) asm volatile("" : "+a"(acc[i][j]));
}

// Everything this wave has asked of memory and LDS has come; ALL: in every
// wave of the workgroup.
template <bool ALL>
__device__ __forceinline__ void arrive() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    if (ALL) {
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }
}

// BM x BN output tile by WI x WJ waves, two LDS stages of kBK contraction
// elements: while one is multiplied the next arrives.
//
// 256 x 256 by four waves of 128 x 128, one a SIMD: the largest accumulator
// that the registers hold (256 a lane), which needs the fewest LDS and L2 bytes
// a product; with eight waves of 128 x 64, which read half as much again, an
// 8192 x 4096 x 4096 weight gradient took 322 us, this way 206 when both were
// new, 193 now.  8192 x 8192 x 8192: 750 us, 1.47 PFLOP/s (the library's
// plain product: 1.42).  What bounds it is power: without any memory traffic it
// takes 5 % fewer cycles, at 2.3 GHz, where with it the clock falls to 1.9; the
// matrix units are busy in 74 % of the cycles of that weight gradient.  Four
// stages of 32 (a longer look ahead) were 6 % slower: twice the barriers, and
// half a cache line a row and load.  A workgroup that stays and fetches its
// next tile during the epilogue was 2 % slower to 3 % faster.
// 128 x 128 by four waves of 64 x 64, two workgroups a CU: one's epilogue and
// waits run beside the other's products; 2048 x 4096 x 4096 59 us (1.16).
//
// KW > 1 (with WI = WJ = 1): KW waves that each take a KW-th of the
// contraction for the whole tile, through stages of their own, without a
// barrier until their sums are added at the end.  It is the form for products
// of few tiles: a wave's tile stays 64 x 64, which needs half the LDS reads a
// product of 32 x 32 ones, while four times as many loads are on their way.
// 1024 x 1024 x 4096: 17 us; bound by L2's bytes (90 GB/s a CU): without
// memory traffic 12.8, and with 32-element stages, half lines, 23.8.
template <int BM, int BN, int WI, int WJ, int KW, bool AL, bool BL, bool DIRECT, bool FP8>
__global__ __launch_bounds__(WI* WJ* KW * 64) void product_kernel(Product g) {
    static_assert(KW == 1 || (WI == 1 && WJ == 1 && BM == 64 && BN == 64 && DIRECT), "waves with parts of the contraction");
    constexpr int kThreads = WI * WJ * 64, kWM = BM / WI, kWN = BN / WJ, kFI = kWM / 16, kFJ = kWN / 16;
    constexpr int kEB = DIRECT && FP8 ? 16 : 8;  // elements of B in 16 bytes of LDS
    constexpr int kStage = (BM + BN) * kBK * 2;  // B's part is half filled by codes
    constexpr bool kShared = KW == 1;  // the waves share their stages
    __shared__ __attribute__((aligned(1024))) uint8_t s0[kStage * KW];
    __shared__ __attribute__((aligned(1024))) uint8_t s1[kStage * KW];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tid = kShared ? threadIdx.x : lane;  // among the threads that fill a stage
    const int part = kShared ? 0 : wave;
    Lds* const l0 = (Lds*)s0 + part * kStage;
    Lds* const l1 = (Lds*)s1 + part * kStage;
    const int tiles = g.tm * g.tn;
    const int id = tile_id(blockIdx.x, tiles * g.splits);
    const int split = id / tiles;
    int ti, tj;
    tile_at(id - split * tiles, g.tm, g.tn, &ti, &tj);
    const int i0 = ti * BM, j0 = tj * BN;
    int kbeg = split * g.kper, kend = min(g.k, kbeg + g.kper);
    if (KW > 1) {
        const int per = (kend - kbeg + kBK * KW - 1) / (kBK * KW) * kBK;
        kbeg += part * per;
        kend = min(kend, kbeg + per);
    }
    const int steps = kend > kbeg ? (kend - kbeg + kBK - 1) / kBK : 0;
    const int wi = kShared ? wave / WJ : 0, wj = kShared ? wave % WJ : 0;

    f32x4 acc[kFI][kFJ];
#pragma unroll
    for (int i = 0; i < kFI; ++i)
#pragma unroll
        for (int j = 0; j < kFJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    Fragments<BM, AL, kFI, 8> fa;
    Fragments<BN, BL, kFJ, kEB> fb;
    fa.init(wi * kWM, lane);
    fb.init(wj * kWN, lane);

    // A step multiplies one LDS stage in two halves of 32 contraction elements.
    // Each half's fragments are read from LDS while the half before is being
    // multiplied, and a stage is refilled as soon as its second half has been
    // read, a whole step ahead of its use; so the one barrier of a step, in
    // its middle, finds everything that it waits for already there.
    bf16x8 a[2][kFI], b[2][kFJ];
    u32x2 codes[kFJ];  // E4M3: the next half's, until they are widened
    // Fragment f of a half, in the order in which multiplying needs them.
    auto read = [&](const Lds* stage, int kk, int f) {
        if (f < kFJ) {
            if constexpr (kEB == 8) b[kk][f] = fb.get(stage + BM * kBK * 2, f, kk);
            else codes[f] = fb.get(stage + BM * kBK * 2, f, kk);
        } else {
            a[kk][f - kFJ] = fa.get(stage, f - kFJ, kk);
        }
    };
    // Instruction c of the 4 kFJ that widen a half's codes.
    auto widen_step = [&](int kk, int c) {
        u32x4 w = __builtin_bit_cast(u32x4, b[kk][c / 4]);
        w[c % 4] = c % 2 ? widen2_e4m3<true>(codes[c / 4][c % 4 / 2]) : widen2_e4m3<false>(codes[c / 4][c % 4 / 2]);
        b[kk][c / 4] = __builtin_bit_cast(bf16x8, w);
    };
    // Half kk, product by product, with the reads of the other half (of
    // `stage`) and a refill's loads between them one at a time: a product
    // keeps the matrix unit for 16 cycles, in which one other access can be
    // issued, and with one wave a SIMD nothing else covers a longer run of
    // them.  The reads end early enough to have come when the half does, B's
    // first, whose codes are widened between the later products.
    auto multiply = [&](int kk, const Lds* stage, auto&& between) {
        constexpr int kAll = kFI * kFJ, kGap = kAll >= 64 ? 3 : 1;
        constexpr int kFirst = kAll >= 64 ? 28 : 8, kWiden = kFJ * 4 / (kAll - kFirst) + (kFJ * 4 % (kAll - kFirst) != 0);
#pragma unroll
        for (int t = 0; t < kAll; ++t) {
            mfma(acc[t / kFJ][t % kFJ], b[kk][t % kFJ], a[kk][t / kFJ]);
            __builtin_amdgcn_sched_barrier(0);
            if (t % kGap == 0 && t / kGap < kFI + kFJ) read(stage, 1 - kk, t / kGap);
            if constexpr (kEB == 16) {
#pragma unroll
                for (int c = (t - kFirst) * kWiden; c < (t - kFirst + 1) * kWiden; ++c)
                    if (c >= 0 && c < kFJ * 4) widen_step(1 - kk, c);
            }
            between(t, kAll);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // refill(stage, i, n): what of a stage's filling belongs to place i of n.
    auto run = [&](auto&& refill) {
        auto step = [&](Lds* cur, Lds* nxt) {
            multiply(0, cur, [](int, int) {});
            arrive<kShared>();
            multiply(1, nxt, [&](int i, int n) { refill(cur, i, n); });
        };
        arrive<kShared>();
        settle(acc);
#pragma unroll
        for (int f = 0; f < kFI + kFJ; ++f) read(l0, 0, f);
        if constexpr (kEB == 16) {
#pragma unroll
            for (int c = 0; c < kFJ * 4; ++c) widen_step(0, c);
            // as settle(): operands that other units wrote, before the first product
#pragma unroll
            for (int j = 0; j < kFJ; ++j) asm volatile("" : "+v"(b[0][j]));
            asm volatile("s_nop 3" ::: "memory");
#pragma unroll
            for (int j = 0; j < kFJ; ++j) asm volatile("" : "+v"(b[0][j]));
        }
        // Two steps a turn, so that each LDS access names its stage.  An odd
        // count takes one more step, over zeros.
        int turns = (steps + 1) / 2;
        do {
            step(l0, l1);
            step(l1, l0);
        } while (--turns > 0);
        settle(acc);
    };
    if (steps > 0) {
        if constexpr (DIRECT) {
            DirectTile<BM, kThreads, AL, 8> ta;
            DirectTile<BN, kThreads, BL, kEB> tb;
            ta.init(g.a, g.lda, i0, g.m, kbeg, kend, tid);
            tb.init(g.b, g.ldb, j0, g.n, kbeg, kend, tid);
            constexpr int kLoads = ta.kLoads + tb.kLoads;
            auto fetch = [&](Lds* stage, int q) {
                if (q < ta.kLoads) ta.load(stage, kShared ? wave : 0, q);
                else tb.load(stage + BM * kBK * 2, kShared ? wave : 0, q - ta.kLoads);
                if (q == kLoads - 1) {
                    ta.advance();
                    tb.advance();
                }
            };
#pragma unroll
            for (int q = 0; q < kLoads; ++q) fetch(l0, q);
#pragma unroll
            for (int q = 0; q < kLoads; ++q) fetch(l1, q);
            run([&](Lds* stage, int i, int n) {
                const int every = n / kLoads;
                if (i % every == every - 1 && i / every < kLoads) fetch(stage, i / every);
            });
        } else {
            StagedTile<BM, kThreads, AL, false> ta;
            StagedTile<BN, kThreads, BL, FP8> tb;
            ta.init(g.a, g.lda, i0, g.m, tid, kend);
            tb.init(g.b, g.ldb, j0, g.n, tid, kend);
            int l = kbeg;
            auto fetch = [&] {
                ta.load(l);
                tb.load(l);
                l += kBK;
            };
            auto store = [&](Lds* stage) {
                ta.store(stage);
                tb.store(stage + BM * kBK * 2);
                fetch();
            };
            fetch();
            store(l0);
            store(l1);
            run([&](Lds* stage, int i, int) {
                if (i == 0) store(stage);
            });
        }
    }

    // Lane l holds of each 16x16 block output row l mod 16 and columns
    // 4 (l / 16) + 0..3.
    const int lo = lane & 15, hi = lane >> 4;
    using Quad = __attribute__((address_space(3))) f32x4;
    const float recip = g.e.scale ? 1.0f / *g.e.scale : 1.0f;
    const uint64_t off = mask_offset(g.e.mask);
    float* const sums = g.part + static_cast<int64_t>(split) * g.m * g.pitch;
    // Rows of 16-byte chunks in LDS are permuted by the row, which spreads the
    // 16 rows that one write touches over the banks.
    if constexpr (KW > 1) {
        arrive<false>();  // this wave's stages are being read and filled until here
#pragma unroll
        for (int i = 0; i < kFI; ++i)
#pragma unroll
            for (int j = 0; j < kFJ; ++j)
                *(Quad*)(l0 + (i * 16 + lo) * 256 + (((j * 4 + hi) ^ lo) << 4)) = acc[i][j];
        __syncthreads();
        // each wave adds the parts of its 64 / KW rows, in order
        constexpr int kBatch = 64 / KW / 8;
        const int c = lane & 7, col = j0 + c * 8, r0 = wave * (64 / KW) + (lane >> 3);
        float v[kBatch][8];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int r = r0 + q * 8;
            f32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
#pragma unroll
            for (int p = 0; p < KW; ++p) {
                const Lds* row = (Lds*)s0 + p * kStage + r * 256;
                x += *(const Quad*)(row + (((c * 2) ^ (r & 15)) << 4));
                y += *(const Quad*)(row + (((c * 2 + 1) ^ (r & 15)) << 4));
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                v[q][t] = x[t];
                v[q][4 + t] = y[t];
            }
        }
        if (g.splits > 1) {
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int row = i0 + r0 + q * 8;
                if (row < g.m && col < g.pitch) store8(sums + static_cast<int64_t>(row) * g.pitch + col, 8, v[q]);
            }
        } else if (col < g.n) {
            epilogue8<kBatch>(g.e, i0 + r0, 8, g.m, col, g.n - col, recip, off, v);
        }
        return;
    }
    if (g.splits > 1) {
#pragma unroll
        for (int i = 0; i < kFI; ++i) {
            const int row = i0 + wi * kWM + i * 16 + lo;
#pragma unroll
            for (int j = 0; j < kFJ; ++j) {
                const int col = j0 + wj * kWN + j * 16 + hi * 4;
                if (row < g.m && col < g.pitch)
                    *reinterpret_cast<f32x4*>(sums + static_cast<int64_t>(row) * g.pitch + col) = acc[i][j];
            }
        }
        return;
    }
    // 64 rows at a time through the wave's own piece of LDS, so that a lane has
    // 8 consecutive columns: one 16-byte store and one mask block.
    arrive<true>();  // the last stages are being read and filled until here
    constexpr int kHalf = (WI * WJ + 1) / 2, kPiece = 64 * kWN * 4, kLanes = kWN / 8;
    static_assert(KW > 1 || (kWM % 64 == 0 && kWN >= 64 && kHalf * kPiece <= kStage), "a piece of 64 x kWN floats a wave");
    Lds* const piece = (wave < kHalf ? l0 : l1) + wave % kHalf * kPiece;
    const int c = lane % kLanes, col = j0 + wj * kWN + c * 8;
#pragma unroll
    for (int h = 0; h < kWM / 64; ++h) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < kFJ; ++j)
                *(Quad*)(piece + (i * 16 + lo) * (kWN * 4) + (((j * 4 + hi) ^ lo) << 4)) = acc[h * 4 + i][j];
        __builtin_amdgcn_wave_barrier();
        constexpr int kBatch = 4, kStep = 64 / kLanes;
#pragma unroll 1
        for (int r = lane / kLanes; r < 64; r += kBatch * kStep) {
            float v[kBatch][8];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int rq = r + q * kStep;
                const f32x4 x = *(const Quad*)(piece + rq * (kWN * 4) + (((c * 2) ^ (rq & 15)) << 4));
                const f32x4 y = *(const Quad*)(piece + rq * (kWN * 4) + (((c * 2 + 1) ^ (rq & 15)) << 4));
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    v[q][t] = x[t];
                    v[q][4 + t] = y[t];
                }
            }
            if (col < g.n)
                epilogue8<kBatch>(g.e, i0 + wi * kWM + h * 64 + r, kStep, g.m, col, g.n - col, recip, off, v);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// The sum of a split product's parts, in order, and the epilogue.  A pass over
// memory, at about 6 TB/s, that takes 3 us even for the smallest output.
constexpr int kJoinBlock = 256;
__global__ __launch_bounds__(kJoinBlock) void join_kernel(Product g) {
    const int chunks = g.pitch / 8;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kJoinBlock + threadIdx.x;
    if (id >= static_cast<int64_t>(g.m) * chunks) return;
    const int64_t i = id / chunks;
    const int j = static_cast<int>(id - i * chunks) * 8;
    const float* p = g.part + id * 8;
    const int64_t stride = static_cast<int64_t>(g.m) * g.pitch;
    f32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = 0; s < g.splits; ++s) {
        x += *reinterpret_cast<const f32x4*>(p + s * stride);
        y += *reinterpret_cast<const f32x4*>(p + s * stride + 4);
    }
    float v[1][8] = {{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]}};
    epilogue8<1>(g.e, i, 0, g.m, j, g.n - j, g.e.scale ? 1.0f / *g.e.scale : 1.0f, mask_offset(g.e.mask), v);
}

// ---------------------------------------------------------------- products of few rows

// The 16 bytes at p.  ODD: where p is off a 4-byte boundary a 16-byte load takes
// several times as long, so they come as the aligned words that hold them (five,
// and no byte outside those that hold some of the 16) and are moved down.
template <bool ODD>
__device__ __forceinline__ u32x4 bytes16(const uint8_t* p) {
    if constexpr (!ODD) return reinterpret_cast<const Bytes16*>(p)->v;
    const uint32_t in = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 3, bits = in * 8;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p - in);
    typedef u32x4 Words __attribute__((aligned(4)));
    const u32x4 w = *reinterpret_cast<const Words*>(q);
    const uint32_t last = q[in ? 4 : 3];
    return u32x4{__builtin_amdgcn_alignbit(w[1], w[0], bits), __builtin_amdgcn_alignbit(w[2], w[1], bits),
                 __builtin_amdgcn_alignbit(w[3], w[2], bits), __builtin_amdgcn_alignbit(last, w[3], bits)};
}

// The same for bytes [at, at + 16) of a row of `len`, zeros from its end on.
// Past the end, the row's last 16 bytes are read and moved down, so that this is
// one load too; of a shorter row, each element.
template <typename T, bool ODD>
__device__ __forceinline__ u32x4 row_end16(const uint8_t* row, int64_t at, int64_t len) {
    u32x4 w = {0, 0, 0, 0};
    if (at >= len) return w;
    if (len < 16) {
#pragma unroll
        for (int s = 0; s < static_cast<int>(16 / sizeof(T)); ++s) {
            const int64_t b = at + s * static_cast<int64_t>(sizeof(T));
            const uint32_t c = b < len ? *reinterpret_cast<const T*>(row + b) : 0u;
            w[s * sizeof(T) / 4] |= c << (8 * (s * sizeof(T) % 4));
        }
        return w;
    }
    const int64_t from = min(at, len - 16);
    w = bytes16<ODD>(row + from);
    const uint32_t back = static_cast<uint32_t>(at - from);
    if (back & 8) w = u32x4{w[2], w[3], 0, 0};
    if (back & 4) w = u32x4{w[1], w[2], w[3], 0};
    const uint32_t bits = (back & 3) * 8;
    return u32x4{__builtin_amdgcn_alignbit(w[1], w[0], bits), __builtin_amdgcn_alignbit(w[2], w[1], bits),
                 __builtin_amdgcn_alignbit(w[3], w[2], bits), __builtin_amdgcn_alignbit(0u, w[3], bits)};
}

// The forward product for at most 16 * MB tokens: bound by reading W once.  One
// token: [4096, 4096] 8.2 us with the call, [28672, 8192] 89 us (5.3 TB/s), from
// E4M3 codes 46; sixteen tokens: 10.4, 101 and 61.  Four waves or sixteen a
// workgroup: 3-15 % slower at most sizes; non-temporal loads of W 8-25 %.  A
// workgroup takes 16 * JB output features; its eight waves take every eighth
// chunk of 64 contraction elements, from memory straight into the fragments
// of the matrix instructions (W is used once, so LDS would only be a detour;
// x comes from L2), several chunks on their way at a time, all of whose loads
// are issued before the first is used (left to the compiler's order, sixteen
// tokens of [11008, 4096] take 24.4 us, this way 21.0; of [8192, 28672] 116 and
// 89; one token of [28672, 8192] 89 both ways).  Nothing is on its way while a
// batch is multiplied.  Their sums are added in LDS, so the call is one launch.
// ODD: rows off 4-byte boundaries; 16 tokens of [4096, 4095] 14 us, by unaligned
// loads 30.
constexpr int kFewWaves = 8;
template <int MB, int JB, bool FP8, bool ODD>
__global__ __launch_bounds__(kFewWaves * 64) void few_rows_kernel(Product g) {
    constexpr int kPitch = 20;  // floats of 16, padded against bank conflicts
    __shared__ __attribute__((aligned(16))) float sums[kFewWaves][MB][JB][16 * kPitch];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lo = lane & 15, q = lane >> 4;
    const int j0 = blockIdx.x * (16 * JB);
    // Rows past the end are read as the last one; what they give is not stored.
    const uint8_t* x[MB];
    const uint8_t* w[JB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
        x[i] = static_cast<const uint8_t*>(g.a) + min(i * 16 + lo, g.m - 1) * g.lda * 2;
#pragma unroll
    for (int j = 0; j < JB; ++j)
        w[j] = static_cast<const uint8_t*>(g.b) + min(j0 + j * 16 + lo, g.n - 1) * g.ldb * (FP8 ? 1 : 2);
    f32x4 acc[MB][JB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    // A chunk is two matrix instructions.  Lane group q takes of the chunk's
    // contraction elements 8 q + 0..7 of each half of 32 (bf16), or 16 q + 0..15
    // (E4M3: one 16-byte load), and the same ones of x.
    struct Chunk {
        u32x4 x[MB][2], w[JB][FP8 ? 1 : 2];
    };
    // END: the chunk may end behind the rows' end.
    auto load = [&](Chunk& c, int k, auto end) {
        auto row16 = [&](const uint8_t* row, int at, auto type) {
            using T = decltype(type);
            constexpr int64_t e = sizeof(T);
            if constexpr (decltype(end)::value) return row_end16<T, ODD>(row, at * e, g.k * e);
            else return bytes16<ODD>(row + at * e);
        };
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            if constexpr (FP8) {
                c.w[j][0] = row16(w[j], k + q * 16, uint8_t());
            } else {
                c.w[j][0] = row16(w[j], k + q * 8, uint16_t());
                c.w[j][1] = row16(w[j], k + 32 + q * 8, uint16_t());
            }
        }
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            c.x[i][0] = row16(x[i], k + q * (FP8 ? 16 : 8), uint16_t());
            c.x[i][1] = row16(x[i], k + (FP8 ? q * 16 + 8 : 32 + q * 8), uint16_t());
        }
    };
    auto multiply = [&](const Chunk& c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            bf16x8 b[JB];
#pragma unroll
            for (int j = 0; j < JB; ++j)
                b[j] = __builtin_bit_cast(bf16x8, FP8 ? widen_e4m3(c.w[j][0][2 * h], c.w[j][0][2 * h + 1])
                                                      : c.w[j][FP8 ? 0 : h]);
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int j = 0; j < JB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        b[j], __builtin_bit_cast(bf16x8, c.x[i][h]), acc[i][j], 0, 0, 0);
        }
    };
    // Eight chunks on their way where they take no more than 160 registers, else
    // four; what is left of a wave's chunks in batches of four and two.  Eight
    // against four: one token of [4096, 4096] 8.1 and 8.4 us, from codes 6.3 and
    // 6.9; [28672, 8192] 89.3 and 86.4, from codes 45.7 and 47.5.  Up to 224
    // registers: codes of [32000, 4096] 3-7 % faster, 16 tokens of bf16
    // [8192, 8192] and [8192, 28672] 4 % slower.  One token of [4096, 11008],
    // whose waves have 21 chunks: 23.7 (codes 16.2), the rest one by one 23.7
    // (16.9), by fours alone 22.2 (14.4); [4096, 14336] 23.9 (14.6), one by one
    // 25.7 (15.7).
    constexpr int kAhead = ((FP8 ? JB : 2 * JB) + 2 * MB) * 32 <= 160 ? 8 : 4;
    const int full = g.k / 64;
    int c = wave;
    auto batches = [&](auto ahead) {
        constexpr int kN = decltype(ahead)::value;
        for (; c + (kN - 1) * kFewWaves < full; c += kN * kFewWaves) {
            Chunk r[kN];
#pragma unroll
            for (int u = 0; u < kN; ++u) load(r[u], (c + u * kFewWaves) * 64, std::false_type{});
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < kN; ++u) multiply(r[u]);
        }
    };
    batches(std::integral_constant<int, kAhead>{});
    if constexpr (kAhead > 4) batches(std::integral_constant<int, 4>{});
    batches(std::integral_constant<int, 2>{});
    for (; c * 64 < g.k; c += kFewWaves) {
        Chunk r;
        if (c < full) load(r, c * 64, std::false_type{});
        else load(r, c * 64, std::true_type{});
        multiply(r);
    }
    // Lane: token lo, features 4 q + 0..3.
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j) *reinterpret_cast<f32x4*>(&sums[wave][i][j][lo * kPitch + q * 4]) = acc[i][j];
    __syncthreads();
    const int t = threadIdx.x, half = t & 1, j = (t >> 1) % JB, i = t / (2 * JB);  // 16 MB rows of 2 JB pieces
    const int col = j0 + j * 16 + half * 8;
    if (i >= g.m || i >= 16 * MB || col >= g.n) return;
    float v[1][8] = {{0, 0, 0, 0, 0, 0, 0, 0}};
#pragma unroll
    for (int p = 0; p < kFewWaves; ++p) {
        const float* s = &sums[p][i >> 4][j][(i & 15) * kPitch + half * 8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[0][u] += s[u];
    }
    epilogue8<1>(g.e, i, 0, g.m, col, g.n - col, g.e.scale ? 1.0f / *g.e.scale : 1.0f, mask_offset(g.e.mask), v);
}

// ---------------------------------------------------------------- operands laid out anew

// A matrix as the direct loads want it: rows whose length is rounded up to 16
// bytes with zeros, on 128-byte boundaries, so that the 128 bytes of a row which
// a stage takes are one cache line (rows 8208 bytes apart took a 4096 x 2048 x
// 4097 product from 60 to 101 us).  5 us for a few megabytes, which is a
// launch's latency, then 4 TB/s; the loads through registers, which need no
// copy, took 25 us instead of 17 for the 1000 x 1024 x 1365 forward product.
// Rows may lie off 4-byte boundaries, which bytes16 takes into account.
struct Pack {
    const void* src;
    uint8_t* dst;
    int64_t ld;
    int32_t rows, cols, chunks, pitch, fp8;  // chunks: 16-byte pieces of a row; pitch: bytes between packed rows
};
constexpr int kPackBlock = 256;
__global__ __launch_bounds__(kPackBlock) void pack_kernel(Pack a, Pack b, int blocks_a) {
    const bool second = static_cast<int>(blockIdx.x) >= blocks_a;
    const Pack p = second ? b : a;
    const int id = (static_cast<int>(blockIdx.x) - (second ? blocks_a : 0)) * kPackBlock + threadIdx.x;
    const int row = id / p.chunks, c = id - row * p.chunks;
    if (row >= p.rows) return;
    u32x4 v;
    const int64_t e = p.fp8 ? 1 : 2;
    const uint8_t* from = static_cast<const uint8_t*>(p.src) + row * p.ld * e;
    if (p.fp8) v = row_end16<uint8_t, true>(from, c * 16, p.cols);
    else v = row_end16<uint16_t, true>(from, c * 16, p.cols * e);
    *reinterpret_cast<u32x4*>(p.dst + static_cast<int64_t>(row) * p.pitch + c * 16) = v;
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

// 2^tx lanes take one row's chunks of 16 bytes (as many as the row has, up
// to a wave), the block's 256 >> tx other places take rows, one at a time: two
// at a time, with twice the loads on their way, were 8 % slower.
constexpr int kElemBlock = 256;
struct Grid {
    int32_t tx, cblocks;  // lanes a row (log2), column blocks
    int64_t rows;         // rows a block takes in all (a multiple of 256 >> tx)
};

struct DropoutArgs {
    void* y;
    const void* x;
    const void* res;
    int64_t ldy, ldx, ldr, m, n;
    Mask mask;
    Grid g;
    int32_t wt;
};

// 16 bytes a lane: in fp32 two lanes draw one mask block, each for its half.
// With 8 elements a lane a store would write half of every line it touches:
// 8192 x 4096 fp32 77.6 us, this way 49.5.
template <typename T>
__global__ __launch_bounds__(kElemBlock) void dropout_kernel(DropoutArgs a) {
    constexpr int kEach = 16 / sizeof(T);
    const int tid = threadIdx.x, per = kElemBlock >> a.g.tx;
    const int64_t rb = blockIdx.x / a.g.cblocks;
    const int64_t j = ((static_cast<int64_t>(blockIdx.x % a.g.cblocks) << a.g.tx) + (tid & ((1 << a.g.tx) - 1))) * kEach;
    if (j >= a.n) return;
    const int cnt = static_cast<int>(min(a.n - j, static_cast<int64_t>(kEach)));
    const int back = chunk_back<T>(cnt, a.n);
    const int64_t chunks = (a.n + 7) >> 3, end = min(a.m, (rb + 1) * a.g.rows);
    const uint64_t off = mask_offset(a.mask);
    for (int64_t i = rb * a.g.rows + (tid >> a.g.tx); i < end; i += per) {
        float v[kEach], r[kEach];
        const u32x4 x = stream_load(static_cast<const T*>(a.x) + i * a.ldx + j, cnt, back);
        u32x4 res = {0, 0, 0, 0};
        if (a.res) res = stream_load(static_cast<const T*>(a.res) + i * a.ldr + j, cnt, back);
        arrange(x, back, v);
        if (a.mask.t) {
            u32x4 w = philox(static_cast<uint64_t>(i * chunks + (j >> 3)), off, a.mask.seed);
            if (kEach == 4 && (j & 4)) w = u32x4{w[2], w[3], 0, 0};
            select(v, a.mask, w);
        }
        if (a.res) {
            arrange(res, back, r);
#pragma unroll
            for (int q = 0; q < kEach; ++q) v[q] += r[q];
        }
        stream_store(static_cast<T*>(a.y) + i * a.ldy + j, cnt, a.wt, v);
    }
}

struct BackwardArgs {
    uint16_t* dz;
    const uint16_t* dy;
    const uint16_t* z;
    int64_t lddz, lddy, ldz, m, n;
    float* part;  // [row blocks][n] column sums, or null
    void* db;     // with one row block: the result
    int32_t db_f32, accumulate, act, sums, wt;
    Mask mask;
    Grid g;
};

__device__ __forceinline__ void put_db(void* db, int f32, int accumulate, int64_t j, float s) {
    if (f32) {
        float* p = static_cast<float*>(db) + j;
        *p = accumulate ? *p + s : s;
    } else {
        uint16_t* p = static_cast<uint16_t*>(db) + j;
        *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(accumulate ? widen(*p) + s : s));
    }
}

// dz and the column sums in one pass.  Bound by memory, with the vector unit
// close behind: 4096 x 11008 with gelu and dropout takes 52 us (5.2 TB/s), of
// which the generator's 83 instructions for 8 elements are about 10, gelu's 184
// 4.  BLOCK 256: a row block's sums of its columns.  BLOCK 1024 is the form for
// few rows, 4 lanes a row and every row in one block, so that the sums need no
// second launch.
constexpr int kTallBlock = 1024;
template <int BLOCK>
__global__ __launch_bounds__(BLOCK) void epilogue_backward_kernel(BackwardArgs a) {
    __shared__ float sums[BLOCK == kElemBlock ? BLOCK : 64][9];
    const int tid = threadIdx.x, per = BLOCK >> a.g.tx, width = 1 << a.g.tx;
    const int64_t rb = blockIdx.x / a.g.cblocks;
    const int64_t j0 = (static_cast<int64_t>(blockIdx.x % a.g.cblocks) << a.g.tx) * 8;
    const int64_t j = j0 + (tid & (width - 1)) * 8;
    const int cnt = static_cast<int>(min(a.n - j, static_cast<int64_t>(8)));  // <= 0 outside
    const int64_t chunks = (a.n + 7) >> 3, end = cnt > 0 ? min(a.m, (rb + 1) * a.g.rows) : 0;
    const int back = chunk_back<uint16_t>(cnt, a.n);
    const uint64_t off = mask_offset(a.mask);
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int64_t i = rb * a.g.rows + (tid >> a.g.tx); i < end; i += per) {
        float v[8], z[8];
        const u32x4 wv = stream_load(a.dy + i * a.lddy + j, cnt, back);
        u32x4 wz = {0, 0, 0, 0};
        if (a.act != FSDP_ACT_NONE) wz = stream_load(a.z + i * a.ldz + j, cnt, back);
        // The bits are drawn while the loads are on their way, and select last, so
        // that a dropped element is 0 whatever dy and z hold (1 % slower than
        // selecting dy).
        u32x4 bits = {0, 0, 0, 0};
        if (a.mask.t) bits = philox(static_cast<uint64_t>(i * chunks + (j >> 3)), off, a.mask.seed);
        arrange(wv, back, v);
        arrange(wz, back, z);
        activation_grad8(v, z, a.act);
        if (a.mask.t) select(v, a.mask, bits);
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] += v[q];
        if (a.dz) stream_store(a.dz + i * a.lddz + j, cnt, a.wt, v);
    }
    if (!a.sums) return;
    int places = per;  // of sums a column in LDS
    if constexpr (BLOCK == kElemBlock) {
#pragma unroll
        for (int q = 0; q < 8; ++q) sums[tid][q] = sum[q];
    } else {
        // first over the wave's rows: lanes of one column chunk are 4 apart
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
            for (int d = 4; d < 64; d <<= 1) sum[q] += __shfl_xor(sum[q], d);
        places = BLOCK / 64;
        if ((tid & 63) < 4)
#pragma unroll
            for (int q = 0; q < 8; ++q) sums[(tid >> 6) * 4 + (tid & 3)][q] = sum[q];
    }
    __syncthreads();
    // thread t of the block's first ones: column t of the block, over its places in order
    for (int t = tid; t < width * 8; t += BLOCK) {
        const int64_t col = j0 + t;
        if (col >= a.n) break;
        float s = 0;
        for (int r = 0; r < places; ++r) s += sums[r * width + (t >> 3)][t & 7];
        if (a.part) a.part[rb * a.n + col] = s;
        else put_db(a.db, a.db_f32, a.accumulate, col, s);
    }
}

// db from the row blocks' sums: 64 columns a block, 16 threads a column, their
// sums added in order.
constexpr int kSumBlock = 1024;
__global__ __launch_bounds__(kSumBlock) void column_sum_kernel(const float* part, int64_t n, int32_t blocks,
                                                               void* db, int32_t f32, int32_t accumulate) {
    __shared__ float sums[16][64];
    const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + c;
    float s = 0;
    if (col < n) {
#pragma unroll 8
        for (int r = q; r < blocks; r += 16) s += part[r * n + col];
    }
    sums[q][c] = s;
    __syncthreads();
    if (q != 0 || col >= n) return;
#pragma unroll
    for (int r = 1; r < 16; ++r) s += sums[r][c];
    put_db(db, f32, accumulate, col, s);
}

// ---------------------------------------------------------------- host: arguments

int32_t make_mask(const fsdp_dropout_mask* d, Mask* out, const char* who) {
    *out = Mask{0, 0, nullptr, 0, 0, 1.0f};
    if (!d) return FSDP_OK;
    if (!(d->p >= 0.0 && d->p <= 1.0)) return fail(FSDP_E_ARG, "%s: dropout p outside [0, 1]", who);
    if (!aligned(d->offset_dev, 8)) return fail(FSDP_E_ALIGN, "%s: offset_dev misaligned", who);
    out->seed = d->seed;
    out->offset = d->offset;
    out->offset_dev = d->offset_dev;
    out->t = static_cast<uint32_t>(std::rint(d->p * 65536.0));
    out->above = static_cast<uint32_t>((static_cast<uint64_t>(out->t) << 16) - 1);
    out->scale = out->t < 65536 ? static_cast<float>(65536.0 / (65536.0 - out->t)) : 0.0f;
    return FSDP_OK;
}

int32_t launched(const char* who) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(FSDP_E_HIP, "%s: launch failed: %s", who, hipGetErrorString(e));
    return FSDP_OK;
}

// ---------------------------------------------------------------- host: products

template <int BM, int BN, int WI, int WJ, int KW, bool AL, bool BL, bool DIRECT, bool FP8>
int32_t launch_product(Product& g, hipStream_t stream, const char* who) {
    g.tm = static_cast<int32_t>(ceil_div(g.m, BM));
    g.tn = static_cast<int32_t>(ceil_div(g.n, BN));
    const int64_t blocks = static_cast<int64_t>(g.tm) * g.tn * g.splits;
    const int64_t joins = ceil_div(static_cast<int64_t>(g.m) * (g.pitch / 8), kJoinBlock);
    if (blocks > kMaxBlocks || (g.splits > 1 && joins > kMaxBlocks))
        return fail(FSDP_E_CAPACITY, "%s: more output tiles than one launch holds", who);
    product_kernel<BM, BN, WI, WJ, KW, AL, BL, DIRECT, FP8>
        <<<dim3(static_cast<uint32_t>(blocks)), dim3(WI * WJ * KW * 64), 0, stream>>>(g);
    int32_t st = launched(who);
    if (st != FSDP_OK || g.splits == 1) return st;
    join_kernel<<<dim3(static_cast<uint32_t>(joins)), dim3(kJoinBlock), 0, stream>>>(g);
    return launched(who);
}

void split(Product& g, int64_t splits, const Space& space) {
    const Parts p = parts_of(g.k, splits);
    g.splits = p.n;
    g.kper = p.k;
    g.part = reinterpret_cast<float*>(space.p);
}

// Columns [j0, j0 + n) of the product.
template <bool BL>
Product columns(const Product& g, bool fp8, int64_t j0, int64_t n) {
    Product s = g;
    s.n = static_cast<int32_t>(n);
    s.pitch = columns_of(g.extent(), n).pitch;
    const int64_t e = fp8 ? 1 : 2, oe = g.e.out_f32 ? 4 : 2;
    s.b = static_cast<const uint8_t*>(g.b) + (BL ? j0 * g.ldb : j0) * e;
    s.e.out = static_cast<uint8_t*>(g.e.out) + j0 * oe;
    if (g.e.res) s.e.res = static_cast<const uint8_t*>(g.e.res) + j0 * oe;
    if (g.e.z) s.e.z = g.e.z + j0;
    if (g.e.bias) s.e.bias = g.e.bias + j0;
    s.e.j0 += j0;
    return s;
}

// Rows [i0, i0 + m) of the product.
template <bool AL>
Product rows(const Product& g, int64_t i0, int64_t m) {
    Product s = g;
    s.m = static_cast<int32_t>(m);
    const int64_t oe = g.e.out_f32 ? 4 : 2;
    s.a = static_cast<const uint8_t*>(g.a) + (AL ? i0 * g.lda : i0) * 2;
    s.e.out = static_cast<uint8_t*>(g.e.out) + i0 * g.e.ldo * oe;
    if (g.e.res) s.e.res = static_cast<const uint8_t*>(g.e.res) + i0 * g.e.ldr * oe;
    if (g.e.z) s.e.z = g.e.z + i0 * g.e.ldz;
    s.e.i0 += i0;
    return s;
}

// The product whole, or its two parts after a cut.
template <bool AL, bool BL, bool FP8>
int32_t run_direct(Product& g, const Space& space, hipStream_t stream, const char* who) {
    const Way best = best_way<BL>(g.extent(), space);
    if (best.us == kNoWay) return fail(FSDP_E_CAPACITY, "%s: more output tiles than one launch holds", who);
    const Cut cut = cut_of<BL>(g.extent(), best, space);
    if (cut.columns + cut.rows > 0) {
        const int64_t cj = cut.columns, ci = cut.rows;
        Product p = cj > 0 ? columns<BL>(g, FP8, 0, cj) : rows<AL>(g, 0, ci);
        Product q = cj > 0 ? columns<BL>(g, FP8, cj, g.n - cj) : rows<AL>(g, ci, g.m - ci);
        const int32_t st = run_direct<AL, BL, FP8>(p, space, stream, who);
        return st != FSDP_OK ? st : run_direct<AL, BL, FP8>(q, space, stream, who);
    }
    split(g, best.splits, space);
    if (best.tile == 256) return launch_product<256, 256, 2, 2, 1, AL, BL, true, FP8>(g, stream, who);
    if (best.tile == 128) return launch_product<128, 128, 2, 2, 1, AL, BL, true, FP8>(g, stream, who);
    return launch_product<64, 64, 1, 1, 4, AL, BL, true, FP8>(g, stream, who);
}

template <int MB, int JB>
int32_t launch_few(const Product& g, bool fp8, hipStream_t stream, const char* who) {
    const dim3 grid(static_cast<uint32_t>(ceil_div(g.n, 16 * JB))), block(kFewWaves * 64);
    const bool odd = !aligned(g.a, 4) || !aligned(g.b, 4) || g.lda % 2 != 0 || g.ldb % (fp8 ? 4 : 2) != 0;
    if (fp8 && odd) few_rows_kernel<MB, JB, true, true><<<grid, block, 0, stream>>>(g);
    else if (fp8) few_rows_kernel<MB, JB, true, false><<<grid, block, 0, stream>>>(g);
    else if (odd) few_rows_kernel<MB, JB, false, true><<<grid, block, 0, stream>>>(g);
    else few_rows_kernel<MB, JB, false, false><<<grid, block, 0, stream>>>(g);
    return launched(who);
}

template <int MB>
int32_t run_few(const Product& g, bool fp8, hipStream_t stream, const char* who) {
    const int best = few_features(g.m, g.n, fp8);
    if (ceil_div(g.n, 16 * best) > kMaxBlocks)
        return fail(FSDP_E_CAPACITY, "%s: more output tiles than one launch holds", who);
    switch (best) {
        case 1: return launch_few<MB, 1>(g, fp8, stream, who);
        case 2: return launch_few<MB, 2>(g, fp8, stream, who);
        case 3: return launch_few<MB, 3>(g, fp8, stream, who);
        default: return launch_few<MB, 4>(g, fp8, stream, who);
    }
}

Pack pack_of(const void* src, int64_t ld, int64_t rows, int64_t cols, bool fp8, void* dst) {
    return Pack{src, static_cast<uint8_t*>(dst), ld, static_cast<int32_t>(rows), static_cast<int32_t>(cols),
                static_cast<int32_t>(ceil_div(cols, fp8 ? 16 : 8)), static_cast<int32_t>(packed_row(cols, fp8)), fp8};
}

// The product with operands that are not as the direct loads want them.
template <bool AL, bool BL>
int32_t run_packed(const Product& g, bool fp8, bool a_ok, bool b_ok, const Space& whole, hipStream_t stream,
                   const char* who) {
    const Pieces p = pieces_of<AL, BL>(g.extent(), fp8, a_ok, b_ok, whole);
    if (p.rows == 0) {
        Product s = g;
        split(s, splits_for(128, 2 * kCus, s.extent(), whole), whole);
        if constexpr (AL) {
            if (fp8) return launch_product<128, 128, 2, 2, 1, AL, BL, false, true>(s, stream, who);
        }
        return launch_product<128, 128, 2, 2, 1, AL, BL, false, false>(s, stream, who);
    }
    Space space = whole;
    void* const pa = space.take(packed_bytes(a_ok, AL, p.rows, g.k, false));
    void* const pb = space.take(packed_bytes(b_ok, BL, p.cols, g.k, fp8));
    // That a piece's launch is possible is known before the first operand is laid out.
    if (best_way<BL>(columns_of(rows_of(g.extent(), p.rows), p.cols), space).us == kNoWay)
        return fail(FSDP_E_CAPACITY, "%s: more output tiles than one launch holds", who);
    const int64_t na = ceil_div(g.m, p.rows), nb = ceil_div(g.n, p.cols);
    int64_t has_a = -1, has_b = -1;  // the pieces that lie there
    for (int64_t t = 0; t < na * nb; ++t) {
        const int64_t ia = p.by_rows ? t / nb : t % na, ib = p.by_rows ? t % nb : t / na;
        const int64_t i0 = ia * p.rows, j0 = ib * p.cols;
        const int64_t m = std::min(p.rows, g.m - i0), n = std::min(p.cols, g.n - j0);
        Product s = columns<BL>(rows<AL>(g, i0, m), fp8, j0, n);
        Pack a{}, b{};
        int64_t blocks_a = 0, blocks_b = 0;
        if (!a_ok) {
            a = pack_of(s.a, g.lda, AL ? m : g.k, AL ? g.k : m, false, pa);
            if (ia != has_a) blocks_a = ceil_div(static_cast<int64_t>(a.rows) * a.chunks, kPackBlock);
            has_a = ia;
            s.a = pa;
            s.lda = a.pitch / 2;
        }
        if (!b_ok) {
            b = pack_of(s.b, g.ldb, BL ? n : g.k, BL ? g.k : n, fp8, pb);
            if (ib != has_b) blocks_b = ceil_div(static_cast<int64_t>(b.rows) * b.chunks, kPackBlock);
            has_b = ib;
            s.b = pb;
            s.ldb = b.pitch / (fp8 ? 1 : 2);
        }
        if (blocks_a + blocks_b > 0) {
            pack_kernel<<<dim3(static_cast<uint32_t>(blocks_a + blocks_b)), dim3(kPackBlock), 0, stream>>>(
                a, b, static_cast<int>(blocks_a));
            const int32_t st = launched(who);
            if (st != FSDP_OK) return st;
        }
        int32_t st;
        if constexpr (AL) st = fp8 ? run_direct<AL, BL, true>(s, space, stream, who) : run_direct<AL, BL, false>(s, space, stream, who);
        else st = run_direct<AL, BL, false>(s, space, stream, who);
        if (st != FSDP_OK) return st;
    }
    return FSDP_OK;
}

template <bool AL, bool BL>
int32_t run_product(Product& g, bool fp8, void* workspace, int64_t bytes, hipStream_t stream, const char* who) {
    if (g.m == 0 || g.n == 0) return FSDP_OK;
    g.pitch = (g.n + 7) / 8 * 8;
    g.e.n = g.n;
    // The stride of a single row says nothing; its length stands for it.
    if ((AL ? g.m : g.k) <= 1) g.lda = ((AL ? g.k : g.m) + 15) / 16 * 16;
    if ((BL ? g.n : g.k) <= 1) g.ldb = ((BL ? g.k : g.n) + 15) / 16 * 16;
    const Space space(workspace, bytes);
    const bool a_ok = direct_ok(g.a, g.lda, AL ? g.m : g.k, AL ? g.k : g.m, 8);
    const bool b_ok = direct_ok(g.b, g.ldb, BL ? g.n : g.k, BL ? g.k : g.n, fp8 ? 16 : 8);
    if constexpr (AL && BL) {
        if (few_tokens(g.m, a_ok, b_ok)) {
            g.splits = 1;
            return g.m <= 16 ? run_few<1>(g, fp8, stream, who) : run_few<2>(g, fp8, stream, who);
        }
    }
    if (a_ok && b_ok) {
        if constexpr (AL) {
            if (fp8) return run_direct<AL, BL, true>(g, space, stream, who);
        }
        return run_direct<AL, BL, false>(g, space, stream, who);
    }
    return run_packed<AL, BL>(g, fp8, a_ok, b_ok, space, stream, who);
}

int32_t check_weight(int32_t w_dtype, const float* w_scale, const char* who) {
    if (w_dtype != FSDP_DT_BF16 && w_dtype != FSDP_DT_E4M3)
        return fail(FSDP_E_DTYPE, "%s: weights are bf16 or E4M3", who);
    if (w_dtype == FSDP_DT_E4M3 && !w_scale) return fail(FSDP_E_ARG, "%s: E4M3 weights need w_scale", who);
    if (w_dtype == FSDP_DT_BF16 && w_scale) return fail(FSDP_E_ARG, "%s: w_scale is for E4M3 weights", who);
    if (!aligned(w_scale, 4)) return fail(FSDP_E_ALIGN, "%s: w_scale misaligned", who);
    return FSDP_OK;
}

int32_t check_act(int32_t act, const char* who) {
    if (act < FSDP_ACT_NONE || act > FSDP_ACT_SILU) return fail(FSDP_E_ARG, "%s: unknown activation", who);
    return FSDP_OK;
}

int32_t check_flag(int32_t v, const char* what, const char* who) {
    if (v != 0 && v != 1) return fail(FSDP_E_ARG, "%s: %s must be 0 or 1", who, what);
    return FSDP_OK;
}

int32_t check_float_dtype(int32_t d, const char* what, const char* who) {
    if (d != FSDP_DT_F32 && d != FSDP_DT_BF16) return fail(FSDP_E_DTYPE, "%s: %s must be fp32 or bf16", who, what);
    return FSDP_OK;
}

#define TRY(x)                                     \
    do {                                           \
        const int32_t st_ = (x);                   \
        if (st_ != FSDP_OK) return st_;            \
    } while (0)

int32_t forward_impl(const fsdp_linear* a, hipStream_t stream) {
    const char* who = "fsdp_linear_forward";
    if (!a) return fail(FSDP_E_ARG, "%s: null argument", who);
    if (a->reserved != 0) return fail(FSDP_E_ARG, "%s: reserved must be 0", who);
    TRY(check_sizes(a->m, a->n, a->k, who));
    TRY(check_weight(a->w_dtype, a->w_scale, who));
    TRY(check_float_dtype(a->y_dtype, "y", who));
    TRY(check_act(a->act, who));
    TRY(check_workspace(a->workspace, a->workspace_bytes, who));
    const int we = a->w_dtype == FSDP_DT_BF16 ? 2 : 1, ye = a->y_dtype == FSDP_DT_BF16 ? 2 : 4;
    const Matrix x{a->x, a->m, a->k, a->ldx, 2, "x", false}, w{a->w, a->n, a->k, a->ldw, we, "w", false};
    const Matrix y{a->y, a->m, a->n, a->ldy, ye, "y", true}, z{a->z, a->m, a->n, a->ldz, 2, "z", true};
    const Matrix r{a->residual, a->m, a->n, a->ldr, ye, "residual", false};
    const Matrix b = vector(a->bias, a->n, 2, "bias");
    TRY(check_matrix(x, false, who));
    TRY(check_matrix(w, false, who));
    TRY(check_matrix(y, false, who));
    TRY(check_matrix(z, true, who));
    TRY(check_matrix(r, true, who));
    TRY(check_matrix(b, true, who));
    Product g{};
    TRY(make_mask(a->dropout, &g.e.mask, who));
    TRY(check_overlaps({y, z, workspace_of(a->workspace, a->workspace_bytes), x, w, r, b, bytes_of(a->w_scale, 4, "w_scale", false),
                        bytes_of(g.e.mask.offset_dev, 8, "offset_dev", false)},
                       who, [&](const Matrix& p, const Matrix& q) { return p.what == y.what && q.what == r.what; }));
    g.a = a->x;
    g.b = a->w;
    g.lda = a->ldx;
    g.ldb = a->ldw;
    g.m = static_cast<int32_t>(a->m);
    g.n = static_cast<int32_t>(a->n);
    g.k = static_cast<int32_t>(a->k);
    g.e.out = a->y;
    g.e.ldo = a->ldy;
    g.e.out_f32 = a->y_dtype == FSDP_DT_F32;
    g.e.res = a->residual;
    g.e.ldr = a->ldr;
    g.e.z = a->z;
    g.e.ldz = a->ldz;
    g.e.bias = a->bias;
    g.e.scale = a->w_scale;
    g.e.act = a->act;
    return run_product<true, true>(g, we == 1, a->workspace, a->workspace_bytes, stream, who);
}

int32_t grad_input_impl(uint16_t* dx, int64_t lddx, const uint16_t* dz, int64_t lddz, const void* w, int64_t ldw,
                        int32_t w_dtype, const float* w_scale, int64_t m, int64_t n, int64_t k, void* workspace,
                        int64_t workspace_bytes, hipStream_t stream) {
    const char* who = "fsdp_linear_grad_input";
    TRY(check_sizes(m, n, k, who));
    TRY(check_weight(w_dtype, w_scale, who));
    TRY(check_workspace(workspace, workspace_bytes, who));
    const int we = w_dtype == FSDP_DT_BF16 ? 2 : 1;
    const Matrix x{dx, m, k, lddx, 2, "dx", true}, z{dz, m, n, lddz, 2, "dz", false}, wm{w, n, k, ldw, we, "w", false};
    TRY(check_matrix(x, false, who));
    TRY(check_matrix(z, false, who));
    TRY(check_matrix(wm, false, who));
    TRY(check_overlaps({x, workspace_of(workspace, workspace_bytes), z, wm, bytes_of(w_scale, 4, "w_scale", false)}, who,
                       [](const Matrix&, const Matrix&) { return false; }));
    Product g{};
    g.a = dz;
    g.b = w;
    g.lda = lddz;
    g.ldb = ldw;
    g.m = static_cast<int32_t>(m);
    g.n = static_cast<int32_t>(k);
    g.k = static_cast<int32_t>(n);
    g.e.out = dx;
    g.e.ldo = lddx;
    g.e.scale = w_scale;
    g.e.mask.scale = 1.0f;
    return run_product<true, false>(g, we == 1, workspace, workspace_bytes, stream, who);
}

int32_t grad_weight_impl(void* dw, int64_t lddw, int32_t dw_dtype, int32_t accumulate, const uint16_t* dz,
                         int64_t lddz, const uint16_t* x, int64_t ldx, int64_t m, int64_t n, int64_t k,
                         void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    const char* who = "fsdp_linear_grad_weight";
    TRY(check_sizes(m, n, k, who));
    TRY(check_float_dtype(dw_dtype, "dw", who));
    TRY(check_flag(accumulate, "accumulate", who));
    TRY(check_workspace(workspace, workspace_bytes, who));
    const int we = dw_dtype == FSDP_DT_BF16 ? 2 : 4;
    const Matrix d{dw, n, k, lddw, we, "dw", true}, z{dz, m, n, lddz, 2, "dz", false}, xm{x, m, k, ldx, 2, "x", false};
    TRY(check_matrix(d, false, who));
    TRY(check_matrix(z, false, who));
    TRY(check_matrix(xm, false, who));
    TRY(check_overlaps({d, workspace_of(workspace, workspace_bytes), z, xm}, who,
                       [](const Matrix&, const Matrix&) { return false; }));
    Product g{};
    g.a = dz;
    g.b = x;
    g.lda = lddz;
    g.ldb = ldx;
    g.m = static_cast<int32_t>(n);
    g.n = static_cast<int32_t>(k);
    g.k = static_cast<int32_t>(m);
    g.e.out = dw;
    g.e.ldo = lddw;
    g.e.out_f32 = dw_dtype == FSDP_DT_F32;
    g.e.res = accumulate ? dw : nullptr;
    g.e.ldr = lddw;
    g.e.mask.scale = 1.0f;
    return run_product<false, false>(g, false, workspace, workspace_bytes, stream, who);
}

// ---------------------------------------------------------------- host: elementwise passes

// Whether rows take written-through stores: 16-byte boundaries, and 64 rows
// within the 31 bits of a buffer offset.
bool stream_ok(const void* p, int64_t ld, int elem) {
    return aligned(p, 16) && ld * elem % 16 == 0 && ld <= (int64_t(1) << 22);
}

// chunks: 16-byte ones of a row; rows_max: the most row blocks wanted.
Grid elementwise_grid(int64_t m, int64_t chunks, int64_t rows_max, int64_t* blocks) {
    Grid g{};
    while (g.tx < 6 && (int64_t(1) << g.tx) < chunks) ++g.tx;
    g.cblocks = static_cast<int32_t>(ceil_div(chunks, int64_t(1) << g.tx));
    const int64_t per = kElemBlock >> g.tx;
    g.rows = std::max<int64_t>(1, ceil_div(ceil_div(m, per), std::max<int64_t>(1, rows_max))) * per;
    *blocks = ceil_div(m, g.rows);
    return g;
}

// Rows up to which one workgroup takes a column block's whole height.  333 x
// 1024: 6.5 us, by row blocks and a second launch 9.0; 600 x 4096: 11.7 and 10.7.
constexpr int64_t kTallRows = 512;

int32_t epilogue_backward_impl(uint16_t* dz, int64_t lddz, void* db, int32_t db_dtype, int32_t accumulate,
                               const uint16_t* dy, int64_t lddy, const uint16_t* z, int64_t ldz, int32_t act,
                               const fsdp_dropout_mask* dropout, int64_t m, int64_t n, void* workspace,
                               int64_t workspace_bytes, hipStream_t stream) {
    const char* who = "fsdp_linear_epilogue_backward";
    TRY(check_sizes(m, n, 0, who));
    TRY(check_act(act, who));
    TRY(check_float_dtype(db_dtype, "db", who));
    TRY(check_flag(accumulate, "accumulate", who));
    TRY(check_workspace(workspace, workspace_bytes, who));
    const int be = db_dtype == FSDP_DT_BF16 ? 2 : 4;
    const Matrix mdz{dz, m, n, lddz, 2, "dz", true}, mdy{dy, m, n, lddy, 2, "dy", false};
    const Matrix mz{act == FSDP_ACT_NONE ? nullptr : z, m, n, ldz, 2, "z", false}, mdb = vector(db, n, be, "db", true);
    TRY(check_matrix(mdz, true, who));
    TRY(check_matrix(mdy, false, who));
    TRY(check_matrix(mz, act == FSDP_ACT_NONE, who));
    TRY(check_matrix(mdb, true, who));
    BackwardArgs a{};
    TRY(make_mask(dropout, &a.mask, who));
    TRY(check_overlaps({mdz, mdb, workspace_of(workspace, workspace_bytes), mdy, mz,
                        bytes_of(a.mask.offset_dev, 8, "offset_dev", false)},
                       who, [&](const Matrix& p, const Matrix& q) {
                           return p.what == mdz.what && (q.what == mdy.what || q.what == mz.what);
                       }));
    if (n == 0 || (m == 0 && (!db || accumulate))) return FSDP_OK;
    if (!dz && !db) return FSDP_OK;
    a.dz = dz;
    a.dy = dy;
    a.z = z;
    a.lddz = lddz;
    a.lddy = lddy;
    a.ldz = ldz;
    a.m = m;
    a.n = n;
    a.db = db;
    a.db_f32 = db_dtype == FSDP_DT_F32;
    a.accumulate = accumulate;
    a.act = act;
    a.sums = db != nullptr;
    a.wt = stream_ok(dz, lddz, 2);
    if (db && m <= kTallRows && n <= 32 * (kMaxBlocks / 2)) {
        a.g = Grid{2, static_cast<int32_t>(ceil_div(n, 32)), kTallRows};
        epilogue_backward_kernel<kTallBlock><<<dim3(static_cast<uint32_t>(a.g.cblocks)), dim3(kTallBlock), 0, stream>>>(a);
        return launched(who);
    }
    const int64_t cblocks = ceil_div(ceil_div(n, 8), 64);
    // 24 workgroups a CU: 59 us for 4096 x 11008; 16 take 62, 8 66, 32 64
    int64_t want = 24 * kCus / cblocks;
    if (db) want = std::min(want, std::min(workspace_bytes, FSDP_LINEAR_WORKSPACE_BYTES) / (4 * n));
    int64_t blocks;
    a.g = elementwise_grid(m, ceil_div(n, 8), std::max<int64_t>(1, want), &blocks);
    a.part = db && blocks > 1 ? static_cast<float*>(workspace) : nullptr;
    if (blocks * a.g.cblocks > kMaxBlocks) return fail(FSDP_E_CAPACITY, "%s: more blocks than one launch holds", who);
    epilogue_backward_kernel<kElemBlock><<<dim3(static_cast<uint32_t>(blocks * a.g.cblocks)), dim3(kElemBlock), 0, stream>>>(a);
    TRY(launched(who));
    if (!a.part) return FSDP_OK;
    column_sum_kernel<<<dim3(static_cast<uint32_t>(ceil_div(n, 64))), dim3(kSumBlock), 0, stream>>>(
        a.part, n, static_cast<int32_t>(blocks), db, a.db_f32, accumulate);
    return launched(who);
}

int32_t dropout_impl(void* y, int64_t ldy, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                     int32_t dtype, int64_t rows, int64_t cols, const fsdp_dropout_mask* mask, hipStream_t stream) {
    const char* who = "fsdp_dropout";
    TRY(check_sizes(rows, cols, 0, who));
    TRY(check_float_dtype(dtype, "dtype", who));
    if (!mask) return fail(FSDP_E_ARG, "%s: null mask", who);
    const int e = dtype == FSDP_DT_BF16 ? 2 : 4;
    const Matrix my{y, rows, cols, ldy, e, "y", true}, mx{x, rows, cols, ldx, e, "x", false};
    const Matrix mr{residual, rows, cols, ldr, e, "residual", false};
    TRY(check_matrix(my, false, who));
    TRY(check_matrix(mx, false, who));
    TRY(check_matrix(mr, true, who));
    DropoutArgs a{};
    TRY(make_mask(mask, &a.mask, who));
    TRY(check_overlaps({my, mx, mr, bytes_of(a.mask.offset_dev, 8, "offset_dev", false)}, who,
                       [&](const Matrix&, const Matrix& q) { return q.what == mx.what || q.what == mr.what; }));
    if (rows == 0 || cols == 0) return FSDP_OK;
    a.y = y;
    a.x = x;
    a.res = residual;
    a.ldy = ldy;
    a.ldx = ldx;
    a.ldr = ldr;
    a.m = rows;
    a.n = cols;
    a.wt = stream_ok(y, ldy, e);
    const int64_t chunks = ceil_div(cols, 16 / e);
    int64_t blocks;
    a.g = elementwise_grid(rows, chunks, 16 * kCus / ceil_div(chunks, 64), &blocks);
    if (blocks * a.g.cblocks > kMaxBlocks) return fail(FSDP_E_CAPACITY, "%s: more blocks than one launch holds", who);
    const dim3 grid(static_cast<uint32_t>(blocks * a.g.cblocks));
    if (e == 2) dropout_kernel<uint16_t><<<grid, dim3(kElemBlock), 0, stream>>>(a);
    else dropout_kernel<float><<<grid, dim3(kElemBlock), 0, stream>>>(a);
    return launched(who);
}

#undef TRY

}  // namespace

// ---------------------------------------------------------------- entry points

extern "C" int32_t fsdp_linear_forward(const fsdp_linear* a, hipStream_t stream) {
    return fsdp::guarded("fsdp_linear_forward", [&] { return forward_impl(a, stream); });
}

extern "C" int32_t fsdp_linear_epilogue_backward(uint16_t* dz, int64_t lddz, void* db, int32_t db_dtype,
                                                 int32_t accumulate, const uint16_t* dy, int64_t lddy,
                                                 const uint16_t* z, int64_t ldz, int32_t act,
                                                 const fsdp_dropout_mask* dropout, int64_t m, int64_t n,
                                                 void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    return fsdp::guarded("fsdp_linear_epilogue_backward", [&] {
        return epilogue_backward_impl(dz, lddz, db, db_dtype, accumulate, dy, lddy, z, ldz, act, dropout, m, n,
                                      workspace, workspace_bytes, stream);
    });
}

extern "C" int32_t fsdp_linear_grad_input(uint16_t* dx, int64_t lddx, const uint16_t* dz, int64_t lddz, const void* w,
                                          int64_t ldw, int32_t w_dtype, const float* w_scale, int64_t m, int64_t n,
                                          int64_t k, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    return fsdp::guarded("fsdp_linear_grad_input", [&] {
        return grad_input_impl(dx, lddx, dz, lddz, w, ldw, w_dtype, w_scale, m, n, k, workspace, workspace_bytes,
                               stream);
    });
}

extern "C" int32_t fsdp_linear_grad_weight(void* dw, int64_t lddw, int32_t dw_dtype, int32_t accumulate,
                                           const uint16_t* dz, int64_t lddz, const uint16_t* x, int64_t ldx,
                                           int64_t m, int64_t n, int64_t k, void* workspace, int64_t workspace_bytes,
                                           hipStream_t stream) {
    return fsdp::guarded("fsdp_linear_grad_weight", [&] {
        return grad_weight_impl(dw, lddw, dw_dtype, accumulate, dz, lddz, x, ldx, m, n, k, workspace, workspace_bytes,
                                stream);
    });
}

extern "C" int32_t fsdp_dropout(void* y, int64_t ldy, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                int32_t dtype, int64_t rows, int64_t cols, const fsdp_dropout_mask* mask,
                                hipStream_t stream) {
    return fsdp::guarded("fsdp_dropout",
                         [&] { return dropout_impl(y, ldy, x, ldx, residual, ldr, dtype, rows, cols, mask, stream); });
}
