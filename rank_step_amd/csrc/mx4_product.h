// The product of two 4-bit matrices (include/fsdp_mx4.h).  Part of linear.hip's
// translation unit, with whose products it shares tiles, epilogue and join.
//
// Every product is C(i, j) = sum_l A(i, l) B(j, l), and both operands' rows run
// along l.  One scaled matrix instruction multiplies 16 x 16 outputs over 128
// contraction elements, four blocks: its lane takes 16 bytes of each operand, a
// block, and that block's scale byte.  That is as many bytes a lane and as many
// cycles as of the bf16 instruction over 32 elements, so the tiles are those of
// the bf16 product with blocks in the place of 8 elements: a stage of kBK 16-bit
// units is 128 bytes of a row, 8 blocks.
#pragma once

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Mx4Product : Product {
    const uint8_t* sa;
    const uint8_t* sb;
    int64_t ldsa, ldsb;
};

// LDS scales of a tile: 16 bytes a row, A's rows and then B's, for two stages.
// 64 rows are one load of a wave; PARTS waves share them.
template <int BM, int BN, int PARTS>
struct Mx4Scales {
    static constexpr int kLoads = (BM + BN) / 64 / PARTS;
    const uint8_t* base[kLoads];
    uint32_t off[kLoads];
    int left;  // bytes from here to the end of this part's scales, may be negative

    __device__ __forceinline__ void init(const Mx4Product& g, int i0, int j0, int lbeg, int lend, int part, int lane) {
        left = (lend - lbeg + 7) / 8;
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int row = (q * PARTS + part) * 64;
            const bool of_a = row < BM;
            const int first = of_a ? i0 + row : j0 + row - BM, rows = of_a ? g.m : g.n;
            const int64_t ld = of_a ? g.ldsa : g.ldsb;
            base[q] = (of_a ? g.sa : g.sb) + first * ld + lbeg / 8;
            off[q] = first + lane < rows ? static_cast<uint32_t>(lane * static_cast<int>(ld)) : kOutside;
        }
    }
    // What is outside comes as zeros: 2^-127, of codes that are zero as well.
    __device__ __forceinline__ void load(Lds* dst, int part, int q) {
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base[q]), 0, 0x7fffffff, 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void*)(dst + (q * PARTS + part) * 1024), 16, left > 0 ? off[q] : kOutside, 0, 0, 0);
        if (q == kLoads - 1) {
            left -= 16;
#pragma unroll
            for (int p = 0; p < kLoads; ++p) base[p] += 16;
        }
    }
};

__device__ __forceinline__ i32x8 mx4_operand(const u32x4& v) {
    return i32x8{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]), static_cast<int>(v[3]), 0, 0, 0, 0};
}

// A lane's 16 bytes of row o0 + lane mod 16 from a stage: block 2 (lane / 16) + kk.
__device__ __forceinline__ u32x4 mx4_fragment(const Lds* tile, int row, int g, int kk) {
    return *(const __attribute__((address_space(3))) u32x4*)(tile + row * 128 + (((2 * g + kk) ^ (row & 7)) << 4));
}

template <int BM, int BN, int WI, int WJ>
__global__ __launch_bounds__(WI* WJ * 64) void mx4_product_kernel(Mx4Product g) {
    constexpr int kThreads = WI * WJ * 64, kWM = BM / WI, kWN = BN / WJ, kFI = kWM / 16, kFJ = kWN / 16;
    constexpr int kStage = (BM + BN) * 128;
    __shared__ __attribute__((aligned(1024))) uint8_t s0[kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t s1[kStage];
    __shared__ __attribute__((aligned(1024))) uint8_t c0[(BM + BN) * 16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = g.tm * g.tn;
    const int id = tile_id(blockIdx.x, tiles * g.splits);
    const int split = id / tiles;
    int ti, tj;
    tile_at(id - split * tiles, g.tm, g.tn, &ti, &tj);
    const int i0 = ti * BM, j0 = tj * BN;
    const int lbeg = split * g.kper, lend = min(g.k, lbeg + g.kper);
    const int wi = wave / WJ, wj = wave % WJ, lo = lane & 15, hi = lane >> 4;
    f32x4 acc[kFI][kFJ];
#pragma unroll
    for (int i = 0; i < kFI; ++i)
#pragma unroll
        for (int j = 0; j < kFJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    DirectTile<BM, kThreads, true, 8> ta;
    DirectTile<BN, kThreads, true, 8> tb;
    Mx4Scales<BM, BN, WI * WJ> ts;
    ta.init(g.a, g.lda, i0, g.m, lbeg, lend, threadIdx.x);
    tb.init(g.b, g.ldb, j0, g.n, lbeg, lend, threadIdx.x);
    ts.init(g, i0, j0, lbeg, lend, wave, lane);
    Lds* const stages[2] = {(Lds*)s0, (Lds*)s1};
    for (int l = lbeg; l < lend; l += 2 * kBK) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int q = 0; q < ta.kLoads; ++q) ta.load(stages[h], wave, q);
#pragma unroll
            for (int q = 0; q < tb.kLoads; ++q) tb.load(stages[h] + BM * 128, wave, q);
            ta.advance();
            tb.advance();
        }
#pragma unroll
        for (int q = 0; q < ts.kLoads; ++q) ts.load((Lds*)c0, wave, q);
        arrive<true>();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            i32x8 a[2][kFI], b[2][kFJ];
            int sa[kFI], sb[kFJ];
            auto scale = [&](int row) {
                return static_cast<int>(*(const __attribute__((address_space(3))) uint16_t*)((Lds*)c0 + row * 16 + h * 8 + hi * 2));
            };
#pragma unroll
            for (int i = 0; i < kFI; ++i) {
                const int row = wi * kWM + i * 16 + lo;
                a[0][i] = mx4_operand(mx4_fragment(stages[h], row, hi, 0));
                a[1][i] = mx4_operand(mx4_fragment(stages[h], row, hi, 1));
                sa[i] = scale(row);
            }
#pragma unroll
            for (int j = 0; j < kFJ; ++j) {
                const int row = wj * kWN + j * 16 + lo;
                b[0][j] = mx4_operand(mx4_fragment(stages[h] + BM * 128, row, hi, 0));
                b[1][j] = mx4_operand(mx4_fragment(stages[h] + BM * 128, row, hi, 1));
                sb[j] = scale(BM + row);
            }
#pragma unroll
            for (int i = 0; i < kFI; ++i)
#pragma unroll
                for (int j = 0; j < kFJ; ++j) {
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[0][j], a[0][i], acc[i][j], 4, 4, 0, sb[j], 0, sa[i]);
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[1][j], a[1][i], acc[i][j], 4, 4, 1, sb[j], 1, sa[i]);
                }
        }
        arrive<true>();
    }
    finish<BM, BN, WI, WJ, 1>(g, acc, (Lds*)s0, (Lds*)s1, (Lds*)s0, split, i0, j0, lane, wave);
}

// ---------------------------------------------------------------- host

template <int BM, int BN, int WI, int WJ>
int32_t launch_mx4(Mx4Product& g, hipStream_t stream, const char* who) {
    g.tm = static_cast<int32_t>(ceil_div(g.m, BM));
    g.tn = static_cast<int32_t>(ceil_div(g.n, BN));
    const int64_t blocks = static_cast<int64_t>(g.tm) * g.tn * g.splits;
    const int64_t joins = ceil_div(static_cast<int64_t>(g.m) * (g.pitch / 8), kJoinBlock);
    if (blocks > kMaxBlocks || (g.splits > 1 && joins > kMaxBlocks))
        return fail(FSDP_E_CAPACITY, "%s: more output tiles than one launch holds", who);
    mx4_product_kernel<BM, BN, WI, WJ><<<dim3(static_cast<uint32_t>(blocks)), dim3(WI * WJ * 64), 0, stream>>>(g);
    const int32_t st = launched(who);
    if (st != FSDP_OK || g.splits == 1) return st;
    join_kernel<<<dim3(static_cast<uint32_t>(joins)), dim3(kJoinBlock), 0, stream>>>(g);
    return launched(who);
}

int32_t mx4_product_impl(const fsdp_mx4_operands* a, hipStream_t stream) {
    const char* who = "fsdp_mx4_product";
    if (!a) return fail(FSDP_E_ARG, "%s: null argument", who);
    TRY(check_sizes(a->m, a->n, a->k, who));
    TRY(check_float_dtype(a->y_dtype, "y", who));
    TRY(check_act(a->act, who));
    TRY(check_workspace(a->workspace, a->workspace_bytes, who));
    const int ye = a->y_dtype == FSDP_DT_BF16 ? 2 : 4;
    const Mx4Matrix ma = mx4_matrix(a->a, a->lda, "a", a->a_scales, a->ldas, "a_scales", a->m, a->k, false);
    const Mx4Matrix mb = mx4_matrix(a->b, a->ldb, "b", a->b_scales, a->ldbs, "b_scales", a->n, a->k, false);
    const Matrix y{a->y, a->m, a->n, a->ldy, ye, "y", true}, z{a->z, a->m, a->n, a->ldz, 2, "z", true};
    const Matrix r{a->residual, a->m, a->n, a->ldr, ye, "residual", false}, b = vector(a->bias, a->n, 2, "bias");
    TRY(check_mx4(ma, who));
    TRY(check_mx4(mb, who));
    TRY(check_matrix(y, false, who));
    for (const Matrix& x : {z, r, b}) TRY(check_matrix(x, true, who));
    Mx4Product g{};
    TRY(make_mask(a->dropout, &g.e.mask, who));
    TRY(check_overlaps({y, z, bytes_of(a->workspace, std::min(a->workspace_bytes, FSDP_MX4_WORKSPACE_BYTES), "workspace", true),
                        ma.codes, ma.scales, mb.codes, mb.scales, r, b, bytes_of(g.e.mask.offset_dev, 8, "offset_dev", false)},
                       who, [&](const Matrix& p, const Matrix& q) { return p.what == y.what && q.what == r.what; }));
    if (a->m == 0 || a->n == 0) return FSDP_OK;
    // The stride of a single row says nothing; its length stands for it.
    const int64_t codes = FSDP_MX4_CODE_BYTES(a->k), scales = FSDP_MX4_SCALE_BYTES(a->k);
    const int64_t lda = a->m > 1 ? a->lda : codes, ldb = a->n > 1 ? a->ldb : codes;
    g.ldsa = a->m > 1 ? a->ldas : scales;
    g.ldsb = a->n > 1 ? a->ldbs : scales;
    for (int64_t ld : {lda, ldb, g.ldsa, g.ldsb})
        if (ld > kMaxMx4Stride) return fail(FSDP_E_CAPACITY, "%s: rows of 4-bit codes or scales more than 2^22 bytes apart", who);
    g.a = a->a;
    g.b = a->b;
    g.sa = a->a_scales;
    g.sb = a->b_scales;
    g.lda = lda / 2;
    g.ldb = ldb / 2;
    g.m = static_cast<int32_t>(a->m);
    g.n = static_cast<int32_t>(a->n);
    g.k = static_cast<int32_t>(codes / 2);
    g.pitch = (g.n + 7) / 8 * 8;
    g.e.n = g.n;
    g.e.out = a->y;
    g.e.ldo = a->ldy;
    g.e.out_f32 = ye == 4;
    g.e.res = a->residual;
    g.e.ldr = a->ldr;
    g.e.z = a->z;
    g.e.ldz = a->ldz;
    g.e.bias = a->bias;
    g.e.act = a->act;
    g.splits = 1;
    g.kper = g.k;
    return launch_mx4<128, 128, 2, 2>(g, stream, who);
}

}  // namespace
