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

// One operand's tile of W rows of a step, 128 bytes each, from memory to LDS as
// DirectTile's l-major ones.  Chunk c of a row, block c, goes to the place of
// bits (c0 c2 c1), then permuted by the row: lane group g of a matrix instruction
// reads blocks 2g and 2g + 1, one after the other, and with neighbouring groups
// at neighbouring places its reads meet no bank twice.
template <int W, int THREADS>
struct Mx4Tile {
    static constexpr int kLoads = W * 8 / THREADS;
    const uint8_t* base;  // the tile's first row at this step
    int left;             // bytes of a row from here to the end, may be negative
    int at;               // this thread's chunk in a row (the same in all its loads)
    uint32_t off[kLoads];

    __device__ __forceinline__ void init(const void* p, int64_t ld, int o0, int no, int l0, int lend, int tid) {
        const int row = static_cast<int>(ld * 2), place = (tid & 7) ^ (tid >> 3 & 7);
        left = (lend - l0) * 2;
        base = static_cast<const uint8_t*>(p) + o0 * (ld * 2) + static_cast<int64_t>(l0) * 2;
        at = ((place & 3) << 1 | place >> 2) * 16;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = (i * THREADS + tid) / 8;
            off[i] = o0 + r < no ? static_cast<uint32_t>(r * row + at) : kOutside;
        }
    }
    __device__ __forceinline__ void load(Lds* dst, int wave, int q) {
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, 0x7fffffff, 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void*)(dst + (q * THREADS + wave * 64) * 16), 16,
            at < left ? off[q] : kOutside, 0, 0, 0);
    }
    __device__ __forceinline__ void advance() {
        base += 128;
        left -= 128;
    }
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
            base[q] = (of_a ? g.sa : g.sb) + first * ld + lbeg / 8;  // the same in the whole wave
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

// acc += the 16x16 product of two fragments over 128 elements; KK: which byte of
// the scale registers.  In assembly for its register classes, as mfma() above.
template <int KK>
__device__ __forceinline__ void mx4_mfma(f32x4& acc, const u32x4& b, const u32x4& a, uint32_t sb, uint32_t sa) {
    if constexpr (KK == 0)
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[0,0,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                     : "+a"(acc) : "v"(b), "v"(a), "v"(sb), "v"(sa));
    else
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                     : "+a"(acc) : "v"(b), "v"(a), "v"(sb), "v"(sa));
}

// f(0), ..., f(N - 1), each a constant.
template <typename F, int... I>
__device__ __forceinline__ void for_each_constant(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void for_constants(F&& f) {
    for_each_constant(f, std::make_integer_sequence<int, N>());
}
// f(q) for those of COUNT accesses that belong to slot T of N.
template <int COUNT, int T, int N, typename F>
__device__ __forceinline__ void for_slot(F&& f) {
    constexpr int kFirst = T * COUNT / N, kEnd = (T + 1) * COUNT / N;
    for_constants<kEnd - kFirst>([&](auto q) { f(std::integral_constant<int, kFirst + decltype(q)::value>()); });
}

// One lane's operands from a stage of W rows: of row o0 + lane mod 16 and every
// 16th behind it, block 2 (lane / 16) + kk, so that the two blocks that a lane
// takes of a stage are neighbours and their scales one 16-bit read.
template <int NF>
struct Mx4Fragments {
    int at, scale;

    __device__ __forceinline__ void init(int o0, int lane) {
        const int lo = lane & 15, g = lane >> 4;
        at = (o0 + lo) * 128 + ((g ^ (lo & 7)) << 4);
        scale = (o0 + lo) * 16 + 2 * g;
    }
    __device__ __forceinline__ u32x4 get(const Lds* tile, int f, int kk) const {
        return *(const __attribute__((address_space(3))) u32x4*)(tile + (at ^ (kk << 6)) + f * 2048);
    }
    // h: which stage of the two whose scales lie together
    __device__ __forceinline__ uint32_t get_scale(const Lds* scales, int f, int h) const {
        return *(const __attribute__((address_space(3))) uint16_t*)(scales + scale + f * 256 + h * 8);
    }
};

// Tiles, waves and stages as product_kernel's.  A step is 256 contraction
// elements; the scales of two steps come together, 16 bytes a row, into a
// buffer of their own, of which there are two as well.
template <int BM, int BN, int WI, int WJ, int KW>
__global__ __launch_bounds__(WI* WJ* KW * 64) void mx4_product_kernel(Mx4Product g) {
    static_assert(KW == 1 || (WI == 1 && WJ == 1 && BM == 64 && BN == 64), "waves with parts of the contraction");
    constexpr int kThreads = WI * WJ * 64, kWM = BM / WI, kWN = BN / WJ, kFI = kWM / 16, kFJ = kWN / 16;
    constexpr int kStage = (BM + BN) * 128, kScale = (BM + BN) * 16;
    constexpr bool kShared = KW == 1;  // the waves share their stages
    __shared__ __attribute__((aligned(1024))) uint8_t s0[kStage * KW];
    __shared__ __attribute__((aligned(1024))) uint8_t s1[kStage * KW];
    __shared__ __attribute__((aligned(1024))) uint8_t c0[kScale * KW];
    __shared__ __attribute__((aligned(1024))) uint8_t c1[kScale * KW];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tid = kShared ? threadIdx.x : lane;  // among the threads that fill a stage
    const int part = kShared ? 0 : wave, filler = kShared ? wave : 0;
    Lds* const l0 = (Lds*)s0 + part * kStage;
    Lds* const l1 = (Lds*)s1 + part * kStage;
    Lds* const e0 = (Lds*)c0 + part * kScale;
    Lds* const e1 = (Lds*)c1 + part * kScale;
    const int tiles = g.tm * g.tn;
    const int id = tile_id(blockIdx.x, tiles * g.splits);
    const int split = id / tiles;
    int ti, tj;
    tile_at(id - split * tiles, g.tm, g.tn, &ti, &tj);
    const int i0 = ti * BM, j0 = tj * BN;
    int lbeg = split * g.kper, lend = min(g.k, lbeg + g.kper);
    if (KW > 1) {
        const int per = (lend - lbeg + 2 * kBK * KW - 1) / (2 * kBK * KW) * (2 * kBK);
        lbeg += part * per;
        lend = min(lend, lbeg + per);
    }
    int turns = lend > lbeg ? (lend - lbeg + 2 * kBK - 1) / (2 * kBK) : 0;
    const int wi = kShared ? wave / WJ : 0, wj = kShared ? wave % WJ : 0;

    f32x4 acc[kFI][kFJ];
#pragma unroll
    for (int i = 0; i < kFI; ++i)
#pragma unroll
        for (int j = 0; j < kFJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    if (turns > 0) {
        Mx4Fragments<kFI> fa;
        Mx4Fragments<kFJ> fb;
        fa.init(wi * kWM, lane);
        fb.init(wj * kWN, lane);
        Mx4Tile<BM, kThreads> ta;
        Mx4Tile<BN, kThreads> tb;
        Mx4Scales<BM, BN, WI * WJ> ts;
        ta.init(g.a, g.lda, i0, g.m, lbeg, lend, tid);
        tb.init(g.b, g.ldb, j0, g.n, lbeg, lend, tid);
        ts.init(g, i0, j0, lbeg, lend, filler, lane);
        constexpr int kLoads = ta.kLoads + tb.kLoads, kSlots = kFI * kFJ;
        auto fetch = [&](Lds* stage, int q) {
            if (q < ta.kLoads) ta.load(stage, filler, q);
            else tb.load(stage + BM * 128, filler, q - ta.kLoads);
            if (q == kLoads - 1) {
                ta.advance();
                tb.advance();
            }
        };

        u32x4 a[2][kFI], b[2][kFJ];
        uint32_t sa[2][kFI], sb[2][kFJ];  // of this step and the next
        // What a half needs, in the order in which it needs it: fragments, and of a
        // step's first half the step's scales.
        auto read = [&](const Lds* stage, int kk, int f) {
            if (f < kFJ) b[kk][f] = fb.get(stage + BM * 128, f, kk);
            else a[kk][f - kFJ] = fa.get(stage, f - kFJ, kk);
        };
        auto read_scale = [&](const Lds* scales, int h, int p, int f) {
            if (f < kFJ) sb[p][f] = fb.get_scale(scales + BM * 16, f, h);
            else sa[p][f - kFJ] = fa.get_scale(scales, f - kFJ, h);
        };
        // Half KK of the step of parity p, product by product, with `between` (slot) in
        // each product's shadow.
        auto multiply = [&](auto kk, int p, auto&& between) {
            constexpr int KK = decltype(kk)::value;
            for_constants<kSlots>([&](auto slot) {
                constexpr int t = decltype(slot)::value;
                mx4_mfma<KK>(acc[t / kFJ][t % kFJ], b[KK][t % kFJ], a[KK][t / kFJ], sb[p][t % kFJ], sa[p][t / kFJ]);
                __builtin_amdgcn_sched_barrier(0);
                between(slot);
                __builtin_amdgcn_sched_barrier(0);
            });
        };
        // The step of parity p in `cur`; the next one is in `nxt`, with its scales the
        // half h of `scales`.  FILL: `more` takes the scales of the two steps from the
        // next but one on.
        auto step = [&](Lds* cur, Lds* nxt, int p, const Lds* scales, int h, auto fill, Lds* more) {
            constexpr int kReads = kFI + kFJ, kFills = kLoads + (decltype(fill)::value ? ts.kLoads : 0);
            multiply(std::integral_constant<int, 0>(), p, [&](auto slot) {
                for_slot<kReads, decltype(slot)::value, kSlots>([&](auto q) { read(cur, 1, decltype(q)::value); });
            });
            arrive<kShared>();
            multiply(std::integral_constant<int, 1>(), p, [&](auto slot) {
                constexpr int t = decltype(slot)::value;
                for_slot<2 * kReads, t, kSlots>([&](auto i) {
                    constexpr int q = decltype(i)::value;
                    if constexpr (q & 1) read_scale(scales, h, 1 - p, q / 2);
                    else read(nxt, 0, q / 2);
                });
                for_slot<kFills, t, kSlots>([&](auto i) {
                    constexpr int q = decltype(i)::value;
                    if constexpr (q < kLoads) fetch(cur, q);
                    else ts.load(more, filler, q - kLoads);
                });
            });
        };

#pragma unroll
        for (int q = 0; q < kLoads; ++q) fetch(l0, q);
#pragma unroll
        for (int q = 0; q < ts.kLoads; ++q) ts.load(e0, filler, q);
#pragma unroll
        for (int q = 0; q < kLoads; ++q) fetch(l1, q);
        arrive<kShared>();
        settle(acc);
#pragma unroll
        for (int f = 0; f < kFI + kFJ; ++f) {
            read(l0, 0, f);
            read_scale(e0, 0, 0, f);
        }
        // Four steps a turn of the loop, so that each LDS access names its buffer.  An
        // odd count takes one more step, over zeros.
        for (;;) {
            step(l0, l1, 0, e0, 1, std::true_type(), e1);
            step(l1, l0, 1, e1, 0, std::false_type(), e1);
            if (--turns <= 0) break;
            step(l0, l1, 0, e1, 1, std::true_type(), e0);
            step(l1, l0, 1, e0, 0, std::false_type(), e0);
            if (--turns <= 0) break;
        }
        settle(acc);
    }
    finish<BM, BN, WI, WJ, KW>(g, acc, l0, l1, (Lds*)s0, split, i0, j0, lane, wave);
}

// ---------------------------------------------------------------- host

template <int BM, int BN, int WI, int WJ, int KW>
int32_t launch_mx4(Mx4Product& g, hipStream_t stream, const char* who) {
    g.tm = static_cast<int32_t>(ceil_div(g.m, BM));
    g.tn = static_cast<int32_t>(ceil_div(g.n, BN));
    const int64_t blocks = static_cast<int64_t>(g.tm) * g.tn * g.splits;
    const int64_t joins = ceil_div(static_cast<int64_t>(g.m) * (g.pitch / 8), kJoinBlock);
    if (blocks > kMaxBlocks || (g.splits > 1 && joins > kMaxBlocks))
        return fail(FSDP_E_CAPACITY, "%s: more output tiles than one launch holds", who);
    mx4_product_kernel<BM, BN, WI, WJ, KW><<<dim3(static_cast<uint32_t>(blocks)), dim3(WI * WJ * KW * 64), 0, stream>>>(g);
    const int32_t st = launched(who);
    if (st != FSDP_OK || g.splits == 1) return st;
    join_kernel<<<dim3(static_cast<uint32_t>(joins)), dim3(kJoinBlock), 0, stream>>>(g);
    return launched(who);
}

// The product whole, or its two parts after a cut.
int32_t run_mx4(Mx4Product& g, const Space& space, hipStream_t stream, const char* who) {
    const Way best = mx4_best_way(g.extent(), space);
    if (best.us == kNoWay) return fail(FSDP_E_CAPACITY, "%s: more output tiles than one launch holds", who);
    const Parts p = mx4_parts_of(g.k, best.splits);
    g.splits = p.n;
    g.kper = p.k;
    g.part = reinterpret_cast<float*>(space.p);
    if (best.tile == 256) return launch_mx4<256, 256, 2, 2, 1>(g, stream, who);
    if (best.tile == 128) return launch_mx4<128, 128, 2, 2, 1>(g, stream, who);
    return launch_mx4<64, 64, 1, 1, 4>(g, stream, who);
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
    return run_mx4(g, Space(a->workspace, a->workspace_bytes), stream, who);
}

}  // namespace
