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

typedef short s16x2 __attribute__((ext_vector_type(2)));

struct Mx4Product : Product {
    const uint8_t* sa;
    const uint8_t* sb;
    int64_t ldsa, ldsb;
};

// One operand's tile of W rows of a step, 128 bytes each, from memory to LDS.
// Chunk c of a row, block c, goes to the place of bits (c0 c2 c1), then permuted
// by the row: lane group g of a matrix instruction reads blocks 2g and 2g + 1, one
// after the other, and with neighbouring groups at neighbouring places its
// reads meet no bank twice (with the blocks in their order 8192 x 28672 x 8192 had
// five times the conflict cycles).
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
        end();
    }
    // Behind the row's end no load touches memory: the chunks that lie there, and
    // lie there from then on, are sent out of range.
    __device__ __forceinline__ void end() {
        if (__builtin_expect(left < 128, 0) && at >= left) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) off[i] = kOutside;
        }
    }
    __device__ __forceinline__ void load(Lds* dst, int wave, int q) {
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, 0x7fffffff, 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rsrc, (__attribute__((address_space(3))) void*)(dst + (q * THREADS + wave * 64) * 16), 16, off[q], 0, 0, 0);
        if (q == kLoads - 1) {
            base += 128;
            left -= 128;
            end();
        }
    }
};

// LDS scales of a tile: 16 bytes a row, A's rows and then B's, for two steps.
// 64 rows are one load of a wave; PARTS waves share them.
template <int BM, int BN, int PARTS>
struct Mx4Scales {
    static constexpr int kLoads = (BM + BN) / 64 / PARTS;
    const uint8_t* base[kLoads];  // each the same in the whole wave
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

// acc += the 16x16 product of two fragments over 128 elements; KK: which byte of
// the scale registers.  In assembly for its register classes, as mfma() above.
template <int KK>
__device__ __forceinline__ void mx4_mfma(f32x4& acc, const u32x4& b, const u32x4& a, s16x2 sb, s16x2 sa) {
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

// One lane's operands from a stage: of row o0 + lane mod 16 and every 16th behind
// it, block 2 (lane / 16) + kk, so that the two blocks that a lane takes of a step
// are neighbours and their scales one 16-bit read.
struct Mx4Fragments {
    int at, scale;

    // slot: the row's among the scales
    __device__ __forceinline__ void init(int o0, int slot, int lane) {
        const int lo = lane & 15, g = lane >> 4;
        at = (o0 + lo) * 128 + ((g ^ (lo & 7)) << 4);
        scale = (slot + lo) * 16 + 2 * g;
    }
    __device__ __forceinline__ u32x4 get(const Lds* tile, int f, int kk) const {
        return *(const __attribute__((address_space(3))) u32x4*)(tile + (at ^ (kk << 6)) + f * 2048);
    }
    // h: which of the two steps whose scales lie together.  The upper half of the
    // register is not used, and left to whatever it holds.
    __device__ __forceinline__ s16x2 get_scale(const Lds* scales, int f, int h) const {
        s16x2 v;
        v[0] = *(const __attribute__((address_space(3))) short*)(scales + scale + f * 256 + h * 8);
        return v;
    }
};

// All but the newest LOADS loads of this wave have come, and all but the newest
// READS of its LDS reads; SHARED: of every wave of the workgroup.
template <bool SHARED, int LOADS, int READS>
__device__ __forceinline__ void mx4_arrive() {
    static_assert(LOADS < 64 && READS < 16, "the counters' ranges");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(%1)" ::"i"(LOADS), "i"(READS) : "memory");
    if (SHARED) {
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }
}
// All its LDS reads have.
template <bool SHARED>
__device__ __forceinline__ void mx4_read() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (SHARED) {
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }
}

// A wave's sums, to memory (a split's part) or through the epilogue: 64 rows at a
// time through a piece of LDS of its own, 64 rows of FJ * 64 bytes, so that a lane
// has 8 consecutive columns and a store takes whole lines.  (Exchanged between
// lanes without LDS, which gives 64 bytes a row and store, it took 274 us of
// 8192 x 28672 x 8192, this way 105.)  A row's 16-byte chunks are permuted by the
// row, which spreads the 16 rows that one write touches over the banks.  fp32
// outputs, of which a lane's two stores are each half of its 32 bytes, with
// ordinary stores: 8192 x 8192 x 4096 181 us, non-temporal 239 (bf16 the other way:
// 8192 x 28672 x 8192 870 and 910).
template <int FI, int FJ>
__device__ __forceinline__ void mx4_finish(const Product& g, f32x4 (&acc)[FI][FJ], Lds* piece, int split, int i0, int j0, int lane) {
    using Quad = __attribute__((address_space(3))) f32x4;
    constexpr int kRow = FJ * 64, kLanes = FJ * 2, kBatch = 4, kStep = 64 / kLanes;
    // Lane l holds of each 16x16 block output row l mod 16 and columns 4 (l / 16) + 0..3.
    const int lo = lane & 15, hi = lane >> 4;
    if (g.splits > 1) {
        float* const sums = g.part + static_cast<int64_t>(split) * g.m * g.pitch;
#pragma unroll
        for (int i = 0; i < FI; ++i) {
            const int row = i0 + i * 16 + lo;
#pragma unroll
            for (int j = 0; j < FJ; ++j) {
                const int col = j0 + j * 16 + hi * 4;
                if (row < g.m && col < g.pitch)
                    *reinterpret_cast<f32x4*>(sums + static_cast<int64_t>(row) * g.pitch + col) = acc[i][j];
            }
        }
        return;
    }
    const uint64_t off = mask_offset(g.e.mask);
    const int c = lane % kLanes, col = j0 + c * 8;
#pragma unroll
    for (int h = 0; h < FI / 4; ++h) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < FJ; ++j) *(Quad*)(piece + (i * 16 + lo) * kRow + (((j * 4 + hi) ^ lo) << 4)) = acc[h * 4 + i][j];
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int r = lane / kLanes; r < 64; r += kBatch * kStep) {
            float v[kBatch][8];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int rq = r + q * kStep;
                const f32x4 x = *(const Quad*)(piece + rq * kRow + (((c * 2) ^ (rq & 15)) << 4));
                const f32x4 y = *(const Quad*)(piece + rq * kRow + (((c * 2 + 1) ^ (rq & 15)) << 4));
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    v[q][t] = x[t];
                    v[q][4 + t] = y[t];
                }
            }
            if (col < g.n) epilogue8<kBatch, true>(g.e, i0 + h * 64 + r, kStep, g.m, col, g.n - col, 1.0f, off, v);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Tiles and waves as product_kernel's.  A step is 256 contraction elements in
// two LDS stages; the scales of two steps come together, 16 bytes a row, into a
// buffer of their own, of which there are two as well.
//
// Bound by power, and next by the way of the operands to LDS.  8192 x 28672 x 8192
// as bf16 823 to 858 us (4.5 to 4.7 PFLOP/s); matrix instructions of random codes
// from registers alone reach 7.2, of zeros 9.8.  A step of a full chip takes 1.49 us
// of random codes, at 1.97 GHz, and 1.15 of zeros, at 2.4: 2750 cycles, of which 2048
// are the matrix instructions'.  With the loads left out it is 1.20 and 0.94; from
// L2 at one place 1.43 and 0.99; with the reads of scales left out 1.45 and 1.07, of
// A and half of B 1.42 and 1.11.  Beside the steps a round of tiles takes 12 us,
// when all CUs store at once (CUs started apart by parts of a tile: 0 to 4 % slower).
template <int BM, int BN, int WI, int WJ, int KW>
__global__ __launch_bounds__(WI* WJ* KW * 64) void mx4_product_kernel(Mx4Product g) {
    static_assert(KW == 1 || (WI == 1 && WJ == 1 && BM == 64 && BN == 64), "waves with parts of the contraction");
    constexpr int kThreads = WI * WJ * 64, kWM = BM / WI, kWN = BN / WJ, kFI = kWM / 16, kFJ = kWN / 16;
    constexpr int kStageA = BM * 128, kStageB = BN * 128, kScale = (BM + BN) * 16;
    constexpr bool kShared = KW == 1;  // the waves share their stages
    // Objects of their own, so that the compiler sees that a load into one and a
    // read of another have nothing to wait for.
    __shared__ __attribute__((aligned(1024))) uint8_t sa0[kStageA * KW];
    __shared__ __attribute__((aligned(1024))) uint8_t sa1[kStageA * KW];
    __shared__ __attribute__((aligned(1024))) uint8_t sb0[kStageB * KW];
    __shared__ __attribute__((aligned(1024))) uint8_t sb1[kStageB * KW];
    __shared__ __attribute__((aligned(1024))) uint8_t c0[kScale * KW];
    __shared__ __attribute__((aligned(1024))) uint8_t c1[kScale * KW];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tid = kShared ? threadIdx.x : lane;  // among the threads that fill a stage
    const int part = kShared ? 0 : wave, filler = kShared ? wave : 0;
    Lds* const a0 = (Lds*)sa0 + part * kStageA;
    Lds* const a1 = (Lds*)sa1 + part * kStageA;
    Lds* const b0 = (Lds*)sb0 + part * kStageB;
    Lds* const b1 = (Lds*)sb1 + part * kStageB;
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
    const int wi = kShared ? wave / WJ : 0, wj = kShared ? wave % WJ : 0, lo = lane & 15;

    f32x4 acc[kFI][kFJ];
#pragma unroll
    for (int i = 0; i < kFI; ++i)
#pragma unroll
        for (int j = 0; j < kFJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    if (turns > 0) {
        Mx4Fragments fa, fb;
        fa.init(wi * kWM, wi * kWM, lane);
        fb.init(wj * kWN, BM + wj * kWN, lane);
        Mx4Tile<BM, kThreads> ta;
        Mx4Tile<BN, kThreads> tb;
        Mx4Scales<BM, BN, WI * WJ> ts;
        ta.init(g.a, g.lda, i0, g.m, lbeg, lend, tid);
        tb.init(g.b, g.ldb, j0, g.n, lbeg, lend, tid);
        ts.init(g, i0, j0, lbeg, lend, filler, lane);
        constexpr int kSlots = kFI * kFJ, kEarly = kSlots / 8, kLag = kSlots / 4, kStop = kSlots * 5 / 4;

        // A's fragments of a step's first half, and of the second half of this step
        // and the next; B's of both halves; the scales of this step and the next.
        u32x4 x[kFI], y[2][kFI], b[2][kFJ];
        s16x2 sa[2][kFI], sb[2][kFJ];
        // One half of the step of parity p, product by product, with `between` (slot)
        // in each product's shadow.
        auto multiply = [&](auto kk, int p, auto&& between) {
            constexpr int KK = decltype(kk)::value;
            for_constants<kSlots>([&](auto slot) {
                constexpr int t = decltype(slot)::value;
                // 2 x 2 blocks, each product with one operand of the one before: a percent less
                // power than row by row, and so time
                constexpr int i = t / 4 / (kFJ / 2) * 2 + t % 4 / 2, j = t / 4 % (kFJ / 2) * 2 + (t % 4 / 2 ? 1 - t % 2 : t % 2);
                mx4_mfma<KK>(acc[i][j], b[KK][j], KK ? y[p][i] : x[i], sb[p][j], sa[p][i]);
                __builtin_amdgcn_sched_barrier(0);
                between(slot);
                __builtin_amdgcn_sched_barrier(0);
            });
        };
        // The step of parity p in a0 and b0 (or whichever are `a` and `bb`); the next one
        // is in `na` and `nb`, with its scales the half h of `scales`.
        //   first half   reads B of the second, at once, then the next step's scales
        //   second half  reads all of A and the first half of B of the next step
        // Before the step's two stages are filled with the step after the next all waves
        // have read them: a barrier stands at slot kLag, when the reads at the end of the
        // step before and those of B have come; another between the halves, where the
        // next step's stages are there.  The loads are spread over the slots from kLag to
        // kStop of the step's 2 kSlots: packed more densely they pass no faster, the last
        // ones later come late (8192 x 28672 x 8192 851 us; to the end of the first half
        // 855, to the middle of the second 859, to its end 863).
        auto step = [&](Lds* a, Lds* bb, Lds* na, Lds* nb, int p, const Lds* scales, int h, auto fill, Lds* more) {
            constexpr int kScales = kFI + kFJ, kAll = ta.kLoads + tb.kLoads + (decltype(fill)::value ? ts.kLoads : 0);
            auto load = [&](auto slot) {  // of the step's
                for_slot<kAll, decltype(slot)::value, kStop - kLag>([&](auto i) {
                    constexpr int q = decltype(i)::value;
                    if constexpr (q < ta.kLoads) ta.load(a, filler, q);
                    else if constexpr (q < ta.kLoads + tb.kLoads) tb.load(bb, filler, q - ta.kLoads);
                    else ts.load(more, filler, q - ta.kLoads - tb.kLoads);
                });
            };
            multiply(std::integral_constant<int, 0>(), p, [&](auto slot) {
                constexpr int t = decltype(slot)::value;
                if constexpr (t < kEarly) for_slot<kFJ, t, kEarly>([&](auto q) { b[1][decltype(q)::value] = fb.get(bb, decltype(q)::value, 1); });
                if constexpr (t == kLag) mx4_read<kShared>();
                if constexpr (t >= kLag) {
                    for_slot<kScales, t - kLag, kSlots - kLag>([&](auto i) {
                        constexpr int q = decltype(i)::value;
                        if constexpr (q < kFJ) sb[1 - p][q] = fb.get_scale(scales, q, h);
                        else sa[1 - p][q - kFJ] = fa.get_scale(scales, q - kFJ, h);
                    });
                    if constexpr (t < kStop) load(std::integral_constant<int, t - kLag>());
                }
            });
            // (the scales are the newest reads)
            constexpr int kIssued = kStop > kSlots ? (kSlots - kLag) * kAll / (kStop - kLag) : kAll;
            mx4_arrive<kShared, kIssued, kScales < 15 ? kScales : 15>();
            multiply(std::integral_constant<int, 1>(), p, [&](auto slot) {
                constexpr int t = decltype(slot)::value;
                for_slot<2 * kFI + kFJ, t, kSlots>([&](auto i) {
                    constexpr int q = decltype(i)::value;
                    if constexpr (q < kFI) x[q] = fa.get(na, q, 0);
                    else if constexpr (q < 2 * kFI) y[1 - p][q - kFI] = fa.get(na, q - kFI, 1);
                    else b[0][q - 2 * kFI] = fb.get(nb, q - 2 * kFI, 0);
                });
                if constexpr (t + kSlots < kStop) load(std::integral_constant<int, t + kSlots - kLag>());
            });
        };

#pragma unroll
        for (int q = 0; q < ta.kLoads; ++q) ta.load(a0, filler, q);
#pragma unroll
        for (int q = 0; q < tb.kLoads; ++q) tb.load(b0, filler, q);
#pragma unroll
        for (int q = 0; q < ts.kLoads; ++q) ts.load(e0, filler, q);
#pragma unroll
        for (int q = 0; q < ts.kLoads; ++q) ts.load(e1, filler, q);
#pragma unroll
        for (int q = 0; q < ta.kLoads; ++q) ta.load(a1, filler, q);
#pragma unroll
        for (int q = 0; q < tb.kLoads; ++q) tb.load(b1, filler, q);
        arrive<kShared>();
        settle(acc);
#pragma unroll
        for (int f = 0; f < kFI; ++f) {
            x[f] = fa.get(a0, f, 0);
            y[0][f] = fa.get(a0, f, 1);
            sa[0][f] = fa.get_scale(e0, f, 0);
        }
#pragma unroll
        for (int f = 0; f < kFJ; ++f) {
            b[0][f] = fb.get(b0, f, 0);
            sb[0][f] = fb.get_scale(e0, f, 0);
        }
        // Four steps a turn of the loop, so that each LDS access names its buffer.  An
        // odd count takes one more step, over zeros.
        for (;;) {
            step(a0, b0, a1, b1, 0, e0, 1, std::false_type(), e0);
            step(a1, b1, a0, b0, 1, e1, 0, std::true_type(), e0);
            if (--turns <= 0) break;
            step(a0, b0, a1, b1, 0, e1, 1, std::false_type(), e1);
            step(a1, b1, a0, b0, 1, e0, 0, std::true_type(), e1);
            if (--turns <= 0) break;
        }
        settle(acc);
    }
    arrive<kShared>();  // the last stages are being read and filled until here
    if constexpr (KW == 1) {
        static_assert(WI * WJ == 4 && kStageA >= 64 * kWN * 4 && kStageB >= 64 * kWN * 4, "a piece of LDS for each wave");
        mx4_finish(g, acc, wave == 0 ? a0 : wave == 1 ? b0 : wave == 2 ? a1 : b1, split, i0 + wi * kWM, j0 + wj * kWN, lane);
    } else {
        // The waves' sums of the tile through LDS, in the waves' order: rows of 256
        // bytes, the first half of them where A's first stage was, the others where B's
        // was, their chunks of 16 bytes permuted by the row.
        using Quad = __attribute__((address_space(3))) f32x4;
        auto at = [&](int w, int r) { return (r < 32 ? (Lds*)sa0 + w * kStageA : (Lds*)sb0 + w * kStageB) + (r & 31) * 256; };
#pragma unroll
        for (int i = 0; i < kFI; ++i)
#pragma unroll
            for (int j = 0; j < kFJ; ++j) *(Quad*)(at(wave, i * 16 + lo) + (((j * 4 + (lane >> 4)) ^ lo) << 4)) = acc[i][j];
        __syncthreads();
        constexpr int kBatch = 64 / KW / 8;
        const int c = lane & 7, col = j0 + c * 8, r0 = wave * (64 / KW) + (lane >> 3);
        float v[kBatch][8];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int r = r0 + q * 8;
            f32x4 s = {0, 0, 0, 0}, u = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                s += *(const Quad*)(at(w, r) + (((c * 2) ^ (r & 15)) << 4));
                u += *(const Quad*)(at(w, r) + (((c * 2 + 1) ^ (r & 15)) << 4));
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                v[q][t] = s[t];
                v[q][4 + t] = u[t];
            }
        }
        if (g.splits > 1) {
            float* const sums = g.part + static_cast<int64_t>(split) * g.m * g.pitch;
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int row = i0 + r0 + q * 8;
                if (row < g.m && col < g.pitch) store8(sums + static_cast<int64_t>(row) * g.pitch + col, 8, v[q]);
            }
        } else if (col < g.n) {
            epilogue8<kBatch>(g.e, i0 + r0, 8, g.m, col, g.n - col, 1.0f, mask_offset(g.e.mask), v);
        }
    }
}

// The product for at most 16 rows of A and not very many of B: bound by reading B
// once, and by a launch's start and end for small ones: 1 x 8192 x 8192 7.3 us (4.9
// TB/s), 16 x 11008 x 4096 7.2 to 7.9, 1 x 4096 x 4096 5.5 to 6.9 (of which 4.6 on the
// card).  As few_rows_kernel, with the eight waves taking every eighth 512
// contraction elements, 256 bytes of a row and 16 scales, from memory straight into
// the fragments: lane group q takes blocks 4q to 4q + 3, whose scales are one word.
template <int JB>
__global__ __launch_bounds__(kFewWaves * 64) void mx4_few_rows_kernel(Mx4Product g) {
    typedef int i32x8 __attribute__((ext_vector_type(8)));
    constexpr int kPitch = 20;  // floats of 16, padded against bank conflicts
    __shared__ __attribute__((aligned(16))) float sums[kFewWaves][JB][16 * kPitch];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lo = lane & 15, q = lane >> 4;
    const int j0 = blockIdx.x * (16 * JB);
    // Rows past the end are read as the last one; what they give is not stored.
    const int64_t ra = min(lo, g.m - 1);
    const uint8_t* const a = static_cast<const uint8_t*>(g.a) + ra * g.lda * 2 + q * 64;
    const uint8_t* const as = g.sa + ra * g.ldsa + q * 4;
    const uint8_t *b[JB], *bs[JB];
#pragma unroll
    for (int j = 0; j < JB; ++j) {
        const int64_t row = min(j0 + j * 16 + lo, g.n - 1);
        b[j] = static_cast<const uint8_t*>(g.b) + row * g.ldb * 2 + q * 64;
        bs[j] = g.sb + row * g.ldsb + q * 4;
    }
    f32x4 acc[JB];
#pragma unroll
    for (int j = 0; j < JB; ++j) acc[j] = f32x4{0, 0, 0, 0};

    struct Chunk {
        u32x4 a[4], b[JB][4];
        int as, bs[JB];
    };
    const int blocks = g.k / 8, full = blocks / 16, all = (blocks + 15) / 16;
    // END: the chunk may end behind the rows' end (its scales are there all the same).
    auto load = [&](Chunk& c, int at, auto end) {
        auto block = [&](const uint8_t* row, int t) {
            if (decltype(end)::value && at * 16 + q * 4 + t >= blocks) return u32x4{0, 0, 0, 0};
            return *reinterpret_cast<const u32x4*>(row + static_cast<int64_t>(at) * 256 + t * 16);
        };
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            c.bs[j] = *reinterpret_cast<const int*>(bs[j] + at * 16);
#pragma unroll
            for (int t = 0; t < 4; ++t) c.b[j][t] = block(b[j], t);
        }
        c.as = *reinterpret_cast<const int*>(as + at * 16);
#pragma unroll
        for (int t = 0; t < 4; ++t) c.a[t] = block(a, t);
    };
    auto multiply = [&](const Chunk& c) {
        auto operand = [](const u32x4& v) {
            return i32x8{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]), static_cast<int>(v[3]), 0, 0, 0, 0};
        };
        for_constants<4>([&](auto which) {
            constexpr int t = decltype(which)::value;
#pragma unroll
            for (int j = 0; j < JB; ++j)
                acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(c.b[j][t]), operand(c.a[t]), acc[j], 4, 4, t,
                                                                          c.bs[j], t, c.as);
        });
    };
    int c = wave;
    auto batches = [&](auto ahead) {
        constexpr int kN = decltype(ahead)::value;
        for (; c + (kN - 1) * kFewWaves < full; c += kN * kFewWaves) {
            Chunk r[kN];
#pragma unroll
            for (int u = 0; u < kN; ++u) load(r[u], c + u * kFewWaves, std::false_type{});
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < kN; ++u) multiply(r[u]);
        }
    };
    if constexpr (JB == 1) batches(std::integral_constant<int, 4>{});
    batches(std::integral_constant<int, 2>{});
    for (; c < all; c += kFewWaves) {
        Chunk r;
        if (c < full) load(r, c, std::false_type{});
        else load(r, c, std::true_type{});
        __builtin_amdgcn_sched_barrier(0);
        multiply(r);
    }
    // Lane: row lo, columns 4 q + 0..3.
#pragma unroll
    for (int j = 0; j < JB; ++j) *reinterpret_cast<f32x4*>(&sums[wave][j][lo * kPitch + q * 4]) = acc[j];
    __syncthreads();
    const int t = threadIdx.x, half = t & 1, j = (t >> 1) % JB, i = t / (2 * JB);  // 16 rows of 2 JB pieces
    const int col = j0 + j * 16 + half * 8;
    if (i >= g.m || col >= g.n) return;
    float v[1][8] = {{0, 0, 0, 0, 0, 0, 0, 0}};
#pragma unroll
    for (int p = 0; p < kFewWaves; ++p) {
        const float* s = &sums[p][j][i * kPitch + half * 8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[0][u] += s[u];
    }
    epilogue8<1>(g.e, i, 0, g.m, col, g.n - col, 1.0f, mask_offset(g.e.mask), v);
}

// ---------------------------------------------------------------- host

// Named, since the compiler otherwise leaves out the host's part of one of the two.
template __global__ void mx4_product_kernel<64, 64, 1, 1, 2>(Mx4Product g);
template __global__ void mx4_product_kernel<64, 64, 1, 1, 4>(Mx4Product g);

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

int32_t run_mx4_few(const Mx4Product& g, hipStream_t stream, const char* who) {
    const int features = mx4_few_features(g.m, g.n);
    const int64_t blocks = ceil_div(g.n, 16 * features);
    if (blocks > kMaxBlocks) return fail(FSDP_E_CAPACITY, "%s: more output tiles than one launch holds", who);
    const dim3 grid(static_cast<uint32_t>(blocks)), block(kFewWaves * 64);
    switch (features) {
        case 1: mx4_few_rows_kernel<1><<<grid, block, 0, stream>>>(g); break;
        case 2: mx4_few_rows_kernel<2><<<grid, block, 0, stream>>>(g); break;
        case 3: mx4_few_rows_kernel<3><<<grid, block, 0, stream>>>(g); break;
        default: mx4_few_rows_kernel<4><<<grid, block, 0, stream>>>(g);
    }
    return launched(who);
}

// Columns [j0, j0 + n) and rows [i0, i0 + m) of the product.
Mx4Product mx4_columns(const Mx4Product& g, int64_t j0, int64_t n) {
    Mx4Product s = g;
    static_cast<Product&>(s) = columns<true>(g, false, j0, n);
    s.sb += j0 * g.ldsb;
    return s;
}
Mx4Product mx4_rows(const Mx4Product& g, int64_t i0, int64_t m) {
    Mx4Product s = g;
    static_cast<Product&>(s) = rows<true>(g, i0, m);
    s.sa += i0 * g.ldsa;
    return s;
}

// The product whole, or its two parts after a cut.
int32_t run_mx4(Mx4Product& g, const Space& space, hipStream_t stream, const char* who) {
    if (mx4_few(g.m, g.n)) return run_mx4_few(g, stream, who);
    const Way best = mx4_best_way(g.extent(), space);
    if (best.us == kNoWay) return fail(FSDP_E_CAPACITY, "%s: more output tiles than one launch holds", who);
    const Cut cut = mx4_cut_of(g.extent(), best, space);
    if (cut.columns + cut.rows > 0) {
        const int64_t cj = cut.columns, ci = cut.rows;
        Mx4Product p = cj > 0 ? mx4_columns(g, 0, cj) : mx4_rows(g, 0, ci);
        Mx4Product q = cj > 0 ? mx4_columns(g, cj, g.n - cj) : mx4_rows(g, ci, g.m - ci);
        const int32_t st = run_mx4(p, space, stream, who);
        return st != FSDP_OK ? st : run_mx4(q, space, stream, who);
    }
    const Parts p = mx4_parts_of(g.k, best.splits);
    g.splits = p.n;
    g.kper = p.k;
    g.part = reinterpret_cast<float*>(space.p);
    if (best.tile == 256) return launch_mx4<256, 256, 2, 2, 1>(g, stream, who);
    if (best.tile == 128) return launch_mx4<128, 128, 2, 2, 1>(g, stream, who);
    const int64_t blocks = ceil_div(g.m, 64) * ceil_div(g.n, 64) * g.splits;
    if (mx4_waves(static_cast<double>(blocks)) == 4) return launch_mx4<64, 64, 1, 1, 4>(g, stream, who);
    return launch_mx4<64, 64, 1, 1, 2>(g, stream, who);
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
    if (a->k > kMaxMx4Contraction) return fail(FSDP_E_CAPACITY, "%s: k exceeds 2^23", who);
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
