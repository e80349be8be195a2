// Host logic of the 4-bit matrices (include/fsdp_mx4.h): their checks, and by
// which launches a product is computed.  Plain C++ without device code, so that
// host tests reach it.
#pragma once

#include "fsdp_mx4.h"
#include "internal.h"
#include "linear_plan.h"

namespace fsdp {
namespace linear {

// A product's rows lie no further apart: a tile's 256 of them are within the 31
// bits of a buffer offset.
constexpr int64_t kMaxMx4Stride = int64_t(1) << 22;
constexpr int64_t kMaxMx4Contraction = 2 * kMaxMx4Stride;  // its codes are such a row

// The two arrays of a 4-bit matrix, as matrices of bytes.
struct Mx4Matrix {
    Matrix codes, scales;
};

inline Mx4Matrix mx4_matrix(const void* codes, int64_t ldc, const char* what, const void* scales, int64_t lds,
                            const char* what_scales, int64_t rows, int64_t cols, bool written) {
    return {{codes, rows, FSDP_MX4_CODE_BYTES(cols), ldc, 1, what, written},
            {scales, rows, FSDP_MX4_SCALE_BYTES(cols), lds, 1, what_scales, written}};
}

inline int32_t check_mx4(const Mx4Matrix& x, const char* who) {
    for (const Matrix* p : {&x.codes, &x.scales}) {
        const int32_t st = check_matrix(*p, false, who);
        if (st != FSDP_OK) return st;
        if (!aligned(p->p, 16) || (p->rows > 1 && p->ld % 16 != 0))
            return fail(FSDP_E_ALIGN, "%s: rows of %s do not start on 16-byte boundaries", who, p->what);
    }
    return FSDP_OK;
}

// ---------------------------------------------------------------- ways to compute a product
//
// The contraction is counted in 16-bit units of codes, eight a block: a step of
// kBK of them is 256 elements.

// The contraction in at most `splits` parts of whole pairs of steps, none empty:
// the scales of two steps are read together.
inline Parts mx4_parts_of(int64_t k, int64_t splits) {
    const int64_t turns = std::max<int64_t>(1, ceil_div(k, 2 * kBK)), per = ceil_div(turns, splits);
    return {static_cast<int32_t>(ceil_div(turns, per)), static_cast<int32_t>(per * 2 * kBK)};
}

// The waves that share the contraction of a 64-tile, in `blocks` workgroups: four,
// one workgroup a CU; or where there are more workgroups than CUs two, and two
// workgroups a CU.  1024 x 2048 x 4096: 10.6 us, by four 13.7; 1024 x 1365 x 2047: 8.3
// and 11.5; 1024 x 1024 x 4096, 256 workgroups: 8.0 and 7.6.
inline int mx4_waves(double blocks) { return blocks > kCus ? 2 : 4; }

// What a product takes in microseconds, as way_of in linear_plan.h: from times
// measured over products of one 64 x 64 tile to 8192 x 11008 x 4096, within a
// sixth of them but for the smallest.
//   256: a step takes 1.1 us on a near empty chip, 1.6 on a full one, where
//     power sets the clock.  4096 x 4096 x 4096: 37.5 us, by 128-tiles 45.2.
//   128: two workgroups a CU, 1.08 us a step for both; alone 0.37 to 0.67.
//     2048 x 2048 x 4096: 13.1 us, by 256-tiles 31.4, by 64-tiles 21.8.
//   64: waves on parts of a step.  1024 x 1024 x 4096: 7.6 us, by 128-tiles 11.7;
//     1024 x 2048 x 4096: 10.6 and 12.0; 1024 x 2048 x 11008: 24.1 and 27.2.  64 x 64 x 16384: 13.2 us, split in four 9.7, in seven 9.2.
inline Way mx4_way_of(int tile, int64_t splits, const Extent& g) {
    const double tiles = static_cast<double>(ceil_div(g.m, tile)) * ceil_div(g.n, tile) * splits;
    const double steps = static_cast<double>(ceil_div(ceil_div(g.k, kBK), splits)), fill = std::min(1.0, tiles / kCus);
    double us;
    if (tile == 256) us = 3 + std::ceil(tiles / kCus) * (10 + (1.1 + 0.5 * fill) * steps);
    else if (tile == 64 && mx4_waves(tiles) == 2) us = 0.5 + std::ceil(tiles / (2 * kCus)) * (4.9 + 0.37 * steps);
    else if (tile == 64) us = 4.9 + 0.135 * steps;
    else if (tiles <= kCus) us = 5.5 + (0.37 + 0.3 * fill) * steps;
    else us = 1 + std::ceil(tiles / (2 * kCus)) * (4.6 + 1.08 * steps);
    if (splits > 1) us += 3 + std::max(8.0 * splits * g.m * g.pitch / 6e6, 0.1 * (splits - 24));
    return Way{tile, splits, tiles > kMaxBlocks ? kNoWay : us};
}

inline Way mx4_best_way(const Extent& g, const Space& space) { return best_way_by<mx4_way_of>(g, space); }

inline Cut mx4_cut_of(const Extent& g, const Way& best, const Space& space) { return cut_by<mx4_way_of>(g, best, space); }

// Whether the product takes the way for few rows of A: what one matrix
// instruction takes, where 64-tiles would not give more than every CU one.  By it
// and by tiles: 16 rows, [4096, 4096] 5.6 and 7.0 us, [8192, 8192] 9.0 and 10.7,
// [16384, 4096] 8.2 and 8.6, [28672, 8192] 26.9 and 21.5, [32000, 4096] 16.4 and 14.0;
// one row, [28672, 8192] 27.1 and 21.0; 32 rows, [11008, 4096] 8.6 and 7.2, [4096, 4096]
// 6.3 and 7.0.
inline bool mx4_few(int64_t m, int64_t n) { return m <= 16 && n <= 64 * kCus; }

// The columns of a workgroup of that way: A is read again by each, B's rows
// once, and the CU with the most workgroups ends last; so the least rounds *
// bytes of one.
inline int mx4_few_features(int64_t m, int64_t n) {
    int best = 0;
    int64_t cost = 0;
    for (int jb = 1; jb <= 4; ++jb) {
        const int64_t c = ceil_div(ceil_div(n, 16 * jb), kCus) * (16 * jb + m);
        if (best == 0 || c < cost) {
            best = jb;
            cost = c;
        }
    }
    return best;
}

}  // namespace linear
}  // namespace fsdp
