// Host logic of the 4-bit matrices (include/fsdp_mx4.h): their checks, and by
// which launches a product is computed.  Plain
// C++ without device code.
#pragma once

#include "fsdp_mx4.h"
#include "internal.h"
#include "linear_plan.h"

namespace fsdp {
namespace linear {

// A product's rows lie no further apart: a tile's 256 of them are within the 31
// bits of a buffer offset.
constexpr int64_t kMaxMx4Stride = int64_t(1) << 22;

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

// Whether the product takes the way for few rows of A.
inline bool mx4_few(int64_t m) { return m <= 32; }

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

inline Way mx4_best_way(const Extent& g, const Space& space) { return best_way<true>(g, space); }

}  // namespace linear
}  // namespace fsdp
