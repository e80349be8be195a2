// The linear layer's host logic (include/fsdp_linear.h): its checks of matrices
// and overlaps, and by which launches a product is computed.  Plain C++ without
// device code, so that host tests reach it; csrc/linear.hip carries it out.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "fsdp_linear.h"
#include "internal.h"

// Returns what x gives unless that is FSDP_OK.
#define TRY(x)                                     \
    do {                                           \
        const int32_t st_ = (x);                   \
        if (st_ != FSDP_OK) return st_;            \
    } while (0)

namespace fsdp {
namespace linear {

constexpr int kXcds = 8;
constexpr int kCus = 256;
constexpr int kBK = 64;  // contraction elements of one LDS tile: 128 bytes of bf16

// A product's output rows and columns and its contraction's length.
struct Extent {
    int32_t m, n, k;
    int32_t pitch;  // n rounded up to 8: columns of a row of partial sums
};

// ---------------------------------------------------------------- arguments

constexpr int64_t kMaxDim = int64_t(1) << 30;

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// One matrix (or vector: rows = 1) of a call.
struct Matrix {
    const void* p;
    int64_t rows, cols, ld;
    int elem;
    const char* what;
    bool written;

    bool empty() const { return !p || rows == 0 || cols == 0; }
    uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
    uintptr_t hi() const { return lo() + static_cast<uintptr_t>(((rows - 1) * ld + cols) * elem); }
};

inline int32_t check_matrix(const Matrix& x, bool may_be_null, const char* who) {
    if (!x.p) {
        if (may_be_null || x.rows == 0 || x.cols == 0) return FSDP_OK;
        return fail(FSDP_E_ARG, "%s: null %s", who, x.what);
    }
    if (x.rows > 1 && x.ld < x.cols)
        return fail(FSDP_E_ARG, "%s: row stride %lld of %s is below its %lld columns", who,
                    static_cast<long long>(x.ld), x.what, static_cast<long long>(x.cols));
    if (!aligned(x.p, static_cast<uintptr_t>(x.elem)))
        return fail(FSDP_E_ALIGN, "%s: %s misaligned", who, x.what);
    int64_t bytes;
    if (x.rows > 0 && (x.ld < 0 || !fsdp::mul_i64(x.rows, x.ld, &bytes) || !fsdp::mul_i64(bytes, x.elem, &bytes) ||
                       !fsdp::add_i64(bytes, x.cols * x.elem, &bytes)))
        return fail(FSDP_E_ARG, "%s: size of %s overflows", who, x.what);
    return FSDP_OK;
}

// Whether two matrices share a byte.  Of one row stride, they do unless their
// columns differ everywhere; of different strides, when their extents meet.
inline bool overlap(const Matrix& a, const Matrix& b) {
    if (a.empty() || b.empty() || a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
    const int64_t row = a.ld * a.elem;
    if (a.rows == 1 || b.rows == 1 || row != b.ld * b.elem) return true;
    const uintptr_t span = static_cast<uintptr_t>(row);
    const uintptr_t d = a.lo() <= b.lo() ? (b.lo() - a.lo()) % span : (span - (a.lo() - b.lo()) % span) % span;
    // columns [0, wa) of a against [d, d + wb) of b, on a circle of one row
    return d < static_cast<uintptr_t>(a.cols * a.elem) || d + static_cast<uintptr_t>(b.cols * b.elem) > span;
}

inline bool same(const Matrix& a, const Matrix& b) { return a.p == b.p && a.ld == b.ld && a.elem == b.elem; }

// twin(a, b): whether written a may be b itself
template <typename F>
inline int32_t check_overlaps(std::initializer_list<Matrix> ms, const char* who, F&& twin) {
    for (auto i = ms.begin(); i != ms.end(); ++i)
        for (auto j = i + 1; j != ms.end(); ++j) {
            const Matrix &a = *i, &b = *j;
            if (!(a.written || b.written) || !overlap(a, b)) continue;
            if (same(a, b) && twin(a, b)) continue;
            return fail(FSDP_E_ALIAS, "%s: %s overlaps %s", who, a.what, b.what);
        }
    return FSDP_OK;
}

inline int32_t check_sizes(int64_t m, int64_t n, int64_t k, const char* who) {
    if (m < 0 || n < 0 || k < 0) return fail(FSDP_E_ARG, "%s: negative size", who);
    if (m > kMaxDim || n > kMaxDim || k > kMaxDim) return fail(FSDP_E_CAPACITY, "%s: a size exceeds 2^30", who);
    return FSDP_OK;
}

inline int32_t check_workspace(const void* p, int64_t bytes, const char* who) {
    if (bytes < 0 || (!p && bytes > 0)) return fail(FSDP_E_ARG, "%s: bad workspace", who);
    if (!aligned(p, 16)) return fail(FSDP_E_ALIGN, "%s: workspace misaligned", who);
    return FSDP_OK;
}

inline int32_t check_flag(int32_t v, const char* what, const char* who) {
    if (v != 0 && v != 1) return fail(FSDP_E_ARG, "%s: %s must be 0 or 1", who, what);
    return FSDP_OK;
}

inline int32_t check_float_dtype(int32_t d, const char* what, const char* who) {
    if (d != FSDP_DT_F32 && d != FSDP_DT_BF16) return fail(FSDP_E_DTYPE, "%s: %s must be fp32 or bf16", who, what);
    return FSDP_OK;
}

inline Matrix vector(const void* p, int64_t n, int elem, const char* what, bool written = false) {
    return Matrix{p, 1, n, n, elem, what, written};
}

inline Matrix bytes_of(const void* p, int64_t bytes, const char* what, bool written) {
    return Matrix{p, 1, bytes, bytes, 1, what, written};
}

// The workspace that the call will actually write is within its first bytes.
inline Matrix workspace_of(const void* p, int64_t bytes) {
    return bytes_of(p, std::min<int64_t>(bytes, FSDP_LINEAR_WORKSPACE_BYTES), "workspace", true);
}

// ---------------------------------------------------------------- ways to compute a product

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int64_t round_up(int64_t x, int64_t a) { return ceil_div(x, a) * a; }

// Workgroups of one launch: its threads are counted in 32 bits.
constexpr int64_t kMaxBlocks = 0x3fffff;

// Rows on 16-byte boundaries and lengths in whole 16-byte chunks of e elements;
// a tile's rows within the 31 bits of a buffer offset.
inline bool direct_ok(const void* p, int64_t ld, int64_t rows, int64_t cols, int e) {
    return aligned(p, 16) && cols % e == 0 && (ld % e == 0 || rows <= 1) && ld <= (int64_t(1) << 21);
}

// The workspace, handed out from its start.
struct Space {
    uint8_t* p;
    int64_t left;

    Space(void* ptr, int64_t bytes)
        : p(static_cast<uint8_t*>(ptr)), left(std::min<int64_t>(bytes, FSDP_LINEAR_WORKSPACE_BYTES)) {}
    void* take(int64_t bytes) {
        bytes = (bytes + 255) / 256 * 256;
        if (bytes > left) return nullptr;
        void* q = p;
        p += bytes;
        left -= bytes;
        return q;
    }
};

// A way to compute a product: the output tile's side and the parts that its
// contraction is split into.
struct Way {
    int tile;
    int64_t splits;
    double us;
};
constexpr double kNoWay = 1e30;

// What a product takes in microseconds, from times measured over products of
// one 64 x 64 tile to 8192 x 8192 x 8192 on MI355X; within a fifth of most of
// them, which is enough to order the ways.  A launch is a number of rounds of
// the chip, each an entry and an epilogue and a time a step of 64.
//   256: one workgroup a CU.  A step takes 1.5 us on a full chip, where power
//     sets the clock, 1.0 on a near empty one.  4096 x 4096 x 4096: 105 us, by
//     128-tiles 130.
//   128: two workgroups a CU share its matrix units.  2048 x 4096 x 4096: 60
//     us, by 256-tiles 81.
//   64: one workgroup a CU, four waves on four parts of a step, which takes
//     more where B is read by its columns.  1024 x 1024 x 4096: 17 us, by
//     128-tiles 42, by those split in four 22.
//   A split's sums go to memory and back at 6 TB/s, and the join is a launch.
//     64 x 1024 x 4096 by 64-tiles: 15.5 us, split in 16 9.8.  The join's
//     threads add the parts one after the other, which over small outputs takes
//     0.1 us for each beyond 24: 33 x 64 x 11008 by 128-tiles in 86 parts 15.1
//     us, by 64-tiles in 20 10.7; but 7 x 16 x 1888 by 128-tiles in 15 7.9, by
//     64-tiles in 3 8.8.
template <bool BL>
inline Way way_of(int tile, int64_t splits, const Extent& g) {
    const double tiles = static_cast<double>(ceil_div(g.m, tile)) * ceil_div(g.n, tile) * splits;
    const double steps = static_cast<double>(ceil_div(ceil_div(g.k, kBK), splits));
    double us = 3;
    if (tile == 256) us += std::ceil(tiles / kCus) * (10 + (1 + 0.5 * std::min(1.0, tiles / kCus)) * steps);
    else if (tile == 64) us += std::ceil(tiles / kCus) * (3 + (BL ? 0.165 : 0.2) * steps);
    else if (tiles <= kCus) us += 3 + 0.57 * steps;
    else us += std::ceil(tiles / (2 * kCus)) * (4 + 0.9 * steps);
    if (splits > 1) us += 3 + std::max(8.0 * splits * g.m * g.pitch / 6e6, 0.1 * (splits - 24));
    return Way{tile, splits, tiles > kMaxBlocks ? kNoWay : us};
}

// The splits that fill `fill` workgroups, at least two steps each, partial sums
// within the workspace.
inline int64_t splits_for(int tile, int64_t fill, const Extent& g, const Space& space) {
    const int64_t tiles = ceil_div(g.m, tile) * ceil_div(g.n, tile);
    const int64_t one = static_cast<int64_t>(g.m) * g.pitch * 4;
    const int64_t splits = std::min(fill / tiles, ceil_div(g.k, kBK) / (tile == 64 ? 8 : 2));
    return std::max<int64_t>(1, std::min(splits, space.left / one));
}

// The contraction in at most `splits` parts of whole steps, none empty.
struct Parts {
    int32_t n, k;  // parts, and the contraction elements of each but the last (a multiple of kBK)
};
inline Parts parts_of(int64_t k, int64_t splits) {
    const int64_t steps = std::max<int64_t>(1, ceil_div(k, kBK)), per = ceil_div(steps, splits);
    return {static_cast<int32_t>(ceil_div(steps, per)), static_cast<int32_t>(per * kBK)};
}

// The least estimate for the whole product.
using Estimate = Way(int tile, int64_t splits, const Extent& g);
template <Estimate WAY>
inline Way best_way_by(const Extent& g, const Space& space) {
    Way best = WAY(256, 1, g);
    for (int tile : {128, 64})
        for (int64_t fill : {int64_t(0), int64_t(kCus), int64_t(2 * kCus)}) {
            const Way w = WAY(tile, splits_for(tile, fill, g, space), g);
            if (w.us < best.us) best = w;
        }
    return best;
}
template <bool BL>
inline Way best_way(const Extent& g, const Space& space) {
    return best_way_by<way_of<BL>>(g, space);
}

// Where to cut `along` output rows (columns) into whole rounds of 256-tiles and
// a rest: 0 if there is no such place.
inline int64_t round_cut(int64_t along, int64_t across) {
    const int64_t tiles = ceil_div(across, 256), all = ceil_div(along, 256);
    const int64_t cut = tiles * all / kCus * kCus / tiles * 256;
    return cut < along ? cut : 0;
}

// Columns (rows) [0, n) of the product's extent.
inline Extent columns_of(const Extent& g, int64_t n) {
    return {g.m, static_cast<int32_t>(n), g.k, static_cast<int32_t>(round_up(n, 8))};
}
inline Extent rows_of(const Extent& g, int64_t m) { return {static_cast<int32_t>(m), g.n, g.k, g.pitch}; }

// Whether the product is cut in two, where a round of the chip would be for a
// few tiles only (4096 x 4104 x 4096: 256 tiles and 16 of 8 columns each: 122
// us, whole 178).  For less than 4 % by the estimate the second launch is not
// worth it (4096 x 11008 x 4096: 2 %, and 1-6 % slower).
struct Cut {
    int64_t columns, rows;  // the first part's (a multiple of 256), or 0; at most one is set
};
template <Estimate WAY>
inline Cut cut_by(const Extent& g, const Way& best, const Space& space) {
    const int64_t cj = round_cut(g.n, g.m), ci = round_cut(g.m, g.n);
    double us = 0.96 * best.us;
    Cut cut{0, 0};
    if (cj > 0) {
        const double c = best_way_by<WAY>(columns_of(g, cj), space).us + best_way_by<WAY>(columns_of(g, g.n - cj), space).us;
        if (c < us) {
            us = c;
            cut = {cj, 0};
        }
    }
    if (ci > 0) {
        const double c = best_way_by<WAY>(rows_of(g, ci), space).us + best_way_by<WAY>(rows_of(g, g.m - ci), space).us;
        if (c < us) cut = {0, ci};
    }
    return cut;
}
template <bool BL>
inline Cut cut_of(const Extent& g, const Way& best, const Space& space) {
    return cut_by<way_of<BL>>(g, best, space);
}

// Whether the forward product takes the way for few tokens.  Up to 16 tokens,
// and up to 32 where the tiles would need operands laid out anew.  32 tokens by
// 64-tiles: [4096, 11008] 23 us, this way 35; [11008, 4096] 23 and 24.  16
// tokens of [4096, 4096]: 13 and 10.
inline bool few_tokens(int64_t m, bool a_ok, bool b_ok) { return m <= 16 || (m <= 32 && !(a_ok && b_ok)); }

// The features of a workgroup: x is read again by each, W's rows once, and the
// CU with the most workgroups ends last; so the least rounds * (bytes of x and
// W of one).  11008 features of 4096 E4M3 codes, 16 tokens: 48 a workgroup (230
// workgroups) take 12.2 us, 32 (344) 17.
inline int few_features(int64_t m, int64_t n, bool fp8) {
    int best = 0;
    int64_t cost = 0;
    for (int jb = 1; jb <= 4; ++jb) {
        const int64_t c = ceil_div(ceil_div(n, 16 * jb), kCus) * (16 * jb * (fp8 ? 1 : 2) + 2 * m);
        if (best == 0 || c < cost) {
            best = jb;
            cost = c;
        }
    }
    return best;
}

// Bytes of a packed row.
inline int64_t packed_row(int64_t cols, bool fp8) { return ceil_div(cols * (fp8 ? 1 : 2), 128) * 128; }

// Bytes that an operand's part of `outputs` rows (columns) of the product takes
// when it is laid out anew; 0 where that isn't needed.
inline int64_t packed_bytes(bool ok, bool lmajor, int64_t outputs, int64_t k, bool fp8) {
    return ok ? 0 : round_up(lmajor ? outputs * packed_row(k, fp8) : k * packed_row(outputs, fp8), 256);
}

// How a product with unaligned operands is computed: its output in pieces of
// rows x cols, whose operands are laid out anew one after the other; rows = 0:
// whole, with the operands staged through registers.
struct Pieces {
    int64_t rows, cols;
    bool by_rows;  // a piece of A serves all pieces of B, not the other way round
};

// Whole operands where they fit in the workspace; else the pieces of least
// estimated time, or none.  Small pieces fill the chip badly, and many lay
// operands out again and again (at 4.5 TB/s and 4 us a launch).  Staged, a
// 128-tile's step takes 1.5 to 1.8 us where both operands are l-major, 1.7 to
// 2.4 with an o-major B (5.5 where only one round of workgroups hides its
// loads), 2.6 to 4.3 with both, against 0.9.  Pieces and staged, with 64 MiB:
// weight gradient of [4095, 11007] over 8192 tokens 1126 and 3300 us, the input
// gradient 670 and 1220; forward of 8191 tokens through [11007, 4095] 670 and
// 1160, but through [4095, 11007], of whose operands only 1500 rows each fit,
// 1180 staged.  Pieces of B alone are taken for 6 % more, and others for 6 %
// less: the estimates are no nearer.
template <bool AL, bool BL>
inline Pieces pieces_of(const Extent& g, bool fp8, bool a_ok, bool b_ok, const Space& space) {
    const auto bytes_a = [&](int64_t r) { return packed_bytes(a_ok, AL, r, g.k, false); };
    const auto bytes_b = [&](int64_t c) { return packed_bytes(b_ok, BL, c, g.k, fp8); };
    if (bytes_a(g.m) + bytes_b(g.n) <= space.left) return {g.m, g.n, true};
    if (bytes_a(std::min(g.m, 256)) + bytes_b(std::min(g.n, 256)) > space.left) return {0, 0, true};
    const Parts s = parts_of(g.k, splits_for(128, 2 * kCus, g, space));
    const double tiles = static_cast<double>(ceil_div(g.m, 128)) * ceil_div(g.n, 128) * s.n;
    const double rounds = std::ceil(tiles / (2 * kCus));
    const double step = AL && BL ? (fp8 ? 1.5 : 1.8) : !AL ? 3.4 : rounds > 1 ? 2.4 : 5.5;
    double least = 3 + rounds * (4 + step * s.k / kBK);
    Pieces best{0, 0, true};
    for (int64_t na = 1; na <= (a_ok ? 1 : 32); ++na) {
        const int64_t r = na == 1 ? g.m : std::min<int64_t>(g.m, round_up(ceil_div(g.m, na), 256));
        const int64_t left = space.left - bytes_a(r);
        for (int64_t nb = 1; left >= 0 && nb <= (b_ok ? 1 : 32); ++nb) {
            const int64_t c = nb == 1 ? g.n : std::min<int64_t>(g.n, round_up(ceil_div(g.n, nb), 256));
            if (bytes_b(c) > left) continue;
            Space rest = space;
            rest.take(bytes_a(r) + bytes_b(c));
            const Extent p = columns_of(rows_of(g, r), c);
            const int64_t ra = ceil_div(g.m, r), cb = ceil_div(g.n, c);
            const double once = static_cast<double>(bytes_a(r)) * ra, other = static_cast<double>(bytes_b(c)) * cb;
            const double by_rows = once + other * (cb > 1 ? ra : 1), by_cols = other + once * (ra > 1 ? cb : 1);
            const double us = ra * cb * (4 + best_way<BL>(p, rest).us) + std::min(by_rows, by_cols) * 2 / 4.5e6;
            if (us < (na == 1 ? 1.06 : 0.94) * least) {
                least = us;
                best = {r, c, by_rows <= by_cols};
            }
            break;  // fewer columns a piece only cost more
        }
    }
    return best;
}

}  // namespace linear
}  // namespace fsdp
