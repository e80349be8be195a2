// The linear layer's host logic (csrc/linear_plan.h) under AddressSanitizer and
// UBSan (CPU only), driven by tests/test_linear_plan.py.
//
//   route < cases    one product per input line:
//                      call fp8 m n k a_aligned b_aligned workspace_bytes
//                    with call forward, grad_input or grad_weight and the
//                    product's own m, n, k (output rows and columns, contraction
//                    length); prints by which launches it is computed.
//   plan SEED K      K random products: whether every part fits its workspace,
//                    covers the contraction, and is a launch; prints
//                    "cases faults".
//   overlap SEED K   K random pairs of matrices against a byte-by-byte brute
//                    force; prints "cases missed refused": overlaps not seen,
//                    and matrices of one stride refused without one.
#include <cinttypes>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <iostream>
#include <random>
#include <sstream>
#include <string>
#include <vector>

#include "linear_plan.h"

namespace {

using namespace fsdp::linear;

int64_t faults = 0;
void expect(bool ok) { faults += !ok; }

// One launch (and its join, for several parts) over g's whole output.
void check_parts(const Extent& g, int tile, int64_t splits, const Space& space) {
    const Parts p = parts_of(g.k, splits);
    expect(p.n >= 1 && p.n <= splits && p.k % kBK == 0);
    expect(static_cast<int64_t>(p.n) * p.k >= g.k && static_cast<int64_t>(p.n - 1) * p.k < std::max(g.k, 1));
    expect(p.n == 1 || static_cast<int64_t>(p.n) * g.m * g.pitch * 4 <= space.left);
    expect(ceil_div(g.m, tile) * ceil_div(g.n, tile) * p.n <= kMaxBlocks);
    expect(p.n == 1 || ceil_div(static_cast<int64_t>(g.m) * (g.pitch / 8), 256) <= kMaxBlocks);
}

template <bool BL>
std::string direct(const Extent& g, const Space& space) {
    const Way best = best_way<BL>(g, space);
    if (best.us == kNoWay) return " refused";
    const Cut cut = cut_of<BL>(g, best, space);
    expect(cut.columns % 256 == 0 && cut.rows % 256 == 0 && cut.columns >= 0 && cut.rows >= 0);
    expect(cut.columns == 0 || cut.rows == 0);
    if (cut.columns > 0) {
        expect(cut.columns < g.n);
        return " columns" + direct<BL>(columns_of(g, cut.columns), space) + direct<BL>(columns_of(g, g.n - cut.columns), space);
    }
    if (cut.rows > 0) {
        expect(cut.rows < g.m);
        return " rows" + direct<BL>(rows_of(g, cut.rows), space) + direct<BL>(rows_of(g, g.m - cut.rows), space);
    }
    check_parts(g, best.tile, best.splits, space);
    return " " + std::to_string(best.tile) + "/" + std::to_string(parts_of(g.k, best.splits).n);
}

template <bool AL, bool BL>
std::string route(Extent g, bool fp8, bool a_ok, bool b_ok, int64_t bytes) {
    const Space space(reinterpret_cast<void*>(uintptr_t(1) << 20), bytes);
    g.pitch = static_cast<int32_t>(round_up(g.n, 8));
    if (AL && BL && few_tokens(g.m, a_ok, b_ok))
        return std::string("few ") + (g.m <= 16 ? "1x" : "2x") + std::to_string(few_features(g.m, g.n, fp8));
    if (a_ok && b_ok) return "direct" + direct<BL>(g, space);
    const Pieces p = pieces_of<AL, BL>(g, fp8, a_ok, b_ok, space);
    if (p.rows == 0) {
        const int64_t splits = splits_for(128, 2 * kCus, g, space);
        if (ceil_div(g.m, 128) * ceil_div(g.n, 128) <= kMaxBlocks) check_parts(g, 128, splits, space);
        return "staged 128/" + std::to_string(parts_of(g.k, splits).n);
    }
    const int64_t a = packed_bytes(a_ok, AL, p.rows, g.k, false), b = packed_bytes(b_ok, BL, p.cols, g.k, fp8);
    expect(a + b <= space.left && p.rows > 0 && p.rows <= g.m && p.cols > 0 && p.cols <= g.n);
    expect(p.rows == g.m || (p.rows % 256 == 0 && !a_ok));
    expect(p.cols == g.n || (p.cols % 256 == 0 && !b_ok));
    // a packed row's length is an int32, and its rows lie within a buffer offset's 31 bits
    expect(a_ok || packed_row(AL ? g.k : p.rows, false) * std::min<int64_t>(AL ? p.rows : g.k, 256) <= INT32_MAX);
    expect(b_ok || packed_row(BL ? g.k : p.cols, fp8) * std::min<int64_t>(BL ? p.cols : g.k, 256) <= INT32_MAX);
    Space rest = space;
    rest.take(a);
    rest.take(b);
    expect(rest.left >= 0 && rest.left == space.left - a - b);
    const int64_t na = ceil_div(g.m, p.rows), nb = ceil_div(g.n, p.cols);
    return "pieces " + std::to_string(na) + "x" + std::to_string(nb) +
           direct<BL>(columns_of(rows_of(g, p.rows), p.cols), rest);
}

std::string route_of(const std::string& call, bool fp8, const Extent& g, bool a_ok, bool b_ok, int64_t bytes) {
    if (call == "forward") return route<true, true>(g, fp8, a_ok, b_ok, bytes);
    if (call == "grad_input") return route<true, false>(g, fp8, a_ok, b_ok, bytes);
    return route<false, false>(g, false, a_ok, b_ok, bytes);
}

int run_route() {
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        std::string call;
        int fp8, a_ok, b_ok;
        int64_t bytes;
        Extent g{};
        in >> call >> fp8 >> g.m >> g.n >> g.k >> a_ok >> b_ok >> bytes;
        std::printf("%s\n", route_of(call, fp8 != 0, g, a_ok != 0, b_ok != 0, bytes).c_str());
    }
    return faults != 0;
}

int run_plan(uint64_t seed, int count) {
    std::mt19937_64 rng(seed);
    auto size = [&](double bits) {
        return static_cast<int32_t>(std::exp2(std::uniform_real_distribution<>(0, bits)(rng)));
    };
    const char* calls[] = {"forward", "grad_input", "grad_weight"};
    for (int i = 0; i < count; ++i) {
        const double bits = i % 4 == 0 ? 30 : 15;
        const Extent g{size(bits), size(bits), rng() % 20 == 0 ? 0 : size(bits), 0};
        const int64_t bytes = rng() % 5 == 0 ? 0 : static_cast<int64_t>(std::exp2(std::uniform_real_distribution<>(0, 27)(rng)));
        route_of(calls[rng() % 3], rng() % 2, g, rng() % 2, rng() % 2, bytes);
    }
    std::printf("%d %" PRId64 "\n", count, faults);
    return 0;
}

int run_overlap(uint64_t seed, int count) {
    std::mt19937_64 rng(seed);
    int64_t missed = 0, refused = 0;
    constexpr int kBytes = 400;
    for (int t = 0; t < count; ++t) {
        Matrix m[2];
        std::vector<char> held[2];
        const int64_t stride = 1 + static_cast<int64_t>(rng() % 12);
        for (int i = 0; i < 2; ++i) {
            const int elem = 1 << rng() % 3;
            const int64_t rows = static_cast<int64_t>(rng() % 5), cols = static_cast<int64_t>(rng() % 9);
            int64_t ld = rng() % 4 == 0 ? cols + static_cast<int64_t>(rng() % 4) : (stride * 4) / elem;
            if (ld < cols) ld = cols;
            const uintptr_t at = 4096 + (rng() % 100) / static_cast<unsigned>(elem) * static_cast<unsigned>(elem);
            m[i] = Matrix{reinterpret_cast<const void*>(at), rows, cols, ld, elem, "m", true};
            held[i].assign(kBytes * 4, 0);
            for (int64_t r = 0; r < rows; ++r)
                for (int64_t c = 0; c < cols * elem; ++c)
                    held[i].at(static_cast<size_t>(at - 4096) + static_cast<size_t>(r * ld * elem + c)) = 1;
            expect(check_matrix(m[i], false, "overlap") == FSDP_OK);
        }
        bool real = false;
        for (size_t b = 0; b < held[0].size(); ++b) real = real || (held[0][b] && held[1][b]);
        const bool said = overlap(m[0], m[1]);
        missed += real && !said;
        // exact where both have several rows of one stride, and for single rows
        const bool one = m[0].rows > 1 && m[1].rows > 1 && m[0].ld * m[0].elem == m[1].ld * m[1].elem;
        refused += !real && said && (one || (m[0].rows == 1 && m[1].rows == 1));
        expect(said == overlap(m[1], m[0]));
    }
    std::printf("%d %" PRId64 " %" PRId64 "\n", count, missed + faults, refused);
    return 0;
}

}  // namespace

int main(int argc, char** argv) {
    if (argc >= 2 && std::strcmp(argv[1], "route") == 0) return run_route();
    if (argc >= 4 && std::strcmp(argv[1], "plan") == 0) return run_plan(std::strtoull(argv[2], nullptr, 10), std::atoi(argv[3]));
    if (argc >= 4 && std::strcmp(argv[1], "overlap") == 0)
        return run_overlap(std::strtoull(argv[2], nullptr, 10), std::atoi(argv[3]));
    std::fprintf(stderr, "usage: %s route < cases | plan SEED K | overlap SEED K\n", argv[0]);
    return 2;
}
