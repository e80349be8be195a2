// The 4-bit product's host logic (csrc/mx4_plan.h) under AddressSanitizer and
// UBSan, for tests/test_mx4_plan.py.
//
//   mx4_plan plan SEED COUNT   random products: parts, cuts and launches hold their bounds
//   mx4_plan route             a line "m n k workspace" each: the way it takes
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>

#include "mx4_plan.h"

using namespace fsdp::linear;

static Extent extent(int64_t m, int64_t n, int64_t k) {
    return {static_cast<int32_t>(m), static_cast<int32_t>(n), static_cast<int32_t>(FSDP_MX4_CODE_BYTES(k) / 2),
            static_cast<int32_t>(round_up(n, 8))};
}

// What run_mx4 does, as text; false if a bound does not hold.
static bool walk(const Extent& g, const Space& space, char* out, size_t room, int depth) {
    if (mx4_few(g.m, g.n)) {
        const int f = mx4_few_features(g.m, g.n);
        snprintf(out, room, "few %d", f);
        return f >= 1 && f <= 4;
    }
    const Way best = mx4_best_way(g, space);
    if (best.us == kNoWay) {
        snprintf(out, room, "none");
        return true;
    }
    const Cut cut = mx4_cut_of(g, best, space);
    if (cut.columns + cut.rows > 0) {
        if ((cut.columns > 0) == (cut.rows > 0) || cut.columns % 256 || cut.rows % 256 || cut.columns >= g.n || cut.rows >= g.m ||
            depth > 8)
            return false;
        const Extent p = cut.columns ? columns_of(g, cut.columns) : rows_of(g, cut.rows);
        const Extent q = cut.columns ? columns_of(g, g.n - cut.columns) : rows_of(g, static_cast<int64_t>(g.m) - cut.rows);
        const int at = snprintf(out, room, "%s ", cut.columns ? "columns" : "rows");
        if (!walk(p, space, out + at, room - at, depth + 1)) return false;
        const size_t used = strlen(out);
        out[used] = ' ';
        return walk(q, space, out + used + 1, room - used - 1, depth + 1);
    }
    const Parts s = mx4_parts_of(g.k, best.splits);
    const double blocks = std::ceil(g.m / 64.0) * std::ceil(g.n / 64.0) * s.n;
    if (best.tile == 64) snprintf(out, room, "64x%d/%d", mx4_waves(blocks), s.n);
    else snprintf(out, room, "%d/%d", best.tile, s.n);
    // whole pairs of steps, none empty, all covered; sums within the workspace; a possible launch
    const int64_t k = g.k, per = s.k;
    if (s.n < 1 || per % (2 * kBK) || per * s.n < k || (s.n > 1 && per * (s.n - 1) >= k) || s.n > best.splits) return false;
    if (s.n > 1 && static_cast<int64_t>(s.n) * g.m * g.pitch * 4 > space.left) return false;
    return ceil_div(g.m, best.tile) * ceil_div(g.n, best.tile) * s.n <= kMaxBlocks;
}

int main(int argc, char** argv) {
    char text[512];
    if (argc == 4 && !strcmp(argv[1], "plan")) {
        std::mt19937_64 r(strtoull(argv[2], nullptr, 10));
        const long count = atol(argv[3]);
        auto size = [&](int bits) {
            const int64_t v = static_cast<int64_t>(r() >> (64 - 1 - r() % bits));
            return std::max<int64_t>(1, std::min<int64_t>(v, kMaxDim));
        };
        long bad = 0;
        for (long i = 0; i < count; ++i) {
            const int64_t m = size(30), n = size(30), k = std::min<int64_t>(size(23), 1 << 23);
            const int64_t bytes = r() % 4 ? static_cast<int64_t>(r() % (128 << 20)) : 0;
            if (!walk(extent(m, n, k), Space(bytes ? &text : nullptr, bytes), text, sizeof text, 0)) {
                if (bad++ < 5) fprintf(stderr, "%lld %lld %lld %lld: %s\n", (long long)m, (long long)n, (long long)k, (long long)bytes, text);
            }
        }
        printf("%ld %ld\n", count, bad);
        return 0;
    }
    long long m, n, k, bytes;
    while (scanf("%lld %lld %lld %lld", &m, &n, &k, &bytes) == 4) {
        if (!walk(extent(m, n, k), Space(bytes ? &text : nullptr, bytes), text, sizeof text, 0)) return 1;
        puts(text);
    }
    return 0;
}
