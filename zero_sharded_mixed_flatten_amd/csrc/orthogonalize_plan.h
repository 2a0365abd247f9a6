// orthogonalize_plan.h -- how zero_orthogonalize runs, by its sizes: which
// kernels, tiles and parts, and what lies where in the workspace; and each
// round's constants, by its coefficients.  Host code without a HIP call.
// Internal.
#ifndef ZERO_SHARD_ORTHOGONALIZE_PLAN_H
#define ZERO_SHARD_ORTHOGONALIZE_PLAN_H

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "linear_plan.h"
#include "zero_muon.h"

namespace zero_muon_impl {

using zero_linear_impl::ceil_div;
using zero_linear_impl::kBK;
using zero_linear_impl::kCUs;

constexpr int kParts = 256;  // partial sums of squares a matrix, at most
constexpr int64_t kMaxSide = 65536, kMaxCount = 65535;

enum Kind { GRAM = 0, SQUARE = 1, APPLY = 2, FINISH = 3 };  // FINISH: the last apply

template <int R>
constexpr int kSmallColumns = R == 64 ? 1024 : 448;  // of the longest rows

inline int64_t up64(int64_t v) { return (v + 63) / 64 * 64; }

struct Work {
    int64_t r, c, rp, cp;
    int64_t parts, d, e, a, q, hi0, hi1, lo, partial, bytes;  // offsets into the workspace
};

inline int64_t partial_bytes(const Work &w, int64_t count);

// by one workgroup a matrix, to which only X's lo is not local
inline bool is_small(const Work &w) {
    return w.rp == 64 ? w.cp <= kSmallColumns<64> : w.rp == 128 && w.cp <= kSmallColumns<128>;
}

inline Work work_of(int64_t count, int64_t rows, int64_t cols) {
    Work w{};
    w.r = std::min(rows, cols);
    w.c = std::max(rows, cols);
    w.rp = up64(w.r);
    w.cp = up64(w.c);
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    if (is_small(w)) {
        w.lo = take(count * w.rp * w.cp * 2);
        w.bytes = at;
        return w;
    }
    w.parts = take(count * kParts * 8);
    w.d = take(count * w.rp * 4);
    w.e = take(count * w.rp * 4);
    w.a = take(count * w.rp * w.rp * 2);
    w.q = take(count * w.rp * w.rp * 2);
    w.hi0 = take(count * w.rp * w.cp * 2);
    w.hi1 = take(count * w.rp * w.cp * 2);
    w.lo = take(count * w.rp * w.cp * 2);
    w.partial = take(partial_bytes(w, count));
    w.bytes = at;
    return w;
}

inline bool sides_ok(int64_t count, int64_t rows, int64_t cols) {
    return count >= 0 && count <= kMaxCount && rows >= 0 && rows <= kMaxSide && cols >= 0 &&
           cols <= kMaxSide;
}

constexpr int64_t kMaxTiles = int64_t(1) << 23;

inline int64_t tiles_of(int kind, const Work &w, int64_t bt) {
    const int64_t ti = ceil_div(w.rp, bt);
    return kind == GRAM || kind == SQUARE ? ti * (ti + 1) / 2 : ti * ceil_div(w.cp, bt);
}

// How a product runs: the side of its tiles, groups of waves a workgroup,
// buffers of steps, and (gram) parts of the contraction.
struct Way {
    int side, groups, buffers, parts;
    int64_t steps;  // of a part
};

// Tiles of 256 from half a round of the CUs on.  Fewer are as many smaller
// ones; one step of the contraction is then over sooner than the next one's
// copies take, so the smallest tiles have four buffers while two workgroups on
// each CU are enough for all, and tiles of 128 two groups of waves while one
// is.  Times of gram, square and apply (us) of one matrix, with
//                  64, 2 buffers   64, 4 buffers   128, 1 group    128, 2 groups
//   512 x 512      6.8  7.6  7.3   5.7  6.4  6.4  11.3 12.5 11.9   9.2 10.6 11.4
//   1024 x 1024   11.1 11.7 11.4   6.9  8.4  9.3  15.4 17.9 17.1  13.0 15.6 15.4
//   1600 x 1600   15.4 16.4 21.0  12.6 13.3 23.4  21.3 22.9 24.4  19.6 18.0 21.1
//   2048 x 2048   20.6 21.8 33.0  23.0 24.5 35.0  26.0 27.8 31.8  21.8 23.5 27.9
// and of a call, tiles of 256 and 128: 3200 x 3200 (91 and 169 tiles of 256)
// 1060 : 940, 4096 x 4096 (136 and 256) 1530 : 1810.
//
// A long contraction of the gram product is divided where its tiles leave CUs
// idle.  Calls, undivided : divided, us: 256 x 8192 264 : 141, 1024 x 4096
// 256 : 235, 128 x 1024 96 : 81, 128 x 2048 137 : 91; 128 x 512 75 : 78 is left
// whole.
inline Way way_of(int kind, const Work &w, int64_t count) {
    const int64_t steps = (kind == GRAM ? w.cp : w.rp) / kBK;
    const int64_t n256 = count * tiles_of(kind, w, 256), n128 = count * tiles_of(kind, w, 128),
                  n64 = count * tiles_of(kind, w, 64);
    const bool narrow = kind == GRAM && w.rp <= 128;
    if (n256 >= kCUs / 2 && !narrow) return Way{256, 1, 2, 1, steps};
    if (n64 > 2 * kCUs && !narrow)
        return steps > 8 ? Way{128, n128 <= kCUs ? 2 : 1, 2, 1, steps} : Way{64, 1, 2, 1, steps};
    Way p{64, 1, 4, 1, steps};
    if (kind == GRAM) {
        // of eight steps and more, or (few rows) of four: what is not divided
        // there is one workgroup's work
        const int64_t parts = narrow ? std::min({steps / 4, 384 / n64, int64_t(8)})
                                     : std::min({steps / 8, 384 / n64, int64_t(10)});
        if (parts > 1 && (narrow ? steps >= 12 : steps - steps / parts > 26))
            p.steps = ceil_div(steps, parts);
        p.parts = static_cast<int>(ceil_div(steps, p.steps));
    }
    return p;
}

inline int64_t partial_bytes(const Work &w, int64_t count) {
    const Way p = way_of(GRAM, w, count);
    return p.parts == 1 ? 0 : p.parts * count * tiles_of(GRAM, w, p.side) * p.side * p.side * 4;
}

// One tile of 256 has a CU to itself.  What is left after the last whole round
// of them, up to half a round, runs as quarters in a second launch: how many
// tiles do.  A call with and without, us: four 4096 x 4096 matrices 5390 : 5700,
// one 8192 x 8192 9470 : 10130, twelve 1600 x 1600 1680 : 1790; not where a few
// short tiles are left: sixteen 1600 x 1600 2120 : 2060.
inline int64_t rest_of(int kind, const Work &w, int64_t count) {
    const Way p = way_of(kind, w, count);
    const int64_t rest =
        p.side == 256 ? zero_linear_impl::quartered(tiles_of(kind, w, 256) * count) : 0;
    return rest * (kind == GRAM ? w.cp : w.rp) < 65536 ? 0 : rest;
}

// Powers of two: A's off-diagonals in fp16 from a product of X, scaled by 2^24,
// and back, and P's.
struct Scales {
    float to_a, from_a, from_aa;  // from_aa: from a product of two A
    float to_p, from_p;
};

struct Round {
    float a, b, c;
    float lo_share, lo_rest;  // lo's factor, as 1 e_i + 0 or 0 e_i + a
    Scales scale;
};

// the largest power of two up to 2^12, X's scale, that keeps magnitudes of
// `most` well inside fp16's range
inline double scale_for(double most) {
    return std::ldexp(1.0, static_cast<int>(std::min(
                               12.0, std::max(-100.0, std::floor(15.0 - std::log2(most))))));
}

// Each round's constants.  `top` bounds X's singular values: 1 at first, then
// what the polynomial makes of those up to it (1 % more for its roundings), and
// 16 by contract.  Off-diagonal elements of a symmetric matrix are at most half
// the difference of two of its eigenvalues.  lo's factor is the diagonal of P
// in the rounds whose error small directions multiply by 4 at most until the
// end, by the coefficients a of the rounds that follow, and a in the others.
inline void rounds_of(const zero_ns_params &k, int64_t r, Round *rounds) {
    const double usual[3] = {3.4445, -4.7750, 2.0315};
    double top = 1.01;
    for (int i = 0; i < k.steps; ++i) {
        const double *given = k.coeffs != nullptr ? k.coeffs + 3 * i : usual;
        Round &q = rounds[i];
        q.a = static_cast<float>(given[0]);
        q.b = static_cast<float>(given[1]);
        q.c = static_cast<float>(given[2]);
        const double a = q.a, b = q.b, c = q.c, t1 = top * top;
        // b t + c t^2 over t = s^2 up to top^2
        const double end = t1 * (b + c * t1), turn = -b / (2.0 * c);
        double low = std::min(0.0, end), high = std::max(0.0, end);
        if (turn > 0.0 && turn < t1) {
            low = std::min(low, 0.5 * b * turn);
            high = std::max(high, 0.5 * b * turn);
        }
        const double scale_a = scale_for(0.5 * t1), scale_p = scale_for(0.5 * (high - low));
        q.scale.to_a = static_cast<float>(scale_a / (4096.0 * 4096.0));
        q.scale.from_a = static_cast<float>(1.0 / scale_a);
        q.scale.from_aa = static_cast<float>(1.0 / (scale_a * scale_a));
        q.scale.to_p = static_cast<float>(scale_p);
        q.scale.from_p = static_cast<float>(1.0 / scale_p);
        // the largest |s (a + b s^2 + c s^4)|: at the end, or where 5 c t^2 + 3 b
        // t + a is zero
        double next = top * std::fabs(a + end);
        const double root = std::sqrt(9.0 * b * b - 20.0 * a * c);
        for (double t : {(-3.0 * b - root) / (10.0 * c), (-3.0 * b + root) / (10.0 * c),
                         -a / (3.0 * b)})
            if (t > 0.0 && t < t1) next = std::max(next, std::sqrt(t) * std::fabs(a + t * (b + c * t)));
        top = std::min(16.0, 1.01 * next);
    }
    double slope = 1.0;
    for (int i = k.steps - 1; i >= 0; --i) {
        const bool diagonal = slope <= 4.0 || r == 1;
        rounds[i].lo_share = diagonal ? 1.0f : 0.0f;
        rounds[i].lo_rest = diagonal ? 0.0f : rounds[i].a;
        slope *= std::fabs(rounds[i].a);
    }
}

}  // namespace zero_muon_impl

#endif
