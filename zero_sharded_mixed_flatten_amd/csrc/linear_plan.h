// linear_plan.h -- which kernel, tile and division of the contraction a layer
// product takes, by its sizes.  Host code without a HIP call.  Internal.
#ifndef ZERO_SHARD_LINEAR_PLAN_H
#define ZERO_SHARD_LINEAR_PLAN_H

#include <algorithm>
#include <cstdint>

#include "zero_linear.h"

namespace zero_linear_impl {

constexpr int kBK = 64;    // contraction elements of one step
constexpr int kCUs = 256;

enum Op { FWD = ZERO_LINEAR, DGRAD = ZERO_LINEAR_DGRAD, WGRAD = ZERO_LINEAR_WGRAD };

struct Plan {
    int bi, bj, parts;  // bi == 16 or 32: the kernel for few rows
    int64_t chunk;
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline Plan plan_for(int op, int64_t ni, int64_t nj, int64_t nc) {
    // Few rows: 16 columns a workgroup, the contraction undivided, against 64 x
    // 128 tiles in parts.  Up to 16 rows the former wins nearly everywhere; from
    // 17 on it multiplies twice for every piece of W, and loses where each CU
    // has much to do alone.  Times (us) few rows : tiles, W from HBM, for 1, 16
    // and 32 rows (24 and more are like 32):
    //   1600 x 1600    4.8 : 11.4     5.9 : 11.8     7.7 : 11.9
    //   4096 x 4096    9.9 : 18.3*   11.6 : 18.4    15.0 : 18.4
    //   1600 x 6400   10.2 : 17.5    13.9 : 18.0    19.9 : 18.1
    //   4096 x 6400   12.4 : 23.3    17.6 : 23.5    21.7 : 23.4
    //   11008 x 4096  23.1 : 26.4*   27.0 : 26.5    37.5 : 27.2
    //   32000 x 6400    87 :   83*    107 :   85     148 :   88
    //   1024 x 12288  16.4 : 21.2    23.8 : 22.3    35.0 : 22.5
    //   48 x 12288    15.1 : 16.7    22.8 : 16.0    33.3 : 16.2
    // (* 8 rows).  With W at an odd element both are slower, the former more:
    //   16 rows, 1600 x 2048 11.3 : 14.4, 4096 x 6400 31 : 29, 6400 x 6400 58 : 32
    // which the rule leaves out, since a product's workspace depends on its
    // sizes only.
    if (op == FWD && ni <= 32 && nj < (int64_t(1) << 26) &&
        (ni <= 16 || ceil_div(nj, 16 * kCUs) * nc <= 6400))
        return Plan{ni <= 16 ? 16 : 32, 16, 1, nc};
    const int64_t steps = std::max<int64_t>(ceil_div(nc, kBK), 1);
    // 256 x 256 tiles read least from shared memory and from memory a
    // product, but one fills a CU.  They pay from five eighths of a round on
    // and where the main loop outweighs the epilogue.  Times (us) with them
    // and with 128 x 128 tiles, on inputs that change from call to call:
    //   2500 x 4096 x 4096 (160 tiles)                 76 :  96
    //   8192 x 6400 x 1600                            152 : 162
    //   wgrad 6400 x 1600 over 8192 rows (175 tiles)  181 : 221
    //   the same over 512 rows                       22.1 : 23.1
    //   wgrad 4096 x 4096 over 512 rows (256 tiles)  27.8 : 31.6
    //   wgrad 11008 x 4096 over 64 rows                47 :  39
    //   256 x 50257 x 1600                             62 :  82
    // and where they would hang further over the edges, the small ones:
    //   333 x 50257 x 1600                            105 : 100
    // Operands that cannot be copied directly (direct_ok below) run as 128 x
    // 128 in one part where the large tiles are chosen here.
    const int64_t large = ceil_div(ni, 256) * ceil_div(nj, 256);
    const int64_t small = ceil_div(ni, 128) * ceil_div(nj, 128);
    if (large >= kCUs * 5 / 8 && 4 * large * 7 <= small * 8 && steps > (large >= kCUs ? 4 : 8))
        return Plan{256, 256, 1, steps * kBK};
    Plan p{ni <= 64 ? 64 : 128, 128, 1, 0};
    // Parts of the contraction, while all of them fit the card at once.  A
    // step takes 0.62 us with one workgroup on a CU and 0.95 with two, and
    // joining costs 4 us and 0.5 a part.  Undivided : divided as this says:
    // 128 x 4096 x 4096 41 : 19.5 us (8 parts; 24 in 16), 64 x 4096 x 11008
    // 122 : 29, wgrad 1600 x 1600 over 4096 rows 46 : 36; 512 x 6400 x 1600
    // is left whole, 20 us (25 in 2).
    const int64_t tiles = ceil_div(ni, p.bi) * ceil_div(nj, p.bj);
    int64_t parts = 1;
    double best = 0.0;
    for (int64_t n = 1; n <= 64 && n <= steps && (n == 1 || tiles * n <= 2 * kCUs); ++n) {
        const double cost = static_cast<double>(ceil_div(steps, n)) * (tiles * n <= kCUs ? 0.62 : 0.95) +
                            (n == 1 ? 0.0 : 4.0 + 0.5 * static_cast<double>(n));
        if (n == 1 || cost < best) {
            best = cost;
            parts = n;
        }
    }
    p.chunk = ceil_div(steps, parts) * kBK;
    p.parts = static_cast<int>(std::max<int64_t>(1, ceil_div(nc, p.chunk)));
    return p;
}

// One of the largest tiles occupies a CU.  What is left after the last whole
// round of them, up to half a round, runs as quarters, two to a CU: how many
// of a product's tiles do.
inline int64_t quartered(int64_t tiles) {
    const int64_t rest = tiles % kCUs;
    return tiles > kCUs && rest <= kCUs / 2 ? rest : 0;
}

// Direct copies move 16-byte pieces: every row 16-byte aligned, and (rows of
// lanes) a whole number of pieces long; a tile's rows span less than 2^32
// bytes.
inline bool direct_ok(const void *p, int64_t ld, int64_t lanes) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0 && lanes % 8 == 0 &&
           ld < (int64_t(1) << 22);
}

}  // namespace zero_linear_impl

#endif
