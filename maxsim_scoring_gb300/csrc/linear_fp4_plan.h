// Which tiles a 4-bit linear takes: host arithmetic on the product's sizes alone.
#pragma once

#include <cstdint>

namespace maxsim {

constexpr int kFp4TileM = 256;      // rows of A per tile: 128 on each CTA of a pair
constexpr int kFp4TileK = 256;      // values of K per stage: 128 bytes of a row
constexpr int kFp4MaxSplits = 4;    // pairs that share a tile's K
constexpr int64_t kFp4Pairs = 76;   // CTA pairs of a GB300 (152 SMs): plans do not depend on the device

struct LinearFp4Plan {
    bool swap = false;  // A is w, B is x
    int tn = 64;
    int64_t tiles = 0, tiles_b = 0;
    int32_t kb = 0, splits = 1, kb_split = 0;
};

// The tile's width, and the pairs of a cluster that share a tile's K where there
// are few tiles, by the time they should take, in cycles: the tiles of the
// busiest pair, each its stages and a start and end. (Fitted to the times of whole
// products: a stage takes 600 cycles with 256 columns, and 490 and 460 with 128 and
// 64, where the MMA warp's issue bounds it; the rest of a tile 2,300, 1,000 and 700.)
// Clusters of four CTAs: a GB300 holds 36 of them; of eight only 15.
inline LinearFp4Plan plan_linear_fp4(int64_t M, int64_t N, int64_t K) {
    LinearFp4Plan p;
    p.swap = N > M;
    p.kb = static_cast<int32_t>((K + kFp4TileK - 1) / kFp4TileK);
    const int64_t rows_a = p.swap ? N : M, rows_b = p.swap ? M : N;
    double best = 0.0;
    for (int tn = 256; tn >= 64; tn /= 2) {
        const int64_t tiles_b = (rows_b + tn - 1) / tn, tiles = (rows_a + kFp4TileM - 1) / kFp4TileM * tiles_b;
        const double stage = tn == 256 ? 600.0 : tn == 128 ? 490.0 : 460.0, ends = tn == 256 ? 2300.0 : tn == 128 ? 1000.0 : 700.0;
        // the first stage's latency, and the last tile's way out
        const double once = tn == 256 ? 6000.0 : tn == 128 ? 3500.0 : 2500.0;
        for (int32_t splits = 1; splits <= kFp4MaxSplits; splits *= 2) {
            const int32_t kb_split = (p.kb + splits - 1) / splits;
            const int64_t clusters = splits == 1 ? kFp4Pairs : splits == 2 ? 36 : 15;
            if (splits > 1 && (tn != 64 || tiles > clusters || kb_split * (splits - 1) >= p.kb)) continue;
            const double cost = static_cast<double>((tiles + clusters - 1) / clusters) * (kb_split * stage + ends) + once + (splits > 1 ? 1500.0 : 0.0);
            if (best == 0.0 || cost < best) {
                best = cost;
                p.tn = tn;
                p.tiles = tiles;
                p.tiles_b = tiles_b;
                p.splits = splits;
                p.kb_split = kb_split;
            }
        }
    }
    return p;
}

}  // namespace maxsim
