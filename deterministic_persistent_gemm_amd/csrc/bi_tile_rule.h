// bi_tile_rule.h -- how a feed-forward product picks its tile shape (host).
//
// The shapes of one product differ only in time, never in bits, so the rule may
// look at everything, M included.  A shape's time is estimated as
//
//   launch + rounds * (per_tile + slices * per_slice)
//
// with the two costs of one workgroup fitted to timings of 32 to 34 problems per
// product, drawn over M 1 .. 4096, widths 128 .. 12288 and k 256 .. 4096, on an
// MI355X (fit within 5 to 20 percent there).  rounds: workgroups per compute unit,
// counted whole where a shape's LDS ring leaves room for one workgroup per
// compute unit and as a fraction where several share it.  Over those problems
// the shapes chosen this way come within 1 to 4 percent of the fastest of 6 to 14
// shapes on average; always taking 64 x 64 costs 1.24 to 1.38 times the fastest,
// always 128 x 128 1.40 to 1.70, always 256 x 256 2.0 to 3.4.
//
// What it does not hold for: contractions far past 4096, as dx has over wide
// layers, are priced too low (290 rows, K 3296, contraction 16032 on 64 x 64 tiles:
// 65 us estimated, 113 taken), and rows of a tile that lie past M count like others.
// Costs refitted on contractions up to 24576 picked dx alone within 1.04 of the
// fastest (1.11 with these) but changed passes with both products by -20 to +20
// percent, so they are not used; the backward pass has two exceptions instead
// (kNumDxApart and the streaming 64 x 64 tiles below 33 rows).
#pragma once

#include <stdint.h>

namespace bi {

struct TileShape {
    int bm, bn;            // outputs per tile: rows, columns
    float per_tile;        // us
    float per_slice;       // us
    float share;           // several workgroups per compute unit: cost of each against alone; 0: one
};

constexpr float kTileLaunch = 1.7f;    // us

inline int64_t tile_count(const TileShape& t, int64_t M, int64_t N)
{
    return ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
}

// One workgroup's time.  The costs were taken with bf16 outputs; fp32 outputs
// write two bytes more each, at the 19 KB a microsecond that a compute unit has
// of the HBM's write rate when all of them write.
inline float tile_once(const TileShape& t, int64_t slices, bool f32_out)
{
    return t.per_tile + t.per_slice * (float)slices + (f32_out ? (float)(t.bm * t.bn) * 2.f / 18750.f : 0.f);
}

inline float tile_time(const TileShape& t, int64_t M, int64_t N, int64_t slices, bool f32_out, int cus)
{
    const int64_t tiles = tile_count(t, M, N);
    float rounds;
    if (t.share > 0.f) {
        rounds = (float)tiles / (float)cus * t.share;
        rounds = rounds < 1.f ? 1.f : rounds;
    } else {
        rounds = (float)((tiles + cus - 1) / cus);
    }
    return kTileLaunch + rounds * tile_once(t, slices, f32_out);
}

// The index of the fastest of n shapes.
inline int pick_tile(const TileShape* t, int n, int64_t M, int64_t N, int64_t slices, bool f32_out, int cus)
{
    int best = 0;
    float best_time = tile_time(t[0], M, N, slices, f32_out, cus);
    for (int i = 1; i < n; ++i) {
        const float time = tile_time(t[i], M, N, slices, f32_out, cus);
        if (time < best_time) {
            best = i;
            best_time = time;
        }
    }
    return best;
}

}  // namespace bi
