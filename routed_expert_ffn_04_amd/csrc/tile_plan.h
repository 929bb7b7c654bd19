// Tile size and k-splits of a product, from its sizes alone (plain C++, no device code).
#pragma once
#include <algorithm>

namespace moe {
namespace gemm {

constexpr int kStage = 128;  // bytes of k per stage

// A grid holds fewer than 2^32 threads.
inline bool grid_fits(long blocks, int threads) { return blocks > 0 && blocks <= 0xffffffffL / threads; }

// Threads of a workgroup: of the tiles, and of the kernel for a few rows (16 MFMA columns a workgroup).
constexpr int tile_threads(int edge) { return edge == 256 ? 512 : 256; }
constexpr int kFewThreads = 512;

// Up to 16 rows (one MFMA block) go to the kernel for a few rows, more to the tiles.
// 16 rows, weights from HBM, there and in tiles: FFN of 256 x 512 5.8 and 7.5 us, of
// 1024 x 512 8.1 and 11.4, 2048 x 1408 12.5 and 19.2, 4096 x 1024 15.3 and 19.1, 7168 x
// 2048 30 to 32 and 30; int8 of 7168 x 4096 11.9 and 12.6.  Fewer rows gain more (4 rows
// of 7168 x 2048 24.7 and 29.3).  Two blocks of 16 rows there do not reach the tiles'
// 33 rows.
constexpr int kFewRows = 16;

// Tile t of mt x nt in bands of 8 m-tiles with n outermost: the 32 tiles that a die
// works on together form a block of about 8 x 4 and share their operands in L2.
constexpr void band_of(int t, int mt, int nt, int& tm, int& tn) {
    const int band = t / (8 * nt);
    const int rows = mt - band * 8 < 8 ? mt - band * 8 : 8;
    t -= band * 8 * nt;
    tn = t / rows;
    tm = band * 8 + t % rows;
}

struct Plan {
    int few;             // the kernel for a few rows
    int edge;            // 256 x 256, 128 x 128 or 64 x 64 tiles; 0 and not few: no kernel's grid holds the product
    int splits, kspan;
    int workgroups;
    double us;           // estimated time
};

// Estimated time of wg workgroups of `span` stages each, in us, fitted to
// sweeps of every edge and number of splits.  64-row tiles share a CU's loads
// (up to four at once, 0.21 us a stage each); 128-row tiles run two to a CU, where
// a stage of each takes 0.95 us, against 0.5 with half of the CUs taken; a 256-row
// tile's stage takes 1.1 us alone and 1.6 when the whole chip draws power.
inline double tiling_us(int edge, long wg, int span) {
    auto rounds = [&](long at_once) { return (double)((wg + at_once - 1) / at_once); };
    if (edge == 256) {
        const double full = std::min(1.0, wg / 256.0);
        return rounds(256) * (span * (1.1 + 0.5 * full * full) + 10);
    }
    if (edge == 128) return wg <= 512 ? span * (0.35 + 0.6 * wg / 512.0) + 5 : rounds(512) * (span * 0.95 + 4) + 1;
    return rounds(256) * (span * 0.21 + 0.25) + 3;
}

// The tiling with the least estimated time, of those whose grid fits.
// mma_cols: MFMA columns of the product (gate/up: both matrices' columns).
// rows: both operands have k contiguous.
inline Plan plan_tiles(long M, long mma_cols, int K, int stage_elems, bool rows) {
    Plan best{};
    const int stages = (K + stage_elems - 1) / stage_elems;
    if (rows && M <= kFewRows && grid_fits((mma_cols + 15) / 16, kFewThreads)) {
        best.few = best.splits = 1;
        best.kspan = stages * stage_elems;
        return best;
    }
    double least = 0;
    for (int edge = 64; edge <= 256; edge *= 2) {
        const long tiles = ((M + edge - 1) / edge) * ((mma_cols + edge - 1) / edge);
        for (int s = 1; s <= 16 && (s == 1 || (stages / s >= 2 && tiles * s <= 512)); ++s) {
            const int span = (stages + s - 1) / s, n = (stages + span - 1) / span;
            const long wg = tiles * n;
            if (!grid_fits(wg, tile_threads(edge))) continue;
            double us = tiling_us(edge, wg, span);
            if (n > 1) us += 4 + (double)n * M * mma_cols * 8 / 4e6;
            if (least == 0 || us < least) {
                least = best.us = us;
                best.edge = edge;
                best.splits = n;
                best.kspan = span * stage_elems;
                best.workgroups = (int)wg;
            }
        }
    }
    return best;
}

// Tile edge of n products that go out as one launch, or 0 where `apart` (us, one
// after the other) is less.  Fitted to 36 shapes like the times above: the work of a
// CU (a stage, a tile's beginning and end) and the uneven end in units of the
// longest tile, at least that tile alone; off by 6 to 11 % (256- to 64-row tiles).
struct Size {
    int M, N, K;
};
inline int plan_together(const Size* p, int n, int stage_elems, double apart) {
    struct { double stage, tile, end, alone; } t;
    int best = 0;
    for (int edge = 64; n > 1 && edge <= 256; edge *= 2) {
        if (edge == 256) t = {1.7, 4.6, 0.41, 1.25};
        else if (edge == 128) t = {0.48, 0.8, 0.39, 0.6};
        else t = {0.2, 0, 0.44, 0.19};
        double work = 0, longest = 0, all = 0;
        for (int i = 0; i < n; ++i) {
            const double tiles = (double)((p[i].M + edge - 1) / edge) * ((p[i].N + edge - 1) / edge);
            const double span = (p[i].K + stage_elems - 1) / stage_elems;
            all += tiles;
            work += tiles * (span * t.stage + t.tile) / 256;
            longest = std::max(longest, span);
        }
        if (!grid_fits((long)all, tile_threads(edge))) continue;
        const double us = std::max(longest * t.alone + 5, work + longest * t.end) + 2;
        if (us < apart) {
            apart = us;
            best = edge;
        }
    }
    return best;
}

inline bool fits(const Plan& p) { return p.few || p.edge; }

}  // namespace gemm
}  // namespace moe
