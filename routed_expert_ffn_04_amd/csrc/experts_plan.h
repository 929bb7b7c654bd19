// Tiles and grids of the experts' products, from their sizes alone (plain C++, no
// device code).  How the rows are spread over the experts is not known to the host: a
// grid has room for any spread, times are estimated for an even one.
#pragma once
#include "tile_plan.h"

namespace moe {
namespace gemm {

constexpr int kDies = 8;
constexpr int kStreamEdge = 256;   // tiles of the streamed weight gradients

// Most of an expert's `tiles` that a die takes.
constexpr int die_share(int tiles) { return (tiles + kDies - 1) / kDies; }

// Row tiles that the experts' rows can fill: one more than they fill together, for
// every expert that has rows; and those of an even spread.
inline long row_tiles(int R, int n, int edge) { return (long)R / edge + std::min(R, n); }
inline int even_rows(int R, int n) { return (R + std::min(R, n) - 1) / std::min(R, n); }
inline long even_tiles(int R, int n, int edge) { return (long)std::min(R, n) * ((even_rows(R, n) + edge - 1) / edge); }

// Position in the order of `total` tiles, of which every die takes one contiguous
// run, of workgroup `block`; -1 past them.
constexpr int in_die_order(int block, int total) {
    const int x = block % kDies, j = block / kDies;
    const int base = total / kDies, extra = total % kDies;
    return j < base + (x < extra ? 1 : 0) ? x * base + (x < extra ? x : extra) + j : -1;
}

// 256-row tiles: where a die's tiles leave half or more of its `cus` CUs without work in
// their last round, the tiles of that round are cut into halves of 128 rows, which
// take 0.6 of a tile's time each.  The workgroup whose tile workgroup `block` takes, and which part of it.
constexpr int kMostCuts = 16;   // of a die
struct Cut {
    int block;
    int half;   // 0: the whole tile, 1: its upper, 2: its lower half
};
constexpr Cut cut_of(int block, int total, int cus) {
    const int x = block % kDies, j = block / kDies;
    const int mine = total / kDies + (x < total % kDies ? 1 : 0), last = mine % cus, whole = mine - last;
    if (2 * last > cus || last > kMostCuts || j < whole) return {block, 0};
    return {(whole + (j - whole) / 2) * kDies + x, 1 + (j - whole) % 2};
}

// Workgroups of a product over the experts' rows: a multiple of the dies, which share
// the tiles that there are evenly, and of 256-row tiles so many more for the second
// halves of those that are cut.
inline long rows_grid(int R, int n, int edge, long nt) {
    return (row_tiles(R, n, edge) * nt + kDies - 1) / kDies * kDies + (edge == 256 ? kDies * kMostCuts : 0);
}

// Estimated time, in us, of a product over the experts' rows by tiles of an edge, for
// rows spread around an even share: fitted to 80 banks and row counts (4 to 128 experts
// of 1024 x 512 to 7168 x 2048, 12 to 1200 rows each, shares that differ by a factor of
// two to three).  Taking the edge with the least of these loses 1.1 % against the best of
// the three (tiling_us of an even spread: 4.9 %).  The last tile of an expert counts for a part of one, of
// 256-row tiles as half a one's 0.6 where few rows fill no more.
inline double rows_us(int edge, int R, int n, long nt, int span) {
    const double experts = std::min(R, n), rows = R / experts;
    if (edge == 256) {
        const double tiles = experts * std::max(rows / 256 + 0.14, 0.6) * nt / 256, full = std::min(1.0, tiles);
        return std::max(rows < 110 ? 0.6 : 1.0, tiles + 0.12) * (span * (0.91 + 0.12 * full * full) + 10.7);
    }
    if (edge == 128) {
        const double tiles = experts * std::max(rows / 128 + 0.55, 1.0) * nt / 512;
        return tiles <= 1 ? span * (0.49 + 0.51 * tiles) + 5 : tiles * (span * 0.88 + 6) + 1;
    }
    const double tiles = experts * std::max(rows / 64 + 0.42, 1.0) * nt / 256;
    return std::max(1.0, tiles + 0.14) * (span * 0.19 + 0.47) + 3;
}

// Tile edge of such a product, by the estimated time; 0: no grid holds it.  cols: MFMA
// columns (gate/up: both matrices').
inline int rows_edge(int R, int n, long cols, int K, int stage_elems) {
    int best = 0;
    double least = 0;
    for (int edge = 64; edge <= 256; edge *= 2) {
        const long nt = (cols + edge - 1) / edge;
        if (!grid_fits(rows_grid(R, n, edge, nt), tile_threads(edge))) continue;
        const double us = rows_us(edge, R, n, nt, (K + stage_elems - 1) / stage_elems);
        if (best == 0 || us < least) {
            least = us;
            best = edge;
        }
    }
    return best;
}

// Half-stages in the ring of tiles: ten where there are no more of them than then run at once.
inline int ring_of(int edge, long tiles) { return (edge == 64 && tiles <= 512) || (edge == 128 && tiles <= 256) ? 10 : 5; }

// The products of the backward pass that do not depend on each other: dx, over the
// rows, and weight gradients (sum), for every expert.
struct GroupSize {
    int M, N, K;   // dx: N, K; a gradient: M, N
    bool sum;
};

// The weight gradients go as a stream of 256 x 256 tiles where these give every CU
// one: with fewer (up to 256 of them were tried), smaller tiles in one launch with dx are faster.
inline long stream_tiles(const GroupSize* p, int m, int n) {
    long tiles = 0;
    for (int i = 0; i < m; ++i)
        if (p[i].sum) tiles += (long)n * ((p[i].M + kStreamEdge - 1) / kStreamEdge) * ((p[i].N + kStreamEdge - 1) / kStreamEdge);
    return tiles;
}

// Workgroups of one of them in a launch together, and how many of these have a tile with rows spread evenly.
inline long group_grid(const GroupSize& p, int R, int n, int edge) {
    const long nt = (p.N + edge - 1) / edge, mt = (p.M + edge - 1) / edge;
    return p.sum ? (long)n * ((mt * nt + kDies - 1) / kDies * kDies) : rows_grid(R, n, edge, nt);
}
inline long group_tiles(const GroupSize& p, int R, int n, int edge) {
    const long nt = (p.N + edge - 1) / edge, mt = (p.M + edge - 1) / edge;
    return p.sum ? n * mt * nt : even_tiles(R, n, edge) * nt;
}

// Tile edge of a launch together (times as in plan_together); 0: no grid holds it.
inline int group_edge(const GroupSize* p, int m, int R, int n, int stage_elems) {
    struct { double stage, tile, end, alone; } t;
    int best = 0;
    double least = 0;
    for (int edge = 64; edge <= 256; edge *= 2) {
        if (edge == 256) t = {1.7, 4.6, 0.41, 1.25};
        else if (edge == 128) t = {0.48, 0.8, 0.39, 0.6};
        else t = {0.2, 0, 0.44, 0.19};
        double work = 0, longest = 0;
        long all = 0;
        for (int i = 0; i < m; ++i) {
            const double span = ((p[i].sum ? even_rows(R, n) : p[i].K) + stage_elems - 1) / stage_elems;
            all += group_grid(p[i], R, n, edge);
            work += group_tiles(p[i], R, n, edge) * (span * t.stage + t.tile) / 256;
            longest = std::max(longest, span);
        }
        if (!grid_fits(all, tile_threads(edge))) continue;
        const double us = std::max(longest * t.alone + 5, work + longest * t.end) + 2;
        if (best == 0 || us < least) {
            least = us;
            best = edge;
        }
    }
    return best;
}

}  // namespace gemm
}  // namespace moe
