// mla_tree_plan.h -- how the tree decode cuts a batch's blocks into ranges, and how many ranges a call has.
// Plain arithmetic, compiled for the device and, by the tests, for the host.
#pragma once

#include "mla_dense_plan.h"

namespace dsa {

constexpr int kTreeSegUnits = 4;     // a request's fixed cost in a range (q, first products, output), in blocks
constexpr int kTreeWholeBlocks = 3;  // requests of at most this many blocks are not split
constexpr int kTreeMaxRanges = 256;  // of a tile
constexpr int kTreeMaxUnits = 512;   // of a call
constexpr int kTreeMaxTiles = 16;
constexpr int kTreeMaxRounds = 8;    // units of a cluster, at most
constexpr int kTreePlanRounds = 4;   // rounds that are tried for a full device

// A request's pages: the live ones of the cache and one of its drafted tokens, where it has any.
DSA_PLAN int tree_cache_pages(int tokens) { return (((tokens + 3) >> 2) + 63) >> 6; }
// Its blocks of two pages.
DSA_PLAN int tree_blocks(int cache_pages, int drafted) { return drafted > 0 ? (cache_pages + 2) >> 1 : 0; }
DSA_PLAN int tree_units(int blocks) { return blocks ? blocks + kTreeSegUnits : 0; }

// Where a cut inside a request of `blocks` blocks, whose units start at u, comes to lie.
DSA_PLAN int tree_settled_cut(int cut, int u, int blocks) {
    const int n = tree_units(blocks);
    return blocks > kTreeWholeBlocks ? cut : ((cut - u) * 2 < n ? u : u + n);
}

// Tiles of drafted tokens, each a unit in every range.
constexpr int kTileTokens = 4, kPairTokens = 2;  // of a cluster of four CTAs, of two
DSA_PLAN int tree_tiles(int tokens) { return (tokens + kTileTokens - 1) / kTileTokens; }
// Partial outputs of a range: places of two each.
DSA_PLAN int tree_places(int tokens) { return tokens <= kPairTokens ? tokens : kTileTokens; }

// The most ranges of a call on `clusters` clusters: as many as fill them in few rounds.  A round more is worth
// it for a twentieth of the device.
DSA_PLAN int tree_ranges(int tiles, int clusters) {
    int best = 1, best_rounds = 0, best_units = 0;  // units: of best_rounds * clusters places
    for (int k = 1; k <= kTreePlanRounds; ++k) {
        int r = k * clusters / tiles;
        if (r > kTreeMaxRanges) r = kTreeMaxRanges;
        if (r < 1) continue;
        // r tiles / (k clusters) against best_units / (best_rounds clusters) + 1 / 20
        if (best_rounds == 0 || 20 * (r * tiles * best_rounds - best_units * k) > k * best_rounds * clusters)
            best = r, best_rounds = k, best_units = r * tiles;
    }
    return best;
}

// What `ranges` of `total` plan units cost, in sixteenths of a block: the units that a cluster does one after
// another, each with its own start and end, and the partial outputs that the merge reads.
constexpr int kTreeUnitCost = 96, kTreeMergeCost = 64;
DSA_PLAN long long tree_cost(int ranges, int total, int tiles, int clusters, int tokens) {
    const long long rounds = (ranges * tiles + clusters - 1) / clusters, each = (total + ranges - 1) / ranges;
    return rounds * (16 * each + kTreeUnitCost) + (ranges > 1 ? kTreeMergeCost + ranges * tokens * 3 / 4 : 0);
}

// Trees of different sizes: tile t has the requests with more than so many tokens, and ranges of its own, of about
// `each` plan units in every tile.  The same costs, for `units` ranges of all tiles.
DSA_PLAN int tree_line_ranges(int total, int each) { return (total + each - 1) / each; }
DSA_PLAN long long tree_cost_ragged(int units, int each, int tiles, int clusters) {
    const long long rounds = (units + clusters - 1) / clusters;
    return rounds * (16 * each + kTreeUnitCost) + (units > tiles ? kTreeMergeCost + 3 * units : 0);
}
// Where range g of tile t comes among all: by how far into its tile its middle lies, so that the tiles of a request
// run at about the same time.  Tile t's ranges are numbered first[t], .., first[t + 1] - 1.  (With equal tiles it is
// g * tiles + t.)
DSA_PLAN int tree_rank(const int* first, int tiles, int t, int g) {
    const int n = first[t + 1] - first[t];
    int rank = 0;
    for (int o = 0; o < tiles; ++o) {  // (2 i + 1) / others < (2 g + 1) / n
        const int others = first[o + 1] - first[o], x = (2 * g + 1) * others;
        const int before = ((o < t ? x : x - 1) / n + 1) / 2;
        rank += x == 0 ? 0 : (before < others ? before : others);
    }
    return rank;
}

}  // namespace dsa
