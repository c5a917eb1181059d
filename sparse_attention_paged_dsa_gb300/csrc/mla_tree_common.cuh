// mla_tree_common.cuh -- what the tree decode's two kernels on clusters share: the
// plan of a call, the walk over it, and the drafted pages.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "cta_pair.cuh"
#include "indexer_kernels.h"
#include "mla_tree_plan.h"

namespace dsa {

constexpr int kTreeThreads = 384;  // (a thirteenth warp would leave the softmax 128 registers)
constexpr int kPg = kPageEntries;      // entries of a page, heads of a token
constexpr int kSoftWarps = 8;
constexpr float kLn2T = 0.69314718055994531f;

struct UnitT {
    int lo, hi;                  // the range, in units of the plan
    int first_req, first_start;  // request of its first unit, and where that request's units start
    int range, tile;             // among the ranges of all tiles
};

// In shared memory: a cluster's units.
struct TreePlan {
    UnitT unit[kTreeMaxRounds];
    int cut[kTreeMaxRounds];     // the request that the range is the second one of, or -1
    int first[kTreeMaxTiles + 1];  // a tile's first range
    int line[kTreeMaxTiles];       // a tile's plan units
    int warp_units[16];
    uint64_t warp_best[16];
};

__device__ __forceinline__ bool soft_or(bool v) {  // over the 256 softmax threads
    __syncwarp();  // (it stands behind waits that spin lane by lane)
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred pi, po;\n\t"
        "setp.ne.u32 pi, %1, 0;\n\t"
        "bar.red.or.pred po, 1, 256, pi;\n\t"
        "selp.u32 %0, 1, 0, po;\n\t}"
        : "=r"(r)
        : "r"(v ? 1u : 0u)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void wait_landed_t(uint64_t* bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(a, parity) && global_timer_ns() - t0 < kWaitLimitNs) {
    }
}

__device__ __forceinline__ int tree_tokens(const MlaTreeParams& p, int b) {  // cached, in [0, max_context]
    const int seq = __ldg(p.seq_lens + b);
    return seq < 0 ? 0 : (int64_t(seq) > p.max_context ? int(p.max_context) : seq);
}
__device__ __forceinline__ int tree_drafted(const MlaTreeParams& p, int b) {  // in [0, tokens]
    if (!p.counts) return p.tokens;
    return min(max(__ldg(p.counts + b), 0), p.tokens);
}
__device__ __forceinline__ uint64_t low_bits(int n) { return n >= 64 ? ~uint64_t(0) : (uint64_t(1) << n) - 1; }

// The cluster's walk over its units: one step per request that has blocks in a unit's range and tokens
// in its tile of kTile.
template <int kTile>
struct TreeWalk {
    int k, rounds;
    int b, u0, lo, hi;
    int range, tile;
    int np, live, drafted, nb, blo, bhi;  // current request: cache pages, entries, drafted tokens, blocks
    __device__ __forceinline__ TreeWalk(int first_, int step_, int units)
        : k(-1), rounds(first_ < units ? (units - first_ + step_ - 1) / step_ : 0), b(0), u0(0), lo(0), hi(0),
          range(0), tile(0), np(0), live(0), drafted(0), nb(0), blo(0), bhi(0) {}
    __device__ __forceinline__ bool next(const MlaTreeParams& p, const TreePlan& plan) {
        while (true) {
            while (b < p.batch && u0 < hi) {
                const int seq = tree_tokens(p, b);
                live = (seq + 3) >> 2;
                np = tree_cache_pages(seq);
                drafted = tree_drafted(p, b);
                nb = tree_blocks(np, drafted);
                const int base = u0 + kTreeSegUnits, end = u0 + (kTile * tile < drafted ? tree_units(nb) : 0);
                blo = max(lo, base) - base;
                bhi = min(hi, end) - base;
                ++b;
                u0 = end;
                if (bhi > blo) return true;
            }
            if (++k >= rounds) return false;
            // (In one build the softmax warps read these while they were still cleared, behind a cluster barrier to which
            // their lanes could come apart; the barriers meet the warp first since, and these are read from memory each time.)
            const volatile UnitT& unit = plan.unit[k];
            range = unit.range, tile = unit.tile, lo = unit.lo, hi = unit.hi, b = unit.first_req, u0 = unit.first_start;
        }
    }
    __device__ __forceinline__ int req() const { return b - 1; }
    // Entries of a page that somebody may see, if its id is good.
    __device__ __forceinline__ int valid(int page) const {
        return page < np ? min(live - page * kPg, kPg) : (page == np ? drafted : 0);
    }
    // Has a page value rows to zero?  (The drafted page always, by the masks.)
    __device__ __forceinline__ bool zeroes(int page) const {
        return page == np || (page < np && ((live - page * kPg) < kPg) && ((live & 15) != 0));
    }
};

// Ids of pages [page0, page0 + 32) of the current request, a lane each: -1 where the table's is outside the
// cache, -2 for the drafted page and those behind it.
template <int kTile>
__device__ __forceinline__ int tree_page_of_lane(const MlaTreeParams& p, const TreeWalk<kTile>& w, int page0,
                                                 int lane) {
    const int page = page0 + lane;
    if (page >= w.np) return -2;
    const int id = __ldg(p.page_table + int64_t(w.req()) * p.table_width + page);
    return (id >= 0 && int64_t(id) < p.num_pages) ? id : -1;
}

__device__ __forceinline__ void clear_plan(const MlaTreeParams& p, TreePlan& plan) {
    for (int k = 0; k < kTreeMaxRounds; ++k) {
        plan.unit[k] = {0, 0, p.batch, 0, 0, 0};
        plan.cut[k] = -1;
    }
    for (int t = 0; t <= kTreeMaxTiles; ++t) plan.first[t] = 0;
}

// Finds the cluster's units, from the prefix sums of the requests' plan units (a tile's: of those that have tokens in
// it); returns how many the call has.  For all threads, the plan cleared; it is there after the caller's next barrier.
template <int kTile>
__device__ __forceinline__ int find_units(const MlaTreeParams& p, TreePlan& plan, int cluster, int clusters) {
    const int warp = int(threadIdx.x) >> 5, lane = threadIdx.x & 31;
    const int per = (p.batch + kTreeThreads - 1) / kTreeThreads;
    const int r0 = min(int(threadIdx.x) * per, p.batch), r1 = min(r0 + per, p.batch);
    const bool ragged = kTile == kTileTokens && p.counts;  // (a pair has one tile)
    const auto blocks_in = [&](int b, int tile) {
        const int drafted = tree_drafted(p, b);
        return kTile * tile < drafted ? tree_blocks(tree_cache_pages(tree_tokens(p, b)), drafted) : 0;
    };
    // The tile whose prefix sums are known: where this thread's requests start, and its plan units.
    int start = 0, total = 0, known = -1;
    const auto scan = [&](int tile) {
        if (known == tile || (known >= 0 && !ragged)) return;
        const bool again = known >= 0;
        known = tile;
        int mine = 0;
#pragma unroll 1
        for (int b = r0; b < r1; ++b) mine += tree_units(blocks_in(b, tile));
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (again) __syncthreads();
        if (lane == 31) plan.warp_units[warp] = incl;
        __syncthreads();
        start = incl - mine, total = 0;
        for (int w = 0; w < kTreeThreads / 32; ++w) {
            if (w < warp) start += plan.warp_units[w];
            total += plan.warp_units[w];
        }
    };
    if (blockIdx.x == 0)
        for (int b = r0; b < r1; ++b) {
            const int seq = __ldg(p.seq_lens + b);
            if (seq < 0 || int64_t(seq) > p.max_context) atomicOr(p.err, kErrSeqLenClamped);
            if (p.counts && tree_drafted(p, b) != __ldg(p.counts + b)) atomicOr(p.err, kErrBadRange);
        }
    scan(0);
    if (ragged) {  // what each tile has
        for (int b = r0; b < r1; ++b)
            if (const int n = tree_units(blocks_in(b, 0)))
                atomicAdd(&plan.first[(tree_drafted(p, b) - 1) / kTile], n);
        __syncthreads();
        if (int(threadIdx.x) < p.tiles) {
            int sum = 0;
            for (int t = threadIdx.x; t < p.tiles; ++t) sum += plan.first[t];
            plan.line[threadIdx.x] = sum;
        }
        __syncthreads();
    }
    // How many ranges (ragged: of tile 0): a thread for each number.
    uint64_t best = ~uint64_t(0);
    for (int r = int(threadIdx.x) + 1; r <= min(ragged ? kTreeMaxRanges : p.ranges, total); r += kTreeThreads) {
        uint64_t cost;
        if (ragged) {
            const int each = (total + r - 1) / r;
            int units = 0;
            for (int t = 0; t < p.tiles; ++t) units += tree_line_ranges(plan.line[t], each);
            if (units > p.ranges * p.tiles) continue;  // (one of each tile never are)
            cost = uint64_t(tree_cost_ragged(units, each, p.tiles, p.clusters));
        } else {
            cost = uint64_t(tree_cost(r, total, p.tiles, p.clusters, p.tokens));
        }
        cost = cost << 16 | uint64_t(r);
        best = cost < best ? cost : best;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const uint64_t y = __shfl_xor_sync(0xffffffffu, best, o);
        best = y < best ? y : best;
    }
    if (lane == 0) plan.warp_best[warp] = best;
    __syncthreads();
    for (int w = 0; w < kTreeThreads / 32; ++w) best = plan.warp_best[w] < best ? plan.warp_best[w] : best;
    const int nranges = total > 0 ? int(best & 0xFFFF) : 1;
    int units = nranges * p.tiles;
    if (ragged) {
        const int each = total > 0 ? (total + nranges - 1) / nranges : 1;
        if (threadIdx.x == 0) {
            int n = 0;
            for (int t = 0; t < p.tiles; ++t) {
                plan.first[t] = n;
                n += tree_line_ranges(plan.line[t], each);
            }
            plan.first[p.tiles] = n;
        }
        __syncthreads();
        units = plan.first[p.tiles];
        for (int i = threadIdx.x; i < units; i += kTreeThreads) {
            int t = 0;
            while (plan.first[t + 1] <= i) ++t;
            const int rank = tree_rank(plan.first, p.tiles, t, i - plan.first[t]);
            if (rank % clusters == cluster) {
                plan.unit[rank / clusters].range = i;
                plan.unit[rank / clusters].tile = t;
            }
        }
        __syncthreads();
    }
    const auto first_of = [&](int tile) { return ragged ? plan.first[tile] : tile * nranges; };
#pragma unroll 1
    for (int k = 0; cluster + k * clusters < units; ++k) {
        int tile, g;
        if (ragged) {
            tile = plan.unit[k].tile, g = plan.unit[k].range - plan.first[tile];
        } else {
            const int u = cluster + k * clusters;
            g = u / p.tiles, tile = u - g * p.tiles;
            if (threadIdx.x == 0) plan.unit[k].range = tile * nranges + g, plan.unit[k].tile = tile;
        }
        scan(tile);
        const Ranges ranges(first_of(tile + 1) - first_of(tile), total);
        const int lo = ranges.cut(g), hi = ranges.cut(g + 1);
        if (threadIdx.x == 0) {  // cuts at the very end lie in no request
            if (lo == total) plan.unit[k].lo = total;
            if (hi == total) plan.unit[k].hi = total;
        }
        int u = start;
        for (int b = r0; b < r1; ++b) {
            const int nb = blocks_in(b, tile), n = tree_units(nb);
            if (lo >= u && lo < u + n) {
                plan.unit[k].lo = tree_settled_cut(lo, u, nb);
                plan.unit[k].first_req = b;
                plan.unit[k].first_start = u;
            }
            if (hi >= u && hi < u + n) plan.unit[k].hi = tree_settled_cut(hi, u, nb);
            // Is this the request's second range?  Its first block lies in the one before.
            if (nb > kTreeWholeBlocks && lo > u + kTreeSegUnits && lo < u + n && ranges.cut(g - 1) <= u + kTreeSegUnits)
                plan.cut[k] = b;
            u += n;
        }
    }
    // The first and last range that hold a request's blocks, for the merge: a tile a CTA.
#pragma unroll 1
    for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        scan(tile);
        const int first = first_of(tile);
        const Ranges ranges(max(first_of(tile + 1) - first, 1), total);
        int u = start;
        for (int b = r0; b < r1; ++b) {
            const int nb = blocks_in(b, tile), n = tree_units(nb);
            p.plan[tile * p.batch + b] = nb > kTreeWholeBlocks ? make_int2(first + ranges.of(u + kTreeSegUnits),
                                                                           first + ranges.of(u + n - 1))
                                                               : make_int2(0, 0);
            u += n;
        }
    }
    __syncthreads();
    return units;
}

// The cuts of the cluster's ranges, and its part of those that no range has, for the merge (16 request + tile, or
// -1); by one thread.
__device__ __forceinline__ void write_cuts(const MlaTreeParams& p, const TreePlan& plan, int cluster, int clusters,
                                           int units) {
    for (int k = 0; cluster + k * clusters < p.ranges * p.tiles; ++k) {
        const int u = cluster + k * clusters;
        const volatile UnitT& unit = plan.unit[k];
        const int b = *const_cast<const volatile int*>(&plan.cut[k]);
        if (u < units)
            p.cuts[unit.range] = b < 0 ? -1 : 16 * b + unit.tile;
        else
            p.cuts[u] = -1;
    }
}

// A box's rows (32 or 64) of one slab of a request's drafted entries (rows behind the last arrive as zeros).
__device__ __forceinline__ void load_drafts(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t row,
                                            int32_t slab, int32_t request, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(slab), "r"(request), "r"(bar), "l"(policy)
        : "memory");
}

// What some token of the current request sees of its drafted entries; by a whole warp.
template <int kTile>
__device__ __forceinline__ uint64_t drafts_seen(const MlaTreeParams& p, const TreeWalk<kTile>& w, int lane) {
    uint64_t any = 0;
    for (int j = lane; j < w.drafted; j += 32) any |= __ldg(p.mask + int64_t(w.req()) * p.tokens + j);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) any |= __shfl_xor_sync(0xffffffffu, any, o);
    return any & low_bits(w.drafted);
}

// Zeroes the value rows of a page (in kSlabs slabs of 64 x 64) that nobody sees, up to the last 16-entry step of the
// product: their weights are 0, but 0 x NaN is not.  By a whole warp, once the page has landed.  Out of line: the
// loops of the roles run side by side and share an instruction cache.
template <int kSlabs>
__device__ __noinline__ void zero_unseen(uint64_t used, int valid, uint8_t* v) {
    const int lane = threadIdx.x & 31;
    const int rows = (valid + 15) & ~15;
#pragma unroll 1
    for (int c = lane; c < rows * 8; c += 32) {
        if ((used >> (c >> 3)) & 1u) continue;
#pragma unroll
        for (int s = 0; s < kSlabs; ++s)
            *reinterpret_cast<uint4*>(v + s * (kPg * 128) + c * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    __syncwarp();
}

}  // namespace dsa
