// mla_prefill_kernel.cu -- latent attention over a ragged batch of prompts or
// prompt chunks (expanded form), sm_103a.
//
//     s[i, t] = sm_scale * (q[i, h, :128] . k_nope[t, h] + q[i, h, 128:] . k_rope[t])
//     o[i, h] = sum_t softmax_t(s[i, :]) v[t, h],   lse[i, h] = log sum_t exp(s[i, t])
//
// Row i of a request with n rows and seq_len tokens sees its first
// ceil((seq_len - (n - 1 - i)) / entry_tokens) entries: whole ones, whatever tokens
// behind the row's own the last of them holds.
//
// A cluster of two CTAs works on two query tiles of 256 rows at a time, each CTA
// holding 128 rows of both.  All MMAs are cta_group::2 (M = 256: 128 rows in each
// CTA's TMEM; N = 128), issued by the leader.  Their second operand is split between
// the two CTAs' shared memory: each loads half of every 128-entry tile's keys (64
// entries) and half of its values (64 dims), so a tile costs an SM 40 KB of loads
// instead of 80, its shared memory holds three tiles, and the operand reads fit its
// bandwidth.
//
// Work.  A unit is 512 rows of a request and one head, whose two tiles share the
// keys and values; or 256 rows and two heads, one a tile (see Cut).  Clusters are
// persistent: the units, longest requests and their last rows first, are dealt out
// back and forth over the clusters that fit the device, and the next unit's loads and
// first product run under the end of the one before (a unit's own set-up and tail cost
// 9 us without that).  The units behind the last whole round of the clusters are cut
// along their entries where that pays (parts_of); parts leave fp32 outputs and a second
// kernel joins them by log-sum-exp (one row of 64 heads over 16,385 entries: 136 us,
// uncut 249; 300 rows of two heads over 33,068: 42, uncut 386; 128 units of 256 key
// tiles: 750, uncut 805).  Units of equal cost laid end to end and cut once per cluster
// balance better, but cost more to find and to join: 735 there, 8192 rows of 32 heads
// 484 against 407.  A scheduler warp looks the units up.  Roles of a CTA (384 threads):
//   * warps 0-3 and 4-7: softmax of query tile 0 and 1, one row per thread: the
//     row of S from TMEM to registers, its maximum (raised only when a tile
//     passes it by more than 2^20; the accumulator is then rescaled in TMEM),
//     2^x, and P (bf16) back into S's columns; at the end the output.
//   * warp 8 (leader): tcgen05.mma.  S = Q . K^T from shared memory (12 steps);
//     O += P . V with P from TMEM and V read in place as an MN-major operand (up to
//     8 steps).  Order per tile: PV of query tile 0, its next QK, PV of query tile
//     1, its next QK, so that one tile's products run while the other's softmax does.
//   * warp 9: TMA.  q; keys (two 64-dim slabs of the head's own, one shared
//     by all heads) and values, three stages each.  Both CTAs' copies count on the
//     leader's barriers.
//   * warp 10: zeroes the value rows behind the last entry (see Unit::tail).
//   * warp 11: the scheduler.
// TMEM: S/P of the two tiles 2 x 128 columns, O 2 x 128: all 512.
//
// The shared 64 rotary key dims are loaded from their one copy per entry, so no
// 192-wide key is ever built, and every operand may be a strided view.
//
// What bounds it: the tensor cores: 20 MMA steps of 128 x 128 x 16 per SM for each
// (128 rows, 128 entries), 1,280 SM cycles at full rate.  8192 rows of 32 heads: 407 us,
// 1690 TFLOP/s, 0.88 of the measured bf16 rate; 1024 rows of 64 heads over 32,768
// entries: 750 us, 0.95.  Short prompts are bound by a unit's ends: 32 prompts of 512
// rows and 32 heads 143 us (0.62), 64 of 100 rows and 64 heads 120 (0.39 of the bytes).
// Every wait is bounded (about 1 s) but the cluster barriers, which every thread
// reaches; a timeout sets an error bit, the roles drain, and TMEM is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "cta_pair.cuh"
#include "indexer_kernels.h"
#include "mla_common.cuh"
#include "mla_prefill_plan.h"
#include "sm103_ptx.cuh"

namespace dsa {
namespace {

constexpr int kTile = 128;                      // rows of a CTA's query tile, entries of a key tile
constexpr int kSlabB = kTile * 128;             // 128 rows x 64 bf16 dims, 16 KiB
constexpr int kHalfB = kSlabB / 2;              // 64 rows x 64 dims: a CTA's half of a key slab
constexpr int kQkSlabs = kPrefillQk / 64;       // 3: two of the head's own, one rotary
constexpr int kStages = 3;                      // key and value tiles in shared memory
constexpr int kStageK = kQkSlabs * kHalfB;      // 24 KiB
constexpr int kStageV = kSlabB;                 // 128 entries x this CTA's 64 value dims
constexpr int kOffQt = 0;                       // q: 2 tiles x 3 slabs
constexpr int kOffK = kOffQt + 2 * kQkSlabs * kSlabB;
constexpr int kOffV = kOffK + kStages * kStageK;
constexpr int kOffCtlP = kOffV + kStages * kStageV;
constexpr int kThreadsP = 384;
static_assert(2 * kTile == kPrefillPair, "a cluster's query tile");
constexpr int kRegsSoftmax = 208, kRegsOther = 88;  // 8 x 208 + 4 x 88 = 12 x 168 a warp lane
constexpr uint32_t kTmemColsP = 512;
constexpr uint32_t kColSP = 0;    // S / P of tile i at 128 i
constexpr uint32_t kColOP = 256;  // O of tile i at 256 + 128 i
constexpr float kRaiseLog2 = 20.0f;  // rounding is relative: weights may pass 1 by this much
constexpr float kLn2P = 0.69314718055994531f;

constexpr int kPartTiles = 4;        // key tiles a part has at least (2: no faster; 8: 64 rows of 20 heads
                                     // over 2,064 entries took 29 us, now 24)
constexpr int kSortMost = 256;       // requests that are ordered by length, one a thread (more: as they come)
constexpr int kInfoSlots = 4;
constexpr int kInfoReaders = 11;     // every warp but the scheduler

// What a cluster works on: two query tiles, or fewer.  Tile i is rows [i step_row, + 256) of the block
// (those of them below `rows`) of head `head` + i step_head.
struct Unit {
    int q_row;               // row of q where the block starts
    int row0;                // the same within the request
    int rows;                // of the block
    int req_rows, seq, live; // of the request: rows, tokens, entries
    int kv0;                 // its first entry
    int head;
    int step_row, step_head; // (256, 0): the tiles share keys and values; (0, 1)
    int limit[2];            // entries that the tile's last row sees; 0 without a tile
    int skip;                // entries before this part's first one (kv0 and limit are the part's)
    int part;                // where its output goes, -1: the output itself
    int last;                // no unit: the list is at its end

    __device__ __forceinline__ bool shared() const { return step_head == 0; }
    __device__ __forceinline__ int tiles(int i) const { return (limit[i] + kTile - 1) / kTile; }
    // Streams of keys and values, and tiles in each.
    __device__ __forceinline__ int streams() const { return shared() || limit[1] == 0 ? 1 : 2; }
    __device__ __forceinline__ int nt() const { return max(tiles(0), tiles(1)); }
    __device__ __forceinline__ int limit_max() const { return max(limit[0], limit[1]); }
    // Value rows behind the last entry that any of these rows sees belong to other requests or hold
    // nothing.  Products stop at a 16-entry step, and where that is not the end of the entries the rows
    // up to it are zeroed (weights there are 0, but 0 x NaN is not): such a last tile's values count on
    // a barrier of each CTA, whose warp 10 zeroes them and tells the leader.  Those barriers are the
    // stage's: the loads run ahead of the products by units, and a barrier takes one fill at a time.
    __device__ __forceinline__ bool tail() const { return (limit_max() & 15) != 0; }
};

struct __align__(8) PrefillCtl {
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], o_empty[2];
    uint64_t tail_landed[kStages], tail_ready[kStages];  // per value stage
    uint64_t info_full[kInfoSlots], info_empty[kInfoSlots];
    uint64_t all_done;
    uint32_t tmem_base;
    int abort;
    int total, list;                   // units; entries of the list below
    int warp_units[kThreadsP / 32];
    Unit info[kInfoSlots];
    int first[kMaxBatch];              // first unit of the i-th entry of the list
    int order[kMaxBatch];              // its request, the kind of order, and its first unit there (ListEntry)
    union {
        int live[kSortMost];
        uint16_t tiles[2 * kSortMost];
    } key;
};
constexpr int kSmemP = 1024 + kOffCtlP + int(sizeof(PrefillCtl));
static_assert(kSmemP <= 232448, "fits one CTA per SM");

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Entries seen by a row whose last visible token is number `len` (from 1).
__device__ __forceinline__ int entries_seen(int len, int entry_tokens) {
    return len > 0 ? (len - 1) / entry_tokens + 1 : 0;
}

// A request's rows, entries and lengths, held to the tensors' extents; 0 rows where cu_q is out of
// order or range.  `bad` collects error bits.
struct Request {
    int q0, rows, kv0, live, seq;
    __device__ __forceinline__ Request(const PrefillParams& p, int b, uint32_t& bad) {
        q0 = __ldg(p.cu_q + b);
        const int q1 = __ldg(p.cu_q + b + 1);
        rows = q1 - q0;
        if (q0 < 0 || q1 < q0 || q1 > p.q_rows) {
            bad |= kErrBadRange;
            q0 = rows = 0;
        }
        kv0 = __ldg(p.cu_kv + b);
        const int kv1 = __ldg(p.cu_kv + b + 1);
        int entries = kv1 - kv0;
        if (kv0 < 0 || kv1 < kv0 || kv1 > p.kv_rows) {
            bad |= kErrBadRange;
            kv0 = entries = 0;
        }
        seq = __ldg(p.seq_lens + b);
        if (seq < 0) {
            bad |= kErrSeqLenClamped;
            seq = 0;
        }
        live = entries_seen(seq, p.entry_tokens);
        if (live > entries) {
            bad |= kErrBadRange;
            live = entries;
        }
    }
    // Entries that row i sees.
    __device__ __forceinline__ int seen(int i, int entry_tokens) const {
        const int64_t len = int64_t(seq) - (int64_t(rows) - 1 - i);
        return min(entries_seen(len > 0 ? int(len) : 0, entry_tokens), live);
    }
};

__device__ __forceinline__ void wait_landed_p(uint64_t* bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(a, parity) && global_timer_ns() - t0 < kWaitLimitNs) {
    }
}

// Do a request's blocks of 512 rows see about equally many entries (a chunk on a long past)?  A head's
// blocks then follow one another, so that its keys and values are in L2 for all but the first (1024 rows of
// 64 heads over 32,768 entries in a long run, which power limits: 871 -> 838 us; alone 756 -> 750).
__device__ __forceinline__ bool blocks_alike(const PrefillParams& p, const Request& rq) {
    return rq.seen(kPrefillBlock - 1, p.entry_tokens) >= rq.live - rq.live / 4;
}
// Groups of a request's units, in their order: a block each, or all the alike ones.
__device__ __forceinline__ int groups_of(const PrefillParams& p, const Request& rq, const Cut& cut) {
    return cut.pair_blocks + (cut.long_blocks > 1 && blocks_alike(p, rq) ? 1 : cut.long_blocks);
}
__device__ __forceinline__ int group_start(const Cut& cut, int group) {
    return min(group, cut.pair_blocks) * cut.pairs() + max(group - cut.pair_blocks, 0) * cut.heads;
}
// Key tiles of a group's (longest) units.
__device__ __forceinline__ int group_tiles(const PrefillParams& p, const Request& rq, const Cut& cut, int group) {
    const int pair = cut.pair_blocks - 1 - group;
    const int end = pair >= 0 ? cut.long_blocks * kPrefillBlock + (pair + 1) * 2 * kTile
                              : (cut.long_blocks + pair + 1) * kPrefillBlock;
    return (rq.seen(min(end, rq.rows) - 1, p.entry_tokens) + kTile - 1) / kTile;
}

// The request's unit number `at`, last rows (the longest) first: the blocks for two heads lie behind the
// long ones.
__device__ __forceinline__ Unit unit_of(const PrefillParams& p, const Request& rq, bool alike, int at) {
    const Cut cut(rq.rows, rq.live, p.heads);
    Unit u = {};
    if (at < cut.pair_blocks * cut.pairs()) {
        u.row0 = cut.long_blocks * kPrefillBlock + (cut.pair_blocks - 1 - at / cut.pairs()) * 2 * kTile;
        u.rows = min(rq.rows - u.row0, 2 * kTile);
        u.head = at % cut.pairs() * 2;
        u.step_head = 1;
    } else {
        at -= cut.pair_blocks * cut.pairs();
        const int block = alike ? at % cut.long_blocks : at / p.heads;
        u.row0 = (cut.long_blocks - 1 - block) * kPrefillBlock;
        u.rows = min(rq.rows - u.row0, kPrefillBlock);
        u.head = alike ? at / cut.long_blocks : at % p.heads;
        u.step_row = 2 * kTile;
    }
    u.q_row = rq.q0 + u.row0;
    u.req_rows = rq.rows, u.seq = rq.seq, u.live = rq.live, u.kv0 = rq.kv0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int from = i * u.step_row, to = min(u.rows, from + 2 * kTile);
        const bool there = to > from && u.head + i * u.step_head < p.heads;
        u.limit[i] = there ? rq.seen(u.row0 + to - 1, p.entry_tokens) : 0;
    }
    u.part = -1;
    return u;
}

// An entry of the list: units of a request from number `start` on (16 bits: of at most 384 groups of 128).
__device__ __forceinline__ int list_entry(int request, bool alike, int start) {
    return request << 17 | int(alike) << 16 | start;
}
// Unit n of the list, for a whole warp.
__device__ __forceinline__ Unit unit_at(const PrefillParams& p, const PrefillCtl& ctl, int n, int lane) {
    int lo = 0;  // the last entry that starts at or before it: 32-way, twice
    for (int span = 32; span >= 1; span /= 32) {
        const int at = lo + lane * span;
        const bool before = at < ctl.list && ctl.first[at] <= n;
        lo += span * (__popc(__ballot_sync(0xffffffffu, before)) - 1);
    }
    // requests without rows start where the next one does: the last of them is the owner
    const int entry = ctl.order[lo];
    uint32_t ignored = 0;
    return unit_of(p, Request(p, entry >> 17, ignored), (entry >> 16) & 1, n - ctl.first[lo] + (entry & 0xFFFF));
}

// Into how many parts to cut each of `units` units of `tiles` key tiles, the last ones, which would leave
// some of the clusters idle.  In key tiles: a unit costs 3 beside its own, a second launch and its reading
// 6 and 1 for every 36 parts.  Parts go round the clusters at most kRounds times.
constexpr int kRounds = 3;
__host__ __device__ __forceinline__ int parts_of(int units, int tiles, int clusters) {
    int best = 1, least = tiles + 3;
    for (int rounds = 1; units > 0 && rounds <= kRounds; ++rounds) {
        int parts = rounds * clusters / units;
        if (parts > tiles / kPartTiles) parts = tiles / kPartTiles;
        if (parts < 2) continue;
        const int goes = (units * parts + clusters - 1) / clusters;
        const int cost = goes * ((tiles + parts - 1) / parts + 3) + 6 + units * parts / 36;
        if (cost < least) best = parts, least = cost;
    }
    return best;
}

// kSplit: units may be cut into parts.  (In a kernel of its own: the choice made at run time in one took
// 64 prompts of 100 rows, which are not cut, from 119 to 131 us.)
// kGroups: several long prompts, whose units are ordered by their groups.
template <bool kSplit, bool kGroups>
__global__ void __launch_bounds__(kThreadsP, 1) __cluster_dims__(2, 1, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kn_map,
                       const __grid_constant__ CUtensorMap kr_map, const __grid_constant__ CUtensorMap v_map,
                       const __grid_constant__ CUtensorMap kn16_map, const __grid_constant__ CUtensorMap kr16_map,
                       const __grid_constant__ CUtensorMap v16_map, const PrefillParams p) {
    extern __shared__ uint8_t smem_raw[];
    // Dynamic shared memory starts at the same offset in both CTAs, so the operands and barriers do too.
    uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    PrefillCtl& ctl = *reinterpret_cast<PrefillCtl*>(tiles + kOffCtlP);
    const uint32_t s_base = smem_u32(tiles);
    const int warp = uniform(int(threadIdx.x) >> 5);
    const int lane = threadIdx.x & 31;
    const int rank = int(cluster_rank());  // 0: the leader

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&ctl.k_full[i], 1);
            mbar_init(&ctl.k_empty[i], 1);
            mbar_init(&ctl.v_full[i], 1);
            mbar_init(&ctl.v_empty[i], 1);
            mbar_init(&ctl.tail_landed[i], 1);
            mbar_init(&ctl.tail_ready[i], 2);  // one arrival of each CTA
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.q_full[i], 1);
            mbar_init(&ctl.q_empty[i], 1);
            mbar_init(&ctl.s_full[i], 1);
            mbar_init(&ctl.p_full[i], 8);   // four warps of each CTA
            mbar_init(&ctl.o_full[i], 1);
            mbar_init(&ctl.o_empty[i], 8);  // the same
        }
        for (int i = 0; i < kInfoSlots; ++i) {
            mbar_init(&ctl.info_full[i], 1);
            mbar_init(&ctl.info_empty[i], kInfoReaders);
        }
        mbar_init(&ctl.all_done, 1);
        ctl.abort = 0;
        fence_mbar_init();
        tma_prefetch_map(&q_map);
        tma_prefetch_map(&kn_map);
        tma_prefetch_map(&kr_map);
        tma_prefetch_map(&v_map);
        tma_prefetch_map(&kn16_map);
        tma_prefetch_map(&kr16_map);
        tma_prefetch_map(&v16_map);
    }
    if (warp == 8) tmem2_alloc(&ctl.tmem_base, kTmemColsP);
    __syncwarp();
    tc_fence_before_sync();
    cluster_arrive();
    pdl_wait_prior_grid();
    pdl_allow_next_grid();

    // The list of the units: longest requests first, their last rows first; several long prompts by their
    // groups of units instead, longest first (four prompts of 2048 rows, 8 heads: 52 us, by requests 56; of
    // 5378 rows, 5 heads: 138, 175).  Many requests as they come.
    uint32_t bad = 0;
    const int me = threadIdx.x;
    int groups = 0;
    for (int b = me; b < p.batch; b += kThreadsP) {
        const Request r(p, b, bad);
        const Cut cut(r.rows, r.live, p.heads);
        ctl.first[b] = cut.units();
        ctl.order[b] = list_entry(b, blocks_alike(p, r), 0);
        if (b < kSortMost) ctl.key.live[b] = r.rows > 0 ? r.live : -1;
        if constexpr (kGroups) groups = groups_of(p, r, cut);  // (a thread has one request)
    }
    if (bad && blockIdx.x == 0) atomicOr(p.err, bad);
    // Sum over the threads before this one, and over all of them.
    const auto scan = [&](int mine, int& total) {
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) ctl.warp_units[warp] = incl;
        __syncthreads();
        int before = incl - mine;
        total = 0;
        for (int w = 0; w < kThreadsP / 32; ++w) {
            if (w < warp) before += ctl.warp_units[w];
            total += ctl.warp_units[w];
        }
        return before;
    };
    int list = p.batch;
    if (p.batch > 1 && p.batch <= kSortMost) {
        bool by_groups = false;
        if constexpr (kGroups) {
            int all = 0;
            const int start = scan(groups, all);
            by_groups = all <= kThreadsP;
            if (by_groups) {
                if (me < p.batch) ctl.order[me] = start;
                list = all;
            }
        }
        __syncthreads();
        int entry = 0, units = 0, key = 0, at = 0;
        if (me < list) {
            if (by_groups) {
                int b = 0;
                for (int step = kSortMost / 2; step > 0; step >>= 1)
                    if (b + step < p.batch && ctl.order[b + step] <= me) b += step;
                const int group = me - ctl.order[b];
                uint32_t ignored = 0;
                const Request r(p, b, ignored);
                const Cut cut(r.rows, r.live, p.heads);
                const bool last = group + 1 == groups_of(p, r, cut);
                const int from = group_start(cut, group);
                units = (last ? cut.units() : group_start(cut, group + 1)) - from;
                key = min(group_tiles(p, r, cut, group), 0xFFFF);
                entry = list_entry(b, blocks_alike(p, r), from);
            } else {
                units = ctl.first[me], entry = ctl.order[me], key = ctl.key.live[me];
            }
        }
        if (by_groups) {
            if (me < list) ctl.key.tiles[me] = uint16_t(key);
            __syncthreads();
            if (me < list)
                for (int o = 0; o < list; ++o) at += ctl.key.tiles[o] > key || (ctl.key.tiles[o] == key && o < me);
        } else if (me < list) {
            for (int o = 0; o < list; ++o) at += ctl.key.live[o] > key || (ctl.key.live[o] == key && o < me);
        }
        __syncthreads();
        if (me < list) {
            ctl.order[at] = entry;
            ctl.first[at] = units;
        }
    }
    __syncthreads();
    const int per = (list + kThreadsP - 1) / kThreadsP;
    const int i0 = min(me * per, list), i1 = min(i0 + per, list);
    int mine = 0, total_units = 0;
    for (int i = i0; i < i1; ++i) mine += ctl.first[i];
    int before = scan(mine, total_units);
    for (int i = i0; i < i1; ++i) {
        const int units = ctl.first[i];
        ctl.first[i] = before;
        before += units;
    }
    if (me == 0) ctl.total = total_units, ctl.list = list;
    __syncwarp();
    cluster_wait();  // the other CTA's barriers are set up too
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = ctl.tmem_base;

    // A warp's next unit, of which `read` takes what the warp needs; false at the end of the list or when
    // a role has given up.
    int taken = 0;
    const auto next_unit = [&](auto&& read) {
        const int slot = taken & (kInfoSlots - 1);
        const bool ok = mbar_await(&ctl.info_full[slot], uint32_t(taken / kInfoSlots) & 1u, &ctl.abort);
        if (!__all_sync(0xffffffffu, ok)) return false;
        read(ctl.info[slot]);
        const bool more = ctl.info[slot].last == 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.info_empty[slot]);
        ++taken;
        return more;
    };

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 11) {
        // ================= scheduler =================
        const int clusters = int(gridDim.x >> 1), cluster = int(blockIdx.x >> 1);
        // Units that go round the clusters whole times, then the parts of the others.
        int total = ctl.total, whole = total, parts = 1;
        if (kSplit && total > 0) {
            const int left = total % clusters;
            if (left > 0) parts = parts_of(left, unit_at(p, ctl, total - left, lane).nt(), clusters);
            if (parts > 1) whole = total - left, total = whole + left * parts;
        }
        if (kSplit && blockIdx.x == 0 && lane == 0) *p.split = make_int2(ctl.total - whole, parts);
        bool ok = true, more = true;
        for (int k = 0; ok && more; ++k) {
            const int slot = k & (kInfoSlots - 1);
            // dealt back and forth: what is longer in one round meets what is shorter in the next
            const int64_t n = int64_t(k) * clusters + ((k & 1) ? clusters - 1 - cluster : cluster);
            more = n < total;
            Unit u = {};
            u.last = more ? 0 : 1;
            if (more) {
                const int past = max(int(n) - whole, 0), part = past % parts;  // (1 part: 0)
                const int at = min(int(n), whole) + past / parts;
                u = unit_at(p, ctl, at, lane);
                if (kSplit && parts > 1 && int(n) >= whole) {
                    u.part = past;
                    if (part == 0 && rank == 0 && lane == 0) {
                        SplitUnit& out = p.split_units[at - whole];
                        out.q_row = u.q_row, out.rows = u.rows, out.head = u.head;
                        out.step_row = u.step_row, out.step_head = u.step_head;
                    }
                    const int nt = u.nt(), j0 = nt * part / parts, j1 = nt * (part + 1) / parts;
                    u.skip = j0 * kTile;
                    u.kv0 += u.skip;
#pragma unroll
                    for (int i = 0; i < 2; ++i) u.limit[i] = min(max(u.limit[i] - u.skip, 0), (j1 - j0) * kTile);
                }
            }
            ok = __all_sync(0xffffffffu, mbar_await(&ctl.info_empty[slot], (uint32_t(k / kInfoSlots) & 1u) ^ 1u,
                                                   &ctl.abort)) != 0;
            if (ok && lane == 0) {
                ctl.info[slot] = u;
                mbar_arrive(&ctl.info_full[slot]);
            }
            __syncwarp();
        }
        if (!ok && lane == 0) {
            atomicOr(p.err, kErrWaitTimeout);
            ctl.abort = 1;
        }
        __syncwarp();
    } else if (warp == 9) {
        // ================= TMA =================
        const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
        const bool issuer = elect_one();
        const uint32_t sb = uint32_t(uniform(int(s_base)));
        bool ok = true;
        int nk = 0, nv = 0;                       // key and value tiles so far
        int nq[2] = {0, 0};                       // q tiles
        uint32_t v_tail = 0, tail_phase = 0;      // value stages whose last fill counts on the tail barrier; its phases
        const auto wait = [&](uint64_t* bar, int fills) {  // the stage's `fills` earlier contents are used
            ok = ok && __all_sync(0xffffffffu, mbar_await(bar, (uint32_t(fills) & 1u) ^ 1u, &ctl.abort));
            return ok;
        };
        Unit u;
        while (ok && next_unit([&](const Unit& from) { u = from; })) {
            const int streams = u.streams(), nt = u.nt();
            const int limit = u.limit_max();
            const auto load_q = [&](int i) {  // a CTA whose 128 rows are all past the block loads none
                if (u.limit[i] == 0 || !wait(&ctl.q_empty[i], nq[i])) return;
                if (issuer) {
                    const uint32_t bar = cluster_addr(&ctl.q_full[i], 0);
                    const int rows = u.rows - i * u.step_row;
                    if (rank == 0)
                        mbar_arrive_expect_tx(&ctl.q_full[i], uint32_t((rows > kTile ? 2 : 1) * kQkSlabs * kSlabB));
                    if (rank == 0 || rows > kTile) {
#pragma unroll
                        for (int s = 0; s < kQkSlabs; ++s)
                            tma2_load_3d(sb + kOffQt + (i * kQkSlabs + s) * kSlabB, &q_map, bar, 64 * s,
                                         u.head + i * u.step_head, u.q_row + i * u.step_row + rank * kTile, pol_q);
                    }
                }
                __syncwarp();
                ++nq[i];
            };
            // Of a request's last tile only what lies before the limit is loaded, 16 entries at a time; the
            // rest of the stage keeps what it held (scores there are masked, value steps left out).
            const auto load_k = [&](int l, int j) {  // this CTA's 64 entries of tile j of stream l
                const int st = nk % kStages;
                if (!wait(&ctl.k_empty[st], nk / kStages)) return;
                if (issuer) {
                    const uint32_t bar = cluster_addr(&ctl.k_full[st], 0);
                    const int steps = min((limit - j * kTile + 15) >> 4, kTile / 16);  // of the tile, both CTAs
                    if (rank == 0) mbar_arrive_expect_tx(&ctl.k_full[st], uint32_t(steps * (2 * kStageK / (kTile / 16))));
                    const uint32_t dst = sb + kOffK + st * kStageK;
                    const int row = u.kv0 + j * kTile + rank * (kTile / 2), head = u.head + l;
                    const int mine = min(max(steps - rank * (kTile / 32), 0), kTile / 32);
                    if (mine == kTile / 32) {
                        tma2_load_3d(dst, &kn_map, bar, 0, head, row, pol_kv);
                        tma2_load_3d(dst + kHalfB, &kn_map, bar, 64, head, row, pol_kv);
                        tma2_load_2d(dst + 2 * kHalfB, &kr_map, bar, 0, row, pol_kv);
                    } else {
                        for (int s = 0; s < mine; ++s) {
                            tma2_load_3d(dst + s * 2048, &kn16_map, bar, 0, head, row + 16 * s, pol_kv);
                            tma2_load_3d(dst + kHalfB + s * 2048, &kn16_map, bar, 64, head, row + 16 * s, pol_kv);
                            tma2_load_2d(dst + 2 * kHalfB + s * 2048, &kr16_map, bar, 0, row + 16 * s, pol_kv);
                        }
                    }
                }
                __syncwarp();
                ++nk;
            };
            const auto load_v = [&](int l, int j) {  // this CTA's 64 value dims of tile j of stream l
                const int st = nv % kStages;
                if (!wait(&ctl.v_empty[st], nv / kStages)) return;
                const bool end = u.tail() && j == nt - 1;
                if (issuer) {
                    const uint32_t bar = end ? cluster_addr(&ctl.tail_landed[st], uint32_t(rank))
                                             : cluster_addr(&ctl.v_full[st], 0);
                    const int steps = min((limit - j * kTile + 15) >> 4, kTile / 16);
                    const uint32_t bytes = uint32_t(steps * (kStageV / (kTile / 16)));
                    if (end) {
                        mbar_arrive_expect_tx(&ctl.tail_landed[st], bytes);
                        if (rank == 0) mbar_arrive(&ctl.v_full[st]);  // the stage's phases go on
                    } else if (rank == 0) {
                        mbar_arrive_expect_tx(&ctl.v_full[st], 2 * bytes);
                    }
                    const uint32_t dst = sb + kOffV + st * kStageV;
                    const int row = u.kv0 + j * kTile, head = u.head + l;
                    if (steps == kTile / 16) {
                        tma2_load_3d(dst, &v_map, bar, 64 * rank, head, row, pol_kv);
                    } else {
                        for (int s = 0; s < steps; ++s)
                            tma2_load_3d(dst + s * 2048, &v16_map, bar, 64 * rank, head, row + 16 * s, pol_kv);
                    }
                }
                __syncwarp();
                v_tail = (v_tail & ~(1u << st)) | (uint32_t(end) << st);
                if (end) tail_phase ^= 1u << st;
                ++nv;
            };
            // In the order of use: q and K(0) of each stream, then V(j) and K(j + 1) of each.  Rolled, so that
            // every kind of load is in the code once.
#pragma unroll 1
            for (int j = -1; j < nt && nt > 0 && ok; ++j) {
#pragma unroll 1
                for (int l = 0; l < 2; ++l) {
                    if (j < 0) load_q(l);
                    if (j >= 0 && l < streams) load_v(l, j);
                    if (j < 0 && l < streams) load_k(l, 0);
                }
                if (j >= 0 && j + 1 < nt)
#pragma unroll 1
                    for (int l = 0; l < streams; ++l) load_k(l, j + 1);
            }
        }
        if (lane == 0) {
            if (!ok) {
                atomicOr(p.err, kErrWaitTimeout);
                ctl.abort = 1;
            }
            // No copy outlives the cluster (bounded waits; they have landed unless a role gave up).  The
            // leader's barriers count both CTAs' copies, and neither CTA leaves before the other.
            if (rank == 0) {
                for (int n = max(nk - kStages, 0); n < nk; ++n)
                    wait_landed_p(&ctl.k_full[n % kStages], uint32_t(n / kStages) & 1u);
                for (int n = max(nv - kStages, 0); n < nv; ++n)
                    if (!((v_tail >> (n % kStages)) & 1u))
                        wait_landed_p(&ctl.v_full[n % kStages], uint32_t(n / kStages) & 1u);
                for (int i = 0; i < 2; ++i)
                    if (nq[i] > 0) wait_landed_p(&ctl.q_full[i], uint32_t(nq[i] - 1) & 1u);
            }
            for (int st = 0; st < kStages; ++st)
                if ((v_tail >> st) & 1u) wait_landed_p(&ctl.tail_landed[st], ((tail_phase >> st) & 1u) ^ 1u);
            // After a timeout the two CTAs may have issued different copies, and what only the other counts
            // cannot be waited for here: a millisecond, a thousand times a copy's latency.
            if (*const_cast<volatile int*>(&ctl.abort)) {
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 1000 * 1000) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 10) {
        // ================= the last tiles' value rows =================
        int nv = 0;
        uint32_t tail_phase = 0;  // per value stage
        bool ok = true;
        int streams = 0, limit = 0;
        while (ok && next_unit([&](const Unit& from) { streams = from.streams(), limit = from.limit_max(); })) {
            const int nt = (limit + kTile - 1) / kTile;
            nv += nt * streams;
            if ((limit & 15) == 0) continue;  // Unit::tail
            const int valid = limit - (nt - 1) * kTile, fill = 16 - (valid & 15);
            for (int l = 0; l < streams && ok; ++l) {
                const int st = (nv - streams + l) % kStages;
                ok = __all_sync(0xffffffffu, mbar_await(&ctl.tail_landed[st], (tail_phase >> st) & 1u, &ctl.abort)) != 0;
                tail_phase ^= 1u << st;
                if (!ok) break;
                uint8_t* v = tiles + kOffV + st * kStageV;
                for (int i = lane; i < fill * 8; i += 32)
                    *reinterpret_cast<uint4*>(v + (valid + (i >> 3)) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                asm volatile("fence.proxy.async;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(cluster_addr(&ctl.tail_ready[st], 0));
            }
        }
        __syncwarp();
    } else if (warp == 8) {
        // ================= MMA (the leader's) =================
        // The whole warp runs the loop on uniform values; one elected lane issues.
        constexpr uint32_t kIdescQk = idesc_bf16_f32(2 * kTile, kTile);
        constexpr uint32_t kIdescPv = idesc_bf16_f32(2 * kTile, kPrefillDv) | (1u << 16);  // B (V) MN-major
        const uint32_t tmem = uint32_t(uniform(int(tmem_base)));
        const uint32_t sb = uint32_t(uniform(int(s_base)));
        const uint64_t q_desc = smem_desc_kmajor_sw128(sb + kOffQt);
        const uint64_t k_desc = smem_desc_kmajor_sw128(sb + kOffK);
        const uint64_t v_desc = desc_mn_sw128(sb + kOffV, kSlabB);
        const bool issuer = elect_one();
        bool ok = true;
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_await(bar, parity, &ctl.abort));
            return ok;
        };
        const auto commit = [&](uint64_t* bar) {
            if (issuer) umma2_commit(bar);
            __syncwarp();
        };
        // Rings of key and value stages, in the order of the loads: a stage and its phase.
        struct Ring {
            int st = 0;
            uint32_t phase = 0;
            __device__ __forceinline__ void next() {
                if (++st == kStages) st = 0, phase ^= 1u;
            }
        };
        Ring kr, vr;
        uint32_t p_phase = 0, o_phase = 3, q_phase = 0, tail_phase = 0;  // bit i: of tile (stage) i
        // What the loop needs of a unit; fetched a unit ahead.
        struct Plan {
            int lim[2], n_of[2], nt;
            bool shared, tail;
        };
        const auto fetch = [&](Plan& w) {
            int step = 0;
            if (!next_unit([&](const Unit& from) {
                    w.lim[0] = uniform(from.limit[0]), w.lim[1] = uniform(from.limit[1]);
                    step = uniform(from.step_head);
                }))
                return false;
            w.n_of[0] = (w.lim[0] + kTile - 1) / kTile, w.n_of[1] = (w.lim[1] + kTile - 1) / kTile;
            w.nt = max(w.n_of[0], w.n_of[1]);
            w.shared = step == 0;
            w.tail = (max(w.lim[0], w.lim[1]) & 15) != 0;
            return true;
        };
        const auto flip = [](uint32_t& phases, int i) {  // the tile's phase, and on to the next
            const uint32_t phase = (phases >> i) & 1u;
            phases ^= 1u << i;
            return phase;
        };
        // S(tile i) = Q_i . K^T, keys in stage st
        const auto qk = [&](int i, int st, bool last) {
            if (issuer) {
                const uint64_t a = refreshed(q_desc + uint32_t(i * kQkSlabs * (kSlabB >> 4)));
                const uint64_t bd = refreshed(k_desc + uint32_t(st * (kStageK >> 4)));
                const uint32_t d = refreshed(tmem + kColSP + 128u * i);
#pragma unroll
                for (int s = 0; s < kQkSlabs; ++s)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma2_bf16_ss(d, a + uint32_t(s * (kSlabB >> 4) + 2 * kk),
                                      bd + uint32_t(s * (kHalfB >> 4) + 2 * kk), kIdescQk, (s | kk) != 0 ? 1u : 0u);
                umma2_commit(&ctl.s_full[i]);
                if (last) umma2_commit(&ctl.q_empty[i]);
            }
            __syncwarp();
        };
        // O(tile i) (+)= P_i . V, values in stage st
        const auto pv = [&](int i, int st, int steps, bool first) {
            const uint64_t bd = refreshed(v_desc + uint32_t(st * (kStageV >> 4)));
            const uint32_t d = refreshed(tmem + kColOP + 128u * i), a = refreshed(tmem + kColSP + 128u * i);
            const auto step = [&](int kk) {
                umma2_bf16_ts(d, a + 8u * kk, bd + 128u * kk, kIdescPv, kk == 0 && first ? 0u : 1u);
            };
            if (steps == kTile / 16) {
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk) step(kk);
            } else {
#pragma unroll 1
                for (int kk = 0; kk < steps; ++kk) step(kk);
            }
        };
        Plan w = {}, next = {};
        bool more = fetch(next);
        if (rank == 0) {
            // One round per key tile: the products of both query tiles with it, each followed by that
            // tile's next scores, be they this unit's or (its keys are all used) the next one's.  The first
            // round is of no unit and has scores only.  Rolled over the tiles: this code runs once or twice
            // a unit where units are short, and out of the instruction cache it is twice as slow.
            int j = 0;
            while (ok && (w.nt > 0 || more)) {
                // Tiles that both query tiles see whole, with another one to come: the long part of a long
                // unit, as straight as it can be (an MMA issued late is tensor core time lost).
                const int whole = w.shared ? min(w.n_of[0], w.n_of[1]) - 1 : 0;
#pragma unroll 1
                for (; j < whole && ok; ++j) {
                    wait(&ctl.v_full[vr.st], vr.phase);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (j == 0) wait(&ctl.o_empty[i], flip(o_phase, i));
                        if (i == 0) wait(&ctl.k_full[kr.st], kr.phase);
                        wait(&ctl.p_full[i], flip(p_phase, i));
                        tc_fence_after_sync();
                        if (ok && issuer) {
                            pv(i, vr.st, kTile / 16, j == 0);
                            if (i == 1) umma2_commit(&ctl.v_empty[vr.st]);
                        }
                        if (ok) qk(i, kr.st, j + 2 == w.n_of[i]);
                    }
                    if (ok) commit(&ctl.k_empty[kr.st]);
                    kr.next();
                    vr.next();
                }
                const bool end = j >= w.nt - 1;
                if (end && w.nt > 0) more = fetch(next);
                // Whose scores come next: of tile j + 1 of this unit, or of the first of the next one.
                const int first_n = more ? next.n_of[0] : 0, second_n = more ? next.n_of[1] : 0;
                const bool s_shared = end ? next.shared : w.shared;
                bool have_k = false, have_v = false;
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    const int n = i ? w.n_of[1] : w.n_of[0], lim = i ? w.lim[1] : w.lim[0];
                    if (ok && j < n) {
                        if (!w.shared || !have_v) {
                            if (w.tail && end)
                                ok = __all_sync(0xffffffffu, mbar_wait_cluster(&ctl.tail_ready[vr.st],
                                                                               flip(tail_phase, vr.st), &ctl.abort)) != 0;
                            else
                                wait(&ctl.v_full[vr.st], vr.phase);
                        }
                        have_v = true;
                        if (j == 0) wait(&ctl.o_empty[i], flip(o_phase, i));
                        wait(&ctl.p_full[i], flip(p_phase, i));
                        tc_fence_after_sync();
                        if (ok && issuer) {
                            pv(i, vr.st, min((lim - j * kTile + 15) >> 4, kTile / 16), j == 0);
                            if (j + 1 == n) umma2_commit(&ctl.o_full[i]);
                        }
                        __syncwarp();
                    }
                    if (ok && w.nt > 0 && (w.shared ? i == 1 : j < n)) {
                        commit(&ctl.v_empty[vr.st]);
                        vr.next();
                    }
                    const int to_come = end ? (i ? second_n : first_n) : n - (j + 1);  // key tiles
                    if (ok && to_come > 0) {
                        if (!s_shared || !have_k) wait(&ctl.k_full[kr.st], kr.phase);
                        have_k = true;
                        if (end) wait(&ctl.q_full[i], flip(q_phase, i));
                        tc_fence_after_sync();
                        if (ok) qk(i, kr.st, to_come == 1);
                    }
                    if (ok && have_k && (s_shared ? i == 1 : to_come > 0)) {
                        commit(&ctl.k_empty[kr.st]);
                        kr.next();
                    }
                }
                ++j;
                if (end) {
                    j = 0;
                    if (more) {
                        w = next;
                        if (w.nt == 0) more = fetch(next);
                    } else {
                        w.nt = 0;
                    }
                }
            }
        } else {
            while (more) more = fetch(w);  // the leader issues for both
        }
        if (rank == 0) {
            if (!ok && issuer) {
                atomicOr(p.err, kErrWaitTimeout);
                ctl.abort = 1;
            }
            commit(&ctl.all_done);
        }
        wait_landed_p(&ctl.all_done, 0);  // every MMA has completed, and every arrival is here
        __syncwarp();
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ================= softmax: warps 0-3 tile 0, warps 4-7 tile 1 =================
        const int i = warp >> 2;
        const int r = rank * kTile + (warp & 3) * 32 + lane;  // row of the tile
        const uint32_t lane_addr = tmem_base + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t s_addr = lane_addr + kColSP + 128u * i;
        const uint32_t o_addr = lane_addr + kColOP + 128u * i;
        const float c2 = p.sm_scale_log2;
        const uint32_t p_bar = cluster_addr(&ctl.p_full[i], 0);
        const uint32_t o_bar = cluster_addr(&ctl.o_empty[i], 0);
        bool failed = false;
        uint32_t ns = 0, no = 0;  // score tiles and outputs so far
        Unit u;
        const auto copy = [&](const Unit& from) { u = from; };
        bool more = next_unit(copy);
        while (more) {
            const int head = u.head + i * u.step_head;
            const bool live_row = i * u.step_row + r < u.rows && head < p.heads;
            const int limit = i ? u.limit[1] : u.limit[0], ntiles = (limit + kTile - 1) / kTile;
            const int64_t token = int64_t(u.q_row) + i * u.step_row + r;
            const int64_t part_row = kSplit && u.part >= 0 ? (int64_t(u.part) * 2 + i) * (2 * kTile) + r : -1;
            int see = limit;
            if (live_row) {
                const int64_t len = int64_t(u.seq) - (int64_t(u.req_rows) - 1 - (u.row0 + i * u.step_row + r));
                see = min(entries_seen(len > 0 ? int(len) : 0, p.entry_tokens), u.live) - (kSplit ? u.skip : 0);
            }
            float m = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int j = 0; j < ntiles; ++j, ++ns) {
                const bool ok = mbar_await(&ctl.s_full[i], ns & 1u, &ctl.abort);
                if (!__all_sync(0xffffffffu, ok)) {
                    failed = true;
                    break;
                }
                tc_fence_after_sync();
                const int here = see - j * kTile;  // entries of this tile that the row sees
                const float2 cc = make_float2(c2, c2);
                // The row's maximum so far, and O and the sum with it (rare after the first tile).
                const auto raise = [&](float mx) {
                    const bool need = mx > m + kRaiseLog2;
                    if (__any_sync(0xffffffffu, need)) {
                        float alpha = 1.f;
                        if (need) {
                            alpha = exp2f(m - mx);
                            m = mx;
                            l2.x *= alpha;
                            l2.y *= alpha;
                        }
                        __syncwarp();
                        // S(j) full means that PV(j - 1), issued before it, has completed: O is at rest.
                        if (j > 0) {
#pragma unroll 1
                            for (int c = 0; c < 4; ++c) {
                                uint32_t o[32];
                                tmem_ld_32x32b_x32(o_addr + 32u * c, o);
                                tmem_ld_wait(o);
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                                tmem_st_x32(o_addr + 32u * c, o);
                            }
                        }
                    }
                };
                // The weights of 32 columns, as 16 pairs of bf16 from pk[at] on.
                const auto weights = [&](const uint32_t (&v)[32], auto& pk, int at, float2 mm) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float2 x =
                            fma_f32x2(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), cc, mm);
                        x.x = ex2_approx(x.x);
                        x.y = ex2_approx(x.y);
                        l2 = add_f32x2(l2, x);
                        const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
                        pk[at + k] = *reinterpret_cast<const uint32_t*>(&b);
                    }
                };
                if (__all_sync(0xffffffffu, here >= kTile)) {
                    uint32_t s[4][32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(s_addr + 32u * c, s[c]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld_wait(s[c]);
                    float mx[4];  // four independent chains
#pragma unroll
                    for (int c = 0; c < 4; ++c) mx[c] = __uint_as_float(s[c][0]);
#pragma unroll
                    for (int k = 1; k < 31; k += 2)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            mx[c] = max3(mx[c], __uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1]));
#pragma unroll
                    for (int c = 0; c < 4; ++c) mx[c] = fmaxf(mx[c], __uint_as_float(s[c][31]));
                    raise(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2);
                    const float nm = m == -INFINITY ? 0.f : -m;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[32];
                        weights(s[2 * h], pk, 0, make_float2(nm, nm));
                        weights(s[2 * h + 1], pk, 16, make_float2(nm, nm));
                        tmem_st_x32(s_addr + 32u * h, pk);
                    }
                } else {
                    // A tile that some row sees in part: 32 columns at a time, read twice (all of them at once
                    // do not fit beside their masks).  Columns that no row of the warp sees are not read, and
                    // their weights are 0 as far as the tile's limit (the products read none past it).
                    const int most = __reduce_max_sync(0xffffffffu, here);
                    const int chunks = min((limit - j * kTile + 31) >> 5, 4), seen = min(max(most + 31, 0) >> 5, chunks);
                    uint32_t v[32];
                    const auto chunk = [&](int c) {
                        tmem_ld_32x32b_x32(s_addr + 32u * c, v);
                        tmem_ld_wait(v);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * c + k >= here) v[k] = 0xFF800000u;  // -inf
                    };
                    float mx = -INFINITY, nm = 0.f;
                    // P's chunk c covers S's columns [16 c, 16 c + 16): behind what later chunks still read.
#pragma unroll 1
                    for (int it = 0; it < 2 * seen; ++it) {
                        const int c = it < seen ? it : it - seen;
                        chunk(c);
                        if (it < seen) {
#pragma unroll
                            for (int k = 0; k < 32; k += 2)
                                mx = max3(mx, __uint_as_float(v[k]), __uint_as_float(v[k + 1]));
                            if (it == seen - 1) {
                                raise(mx * c2);
                                nm = m == -INFINITY ? 0.f : -m;
                            }
                        } else {
                            uint32_t pk[16];
                            weights(v, pk, 0, make_float2(nm, nm));
                            tmem_st_x16(s_addr + 16u * c, pk);
                        }
                    }
#pragma unroll 1
                    for (int c = seen; c < chunks; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) pk[k] = 0;
                        tmem_st_x16(s_addr + 16u * c, pk);
                    }
                }
                tmem_st_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(p_bar);
            }
            if (failed) break;
            more = next_unit(copy);
            // ---- output
            __nv_bfloat16* o_row = reinterpret_cast<__nv_bfloat16*>(p.out) + (token * p.heads + head) * kPrefillDv;
            if (ntiles == 0) {  // rows that see nothing
                if (kSplit && live_row && part_row >= 0) {
                    p.lse_part[part_row] = -INFINITY;
                } else if (live_row) {
                    for (int c = 0; c < kPrefillDv / 8; ++c)
                        *reinterpret_cast<uint4*>(o_row + 8 * c) = make_uint4(0, 0, 0, 0);
                    p.lse[token * p.heads + head] = -INFINITY;
                }
                __syncwarp();
                continue;
            }
            const bool ok = mbar_await(&ctl.o_full[i], no & 1u, &ctl.abort);
            if (!__all_sync(0xffffffffu, ok)) {
                failed = true;
                break;
            }
            ++no;
            tc_fence_after_sync();
            const float l = l2.x + l2.y;
            const float inv = l == 0.f ? 0.f : 1.f / l;  // (0: nothing was seen; a NaN goes on to both outputs)
            const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2P;
            if (kSplit && live_row && part_row >= 0) {
                p.lse_part[part_row] = lse;
            } else if (live_row) {
                p.lse[token * p.heads + head] = lse;
            }
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld_32x32b_x32(o_addr + 32u * c, o);
                tmem_ld_wait(o);
                if (c == 3) {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(o_bar);  // O may be overwritten
                }
                if (kSplit && live_row && part_row >= 0) {
                    float* d = p.o_part + part_row * kPrefillDv + 32 * c;
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(__uint_as_float(o[8 * h + k]) * inv);
                        st_global_v8(d + 8 * h, w);
                    }
                } else if (live_row) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // a whole sector a lane
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[16 * h + 2 * k]) * inv,
                                                                           __uint_as_float(o[16 * h + 2 * k + 1]) * inv);
                            w[k] = *reinterpret_cast<const uint32_t*>(&v);
                        }
                        __nv_bfloat16* d = o_row + 32 * c + 16 * h;
                        if (p.out_aligned32) {
                            st_global_v8(d, w);
                        } else {
                            reinterpret_cast<uint4*>(d)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            reinterpret_cast<uint4*>(d)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                }
            }
            __syncwarp();
        }
        if (failed && lane == 0) {
            atomicOr(p.err, kErrWaitTimeout);
            ctl.abort = 1;
        }
    }

    __syncwarp();
    tc_fence_before_sync();
    cluster_sync_all();  // no CTA leaves while the other may read its memory or arrive on its barriers
    tc_fence_after_sync();
    if (warp == 8) tmem2_dealloc(tmem_base, kTmemColsP);
}

// out = sum_s exp(lse_s - lse) o_s over a unit's parts, lse = log sum_s exp(lse_s).  One warp per row; grid
// (units, 64 groups of 8 rows).
__global__ void __launch_bounds__(256) mla_prefill_merge_kernel(const PrefillParams p) {
    pdl_wait_prior_grid();
    pdl_allow_next_grid();
    const int2 split = *p.split;  // units, parts of each
    const int unit = blockIdx.x, parts = split.y;
    if (unit >= split.x || parts < 2) return;
    const SplitUnit u = p.split_units[unit];
    const int lane = threadIdx.x & 31;
    const int at = int(blockIdx.y) * 8 + (threadIdx.x >> 5), i = at / (2 * kTile), r = at % (2 * kTile);
    const int head = u.head + i * u.step_head;
    if (i * u.step_row + r >= u.rows || head >= p.heads) return;
    const auto part_row = [&](int s) { return (int64_t(unit) * parts + s) * 4 * kTile + at; };
    float mx = -INFINITY, sum = 0.f;
    for (int s = lane; s < parts; s += 32) mx = fmaxf(mx, p.lse_part[part_row(s)]);
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
        const float lse = p.lse_part[part_row(s)];
        if (lse == -INFINITY) continue;  // a part without entries has written no output
        const float w = expf(lse - mx);  // (a NaN, which the maximum passes by, stays)
        sum += w;
        const float4 v = *reinterpret_cast<const float4*>(p.o_part + part_row(s) * kPrefillDv + 4 * lane);
        acc.x = fmaf(w, v.x, acc.x), acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z), acc.w = fmaf(w, v.w, acc.w);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t row = (int64_t(u.q_row) + i * u.step_row + r) * p.heads + head;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(p.out + row * kPrefillDv + 4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    if (lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : mx + logf(sum);
}

}  // namespace

size_t prefill_split_bytes(int sms) {  // a slot of 512 rows for each part
    return prefill_part_offset(sms) + prefill_max_parts(sms) * 4 * kTile * (kPrefillDv + 1) * sizeof(float);
}
size_t prefill_part_offset(int sms) {  // the pair of counts and the units, before the parts
    return (16 + size_t(sms) / 2 * sizeof(SplitUnit) + 255) / 256 * 256;
}
size_t prefill_max_parts(int sms) { return size_t(sms) / 2 * kRounds; }

cudaError_t launch_mla_prefill(const PrefillMaps& m, const PrefillParams& p, cudaStream_t stream) {
    static SmemLimitOnce smem_limit, smem_limit_split, smem_limit_groups;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = smem_limit.apply(dev, mla_prefill_kernel<false, false>, kSmemP);
    if (e == cudaSuccess) e = smem_limit_split.apply(dev, mla_prefill_kernel<true, false>, kSmemP);
    if (e == cudaSuccess) e = smem_limit_groups.apply(dev, mla_prefill_kernel<false, true>, kSmemP);
    if (e != cudaSuccess) return e;
    // Persistent clusters: as many as the device holds (its SMs do not all pair up), or one per unit.
    static std::atomic<int> resident[kMaxDevices];
    int fit = resident[dev].load(std::memory_order_relaxed);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreadsP);
    cfg.dynamicSmemBytes = size_t(kSmemP);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (fit == 0) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        e = cudaOccupancyMaxActiveClusters(&fit, mla_prefill_kernel<false, false>, &cfg);
        if (e != cudaSuccess) return e;
        if (fit < 1) return cudaErrorInvalidConfiguration;
        resident[dev].store(fit, std::memory_order_relaxed);
    }
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const int64_t most = prefill_most_units(p.slots, p.heads);
    // Cut where a batch of this batch's average request would be; the kernel, which sees the lengths, decides.
    bool split = false;
    if (p.o_part) {
        const int rows = int((p.q_rows + p.batch - 1) / p.batch), entries = int(p.kv_rows / p.batch);
        const int64_t units = Cut(rows, entries, p.heads).units() * int64_t(p.batch);
        const int first = units > fit && rows > kPrefillBlock ? kPrefillBlock : rows;  // the last units are of
        const int tiles = (entries - (rows - first) / p.entry_tokens + kTile - 1) / kTile;  // a prompt's first rows
        split = parts_of(int(units % fit), tiles, fit) > 1;
    }
    cfg.gridDim = dim3(2u * unsigned(most < fit && !split ? most : fit));
    if (!split) {
        // Several prompts of more than a block on average (shorter ones lose what finding the groups takes).
        const bool groups = p.batch > 1 && p.batch <= kSortMost && p.q_rows > p.batch * kPrefillBlock;
        return cudaLaunchKernelEx(&cfg, groups ? mla_prefill_kernel<false, true> : mla_prefill_kernel<false, false>, m.q,
                                  m.kn, m.kr, m.v, m.kn16, m.kr16, m.v16, p);
    }
    e = cudaLaunchKernelEx(&cfg, mla_prefill_kernel<true, false>, m.q, m.kn, m.kr, m.v, m.kn16, m.kr16, m.v16, p);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(unsigned(fit), 4 * kTile / 8);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, mla_prefill_merge_kernel, p);
}

}  // namespace dsa
