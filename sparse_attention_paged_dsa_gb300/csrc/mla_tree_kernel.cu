// mla_tree_kernel.cu -- latent attention decode (absorbed form) for trees of more
// than two drafted tokens, sm_103a.
//
//     s[h, t] = sm_scale * q[b, j, h] . e_t                  (576-wide entries)
//     o[b, j, h] = sum_t softmax_t(s[h, :]) e_t[:512],  lse = log sum_t exp(s[h, t])
//
// over the ceil(seq_len / 4) live entries of the request's paged cache and the drafted
// entries i whose bit of the token's mask is set.  (Two tokens: mla_tree_pair_kernel.cu.  One,
// and small calls: mla_dense_kernel.cu.)
//
// What an SM takes in is 33 bytes a cycle, from L2 by plain or multicast loads alike
// (measured).  A token's 64 heads on an SM of their own need an entry's 1,152 bytes, 35
// cycles, for 17 of multiply-adds.  So four tokens share a cluster of four CTAs:
//   * rows: tokens 0 and 1 of the tile are the 128 rows of CTAs 0 and 2, tokens 2 and 3 of
//     CTAs 1 and 3.  CTAs 0, 1 and CTAs 2, 3 are pairs (cta_group::2, M = 256: all tokens);
//   * S = Q . K^T    pair p takes page p of a block of two: N = 64, 32 entries in each CTA;
//   * O += P . V     pair p takes value dims [256 p, 256 p + 256) of both pages: N = 256, 128
//                    dims in each CTA.  P of the other page comes from the CTA with the same
//                    rows in the other pair, by bulk copies between their shared memories.
// A block's entry then costs an SM 288 bytes as key, 256 as value and 128 of weights: 20 cycles.
// The multiply-adds of a block take 2,464 (36 products of N = 64 at 40, bound by their reads
// of shared memory, and 8 of N = 256 at 128); the loop runs at 2,490.
//
// Work.  A request's blocks are those of its pages followed by a page of its drafted
// entries.  Requests laid end to end, kTreeSegUnits units of fixed cost before each, are cut
// into ranges (how many: tree_cost); a unit is a range and a tile of four tokens.  Units are
// dealt out range by range, so that the tiles of one request run at the same time and all but
// the first read its pages from L2.  A request inside one range is written straight to the
// output, one that crosses ranges leaves fp32 partials that a second kernel joins.  Trees of
// different sizes: each tile has a line of its own, of the requests that reach into it, cut
// into ranges of about one size in all tiles, and the units go out by how far into its line
// each lies (tree_rank).  64 requests of 16384 tokens with 0 to 32 drafted ones 545 us (700 with
// the same ranges in all tiles, 735 for 32 of each), 5 of 100000 with up to 33 150 (366), 8 of
// up to 32768 with up to 64 52 (94); 13 x 27 of up to 8192 45 (44).
//
// No running maximum.  Both CTAs that hold a row must use one reference, and agreeing on a new
// one block by block would cost a round trip each.  They agree once, on the first block's
// maximum.  Weights may then pass 1 as far as fp32 and bf16 reach (their rounding is relative:
// nothing is lost).  A request one of whose sums passes 2^58, or one of whose outputs is not finite,
// is flagged, and the dense kernel, which keeps a running maximum, then does the flagged requests
// again (the others keep their results); it leaves at once (3 us) where there is none.
//
// Memory.  q: five slabs of 64 dims in shared memory (80 KB), four in tensor memory beside S
// (two blocks) and O; keys: a ring of four groups of three slabs; values: one block; weights of both
// pages: two blocks.  One block's weights less in flight: 2,144 us for 16 x 32 tokens at
// 128K context, now 1,275 (1,833 TFLOP/s, 0.96 of the measured bf16 rate; in a long run, which
// power limits, 1,428: 0.97 of the sustained rate).
//
// Roles of a CTA (384 threads):
//   * warps 0-7: softmax, one row and 32 entries a thread; q's slabs into tensor memory; outputs.
//   * warp 8 of each pair's leader: S.  Warp 11: O.  (One warp for both was late with every
//     product: 4,650 cycles a block, of them 2,000 in waits for barriers that were complete.)
//   * warp 11 of the other CTAs: tells the leader of weights that have come there.  Both zero
//     value rows that nobody sees (behind the last live entry, drafts outside every mask).
//   * warps 9 and 10: TMA of q and keys, and of values.
// The roles' loops run side by side and share an instruction cache: with a few hundred
// instructions more, the loop ran a quarter slower on most of the device.
//
// What bounds it: the tensor cores in long requests; in short ones a request's start and end
// (about 8,000 cycles: q, the first block's maxima, sums, outputs).  64 x 8 tokens at 8192: 134 us
// (0.57); 64 x 64 at 512: 251 us, of them 86 the bytes of q and the output.
// Every wait is bounded (about 1 s) but the cluster barriers, which every thread reaches, and the
// softmax warps' own, which they meet in step whatever fails; a timeout sets an error bit, the
// roles drain, and TMEM is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "cta_pair.cuh"
#include "indexer_kernels.h"
#include "mla_common.cuh"
#include "mla_tree_common.cuh"
#include "sm103_ptx.cuh"

namespace dsa {
namespace {

constexpr int kRowsQ = 128;                     // rows of a CTA: two tokens' heads
constexpr int kHalfPg = kPg / 2;                // entries of a CTA's half page
constexpr int kSlabsQ = kMlaDim / 64;           // 9
constexpr int kSlabQ = kRowsQ * 128;            // 16 KiB
constexpr int kSlabK = kHalfPg * 128;           // 4 KiB
constexpr int kSlabsTm = 4;                     // of q in tensor memory, the last ones
constexpr int kSlabsSm = kSlabsQ - kSlabsTm;    // in shared memory
constexpr int kSlabsK = 3;                      // key slabs that are loaded together
constexpr int kGroupK = kSlabsK * kSlabK;
constexpr int kGroupsK = kSlabsQ / kSlabsK;     // of a block
constexpr int kRingK = 4;                       // groups in shared memory
constexpr int kSlabV = kPg * 128;               // values of a page: two slabs of 64 entries x 64 dims
constexpr int kGroupQ = 2 * kSlabV;
constexpr int kSlabsLand = kRingK * kGroupK / kSlabQ;  // of q's slabs for tensor memory, by way of the idle ring
static_assert(kSlabsLand == kSlabsTm - 1, "the last one goes through registers");
constexpr int kOffQq = 0;
constexpr int kOffKq = kOffQq + kSlabsSm * kSlabQ;
constexpr int kOffVq = kOffKq + kRingK * kGroupK;
constexpr int kOffRq = kOffVq + 2 * kGroupQ;    // weights of the other page, 128 rows x 64 entries
constexpr int kOffPq = kOffRq + 2 * kSlabQ;     // and of the own page; two blocks' of both
constexpr int kOffCtlQ = kOffPq + 2 * kSlabQ;
constexpr uint32_t kColSQ = 0;     // S: 2 x 64 columns
constexpr uint32_t kColQQ = 128;   // q: 32 columns a slab
constexpr uint32_t kColOQ = 256;   // O: 256 columns
constexpr float kSumMost = 288230376151711744.0f;  // 2^58: |O| is at most that times the largest |value|, finite for
                                                   // values below 2^69; what larger ones make infinite is flagged too
constexpr float kSumLeast = 8.4703294725430034e-22f;  // 2^-70, where the reference is not the row's own

struct __align__(16) TreeCtl {
    uint64_t k_full[kRingK], k_empty[kRingK];  // full: the pair's leader's, of both CTAs' copies
    uint64_t v_full[2], v_empty[2];            // per page of a block
    uint64_t vz_full[2], vz_ready[2];
    uint64_t s_full[2], s_empty[2];
    uint64_t q_full, q_empty, ql_full, ql_read, qt_full, o_empty, all_done;
    uint64_t p_own[2], p_other[2], r_full[2], pv_done[2];  // of every other block
    uint64_t m_full, l_full;                   // the other pair's row maxima, and sums, are here
    uint32_t tmem_base;
    int abort;
    TreePlan plan;
    float part[2][kRowsQ];                     // per half of the entries: maxima of the first block, then sums
    float peer[2][kRowsQ];                     // the other pair's maxima, and sums
};
constexpr int kSmemQ = kOffCtlQ + int(sizeof(TreeCtl));
static_assert(kSmemQ <= 232448, "fits one CTA per SM");

// Arrive once on the barrier at this offset in the CTAs of `mask` when every MMA this thread issued has completed.
__device__ __forceinline__ void commit_to(uint64_t* bar, uint16_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(mask)
        : "memory");
}

// Copy to another CTA's shared memory, counted on a barrier there.
__device__ __forceinline__ void bulk_to_cta(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     dst),
                 "r"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
// Store to another CTA's shared memory, counted (four bytes) on a barrier there: no release to wait for.
__device__ __forceinline__ void st_async_f32(uint32_t addr, float v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(addr), "f"(v),
                 "r"(bar)
                 : "memory");
}

// The two warps of a quadrant: both halves of its 32 rows.
__device__ __forceinline__ void quad_sync(int quad) {
    __syncwarp();
    asm volatile("bar.sync %0, 64;" ::"r"(2 + quad) : "memory");
}

__global__ void __launch_bounds__(kTreeThreads, 1) __cluster_dims__(4, 1, 1)
    mla_tree_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap d_map,
                    const __grid_constant__ CUtensorMap o_map, const __grid_constant__ MlaTreeParams p) {
    extern __shared__ uint8_t smem_raw[];  // at the same offset in all CTAs; on a 1,024-byte boundary, checked below
    uint8_t* tiles = smem_raw;
    TreeCtl& ctl = *reinterpret_cast<TreeCtl*>(tiles + kOffCtlQ);
    const uint32_t s_base = smem_u32(tiles);
    const int warp = uniform(int(threadIdx.x) >> 5);
    const int lane = threadIdx.x & 31;
    const int rank = int(cluster_rank());
    const int pair = rank >> 1, side = rank & 1;   // side 0: the pair's leader
    const uint32_t leader = uint32_t(rank & 2);
    const uint16_t both = uint16_t(3u << (rank & 2));
    const int cluster = int(blockIdx.x) >> 2, clusters = int(gridDim.x) >> 2;

    if (s_base & 1023u) {  // (the same in every CTA; shared memory has always started on such a boundary)
        pdl_wait_prior_grid();
        if (int(threadIdx.x) < (p.batch + 31) / 32) atomicOr(p.flags + threadIdx.x, 0xffffffffu);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRingK; ++i) {
            mbar_init(&ctl.k_full[i], 1);
            mbar_init(&ctl.k_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.v_full[i], 1);
            mbar_init(&ctl.v_empty[i], 1);
            mbar_init(&ctl.vz_full[i], 1);
            mbar_init(&ctl.vz_ready[i], 1);  // the leader's: of the other CTA
            mbar_init(&ctl.s_full[i], 1);
            mbar_init(&ctl.p_own[i], 2 * kSoftWarps);
            mbar_init(&ctl.p_other[i], 1);   // the other CTA of the pair has its part
            mbar_init(&ctl.r_full[i], 1);
            mbar_init(&ctl.pv_done[i], 2);   // of both pairs
            mbar_init(&ctl.s_empty[i], 2 * kSoftWarps);
        }
        mbar_init(&ctl.q_full, 1);
        mbar_init(&ctl.q_empty, 1);
        mbar_init(&ctl.ql_full, 1);          // slabs for tensor memory landed in this CTA's key ring; read from it
        mbar_init(&ctl.ql_read, kSoftWarps);
        mbar_init(&ctl.qt_full, 2 * kSoftWarps);
        mbar_init(&ctl.o_empty, 2 * kSoftWarps);
        mbar_init(&ctl.all_done, 4);         // of both pairs' two issuing warps
        mbar_init(&ctl.m_full, 1);
        mbar_init(&ctl.l_full, 1);
        ctl.abort = 0;
        clear_plan(p, ctl.plan);
        fence_mbar_init();
        tma_prefetch_map(&q_map);
        tma_prefetch_map(&k_map);
        tma_prefetch_map(&v_map);
        tma_prefetch_map(&d_map);
        tma_prefetch_map(&o_map);
    }
    if (warp == 8) tmem2_alloc(&ctl.tmem_base, 512);
    __syncwarp();
    pdl_wait_prior_grid();
    pdl_allow_next_grid();

    const int units = find_units<kTileTokens>(p, ctl.plan, cluster, clusters);
    tc_fence_before_sync();
    cluster_sync_all();  // the barriers and the plan are there, in all CTAs
    tc_fence_after_sync();
    if (threadIdx.x == 0 && rank == 0) write_cuts(p, ctl.plan, cluster, clusters, units);
    __syncwarp();
    const uint32_t tmem_base = ctl.tmem_base;
    TreeWalk<kTileTokens> w(cluster, clusters, units);

    if (warp == 9) {
        // ================= TMA: q and keys =================
        // Whole warps run the loops on uniform values; one elected lane issues.
        const bool issuer = elect_one();
        const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
        const uint32_t sb = uint32_t(uniform(int(s_base)));
        bool ok = true;
        int n = 0, seg = 0, slot = 0;  // key groups, requests so far; the ring's place
        uint32_t phase = 0;
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_await(bar, parity, &ctl.abort));
            return ok;
        };
        while (ok && w.next(p, ctl.plan)) {
            int id_l = tree_page_of_lane(p, w, 2 * w.blo, lane);
            if (id_l == -1 && 2 * w.blo + lane < 2 * w.bhi) atomicOr(p.err, kErrBadPage);
            const int row = (w.req() * p.tokens + 4 * w.tile + 2 * side) * kMlaHeads;
            if (issuer) {  // into L2, while the products of the request before use its q
#pragma unroll 1
                for (int s = 0; s < kSlabsQ; ++s)
                    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                                     reinterpret_cast<uint64_t>(&q_map)),
                                 "r"(0), "r"(row), "r"(s)
                                 : "memory");
            }
            __syncwarp();
            if (!wait(&ctl.q_empty, uint32_t(seg & 1) ^ 1u)) break;
            if (issuer) {
                const uint32_t bar = cluster_addr(&ctl.q_full, leader);
                if (side == 0) mbar_arrive_expect_tx(&ctl.q_full, uint32_t(2 * kSlabsSm * kSlabQ));
                // Rows behind the request's tokens are others' or zeros, and their outputs are not written.  The slabs
                // for tensor memory first, by way of the ring, whose keys are used.
                mbar_arrive_expect_tx(&ctl.ql_full, uint32_t(kSlabsLand * kSlabQ));
#pragma unroll 1
                for (int s = 0; s < kSlabsLand; ++s)
                    tma_load_3d(tiles + kOffKq + s * kSlabQ, &q_map, &ctl.ql_full, 0, row, kSlabsSm + s, pol_q);
#pragma unroll 1
                for (int s = 0; s < kSlabsSm; ++s)
                    tma2_load_3d(sb + kOffQq + s * kSlabQ, &q_map, bar, 0, row, s, pol_q);
            }
            __syncwarp();
            ++seg;
            if (!wait(&ctl.ql_read, uint32_t(seg - 1) & 1u)) break;
            const int blocks = uniform(w.bhi - w.blo);
#pragma unroll 1
            for (int i = 0; i < blocks && ok; ++i) {
                if (i > 0 && (i & 15) == 0) {
                    id_l = tree_page_of_lane(p, w, 2 * (w.blo + i), lane);
                    if (id_l == -1 && 2 * (w.blo + i) + lane < 2 * w.bhi) atomicOr(p.err, kErrBadPage);
                }
                // the pair's page; -1: page 0 stands in, its entries are not used
                const int id = __shfl_sync(0xffffffffu, id_l, 2 * (i & 15) + pair);
                const int row = max(id, 0) * kPg + kHalfPg * side;
#pragma unroll 1
                for (int j = 0; j < kGroupsK; ++j, ++n) {
                    if (!wait(&ctl.k_empty[slot], phase ^ 1u)) break;
                    if (issuer) {
                        const uint32_t bar = cluster_addr(&ctl.k_full[slot], leader);
                        const uint32_t dst = sb + kOffKq + slot * kGroupK;
                        if (side == 0) mbar_arrive_expect_tx(&ctl.k_full[slot], uint32_t(2 * kGroupK));
                        if (id == -2) {
#pragma unroll
                            for (int k = 0; k < kSlabsK; ++k)
                                load_drafts(dst + k * kSlabK, &d_map, bar, kHalfPg * side, kSlabsK * j + k, w.req(),
                                            pol_kv);
                        } else {
                            tma2_load_3d(dst, &k_map, bar, 0, row, kSlabsK * j, pol_kv);
                        }
                    }
                    __syncwarp();
                    if (++slot == kRingK) slot = 0, phase ^= 1u;
                }
            }
        }
        if (lane == 0) {
            if (!ok) {
                atomicOr(p.err, kErrWaitTimeout);
                ctl.abort = 1;
            }
            // No copy outlives the cluster (bounded waits; they have landed unless a role gave up).
            if (side == 0) {
                for (int i = max(n - kRingK, 0); i < n; ++i)
                    wait_landed_t(&ctl.k_full[i % kRingK], uint32_t(i / kRingK) & 1u);
                if (seg > 0) wait_landed_t(&ctl.q_full, uint32_t(seg - 1) & 1u);
            }
            if (seg > 0) wait_landed_t(&ctl.ql_full, uint32_t(seg - 1) & 1u);
        }
        __syncwarp();
    } else if (warp == 10) {
        // ================= TMA: values =================
        const bool issuer = elect_one();
        const uint64_t pol_kv = l2_policy_evict_last();
        const uint32_t sb = uint32_t(uniform(int(s_base)));
        bool ok = true;
        int n = 0;
        uint32_t zero_fills[2] = {0, 0}, issued = 0;
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_await(bar, parity, &ctl.abort));
            return ok;
        };
        while (ok && w.next(p, ctl.plan)) {
            int id_l = 0;
            const int blocks = uniform(w.bhi - w.blo);
#pragma unroll 1
            for (int i = 0; i < blocks; ++i, ++n) {
                if ((i & 15) == 0) id_l = tree_page_of_lane(p, w, 2 * (w.blo + i), lane);
#pragma unroll
                for (int s = 0; s < 2; ++s) {  // the pair's own page first, as its product goes
                    const int pg = s ^ pair;
                    const int id = __shfl_sync(0xffffffffu, id_l, 2 * (i & 15) + pg);
                    const bool zeroes = id != -1 && w.zeroes(2 * (w.blo + i) + pg);
                    if (!wait(&ctl.v_empty[pg], uint32_t(n & 1) ^ 1u)) break;
                    if (issuer) {
                        uint32_t bar = cluster_addr(&ctl.v_full[pg], leader);
                        if (zeroes) {
                            bar = cluster_addr(&ctl.vz_full[pg], uint32_t(rank));
                            mbar_arrive_expect_tx(&ctl.vz_full[pg], uint32_t(kGroupQ));
                            if (side == 0) mbar_arrive(&ctl.v_full[pg]);  // the page's phases go on
                        } else if (side == 0) {
                            mbar_arrive_expect_tx(&ctl.v_full[pg], uint32_t(2 * kGroupQ));
                        }
                        const uint32_t dst = sb + kOffVq + pg * kGroupQ;
                        const int slab = 4 * pair + 2 * side;  // dims 256 pair + 128 side
                        if (id == -2) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)  // 32 entries of a slab at a time
                                load_drafts(dst + k * kSlabK, &d_map, bar, kHalfPg * (k & 1), slab + (k >> 1), w.req(),
                                            pol_kv);
                        } else {
                            tma2_load_3d(dst, &v_map, bar, 0, max(id, 0) * kPg, slab, pol_kv);
                        }
                    }
                    __syncwarp();
                    issued |= 1u << pg;
                    if (ok && zeroes) ++zero_fills[pg];
                }
                if (!ok) break;
                issued = 0;
            }
        }
        if (lane == 0) {
            if (!ok) {
                atomicOr(p.err, kErrWaitTimeout);
                ctl.abort = 1;
            }
            if (side == 0)
                for (int g = 0; g < 2; ++g) {
                    const int fills = n + int((issued >> g) & 1u);
                    if (fills > 0) wait_landed_t(&ctl.v_full[g], uint32_t(fills - 1) & 1u);
                }
            for (int pg = 0; pg < 2; ++pg)
                if (zero_fills[pg] > 0) wait_landed_t(&ctl.vz_full[pg], (zero_fills[pg] - 1) & 1u);
            // After a timeout the CTAs may have issued different copies, and what only another counts
            // cannot be waited for here: a millisecond, a thousand times a copy's latency.
            if (*const_cast<volatile int*>(&ctl.abort)) {
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 1000 * 1000) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 8 || warp == 11) {
        // ================= MMA (the pairs' leaders') =================
        if (side == 0) {
            constexpr uint32_t kIdescQk = idesc_bf16_f32(256, 64);
            constexpr uint32_t kIdescPv = idesc_bf16_f32(256, 256) | (1u << 16);  // B (V) MN-major
            const uint32_t tmem = uint32_t(uniform(int(tmem_base)));
            const uint32_t sb = uint32_t(uniform(int(s_base)));
            const bool issuer = elect_one();
            bool ok = true;
            const auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok = ok && __all_sync(0xffffffffu, mbar_await(bar, parity, &ctl.abort));
                return ok;
            };
            int n = 0, seg = 0;  // blocks, requests so far
            if (warp == 8) {
                // ---- scores
                const uint64_t q_desc = smem_desc_kmajor_sw128(sb + kOffQq);
                const uint64_t k_desc = smem_desc_kmajor_sw128(sb + kOffKq);
                int slot = 0;
                uint32_t phase = 0;
                while (ok && w.next(p, ctl.plan)) {
                    if (!wait(&ctl.q_full, uint32_t(seg & 1)) || !wait(&ctl.qt_full, uint32_t(seg & 1))) break;
                    const int blocks = uniform(w.bhi - w.blo);
#pragma unroll 1
                    for (int i = 0; i < blocks && ok; ++i, ++n) {
                        const int buf = n & 1;
                        const uint32_t d = tmem + kColSQ + 64u * buf;
                        wait(&ctl.s_empty[buf], (uint32_t(n >> 1) & 1u) ^ 1u);
#pragma unroll
                        for (int j = 0; j < kGroupsK; ++j) {
                            wait(&ctl.k_full[slot], phase);
                            tc_fence_after_sync();
                            if (ok && issuer) {
                                const uint64_t bd = refreshed(k_desc + uint32_t(slot * (kGroupK >> 4)));
                                const uint64_t a = refreshed(q_desc + uint32_t(kSlabsK * j * (kSlabQ >> 4)));
                                const uint32_t at = refreshed(tmem + kColQQ), dd = refreshed(d);
#pragma unroll
                                for (int k = 0; k < kSlabsK; ++k)
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk) {
                                        const uint64_t b = bd + uint32_t(k * (kSlabK >> 4) + 2 * kk);
                                        if (kSlabsK * j + k < kSlabsSm)
                                            umma2_bf16_ss(dd, a + uint32_t(k * (kSlabQ >> 4) + 2 * kk), b, kIdescQk,
                                                          (j | k | kk) != 0 ? 1u : 0u);
                                        else
                                            umma2_bf16_ts(dd, at + uint32_t(32 * (kSlabsK * j + k - kSlabsSm) + 8 * kk), b,
                                                          kIdescQk, 1u);
                                    }
                                commit_to(&ctl.k_empty[slot], both);
                                if (j == kGroupsK - 1) {
                                    commit_to(&ctl.s_full[buf], both);
                                    if (i + 1 == blocks) commit_to(&ctl.q_empty, both);
                                }
                            }
                            __syncwarp();
                            if (++slot == kRingK) slot = 0, phase ^= 1u;
                        }
                    }
                    ++seg;
                }
            } else {
                // ---- outputs
                const uint64_t r_desc = smem_desc_kmajor_sw128(sb + kOffRq);
                const uint64_t p_desc = smem_desc_kmajor_sw128(sb + kOffPq);
                const uint64_t v_desc = desc_mn_sw128(sb + kOffVq, kSlabV);
                uint32_t zero_phase = 0;
                while (ok && w.next(p, ctl.plan)) {
                    const int blocks = uniform(w.bhi - w.blo);
                    const uint64_t drafts = drafts_seen(p, w, lane);
                    uint32_t fresh = 1, bad = 0;
#pragma unroll 1
                    for (int i = 0; i < blocks && ok; ++i, ++n) {
                        if ((i & 15) == 0)
                            bad = __ballot_sync(0xffffffffu, tree_page_of_lane(p, w, 2 * (w.blo + i), lane) == -1);
                        const int buf = n & 1;
                        const uint32_t phase = uint32_t(n >> 1) & 1u;
                        if (issuer) mbar_arrive_expect_tx(&ctl.r_full[buf], uint32_t(kSlabQ));
                        __syncwarp();
                        if (i == 0) wait(&ctl.o_empty, uint32_t(seg & 1) ^ 1u);
#pragma unroll 1
                        for (int s = 0; s < 2; ++s) {  // the own page, then the other
                            const int pg = s ^ pair;
                            const int page = 2 * (w.blo + i) + pg;
                            const bool good = !((bad >> (2 * (i & 15) + pg)) & 1u);
                            const int steps = good ? uniform((w.valid(page) + 15) >> 4) : 0;
                            if (good && w.zeroes(page)) {
                                wait(&ctl.vz_full[pg], (zero_phase >> pg) & 1u);
                                zero_unseen<2>(page == w.np ? drafts : low_bits(w.valid(page)), w.valid(page),
                                               tiles + kOffVq + pg * kGroupQ);
                                ok = ok && __all_sync(0xffffffffu, mbar_wait_cluster(&ctl.vz_ready[pg],
                                                                                     (zero_phase >> pg) & 1u, &ctl.abort));
                                zero_phase ^= 1u << pg;
                            }
                            wait(&ctl.v_full[pg], uint32_t(n & 1));
                            if (s == 0) {
                                wait(&ctl.p_own[buf], phase);
                            } else {
                                wait(&ctl.r_full[buf], phase);
                                wait(&ctl.p_other[buf], phase);
                            }
                            tc_fence_after_sync();
                            if (ok && issuer) {
                                const uint64_t bd = refreshed(v_desc + uint32_t(pg * (kGroupQ >> 4)));
                                const uint32_t d = refreshed(tmem + kColOQ);
                                const uint64_t a =
                                    refreshed((s == 0 ? p_desc : r_desc) + uint32_t(buf * (kSlabQ >> 4)));
                                const auto step = [&](int kk) {
                                    umma2_bf16_ss(d, a + 2u * kk, bd + uint32_t(kk * (2048 >> 4)), kIdescPv,
                                                  (kk == 0 && fresh) ? 0u : 1u);
                                };
                                if (steps == 4) {
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk) step(kk);
                                } else {
#pragma unroll 1
                                    for (int kk = 0; kk < steps; ++kk) step(kk);
                                }
                                commit_to(&ctl.v_empty[pg], both);
                                if (s == 1) commit_to(&ctl.pv_done[buf], uint16_t(15));
                            }
                            __syncwarp();
                            if (steps > 0) fresh = 0;
                        }
                    }
                    ++seg;
                }
            }
            if (issuer) {
                if (!ok) {
                    atomicOr(p.err, kErrWaitTimeout);
                    ctl.abort = 1;
                }
                commit_to(&ctl.all_done, uint16_t(15));  // every MMA this thread issued has completed when this arrives
            }
            __syncwarp();
        } else if (warp == 11) {
            // ---- the other CTA's: zeroes its value rows that nobody sees, and tells the leader of that and of
            // the weights that have come here
            const bool issuer = elect_one();
            bool ok = true;
            const auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok = ok && __all_sync(0xffffffffu, mbar_await(bar, parity, &ctl.abort));
                return ok;
            };
            int n = 0;
            uint32_t zero_phase = 0, bad = 0;
            while (ok && w.next(p, ctl.plan)) {
                const int blocks = uniform(w.bhi - w.blo);
                const uint64_t drafts = drafts_seen(p, w, lane);
#pragma unroll 1
                for (int i = 0; i < blocks && ok; ++i, ++n) {
                    if ((i & 15) == 0)
                        bad = __ballot_sync(0xffffffffu, tree_page_of_lane(p, w, 2 * (w.blo + i), lane) == -1);
                    if (issuer) mbar_arrive_expect_tx(&ctl.r_full[n & 1], uint32_t(kSlabQ));
                    __syncwarp();
#pragma unroll 1
                    for (int s = 0; s < 2; ++s) {
                        const int pg = s ^ pair, page = 2 * (w.blo + i) + pg;
                        if (((bad >> (2 * (i & 15) + pg)) & 1u) || !w.zeroes(page)) continue;
                        if (!wait(&ctl.vz_full[pg], (zero_phase >> pg) & 1u)) break;
                        zero_phase ^= 1u << pg;
                        zero_unseen<2>(page == w.np ? drafts : low_bits(w.valid(page)), w.valid(page),
                                       tiles + kOffVq + pg * kGroupQ);
                        if (issuer) mbar_arrive_cluster(cluster_addr(&ctl.vz_ready[pg], leader));
                        __syncwarp();
                    }
                    wait(&ctl.r_full[n & 1], uint32_t(n >> 1) & 1u);
                    if (ok && issuer) mbar_arrive_remote(cluster_addr(&ctl.p_other[n & 1], leader));
                    __syncwarp();
                }
            }
        }
    } else if (warp < kSoftWarps) {
        // ================= softmax and output =================
        const int quad = warp & 3, half = warp >> 2;     // entries [32 half, 32 half + 32) of the pair's page
        const int row = quad * 32 + lane;
        const uint32_t lane_addr = tmem_base + (uint32_t(quad * 32) << 16);
        const uint32_t peer = uint32_t(rank ^ 2);        // the same rows, the other page and value dims
        const uint32_t s_bar = cluster_addr(ctl.s_empty, leader), p_bar = cluster_addr(ctl.p_own, leader),
                       o_bar = cluster_addr(&ctl.o_empty, leader), qt_bar = cluster_addr(&ctl.qt_full, leader);
        const uint32_t r_rows = cluster_addr(tiles + kOffRq, peer) + quad * 4096;
        const uint32_t r_bar = cluster_addr(ctl.r_full, peer);
        uint8_t* const pbuf = tiles + kOffPq + row * 128;
        const uint32_t peer_max = cluster_addr(ctl.peer[0], peer) + 4 * row;
        const uint32_t peer_sum = cluster_addr(ctl.peer[1], peer) + 4 * row;
        const uint32_t m_bar = cluster_addr(&ctl.m_full, peer), l_bar = cluster_addr(&ctl.l_full, peer);
        const float c2 = p.sm_scale_log2;
        const bool q_aligned = (reinterpret_cast<uintptr_t>(p.q) & 31) == 0;
        bool failed = false;
        int n = 0, seg = 0;
        // One request after another, the start of each under the last products of the one before.
        bool more = w.next(p, ctl.plan), had = false;
        int q_seg = 0;
        // of the request before: its sums, where its outputs go, and what is known of them
        float m = 0.f, l = 0.f;
        bool own = true, fresh = true, live_token = false, whole = false;
        uint32_t any = 0;
        int64_t at = 0, first_row = 0;
        int tokens_here = 0;
        while (true) {
            float sum = 0.f;
            if (had) {
                ctl.part[half][row] = l;
                if (soft_or(failed)) break;
                sum = ctl.part[0][row] + ctl.part[1][row];
                if (half == 0) st_async_f32(peer_sum, sum, l_bar);
            }
            // q's slabs for tensor memory, half of each a thread: the last one straight from global memory, the others
            // by way of the key ring.
            if (more) {
                const int token = min(kTileTokens * w.tile + 2 * side + (row >> 6), p.tokens - 1);
                const __nv_bfloat16_raw* q = p.q +
                                             ((int64_t(w.req()) * p.tokens + token) * kMlaHeads + (row & 63)) * kMlaDim +
                                             64 * (kSlabsQ - 1) + 32 * half;
                uint32_t last[16];
                if (q_aligned) {  // a sector a lane
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t v[8];
                        ld_global_v8(v, q + 16 * k);
#pragma unroll
                        for (int e = 0; e < 8; ++e) last[8 * k + e] = v[e];
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 v = __ldg(reinterpret_cast<const uint4*>(q) + k);
                        last[4 * k] = v.x, last[4 * k + 1] = v.y, last[4 * k + 2] = v.z, last[4 * k + 3] = v.w;
                    }
                }
                const bool ok = mbar_await(&ctl.ql_full, uint32_t(q_seg & 1), &ctl.abort);
                ++q_seg;
                if (!__all_sync(0xffffffffu, ok)) {
                    failed = true;  // (all warps meet at the next barrier)
                    if (lane == 0) ctl.abort = 1;
                    __syncwarp();
                }
                tc_fence_after_sync();  // (behind q_empty: the products have read what was there)
#pragma unroll 1
                for (int c = 0; c < kSlabsLand; ++c) {
                    uint32_t r[16];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 v = *reinterpret_cast<const uint4*>(tiles + kOffKq + c * kSlabQ + row * 128 +
                                                                        (((4 * half + k) ^ (row & 7)) << 4));
                        r[4 * k] = v.x, r[4 * k + 1] = v.y, r[4 * k + 2] = v.z, r[4 * k + 3] = v.w;
                    }
                    tmem_st_x16(lane_addr + kColQQ + 32u * c + 16u * half, r);
                }
                tmem_st_x16(lane_addr + kColQQ + 32u * kSlabsLand + 16u * half, last);
                // the ring's next contents come by TMA: behind these reads
                fence_proxy_async_smem();
                tmem_st_wait();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&ctl.ql_read);
                    mbar_arrive_remote(qt_bar);
                }
            }
            if (had) {
                // ---- the output (or partial)
                bool done = mbar_await(&ctl.pv_done[(n - 1) & 1], uint32_t((n - 1) >> 1) & 1u, &ctl.abort);
                done = done && mbar_wait_cluster(&ctl.l_full, uint32_t(seg & 1), &ctl.abort);
                if (soft_or(!done || failed)) {  // (and the sums are read)
                    failed = true;
                    break;
                }
                tc_fence_after_sync();
                ++seg;
                {   // in one order, so that both pairs have the same sum
                    const float other = *const_cast<volatile float*>(&ctl.peer[1][row]);
                    sum = pair == 0 ? sum + other : other + sum;
                }
                bool flagged = live_token && (!(sum <= kSumMost) || (!own && any != 0 && !(sum >= kSumLeast)));
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const int head = row & 63;
                if (live_token && pair == 0 && half == 0)
                    (whole ? p.lse : p.lse_part)[at * kMlaHeads + head] =
                        sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2T;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32];
                    __syncwarp();
                    if (fresh) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0u;
                    } else {
                        tmem_ld_32x32b_x32(lane_addr + kColOQ + 128u * half + 32u * c, o);
                        tmem_ld_wait(o);
                    }
                    if (c == 3) {
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote(o_bar);  // O may be overwritten
                    }
                    if (!live_token) continue;
                    float most = 0.f;  // (0 x inf and 0 x NaN are NaN, and any other product 0)
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float v = __uint_as_float(o[i]) * inv;
                        most = fmaf(v, 0.f, most);
                        o[i] = __float_as_uint(v);
                    }
                    if (most != 0.f) flagged = true;
                    if (whole) {  // 64 heads x 64 dims a tile, 128-byte-swizzled, where the weights were
                        uint8_t* const tile =
                            tiles + kOffRq + ((row >> 6) * 4 + 2 * half + (c >> 1)) * kSlabV + head * 128;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t v[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(o[8 * k + 2 * e]),
                                                                                __uint_as_float(o[8 * k + 2 * e + 1]));
                                v[e] = *reinterpret_cast<const uint32_t*>(&b2);
                            }
                            *reinterpret_cast<uint4*>(tile + (((4 * (c & 1) + k) ^ (head & 7)) << 4)) =
                                make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    } else {  // eight dims of a head after those of the head before: a warp's stores are contiguous
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t v[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = o[8 * k + e];
                            st_global_v8(p.o_part + tiled_part(at, head, 256 * pair + 128 * half + 32 * c + 8 * k), v);
                        }
                    }
                }
                if (__any_sync(0xffffffffu, flagged) && lane == 0) {  // (rows of the request's: live ones)
                    const int b = int(first_row / p.tokens);
                    atomicOr(p.flags + (b >> 5), 1u << (b & 31));
                }
                if (whole) {
                    fence_proxy_async_smem();
                    soft_or(false);
                    if (threadIdx.x == 0) {
#pragma unroll 1
                        for (int i = 0; i < 4 * tokens_here; ++i)
                            tma_store_2d(&o_map, s_base + kOffRq + i * kSlabV, 256 * pair + 64 * (i & 3),
                                         int(first_row + (i >> 2)) * kMlaHeads);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                    __syncwarp();
                }
            }
            if (!more) break;

            // ---- the request's weights
            const int token = kTileTokens * w.tile + 2 * side + (row >> 6);
            live_token = token < w.drafted;
            const int64_t q_row = int64_t(w.req()) * p.tokens + min(token, p.tokens - 1);
            const uint64_t drafts = __ldg(p.mask + q_row) & low_bits(w.drafted);
            bool ok = true;
            if (threadIdx.x == 0) {  // what the other pair will send: a maximum and a sum of each row
                mbar_arrive_expect_tx(&ctl.m_full, uint32_t(kRowsQ * sizeof(float)));
                mbar_arrive_expect_tx(&ctl.l_full, uint32_t(kRowsQ * sizeof(float)));
            }
            m = l = 0.f;
            own = true;    // the reference is a score of the row's
            any = 0;       // entries seen
            fresh = true;  // no product of this request yet: O holds nothing of it
            uint32_t bad = 0;
#pragma unroll 1
            for (int blk = w.blo; blk < w.bhi; ++blk, ++n) {
                if (((blk - w.blo) & 15) == 0)
                    bad = __ballot_sync(0xffffffffu, tree_page_of_lane(p, w, 2 * blk, lane) == -1);
                const uint32_t bad_here = bad >> (2 * ((blk - w.blo) & 15));
                const int page = 2 * blk + pair;
                uint64_t seen = page == w.np ? drafts : low_bits(w.valid(page));
                if ((bad_here >> pair) & 1u) seen = 0;
                const uint32_t bits = uint32_t(seen >> (32 * half));
                any |= bits;
                const int buf = n & 1;
                ok = __all_sync(0xffffffffu, mbar_await(&ctl.s_full[buf], uint32_t(n >> 1) & 1u, &ctl.abort)) != 0;
                float x[32];
                {
                    uint32_t r[32];
                    tc_fence_after_sync();
                    tmem_ld_32x32b_x32(lane_addr + kColSQ + 64u * buf + 32u * half, r);
                    tmem_ld_wait(r);
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(s_bar + 8u * buf);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 y = mul_f32x2(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])),
                                                   make_float2(c2, c2));
                        x[i] = y.x, x[i + 1] = y.y;
                    }
                }
                if (__any_sync(0xffffffffu, bits != 0xffffffffu)) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!((bits >> i) & 1u)) x[i] = -INFINITY;
                }
                if (blk == w.blo) {  // the reference: the block's maximum, of both pages
                    float mx = x[0];
#pragma unroll
                    for (int i = 1; i < 32; ++i) mx = fmaxf(mx, x[i]);
                    ctl.part[half][row] = mx;
                    // The outputs of the request before have left the buffers that weights come to again, this CTA's
                    // own and, once its maxima are sent, the other pair's.
                    if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    __syncwarp();
                    soft_or(false);
                    mx = fmaxf(ctl.part[0][row], ctl.part[1][row]);
                    if (half == 0) st_async_f32(peer_max, mx, m_bar);
                    ok = ok && mbar_wait_cluster(&ctl.m_full, uint32_t(seg & 1), &ctl.abort);
                    if (soft_or(!ok)) {
                        failed = true;
                        break;
                    }
                    m = fmaxf(mx, *const_cast<volatile float*>(&ctl.peer[0][row]));
                    own = m != -INFINITY;
                    if (!own) m = 0.f;
                }
                uint32_t packed[16];
                float2 sums = make_float2(0.f, 0.f);
                const float2 m2 = make_float2(-m, -m);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 y = add_f32x2(make_float2(x[2 * i], x[2 * i + 1]), m2);
                    const float p0 = ex2_approx(y.x), p1 = ex2_approx(y.y);
                    sums = add_f32x2(sums, make_float2(p0, p1));
                    const __nv_bfloat162 v = __floats2bfloat162_rn(p0, p1);
                    packed[i] = *reinterpret_cast<const uint32_t*>(&v);
                }
                l += sums.x + sums.y;
                // The products of the block before the last, of both pairs, have read their weights.
                ok = ok && mbar_await(&ctl.pv_done[buf], (uint32_t(n >> 1) & 1u) ^ 1u, &ctl.abort);
                if (!__all_sync(0xffffffffu, ok)) {
                    failed = true;  // (the others' waits end the same way; the barriers are met by all)
                    if (lane == 0) ctl.abort = 1;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<uint4*>(pbuf + buf * kSlabQ + (((4 * half + k) ^ (row & 7)) << 4)) =
                        make_uint4(packed[4 * k], packed[4 * k + 1], packed[4 * k + 2], packed[4 * k + 3]);
                fence_proxy_async_smem();
                // Both halves of these 32 rows are there, for the async proxy too: the products and the copy read them in
                // this SM, behind each writer's fence.  (No thread of another CTA does: the arrivals need no
                // cluster-scope release, which took 1,900 cycles here and bound the loop: 1662 us for 16 x 32
                // tokens at 128K context.)
                quad_sync(quad);
                if (lane == 0) {
                    if (half == 0)
                        bulk_to_cta(r_rows + buf * kSlabQ, s_base + kOffPq + buf * kSlabQ + quad * 4096, 4096u,
                                    r_bar + 8u * buf);
                    mbar_arrive_remote(p_bar + 8u * buf);
                }
                if (w.valid(2 * blk) > 0 && !(bad_here & 1u)) fresh = false;
                if (w.valid(2 * blk + 1) > 0 && !(bad_here & 2u)) fresh = false;
            }
            whole = w.blo == 0 && w.bhi == w.nb;
            at = whole ? q_row : (int64_t(w.range) * kTileTokens + token % kTileTokens) * 2 + (w.blo == 0 ? 1 : 0);
            tokens_here = min(w.drafted - kTileTokens * w.tile - 2 * side, 2);  // of this CTA's two
            first_row = int64_t(w.req()) * p.tokens + kTileTokens * w.tile + 2 * side;
            had = true;
            more = w.next(p, ctl.plan);
        }
        if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (failed && lane == 0) {
            atomicOr(p.err, kErrWaitTimeout);
            ctl.abort = 1;
        }
        __syncwarp();
    }

    __syncwarp();
    tc_fence_before_sync();
    cluster_sync_all();  // no CTA leaves while another may read its memory or arrive on its barriers
    tc_fence_after_sync();
    if (warp == 8) {
        wait_landed_t(&ctl.all_done, 0);  // the leaders' last arrivals here
        __syncwarp();
        tmem2_dealloc(tmem_base, 512);
    }
}

}  // namespace

cudaError_t mla_tree_quads(int* quads) {
    static SmemLimitOnce smem_limit;
    static std::atomic<int> resident[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    e = smem_limit.apply(dev, mla_tree_kernel, kSmemQ);
    if (e != cudaSuccess) return e;
    *quads = resident[dev].load(std::memory_order_relaxed);
    if (*quads > 0) return cudaSuccess;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 4;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(4);
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = size_t(kSmemQ);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(quads, mla_tree_kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (*quads < 1) return cudaErrorInvalidConfiguration;
    resident[dev].store(*quads, std::memory_order_relaxed);
    return cudaSuccess;
}

cudaError_t launch_mla_tree(const MlaTreeMaps& m, MlaTreeParams p, int quads, cudaStream_t stream) {
    p.clusters = quads;
    const int units = p.ranges * p.tiles;
    if (p.ranges < 1 || p.ranges > kTreeMaxRanges || units > kTreeMaxRounds * quads || units > kTreeMaxUnits)
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(4u * unsigned(units < quads ? units : quads));
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = size_t(kSmemQ);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mla_tree_kernel, m.q, m.k, m.v, m.d, m.o, p);
}

}  // namespace dsa
