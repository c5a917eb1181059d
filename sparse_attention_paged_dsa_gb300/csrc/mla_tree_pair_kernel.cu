// mla_tree_pair_kernel.cu -- latent attention decode (absorbed form) for two drafted
// tokens, sm_103a.
//
//     s[h, t] = sm_scale * q[b, j, h] . e_t                  (576-wide entries)
//     o[b, j, h] = sum_t softmax_t(s[h, :]) e_t[:512],  lse = log sum_t exp(s[h, t])
//
// over the ceil(seq_len / 4) live entries of the request's paged cache and the drafted
// entries i whose bit of the token's mask is set.
//
// Two tokens leave half the rows of a cluster of four (mla_tree_kernel.cu) empty, and a CTA
// for each (mla_dense_kernel.cu) reads every entry twice.  Here a cluster of two CTAs has one
// token in each, and cta_group::2 products (M = 128: 64 rows in each CTA) whose second operand
// is split between the CTAs' shared memory:
//     S = Q . K^T    N = 128 entries: a block of two pages, one page's 576 dims in each CTA
//     O += P . V     N = 256 dims, twice: of both pages 2 x 128 dims in each CTA, read
//                    in place as an MN-major operand
// An entry is key in one of the CTAs and half a value row in both: 1,088 bytes of loads a
// CTA for two tokens, 1,152 for one otherwise.  D of an M = 128 pair lies in each CTA as 64
// rows x two halves of the columns: lanes 0-63 the first half, 64-127 the second.
//
// Work: ranges of blocks as in mla_tree_kernel.cu, with one tile.
//
// Roles of a CTA (384 threads):
//   * warps 0-7: softmax.  Warp w reads TMEM quadrant w % 4 (rows 32 (w & 1) + lane of
//     page (w >> 1) & 1) and half of the page's entries: one row and 32 entries a
//     thread.  All of a row is in this CTA, so there is a running maximum; it is raised only
//     when a block passes it by more than 2^20, and O is then rescaled in tensor memory.  At
//     the end the output, from tensor memory to global memory.
//   * warp 8 (of the leader): S.  Warp 11: O; in the other CTA, zeroes value rows that nobody
//     sees (behind the last live entry, drafts outside every mask), as it does in the leader's.
//   * warps 9 and 10: TMA of q and keys, and of values.
// Row sums add the unrounded fp32 weights; the weights are rounded to bf16 only as the
// second product's operand.
//
// What bounds it: what an SM takes in, 33 bytes a cycle: 4,220 cycles a block, and the loop runs
// at about that; of HBM's time it needs 1.4 (64 requests of 65536 tokens 244 us, 4,950 GB/s; a
// CTA for each token took 354).  16 x 131072 131 us (183), 64 x 8192 65 (75), 1 x 1048576 80
// (99).  The loops of the roles run side by side and share an instruction cache: loaders and
// issuers are rolled (311 us with them unrolled, and up to 15 % more or less with each change
// anywhere else in the kernel).
// Not kept: the next pages fetched into L2 one to three blocks ahead (a twentieth more; the copy
// engine issues that traffic too); half of a CTA's keys kept as its values, the other half
// loaded over with the rest of them (832 bytes an entry and CTA, but a block's buffers go
// through load, scores, load, product before the next but one can come: 256 us).
//
// Every wait is bounded (about 1 s) but the cluster barriers, which every thread reaches, and
// the softmax warps' own, which they meet in step whatever fails; a timeout sets an error bit,
// the roles drain, and TMEM is freed.
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

constexpr int kSlabT = kPg * 128;             // 64 rows x 64 bf16 dims, 8 KiB
constexpr int kSlabsT = kMlaDim / 64;         // 9
constexpr int kKeyGroups = 5;                 // slab pairs of the value dims, and the last slab
constexpr int kValGroups = 4;                 // (page, 256 dims): 2 page + half
constexpr int kGroupV = 2 * kSlabT;           // this CTA's 128 of a group's 256 dims
constexpr int kOffQT = 0;
constexpr int kOffKT = kOffQT + kSlabsT * kSlabT;
constexpr int kOffVT = kOffKT + kSlabsT * kSlabT;
constexpr int kOffPT = kOffVT + kValGroups * kGroupV;  // P: 64 rows x 64 entries of each page
constexpr int kOffCtlT = kOffPT + 2 * kSlabT;
constexpr uint32_t kTmemColsT = 512;
constexpr uint32_t kColST = 0;    // S: 2 x 64 columns
constexpr uint32_t kColOT = 128;  // O: 2 x 128 columns
constexpr float kRaise = 20.0f;   // log2; a weight's rounding is relative, so nothing is lost below it

struct __align__(16) PairCtl {
    uint64_t k_full[kKeyGroups], k_empty[kKeyGroups];  // full: the leader's, of both CTAs' copies
    uint64_t v_full[kValGroups], v_empty[kValGroups];
    uint64_t vz_full[2], vz_ready[2];  // of pages with rows to zero: landed in this CTA; zeroed in both
    uint64_t s_full[2], s_empty[2];
    uint64_t q_full, q_empty, p_full, pv_done, o_empty, all_done;
    uint32_t tmem_base;
    int abort;
    TreePlan plan;
    float part[4][kPg];          // per row and quarter of the block: maxima, at the end sums
};
constexpr int kSmemT = 1024 + kOffCtlT + int(sizeof(PairCtl));
static_assert(kSmemT <= 232448, "fits one CTA per SM");

__global__ void __launch_bounds__(kTreeThreads, 1) __cluster_dims__(2, 1, 1)
    mla_tree_pair_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kv_map,
                         const __grid_constant__ CUtensorMap kr_map, const __grid_constant__ CUtensorMap d_map,
                         const __grid_constant__ MlaTreeParams p) {
    extern __shared__ uint8_t smem_raw[];
    // Dynamic shared memory starts at the same offset in both CTAs, so the operands and barriers do too.
    uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    PairCtl& ctl = *reinterpret_cast<PairCtl*>(tiles + kOffCtlT);
    const uint32_t s_base = smem_u32(tiles);
    const int warp = uniform(int(threadIdx.x) >> 5);
    const int lane = threadIdx.x & 31;
    const int rank = int(cluster_rank());  // 0: the leader
    const int cluster = int(blockIdx.x) >> 1, clusters = int(gridDim.x) >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kKeyGroups; ++i) {
            mbar_init(&ctl.k_full[i], 1);
            mbar_init(&ctl.k_empty[i], 1);
        }
        for (int i = 0; i < kValGroups; ++i) {
            mbar_init(&ctl.v_full[i], 1);
            mbar_init(&ctl.v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.vz_full[i], 1);
            mbar_init(&ctl.vz_ready[i], 1);  // the leader's: of the other CTA
            mbar_init(&ctl.s_full[i], 1);
            mbar_init(&ctl.s_empty[i], 2 * kSoftWarps);
        }
        mbar_init(&ctl.q_full, 1);
        mbar_init(&ctl.q_empty, 1);
        mbar_init(&ctl.p_full, 2 * kSoftWarps);
        mbar_init(&ctl.pv_done, 1);
        mbar_init(&ctl.o_empty, 2 * kSoftWarps);
        mbar_init(&ctl.all_done, 2);
        ctl.abort = 0;
        clear_plan(p, ctl.plan);
        fence_mbar_init();
        tma_prefetch_map(&q_map);
        tma_prefetch_map(&kv_map);
        tma_prefetch_map(&kr_map);
        tma_prefetch_map(&d_map);
    }
    if (warp == 8) tmem2_alloc(&ctl.tmem_base, kTmemColsT);
    __syncwarp();
    pdl_wait_prior_grid();
    pdl_allow_next_grid();

    const int units = find_units<kPairTokens>(p, ctl.plan, cluster, clusters);
    tc_fence_before_sync();
    cluster_sync_all();  // the barriers and the plan are there, in both CTAs
    tc_fence_after_sync();
    if (threadIdx.x == 0 && rank == 0) write_cuts(p, ctl.plan, cluster, clusters, units);
    __syncwarp();
    const uint32_t tmem_base = ctl.tmem_base;
    TreeWalk<kPairTokens> w(cluster, clusters, units);

    if (warp == 9) {
        // ================= TMA: q and keys =================
        // Whole warps run the loops on uniform values; one elected lane issues.
        const bool issuer = elect_one();
        const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
        const uint32_t sb = uint32_t(uniform(int(s_base)));
        bool ok = true;
        int n = 0, seg = 0;
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_await(bar, parity, &ctl.abort));
            return ok;
        };
        uint32_t issued = 0;  // fills of each key group beyond the n whole blocks (bit j), for the drain
        while (ok && w.next(p, ctl.plan)) {
            int id_l = tree_page_of_lane(p, w, 2 * w.blo, lane);
            if (id_l == -1 && 2 * w.blo + lane < 2 * w.bhi) atomicOr(p.err, kErrBadPage);
            if (!wait(&ctl.q_empty, uint32_t(seg & 1) ^ 1u)) break;
            if (issuer) {
                const uint32_t bar = cluster_addr(&ctl.q_full, 0);
                if (rank == 0) mbar_arrive_expect_tx(&ctl.q_full, uint32_t(2 * kSlabsT * kSlabT));
                const int row = (w.req() * kPairTokens + rank) * kMlaHeads;
#pragma unroll
                for (int s = 0; s < kSlabsT; s += 3)
                    tma2_load_3d(sb + kOffQT + s * kSlabT, &q_map, bar, 0, row, s, pol_q);
            }
            __syncwarp();
            ++seg;
            const int blocks = uniform(w.bhi - w.blo);
#pragma unroll 1
            for (int i = 0; i < blocks; ++i, ++n) {
                if (i > 0 && (i & 15) == 0) {
                    id_l = tree_page_of_lane(p, w, 2 * (w.blo + i), lane);
                    if (id_l == -1 && 2 * (w.blo + i) + lane < 2 * w.bhi) atomicOr(p.err, kErrBadPage);
                }
                // this CTA's page; -1: page 0 stands in, its entries are not used
                const int id = __shfl_sync(0xffffffffu, id_l, 2 * (i & 15) + rank);
                const int row = max(id, 0) * kPg;
#pragma unroll 1
                for (int j = 0; j < kKeyGroups; ++j) {
                    if (!wait(&ctl.k_empty[j], uint32_t(n & 1) ^ 1u)) break;
                    if (issuer) {
                        const uint32_t bar = cluster_addr(&ctl.k_full[j], 0), dst = sb + kOffKT + 2 * j * kSlabT;
                        if (rank == 0) mbar_arrive_expect_tx(&ctl.k_full[j], uint32_t((j < 4 ? 4 : 2) * kSlabT));
                        if (id == -2) {
                            load_drafts(dst, &d_map, bar, 0, 2 * j, w.req(), pol_kv);
                            if (j < 4) load_drafts(dst + kSlabT, &d_map, bar, 0, 2 * j + 1, w.req(), pol_kv);
                        } else if (j < 4) {
                            tma2_load_3d(dst, &kv_map, bar, 0, row, 2 * j, pol_kv);
                        } else {
                            tma2_load_2d(dst, &kr_map, bar, kMlaDv, row, pol_kv);
                        }
                    }
                    __syncwarp();
                    issued |= 1u << j;
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
            // No copy outlives the cluster (bounded waits; they have landed unless a role gave up).
            if (rank == 0) {
                for (int j = 0; j < kKeyGroups; ++j) {
                    const int fills = n + int((issued >> j) & 1u);
                    if (fills > 0) wait_landed_t(&ctl.k_full[j], uint32_t(fills - 1) & 1u);
                }
                if (seg > 0) wait_landed_t(&ctl.q_full, uint32_t(seg - 1) & 1u);
            }
        }
        __syncwarp();
    } else if (warp == 10) {
        // ================= TMA: values =================
        const bool issuer = elect_one();
        const uint64_t pol_kv = l2_policy_evict_last();
        const uint32_t sb = uint32_t(uniform(int(s_base)));
        bool ok = true;
        int n = 0;
        uint32_t zero_fills = 0;  // 16 bits for each page of a block (a request has one at most)
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_await(bar, parity, &ctl.abort));
            return ok;
        };
        uint32_t issued = 0;
        while (ok && w.next(p, ctl.plan)) {
            int id_l = 0;
            const int blocks = uniform(w.bhi - w.blo);
#pragma unroll 1
            for (int i = 0; i < blocks; ++i, ++n) {
                if ((i & 15) == 0) id_l = tree_page_of_lane(p, w, 2 * (w.blo + i), lane);
#pragma unroll 1
                for (int pg = 0; pg < 2; ++pg) {
                    const int id = __shfl_sync(0xffffffffu, id_l, 2 * (i & 15) + pg);
                    const int row = max(id, 0) * kPg;
                    const bool zeroes = id != -1 && w.zeroes(2 * (w.blo + i) + pg);
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        const int g = 2 * pg + h;
                        if (!wait(&ctl.v_empty[g], uint32_t(n & 1) ^ 1u)) break;
                        if (issuer) {
                            uint32_t bar = cluster_addr(&ctl.v_full[g], 0);
                            if (zeroes) {
                                bar = cluster_addr(&ctl.vz_full[pg], uint32_t(rank));
                                if (h == 0) mbar_arrive_expect_tx(&ctl.vz_full[pg], uint32_t(2 * kGroupV));
                                if (rank == 0) mbar_arrive(&ctl.v_full[g]);  // the group's phases go on
                            } else if (rank == 0) {
                                mbar_arrive_expect_tx(&ctl.v_full[g], uint32_t(2 * kGroupV));
                            }
                            const uint32_t dst = sb + kOffVT + g * kGroupV;
                            const int slab = 4 * h + 2 * rank;  // dims 256 h + 128 rank
                            if (id == -2) {
                                load_drafts(dst, &d_map, bar, 0, slab, w.req(), pol_kv);
                                load_drafts(dst + kSlabT, &d_map, bar, 0, slab + 1, w.req(), pol_kv);
                            } else {
                                tma2_load_3d(dst, &kv_map, bar, 0, row, slab, pol_kv);
                            }
                        }
                        __syncwarp();
                        issued |= 1u << g;
                    }
                    if (ok && zeroes) zero_fills += 1u << (16 * pg);
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
            if (rank == 0)
                for (int g = 0; g < kValGroups; ++g) {
                    const int fills = n + int((issued >> g) & 1u);
                    if (fills > 0) wait_landed_t(&ctl.v_full[g], uint32_t(fills - 1) & 1u);
                }
            for (int pg = 0; pg < 2; ++pg)
                if (const uint32_t fills = (zero_fills >> (16 * pg)) & 0xFFFFu)
                    wait_landed_t(&ctl.vz_full[pg], (fills - 1) & 1u);
            // After a timeout the two CTAs may have issued different copies, and what only the other counts
            // cannot be waited for here: a millisecond, a thousand times a copy's latency.
            if (*const_cast<volatile int*>(&ctl.abort)) {
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 1000 * 1000) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 8 || warp == 11) {
        // ================= MMA (the leader's) =================
        if (rank == 0) {
            constexpr uint32_t kIdescQk = idesc_bf16_f32(128, 128);
            constexpr uint32_t kIdescPv = idesc_bf16_f32(128, 256) | (1u << 16);  // B (V) MN-major
            const uint32_t tmem = uint32_t(uniform(int(tmem_base)));
            const uint32_t sb = uint32_t(uniform(int(s_base)));
            const uint64_t q_desc = smem_desc_kmajor_sw128(sb + kOffQT);
            const uint64_t k_desc = smem_desc_kmajor_sw128(sb + kOffKT);
            const uint64_t p_desc = smem_desc_kmajor_sw128(sb + kOffPT);
            const uint64_t v_desc = desc_mn_sw128(sb + kOffVT, kSlabT);
            const bool issuer = elect_one();
            bool ok = true;
            const auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok = ok && __all_sync(0xffffffffu, mbar_await(bar, parity, &ctl.abort));
                return ok;
            };
            int nq = 0, nv = 0, seg = 0;  // S products, O products, requests so far
            uint32_t zero_phase = 0;
            // S of the next block
            const auto qk = [&](bool last) {
                const int buf = nq & 1;
                const uint32_t phase = uint32_t(nq & 1);
                wait(&ctl.s_empty[buf], (uint32_t(nq >> 1) & 1u) ^ 1u);
                const uint32_t d = tmem + kColST + 64u * buf;
#pragma unroll 1
                for (int j = 0; j < kKeyGroups; ++j) {
                    if (!wait(&ctl.k_full[j], phase)) return;
                    tc_fence_after_sync();
                    if (issuer) {
                        const uint64_t a = refreshed(q_desc + uint32_t(2 * j * (kSlabT >> 4)));
                        const uint64_t bd = refreshed(k_desc + uint32_t(2 * j * (kSlabT >> 4)));
#pragma unroll
                        for (int hs = 0; hs < (j < 4 ? 2 : 1); ++hs)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma2_bf16_ss(refreshed(d), a + uint32_t(hs * (kSlabT >> 4) + 2 * kk),
                                              bd + uint32_t(hs * (kSlabT >> 4) + 2 * kk), kIdescQk,
                                              (j | hs | kk) != 0 ? 1u : 0u);
                        umma2_commit(&ctl.k_empty[j]);
                        if (j == kKeyGroups - 1) {
                            umma2_commit(&ctl.s_full[buf]);
                            if (last) umma2_commit(&ctl.q_empty);
                        }
                    }
                    __syncwarp();
                }
                ++nq;
            };
            if (warp == 8) {
                while (ok && w.next(p, ctl.plan)) {
                    if (!wait(&ctl.q_full, uint32_t(seg & 1))) break;
                    const int blocks = uniform(w.bhi - w.blo);
#pragma unroll 1
                    for (int i = 0; i < blocks && ok; ++i) qk(i + 1 == blocks);
                    ++seg;
                }
            } else {
                while (ok && w.next(p, ctl.plan)) {
                    const int blocks = uniform(w.bhi - w.blo);
                    const uint64_t drafts = drafts_seen(p, w, lane);
                    uint32_t fresh = 1, bad = 0;
#pragma unroll 1
                    for (int i = 0; i < blocks && ok; ++i, ++nv) {
                        if ((i & 15) == 0)
                            bad = __ballot_sync(0xffffffffu, tree_page_of_lane(p, w, 2 * (w.blo + i), lane) == -1);
                        if (i == 0) wait(&ctl.o_empty, uint32_t(seg & 1) ^ 1u);
                        // (the weights are read in their writers' SMs, behind the writers' fences: no cluster scope)
                        wait(&ctl.p_full, uint32_t(nv & 1));
#pragma unroll 1
                        for (int pg = 0; pg < 2; ++pg) {
                            const int page = 2 * (w.blo + i) + pg;
                            const bool good = !((bad >> (2 * (i & 15) + pg)) & 1u);
                            const int steps = good ? uniform((w.valid(page) + 15) >> 4) : 0;
                            if (good && w.zeroes(page)) {
                                wait(&ctl.vz_full[pg], (zero_phase >> pg) & 1u);
                                zero_unseen<4>(page == w.np ? drafts : low_bits(w.valid(page)), w.valid(page),
                                               tiles + kOffVT + 2 * (page & 1) * kGroupV);
                                ok = ok && __all_sync(0xffffffffu, mbar_wait_cluster(&ctl.vz_ready[pg],
                                                                                     (zero_phase >> pg) & 1u, &ctl.abort));
                                zero_phase ^= 1u << pg;
                            }
#pragma unroll 1
                            for (int h = 0; h < 2; ++h) {
                                const int g = 2 * pg + h;
                                if (!wait(&ctl.v_full[g], uint32_t(nv & 1))) break;
                                tc_fence_after_sync();
                                if (issuer) {
                                    const uint64_t a = refreshed(p_desc + uint32_t(pg * (kSlabT >> 4)));
                                    const uint64_t bd = refreshed(v_desc + uint32_t(g * (kGroupV >> 4)));
                                    const uint32_t d = refreshed(tmem + kColOT + 128u * h);
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
                                    umma2_commit(&ctl.v_empty[g]);
                                    if (g == kValGroups - 1) umma2_commit(&ctl.pv_done);
                                }
                                __syncwarp();
                            }
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
                umma2_commit(&ctl.all_done);  // every MMA this thread issued has completed when this arrives
            }
            __syncwarp();
            if (warp == 8) wait_landed_t(&ctl.all_done, 0);
            __syncwarp();
        } else if (warp == 11) {
            bool ok = true;
            uint32_t phase = 0;
            while (ok && w.next(p, ctl.plan)) {
                const uint64_t drafts = drafts_seen(p, w, lane);
                for (int page = max(w.np - 1, 0); page <= w.np && ok; ++page) {
                    if (page < 2 * w.blo || page >= 2 * w.bhi || !w.zeroes(page)) continue;
                    if (page < w.np && tree_page_of_lane(p, w, page, 0) == -1) continue;
                    const int pg = page & 1;
                    ok = __all_sync(0xffffffffu, mbar_await(&ctl.vz_full[pg], (phase >> pg) & 1u, &ctl.abort)) != 0;
                    phase ^= 1u << pg;
                    if (!ok) break;
                    zero_unseen<4>(page == w.np ? drafts : low_bits(w.valid(page)), w.valid(page),
                                   tiles + kOffVT + 2 * (page & 1) * kGroupV);
                    if (lane == 0) mbar_arrive_cluster(cluster_addr(&ctl.vz_ready[pg], 0));
                    __syncwarp();
                }
            }
            __syncwarp();
        }
    } else if (warp < 8) {
        // ================= softmax and output =================
        const int quad = warp & 3, half = warp >> 2;     // entries [32 half, 32 half + 32) of the page
        const int pg = quad >> 1;
        const int row = (quad & 1) * 32 + lane;          // the head
        const int part = 2 * pg + half;
        const uint32_t lane_addr = tmem_base + (uint32_t(quad * 32) << 16);
        const uint32_t s_bar = cluster_addr(ctl.s_empty, 0), p_bar = cluster_addr(&ctl.p_full, 0),
                       o_bar = cluster_addr(&ctl.o_empty, 0);
        const float c2 = p.sm_scale_log2;
        uint8_t* const pbuf = tiles + kOffPT + pg * kSlabT + row * 128;
        bool failed = false;
        int n = 0;
        while (!failed && w.next(p, ctl.plan)) {
            const bool live_token = rank < w.drafted;
            const int64_t q_row = int64_t(w.req()) * kPairTokens + rank;
            const uint64_t drafts = __ldg(p.mask + q_row) & low_bits(w.drafted);
            float m = -INFINITY, l = 0.f;
            bool fresh = true;  // no product of this request yet: O holds nothing of it
            uint32_t bad = 0;
#pragma unroll 1
            for (int blk = w.blo; blk < w.bhi; ++blk, ++n) {
                if (((blk - w.blo) & 15) == 0)
                    bad = __ballot_sync(0xffffffffu, tree_page_of_lane(p, w, 2 * blk, lane) == -1);
                const uint32_t bad_here = bad >> (2 * ((blk - w.blo) & 15));
                const int page = 2 * blk + pg;
                uint64_t seen = page == w.np ? drafts : low_bits(w.valid(page));
                if ((bad_here >> pg) & 1u) seen = 0;
                const uint32_t bits = uint32_t(seen >> (32 * half));
                const int buf = n & 1;
                bool ok = mbar_await(&ctl.s_full[buf], uint32_t(n >> 1) & 1u, &ctl.abort);
                ok = __all_sync(0xffffffffu, ok);
                float x[32];
                {
                    uint32_t r[32];
                    tc_fence_after_sync();
                    tmem_ld_32x32b_x32(lane_addr + kColST + 64u * buf + 32u * half, r);
                    tmem_ld_wait(r);
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(s_bar + 8u * buf);
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]) * c2;
                }
                if (bits != 0xffffffffu) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!((bits >> i) & 1u)) x[i] = -INFINITY;
                }
                float mx = x[0];
#pragma unroll
                for (int i = 1; i < 32; ++i) mx = fmaxf(mx, x[i]);
                const bool need = mx > m + kRaise;
                if (soft_or(need || !ok)) {  // raise the running maximum (rare), or give up
                    ctl.part[part][row] = mx;
                    // O is at rest behind the previous block's product
                    ok = ok && (n == 0 || mbar_await(&ctl.pv_done, uint32_t(n & 1) ^ 1u, &ctl.abort));
                    if (soft_or(!ok)) {
                        failed = true;
                        break;
                    }
                    const float top = fmaxf(fmaxf(ctl.part[0][row], ctl.part[1][row]),
                                            fmaxf(ctl.part[2][row], ctl.part[3][row]));
                    float alpha = 1.f;
                    if (top > m + kRaise) {
                        alpha = exp2f(m - top);
                        m = top;
                        l *= alpha;
                    }
                    __syncwarp();
                    if (!fresh) {
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t r[32];
                            const uint32_t col = kColOT + 128u * half + 32u * c;
                            tmem_ld_32x32b_x32(lane_addr + col, r);
                            tmem_ld_wait(r);
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
                            tmem_st_x32(lane_addr + col, r);
                        }
                        tmem_st_wait();
                        tc_fence_before_sync();
                    }
                    soft_or(false);  // the maxima are read
                }
                uint32_t packed[16];
                const float mr = m == -INFINITY ? 0.f : m;
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float p0 = ex2_approx(x[2 * i] - mr), p1 = ex2_approx(x[2 * i + 1] - mr);
                    sum = add_f32x2(sum, make_float2(p0, p1));
                    const __nv_bfloat162 v = __floats2bfloat162_rn(p0, p1);
                    packed[i] = *reinterpret_cast<const uint32_t*>(&v);
                }
                l += sum.x + sum.y;
                // The previous block's product has read P.
                if (!__all_sync(0xffffffffu, n == 0 || mbar_await(&ctl.pv_done, uint32_t(n & 1) ^ 1u, &ctl.abort))) {
                    failed = true;  // (the others' waits end the same way)
                    if (lane == 0) ctl.abort = 1;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<uint4*>(pbuf + (((4 * half + k) ^ (row & 7)) << 4)) =
                        make_uint4(packed[4 * k], packed[4 * k + 1], packed[4 * k + 2], packed[4 * k + 3]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(p_bar);
                if (w.valid(2 * blk) > 0 && !(bad_here & 1u)) fresh = false;
                if (w.valid(2 * blk + 1) > 0 && !(bad_here & 2u)) fresh = false;
            }
            // ---- the request's output (or partial)
            const bool done = !failed && mbar_await(&ctl.pv_done, uint32_t(n & 1) ^ 1u, &ctl.abort);
            ctl.part[part][row] = l;
            if (soft_or(!done)) {
                failed = true;
                break;
            }
            tc_fence_after_sync();
            const float sum = (ctl.part[0][row] + ctl.part[1][row]) + (ctl.part[2][row] + ctl.part[3][row]);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (0: nothing was seen; a NaN goes on to both outputs)
            const bool whole = w.blo == 0 && w.bhi == w.nb;
            const int64_t at = whole ? q_row : (int64_t(w.range) * kPairTokens + rank) * 2 + (w.blo == 0 ? 1 : 0);
            if (live_token && part == 0)
                (whole ? p.lse : p.lse_part)[at * kMlaHeads + row] =
                    sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2T;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                __syncwarp();
                if (fresh) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                } else {
                    tmem_ld_32x32b_x32(lane_addr + kColOT + 128u * half + 32u * c, o);
                    tmem_ld_wait(o);
                }
                if (c == 3) {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(o_bar);  // O may be overwritten
                }
                if (!live_token) continue;
                const int d = 256 * half + 128 * pg + 32 * c;
                if (whole) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __nv_bfloat162 b2 =
                                __floats2bfloat162_rn(__uint_as_float(o[8 * k + 2 * e]) * inv,
                                                      __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
                            v[e] = *reinterpret_cast<const uint32_t*>(&b2);
                        }
                        *reinterpret_cast<uint4*>(p.out + (at * kMlaHeads + row) * kMlaDv + d + 8 * k) =
                            make_uint4(v[0], v[1], v[2], v[3]);
                    }
                } else {  // eight dims of a head after those of the head before: a warp's stores are contiguous
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(__uint_as_float(o[8 * k + e]) * inv);
                        st_global_v8(p.o_part + tiled_part(at, row, d + 8 * k), v);
                    }
                }
            }
            soft_or(false);  // the sums are read
        }
        if (failed && lane == 0) {
            atomicOr(p.err, kErrWaitTimeout);
            ctl.abort = 1;
        }
        __syncwarp();
    }

    __syncwarp();
    tc_fence_before_sync();
    cluster_sync_all();  // no CTA leaves while the other may read its memory or arrive on its barriers
    tc_fence_after_sync();
    if (warp == 8) {
        if (rank != 0) wait_landed_t(&ctl.all_done, 0);  // the leader's last arrival here
        __syncwarp();
        tmem2_dealloc(tmem_base, kTmemColsT);
    }
}

}  // namespace

cudaError_t mla_tree_pairs(int* pairs) {
    static SmemLimitOnce smem_limit;
    static std::atomic<int> resident[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    e = smem_limit.apply(dev, mla_tree_pair_kernel, kSmemT);
    if (e != cudaSuccess) return e;
    *pairs = resident[dev].load(std::memory_order_relaxed);
    if (*pairs > 0) return cudaSuccess;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = size_t(kSmemT);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(pairs, mla_tree_pair_kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (*pairs < 1) return cudaErrorInvalidConfiguration;
    resident[dev].store(*pairs, std::memory_order_relaxed);
    return cudaSuccess;
}

cudaError_t launch_mla_tree_pair(const MlaTreeMaps& m, MlaTreeParams p, int pairs, cudaStream_t stream) {
    p.clusters = pairs;
    if (p.tokens != kPairTokens || p.tiles != 1 || p.ranges < 1 || p.ranges > kTreeMaxRanges ||
        p.ranges > kTreeMaxRounds * pairs)
        return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2u * unsigned(p.ranges < pairs ? p.ranges : pairs));
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = size_t(kSmemT);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, mla_tree_pair_kernel, m.q, m.v, m.k, m.d, p);
    if (e != cudaSuccess) return e;
    // No request is split where none can have more blocks than are kept together.
    if (tree_blocks(p.table_width, 1) <= kTreeWholeBlocks) return cudaSuccess;
    MlaMergeParams g{};
    g.plan = p.plan;
    g.cuts = p.cuts;
    g.o_part = p.o_part;
    g.lse_part = p.lse_part;
    g.out = p.out;
    g.lse = p.lse;
    g.counts = p.counts;
    g.tokens = p.tokens;
    g.batch = p.batch;
    g.tiled = 1;
    g.by_cut = p.batch > p.ranges;
    g.rows = (g.by_cut ? p.ranges : p.batch) * p.tokens;
    g.one_head = g.rows <= 16 && p.ranges >= 32 * p.batch;
    return launch_mla_merge(g, stream);
}

}  // namespace dsa
