// mla_prefill_kernel.cu -- latent attention over a ragged batch of prompts or
// prompt chunks (expanded form), sm_103a.
//
//     s[i, t] = sm_scale * (q[i, h, :128] . k_nope[t, h] + q[i, h, 128:] . k_rope[t])
//     o[i, h] = sum_t softmax_t(s[i, :]) v[t, h],   lse[i, h] = log sum_t exp(s[i, t])
//
// Row i of a request with n rows and seq_len tokens sees its first
// ceil((seq_len - (n - 1 - i)) / entry_tokens) entries.
//
// A cluster of two CTAs takes 512 rows of a request and one head: two query tiles
// of 256 rows, each CTA holding 128 rows of both.  All MMAs are cta_group::2
// (M = 256: 128 rows in each CTA's TMEM; N = 128), issued by the leader.  Their
// second operand is split between the two CTAs' shared memory: each loads half of
// every 128-entry tile's keys (64 entries) and half of its values (64 dims), so a
// tile costs an SM 40 KB of loads instead of 80, its shared memory holds three
// tiles, and the operand reads fit its bandwidth.  Roles of a CTA (384 threads):
//   * warps 0-3 and 4-7: softmax of query tile 0 and 1, one row per thread: the
//     row of S from TMEM to registers, its maximum (raised only when a tile
//     passes it by more than 2^8; the accumulator is then rescaled in TMEM),
//     2^x, and P (bf16) back into S's columns.
//   * warp 8 (leader): tcgen05.mma.  S = Q . K^T from shared memory (12 steps);
//     O += P . V with P from TMEM and V read in place as an MN-major operand (up to
//     8 steps).  Order per tile: PV of query tile 0, its next QK, PV of query tile
//     1, its next QK, so that one tile's products run while the other's softmax does.
//   * warp 9: TMA.  q once; keys (two 64-dim slabs of the head's own, one shared
//     by all heads) and values, three stages each.  Both CTAs' copies count on the
//     leader's barriers.
//   * warp 10: zeroes the value rows behind the last entry (see below).
// TMEM: S/P of the two tiles 2 x 128 columns, O 2 x 128: all 512.
//
// The shared 64 rotary key dims are loaded from their one copy per entry, so no
// 192-wide key is ever built, and every operand may be a strided view.
//
// What bounds it: the tensor cores: 20 MMA steps of 128 x 128 x 16 per SM for each
// (128 rows, 128 entries), 1,280 SM cycles at full rate.
// Every wait is bounded (about 1 s) but the cluster barriers, which every thread
// reaches; a timeout sets an error bit, the roles drain, and TMEM is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "indexer_kernels.h"
#include "mla_common.cuh"
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
constexpr int kRegsSoftmax = 200, kRegsOther = 104;  // 8 x 200 + 4 x 104 = 12 x 168 a warp lane
constexpr uint32_t kTmemColsP = 512;
constexpr uint32_t kColSP = 0;    // S / P of tile i at 128 i
constexpr uint32_t kColOP = 256;  // O of tile i at 256 + 128 i
constexpr float kRaiseLog2 = 8.0f;
constexpr float kLn2P = 0.69314718055994531f;

struct __align__(8) PrefillCtl {
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
    uint64_t tail_landed, tail_ready, all_done;
    uint32_t tmem_base;
    int abort;
    int req, block;  // this slot's request (-1: none) and block of rows
};
constexpr int kSmemP = 1024 + kOffCtlP + int(sizeof(PrefillCtl));
static_assert(kSmemP <= 232448, "fits one CTA per SM");

// Two-CTA MMAs, issued by one thread of the leader: M = 256 (128 rows of A and D in each CTA), each
// CTA's shared memory (at the same offsets) holding half of B.  A from shared memory:
__device__ __forceinline__ void umma2_bf16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// A from TMEM: row r in lane r, column c the bf16 pair (2 c, 2 c + 1).
__device__ __forceinline__ void umma2_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive once on the barrier at this offset in both CTAs when every MMA this thread issued has completed.
__device__ __forceinline__ void umma2_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(uint16_t(3))
        : "memory");
}

// TMA loads into this CTA that count on a barrier given by its shared::cluster address.
__device__ __forceinline__ void tma2_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y,
                                             int32_t z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma2_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y,
                                             uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy)
        : "memory");
}

// Arrive on a barrier of either CTA (shared::cluster address).  What the arrivals on p_full order is
// tensor memory, through the tcgen05 fences; the cluster-scope release and acquire below cost 250 to 470
// cycles a time on the MMA's path and are kept for ordinary stores (the zeroed value rows).
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// mbar_wait that also orders what the other CTA did before its arrivals.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, const volatile int* abort) {
    const uint32_t a = smem_u32(bar);
    const auto try_wait = [&] {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(a), "r"(parity)
            : "memory");
        return ok != 0;
    };
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (try_wait()) return true;
    const uint64_t t0 = global_timer_ns();
#pragma unroll 1
    while (true) {
        if (try_wait()) return true;
        if (*abort) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) return false;
    }
}

__device__ __forceinline__ void tmem2_alloc(uint32_t* dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem2_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
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

__global__ void __launch_bounds__(kThreadsP, 1) __cluster_dims__(2, 1, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kn_map,
                       const __grid_constant__ CUtensorMap kr_map, const __grid_constant__ CUtensorMap v_map,
                       const PrefillParams p) {
    extern __shared__ uint8_t smem_raw[];
    // Dynamic shared memory starts at the same offset in both CTAs, so the operands and barriers do too.
    uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    PrefillCtl& ctl = *reinterpret_cast<PrefillCtl*>(tiles + kOffCtlP);
    const uint32_t s_base = smem_u32(tiles);
    const int warp = uniform(int(threadIdx.x) >> 5);
    const int lane = threadIdx.x & 31;
    const int rank = int(cluster_rank());  // 0: the leader

    // Heads vary fastest, and the last (longest) row blocks come first.
    const unsigned unit = blockIdx.x >> 1;
    const int head = int(unit % unsigned(p.heads));
    const int slot_t = p.slots - 1 - int(unit / unsigned(p.heads));
    if (threadIdx.x == 0) {
        ctl.req = -1;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&ctl.k_full[i], 1);
            mbar_init(&ctl.k_empty[i], 1);
            mbar_init(&ctl.v_full[i], 1);
            mbar_init(&ctl.v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.q_full[i], 1);
            mbar_init(&ctl.s_full[i], 1);
            mbar_init(&ctl.p_full[i], 8);  // four warps of each CTA
            mbar_init(&ctl.o_full[i], 1);
        }
        mbar_init(&ctl.tail_landed, 1);
        mbar_init(&ctl.tail_ready, 2);
        mbar_init(&ctl.all_done, 1);
        ctl.abort = 0;
        fence_mbar_init();
        tma_prefetch_map(&q_map);
        tma_prefetch_map(&kn_map);
        tma_prefetch_map(&kr_map);
        tma_prefetch_map(&v_map);
    }
    if (warp == 8) tmem2_alloc(&ctl.tmem_base, kTmemColsP);
    __syncwarp();
    tc_fence_before_sync();
    cluster_arrive();
    __syncthreads();
    pdl_wait_prior_grid();
    pdl_allow_next_grid();

    // Request b owns the slots [cu_q[b] / 512 + b, cu_q[b + 1] / 512 + b + 1): at least as many as it
    // has blocks of 512 rows, so the launch depends on the row count and the batch alone.
    uint32_t bad = 0;
    for (int b = threadIdx.x; b < p.batch; b += kThreadsP) {
        const Request r(p, b, bad);  // loaded by the way, so that the owner's lines are in L1 below
        const int64_t s0 = int64_t(__ldg(p.cu_q + b)) / kPrefillBlock + b;
        const int64_t s1 = int64_t(__ldg(p.cu_q + b + 1)) / kPrefillBlock + b + 1;
        if (slot_t >= s0 && slot_t < s1 && slot_t - s0 < (r.rows + kPrefillBlock - 1) / kPrefillBlock) {
            ctl.req = b;
            ctl.block = int(slot_t - s0);
        }
    }
    if (bad && blockIdx.x == 0) atomicOr(p.err, bad);  // every request is checked, also those without rows
    __syncwarp();
    cluster_wait();  // the other CTA's barriers are set up too
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = ctl.tmem_base;
    const int b = ctl.req;
    if (b < 0) {  // a slot without rows; both CTAs alike
        cluster_sync_all();
        if (warp == 8) tmem2_dealloc(tmem_base, kTmemColsP);
        return;
    }
    const Request rq(p, b, bad);
    // Query tile i: rows [row0 + 256 i, + 256) of the request, the second 128 of them in CTA 1.
    const int row0 = ctl.block * kPrefillBlock;
    int limit[2], ntiles[2];  // entries that the tile's last row sees
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int last = min(rq.rows, row0 + (i + 1) * 2 * kTile) - 1;
        limit[i] = last >= row0 + i * 2 * kTile ? rq.seen(last, p.entry_tokens) : 0;
        ntiles[i] = (limit[i] + kTile - 1) / kTile;
    }
    const int nt = max(ntiles[0], ntiles[1]);
    const int limit_max = max(limit[0], limit[1]);
    // Value rows behind the last entry that any of these rows sees belong to other requests or hold
    // nothing.  Products stop at a 16-entry step, and where that is not the end of the entries the rows
    // up to it are zeroed (weights there are 0, but 0 x NaN is not): the last tile's values count on a
    // barrier of each CTA, whose warp 10 zeroes them and tells the leader.
    const bool tail = (limit_max & 15) != 0;

    if (warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 9) {
        // ================= TMA =================
        if (lane == 0 && nt > 0) {
            const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
            bool stop = false;
            const auto load_q = [&](int i) {
                const uint32_t bar = cluster_addr(&ctl.q_full[i], 0);
                if (rank == 0) mbar_arrive_expect_tx(&ctl.q_full[i], uint32_t(2 * kQkSlabs * kSlabB));
                for (int s = 0; s < kQkSlabs; ++s)
                    tma2_load_3d(s_base + kOffQt + (i * kQkSlabs + s) * kSlabB, &q_map, bar, 64 * s, head,
                                 rq.q0 + row0 + i * 2 * kTile + rank * kTile, pol_q);
            };
            const auto load_k = [&](int j) {  // this CTA's 64 entries of tile j
                const int st = j % kStages;
                if (stop || !mbar_wait(&ctl.k_empty[st], uint32_t((j / kStages) & 1) ^ 1u, &ctl.abort)) {
                    stop = true;
                    return;
                }
                const uint32_t bar = cluster_addr(&ctl.k_full[st], 0);
                if (rank == 0) mbar_arrive_expect_tx(&ctl.k_full[st], uint32_t(2 * kStageK));
                const uint32_t dst = s_base + kOffK + st * kStageK;
                const int row = rq.kv0 + j * kTile + rank * (kTile / 2);
                tma2_load_3d(dst, &kn_map, bar, 0, head, row, pol_kv);
                tma2_load_3d(dst + kHalfB, &kn_map, bar, 64, head, row, pol_kv);
                tma2_load_2d(dst + 2 * kHalfB, &kr_map, bar, 0, row, pol_kv);
            };
            const auto load_v = [&](int j) {  // this CTA's 64 value dims of tile j
                const int st = j % kStages;
                if (stop || !mbar_wait(&ctl.v_empty[st], uint32_t((j / kStages) & 1) ^ 1u, &ctl.abort)) {
                    stop = true;
                    return;
                }
                const bool last = tail && j == nt - 1;
                const uint32_t bar = last ? cluster_addr(&ctl.tail_landed, uint32_t(rank)) : cluster_addr(&ctl.v_full[st], 0);
                if (last)
                    mbar_arrive_expect_tx(&ctl.tail_landed, uint32_t(kStageV));
                else if (rank == 0)
                    mbar_arrive_expect_tx(&ctl.v_full[st], uint32_t(2 * kStageV));
                tma2_load_3d(s_base + kOffV + st * kStageV, &v_map, bar, 64 * rank, head, rq.kv0 + j * kTile, pol_kv);
            };
            if (ntiles[0] > 0) load_q(0);
            load_k(0);
            if (ntiles[1] > 0) load_q(1);
            for (int j = 0; j < nt && !stop; ++j) {
                load_v(j);
                if (j + 1 < nt) load_k(j + 1);
            }
            if (stop) {
                atomicOr(p.err, kErrWaitTimeout);
                ctl.abort = 1;
            }
            // No copy outlives the cluster (bounded waits; they have landed unless a role gave up).  The
            // leader's barriers count both CTAs' copies, and neither CTA leaves before the other.
            if (rank == 0) {
                for (int j = max(nt - kStages, 0); j < nt; ++j) {
                    wait_landed_p(&ctl.k_full[j % kStages], uint32_t(j / kStages) & 1u);
                    if (!(tail && j == nt - 1)) wait_landed_p(&ctl.v_full[j % kStages], uint32_t(j / kStages) & 1u);
                }
                for (int i = 0; i < 2; ++i)
                    if (ntiles[i] > 0) wait_landed_p(&ctl.q_full[i], 0);
            }
            if (tail) wait_landed_p(&ctl.tail_landed, 0);
        }
        __syncwarp();
    } else if (warp == 10) {
        // ================= the last tile's value rows =================
        if (tail) {
            const bool ok = mbar_wait(&ctl.tail_landed, 0, &ctl.abort);
            if (__all_sync(0xffffffffu, ok)) {
                const int valid = limit_max - (nt - 1) * kTile;
                const int fill = 16 - (valid & 15);
                uint8_t* v = tiles + kOffV + ((nt - 1) % kStages) * kStageV;
                for (int i = lane; i < fill * 8; i += 32)
                    *reinterpret_cast<uint4*>(v + (valid + (i >> 3)) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                asm volatile("fence.proxy.async;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(cluster_addr(&ctl.tail_ready, 0));
            }
        }
    } else if (warp == 8 && rank == 0) {
        // ================= MMA (the leader's) =================
        // The whole warp runs the loop; one elected lane issues.
        constexpr uint32_t kIdescQk = idesc_bf16_f32(2 * kTile, kTile);
        constexpr uint32_t kIdescPv = idesc_bf16_f32(2 * kTile, kPrefillDv) | (1u << 16);  // B (V) MN-major
        const uint32_t tmem = uint32_t(uniform(int(tmem_base)));
        const uint32_t sb = uint32_t(uniform(int(s_base)));
        const int n_all = uniform(nt);
        const int n_of[2] = {uniform(ntiles[0]), uniform(ntiles[1])};
        const int lim[2] = {uniform(limit[0]), uniform(limit[1])};
        const uint64_t q_desc = smem_desc_kmajor_sw128(sb + kOffQt);
        const uint64_t k_desc = smem_desc_kmajor_sw128(sb + kOffK);
        const uint64_t v_desc = desc_mn_sw128(sb + kOffV, kSlabB);
        const bool issuer = elect_one();
        // S(tile i) = Q_i . K^T, keys in stage st
        const auto qk = [&](int i, int st) {
            if (issuer) {
                const uint64_t a = q_desc + uint32_t(i * kQkSlabs * (kSlabB >> 4));
                const uint64_t bd = k_desc + uint32_t(st * (kStageK >> 4));
#pragma unroll
                for (int s = 0; s < kQkSlabs; ++s)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma2_bf16_ss(tmem + kColSP + 128u * i, a + uint32_t(s * (kSlabB >> 4) + 2 * kk),
                                      bd + uint32_t(s * (kHalfB >> 4) + 2 * kk), kIdescQk, (s | kk) != 0 ? 1u : 0u);
                umma2_commit(&ctl.s_full[i]);
            }
            __syncwarp();
        };
        // O(tile i) += P_i . V, values in stage st, over the 16-entry steps below the tile's limit
        const auto pv = [&](int i, int j, int st) {
            const int steps = min((lim[i] - j * kTile + 15) >> 4, kTile / 16);
            if (issuer) {
                const uint64_t bd = v_desc + uint32_t(st * (kStageV >> 4));
                const auto step = [&](int kk) {
                    umma2_bf16_ts(tmem + kColOP + 128u * i, tmem + kColSP + 128u * i + 8u * kk, bd + 128u * kk, kIdescPv,
                                  (j | kk) != 0 ? 1u : 0u);
                };
                if (steps == kTile / 16) {
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk) step(kk);
                } else {
#pragma unroll 1
                    for (int kk = 0; kk < steps; ++kk) step(kk);
                }
                if (j + 1 == n_of[i]) umma2_commit(&ctl.o_full[i]);
            }
            __syncwarp();
        };
        const auto commit = [&](uint64_t* bar) {
            if (issuer) umma2_commit(bar);
            __syncwarp();
        };
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, &ctl.abort)) != 0;
        };
        bool ok = n_all == 0 || wait(&ctl.k_full[0], 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (ok && n_of[i] > 0) {
                ok = wait(&ctl.q_full[i], 0);
                tc_fence_after_sync();
                if (ok) qk(i, 0);
            }
        }
        if (ok && n_all > 0) commit(&ctl.k_empty[0]);
        int st = 0, st_next = 1;          // stages of tiles j and j + 1, and their phases
        uint32_t phase = 0, phase_next = 0;
#pragma unroll 1
        for (int j = 0; j < n_all && ok; ++j) {
            bool have_k = false, have_v = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (ok && j < n_of[i]) {
                    if (!have_v) {
                        if (tail && j == n_all - 1)
                            ok = __all_sync(0xffffffffu, mbar_wait_cluster(&ctl.tail_ready, 0, &ctl.abort)) != 0;
                        else
                            ok = wait(&ctl.v_full[st], phase);
                    }
                    have_v = true;
                    if (ok) ok = wait(&ctl.p_full[i], uint32_t(j & 1));
                    tc_fence_after_sync();
                    if (ok) pv(i, j, st);
                }
                if (ok && i == 1) commit(&ctl.v_empty[st]);
                if (ok && j + 1 < n_of[i]) {
                    if (!have_k) ok = wait(&ctl.k_full[st_next], phase_next);
                    have_k = true;
                    tc_fence_after_sync();
                    if (ok) qk(i, st_next);
                }
            }
            if (ok && j + 1 < n_all) commit(&ctl.k_empty[st_next]);
            st = st_next;
            phase = phase_next;
            if (++st_next == kStages) {
                st_next = 0;
                phase_next ^= 1u;
            }
        }
        if (!ok && issuer) {
            atomicOr(p.err, kErrWaitTimeout);
            ctl.abort = 1;
        }
        commit(&ctl.all_done);
        wait_landed_p(&ctl.all_done, 0);  // every MMA issued has completed
        __syncwarp();
    } else if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ================= softmax: warps 0-3 tile 0, warps 4-7 tile 1 =================
        const int i = warp >> 2;
        const int r = (warp & 3) * 32 + lane;  // row of the tile
        const uint32_t lane_addr = tmem_base + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t s_addr = lane_addr + kColSP + 128u * i;
        const uint32_t o_addr = lane_addr + kColOP + 128u * i;
        const float c2 = p.sm_scale_log2;
        const int row = row0 + i * 2 * kTile + rank * kTile + r;  // of the request
        const bool live_row = row < rq.rows;
        const uint32_t p_bar = cluster_addr(&ctl.p_full[i], 0);
        const int see = live_row ? rq.seen(row, p.entry_tokens) : limit[i];
        float m = -INFINITY;
        float2 l2 = make_float2(0.f, 0.f);
        bool failed = false;
#pragma unroll 1
        for (int j = 0; j < ntiles[i]; ++j) {
            const bool ok = mbar_wait(&ctl.s_full[i], uint32_t(j & 1), &ctl.abort);
            if (!__all_sync(0xffffffffu, ok)) {
                failed = true;
                break;
            }
            tc_fence_after_sync();
            uint32_t s[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(s_addr + 32u * c, s[c]);
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_wait(s[c]);
            const int here = see - j * kTile;  // entries of this tile that the row sees
            if (__any_sync(0xffffffffu, here < kTile)) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (32 * c + k >= here) s[c][k] = 0xFF800000u;  // -inf
            }
            float mx4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                mx4[c] = __uint_as_float(s[c][0]);
#pragma unroll
                for (int k = 1; k < 32; ++k) mx4[c] = fmaxf(mx4[c], __uint_as_float(s[c][k]));
            }
            const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * c2;
            const bool need = mx > m + kRaiseLog2;
            if (__any_sync(0xffffffffu, need)) {  // rare after the first tile
                float alpha = 1.f;
                if (need) {
                    alpha = exp2f(m - mx);
                    m = mx;
                    l2.x *= alpha;
                    l2.y *= alpha;
                }
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
            const float2 cc = make_float2(c2, c2);
            const float nm = m == -INFINITY ? 0.f : -m;
            const float2 mm = make_float2(nm, nm);
#pragma unroll
            for (int hp = 0; hp < 2; ++hp) {
                uint32_t pk[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const int c = 2 * hp + (k >> 4), e = 2 * (k & 15);
                    float2 x = fma_f32x2(make_float2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), cc, mm);
                    x.x = ex2_approx(x.x);
                    x.y = ex2_approx(x.y);
                    l2 = add_f32x2(l2, x);
                    const __nv_bfloat162 v = __floats2bfloat162_rn(x.x, x.y);
                    pk[k] = *reinterpret_cast<const uint32_t*>(&v);
                }
                tmem_st_x32(s_addr + 32u * hp, pk);
            }
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(p_bar);
        }
        // ---- output
        if (!failed && ntiles[i] > 0) {
            const bool ok = mbar_wait(&ctl.o_full[i], 0, &ctl.abort);
            failed = !__all_sync(0xffffffffu, ok);
        }
        if (failed) {
            if (lane == 0) {
                atomicOr(p.err, kErrWaitTimeout);
                ctl.abort = 1;
            }
        } else if (__any_sync(0xffffffffu, live_row)) {
            tc_fence_after_sync();
            const float l = l2.x + l2.y;
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const int64_t token = int64_t(rq.q0) + row;
            __nv_bfloat16* o_row = reinterpret_cast<__nv_bfloat16*>(p.out) + (token * p.heads + head) * kPrefillDv;
            if (live_row) p.lse[token * p.heads + head] = l > 0.f ? (m + log2f(l)) * kLn2P : -INFINITY;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                if (ntiles[i] > 0) {
                    tmem_ld_32x32b_x32(o_addr + 32u * c, o);
                    tmem_ld_wait(o);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0u;
                }
                if (live_row) {
#pragma unroll
                    for (int q4 = 0; q4 < 2; ++q4) {  // a whole sector a lane
                        uint32_t u[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[16 * q4 + 2 * k]) * inv,
                                                                           __uint_as_float(o[16 * q4 + 2 * k + 1]) * inv);
                            u[k] = *reinterpret_cast<const uint32_t*>(&v);
                        }
                        if (p.out_aligned32) {
                            st_global_v8(o_row + 32 * c + 16 * q4, u);
                        } else {
                            uint4* d = reinterpret_cast<uint4*>(o_row + 32 * c + 16 * q4);
                            d[0] = make_uint4(u[0], u[1], u[2], u[3]);
                            d[1] = make_uint4(u[4], u[5], u[6], u[7]);
                        }
                    }
                }
            }
        }
    }

    // The leader's last arrival here: none of its earlier ones is still under way to this CTA.
    if (warp == 8 && rank == 1) wait_landed_p(&ctl.all_done, 0);
    __syncwarp();
    tc_fence_before_sync();
    cluster_sync_all();  // no CTA leaves while the other may read its memory or arrive on its barriers
    tc_fence_after_sync();
    if (warp == 8) tmem2_dealloc(tmem_base, kTmemColsP);
}

}  // namespace

cudaError_t launch_mla_prefill(const CUtensorMap& q_map, const CUtensorMap& kn_map, const CUtensorMap& kr_map,
                               const CUtensorMap& v_map, const PrefillParams& p, cudaStream_t stream) {
    static SmemLimitOnce smem_limit;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = smem_limit.apply(dev, mla_prefill_kernel, kSmemP);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2u * unsigned(p.slots) * unsigned(p.heads));
    cfg.blockDim = dim3(kThreadsP);
    cfg.dynamicSmemBytes = size_t(kSmemP);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mla_prefill_kernel, q_map, kn_map, kr_map, v_map, p);
}

}  // namespace dsa
