// mla_dense_kernel.cu -- latent attention decode over every live entry of the
// paged cache (absorbed form), one to four query tokens per request, sm_103a; and for
// trees of drafted tokens (kTree) where they are small, or again with a running maximum
// for the requests that mla_tree_kernel.cu, which keeps none, has given up.
//
//     s[h, t] = sm_scale * q[b, j, h] . kv_t                 (576-wide entries)
//     o[b, j, h] = sum_t softmax_t(s[h, :]) kv_t[:512],  lse = log sum_t exp(s[h, t])
//
// over t < ceil((seq_len - (next_n - 1 - j)) / 4).  A tree's tokens see all ceil(seq_len / 4)
// entries, and of one more block, their own entries, those of their masks.
//
// Work split.  A block is one page: 64 entries, 73,728 contiguous bytes.  The
// requests' blocks, laid end to end with kMlaSegUnits units of fixed cost before
// each request, are cut into equal ranges, one per group of next_n CTAs (one CTA
// per SM; token j of a group's requests belongs to its CTA j, so the tokens read
// a page at about the same time and all but the first from L2).  A cut inside a
// request of at most kMlaWholeBlocks blocks moves to its nearer end: joining its parts
// would cost more than reading them one after another.  Every CTA finds its range
// from seq_lens alone.  A request inside one range is written straight to the
// output; one that crosses ranges leaves an fp32 partial per range, and the merge
// kernel joins them by log-sum-exp.
//
// Roles of a CTA (384 threads):
//   * warp 0: TMA.  Each page into nine 64 x 64 slabs of 128-byte-swizzled rows
//     (a ring of 8 slab pairs for the 512 value dims, 2 slabs for the last 64:
//     two blocks), and each request's q.
//   * warp 1: S[head, entry] = Q . K^T, M = 64, N = 64, K = 576, as slabs land;
//     two S accumulators.
//   * warp 2: O^T[dim, head] += V^T . P^T, M = 128 dims x 4, N = 64 heads, K = 64
//     entries, V read in place as an MN-major operand.
//   * warps 4-11: softmax.  Warp w reads the 16 heads of TMEM quadrant w % 4 and
//     half of the block's entries with 16-lane loads that spread them over all 32
//     lanes: 2 heads x 8 entries per thread.  The running maximum is raised only
//     when a block passes it by more than 2^20; then the accumulators are rescaled
//     in TMEM.  At a request's end the warps normalise O^T into the ring half of its
//     last block (released only then), a range's last partial into the whole ring
//     (stage_whole_ring: where the other half is known to be at rest).
//   * warp 3: stores from there with bulk copies; zeroes the outputs of empty requests.
// Row sums add the unrounded fp32 weights; the weights are rounded to bf16 only
// as the second product's operand.
//
// Entries past the live length, or on a page outside the cache, have weight 0
// and their value rows are left out of the product (whole 16-entry steps) or
// zeroed in shared memory, so that nothing stored there, NaN included, matters.
//
// What bounds it: bytes in flight.  A block's slots turn over after its landing
// (loaded latency plus 73.7 KB at an SM's share of HBM) and the chain MMA1 tail,
// softmax, MMA2; the ring holds two blocks, all the shared memory beside q.  64
// requests of 131072 tokens: 373 us, 6480 GB/s, 0.96 of the measured copy rate; one
// of 1M: 66 us, 0.68 (ramp, tail, and 11 us of launch and merge); 64 of 8192: 46.
// Several tokens are bound by the MMAs' rate: 52 a block at about 50 cycles each (their
// operands' reads of shared memory), 2,750 cycles a block and token, of which they run
// 2,270 (64 x 131072, four tokens: 1230 us; the pipe's own figure is 53 %).  Tokens of a
// request in one cluster, its pages loaded once and multicast, took 1352, pages fetched
// into L2 ahead of the ring 1225 (and one token up to 10 % more): bytes are not the bound.
// Shares of at least 2, 3 or 4 units for small batches were slower throughout.
// Every wait is bounded (about 1 s); a timeout sets an error bit, the roles
// drain, and TMEM is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "indexer_kernels.h"
#include "mla_common.cuh"
#include "mla_tree_plan.h"
#include "sm103_ptx.cuh"

namespace dsa {
namespace {

constexpr int kBlk = kPageEntries;             // entries per block: one page
constexpr int kSlabBytes = kBlk * 128;         // 64 rows x 64 bf16 dims, 8 KiB
constexpr int kPairBytes = 2 * kSlabBytes;     // value dims [128 j, 128 j + 128)
constexpr int kVRing = 8;                      // slab pairs (two blocks' values)
constexpr int kRRing = 2;                      // slabs of the last 64 dims
constexpr int kQSlabs = kMlaDim / 64;          // 9
constexpr int kQBox = 3;                       // q slabs per copy
constexpr int kOffQ = 0;
constexpr int kOffP = kOffQ + kQSlabs * kSlabBytes;  // P [64 heads x 64 entries] bf16 (follows q's last
                                                     // slab, whose rows 64..127 an M = 64 MMA may touch)
constexpr int kOffV = kOffP + kSlabBytes;
constexpr int kOffR = kOffV + kVRing * kPairBytes;
constexpr int kOffCtl = kOffR + kRRing * kSlabBytes;
constexpr int kThreadsD = 384;
constexpr int kWarpsD = kThreadsD / 32;
constexpr int kSoftWarp0 = 4;
constexpr int kSoftThreads = 256;
constexpr uint32_t kTmemColsD = 512;
constexpr uint32_t kColS = 0;    // S: 2 x 64 columns
constexpr uint32_t kColO = 128;  // O^T: 4 x 64 columns
// A weight may pass 1 by this much (its rounding is relative, so nothing is lost) before the running
// maximum is raised: ordinary scores never rescale after the first block.  At 2^8 about every second
// request of 256 random entries did, 2,000 cycles each.
constexpr float kRescaleLog2 = 20.0f;
constexpr float kLn2 = 0.69314718055994531f;

struct __align__(16) DenseCtl {
    uint64_t v_full[kVRing], v_empty[kVRing];
    uint64_t r_full[kRRing], r_empty[kRRing];
    uint64_t s_full[2], s_empty[2];
    uint64_t q_full, q_empty, p_full, pv_done, o_empty, all_done;
    uint64_t stage_full, stage_free;  // the output staged in the ring; its first half stored
    uint32_t tmem_base;
    int abort;
    int first_req, first_start;  // request of the range's first unit, and where its units start
    int lo, hi;                  // the range, in units
    int cut;                     // the request that this range is the second one of, or -1
    uint32_t todo[kAgainWords];  // of a tree: a bit for each request that is this call's
    int warp_units[kWarpsD];
    float row_max[2][kMlaHeads];  // per half of the entries; the row sums at a request's end
    alignas(16) float alpha[kMlaHeads];
};
constexpr int kSmemD = 1024 + kOffCtl + int(sizeof(DenseCtl));
static_assert(kSmemD <= 232448, "fits one CTA per SM");

// Named barrier over the 256 softmax threads returning the OR of `v`.
__device__ __forceinline__ bool soft_bar_or(bool v) {
    __syncwarp();
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
__device__ __forceinline__ void soft_bar_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, 256;" ::: "memory");
}

// 16 TMEM lanes x 32 consecutive 32-bit columns over the warp's 32 threads: thread t gets rows
// t / 4 and t / 4 + 8; r[4 k], r[4 k + 1] are row t / 4, columns 8 k + 2 (t % 4) and the next,
// r[4 k + 2], r[4 k + 3] the same columns of row t / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// The same with 64 columns.
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// Four 8 x 8 matrices of 16-bit elements, stored transposed: lane 4 i + k holds row i, columns 2 k and
// 2 k + 1; lane 8 m + c gives the 16-byte address of column c of matrix m.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, const uint32_t (&v)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}

// Rows [row, row + 64) of the map's slabs [slab, ...) (a (dim in slab, row, slab) view of 576-wide rows)
// into consecutive 64 x 64 slabs.
__device__ __forceinline__ void tma_load_slabs(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int32_t row,
                                               int32_t slab, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(slab), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// 64 rows of one slab of a request's drafted entries (rows behind the last arrive as zeros).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int32_t slab,
                                            int32_t request, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(slab), "r"(request), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ uint64_t low_bits(int n) { return n >= 64 ? ~uint64_t(0) : (uint64_t(1) << n) - 1; }

// Bounded wait for a phase of `bar`, whatever the other roles do.
__device__ __forceinline__ void wait_landed(uint64_t* bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(a, parity) && global_timer_ns() - t0 < kWaitLimitNs) {
    }
}

// Tokens of a request, held to [0, max_context].
__device__ __forceinline__ int seq_tokens(const MlaDenseParams& p, int b) {
    const int seq = __ldg(p.seq_lens + b);
    return seq < 0 ? 0 : (int64_t(seq) > p.max_context ? int(p.max_context) : seq);
}
__device__ __forceinline__ int cache_blocks(int seq) { return (((seq + 3) >> 2) + kBlk - 1) / kBlk; }
// A tree's tokens of a request, held to [0, tokens].
__device__ __forceinline__ int drafted_tokens(const MlaDenseParams& p, int b) {
    return p.counts ? min(max(__ldg(p.counts + b), 0), p.tokens) : p.tokens;
}
// A request's blocks: its pages, and of a tree (if it has any tokens) one of their own entries behind them.
template <bool kTree>
__device__ __forceinline__ int blocks_of(const MlaDenseParams& p, int b) {
    const int nb = cache_blocks(seq_tokens(p, b));
    if constexpr (kTree) return drafted_tokens(p, b) > 0 ? nb + 1 : 0;
    return nb;
}

// The CTA's walk over its range: one step per request that has blocks in it.
template <bool kTree>
struct Walk {
    int b, u0, lo, hi, batch;  // request b starts at unit u0; range [lo, hi)
    int seq, nb, blo, bhi;     // current request: tokens, blocks, and this range's blocks [blo, bhi)
    int token, drafted;        // of a tree: this CTA's, and the request's tokens
    const uint32_t* todo;
    __device__ __forceinline__ Walk(const DenseCtl& ctl, const MlaDenseParams& p)
        : b(ctl.first_req), u0(ctl.first_start), lo(ctl.lo), hi(ctl.hi), batch(p.batch), token(blockIdx.x),
          todo(ctl.todo) {}
    __device__ __forceinline__ bool next(const MlaDenseParams& p) {
        while (b < batch && u0 < hi) {
            seq = seq_tokens(p, b);
            nb = blocks_of<kTree>(p, b);
            drafted = kTree ? drafted_tokens(p, b) : 0;
            const int base = u0 + kMlaSegUnits, end = u0 + units_of(nb);
            blo = max(lo, base) - base;
            bhi = min(hi, end) - base;
            ++b;
            u0 = end;
            if (nb > 0 && bhi > blo && (!kTree || (token < drafted && (todo[(b - 1) >> 5] >> ((b - 1) & 31) & 1u))))
                return true;
        }
        return false;
    }
    __device__ __forceinline__ int req() const { return b - 1; }
    // Nothing follows the current request (false if the range ends in units without blocks).
    __device__ __forceinline__ bool last() const { return b >= batch || u0 >= hi; }
    // The block of a tree's own entries.
    __device__ __forceinline__ bool own(int blk) const { return kTree && blk == nb - 1; }
    // Entries of block `blk` that token `back` from the end sees (of a tree's own block: that some token may).
    __device__ __forceinline__ int valid(int blk, int back) const {
        if (own(blk)) return drafted;
        const int n = (max(seq - back, 0) + 3) >> 2;
        return min(max(n - blk * kBlk, 0), kBlk);
    }
};

// The pages of blocks [blk0, blk0 + 32) of the current request: lane's page id, -1 when outside
// the cache or past the range, -2 of a tree's own block.
template <bool kTree>
__device__ __forceinline__ int page_of_lane(const MlaDenseParams& p, const Walk<kTree>& w, int blk0, int lane) {
    const int blk = blk0 + lane;
    if (blk >= w.bhi) return -1;
    if (w.own(blk)) return -2;
    const int page = __ldg(p.page_table + int64_t(w.req()) * p.table_width + blk);
    return (page >= 0 && int64_t(page) < p.num_pages) ? page : -1;
}

template <bool kTree>
__global__ void __launch_bounds__(kThreadsD, 1)
    mla_dense_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kv_map,
                     const __grid_constant__ CUtensorMap kr_map, const __grid_constant__ CUtensorMap o_map,
                     const __grid_constant__ CUtensorMap d_map, const MlaDenseParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    DenseCtl& ctl = *reinterpret_cast<DenseCtl*>(tiles + kOffCtl);
    if (kTree) {
        // The call of another kernel: the requests that it has given up, if there are any.  The plan is that of the whole
        // batch, so that a request's sums do not depend on which others are done again.
        const bool has_word = int(threadIdx.x) < kAgainWords;
        uint32_t word = 0xffffffffu;
        if (p.redo) {
            pdl_wait_prior_grid();
            word = has_word ? p.flags[threadIdx.x] : 0u;
        }
        const int any = __syncthreads_or(has_word && word != 0);
        if (p.redo && blockIdx.x == 0 && blockIdx.y == 0) {
            if (has_word) p.again[threadIdx.x] = word;
            if (threadIdx.x == 0) p.again[kAgainWords] = any ? 1 : 0;
        }
        if (!any) return;
        if (has_word) ctl.todo[threadIdx.x] = word;
        if (p.redo && threadIdx.x == 0) {  // every thread's word is here: the last CTA clears them
            if (atomicAdd(p.ticket, 1u) == gridDim.x * gridDim.y - 1) {
                for (int i = 0; i < kAgainWords; ++i) p.flags[i] = 0;
                *p.ticket = 0;
            }
        }
    }
    const uint32_t s_base = smem_u32(tiles);

    const int warp = uniform(int(threadIdx.x) >> 5);
    const int lane = threadIdx.x & 31;
    const int token = blockIdx.x;  // of the group
    const int group = blockIdx.y;
    const int back = kTree ? 0 : p.tokens - 1 - token;  // (a tree's tokens are not in the cache)

    if (threadIdx.x == 0) {
        for (int i = 0; i < kVRing; ++i) {
            mbar_init(&ctl.v_full[i], 1);
            mbar_init(&ctl.v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.r_full[i], 1);
            mbar_init(&ctl.r_empty[i], 1);
            mbar_init(&ctl.s_full[i], 1);
            mbar_init(&ctl.s_empty[i], kSoftThreads / 32);
        }
        mbar_init(&ctl.q_full, 1);
        mbar_init(&ctl.q_empty, 1);
        mbar_init(&ctl.p_full, kSoftThreads / 32);
        mbar_init(&ctl.pv_done, 1);
        mbar_init(&ctl.o_empty, kSoftThreads / 32);
        mbar_init(&ctl.stage_full, kSoftThreads / 32);
        mbar_init(&ctl.stage_free, 1);
        mbar_init(&ctl.all_done, 2);
        ctl.abort = 0;
        ctl.first_req = p.batch;
        ctl.first_start = 0;
        ctl.cut = -1;
        fence_mbar_init();
        tma_prefetch_map(&q_map);
        tma_prefetch_map(&kv_map);
        tma_prefetch_map(&kr_map);
        if (kTree) tma_prefetch_map(&d_map);
    }
    if (warp == 1) {
        tmem_alloc(&ctl.tmem_base, kTmemColsD);
        tmem_relinquish();
    }
    pdl_wait_prior_grid();
    pdl_allow_next_grid();

    // The range of this group, from the prefix sums of the requests' units.
    const int per = (p.batch + kThreadsD - 1) / kThreadsD;
    const int r0 = min(int(threadIdx.x) * per, p.batch), r1 = min(r0 + per, p.batch);
    int mine = 0;
    for (int b = r0; b < r1; ++b) {
        const int seq = __ldg(p.seq_lens + b);
        if ((seq < 0 || int64_t(seq) > p.max_context) && group == 0 && token == 0) atomicOr(p.err, kErrSeqLenClamped);
        if (kTree && p.counts && __ldg(p.counts + b) != drafted_tokens(p, b) && group == 0 && token == 0)
            atomicOr(p.err, kErrBadRange);
        mine += units_of(blocks_of<kTree>(p, b));
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) ctl.warp_units[warp] = incl;
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    int before = 0, total = 0;
    for (int w = 0; w < kWarpsD; ++w) {
        if (w < warp) before += ctl.warp_units[w];
        total += ctl.warp_units[w];
    }
    const int ngroups = max(min(p.groups, total), 1);
    const Ranges ranges(ngroups, total);
    const int lo = group < ngroups ? ranges.cut(group) : total;
    const int hi = group < ngroups ? ranges.cut(group + 1) : total;
    if (threadIdx.x == 0) {  // cuts at the very end lie in no request
        if (lo == total) ctl.lo = total;
        if (hi == total) ctl.hi = total;
    }
    {
        int u = before + incl - mine;
        for (int b = r0; b < r1; ++b) {
            const int nb = blocks_of<kTree>(p, b), n = units_of(nb);
            if (lo >= u && lo < u + n) {
                ctl.lo = settled_cut(lo, u, nb);
                ctl.first_req = b;
                ctl.first_start = u;
            }
            if (hi >= u && hi < u + n) ctl.hi = settled_cut(hi, u, nb);
            // Is this the request's second range?  Its first block lies in the one before.
            if (nb > kMlaWholeBlocks && lo > u + kMlaSegUnits && lo < u + n && ranges.cut(group - 1) <= u + kMlaSegUnits)
                ctl.cut = b;
            if (group == 0 && token == 0)  // the first and last range that hold its blocks, for the merge
                p.plan[b] = nb > kMlaWholeBlocks ? make_int2(ranges.of(u + kMlaSegUnits), ranges.of(u + n - 1))
                                                 : make_int2(0, 0);
            u += n;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && token == 0) p.cuts[group] = ctl.cut;
    const uint32_t tmem_base = ctl.tmem_base;

    if (warp == 0) {
        // ================= TMA =================
        // The whole warp runs the loop on uniform values; one elected lane issues.
        Walk<kTree> w(ctl, p);
        bool stop = false;
        int n = 0, seg = 0;                         // blocks and requests so far
        int last_v = -1, last_r = -1, last_q = -1;  // the last fills issued
        const bool issuer = elect_one();
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_await(bar, parity, &ctl.abort)) != 0;
        };
        const uint64_t pol_q = l2_policy_evict_first();
        // Tokens of a group share a page through L2; a single token reads it once.
        const uint64_t pol_kv = p.tokens > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
        const uint32_t sb = uint32_t(uniform(int(s_base)));
        while (!stop && w.next(p)) {
            int page_l = page_of_lane(p, w, w.blo, lane);
            if (w.blo + lane < w.bhi && page_l == -1) atomicOr(p.err, kErrBadPage);
            stop = !wait(&ctl.q_empty, uint32_t(seg & 1) ^ 1u);
            if (stop) break;
            if (issuer) {
                mbar_arrive_expect_tx(&ctl.q_full, uint32_t(kQSlabs * kSlabBytes));
                const int row = (w.req() * p.tokens + token) * kMlaHeads;
#pragma unroll
                for (int s = 0; s < kQSlabs; s += kQBox)
                    tma_load_slabs(sb + kOffQ + s * kSlabBytes, &q_map, &ctl.q_full, row, s, pol_q);
            }
            __syncwarp();
            last_q = seg++;
            const int blocks = uniform(w.bhi - w.blo);
#pragma unroll 1
            for (int i = 0; i < blocks; ++i, ++n) {
                if (i > 0 && (i & 31) == 0) {
                    page_l = page_of_lane(p, w, w.blo + i, lane);
                    if (w.blo + i + lane < w.bhi && page_l == -1) atomicOr(p.err, kErrBadPage);
                }
                // a page outside the cache: page 0 stands in, its entries are not used
                const int page = __shfl_sync(0xffffffffu, page_l, i & 31);
                const int row = max(page, 0) * kBlk;
                const bool own = kTree && page == -2;
                const int buf = n & 1;  // half of the ring and rotary slab
                const uint32_t phase = uint32_t((n >> 1) & 1) ^ 1u;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    stop = stop || !wait(&ctl.v_empty[4 * buf + j], phase);
                    if (!stop && issuer) {
                        mbar_arrive_expect_tx(&ctl.v_full[4 * buf + j], uint32_t(kPairBytes));
                        const uint32_t dst = sb + kOffV + (4 * buf + j) * kPairBytes;
                        if (own) {
                            tma_load_4d(dst, &d_map, &ctl.v_full[4 * buf + j], 2 * j, w.req(), pol_kv);
                            tma_load_4d(dst + kSlabBytes, &d_map, &ctl.v_full[4 * buf + j], 2 * j + 1, w.req(), pol_kv);
                        } else {
                            tma_load_slabs(dst, &kv_map, &ctl.v_full[4 * buf + j], row, 2 * j, pol_kv);
                        }
                    }
                    __syncwarp();
                    if (!stop) last_v = 4 * n + j;
                }
                stop = stop || !wait(&ctl.r_empty[buf], phase);
                if (stop) break;
                if (issuer) {
                    mbar_arrive_expect_tx(&ctl.r_full[buf], uint32_t(kSlabBytes));
                    if (own)
                        tma_load_4d(sb + kOffR + buf * kSlabBytes, &d_map, &ctl.r_full[buf], 8, w.req(), pol_kv);
                    else
                        tma_load_2d(tiles + kOffR + buf * kSlabBytes, &kr_map, &ctl.r_full[buf], kMlaDv, row, pol_kv);
                }
                __syncwarp();
                last_r = n;
            }
        }
        if (stop && lane == 0) {
            atomicOr(p.err, kErrWaitTimeout);
            ctl.abort = 1;
        }
        if (lane == 0) {  // no copy outlives the CTA (bounded waits; they have landed unless a role gave up)
            for (int pos = last_v; pos >= 0 && pos > last_v - kVRing; --pos)
                wait_landed(&ctl.v_full[pos & (kVRing - 1)], uint32_t(pos / kVRing) & 1u);
            for (int i = last_r; i >= 0 && i > last_r - kRRing; --i)
                wait_landed(&ctl.r_full[i & (kRRing - 1)], uint32_t(i / kRRing) & 1u);
            if (last_q >= 0) wait_landed(&ctl.q_full, uint32_t(last_q) & 1u);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================= MMA1: S = Q . K^T =================
        // The whole warp runs the loop on uniform values; one elected lane issues.
        constexpr uint32_t kIdesc1 = idesc_bf16_f32(64, 64);
        const uint32_t tmem = uint32_t(uniform(int(tmem_base)));
        const uint32_t sb = uint32_t(uniform(int(s_base)));
        const uint64_t q_desc = smem_desc_kmajor_sw128(sb + kOffQ);
        const uint64_t v_desc = smem_desc_kmajor_sw128(sb + kOffV);
        const uint64_t r_desc = smem_desc_kmajor_sw128(sb + kOffR);
        const bool issuer = elect_one();
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_await(bar, parity, &ctl.abort)) != 0;
        };
        Walk<kTree> w(ctl, p);
        bool ok = true;
        int n = 0, seg = 0;
        while (ok && w.next(p)) {
            ok = wait(&ctl.q_full, uint32_t(seg & 1));
            ++seg;
            const int blocks = uniform(w.bhi - w.blo);
#pragma unroll 1
            for (int i = 0; i < blocks && ok; ++i, ++n) {
                const int buf = n & 1;  // S accumulator, half of the ring and rotary slab
                const uint32_t phase = uint32_t((n >> 1) & 1);
                ok = wait(&ctl.s_empty[buf], phase ^ 1u);
                const uint32_t s_col = tmem + kColS + 64u * buf;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ok = ok && wait(&ctl.v_full[4 * buf + j], phase);
                    tc_fence_after_sync();
                    if (ok && issuer) {
                        const uint64_t a = refreshed(q_desc + uint32_t(2 * j * (kSlabBytes >> 4)));
                        const uint64_t bd = refreshed(v_desc + uint32_t((buf * 4 + j) * (kPairBytes >> 4)));
                        const uint32_t d = refreshed(s_col);
#pragma unroll
                        for (int hs = 0; hs < 2; ++hs)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_bf16_ss(d, a + uint32_t(hs * (kSlabBytes >> 4) + 2 * kk),
                                             bd + uint32_t(hs * (kSlabBytes >> 4) + 2 * kk), kIdesc1,
                                             (j | hs | kk) != 0 ? 1u : 0u);
                    }
                    __syncwarp();
                }
                ok = ok && wait(&ctl.r_full[buf], phase);
                tc_fence_after_sync();
                if (ok && issuer) {
                    const uint64_t a = refreshed(q_desc + uint32_t(8 * (kSlabBytes >> 4)));
                    const uint64_t bd = refreshed(r_desc + uint32_t(buf * (kSlabBytes >> 4)));
                    const uint32_t d = refreshed(s_col);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) umma_bf16_ss(d, a + 2u * kk, bd + 2u * kk, kIdesc1, 1u);
                    umma_commit(&ctl.s_full[buf]);
                    umma_commit(&ctl.r_empty[buf]);
                }
                __syncwarp();
            }
            if (ok && issuer) umma_commit(&ctl.q_empty);
            __syncwarp();
        }
        if (issuer) {
            if (!ok) {
                atomicOr(p.err, kErrWaitTimeout);
                ctl.abort = 1;
            }
            umma_commit(&ctl.all_done);  // every MMA this thread issued has completed when this arrives
        }
        __syncwarp();
    } else if (warp == 2) {
        // ================= MMA2: O^T += V^T . P^T =================
        constexpr uint32_t kIdesc2 = idesc_bf16_f32(128, 64) | (1u << 15);  // A (V^T) MN-major
        const uint32_t tmem = uint32_t(uniform(int(tmem_base)));
        const uint32_t sb = uint32_t(uniform(int(s_base)));
        const uint64_t p_desc = smem_desc_kmajor_sw128(sb + kOffP);
        const uint64_t v_desc = desc_mn_sw128(sb + kOffV, kSlabBytes);
        const bool issuer = elect_one();
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_await(bar, parity, &ctl.abort)) != 0;
        };
        Walk<kTree> w(ctl, p);
        bool ok = true;
        int n = 0, seg = 0;
        while (ok && w.next(p)) {
            uint32_t fresh = 1;  // no product of this request yet
            uint32_t bad = 0;
            const int blocks = uniform(w.bhi - w.blo);
#pragma unroll 1
            for (int i = 0; i < blocks; ++i, ++n) {
                const int blk = w.blo + i;
                if ((i & 31) == 0) bad = __ballot_sync(0xffffffffu, page_of_lane(p, w, blk, lane) == -1);
                const int valid = uniform(((bad >> (i & 31)) & 1u) ? 0 : w.valid(blk, back));
                const int buf = n & 1;  // half of the ring
                if (i == 0) ok = wait(&ctl.o_empty, uint32_t(seg & 1) ^ 1u);
                ok = ok && wait(&ctl.p_full, uint32_t(n & 1));
                if (!ok) break;
                tc_fence_after_sync();
                const bool own = w.own(blk);
                if (own) {  // zero the value rows of drafted entries that nobody sees
                    uint64_t used = 0;
                    for (int j = lane; j < w.drafted; j += 32) used |= __ldg(p.mask + int64_t(w.req()) * p.tokens + j);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) used |= __shfl_xor_sync(0xffffffffu, used, o);
                    used &= low_bits(w.drafted);
                    for (int j = 0; j < 4; ++j)
                        wait_landed(&ctl.v_full[4 * buf + j], uint32_t((n >> 1) & 1));
                    for (int c = lane; c < ((valid + 15) & ~15) * 8; c += 32) {
                        if ((used >> (c >> 3)) & 1u) continue;
#pragma unroll
                        for (int s = 0; s < 8; ++s)
                            *reinterpret_cast<uint4*>(tiles + kOffV + buf * 4 * kPairBytes + s * kSlabBytes + c * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                } else if (valid & 15) {  // zero the value rows behind the live ones in the last 16-entry step
                    const int rows = 16 - (valid & 15);
                    for (int j = 0; j < 4; ++j)  // landed long ago: orders these stores behind the copies
                        wait_landed(&ctl.v_full[4 * buf + j], uint32_t((n >> 1) & 1));
                    for (int c = lane; c < rows * 64; c += 32) {  // 8 slabs x 8 chunks of 16 bytes per row
                        const int row = valid + (c >> 6), slab = (c >> 3) & 7, ch = c & 7;
                        *reinterpret_cast<uint4*>(tiles + kOffV + buf * 4 * kPairBytes + slab * kSlabBytes + row * 128 +
                                                  ch * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (issuer) {
                    // pair by pair, so that the first slots are free (and refilled) early
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint64_t vd = refreshed(v_desc + uint32_t((buf * 4 + j) * (kPairBytes >> 4)));
                        const uint64_t pd = refreshed(p_desc);
                        const uint32_t d = refreshed(tmem + kColO + 64u * j);
                        const auto step = [&](int kk) {
                            umma_bf16_ss(d, vd + uint32_t(kk * (2048 >> 4)), pd + 2u * kk, kIdesc2,
                                         (kk == 0 && fresh) ? 0u : 1u);
                        };
                        if (valid > 48) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) step(kk);
                        } else {
#pragma unroll 1
                            for (int kk = 0; 16 * kk < valid; ++kk) step(kk);
                        }
                        if (i + 1 < blocks) umma_commit(&ctl.v_empty[4 * buf + j]);
                    }
                    umma_commit(&ctl.pv_done);
                }
                __syncwarp();
                if (valid > 0) fresh = 0;
            }
            ++seg;
        }
        if (issuer) {
            if (!ok) {
                atomicOr(p.err, kErrWaitTimeout);
                ctl.abort = 1;
            }
            umma_commit(&ctl.all_done);
        }
        __syncwarp();
    } else if (warp == 3) {
        // ================= output stores =================
        // Requests without entries: out = 0, lse = -inf.
        for (int b = group; b < p.batch && !kTree; b += p.groups) {
            if (blocks_of<kTree>(p, b) > 0) continue;
            const int64_t row = int64_t(b) * p.tokens + token;
            uint4* o = reinterpret_cast<uint4*>(p.out + row * kMlaHeads * kMlaDv);
            for (int i = lane; i < kMlaHeads * kMlaDv / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
            for (int h = lane; h < kMlaHeads; h += 32) p.lse[row * kMlaHeads + h] = -INFINITY;
        }
        const bool issuer = elect_one();
        Walk<kTree> w(ctl, p);
        bool ok = true;
        int n = 0, staged = 0;  // blocks so far, and stagings
        while (ok && w.next(p)) {
            n += w.bhi - w.blo;
            const int buf = (n - 1) & 1;  // the ring half of the request's last block
            const bool whole = w.blo == 0 && w.bhi == w.nb;
            const int64_t row = int64_t(w.req()) * p.tokens + token;
            const int64_t part = int64_t(group * p.tokens + token) * 2 + (w.blo == 0 ? 1 : 0);
            uint8_t* dst = reinterpret_cast<uint8_t*>(p.o_part + part * kMlaHeads * kMlaDv);
            const int rounds = whole || stage_whole_ring(w.last(), w.bhi - w.blo, n) ? 1 : 2;
            for (int r = 0; r < rounds && ok; ++r, ++staged) {
                ok = __all_sync(0xffffffffu, mbar_await(&ctl.stage_full, uint32_t(staged & 1), &ctl.abort)) != 0;
                if (ok && issuer) {
                    if (whole) {
#pragma unroll
                        for (int t = 0; t < 8; ++t)
                            tma_store_2d(&o_map, s_base + kOffV + 4 * buf * kPairBytes + t * kSlabBytes, 64 * t,
                                         int(row) * kMlaHeads);
                    } else if (rounds == 1) {  // the whole ring
                        for (int c = 0; c < 8; ++c)
                            bulk_store(dst + c * kPairBytes, s_base + kOffV + c * kPairBytes, uint32_t(kPairBytes));
                    } else {
                        for (int c = 0; c < 4; ++c)
                            bulk_store(dst + r * 4 * kPairBytes + c * kPairBytes,
                                       s_base + kOffV + (4 * buf + c) * kPairBytes, uint32_t(kPairBytes));
                    }
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    if (r + 1 < rounds) {
                        mbar_arrive(&ctl.stage_free);
                    } else {
                        for (int j = 0; j < 4; ++j) mbar_arrive(&ctl.v_empty[4 * buf + j]);
                    }
                }
                __syncwarp();
            }
        }
        if (issuer) {
            if (!ok) {
                atomicOr(p.err, kErrWaitTimeout);
                ctl.abort = 1;
            }
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
        __syncwarp();
    } else if (warp >= kSoftWarp0) {
        // ================= softmax and output =================
        const int quad = warp & 3;
        const int half = (warp - kSoftWarp0) >> 2;        // entries [32 half, 32 half + 32)
        const int h0 = quad * 16 + (lane >> 2);           // this thread's heads: h0 and h0 + 8
        const uint32_t lane_addr = tmem_base + (uint32_t(quad * 32) << 16);
        const float c2 = p.sm_scale_log2;
        uint8_t* const pbuf = tiles + kOffP;
        Walk<kTree> w(ctl, p);
        bool failed = false;
        int n = 0, halves = 0;  // blocks so far, and outputs staged in two halves
        while (!failed && w.next(p)) {
            const uint64_t drafts =
                kTree ? __ldg(p.mask + int64_t(w.req()) * p.tokens + token) & low_bits(w.drafted) : 0;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
            bool fresh = true;  // no product of this request yet: O^T holds nothing of it
            uint32_t bad = 0;
#pragma unroll 1
            for (int blk = w.blo; blk < w.bhi; ++blk, ++n) {
                if (((blk - w.blo) & 31) == 0)
                    bad = __ballot_sync(0xffffffffu, page_of_lane(p, w, blk, lane) == -1);
                const int valid = ((bad >> ((blk - w.blo) & 31)) & 1u) ? 0 : w.valid(blk, back);
                const int buf = n & 1;
                // The previous block's product has read P (and O^T is at rest) long before the next scores
                // are there: waiting for it first costs nothing.
                bool ok = n == 0 || mbar_await(&ctl.pv_done, uint32_t(n & 1) ^ 1u, &ctl.abort);
                ok = ok && mbar_await(&ctl.s_full[buf], uint32_t((n >> 1) & 1), &ctl.abort);
                ok = __all_sync(0xffffffffu, ok);
                float x[16];
                {
                    uint32_t r[16];
                    tc_fence_after_sync();
                    tmem_ld_16x256b_x4(lane_addr + kColS + 64u * buf + 32u * half, r);
                    tmem_ld_wait16(r);
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.s_empty[buf]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]) * c2;
                }
                if (w.own(blk)) {
                    const uint32_t bits = uint32_t(drafts >> (32 * half)) >> (2 * (lane & 3));
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (!((bits >> (8 * (i >> 2) + (i & 1))) & 1u)) x[i] = -INFINITY;
                } else if (valid < kBlk) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int col = 32 * half + 8 * (i >> 2) + 2 * (lane & 3) + (i & 1);
                        if (col >= valid) x[i] = -INFINITY;
                    }
                }
                float mx[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float a = fmaxf(x[2 * r], x[2 * r + 1]);
#pragma unroll
                    for (int k = 1; k < 4; ++k) a = fmaxf(a, fmaxf(x[4 * k + 2 * r], x[4 * k + 2 * r + 1]));
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
                    mx[r] = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
                }
                const bool need = mx[0] > m[0] + kRescaleLog2 || mx[1] > m[1] + kRescaleLog2;
                if (soft_bar_or(need || !ok)) {  // raise the running maximum (rare), or give up
                    if (lane % 4 == 0) {
                        ctl.row_max[half][h0] = ok ? mx[0] : NAN;
                        ctl.row_max[half][h0 + 8] = mx[1];
                    }
                    if (soft_bar_or(!ok)) {
                        failed = true;
                        break;
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int h = h0 + 8 * r;
                        const float top = fmaxf(ctl.row_max[0][h], ctl.row_max[1][h]);
                        float alpha = 1.f;
                        if (top > m[r] + kRescaleLog2) {
                            alpha = exp2f(m[r] - top);
                            m[r] = top;
                            l[r] *= alpha;
                        }
                        if (half == 0 && lane % 4 == 0) ctl.alpha[h] = alpha;
                    }
                    soft_bar_sync();
                    if (!fresh) {
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int j = 0; j < 4; ++j) {
                            uint32_t r[32];
                            const uint32_t col = kColO + 64u * (2 * half + (j >> 1)) + 32u * (j & 1);
                            tmem_ld_32x32b_x32(lane_addr + col, r);
                            tmem_ld_wait(r);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                r[i] = __float_as_uint(__uint_as_float(r[i]) * ctl.alpha[(j & 1) * 32 + i]);
                            tmem_st_x32(lane_addr + col, r);
                        }
                        tmem_st_wait();
                        tc_fence_before_sync();
                    }
                }
                uint32_t packed[8];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float mr = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float p0 = ex2_approx(x[4 * k + 2 * r] - mr);
                        const float p1 = ex2_approx(x[4 * k + 2 * r + 1] - mr);
                        l[r] += p0 + p1;
                        const __nv_bfloat162 v = __floats2bfloat162_rn(p0, p1);
                        packed[4 * r + k] = *reinterpret_cast<const uint32_t*>(&v);
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int h = h0 + 8 * r;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<uint32_t*>(pbuf + h * 128 + (((4 * half + k) ^ (h & 7)) << 4) +
                                                     4 * (lane & 3)) = packed[4 * r + k];
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.p_full);
                if (valid > 0) fresh = false;
            }
            if (failed) break;
            // ---- the request's output (or partial)
            bool ok = mbar_await(&ctl.pv_done, uint32_t(n & 1) ^ 1u, &ctl.abort);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            }
            if (lane % 4 == 0) {
                ctl.row_max[half][h0] = l[0];
                ctl.row_max[half][h0 + 8] = l[1];
            }
            if (soft_bar_or(!ok)) {
                failed = true;
                break;
            }
            tc_fence_after_sync();
            const int64_t row = int64_t(w.req()) * p.tokens + token;
            const bool whole = w.blo == 0 && w.bhi == w.nb;
            const int64_t part = int64_t(group * p.tokens + token) * 2 + (w.blo == 0 ? 1 : 0);
            if (half == 0 && lane % 4 == 0) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int h = h0 + 8 * r;
                    const float sum = ctl.row_max[0][h] + ctl.row_max[1][h];
                    // (0: nothing was seen; a NaN goes on to both outputs)
                    ctl.alpha[h] = sum == 0.f ? 0.f : 1.f / sum;
                    const float lse = sum == 0.f ? -INFINITY : (m[r] + log2f(sum)) * kLn2;
                    if (whole)
                        p.lse[row * kMlaHeads + h] = lse;
                    else
                        p.lse_part[part * kMlaHeads + h] = lse;
                }
            }
            soft_bar_sync();
            const auto o_read = [&] {  // the last of O^T is in registers
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.o_empty);
            };
            const auto staged = [&] {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl.stage_full);
            };
            if (whole) {
                // bf16, into the ring half of the request's last block: eight 128-byte-swizzled tiles of
                // 64 heads x 64 dims.  This warp: 16-dim strips 128 j + 32 quad + 16 s of j = 2 half,
                // 2 half + 1; each 8 x 8 (dims x heads) piece of a strip is stored transposed.
                const uint32_t stage = s_base + kOffV + ((n - 1) & 1) * 4 * kPairBytes;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t r[32];
                    const int j = 2 * half + (c >> 1), s16 = c & 1;
                    __syncwarp();
                    if (fresh) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] = 0u;
                    } else {
                        tmem_ld_16x256b_x8(lane_addr + (uint32_t(16 * s16) << 16) + kColO + 64u * j, r);
                        tmem_ld_wait(r);
                    }
                    if (c == 3) o_read();
                    // Tile 2 j + quad / 2, 16-byte chunks ch0 (dims 0-7 of the strip) and ch0 + 1.
                    const uint32_t tile = stage + (2 * j + (quad >> 1)) * kSlabBytes;
                    const int ch0 = 4 * (quad & 1) + 2 * s16;
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {  // heads [8 k, 8 k + 16)
                        uint32_t v[4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 f = *reinterpret_cast<const float2*>(ctl.alpha + 8 * (k + e) + 2 * (lane & 3));
#pragma unroll
                            for (int d8 = 0; d8 < 2; ++d8) {
                                const int q = 4 * (k + e) + 2 * d8;
                                const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(r[q]) * f.x,
                                                                                __uint_as_float(r[q + 1]) * f.y);
                                v[2 * e + d8] = *reinterpret_cast<const uint32_t*>(&b2);
                            }
                        }
                        // lane's row address: piece lane / 8 is (heads + 8 (piece / 2), dims + 8 (piece % 2))
                        const int h = 8 * k + 8 * (lane >> 4) + (lane & 7);
                        const int ch = ch0 + ((lane >> 3) & 1);
                        stmatrix_x4_trans(tile + h * 128 + ((ch ^ (h & 7)) << 4), v);
                    }
                }
                staged();
            } else {
                // fp32: the whole ring (stage_whole_ring), or 32 heads at a time in the half of the
                // request's last block.  This warp: dims 128 j + 32 quad + lane of the same j.
                const int rounds = stage_whole_ring(w.last(), w.bhi - w.blo, n) ? 1 : 2;
                float* const stage =
                    reinterpret_cast<float*>(tiles + kOffV + (rounds == 1 ? 0 : ((n - 1) & 1) * 4 * kPairBytes));
#pragma unroll 1
                for (int rd = 0; rd < rounds; ++rd) {
                    if (rd > 0) {
                        ok = mbar_await(&ctl.stage_free, uint32_t(halves & 1), &ctl.abort);
                        ++halves;
                        if (!__all_sync(0xffffffffu, ok)) break;
                    }
                    const int chunks = rounds == 1 ? 4 : 2;
#pragma unroll 1
                    for (int c = 0; c < chunks; ++c) {
                        uint32_t r[32];
                        const int j = 2 * half + (c & 1);
                        const int hb = 32 * (rounds == 1 ? c >> 1 : rd);
                        __syncwarp();
                        if (fresh) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[i] = 0u;
                        } else {
                            tmem_ld_32x32b_x32(lane_addr + kColO + 64u * j + hb, r);
                            tmem_ld_wait(r);
                        }
                        if (rd + 1 == rounds && c + 1 == chunks) o_read();
                        float* o = stage + (rounds == 1 ? hb * kMlaDv : 0) + 128 * j + 32 * quad + lane;
                        const float4* scale = reinterpret_cast<const float4*>(ctl.alpha + hb);
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 f = scale[i / 4];
                            o[i * kMlaDv] = __uint_as_float(r[i]) * f.x;
                            o[(i + 1) * kMlaDv] = __uint_as_float(r[i + 1]) * f.y;
                            o[(i + 2) * kMlaDv] = __uint_as_float(r[i + 2]) * f.z;
                            o[(i + 3) * kMlaDv] = __uint_as_float(r[i + 3]) * f.w;
                        }
                    }
                    staged();
                }
            }
            // alpha and row_max are written again only behind the next block's first barrier
        }
        if (failed && threadIdx.x == kSoftWarp0 * 32) {
            atomicOr(p.err, kErrWaitTimeout);
            ctl.abort = 1;
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        const uint32_t addr = smem_u32(&ctl.all_done);
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(addr, 0) && global_timer_ns() - t0 < kWaitLimitNs) {
        }
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, kTmemColsD);
    }
}

}  // namespace

namespace {

template <bool kTree>
cudaError_t launch(const CUtensorMap& q_map, const CUtensorMap& kv_map, const CUtensorMap& kr_map,
                   const CUtensorMap& o_map, const CUtensorMap& d_map, const MlaDenseParams& p, cudaStream_t stream) {
    static SmemLimitOnce smem_limit;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = smem_limit.apply(dev, mla_dense_kernel<kTree>, kSmemD);
    if (e != cudaSuccess) return e;
    if (p.groups < 1 || p.groups > kMlaMaxGroups || p.tokens < 1) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.tokens), unsigned(p.groups));
    cfg.blockDim = dim3(kThreadsD);
    cfg.dynamicSmemBytes = size_t(kSmemD);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, mla_dense_kernel<kTree>, q_map, kv_map, kr_map, o_map, d_map, p);
    if (e != cudaSuccess) return e;
    // No request is split where none can have more blocks than are kept together.
    if (p.table_width + (kTree ? 1 : 0) <= kMlaWholeBlocks) return cudaSuccess;
    MlaMergeParams m{};
    m.plan = p.plan;
    m.cuts = p.cuts;
    m.o_part = p.o_part;
    m.lse_part = p.lse_part;
    m.out = p.out;
    m.lse = p.lse;
    m.counts = p.counts;
    m.tokens = p.tokens;
    m.by_cut = p.merge_by_cut;
    m.rows = (p.merge_by_cut ? p.groups : p.batch) * p.tokens;
    m.one_head = m.rows <= 16;
    if (p.redo) {  // one merge, for this kernel's partials and those of the one before
        m.again = p.again;
        m.plan_again = m.plan, m.cuts_again = m.cuts, m.o_again = m.o_part, m.lse_again = m.lse_part;
        m.plan = p.first.plan, m.cuts = p.first.cuts, m.o_part = p.first.o_part, m.lse_part = p.first.lse_part;
        m.tiled = 1;
        m.batch = p.batch;
        m.by_cut_again = m.by_cut, m.rows_again = m.rows;
        const int places = p.first.ranges * tree_tiles(p.tokens) * tree_places(p.tokens);
        m.by_cut = p.batch * p.tokens > places;
        m.rows = m.by_cut ? places : p.batch * p.tokens;
        m.one_head = m.rows <= 16 && p.first.ranges >= 32 * p.batch;
    }
    return launch_mla_merge(m, stream);
}

}  // namespace

cudaError_t launch_mla_dense(const CUtensorMap& q_map, const CUtensorMap& kv_map, const CUtensorMap& kr_map,
                             const CUtensorMap& o_map, const MlaDenseParams& p, cudaStream_t stream) {
    return launch<false>(q_map, kv_map, kr_map, o_map, q_map, p, stream);
}

cudaError_t launch_mla_dense_tree(const CUtensorMap& q_map, const CUtensorMap& kv_map, const CUtensorMap& kr_map,
                                  const CUtensorMap& o_map, const CUtensorMap& d_map, const MlaDenseParams& p,
                                  cudaStream_t stream) {
    return launch<true>(q_map, kv_map, kr_map, o_map, d_map, p, stream);
}

}  // namespace dsa
