// mla_prefill_kernel.cu -- latent attention over a ragged batch of prompts or
// prompt chunks (expanded form), sm_103a.
//
//     s[i, t] = sm_scale * (q[i, h, :128] . k_nope[t, h] + q[i, h, 128:] . k_rope[t])
//     o[i, h] = sum_t softmax_t(s[i, :]) v[t, h],   lse[i, h] = log sum_t exp(s[i, t])
//
// Row i of a request with n rows and seq_len tokens sees its first
// ceil((seq_len - (n - 1 - i)) / entry_tokens) entries.
//
// One CTA per (256 rows of a request, head): two 128-row query tiles share each
// 128-entry tile of keys and values.  Roles (320 threads):
//   * warps 0-3 and 4-7: softmax of query tile 0 and 1, one row per thread: the
//     row of S from TMEM to registers, its maximum (raised only when a tile
//     passes it by more than 2^8; the accumulator is then rescaled in TMEM),
//     2^x, and P (bf16) back into S's columns.
//   * warp 8: tcgen05.mma, all M = 128, N = 128.  S = Q . K^T from shared memory
//     (12 steps); O += P . V with P from TMEM and V read in place as an MN-major
//     operand (up to 8 steps).  Order per tile: PV of tile 0, next QK of tile 0,
//     PV of tile 1, next QK of tile 1, so that one tile's products run while the
//     other tile's softmax does.
//   * warp 9: TMA.  q once; keys (two 64-dim slabs of the head's own, one shared
//     by all heads) and values (two slabs) through a ring of eight 16 KB slabs.
// TMEM: S/P of the two tiles 2 x 128 columns, O 2 x 128: all 512.
//
// The shared 64 rotary key dims are loaded from their one copy per entry, so no
// 192-wide key is ever built, and every operand may be a strided view.
//
// What bounds it: the tensor cores: 20 MMAs of 128 x 128 x 16 per (128 rows, 128
// entries), 1,280 SM cycles at full rate, of which the 12 with both operands in
// shared memory also take all of its bandwidth.
// Every wait is bounded (about 1 s); a timeout sets an error bit, the roles
// drain, and TMEM is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "indexer_kernels.h"
#include "mla_common.cuh"
#include "sm103_ptx.cuh"

namespace dsa {
namespace {

constexpr int kTile = 128;                      // rows of a query tile, entries of a key tile
constexpr int kSlabB = kTile * 128;             // 128 rows x 64 bf16 dims, 16 KiB
constexpr int kQkSlabs = kPrefillQk / 64;       // 3: two of the head's own, one rotary
constexpr int kRing = 8;
constexpr int kOffQt = 0;                       // q: 2 tiles x 3 slabs
constexpr int kOffRing = kOffQt + 2 * kQkSlabs * kSlabB;
constexpr int kOffCtlP = kOffRing + kRing * kSlabB;
constexpr int kThreadsP = 320;
constexpr uint32_t kTmemColsP = 512;
constexpr uint32_t kColSP = 0;    // S / P of tile i at 128 i
constexpr uint32_t kColOP = 256;  // O of tile i at 256 + 128 i
constexpr float kRaiseLog2 = 8.0f;
constexpr float kLn2P = 0.69314718055994531f;

struct __align__(8) PrefillCtl {
    uint64_t full[kRing], empty[kRing];
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
    uint64_t all_done;
    uint32_t tmem_base;
    int abort;
    int req;
};
constexpr int kSmemP = 1024 + kOffCtlP + int(sizeof(PrefillCtl));
static_assert(kSmemP <= 232448, "fits one CTA per SM");

__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 ra, ra, rb, rc;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// D[tmem] (+)= A[tmem] * B[smem], issued by one thread: A row r in TMEM lane r, column c the bf16
// pair (2 c, 2 c + 1).
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
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

__global__ void __launch_bounds__(kThreadsP, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kn_map,
                       const __grid_constant__ CUtensorMap kr_map, const __grid_constant__ CUtensorMap v_map,
                       const PrefillParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* tiles = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    PrefillCtl& ctl = *reinterpret_cast<PrefillCtl*>(tiles + kOffCtlP);
    const uint32_t s_base = smem_u32(tiles);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // Heads vary fastest, and the last (longest) row blocks come first.
    const int head = int(blockIdx.x % unsigned(p.heads));
    const int slot_t = p.slots - 1 - int(blockIdx.x / unsigned(p.heads));
    if (threadIdx.x == 0) ctl.req = -1;
    __syncthreads();
    pdl_wait_prior_grid();
    pdl_allow_next_grid();

    // Request b owns the slots [cu_q[b] / 256 + b, cu_q[b + 1] / 256 + b + 1): at least as many as it
    // has blocks of 256 rows, so the launch depends on the row count and the batch alone.
    uint32_t bad = 0;
    for (int b = threadIdx.x; b < p.batch; b += kThreadsP) {
        const int64_t s0 = int64_t(__ldg(p.cu_q + b)) / (2 * kTile) + b;
        const int64_t s1 = int64_t(__ldg(p.cu_q + b + 1)) / (2 * kTile) + b + 1;
        if (slot_t >= s0 && slot_t < s1) ctl.req = b;
        if (blockIdx.x == 0) Request(p, b, bad);  // every request is checked, also those without rows
    }
    if (bad) atomicOr(p.err, bad);
    __syncthreads();
    const int b = ctl.req;
    if (b < 0) return;
    const Request rq(p, b, bad);
    const int64_t block = slot_t - (int64_t(__ldg(p.cu_q + b)) / (2 * kTile) + b);
    if (block < 0 || block * 2 * kTile >= rq.rows) return;
    const int row0 = int(block) * 2 * kTile;              // of the request
    const int nrows[2] = {min(rq.rows - row0, kTile), min(max(rq.rows - row0 - kTile, 0), kTile)};
    int limit[2], ntiles[2];                              // entries the tile's last row sees
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        limit[i] = nrows[i] > 0 ? rq.seen(row0 + i * kTile + nrows[i] - 1, p.entry_tokens) : 0;
        ntiles[i] = (limit[i] + kTile - 1) / kTile;
    }
    const int nt = max(ntiles[0], ntiles[1]);
    const int limit_max = max(limit[0], limit[1]);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&ctl.full[i], 1);
            mbar_init(&ctl.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.q_full[i], 1);
            mbar_init(&ctl.s_full[i], 1);
            mbar_init(&ctl.p_full[i], 4);
            mbar_init(&ctl.o_full[i], 1);
        }
        mbar_init(&ctl.all_done, 1);
        ctl.abort = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&ctl.tmem_base, kTmemColsP);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = ctl.tmem_base;

    if (warp == 9) {
        // ================= TMA =================
        if (lane == 0 && nt > 0) {
            const uint64_t pol_q = l2_policy_evict_first(), pol_kv = l2_policy_evict_last();
            int pos = 0;  // slabs issued
            bool stop = false;
            const auto slab = [&](const CUtensorMap* map, bool shared_dims, int x, int row) {
                const int slot = pos & (kRing - 1);
                if (stop || !mbar_wait(&ctl.empty[slot], uint32_t((pos / kRing) & 1) ^ 1u, &ctl.abort)) {
                    stop = true;
                    return;
                }
                mbar_arrive_expect_tx(&ctl.full[slot], uint32_t(kSlabB));
                uint8_t* dst = tiles + kOffRing + slot * kSlabB;
                if (shared_dims)
                    tma_load_2d(dst, map, &ctl.full[slot], x, row, pol_kv);
                else
                    tma_load_3d(dst, map, &ctl.full[slot], x, head, row, pol_kv);
                ++pos;
            };
            const auto load_q = [&](int i) {
                mbar_arrive_expect_tx(&ctl.q_full[i], uint32_t(kQkSlabs * kSlabB));
                for (int s = 0; s < kQkSlabs; ++s)
                    tma_load_3d(tiles + kOffQt + (i * kQkSlabs + s) * kSlabB, &q_map, &ctl.q_full[i], 64 * s, head,
                                rq.q0 + row0 + i * kTile, pol_q);
            };
            const auto load_k = [&](int j) {
                slab(&kn_map, false, 0, rq.kv0 + j * kTile);
                slab(&kn_map, false, 64, rq.kv0 + j * kTile);
                slab(&kr_map, true, 0, rq.kv0 + j * kTile);
            };
            if (ntiles[0] > 0) load_q(0);
            load_k(0);
            if (ntiles[1] > 0) load_q(1);
            for (int j = 0; j < nt && !stop; ++j) {  // in the order of use: K(0) V(0) K(1) V(1) ...
                slab(&v_map, false, 0, rq.kv0 + j * kTile);
                slab(&v_map, false, 64, rq.kv0 + j * kTile);
                if (j + 1 < nt) load_k(j + 1);
            }
            if (stop) {
                atomicOr(p.err, kErrWaitTimeout);
                ctl.abort = 1;
            }
            // no copy outlives the CTA (bounded waits; they have landed unless a role gave up)
            for (int i = pos - 1; i >= 0 && i >= pos - kRing; --i)
                wait_landed_p(&ctl.full[i & (kRing - 1)], uint32_t(i / kRing) & 1u);
            for (int i = 0; i < 2; ++i)
                if (ntiles[i] > 0) wait_landed_p(&ctl.q_full[i], 0);
        }
        __syncwarp();
    } else if (warp == 8) {
        // ================= MMA =================
        constexpr uint32_t kIdescQk = idesc_bf16_f32(kTile, kTile);
        constexpr uint32_t kIdescPv = idesc_bf16_f32(kTile, kPrefillDv) | (1u << 16);  // B (V) MN-major
        bool stop = false;
        const auto ring_wait = [&](int pos) {
            const bool ok = mbar_wait(&ctl.full[pos & (kRing - 1)], uint32_t(pos / kRing) & 1u, &ctl.abort);
            if (!__all_sync(0xffffffffu, ok)) stop = true;
        };
        const auto ring_free = [&](int pos) { umma_commit(&ctl.empty[pos & (kRing - 1)]); };
        const auto ring_addr = [&](int pos) { return s_base + kOffRing + (pos & (kRing - 1)) * kSlabB; };
        // S(tile i) = Q_i . K(j)^T
        const auto qk = [&](int i, int j) {
            if (lane == 0) {
#pragma unroll
                for (int s = 0; s < kQkSlabs; ++s) {
                    const uint64_t a = smem_desc_kmajor_sw128(s_base + kOffQt + (i * kQkSlabs + s) * kSlabB);
                    const uint64_t bd = smem_desc_kmajor_sw128(ring_addr(5 * j + s));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16_ss(tmem_base + kColSP + 128u * i, a + 2u * kk, bd + 2u * kk, kIdescQk,
                                     (s | kk) != 0 ? 1u : 0u);
                }
                umma_commit(&ctl.s_full[i]);
            }
            __syncwarp();
        };
        // O(tile i) += P_i . V(j), over the 16-entry steps below the tile's limit
        const auto pv = [&](int i, int j) {
            if (lane == 0) {
                const int steps = min((limit[i] - j * kTile + 15) >> 4, kTile / 16);
                // Slabs 5 j + 3 and 5 j + 4 may sit at the two ends of the ring: one N = 64 half each.
                const uint32_t v0 = ring_addr(5 * j + 3), v1 = ring_addr(5 * j + 4);
                if (v1 > v0) {
                    for (int kk = 0; kk < steps; ++kk)
                        umma_bf16_ts(tmem_base + kColOP + 128u * i, tmem_base + kColSP + 128u * i + 8u * kk,
                                     desc_mn_sw128(v0 + kk * 2048, kSlabB), kIdescPv, (j | kk) != 0 ? 1u : 0u);
                } else {
                    constexpr uint32_t kIdescHalf = idesc_bf16_f32(kTile, 64) | (1u << 16);
                    for (int kk = 0; kk < steps; ++kk) {
                        umma_bf16_ts(tmem_base + kColOP + 128u * i, tmem_base + kColSP + 128u * i + 8u * kk,
                                     desc_mn_sw128(v0 + kk * 2048, kSlabB), kIdescHalf, (j | kk) != 0 ? 1u : 0u);
                        umma_bf16_ts(tmem_base + kColOP + 128u * i + 64u, tmem_base + kColSP + 128u * i + 8u * kk,
                                     desc_mn_sw128(v1 + kk * 2048, kSlabB), kIdescHalf, (j | kk) != 0 ? 1u : 0u);
                    }
                }
                if (j + 1 == ntiles[i]) umma_commit(&ctl.o_full[i]);
            }
            __syncwarp();
        };
        const auto wait_p = [&](int i, int j) {
            const bool ok = mbar_wait(&ctl.p_full[i], uint32_t(j & 1), &ctl.abort);
            if (!__all_sync(0xffffffffu, ok)) stop = true;
            tc_fence_after_sync();
        };
        if (nt > 0) {
            for (int s = 0; s < kQkSlabs && !stop; ++s) ring_wait(s);
            for (int i = 0; i < 2 && !stop; ++i) {
                if (ntiles[i] == 0) continue;
                if (!__all_sync(0xffffffffu, mbar_wait(&ctl.q_full[i], 0, &ctl.abort))) {
                    stop = true;
                    break;
                }
                tc_fence_after_sync();
                qk(i, 0);
            }
            if (!stop && lane == 0)
                for (int s = 0; s < kQkSlabs; ++s) ring_free(s);
            __syncwarp();
            for (int j = 0; j < nt && !stop; ++j) {
                ring_wait(5 * j + 3);
                if (!stop) ring_wait(5 * j + 4);
                if (stop) break;
                // Value rows behind the last entry that any of these rows sees belong to other requests
                // or hold nothing: zeroed up to the end of the last step (weights there are 0, but 0 x NaN is not).
                const int valid = limit_max - j * kTile;
                if (valid < kTile && (valid & 15)) {
                    const int fill = 16 - (valid & 15);
                    for (int i = lane; i < fill * 16; i += 32) {
                        const int row = valid + (i >> 4), half = (i >> 3) & 1, ch = i & 7;
                        *reinterpret_cast<uint4*>(tiles + kOffRing + ((5 * j + 3 + half) & (kRing - 1)) * kSlabB +
                                                  row * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                bool next_k = false;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (j < ntiles[i]) {
                        wait_p(i, j);
                        if (stop) break;
                        pv(i, j);
                    }
                    if (i == 1 && lane == 0) {
                        ring_free(5 * j + 3);
                        ring_free(5 * j + 4);
                    }
                    if (j + 1 < ntiles[i]) {
                        if (!next_k) {
                            next_k = true;
                            for (int s = 0; s < kQkSlabs && !stop; ++s) ring_wait(5 * (j + 1) + s);
                            if (stop) break;
                            tc_fence_after_sync();
                        }
                        qk(i, j + 1);
                    }
                }
                if (!stop && j + 1 < nt && lane == 0)
                    for (int s = 0; s < kQkSlabs; ++s) ring_free(5 * (j + 1) + s);
                __syncwarp();
            }
        }
        if (lane == 0) {
            if (stop) {
                atomicOr(p.err, kErrWaitTimeout);
                ctl.abort = 1;
            }
            umma_commit(&ctl.all_done);  // every MMA issued has completed when this arrives
        }
        __syncwarp();
    } else {
        // ================= softmax: warps 0-3 tile 0, warps 4-7 tile 1 =================
        const int i = warp >> 2;
        const int r = (warp & 3) * 32 + lane;  // row of the tile
        const uint32_t lane_addr = tmem_base + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t s_addr = lane_addr + kColSP + 128u * i;
        const uint32_t o_addr = lane_addr + kColOP + 128u * i;
        const float c2 = p.sm_scale_log2;
        const int row = row0 + i * kTile + r;
        const bool live_row = r < nrows[i];
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
            if (lane == 0) mbar_arrive(&ctl.p_full[i]);
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
        } else if (nrows[i] > 0) {
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
                    for (int q4 = 0; q4 < 4; ++q4) {
                        uint32_t u[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[8 * q4 + 2 * k]) * inv,
                                                                           __uint_as_float(o[8 * q4 + 2 * k + 1]) * inv);
                            u[k] = *reinterpret_cast<const uint32_t*>(&v);
                        }
                        *reinterpret_cast<uint4*>(o_row + 32 * c + 8 * q4) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 8) {
        const uint32_t addr = smem_u32(&ctl.all_done);
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(addr, 0) && global_timer_ns() - t0 < kWaitLimitNs) {
        }
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, kTmemColsP);
    }
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
    cfg.gridDim = dim3(unsigned(p.slots) * unsigned(p.heads));
    cfg.blockDim = dim3(kThreadsP);
    cfg.dynamicSmemBytes = size_t(kSmemP);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mla_prefill_kernel, q_map, kn_map, kr_map, v_map, p);
}

}  // namespace dsa
