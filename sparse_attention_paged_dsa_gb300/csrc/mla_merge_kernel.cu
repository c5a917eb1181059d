// mla_merge_kernel.cu -- joins the partial outputs of requests whose entries the
// dense and the tree decode cut between ranges.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "indexer_kernels.h"
#include "mla_tree_plan.h"
#include "sm103_ptx.cuh"

namespace dsa {
namespace {

// o[r] = sum_i exp(lse_i - lse) o_i over the partials of a split request, lse = log sum_i exp(lse_i).
// 512 threads.  128 of them per 512 dims, four heads a CTA; or (kOneHead: few rows, each split many ways)
// 64 per 256 dims, half a head a CTA, whose partials go to the eight groups in turn.  Grid (heads / 4 or
// heads x 2, requests or cuts x tokens).
// kTiled: of the kernels on clusters.  kAgain: of requests that the dense kernel has done again.
template <bool kOneHead>
using Weights = float[kOneHead ? 1 : 4][kMlaMaxGroups];
template <bool kOneHead>
using Sums = float4[kOneHead ? 7 : 1][64];
template <bool kOneHead, bool kTiled, bool kAgain>
__device__ __forceinline__ void merge_row(const MlaMergeParams& p, int at, bool any_again, Weights<kOneHead>& wgt,
                                          Sums<kOneHead>& acc_s) {
    const int2* const plan = kAgain ? p.plan_again : p.plan;
    const int32_t* const cuts = kAgain ? p.cuts_again : p.cuts;
    const float* const o_part = kAgain ? p.o_again : p.o_part;
    const float* const lse_part = kAgain ? p.lse_again : p.lse_part;
    const bool by_cut = kAgain ? p.by_cut_again : p.by_cut;
    const int quarter = threadIdx.x >> (kOneHead ? 6 : 7);
    const int d4 = kOneHead ? (int(blockIdx.x) & 1) * 64 + (threadIdx.x & 63) : threadIdx.x & 127;
    const int h = kOneHead ? int(blockIdx.x) >> 1 : int(blockIdx.x) * 4 + quarter;
    const int places = kTiled ? tree_places(p.tokens) : p.tokens;  // of a range's partials
    int token = at % p.tokens, b;
    if constexpr (kTiled) {
        b = at / p.tokens;
        if (by_cut) {
            b = cuts[at / places];
            if (b < 0) return;
            token = kTileTokens * (b & 15) + at % places, b >>= 4;
            if (token >= p.tokens) return;
        }
    } else {
        b = by_cut ? cuts[at / p.tokens] : at / p.tokens;
        if (b < 0) return;
    }
    if (p.counts && token >= __ldg(p.counts + b)) return;
    // a request's partials are those of the kernel that has done it last
    if ((kTiled || kAgain) && any_again && bool(p.again[b >> 5] >> (b & 31) & 1u) != kAgain) return;
    const int64_t row = int64_t(b) * p.tokens + token;
    const int2 g = plan[kTiled ? token / kTileTokens * p.batch + b : b];
    if (g.x == g.y) return;  // one range: written by the attention kernel
    const int S = g.y - g.x + 1;
    // partial i: range g.x + i; the first one ends in the next range, the others began earlier
    const int place = kTiled ? token % kTileTokens : token;
    const auto part = [&](int i) { return (int64_t(g.x + i) * places + place) * 2 + (i == 0 ? 1 : 0); };
    // The first partials are on their way while the weights are made.
    const auto value = [&](int i) {
        return *reinterpret_cast<const float4*>(o_part + (kTiled ? tiled_part(part(i), h, 4 * d4)
                                                                   : (part(i) * kMlaHeads + h) * kMlaDv + 4 * d4));
    };
    constexpr int kStep = kOneHead ? 8 : 1;
    const int first = kOneHead ? quarter : 0;
    // (not for the dense kernel's many requests of two parts each: 200 of 4096 tokens took 71 us, 68 without)
    constexpr int kEarly = kOneHead || kTiled ? 4 : 0;
    float4 early[kEarly + 1];
#pragma unroll
    for (int k = 0; k < kEarly; ++k) early[k] = value(min(first + k * kStep, S - 1));
    if ((threadIdx.x & 127) < 32 && (!kOneHead || quarter == 0)) {
        float* const w = wgt[kOneHead ? 0 : quarter];
        const int lane = threadIdx.x & 31;
        float mx = -INFINITY;
        for (int i = lane; i < S; i += 32) {
            w[i] = lse_part[part(i) * kMlaHeads + h];
            mx = fmaxf(mx, w[i]);
        }
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        float sum = 0.f;
        for (int i = lane; i < S; i += 32) {
            const float e = w[i] == -INFINITY ? 0.f : expf(w[i] - mx);  // (a NaN, which the maximum passes by, stays)
            w[i] = e;
            sum += e;
        }
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        for (int i = lane; i < S; i += 32) w[i] *= inv;
        if (lane == 0 && (!kOneHead || (blockIdx.x & 1) == 0))
            p.lse[row * kMlaHeads + h] = sum == 0.f ? -INFINITY : mx + logf(sum);
    }
    __syncthreads();
    const float* const w = wgt[kOneHead ? 0 : quarter];
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto add = [&](int i, const float4& v) {
        acc.x = fmaf(w[i], v.x, acc.x), acc.y = fmaf(w[i], v.y, acc.y);
        acc.z = fmaf(w[i], v.z, acc.z), acc.w = fmaf(w[i], v.w, acc.w);
    };
#pragma unroll
    for (int k = 0; k < kEarly; ++k)
        if (first + k * kStep < S) add(first + k * kStep, early[k]);
#pragma unroll 8
    for (int i = first + kEarly * kStep; i < S; i += kStep) add(i, value(i));
    if constexpr (kOneHead) {
        if (quarter > 0) acc_s[quarter - 1][threadIdx.x & 63] = acc;
        __syncthreads();
        if (quarter > 0) return;
#pragma unroll
        for (int q = 0; q < 7; ++q) {
            const float4 v = acc_s[q][threadIdx.x & 63];
            acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
        }
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y), hi = __floats2bfloat162_rn(acc.z, acc.w);
    *reinterpret_cast<uint2*>(p.out + (row * kMlaHeads + h) * kMlaDv + 4 * d4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

template <bool kOneHead>
__global__ void __launch_bounds__(512) mla_merge_kernel(const MlaMergeParams p) {
    __shared__ Weights<kOneHead> wgt;
    __shared__ Sums<kOneHead> acc;
    pdl_wait_prior_grid();
    pdl_allow_next_grid();
    if (int(blockIdx.y) < p.rows) merge_row<kOneHead, false, false>(p, blockIdx.y, false, wgt, acc);
}

// Of the tree decode's kernels on clusters.  Of one of them the dense kernel may have done some requests again, with a
// plan and partials of its own: a copy of the code for each (one with its pointers in registers took 64 of them for
// 40, and so two CTAs an SM for three).
template <bool kOneHead>
__global__ void __launch_bounds__(512, 3) mla_tree_merge_kernel(const MlaMergeParams p) {
    __shared__ Weights<kOneHead> wgt;
    __shared__ Sums<kOneHead> acc;
    pdl_wait_prior_grid();
    pdl_allow_next_grid();
    const bool again = p.again && p.again[kAgainWords] != 0;
    if (int(blockIdx.y) < p.rows) merge_row<kOneHead, true, false>(p, blockIdx.y, again, wgt, acc);
    if (!again) return;
    __syncthreads();  // (the weights and sums of the row before)
    if (int(blockIdx.y) < p.rows_again) merge_row<kOneHead, false, true>(p, blockIdx.y, true, wgt, acc);
}

}  // namespace

cudaError_t launch_mla_merge(const MlaMergeParams& p, cudaStream_t stream) {
    const int rows = p.again && p.rows_again > p.rows ? p.rows_again : p.rows;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.one_head ? kMlaHeads * 2 : kMlaHeads / 4, unsigned(rows));
    cfg.blockDim = dim3(512);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.tiled)
        return p.one_head ? cudaLaunchKernelEx(&cfg, mla_tree_merge_kernel<true>, p)
                          : cudaLaunchKernelEx(&cfg, mla_tree_merge_kernel<false>, p);
    return p.one_head ? cudaLaunchKernelEx(&cfg, mla_merge_kernel<true>, p)
                      : cudaLaunchKernelEx(&cfg, mla_merge_kernel<false>, p);
}

}  // namespace dsa
