// rmsnorm_kernel.cu -- residual addition and RMS norm of bf16 rows, with a bf16
// output, an e4m3 output with fp32 scales, or both.
//
//     h = x + residual,   y = h / sqrt(mean(h^2) + eps) * weight
//     residual_out = bf16(h),  out = bf16(y)
//     scale_G = max_G |y| / 448,  code = e4m3(y / scale_G)   over groups G of a row
//
// h stays in fp32 registers from its one load to the stores (the norm is that of
// the unrounded sum; each output is rounded once), so a row is read and written
// once: HBM-bound for many rows, launch latency for few.
//
// A row belongs to T threads; vector v (8 consecutive elements, one 16-byte load)
// belongs to thread v % T, so neighbouring lanes hold neighbouring vectors and a
// quantisation group of 64 or 128 elements is 8 or 16 neighbouring lanes.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "indexer_kernels.h"
#include "sm103_ptx.cuh"

namespace dsa {
namespace {

constexpr int kVec = 8;           // elements per vector
constexpr int kCta = 256;         // threads of a CTA whose rows have at most one warp each
constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Eight consecutive bf16 from `p`; the last `kVec - n` read as 0.  Wide: one 16-byte load.
template <bool kWide>
__device__ __forceinline__ void load8(float (&v)[kVec], const __nv_bfloat16* p, int n) {
    if constexpr (kWide) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.f;
    }
}

template <bool kWide>
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[kVec], int n) {
    if constexpr (kWide) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < n) p[i] = __float2bfloat16_rn(v[i]);
    }
}

// A correctly rounded quotient, kept out of line: only groups at the ends of fp32's range take it.
__device__ __noinline__ float divide(float a, float b) { return a / b; }

// Sum or maximum over the `lanes` (a power of two) neighbouring lanes of each group.
template <bool kMax>
__device__ __forceinline__ float lanes_reduce(float x, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, o);
        x = kMax ? fmaxf(x, y) : x + y;
    }
    return x;
}

// The same over the row's T threads (T <= 32: part of a warp; else the whole CTA).
template <bool kMax>
__device__ __forceinline__ float row_reduce(float x, int T, float* scratch) {
    if (T <= 32) return lanes_reduce<kMax>(x, T);
    x = lanes_reduce<kMax>(x, 32);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return lanes_reduce<kMax>(lane < (T >> 5) ? scratch[lane] : 0.f, 32);  // sums and |y| maxima: 0 is neutral
}

// kNV vectors per thread.  kWide: every row of every array starts on a 16-byte
// boundary (codes: 8-byte) and d is a multiple of 8.
template <int kNV, bool kWide>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const RmsNormParams p) {
    __shared__ float scratch[2][32];
    const int T = p.row_threads;
    const int t = T <= 32 ? int(threadIdx.x) & (T - 1) : int(threadIdx.x);
    const int64_t row = T <= 32 ? int64_t(blockIdx.x) * (kCta / T) + int(threadIdx.x) / T : int64_t(blockIdx.x);
    const bool live = row < p.rows;  // every thread takes part in the shuffles
    const int nvec = (p.d + kVec - 1) / kVec;
    const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(p.x) + row * p.x_stride;
    const __nv_bfloat16* res = reinterpret_cast<const __nv_bfloat16*>(p.residual) + row * p.d;

    float h[kNV][kVec];
    pdl_wait_prior_grid();
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
        const int v = j * T + t;
        if (live && v < nvec) {
            load8<kWide>(h[j], x + v * kVec, p.d - v * kVec);
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i) h[j][i] = 0.f;
        }
    }
    if (p.residual) {
#pragma unroll
        for (int j = 0; j < kNV; ++j) {
            const int v = j * T + t;
            if (live && v < nvec) {
                float r[kVec];
                load8<kWide>(r, res + v * kVec, p.d - v * kVec);
#pragma unroll
                for (int i = 0; i < kVec; ++i) h[j][i] += r[i];
            }
        }
    }
    pdl_allow_next_grid();

    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < kNV; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) sq = fmaf(h[j][i], h[j][i], sq);
    sq = row_reduce<false>(sq, T, scratch[0]);
    const float rstd = rsqrtf(sq / float(p.d) + p.eps);

    float row_max = 0.f;
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
        const int v = j * T + t;
        if (!live || v >= nvec) continue;
        const int n = p.d - v * kVec;
        if (p.residual_out) store8<kWide>(reinterpret_cast<__nv_bfloat16*>(p.residual_out) + row * p.d + v * kVec, h[j], n);
        float g[kVec];
        if (p.weight_fp32) {
            const float* w = static_cast<const float*>(p.weight) + v * kVec;
            if constexpr (kWide) {
                const float4 a = __ldg(reinterpret_cast<const float4*>(w)), b = __ldg(reinterpret_cast<const float4*>(w) + 1);
                g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w, g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
            } else {
#pragma unroll
                for (int i = 0; i < kVec; ++i) g[i] = i < n ? w[i] : 0.f;
            }
        } else {
            load8<kWide>(g, static_cast<const __nv_bfloat16*>(p.weight) + v * kVec, n);
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) h[j][i] = h[j][i] * rstd * g[i];
        if (p.out) store8<kWide>(reinterpret_cast<__nv_bfloat16*>(p.out) + row * p.d + v * kVec, h[j], n);
    }
    if (!p.codes) return;

    // 8-bit output: one scale per group of 64 or 128 elements (8 or 16 lanes) or per row.
    if (p.group == 0) {
#pragma unroll
        for (int j = 0; j < kNV; ++j)
#pragma unroll
            for (int i = 0; i < kVec; ++i) row_max = fmaxf(row_max, fabsf(h[j][i]));
        row_max = row_reduce<true>(row_max, T, scratch[1]);
    }
    const int glanes = min(p.group / kVec, T);  // a row shorter than a group lies in its T lanes
    const int nscale = p.group ? (p.d + p.group - 1) / p.group : 1;
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
        const int v = j * T + t;
        float amax = row_max;
        if (p.group) {
            amax = 0.f;  // vectors past the row hold zeros
#pragma unroll
            for (int i = 0; i < kVec; ++i) amax = fmaxf(amax, fabsf(h[j][i]));
            amax = lanes_reduce<true>(amax, glanes);
        }
        if (!live || v >= nvec) continue;
        float scale = amax * (1.f / kE4m3Max);
        if (!(scale > 0.f)) scale = 1.f;  // an all-zero group (or one below fp32's range): codes 0
        uint8_t* codes = p.codes + row * p.d + v * kVec;
        float c[kVec];
        if (amax > 1e-30f && amax < 1e30f) {
            const float inv = __fdividef(kE4m3Max, amax);
#pragma unroll
            for (int i = 0; i < kVec; ++i) c[i] = h[j][i] * inv;
        } else {  // 448 / amax or its approximation would leave fp32's range
#pragma unroll
            for (int i = 0; i < kVec; ++i) c[i] = divide(h[j][i], scale);
        }
        uint32_t pk[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t e = __nv_cvt_float2_to_fp8x2(make_float2(c[2 * i], c[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
            pk[i >> 1] = (i & 1) ? pk[i >> 1] | (e << 16) : e;
        }
        if constexpr (kWide) {
            *reinterpret_cast<uint2*>(codes) = make_uint2(pk[0], pk[1]);
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (v * kVec + i < p.d) codes[i] = uint8_t(pk[i >> 2] >> (8 * (i & 3)));
        }
        const bool first = p.group ? (v * kVec) % p.group == 0 : v == 0;
        if (first) p.scales[row * nscale + (p.group ? (v * kVec) / p.group : 0)] = scale;
    }
}

template <int kNV>
cudaError_t launch_nv(const RmsNormParams& p, bool wide, unsigned grid, unsigned threads, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return wide ? cudaLaunchKernelEx(&cfg, rmsnorm_kernel<kNV, true>, p)
                : cudaLaunchKernelEx(&cfg, rmsnorm_kernel<kNV, false>, p);
}

}  // namespace

cudaError_t launch_rmsnorm(RmsNormParams p, bool wide, int sms, cudaStream_t stream) {
    const int nvec = (p.d + kVec - 1) / kVec;
    int nv;
    if (nvec <= 32) {  // a row in part of a warp
        nv = 1;
        p.row_threads = 1;
        while (p.row_threads < nvec) p.row_threads *= 2;
    } else if (nvec <= 128) {  // one warp per row
        p.row_threads = 32;
        nv = nvec <= 64 ? 2 : 4;
    } else {
        // One CTA per row.  Few rows: as many threads as vectors (one load each, shortest chain);
        // many rows: four vectors per thread (smaller CTAs, more of them resident).
        const int least = p.rows > 4 * int64_t(sms) ? 4 : 1;
        nv = least;
        while ((nvec + nv - 1) / nv > 1024) nv *= 2;
        p.row_threads = ((nvec + nv - 1) / nv + 31) / 32 * 32;
    }
    const int T = p.row_threads;
    const int64_t grid = T <= 32 ? (p.rows + kCta / T - 1) / (kCta / T) : p.rows;
    const unsigned threads = T <= 32 ? kCta : T;
    switch (nv) {
        case 1: return launch_nv<1>(p, wide, unsigned(grid), threads, stream);
        case 2: return launch_nv<2>(p, wide, unsigned(grid), threads, stream);
        default: return launch_nv<4>(p, wide, unsigned(grid), threads, stream);
    }
}

}  // namespace dsa
