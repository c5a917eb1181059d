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
// A row belongs to T threads; unit v (16 consecutive elements, one 32-byte load)
// belongs to thread v % T, so neighbouring lanes hold neighbouring units and a
// quantisation group of 64 or 128 elements is 4 or 8 neighbouring lanes.
//
// What bounds it.  16384 x 7168, residual, e4m3 out: 123 us, 0.99 of the measured
// copy rate (bf16 out: 140 us, 0.99).  Steps there: 8-element units, reductions over
// run-time lane counts and scalar arithmetic, 35 instructions an element: 242 us;
// 16-element units and packed fp32 pairs: 156; 40 registers, so that three CTAs of
// one unit a thread are resident: 143; the next row fetched into L2: 123.  Without
// a residual the e4m3 output is bound by its instructions (73 us, 0.72).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "indexer_kernels.h"
#include "sm103_ptx.cuh"

namespace dsa {
namespace {

constexpr int kUnit = 16;         // elements per unit
constexpr int kPairs = kUnit / 2;
constexpr int kCta = 256;         // threads of a CTA whose rows have at most one warp each
constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ float2 unpack_bf16(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// A row's rows of the arrays, moved by its T threads.  kAlign: the boundary, in bytes, that every unit of
// every array starts on.  32: one access a unit; 16: two (d a multiple of 8).  2: the row passes through
// shared memory, so that global accesses are of neighbouring elements (unit by unit, 32 lanes touch
// 32 sectors an access: 16384 x 7001 took 891 us, now 520).
template <int kNV, bool kCtaRow, int kAlign>
struct RowIo {
    int T, t, d, units;  // units: 0 for threads past the last row
    uint16_t* stage;     // kAlign 2: T x kNV x 16 elements of shared memory

    __device__ __forceinline__ int unit(int j) const { return j * T + t; }
    // Where the 8-element half `f` of this thread's unit j starts.  With 16-byte accesses two neighbouring
    // threads share their units' halves alternately, so that each access is of whole sectors.
    __device__ __forceinline__ int half_at(int j, int f) const {
        const int v = unit(j);
        return kAlign == 16 ? ((v >> 1) * 4 + (v & 1) + 2 * f) * 8 : v * kUnit + 8 * f;
    }
    __device__ __forceinline__ void sync() const {
        if constexpr (kCtaRow)
            __syncthreads();
        else
            __syncwarp();
    }
    // Elements past the row read as 0.
    __device__ __forceinline__ void load(float2 (&v)[kNV][kPairs], const uint16_t* p) const {
        if constexpr (kAlign == 2) {
#pragma unroll 4
            for (int i = 0; i < kNV * kUnit; ++i) {
                const int e = i * T + t;
                stage[e] = units && e < d ? p[e] : uint16_t(0);
            }
            sync();
        }
#pragma unroll
        for (int j = 0; j < kNV; ++j) {
            uint32_t u[kPairs] = {};
            if constexpr (kAlign == 2) {
                const uint4* q = reinterpret_cast<const uint4*>(stage + unit(j) * kUnit);
                const uint4 a = q[0], b = q[1];
                u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w, u[4] = b.x, u[5] = b.y, u[6] = b.z, u[7] = b.w;
            } else if constexpr (kAlign == 32) {
                if (unit(j) < units) ld_global_v8(u, p + unit(j) * kUnit);
            } else {
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    uint4 a = make_uint4(0, 0, 0, 0);
                    if (units && half_at(j, f) < d) a = *reinterpret_cast<const uint4*>(p + half_at(j, f));
                    u[4 * f] = a.x, u[4 * f + 1] = a.y, u[4 * f + 2] = a.z, u[4 * f + 3] = a.w;
                }
            }
#pragma unroll
            for (int i = 0; i < kPairs; ++i) v[j][i] = unpack_bf16(u[i]);
        }
        if constexpr (kAlign == 2) sync();
    }
    __device__ __forceinline__ void store(uint16_t* p, const float2 (&v)[kNV][kPairs]) const {
#pragma unroll
        for (int j = 0; j < kNV; ++j) {
            uint32_t u[kPairs];
#pragma unroll
            for (int i = 0; i < kPairs; ++i) u[i] = pack_bf16(v[j][i]);
            if constexpr (kAlign == 32) {
                if (unit(j) < units) st_global_v8(p + unit(j) * kUnit, u);
            } else {
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    if (kAlign == 2 || (units && half_at(j, f) < d))
                        *reinterpret_cast<uint4*>((kAlign == 2 ? stage : p) + half_at(j, f)) =
                            make_uint4(u[4 * f], u[4 * f + 1], u[4 * f + 2], u[4 * f + 3]);
            }
        }
        if constexpr (kAlign == 2) {
            sync();
#pragma unroll 4
            for (int i = 0; i < kNV * kUnit; ++i) {
                const int e = i * T + t;
                if (units && e < d) p[e] = stage[e];
            }
            sync();
        }
    }
    __device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&pk)[kNV][4]) const {
        uint8_t* const bytes = reinterpret_cast<uint8_t*>(stage);
#pragma unroll
        for (int j = 0; j < kNV; ++j) {
            if constexpr (kAlign == 16) {
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    if (units && half_at(j, f) < d)
                        *reinterpret_cast<uint2*>(p + half_at(j, f)) = make_uint2(pk[j][2 * f], pk[j][2 * f + 1]);
            } else if (kAlign == 2 || unit(j) < units) {
                *reinterpret_cast<uint4*>((kAlign == 2 ? bytes : p) + unit(j) * kUnit) =
                    make_uint4(pk[j][0], pk[j][1], pk[j][2], pk[j][3]);
            }
        }
        if constexpr (kAlign == 2) {
            sync();
#pragma unroll 4
            for (int i = 0; i < kNV * kUnit; ++i) {
                const int e = i * T + t;
                if (units && e < d) p[e] = bytes[e];
            }
        }
    }
    __device__ __forceinline__ void load_weight_fp32(float2 (&v)[kNV][kPairs], const float* w) const {
#pragma unroll
        for (int j = 0; j < kNV; ++j) {
#pragma unroll
            for (int i = 0; i < kPairs; i += 2) {
                const int e = half_at(j, i >> 2) + 2 * (i & 3);
                const int n = units ? d - e : 0;
                if constexpr (kAlign == 2) {
                    v[j][i] = make_float2(0 < n ? w[e] : 0.f, 1 < n ? w[e + 1] : 0.f);
                    v[j][i + 1] = make_float2(2 < n ? w[e + 2] : 0.f, 3 < n ? w[e + 3] : 0.f);
                } else {
                    const float4 a =
                        0 < n ? __ldg(reinterpret_cast<const float4*>(w + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
                    v[j][i] = make_float2(a.x, a.y), v[j][i + 1] = make_float2(a.z, a.w);
                }
            }
        }
    }
};

// max(m, |v.x|, |v.y|); a NaN loses.
__device__ __forceinline__ float max_abs3(float m, float2 v) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(v.x), "f"(v.y));
    return r;
}

// Fetch `bytes` (a multiple of 16) from a 16-byte aligned address into L2.
__device__ __forceinline__ void l2_prefetch(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// A correctly rounded quotient, kept out of line: only groups at the ends of fp32's range take it.
__device__ __noinline__ float divide(float a, float b) { return a / b; }

constexpr int kResident = 3;  // CTAs of up to 512 threads per SM (40 registers; two at 64 were slower throughout)

// Sum or maximum over each group of kLanes neighbouring lanes.
template <bool kMax, int kLanes>
__device__ __forceinline__ float lanes_reduce(float x) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, o);
        x = kMax ? fmaxf(x, y) : x + y;
    }
    return x;
}
// The same over T lanes (a power of two up to 32).  0 is neutral: the maxima are of |y|.
template <bool kMax>
__device__ __forceinline__ float part_reduce(float x, int T) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        float y = __shfl_xor_sync(0xffffffffu, x, o);
        y = o < T ? y : 0.f;
        x = kMax ? fmaxf(x, y) : x + y;
    }
    return x;
}
// Over a row's T threads: part of a warp, or (kCtaRow) the whole CTA.
template <bool kMax, bool kCtaRow>
__device__ __forceinline__ float row_reduce(float x, int T, float* scratch) {
    if constexpr (!kCtaRow) return part_reduce<kMax>(x, T);
    x = lanes_reduce<kMax, 32>(x);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return lanes_reduce<kMax, 32>(lane < (T >> 5) ? scratch[lane] : 0.f);
}

// The 8-bit output of a row: one scale per group of kGroupLanes lanes (4 or 8), or (32) per row.
template <int kNV, bool kCtaRow, int kGroupLanes, typename Io>
__device__ __forceinline__ void quantise(const RmsNormParams& p, const Io& io, float2 (&h)[kNV][kPairs], int64_t row,
                                         float* scratch) {
    float amax[kNV];
#pragma unroll
    for (int j = 0; j < kNV; ++j) {  // units past the row hold zeros
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int i = 0; i < kPairs; i += 2) a = max_abs3(a, h[j][i]), b = max_abs3(b, h[j][i + 1]);
        amax[j] = fmaxf(a, b);
    }
    if constexpr (kGroupLanes == 32) {
#pragma unroll
        for (int j = 1; j < kNV; ++j) amax[0] = fmaxf(amax[0], amax[j]);
        amax[0] = row_reduce<true, kCtaRow>(amax[0], io.T, scratch);
#pragma unroll
        for (int j = 1; j < kNV; ++j) amax[j] = amax[0];
    } else {
#pragma unroll
        for (int j = 0; j < kNV; ++j) {
            if constexpr (kCtaRow)
                amax[j] = lanes_reduce<true, kGroupLanes>(amax[j]);
            else  // a row shorter than a group lies in its T lanes
                amax[j] = part_reduce<true>(amax[j], min(io.T, kGroupLanes));
        }
    }
    const int nscale = kGroupLanes == 32 ? 1 : (p.d + kGroupLanes * kUnit - 1) / (kGroupLanes * kUnit);
    uint32_t pk[kNV][4];
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
        float scale = amax[j] * (1.f / kE4m3Max);
        if (!(scale > 0.f)) scale = 1.f;  // an all-zero group (or one below fp32's range): codes 0
        if (amax[j] > 1e-30f && amax[j] < 1e30f) {
            const float inv = __fdividef(kE4m3Max, amax[j]);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) h[j][i] = mul_f32x2(h[j][i], make_float2(inv, inv));
        } else {  // 448 / amax or its approximation would leave fp32's range
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                h[j][i] = make_float2(divide(h[j][i].x, scale), divide(h[j][i].y, scale));
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const uint32_t e = __nv_cvt_float2_to_fp8x2(h[j][i], __NV_SATFINITE, __NV_E4M3);
            pk[j][i >> 1] = (i & 1) ? pk[j][i >> 1] | (e << 16) : e;
        }
        const int v = io.unit(j);
        const bool first = kGroupLanes == 32 ? v == 0 : (v & (kGroupLanes - 1)) == 0;
        if (v < io.units && first) p.scales[row * nscale + (kGroupLanes == 32 ? 0 : v / kGroupLanes)] = scale;
    }
    io.store_codes(p.codes + row * p.d, pk);
}

// kNV units per thread; kCtaRow: one row per CTA, else rows of T <= 32 threads.  kGroupLanes: lanes of a
// quantisation group (4 or 8), 32 for one scale per row, 0 without 8-bit output.
template <int kNV, bool kCtaRow, int kGroupLanes, int kAlign, int kMaxT>
__global__ void __launch_bounds__(kMaxT, kMaxT == 512 ? kResident : 1) rmsnorm_kernel(const RmsNormParams p) {
    __shared__ float scratch[2][32];
    const int T = p.row_threads;
    const int t = kCtaRow ? int(threadIdx.x) : int(threadIdx.x) & (T - 1);
    const int64_t row =
        kCtaRow ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * (kCta >> p.log2_threads) + (threadIdx.x >> p.log2_threads);
    const bool live = kCtaRow || row < p.rows;  // every thread takes part in the shuffles
    extern __shared__ uint4 stage_raw[];
    uint16_t* const stage = reinterpret_cast<uint16_t*>(stage_raw) + (int(threadIdx.x) - t) * kNV * kUnit;
    const RowIo<kNV, kCtaRow, kAlign> io{T, t, p.d, live ? (p.d + kUnit - 1) / kUnit : 0, stage};
    const int64_t at = row * p.d;

    float2 h[kNV][kPairs];
    pdl_wait_prior_grid();
    // The row that takes this CTA's place is fetched into L2 now: what is in flight no longer ends with
    // the resident CTAs' registers.
    if (kCtaRow && kAlign >= 16 && threadIdx.x == 0 && row + p.ahead < p.rows) {
        const uint32_t bytes = uint32_t(p.d) * 2u;
        l2_prefetch(static_cast<const uint16_t*>(p.x) + (row + p.ahead) * p.x_stride, bytes);
        if (p.residual) l2_prefetch(static_cast<const uint16_t*>(p.residual) + (row + p.ahead) * p.d, bytes);
    }
    {
        float2 r[kNV][kPairs];
        io.load(h, static_cast<const uint16_t*>(p.x) + row * p.x_stride);
        if (p.residual) {
            io.load(r, static_cast<const uint16_t*>(p.residual) + at);
#pragma unroll
            for (int j = 0; j < kNV; ++j)
#pragma unroll
                for (int i = 0; i < kPairs; ++i) h[j][i] = add_f32x2(h[j][i], r[j][i]);
        }
    }
    pdl_allow_next_grid();

    float2 sq2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kNV; ++j)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) sq2 = fma_f32x2(h[j][i], h[j][i], sq2);
    const float sq = row_reduce<false, kCtaRow>(sq2.x + sq2.y, T, scratch[0]);
    const float rstd = rsqrtf(sq / float(p.d) + p.eps);
    const float2 rstd2 = make_float2(rstd, rstd);

    if (p.residual_out) io.store(static_cast<uint16_t*>(p.residual_out) + at, h);
    {
        float2 g[kNV][kPairs];
        if (p.weight_fp32)
            io.load_weight_fp32(g, static_cast<const float*>(p.weight));
        else
            io.load(g, static_cast<const uint16_t*>(p.weight));
#pragma unroll
        for (int j = 0; j < kNV; ++j)
#pragma unroll
            for (int i = 0; i < kPairs; ++i) h[j][i] = mul_f32x2(mul_f32x2(h[j][i], rstd2), g[j][i]);
    }
    if (p.out) io.store(static_cast<uint16_t*>(p.out) + at, h);
    if constexpr (kGroupLanes > 0) {
        quantise<kNV, kCtaRow, kGroupLanes>(p, io, h, row, scratch[1]);
    }
}
template <int kNV, bool kCtaRow, int kGroupLanes, int kMaxT>
cudaError_t launch_aligned(const RmsNormParams& p, int align, cudaLaunchConfig_t cfg) {
    if (align == 2) {  // the rows' staging; above 48 KB the limit is raised once
        cfg.dynamicSmemBytes = size_t(cfg.blockDim.x) * kNV * kUnit * sizeof(uint16_t);
        if (kNV > 1 && cfg.dynamicSmemBytes > 48 * 1024) {
            static SmemLimitOnce limit;
            int dev = 0;
            cudaError_t e = cudaGetDevice(&dev);
            if (e == cudaSuccess) e = limit.apply(dev, rmsnorm_kernel<kNV, kCtaRow, kGroupLanes, 2, kMaxT>, 65536);
            if (e != cudaSuccess) return e;
        }
    }
    switch (align) {
        case 32: return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<kNV, kCtaRow, kGroupLanes, 32, kMaxT>, p);
        case 16: return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<kNV, kCtaRow, kGroupLanes, 16, kMaxT>, p);
        default: return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<kNV, kCtaRow, kGroupLanes, 2, kMaxT>, p);
    }
}

template <int kNV, bool kCtaRow, int kMaxT>
cudaError_t launch_nv(const RmsNormParams& p, int align, unsigned grid, unsigned threads, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!p.codes) return launch_aligned<kNV, kCtaRow, 0, kMaxT>(p, align, cfg);
    switch (p.group) {
        case 64: return launch_aligned<kNV, kCtaRow, 64 / kUnit, kMaxT>(p, align, cfg);
        case 128: return launch_aligned<kNV, kCtaRow, 128 / kUnit, kMaxT>(p, align, cfg);
        default: return launch_aligned<kNV, kCtaRow, 32, kMaxT>(p, align, cfg);
    }
}

}  // namespace

cudaError_t launch_rmsnorm(RmsNormParams p, int align, int sms, cudaStream_t stream) {
    const int units = (p.d + kUnit - 1) / kUnit;
    if (units <= 64) {  // at most one warp per row, two units a thread above 32
        int T = align == 16 ? 2 : 1;  // 16-byte halves are shared by pairs of threads
        while (T < units && T < 32) T *= 2;
        p.row_threads = T;
        p.log2_threads = 31 - __builtin_clz(unsigned(T));
        const unsigned grid = unsigned((p.rows + kCta / T - 1) / (kCta / T));
        return units <= 32 ? launch_nv<1, false, kCta>(p, align, grid, kCta, stream)
                           : launch_nv<2, false, kCta>(p, align, grid, kCta, stream);
    }
    const int nv = units <= 1024 ? 1 : 2;  // one CTA per row
    const unsigned T = unsigned((units + nv - 1) / nv + 31) / 32 * 32, grid = unsigned(p.rows);
    p.row_threads = int(T);
    p.ahead = sms * (T <= 512 ? kResident : 1);  // the CTAs resident at a time
    if (nv == 2) return launch_nv<2, true, 1024>(p, align, grid, T, stream);
    return T <= 512 ? launch_nv<1, true, 512>(p, align, grid, T, stream)
                    : launch_nv<1, true, 1024>(p, align, grid, T, stream);
}

}  // namespace dsa
