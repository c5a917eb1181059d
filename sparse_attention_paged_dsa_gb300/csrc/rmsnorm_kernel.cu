// rmsnorm_kernel.cu -- residual addition and RMS norm of bf16 rows, with a bf16
// output, an e4m3 output with fp32 scales, or both.
//
//     h = x + residual,   u = h * weight,   y = u / sqrt(mean(h^2) + eps)
//     residual_out = bf16(h),  out = bf16(y)
//     scale_G = max_G |y| / 448,  code = e4m3(u * 448 / max_G |u|)   over groups G of a row
//
// h stays in fp32 registers from its one load to the stores (the norm is that of
// the unrounded sum; each output is rounded once), so a row is read and written
// once: HBM-bound for many rows, launch latency for few.  The codes do not depend
// on the row's norm, so they are made while its sum is under way, and from fewer
// roundings than y / scale would take.
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
// a residual the e4m3 output is bound by its instructions (63 us, 0.83; one unit a
// thread, and the codes after the norm: 73; 131072 x 512: 36 us, 0.82, from 46).  Rows
// off 16-byte boundaries are, too: 16384 x 7001, residual, e4m3 out: 231 us, 0.51, 750
// instructions a unit and warp for 300, the ALU pipe at 71 % and DRAM at 39.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>

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

// out[i] = in[i + by] for by in [0, 2 kMost), a power of two at a time (registers have no run-time index).
template <int kMost, int kIn>
__device__ __forceinline__ void shift_words(uint32_t (&w)[kIn], int by) {
#pragma unroll
    for (int o = kMost; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < kIn; ++i) w[i] = (by & o) ? (i + o < kIn ? w[i + o] : 0u) : w[i];
}

// A row's part of the arrays, moved by its T threads.  kAlign: the boundary, in bytes, that every unit of
// every array starts on.  32: one access a unit; 16: two (d a multiple of 8).  2: 16-byte accesses on
// their own boundaries all the same, a unit being shifted out of (into) the three that it lies in; what
// two threads share is put together by a shuffle, and elements at the ends of a warp's part move one by
// one (16384 x 7001 element by element, through shared memory: 520 us).
template <int kNV, bool kCtaRow, int kAlign>
struct RowIo {
    int T, t, d, units;  // units: 0 for threads past the last row

    __device__ __forceinline__ int unit(int j) const { return j * T + t; }
    // Where the 8-element half `f` of this thread's unit j starts.  With 16-byte accesses four neighbouring
    // threads share their units' halves, so that each access, the codes' 8 bytes too, is of whole sectors.
    __device__ __forceinline__ int half_at(int j, int f) const {
        const int v = unit(j);
        return kAlign == 16 ? ((v >> 2) * 8 + (v & 3) + 4 * f) * 8 : v * kUnit + 8 * f;
    }
    // The bf16 pairs of this thread's units; elements past the row read as 0.
    __device__ __forceinline__ void load(uint32_t (&v)[kNV][kPairs], const uint16_t* p) const {
#pragma unroll
        for (int j = 0; j < kNV; ++j) {
            uint32_t (&u)[kPairs] = v[j];
            if constexpr (kAlign == 2) {
                // Only 16-byte pieces that hold an element of the row are read.
                const uintptr_t at = reinterpret_cast<uintptr_t>(p + unit(j) * kUnit);
                const uintptr_t end = unit(j) < units ? reinterpret_cast<uintptr_t>(p + d) : 0;
                const int m = int(at & 15);
                uint32_t w[12];
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    uint4 a = make_uint4(0, 0, 0, 0);
                    if (at - m + 16 * i < end && (i < 2 || m > 0)) a = *reinterpret_cast<const uint4*>(at - m + 16 * i);
                    w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
                }
                shift_words<2>(w, m >> 2);
                const int n = d - unit(j) * kUnit;
#pragma unroll
                for (int i = 0; i < kPairs; ++i) u[i] = __funnelshift_r(w[i], w[i + 1], 8 * (m & 3));
                if (n < kUnit)
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) u[i] = n > 2 * i + 1 ? u[i] : n > 2 * i ? u[i] & 0xFFFFu : 0u;
            } else if constexpr (kAlign == 32) {
#pragma unroll
                for (int i = 0; i < kPairs; ++i) u[i] = 0;
                if (unit(j) < units) ld_global_v8(u, p + unit(j) * kUnit);
            } else {
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    uint4 a = make_uint4(0, 0, 0, 0);
                    if (units && half_at(j, f) < d) a = *reinterpret_cast<const uint4*>(p + half_at(j, f));
                    u[4 * f] = a.x, u[4 * f + 1] = a.y, u[4 * f + 2] = a.z, u[4 * f + 3] = a.w;
                }
            }
        }
    }
    // kAlign 2: the elements of a unit (kWords words of them, of type E), to p + unit(j) * kUnit.  16-byte
    // pieces that this thread and the one before share are written here.
    template <typename E, int kWords>
    __device__ __forceinline__ void store_shifted(E* p, int j, const uint32_t (&own)[kWords]) const {
        constexpr int kBytes = 4 * kWords, kPieces = kBytes / 16 + 1;
        const uintptr_t at = reinterpret_cast<uintptr_t>(p + unit(j) * kUnit);
        const int m = int(at & 15), lane = threadIdx.x & 31;
        uint32_t w[kWords + 8];  // the 16 bytes before the unit, the unit, and nothing
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(0xffffffffu, own[kWords - 4 + i], 1);
#pragma unroll
        for (int i = 0; i < kWords + 4; ++i) w[4 + i] = i < kWords ? own[i] : 0u;
        // The first piece starts m bytes before the unit.
        shift_words<4>(w, (16 - m) >> 2);
#pragma unroll
        for (int i = 0; i < kWords + 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * ((16 - m) & 3));
        const bool before = lane > 0 && t > 0, after = lane < 31 && t + 1 < T && unit(j) + 1 < units;
        const int n = min(d - unit(j) * kUnit, kUnit) * int(sizeof(E));
        const int from = before ? 0 : m, to = unit(j) < units ? (after ? kBytes : m + n) : 0;  // of the pieces
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            if (from <= 16 * i && to >= 16 * i + 16) {
                *reinterpret_cast<uint4*>(at - m + 16 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            } else if (from < 16 * i + 16 && to > 16 * i) {
#pragma unroll
                for (int e = 0; e < 16; e += int(sizeof(E)))
                    if (16 * i + e >= from && 16 * i + e < to)
                        *reinterpret_cast<E*>(at - m + 16 * i + e) = E(w[4 * i + e / 4] >> (8 * (e & 3)));
            }
        }
    }
    // bf16(v), or (kScaled) bf16(v * by).
    template <bool kScaled>
    __device__ __forceinline__ void store(uint16_t* p, const float2 (&v)[kNV][kPairs], float2 by = {}) const {
#pragma unroll
        for (int j = 0; j < kNV; ++j) {
            uint32_t u[kPairs];
#pragma unroll
            for (int i = 0; i < kPairs; ++i) u[i] = pack_bf16(kScaled ? mul_f32x2(v[j][i], by) : v[j][i]);
            if constexpr (kAlign == 2) {
                store_shifted(p, j, u);
            } else if constexpr (kAlign == 32) {
                if (unit(j) < units) st_global_v8(p + unit(j) * kUnit, u);
            } else {
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    if (units && half_at(j, f) < d)
                        *reinterpret_cast<uint4*>(p + half_at(j, f)) =
                            make_uint4(u[4 * f], u[4 * f + 1], u[4 * f + 2], u[4 * f + 3]);
            }
        }
    }
    __device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&pk)[kNV][4]) const {
#pragma unroll
        for (int j = 0; j < kNV; ++j) {
            if constexpr (kAlign == 2) {
                store_shifted(p, j, pk[j]);
            } else if constexpr (kAlign == 16) {
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    if (units && half_at(j, f) < d)
                        *reinterpret_cast<uint2*>(p + half_at(j, f)) = make_uint2(pk[j][2 * f], pk[j][2 * f + 1]);
            } else if (unit(j) < units) {
                *reinterpret_cast<uint4*>(p + unit(j) * kUnit) = make_uint4(pk[j][0], pk[j][1], pk[j][2], pk[j][3]);
            }
        }
    }
    __device__ __forceinline__ void load_weight_fp32(float2 (&v)[kNV][kPairs], const float* w) const {
        const bool whole = kAlign != 2 || (reinterpret_cast<uintptr_t>(w) & 15) == 0;
#pragma unroll
        for (int j = 0; j < kNV; ++j) {
#pragma unroll
            for (int i = 0; i < kPairs; i += 2) {
                const int e = half_at(j, i >> 2) + 2 * (i & 3);
                const int n = units ? d - e : 0;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                if (whole && n > 3) {
                    a = __ldg(reinterpret_cast<const float4*>(w + e));
                } else if (kAlign == 2) {
                    if (n > 0) a.x = w[e];
                    if (n > 1) a.y = w[e + 1];
                    if (n > 2) a.z = w[e + 2];
                    if (n > 3) a.w = w[e + 3];
                }
                v[j][i] = make_float2(a.x, a.y), v[j][i + 1] = make_float2(a.z, a.w);
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

// Fetch the whole 16-byte pieces of n elements into L2.
__device__ __forceinline__ void l2_prefetch(const uint16_t* p, int n) {
    const uintptr_t from = (reinterpret_cast<uintptr_t>(p) + 15) & ~uintptr_t(15);
    const uintptr_t to = reinterpret_cast<uintptr_t>(p + n) & ~uintptr_t(15);
    if (to > from)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(uint32_t(to - from)) : "memory");
}

// CTAs per SM that the registers have to allow: 40 a thread with one unit (with 56, and fewer CTAs, 131072
// x 512 took 46 us, now 42), 64 with two; more for shifting.
template <int kNV, int kMaxT, int kAlign>
constexpr int kResidentOf = kMaxT == 1024 ? 1 : (kMaxT == 512 ? 3 : kNV == 1 ? 6 : 4) * (kAlign == 2 ? 2 : 3) / 3;

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
// A reduction over a row's T threads, which are part of a warp or (kCtaRow) the whole CTA, in two halves
// with a barrier between them.
template <bool kMax, bool kCtaRow>
__device__ __forceinline__ float row_begin(float x, int T, float* scratch) {
    if constexpr (!kCtaRow) return part_reduce<kMax>(x, T);
    x = lanes_reduce<kMax, 32>(x);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
    return x;
}
template <bool kMax, bool kCtaRow>
__device__ __forceinline__ float row_end(float x, int T, const float* scratch) {
    if constexpr (!kCtaRow) return x;
    const int lane = threadIdx.x & 31;
    return lanes_reduce<kMax, 32>(lane < (T >> 5) ? scratch[lane] : 0.f);
}

// Largest magnitude of a unit; units past the row hold zeros.
__device__ __forceinline__ float unit_max(const float2 (&u)[kPairs]) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < kPairs; i += 2) a = max_abs3(a, u[i]), b = max_abs3(b, u[i + 1]);
    return fmaxf(a, b);
}
// Four elements to e4m3 (to nearest even, held to 448, NaN to NaN), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3_x4(float2 a, float2 b) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
// The codes of a unit's elements, each passed through f first.
template <typename F>
__device__ __forceinline__ void pack_e4m3(uint32_t (&pk)[4], const float2 (&u)[kPairs], F&& f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) pk[i] = e4m3_x4(f(u[2 * i]), f(u[2 * i + 1]));
}
// The codes of v * by * (q + lo), out of line.
__device__ __noinline__ uint32_t e4m3_x4_moved(float2 a, float2 b, float by, float q, float lo) {
    const auto f = [&](float v) { return v *= by, fmaf(v, q, v * lo); };
    return e4m3_x4(make_float2(f(a.x), f(a.y)), make_float2(f(b.x), f(b.y)));
}
// The codes of a unit whose group's largest magnitude is amax: u * 448 / amax, with the quotient in two
// parts, so that the result is off by little more than its last rounding (a one-part quotient moves half
// as many more codes to a neighbour: they lie where u is just between two).  kTight: groups at the ends of
// fp32's range go out of line, where the registers are short (in line, 65536 x 1000 without a residual
// takes 40.5 us, not 38.2, and 8192 x 32001 537, not 520; but 16384 x 7168 out of line 62.4, not 61.6).
template <bool kTight>
__device__ __forceinline__ void codes_of(uint32_t (&pk)[4], const float2 (&u)[kPairs], float amax) {
    float q, lo;
    const auto quotient = [&](float most) {
        q = __fdividef(kE4m3Max, most);
        lo = fmaf(-q, most, kE4m3Max) * (q * (1.f / kE4m3Max));
    };
    const auto times = [&](float2 v) {
        return fma_f32x2(v, make_float2(q, q), mul_f32x2(v, make_float2(lo, lo)));
    };
    if (amax > 1e-30f && amax < 1e30f) {
        quotient(amax);
        pack_e4m3(pk, u, times);
    } else if (!(amax > 0.f)) {  // zeros (a row's last warp may hold nothing else) and NaN
        pack_e4m3(pk, u, [](float2 v) { return v; });
    } else {  // a quotient that would leave fp32's range: moved by 2^64, which is exact where it counts
        const float by = amax < 1.f ? 0x1p64f : 0x1p-64f;
        quotient(amax * by);
        if constexpr (kTight) {
#pragma unroll
            for (int i = 0; i < 4; ++i) pk[i] = e4m3_x4_moved(u[2 * i], u[2 * i + 1], by, q, lo);
        } else {
            pack_e4m3(pk, u, [&](float2 v) { return times(mul_f32x2(v, make_float2(by, by))); });
        }
    }
}

// kNV units per thread; kCtaRow: one row per CTA, else rows of T <= 32 threads.  kGroupLanes: lanes of a
// quantisation group (4 or 8), 32 for one scale per row, 0 without 8-bit output.
template <int kNV, bool kCtaRow, int kGroupLanes, int kAlign, int kMaxT>
__global__ void __launch_bounds__(kMaxT, kResidentOf<kNV, kMaxT, kAlign>) rmsnorm_kernel(const RmsNormParams p) {
    __shared__ float scratch[2][32];
    const int T = p.row_threads;
    const int t = kCtaRow ? int(threadIdx.x) : int(threadIdx.x) & (T - 1);
    const int64_t row =
        kCtaRow ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * (kCta >> p.log2_threads) + (threadIdx.x >> p.log2_threads);
    const bool live = kCtaRow || row < p.rows;  // every thread takes part in the shuffles
    const RowIo<kNV, kCtaRow, kAlign> io{T, t, p.d, live ? (p.d + kUnit - 1) / kUnit : 0};
    const int64_t at = row * p.d;

    float2 h[kNV][kPairs];
    uint32_t g[kNV][kPairs];
    pdl_wait_prior_grid();
    // The rows of the CTA that takes this one's place are fetched into L2 now: what is in flight no longer
    // ends with the resident CTAs' registers.  (Short rows without codes leave by themselves soon enough:
    // 131072 x 512 44 us with it, 41 without; with codes 36 against 42.  `ahead` counts on the variant's
    // largest CTAs: of smaller ones more are resident, and part of what is fetched is under way already.)
    if ((kCtaRow || kGroupLanes > 0) && threadIdx.x == 0) {
        const int64_t rows = kCtaRow ? 1 : kCta >> p.log2_threads, next = int64_t(blockIdx.x) * rows + p.ahead;
        if (next < p.rows && (kCtaRow || p.x_stride < 2 * p.d)) {
            const int64_t more = (rows < p.rows - next ? rows : p.rows - next) - 1;
            l2_prefetch(static_cast<const uint16_t*>(p.x) + next * p.x_stride, int(more * p.x_stride) + p.d);
            if (p.residual)
                l2_prefetch(static_cast<const uint16_t*>(p.residual) + next * p.d, int(more + 1) * p.d);
        }
    }
    {
        uint32_t x[kNV][kPairs], r[kNV][kPairs];
        io.load(x, static_cast<const uint16_t*>(p.x) + row * p.x_stride);
        if (p.residual) io.load(r, static_cast<const uint16_t*>(p.residual) + at);
        if (kNV == 1 && !p.weight_fp32) io.load(g, static_cast<const uint16_t*>(p.weight));
#pragma unroll
        for (int j = 0; j < kNV; ++j)
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                h[j][i] = unpack_bf16(x[j][i]);
                if (p.residual) h[j][i] = add_f32x2(h[j][i], unpack_bf16(r[j][i]));
            }
    }
    pdl_allow_next_grid();

    float2 sq2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kNV; ++j)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) sq2 = fma_f32x2(h[j][i], h[j][i], sq2);
    float sq = row_begin<false, kCtaRow>(sq2.x + sq2.y, T, scratch[0]);
    if (p.residual_out) io.template store<false>(static_cast<uint16_t*>(p.residual_out) + at, h);

    // u = h * weight from here on: y = u * rstd, and the codes, which are of u / max|u|, need no rstd.
    if (p.weight_fp32) {
        float2 w[kNV][kPairs];
        io.load_weight_fp32(w, static_cast<const float*>(p.weight));
#pragma unroll
        for (int j = 0; j < kNV; ++j)
#pragma unroll
            for (int i = 0; i < kPairs; ++i) h[j][i] = mul_f32x2(h[j][i], w[j][i]);
    } else {
        if (kNV > 1) io.load(g, static_cast<const uint16_t*>(p.weight));  // (registers)
#pragma unroll
        for (int j = 0; j < kNV; ++j)
#pragma unroll
            for (int i = 0; i < kPairs; ++i) h[j][i] = mul_f32x2(h[j][i], unpack_bf16(g[j][i]));
    }
    constexpr bool kRowScale = kGroupLanes == 32, kTight = kAlign == 2 || (kAlign == 16 && !kCtaRow);
    float amax[kNV];
    uint32_t pk[kNV][4];
    if constexpr (kGroupLanes > 0) {
#pragma unroll
        for (int j = 0; j < kNV; ++j) amax[j] = unit_max(h[j]);
        if constexpr (kRowScale) {
#pragma unroll
            for (int j = 1; j < kNV; ++j) amax[0] = fmaxf(amax[0], amax[j]);
            amax[0] = row_begin<true, kCtaRow>(amax[0], T, scratch[1]);
        } else {
#pragma unroll
            for (int j = 0; j < kNV; ++j) {
                if constexpr (kCtaRow)
                    amax[j] = lanes_reduce<true, kGroupLanes>(amax[j]);
                else  // a row shorter than a group lies in its T lanes
                    amax[j] = part_reduce<true>(amax[j], min(T, kGroupLanes));
                codes_of<kTight>(pk[j], h[j], amax[j]);
            }
        }
    }
    if constexpr (kCtaRow) __syncthreads();
    sq = row_end<false, kCtaRow>(sq, T, scratch[0]);
    const float rstd = rsqrtf(fmaf(sq, p.inv_d, p.eps));
    if (p.out) io.template store<true>(static_cast<uint16_t*>(p.out) + at, h, make_float2(rstd, rstd));
    if constexpr (kGroupLanes > 0) {
        if constexpr (kRowScale) {
            amax[0] = row_end<true, kCtaRow>(amax[0], T, scratch[1]);
#pragma unroll
            for (int j = 0; j < kNV; ++j) {
                amax[j] = amax[0];
                codes_of<kTight>(pk[j], h[j], amax[j]);
            }
        }
        const int nscale = kRowScale ? 1 : (p.d + kGroupLanes * kUnit - 1) / (kGroupLanes * kUnit);
#pragma unroll
        for (int j = 0; j < kNV; ++j) {
            float scale = amax[j] * rstd * (1.f / kE4m3Max);
            if (__float_as_uint(scale) - 0x00800000u >= 0x7F000000u) {  // not a positive normal number
                if (amax[j] == 0.f && rstd <= FLT_MAX) {  // zeros: their codes stand
                    scale = 1.f;
                } else {  // an end of fp32's range, or no finite norm
                    const bool over = scale > FLT_MAX;  // y alone may pass fp32's range: these codes stand
                    if (over) scale = amax[j] * (1.f / kE4m3Max) * rstd;
                    const bool one = !(scale > 0.f && scale <= FLT_MAX);
                    if (one) scale = 1.f;
                    if (one || !over) {  // the codes of y / scale itself, whose rounding counts below 2^-126
                        const float by = one ? rstd : rstd * 0x1p64f, inv = one ? 1.f : __fdividef(1.f, scale * 0x1p64f);
                        pack_e4m3(pk[j], h[j], [&](float2 v) {
                            return mul_f32x2(mul_f32x2(v, make_float2(by, by)), make_float2(inv, inv));
                        });
                    }
                }
            }
            const int v = io.unit(j);
            const bool first = kRowScale ? v == 0 : (v & (kGroupLanes - 1)) == 0;
            if (v < io.units && first) p.scales[row * nscale + (kRowScale ? 0 : v / kGroupLanes)] = scale;
        }
        io.store_codes(p.codes + row * p.d, pk);
    }
}

template <int kNV, bool kCtaRow, int kGroupLanes, int kMaxT>
cudaError_t launch_aligned(const RmsNormParams& p, int align, const cudaLaunchConfig_t& cfg) {
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
    p.inv_d = 1.f / float(p.d);
    const bool bare = p.codes && !p.residual;  // little to load for what there is to compute
    // At most one warp per row, two units a thread above 32; with a residual, rows that fill two warps take
    // them (65536 x 1024, e4m3 out: 70 us against 76; 131072 x 640 135 against 89).
    if (units <= (p.residual ? 48 : 64)) {
        const int nv = units > 32 || (bare && units > 8) ? 2 : 1;  // (see below)
        // 16-byte halves are shared by four threads; a group of 128 elements is eight with a unit each
        int T = nv == 2 ? 8 : align == 16 ? 4 : 1;
        while (T * nv < units && T < 32) T *= 2;
        p.row_threads = T;
        p.log2_threads = 31 - __builtin_clz(unsigned(T));
        const unsigned grid = unsigned((p.rows + kCta / T - 1) / (kCta / T));
        p.ahead = sms * (nv == 1 ? kResidentOf<1, kCta, 32> : kResidentOf<2, kCta, 32>) * (kCta / T);
        return nv == 1 ? launch_nv<1, false, kCta>(p, align, grid, kCta, stream)
                       : launch_nv<2, false, kCta>(p, align, grid, kCta, stream);
    }
    // One CTA per row.  Two units a thread where a row does not fit one, and where instructions are the
    // bound, which two share (16384 x 7168 without a residual, e4m3 out: 63 us against 71, 262144 x 256 39
    // against 43; with one, and so more to load, 129 against 123).
    const int nv = units > 1024 || (units <= 512 && bare) ? 2 : 1;
    const unsigned T = unsigned((units + nv - 1) / nv + 31) / 32 * 32, grid = unsigned(p.rows);
    p.row_threads = int(T);
    const auto run = [&](auto kernel_nv, auto max_t) {
        constexpr int kNV = decltype(kernel_nv)::value, kMaxT = decltype(max_t)::value;
        p.ahead = sms * kResidentOf<kNV, kMaxT, 32>;
        return launch_nv<kNV, true, kMaxT>(p, align, grid, T, stream);
    };
    using std::integral_constant;
    if (nv == 2 && T <= kCta) return run(integral_constant<int, 2>{}, integral_constant<int, kCta>{});
    if (nv == 2) return run(integral_constant<int, 2>{}, integral_constant<int, 1024>{});
    if (T <= 512) return run(integral_constant<int, 1>{}, integral_constant<int, 512>{});
    return run(integral_constant<int, 1>{}, integral_constant<int, 1024>{});
}

}  // namespace dsa
