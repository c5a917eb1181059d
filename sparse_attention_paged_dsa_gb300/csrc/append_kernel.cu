// append_kernel.cu -- new entries into the paged caches at their slots: RMS norm of
// the latent part, rotation of the rotary part, RMS norm and 8-bit quantisation of
// the index key.  One pass, one launch.
//
//     c = x[0:512] * weight / sqrt(mean(x[0:512]^2) + eps)           (without a weight: x)
//     r[2j], r[2j + 1] = a cos - b sin, a sin + b cos                 (a, b = x[512 + 2j], x[513 + 2j])
//     y = k * key_weight / sqrt(mean(k^2) + eps),  scale = max|y| / 448,  code = e4m3(u * 448 / max|u|)
//
// with u = k * key_weight: the codes do not depend on the norm, and from u, with the quotient in two parts, they are
// those of the 8-bit RMS norm (rmsnorm_kernel.cu) bit for bit.  (y * (448 / max|y|) by one approximate quotient moved
// half as many more codes to a neighbour.)
//
// A warp has a row at a time: 8-element chunks lane and lane + 32 of the latent part
// (16-byte accesses, whole 512-byte lines of the warp), one pair of the rotary dims and
// of the key a lane.  Both sums of squares and the key's maximum are one set of
// butterflies over the warp, side by side: the norm does not change which product of key
// and weight is largest.  fp32 throughout, one rounding per output.  A row's place is
// fetched two rows ahead, its data (and its row of the rotation's table) one.  Rows whose squares leave fp32's range are
// left for the end of the kernel: with their code called from the loop 262144 rows took 150 us.
//
// What bounds it: HBM and the rows' places.  262144 rows, norms, rotation, fp8 keys: 117 us in
// a loop of calls, 123 after other writes to all of L2 (6200 and 5900 GB/s, 0.91 and 0.87 of
// the measured copy rate; 119 for 123 with the slots in order; the latents alone 101, a copy
// of them 95), at 324 instructions a row (61 % of issue slots).  At 400 it was bound by them
// (132 us, 71 %); the sums one after another took 136; 24 warps an SM, with the weights in
// registers, 142; five CTAs an SM spill (181).  Few rows: launch latency, 2.5 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "indexer_kernels.h"
#include "sm103_ptx.cuh"

namespace dsa {
namespace {

constexpr int kWarpsA = 8;
constexpr int kCtasA = 4;  // per SM, by their registers
constexpr float kE4m3Max = 448.0f;

__device__ __forceinline__ float2 widen(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t narrow(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// The quotient 448 / most in two parts, q + lo.
__device__ __forceinline__ float2 code_quotient(float most) {
    const float q = __fdividef(kE4m3Max, most);
    return make_float2(q, fmaf(-q, most, kE4m3Max) * (q * (1.f / kE4m3Max)));
}
// A row whose sum of squares lies past fp32's range, or below what fp32 holds of it where eps does not cover that.
constexpr float kSumMost = 1e37f, kSumLeast = 1e-30f;
__device__ __forceinline__ bool far_sum(float sum, float eps) {
    return !(sum <= kSumMost) || (sum < kSumLeast && eps < kSumLeast);
}
// Factors `first` and `second` of the norm's reciprocal for such a row, from its squares moved by a power of two: x *
// first * second leaves the range nowhere.
struct FarNorm {
    float by, first, second;
    __device__ __forceinline__ explicit FarNorm(float sum)
        : by(sum < 1.f ? 0x1p100f : 0x1p-70f), first(1.f), second(1.f) {}
    __device__ __forceinline__ float square(float x) const { return x * by * (x * by); }
    __device__ __forceinline__ void settle(float sum, float over_n, float eps) {
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = rsqrtf(sum * over_n + eps * by * by);
        first = by < 1.f ? inv * by : by;
        second = by < 1.f ? 1.f : inv;
    }
    __device__ __forceinline__ float of(float x) const { return x * first * second; }
};
struct Place {
    int64_t slot;
    int pos;
};
struct Row {
    uint4 c[2];     // latent chunks
    uint32_t r, k;  // rotary pair, key pair
    float cs, sn;
};

// The codes and the scale of a key: y, two elements a lane, with top = max|y|, of which u with most = max|u| is a multiple.
__device__ __forceinline__ void store_codes(const AppendParams& p, int64_t slot, int lane, float2 y, float2 u, float top,
                                            float most) {
    float scale = top / kE4m3Max;
    float2 q;
    if (top > 0x1p-100f && top < 0x1p100f && most > 1e-30f && most < 1e30f) {
        const float2 by = code_quotient(most);
        q = fma_f32x2(u, make_float2(by.x, by.x), mul_f32x2(u, make_float2(by.y, by.y)));
    } else {
        if (!(scale > 0.f) || scale > 3.0e38f) scale = 1.f;
        q = make_float2(y.x / scale, y.y / scale);
    }
    uint16_t code;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(code) : "f"(q.y), "f"(q.x));
    *reinterpret_cast<uint16_t*>(p.key_codes + slot * kHeadDim + 2 * lane) = code;
    if (lane == 0) p.key_scales[slot] = scale;
}

// kKeys: 0 none, 1 bf16, 2 fp8.
template <bool kLatent, int kKeys>
__global__ void __launch_bounds__(kWarpsA * 32, kCtasA) append_kernel(const AppendParams p) {
    const int lane = threadIdx.x & 31;
    const uint32_t warp = blockIdx.x * kWarpsA + (threadIdx.x >> 5), warps = gridDim.x * kWarpsA;
    const uint32_t rows = uint32_t(p.rows);  // (below 2^31, and two rounds of warps more below 2^32)
    __shared__ __align__(16) float wc[kMlaDv];
    __shared__ __align__(16) float wk[kHeadDim];
    pdl_wait_prior_grid();
    pdl_allow_next_grid();

    const bool norm = kLatent && p.latent_weight, rotate = kLatent && p.cos_sin, key_norm = kKeys > 0 && p.key_weight;
    const auto place = [&](uint32_t i) {
        Place at = {-1, 0};
        if (i < rows) {
            at.slot = __ldg(p.slots + i);
            if (rotate) at.pos = __ldg(p.positions + i);
        }
        return at;
    };
    const auto in_table = [&](int pos) { return pos >= 0 && int64_t(pos) < p.cos_rows; };
    // Where the next row to load starts, for this lane.
    const uint8_t* x = p.latent + int64_t(warp) * p.latent_stride * 2 + 16 * lane;
    const uint8_t* key = p.keys + int64_t(warp) * p.key_stride * 2 + 4 * lane;
    const int64_t x_step = int64_t(warps) * p.latent_stride * 2, key_step = int64_t(warps) * p.key_stride * 2;
    const auto load = [&](const Place& at) {
        Row row;
        row.cs = 1.f, row.sn = 0.f;
        if (at.slot != -1) {
            if (kLatent) {
                row.c[0] = __ldcs(reinterpret_cast<const uint4*>(x));
                row.c[1] = __ldcs(reinterpret_cast<const uint4*>(x + 512));
                row.r = __ldcs(reinterpret_cast<const uint32_t*>(x + kMlaDv * 2 - 12 * lane));
                if (rotate && in_table(at.pos)) {
                    const float* t = p.cos_sin + int64_t(at.pos) * 64 + lane;
                    row.cs = __ldg(t);
                    row.sn = __ldg(t + 32);
                }
            }
            if (kKeys) row.k = __ldcs(reinterpret_cast<const uint32_t*>(key));
        }
        if (kLatent) x += x_step;
        if (kKeys) key += key_step;
        return row;
    };
    const auto weight_at = [&](const void* w, int fp32, int i) {
        return fp32 ? __ldg(static_cast<const float*>(w) + i)
                    : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(w) + i));
    };
    Place at = place(warp), next = place(warp + warps);
    if (norm)
        for (int i = threadIdx.x; i < kMlaDv; i += kWarpsA * 32)
            wc[i] = weight_at(p.latent_weight, p.latent_weight_fp32, i);
    if (key_norm)
        for (int i = threadIdx.x; i < kHeadDim; i += kWarpsA * 32)
            wk[i] = weight_at(p.key_weight, p.key_weight_fp32, i);
    __syncthreads();

    // A row's place is fetched two rows ahead, its data (and its row of the table) one.
    const int64_t slots = p.num_pages * kPageEntries;
    Row row = load(at);
    bool late = false;  // rows left for the end: far_sum
    for (uint32_t i = warp; i < rows; i += warps) {
        const Row now = row;
        const Place to = at;
        at = next;
        next = place(i + 2 * warps);
        row = load(at);
        if (to.slot == -1) continue;
        const bool bad_slot = uint64_t(to.slot) >= uint64_t(slots), bad_pos = rotate && !in_table(to.pos);
        if (bad_slot || bad_pos) {
            if (lane == 0) atomicOr(p.err, (bad_slot ? kErrBadPage : 0u) | (bad_pos ? kErrBadRange : 0u));
            continue;
        }
        uint4 c[2] = {now.c[0], now.c[1]};
        uint32_t* const u = reinterpret_cast<uint32_t*>(c);
        // What the row needs of the whole warp, three butterflies side by side: both sums of squares, and the
        // largest key times its weight (the norm is the same for all of them).
        float2 sums = make_float2(0.f, 0.f), y = make_float2(0.f, 0.f);  // of the entry, of the key
        float top = 0.f;
        if (norm) {
            float2 ss = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 v = widen(u[j]);
                ss = fma_f32x2(v, v, ss);
            }
            sums.x = ss.x + ss.y;
        }
        if (kKeys) {
            y = widen(now.k);
            if (key_norm) {
                sums.y = fmaf(y.x, y.x, y.y * y.y);
                y = mul_f32x2(y, *reinterpret_cast<const float2*>(wk + 2 * lane));
            }
            if (kKeys == 2) top = fmaxf(fabsf(y.x), fabsf(y.y));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            float2 other = make_float2(0.f, 0.f);
            if (kLatent) other.x = __shfl_xor_sync(0xffffffffu, sums.x, o);
            if (kKeys) other.y = __shfl_xor_sync(0xffffffffu, sums.y, o);
            if (kKeys == 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            sums = add_f32x2(sums, other);
        }
        if ((norm && far_sum(sums.x, p.eps)) || (key_norm && far_sum(sums.y, p.eps))) {
            late = true;
            continue;
        }
        if (kLatent) {
            if (norm) {
                const float inv = rsqrtf(sums.x * (1.f / kMlaDv) + p.eps);
                const float2 by = make_float2(inv, inv);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float4 w = *reinterpret_cast<const float4*>(wc + (j >> 2) * 256 + lane * 8 + 2 * (j & 3));
                    const float2 a = mul_f32x2(mul_f32x2(widen(u[j]), make_float2(w.x, w.y)), by);
                    const float2 b = mul_f32x2(mul_f32x2(widen(u[j + 1]), make_float2(w.z, w.w)), by);
                    u[j] = narrow(a.x, a.y);
                    u[j + 1] = narrow(b.x, b.y);
                }
            }
            uint32_t r = now.r;
            if (rotate) {
                const float2 v = widen(r);
                r = narrow(v.x * now.cs - v.y * now.sn, v.x * now.sn + v.y * now.cs);
            }
            uint8_t* out = p.kv_cache + to.slot * (kMlaDim * 2) + 16 * lane;
            *reinterpret_cast<uint4*>(out) = c[0];
            *reinterpret_cast<uint4*>(out + 512) = c[1];
            *reinterpret_cast<uint32_t*>(out + kMlaDv * 2 - 12 * lane) = r;
        }
        if (kKeys) {
            const float2 u = y;  // before the norm
            const float most = top;
            if (key_norm) {
                const float inv = rsqrtf(sums.y * (1.f / kHeadDim) + p.eps);
                y = mul_f32x2(y, make_float2(inv, inv));
                top *= inv;
            }
            if (kKeys == 1) {
                *reinterpret_cast<uint32_t*>(p.key_pool + to.slot * (kHeadDim * 2) + 4 * lane) =
                    key_norm ? narrow(y.x, y.y) : now.k;
            } else {
                store_codes(p, to.slot, lane, y, u, top, most);
            }
        }
    }
    // Rows left for the end (rare), one after another: the whole row, whichever of its norms is far.
    if (!late) return;
#pragma unroll 1
    for (uint32_t i = warp; i < rows; i += warps) {
        const Place to = place(i);
        if (to.slot == -1 || uint64_t(to.slot) >= uint64_t(slots) || (rotate && !in_table(to.pos))) continue;
        x = p.latent + int64_t(i) * p.latent_stride * 2 + 16 * lane;
        key = p.keys + int64_t(i) * p.key_stride * 2 + 4 * lane;
        const Row now = load(to);
        const uint4 c[2] = {now.c[0], now.c[1]};
        const float2 k = widen(now.k);
        // The sums as above, in the same order: the same rows are far.
        float2 sums = make_float2(0.f, 0.f);
        const auto word = [&](int j) {
            const uint4& w = c[j >> 2];
            return (j & 3) == 0 ? w.x : (j & 3) == 1 ? w.y : (j & 3) == 2 ? w.z : w.w;
        };
        const auto part = [&](int j) { return widen(word(j)); };
        if (norm) {
            float2 ss = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fma_f32x2(part(j), part(j), ss);
            sums.x = ss.x + ss.y;
        }
        if (key_norm) sums.y = fmaf(k.x, k.x, k.y * k.y);
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1)
            sums = add_f32x2(sums, make_float2(__shfl_xor_sync(0xffffffffu, sums.x, o), __shfl_xor_sync(0xffffffffu, sums.y, o)));
        const bool far_c = norm && far_sum(sums.x, p.eps), far_k = key_norm && far_sum(sums.y, p.eps);
        if (!far_c && !far_k) continue;
        if (kLatent) {
            FarNorm f(sums.x);
            if (far_c) {
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += f.square(part(j).x) + f.square(part(j).y);
                f.settle(sum, 1.f / kMlaDv, p.eps);
            } else if (norm) {
                f.first = rsqrtf(sums.x * (1.f / kMlaDv) + p.eps);
            }
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float* by = wc + (j >> 2) * 256 + lane * 8 + 2 * (j & 3);
                w[j] = norm ? narrow(f.of(part(j).x) * by[0], f.of(part(j).y) * by[1]) : word(j);
            }
            uint32_t r = now.r;
            if (rotate) {
                const float2 v = widen(r);
                r = narrow(v.x * now.cs - v.y * now.sn, v.x * now.sn + v.y * now.cs);
            }
            uint8_t* out = p.kv_cache + to.slot * (kMlaDim * 2) + 16 * lane;
            *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(out + 512) = make_uint4(w[4], w[5], w[6], w[7]);
            *reinterpret_cast<uint32_t*>(out + kMlaDv * 2 - 12 * lane) = r;
        }
        if (kKeys) {
            FarNorm f(sums.y);
            if (far_k)
                f.settle(f.square(k.x) + f.square(k.y), 1.f / kHeadDim, p.eps);
            else if (key_norm)
                f.first = rsqrtf(sums.y * (1.f / kHeadDim) + p.eps);
            const float2 y = key_norm ? make_float2(f.of(k.x) * wk[2 * lane], f.of(k.y) * wk[2 * lane + 1]) : k;
            if (kKeys == 1) {
                *reinterpret_cast<uint32_t*>(p.key_pool + to.slot * (kHeadDim * 2) + 4 * lane) =
                    key_norm ? narrow(y.x, y.y) : now.k;
            } else {
                float top = fmaxf(fabsf(y.x), fabsf(y.y));
#pragma unroll 1
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                store_codes(p, to.slot, lane, y, y, top, top);
            }
        }
    }
}

}  // namespace

namespace {

template <bool kLatent, int kKeys>
cudaError_t launch(const AppendParams& p, int sms, cudaStream_t stream) {
    const int64_t ctas = (p.rows + kWarpsA - 1) / kWarpsA, most = int64_t(sms) * kCtasA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(ctas < most ? ctas : most));
    cfg.blockDim = dim3(kWarpsA * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, append_kernel<kLatent, kKeys>, p);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, int sms, cudaStream_t stream) {
    const int keys = p.keys ? (p.key_pool ? 1 : 2) : 0;
    if (p.latent)
        return keys == 0 ? launch<true, 0>(p, sms, stream)
                         : (keys == 1 ? launch<true, 1>(p, sms, stream) : launch<true, 2>(p, sms, stream));
    return keys == 1 ? launch<false, 1>(p, sms, stream) : launch<false, 2>(p, sms, stream);
}

}  // namespace dsa
