// append_kernel.cu -- new entries into the paged caches at their slots: RMS norm of
// the latent part, rotation of the rotary part, RMS norm and 8-bit quantisation of
// the index key.  One pass, one launch.
//
//     c = x[0:512] * weight / sqrt(mean(x[0:512]^2) + eps)           (without a weight: x)
//     r[2j], r[2j + 1] = a cos - b sin, a sin + b cos                 (a, b = x[512 + 2j], x[513 + 2j])
//     y = k * key_weight / sqrt(mean(k^2) + eps),  scale = max|y| / 448,  code = y / scale
//
// A warp has a row at a time: 8-element chunks lane and lane + 32 of the latent part
// (16-byte accesses, whole 512-byte lines of the warp), one pair of the rotary dims and
// of the key a lane.  Both sums of squares and the key's maximum are one set of
// butterflies over the warp, side by side: the norm does not change which product of key
// and weight is largest.  fp32 throughout, one rounding per output.  A row's place is
// fetched two rows ahead, its data (and its row of the rotation's table) one.
//
// What bounds it: HBM and, by half, instructions.  262144 rows, norms, rotation, fp8 keys: 132
// us, 5490 GB/s, 0.81 of the measured copy rate; the latents alone 101 us (a copy of them 95);
// the keys' 4-byte scales and 64-byte rows are written where the slots say.  One after another
// the sums took 136 us; weights in registers 142 (24 warps an SM, now 32); five CTAs an SM
// spill (181).  Few rows: launch latency, 2.5 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "indexer_kernels.h"
#include "sm103_ptx.cuh"

namespace dsa {
namespace {

constexpr int kWarpsA = 8;
constexpr int kCtasA = 4;  // per SM
constexpr float kE4m3Max = 448.0f;

__device__ __forceinline__ float2 widen(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t narrow(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
struct Place {
    int64_t slot;
    int pos;
};
struct Row {
    uint4 c[2];     // latent chunks
    uint32_t r, k;  // rotary pair, key pair
    float cs, sn;
};

__global__ void __launch_bounds__(kWarpsA * 32, kCtasA) append_kernel(const AppendParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t warp = int64_t(blockIdx.x) * kWarpsA + (threadIdx.x >> 5), warps = int64_t(gridDim.x) * kWarpsA;
    __shared__ __align__(16) float wc[kMlaDv];
    __shared__ __align__(16) float wk[kHeadDim];
    pdl_wait_prior_grid();
    pdl_allow_next_grid();

    const auto place = [&](int64_t i) {
        Place at = {-1, 0};
        if (i < p.rows) {
            at.slot = __ldg(p.slots + i);
            if (p.cos_sin) at.pos = __ldg(p.positions + i);
        }
        return at;
    };
    const auto in_table = [&](int pos) { return pos >= 0 && int64_t(pos) < p.cos_rows; };
    const auto load = [&](int64_t i, const Place& at) {
        Row row;
        row.cs = 1.f, row.sn = 0.f;
        if (i >= p.rows || at.slot == -1) return row;
        if (p.latent) {
            const uint8_t* x = p.latent + i * p.latent_stride * 2;
            row.c[0] = __ldcs(reinterpret_cast<const uint4*>(x) + lane);
            row.c[1] = __ldcs(reinterpret_cast<const uint4*>(x) + 32 + lane);
            row.r = __ldcs(reinterpret_cast<const uint32_t*>(x + kMlaDv * 2) + lane);
            if (p.cos_sin && in_table(at.pos)) {
                row.cs = __ldg(p.cos_sin + int64_t(at.pos) * 64 + lane);
                row.sn = __ldg(p.cos_sin + int64_t(at.pos) * 64 + 32 + lane);
            }
        }
        if (p.keys) row.k = __ldcs(reinterpret_cast<const uint32_t*>(p.keys + i * p.key_stride * 2) + lane);
        return row;
    };
    const auto weight_at = [&](const void* w, int fp32, int i) {
        return fp32 ? __ldg(static_cast<const float*>(w) + i)
                    : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(w) + i));
    };
    Place at = place(warp), next = place(warp + warps);
    if (p.latent_weight)
        for (int i = threadIdx.x; i < kMlaDv; i += kWarpsA * 32)
            wc[i] = weight_at(p.latent_weight, p.latent_weight_fp32, i);
    if (p.key_weight)
        for (int i = threadIdx.x; i < kHeadDim; i += kWarpsA * 32)
            wk[i] = weight_at(p.key_weight, p.key_weight_fp32, i);
    __syncthreads();

    // A row's place is fetched two rows ahead, its data (and its row of the table) one.
    Row row = load(warp, at);
    for (int64_t i = warp; i < p.rows; i += warps) {
        const Row now = row;
        const Place to = at;
        at = next;
        next = place(i + 2 * warps);
        row = load(i + warps, at);
        if (to.slot == -1) continue;
        const bool bad_slot = to.slot < -1 || to.slot >= p.num_pages * kPageEntries;
        const bool bad_pos = p.cos_sin && !in_table(to.pos);
        if (bad_slot || bad_pos) {
            if (lane == 0) atomicOr(p.err, (bad_slot ? kErrBadPage : 0u) | (bad_pos ? kErrBadRange : 0u));
            continue;
        }
        uint4 c[2] = {now.c[0], now.c[1]};
        uint32_t* const u = reinterpret_cast<uint32_t*>(c);
        // What the row needs of the whole warp, three butterflies side by side: both sums of squares, and the
        // largest key times its weight (the norm is the same for all of them).
        float ss = 0.f, ks = 0.f, top = 0.f;
        float2 y = make_float2(0.f, 0.f);
        if (p.latent_weight) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 v = widen(u[j]);
                ss = fmaf(v.x, v.x, fmaf(v.y, v.y, ss));
            }
        }
        if (p.keys) {
            y = widen(now.k);
            if (p.key_weight) {
                ks = fmaf(y.x, y.x, y.y * y.y);
                const float2 w = *reinterpret_cast<const float2*>(wk + 2 * lane);
                y = make_float2(y.x * w.x, y.y * w.y);
            }
            top = fmaxf(fabsf(y.x), fabsf(y.y));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float a = __shfl_xor_sync(0xffffffffu, ss, o), b = __shfl_xor_sync(0xffffffffu, ks, o),
                        d = __shfl_xor_sync(0xffffffffu, top, o);
            ss += a, ks += b, top = fmaxf(top, d);
        }
        if (p.latent) {
            if (p.latent_weight) {
                const float inv = 1.f / sqrtf(ss * (1.f / kMlaDv) + p.eps);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float4 w = *reinterpret_cast<const float4*>(wc + (j >> 2) * 256 + lane * 8 + 2 * (j & 3));
                    const float2 a = widen(u[j]), b = widen(u[j + 1]);
                    u[j] = narrow(a.x * w.x * inv, a.y * w.y * inv);
                    u[j + 1] = narrow(b.x * w.z * inv, b.y * w.w * inv);
                }
            }
            uint32_t r = now.r;
            if (p.cos_sin) {
                const float2 v = widen(r);
                r = narrow(v.x * now.cs - v.y * now.sn, v.x * now.sn + v.y * now.cs);
            }
            uint8_t* out = p.kv_cache + to.slot * (kMlaDim * 2);
            reinterpret_cast<uint4*>(out)[lane] = c[0];
            reinterpret_cast<uint4*>(out)[32 + lane] = c[1];
            reinterpret_cast<uint32_t*>(out + kMlaDv * 2)[lane] = r;
        }
        if (p.keys) {
            if (p.key_weight) {
                const float inv = 1.f / sqrtf(ks * (1.f / kHeadDim) + p.eps);
                y = make_float2(y.x * inv, y.y * inv);
                top *= inv;
            }
            if (p.key_pool) {
                reinterpret_cast<uint32_t*>(p.key_pool + to.slot * (kHeadDim * 2))[lane] =
                    p.key_weight ? narrow(y.x, y.y) : now.k;
            } else {
                float scale = top / kE4m3Max;
                if (!(scale > 0.f) || scale > 3.0e38f) scale = 1.f;
                uint16_t code;
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(code) : "f"(y.y / scale), "f"(y.x / scale));
                reinterpret_cast<uint16_t*>(p.key_codes + to.slot * kHeadDim)[lane] = code;
                if (lane == 0) p.key_scales[to.slot] = scale;
            }
        }
    }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, int sms, cudaStream_t stream) {
    static std::atomic<int> resident[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    int per_sm = resident[dev].load(std::memory_order_relaxed);
    if (per_sm == 0) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, append_kernel, kWarpsA * 32, 0);
        if (e != cudaSuccess) return e;
        resident[dev].store(per_sm, std::memory_order_relaxed);
    }
    const int64_t ctas = (p.rows + kWarpsA - 1) / kWarpsA, most = int64_t(sms) * per_sm;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(ctas < most ? ctas : most));
    cfg.blockDim = dim3(kWarpsA * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, append_kernel, p);
}

}  // namespace dsa
