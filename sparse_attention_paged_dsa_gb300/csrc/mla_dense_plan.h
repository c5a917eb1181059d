// mla_dense_plan.h -- how the dense latent decode cuts a batch's units into ranges, and where a range stages
// its outputs.  Plain arithmetic, compiled for the device and, by the tests, for the host.
#pragma once

#if defined(__CUDACC__)
#define DSA_PLAN __host__ __device__ __forceinline__
#else
#define DSA_PLAN inline
#endif

namespace dsa {

constexpr int kMlaSegUnits = 2;     // a request's fixed cost in a range (q, output), in blocks
constexpr int kMlaWholeBlocks = 4;  // requests of at most this many blocks are not split

DSA_PLAN int units_of(int blocks) { return blocks ? blocks + kMlaSegUnits : 0; }

// Equal ranges of `total` units: range g is [cut(g), cut(g + 1)).  32-bit arithmetic only.
struct Ranges {
    int n, total, q, r;
    DSA_PLAN Ranges(int n_, int total_) : n(n_), total(total_), q(total_ / n_), r(total_ % n_) {}
    DSA_PLAN int cut(int g) const { return q * g + r * g / n; }  // r * g < 2^16
    DSA_PLAN int of(int unit) const {                           // the range that holds a unit
        int g = int(float(unit) * float(n) / float(total));
        if (g > n - 1) g = n - 1;
        while (g > 0 && cut(g) > unit) --g;
        while (g + 1 < n && cut(g + 1) <= unit) ++g;
        return g;
    }
};

// Where a cut inside a request of `blocks` blocks, whose units start at u, comes to lie.
DSA_PLAN int settled_cut(int cut, int u, int blocks) {
    const int n = units_of(blocks);
    return blocks > kMlaWholeBlocks ? cut : ((cut - u) * 2 < n ? u : u + n);
}

// May a partial output be staged over the whole ring, in one round, rather than 32 heads at a time in the half
// of its request's last block?  Nothing may follow in the range, and the other half must be at rest: the
// output of the request before is staged there, and what orders that store's reads before new writes is the
// half's refill.  So the request has a second block here, or it is the range's first one.  `blocks`: the
// request's in this range; `so_far`: the range's, this request's included.
DSA_PLAN bool stage_whole_ring(bool last, int blocks, int so_far) { return last && (blocks > 1 || so_far == blocks); }

}  // namespace dsa
