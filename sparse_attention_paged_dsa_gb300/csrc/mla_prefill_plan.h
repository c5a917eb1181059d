// mla_prefill_plan.h -- how the prompt attention cuts a request's rows into units.  Plain arithmetic, compiled
// for the device and, by the tests, for the host.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define DSA_PREFILL_PLAN __host__ __device__ __forceinline__
#else
#define DSA_PREFILL_PLAN inline
#endif

namespace dsa {

constexpr int kPrefillBlock = 512;  // rows of a request that share a pass over its entries
constexpr int kPrefillPair = 256;   // rows of a query tile: of a unit of two heads
constexpr int kFewEntries = 768;    // see Cut: two heads a unit up to here (prompts of 512 rows: 146 us
                                    // against 155), one above (of 1024: 80 against 100)

// How a request's rows are cut.  Few entries: 256 rows at a time, two heads a unit, whose tiles run for
// equally many key tiles (the halves of 512 rows do not, and a tile alone waits out its own softmax).
// Many: 512 rows of one head, whose tiles share keys and values, and at most 256 rows left as above.
struct Cut {
    int rows, heads, pair_blocks, long_blocks;  // blocks of 256 rows for two heads, and of 512 for one
    DSA_PREFILL_PLAN Cut(int rows_, int live, int heads_) : rows(rows_), heads(heads_) {
        const bool few = live <= kFewEntries && heads_ > 1;
        const int left = few ? rows : rows % kPrefillBlock;
        pair_blocks = few || left <= kPrefillPair ? (left + kPrefillPair - 1) / kPrefillPair : 0;
        long_blocks = few ? 0 : (rows + kPrefillPair - 1) / kPrefillBlock;
    }
    DSA_PREFILL_PLAN int pairs() const { return (heads + 1) / 2; }
    DSA_PREFILL_PLAN int units() const { return pair_blocks * pairs() + long_blocks * heads; }
};

// At least the blocks of up to 512 rows of any batch, and at least its units, whatever its lengths: a block is
// a unit per head, or two halves with a unit for every two heads each (an odd last head's is a unit all the same).
DSA_PREFILL_PLAN int64_t prefill_slots(int64_t q_rows, int batch) { return q_rows / kPrefillBlock + batch; }
DSA_PREFILL_PLAN int64_t prefill_most_units(int64_t slots, int heads) {
    return slots * (heads > 1 ? heads + heads % 2 : 1);
}

}  // namespace dsa
