// indexer_kernels.h -- host-side launch interface of the indexer kernels
// (internal to the library; the public ABI is include/dsa_indexer.h).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <mutex>

namespace dsa {

constexpr int kMaxDevices = 64;

// A kernel's dynamic shared-memory limit, set once per device.  Safe when
// several host threads make their first calls at the same time (call_once
// per device); every later call returns the first call's result.  One
// static instance per kernel, used on the launching thread's current device.
struct SmemLimitOnce {
    std::once_flag flag[kMaxDevices];
    cudaError_t result[kMaxDevices] = {};

    template <typename Kernel>
    cudaError_t apply(int dev, Kernel* kernel, int bytes) {
        if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
        std::call_once(flag[dev], [&] {
            result[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        });
        return result[dev];
    }
};

// Fixed problem geometry.
constexpr int kHeads = 32;
constexpr int kHeadDim = 64;
constexpr int kPageEntries = 64;                          // C4 keys per page
constexpr int kPageBytes = kPageEntries * kHeadDim * 2;   // 8 KiB of bf16
constexpr int kPageCodeBytes = kPageEntries * kHeadDim;   // 4 KiB of e4m3 codes (fp8 cache)
constexpr int kPageScaleBytes = kPageEntries * 4;         // 256 B of fp32 key scales (fp8 cache)
constexpr int kQRowBytes = kHeads * kHeadDim * 2;         // 4 KiB of bf16
constexpr int kUnitPositions = 2 * kPageEntries;          // one work unit = 2 pages = 128 keys
constexpr int kMaxBatch = 1024;
constexpr size_t kWorkspaceHeaderBytes = 256;
// Words of the header beside the error word (word 0); all of them are 0 between calls.
constexpr int kAgainWord = 1;    // 32 of them: the requests (a bit each) that a tree decode has to do again
constexpr int kTicketWord = 33;  // of CTAs that count themselves
constexpr int kAgainWords = kMaxBatch / 32;
static_assert(size_t(kTicketWord + 1) * 4 <= kWorkspaceHeaderBytes && kAgainWord + kAgainWords <= kTicketWord, "they fit");

// Device error bits (same values as DSA_DEVERR_* in the public header).
constexpr uint32_t kErrSeqLenClamped = 0x1u;
constexpr uint32_t kErrBadPage = 0x2u;
constexpr uint32_t kErrWaitTimeout = 0x4u;
constexpr uint32_t kErrBadRange = 0x8u;
constexpr uint32_t kErrNoPages = 0x10u;

struct ScoresParams {
    const int32_t* page_table;  // [batch, table_width]
    const int32_t* seq_lens;    // [batch]
    const float* w;             // [batch, 32]
    float* out;                 // [batch, row_width]
    uint32_t* err;              // device error word
    int64_t num_pages;
    int64_t max_context;        // tokens
    int64_t row_width;          // max_context / 4
    int32_t table_width;        // max_context / 256
    int32_t batch;
    int32_t fill_dead;          // 1: write -inf from the live extent to the row end
    int32_t tokens;             // query tokens per request (q [batch, tokens, 32, 64], rows batch x tokens)
    const float* key_scales;    // [num_pages, 64] per-key scales of the fp8 cache (fp8 kernel only)
};

struct TopkParams {
    const float* scores;  // [batch x tokens, row_width]
    const int32_t* seq_lens;  // [batch]
    int32_t* out;         // [batch x tokens, k]
    uint32_t* err;
    int64_t max_context;
    int64_t row_width;
    int32_t batch;
    int32_t k;
    int32_t tokens;       // query tokens per request: row r is token r % tokens of request r / tokens
};

// Scores kernel: persistent, one CTA per SM, TMA page gather + tcgen05 QK.
cudaError_t launch_scores(const CUtensorMap& keys_map, const CUtensorMap& q_map, const ScoresParams& p,
                          cudaStream_t stream);

// Scores kernel on the fp8 key cache (e4m3 codes + per-key fp32 scale in
// p.key_scales): the codes feed tcgen05.mma kind::f8f6f4 directly, against
// each query split into two e4m3 terms in the kernel.  qraw_map: bf16
// queries, unswizzled; w_map: head weights.
cudaError_t launch_scores_fp8(const CUtensorMap& codes_map, const CUtensorMap& qraw_map, const CUtensorMap& w_map,
                              const ScoresParams& p, cudaStream_t stream);

// Top-k kernel: one CTA per request row, radix select over live positions.
cudaError_t launch_topk(const TopkParams& p, cudaStream_t stream);

// Query / head-weight projection (split-K weight stream over a thread-block
// cluster, deterministic reduction through distributed shared memory).
struct ProjParams {
    __nv_bfloat16_raw* q_out; // [batch, 32, 64] bf16
    float* w_out;             // [batch, 32]
    uint32_t* err;            // device error word
    int32_t batch;
    int32_t batch_pad;        // tokens padded to the MMA's N: 32, 64, 128 or 256
    int32_t d_model;          // multiple of 64
    int32_t q_tiles;          // 2048 / 128
    int32_t k_split;          // CTAs along d (one cluster), 1..8, <= d_model / 64
};
int proj_batch_pad(int batch);
cudaError_t launch_proj(const CUtensorMap& wq_map, const CUtensorMap& ww_map, const CUtensorMap& x_map,
                        const ProjParams& p, cudaStream_t stream);

// Sparse multi-head latent attention decode over the top-k entries: 64 heads,
// 576-wide bf16 cache entries paged like the index keys, value = first 512 dims.
constexpr int kMlaHeads = 64;
constexpr int kMlaDim = 576;
constexpr int kMlaDv = 512;
constexpr int kMlaMaxTopk = 2048;
constexpr int kMlaMaxSplits = 32;
struct MlaParams {
    const uint8_t* kv;         // [num_pages, 64, 576] bf16
    const int32_t* page_table; // [batch, table_width]
    const int32_t* seq_lens;   // [batch] tokens
    const int32_t* topk;       // [batch, k] C4 positions, -1 = unused
    float* out;                // [batch, 64, 512]
    float* lse;                // [batch, 64]
    float* o_part;             // [batch, splits, 64, 512] (splits > 1)
    float* lse_part;           // [batch, splits, 64]
    uint32_t* err;             // device error word
    int64_t num_pages;
    int64_t max_context;
    int32_t table_width;
    int32_t batch;
    int32_t k;
    int32_t splits;            // CTAs per request, 1..32
    float sm_scale_log2;       // sm_scale * log2(e)
};
size_t mla_smem_bytes();
// Decode kernel (grid splits x batch) and, for splits > 1, the log-sum-exp merge.
// q_map: q [batch * 64, 576] bf16, 128-byte-swizzled boxes of 64 x 64.
// kv_map: the cache as [num_pages * 64, 576] bf16 rows, 128-byte-swizzled boxes of
// one row x 64 (the row gathers' map).
cudaError_t launch_mla(const CUtensorMap& q_map, const CUtensorMap& kv_map, const MlaParams& p, cudaStream_t stream);

// Latent attention decode over every live entry, 1-4 tokens per request.
constexpr int kMlaMaxGroups = 256;
// Where a tree decode's kernel on clusters has left its partial outputs (see MlaMergeParams).
struct MlaTreeOutputs {
    const int2* plan;
    const int32_t* cuts;
    const float* o_part;
    const float* lse_part;
    int32_t ranges;
};
struct MlaDenseParams {
    const int32_t* page_table; // [batch, table_width]
    const int32_t* seq_lens;   // [batch] tokens
    __nv_bfloat16_raw* out;    // [batch, tokens, 64, 512]
    float* lse;                // [batch, tokens, 64]
    int2* plan;                // [batch] first and last range of each request (equal: one)
    int32_t* cuts;             // [groups] the request that the range is the second one of, or -1
    float* o_part;             // [groups * tokens * 2, 64, 512] partial outputs
    float* lse_part;           // [groups * tokens * 2, 64]
    uint32_t* err;             // device error word
    int64_t num_pages;
    int64_t max_context;
    int32_t table_width;
    int32_t batch;
    int32_t tokens;            // query tokens per request
    int32_t groups;            // ranges: SMs / tokens
    int32_t merge_by_cut;      // the merge goes by cuts (there are fewer ranges than requests)
    float sm_scale_log2;       // sm_scale * log2(e)
    // of a tree of drafted tokens:
    const uint64_t* mask;      // [batch, tokens] bit i: the token sees drafted entry i
    const int32_t* counts;     // [batch] drafted tokens, or null: all `tokens`
    uint32_t* flags;           // [kAgainWords] with redo: requests whose outputs of that kernel are not to be used; cleared
    uint32_t* ticket;          // with redo, 0 between calls
    uint32_t* again;           // [kAgainWords + 1] with redo: a copy of the flags for the merge, and whether any is set
    int32_t redo;              // another kernel has done the call: only flagged requests are done here
    MlaTreeOutputs first;      // with redo: of that kernel, for the merge
};
// q_map and kv_map: 576-wide bf16 rows (q: batch * tokens * 64 of them; the cache: num_pages * 64) as
// (dim in slab, row, slab of 64 dims), boxes of 64 rows x 3 slabs and 64 rows x 2 slabs; kr_map: the
// cache's rows as (dim, row), boxes of 64 x 64; o_map: out as [batch * tokens * 64, 512] rows, boxes of
// 64 x 64.  All 128-byte-swizzled.
cudaError_t launch_mla_dense(const CUtensorMap& q_map, const CUtensorMap& kv_map, const CUtensorMap& kr_map,
                             const CUtensorMap& o_map, const MlaDenseParams& p, cudaStream_t stream);

// The same for a tree of drafted tokens (1-64 per request), each of which sees all of the cache and the drafted
// entries of its mask.  d_map: the drafted entries as (dim in slab, token, slab, request), boxes of 64 tokens x 1 slab.
cudaError_t launch_mla_dense_tree(const CUtensorMap& q_map, const CUtensorMap& kv_map, const CUtensorMap& kr_map,
                                  const CUtensorMap& o_map, const CUtensorMap& d_map, const MlaDenseParams& p,
                                  cudaStream_t stream);

// The log-sum-exp merge of requests that cross ranges (of the dense and the tree decode).  Rows go by requests, or by
// cuts between ranges where those are fewer.
struct MlaMergeParams {
    const int2* plan;          // [batch] first and last range of each request (equal: one)
    const int32_t* cuts;       // [ranges] the request that the range is the second one of, or -1
    const float* o_part;       // [ranges * tokens * 2, 64, 512] partial outputs: of a range and token the one
    const float* lse_part;     // [ranges * tokens * 2, 64]      that began earlier, then the one that begins here
    __nv_bfloat16_raw* out;    // [batch, tokens, 64, 512]
    float* lse;                // [batch, tokens, 64]
    const int32_t* counts;     // [batch] tokens of each request, or null: all
    const uint32_t* again;     // [kAgainWords + 1] the requests that the dense kernel has done again (null: none), whose
                               // partials are these four:
    const int2* plan_again;
    const int32_t* cuts_again;
    const float* o_again;
    const float* lse_again;
    int32_t tokens, batch;
    int32_t by_cut, rows;              // requests (or cuts) x tokens (cuts of tiled partials: x places)
    int32_t by_cut_again, rows_again;  // of the dense kernel's second try
    int32_t tiled;             // the partials are of tiles of four tokens (tree_places of them a range, plans
                               // [tiles, batch], cuts 16 request + tile) and lie as tiled_part says (those of a
                               // second try never do)
    int32_t one_head;          // few rows that are split many ways: more threads a row
};
cudaError_t launch_mla_merge(const MlaMergeParams& p, cudaStream_t stream);
// Where a dim (a multiple of 4) of a head lies in a tiled partial: eight dims of all 64 heads after one another.
__host__ __device__ inline int64_t tiled_part(int64_t part, int head, int dim) {
    return ((part * (kMlaDv / 8) + dim / 8) * kMlaHeads + head) * 8 + dim % 8;
}

// Latent attention decode for trees of drafted tokens, on clusters of four CTAs.
struct MlaTreeParams {
    const __nv_bfloat16_raw* q; // [batch, tokens, 64, 576]
    const int32_t* page_table; // [batch, table_width]
    const int32_t* seq_lens;   // [batch] tokens in the cache
    const uint64_t* mask;      // [batch, tokens] bit i: the token sees drafted entry i
    const int32_t* counts;     // [batch] drafted tokens, or null: all `tokens`
    __nv_bfloat16_raw* out;    // [batch, tokens, 64, 512]
    float* lse;                // [batch, tokens, 64]
    int2* plan;                // these four as for the merge
    int32_t* cuts;
    float* o_part;
    float* lse_part;
    uint32_t* err;             // device error word
    uint32_t* flags;           // [kAgainWords] a bit each, 0 at first: requests whose outputs are not to be used
    int64_t num_pages;
    int64_t max_context;
    int32_t table_width;
    int32_t batch;
    int32_t tokens;
    int32_t tiles;             // tree_tiles: of four tokens
    int32_t ranges;            // tree_ranges: at most
    int32_t clusters;          // of the device (set by the launch)
    float sm_scale_log2;       // sm_scale * log2(e)
};
// 576-wide bf16 rows as (dim in slab, row, slab), boxes of rows x slabs: q 128 x 1; the cache's, k 32 x 3, v 64 x
// 2; the drafted entries as (dim in slab, token, slab, request), d 32 tokens x 1; o, out as [batch * tokens * 64, 512]
// rows, boxes of 64 x 64.  All 128-byte-swizzled.
struct MlaTreeMaps {
    CUtensorMap q, k, v, d, o;
};
cudaError_t mla_tree_quads(int* quads);                    // clusters that the current device holds
cudaError_t launch_mla_tree(const MlaTreeMaps& m, MlaTreeParams p, int quads, cudaStream_t stream);

// The same for two tokens, on clusters of two CTAs, with a running maximum (flags are not used), and its merge.
// q and v: boxes of 64 rows x 3 slabs and x 2; k: the cache's rows as (dim, row), 64 x 64; d: 64 tokens x 1.
cudaError_t mla_tree_pairs(int* pairs);                    // clusters that the current device holds
cudaError_t launch_mla_tree_pair(const MlaTreeMaps& m, MlaTreeParams p, int pairs, cudaStream_t stream);

// Latent attention over ragged prompts, expanded form: per-head 128 + 64 shared key dims, 128 value dims.
constexpr int kPrefillQk = 192;
constexpr int kPrefillDv = 128;
struct SplitUnit {             // rows that several parts of their entries leave outputs for
    int32_t q_row, rows, head, step_row, step_head;
};
struct PrefillParams {
    const int32_t* cu_q;       // [batch + 1] first row of each request
    const int32_t* cu_kv;      // [batch + 1] first entry of each request
    const int32_t* seq_lens;   // [batch] tokens, the request's rows included
    __nv_bfloat16_raw* out;    // [q_rows, heads, 128]
    float* lse;                // [q_rows, heads]
    uint32_t* err;             // device error word
    int32_t q_rows;
    int32_t kv_rows;
    int32_t batch;
    int32_t heads;
    int32_t entry_tokens;      // tokens per entry
    int32_t slots;             // prefill_slots: at least the blocks of up to 512 rows
    int2* split;               // cut units, and parts of each (1: none is cut)
    SplitUnit* split_units;    // [clusters]
    float* o_part;             // [parts, 2 tiles, 256 rows, 128]; null: no splitting
    float* lse_part;           // [parts, 2, 256]
    int32_t out_aligned32;     // out starts on a 32-byte boundary
    float sm_scale_log2;       // sm_scale * log2(e), above 0
};
// 128-byte-swizzled boxes of 64 dims x 128 rows (q, v) or 64 rows (kn, kr), and of 16 rows for a request's
// last tile; q, k_nope and v as (dim, head, row), k_rope as (dim, row).
struct PrefillMaps {
    CUtensorMap q, kn, kr, v, kn16, kr16, v16;
};
size_t prefill_split_bytes(int sms);  // workspace behind the header, with splitting
size_t prefill_part_offset(int sms);  // where in it the parts' outputs start
size_t prefill_max_parts(int sms);
cudaError_t launch_mla_prefill(const PrefillMaps& m, const PrefillParams& p, cudaStream_t stream);

// Residual addition + RMS norm of bf16 rows.
struct RmsNormParams {
    const void* x;            // bf16, rows x_stride elements apart
    const void* residual;     // bf16 [rows, d] or null
    const void* weight;       // bf16 or fp32 [d]
    void* residual_out;       // bf16 [rows, d], null without a residual
    void* out;                // bf16 [rows, d] or null
    uint8_t* codes;           // e4m3 [rows, d] or null
    float* scales;            // [rows, groups of a row]
    int64_t x_stride;
    int64_t rows;
    int32_t d;
    int32_t group;            // 64, 128 or 0 (one scale per row)
    int32_t weight_fp32;
    int32_t row_threads;      // threads that share a row (set by the launch)
    int32_t log2_threads;     // of row_threads, where several rows share a CTA
    int32_t ahead;            // how many rows ahead a CTA fetches into L2 (set by the launch)
    float eps;
    float inv_d;              // 1 / d (set by the launch)
};
// align: 32, 16 or 2, the boundary in bytes of every 16-element unit (codes: half of it); d is a multiple
// of align / 2.
cudaError_t launch_rmsnorm(RmsNormParams p, int align, int sms, cudaStream_t stream);

// Page tables, lengths, free pages and slots, from the lengths now and those wanted.
struct PagesParams {
    const int32_t* seq_lens;   // [batch] tokens now
    const int32_t* new_lens;   // [batch] tokens wanted
    int32_t* page_table;       // [batch, table_width]
    int32_t* free_pages;       // [num_pages] a stack
    const int32_t* free_count; // [1]
    int32_t* seq_lens_out;     // [batch] (may be seq_lens)
    int32_t* free_count_out;   // [1] (may be free_count)
    int32_t* cu_slots;         // [batch + 1]
    int64_t* slots;            // [max_slots], 16-byte aligned like positions
    int32_t* positions;        // [max_slots]
    uint32_t* err;             // device error word
    uint32_t* ticket;          // in the workspace header, 0 between calls
    int64_t num_pages;
    int64_t max_context;
    int64_t max_slots;
    int32_t table_width;
    int32_t batch;
    int32_t in_place;          // seq_lens_out or free_count_out is an input
};
cudaError_t launch_pages_update(const PagesParams& p, int sms, cudaStream_t stream);

// New entries into the paged caches at their slots.
struct AppendParams {
    const int64_t* slots;      // [rows], -1: skipped
    const uint8_t* latent;     // bf16 [rows, 576], rows latent_stride elements apart, or null
    const void* latent_weight; // [512] bf16 or fp32, or null: no norm
    const float* cos_sin;      // [cos_rows, 64], or null: no rotation
    const int32_t* positions;  // [rows]
    const uint8_t* keys;       // bf16 [rows, 64], rows key_stride elements apart, or null
    const void* key_weight;    // [64] bf16 or fp32, or null: no norm
    uint8_t* kv_cache;         // bf16 [num_pages, 64, 576]
    uint8_t* key_pool;         // bf16 [num_pages, 64, 64], or null: the two below
    uint8_t* key_codes;        // e4m3 [num_pages, 64, 64]
    float* key_scales;         // [num_pages, 64]
    uint32_t* err;             // device error word
    int64_t rows;
    int64_t latent_stride;
    int64_t key_stride;
    int64_t cos_rows;
    int64_t num_pages;
    int32_t latent_weight_fp32;
    int32_t key_weight_fp32;
    float eps;
};
cudaError_t launch_append(const AppendParams& p, int sms, cudaStream_t stream);

}  // namespace dsa
