// dsa_indexer_api.cu -- the C ABI (include/dsa_indexer.h): argument checks,
// TMA descriptor set-up, and kernel launches on the caller's stream.
// Nothing here allocates, frees or synchronises during a compute call.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../include/dsa_indexer.h"
#include "api_checks.h"
#include "indexer_kernels.h"
#include "mla_prefill_plan.h"
#include "mla_tree_plan.h"

namespace {

using dsa::kHeadDim;
using dsa::kHeads;
using dsa::kPageEntries;

constexpr int64_t kMaxContext = int64_t(1) << 24;  // 16M tokens per request row
constexpr int64_t kMaxPages = (int64_t(1) << 31) - 1;

thread_local char g_last_cuda_error[256] = "";

dsa_status_t cuda_fail(cudaError_t e, const char* where) {
    std::snprintf(g_last_cuda_error, sizeof g_last_cuda_error, "%s: %s (%d)", where, cudaGetErrorString(e),
                  int(e));
    return DSA_ERR_CUDA;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

PFN_cuTensorMapEncodeTiled_v12000 encode_tiled() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// Key pool [num_pages, 64, 64] bf16 as a 3-D tensor (dim, entry, page); one
// box = one whole page, stored with the 128-byte swizzle the MMA reads.
dsa_status_t make_keys_map(CUtensorMap* map, const void* key_pool, int64_t num_pages) {
    auto enc = encode_tiled();
    if (!enc) return cuda_fail(cudaErrorNotSupported, "cuTensorMapEncodeTiled lookup");
    const cuuint64_t dims[3] = {cuuint64_t(kHeadDim), cuuint64_t(kPageEntries), cuuint64_t(num_pages)};
    const cuuint64_t strides[2] = {cuuint64_t(kHeadDim * 2), cuuint64_t(kPageEntries * kHeadDim * 2)};
    const cuuint32_t box[3] = {cuuint32_t(kHeadDim), cuuint32_t(kPageEntries), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(key_pool), dims, strides,
                           box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        std::snprintf(g_last_cuda_error, sizeof g_last_cuda_error, "cuTensorMapEncodeTiled(keys): CUresult %d",
                      int(r));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

// fp8 key cache: codes [num_pages, 64, 64] uint8 as a 3-D tensor (dim, entry,
// page), one box = one page of codes stored with the 64-byte swizzle the
// 8-bit MMA reads.  (The scales are copied by the kernel with cp.async.)
dsa_status_t make_codes_map(CUtensorMap* codes_map, const void* key_codes, int64_t num_pages) {
    auto enc = encode_tiled();
    if (!enc) return cuda_fail(cudaErrorNotSupported, "cuTensorMapEncodeTiled lookup");
    const cuuint64_t cdims[3] = {cuuint64_t(kHeadDim), cuuint64_t(kPageEntries), cuuint64_t(num_pages)};
    const cuuint64_t cstrides[2] = {cuuint64_t(kHeadDim), cuuint64_t(kPageEntries * kHeadDim)};
    const cuuint32_t cbox[3] = {cuuint32_t(kHeadDim), cuuint32_t(kPageEntries), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = enc(codes_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(key_codes), cdims, cstrides,
                     cbox, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        std::snprintf(g_last_cuda_error, sizeof g_last_cuda_error, "cuTensorMapEncodeTiled(codes): CUresult %d",
                      int(r));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

// Query [batch * tokens * 32, 64] bf16; one box = the tokens x 32 heads of one request.
dsa_status_t make_q_map(CUtensorMap* map, const void* q, int32_t batch, int32_t tokens = 1) {
    auto enc = encode_tiled();
    if (!enc) return cuda_fail(cudaErrorNotSupported, "cuTensorMapEncodeTiled lookup");
    const cuuint64_t dims[2] = {cuuint64_t(kHeadDim), cuuint64_t(batch) * cuuint64_t(tokens) * kHeads};
    const cuuint64_t strides[1] = {cuuint64_t(kHeadDim * 2)};
    const cuuint32_t box[2] = {cuuint32_t(kHeadDim), cuuint32_t(kHeads * tokens)};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(q), dims, strides, box,
                           estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        std::snprintf(g_last_cuda_error, sizeof g_last_cuda_error, "cuTensorMapEncodeTiled(q): CUresult %d",
                      int(r));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

// Plain (unswizzled) maps for the fp8 kernel's query splitter: q [batch * 32,
// 64] bf16 with one request's 32 heads per box, and w [batch, 32] fp32 with
// one request's weights per box.
dsa_status_t make_plain_q_w_maps(CUtensorMap* q_map, CUtensorMap* w_map, const void* q, const float* w,
                                 int32_t batch) {
    auto enc = encode_tiled();
    if (!enc) return cuda_fail(cudaErrorNotSupported, "cuTensorMapEncodeTiled lookup");
    const cuuint64_t qdims[2] = {cuuint64_t(kHeadDim), cuuint64_t(batch) * kHeads};
    const cuuint64_t qstrides[1] = {cuuint64_t(kHeadDim * 2)};
    const cuuint32_t qbox[2] = {cuuint32_t(kHeadDim), cuuint32_t(kHeads)};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(q), qdims, qstrides, qbox, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        std::snprintf(g_last_cuda_error, sizeof g_last_cuda_error, "cuTensorMapEncodeTiled(q plain): CUresult %d",
                      int(r));
        return DSA_ERR_CUDA;
    }
    const cuuint64_t wdims[2] = {cuuint64_t(kHeads), cuuint64_t(batch)};
    const cuuint64_t wstrides[1] = {cuuint64_t(kHeads * sizeof(float))};
    const cuuint32_t wbox[2] = {cuuint32_t(kHeads), 1};
    r = enc(w_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float*>(w), wdims, wstrides, wbox, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        std::snprintf(g_last_cuda_error, sizeof g_last_cuda_error, "cuTensorMapEncodeTiled(w): CUresult %d", int(r));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

// bf16 2-D tensor [rows, cols] (cols contiguous, rows `row_stride` elements apart, by default cols) with a 128-byte-swizzled box of box_rows x 64.
dsa_status_t make_rows_map(CUtensorMap* map, const void* ptr, int64_t rows, int64_t cols, uint32_t box_rows,
                           const char* what, int64_t row_stride = 0) {
    auto enc = encode_tiled();
    if (!enc) return cuda_fail(cudaErrorNotSupported, "cuTensorMapEncodeTiled lookup");
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(row_stride ? row_stride : cols) * 2};
    const cuuint32_t box[2] = {64, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box,
                           estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        std::snprintf(g_last_cuda_error, sizeof g_last_cuda_error, "cuTensorMapEncodeTiled(%s): CUresult %d", what,
                      int(r));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

// 576-wide bf16 rows as (dim in slab, row, slab of 64 dims): boxes of box_rows rows x box_slabs slabs, 128-byte
// swizzle, so that one copy fills several slabs.
dsa_status_t make_slabs_map(CUtensorMap* map, const void* ptr, int64_t rows, uint32_t box_slabs, const char* what,
                            uint32_t box_rows = 64) {
    auto enc = encode_tiled();
    if (!enc) return cuda_fail(cudaErrorNotSupported, "cuTensorMapEncodeTiled lookup");
    const cuuint64_t dims[3] = {64, cuuint64_t(rows), DSA_MLA_DIM / 64};
    const cuuint64_t strides[2] = {DSA_MLA_DIM * 2, 128};
    const cuuint32_t box[3] = {64, box_rows, box_slabs};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box,
                           estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        std::snprintf(g_last_cuda_error, sizeof g_last_cuda_error, "cuTensorMapEncodeTiled(%s): CUresult %d", what,
                      int(r));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

// bf16 [rows, heads, dim] with element strides (dim contiguous) as (dim, head, row): boxes of
// 64 dims x 1 head x box_rows, 128-byte swizzle.
dsa_status_t make_heads_map(CUtensorMap* map, const void* ptr, int64_t rows, int32_t heads, int32_t dim,
                            int64_t row_stride, int64_t head_stride, uint32_t box_rows, const char* what) {
    auto enc = encode_tiled();
    if (!enc) return cuda_fail(cudaErrorNotSupported, "cuTensorMapEncodeTiled lookup");
    const cuuint64_t dims[3] = {cuuint64_t(dim), cuuint64_t(heads), cuuint64_t(rows)};
    const cuuint64_t strides[2] = {cuuint64_t(head_stride) * 2, cuuint64_t(row_stride) * 2};
    const cuuint32_t box[3] = {64, 1, box_rows};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box,
                           estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        std::snprintf(g_last_cuda_error, sizeof g_last_cuda_error, "cuTensorMapEncodeTiled(%s): CUresult %d", what,
                      int(r));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

// Drafted entries [batch, tokens, 576] bf16 as (dim in slab, token, slab of 64 dims, request): boxes of one slab of
// box_rows tokens, those behind the request's arriving as zeros.
dsa_status_t make_drafts_map(CUtensorMap* map, const void* ptr, int32_t batch, int32_t tokens, uint32_t box_rows) {
    auto enc = encode_tiled();
    if (!enc) return cuda_fail(cudaErrorNotSupported, "cuTensorMapEncodeTiled lookup");
    const cuuint64_t dims[4] = {64, cuuint64_t(tokens), DSA_MLA_DIM / 64, cuuint64_t(batch)};
    const cuuint64_t strides[3] = {DSA_MLA_DIM * 2, 128, cuuint64_t(tokens) * DSA_MLA_DIM * 2};
    const cuuint32_t box[4] = {64, box_rows, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box,
                           estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        std::snprintf(g_last_cuda_error, sizeof g_last_cuda_error, "cuTensorMapEncodeTiled(drafts): CUresult %d",
                      int(r));
        return DSA_ERR_CUDA;
    }
    return DSA_OK;
}

constexpr int kProjMaxSplit = 8;  // CTAs per cluster (portable size)
constexpr int kProjQTiles = (DSA_HEADS * DSA_HEAD_DIM) / 128;
constexpr int64_t kProjMaxModel = 65536;

dsa_status_t check_shape(int32_t batch, int64_t max_context) {
    if (batch < 1 || max_context < 1 || max_context % DSA_PAGE_TOKENS != 0) return DSA_ERR_INVALID_ARG;
    if (batch > DSA_MAX_BATCH || max_context > kMaxContext) return DSA_ERR_UNSUPPORTED;
    return DSA_OK;
}

dsa_status_t check_workspace(const void* ws, size_t bytes, size_t need) {
    if (ws == nullptr || !aligned(ws, 256) || bytes < need) return DSA_ERR_WORKSPACE;
    return DSA_OK;
}

dsa_status_t check_score_inputs(const void* q, const float* w, const void* key_pool, int64_t num_pages,
                                const int32_t* page_table, const int32_t* seq_lens) {
    if (!q || !w || !key_pool || !page_table || !seq_lens) return DSA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(w, 16) || !aligned(key_pool, 16) || !aligned(page_table, 4) ||
        !aligned(seq_lens, 4))
        return DSA_ERR_INVALID_ARG;
    if (num_pages < 1 || num_pages > kMaxPages) return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

dsa::ScoresParams score_params(const float* w, int64_t num_pages, const int32_t* page_table,
                               const int32_t* seq_lens, int32_t batch, int64_t max_context, float* out,
                               int fill_dead, void* workspace, int32_t tokens = 1) {
    dsa::ScoresParams p{};
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.w = w;
    p.out = out;
    p.err = static_cast<uint32_t*>(workspace);
    p.num_pages = num_pages;
    p.max_context = max_context;
    p.row_width = max_context / 4;
    p.table_width = int32_t(max_context / DSA_PAGE_TOKENS);
    p.batch = batch;
    p.fill_dead = fill_dead;
    p.tokens = tokens;
    return p;
}

dsa_status_t run_scores(const void* q, const float* w, const void* key_pool, int64_t num_pages,
                        const int32_t* page_table, const int32_t* seq_lens, int32_t batch, int64_t max_context,
                        float* out, int fill_dead, void* workspace, cudaStream_t stream, int32_t tokens = 1) {
    CUtensorMap keys_map, q_map;
    dsa_status_t st = make_keys_map(&keys_map, key_pool, num_pages);
    if (st != DSA_OK) return st;
    st = make_q_map(&q_map, q, batch, tokens);
    if (st != DSA_OK) return st;
    const dsa::ScoresParams p =
        score_params(w, num_pages, page_table, seq_lens, batch, max_context, out, fill_dead, workspace, tokens);
    const cudaError_t e = dsa::launch_scores(keys_map, q_map, p, stream);
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "scores kernel launch");
}

dsa_status_t run_scores_fp8(const void* q, const float* w, const void* key_codes, const float* key_scales,
                            int64_t num_pages, const int32_t* page_table, const int32_t* seq_lens, int32_t batch,
                            int64_t max_context, float* out, int fill_dead, void* workspace, cudaStream_t stream) {
    CUtensorMap codes_map, q_map, w_map;
    dsa_status_t st = make_codes_map(&codes_map, key_codes, num_pages);
    if (st != DSA_OK) return st;
    st = make_plain_q_w_maps(&q_map, &w_map, q, w, batch);
    if (st != DSA_OK) return st;
    dsa::ScoresParams p =
        score_params(w, num_pages, page_table, seq_lens, batch, max_context, out, fill_dead, workspace);
    p.key_scales = key_scales;
    const cudaError_t e = dsa::launch_scores_fp8(codes_map, q_map, w_map, p, stream);
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "fp8 scores kernel launch");
}

dsa_status_t run_topk(const float* scores, const int32_t* seq_lens, int32_t batch, int64_t max_context, int32_t k,
                      int32_t* topk_idx, void* workspace, cudaStream_t stream, int32_t tokens = 1) {
    dsa::TopkParams p{};
    p.scores = scores;
    p.seq_lens = seq_lens;
    p.out = topk_idx;
    p.err = static_cast<uint32_t*>(workspace);
    p.max_context = max_context;
    p.row_width = max_context / 4;
    p.batch = batch;
    p.k = k;
    p.tokens = tokens;
    const cudaError_t e = dsa::launch_topk(p, stream);
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "top-k kernel launch");
}

// Workspace of a fused call over `nrows` score rows: the header, plus the
// live-score slots when no scores row is given.
size_t fused_workspace_bytes(int64_t nrows, int64_t max_context, bool with_slots) {
    return dsa::kWorkspaceHeaderBytes + (with_slots ? size_t(nrows) * size_t(max_context / 4) * sizeof(float) : 0);
}

float* fused_rows(void* workspace, float* scores_opt) {
    return scores_opt ? scores_opt
                      : reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + dsa::kWorkspaceHeaderBytes);
}

// Splits of a request's top-k row across CTAs (one CTA per SM): enough to fill
// the current device once, at most one per 64-entry block and kMlaMaxSplits.
int mla_splits(int32_t batch, int32_t k) {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) !=
                                                   cudaSuccess)
        sms = 148;
    const int blocks = (k + 63) / 64;
    int s = sms / batch;
    if (s > blocks) s = blocks;
    if (s > dsa::kMlaMaxSplits) s = dsa::kMlaMaxSplits;
    return s < 1 ? 1 : s;
}
size_t mla_partial_floats(int32_t batch, int splits) {
    return splits > 1 ? size_t(batch) * size_t(splits) * dsa::kMlaHeads * (dsa::kMlaDv + 1) : 0;
}

// SMs of the current device (cached per device: the query is on every launch's path).
cudaError_t sm_count(int* sms) {
    static std::atomic<int> known[dsa::kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= dsa::kMaxDevices) return cudaErrorInvalidDevice;
    *sms = known[dev].load(std::memory_order_relaxed);
    if (*sms > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) known[dev].store(*sms, std::memory_order_relaxed);
    return e;
}

// Dense latent decode: one range of work per group of next_n CTAs, one CTA per SM.
int dense_groups(int sms, int32_t next_n) {
    const int g = sms / next_n;
    return g < 1 ? 1 : (g > dsa::kMlaMaxGroups ? dsa::kMlaMaxGroups : g);
}
constexpr size_t kDenseCutBytes = size_t(dsa::kMlaMaxGroups) * sizeof(int32_t);
constexpr size_t kDensePlanBytes = size_t(DSA_MAX_BATCH) * sizeof(int2) + kDenseCutBytes;
size_t dense_parts(int groups, int32_t next_n) { return size_t(groups) * size_t(next_n) * 2; }
size_t dense_workspace_bytes(int groups, int32_t next_n) {
    return dsa::kWorkspaceHeaderBytes + kDensePlanBytes +
           dense_parts(groups, next_n) * dsa::kMlaHeads * (dsa::kMlaDv + 1) * sizeof(float);
}

// From this many tokens x context on, a tree of two tokens or more is worth a kernel on clusters.  Of two CTAs (us,
// dense kernel and that one, two tokens each: 4 x 65536 context 41.5, 41.5; 1 x 262144 38, 37; 16 x 131072 183, 131;
// 64 x 8192 75, 65; 64 x 65536 354, 244), or of four (1 request, 4 tokens, 131072 context 44, 46; 4 x 8, 8192 36, 40;
// 16 x 8, 4096 58, 58; 1 x 16, 32768 52, 46; 64 x 8, 8192 212, 134; 16 x 32, 131072 2996, 1275).
constexpr int64_t kTreeWork = int64_t(1) << 19;
// But not two tokens of requests of a page or two, where a request's start and end count (512: 600 of them 73, 85,
// 1024 121, 140; 768: 85, 84 and 141, 136).
constexpr int64_t kPairContext = 512;

// Tree decode: header, cuts, plan (of each tile), the same of the dense kernel, then two partial outputs per range
// and token, of the kernel that the call takes.  (Of more than two tokens the dense one may have to do some requests
// again while the others' partials wait for the merge: room for both.)
struct TreeShape {
    int groups;                   // of the dense kernel
    int clusters, tiles, ranges;  // of the one on clusters: of two CTAs for two tokens, of four for more
    TreeShape(int32_t tokens, int sms, int quads, int pairs)
        : groups(dense_groups(sms, tokens)), clusters(tokens > dsa::kPairTokens ? quads : pairs),
          tiles(tokens > dsa::kPairTokens ? dsa::tree_tiles(tokens) : 1),
          ranges(tokens < dsa::kPairTokens ? 0 : dsa::tree_ranges(tiles, clusters)) {}
    size_t tiled_parts(int32_t tokens) const { return dense_parts(ranges * tiles, dsa::tree_places(tokens)); }
    size_t parts(int32_t tokens) const {
        const size_t dense = dense_parts(groups, tokens), tiled = tiled_parts(tokens);
        return tokens > dsa::kPairTokens ? dense + tiled : (dense > tiled ? dense : tiled);
    }
    size_t workspace_bytes(int32_t tokens) const {
        return dsa::kWorkspaceHeaderBytes + kTreePlanBytes +
               parts(tokens) * dsa::kMlaHeads * (dsa::kMlaDv + 1) * sizeof(float);
    }
    static constexpr size_t kCutBytes = size_t(dsa::kTreeMaxUnits) * sizeof(int32_t);
    static constexpr size_t kDenseAt = kCutBytes + size_t(dsa::kTreeMaxTiles) * DSA_MAX_BATCH * sizeof(int2);
    static constexpr size_t kAgainAt = kDenseAt + kDensePlanBytes;
    static constexpr size_t kTreePlanBytes = (kAgainAt + (dsa::kAgainWords + 1) * sizeof(uint32_t) + 255) / 256 * 256;
};

dsa_status_t run_rmsnorm(dsa::RmsNormParams p, void* stream) {
    if (p.rows < 0 || p.rows > INT32_MAX || p.d < 1 || p.x_stride < 0 || !std::isfinite(p.eps) || p.eps < 0.f ||
        (p.weight_fp32 != 0 && p.weight_fp32 != 1))
        return DSA_ERR_INVALID_ARG;
    if (p.d > DSA_NORM_MAX_DIM) return DSA_ERR_UNSUPPORTED;
    if (p.rows == 0) return DSA_OK;
    if (p.rows == 1) p.x_stride = p.d;  // no second row: the stride means nothing
    if (!p.x || !p.weight || (p.residual == nullptr) != (p.residual_out == nullptr) || (!p.out && !p.codes))
        return DSA_ERR_INVALID_ARG;
    if (!aligned(p.x, 2) || !aligned(p.residual, 2) || !aligned(p.residual_out, 2) || !aligned(p.out, 2) ||
        !aligned(p.weight, p.weight_fp32 ? 4 : 2) || !aligned(p.scales, 4))
        return DSA_ERR_INVALID_ARG;
    if (p.out && p.out == p.residual_out) return DSA_ERR_INVALID_ARG;
    if ((p.out == p.x || p.residual_out == p.x) && p.x_stride != p.d) return DSA_ERR_INVALID_ARG;
    // The boundary that every 16-element unit of every array starts on (its codes: half of it), in bytes.
    const auto on = [&](uintptr_t bytes) {
        const int64_t n = int64_t(bytes) / 2;
        return p.d % n == 0 && p.x_stride % n == 0 && aligned(p.x, bytes) && aligned(p.residual, bytes) &&
               aligned(p.weight, p.weight_fp32 ? 16 : bytes) && aligned(p.residual_out, bytes) &&
               aligned(p.out, bytes) && aligned(p.codes, bytes / 2);
    };
    const int align = on(32) ? 32 : on(16) ? 16 : 2;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return cuda_fail(e, "device query");
    e = dsa::launch_rmsnorm(p, align, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "RMS norm launch");
}

dsa::RmsNormParams norm_params(const void* x, int64_t x_stride, const void* residual, const void* weight,
                               int32_t weight_fp32, int64_t rows, int32_t d, float eps, void* residual_out,
                               void* out) {
    dsa::RmsNormParams p{};
    p.x = x;
    p.residual = residual;
    p.weight = weight;
    p.residual_out = residual_out;
    p.out = out;
    p.x_stride = x_stride;
    p.rows = rows;
    p.d = d;
    p.weight_fp32 = weight_fp32;
    p.eps = eps;
    return p;
}

}  // namespace

namespace dsa {

dsa_status_t check_fused_args(const void* q, const float* w, const void* key_pool, int64_t num_pages,
                              const int32_t* page_table, const int32_t* seq_lens, int32_t batch,
                              int64_t max_context, int32_t k, const int32_t* topk_idx, const float* scores_opt) {
    dsa_status_t st = check_shape(batch, max_context);
    if (st != DSA_OK) return st;
    st = check_score_inputs(q, w, key_pool, num_pages, page_table, seq_lens);
    if (st != DSA_OK) return st;
    if (!topk_idx || !aligned(topk_idx, 4)) return DSA_ERR_INVALID_ARG;
    if (scores_opt && !aligned(scores_opt, 16)) return DSA_ERR_INVALID_ARG;
    if (k < 1 || int64_t(k) > max_context / 4) return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

}  // namespace dsa

extern "C" {

size_t dsa_indexer_workspace_size(int32_t batch, int64_t max_context, int32_t k) {
    (void)k;
    if (check_shape(batch, max_context) != DSA_OK) return 0;
    return fused_workspace_bytes(batch, max_context, true);
}

dsa_status_t dsa_indexer_workspace_init(void* workspace, size_t workspace_bytes, void* stream) {
    if (check_workspace(workspace, workspace_bytes, dsa::kWorkspaceHeaderBytes) != DSA_OK) return DSA_ERR_WORKSPACE;
    const cudaError_t e =
        cudaMemsetAsync(workspace, 0, dsa::kWorkspaceHeaderBytes, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "workspace init");
}

dsa_status_t dsa_indexer_scores(const void* q, const float* w, const void* key_pool, int64_t num_pages,
                                const int32_t* page_table, const int32_t* seq_lens, int32_t batch,
                                int64_t max_context, float* scores, void* workspace, size_t workspace_bytes,
                                void* stream) {
    dsa_status_t st = check_shape(batch, max_context);
    if (st != DSA_OK) return st;
    st = check_score_inputs(q, w, key_pool, num_pages, page_table, seq_lens);
    if (st != DSA_OK) return st;
    if (!scores || !aligned(scores, 16)) return DSA_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, dsa::kWorkspaceHeaderBytes);
    if (st != DSA_OK) return st;
    return run_scores(q, w, key_pool, num_pages, page_table, seq_lens, batch, max_context, scores, 1, workspace,
                      static_cast<cudaStream_t>(stream));
}

dsa_status_t dsa_indexer_topk(const float* scores, const int32_t* seq_lens, int32_t batch, int64_t max_context,
                              int32_t k, int32_t* topk_idx, void* workspace, size_t workspace_bytes,
                              void* stream) {
    dsa_status_t st = check_shape(batch, max_context);
    if (st != DSA_OK) return st;
    if (!scores || !seq_lens || !topk_idx || !aligned(scores, 16) || !aligned(seq_lens, 4) || !aligned(topk_idx, 4))
        return DSA_ERR_INVALID_ARG;
    if (k < 1 || int64_t(k) > max_context / 4) return DSA_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, dsa::kWorkspaceHeaderBytes);
    if (st != DSA_OK) return st;
    return run_topk(scores, seq_lens, batch, max_context, k, topk_idx, workspace, static_cast<cudaStream_t>(stream));
}

dsa_status_t dsa_indexer_fused(const void* q, const float* w, const void* key_pool, int64_t num_pages,
                               const int32_t* page_table, const int32_t* seq_lens, int32_t batch,
                               int64_t max_context, int32_t k, int32_t* topk_idx, float* scores_opt,
                               void* workspace, size_t workspace_bytes, void* stream) {
    dsa_status_t st = dsa::check_fused_args(q, w, key_pool, num_pages, page_table, seq_lens, batch, max_context, k,
                                            topk_idx, scores_opt);
    if (st != DSA_OK) return st;
    st = check_workspace(workspace, workspace_bytes, fused_workspace_bytes(batch, max_context, !scores_opt));
    if (st != DSA_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    float* rows = fused_rows(workspace, scores_opt);
    st = run_scores(q, w, key_pool, num_pages, page_table, seq_lens, batch, max_context, rows, scores_opt ? 1 : 0,
                    workspace, s);
    if (st != DSA_OK) return st;
    return run_topk(rows, seq_lens, batch, max_context, k, topk_idx, workspace, s);
}

dsa_status_t dsa_indexer_scores_fp8(const void* q, const float* w, const void* key_codes, const float* key_scales,
                                    int64_t num_pages, const int32_t* page_table, const int32_t* seq_lens,
                                    int32_t batch, int64_t max_context, float* scores, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    dsa_status_t st = check_shape(batch, max_context);
    if (st != DSA_OK) return st;
    st = check_score_inputs(q, w, key_codes, num_pages, page_table, seq_lens);
    if (st != DSA_OK) return st;
    if (!key_scales || !aligned(key_scales, 16)) return DSA_ERR_INVALID_ARG;
    if (!scores || !aligned(scores, 16)) return DSA_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, dsa::kWorkspaceHeaderBytes);
    if (st != DSA_OK) return st;
    return run_scores_fp8(q, w, key_codes, key_scales, num_pages, page_table, seq_lens, batch, max_context, scores, 1,
                          workspace, static_cast<cudaStream_t>(stream));
}

dsa_status_t dsa_indexer_fused_fp8(const void* q, const float* w, const void* key_codes, const float* key_scales,
                                   int64_t num_pages, const int32_t* page_table, const int32_t* seq_lens,
                                   int32_t batch, int64_t max_context, int32_t k, int32_t* topk_idx,
                                   float* scores_opt, void* workspace, size_t workspace_bytes, void* stream) {
    dsa_status_t st = check_shape(batch, max_context);
    if (st != DSA_OK) return st;
    st = check_score_inputs(q, w, key_codes, num_pages, page_table, seq_lens);
    if (st != DSA_OK) return st;
    if (!key_scales || !aligned(key_scales, 16)) return DSA_ERR_INVALID_ARG;
    if (!topk_idx || !aligned(topk_idx, 4)) return DSA_ERR_INVALID_ARG;
    if (scores_opt && !aligned(scores_opt, 16)) return DSA_ERR_INVALID_ARG;
    if (k < 1 || int64_t(k) > max_context / 4) return DSA_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, fused_workspace_bytes(batch, max_context, !scores_opt));
    if (st != DSA_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    float* rows = fused_rows(workspace, scores_opt);
    st = run_scores_fp8(q, w, key_codes, key_scales, num_pages, page_table, seq_lens, batch, max_context, rows,
                        scores_opt ? 1 : 0, workspace, s);
    if (st != DSA_OK) return st;
    return run_topk(rows, seq_lens, batch, max_context, k, topk_idx, workspace, s);
}

size_t dsa_indexer_workspace_size_mtp(int32_t batch, int32_t next_n, int64_t max_context, int32_t k) {
    (void)k;
    if (check_shape(batch, max_context) != DSA_OK || next_n < 1 || next_n > DSA_MAX_NEXT_N) return 0;
    return fused_workspace_bytes(int64_t(batch) * next_n, max_context, true);
}

dsa_status_t dsa_indexer_scores_mtp(const void* q, const float* w, const void* key_pool, int64_t num_pages,
                                    const int32_t* page_table, const int32_t* seq_lens, int32_t batch,
                                    int32_t next_n, int64_t max_context, float* scores, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    dsa_status_t st = check_shape(batch, max_context);
    if (st != DSA_OK) return st;
    if (next_n < 1 || next_n > DSA_MAX_NEXT_N) return DSA_ERR_INVALID_ARG;
    st = check_score_inputs(q, w, key_pool, num_pages, page_table, seq_lens);
    if (st != DSA_OK) return st;
    if (!scores || !aligned(scores, 16)) return DSA_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, dsa::kWorkspaceHeaderBytes);
    if (st != DSA_OK) return st;
    return run_scores(q, w, key_pool, num_pages, page_table, seq_lens, batch, max_context, scores, 1, workspace,
                      static_cast<cudaStream_t>(stream), next_n);
}

dsa_status_t dsa_indexer_topk_mtp(const float* scores, const int32_t* seq_lens, int32_t batch, int32_t next_n,
                                  int64_t max_context, int32_t k, int32_t* topk_idx, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    dsa_status_t st = check_shape(batch, max_context);
    if (st != DSA_OK) return st;
    if (next_n < 1 || next_n > DSA_MAX_NEXT_N) return DSA_ERR_INVALID_ARG;
    if (!scores || !seq_lens || !topk_idx || !aligned(scores, 16) || !aligned(seq_lens, 4) || !aligned(topk_idx, 4))
        return DSA_ERR_INVALID_ARG;
    if (k < 1 || int64_t(k) > max_context / 4) return DSA_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, dsa::kWorkspaceHeaderBytes);
    if (st != DSA_OK) return st;
    return run_topk(scores, seq_lens, batch, max_context, k, topk_idx, workspace, static_cast<cudaStream_t>(stream),
                    next_n);
}

dsa_status_t dsa_indexer_fused_mtp(const void* q, const float* w, const void* key_pool, int64_t num_pages,
                                   const int32_t* page_table, const int32_t* seq_lens, int32_t batch,
                                   int32_t next_n, int64_t max_context, int32_t k, int32_t* topk_idx,
                                   float* scores_opt, void* workspace, size_t workspace_bytes, void* stream) {
    dsa_status_t st = check_shape(batch, max_context);
    if (st != DSA_OK) return st;
    if (next_n < 1 || next_n > DSA_MAX_NEXT_N) return DSA_ERR_INVALID_ARG;
    st = check_score_inputs(q, w, key_pool, num_pages, page_table, seq_lens);
    if (st != DSA_OK) return st;
    if (!topk_idx || !aligned(topk_idx, 4)) return DSA_ERR_INVALID_ARG;
    if (scores_opt && !aligned(scores_opt, 16)) return DSA_ERR_INVALID_ARG;
    if (k < 1 || int64_t(k) > max_context / 4) return DSA_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes,
                         fused_workspace_bytes(int64_t(batch) * next_n, max_context, !scores_opt));
    if (st != DSA_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    float* rows = fused_rows(workspace, scores_opt);
    st = run_scores(q, w, key_pool, num_pages, page_table, seq_lens, batch, max_context, rows, scores_opt ? 1 : 0,
                    workspace, s, next_n);
    if (st != DSA_OK) return st;
    return run_topk(rows, seq_lens, batch, max_context, k, topk_idx, workspace, s, next_n);
}

size_t dsa_indexer_qw_proj_workspace_size(int32_t batch, int64_t d_model) {
    if (batch < 1 || batch > DSA_PROJ_MAX_TOKENS || d_model < 64 || d_model % 64 != 0 || d_model > kProjMaxModel)
        return 0;
    return dsa::kWorkspaceHeaderBytes;  // the error word only: partial sums stay on chip
}

dsa_status_t dsa_indexer_qw_proj(const void* x, const void* w_q, const void* w_w, int32_t batch, int64_t d_model,
                                 void* q_out, float* w_out, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    const size_t need = dsa_indexer_qw_proj_workspace_size(batch, d_model);
    if (need == 0) return DSA_ERR_INVALID_ARG;
    if (!x || !w_q || !w_w || !q_out || !w_out) return DSA_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w_q, 16) || !aligned(w_w, 16) || !aligned(q_out, 4) || !aligned(w_out, 4))
        return DSA_ERR_INVALID_ARG;
    dsa_status_t st = check_workspace(workspace, workspace_bytes, need);
    if (st != DSA_OK) return st;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "device query");
    const int atoms = int(d_model / 64);
    int k_split = sms / (kProjQTiles + 1);  // about one weight-streaming CTA per SM
    k_split = k_split < 1 ? 1 : (k_split > kProjMaxSplit ? kProjMaxSplit : k_split);
    k_split = k_split > atoms ? atoms : k_split;
    const int bp = dsa::proj_batch_pad(batch);
    CUtensorMap wq_map, ww_map, x_map;
    st = make_rows_map(&wq_map, w_q, kProjQTiles * 128, d_model, 128, "w_q");
    if (st != DSA_OK) return st;
    st = make_rows_map(&ww_map, w_w, DSA_HEADS, d_model, 128, "w_w");
    if (st != DSA_OK) return st;
    st = make_rows_map(&x_map, x, batch, d_model, uint32_t(bp), "x");
    if (st != DSA_OK) return st;
    dsa::ProjParams p{};
    p.q_out = static_cast<__nv_bfloat16_raw*>(q_out);
    p.w_out = w_out;
    p.err = static_cast<uint32_t*>(workspace);
    p.batch = batch;
    p.batch_pad = bp;
    p.d_model = int32_t(d_model);
    p.q_tiles = kProjQTiles;
    p.k_split = k_split;
    e = dsa::launch_proj(wq_map, ww_map, x_map, p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "projection kernel launch");
}

dsa_status_t dsa_indexer_get_error(void* workspace, uint32_t* code, int clear, void* stream) {
    if (!workspace || !code || !aligned(workspace, 256)) return DSA_ERR_INVALID_ARG;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyAsync(&v, workspace, sizeof v, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess && clear) e = cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "read error word");
    *code = v;
    return DSA_OK;
}

const char* dsa_status_string(dsa_status_t status) {
    switch (status) {
        case DSA_OK: return "ok";
        case DSA_ERR_INVALID_ARG: return "invalid argument";
        case DSA_ERR_UNSUPPORTED: return "unsupported shape";
        case DSA_ERR_WORKSPACE: return "workspace missing, misaligned or too small";
        case DSA_ERR_CUDA: return "CUDA error";
    }
    return "unknown status";
}

const char* dsa_indexer_last_cuda_error(void) { return g_last_cuda_error; }

size_t dsa_sparse_mla_workspace_size(int32_t batch, int32_t k) {
    if (batch < 1 || batch > DSA_MAX_BATCH || k < 1 || k > DSA_MLA_MAX_TOPK) return 0;
    return dsa::kWorkspaceHeaderBytes + mla_partial_floats(batch, mla_splits(batch, k)) * sizeof(float);
}
dsa_status_t dsa_sparse_mla_decode(const void* q, const void* kv_cache, int64_t num_pages,
                                   const int32_t* page_table, const int32_t* seq_lens, int32_t batch,
                                   int64_t max_context, const int32_t* topk_idx, int32_t k, float sm_scale,
                                   float* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    dsa_status_t st = check_shape(batch, max_context);
    if (st != DSA_OK) return st;
    if (!q || !kv_cache || !page_table || !seq_lens || !topk_idx || !out || !lse) return DSA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(topk_idx, 4) || !aligned(out, 16) || !aligned(lse, 16))
        return DSA_ERR_INVALID_ARG;
    if (num_pages < 1 || num_pages > kMaxPages) return DSA_ERR_INVALID_ARG;
    if (k < 1 || k > DSA_MLA_MAX_TOPK || !std::isfinite(sm_scale))
        return DSA_ERR_INVALID_ARG;
    const int splits = mla_splits(batch, k);
    st = check_workspace(workspace, workspace_bytes,
                         dsa::kWorkspaceHeaderBytes + mla_partial_floats(batch, splits) * sizeof(float));
    if (st != DSA_OK) return st;
    // The row gathers address cache rows with 32-bit coordinates.
    if (num_pages > (int64_t(1) << 31) / dsa::kPageEntries - 1) return DSA_ERR_UNSUPPORTED;
    CUtensorMap q_map, kv_map;
    st = make_rows_map(&q_map, q, int64_t(batch) * DSA_MLA_HEADS, DSA_MLA_DIM, 64, "mla q");
    if (st != DSA_OK) return st;
    st = make_rows_map(&kv_map, kv_cache, num_pages * dsa::kPageEntries, DSA_MLA_DIM, 1, "mla kv");
    if (st != DSA_OK) return st;
    dsa::MlaParams p{};
    p.kv = static_cast<const uint8_t*>(kv_cache);
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.topk = topk_idx;
    p.out = out;
    p.lse = lse;
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + dsa::kWorkspaceHeaderBytes);
    p.o_part = splits > 1 ? part : nullptr;
    p.lse_part = splits > 1 ? part + size_t(batch) * splits * dsa::kMlaHeads * dsa::kMlaDv : nullptr;
    p.err = static_cast<uint32_t*>(workspace);
    p.num_pages = num_pages;
    p.max_context = max_context;
    p.table_width = int32_t(max_context / DSA_PAGE_TOKENS);
    p.batch = batch;
    p.k = k;
    p.splits = splits;
    p.sm_scale_log2 = sm_scale * 1.4426950408889634f;
    const cudaError_t e = dsa::launch_mla(q_map, kv_map, p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "sparse MLA decode launch");
}

dsa_status_t dsa_rmsnorm(const void* x, int64_t x_stride, const void* residual_opt, const void* weight,
                         int32_t weight_fp32, int64_t rows, int32_t d, float eps, void* residual_out, void* out,
                         void* stream) {
    return run_rmsnorm(norm_params(x, x_stride, residual_opt, weight, weight_fp32, rows, d, eps, residual_out, out),
                       stream);
}

dsa_status_t dsa_rmsnorm_fp8(const void* x, int64_t x_stride, const void* residual_opt, const void* weight,
                             int32_t weight_fp32, int64_t rows, int32_t d, float eps, int32_t group,
                             void* residual_out, void* out_opt, void* codes, float* scales, void* stream) {
    dsa::RmsNormParams p =
        norm_params(x, x_stride, residual_opt, weight, weight_fp32, rows, d, eps, residual_out, out_opt);
    if (group != 0 && group != 64 && group != 128) return DSA_ERR_INVALID_ARG;
    if (rows > 0 && (!codes || !scales)) return DSA_ERR_INVALID_ARG;
    p.group = group;
    p.codes = static_cast<uint8_t*>(codes);
    p.scales = scales;
    return run_rmsnorm(p, stream);
}

size_t dsa_mla_decode_workspace_size(int32_t batch, int32_t next_n) {
    int sms = 0;
    if (batch < 1 || batch > DSA_MAX_BATCH || next_n < 1 || next_n > DSA_MAX_NEXT_N) return 0;
    if (sm_count(&sms) != cudaSuccess) sms = 160;  // no device: what a large part needs
    return dense_workspace_bytes(dense_groups(sms, next_n), next_n);
}

dsa_status_t dsa_mla_decode(const void* q, const void* kv_cache, int64_t num_pages, const int32_t* page_table,
                            const int32_t* seq_lens, int32_t batch, int32_t next_n, int64_t max_context,
                            float sm_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                            void* stream) {
    dsa_status_t st = check_shape(batch, max_context);
    if (st != DSA_OK) return st;
    if (next_n < 1 || next_n > DSA_MAX_NEXT_N) return DSA_ERR_INVALID_ARG;
    if (!q || !kv_cache || !page_table || !seq_lens || !out || !lse) return DSA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(out, 16) || !aligned(lse, 16))
        return DSA_ERR_INVALID_ARG;
    if (num_pages < 1 || num_pages > kMaxPages || !std::isfinite(sm_scale)) return DSA_ERR_INVALID_ARG;
    // The tile loads address cache rows with 32-bit coordinates.
    if (num_pages > (int64_t(1) << 31) / dsa::kPageEntries - 1) return DSA_ERR_UNSUPPORTED;
    st = check_workspace(workspace, workspace_bytes, dsa::kWorkspaceHeaderBytes);
    if (st != DSA_OK) return st;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return cuda_fail(e, "device query");
    const int groups = dense_groups(sms, next_n);
    st = check_workspace(workspace, workspace_bytes, dense_workspace_bytes(groups, next_n));
    if (st != DSA_OK) return st;
    CUtensorMap q_map, kv_map, kr_map, o_map;
    st = make_slabs_map(&q_map, q, int64_t(batch) * next_n * DSA_MLA_HEADS, 3, "mla q");
    if (st != DSA_OK) return st;
    st = make_slabs_map(&kv_map, kv_cache, num_pages * dsa::kPageEntries, 2, "mla kv");
    if (st != DSA_OK) return st;
    st = make_rows_map(&kr_map, kv_cache, num_pages * dsa::kPageEntries, DSA_MLA_DIM, 64, "mla kv");
    if (st != DSA_OK) return st;
    st = make_rows_map(&o_map, out, int64_t(batch) * next_n * DSA_MLA_HEADS, DSA_MLA_DV, 64, "mla out");
    if (st != DSA_OK) return st;
    dsa::MlaDenseParams p{};
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.out = static_cast<__nv_bfloat16_raw*>(out);
    p.lse = lse;
    p.cuts = reinterpret_cast<int32_t*>(ws + dsa::kWorkspaceHeaderBytes);
    p.plan = reinterpret_cast<int2*>(ws + dsa::kWorkspaceHeaderBytes + kDenseCutBytes);
    p.o_part = reinterpret_cast<float*>(ws + dsa::kWorkspaceHeaderBytes + kDensePlanBytes);
    p.lse_part = p.o_part + dense_parts(groups, next_n) * dsa::kMlaHeads * dsa::kMlaDv;
    p.err = static_cast<uint32_t*>(workspace);
    p.num_pages = num_pages;
    p.max_context = max_context;
    p.table_width = int32_t(max_context / DSA_PAGE_TOKENS);
    p.batch = batch;
    p.tokens = next_n;
    p.groups = groups;
    p.merge_by_cut = batch > groups ? 1 : 0;
    p.sm_scale_log2 = sm_scale * 1.4426950408889634f;
    e = dsa::launch_mla_dense(q_map, kv_map, kr_map, o_map, p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "MLA decode launch");
}

size_t dsa_mla_prefill_workspace_size(void) {
    int sms = 0;
    if (sm_count(&sms) != cudaSuccess) sms = 160;  // no device: what a large part needs
    return dsa::kWorkspaceHeaderBytes + dsa::prefill_split_bytes(sms);
}

dsa_status_t dsa_mla_prefill(const void* q, int64_t q_row_stride, int64_t q_head_stride, const void* k_nope,
                             int64_t k_row_stride, int64_t k_head_stride, const void* k_rope, int64_t k_rope_stride,
                             const void* v, int64_t v_row_stride, int64_t v_head_stride, const int32_t* cu_q,
                             const int32_t* cu_kv, const int32_t* seq_lens, int32_t batch, int32_t heads,
                             int64_t q_rows, int64_t kv_rows, int32_t entry_tokens, float sm_scale, void* out,
                             float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    if (batch < 1 || heads < 1 || q_rows < 0 || kv_rows < 0 || entry_tokens < 1) return DSA_ERR_INVALID_ARG;
    if (batch > DSA_MAX_BATCH || heads > DSA_PREFILL_MAX_HEADS || entry_tokens > 64 || q_rows > INT32_MAX ||
        kv_rows > INT32_MAX)
        return DSA_ERR_UNSUPPORTED;
    if (!std::isfinite(sm_scale) || sm_scale < 0.f) return DSA_ERR_INVALID_ARG;
    const int64_t slots = dsa::prefill_slots(q_rows, batch);
    if (2 * dsa::prefill_most_units(slots, heads) > INT32_MAX) return DSA_ERR_UNSUPPORTED;
    if (!cu_q || !cu_kv || !seq_lens || !aligned(cu_q, 4) || !aligned(cu_kv, 4) || !aligned(seq_lens, 4))
        return DSA_ERR_INVALID_ARG;
    if (q_rows > 0 && (!q || !out || !lse || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4)))
        return DSA_ERR_INVALID_ARG;
    if (kv_rows > 0 && (!k_nope || !k_rope || !v || !aligned(k_nope, 16) || !aligned(k_rope, 16) || !aligned(v, 16)))
        return DSA_ERR_INVALID_ARG;
    // A dimension of size 1 has no stride to speak of.
    if (heads == 1) q_head_stride = k_head_stride = v_head_stride = DSA_PREFILL_QK_DIM;
    if (q_rows <= 1) q_row_stride = DSA_PREFILL_QK_DIM;
    if (kv_rows <= 1) k_row_stride = k_rope_stride = v_row_stride = DSA_PREFILL_QK_DIM;
    for (int64_t s : {q_row_stride, q_head_stride, k_row_stride, k_head_stride, k_rope_stride, v_row_stride,
                      v_head_stride})
        if (s < 1 || s % 8 != 0 || s >= (int64_t(1) << 39)) return DSA_ERR_INVALID_ARG;
    dsa_status_t st = check_workspace(workspace, workspace_bytes, DSA_PREFILL_WORKSPACE_BYTES);
    if (st != DSA_OK) return st;
    if (q_rows == 0) return DSA_OK;
    dsa::PrefillMaps m;
    st = make_heads_map(&m.q, q, q_rows, heads, DSA_PREFILL_QK_DIM, q_row_stride, q_head_stride, 128, "prefill q");
    if (st != DSA_OK) return st;
    if (kv_rows > 0) {
        for (uint32_t few : {0u, 16u}) {  // whole tiles, and the 16 entries that the last ones are loaded by
            st = make_heads_map(few ? &m.kn16 : &m.kn, k_nope, kv_rows, heads, DSA_PREFILL_NOPE_DIM, k_row_stride,
                                k_head_stride, few ? few : 64, "prefill k_nope");
            if (st != DSA_OK) return st;
            st = make_heads_map(few ? &m.v16 : &m.v, v, kv_rows, heads, DSA_PREFILL_V_DIM, v_row_stride, v_head_stride,
                                few ? few : 128, "prefill v");
            if (st != DSA_OK) return st;
            st = make_rows_map(few ? &m.kr16 : &m.kr, k_rope, kv_rows, DSA_PREFILL_ROPE_DIM, few ? few : 64,
                               "prefill k_rope", k_rope_stride);
            if (st != DSA_OK) return st;
        }
    } else {
        m.kn = m.kr = m.v = m.kn16 = m.kr16 = m.v16 = m.q;  // no entry: the kernel loads none
    }
    dsa::PrefillParams p{};
    p.cu_q = cu_q;
    p.cu_kv = cu_kv;
    p.seq_lens = seq_lens;
    p.out = static_cast<__nv_bfloat16_raw*>(out);
    p.lse = lse;
    p.err = static_cast<uint32_t*>(workspace);
    p.q_rows = int32_t(q_rows);
    p.kv_rows = int32_t(kv_rows);
    p.batch = batch;
    p.heads = heads;
    p.entry_tokens = entry_tokens;
    p.slots = int32_t(slots);
    p.out_aligned32 = aligned(out, 32) ? 1 : 0;
    // A scale of 0 becomes one whose products vanish next to 1: hidden scores stay -inf times it.
    p.sm_scale_log2 = std::fmax(sm_scale * 1.4426950408889634f, 1e-30f);
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return cuda_fail(e, "device query");
    if (workspace_bytes >= dsa::kWorkspaceHeaderBytes + dsa::prefill_split_bytes(sms)) {
        uint8_t* ws = static_cast<uint8_t*>(workspace) + dsa::kWorkspaceHeaderBytes;
        p.split = reinterpret_cast<int2*>(ws);
        p.split_units = reinterpret_cast<dsa::SplitUnit*>(ws + 16);
        p.o_part = reinterpret_cast<float*>(ws + dsa::prefill_part_offset(sms));
        p.lse_part = p.o_part + dsa::prefill_max_parts(sms) * dsa::kPrefillBlock * DSA_PREFILL_V_DIM;
    }
    e = dsa::launch_mla_prefill(m, p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "MLA prefill launch");
}

size_t dsa_mla_tree_decode_workspace_size(int32_t batch, int32_t tokens) {
    int sms = 0, quads = 0, pairs = 0;
    if (batch < 1 || batch > DSA_MAX_BATCH || tokens < 1 || tokens > DSA_MAX_TREE_TOKENS) return 0;
    if (sm_count(&sms) != cudaSuccess || dsa::mla_tree_quads(&quads) != cudaSuccess ||
        dsa::mla_tree_pairs(&pairs) != cudaSuccess)
        sms = 160, quads = 40, pairs = 80;  // no device: what a large part needs
    return TreeShape(tokens, sms, quads, pairs).workspace_bytes(tokens);
}

dsa_status_t dsa_mla_tree_decode(const void* q, const void* kv_cache, int64_t num_pages, const int32_t* page_table,
                                 const int32_t* seq_lens, const void* draft_kv, const uint64_t* tree_mask,
                                 const int32_t* token_counts_opt, int32_t batch, int32_t tokens, int64_t max_context,
                                 float sm_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    dsa_status_t st = check_shape(batch, max_context);
    if (st != DSA_OK) return st;
    if (tokens < 1) return DSA_ERR_INVALID_ARG;
    if (tokens > DSA_MAX_TREE_TOKENS) return DSA_ERR_UNSUPPORTED;
    if (!q || !kv_cache || !page_table || !seq_lens || !draft_kv || !tree_mask || !out || !lse)
        return DSA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(draft_kv, 16) || !aligned(page_table, 4) ||
        !aligned(seq_lens, 4) || !aligned(token_counts_opt, 4) || !aligned(tree_mask, 8) || !aligned(out, 16) ||
        !aligned(lse, 4))
        return DSA_ERR_INVALID_ARG;
    if (num_pages < 1 || num_pages > kMaxPages || !std::isfinite(sm_scale)) return DSA_ERR_INVALID_ARG;
    // The tile loads address cache rows with 32-bit coordinates.
    if (num_pages > (int64_t(1) << 31) / dsa::kPageEntries - 1) return DSA_ERR_UNSUPPORTED;
    st = check_workspace(workspace, workspace_bytes, dsa::kWorkspaceHeaderBytes);
    if (st != DSA_OK) return st;
    int sms = 0, quads = 0, pairs = 0;
    cudaError_t e = sm_count(&sms);
    if (e == cudaSuccess) e = dsa::mla_tree_quads(&quads);
    if (e == cudaSuccess) e = dsa::mla_tree_pairs(&pairs);
    if (e != cudaSuccess) return cuda_fail(e, "device query");
    const TreeShape shape(tokens, sms, quads, pairs);
    st = check_workspace(workspace, workspace_bytes, shape.workspace_bytes(tokens));
    if (st != DSA_OK) return st;
    uint8_t* ws = static_cast<uint8_t*>(workspace) + dsa::kWorkspaceHeaderBytes;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const int64_t q_rows = int64_t(batch) * tokens * DSA_MLA_HEADS, kv_rows = num_pages * dsa::kPageEntries;
    dsa::MlaDenseParams p{};
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.out = static_cast<__nv_bfloat16_raw*>(out);
    p.lse = lse;
    p.cuts = reinterpret_cast<int32_t*>(ws + TreeShape::kDenseAt);
    p.plan = reinterpret_cast<int2*>(ws + TreeShape::kDenseAt + kDenseCutBytes);
    p.again = reinterpret_cast<uint32_t*>(ws + TreeShape::kAgainAt);
    p.o_part = reinterpret_cast<float*>(ws + TreeShape::kTreePlanBytes);
    p.lse_part = p.o_part + shape.parts(tokens) * dsa::kMlaHeads * dsa::kMlaDv;
    p.err = static_cast<uint32_t*>(workspace);
    p.flags = p.err + dsa::kAgainWord;
    p.ticket = p.err + dsa::kTicketWord;
    p.num_pages = num_pages;
    p.max_context = max_context;
    p.table_width = int32_t(max_context / DSA_PAGE_TOKENS);
    p.batch = batch;
    p.tokens = tokens;
    p.groups = shape.groups;
    p.merge_by_cut = batch > shape.groups ? 1 : 0;
    p.sm_scale_log2 = sm_scale * 1.4426950408889634f;
    p.mask = tree_mask;
    p.counts = token_counts_opt;
    if (tokens >= dsa::kPairTokens && int64_t(batch) * tokens * max_context > kTreeWork &&
        (tokens > dsa::kPairTokens || max_context > kPairContext) &&
        shape.ranges * shape.tiles <= dsa::kTreeMaxRounds * shape.clusters &&
        shape.ranges * shape.tiles <= dsa::kTreeMaxUnits) {
        dsa::MlaTreeParams t{};
        t.q = static_cast<const __nv_bfloat16_raw*>(q);
        t.page_table = page_table;
        t.seq_lens = seq_lens;
        t.mask = tree_mask;
        t.counts = token_counts_opt;
        t.out = p.out;
        t.lse = lse;
        t.plan = reinterpret_cast<int2*>(ws + TreeShape::kCutBytes);
        t.cuts = reinterpret_cast<int32_t*>(ws);
        t.o_part = p.o_part;
        t.lse_part = p.lse_part;
        t.err = p.err;
        t.flags = p.flags;
        t.num_pages = num_pages;
        t.max_context = max_context;
        t.table_width = p.table_width;
        t.batch = batch;
        t.tokens = tokens;
        t.tiles = shape.tiles;
        t.ranges = shape.ranges;
        t.sm_scale_log2 = p.sm_scale_log2;
        dsa::MlaTreeMaps m;
        if (tokens == dsa::kPairTokens) {
            st = make_slabs_map(&m.q, q, q_rows, 3, "mla q");
            if (st == DSA_OK) st = make_rows_map(&m.k, kv_cache, kv_rows, DSA_MLA_DIM, 64, "mla kv");
            if (st == DSA_OK) st = make_slabs_map(&m.v, kv_cache, kv_rows, 2, "mla kv");
            if (st == DSA_OK) st = make_drafts_map(&m.d, draft_kv, batch, tokens, 64);
            if (st != DSA_OK) return st;
            e = dsa::launch_mla_tree_pair(m, t, pairs, cs);
            return e == cudaSuccess ? DSA_OK : cuda_fail(e, "MLA tree decode launch");
        }
        st = make_slabs_map(&m.q, q, q_rows, 1, "mla q", 128);
        if (st == DSA_OK) st = make_slabs_map(&m.k, kv_cache, kv_rows, 3, "mla kv", 32);
        if (st == DSA_OK) st = make_slabs_map(&m.v, kv_cache, kv_rows, 2, "mla kv");
        if (st == DSA_OK) st = make_drafts_map(&m.d, draft_kv, batch, tokens, 32);
        if (st == DSA_OK) st = make_rows_map(&m.o, out, q_rows, DSA_MLA_DV, 64, "mla out");
        if (st != DSA_OK) return st;
        e = dsa::launch_mla_tree(m, t, quads, cs);
        if (e != cudaSuccess) return cuda_fail(e, "MLA tree decode launch");
        p.redo = 1;
        p.first = {t.plan, t.cuts, t.o_part, t.lse_part, shape.ranges};
        p.o_part += shape.tiled_parts(tokens) * dsa::kMlaHeads * dsa::kMlaDv;
        p.lse_part += shape.tiled_parts(tokens) * dsa::kMlaHeads;
    }
    CUtensorMap q_map, kv_map, kr_map, o_map, d_map;
    st = make_slabs_map(&q_map, q, q_rows, 3, "mla q");
    if (st == DSA_OK) st = make_slabs_map(&kv_map, kv_cache, kv_rows, 2, "mla kv");
    if (st == DSA_OK) st = make_rows_map(&kr_map, kv_cache, kv_rows, DSA_MLA_DIM, 64, "mla kv");
    if (st == DSA_OK) st = make_rows_map(&o_map, out, q_rows, DSA_MLA_DV, 64, "mla out");
    if (st == DSA_OK) st = make_drafts_map(&d_map, draft_kv, batch, tokens, 64);
    if (st != DSA_OK) return st;
    e = dsa::launch_mla_dense_tree(q_map, kv_map, kr_map, o_map, d_map, p, cs);
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "MLA tree decode launch");
}

dsa_status_t dsa_pages_update(const int32_t* seq_lens, const int32_t* new_lens, int32_t batch, int64_t max_context,
                              int32_t* page_table, int32_t* free_pages, int64_t num_pages, const int32_t* free_count,
                              int64_t max_slots, int32_t* seq_lens_out, int32_t* free_count_out, int32_t* cu_slots,
                              int64_t* slots, int32_t* positions, void* workspace, size_t workspace_bytes,
                              void* stream) {
    dsa_status_t st = check_shape(batch, max_context);
    if (st != DSA_OK) return st;
    if (!seq_lens || !new_lens || !page_table || !free_pages || !free_count || !seq_lens_out || !free_count_out ||
        !cu_slots || max_slots < 0 || (max_slots > 0 && (!slots || !positions)))
        return DSA_ERR_INVALID_ARG;
    for (const void* a : {static_cast<const void*>(seq_lens), static_cast<const void*>(new_lens),
                          static_cast<const void*>(page_table), static_cast<const void*>(free_pages),
                          static_cast<const void*>(free_count), static_cast<const void*>(seq_lens_out),
                          static_cast<const void*>(free_count_out), static_cast<const void*>(cu_slots)})
        if (!aligned(a, 4)) return DSA_ERR_INVALID_ARG;
    if (!aligned(slots, 16) || !aligned(positions, 16)) return DSA_ERR_INVALID_ARG;
    if (num_pages < 1 || num_pages > kMaxPages) return DSA_ERR_INVALID_ARG;
    if (max_slots > kMaxPages) return DSA_ERR_UNSUPPORTED;
    st = check_workspace(workspace, workspace_bytes, dsa::kWorkspaceHeaderBytes);
    if (st != DSA_OK) return st;
    dsa::PagesParams p{};
    p.seq_lens = seq_lens;
    p.new_lens = new_lens;
    p.page_table = page_table;
    p.free_pages = free_pages;
    p.free_count = free_count;
    p.seq_lens_out = seq_lens_out;
    p.free_count_out = free_count_out;
    p.cu_slots = cu_slots;
    p.slots = slots;
    p.positions = positions;
    p.err = static_cast<uint32_t*>(workspace);
    p.ticket = p.err + dsa::kTicketWord;
    p.in_place = seq_lens_out == seq_lens || seq_lens_out == new_lens || free_count_out == free_count;
    p.num_pages = num_pages;
    p.max_context = max_context;
    p.max_slots = max_slots;
    p.table_width = int32_t(max_context / DSA_PAGE_TOKENS);
    p.batch = batch;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return cuda_fail(e, "device query");
    e = dsa::launch_pages_update(p, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "page update launch");
}

dsa_status_t dsa_cache_append(const int64_t* slots, int64_t rows, const void* latent_opt, int64_t latent_stride,
                              const void* latent_weight_opt, int32_t latent_weight_fp32, const float* cos_sin_opt,
                              int64_t cos_rows, const int32_t* positions, void* kv_cache, const void* index_keys_opt,
                              int64_t key_stride, const void* index_weight_opt, int32_t index_weight_fp32,
                              void* key_pool_opt, void* key_codes_opt, float* key_scales_opt, int64_t num_pages,
                              float eps, void* workspace, size_t workspace_bytes, void* stream) {
    const auto flag = [](int32_t v) { return v == 0 || v == 1; };
    if (rows < 0 || num_pages < 1 || num_pages > kMaxPages || !std::isfinite(eps) || eps < 0.f ||
        !flag(latent_weight_fp32) || !flag(index_weight_fp32))
        return DSA_ERR_INVALID_ARG;
    if (rows > INT32_MAX) return DSA_ERR_UNSUPPORTED;
    if (rows == 0) return DSA_OK;
    // What each part comes with.
    if (!slots || (!latent_opt && !index_keys_opt)) return DSA_ERR_INVALID_ARG;
    if (latent_opt && !kv_cache) return DSA_ERR_INVALID_ARG;
    if (!latent_opt && (kv_cache || latent_weight_opt || cos_sin_opt)) return DSA_ERR_INVALID_ARG;
    if (cos_sin_opt && (cos_rows < 1 || !positions)) return DSA_ERR_INVALID_ARG;
    if ((key_codes_opt == nullptr) != (key_scales_opt == nullptr) || (key_pool_opt && key_codes_opt))
        return DSA_ERR_INVALID_ARG;
    if (index_keys_opt ? !key_pool_opt && !key_codes_opt : key_pool_opt || key_codes_opt || index_weight_opt)
        return DSA_ERR_INVALID_ARG;
    if (rows == 1) latent_stride = DSA_MLA_DIM, key_stride = DSA_HEAD_DIM;  // no second row: no stride
    if ((latent_opt && (latent_stride < 0 || latent_stride % 8 != 0)) ||
        (index_keys_opt && (key_stride < 0 || key_stride % 2 != 0)))
        return DSA_ERR_INVALID_ARG;
    if (!aligned(slots, 8) || !aligned(latent_opt, 16) || !aligned(kv_cache, 16) || !aligned(index_keys_opt, 4) ||
        !aligned(key_pool_opt, 4) || !aligned(key_codes_opt, 2) || !aligned(key_scales_opt, 4) ||
        !aligned(cos_sin_opt, 4) || !aligned(positions, 4) ||
        !aligned(latent_weight_opt, latent_weight_fp32 ? 4 : 2) ||
        !aligned(index_weight_opt, index_weight_fp32 ? 4 : 2))
        return DSA_ERR_INVALID_ARG;
    dsa_status_t st = check_workspace(workspace, workspace_bytes, dsa::kWorkspaceHeaderBytes);
    if (st != DSA_OK) return st;
    dsa::AppendParams p{};
    p.slots = slots;
    p.latent = static_cast<const uint8_t*>(latent_opt);
    p.latent_weight = latent_weight_opt;
    p.cos_sin = cos_sin_opt;
    p.positions = positions;
    p.keys = static_cast<const uint8_t*>(index_keys_opt);
    p.key_weight = index_weight_opt;
    p.kv_cache = static_cast<uint8_t*>(kv_cache);
    p.key_pool = static_cast<uint8_t*>(key_pool_opt);
    p.key_codes = static_cast<uint8_t*>(key_codes_opt);
    p.key_scales = key_scales_opt;
    p.err = static_cast<uint32_t*>(workspace);
    p.rows = rows;
    p.latent_stride = latent_stride;
    p.key_stride = key_stride;
    p.cos_rows = cos_rows;
    p.num_pages = num_pages;
    p.latent_weight_fp32 = latent_weight_fp32;
    p.key_weight_fp32 = index_weight_fp32;
    p.eps = eps;
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return cuda_fail(e, "device query");
    e = dsa::launch_append(p, sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? DSA_OK : cuda_fail(e, "cache append launch");
}

}  // extern "C"
