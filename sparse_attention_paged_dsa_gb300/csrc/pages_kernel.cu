// pages_kernel.cu -- page tables, lengths, free pages and slots of a batch, from
// its lengths now and those wanted.
//
// Request b goes from n to w tokens (256 a page, 4 an entry).  With w < n its last
// pages return to the top of the stack of free pages; with w > n it takes pages
// from the top and its new entries [n / 4, ceil(w / 4)) get slots (page x 64 + entry
// in page).  Requests are served in order, the returned pages of all of them first;
// one that grows is left as it was when the pages or the room for slots end, and so
// is each later one that grows.
//
// With the prefix sums of pages returned, pages taken and entries (at most 1024
// requests: every CTA forms all of them), everything else is independent: the k-th
// page taken is number avail - 1 - k of the stack, where positions from the old count
// on are the returned pages, found in the tables by a search in the prefix sums.
// Reads and writes meet nowhere: the stack is written from the old count on and read
// below it, table rows are written behind their old pages only.  Lengths and the
// count, where they are updated in place, are written by the last CTA to finish
// (a ticket in the workspace header, which it sets back).  Nothing depends on the
// order of the CTAs.
//
// What bounds it: latency (a chain of the lengths, the scan, a page id and a store).  64 requests with one
// to four tokens more: 4.9 us; 257 that end, grow and arrive, 22,000 slots: 7.2 (9.2 with
// one kind of work after another and a ticket each time); 1024 prompts, 224,000 slots: 6.3.
#include <cuda_runtime.h>

#include <cstdint>

#include "indexer_kernels.h"
#include "sm103_ptx.cuh"

namespace dsa {
namespace {

constexpr int kThreadsPg = 512;
constexpr int kWarpsPg = kThreadsPg / 32;
constexpr int kReqs = kMaxBatch / kThreadsPg;  // requests a thread
static_assert(kReqs * kThreadsPg == kMaxBatch, "every request has a thread");
constexpr int kRun = 4;                        // consecutive slots a thread

// Pages taken (low half) and returned (high half) of a request or before it; below 2^27 together.
__device__ __forceinline__ uint64_t pair_of(int take, int give) {
    return uint64_t(uint32_t(give)) << 32 | uint32_t(take);
}

struct PagesShared {
    int take[kMaxBatch + 1], give[kMaxBatch + 1];  // prefix sums; of pages taken, those of requests served
    int slot[kMaxBatch + 1];                       // first slot, the same
    int now[kMaxBatch], want[kMaxBatch];
    uint64_t warp_pages[kWarpsPg];
    int64_t warp_slots[kWarpsPg];
    int refused;                                   // the first request that is not served
    int last;
};

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + 255) >> 8; }

// The last i in [0, n) with start[i] <= at, for start[0] <= at: the owner of number `at` (those without any
// share their start with the next).
__device__ __forceinline__ int owner(const int* start, int n, int at) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        (start[mid] <= at ? lo : hi) = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreadsPg) pages_update_kernel(const PagesParams p) {
    __shared__ PagesShared s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait_prior_grid();
    pdl_allow_next_grid();

    uint32_t bad = 0;
    const auto length = [&](int v) {
        if (v < 0 || int64_t(v) > p.max_context) bad |= kErrSeqLenClamped;
        return v < 0 ? 0 : (int64_t(v) > p.max_context ? int(p.max_context) : v);
    };
    if (tid == 0) s.refused = p.batch;
    uint64_t pages = 0;
    int64_t slots = 0;
#pragma unroll
    for (int i = 0; i < kReqs; ++i) {
        const int b = tid * kReqs + i;
        if (b >= p.batch) break;
        const int n = length(p.seq_lens[b]), w = length(p.new_lens[b]);  // (may be written below: no ld.global.nc)
        s.now[b] = n;
        s.want[b] = w;
        const int d = pages_of(w) - pages_of(n);
        pages += pair_of(max(d, 0), max(-d, 0));
        if (w > n) slots += ((w + 3) >> 2) - (n >> 2);
    }
    uint64_t pages_to = pages;
    int64_t slots_to = slots;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t a = __shfl_up_sync(0xffffffffu, pages_to, o);
        const int64_t c = __shfl_up_sync(0xffffffffu, slots_to, o);
        if (lane >= o) pages_to += a, slots_to += c;
    }
    if (lane == 31) s.warp_pages[warp] = pages_to, s.warp_slots[warp] = slots_to;
    __syncthreads();
    uint64_t pages_all = 0;
    pages_to -= pages;  // before this thread's requests
    slots_to -= slots;
#pragma unroll
    for (int w = 0; w < kWarpsPg; ++w) {
        if (w < warp) pages_to += s.warp_pages[w], slots_to += s.warp_slots[w];
        pages_all += s.warp_pages[w];
    }
    int count = *p.free_count;
    if (count < 0 || int64_t(count) > p.num_pages) {
        bad |= kErrBadRange;
        count = count < 0 ? 0 : int(p.num_pages);
    }
    const int returned = int(pages_all >> 32);
    const int64_t avail64 = int64_t(count) + returned;
    if (avail64 > p.num_pages) bad |= kErrBadRange;  // more pages than there are
    const int avail = int(avail64 < p.num_pages ? avail64 : p.num_pages);
#pragma unroll
    for (int i = 0; i < kReqs; ++i) {
        const int b = tid * kReqs + i;
        if (b > p.batch) break;
        // (no slot past the room is ever used: its number is cut, so that it stays in 32 bits)
        s.take[b] = int(uint32_t(pages_to));
        s.give[b] = int(pages_to >> 32);
        s.slot[b] = int(slots_to < p.max_slots ? slots_to : p.max_slots);
        if (b == p.batch) break;
        const int n = s.now[b], w = s.want[b], d = pages_of(w) - pages_of(n);
        pages_to += pair_of(max(d, 0), max(-d, 0));
        if (w > n) {
            slots_to += ((w + 3) >> 2) - (n >> 2);
            if (int(uint32_t(pages_to)) > avail || slots_to > p.max_slots) atomicMin(&s.refused, b);
        }
        if (b + 1 == kMaxBatch) {  // (no thread has a request of this number)
            s.take[kMaxBatch] = int(uint32_t(pages_to));
            s.give[kMaxBatch] = int(pages_to >> 32);
            s.slot[kMaxBatch] = int(slots_to < p.max_slots ? slots_to : p.max_slots);
        }
    }
    __syncthreads();
    const int refused = s.refused;  // what grows from here on is not served
    if (refused < p.batch) {
        bad |= kErrNoPages;
        const int take = s.take[refused], slot = s.slot[refused];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kReqs; ++i) {
            const int b = tid * kReqs + i + 1;
            if (b <= refused || b > p.batch) continue;
            s.take[b] = take;
            s.slot[b] = slot;
        }
        __syncthreads();
    }
    const int taken = s.take[p.batch], total = s.slot[p.batch], left = avail - taken;
    const int64_t first = int64_t(blockIdx.x) * kThreadsPg + tid, step = int64_t(gridDim.x) * kThreadsPg;

    // Page number `at` of the stack before pages are taken, -1 if it is none.
    const auto stack = [&](int at) {
        int page;
        if (at < count) {
            page = p.free_pages[at];
        } else {
            const int b = owner(s.give, p.batch, at - count);
            page = p.page_table[int64_t(b) * p.table_width + pages_of(s.want[b]) + (at - count - s.give[b])];
        }
        if (page >= 0 && int64_t(page) < p.num_pages) return page;
        bad |= kErrBadPage;
        return -1;
    };
    // What there is to do, one after another over all threads, so that a small call's chains of loads run side by
    // side: runs of slots, pages taken, and returned pages that stay.
    const int64_t runs = (p.max_slots + kRun - 1) / kRun, stays = left > count ? left - count : 0;
    for (int64_t job = first; job < runs + taken + stays; job += step) {
        if (job >= runs + taken) {
            const int64_t to = count + (job - runs - taken);
            p.free_pages[to] = stack(int(to));
            continue;
        }
        if (job >= runs) {
            const int k = int(job - runs), b = owner(s.take, p.batch, k);
            p.page_table[int64_t(b) * p.table_width + pages_of(s.now[b]) + (k - s.take[b])] = stack(avail - 1 - k);
            continue;
        }
        const int64_t i0 = kRun * job;
        int64_t slot[kRun];
        int pos[kRun];
        int b = i0 < total ? owner(s.slot, p.batch, int(i0)) : 0;
        int page_at = -1, page = -1;  // the page looked up last
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            const int64_t i = i0 + j;
            slot[j] = pos[j] = -1;
            if (i >= total) continue;
            if (i >= s.slot[b + 1]) {
                b = owner(s.slot, p.batch, int(i));
                page_at = -1;
            }
            const int entry = (s.now[b] >> 2) + int(i - s.slot[b]), w = entry >> 6, have = pages_of(s.now[b]);
            if (w != page_at) {
                page_at = w;
                if (w < have) {
                    page = p.page_table[int64_t(b) * p.table_width + w];
                    if (page < 0 || int64_t(page) >= p.num_pages) {
                        bad |= kErrBadPage;
                        page = -1;
                    }
                } else {
                    page = stack(avail - 1 - (s.take[b] + w - have));
                }
            }
            slot[j] = page < 0 ? -1 : int64_t(page) * kPageEntries + (entry & 63);
            pos[j] = entry;
        }
        if (i0 + kRun <= p.max_slots) {
            reinterpret_cast<longlong2*>(p.slots + i0)[0] = make_longlong2(slot[0], slot[1]);
            reinterpret_cast<longlong2*>(p.slots + i0)[1] = make_longlong2(slot[2], slot[3]);
            *reinterpret_cast<int4*>(p.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (int j = 0; j < kRun; ++j)
                if (i0 + j < p.max_slots) p.slots[i0 + j] = slot[j], p.positions[i0 + j] = pos[j];
        }
    }
    if (bad) atomicOr(p.err, bad);
    if (blockIdx.x == 0)
        for (int b = tid; b <= p.batch; b += kThreadsPg) p.cu_slots[b] = s.slot[b];

    // Updated in place: by the last CTA to get here, when nobody reads the lengths or the count any more.
    if (!p.in_place) {
        if (blockIdx.x != 0) return;
    } else if (gridDim.x > 1) {
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            s.last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
            if (s.last) *p.ticket = 0;
        }
        __syncthreads();
        if (!s.last) return;
        __threadfence();
    } else {
        __syncthreads();
    }
    for (int b = tid; b < p.batch; b += kThreadsPg)
        p.seq_lens_out[b] = b >= refused && s.want[b] > s.now[b] ? s.now[b] : s.want[b];
    if (tid == 0) *p.free_count_out = left;
}

}  // namespace

cudaError_t launch_pages_update(const PagesParams& p, int sms, cudaStream_t stream) {
    // A CTA for every 2,048 slots or 8,192 pages: fewer would be waited for, and one alone needs no ticket.
    const int64_t by_slots = (p.max_slots + kThreadsPg * kRun - 1) / (kThreadsPg * kRun);
    const int64_t by_pages = (p.num_pages + 16 * kThreadsPg - 1) / (16 * kThreadsPg);
    const int64_t ctas = by_slots > by_pages ? by_slots : by_pages;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(ctas < 1 ? 1 : (ctas > sms ? sms : ctas)));
    cfg.blockDim = dim3(kThreadsPg);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pages_update_kernel, p);
}

}  // namespace dsa
