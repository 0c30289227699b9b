// Device code shared by the tree-verification kernels: a token's request, a
// request's nodes, and cached slots' addresses.
#pragma once

#include <stdint.h>

#include "ple_tree_internal.h"

namespace ple {
namespace {

// Every kernel of the library waits for the grid before it in the stream
// before its first global access (see launch_kernel).
__device__ __forceinline__ void wait_grid_before() { cudaGridDependencySynchronize(); }

// Request r's nodes [begin, end), within [0, T) whatever cu_seqlens holds.
__device__ __forceinline__ void request_nodes(const int32_t* __restrict__ cu, int r, int64_t T,
                                              int32_t& begin, int32_t& end) {
    begin = (int32_t)min((int64_t)max(__ldg(cu + r), 0), T);
    end = (int32_t)min((int64_t)max(__ldg(cu + r + 1), begin), T);
}

// The last request r with cu[r] <= t, found by a whole warp for a uniform t:
// 32 probes a round, two rounds up to 1024 requests.  Reads cu[0..B-1] only.
__device__ __forceinline__ int warp_request(const int32_t* __restrict__ cu, int B, int64_t t,
                                            int lane) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int k = lo + lane * step;
        const unsigned m =
            __ballot_sync(0xffffffffu, k < hi && (int64_t)__ldg(cu + k) <= t);
        lo += (m ? 31 - __clz((int)m) : 0) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// The element offset of head 0 of cached token `slot` of request r, or -1
// where the page table has no page of the cache for it.
__device__ __forceinline__ int64_t slot_offset(const int32_t* __restrict__ table,
                                               int32_t max_pages, int32_t page_size,
                                               int64_t num_pages, int64_t page_stride,
                                               int64_t slot_stride, int r, int64_t slot) {
    if (slot < 0) return -1;
    const int64_t page_at = slot / page_size;
    if (page_at >= max_pages) return -1;
    const int32_t page = __ldg(table + (int64_t)r * max_pages + page_at);
    if (page < 0 || page >= num_pages) return -1;
    return page * page_stride + (slot - page_at * page_size) * slot_stride;
}

}  // namespace
}  // namespace ple
