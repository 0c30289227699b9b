// Pages of a cache, on sm_103a: the commit of accepted branches from block to block of
// a cache in 8 bits, the plan of the next step's page tables, and the copy of pages.
#include "ple_fp8.cuh"
#include "ple_tree_common.cuh"
#include "ple_tree_fp8_internal.h"

namespace ple {
namespace {

// ------------------------------------------------------------------- commit

// Threads of a block: a warp a head where few blocks run, and their latency is the call's;
// two warps where they fill the device several times over.  One branch in one layer of 8
// heads 3.6 us with 256 threads (7.1 with 64); 64 branches in 16 layers 14.5 us with 64
// (16.6 with 256).
constexpr int kCommitThreads = 256, kManyCommitThreads = 64;
constexpr int kCommitAhead = 4;    // rows of a lane in flight
// resident blocks of 256 threads, or as many threads: with more registers 64 branches in 16
// layers take 18 us
constexpr int kCommitBlocks = 4;

// Sixteen elements kept under a scale `under` of at most `top`, which is no power of two, as a
// cache may have been filled with.  The quotient is taken in two parts: its first 20 bits, a
// little low, and what they lack.  A call, so that its registers are not the common path's.
__device__ __noinline__ uint4 odd_elements(uint4 x, float under, float top) {
    const float to_one = scale_to_one(top);
    under *= to_one;
    top *= to_one;
    const float inv = 1.0f / top;
    const float f = __uint_as_float((max(__float_as_uint(under * inv), 16u) - 8) & ~15u);
    const float rest = fmaf(-f, top, under) * inv;
    return make_uint4(scaled_elements(x.x, f, rest), scaled_elements(x.y, f, rest),
                      scaled_elements(x.z, f, rest), scaled_elements(x.w, f, rest));
}

// The accepted rows of one request, one layer and one cache move to the front of the
// tree's slots, block by block of slots under one scale: what a block will hold is
// known first (from which slot each row comes), then a warp takes a head, finds the
// largest of the rows' scales, and moves its rows some at a time, elements scaled to
// it.  Row j comes from node path[j] >= j, so no later source lies below a block that
// was written, nor below a row that was.  Bound by latencies: a few dependent reads a
// block (64 branches in 16 layers move 15 MB in 14.5 us).
__global__ void __launch_bounds__(kCommitThreads, kCommitBlocks)
tree_commit_fp8_kernel(const __grid_constant__ ple_tree_commit_fp8_args f, const int shift) {
    __shared__ int64_t from_s[kMostBlock], scale_s[kMostBlock];
    wait_grid_before();
    const ple_tree_commit_args& a = f.base;
    const int r = blockIdx.x, layer = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t begin, end;
    request_nodes(a.cu_seqlens, r, a.num_tokens, begin, end);
    const int n = end - begin;
    const int kept = min(min(max(__ldg(a.accepted + r), 0), a.path_len), n);
    const int64_t ctx = __ldg(a.ctx_lens + r);
    const int32_t* path = a.path + (int64_t)r * a.path_len;

    if (layer == 0 && blockIdx.z == 0) {
        if (threadIdx.x == 0) a.next_ctx_lens[r] = (int32_t)(ctx + kept);
        if (a.ngram_context != nullptr && threadIdx.x < a.ctx_len) {
            // id number kept + i of (context row, accepted ids)
            const int C = a.ctx_len;
            const int i = kept + threadIdx.x;
            const int64_t src =
                i < C ? (int64_t)r * C + i
                      : begin + (int64_t)min(max(__ldg(path + i - C), 0), max(n - 1, 0));
            const int64_t dst = (int64_t)r * C + threadIdx.x;
            const void* row = i < C ? a.ngram_context : a.input_ids;
            if (a.id_dtype == PLE_I64)
                static_cast<int64_t*>(a.next_context)[dst] = static_cast<const int64_t*>(row)[src];
            else
                static_cast<int32_t*>(a.next_context)[dst] = static_cast<const int32_t*>(row)[src];
        }
    }
    if (kept == 0 || ctx < 0) return;

    const int size = 1 << shift;
    const int lanes = a.head_dim >> 4;   // of 16 bytes a row, at most 16
    const int sub = lane % lanes, group = lane / lanes;
    const int rows_at_once = 32 / lanes;
    const bool working = group < rows_at_once;
    uint8_t* cache = static_cast<uint8_t*>(blockIdx.z == 0 ? a.k_cache : a.v_cache) +
                     layer * a.layer_stride;
    unsigned short* scales =
        static_cast<unsigned short*>(blockIdx.z == 0 ? f.scales.k : f.scales.v) +
        layer * f.scales.layer_stride;
    // a slot's place among the rows and among the scales; -1: it has none
    auto place = [&](int64_t slot, int64_t& scale_at) -> int64_t {
        const int64_t page_at = slot / a.page_size;
        if (page_at >= a.max_pages) return -1;
        const int32_t page = __ldg(a.page_table + (int64_t)r * a.max_pages + page_at);
        if (page < 0 || page >= a.num_pages) return -1;
        const int in_page = (int)(slot - page_at * a.page_size);
        scale_at = page * f.scales.page_stride + (in_page >> shift);
        return page * a.page_stride + in_page * a.slot_stride;
    };
    for (int64_t first = ctx & -(int64_t)size; first < ctx + kept; first += size) {
        const int live = (int)min((int64_t)size, ctx + kept - first);
        int64_t to_scale = 0;
        const int64_t to = place(first, to_scale);
        if (to < 0) continue;
        __syncthreads();
        for (int i = threadIdx.x; i < live; i += blockDim.x) {
            const int64_t slot = first + i;
            int64_t from = to + i * a.slot_stride, scale_at = to_scale;
            if (slot >= ctx) {
                const int j = (int)(slot - ctx), node = __ldg(path + j);
                if (node > j && node < n) {
                    int64_t s = 0;
                    const int64_t at = place(ctx + node, s);
                    if (at >= 0) {
                        from = at;
                        scale_at = s;
                    }
                }
            }
            from_s[i] = from;
            scale_s[i] = scale_at;
        }
        __syncthreads();
        for (int head = warp; head < a.kv_heads; head += blockDim.x / 32) {
            const unsigned short* head_scales = scales + head * f.scales.head_stride;
            float most = 0.f;
            for (int i = lane; i < live; i += 32)
                most = fmaxf(most, scale_value(head_scales[scale_s[i]]));
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1)
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
            // a quotient by a power of two, as every scale is that the library writes, is exact
            const bool odd = (__float_as_uint(most) & 0x7FFFFFu) != 0;
            uint8_t* rows = cache + head * a.head_stride + sub * 16;
            for (int i0 = 0; i0 < live; i0 += kCommitAhead * rows_at_once) {
                uint4 v[kCommitAhead];
                float by[kCommitAhead];   // below 0: the row stays
#pragma unroll
                for (int k = 0; k < kCommitAhead; ++k) {
                    const int i = i0 + k * rows_at_once + group;
                    by[k] = -1.f;
                    if (!working || i >= live) continue;
                    const float scale = scale_value(head_scales[scale_s[i]]);
                    if (from_s[i] == to + i * a.slot_stride && scale == most) continue;
                    by[k] = scale / most;
                    v[k] = *reinterpret_cast<const uint4*>(rows + from_s[i]);
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < kCommitAhead; ++k) {
                    const int i = i0 + k * rows_at_once + group;
                    if (by[k] < 0.f) continue;
                    uint4 x = v[k];
                    if (by[k] != 1.f && odd)
                        x = odd_elements(x, scale_value(head_scales[scale_s[i]]), most);
                    else if (by[k] != 1.f)
                        x = make_uint4(scaled_elements(x.x, by[k]), scaled_elements(x.y, by[k]),
                                       scaled_elements(x.z, by[k]), scaled_elements(x.w, by[k]));
                    *reinterpret_cast<uint4*>(rows + to + i * a.slot_stride) = x;
                }
                __syncwarp();
            }
            if (lane == 0)
                scales[head * f.scales.head_stride + to_scale] =
                    (unsigned short)(__float_as_uint(most) >> 16);
        }
    }
}

// --------------------------------------------------------------------- plan

constexpr int kPlanThreads = 1024;
constexpr int kPlanBlocks = 8;

// The workspace: for each page a byte whether it is carried unwritten and one whether a
// row writes it, the lowest row that does, the free pages by rank, and a moving page's
// rank; for each row the rank of its first new page and of its doubled one; each block's
// sums.
struct PlanSpace {
    uint8_t *carried, *written;
    int32_t *writer, *frees, *rank, *first_new, *first_double, *sums;
};

constexpr int kPlanChunk = 16;   // pages whose bytes a thread reads at once

__host__ __device__ inline int64_t plan_chunks(int64_t pages) {
    return (pages + kPlanChunk - 1) / kPlanChunk;
}

__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A row of the next tables.
struct PlanRow {
    int32_t source, ctx;
    int32_t held;      // entries that it carries
    int32_t need;      // entries that it will have
    int32_t written;   // the entry that new tokens are written to, or -1
};

__device__ __forceinline__ PlanRow plan_row(const ple_plan_pages_args& a, int64_t i) {
    PlanRow p;
    const int32_t s = __ldg(a.source + i);
    p.source = s >= 0 && s < a.num_requests ? s : -1;
    const int32_t most = a.max_pages * a.page_size;
    p.ctx = p.source < 0 ? 0 : min(max(__ldg(a.ctx_lens + p.source), 0), most);
    const int64_t want = max(__ldg(a.want + i), 0);
    p.held = (int32_t)(((int64_t)p.ctx + a.page_size - 1) / a.page_size);
    p.need = (int32_t)min((p.ctx + want + a.page_size - 1) / a.page_size, (int64_t)a.max_pages);
    p.written = want > 0 && p.ctx % a.page_size != 0 ? p.held - 1 : -1;
    return p;
}

// The page of an entry that a row carries, or -1.
__device__ __forceinline__ int32_t carried_page(const ple_plan_pages_args& a, const PlanRow& p,
                                                int32_t entry) {
    const int32_t page = __ldg(a.page_table + (int64_t)p.source * a.max_pages + entry);
    return page >= 0 && page < a.num_pages ? page : -1;
}

// Sums of `n` numbers a thread over the threads before it in the block; the block's in
// all[].
template <int N>
__device__ __forceinline__ void block_scan(int32_t (&v)[N], int32_t (&all)[N],
                                           int32_t (*scratch)[N]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t own[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        own[k] = v[k];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, v[k], d);
            if (lane >= d) v[k] += o;
        }
        if (lane == 31) scratch[warp][k] = v[k];
    }
    __syncthreads();
    if (warp == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            int32_t x = scratch[lane][k];
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t o = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += o;
            }
            scratch[lane][k] = x;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] += (warp ? scratch[warp - 1][k] : 0) - own[k];
        all[k] = scratch[31][k];
    }
}

// The bytes of a chunk's pages that are not 0, as bits.
__device__ __forceinline__ uint32_t byte_bits(const uint8_t* bytes, int64_t chunk) {
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(bytes) + chunk);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // bytes are 0 or 1: they add up in the product's top byte, each at its place
        bits |= (w[i] * 0x01020408u >> 24 & 0xF) << (4 * i);
    }
    return bits;
}

// One cluster of eight blocks, in phases with a barrier between them: rows mark the
// pages that they carry or write, a byte each; bytes are read sixteen at a time, pages and
// rows counted, each thread its part in order, and ranked; rows and copies are written.
// Every result follows from ranks, none from who came first.  A latency: four barriers, and
// a few dependent reads in each phase, eight entries of a row in flight a lane: 4 rows of one
// prompt 12.6 us; 256 requests of up to 512 pages in 130000, of which 20000 move, 39 us (77
// with a word a page for marks, read one by one).
__global__ void __cluster_dims__(kPlanBlocks, 1, 1) __launch_bounds__(kPlanThreads)
plan_pages_kernel(const __grid_constant__ ple_plan_pages_args a,
                  const __grid_constant__ PlanSpace space) {
    __shared__ int32_t scratch[32][5];
    const int block = blockIdx.x;
    const int64_t thread = (int64_t)block * kPlanThreads + threadIdx.x;
    constexpr int64_t kAll = (int64_t)kPlanBlocks * kPlanThreads;
    // a row's warp: rows spread over the blocks
    const int64_t warp = (int64_t)(threadIdx.x >> 5) * kPlanBlocks + block;
    const int lane = threadIdx.x & 31;
    const int64_t P = a.num_pages, N = a.num_rows;
    const int64_t copies = N + P - a.page_limit, chunks = plan_chunks(P);
    constexpr int kAhead = 8;

    wait_grid_before();
    // the first row of this warp, and of this thread
    PlanRow of_warp = {}, of_thread = {};
    if (warp < N) of_warp = plan_row(a, warp);
    const int64_t r0 = N * thread / kAll, r1 = N * (thread + 1) / kAll;
    if (r0 < r1) of_thread = plan_row(a, r0);
    for (int64_t c = thread; c < chunks; c += kAll) {
        reinterpret_cast<uint4*>(space.carried)[c] = make_uint4(0, 0, 0, 0);
        reinterpret_cast<uint4*>(space.written)[c] = make_uint4(0, 0, 0, 0);
    }
    for (int64_t i = r0; i < r1; ++i) {
        const PlanRow p = i == r0 ? of_thread : plan_row(a, i);
        a.next_ctx_lens[i] = p.ctx;
        if (p.written < 0) continue;
        const int32_t page = carried_page(a, p, p.written);
        if (page >= 0) space.writer[page] = INT32_MAX;
    }
    for (int64_t i = thread; i < 2 * copies; i += kAll) a.copies[i] = -1;
    if (thread == 0) a.counts[0] = 0;
    cluster_barrier();

    for (int64_t i = warp; i < N; i += kAll / 32) {
        const PlanRow p = i == warp ? of_warp : plan_row(a, i);
        for (int64_t e0 = lane; e0 < p.held; e0 += 32 * kAhead) {
            int32_t page[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                page[u] = p.held - e0 > 32 * u ? carried_page(a, p, (int32_t)e0 + 32 * u) : -1;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (page[u] < 0) continue;
                if (e0 + 32 * u == p.written) {
                    space.written[page[u]] = 1;
                    atomicMin(space.writer + page[u], (int32_t)i);
                } else {
                    space.carried[page[u]] = 1;
                }
            }
        }
    }
    cluster_barrier();

    // this thread's pages, in order
    auto part = [](int64_t n, int64_t k) { return n * k / kAll; };
    const int64_t c0 = part(chunks, thread), c1 = part(chunks, thread + 1);
    // of a chunk: pages in use, and those below the limit
    auto used = [&](int64_t c) {
        return byte_bits(space.carried, c) | byte_bits(space.written, c);
    };
    auto below = [&](int64_t c) {
        const int64_t n = a.page_limit - c * kPlanChunk;
        return n <= 0 ? 0u : n >= kPlanChunk ? 0xFFFFu : (1u << (int)n) - 1;
    };
    // whether row i keeps the page that it writes
    auto keeps = [&](int64_t i, int32_t page) {
        return page >= 0 && __ldcg(space.carried + page) == 0 && __ldcg(space.writer + page) == i;
    };
    // free pages, pages that move, pages in use; new pages, doubled pages
    int32_t mine[5] = {}, all[5];
    auto count_row = [&](int64_t i) {
        const PlanRow p = i == r0 ? of_thread : plan_row(a, i);
        mine[3] += max(p.need - p.held, 0);
        if (p.written >= 0) {
            const int32_t page = carried_page(a, p, p.written);
            if (!keeps(i, page)) {
                mine[3] += 1;
                mine[4] += page >= 0;
            }
        }
    };
    for (int64_t c = c0; c < c1; ++c) {
        const uint32_t u = used(c), low = below(c);
        mine[0] += __popc(~u & low);
        mine[1] += __popc(u & ~low);
        mine[2] += __popc(u);
    }
    for (int64_t i = r0; i < r1; ++i) count_row(i);
    block_scan(mine, all, scratch);
    if (threadIdx.x == 0) {
#pragma unroll
        for (int k = 0; k < 5; ++k) space.sums[block * 8 + k] = all[k];
    }
    cluster_barrier();

    int32_t total[5] = {};
#pragma unroll
    for (int b = 0; b < kPlanBlocks; ++b) {
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            const int32_t x = __ldcg(space.sums + b * 8 + k);
            if (b < block) mine[k] += x;
            total[k] += x;
        }
    }
    const int32_t room = total[0], moving = total[1], moved = min(moving, room);
    const int64_t asked = (int64_t)moving + total[3];
    for (int64_t c = c0; c < c1; ++c) {
        const uint32_t u = used(c), low = below(c);
        for (uint32_t left = ~u & low; left && mine[0] < asked; left &= left - 1)
            space.frees[mine[0]++] = (int32_t)(c * kPlanChunk) + __ffs((int)left) - 1;
        for (uint32_t left = u & ~low; left; left &= left - 1, ++mine[1]) {
            const int32_t page = (int32_t)(c * kPlanChunk) + __ffs((int)left) - 1;
            space.rank[page] = mine[1];
            if (mine[1] < room) a.copies[2 * (int64_t)mine[1]] = page;
        }
    }
    for (int64_t i = r0; i < r1; ++i) {
        space.first_new[i] = mine[3];
        space.first_double[i] = mine[4];
        count_row(i);
    }
    cluster_barrier();

    for (int64_t k = thread; k < moved; k += kAll) a.copies[2 * k + 1] = __ldcg(space.frees + k);
    for (int64_t i = warp; i < N; i += kAll / 32) {
        const PlanRow p = i == warp ? of_warp : plan_row(a, i);
        const int64_t fresh = (int64_t)moving + __ldcg(space.first_new + i);
        auto new_page = [&](int64_t k) {
            return fresh + k < room ? __ldcg(space.frees + fresh + k) : -1;
        };
        int32_t page = -1;
        bool renewed = false;
        if (p.written >= 0) {
            page = carried_page(a, p, p.written);
            renewed = !keeps(i, page);
        }
        for (int64_t e0 = lane; e0 < a.max_pages; e0 += 32 * kAhead) {
            int32_t to[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                to[u] = p.held - e0 > 32 * u ? carried_page(a, p, (int32_t)e0 + 32 * u) : -1;
            int32_t k[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                k[u] = to[u] >= a.page_limit ? __ldcg(space.rank + to[u]) : room;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (a.max_pages - e0 <= 32 * u) break;
                const int32_t e = (int32_t)e0 + 32 * u;
                if (k[u] < room) to[u] = __ldcg(space.frees + k[u]);
                if (e == p.written && renewed)
                    to[u] = new_page(0);
                else if (e >= p.held && e < p.need)
                    to[u] = new_page(e - p.held + renewed);
                a.next_table[i * a.max_pages + e] = to[u];
            }
        }
        if (lane == 0 && renewed && page >= 0 && new_page(0) >= 0) {
            const int64_t k = (int64_t)moved + __ldcg(space.first_double + i);
            a.copies[2 * k] = page;
            a.copies[2 * k + 1] = new_page(0);
            atomicAdd(a.counts, 1);
        }
    }
    if (thread == 0) {
        const int32_t taken = (int32_t)min(asked, (int64_t)room);
        atomicAdd(a.counts, moved);
        a.counts[1] = total[2] + taken - moved;
        a.counts[2] = (int32_t)(asked - taken);
    }
}

// --------------------------------------------------------------------- copy

constexpr int kCopyThreads = 256;
constexpr int kCopyAhead = 4;                               // 16-byte pieces of a thread
constexpr int kCopyPart = kCopyThreads * kCopyAhead;        // of a page, a block's share

// A block takes a share of 16 KB of one page of one layer's keys or values, for some of
// the copies in turn (as many blocks as keep the device busy, whatever the list's
// length), four pieces a thread in flight.  Bound by the pages' bytes: 97 pages of 256 KB in
// 48 layers, 2.4 GB moved, 364 us (6.7 TB/s, 99% of the measured copy); one page of one layer
// 2.5 us, a launch.
__global__ void __launch_bounds__(kCopyThreads)
copy_pages_kernel(const __grid_constant__ ple_copy_pages_args a, const int row_pieces,
                  const int parts, const int scale_blocks) {
    wait_grid_before();
    const int layer = blockIdx.y;
    const int part = blockIdx.z >> 1;
    const bool keys = !(blockIdx.z & 1);
    const int64_t bytes = a.element_bytes;
    uint8_t* cache = static_cast<uint8_t*>(keys ? a.k_cache : a.v_cache) +
                     layer * a.layer_stride * bytes;
    const int64_t pieces = (int64_t)a.kv_heads * a.page_size * row_pieces;
    // where this thread's pieces lie in a page
    int64_t at[kCopyAhead];
#pragma unroll
    for (int k = 0; k < kCopyAhead; ++k) {
        const int64_t i = (int64_t)part * kCopyPart + k * kCopyThreads + threadIdx.x;
        const int64_t row = i / row_pieces;
        const int64_t head = row / a.page_size;
        at[k] = i < pieces ? head * a.head_stride * bytes +
                                 (row - head * a.page_size) * a.slot_stride * bytes +
                                 (i - row * row_pieces) * 16
                           : -1;
    }
    for (int64_t base = 0; base < a.num_copies; base += (int64_t)gridDim.x * 32) {
        // a warp looks at 32 of this block's entries at a time
        const int64_t mine = base + (int64_t)(threadIdx.x & 31) * gridDim.x + blockIdx.x;
        int2 entry = make_int2(-1, -1);
        if (mine < a.num_copies) entry = __ldg(reinterpret_cast<const int2*>(a.copies) + mine);
        const bool good = entry.x >= 0 && entry.x < a.num_pages && entry.y >= 0 &&
                          entry.y < a.num_pages;
        for (unsigned left = __ballot_sync(0xffffffffu, good); left; left &= left - 1) {
            const int which = __ffs((int)left) - 1;
            const int64_t from = __shfl_sync(0xffffffffu, entry.x, which);
            const int64_t to = __shfl_sync(0xffffffffu, entry.y, which);
            uint4 v[kCopyAhead];
#pragma unroll
            for (int k = 0; k < kCopyAhead; ++k)
                if (at[k] >= 0)
                    v[k] = __ldcs(reinterpret_cast<const uint4*>(
                        cache + from * a.page_stride * bytes + at[k]));
#pragma unroll
            for (int k = 0; k < kCopyAhead; ++k)
                if (at[k] >= 0)
                    __stcs(reinterpret_cast<uint4*>(cache + to * a.page_stride * bytes + at[k]),
                           v[k]);
            if (part == 0 && scale_blocks) {
                unsigned short* scales =
                    static_cast<unsigned short*>(keys ? a.scales.k : a.scales.v) +
                    layer * a.scales.layer_stride;
                for (int64_t i = threadIdx.x; i < (int64_t)a.kv_heads * scale_blocks;
                     i += kCopyThreads) {
                    const int64_t head = i / scale_blocks;
                    const int64_t in = head * a.scales.head_stride + (i - head * scale_blocks);
                    scales[to * a.scales.page_stride + in] =
                        scales[from * a.scales.page_stride + in];
                }
            }
        }
    }
}

int64_t page_parts(const ple_copy_pages_args& a) {
    const int64_t pieces =
        (int64_t)a.kv_heads * a.page_size * (a.head_dim * a.element_bytes / 16);
    return (pieces + kCopyPart - 1) / kCopyPart;
}

}  // namespace

cudaError_t launch_tree_commit_fp8(const ple_tree_commit_fp8_args& f, const DeviceFacts& dev,
                                   cudaStream_t stream) {
    const int64_t blocks = 2 * (int64_t)f.base.num_requests * f.base.num_layers;
    const int threads = blocks * kCommitThreads <= 2048 * (int64_t)dev.sm_count
                            ? kCommitThreads
                            : kManyCommitThreads;
    return launch_kernel(tree_commit_fp8_kernel,
                         dim3((unsigned)f.base.num_requests, (unsigned)f.base.num_layers, 2),
                         dim3(threads), 0, stream, programmatic_launch(), f,
                         block_shift(f.scales.block));
}

int64_t plan_pages_workspace(int32_t num_rows, int32_t num_pages) {
    return 2 * kPlanChunk * plan_chunks(num_pages) +
           4 * (3 * (int64_t)num_pages + 2 * (int64_t)num_rows + kPlanBlocks * 8);
}

cudaError_t launch_plan_pages(const ple_plan_pages_args& a, cudaStream_t stream) {
    PlanSpace s;
    s.carried = static_cast<uint8_t*>(a.workspace);
    s.written = s.carried + kPlanChunk * plan_chunks(a.num_pages);
    s.writer = reinterpret_cast<int32_t*>(s.written + kPlanChunk * plan_chunks(a.num_pages));
    s.frees = s.writer + a.num_pages;
    s.rank = s.frees + a.num_pages;
    s.first_new = s.rank + a.num_pages;
    s.first_double = s.first_new + a.num_rows;
    s.sums = s.first_double + a.num_rows;
    return launch_kernel(plan_pages_kernel, dim3(kPlanBlocks), dim3(kPlanThreads), 0, stream,
                         programmatic_launch(), a, s);
}

bool copy_page_ok(const ple_copy_pages_args& a) { return 2 * page_parts(a) <= 65535; }

cudaError_t launch_copy_pages(const ple_copy_pages_args& a, const DeviceFacts& dev,
                              cudaStream_t stream) {
    const int row_pieces = a.head_dim * a.element_bytes / 16;
    const int64_t parts = page_parts(a);
    const int scale_blocks = a.scales.k ? a.page_size / a.scales.block : 0;
    // blocks enough for several waves; the rest of a long list in turn
    const int64_t others = 2 * parts * a.num_layers;
    int64_t lanes = 64 * (int64_t)dev.sm_count / others;
    if (lanes < 64) lanes = 64;
    if (lanes > a.num_copies) lanes = a.num_copies;
    return launch_kernel(copy_pages_kernel,
                         dim3((unsigned)lanes, (unsigned)a.num_layers, (unsigned)(2 * parts)),
                         dim3(kCopyThreads), 0, stream, programmatic_launch(), a, row_pieces,
                         (int)parts, scale_blocks);
}

}  // namespace ple
