// Bookkeeping of drafted trees on sm_103a: the tree index (positions and
// ancestor masks) and the commit of accepted branches.
#include "ple_tree_common.cuh"

namespace ple {
namespace {

// ---------------------------------------------------------------- tree index

// sees(i) = {i} + sees(parent(i)), and the depth is |sees(i)| - 1.  One block
// for a request, one thread for a node, masks and jumps in shared memory: each
// round joins a node's mask with its jump's mask and doubles the jump, so a
// tree of depth d is done after log2(d) + 1 rounds, however it branches.  The
// call is a latency: parents are read once and the outputs written once (one tree
// of 4 nodes 1.4 us, 256 of up to 127 nodes 2.0 us).
template <int W>
__global__ void __launch_bounds__(64 * W)
tree_index_kernel(const int32_t* __restrict__ parent, const int32_t* __restrict__ cu,
                  const int32_t* __restrict__ ctx_lens, int64_t T,
                  int32_t* __restrict__ positions, uint64_t* __restrict__ mask) {
    __shared__ uint64_t seen[W][64 * W];
    __shared__ int32_t jump[64 * W];
    wait_grid_before();
    const int r = blockIdx.x;
    const int i = threadIdx.x;
    int32_t begin, end;
    request_nodes(cu, r, T, begin, end);
    const int n = end - begin;
    const int32_t ctx = __ldg(ctx_lens + r);
    int32_t up = -1;
    if (i < n) up = __ldg(parent + begin + i);
    if (up >= i) up = -1;
    uint64_t m[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
        m[w] = (i >> 6) == w ? 1ull << (i & 63) : 0;
        seen[w][i] = m[w];
    }
    jump[i] = up;
    while (__syncthreads_or(up >= 0)) {
        int32_t next = -1;
        if (up >= 0) {
#pragma unroll
            for (int w = 0; w < W; ++w) m[w] |= seen[w][up];
            next = jump[up];
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) seen[w][i] = m[w];
        jump[i] = up = next;
    }
    if (i < n) {
        int depth = -1;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            mask[(int64_t)(begin + i) * W + w] = m[w];
            depth += __popcll(m[w]);
        }
        positions[begin + i] = ctx + depth;
    }
    // nodes that have no bit
    for (int j = i + 64 * W; j < n; j += 64 * W) {
        for (int w = 0; w < W; ++w) mask[(int64_t)(begin + j) * W + w] = 0;
        positions[begin + j] = ctx;
    }
}

// ------------------------------------------------------------------- commit

constexpr int kCommitThreads = 128;
constexpr int kCommitSteps = 64;  // path entries staged at a time

// The accepted rows of one request, one layer and one cache move to the front
// of the tree's slots.  A thread owns one 16-byte column of one head and walks
// the path in order, loading a few rows before it stores them: entry j comes
// from node path[j] >= j, so no later source lies at or below slot j and the
// moves in place read nothing that was overwritten.  Bound by the rows' bytes,
// read once and written once (each 16-byte lane of a head's row in one
// transaction with its neighbours): one branch 2.7 us, 64 branches x 48 layers
// 11.8 us (88 MB moved, part of it in L2) and 17 from a cold cache.
__global__ void __launch_bounds__(kCommitThreads)
tree_commit_kernel(const ple_tree_commit_args a) {
    __shared__ int64_t from[kCommitSteps], to[kCommitSteps];
    wait_grid_before();
    const int r = blockIdx.x;
    const int layer = blockIdx.y;
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

    const int per_head = a.head_dim >> 3;
    const int columns = a.kv_heads * per_head;
    unsigned short* cache = static_cast<unsigned short*>(blockIdx.z == 0 ? a.k_cache : a.v_cache) +
                            layer * a.layer_stride;
    for (int j0 = 0; j0 < kept; j0 += kCommitSteps) {
        const int steps = min(kCommitSteps, kept - j0);
        __syncthreads();
        if (threadIdx.x < steps) {
            const int j = j0 + threadIdx.x;
            const int node = __ldg(path + j);
            int64_t s = -1, d = -1;
            if (node > j && node < n) {
                s = slot_offset(a.page_table, a.max_pages, a.page_size, a.num_pages,
                                a.page_stride, a.slot_stride, r, ctx + node);
                d = slot_offset(a.page_table, a.max_pages, a.page_size, a.num_pages,
                                a.page_stride, a.slot_stride, r, ctx + j);
            }
            from[threadIdx.x] = d < 0 ? -1 : s;
            to[threadIdx.x] = d;
        }
        __syncthreads();
        for (int c = threadIdx.x; c < columns; c += kCommitThreads) {
            unsigned short* base = cache + (c / per_head) * a.head_stride + (c % per_head) * 8;
            for (int j = 0; j < steps; j += 4) {
                uint4 row[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (j + k < steps && from[j + k] >= 0)
                        row[k] = *reinterpret_cast<const uint4*>(base + from[j + k]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (j + k < steps && from[j + k] >= 0)
                        *reinterpret_cast<uint4*>(base + to[j + k]) = row[k];
            }
        }
    }
}

template <int W>
cudaError_t launch_index_words(const int32_t* parent, const int32_t* cu, const int32_t* ctx_lens,
                               int32_t B, int64_t T, int32_t* positions, uint64_t* mask,
                               cudaStream_t stream) {
    return launch_kernel(tree_index_kernel<W>, dim3((unsigned)B), dim3(64 * W), 0, stream,
                         programmatic_launch(), parent, cu, ctx_lens, T, positions, mask);
}

}  // namespace

cudaError_t launch_tree_index(const int32_t* parent, const int32_t* cu, const int32_t* ctx_lens,
                              int32_t B, int64_t T, int32_t words, int32_t* positions,
                              uint64_t* mask, cudaStream_t stream) {
    switch (words) {
        case 1: return launch_index_words<1>(parent, cu, ctx_lens, B, T, positions, mask, stream);
        case 2: return launch_index_words<2>(parent, cu, ctx_lens, B, T, positions, mask, stream);
        case 3: return launch_index_words<3>(parent, cu, ctx_lens, B, T, positions, mask, stream);
        case 4: return launch_index_words<4>(parent, cu, ctx_lens, B, T, positions, mask, stream);
        case 5: return launch_index_words<5>(parent, cu, ctx_lens, B, T, positions, mask, stream);
        case 6: return launch_index_words<6>(parent, cu, ctx_lens, B, T, positions, mask, stream);
        case 7: return launch_index_words<7>(parent, cu, ctx_lens, B, T, positions, mask, stream);
        default: return launch_index_words<8>(parent, cu, ctx_lens, B, T, positions, mask, stream);
    }
}

cudaError_t launch_tree_commit(const ple_tree_commit_args& a, const DeviceFacts&,
                               cudaStream_t stream) {
    return launch_kernel(tree_commit_kernel,
                         dim3((unsigned)a.num_requests, (unsigned)a.num_layers, 2),
                         dim3(kCommitThreads), 0, stream, programmatic_launch(), a);
}

}  // namespace ple
