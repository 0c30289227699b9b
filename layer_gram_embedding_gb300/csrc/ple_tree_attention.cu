// Attention of drafted nodes over the paged cache and their own branch, on
// sm_103a: the kernel for every page size and stride.
//
//   out = sum_j p_j v_j,  p = softmax_j(scale q . k_j)
// over the slots that a node sees, in one pass over the keys with the running
// maximum and sum of the softmax (Milakov and Gimelshein 2018): a block takes
// one node and up to eight query heads of one key head, its warps take the
// keys 32 at a time in turn, and the warps' states are joined at the end.  Calls
// with few blocks split the slots over several; those leave their states in
// the workspace and a second kernel joins them in the slots' order.
//
// It serves what the tensor-core kernel does not take: page sizes that are no
// multiple of 8 and caches with strides that a tensor map refuses.  Bound by its
// 32-bit multiply-adds, 4 D operations a row and slot, and by every node reading
// the keys for itself.  20-slot pages, 8 key heads of 4 query heads: 8 requests of
// 1 node over 8192 slots, heads of 128, 368 us (0.7 TB/s); 4 requests of 16 nodes
// over 8192 slots, heads of 256, 4.8 ms.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ple_tree_common.cuh"

namespace ple {
namespace {

constexpr int kWarps = 4;
constexpr int kRows = 8;                          // query heads a block
constexpr int kPieces = PLE_MAX_HEAD_DIM / 64;    // pairs of elements a lane holds

__device__ __forceinline__ float2 widen(__nv_bfloat162 v) { return __bfloat1622float2(v); }
__device__ __forceinline__ float2 widen(__half2 v) { return __half22float2(v); }
__device__ __forceinline__ void narrow(float2 v, __nv_bfloat162* out) {
    *out = __float22bfloat162_rn(v);
}
__device__ __forceinline__ void narrow(float2 v, __half2* out) { *out = __float22half2_rn(v); }

// Blocks along a row's slots: enough that the grid has kSplitBlocks an SM, with
// one part of every row if it has them anyway.
constexpr int kSplitBlocks = 4;
int any_splits(int64_t T, int32_t q_heads, int32_t kv_heads, const DeviceFacts& dev) {
    const int group = q_heads / kv_heads;
    const int64_t blocks = T * kv_heads * ((group + kRows - 1) / kRows);
    const int64_t splits = blocks > 0 ? kSplitBlocks * (int64_t)dev.sm_count / blocks : 1;
    return (int)(splits < 1 ? 1 : splits);
}

// A part's state of row `row` (token-major): maximum, sum, D accumulators.
__host__ __device__ __forceinline__ int64_t part_at(int64_t row, int part, int splits, int D) {
    return (row * splits + part) * (int64_t)(D + 2);
}

template <typename E2>
__global__ void __launch_bounds__(kWarps * 32)
tree_attention_any_kernel(const ple_tree_attention_args a, const int splits) {
    __shared__ __align__(16) float q_s[kRows][PLE_MAX_HEAD_DIM];
    __shared__ float p_s[kWarps][kRows][32];
    __shared__ float top_s[kWarps][kRows], sum_s[kWarps][kRows];
    __shared__ float acc_s[kWarps][kRows][PLE_MAX_HEAD_DIM];
    wait_grid_before();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int D = a.head_dim;
    const int64_t t = blockIdx.x;
    const int kv = blockIdx.y;
    const int group = a.q_heads / a.kv_heads;
    const int part = blockIdx.z % splits;
    const int h0 = kv * group + blockIdx.z / splits * kRows;
    const int rows = min(kRows, (kv + 1) * group - h0);

    const int r = warp_request(a.cu_seqlens, a.num_requests, t, lane);
    int32_t begin, end;
    request_nodes(a.cu_seqlens, r, a.num_tokens, begin, end);
    const int64_t ctx = max(__ldg(a.ctx_lens + r), 0);
    const int64_t slots = min(ctx + (end - begin), (int64_t)a.max_pages * a.page_size);
    // this part's slots, whole rounds of the block's warps
    const int64_t round = splits * kWarps * 32;
    const int64_t span = (slots + round - 1) / round * (kWarps * 32);
    const int64_t last = min(slots, (part + 1) * span);
    for (int i = threadIdx.x; i < rows * (D / 2); i += kWarps * 32) {
        const int row = i / (D / 2), c = i % (D / 2);
        const float2 v = widen(reinterpret_cast<const E2*>(
            static_cast<const unsigned short*>(a.q) + t * a.q_token + (h0 + row) * a.q_head)[c]);
        q_s[row][2 * c] = v.x * a.scale;
        q_s[row][2 * c + 1] = v.y * a.scale;
    }
    __syncthreads();

    float top[kRows], sum[kRows];
    float2 acc[kRows][kPieces];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        top[i] = -INFINITY;
        sum[i] = 0.f;
#pragma unroll
        for (int c = 0; c < kPieces; ++c) acc[i][c] = make_float2(0.f, 0.f);
    }
    const int64_t head = kv * a.head_stride;
    for (int64_t s0 = part * span + warp * 32; s0 < last; s0 += kWarps * 32) {
        // a lane's key
        const int64_t s = s0 + lane;
        bool seen = s < last;
        if (seen && s >= ctx) {
            const int j = (int)(s - ctx);
            seen = j < 64 * a.mask_words &&
                   ((__ldg(reinterpret_cast<const unsigned long long*>(a.tree_mask) +
                           t * a.mask_words + (j >> 6)) >> (j & 63)) & 1);
        }
        const int64_t at = seen ? slot_offset(a.page_table, a.max_pages, a.page_size, a.num_pages,
                                              a.page_stride, a.slot_stride, r, s)
                                : -1;
        float score[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) score[i] = 0.f;
        if (at >= 0) {
            const uint4* k = reinterpret_cast<const uint4*>(
                static_cast<const unsigned short*>(a.k_cache) + at + head);
            for (int c = 0; c < D / 8; ++c) {
                const uint4 w = __ldg(k + c);
                const E2* e = reinterpret_cast<const E2*>(&w);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float2 f = widen(e[x]);
#pragma unroll
                    for (int i = 0; i < kRows; ++i)
                        if (i < rows) {
                            score[i] = fmaf(q_s[i][8 * c + 2 * x], f.x, score[i]);
                            score[i] = fmaf(q_s[i][8 * c + 2 * x + 1], f.y, score[i]);
                        }
                }
            }
        }
        const unsigned any = __ballot_sync(0xffffffffu, seen);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (i >= rows) break;
            const float x = seen ? score[i] : -INFINITY;
            float m = x;
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            m = fmaxf(m, top[i]);
            // -infinity everywhere so far: exponents relative to 0, all zero
            const float base = m == -INFINITY ? 0.f : m;
            const float p = seen ? expf(x - base) : 0.f;
            float l = p;
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
            const float keep = expf(top[i] - base);
            sum[i] = sum[i] * keep + l;
            top[i] = m;
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
                acc[i][c].x *= keep;
                acc[i][c].y *= keep;
            }
            p_s[warp][i][lane] = p;
        }
        __syncwarp();
        // values of the seen keys only: what another slot holds is not read
        for (unsigned left = any; left; left &= left - 1) {
            const int j = __ffs((int)left) - 1;
            const int64_t vat = __shfl_sync(0xffffffffu, at, j);
            if (vat < 0) continue;
            const E2* v = reinterpret_cast<const E2*>(
                static_cast<const unsigned short*>(a.v_cache) + vat + head);
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
                if (2 * lane + 64 * c >= D) break;
                const float2 f = widen(v[lane + 32 * c]);
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    if (i < rows) {
                        acc[i][c].x = fmaf(p_s[warp][i][j], f.x, acc[i][c].x);
                        acc[i][c].y = fmaf(p_s[warp][i][j], f.y, acc[i][c].y);
                    }
            }
        }
        __syncwarp();
    }

#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (lane == 0) {
            top_s[warp][i] = top[i];
            sum_s[warp][i] = sum[i];
        }
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
            if (2 * lane + 64 * c < D)
                *reinterpret_cast<float2*>(&acc_s[warp][i][2 * lane + 64 * c]) = acc[i][c];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (D / 2); i += kWarps * 32) {
        const int row = i / (D / 2), c = i % (D / 2);
        float m = -INFINITY;
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, top_s[w][row]);
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f, x = 0.f, y = 0.f;
        for (int w = 0; w < kWarps; ++w) {
            const float f = expf(top_s[w][row] - base);
            l += f * sum_s[w][row];
            x += f * acc_s[w][row][2 * c];
            y += f * acc_s[w][row][2 * c + 1];
        }
        const int64_t o = t * a.q_heads + h0 + row;
        if (splits > 1) {
            float* state = static_cast<float*>(a.workspace) + part_at(o, part, splits, D);
            if (c == 0) {
                state[0] = m;
                state[1] = l;
            }
            state[2 + 2 * c] = x;
            state[3 + 2 * c] = y;
            continue;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        narrow(make_float2(x * inv, y * inv),
               reinterpret_cast<E2*>(static_cast<unsigned short*>(a.out) + o * D) + c);
        if (c == 0 && a.lse != nullptr) a.lse[o] = l == 0.f ? -INFINITY : m + logf(l);
    }
}

// A warp joins a row's parts, D floats a part read once: a latency of a few us.
template <typename E2>
__global__ void __launch_bounds__(kWarps * 32)
tree_attention_any_join_kernel(const ple_tree_attention_args a, const int splits) {
    wait_grid_before();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int D = a.head_dim;
    if (row >= a.num_tokens * a.q_heads) return;
    const float* state = static_cast<const float*>(a.workspace) + part_at(row, 0, splits, D);
    float m = -INFINITY;
    for (int i = lane; i < splits; i += 32) m = fmaxf(m, __ldcg(state + i * (int64_t)(D + 2)));
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float2 acc[kPieces];
#pragma unroll
    for (int c = 0; c < kPieces; ++c) acc[c] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < splits; ++i) {
        const float* part = state + i * (int64_t)(D + 2);
        const float f = expf(__ldcg(part) - base);
        l = fmaf(f, __ldcg(part + 1), l);
#pragma unroll
        for (int c = 0; c < kPieces; ++c) {
            if (2 * lane + 64 * c < D) {
                const float2 v = __ldcg(reinterpret_cast<const float2*>(part + 2) + lane + 32 * c);
                acc[c].x = fmaf(f, v.x, acc[c].x);
                acc[c].y = fmaf(f, v.y, acc[c].y);
            }
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    E2* out = reinterpret_cast<E2*>(static_cast<unsigned short*>(a.out) + row * D);
#pragma unroll
    for (int c = 0; c < kPieces; ++c)
        if (2 * lane + 64 * c < D)
            narrow(make_float2(acc[c].x * inv, acc[c].y * inv), out + lane + 32 * c);
    if (lane == 0 && a.lse != nullptr) a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

template <typename E2>
cudaError_t launch_any(const ple_tree_attention_args& a, int splits, cudaStream_t stream) {
    const int group = a.q_heads / a.kv_heads;
    const dim3 grid((unsigned)a.num_tokens, (unsigned)a.kv_heads,
                    (unsigned)((group + kRows - 1) / kRows * splits));
    cudaError_t e = launch_kernel(tree_attention_any_kernel<E2>, grid, dim3(kWarps * 32), 0, stream,
                                  programmatic_launch(), a, splits);
    if (e != cudaSuccess || splits == 1) return e;
    const int64_t rows = a.num_tokens * a.q_heads;
    return launch_kernel(tree_attention_any_join_kernel<E2>,
                         dim3((unsigned)((rows + kWarps - 1) / kWarps)), dim3(kWarps * 32), 0,
                         stream, programmatic_launch(), a, splits);
}

}  // namespace

int64_t tree_attention_workspace(int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                 const DeviceFacts& dev) {
    // the tensor-core kernel's states, or this one's
    const int64_t tc = tree_attention_tc_workspace(T, q_heads, kv_heads, head_dim, dev);
    const int splits = any_splits(T, q_heads, kv_heads, dev);
    const int64_t any = splits > 1 ? 4 * part_at(T * q_heads, 0, splits, head_dim) : 0;
    return tc > any ? tc : any;
}

cudaError_t launch_tree_attention(const ple_tree_attention_args& a, const DeviceFacts& dev,
                                  cudaStream_t stream) {
    if (tree_attention_tc_fits(a)) {
        bool taken;
        const cudaError_t e = launch_tree_attention_tc(a, dev, stream, &taken);
        if (e != cudaSuccess || taken) return e;
    }
    const int splits = any_splits(a.num_tokens, a.q_heads, a.kv_heads, dev);
    return a.dtype == PLE_BF16 ? launch_any<__nv_bfloat162>(a, splits, stream)
                               : launch_any<__half2>(a, splits, stream);
}

}  // namespace ple
