// The PLE n-gram row-id hash of drafted trees on sm_103a.
//
// The hash of ple_rowids_common.cuh with every window taken along the node's
// branch: W(t, s) is the id of the node's s-th ancestor, and past the branch's
// root the carried context, newest id first.  Small batches take one thread for
// a row id, which finds the node's request, walks the branch and folds its
// head's order (ple_rowids_small.cu's division of the work, and its limit): a chain
// of dependent reads, 2.1 us for a tree of 9 nodes.  Larger ones take a warp for
// 32 nodes: 20.4 us for 8065 nodes x 48 layers x 32 heads, where int32 rows, half the
// bytes, take 19.5 and 46% of the issue slots are used, so neither bounds it (a
// kernel of compiled-in shapes writes as many rows of the prefill in 15.3).
#include "ple_rowids_common.cuh"
#include "ple_tree_common.cuh"

namespace ple {
namespace {

constexpr int kTreeThreads = 256;
// Blocks an SM that the tiled kernel's layer groups aim for.  Longer groups walk a
// branch and divide for a head's reciprocal less often, more blocks hide those
// better: 8065 nodes x 48 layers x 32 heads take 28.3 us at 2, 24.3 at 4, 20.4
// at 8, 21.8 at 12 and 16 (99 MB written: 4.9 TB/s).
constexpr int kTreeBlocksPerSm = 8;

template <typename IdT>
__global__ void __launch_bounds__(kTreeThreads)
tree_row_ids_kernel(const RowIdsParams p, const int32_t* __restrict__ parent) {
    wait_prior_grid();
    const int64_t per_layer = p.T * p.H;
    const int64_t e = (int64_t)blockIdx.x * kTreeThreads + threadIdx.x;
    if (e >= per_layer) return;
    const int64_t t = e / p.H;
    const int h = (int)(e - t * p.H);
    const int order = h / p.hpn + 1;  // ancestors that the head's order folds
    int32_t r, place;
    load_index<kIdxCu>(p, t, true, r, place);
    const int64_t first = t - place;
    const IdT* ids = static_cast<const IdT*>(p.ids);
    const IdT* ctx = static_cast<const IdT*>(p.ctx) + (int64_t)r * (p.N - 1);
    const int l = blockIdx.y;
    const int64_t* ml = p.mult + (int64_t)l * p.N;
    uint64_t mix = (uint64_t)load_id<IdT>(ids, t) * (uint64_t)ml[0];
    int at = place, back = p.N - 1;
    bool valid = true;
    for (int s = 1; s <= order; ++s) {
        if (at >= 0) {
            const int up = __ldg(parent + first + at);
            at = up < at ? max(up, -1) : -1;
        }
        const int64_t w = at >= 0 ? load_id<IdT>(ids, first + at) : load_id<IdT>(ctx, --back);
        valid = valid && w != p.boundary;
        mix ^= (uint64_t)(valid ? w : p.boundary) * (uint64_t)ml[s];
    }
    const int64_t k = (int64_t)l * p.H + h;
    const HeadConst c = p.heads != nullptr ? load_head_const(p.heads, k)
                                           : make_head_const(p.vocab[k], p.offsets[k]);
    const OffsetBinary u = offset_binary(mix);
    const int64_t row = (c.ext.z & kHeadFast) ? row_fast(u, c.fast, c.off)
                                              : row_general(u, c.fast, c.off, c.ext);
    const int64_t o = (int64_t)l * per_layer + e;
    if (p.out_bytes == 8)
        __stcs(static_cast<long long*>(p.out) + o, (long long)row);
    else
        __stcs(static_cast<int*>(p.out) + o, (int)row);
}

// ------------------------------------------------------- larger batches, tiled

constexpr int kTileWarps = 4;
constexpr int kTileRows = 32;  // nodes a warp's tile, one a lane

// Staged mixes of a tile: a row of N - 1 orders and padding to an odd pitch for
// each node, so that the lanes' stores of one order meet distinct banks.
__host__ __device__ constexpr size_t mix_bytes(int N) { return (size_t)kTileRows * (N | 1) * 8; }

template <typename OutT>
__device__ __forceinline__ void store_row(OutT* p, int64_t v) {
    if constexpr (sizeof(OutT) == 8)
        __stcs(reinterpret_cast<long long*>(p), (long long)v);
    else
        __stcs(reinterpret_cast<int*>(p), (int)v);
}

// A warp takes 32 nodes through a group of layers.  Every lane walks one node's
// branch once, N - 1 dependent reads of parents (L1 and L2 hits: a tree is a few
// lines), and keeps its window in registers for all layers of the group.  For a
// layer each lane folds its node's mixes, one an order, into shared memory; then
// the warp writes the tile's [nodes, H] row ids 32 at a time in global order,
// one contiguous store a step, each lane hashing the row it stores.
// The layer group's head constants are staged in shared memory by the block: a
// reciprocal is a 64-bit division, worth sharing among the block's four tiles.
// kLaneHeads: H divides 32 or is a multiple of it, so a lane meets one head for
// all nodes (of 32 heads) and holds its constants in registers; otherwise the
// head changes from step to step.
template <typename IdT, typename OutT, int NT, bool kLaneHeads>
__global__ void __launch_bounds__(kTileWarps * 32, 8)
tree_row_ids_tiled_kernel(const RowIdsParams p, const int32_t* __restrict__ parent) {
    constexpr int NMAX = NT > 0 ? NT : PLE_MAX_NGRAM;
    const int N = NT > 0 ? NT : p.N;
    const int H = p.H, pitch = N | 1;
    const int l0 = blockIdx.y * p.group_layers;
    const int gl = min(p.group_layers, p.L - l0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    extern __shared__ __align__(16) unsigned char smem[];
    wait_prior_grid();
    uint2* mix_s = reinterpret_cast<uint2*>(smem + (size_t)warp * mix_bytes(N));
    const SmemLayout sm = carve_smem(smem + kTileWarps * mix_bytes(N), p.group_layers, H, N, 0);
    load_group_constants(p, sm, l0, gl, H, N);
    const int64_t t0 = ((int64_t)blockIdx.x * kTileWarps + warp) * kTileRows;
    const int ntile = (int)max((int64_t)0, min((int64_t)kTileRows, p.T - t0));
    int64_t V[NMAX];
    if (ntile > 0) {
        const bool live = lane < ntile;
        const int64_t t = t0 + lane;
        int ra, rb;
        int32_t r, place, unused_r, unused_q;
        warp_owners(p, t0, t0 + ntile - 1, lane, ra, rb);
        if (rb - ra <= 32)
            tile_owners(p, ra, rb, t, live, t, false, lane, r, place, unused_r, unused_q);
        else
            load_index<kIdxCu>(p, t, live, r, place, ra, rb);
        const IdT* ids = static_cast<const IdT*>(p.ids);
        const IdT* ctx = static_cast<const IdT*>(p.ctx) + (int64_t)r * (N - 1);
        const int64_t first = live ? t - place : 0;
        int at = live ? place : -1, back = N - 1;
        bool valid = true;
        V[0] = live ? load_id<IdT>(ids, t) : 0;
#pragma unroll
        for (int s = 1; s < NMAX; ++s) {
            if (NT == 0 && s >= N) break;
            if (at >= 0) {
                const int up = __ldg(parent + first + at);
                at = up < at ? max(up, -1) : -1;
            }
            const int64_t w = at >= 0 ? load_id<IdT>(ids, first + at) : load_id<IdT>(ctx, --back);
            valid = valid && w != p.boundary;
            V[s] = valid ? w : p.boundary;
        }
    }
    __syncthreads();
    if (ntile == 0) return;

#pragma unroll 1
    for (int l = 0; l < gl; ++l) {
        const int64_t layer = (int64_t)l0 + l;
        const int64_t* ml = sm.mul + l * N;
        const uint4* fasts = sm.fast + l * H;
        const int64_t* offs = sm.off + l * H;
        const uint4* exts = sm.ext + l * H;
        uint64_t mix = (uint64_t)V[0] * (uint64_t)ml[0];
#pragma unroll
        for (int s = 1; s < NMAX; ++s) {
            if (NT == 0 && s >= N) break;
            mix ^= (uint64_t)V[s] * (uint64_t)ml[s];
            const OffsetBinary u = offset_binary(mix);
            mix_s[lane * pitch + s - 1] = make_uint2(u.lo, u.hi);
        }
        __syncwarp();
        OutT* out = static_cast<OutT*>(p.out) + (layer * p.T + t0) * H;
        if constexpr (kLaneHeads) {
            const int step = H >= 32 ? 1 : 32 / H;  // nodes a store covers
            const int sub = H >= 32 ? 0 : lane / H;
#pragma unroll 1
            for (int h = H >= 32 ? lane : lane % H; h < H; h += 32) {
                const HeadConst c = {fasts[h], offs[h], exts[h]};
                const uint2* m = mix_s + sub * pitch + h / p.hpn;
                OutT* dst = out + sub * H + h;
                const bool fast = c.ext.z == kHeadFast;
                const uint32_t nv = (uint32_t)((int32_t)c.fast.z >> 1);  // -v
                if (fast) {
#pragma unroll 8
                    for (int i = sub; i < ntile; i += step) {
                        const uint2 w = m[(i - sub) * pitch];
                        store_row(dst + (int64_t)(i - sub) * H,
                                  (int64_t)((uint64_t)c.off +
                                            floormod_fast_alu(OffsetBinary{w.x, w.y}, c.fast, nv,
                                                              p.ones)));
                    }
                } else {
#pragma unroll 1
                    for (int i = sub; i < ntile; i += step) {
                        const uint2 w = m[(i - sub) * pitch];
                        store_row(dst + (int64_t)(i - sub) * H,
                                  row_general(OffsetBinary{w.x, w.y}, c.fast, c.off, c.ext));
                    }
                }
            }
        } else {
            const int dq = 32 / H, dr = 32 % H;
            int node = lane / H, h = lane % H;
#pragma unroll 4
            for (int e = lane; e < ntile * H; e += 32) {
                const uint2 w = mix_s[node * pitch + h / p.hpn];
                const OffsetBinary u{w.x, w.y};
                const uint4 x = exts[h];
                store_row(out + e, x.z == kHeadFast ? row_fast(u, fasts[h], offs[h])
                                                    : row_general(u, fasts[h], offs[h], x));
                h += dr;
                node += dq;
                if (h >= H) {
                    h -= H;
                    ++node;
                }
            }
        }
        __syncwarp();  // the next layer overwrites the mixes
    }
}

using TreeFn = void (*)(const RowIdsParams, const int32_t*);

template <typename IdT, typename OutT, bool kLaneHeads>
TreeFn pick_tiled(int N) {
    switch (N) {
        case 2: return tree_row_ids_tiled_kernel<IdT, OutT, 2, kLaneHeads>;
        case 3: return tree_row_ids_tiled_kernel<IdT, OutT, 3, kLaneHeads>;
        case 4: return tree_row_ids_tiled_kernel<IdT, OutT, 4, kLaneHeads>;
        case 5: return tree_row_ids_tiled_kernel<IdT, OutT, 5, kLaneHeads>;
        default: return tree_row_ids_tiled_kernel<IdT, OutT, 0, kLaneHeads>;
    }
}

template <typename IdT, typename OutT>
TreeFn pick_tiled(int N, bool lane_heads) {
    return lane_heads ? pick_tiled<IdT, OutT, true>(N) : pick_tiled<IdT, OutT, false>(N);
}

}  // namespace

cudaError_t launch_tree_row_ids(RowIdsParams p, const int32_t* parent, int id_bytes,
                                const DeviceFacts& dev, cudaStream_t stream) {
    if (small_batch_fits(p)) {
        const int64_t blocks = (p.T * p.H + kTreeThreads - 1) / kTreeThreads;
        auto* fn = id_bytes == 4 ? tree_row_ids_kernel<int32_t> : tree_row_ids_kernel<int64_t>;
        return launch_kernel(fn, dim3((unsigned)blocks, (unsigned)p.L), dim3(kTreeThreads), 0,
                             stream, programmatic_launch(), p, parent);
    }
    const bool lane_heads = 32 % p.H == 0 || p.H % 32 == 0;
    const int64_t blocks =
        (p.T + kTileRows * kTileWarps - 1) / (kTileRows * kTileWarps);
    // layer groups: as long as every SM gets kTreeBlocksPerSm blocks, so that a
    // branch is walked for several layers; the staged constants within 48 KB and
    // the groups within a grid's second extent
    int64_t groups = (kTreeBlocksPerSm * (int64_t)dev.sm_count + blocks - 1) / blocks;
    groups = groups < 1 ? 1 : groups > p.L ? p.L : groups;
    int64_t G = (p.L + groups - 1) / groups;
    const size_t per_layer = head_const_bytes(p.H) + 8 * (size_t)(p.N + 1);
    if (G > (int64_t)(kConstBudgetBytes / per_layer))
        G = kConstBudgetBytes / per_layer > 0 ? kConstBudgetBytes / per_layer : 1;
    if ((p.L + G - 1) / G > 65535) return cudaErrorInvalidConfiguration;
    p.group_layers = (int)G;
    const size_t smem = kTileWarps * mix_bytes(p.N) + head_const_bytes((int)G * p.H) +
                        ((size_t)G * p.N + 1) * 8;
    TreeFn fn;
    if (p.out_bytes == 4)
        fn = id_bytes == 4 ? pick_tiled<int32_t, int32_t>(p.N, lane_heads)
                           : pick_tiled<int64_t, int32_t>(p.N, lane_heads);
    else
        fn = id_bytes == 4 ? pick_tiled<int32_t, int64_t>(p.N, lane_heads)
                           : pick_tiled<int64_t, int64_t>(p.N, lane_heads);
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(fn, dim3((unsigned)blocks, (unsigned)((p.L + G - 1) / G)),
                         dim3(kTileWarps * 32), smem, stream, programmatic_launch(), p, parent);
}

}  // namespace ple
