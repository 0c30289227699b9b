// The PLE n-gram row-id hash of drafted trees on sm_103a.
//
// The hash of ple_rowids_common.cuh with every window taken along the node's
// branch: W(t, s) is the id of the node's s-th ancestor, and past the branch's
// root the carried context, newest id first.  One thread for a row id: it
// finds the node's request, walks the branch and folds its head's order.
#include "ple_rowids_common.cuh"
#include "ple_tree_common.cuh"

namespace ple {
namespace {

constexpr int kTreeThreads = 256;

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
    for (int l = blockIdx.y; l < p.L; l += gridDim.y) {
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
}

}  // namespace

cudaError_t launch_tree_row_ids(const RowIdsParams& p, const int32_t* parent, int id_bytes,
                                const DeviceFacts&, cudaStream_t stream) {
    const int64_t blocks = (p.T * p.H + kTreeThreads - 1) / kTreeThreads;
    auto* fn = id_bytes == 4 ? tree_row_ids_kernel<int32_t> : tree_row_ids_kernel<int64_t>;
    return launch_kernel(fn, dim3((unsigned)blocks, (unsigned)(p.L < 65535 ? p.L : 65535)), dim3(kTreeThreads), 0, stream,
                         programmatic_launch(), p, parent);
}

}  // namespace ple
