// Norms of queries and keys for each head, the position rotation and the
// append to the paged cache, in one pass, on sm_103a; and the rotation's
// per-position turns.
//
// A head row x of D elements becomes y = x / sqrt(mean(x^2) + eps) * weight, and
// its first R elements turn in pairs by the position's angle.  Everything is
// computed in 32 bits and rounded once.
//
// Angles.  Pair i turns F_i * 2^-64 of a full turn per position, F_i a whole
// number (ple_prepare_rope).  The angle at position m is then the wrapping
// product m * F_i: the whole turns fall off the top, and its upper 32 bits as a
// signed fraction of a turn go to sincospif.  The rounding of F_i to 2^-64
// turns and the 24 bits of the float leave about 2e-7 radians at any position,
// where m * w_i in 32 bits loses 2^-24 of the whole angle (0.008 radians at
// position 131072).
//
// Layout.  Eight elements a lane and D / 8 lanes a row, rounded up to a power of
// two, so a warp holds one to four rows and a row's sum of squares is a few
// shuffles.  A lane holds both elements of its pairs: eight in a row where pairs lie
// side by side, else four and the four half the rotary part behind them.  A block
// takes up to eight tokens: their sines and cosines are computed once and shared
// by all their heads.  Bound by the rows' bytes, each read and written once: 64
// drafted trees (43 MB, in L2) take 13.5 us, one token 3.0.  The trees' 1057 tokens
// go one to a block, and as many blocks are 1.4 times what the device holds at once:
// the second wave, mostly empty, is a part of that time.
#include "ple_norm_rope.cuh"

namespace ple {
namespace {

template <typename E, int LPR, int kLayout>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks)
qk_norm_rope_kernel(const __grid_constant__ ple_qk_norm_rope_args a, const RowPlan plan) {
    norm_rope_rows<E, LPR, kLayout>(a, plan, blockIdx.x, blockIdx.y, gridDim.y);
}

// F_i = w_i / 2 pi * 2^64, w_i the pair's angle per position (base^(-2i/R),
// scaled).  w_i <= 1, so F_i stays below 2^62 and its 53 bits are exact to
// 2^-53 of the turn a position makes.
__global__ void prepare_rope_kernel(int R, double base, int scaling, double factor,
                                    double trained, double beta_fast, double beta_slow,
                                    int64_t* __restrict__ rope) {
    wait_grid_before();
    const int i = threadIdx.x;
    if (i >= R / 2) return;
    const double two_pi = 6.283185307179586476925286766559;
    if (scaling == PLE_ROPE_BASE && R > 2) base *= pow(factor, (double)R / (double)(R - 2));
    double w = pow(base, -2.0 * i / R);
    if (scaling == PLE_ROPE_LINEAR) w /= factor;
    if (scaling == PLE_ROPE_PARTS) {
        const double turns = trained * w / two_pi;
        const double g = fmin(fmax((turns - beta_slow) / (beta_fast - beta_slow), 0.0), 1.0);
        w = g * w + (1.0 - g) * (w / factor);
    }
    rope[i] = (int64_t)(w / two_pi * 0x1p64);
}

template <typename E, int LPR>
cudaError_t launch_rows(const ple_qk_norm_rope_args& a, const DeviceFacts& dev,
                        cudaStream_t stream) {
    constexpr int RPW = 32 / LPR;
    constexpr int kWarps = kNormThreads / 32;
    RowPlan plan;
    plan.q_groups = (a.q_heads + RPW - 1) / RPW;
    plan.kv_groups = (a.kv_heads + RPW - 1) / RPW;
    // one token a block until that makes as many blocks as the device holds
    // at once, then up to kNormTokens; while there are fewer blocks than that,
    // a token's groups spread over several blocks too
    const int64_t resident = kNormBlocks * (int64_t)dev.sm_count;
    const int64_t tokens = a.num_tokens / resident;
    plan.tokens = (int)(tokens < 1 ? 1 : tokens > kNormTokens ? kNormTokens : tokens);
    const int64_t blocks = (a.num_tokens + plan.tokens - 1) / plan.tokens;
    const int groups = plan.q_groups + plan.kv_groups * (a.k_cache != nullptr ? 2 : 1);
    int64_t split = resident / blocks;
    const int64_t most = (groups + kWarps - 1) / kWarps;
    split = split < 1 ? 1 : split > most ? most : split;
    const dim3 grid((unsigned)blocks, (unsigned)split);
    auto* fn = a.interleaved           ? qk_norm_rope_kernel<E, LPR, kPairsInterleaved>
               : a.rotary_dim % 8 == 0 ? qk_norm_rope_kernel<E, LPR, kPairsHalves>
                                        : qk_norm_rope_kernel<E, LPR, kPairsAnyHalves>;
    return launch_kernel(fn, grid, dim3(kNormThreads), 0, stream, programmatic_launch(), a,
                         plan);
}

template <typename E>
cudaError_t launch_element(const ple_qk_norm_rope_args& a, const DeviceFacts& dev,
                           cudaStream_t stream) {
    if (a.head_dim <= 64) return launch_rows<E, 8>(a, dev, stream);
    if (a.head_dim <= 128) return launch_rows<E, 16>(a, dev, stream);
    return launch_rows<E, 32>(a, dev, stream);
}

}  // namespace

cudaError_t launch_prepare_rope(int32_t rotary_dim, double base, int32_t scaling, double factor,
                                double trained, double beta_fast, double beta_slow,
                                int64_t* rope, cudaStream_t stream) {
    return launch_kernel(prepare_rope_kernel, dim3(1), dim3(kMaxPairs), 0, stream,
                         programmatic_launch(), rotary_dim, base, scaling, factor, trained,
                         beta_fast, beta_slow, rope);
}

cudaError_t launch_qk_norm_rope(const ple_qk_norm_rope_args& a, const DeviceFacts& dev,
                                cudaStream_t stream) {
    return a.dtype == PLE_BF16 ? launch_element<__nv_bfloat16>(a, dev, stream)
                               : launch_element<__half>(a, dev, stream);
}

}  // namespace ple
