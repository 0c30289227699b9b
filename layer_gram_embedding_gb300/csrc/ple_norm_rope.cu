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
// Layout.  Eight elements (16 bytes) a lane and D / 8 lanes a row, rounded up to
// a power of two, so a warp holds one to four rows and a row's sum of squares
// is a few shuffles.  A pair's other half is in the same lane (interleaved), or
// R / 16 lanes away (halves).  A block takes up to four tokens: their
// sines and cosines are computed once, one pair a thread, and shared by all
// their heads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ple_tree_common.cuh"

namespace ple {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormTokens = 4;    // tokens a block, for batches that fill the device
constexpr int kMaxPairs = PLE_MAX_HEAD_DIM / 2;

template <typename E>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <typename E>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename E>
__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<E>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

template <typename E>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack2<E>(x[0], x[1]), pack2<E>(x[2], x[3]), pack2<E>(x[4], x[5]),
                      pack2<E>(x[6], x[7]));
}

// How a pair's two elements lie: side by side, half the rotary part apart with
// both in whole lanes (R / 2 a multiple of 8), or half of it apart anyhow.
enum PairLayout { kPairsInterleaved = 0, kPairsHalves = 1, kPairsAnyHalves = 2 };

// Pair p's (cos, sin) is float2 number (2 * ((p % 8) / 2) + ...) of four planes:
// plane k holds, for every chunk of eight pairs, pairs 2k and 2k + 1, so that
// the lanes of a row read consecutive 16-byte words.
__device__ __forceinline__ int pair_slot(int p, int chunks) {
    return (((p & 7) >> 1) * chunks + (p >> 3)) * 2 + (p & 1);
}

template <typename E, int LPR, int kLayout>
__global__ void __launch_bounds__(kNormThreads)
qk_norm_rope_kernel(const ple_qk_norm_rope_args a, const int tokens) {
    constexpr int RPW = 32 / LPR;                      // rows a warp
    constexpr int RPB = RPW * (kNormThreads / 32);     // rows a block and step
    constexpr int U = 3;                               // steps whose loads are in flight
    __shared__ __align__(16) float2 turn[kNormTokens][kMaxPairs + 8];
    __shared__ int64_t dst_s[kNormTokens];
    __shared__ float row_s[kLayout == kPairsAnyHalves ? kNormThreads * 8 : 1];

    wait_grid_before();
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int nt = (int)min((int64_t)tokens, a.num_tokens - t0);
    const bool cached = a.k_cache != nullptr;
    const int heads = a.q_heads + a.kv_heads * (cached ? 2 : 1);
    const int rows = nt * heads;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int sub = lane % LPR;
    const int D = a.head_dim;
    const bool live = sub * 8 < D;
    const int R = a.rotary_dim;
    const int pairs = R >> 1;
    const int chunks = (pairs + 7) >> 3;

    // the rows' loads first: they are in flight while the angles are computed
    auto source = [&](int row, int& tok, int& head) -> const uint4* {
        tok = row / heads;
        head = row - tok * heads;
        const int64_t t = t0 + tok;
        const unsigned short* base;
        int64_t at;
        if (head < a.q_heads) {
            base = static_cast<const unsigned short*>(a.q);
            at = t * a.q_token + head * a.q_head;
        } else if (head < a.q_heads + a.kv_heads) {
            base = static_cast<const unsigned short*>(a.k);
            at = t * a.k_token + (head - a.q_heads) * a.k_head;
        } else {
            base = static_cast<const unsigned short*>(a.v);
            at = t * a.v_token + (head - a.q_heads - a.kv_heads) * a.v_head;
        }
        return reinterpret_cast<const uint4*>(base + at) + sub;
    };
    const int row0 = warp * RPW + lane / LPR;
    uint4 raw[U];
    int tok[U], head[U];
    auto fetch = [&](int first) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = first + u * RPB;
            if (row < rows && live) raw[u] = *source(row, tok[u], head[u]);
        }
    };
    fetch(row0);
    uint4 qw = make_uint4(0, 0, 0, 0), kw = qw;
    if (a.q_weight != nullptr && live) qw = __ldg(static_cast<const uint4*>(a.q_weight) + sub);
    if (a.k_weight != nullptr && live) kw = __ldg(static_cast<const uint4*>(a.k_weight) + sub);

    for (int i = threadIdx.x; i < nt * pairs; i += kNormThreads) {
        const int k = i / pairs;
        const int p = i - k * pairs;
        const uint64_t phase = (uint64_t)(int64_t)__ldg(a.positions + t0 + k) *
                               (uint64_t)__ldg(reinterpret_cast<const long long*>(a.rope) + p);
        // 2^-32 turns, signed; sincospif takes half turns
        const float half_turns = (float)(int32_t)(uint32_t)(phase >> 32) * 0x1p-31f;
        float sn, cs;
        sincospif(half_turns, &sn, &cs);
        turn[k][pair_slot(p, chunks)] = make_float2(cs * a.rope_scale, sn * a.rope_scale);
    }
    if (cached) {
        for (int k = warp; k < nt; k += kNormThreads / 32) {
            const int r = warp_request(a.cu_seqlens, a.num_requests, t0 + k, lane);
            if (lane == 0) {
                const int64_t place = t0 + k - max(__ldg(a.cu_seqlens + r), 0);
                dst_s[k] = place < 0 ? -1
                                     : slot_offset(a.page_table, a.max_pages, a.page_size,
                                                   a.num_pages, a.page_stride, a.slot_stride, r,
                                                   __ldg(a.ctx_lens + r) + place);
            }
        }
    }
    __syncthreads();

    const float inv_d = 1.0f / (float)D;
    for (int first = row0; first - lane / LPR < rows; first += U * RPB) {
        if (first != row0) fetch(first);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = first + u * RPB;
            // a warp's rows go on together: its shuffles need every lane
            if (row - lane / LPR >= rows) break;
            const bool here = row < rows && live;
            const bool is_q = here && head[u] < a.q_heads;
            const bool is_v = here && head[u] >= a.q_heads + a.kv_heads;
            float x[8];
            if (here) {
                unpack8<E>(raw[u], x);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = 0.f;
            }
            float sq = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
#pragma unroll
            for (int m = LPR / 2; m >= 1; m >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, m);
            if ((is_q ? a.q_weight : a.k_weight) != nullptr) {
                const float inv = rsqrtf(fmaf(sq, inv_d, a.eps));
                float w[8];
                unpack8<E>(is_q ? qw : kw, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
            }
            const float2* cs = turn[here ? tok[u] : 0];
            if constexpr (kLayout == kPairsInterleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int p = sub * 4 + i;
                    if (p < pairs) {
                        const float2 c = cs[pair_slot(p, chunks)];
                        const float y0 = x[2 * i], y1 = x[2 * i + 1];
                        x[2 * i] = fmaf(y0, c.x, -y1 * c.y);
                        x[2 * i + 1] = fmaf(y1, c.x, y0 * c.y);
                    }
                }
            } else if constexpr (kLayout == kPairsHalves) {
                const int per = pairs >> 3;  // lanes of half the rotary part
                const int mate = sub < per ? lane + per : sub < 2 * per ? lane - per : lane;
                const int chunk = sub < per ? sub : sub - per;
                const float sign = sub < per ? -1.f : 1.f;
                const float4* plane = reinterpret_cast<const float4*>(cs);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float o0 = __shfl_sync(0xffffffffu, x[2 * i], mate);
                    const float o1 = __shfl_sync(0xffffffffu, x[2 * i + 1], mate);
                    if (sub < 2 * per) {
                        const float4 c = plane[i * chunks + chunk];
                        x[2 * i] = fmaf(x[2 * i], c.x, sign * o0 * c.y);
                        x[2 * i + 1] = fmaf(x[2 * i + 1], c.z, sign * o1 * c.w);
                    }
                }
            } else {
                float* mine = row_s + (threadIdx.x - sub) * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) mine[sub * 8 + i] = x[i];
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = sub * 8 + i;
                    if (e < R) {
                        const int p = e < pairs ? e : e - pairs;
                        const float2 c = cs[pair_slot(p, chunks)];
                        const float o = mine[e < pairs ? e + pairs : p];
                        x[i] = fmaf(x[i], c.x, (e < pairs ? -o : o) * c.y);
                    }
                }
                __syncwarp();
            }
            if (!here) continue;
            const uint4 y = is_v ? raw[u] : pack8<E>(x);
            unsigned short* dst;
            if (is_q) {
                dst = static_cast<unsigned short*>(a.q_out) + (t0 + tok[u]) * a.q_out_token +
                      head[u] * a.q_out_head;
            } else if (cached) {
                const int64_t at = dst_s[tok[u]];
                if (at < 0) continue;
                dst = is_v ? static_cast<unsigned short*>(a.v_cache) + at +
                                 (head[u] - a.q_heads - a.kv_heads) * a.head_stride
                           : static_cast<unsigned short*>(a.k_cache) + at +
                                 (head[u] - a.q_heads) * a.head_stride;
            } else {
                dst = static_cast<unsigned short*>(a.k_out) + (t0 + tok[u]) * a.k_out_token +
                      (head[u] - a.q_heads) * a.k_out_head;
            }
            reinterpret_cast<uint4*>(dst)[sub] = y;
        }
    }
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
    // one token a block until that makes as many blocks as the device holds
    // at once, then up to four
    int tokens = (int)(a.num_tokens / (8 * (int64_t)dev.sm_count));
    tokens = tokens < 1 ? 1 : tokens > kNormTokens ? kNormTokens : tokens;
    const dim3 grid((unsigned)((a.num_tokens + tokens - 1) / tokens));
    auto* fn = a.interleaved           ? qk_norm_rope_kernel<E, LPR, kPairsInterleaved>
               : a.rotary_dim % 16 == 0 ? qk_norm_rope_kernel<E, LPR, kPairsHalves>
                                        : qk_norm_rope_kernel<E, LPR, kPairsAnyHalves>;
    return launch_kernel(fn, grid, dim3(kNormThreads), 0, stream, programmatic_launch(), a,
                         tokens);
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
