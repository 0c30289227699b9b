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

// How a pair's two elements lie: side by side, half the rotary part apart with
// both in whole lanes (R / 2 a multiple of 8), or half of it apart anyhow.
enum PairLayout { kPairsInterleaved = 0, kPairsHalves = 1, kPairsAnyHalves = 2 };

// The table of a token's angles.  Pairs 2m and 2m + 1 make one 16-byte word
// (cos, cos, sin, sin), ready for paired arithmetic; word m of a chunk of eight
// pairs lies in plane m % 4, so that the lanes of a row read consecutive words.
__device__ __forceinline__ int turn_word(int pair, int chunks) {
    return ((pair & 7) >> 1) * chunks + (pair >> 3);
}

// Two 32-bit floats to a register pair: one instruction for both on sm_103a.
struct Pair {
    uint64_t v;
};
__device__ __forceinline__ Pair make_pair(float lo, float hi) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(Pair a, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair fma_pair(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

template <typename E>
__device__ __forceinline__ void unpack_row(uint4 v, Pair (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<E>(w[i]);
        x[i] = make_pair(f.x, f.y);
    }
}

template <typename E>
__device__ __forceinline__ uint4 pack_row(const Pair (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        split(x[i], lo, hi);
        w[i] = pack2<E>(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// How the block's warps meet the rows: `abreast` tokens at a time with
// 8 / abreast warps each, a warp taking every (8 / abreast)-th group of rows.
struct RowPlan {
    int32_t tokens;   // of a block, at most kNormTokens
    int32_t abreast;
    int32_t groups;   // of 32 / lanes-a-row rows, of a token
};

template <typename E, int LPR, int kLayout>
__global__ void __launch_bounds__(kNormThreads, 4)
qk_norm_rope_kernel(const __grid_constant__ ple_qk_norm_rope_args a, const RowPlan plan) {
    constexpr int RPW = 32 / LPR;     // rows a warp
    constexpr int kWarps = kNormThreads / 32;
    constexpr int U = 3;              // rows whose loads are in flight, a lane
    // cosines with sines, and with negated sines for the first half's elements
    __shared__ __align__(16) float4 turn[2][kNormTokens][kMaxPairs / 2];
    __shared__ int64_t dst_s[kNormTokens];
    __shared__ float row_s[kLayout == kPairsAnyHalves ? kNormThreads * 8 : 1];

    wait_grid_before();
    const int64_t t0 = (int64_t)blockIdx.x * plan.tokens;
    const int nt = (int)min((int64_t)plan.tokens, a.num_tokens - t0);
    const bool cached = a.k_cache != nullptr;
    const int qk_heads = a.q_heads + a.kv_heads;
    const int heads = qk_heads + (cached ? a.kv_heads : 0);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int sub = lane % LPR;
    const int in_group = lane / LPR;
    const bool live = sub * 8 < a.head_dim;
    const int pairs = a.rotary_dim >> 1;
    const int chunks = (pairs + 7) >> 3;
    const int per_token = kWarps / plan.abreast;   // warps of a token
    const int group0 = warp % per_token;

    // a row's elements of this lane; q, k and v rows follow one another
    auto load = [&](int tok, int group) -> uint4 {
        const int head = group * RPW + in_group;
        if (head >= heads || !live) return make_uint4(0, 0, 0, 0);
        const bool is_q = head < a.q_heads, is_k = head < qk_heads;
        const unsigned short* base =
            static_cast<const unsigned short*>(is_q ? a.q : is_k ? a.k : a.v);
        const int64_t at = (t0 + tok) * (is_q ? a.q_token : is_k ? a.k_token : a.v_token) +
                           (head - (is_q ? 0 : is_k ? a.q_heads : qk_heads)) *
                               (is_q ? a.q_head : is_k ? a.k_head : a.v_head);
        return __ldcs(reinterpret_cast<const uint4*>(base + at) + sub);
    };
    // the rows' loads first: they are in flight while the angles are computed
    int ltok = warp / per_token, lgroup = group0;
    auto next = [&](int& tok, int& group) {
        group += per_token;
        if (group >= plan.groups) {
            group = group0;
            tok += plan.abreast;
        }
    };
    int tok = ltok, group = lgroup;
    uint4 raw[U];
    const bool any = group0 < plan.groups;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (any && ltok < nt) raw[u] = load(ltok, lgroup);
        next(ltok, lgroup);
    }
    Pair qw[4], kw[4];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const uint4* from = static_cast<const uint4*>(side == 0 ? a.q_weight : a.k_weight);
        Pair(&w)[4] = side == 0 ? qw : kw;
        if (from != nullptr && live) {
            unpack_row<E>(__ldg(from + sub), w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = make_pair(1.f, 1.f);
        }
    }
    const bool norms = a.q_weight != nullptr || a.k_weight != nullptr;

    for (int i = threadIdx.x; i < nt * pairs; i += kNormThreads) {
        const int k = i / pairs;
        const int p = i - k * pairs;
        const uint64_t phase = (uint64_t)(int64_t)__ldg(a.positions + t0 + k) *
                               (uint64_t)__ldg(reinterpret_cast<const long long*>(a.rope) + p);
        // 2^-32 turns, signed; sincospif takes half turns
        const float half_turns = (float)(int32_t)(uint32_t)(phase >> 32) * 0x1p-31f;
        float sn, cs;
        sincospif(half_turns, &sn, &cs);
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            float* word = reinterpret_cast<float*>(&turn[side][k][turn_word(p, chunks)]);
            word[p & 1] = cs * a.rope_scale;
            word[2 + (p & 1)] = side == 0 ? sn * a.rope_scale : -sn * a.rope_scale;
        }
    }
    if (cached) {
        for (int k = warp; k < nt; k += kWarps) {
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
    if (!any) return;

    const float inv_d = 1.0f / (float)a.head_dim;
    while (tok < nt) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (tok >= nt) break;  // a warp's rows go on together
            const int head = group * RPW + in_group;
            const uint4 mine = raw[u];
            if (ltok < nt) raw[u] = load(ltok, lgroup);
            next(ltok, lgroup);
            const bool here = head < heads && live;
            const bool is_q = head < a.q_heads;
            uint4 y = mine;
            if (group * RPW < qk_heads) {  // else value rows alone
                Pair x[4];
                unpack_row<E>(mine, x);
                if (norms) {
                    Pair sq = x[0] * x[0];
#pragma unroll
                    for (int i = 1; i < 4; ++i) sq = fma_pair(x[i], x[i], sq);
                    float lo, hi;
                    split(sq, lo, hi);
                    lo += hi;
#pragma unroll
                    for (int m = LPR / 2; m >= 1; m >>= 1)
                        lo += __shfl_xor_sync(0xffffffffu, lo, m);
                    // rows with a norm and rows without may share a warp
                    const bool norm = (is_q ? a.q_weight : a.k_weight) != nullptr;
                    const float inv = norm ? rsqrtf(fmaf(lo, inv_d, a.eps)) : 1.f;
                    const Pair inv2 = make_pair(inv, inv);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = x[i] * (inv2 * (is_q ? qw[i] : kw[i]));
                }
                if constexpr (kLayout == kPairsInterleaved) {
                    const float4* word = turn[0][tok];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int p = sub * 4 + i;
                        if (p < pairs) {
                            const float* w = reinterpret_cast<const float*>(
                                &word[turn_word(p, chunks)]);
                            const float c = w[p & 1], sn = w[2 + (p & 1)];
                            float y0, y1;
                            split(x[i], y0, y1);
                            x[i] = make_pair(fmaf(y0, c, -y1 * sn), fmaf(y1, c, y0 * sn));
                        }
                    }
                } else if constexpr (kLayout == kPairsHalves) {
                    const int per = pairs >> 3;  // lanes of half the rotary part
                    const bool low = sub < per;
                    const int mate = low ? lane + per : sub < 2 * per ? lane - per : lane;
                    const float4* word = &turn[low ? 1 : 0][tok][low ? sub : sub - per];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float lo, hi;
                        split(x[i], lo, hi);
                        const Pair o = make_pair(__shfl_sync(0xffffffffu, lo, mate),
                                                 __shfl_sync(0xffffffffu, hi, mate));
                        if (sub < 2 * per) {
                            const float4 w = word[i * chunks];
                            x[i] = fma_pair(x[i], make_pair(w.x, w.y), o * make_pair(w.z, w.w));
                        }
                    }
                } else {
                    float* row = row_s + (threadIdx.x - sub) * 8;
                    float z[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        split(x[i], z[2 * i], z[2 * i + 1]);
                        row[sub * 8 + 2 * i] = z[2 * i];
                        row[sub * 8 + 2 * i + 1] = z[2 * i + 1];
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int e = sub * 8 + i;
                        if (e < 2 * pairs) {
                            const int p = e < pairs ? e : e - pairs;
                            const float* w = reinterpret_cast<const float*>(
                                &turn[e < pairs ? 1 : 0][tok][turn_word(p, chunks)]);
                            z[i] = fmaf(z[i], w[p & 1],
                                        row[e < pairs ? e + pairs : p] * w[2 + (p & 1)]);
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = make_pair(z[2 * i], z[2 * i + 1]);
                }
                if (head < qk_heads) y = pack_row<E>(x);
            }
            if (here) {
                const int64_t slot = cached ? dst_s[tok] : 0;
                unsigned short* dst;
                int64_t at;
                if (is_q) {
                    dst = static_cast<unsigned short*>(a.q_out);
                    at = (t0 + tok) * a.q_out_token + head * a.q_out_head;
                } else if (cached) {
                    const bool is_k = head < qk_heads;
                    dst = static_cast<unsigned short*>(is_k ? a.k_cache : a.v_cache);
                    at = slot + (head - (is_k ? a.q_heads : qk_heads)) * a.head_stride;
                } else {
                    dst = static_cast<unsigned short*>(a.k_out);
                    at = (t0 + tok) * a.k_out_token + (head - a.q_heads) * a.k_out_head;
                }
                if (is_q || slot >= 0) reinterpret_cast<uint4*>(dst + at)[sub] = y;
            }
            next(tok, group);
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
    constexpr int RPW = 32 / LPR;
    constexpr int kWarps = kNormThreads / 32;
    RowPlan plan;
    // one token a block until that makes as many blocks as the device holds
    // at once, then up to four
    const int64_t tokens = a.num_tokens / (4 * (int64_t)dev.sm_count);
    plan.tokens = (int)(tokens < 1 ? 1 : tokens > kNormTokens ? kNormTokens : tokens);
    const int heads = a.q_heads + a.kv_heads * (a.k_cache != nullptr ? 2 : 1);
    plan.groups = (heads + RPW - 1) / RPW;
    // as few warps a token as leave none idle in its last step, but all of them
    // on a block's only token
    plan.abreast = 1;
    int best = 0;
    for (int abreast = 1; abreast <= plan.tokens && abreast <= kWarps; abreast *= 2) {
        const int per = kWarps / abreast;
        const int used = plan.groups * 1000 / ((plan.groups + per - 1) / per * per);
        if (used > best) {
            best = used;
            plan.abreast = abreast;
        }
    }
    const dim3 grid((unsigned)((a.num_tokens + plan.tokens - 1) / plan.tokens));
    auto* fn = a.interleaved           ? qk_norm_rope_kernel<E, LPR, kPairsInterleaved>
               : a.rotary_dim % 16 == 0 ? qk_norm_rope_kernel<E, LPR, kPairsHalves>
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
