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
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "ple_tree_common.cuh"

namespace ple {
namespace {

constexpr int kNormThreads = 256;
// Tokens a block, for batches that fill the device; resident blocks an SM.  On the
// 32004-token prompts (786 MB) 145 us with five blocks and eight tokens (5.4 TB/s);
// four blocks 157, six 149, four tokens 148, sixteen 173.  Two to four rows in flight
// a warp instead of one ahead measured no faster (153 to 157), and the kernel
// with its arithmetic taken out, the copies alone, takes 138: what is left is how
// fast rows of 256 bytes between the product's, the queries' and the pages' layouts
// move at all.
constexpr int kNormTokens = 8;
constexpr int kNormBlocks = 5;
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
// R a multiple of 8, or half of it apart anyhow.
enum PairLayout { kPairsInterleaved = 0, kPairsHalves = 1, kPairsAnyHalves = 2 };

// The table of a token's angles: pairs 2m and 2m + 1 make 16-byte word m, (cos, cos,
// sin, sin), ready for paired arithmetic.

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

// A lane's eight elements, as two pieces of four.
struct Row {
    uint2 a, b;
};
__device__ __forceinline__ Row load_row(const unsigned short* p, int second) {
    Row r;
    r.a = __ldcg(reinterpret_cast<const uint2*>(p));
    r.b = __ldcg(reinterpret_cast<const uint2*>(p + second));
    return r;
}
__device__ __forceinline__ void store_row(unsigned short* p, int second, Row r) {
    *reinterpret_cast<uint2*>(p) = r.a;
    *reinterpret_cast<uint2*>(p + second) = r.b;
}

template <typename E>
__device__ __forceinline__ void unpack_row(Row v, Pair (&x)[4]) {
    const uint32_t w[4] = {v.a.x, v.a.y, v.b.x, v.b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<E>(w[i]);
        x[i] = make_pair(f.x, f.y);
    }
}

template <typename E>
__device__ __forceinline__ Row pack_row(const Pair (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        split(x[i], lo, hi);
        w[i] = pack2<E>(lo, hi);
    }
    return Row{make_uint2(w[0], w[1]), make_uint2(w[2], w[3])};
}

// A token's rows come in groups of as many as a warp holds, all of one kind:
// queries, then keys, then values.  A warp takes one group after another, each for
// all tokens of the block, so that a group's addresses are set up once and only
// step from token to token.
struct RowPlan {
    int32_t tokens;   // of a block, at most kNormTokens
    int32_t q_groups, kv_groups;
};

template <typename E, int LPR, int kLayout>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks)
qk_norm_rope_kernel(const __grid_constant__ ple_qk_norm_rope_args a, const RowPlan plan) {
    constexpr int RPW = 32 / LPR;     // rows a warp
    constexpr int kWarps = kNormThreads / 32;
    __shared__ __align__(16) float4 turn[kNormTokens][kMaxPairs / 2];
    __shared__ int64_t dst_s[kNormTokens];
    __shared__ float row_s[kLayout == kPairsAnyHalves ? kNormThreads * 8 : 1];

    wait_grid_before();
    const int64_t t0 = (int64_t)blockIdx.x * plan.tokens;
    const int nt = (int)min((int64_t)plan.tokens, a.num_tokens - t0);
    const bool cached = a.k_cache != nullptr;
    const int k_end = plan.q_groups + plan.kv_groups;
    const int groups = k_end + (cached ? plan.kv_groups : 0);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int sub = lane % LPR;
    const int in_group = lane / LPR;
    const bool live = sub * 8 < a.head_dim;
    const int pairs = a.rotary_dim >> 1;
    // A lane's eight elements: four and the four that they turn with (halves),
    // or eight in a row (side by side, and what is not turned).
    const bool turns = kLayout == kPairsHalves ? sub * 8 < a.rotary_dim : true;
    const int first = kLayout == kPairsHalves && turns ? sub * 4 : sub * 8;
    const int second = kLayout == kPairsHalves && turns ? pairs : 4;

    // a lane's row of a group, at the block's first token: its address, the step
    // to the next token's, and whether there is such a row
    const unsigned short* src;
    int64_t src_step;
    bool here;
    auto open_group = [&](int group) {
        const bool is_q = group < plan.q_groups, is_k = group < k_end;
        const int head = (group - (is_q ? 0 : is_k ? plan.q_groups : k_end)) * RPW + in_group;
        src_step = is_q ? a.q_token : is_k ? a.k_token : a.v_token;
        src = static_cast<const unsigned short*>(is_q ? a.q : is_k ? a.k : a.v) + t0 * src_step +
              head * (is_q ? a.q_head : is_k ? a.k_head : a.v_head) + first;
        here = live && group < groups && head < (is_q ? a.q_heads : a.kv_heads);
    };
    // the first rows' loads are in flight while the angles are computed, and every
    // later row's while the one before it is
    int group = blockIdx.y * kWarps + warp;
    open_group(group);
    Row ahead = {};
    if (here) ahead = load_row(src, second);

    for (int i = threadIdx.x; i < nt * pairs; i += kNormThreads) {
        const int k = i / pairs;
        const int p = i - k * pairs;
        const uint64_t phase = (uint64_t)(int64_t)__ldg(a.positions + t0 + k) *
                               (uint64_t)__ldg(reinterpret_cast<const long long*>(a.rope) + p);
        // 2^-32 turns, signed; sincospif takes half turns
        const float half_turns = (float)(int32_t)(uint32_t)(phase >> 32) * 0x1p-31f;
        float sn, cs;
        sincospif(half_turns, &sn, &cs);
        float* word = reinterpret_cast<float*>(&turn[k][p >> 1]);
        word[p & 1] = cs * a.rope_scale;
        word[2 + (p & 1)] = sn * a.rope_scale;
    }
    if (cached) {
        for (int k = warp; k < nt; k += kWarps) {
            const int r = warp_request(a.cu_seqlens, a.num_requests, t0 + k, lane);
            if (lane == 0) {
                // a token past the last request's is padding: it has no slot
                const int64_t place = t0 + k - max(__ldg(a.cu_seqlens + r), 0);
                const bool node = place >= 0 && t0 + k < __ldg(a.cu_seqlens + r + 1);
                dst_s[k] = node ? slot_offset(a.page_table, a.max_pages, a.page_size, a.num_pages,
                                              a.page_stride, a.slot_stride, r,
                                              __ldg(a.ctx_lens + r) + place)
                                : -1;
            }
        }
    }
    __syncthreads();

    const float inv_d = 1.0f / (float)a.head_dim;
    // rows of one group through all tokens: turned (queries, keys) or copied, to
    // `dst` stepping from token to token or to the tokens' slots behind it
    auto run = [&](auto turned, auto slots, unsigned short* dst, int64_t dst_step,
                   const void* weight) {
        const bool here_now = here;
        // behind this group's last row comes the next group's first
        group += kWarps * gridDim.y;
        const unsigned short* at = src;
        const int64_t at_step = src_step;
        open_group(group);
        Pair w[4];
        if constexpr (turned) {
            Row r = {};
            if (weight != nullptr && live) {
                const unsigned short* from = static_cast<const unsigned short*>(weight) + first;
                r.a = __ldg(reinterpret_cast<const uint2*>(from));
                r.b = __ldg(reinterpret_cast<const uint2*>(from + second));
            }
            unpack_row<E>(r, w);
        }
        for (int tok = 0; tok < nt; ++tok) {
            Row y = ahead;
            at += at_step;
            if (tok + 1 == nt) {
                if (here) ahead = load_row(src, second);
            } else if (here_now) {
                ahead = load_row(at, second);
            }
            if constexpr (turned) {
                Pair x[4];
                unpack_row<E>(y, x);
                if (weight != nullptr) {
                    Pair sq = x[0] * x[0];
#pragma unroll
                    for (int i = 1; i < 4; ++i) sq = fma_pair(x[i], x[i], sq);
                    float lo, hi;
                    split(sq, lo, hi);
                    lo += hi;
#pragma unroll
                    for (int m = LPR / 2; m >= 1; m >>= 1)
                        lo += __shfl_xor_sync(0xffffffffu, lo, m);
                    const float inv = rsqrtf(fmaf(lo, inv_d, a.eps));
                    const Pair inv2 = make_pair(inv, inv);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = x[i] * (inv2 * w[i]);
                }
                if constexpr (kLayout == kPairsHalves) {
                    if (turns) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float4 v = turn[tok][sub * 2 + i];
                            const Pair c = make_pair(v.x, v.y), n = make_pair(v.z, v.w);
                            const Pair lo = x[i], hi = x[i + 2];
                            x[i] = fma_pair(lo, c, hi * make_pair(-v.z, -v.w));
                            x[i + 2] = fma_pair(hi, c, lo * n);
                        }
                    }
                } else if constexpr (kLayout == kPairsInterleaved) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float4 v = turn[tok][sub * 2 + i];
                        const int p = sub * 4 + 2 * i;
                        float y0, y1;
                        if (p < pairs) {
                            split(x[2 * i], y0, y1);
                            x[2 * i] = make_pair(fmaf(y0, v.x, -y1 * v.z), fmaf(y1, v.x, y0 * v.z));
                        }
                        if (p + 1 < pairs) {
                            split(x[2 * i + 1], y0, y1);
                            x[2 * i + 1] =
                                make_pair(fmaf(y0, v.y, -y1 * v.w), fmaf(y1, v.y, y0 * v.w));
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
                            const float* v = reinterpret_cast<const float*>(&turn[tok][p >> 1]);
                            const float o = row[e < pairs ? e + pairs : p];
                            z[i] = fmaf(z[i], v[p & 1], (e < pairs ? -o : o) * v[2 + (p & 1)]);
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = make_pair(z[2 * i], z[2 * i + 1]);
                }
                y = pack_row<E>(x);
            }
            if constexpr (slots) {
                const int64_t slot = dst_s[tok];
                if (here_now && slot >= 0) store_row(dst + slot, second, y);
            } else {
                if (here_now) store_row(dst, second, y);
                dst += dst_step;
            }
        }
    };
    using Yes = std::true_type;
    using No = std::false_type;
    while (group < groups) {
        if (group < plan.q_groups) {
            const int head = group * RPW + in_group;
            run(Yes{}, No{},
                static_cast<unsigned short*>(a.q_out) + t0 * a.q_out_token + head * a.q_out_head +
                    first,
                a.q_out_token, a.q_weight);
        } else if (group < k_end) {
            const int head = (group - plan.q_groups) * RPW + in_group;
            if (cached)
                run(Yes{}, Yes{},
                    static_cast<unsigned short*>(a.k_cache) + head * a.head_stride + first, 0,
                    a.k_weight);
            else
                run(Yes{}, No{},
                    static_cast<unsigned short*>(a.k_out) + t0 * a.k_out_token +
                        head * a.k_out_head + first,
                    a.k_out_token, a.k_weight);
        } else {
            const int head = (group - k_end) * RPW + in_group;
            run(No{}, Yes{},
                static_cast<unsigned short*>(a.v_cache) + head * a.head_stride + first, 0,
                nullptr);
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
