// Norms of queries and keys, their rotation, and the append of keys and values in 8
// bits to the paged cache, in one pass, on sm_103a.
//
// Query rows are those of ple_norm_rope.cuh.  Keys (after norm and rotation, in 32
// bits) and values become elements of e4m3 under one scale for each block of slots and
// head: the least power of two that takes the block's largest finite amount to at most
// 448.  Where a block held tokens before, its scale never falls, and where it grows
// their elements are rounded anew: a power of two only moves their exponents, so all
// but those near the elements' least keep their values.
//
// Layout.  A block of threads takes the cache's blocks that begin among its tokens (or
// go on with a request's first one): their tokens' sines and cosines are computed once,
// and a warp takes one head's keys or values of a cache block, rows as in
// ple_norm_rope.cuh, twice: once for the largest amount and, with the scale known, once
// for the elements, the factors of the norms kept in between.  Values' amounts are
// compared as bits, two at a time.
//
// 32003 prompt tokens, 32 and 2 x 8 heads of 128 in blocks of 16: 166 us, 4.3 TB/s of the
// rows' 721 MB (106 us at the measured copy's rate; the copy of 16-bit rows 146).  Bound by
// instructions: appended rows alone take 73 us (29 of bytes) at 57% of the issue slots, 110
// instructions for a warp's two rows.  One decoded token 4.0 us, a launch and a few
// dependent reads.  Not kept: several warps to a head, so that its rows are read once (alone
// 97 us against 87: registers run out), and turned keys kept in registers (the same).
#include "ple_fp8.cuh"
#include "ple_norm_rope.cuh"
#include "ple_tree_fp8_internal.h"

namespace ple {
namespace {

constexpr int kAppendBlocks = 4;    // resident blocks an SM
constexpr int kHeldRows = 4;        // of a lane, in registers
constexpr int kAppendTokens = 16;   // most tokens a block of threads looks for blocks among
constexpr int kWalkTasks = 32;      // of a warp, between whose two walks others' come

// Tokens whose angles a block of threads holds: all of a cache block's, or, where they would
// take more than 48 KB, 16 KB of them (kWalk).  The 32003-token prompts, all at once and in
// walks: heads of 256 in blocks of 128 tokens (128 KB) 834 and 396 us, in blocks of 64
// (64 KB) 484 and 346; of 128 in blocks of 128 (64 KB) 247 and 191, in blocks of 64 (32 KB)
// 165 and 191.
constexpr int kMostTable = 48 * 1024;
template <int LPR, bool kWalk>
constexpr int kTableTokens = kWalk ? 512 / LPR : kMostBlock;

struct AppendPlan {
    RowPlan rows;          // the queries'
    int32_t kv_blocks;     // blocks of threads that append; behind them those of queries
    int32_t kv_tokens;     // each one's tokens
    int32_t shift;         // log2 of a cache block's tokens
};

// Sine and cosine of a phase in 2^-64 turns, rounded about once, so that few keys near the
// border between two elements come to the other side: of 4 * 10^8 phases worked through in
// these steps each came to 0.73 units of its last place or less where it is 2^-27 or more,
// and below that, next to a zero, to 2^-51.  The angle from the nearest quarter turn, at
// most pi / 4, is p + e in two floats; Taylor's series give what is added to p and to 1.
__device__ __forceinline__ void sine_cosine(uint64_t phase, float& sn, float& cs) {
    constexpr float kPi = 3.14159274f, kPiRest = -8.74227766e-8f;   // their sum is pi
    const uint32_t turn = (uint32_t)(phase >> 32);                  // 2^-32 turns
    const uint32_t quarter = (turn + (1u << 29)) >> 30;
    const int32_t rest = (int32_t)(turn - (quarter << 30));
    const float near = (float)rest;                                 // below 2^30: converts back
    const float y = near * 0x1p-31f;                                // half turns
    const float y_rest = ((float)(rest - (int32_t)near) + (float)(uint32_t)phase * 0x1p-32f) *
                         0x1p-31f;
    const float p = y * kPi;
    const float e = fmaf(y_rest, kPi, fmaf(y, kPiRest, fmaf(y, kPi, -p)));
    const float z = p * p, z_rest = fmaf(p, p, -z);
    const float odd = fmaf(fmaf(fmaf(1.f / 362880, z, -1.f / 5040), z, 1.f / 120), z, -1.f / 6);
    const float even = fmaf(fmaf(fmaf(-1.f / 3628800, z, 1.f / 40320), z, -1.f / 720), z, 1.f / 24);
    const float sine = p + fmaf(p * z, odd, fmaf(-0.5f * z, e, e));
    const float one = fmaf(-0.5f, z, 1.f);
    const float lost = fmaf(-0.5f, z, 1.f - one);
    const float cosine = one + (lost + fmaf(z * z, even, fmaf(-0.5f, z_rest, -p * e)));
    sn = quarter & 1 ? cosine : sine;
    cs = quarter & 1 ? sine : cosine;
    if (quarter & 2) sn = -sn;
    if ((quarter + 1) & 2) cs = -cs;
}

// A lane's eight finite values as elements, four and four; inv: the reciprocal of a power
// of two.
__device__ __forceinline__ uint2 row_elements(const Pair (&x)[4], float inv) {
    const Pair up = make_pair(inv, inv);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        split(x[i] * up, lo, hi);
        w[i] = elements_of(lo, hi);
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// Any eight values: what is not finite becomes NaN, and under a scale that is no power of
// two, as a cache may have been filled with, the product is mended by what it lacks
// (Markstein 1990): a quotient on the border of two elements has to be met exactly.
__device__ __forceinline__ uint2 any_row_elements(const Pair (&x)[4], float scale, float inv) {
    const Pair whole = make_pair(scale, scale), up = make_pair(inv, inv);
    const Pair less = make_pair(-inv, -inv), minus = make_pair(-1.f, -1.f);
    const bool power = (__float_as_uint(scale) & 0x7FFFFFu) == 0;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        Pair y = x[i] * up;
        // (what y is above the quotient, times less: so that a zero keeps its sign)
        if (!power) y = fma_pair(fma_pair(y, whole, x[i] * minus), less, y);
        float lo, hi, lo_x, hi_x;
        split(y, lo, hi);
        split(x[i], lo_x, hi_x);
        lo = fabsf(lo_x) < INFINITY ? lo : __int_as_float(0x7FC00000);
        hi = fabsf(hi_x) < INFINITY ? hi : __int_as_float(0x7FC00000);
        w[i] = elements_of(lo, hi);
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// The largest amount of a lane's values, NaN passed over.
__device__ __forceinline__ float amount(const Pair (&x)[4]) {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        split(x[i], lo, hi);
        most = fmaxf(most, fmaxf(fabsf(lo), fabsf(hi)));
    }
    return most;
}

// The same of values of 16 bits, which without their signs are in the order of their bits,
// two at a time; a NaN is above infinity.
__device__ __forceinline__ uint32_t amount_bits(uint32_t most, const Row& row) {
    most = __vmaxu2(most, row.a.x & 0x7FFF7FFFu);
    most = __vmaxu2(most, row.a.y & 0x7FFF7FFFu);
    most = __vmaxu2(most, row.b.x & 0x7FFF7FFFu);
    return __vmaxu2(most, row.b.y & 0x7FFF7FFFu);
}

// Of finite values alone.
__device__ __forceinline__ float finite_amount(const Pair (&x)[4]) {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        split(x[i], lo, hi);
        lo = fabsf(lo);
        hi = fabsf(hi);
        most = fmaxf(most, fmaxf(lo < INFINITY ? lo : 0.f, hi < INFINITY ? hi : 0.f));
    }
    return most;
}

template <typename E, int LPR, int kLayout, bool kWalk>
__device__ __forceinline__ void append_blocks(const ple_qk_norm_rope_fp8_args& f,
                                              const AppendPlan& plan, int block_x, int block_y,
                                              int grid_y) {
    constexpr int RPW = 32 / LPR;
    constexpr int kWarps = kNormThreads / 32;
    constexpr int kPitch = 2 * LPR;   // a token's angles, 16-byte words
    extern __shared__ __align__(16) float4 angles[];
    __shared__ float row_s[kLayout == kPairsAnyHalves ? kNormThreads * 8 : 1];
    const ple_qk_norm_rope_args& a = f.base;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane % LPR, in_group = lane / LPR;
    const bool live = sub * 8 < a.head_dim;
    const int pairs = a.rotary_dim >> 1;
    const bool turns = kLayout == kPairsHalves ? sub * 8 < a.rotary_dim : true;
    const int first = kLayout == kPairsHalves && turns ? sub * 4 : sub * 8;
    const int second = kLayout == kPairsHalves && turns ? pairs : 4;
    const float inv_d = 1.0f / (float)a.head_dim;
    const int size = 1 << plan.shift;
    // a thread's tokens and pairs, when it works out angles
    const int k0 = pairs ? threadIdx.x / pairs : 0, p0 = threadIdx.x - k0 * pairs;
    const int k_step = pairs ? kNormThreads / pairs : 0, p_step = kNormThreads - k_step * pairs;
    // the factors of keys' norms, for their second turn
    __shared__ float factor_s[kWarps][kTableTokens<LPR, kWalk> + RPW];
    // what is known of a warp's heads between two walks over a block's rows: the largest
    // amount, then the scale; whether a value is infinite
    __shared__ float known_s[kWarps][kWalk ? kWalkTasks : 1];
    __shared__ bool infinite_s[kWarps][kWalk ? kWalkTasks : 1];

    wait_grid_before();
    int64_t t = (int64_t)block_x * plan.kv_tokens;
    const int64_t t_end = min(t + plan.kv_tokens, a.num_tokens);
    int r = warp_request(a.cu_seqlens, a.num_requests, t, lane);
    int32_t begin, end;
    request_nodes(a.cu_seqlens, r, a.num_tokens, begin, end);
    while (t < t_end) {
        while (t >= end && r + 1 < a.num_requests)
            request_nodes(a.cu_seqlens, ++r, a.num_tokens, begin, end);
        if (t >= end) break;                      // padding
        if (t < begin) {
            t = begin;
            continue;
        }
        const int64_t ctx = max(__ldg(a.ctx_lens + r), 0);
        const int64_t slot = ctx + (t - begin);
        const int into = (int)(slot & (size - 1));
        if (t > begin && into != 0) {             // another block of threads has it
            t = min(t + (size - into), (int64_t)end);
            continue;
        }
        const int count = (int)min((int64_t)(size - into), end - t);
        const int64_t page_at = slot / a.page_size;
        int32_t page = -1;
        if (page_at < a.max_pages) page = __ldg(a.page_table + (int64_t)r * a.max_pages + page_at);
        if (page < 0 || page >= a.num_pages) {    // dropped
            t += count;
            continue;
        }
        const int in_page = (int)(slot - page_at * a.page_size);
        // the angles of rows c0 .. c1 - 1
        auto work_out_angles = [&](int c0, int c1) {
            if (pairs == 0) return;
            __syncthreads();
            for (int k = k0, p = p0; k < c1 - c0; k += k_step, p += p_step) {
                if (p >= pairs) {
                    p -= pairs;
                    if (++k >= c1 - c0) break;
                }
                const uint64_t phase = (uint64_t)(int64_t)__ldg(a.positions + t + c0 + k) *
                                       (uint64_t)__ldg(
                                           reinterpret_cast<const long long*>(a.rope) + p);
                float sn, cs;
                sine_cosine(phase, sn, cs);
                float* word = reinterpret_cast<float*>(&angles[k * kPitch + (p >> 1)]);
                word[p & 1] = cs * a.rope_scale;
                word[2 + (p & 1)] = sn * a.rope_scale;
            }
            __syncthreads();
        };
        // One head's keys, or values, rows c0 .. c1 - 1: their largest amount is looked for, the
        // block's scale settled, elements stored; number: of the warp's tasks.
        auto append = [&](auto keys, int head, int number, int c0, int c1, bool look, bool settle,
                          bool store) {
            constexpr bool is_k = keys;
            // values do not turn: a lane's eight elements stand together
            const int at0 = is_k ? first : sub * 8, at1 = is_k ? second : 4;
            const int64_t step = is_k ? a.k_token : a.v_token;
            const unsigned short* src = static_cast<const unsigned short*>(is_k ? a.k : a.v) +
                                        (t + in_group) * step +
                                        head * (is_k ? a.k_head : a.v_head) + at0;
            uint8_t* dst = static_cast<uint8_t*>(is_k ? a.k_cache : a.v_cache) +
                           page * a.page_stride + head * a.head_stride +
                           (in_page + in_group) * a.slot_stride + at0;
            unsigned short* scale_at =
                static_cast<unsigned short*>(is_k ? f.scales.k : f.scales.v) +
                page * f.scales.page_stride + head * f.scales.head_stride +
                (in_page >> plan.shift);
            const bool normed = is_k && a.k_weight != nullptr;
            Pair w[4];
            if constexpr (is_k) {
                Row row = {};
                if (normed && live) {
                    const unsigned short* from =
                        static_cast<const unsigned short*>(a.k_weight) + first;
                    row.a = __ldg(reinterpret_cast<const uint2*>(from));
                    row.b = __ldg(reinterpret_cast<const uint2*>(from + second));
                }
                unpack_row<E>(row, w);
            }
            unsigned short before = 0;
            if (settle && into != 0) before = *scale_at;
            Row held[kHeldRows];
            auto load = [&](const unsigned short* from, int i0) {
#pragma unroll
                for (int i = 0; i < kHeldRows; ++i) {
                    held[i] = Row{};
                    if (live && i0 + i * RPW + in_group < c1) held[i] = load_row(from, at1);
                    from += RPW * step;
                }
            };
            auto turned = [&](bool again, const Row& row, int k, Pair (&x)[4]) {
                unpack_row<E>(row, x);
                if constexpr (is_k) {
                    if (normed) {
                        float* kept = &factor_s[warp][k - c0 + in_group];
                        float factor;
                        if (again) {
                            factor = *kept;
                        } else {
                            factor = norm_factor<LPR>(x, inv_d, a.eps);
                            if (sub == 0) *kept = factor;
                        }
                        scale_row(x, w, factor);
                    }
                    rotate_row<LPR, kLayout>(
                        x, angles + min(k - c0 + in_group, c1 - c0 - 1) * kPitch, sub, pairs, turns,
                        row_s);
                }
            };
            auto put = [&](uint8_t* to, int k, uint2 e) {
                if (!live || k + in_group >= c1) return;
                if constexpr (is_k) {
                    *reinterpret_cast<uint32_t*>(to) = e.x;
                    *reinterpret_cast<uint32_t*>(to + second) = e.y;
                } else {
                    *reinterpret_cast<uint2*>(to) = e;
                }
            };
            float most = 0.f;
            bool infinite = false;
            if (look) {
                uint32_t most_bits = 0;
                for (int i0 = c0; i0 < c1; i0 += kHeldRows * RPW) {
                    load(src + i0 * step, i0);
#pragma unroll
                    for (int i = 0; i < kHeldRows; ++i) {
                        if (i0 + i * RPW >= c1) break;
                        if constexpr (is_k) {
                            Pair x[4];
                            turned(false, held[i], i0 + i * RPW, x);
                            most = fmaxf(most, amount(x));
                        } else {
                            most_bits = amount_bits(most_bits, held[i]);
                        }
                    }
                }
                if constexpr (!is_k) {
                    const float2 both = unpack2<E>(most_bits);
                    // a NaN is looked at too: it says that there is one
                    most = both.x < INFINITY && both.y < INFINITY ? fmaxf(both.x, both.y)
                                                                  : INFINITY;
                }
#pragma unroll
                for (int d = 16; d >= 1; d >>= 1)
                    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                __syncwarp();   // factors
                infinite = !(most < INFINITY);
                if (infinite) {
                    most = 0.f;
#pragma unroll 1
                    for (int k = c0; k < c1; k += RPW) {
                        load(src + k * step, k);
                        Pair x[4];
                        turned(true, held[0], k, x);
                        most = fmaxf(most, finite_amount(x));
                    }
#pragma unroll
                    for (int d = 16; d >= 1; d >>= 1)
                        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                }
                if (c0 != 0) {
                    most = fmaxf(most, known_s[warp][number]);
                    infinite = infinite || infinite_s[warp][number];
                }
            } else {
                most = known_s[warp][number];
                infinite = infinite_s[warp][number];
            }
            float scale = most;
            if (settle) {
                scale = __uint_as_float((uint32_t)(127 + exponent_for(most)) << 23);
                if (into != 0) {
                    const float old = scale_value(before);
                    if (scale > old) {
                        // the tokens that the block holds, under the new scale
                        const float shrink = old / scale;
                        uint8_t* row = dst - (int64_t)into * a.slot_stride - at0 + sub * 8;
#pragma unroll 1
                        for (int k = 0; k + in_group < into; k += RPW) {
                            if (!live) break;
                            uint2* at = reinterpret_cast<uint2*>(row + k * a.slot_stride);
                            const uint2 v = *at;
                            *at = make_uint2(scaled_elements(v.x, shrink),
                                             scaled_elements(v.y, shrink));
                        }
                    } else {
                        scale = old;
                    }
                }
                __syncwarp();   // all lanes have read what lies there
                if (lane == 0) *scale_at = (unsigned short)(__float_as_uint(scale) >> 16);
            }
            if (!(look && store)) {
                __syncwarp();
                if (lane == 0) {
                    known_s[warp][number] = scale;
                    infinite_s[warp][number] = infinite;
                }
                __syncwarp();
            }
            if (!store) return;
            const float inv = 1.0f / scale;
            if (infinite || (__float_as_uint(scale) & 0x7FFFFFu) != 0) {
#pragma unroll 1
                for (int k = c0; k < c1; k += RPW) {
                    load(src + k * step, k);
                    Pair x[4];
                    turned(look, held[0], k, x);
                    put(dst + k * a.slot_stride, k, any_row_elements(x, scale, inv));
                }
            } else {
                for (int i0 = c0; i0 < c1; i0 += kHeldRows * RPW) {
                    if (!look || c1 > kHeldRows * RPW) load(src + i0 * step, i0);
                    uint8_t* to = dst + i0 * a.slot_stride;
#pragma unroll
                    for (int i = 0; i < kHeldRows; ++i) {
                        if (i0 + i * RPW >= c1) break;
                        Pair x[4];
                        turned(look, held[i], i0 + i * RPW, x);
                        put(to, i0 + i * RPW, row_elements(x, inv));
                        to += RPW * a.slot_stride;
                    }
                }
            }
        };
        const int task = block_y * kWarps + warp, task_step = kWarps * grid_y;
        auto append_task = [&](int task, int number, int c0, int c1, bool look, bool settle,
                               bool store) {
            if (task < a.kv_heads)
                append(std::true_type{}, task, number, c0, c1, look, settle, store);
            else
                append(std::false_type{}, task - a.kv_heads, number, c0, c1, look, settle, store);
        };
        if constexpr (!kWalk) {
            // a warp looks at a head's rows and stores them at once
            work_out_angles(0, count);
            for (int i = task; i < 2 * a.kv_heads; i += task_step)
                append_task(i, 0, 0, count, true, true, true);
        } else {
            // all of a warp's heads, some at a time, walk over the rows twice, a table after
            // the other
            constexpr int kTable = kTableTokens<LPR, kWalk>;
            const int all = (2 * a.kv_heads - block_y * kWarps + task_step - 1) / task_step;
            for (int task0 = 0; task0 < all; task0 += kWalkTasks) {
                const int tasks = min(all - task0, kWalkTasks);
                for (int walk = 0; walk < 2; ++walk) {
                    for (int c0 = 0; c0 < count; c0 += kTable) {
                        const int c1 = min(c0 + kTable, count);
                        work_out_angles(c0, c1);
                        for (int number = 0; number < tasks; ++number) {
                            const int i = task + (task0 + number) * task_step;
                            if (i >= 2 * a.kv_heads) break;
                            append_task(i, number, c0, c1, walk == 0, walk == 1 && c0 == 0,
                                        walk == 1);
                        }
                    }
                }
            }
        }
        t += count;
    }
}

template <typename E, int LPR, int kLayout, bool kWalk>
__global__ void __launch_bounds__(kNormThreads, kAppendBlocks)
qk_norm_rope_fp8_kernel(const __grid_constant__ ple_qk_norm_rope_fp8_args f,
                        const __grid_constant__ ple_qk_norm_rope_args queries,
                        const __grid_constant__ AppendPlan plan) {
    if ((int)blockIdx.x < plan.kv_blocks)
        append_blocks<E, LPR, kLayout, kWalk>(f, plan, blockIdx.x, blockIdx.y, gridDim.y);
    else
        norm_rope_rows<E, LPR, kLayout>(queries, plan.rows, blockIdx.x - plan.kv_blocks,
                                        blockIdx.y, gridDim.y);
}

template <typename E, int LPR>
cudaError_t launch_rows(const ple_qk_norm_rope_fp8_args& f, const DeviceFacts& dev,
                        cudaStream_t stream) {
    constexpr int RPW = 32 / LPR;
    constexpr int kWarps = kNormThreads / 32;
    const ple_qk_norm_rope_args& a = f.base;
    AppendPlan plan;
    plan.shift = block_shift(f.scales.block);
    plan.rows.q_groups = (a.q_heads + RPW - 1) / RPW;
    plan.rows.kv_groups = 0;
    const int64_t resident = kAppendBlocks * (int64_t)dev.sm_count;
    auto tokens = [&](int64_t most) {
        const int64_t n = a.num_tokens / resident;
        return n < 1 ? 1 : n > most ? most : n;
    };
    plan.rows.tokens = (int)tokens(kNormTokens);
    plan.kv_tokens = (int)tokens(kAppendTokens);
    const int64_t q_blocks =
        a.q_heads ? (a.num_tokens + plan.rows.tokens - 1) / plan.rows.tokens : 0;
    plan.kv_blocks = (int)((a.num_tokens + plan.kv_tokens - 1) / plan.kv_tokens);
    const int64_t blocks = q_blocks + plan.kv_blocks;
    // few tokens: a token's heads spread over several blocks too
    int64_t split = resident / blocks;
    const int groups = plan.rows.q_groups > 2 * a.kv_heads ? plan.rows.q_groups : 2 * a.kv_heads;
    const int64_t most = (groups + kWarps - 1) / kWarps;
    split = split < 1 ? 1 : split > most ? most : split;
    const int table = f.scales.block * 2 * LPR * 16;
    const bool walk = LPR > 8 && a.rotary_dim && table > kMostTable;
    auto pick = [&](auto walks) {
        constexpr bool kWalk = walks;
        return a.rotary_dim && a.interleaved
                   ? qk_norm_rope_fp8_kernel<E, LPR, kPairsInterleaved, kWalk>
               : a.rotary_dim % 8 == 0 ? qk_norm_rope_fp8_kernel<E, LPR, kPairsHalves, kWalk>
                                       : qk_norm_rope_fp8_kernel<E, LPR, kPairsAnyHalves, kWalk>;
    };
    auto* fn = pick(std::false_type{});
    int smem = a.rotary_dim ? table : 0;
    if constexpr (LPR > 8) {
        if (walk) {
            fn = pick(std::true_type{});
            smem = kTableTokens<LPR, true> * 2 * LPR * 16;
        }
    }
    if (smem > 16384) {
        const cudaError_t e =
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    ple_qk_norm_rope_args queries = a;
    queries.kv_heads = 0;
    queries.k_cache = queries.v_cache = nullptr;
    return launch_kernel(fn, dim3((unsigned)blocks, (unsigned)split), dim3(kNormThreads), smem,
                         stream, programmatic_launch(), f, queries, plan);
}

template <typename E>
cudaError_t launch_element(const ple_qk_norm_rope_fp8_args& f, const DeviceFacts& dev,
                           cudaStream_t stream) {
    if (f.base.head_dim <= 64) return launch_rows<E, 8>(f, dev, stream);
    if (f.base.head_dim <= 128) return launch_rows<E, 16>(f, dev, stream);
    return launch_rows<E, 32>(f, dev, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope_fp8(const ple_qk_norm_rope_fp8_args& f, const DeviceFacts& dev,
                                    cudaStream_t stream) {
    return f.base.dtype == PLE_BF16 ? launch_element<__nv_bfloat16>(f, dev, stream)
                                    : launch_element<__half>(f, dev, stream);
}

}  // namespace ple
