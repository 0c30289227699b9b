// What the attention kernels that split their work evenly over the device share:
// the cut of all units' tiles into one share a block, the walk through a share's
// pieces, nodes' masks, paired 32-bit arithmetic, and the join of rows whose unit
// was cut.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ple_tree_common.cuh"

namespace ple {
namespace {

constexpr int kTile = 128;           // keys a tile
constexpr int kMaxBlocks = 1024;     // blocks of a launch: an SM's number of them is far below

// D is a head's width in shared memory: 64, 128 or 256.
__host__ __device__ constexpr int padded_width(int head_dim) {
    return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256;
}

// Rows of a key head that go together on the tensor cores: 256, or as many as there is
// tensor memory for accumulators of.
__host__ __device__ constexpr int unit_rows(int width) {
    return width > 128 ? kTile : 2 * kTile;
}

struct TcArgs {
    ple_tree_attention_args a;
    int32_t blocks;      // shares
    int32_t rows_cap;    // rows of a state in the workspace, a multiple of 4
    int32_t unit_rows;   // rows of a key head that go together
    int32_t group;       // query heads a key head
    float c;             // |scale| * log2(e)
    uint32_t flip;       // sign bits to turn in Q: scale < 0
};

// a / b for a >= 0, b > 0; most are small, and a 64-bit division is a routine.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// What a unit costs besides its tiles (queries in, rows out), in tiles.  Without it
// the share with the most short units ends last: 32 ragged requests of 17 to 32749
// slots take 380 us at 0, 352 at 2, 346 at 4, 344 at 6, 345 at 8.
constexpr int kUnitCost = 6;

// One request's work, in tiles: that of all its units, kUnitCost each ahead of
// their tiles.
struct Request {
    int64_t work;
    int32_t begin, nodes;
    int32_t ctx, length;     // cached slots all rows see; slots with the nodes'
    int32_t tiles, units;    // key tiles of a unit; units a key head
};

__device__ __forceinline__ Request request_of(const TcArgs& args, int r) {
    const ple_tree_attention_args& a = args.a;
    Request q;
    int32_t end;
    request_nodes(a.cu_seqlens, r, a.num_tokens, q.begin, end);
    q.nodes = end - q.begin;
    const int64_t cap = (int64_t)a.max_pages * a.page_size;
    const int64_t ctx = max(__ldg(a.ctx_lens + r), 0);
    q.ctx = (int32_t)min(ctx, cap);
    q.length = (int32_t)min(ctx + q.nodes, cap);
    q.tiles = (q.length + kTile - 1) / kTile;
    const int64_t rows = (int64_t)q.nodes * args.group;
    q.units = (int32_t)((rows + args.unit_rows - 1) / args.unit_rows);
    q.work = (int64_t)q.units * (q.tiles + kUnitCost) * a.kv_heads;
    return q;
}

// Where share c of `shares` begins, and the share of a place.
__device__ __forceinline__ int64_t share_begin(int64_t total, int c, int shares) {
    return quotient(total * c, shares);
}
__device__ __forceinline__ int share_of(int64_t total, int64_t tile, int shares) {
    return (int)quotient((tile + 1) * shares - 1, total);
}

// A block's part [lo, hi) of the work `total`, the request that owns its first
// place, and the work before that request.  No share is empty.
struct Share {
    int64_t lo, hi, total, before;
    int32_t first, shares;
};

// Every thread of the block calls it; the answer is in *share.  Requests are
// scanned a block's width at a time: once where they fit, else once for the
// total and once for the owner.
template <int kBlock>
__device__ __forceinline__ void find_share(const TcArgs& args, int64_t* scratch, Share* share) {
    const ple_tree_attention_args& a = args.a;
    const int blocks = args.blocks;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int B = a.num_requests;
    int64_t total = 0;
    if (B > kBlock) {
        int64_t mine = 0;
        for (int r = threadIdx.x; r < B; r += kBlock) mine += request_of(args, r).work;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
        if (lane == 0) scratch[warp] = mine;
        __syncthreads();
        for (int k = 0; k < kBlock / 32; ++k) total += scratch[k];
    }
    int64_t base = 0;
    for (int from = 0; from < B; from += kBlock) {
        const int r = from + threadIdx.x;
        const int64_t w = r < B ? request_of(args, r).work : 0;
        int64_t upto = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += o;
        }
        __syncthreads();
        if (lane == 31) scratch[warp] = upto;
        __syncthreads();
        int64_t before = base, all = base;
#pragma unroll
        for (int k = 0; k < kBlock / 32; ++k) {
            const int64_t x = scratch[k];
            if (k < warp) before += x;
            all += x;
        }
        if (B <= kBlock) total = all;
        const int shares = (int)min(total, (int64_t)blocks);
        const bool none = (int)blockIdx.x >= shares;
        const int64_t lo = none ? total : share_begin(total, blockIdx.x, shares);
        if (none ? r == 0 : (w > 0 && before + upto - w <= lo && lo < before + upto)) {
            share->lo = lo;
            share->hi = none ? total : share_begin(total, blockIdx.x + 1, shares);
            share->total = total;
            share->before = before + upto - w;
            share->first = r;
            share->shares = shares;
        }
        base = all;
        if (lo < base) break;
    }
}

// A block's piece of one unit: keys tiles [k0, k1) of `tiles`.
struct Segment {
    Request q;
    int32_t head, unit;
    int32_t k0, k1;
    int32_t r;        // the request
    int32_t rows;     // of the unit, at most unit_rows
    bool pair;        // more than 128 rows, a group each, or the same for both
};

// The block's segments in order; every role walks them alike.
template <int kParts>
struct Walk {
    int64_t at, end;     // what is still to do
    int64_t base;        // the work before request r
    int r;
    Request q;
    __device__ __forceinline__ void begin(const TcArgs& args, const Share& share) {
        at = share.lo;
        end = share.hi;
        base = share.before;
        r = share.first;
        if (at < end) q = request_of(args, r);
    }
    __device__ __forceinline__ bool next(const TcArgs& args, Segment& s) {
        while (at < end) {
            while (at >= base + q.work) {
                base += q.work;
                q = request_of(args, ++r);
            }
            const int32_t span = q.tiles + kUnitCost;
            const int64_t rel = at - base;
            const int32_t u = (int32_t)quotient(rel, span);
            const int32_t from = (int32_t)(rel - (int64_t)u * span);
            const int32_t upto = (int32_t)min((int64_t)span, from + (end - at));
            at += upto - from;
            if (upto <= kUnitCost) continue;  // its first tile is the next share's
            s.q = q;
            s.r = r;
            s.k0 = max(from - kUnitCost, 0);
            s.k1 = upto - kUnitCost;
            s.head = u / q.units;
            s.unit = u - s.head * q.units;
            s.rows = (int32_t)min((int64_t)args.unit_rows,
                                  (int64_t)q.nodes * args.group -
                                      (int64_t)s.unit * args.unit_rows);
            s.pair = kParts == 2 || s.rows > kTile;
            return true;
        }
        return false;
    }
};

// Slots a box: the largest power of two that cuts pages and tiles evenly.
__host__ __device__ __forceinline__ int page_box(int page_size) {
    const int two = page_size & -page_size;
    return two < kTile ? two : kTile;
}

// The offset of the query of a key head's row.
template <typename S>
__device__ __forceinline__ int64_t query_row(const TcArgs& args, const S& s, int row) {
    const ple_tree_attention_args& a = args.a;
    const uint32_t group = args.group;
    const uint32_t node = (uint32_t)row / group;
    return (s.q.begin + (int64_t)node) * a.q_token +
           (int64_t)(s.head * group + (row - node * group)) * a.q_head;
}

// The unit that a block starts and leaves unfinished: what the join has to know.
struct Cut {
    int32_t last;          // the block that finishes it; below the first one: there is none
    int32_t rows;
    int32_t begin;         // the request's first token
    int32_t first_row;     // the unit's among the key head's rows
    int32_t head;
    int32_t unused[3];
};

// The workspace: each block's cut, then two states a block (0: a unit begun
// before the block, 1: a unit that starts in it).  A state is a pair
// (row reference in the exponent of 2, row sum) for each row, then the accumulators
// as [D / 8][row][8]: neighbouring threads write, and a row's readers read, whole
// 32-byte sectors.
__host__ __device__ __forceinline__ int64_t state_at(int64_t block, int slot, int rows_cap,
                                                     int D) {
    return kMaxBlocks * (int64_t)(sizeof(Cut) / 4) +
           (block * 2 + slot) * (int64_t)rows_cap * (D + 2);
}

// K_j's and V_j's places in the order of copies K_0, K_1, V_0, K_2, V_1, ... of
// a segment of n tiles: the order in which the issuing warp wants them.  Of heads
// in parts five places hold no three tiles: K_0, V_0, K_1, V_1, ..., a part after
// the other.
template <int kParts>
__device__ __forceinline__ int key_item(int j) {
    return kParts == 2 ? 4 * j : j == 0 ? 0 : 2 * j - 1;
}
template <int kParts>
__device__ __forceinline__ int value_item(int j, int n) {
    return kParts == 2 ? 4 * j + 2 : j < n - 1 ? 2 * j + 2 : 2 * j + 1;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float as_float(uint32_t v) { return __uint_as_float(v); }

// Two 32-bit floats to a register pair: one instruction for both on sm_103a.
__device__ __forceinline__ uint64_t pack_f32(float lo, float hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ void unpack_f32(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float v;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(v) : "f"(a), "f"(b), "f"(c));
    return v;
}

// The weights are rounded to the element type before the second product, since a
// matrix instruction's operands share the values' type; the row sums take them as
// they were.  Two products, the rest of each weight in the second, would cost what
// the first costs, which is what bounds calls of many rows.
template <bool kBf16>
__device__ __forceinline__ uint32_t round_pair(float lo, float hi) {
    uint32_t v;
    if constexpr (kBf16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(hi), "f"(lo));
    return v;
}

// A node's mask where a tile's slots from `slot` on meet it: three words, all
// that 128 bits may reach, from word `base` on.
struct MaskWindow {
    uint64_t w[3];
    int base;
};

__device__ __forceinline__ MaskWindow mask_window(const unsigned long long* __restrict__ mask,
                                                  uint64_t first_word, int words, int ctx,
                                                  int slot) {
    MaskWindow m;
    m.base = max(slot - ctx, 0) >> 6;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        m.w[k] = m.base + k == 0 ? first_word : 0;
        if (m.base + k > 0 && m.base + k < words) m.w[k] = __ldg(mask + m.base + k);
    }
    return m;
}

// Which of 32 slots from `slot` on a node sees, as bits: all below ctx, above it
// those of its mask.
__device__ __forceinline__ uint32_t seen_bits(const MaskWindow& m, int words, int ctx, int length,
                                              int slot) {
    const int b = slot - ctx;
    if (b + 32 <= 0) return 0xffffffffu;
    const int lo = max(b, 0);
    const int limit = min(length - ctx, 64 * words);
    if (lo >= limit) return b < 0 ? (1u << -b) - 1 : 0u;
    const int k = (lo >> 6) - m.base, s = lo & 63;
    uint64_t v = (k == 0 ? m.w[0] : k == 1 ? m.w[1] : m.w[2]) >> s;
    if (s > 32) v |= (k == 0 ? m.w[1] : m.w[2]) << (64 - s);
    uint32_t bits = (uint32_t)v;
    if (limit - lo < 32) bits &= (1u << (limit - lo)) - 1;
    return b < 0 ? bits << -b | ((1u << -b) - 1) : bits;
}

template <bool kBf16>
__device__ __forceinline__ float widen16(uint32_t v) {
    if constexpr (kBf16)
        return __uint_as_float(v << 16);
    else
        return __half2float(__ushort_as_half((unsigned short)v));
}

// ------------------------------------------------------------------- the join

constexpr int kJoinThreads = 128;
constexpr int kJoinRows = kJoinThreads / 16;  // rows a block

// The cut units' rows: for a row, the states of the blocks that share its unit,
// in block order.  The first grid dimension is the block that started a unit, the
// second its rows.  Sixteen lanes take a row: they read up to 16 states' pairs at
// once, then every lane D / 16 accumulators of each state, eight states' loads in
// flight (four of 256).  The work is a few bytes a row behind three dependent reads, a
// latency, so it is spread thin and wide: 6 us behind the main kernel's 95 for 8
// requests of 4 rows over 16384 slots, 16 with 256 rows (states of 39 MB).
template <int D, bool kBf16>
__global__ void __launch_bounds__(kJoinThreads)
tree_attention_join_kernel(const __grid_constant__ TcArgs args) {
    constexpr int E = D / 16;
    constexpr int kJoinAhead = D > 128 ? 4 : 8;
    const ple_tree_attention_args& a = args.a;
    wait_grid_before();
    const int c0 = blockIdx.x;
    const int4* told = reinterpret_cast<const int4*>(static_cast<const Cut*>(a.workspace) + c0);
    const int4 cut = __ldcg(told);
    const int cut_head = __ldcg(&told[1].x);
    const int c1 = cut.x;
    const int local = blockIdx.y * kJoinRows + threadIdx.x / 16;
    const int lane = threadIdx.x & 15;
    if (c1 <= c0 || local - (threadIdx.x & 31) / 16 >= cut.y) return;
    const bool live = local < cut.y;  // the warp's other row may be there alone
    const float* space = static_cast<const float*>(a.workspace);
    float m = -INFINITY, sum = 0.f, acc[E] = {};
    for (int from = c0; from <= c1; from += 16) {
        const int c = from + lane;
        // the unit starts in the first of its blocks and is begun in the others
        const int64_t mine = state_at(c, c == c0 ? 1 : 0, args.rows_cap, D);
        float2 p = make_float2(-INFINITY, 0.f);
        if (c <= c1 && live) p = __ldcg(reinterpret_cast<const float2*>(space + mine) + local);
        float now = fmaxf(m, p.x);
#pragma unroll
        for (int d = 8; d >= 1; d >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, d));
        // no maximum: nothing seen (zeros), or only NaN, which stays
        const float keep = m == -INFINITY ? 1.f : exp2_fast(m - now);
        const float f = p.x == -INFINITY ? 1.f : exp2_fast(p.x - now);
        float part = p.y * f;
#pragma unroll
        for (int d = 8; d >= 1; d >>= 1) part += __shfl_xor_sync(0xffffffffu, part, d);
        sum = sum * keep + part;
        m = now;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= keep;
        const int n = min(16, c1 - from + 1);
        const int at =
            2 * args.rows_cap + ((lane * E / 8) * args.rows_cap + local) * 8 + lane * E % 8;
        for (int i0 = 0; i0 < n; i0 += kJoinAhead) {
            float4 x[kJoinAhead][E / 4];
#pragma unroll
            for (int i = 0; i < kJoinAhead; ++i) {
                if (i0 + i < n && live) {
                    const float* theirs =
                        space + at +
                        state_at(from + i0 + i, from + i0 + i == c0 ? 1 : 0, args.rows_cap, D);
#pragma unroll
                    for (int e = 0; e < E / 4; ++e)
                        x[i][e] = __ldcg(reinterpret_cast<const float4*>(
                            theirs + e / 2 * 8 * args.rows_cap + e % 2 * 4));
                }
            }
#pragma unroll
            for (int i = 0; i < kJoinAhead; ++i) {
                const float g = __shfl_sync(0xffffffffu, f, (i0 + i) & 15, 16);
                if (i0 + i < n && live) {
#pragma unroll
                    for (int e = 0; e < E / 4; ++e) {
                        acc[4 * e] = fmaf(x[i][e].x, g, acc[4 * e]);
                        acc[4 * e + 1] = fmaf(x[i][e].y, g, acc[4 * e + 1]);
                        acc[4 * e + 2] = fmaf(x[i][e].z, g, acc[4 * e + 2]);
                        acc[4 * e + 3] = fmaf(x[i][e].w, g, acc[4 * e + 3]);
                    }
                }
            }
        }
    }
    if (!live) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const uint32_t group = args.group;
    const uint32_t row = cut.w + local;
    const uint32_t node = row / group;
    const int64_t o = (cut.z + (int64_t)node) * a.q_heads + cut_head * group + row - node * group;
    uint32_t y[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e)
        y[e] = round_pair<kBf16>(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    uint32_t* dst =
        reinterpret_cast<uint32_t*>(static_cast<unsigned short*>(a.out) + o * a.head_dim) +
        lane * (E / 2);
    if constexpr (E == 4) {
        if (lane * E < a.head_dim) *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
    } else {
#pragma unroll
        for (int e = 0; e < E; e += 8)
            if (lane * E + e < a.head_dim)
                *reinterpret_cast<uint4*>(dst + e / 2) =
                    make_uint4(y[e / 2], y[e / 2 + 1], y[e / 2 + 2], y[e / 2 + 3]);
    }
    if (lane == 0 && a.lse != nullptr)
        a.lse[o] = sum == 0.f ? -INFINITY : m * 0.69314718055994531f + logf(sum);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

int tc_blocks(const DeviceFacts& dev) {
    return dev.sm_count < kMaxBlocks ? dev.sm_count : kMaxBlocks;
}

int tc_rows_cap(int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    const int64_t rows = T * (q_heads / kv_heads);
    const int most = unit_rows(padded_width(head_dim));
    return (int)(rows < most ? (rows + 3) / 4 * 4 : most);  // 16-byte rows
}

}  // namespace
}  // namespace ple
