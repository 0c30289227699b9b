// Attention of drafted nodes over a paged cache in 8 bits, on sm_103a: the kernel for
// few rows a key head.
//
//   out = sum_j p_j v_j,  p = softmax_j(scale q . k_j),  k_j = a_j e_j,  v_j = b_j f_j
// with elements e, f (e4m3) and a scale a, b for each block of slots and head, over the
// slots that a node sees, in one pass over the keys with the running maximum and sum of
// the softmax (Milakov and Gimelshein 2018).
//
// Scales.  A block's key scale multiplies its scores in 32 bits.  Its value scale
// multiplies its weights, so that elements enter the products as they are.  A row
// keeps two references, in the exponent of 2: `top`, the maximum of its scores, which its
// sum is relative to, and `ref`, near the maximum of score plus log2 of the value
// scale, which its weights and accumulators are relative to.  Any `ref` will do that
// weights and accumulators share, so accumulators are scaled anew only when a slice's
// maximum is a few binades away from it.
//
// Blocks.  One block an SM: a warp that copies tiles of 128 keys and their values into a
// ring (tiled bulk copies, page by page, swizzled), one that hands their scales over, one
// that works out the next segment, and teams of eight warps.  A warp of a team takes 16
// slots of a tile, for all rows, with a softmax state and accumulators of its own; the
// team's meet at a segment's end.  A slice of 16 slots has one scale.  With up to eight
// rows a key head two teams take the tiles in turn (heads above 128: one), since a team
// alone does not keep up with the memory; with up to sixteen one team does two products
// a slice.  Elements become halves in registers (one conversion for two, exact) on their
// way to m16n8k16 products: the order of a head's elements in the reduction, and of
// columns in the output, is free, so a lane takes 16 consecutive bytes of a key, and of a
// value, wherever a product wants one element of them.  Keys and values are the products'
// 16 rows, queries and weights the eight columns, so that eight rows waste nothing.
//
// Measured (bf16, heads of 128, 32 query and 8 key heads, 64-slot pages, the join with
// it).  The bytes bound it: 64 requests of one token over 257 to 16385 slots 183 us (161
// of bytes at the measured copy's rate), 32 of one or two nodes over 16384 192 (5.6 TB/s;
// the cache in 16 bits takes 318), of four nodes 225.  Few keys are a latency: one token
// over 701 slots 9.3 us, two launches of it.
//
// Split and join: ple_tree_split.cuh.
#include <cuda_fp16.h>

#include "ple_fp8.cuh"
#include "ple_tc.cuh"
#include "ple_tree_fp8_internal.h"
#include "ple_tree_split.cuh"

namespace ple {
namespace {

constexpr int kSlice = 16;                // slots a warp takes of a tile
constexpr int kTeam = kTile / kSlice;     // warps of a tile

// How far a slice's largest weight (times its value scale) may lie above and below the
// row's reference before that moves, and where weights are placed as halves: between
// 2^2 and 2^15 with these, and a scale's significand below 2.
constexpr float kRise = 5.0f, kFall = 7.0f, kBias = 9.0f;
// A reference falls only where the row's weights, relative to the new one, sum up to less than
// this.  That sum is taken as the most that each slice's (or tile's) largest weight allows: up to
// 2^8 times what it is.  So a tile whose largest weight is 2^-50 of the row's sum or more is still
// followed (2^(50 + 8 + kBias) is below it), and accumulators, 448 times the sum at most, stay far
// inside 32 bits.
constexpr float kMostSum = 0x1p68f;

// W: a head's width in shared memory (64, 128 or 256); NT: tiles of eight rows; Teams: of
// eight warps, which take the tiles in turn.
template <int W, int NT, int Teams>
struct RowShape {
    static constexpr int kWarps = Teams * kTeam;
    // a warp that copies, one that walks ahead, one for the scales, and one that fills the
    // warpgroup up: a register split is by warpgroups
    static constexpr int kThreads = 32 * (kWarps + 4);
    static constexpr int kCopyWarp = kWarps, kWalkWarp = kWarps + 1, kScaleWarp = kWarps + 2;
    static constexpr int kRegisters = Teams == 2 ? 104 : 216, kFewRegisters = Teams == 2 ? 64 : 72;
    static constexpr int kHalves = W > 128 ? 2 : 1;     // boxes of a row
    static constexpr int kRowBytes = W / kHalves;       // 64 or 128: the swizzle's span
    static constexpr int kTileBytes = kTile * W;
    // tiles of keys and values in flight: an SM's share of the measured bandwidth is
    // 45 GB/s, and a loaded memory answers in 2 us.  An even number, so that a team that
    // takes every second tile sees every round of its places
    static constexpr int kStages = W == 64 ? 10 : W == 128 ? 4 : 3;
    static constexpr int kColumns = W / 8;              // of a lane
    // of them meet at a time: in rounds of 4, for two more tiles in flight, 256 decodes over
    // 512 slots take 128 us instead of 96, and long contexts what they took
    static constexpr int kRound = W == 128 ? 16 : 8;
    static constexpr int kRounds = kColumns / kRound;
    // eight rows of every warp meet here; queries before that
    static constexpr int kMeetBytes = kWarps * 8 * 8 * kRound * 4;
    static constexpr int kSmem = kStages * 2 * kTileBytes + kMeetBytes + 1024;
};

__device__ __forceinline__ void mma_halves(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A warp's 8 x 8 halves, a lane's two of row lane / 4, turned about the diagonal.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// A 16-byte piece's place in a swizzled row of a tile.
template <int W>
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
    if constexpr (W == 64)
        return row * 64 + ((piece ^ (row >> 1 & 3)) << 4);
    else  // rows of 256 bytes are two halves
        return (piece >> 3) * (kTile * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}

// The same for a row of queries (halves), which lanes read 16 bytes at a time: the
// eight lanes of a transaction, two rows and four columns, meet eight banks.
template <int W>
__device__ __forceinline__ uint32_t query_at(int row, int piece) {
    const int x = W == 64 ? row & 1 : (piece >> 3 & 1) ^ (row & 1) << 1;
    return row * (2 * W) + ((piece ^ x) << 4);
}

// And for 16 bytes of a row of accumulators on their way to meet: lanes that write
// together have two pieces and four rows, every second one.
template <int kRound>
__device__ __forceinline__ int meet_at(int row, int f) {
    return kRound == 16 ? f ^ (row >> 1 & 3) : f ^ (row >> 1 & 1) ^ (row & 4);
}

template <int W, int NT, int Teams, bool kBf16>
__global__ void __launch_bounds__(RowShape<W, NT, Teams>::kThreads, 1)
tree_attention_fp8_kernel(const __grid_constant__ TcArgs args, const __grid_constant__ Scales sc,
                          const __grid_constant__ CUtensorMap k_map,
                          const __grid_constant__ CUtensorMap v_map) {
    using S = RowShape<W, NT, Teams>;
    constexpr int kWarps = S::kWarps;
    const ple_tree_attention_args& a = args.a;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages];
    // a tile's scales, (a, log2 b) for each slice
    __shared__ float2 scale_s[S::kStages][kTeam];
    __shared__ int64_t scratch[S::kThreads / 32];
    __shared__ Share share_s;
    __shared__ int failed_s;
    __shared__ float top_s[kWarps][8 * NT], sum_s[kWarps][8 * NT];
    __shared__ int shift_s[8 * NT];
    __shared__ Segment seg_s[2];
    __shared__ int more_s[2];
    __shared__ int64_t end_s[2];
    volatile int* failed = &failed_s;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* smem = smem_raw + (((smem_addr(smem_raw) + 1023) & ~1023u) - smem_addr(smem_raw));
    uint8_t* ring = smem;
    uint8_t* meet = smem + S::kStages * 2 * S::kTileBytes;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&full[i], 2);
            mbar_init(&empty[i], kTeam);
        }
        failed_s = 0;
        fence_barrier_init();
    }
    if (warp == S::kCopyWarp && lane == 0) {
        prefetch_map(&k_map);
        prefetch_map(&v_map);
    }
    wait_grid_before();
    find_share<S::kThreads>(args, scratch, &share_s);
    __syncthreads();

    if (warp >= kWarps) {
        fewer_registers<S::kFewRegisters>();
        Walk<1> walk;
        walk.begin(args, share_s);
        Segment s;
        if (warp == S::kWalkWarp) {
            // --------------------------- the others' segments, one ahead
            bool more;
            uint32_t seg = 0;
            do {
                more = walk.next(args, s);
                if (lane == 0) {
                    seg_s[seg & 1] = s;
                    end_s[seg & 1] = walk.at;
                    more_s[seg & 1] = more;
                }
                ++seg;
                named_barrier<32 * (kWarps + 1)>(3);
            } while (more);
        } else if (warp == S::kScaleWarp) {
            // ------------------------------------------------------- scales
            // lanes 0 to 7 a slice's each: asked for a tile ahead, their page two
            int stage = 0;
            uint32_t round = 0;
            bool ended = false;
            while (!ended && walk.next(args, s)) {
                const int32_t* table = a.page_table + (int64_t)s.r * a.max_pages;
                auto slice_page = [&](int k) -> int {
                    const uint32_t slot = k * kTile + (lane & 7) * kSlice;
                    int number = -1;
                    if (k < s.k1 && (int)slot < s.q.length)
                        number = load_now(table + sc.page_of(slot));
                    return number;
                };
                uint32_t k_ahead, v_ahead;
                auto ask = [&](int k, int number) {
                    sc.ask(number, a.num_pages, s.head, k * kTile + (lane & 7) * kSlice,
                           a.page_size, k_ahead, v_ahead);
                };
                ask(s.k0, slice_page(s.k0));
                int number = slice_page(s.k0 + 1);
                for (int k = s.k0; k < s.k1; ++k) {
                    const float2 mine = make_float2(scale_value(k_ahead), scale_log(v_ahead));
                    ask(k + 1, number);
                    number = slice_page(k + 2);
                    if (!mbar_wait(&empty[stage], (round & 1) ^ 1, failed)) {
                        ended = true;
                        break;
                    }
                    if (lane < 8) scale_s[stage][lane] = mine;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[stage]);
                    if (++stage == S::kStages) {
                        stage = 0;
                        ++round;
                    }
                }
            }
        } else if (warp == S::kCopyWarp) {
            // ------------------------------------------------------- copies
            const int box = page_box(a.page_size);
            const int boxes = kTile / box;
            const bool keys = lane & 1;
            const int half = lane / 2 % S::kHalves, which = lane / 2 / S::kHalves;
            const bool mine = which < boxes;
            int stage = 0;
            uint32_t round = 0;
            bool ended = false;
            while (!ended && walk.next(args, s)) {
                const int32_t* table = a.page_table + (int64_t)s.r * a.max_pages;
                // a box past the tokens, or of a page outside the cache, is filled
                // with zeros: its page number is outside the map
                auto page_of = [&](int k) -> int {
                    const int slot = k * kTile + which * box;
                    if (!mine || k >= s.k1 || slot >= s.q.length) return (int)a.num_pages;
                    const int p = __ldg(table + sc.page_of(slot));
                    return p < 0 || p >= a.num_pages ? (int)a.num_pages : p;
                };
                int page = page_of(s.k0);
                for (int k = s.k0; k < s.k1; ++k) {
                    const int after = page_of(k + 1);
                    if (!mbar_wait(&empty[stage], (round & 1) ^ 1, failed)) {
                        ended = true;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect(&full[stage], 2 * S::kTileBytes);
                    __syncwarp();
                    if (mine)
                        copy_box(keys ? &k_map : &v_map,
                                 smem_addr(ring) + (2 * stage + !keys) * S::kTileBytes +
                                     half * (kTile * 128) + which * box * S::kRowBytes,
                                 &full[stage], half * 128,
                                 sc.in_page(k * kTile + which * box, a.page_size), s.head, page);
                    page = after;
                    if (++stage == S::kStages) {
                        stage = 0;
                        ++round;
                    }
                }
            }
            if (ended) {
                // copies may be in flight: they land before the block ends
                for (int i = 0; i < S::kStages; ++i) {
                    const uint32_t rounds = round + (i < stage);
                    const long long start = clock64();
                    while (rounds != 0 && !mbar_try(&full[i], (rounds - 1) & 1) &&
                           clock64() - start < kWaitClocks) {
                    }
                }
            }
        }
        return;
    }

    // ----------------------------------------------------------- products
    more_registers<S::kRegisters>();
    constexpr int kSteps = W / 16;                       // of a score's reduction
    constexpr bool kHeld = NT * W <= 256 && Teams * NT < 4;   // queries in registers
    constexpr int kTiles = W / 16;                       // of 16 columns
    const int g = lane >> 2, c = lane & 3;
    const int team = warp / kTeam, slice = warp % kTeam;
    const int group = args.group;
    if (threadIdx.x == 0) static_cast<Cut*>(a.workspace)[blockIdx.x].last = -1;
    int stage = 0;
    uint32_t round = 0, seg = 0;
    for (;;) {
        named_barrier<32 * (kWarps + 1)>(3);
        if (!*static_cast<volatile int*>(&more_s[seg & 1])) break;
        const Segment& s = seg_s[seg & 1];
        const int k0 = s.k0, k1 = s.k1, rows = s.rows, head = s.head;
        const int ctx = s.q.ctx, length = s.q.length;
        const int first_row = s.unit * args.unit_rows;
        // the rows' queries as halves in shared memory: a warp a row at a time
        for (int r = warp; r < 8 * NT; r += kWarps) {
            constexpr int kPer = W / 32;                 // elements a lane: 2, 4 or 8
            uint32_t x[kPer / 2] = {};
            const int at = lane * kPer;
            if (r < rows && at < a.head_dim) {
                const unsigned short* from = static_cast<const unsigned short*>(a.q) +
                                             query_row(args, s, first_row + r) + at;
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i)
                    x[i] = __ldg(reinterpret_cast<const unsigned int*>(from) + i) ^ args.flip;
            }
            int shift = 0;
            if constexpr (kBf16) {
                uint32_t most = 0;
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i)
                    most = max(most, max(x[i] << 16 & 0x7FFF0000u, x[i] & 0x7FFF0000u));
#pragma unroll
                for (int d = 16; d >= 1; d >>= 1)
                    most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
                shift = query_shift(most);
                const float f = __uint_as_float((uint32_t)(127 - shift) << 23);
#pragma unroll
                for (int i = 0; i < kPer / 2; ++i) {
                    const __half2 h = __floats2half2_rn(__uint_as_float(x[i] << 16) * f,
                                                        __uint_as_float(x[i] & 0xFFFF0000u) * f);
                    x[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
            if (lane == 0) shift_s[r] = shift;
            uint32_t* to = reinterpret_cast<uint32_t*>(meet + query_at<W>(r, at >> 3) +
                                                       2 * (at & 7));
#pragma unroll
            for (int i = 0; i < kPer / 2; ++i) to[i] = x[i];
        }
        named_barrier<32 * kWarps>(1);

        // Rows 8 n + 2 c and the next one are a lane's: their factors from score to
        // exponent of 2, and their states (a lane's own part of the sums).
        float factor[NT][2];
        float top[NT][2], sum[NT][2], ref[NT][2], heap[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                factor[n][e] =
                    args.c * __uint_as_float((uint32_t)(127 + shift_s[8 * n + 2 * c + e]) << 23);
                top[n][e] = ref[n][e] = -INFINITY;
                sum[n][e] = heap[n][e] = 0.f;
            }
        // a lane's queries of two steps, of row 8 n + g
        auto query_words = [&](int n, int two) {
            return *reinterpret_cast<const uint4*>(
                meet + query_at<W>(8 * n + g, c * (W / 32) + two));
        };
        uint4 held[kHeld ? NT : 1][kHeld ? kSteps / 2 : 1];
        if constexpr (kHeld) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < kSteps / 2; ++i) held[n][i] = query_words(n, i);
        }
        // columns (W / 8) g + 2 t and the next one, of rows 8 n + 2 c and the next one
        float o[NT][kTiles][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][t][e] = 0.f;

        for (int k = k0; k < k1; ++k) {
            if (Teams == 1 || (stage & 1) == team) {
                if (!mbar_wait(&full[stage], round & 1, failed)) break;
                const uint8_t* keys = ring + 2 * stage * S::kTileBytes;
                const uint8_t* vals = keys + S::kTileBytes;
                const int first = k * kTile + slice * kSlice;
                if (first < length) {
                    const bool masked = first + kSlice > ctx;
                    // -------------------------------------------- scores
                    // of slots g and g + 8, even and odd steps apart
                    float s0[NT][4] = {}, s1[NT][4] = {};
#pragma unroll
                    for (int i = 0; i < kSteps; i += 4) {
                        const uint4 low = *reinterpret_cast<const uint4*>(
                            keys + piece_at<W>(slice * kSlice + g, c * (W / 64) + i / 4));
                        const uint4 high = *reinterpret_cast<const uint4*>(
                            keys + piece_at<W>(slice * kSlice + 8 + g, c * (W / 64) + i / 4));
#pragma unroll
                        for (int two = 0; two < 2; ++two) {
                            uint32_t b[2][4];   // step; both slots, first and second half
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                halves_of(two ? (z ? low.w : low.z) : (z ? low.y : low.x), b[z][0],
                                          b[z][2]);
                                halves_of(two ? (z ? high.w : high.z) : (z ? high.y : high.x),
                                          b[z][1], b[z][3]);
                            }
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                uint4 q;
                                if constexpr (kHeld)
                                    q = held[n][i / 2 + two];
                                else
                                    q = query_words(n, i / 2 + two);
                                mma_halves(s0[n], b[0][0], b[0][1], b[0][2], b[0][3], q.x, q.y);
                                mma_halves(s1[n], b[1][0], b[1][1], b[1][2], b[1][3], q.z, q.w);
                            }
                        }
                    }
                    // the values' words of this lane's four slots
                    constexpr int kWords = W / 32;
                    uint32_t vw[4][kWords];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int row = slice * kSlice + 2 * c + (i & 1) + 8 * (i >> 1);
                        if constexpr (W == 64) {
                            const uint2 x = *reinterpret_cast<const uint2*>(
                                vals + piece_at<W>(row, g >> 1) + 8 * (g & 1));
                            vw[i][0] = x.x;
                            vw[i][1] = x.y;
                        } else {
#pragma unroll
                            for (int p = 0; p < kWords / 4; ++p) {
                                const uint4 x = *reinterpret_cast<const uint4*>(
                                    vals + piece_at<W>(row, g * (kWords / 4) + p));
                                vw[i][4 * p] = x.x;
                                vw[i][4 * p + 1] = x.y;
                                vw[i][4 * p + 2] = x.z;
                                vw[i][4 * p + 3] = x.w;
                            }
                        }
                    }
                    // ------------------------------------------- softmax
                    const float2 scales = scale_s[stage][slice];
                    const float k_scale = scales.x, v_log = scales.y;
                    uint32_t seen[NT][2];
                    if (masked) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int row = 8 * n + 2 * c + e;
                                seen[n][e] = 0;
                                if (row < rows) {
                                    const int64_t token = s.q.begin + (first_row + row) / group;
                                    const unsigned long long* mask =
                                        reinterpret_cast<const unsigned long long*>(a.tree_mask) +
                                        token * a.mask_words;
                                    const MaskWindow w = mask_window(mask, __ldg(mask),
                                                                     a.mask_words, ctx, first);
                                    seen[n][e] =
                                        seen_bits(w, a.mask_words, ctx, length, first) & 0xFFFFu;
                                }
                            }
                        __syncwarp();
                    }
                    float x[NT][2][2];   // row, slot g and g + 8
                    float to[NT][2], reach[NT][2];
                    bool move = false;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float f = factor[n][e] * k_scale;
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                x[n][e][z] = (s0[n][2 * z + e] + s1[n][2 * z + e]) * f;
                                if (masked && !(seen[n][e] >> (g + 8 * z) & 1))
                                    x[n][e][z] = -INFINITY;
                            }
                            reach[n][e] = fmaxf(x[n][e][0], x[n][e][1]);
                        }
#pragma unroll
                    for (int d = 4; d <= 16; d <<= 1)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                reach[n][e] = fmaxf(reach[n][e],
                                                    __shfl_xor_sync(0xffffffffu, reach[n][e], d));
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float now = fmaxf(top[n][e], reach[n][e]);
                            const float base = now == -INFINITY ? 0.f : now;
                            sum[n][e] *= exp2_fast(top[n][e] - base);
                            top[n][e] = now;
                            // where the row's weights should be relative to
                            reach[n][e] += v_log;
                            const float fall = ref[n][e] - reach[n][e];
                            const bool rise = -fall > kRise;
                            const bool sink =
                                fall > kFall && heap[n][e] * exp2_fast(fall) < kMostSum;
                            to[n][e] = rise || sink ? reach[n][e] : ref[n][e];
                            move |= rise || sink;
                        }
                    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float f = ref[n][e] == to[n][e] ? 1.f
                                                : ref[n][e] == -INFINITY
                                                    ? 0.f
                                                    : exp2_fast(ref[n][e] - to[n][e]);
                                ref[n][e] = to[n][e];
                                heap[n][e] *= f;
#pragma unroll
                                for (int t = 0; t < kTiles; ++t) {
                                    o[n][t][e] *= f;
                                    o[n][t][2 + e] *= f;
                                }
                            }
                    }
                    uint32_t p[NT][2];   // slots 2 c, 2 c + 1 and 8 more, of row 8 n + g
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float w[2][2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float base = top[n][e] == -INFINITY ? 0.f : top[n][e];
                            const float f =
                                exp2_fast(fminf(base + v_log - ref[n][e] + kBias, 126.f));
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const float weight = exp2_fast(x[n][e][z] - base);
                                sum[n][e] += weight;
                                w[e][z] = weight * f;
                                // what is not seen has no part, whatever the scale
                                if (masked && x[n][e][z] == -INFINITY) w[e][z] = 0.f;
                            }
                            // at most this much for the slice's 16 weights, the same
                            // in all lanes of a row
                            if (ref[n][e] != -INFINITY)
                                heap[n][e] += exp2_fast(reach[n][e] - ref[n][e] + kBias + 5.f);
                        }
#pragma unroll
                        for (int z = 0; z < 2; ++z)
                            p[n][z] = transposed(round_pair<false>(w[0][z], w[1][z]));
                    }
                    // ------------------------------------------ products
                    // Zero weights would not stop a NaN among values that not all
                    // rows see: such elements are cleared, and where a row sees one
                    // its column becomes NaN.
                    bool bad = false;
                    if (masked) {
                        uint32_t any = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int q = 0; q < kWords; ++q) any |= nan_flags(vw[i][q]);
                        bad = __any_sync(0xffffffffu, any != 0);
                    }
                    if (bad) {
                        uint32_t sees[NT][2];
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint32_t even = __shfl_sync(0xffffffffu, seen[n][0], g >> 1);
                            const uint32_t odd = __shfl_sync(0xffffffffu, seen[n][1], g >> 1);
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const uint32_t b = (g & 1 ? odd : even) >> (2 * c + 8 * z);
                                sees[n][z] = (b & 1 ? 0x3C00u : 0u) | (b & 2 ? 0x3C000000u : 0u);
                            }
                        }
#pragma unroll
                        for (int q = 0; q < kWords; ++q) {
                            uint32_t flag[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t one = nan_flags(vw[i][q]) >> 7;
                                vw[i][q] &= ~(one * 0xFFu);
                                flag[i] = one * 0x38u;   // an element of 1
                            }
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                uint32_t b[4];
                                halves_of(__byte_perm(flag[0], flag[1], t ? 0x7362 : 0x5140), b[0],
                                          b[1]);
                                halves_of(__byte_perm(flag[2], flag[3], t ? 0x7362 : 0x5140), b[2],
                                          b[3]);
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    float hit[4] = {};
                                    mma_halves(hit, b[0], b[1], b[2], b[3], sees[n][0], sees[n][1]);
#pragma unroll
                                    for (int z = 0; z < 4; ++z)
                                        if (hit[z] > 0.f)
                                            o[n][2 * q + t][z] = __int_as_float(0x7FC00000);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int q = 0; q < kWords; ++q)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            // two slots' bytes side by side, two columns a word
                            uint32_t b[4];
                            halves_of(__byte_perm(vw[0][q], vw[1][q], t ? 0x7362 : 0x5140), b[0],
                                      b[1]);
                            halves_of(__byte_perm(vw[2][q], vw[3][q], t ? 0x7362 : 0x5140), b[2],
                                      b[3]);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma_halves(o[n][2 * q + t], b[0], b[1], b[2], b[3], p[n][0],
                                           p[n][1]);
                        }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[stage]);
            }
            if (++stage == S::kStages) {
                stage = 0;
                ++round;
            }
        }

        // --------------------------------------------- the warps' states meet
        const bool whole = k0 == 0 && k1 == s.q.tiles;
        if (threadIdx.x == 0 && k0 == 0 && !whole) {
            Cut cut = {};
            cut.last = share_of(share_s.total, end_s[seg & 1] - 1 + (s.q.tiles - k1),
                                share_s.shares);
            cut.rows = rows;
            cut.begin = s.q.begin;
            cut.first_row = first_row;
            cut.head = head;
            static_cast<Cut*>(a.workspace)[blockIdx.x] = cut;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float t = sum[n][e];
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
                if (g == 0) {
                    top_s[warp][8 * n + 2 * c + e] = top[n][e];
                    sum_s[warp][8 * n + 2 * c + e] = t;
                }
            }
        float* state = static_cast<float*>(a.workspace) +
                       state_at(blockIdx.x, k0 == 0 ? 1 : 0, args.rows_cap, W);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (8 * n >= rows) break;
#pragma unroll
            for (int part = 0; part < S::kRounds; ++part) {
                // the tops are there, and who read the queries, or the rows before
                // these, is done
                named_barrier<32 * kWarps>(1);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float most = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w)
                        most = fmaxf(most, top_s[w][8 * n + 2 * c + e]);
                    const float f = ref[n][e] == -INFINITY
                                        ? 0.f
                                        : exp2_fast(fminf(ref[n][e] - kBias - most, 126.f));
                    float4* put = reinterpret_cast<float4*>(meet) +
                                  (warp * 8 + 2 * c + e) * (2 * S::kRound);
#pragma unroll
                    for (int q = 0; q < S::kRound / 4; ++q) {
                        const int t = (part * S::kRound + 4 * q) / 2;
                        put[meet_at<S::kRound>(2 * c + e, (S::kRound / 4) * g + q)] =
                            make_float4(o[n][t][e] * f, o[n][t][2 + e] * f, o[n][t + 1][e] * f,
                                        o[n][t + 1][2 + e] * f);
                    }
                }
                named_barrier<32 * kWarps>(1);
                constexpr int kAcross = 2 * S::kRound;   // 16-byte pieces of a row
                const int r = threadIdx.x / kAcross, piece = threadIdx.x % kAcross;
                const int row = 8 * n + r;
                if (r < 8 && row < rows) {
                    float best = -INFINITY, total = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) best = fmaxf(best, top_s[w][row]);
                    const float base = best == -INFINITY ? 0.f : best;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        total = fmaf(sum_s[w][row], exp2_fast(top_s[w][row] - base), total);
                        const float4 v = reinterpret_cast<const float4*>(
                            meet)[(w * 8 + r) * kAcross + meet_at<S::kRound>(r, piece)];
                        acc.x += v.x;
                        acc.y += v.y;
                        acc.z += v.z;
                        acc.w += v.w;
                    }
                    if (*failed) total = __int_as_float(0x7FC00000);
                    const int column = piece / (S::kRound / 4) * S::kColumns + part * S::kRound +
                                       piece % (S::kRound / 4) * 4;
                    if (whole) {
                        const int node = (first_row + row) / group;
                        const int64_t at = (s.q.begin + (int64_t)node) * a.q_heads +
                                           (int64_t)head * group + (first_row + row) - node * group;
                        const float inv = total == 0.f ? 0.f : 1.f / total;
                        if (column < a.head_dim)
                            *reinterpret_cast<uint2*>(static_cast<unsigned short*>(a.out) +
                                                      at * a.head_dim + column) =
                                make_uint2(round_pair<kBf16>(acc.x * inv, acc.y * inv),
                                           round_pair<kBf16>(acc.z * inv, acc.w * inv));
                        if (part == 0 && piece == 0 && a.lse != nullptr)
                            a.lse[at] = total == 0.f
                                            ? -INFINITY
                                            : best * 0.69314718055994531f + logf(total);
                    } else {
                        *reinterpret_cast<float4*>(state + 2 * args.rows_cap +
                                                   (column / 8 * args.rows_cap + row) * 8 +
                                                   column % 8) = acc;
                        if (part == 0 && piece == 0) {
                            state[2 * row] = best;
                            state[2 * row + 1] = total;
                        }
                    }
                }
            }
        }
        // the next segment's queries go where these rows met
        named_barrier<32 * kWarps>(1);
        ++seg;
    }
}

// A cache as a map of (element, slot, head, page); boxes of 64 or 128 elements by the
// slots of page_box.  Pages outside read as zeros, and so do elements past a head
// narrower than the tile.
bool encode_cache(CUtensorMap* map, const ple_tree_attention_args& a, const void* cache) {
    const EncodeTiled fn = encode_tiled();
    if (fn == nullptr) return false;
    auto stride = [](int64_t elements, int64_t n) {
        return (cuuint64_t)(n == 1 ? 16 : elements);
    };
    const bool narrow = a.head_dim <= 64;
    const cuuint64_t sizes[4] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.page_size,
                                 (cuuint64_t)a.kv_heads, (cuuint64_t)a.num_pages};
    const cuuint64_t strides[3] = {stride(a.slot_stride, a.page_size),
                                   stride(a.head_stride, a.kv_heads),
                                   stride(a.page_stride, a.num_pages)};
    const cuuint32_t box[4] = {narrow ? 64u : 128u, (cuuint32_t)page_box(a.page_size), 1, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(cache), sizes, strides, box,
              ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int W, int NT, int Teams, bool kBf16>
cudaError_t launch_rows(const TcArgs& args, const Scales& sc, const CUtensorMap& k,
                        const CUtensorMap& v, cudaStream_t stream) {
    using S = RowShape<W, NT, Teams>;
    auto* fn = tree_attention_fp8_kernel<W, NT, Teams, kBf16>;
    cudaError_t e =
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_kernel(fn, dim3((unsigned)args.blocks), dim3(S::kThreads), S::kSmem, stream,
                      programmatic_launch(), args, sc, k, v);
    if (e != cudaSuccess) return e;
    return launch_kernel(
        tree_attention_join_kernel<W, kBf16>,
        dim3((unsigned)args.blocks, (unsigned)((args.rows_cap + kJoinRows - 1) / kJoinRows)),
        dim3(kJoinThreads), 0, stream, programmatic_launch(), args);
}

template <int W, bool kBf16>
cudaError_t launch_width(const TcArgs& args, const Scales& sc, const CUtensorMap& k,
                         const CUtensorMap& v, cudaStream_t stream) {
    if (args.unit_rows <= 8)
        return launch_rows<W, 1, W == 256 ? 1 : 2, kBf16>(args, sc, k, v, stream);
    return launch_rows<W, 2, 1, kBf16>(args, sc, k, v, stream);
}

template <bool kBf16>
cudaError_t launch_dtype(const TcArgs& args, const Scales& sc, const CUtensorMap& k,
                         const CUtensorMap& v, cudaStream_t stream) {
    switch (padded_width(args.a.head_dim)) {
        case 64: return launch_width<64, kBf16>(args, sc, k, v, stream);
        case 128: return launch_width<128, kBf16>(args, sc, k, v, stream);
        default: return launch_width<256, kBf16>(args, sc, k, v, stream);
    }
}

// Whether a call's key heads have so many rows that the tensor cores' kernel takes it.  32
// rows over 32 x 16384 slots, as four products a slice, take 489 us here and 214 there.
// With 9 to 16 rows a slot costs less there and a unit more: 32 x 16384 slots 226 and 207
// us, 32 of 100 to 9000 100 and 84, 64 x 512 41 and 53 (heads of 256, 32 x 8192: 238 and
// 285), so it takes them where the page tables have room for some 100 tiles a block.
bool many_rows(const ple_tree_attention_args& a, const DeviceFacts& dev) {
    const int64_t rows = a.num_tokens * (a.q_heads / a.kv_heads), B = a.num_requests;
    if (rows > 16 * B) return true;
    const int64_t tiles = ((int64_t)a.max_pages * a.page_size + kTile - 1) / kTile;
    return rows > 8 * B && a.head_dim <= 128 &&
           B * a.kv_heads * tiles >= 96 * (int64_t)tc_blocks(dev);
}

}  // namespace

int64_t tree_attention_fp8_workspace(int64_t T, int32_t q_heads, int32_t kv_heads, int32_t D,
                                     const DeviceFacts& dev) {
    // the other kernel's states are of more rows
    return tree_attention_fp8_tc_workspace(T, q_heads, kv_heads, D, dev);
}

cudaError_t launch_tree_attention_fp8(const ple_tree_attention_fp8_args& f,
                                      const DeviceFacts& dev, cudaStream_t stream) {
    const ple_tree_attention_args& a = f.base;
    CUtensorMap k, v;
    if (!encode_cache(&k, a, a.k_cache) || !encode_cache(&v, a, a.v_cache))
        return cudaErrorInvalidValue;
    if (many_rows(a, dev)) return launch_tree_attention_fp8_tc(f, k, v, dev, stream);
    TcArgs args;
    args.a = a;
    args.blocks = tc_blocks(dev);
    args.group = a.q_heads / a.kv_heads;
    // rows that go together: as many as a request's key heads have on the average (of a
    // request with more, several units).  With 4 rows a key head, in units of 8 and of 16:
    // 64 decodes of 257 to 16385 slots 183 and 234 us, 256 over 512 slots 96 and 110; with
    // 16 rows, units of 8 would read every key twice
    const int64_t rows = a.num_tokens * args.group;
    args.unit_rows = rows <= 8 * (int64_t)a.num_requests ? 8 : 16;
    args.rows_cap = (int)(rows < args.unit_rows ? (rows + 3) / 4 * 4 : args.unit_rows);
    // a scale of 0 as the least normal number, so that exponents stay numbers
    args.c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1.17549435e-38f);
    args.flip = a.scale < 0 ? 0x80008000u : 0u;
    const Scales sc = scales_of(f);
    return a.dtype == PLE_BF16 ? launch_dtype<true>(args, sc, k, v, stream)
                               : launch_dtype<false>(args, sc, k, v, stream);
}

}  // namespace ple
