// Attention of drafted nodes over a paged cache in 8 bits, on the tensor cores of
// sm_103a: the kernel for many rows a key head.
//
// The mathematics, scales and references are those of ple_tree_attention_fp8.cu, the
// rows, tiles, segments and the two softmax groups those of ple_tree_attention_tc.cu:
//   S = Q E^T           (in products of elements, accumulated in tensor memory)
//   x = c a S           (a the key scale of a column's block, 16 columns or more)
//   w = b exp2(x - top) * 2^(top - ref)   (b the value scale; as halves over S)
//   O = O + w F         (value elements F as halves)
// with the row's sum of exp2(x - top) in registers.
//
// Queries.  Keys enter their product as they are kept.  A row of queries, times a power
// of two that takes its largest element to [128, 256), is written as a sum of elements:
// the nearest one, the nearest to the rest, and for float16 the nearest to what is left
// then.  Two hold the eight significant bits of bfloat16, three the eleven of float16, but
// for what lies below 2^-10, 2^-17 of the row's largest.  The parts follow each other in
// the reduction; elements multiply at twice the rate of halves, so two cost what halves
// would, and keys need no other form.
//
// Blocks.  One block an SM, four warpgroups: two of softmax, a row a thread; one that
// turns values into halves, from one ring of shared memory into another (a conversion of
// two is one instruction, and every element is a half exactly); and a warp each to copy
// tiles of keys, of values (tiled bulk copies, page by page), to issue the matrix
// instructions and to walk the segments ahead.  Registers are dealt out anew among them.
//
// Copies.  The lanes of a warp hold 32 rows' scores and no other warp can read them, so
// with 32 rows one warp of four would do all exponentials.  Up to 64 rows stand two times
// in their tile, up to 32 four times, and each copy takes its part of a tile's columns (the
// others' weights are zeros), a row of its own until the copies meet at the segment's end.
// 8 nodes of 4 heads over 32 x 16384 slots: 241 us without, 214 with four copies; 16 nodes
// 261 and 238 with two; heads of 64, 8 nodes, 210 and 169.  Units of 64 rows where requests
// have more on the average read keys twice: 32 ragged requests of 66 on the average 360 us
// instead of 288.
//
// Measured (bf16, heads of 128, 32 query and 8 key heads, 64-slot pages, the join with
// it; in brackets the cache in 16 bits).  32 requests over 16384 slots: 4 nodes 207 us, 8
// nodes 211 (324), 32 nodes 289 (337), 64 nodes 493 (421); 64 nodes of 64 heads over
// 130981 slots, float16, 268 (221); 32 ragged requests of 17 to 32749 slots 286 to 306, as
// long contexts meet large trees or not (343).  160 us are the bytes.  512 nodes, a prompt's
// chunk, over 0, 4096 and 16384 slots 37, 69 and 142; four such 62, 177 and 476.  A tile is some 2000 clocks at few rows, where shared memory alone
// is read and written for 1400; with 128 rows the chain of a group: some 1900 clocks of
// softmax for 128 rows of 128 keys, and 1400 from the weights to the next scores.  With
// 256 rows a tile's products read more shared memory than those of the cache in 16 bits
// (the queries' terms), and the turned values are written and read once more: that is what
// the halved bytes cost.
//
// What is not seen: as in ple_tree_attention_tc.cu.  Values past the request's tokens and
// elements of drafted nodes that are NaN are cleared as they are converted; rows that
// see the latter become NaN at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "ple_fp8.cuh"
#include "ple_tc.cuh"
#include "ple_tree_fp8_internal.h"
#include "ple_tree_split.cuh"

namespace ple {
namespace {

constexpr int kThreads = 512;
constexpr int kKeyWarp = 8, kIssueWarp = 9, kValueWarp = 10, kWalkWarp = 11;
constexpr int kTurnWarp = 12;                                  // the first of four
// 512 threads are launched with 128 registers each
constexpr int kSoftmaxRegisters = 176, kOneTaskRegisters = 64, kTurnRegisters = 96;
static_assert(2 * kSoftmaxRegisters + kOneTaskRegisters + kTurnRegisters == 4 * 128, "");

constexpr int kScaleTiles = 16;
constexpr int kBadSegments = 8;

// As in ple_tree_attention_fp8.cu.
constexpr float kRise = 5.0f, kFall = 7.0f, kBias = 9.0f;
constexpr float kMostSum = 0x1p68f;

// kPairs: units of up to 256 rows (heads of up to 128 elements), 128 for each group; else
// of up to 128 / kCopies, and the groups take the tiles in turn.
template <int D, bool kBf16, bool kPairs, int kCopies>
struct Shape {
    static constexpr int kParts = D > 128 ? 2 : 1;       // of a head
    static constexpr int kWidth = D / kParts;            // elements a part
    static constexpr int kTerms = kBf16 ? 2 : 3;         // of a query
    static constexpr int kBytes = kTile * kWidth;        // of a part's tile of elements
    static constexpr int kTileBytes = 2 * kBytes;        // and of halves
    static constexpr int kHalfBytes = kTile * 128;       // a swizzled block of 64 halves a row
    static constexpr int kTermBytes = (kPairs ? 2 : 1) * kTerms * kBytes;
    // (at least what 32 columns of all copies take when they meet)
    static constexpr int kQueryBytes = kCopies > 1 && kTermBytes < 32768 ? 32768 : kTermBytes;
    // rings of values as halves, those at work and the next ones, and of keys and values as
    // they come, with what is left (an SM's share of the measured bandwidth is 45 GB/s,
    // and a loaded memory answers in 2 us)
    static constexpr int kSlots = kWidth == 64 ? 4 : 2;
    // 227 KB less the barriers and what else is shared
    static constexpr int kRings = (kWidth == 64 ? 216 : 208) * 1024;
    static constexpr int kPlaces = (kRings - kQueryBytes - kSlots * kTileBytes) / kBytes;
    static constexpr int kKeys = (kPlaces + 1) / 2 + (kPlaces > 6 ? 1 : 0);
    static constexpr int kValues = kPlaces - kKeys;
    static constexpr int kSmem = kQueryBytes + kSlots * kTileBytes + kPlaces * kBytes + 1024;
    // half of the 512 columns for each group: S (and the weights over it), O behind it
    static constexpr uint32_t kGroupColumns = 256;
    static constexpr uint32_t kOut = 128;
    // rows of elements span a swizzle of 128 bytes, or of 64
    static constexpr uint32_t kAtom = 8 * kWidth;
};

// A 16-byte piece's place in a tile of elements.
template <int kWidth>
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
    return row * kWidth + ((kWidth == 128 ? piece ^ (row & 7) : piece ^ (row >> 1 & 3)) << 4);
}

__device__ __forceinline__ uint4 load_shared(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at));
    return v;
}
__device__ __forceinline__ void store_shared(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}

// The weights of 32 columns, two blocks: exp2(f x + at), as halves, and their share of the
// row's sum.
__device__ __forceinline__ void weigh(const uint32_t (&x)[32], float f_low, float f_high,
                                      float at_low, float at_high, float base, float& sum,
                                      uint32_t (&p)[16]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float f = h ? f_high : f_low, at = h ? at_high : at_low;
        const uint64_t f2 = pack_f32(f, f), at2 = pack_f32(at, at);
        uint64_t part[2];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t pair =
                pack_f32(as_float(x[16 * h + 2 * i]), as_float(x[16 * h + 2 * i + 1]));
            float x0, x1;
            unpack_f32(fma_f32x2(pair, f2, at2), x0, x1);
            x0 = exp2_fast(x0);
            x1 = exp2_fast(x1);
            const uint64_t e2 = pack_f32(x0, x1);
            part[i & 1] = i < 2 ? e2 : add_f32x2(part[i & 1], e2);
            p[8 * h + i] = round_pair<false>(x0, x1);
        }
        float p0, p1;
        unpack_f32(add_f32x2(part[0], part[1]), p0, p1);
        sum = fmaf(p0 + p1, exp2_fast(-(at + base)), sum);
    }
}

// A place in a ring, and how often it was filled before.
template <int kPlaces>
struct Turn {
    int at = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void next() {
        if (++at == kPlaces) {
            at = 0;
            ++round;
        }
    }
};

template <int D, bool kBf16, bool kPairs, int kCopies>
__global__ void __launch_bounds__(kThreads, 1)
tree_attention_fp8_tc_kernel(const __grid_constant__ TcArgs args,
                             const __grid_constant__ Scales sc,
                             const __grid_constant__ CUtensorMap k_map,
                             const __grid_constant__ CUtensorMap v_map) {
    using S = Shape<D, kBf16, kPairs, kCopies>;
    const ple_tree_attention_args& a = args.a;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t key_full[S::kKeys], key_empty[S::kKeys];
    __shared__ __align__(8) uint64_t stage_full[S::kValues], stage_empty[S::kValues];
    __shared__ __align__(8) uint64_t full[S::kSlots], empty[S::kSlots];
    __shared__ __align__(8) uint64_t q_full[2], q_empty, s_full[2], p_low[2], p_high[2], pv_done[2];
    __shared__ __align__(8) uint64_t last;
    // Tiles' scales, (a, log2 b) for each block of 16 slots, written as a tile is copied:
    // more tiles than are ever on their way from there to the softmax.
    __shared__ __align__(16) float2 scale_s[kScaleTiles][kTile / 16];
    __shared__ __align__(8) uint64_t scale_full[kScaleTiles];
    static_assert(S::kKeys + 4 <= kScaleTiles, "");
    __shared__ int64_t scratch[kThreads / 32];
    __shared__ Share share_s;
    __shared__ uint32_t tmem_s;
    __shared__ int failed_s;
    // Whether drafted values of a segment hold NaN, as each converting warp found.  A segment's
    // flags are read while its rows go out: until then no place of the next ones' values is given
    // back, so that warpgroup has converted kSlots segments of one tile at most behind it, and
    // cleared the flags of one more.
    __shared__ int bad_s[kBadSegments][4];
    static_assert(S::kSlots + 2 <= kBadSegments, "");
    __shared__ float join_s[kCopies > 1 ? 2 * kTile : kTile][2];
    __shared__ int8_t shift_s[2][kTile];   // of a group's rows
    __shared__ Segment seg_s[2];
    __shared__ int more_s[2];
    __shared__ int64_t end_s[2];      // the place behind the segment
    volatile int* failed = &failed_s;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* smem = smem_raw + (((smem_addr(smem_raw) + 1023) & ~1023u) - smem_addr(smem_raw));
    uint8_t* q_tiles = smem;
    uint8_t* ring = smem + S::kQueryBytes;                    // values as halves
    uint8_t* key_ring = ring + S::kSlots * S::kTileBytes;
    uint8_t* stages = key_ring + S::kKeys * S::kBytes;         // values as they come

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kKeys; ++i) {
            mbar_init(&key_full[i], 1);
            mbar_init(&key_empty[i], 1);
        }
        for (int i = 0; i < S::kValues; ++i) {
            mbar_init(&stage_full[i], 1);
            mbar_init(&stage_empty[i], 4);
        }
        for (int i = 0; i < kScaleTiles; ++i) mbar_init(&scale_full[i], 1);
        for (int i = 0; i < S::kSlots; ++i) {
            mbar_init(&full[i], 4);
            mbar_init(&empty[i], 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(&q_full[w], 128);
            mbar_init(&s_full[w], 1);
            mbar_init(&p_low[w], 4);
            mbar_init(&p_high[w], 4);
            mbar_init(&pv_done[w], 1);
        }
        mbar_init(&q_empty, 1);
        mbar_init(&last, 1);
        failed_s = 0;
        fence_barrier_init();
    }
    if (warp == kIssueWarp) tmem_alloc(&tmem_s, 512);
    if (warp == kKeyWarp && lane == 0) {
        prefetch_map(&k_map);
        prefetch_map(&v_map);
    }
    wait_grid_before();

    find_share<kThreads>(args, scratch, &share_s);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_s;
    const int group = args.group;
    if (warp >= kTurnWarp) {
        // ---------------------------------------------------- values to halves
        fewer_registers<kTurnRegisters>();
        const int mine = warp - kTurnWarp;
        Walk<S::kParts> walk;
        walk.begin(args, share_s);
        Segment s;
        Turn<S::kValues> stage;
        Turn<S::kSlots> slot;
        uint32_t seg = 0;
        // A lane's 16 elements of a row, and its rows: of each eight in turn the rows first
        // and first ^ 2 (of rows of 64 bytes: first alone).  Eight lanes that access
        // memory together have four pieces of rows r and r ^ 5, and so meet eight banks in
        // both tiles; a row two further on is an exclusive or on every address.
        constexpr bool kWide = S::kWidth == 128;
        const int piece = kWide ? (lane & 3) + (lane >> 1 & 4) : lane & 3;
        const int first_row = mine * (kTile / 4) +
                              (kWide ? (lane >> 4) ^ (lane >> 2 & 1) * 5 : lane >> 2);
        const uint32_t from0 = piece_at<S::kWidth>(first_row, piece);
        const uint32_t to0 = piece / 4 * S::kHalfBytes + first_row * 128 +
                             ((2 * (piece & 3) ^ (first_row & 7)) << 4);
        const uint32_t stages_at = smem_addr(stages), ring_at = smem_addr(ring);
        bool ended = false;
        while (!ended && walk.next(args, s)) {
            if (lane == 0) bad_s[seg % kBadSegments][mine] = 0;
            __syncwarp();
            for (int i = 0; i < (s.k1 - s.k0) * S::kParts; ++i) {
                if (!mbar_wait(&stage_full[stage.at], stage.round & 1, failed) ||
                    !mbar_wait(&empty[slot.at], (slot.round & 1) ^ 1, failed)) {
                    ended = true;
                    break;
                }
                const uint32_t from = stages_at + stage.at * S::kBytes + from0;
                const uint32_t to = ring_at + slot.at * S::kTileBytes + to0;
                const int first = (s.k0 + i / S::kParts) * kTile;
                if (first + kTile > s.q.ctx) {
                    // Values past the request's tokens, and NaN of drafted ones, cleared
                    // where they lie, in a walk of their own: few tiles have any
                    const int seen_to = s.q.length - first, known_to = s.q.ctx - first;
                    bool bad = false;
#pragma unroll 1
                    for (int k = 0; k < 32; ++k) {
                        const int row = mine * (kTile / 4) + k;
                        if (row < known_to || lane >= S::kWidth / 16) continue;
                        uint4* at = reinterpret_cast<uint4*>(stages + stage.at * S::kBytes +
                                                             row * S::kWidth) + lane;
                        if (row >= seen_to) {
                            *at = make_uint4(0, 0, 0, 0);
                        } else {
                            const uint4 v = *at;
                            const uint32_t n[4] = {nan_flags(v.x), nan_flags(v.y), nan_flags(v.z),
                                                   nan_flags(v.w)};
                            if (n[0] | n[1] | n[2] | n[3]) {
                                bad = true;
                                *at = make_uint4(v.x & ~((n[0] >> 7) * 0xFFu),
                                                 v.y & ~((n[1] >> 7) * 0xFFu),
                                                 v.z & ~((n[2] >> 7) * 0xFFu),
                                                 v.w & ~((n[3] >> 7) * 0xFFu));
                            }
                        }
                    }
                    if (__any_sync(0xffffffffu, bad) && lane == 0)
                        bad_s[seg % kBadSegments][mine] = 1;
                    __syncwarp();
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
#pragma unroll
                    for (int odd = 0; odd < (kWide ? 2 : 1); ++odd) {
                        const uint32_t turn = odd ? 2 * 128 + (2 << 4) : 0;
                        const uint4 v = load_shared((from ^ turn) + k * 8 * S::kWidth);
                        uint4 low, high;
                        halves_of(v.x, low.x, low.y);
                        halves_of(v.y, low.z, low.w);
                        halves_of(v.z, high.x, high.y);
                        halves_of(v.w, high.z, high.w);
                        store_shared((to ^ turn) + k * 8 * 128, low);
                        store_shared((to ^ turn ^ 16) + k * 8 * 128, high);
                    }
                }
                fence_async_proxy();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&full[slot.at]);
                    mbar_arrive(&stage_empty[stage.at]);
                }
                stage.next();
                slot.next();
            }
            ++seg;
        }
    } else if (warp >= 8) {
        fewer_registers<kOneTaskRegisters>();
        Walk<S::kParts> walk;
        walk.begin(args, share_s);
        Segment s;
        if (warp == kWalkWarp) {
            // --------------------------- the groups' segments, one ahead
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
                named_barrier<288>(3);
            } while (more);
        } else if (warp == kKeyWarp || warp == kValueWarp) {
            // ------------------------------------------------------- copies
            const bool keys = warp == kKeyWarp;
            const CUtensorMap* map = keys ? &k_map : &v_map;
            uint64_t* filled = keys ? key_full : stage_full;
            uint64_t* freed = keys ? key_empty : stage_empty;
            uint8_t* places = keys ? key_ring : stages;
            const int most = keys ? S::kKeys : S::kValues;
            const int box = page_box(a.page_size);
            const int boxes = kTile / box;     // of a tile, each in one page
            const bool mine = lane < boxes;
            int at = 0;
            uint32_t round = 0, tiles = 0;
            bool ended = false;
            while (!ended && walk.next(args, s)) {
                const int n = s.k1 - s.k0;
                const int32_t* table = a.page_table + (int64_t)s.r * a.max_pages;
                // a box past the tokens, or of a page outside the cache, is filled
                // with zeros: its page number is outside the map
                auto page_of = [&](int j) -> int {
                    const int slot = (s.k0 + j) * kTile + lane * box;
                    if (!mine || j >= n || slot >= s.q.length) return (int)a.num_pages;
                    const int p = __ldg(table + sc.page_of(slot));
                    return p < 0 || p >= a.num_pages ? (int)a.num_pages : p;
                };
                // the queries come to the L2 cache before the groups read them
                if (!keys) {
                    const int first_row = s.unit * args.unit_rows;
                    for (int r = lane; r < s.rows; r += 32) {
                        const unsigned short* at = static_cast<const unsigned short*>(a.q) +
                                                   query_row(args, s, first_row + r);
#pragma unroll
                        for (int h = 0; h < D / 64; ++h)
                            if (64 * h < a.head_dim) prefetch_l2(at + 64 * h);
                    }
                }
                // the warp of the keys also hands over the scales: lanes 0 to 7 a block of 16
                // slots each, asked for a tile ahead, their page two
                auto block_slot = [&](int j) -> uint32_t {
                    return (s.k0 + j) * kTile + (lane & 7) * 16;
                };
                auto block_page = [&](int j) -> int {
                    const uint32_t slot = block_slot(j);
                    int number = -1;
                    if (keys && j < n && (int)slot < s.q.length)
                        number = load_now(table + sc.page_of(slot));
                    return number;
                };
                uint32_t k_ahead, v_ahead;
                auto ask = [&](int j, int number) {
                    sc.ask(number, a.num_pages, s.head, block_slot(j), a.page_size, k_ahead,
                           v_ahead);
                };
                ask(0, block_page(0));
                int number = block_page(1);
                int page = page_of(0);
                for (int j = 0; j < n && !ended; ++j) {
                    const int after = page_of(j + 1);
                    if (keys) {
                        const uint32_t entry = tiles++ % kScaleTiles;
                        if (lane < 8)
                            scale_s[entry][lane] =
                                make_float2(scale_value(k_ahead), scale_log(v_ahead));
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&scale_full[entry]);
                        ask(j + 1, number);
                        number = block_page(j + 2);
                    }
#pragma unroll
                    for (int part = 0; part < S::kParts; ++part) {
                        if (!mbar_wait(&freed[at], (round & 1) ^ 1, failed)) {
                            ended = true;
                            break;
                        }
                        if (lane == 0) mbar_arrive_expect(&filled[at], S::kBytes);
                        __syncwarp();
                        if (mine)
                            copy_box(map,
                                     smem_addr(places) + at * S::kBytes +
                                         lane * box * S::kWidth,
                                     &filled[at], part * S::kWidth,
                                     sc.in_page((s.k0 + j) * kTile + lane * box, a.page_size),
                                     s.head, page);
                        if (++at == most) {
                            at = 0;
                            ++round;
                        }
                    }
                    page = after;
                }
            }
            if (ended) {
                // copies may be in flight: they land before the block ends
                for (int i = 0; i < most; ++i) {
                    const uint32_t rounds = round + (i < at);
                    const long long start = clock64();
                    while (rounds != 0 && !mbar_try(&filled[i], (rounds - 1) & 1) &&
                           clock64() - start < kWaitClocks) {
                    }
                }
                __syncwarp();
            }
        } else if (warp == kIssueWarp) {
            // -------------------------------------------- matrix instructions
            // One lane does all of it.  A tile is 32 instructions and six waits, and what
            // stands between them is what the tensor cores wait for: descriptors are a
            // base and constants, and nothing is shared with the warp's other lanes.
            // The type of an element has the number that a half has among wider types.
            constexpr uint32_t kScoreWord = mma_word(false, false, kTile, kTile);
            constexpr uint32_t kOutWord = mma_word(false, true, kTile, S::kWidth);
            if (elect_lane()) {
                const uint32_t values_at = half_desc_low(smem_addr(ring), S::kHalfBytes);
                const uint32_t keys_at = element_desc_low(smem_addr(key_ring));
                const uint32_t q_at = element_desc_low(smem_addr(q_tiles));
                uint32_t p_count[2] = {0, 0}, pairs = 0, seg = 0;
                Turn<S::kKeys> key;
                Turn<S::kSlots> value;
                auto wait_key = [&]() -> uint32_t {
                    const uint32_t at = key.at;
                    lane_wait(&key_full[at], key.round & 1, failed);
                    key.next();
                    return at;
                };
                auto wait_value = [&]() -> uint32_t {
                    const uint32_t at = value.at;
                    lane_wait(&full[at], value.round & 1, failed);
                    value.next();
                    return at;
                };
                while (walk.next(args, s)) {
                    const int n = s.k1 - s.k0;
                    lane_wait(&q_full[0], seg & 1, failed);
                    if (s.pair) lane_wait(&q_full[1], pairs++ & 1, failed);
                    tmem_fence_after();
                    // Every step takes a group's weights and gives it its next scores: a
                    // tile for both groups in two steps, or tiles in turn
                    const bool both = S::kParts == 2 || (kPairs && s.pair);
                    const int steps = both ? 2 * n : n;
                    uint32_t k = 0, k2 = 0, v = 0;
#pragma unroll 1
                    for (int i = -2; i < steps; ++i) {
                        const int w = i & 1;
                        const uint32_t at = tmem + w * S::kGroupColumns;
                        if (i >= 0) {
                            if (!both || S::kParts == 2 || w == 0) v = wait_value();
                            const uint32_t vd = values_at + (v * S::kTileBytes >> 4);
                            const uint32_t parity = p_count[w]++ & 1;
                            // the first half's product runs while the second's weights
                            // are computed
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                if (!lane_wait(half ? &p_high[w] : &p_low[w], parity, failed))
                                    break;
                                tmem_fence_after();
#pragma unroll
                                for (int c = 0; c < kTile / 32; ++c)
                                    mma_tmem_at<kOutWord, half_desc_high()>(
                                        at + S::kOut, at + half * (kTile / 4) + c * 8,
                                        vd + ((half * (kTile / 2) + c * 16) * 128 >> 4),
                                        half != 0 || c != 0 || i >= 2);
                            }
                            if (*failed) break;
                            mma_commit(&pv_done[w]);
                            if (!both || S::kParts == 2 || w == 1) mma_commit(&empty[v]);
                        }
                        if (i + 2 < steps) {
                            if (!both || w == 0) {
                                k = wait_key();
                                if (S::kParts == 2) k2 = wait_key();
                            }
                            const uint32_t q_tile = both && S::kParts == 1 ? w : 0;
#pragma unroll
                            for (int part = 0; part < S::kParts; ++part) {
                                const uint32_t kd = keys_at + ((part ? k2 : k) * S::kBytes >> 4);
                                const uint32_t qd =
                                    q_at + ((q_tile + part) * S::kTerms * S::kBytes >> 4);
#pragma unroll
                                for (int term = 0; term < S::kTerms; ++term)
#pragma unroll
                                    for (int c = 0; c < S::kWidth / 32; ++c)
                                        mma_elements_at<kScoreWord, element_desc_high<S::kAtom>()>(
                                            at, qd + (term * S::kBytes >> 4) + 2 * c, kd + 2 * c,
                                            part != 0 || term != 0 || c != 0);
                            }
                            mma_commit(&s_full[w]);
                            if (!both || w == 1) {
                                mma_commit(&key_empty[k]);
                                if (S::kParts == 2) mma_commit(&key_empty[k2]);
                            }
                        }
                    }
                    mma_commit(&q_empty);
                    ++seg;
                }
                // everything issued is done before the block ends, also after a failure
                mma_commit(&last);
                const long long start = clock64();
                while (!mbar_try(&last, 0) && clock64() - start < kWaitClocks) {
                }
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------- softmax
        more_registers<kSoftmaxRegisters>();
        const int w = warp >> 2;
        const int row = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + w * S::kGroupColumns + lanes;
        const uint32_t o_at = s_at + S::kOut;
        uint32_t seg = 0, count = 0, tiles = 0;   // tiles: of the segments before
        if (threadIdx.x == 0) static_cast<Cut*>(a.workspace)[blockIdx.x].last = -1;
        for (;;) {
            named_barrier<288>(3);
            if (!*static_cast<volatile int*>(&more_s[seg & 1])) break;
            const volatile Segment& s = seg_s[seg & 1];
            const int n = s.k1 - s.k0;
            constexpr bool kSplit = S::kParts == 2;   // both groups have the same rows
            const int row0 = s.pair && !kSplit ? w * kTile : 0;   // the group's in the unit
            const int first_row = s.unit * args.unit_rows + row0;
            const int rows = s.pair && !kSplit ? (w == 0 ? kTile : s.rows - kTile) : s.rows;
            const int column0 = kSplit ? w * S::kWidth : 0;       // of the group's accumulators
            constexpr int span = kTile / kCopies;
            const int own = row % span, copy = row / span;     // the row, and which copy of it
            constexpr int quarters = 4 / kCopies;              // of the columns
            const int quarter0 = copy * quarters;
            const bool active = (own & ~31) < rows;   // a warp with no row only keeps step
            const bool here = own < rows;
            const int node = (first_row + own) / group;
            const int64_t token = s.q.begin + node;
            const int64_t head = (int64_t)s.head * group + (first_row + own) - node * group;
            const unsigned long long* mask =
                reinterpret_cast<const unsigned long long*>(a.tree_mask) +
                (here ? token : 0) * a.mask_words;
            // asked for long before the tiles that need it
            const uint64_t mask_word = here ? __ldg(mask) : 0;

            const int step = s.pair ? 1 : 2;
            // what every tile asks for stays in registers: shared memory is busy
            const int k0 = s.k0, ctx = s.q.ctx, length = s.q.length;
            const int j0 = s.pair ? 0 : w;

            // this group's queries, rows of the unit, into swizzled shared memory, or
            // its part of all of them
            if (s.pair || w == 0) {
                if (seg > 0) mbar_wait(&q_empty, (seg - 1) & 1, failed);
                uint8_t* tile = q_tiles + (s.pair ? w : 0) * S::kTerms * S::kBytes;
                constexpr int kPer = S::kWidth / 8;      // lanes a row
                constexpr int kAtOnce = 128 / kPer;      // rows
                // rows in flight: one by one, a segment's queries took 10 us
                constexpr int kAhead = kSplit ? 4 : 8;
                const int ch = row % kPer;
                const unsigned short* from =
                    static_cast<const unsigned short*>(a.q) + ch * 8;
                const bool inside = column0 + ch * 8 < a.head_dim;
                const int q_rows = rows;
                // (rows of the warp together, so that the lanes of a row meet)
#pragma unroll 1
                for (int base = 0; base < q_rows; base += kAhead * kAtOnce) {
                    uint4 x[kAhead], y[kSplit ? kAhead : 1];
#pragma unroll
                    for (int z = 0; z < kAhead; ++z) {
                        const int r = base + z * kAtOnce + row / kPer;
                        x[z] = make_uint4(0, 0, 0, 0);
                        if constexpr (kSplit) y[z] = make_uint4(0, 0, 0, 0);
                        if (r < q_rows) {
                            const unsigned short* at = from + query_row(args, s, first_row + r);
                            if (inside) x[z] = __ldg(reinterpret_cast<const uint4*>(at + column0));
                            // of a head in parts the other part's, for the row's largest
                            if constexpr (kSplit)
                                if (S::kWidth - column0 + ch * 8 < a.head_dim)
                                    y[z] = __ldg(reinterpret_cast<const uint4*>(at + S::kWidth -
                                                                                column0));
                        }
                    }
#pragma unroll
                    for (int z = 0; z < kAhead; ++z) {
                        const int r = base + z * kAtOnce + row / kPer;
                        if (base + z * kAtOnce >= q_rows) break;
                        float q[8], most = 0.f;
                        const uint32_t words[4] = {x[z].x, x[z].y, x[z].z, x[z].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            widen_pair<kBf16>(words[i] ^ args.flip, q[2 * i], q[2 * i + 1]);
                            most = fmaxf(most, fmaxf(fabsf(q[2 * i]), fabsf(q[2 * i + 1])));
                        }
                        if constexpr (kSplit) {
                            const uint32_t others[4] = {y[z].x, y[z].y, y[z].z, y[z].w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float z0, z1;
                                widen_pair<kBf16>(others[i], z0, z1);
                                most = fmaxf(most, fmaxf(fabsf(z0), fabsf(z1)));
                            }
                        }
#pragma unroll
                        for (int d = kPer / 2; d >= 1; d >>= 1)
                            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                        const int shift = term_shift(most);
                        const float f = __uint_as_float((uint32_t)(127 - shift) << 23);
#pragma unroll
                        for (int i = 0; i < 8; ++i) q[i] *= f;
                        if (r < q_rows) {
                            if (ch == 0) shift_s[w][r] = (int8_t)shift;
                            uint8_t* to = tile + piece_at<S::kWidth>(r, ch >> 1) + 8 * (ch & 1);
#pragma unroll
                            for (int term = 0; term < S::kTerms; ++term) {
                                uint32_t e[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    e[i] = nearest_elements(q[2 * i], q[2 * i + 1]);
                                    // what this term leaves
                                    const uint32_t h = halves_of((uint16_t)e[i]);
                                    const float2 left =
                                        __half22float2(*reinterpret_cast<const __half2*>(&h));
                                    q[2 * i] -= left.x;
                                    q[2 * i + 1] -= left.y;
                                }
                                const uint2 two =
                                    make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
                                *reinterpret_cast<uint2*>(to + term * S::kBytes) = two;
#pragma unroll
                                for (int i = 1; i < kCopies; ++i)
                                    *reinterpret_cast<uint2*>(to + term * S::kBytes +
                                                              i * span * S::kWidth) = two;
                            }
                        }
                    }
                }
                fence_async_proxy();
                mbar_arrive(&q_full[w]);
            }

            float top = -INFINITY, sum = 0.f, ref = -INFINITY, heap = 0.f;
            float c = 0.f;
            bool begun = false;
            for (int j = j0; j < n; j += step) {
                const int first = (k0 + j) * kTile;
                const bool masked = first + kTile > ctx;
                MaskWindow window;
                if (masked && here)
                    window = mask_window(mask, mask_word, a.mask_words, ctx, first);
                if (!mbar_wait(&s_full[w], count & 1, failed)) break;
                // these came before the keys that the scores are of
                const uint32_t entry = (tiles + j) % kScaleTiles;
                if (!mbar_wait(&scale_full[entry], (tiles + j) / kScaleTiles & 1, failed)) break;
                const float4* scales = reinterpret_cast<const float4*>(scale_s[entry]);
                tmem_fence_after();
                if (active) {
                    // the queries, and with them their shifts, were there before the scores
                    if (!begun)
                        c = args.c *
                            __uint_as_float(
                                (uint32_t)(127 + *static_cast<volatile int8_t*>(
                                                     &shift_s[s.pair ? w : 0][own])) << 23);
                    // Scores of what is not seen become -infinity in tensor memory, in a walk
                    // of their own: few tiles have any, and the loops below stay short
                    if (masked) {
#pragma unroll 1
                        for (int q = quarter0; q < quarter0 + quarters; ++q) {
                            const uint32_t bits =
                                here ? seen_bits(window, a.mask_words, ctx, length,
                                                 first + 32 * q)
                                     : 0u;
                            __syncwarp();
                            uint32_t x[32];
                            tmem_load(s_at + 32 * q, x);
                            tmem_wait_load(x);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(bits >> i & 1)) x[i] = 0xFF800000u;
                            tmem_store(s_at + 32 * q, x);
                        }
                        tmem_wait_store();
                    }
                    // The row's scores are walked twice, 64 columns at a time: the
                    // upper half and then the lower for the maximum, the lower, still in
                    // registers, and the upper again for the weights.  A block that the row
                    // sees nothing of is -infinity whatever its scales (a minimum or
                    // maximum with NaN is the other number).
                    // a block's factor from score to exponent of 2, and that log
                    float factor[8], place[8];
                    uint32_t v[2][32];
                    float now = top, reach = -INFINITY;
                    if constexpr (kCopies > 1) {
                        // the copy's columns alone, 32 or 64
                        float m[4];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (k < quarters) {
                                const uint32_t at = s_at + 32 * (quarter0 + k);
                                tmem_load_max16(at, v[k], 0, m[2 * k]);
                                tmem_load_max16(at + 16, v[k], 16, m[2 * k + 1]);
                                const float4 two = scales[quarter0 + k];
                                factor[2 * k] = fmaxf(c * two.x, 1.17549435e-38f);
                                place[2 * k] = two.y;
                                factor[2 * k + 1] = fmaxf(c * two.z, 1.17549435e-38f);
                                place[2 * k + 1] = two.w;
                                tmem_wait_load(v[k]);
                                asm volatile("" : "+f"(m[2 * k]), "+f"(m[2 * k + 1]));
#pragma unroll
                                for (int b = 2 * k; b < 2 * k + 2; ++b) {
                                    const float x = m[b] * factor[b];
                                    now = fmaxf(now, x);
                                    reach = fmaxf(reach, x + place[b]);
                                }
                            }
                        }
                    } else {
#pragma unroll
                        for (int h = 1; h >= 0; --h) {
                            float m[4];
                            tmem_load_max16(s_at + 64 * h, v[0], 0, m[0]);
                            tmem_load_max16(s_at + 64 * h + 16, v[0], 16, m[1]);
                            tmem_load_max16(s_at + 64 * h + 32, v[1], 0, m[2]);
                            tmem_load_max16(s_at + 64 * h + 48, v[1], 16, m[3]);
#pragma unroll
                            for (int b = 4 * h; b < 4 * h + 4; b += 2) {
                                const float4 two = scales[b / 2];
                                factor[b] = fmaxf(c * two.x, 1.17549435e-38f);
                                place[b] = two.y;
                                factor[b + 1] = fmaxf(c * two.z, 1.17549435e-38f);
                                place[b + 1] = two.w;
                            }
                            tmem_wait_load(v[0]);
                            tmem_settle(v[0], m[0]);
                            tmem_settle(v[1], m[1]);
                            asm volatile("" : "+f"(m[2]), "+f"(m[3]));
#pragma unroll
                            for (int b = 0; b < 4; ++b) {
                                const float x = m[b] * factor[4 * h + b];
                                now = fmaxf(now, x);
                                reach = fmaxf(reach, x + place[4 * h + b]);
                            }
                        }
                    }
                    const float base = now == -INFINITY ? 0.f : now;
                    sum *= exp2_fast(top - base);
                    top = now;
                    // a new reference only where the tile's largest weight is far from it
                    const float fall = ref - reach;
                    const bool move =
                        here && (-fall > kRise ||
                                 (fall > kFall && heap * exp2_fast(fall) < kMostSum));
                    if (__any_sync(0xffffffffu, move)) {
                        const float f =
                            move ? (ref == -INFINITY ? 0.f : exp2_fast(ref - reach)) : 1.f;
                        if (move) ref = reach;
                        heap *= f;
                        if (begun) {
                            mbar_wait(&pv_done[w], (count - 1) & 1, failed);
                            tmem_fence_after();
#pragma unroll 1
                            for (int q = 0; q < S::kWidth / 32; ++q) {
                                uint32_t o[32];
                                tmem_load(o_at + 32 * q, o);
                                tmem_wait_load(o);
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tmem_store(o_at + 32 * q, o);
                            }
                        }
                    }
                    // at most this much for the tile's 128 weights
                    if (ref != -INFINITY) heap += exp2_fast(reach - ref + kBias + 8.f);
                    // Weights with their value scale relative to the row's reference; the
                    // sum takes a block's together, that scale out again.  A scale 2^-100
                    // of what the reference stands for counts as that: its weights, which
                    // the sum needs, would be lost, and its values are nothing to the row.
                    const float to_ref = ref == -INFINITY ? 0.f : kBias - ref;
                    const float least = -100.f - base;
                    if constexpr (kCopies > 1) {
                        // no weights for the other copies' columns
                        const uint32_t none[16] = {};
#pragma unroll 1
                        for (int q = 0; q < 4; ++q)
                            if (q / quarters != copy) tmem_store(s_at + 16 * q, none);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (k < quarters) {
                                uint32_t p[16];
                                weigh(v[k], factor[2 * k], factor[2 * k + 1],
                                      fmaxf(place[2 * k] + to_ref, least),
                                      fmaxf(place[2 * k + 1] + to_ref, least), base, sum, p);
                                tmem_store(s_at + 16 * (quarter0 + k), p);
                            }
                        }
                        tmem_wait_store();
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&p_low[w]);
                            mbar_arrive(&p_high[w]);
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t (&x)[32] = v[q & 1];
                            if (q > 1) tmem_wait_load(x);
                            uint32_t p[16];
                            weigh(x, factor[2 * q], factor[2 * q + 1],
                                  fmaxf(place[2 * q] + to_ref, least),
                                  fmaxf(place[2 * q + 1] + to_ref, least), base, sum, p);
                            if (q < 2) tmem_load(s_at + 32 * (q + 2), x);
                            // over columns whose scores have been read
                            tmem_store(s_at + 16 * q, p);
                            if (q & 1) {
                                tmem_wait_store();
                                tmem_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(q == 1 ? &p_low[w] : &p_high[w]);
                            }
                        }
                    }
                } else {
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&p_low[w]);
                        mbar_arrive(&p_high[w]);
                    }
                }
                begun = true;
                ++count;
            }
            if (begun) mbar_wait(&pv_done[w], (count - 1) & 1, failed);
            tmem_fence_after();
            tiles += n;

            // ------------------------------------ the segment's rows go out
            // Where both groups hold states of the same rows, group 1's go to group 0
            // through the queries' memory, half the columns at a time.
            // Copies of rows all meet there, 32 columns at a time.
            constexpr bool meet = kCopies > 1;
            const bool join = !meet && !s.pair && n > 1;
            float4* exchange = reinterpret_cast<float4*>(q_tiles);
            constexpr int kChunks = S::kWidth / 64;   // of 32 columns, in a half
            auto hand_over = [&](int part) {
                if (w == 1 && active) {
                    const float f =
                        ref == -INFINITY ? 0.f : exp2_fast(fminf(ref - kBias - top, 126.f));
#pragma unroll 1
                    for (int q = 0; q < kChunks; ++q) {
                        uint32_t o[32];
                        tmem_load(o_at + 32 * (part * kChunks + q), o);
                        tmem_wait_load(o);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            exchange[(q * 8 + i) * kTile + row] = make_float4(
                                __uint_as_float(o[4 * i]) * f, __uint_as_float(o[4 * i + 1]) * f,
                                __uint_as_float(o[4 * i + 2]) * f,
                                __uint_as_float(o[4 * i + 3]) * f);
                    }
                }
                named_barrier<256>(1);
            };
            if (join) {
                if (w == 1) {
                    mbar_wait(&q_empty, seg & 1, failed);   // the queries have been read
                    if (active) {
                        join_s[row][0] = top;
                        join_s[row][1] = sum;
                    }
                }
                hand_over(0);
            }
            // a row's states lie `span` threads apart
            constexpr int states = 2 * kCopies;
            float meet_f = 0.f;
            if constexpr (meet) {
                mbar_wait(&q_empty, seg & 1, failed);
                const int me = w * kTile + row;
                join_s[me][0] = top;
                join_s[me][1] = sum;
                named_barrier<256>(1);
                for (int i = 0; i < states; ++i) top = fmaxf(top, join_s[i * span + own][0]);
                const float base = top == -INFINITY ? 0.f : top;
                sum = 0.f;
                for (int i = 0; i < states; ++i)
                    sum = fmaf(join_s[i * span + own][1],
                               exp2_fast(join_s[i * span + own][0] - base), sum);
                meet_f = ref == -INFINITY ? 0.f : exp2_fast(fminf(ref - kBias - top, 126.f));
            }
            // the accumulators of all states of a row, 32 columns, to its first one's thread
            auto meet_columns = [&](int q, float (&x)[32]) {
                const int me = w * kTile + row;
                if (begun) {
                    uint32_t o[32];
                    tmem_load(o_at + 32 * q, o);
                    tmem_wait_load(o);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        exchange[i * 2 * kTile + me] = make_float4(
                            __uint_as_float(o[4 * i]) * meet_f,
                            __uint_as_float(o[4 * i + 1]) * meet_f,
                            __uint_as_float(o[4 * i + 2]) * meet_f,
                            __uint_as_float(o[4 * i + 3]) * meet_f);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        exchange[i * 2 * kTile + me] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
                named_barrier<256>(1);
                for (int i = me / span; i < 8; i += states) {
                    float4* at = exchange + i * 2 * kTile + own;
                    float4 y = at[0];
                    for (int k = 1; k < states; ++k) {
                        const float4 z = at[k * span];
                        y.x += z.x;
                        y.y += z.y;
                        y.z += z.z;
                        y.w += z.w;
                    }
                    at[0] = y;
                }
                named_barrier<256>(1);
                if (me < span) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 y = exchange[i * 2 * kTile + own];
                        x[4 * i] = y.x;
                        x[4 * i + 1] = y.y;
                        x[4 * i + 2] = y.z;
                        x[4 * i + 3] = y.w;
                    }
                }
                named_barrier<256>(1);
            };
            {
                // whether these rows are this group's
                const bool out = s.pair || (w == 0 && copy == 0);
                // accumulators relative to the row's top
                float f1 = 0.f;
                if (join && w == 0 && here) {
                    const float other = join_s[row][0];
                    const float m = fmaxf(top, other);
                    const float base = m == -INFINITY ? 0.f : m;
                    f1 = exp2_fast(other - base);
                    sum = sum * exp2_fast(top - base) + join_s[row][1] * f1;
                    top = m;
                }
                const float f0 =
                    ref == -INFINITY ? 0.f : exp2_fast(fminf(ref - kBias - top, 126.f));
                const bool whole = s.k0 == 0 && s.k1 == s.q.tiles;
                if (threadIdx.x == 0 && s.k0 == 0 && !whole) {
                    Cut cut = {};
                    cut.last = share_of(share_s.total, end_s[seg & 1] - 1 + (s.q.tiles - s.k1),
                                        share_s.shares);
                    cut.rows = s.rows;
                    cut.begin = s.q.begin;
                    cut.first_row = s.unit * args.unit_rows;
                    cut.head = s.head;
                    static_cast<Cut*>(a.workspace)[blockIdx.x] = cut;
                }
                const bool spoiled = *failed;
                if (spoiled) sum = __int_as_float(0x7FC00000);  // NaN, not an unfinished sum
                const volatile int* found = bad_s[seg % kBadSegments];
                const bool bad = found[0] | found[1] | found[2] | found[3];
                const int64_t o_row = token * a.q_heads + head;
                float* state = static_cast<float*>(a.workspace) +
                               state_at(blockIdx.x, s.k0 == 0 ? 1 : 0, args.rows_cap, D);
                const int state_row = row0 + own;
                float* pairs = state + 2 * state_row;
                float* acc = state + (2 + column0) * args.rows_cap + 8 * state_row;
                const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
                    if (join && part == 1) {
                        named_barrier<256>(1);
                        hand_over(1);
                    }
                    if (!meet && (!out || !active)) continue;
#pragma unroll 1
                    for (int q = part * kChunks; q < (part + 1) * kChunks; ++q) {
                        const int column = column0 + 32 * q;
                        float x[32];
                        if constexpr (meet) {
                            meet_columns(q, x);
                            if (!out || !active) continue;
                        } else {
                            uint32_t o[32];
                            if (begun) {
                                tmem_load(o_at + 32 * q, o);
                                tmem_wait_load(o);
                            }
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(o[i]) * f0;
                        }
                        if (kSplit && spoiled) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = __int_as_float(0x7FC00000);
                        }
                        if (join) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float4 y = exchange[(q % kChunks * 8 + i) * kTile + row];
                                x[4 * i] = fmaf(y.x, f1, x[4 * i]);
                                x[4 * i + 1] = fmaf(y.y, f1, x[4 * i + 1]);
                                x[4 * i + 2] = fmaf(y.z, f1, x[4 * i + 2]);
                                x[4 * i + 3] = fmaf(y.w, f1, x[4 * i + 3]);
                            }
                        }
                        if (bad && here) {
                            // the drafted values that were cleared, to the rows
                            // that see them
                            for (int slot = max(s.q.ctx, s.k0 * kTile);
                                 slot < min(s.q.length, s.k1 * kTile); ++slot) {
                                const MaskWindow one = mask_window(mask, mask_word, a.mask_words,
                                                                   s.q.ctx, slot);
                                if (!(seen_bits(one, a.mask_words, s.q.ctx, s.q.length, slot) & 1))
                                    continue;
                                const int64_t at = slot_offset(
                                    a.page_table, a.max_pages, a.page_size, a.num_pages,
                                    a.page_stride, a.slot_stride, s.r, slot);
                                if (at < 0) continue;
                                const uint8_t* vrow = static_cast<const uint8_t*>(a.v_cache) + at +
                                                      s.head * a.head_stride + column;
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    if (column + i >= a.head_dim) break;
                                    if ((vrow[i] & 0x7F) == 0x7F) x[i] = __int_as_float(0x7FC00000);
                                }
                            }
                        }
                        if (here && whole) {
                            uint4* dst = reinterpret_cast<uint4*>(
                                static_cast<unsigned short*>(a.out) + o_row * a.head_dim + column);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (column + 8 * i >= a.head_dim) break;
                                uint32_t y[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    y[e] = round_pair<kBf16>(x[8 * i + 2 * e] * inv,
                                                             x[8 * i + 2 * e + 1] * inv);
                                dst[i] = make_uint4(y[0], y[1], y[2], y[3]);
                            }
                        } else if (here) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<float4*>(
                                    acc + (q * 4 + i / 2) * 8 * args.rows_cap + (i & 1) * 4) =
                                    make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                        }
                        __syncwarp();  // the next load is the whole warp's
                    }
                }
                if (out && here && column0 == 0) {
                    if (!whole) {
                        pairs[0] = top;
                        pairs[1] = sum;
                    } else if (a.lse != nullptr) {
                        a.lse[o_row] =
                            sum == 0.f ? -INFINITY : top * 0.69314718055994531f + logf(sum);
                    }
                }
            }
            tmem_fence_before();
            named_barrier<256>(2);
            ++seg;
        }
    }

    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == kIssueWarp) tmem_free(tmem, 512);
}

template <int D, bool kBf16, bool kPairs, int kCopies>
cudaError_t launch_tc(const TcArgs& args, const Scales& sc, const CUtensorMap& k,
                      const CUtensorMap& v, cudaStream_t stream) {
    using S = Shape<D, kBf16, kPairs, kCopies>;
    auto* fn = tree_attention_fp8_tc_kernel<D, kBf16, kPairs, kCopies>;
    cudaError_t e =
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_kernel(fn, dim3((unsigned)args.blocks), dim3(kThreads), S::kSmem, stream,
                      programmatic_launch(), args, sc, k, v);
    if (e != cudaSuccess) return e;
    return launch_kernel(
        tree_attention_join_kernel<D, kBf16>,
        dim3((unsigned)args.blocks, (unsigned)((args.rows_cap + kJoinRows - 1) / kJoinRows)),
        dim3(kJoinThreads), 0, stream, programmatic_launch(), args);
}

template <bool kBf16>
cudaError_t launch_dtype(const TcArgs& args, const Scales& sc, const CUtensorMap& k,
                         const CUtensorMap& v, cudaStream_t stream) {
    auto width = [&](auto d) {
        constexpr int D = d;
        auto* launch = args.unit_rows > kTile        ? launch_tc<D, kBf16, true, 1>
                       : args.unit_rows == kTile     ? launch_tc<D, kBf16, false, 1>
                       : args.unit_rows == kTile / 2 ? launch_tc<D, kBf16, false, 2>
                                                     : launch_tc<D, kBf16, false, 4>;
        return launch(args, sc, k, v, stream);
    };
    switch (padded_width(args.a.head_dim)) {
        case 64: return width(std::integral_constant<int, 64>{});
        case 128: return width(std::integral_constant<int, 128>{});
        // both parts' queries, as of two groups
        default: return launch_tc<256, kBf16, true, 1>(args, sc, k, v, stream);
    }
}

}  // namespace

int64_t tree_attention_fp8_tc_workspace(int64_t T, int32_t q_heads, int32_t kv_heads, int32_t D,
                                        const DeviceFacts& dev) {
    return 4 * state_at(tc_blocks(dev), 0, tc_rows_cap(T, q_heads, kv_heads, D), padded_width(D));
}

cudaError_t launch_tree_attention_fp8_tc(const ple_tree_attention_fp8_args& f,
                                         const CUtensorMap& k, const CUtensorMap& v,
                                         const DeviceFacts& dev, cudaStream_t stream) {
    const ple_tree_attention_args& a = f.base;
    TcArgs args;
    args.a = a;
    args.blocks = tc_blocks(dev);
    args.group = a.q_heads / a.kv_heads;
    args.rows_cap = tc_rows_cap(a.num_tokens, a.q_heads, a.kv_heads, a.head_dim);
    // units of two groups' rows where a request's are so many on the average
    args.unit_rows = unit_rows(padded_width(a.head_dim));
    const int64_t rows = a.num_tokens * args.group, B = a.num_requests;
    if (rows <= kTile * B) args.unit_rows = kTile;
    // (a prompt of 512 nodes among 64 decodes over 8192 slots each, whose keys small units
    // read four times as often, takes 369 us instead of 360; 65 nodes among 32, 139 for 152)
    if (padded_width(a.head_dim) <= 128) {
        if (rows <= kTile / 2 * B) args.unit_rows = kTile / 2;
        if (rows <= kTile / 4 * B) args.unit_rows = kTile / 4;
    }
    if (args.rows_cap > args.unit_rows) args.rows_cap = args.unit_rows;
    args.c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1.17549435e-38f);
    args.flip = a.scale < 0 ? 0x80008000u : 0u;
    const Scales sc = scales_of(f);
    return a.dtype == PLE_BF16 ? launch_dtype<true>(args, sc, k, v, stream)
                               : launch_dtype<false>(args, sc, k, v, stream);
}

}  // namespace ple
