// Attention of drafted nodes over the paged cache and their own branch, on the
// tensor cores of sm_103a, for heads of up to 256 elements (narrower ones are filled
// up with zeros to 64, 128 or 256 in shared memory).
//
// Rows.  The query heads of one key head share its keys, so for a request of n
// nodes and G = q_heads / kv_heads a key head has n * G rows (node-major).  A
// matrix instruction takes 128 of them.  For every tile of 128 keys
//   S = Q K^T        (accumulated in tensor memory)
//   P = exp2(c S - c m), m the running row maximum, c = scale * log2(e)
//   O = O + P V      (P written over S in tensor memory, O beside it)
// with the row sums of P kept in registers: the one-pass softmax of Milakov and
// Gimelshein (2018).  As is known of it, m need not be the maximum: any reference
// that the sum and O share will do, so O is scaled anew only when a tile's maximum
// is more than a few binades away from the row's reference (Reference below).
//
// Blocks.  One block an SM: two warps that copy key and value tiles into a ring
// of shared memory (tiled bulk copies, page by page, 128-byte swizzle), a warp
// that issues the matrix instructions, one that works out the next segment (a unit's
// tiles in this block) ahead of the softmax, and two groups of four warps that do
// the softmax, one row a thread.  With more than 128 rows the two groups take 128
// each over the same tiles, so that a key is read once for 256 rows; with fewer
// they take the tiles in turn over the same rows and are joined in shared memory.
// Either way one group's softmax runs while the tensor cores work for the other.
// Heads above 128 are two parts of 128 elements, a part a place of the ring, and a
// unit is 128 rows: tensor memory holds no two accumulators of 256.  Both groups
// take the same rows and tiles, each forms the scores and weights for itself
// and group w the product with the values' part w, so a key is still read
// once and the groups never meet.
//
// Split.  All tiles of all (request, key head, 256 rows) are laid end to end, each
// unit behind a few places for what it costs besides its tiles, and cut into equal
// shares, one a block, so ragged requests and few long ones fill the device
// alike.  A block writes a unit that it has whole; of a cut unit it writes the
// state (row reference, sum, O in 32 bits) to the workspace, and a second kernel
// joins the states in block order: results do not depend on timing.
//
// Measured (bf16, heads of 128, 8 key heads, 64-slot pages, the join with it).  Up
// to 128 rows a unit the keys' and values' bytes bound it: 4 rows over 32 x 16384
// slots 316 us (6.8 TB/s), 128 rows 335 us.  Above, the chain of one group's softmax, its second
// product and its next first one does (some 3500 clocks a tile, 2048 of them the
// tensor cores' for both groups): 256 rows 399 to 409 us (1.4 PFLOP/s), 512 rows over
// 1 x 131000 slots 204 to 215 us (1.3 PFLOP/s).  Few keys are a latency: 4 rows over 701
// slots 11 us.  Heads of 256: 4 rows over 32 x 8192 slots 350 us (6.1 TB/s), 128
// rows 380, 64 rows over 4 x 8192 slots 69 (4.8 ms on the kernel without tensor
// cores).
//
// What is not seen.  Scores outside the mask are replaced by -infinity before
// the maximum, so what their keys hold does not matter.  Zero weights would
// not stop an infinity or a NaN among the values in the matrix product:
// values past the request's tokens are cleared in shared memory, and values of
// drafted nodes (seen by some rows only) that are not finite are cleared there
// and added to the rows that see them at the end.
#include "ple_tc.cuh"
#include "ple_tree_split.cuh"

namespace ple {
namespace {

constexpr int kThreads = 384;        // two groups of 128 and four warps of a task each
constexpr int kKeyWarp = 8, kIssueWarp = 9, kValueWarp = 10, kWalkWarp = 11;

// How far a tile's largest weight may lie above and below 1 (in the exponent of 2)
// before the row's reference moves to it, and where weights are placed in the element
// type: P = 2^kBias times the weight.  bfloat16 has the exponents of 32 bits, so a
// reference only ever rises.  float16 ends at 2^16 and 2^-25: weights are placed
// under its upper end, and the reference also falls to a tile whose largest weight is
// small, so that a weight enters the product to 2^-11 of itself or to 2^-28 of its
// tile's largest, however far below the row's largest that lies (behind an attention
// sink all of them do).  Closer limits cost more moves, wider ones more of the small
// weights.  512 rows over 131000 slots in float16, scores of a standard deviation of
// 1.5: 212 us with these limits and with a rise of 8 alone; of 6: 231 to 243 against 217
// to 226.
template <bool kBf16>
struct Reference {
    static constexpr float kRise = kBf16 ? 8.0f : 5.0f;
    static constexpr float kFall = 7.0f;
    static constexpr float kBias = kBf16 ? 0.0f : 10.0f;
};
// A reference falls only while the row's sum stays below this: a tile that would take
// it further has no weight above 2^-50 of the row's, and O stays far inside 32 bits.
constexpr float kMostSum = 0x1p60f;

template <int D>
struct Shape {
    static constexpr int kParts = D > 128 ? 2 : 1;   // of a head
    static constexpr int kWidth = D / kParts;        // elements a part
    static constexpr int kTileBytes = kTile * kWidth * 2;
    static constexpr int kHalves = kWidth / 64;
    static constexpr int kHalfBytes = kTile * 128;
    // as many tiles as fit beside the two query tiles: five of 32 KB,
    // more in flight than the 54 KB that an SM's share of the measured
    // bandwidth times a memory latency of 1.2 us asks for
    static constexpr int kSlots = kWidth == 128 ? 5 : 10;
    static constexpr int kSmem = (2 + kSlots) * kTileBytes + 1024;
    // half of the 512 columns for each group: S (and P over it), O behind it
    static constexpr uint32_t kGroupColumns = 256;
    static constexpr uint32_t kOut = 128;
};

template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
tree_attention_tc_kernel(const __grid_constant__ TcArgs args,
                         const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map) {
    using S = Shape<D>;
    using R = Reference<kBf16>;
    const ple_tree_attention_args& a = args.a;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t full[S::kSlots], empty[S::kSlots];
    __shared__ __align__(8) uint64_t q_full[2], q_empty, s_full[2], p_low[2], p_high[2], pv_done[2];
    __shared__ __align__(8) uint64_t last;
    // How often a slot was armed for a tile.  A barrier tells only the parity of
    // its phase, and neither copying warp sees every tile of a slot: before it
    // waits for the end of the slot's round r - 1 it waits here for r, which says
    // that all rounds before are over.
    __shared__ uint32_t armed_s[S::kSlots];
    __shared__ int64_t scratch[kThreads / 32];
    __shared__ Share share_s;
    __shared__ uint32_t tmem_s;
    __shared__ int failed_s;
    __shared__ int bad_s[2];          // a segment's drafted values hold infinities or NaN
    __shared__ float join_s[kTile][2];
    // The softmax groups' segments, the one that they work on and the next, and
    // whether there is one.  They read them here where they need them: registers are
    // short, and what they spill goes through the little cache that the ring leaves.
    __shared__ Segment seg_s[2];
    __shared__ int more_s[2];
    __shared__ int64_t end_s[2];      // the place behind the segment
    volatile int* failed = &failed_s;
    volatile uint32_t* armed = armed_s;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* smem = smem_raw + (((smem_addr(smem_raw) + 1023) & ~1023u) - smem_addr(smem_raw));
    uint8_t* q_tiles = smem;
    uint8_t* ring = smem + 2 * S::kTileBytes;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kSlots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            armed_s[i] = 0;
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(&q_full[w], 128);
            mbar_init(&s_full[w], 1);
            mbar_init(&p_low[w], 4);
            mbar_init(&p_high[w], 4);
            mbar_init(&pv_done[w], 1);
            bad_s[w] = 0;
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
    if (warp >= 8) {
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
            // a tile is `boxes` boxes of slots, each in one page
            const int box = page_box(a.page_size);
            const int boxes = kTile / box;
            const int which = lane / S::kHalves, half = lane % S::kHalves;
            const bool mine = which < boxes;
            uint32_t items = 0;
            while (walk.next(args, s)) {
                const int n = s.k1 - s.k0;
                const int32_t* table = a.page_table + (int64_t)s.r * a.max_pages;
                // a box past the tokens, or of a page outside the cache, is filled
                // with zeros: its page number is outside the map
                auto page_of = [&](int j) -> int {
                    const int slot = (s.k0 + j) * kTile + which * box;
                    if (!mine || j >= n || slot >= s.q.length) return (int)a.num_pages;
                    const int p = __ldg(table + (box == a.page_size ? (s.k0 + j) * boxes + which
                                                                    : slot / a.page_size));
                    return p < 0 || p >= a.num_pages ? (int)a.num_pages : p;
                };
                // this warp is some tiles ahead: the queries come to the L2 cache
                // before the groups read them
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
                int page = page_of(0);
                bool ended = false;
                for (int j = 0; j < n && !ended; ++j) {
                    const int after = page_of(j + 1);
#pragma unroll
                    for (int part = 0; part < S::kParts; ++part) {
                        const uint32_t item = items + part +
                                              (keys ? key_item<S::kParts>(j)
                                                    : value_item<S::kParts>(j, n));
                        const uint32_t slot = item % S::kSlots, round = item / S::kSlots;
                        count_wait(&armed[slot], round, failed);
                        if (!mbar_wait(&empty[slot], (round & 1) ^ 1, failed) ||
                            __any_sync(0xffffffffu, *failed)) {
                            ended = true;
                            break;
                        }
                        if (lane == 0) {
                            mbar_arrive_expect(&full[slot], S::kTileBytes);
                            armed[slot] = round + 1;
                        }
                        __syncwarp();
                        if (mine)
                            copy_box(map,
                                     smem_addr(ring) + slot * S::kTileBytes +
                                         half * S::kHalfBytes + which * box * 128,
                                     &full[slot], part * S::kWidth + half * 64,
                                     box == a.page_size
                                         ? 0
                                         : ((s.k0 + j) * kTile + which * box) % a.page_size,
                                     s.head, page);
                    }
                    page = after;
                }
                items += 2 * S::kParts * n;
            }
            if (*failed) {
                // copies may be in flight: they end before the block does
                for (int i = 0; i < S::kSlots; ++i) {
                    const uint32_t rounds = armed[i];
                    const long long start = clock64();
                    while (rounds != 0 && !mbar_try(&full[i], (rounds - 1) & 1) &&
                           clock64() - start < kWaitClocks) {
                    }
                }
                __syncwarp();
            }
        } else if (warp == kIssueWarp) {
            // -------------------------------------------- matrix instructions
            // one lane issues for both groups (tcgen05 work of one thread stays
            // in order: a group's next scores follow the product that reads its
            // weights).  A second issuing warp, one a group, measured slower: the
            // two groups' instructions then interleave one by one (256 rows over
            // 32 x 16384 slots, measured before the weights came in halves: 515 us
            // with one, 597 with two)
            constexpr uint32_t kScoreWord = mma_word(kBf16, false, kTile, kTile);
            constexpr uint32_t kOutWord = mma_word(kBf16, true, kTile, S::kWidth);
            const bool elected = elect_lane();
            const uint32_t ring_at = smem_addr(ring), q_at = smem_addr(q_tiles);
            uint32_t items = 0, p_count[2] = {0, 0}, pairs = 0, seg = 0;
            auto wait_item = [&](uint32_t item) -> uint32_t {
                const uint32_t slot = item % S::kSlots;
                mbar_wait(&full[slot], item / S::kSlots & 1, failed);
                return slot;
            };
            // a descriptor's address counts 16 bytes and stays below 2^14, so
            // steps within a tile add to it
            // (the first keys' part in `slot`, a second one in `slot2`)
            auto scores = [&](int w, uint32_t slot, uint32_t slot2, uint32_t q_tile, bool free) {
                if (elected) {
#pragma unroll
                    for (int part = 0; part < S::kParts; ++part) {
                        const uint64_t qd =
                            operand_desc(q_at + (q_tile + part) * S::kTileBytes, 16);
                        const uint64_t kd =
                            operand_desc(ring_at + (part ? slot2 : slot) * S::kTileBytes, 16);
#pragma unroll
                        for (int k = 0; k < S::kWidth / 16; ++k) {
                            const uint32_t at = ((k / 4) * S::kHalfBytes + (k % 4) * 32) >> 4;
                            mma_smem(tmem + w * S::kGroupColumns, qd + at, kd + at, kScoreWord,
                                     part != 0 || k != 0);
                        }
                    }
                    mma_commit(&s_full[w]);
                    if (free) {
                        mma_commit(&empty[slot]);
                        if (S::kParts == 2) mma_commit(&empty[slot2]);
                    }
                }
                __syncwarp();
            };
            // the product of half a tile's weights
            auto values = [&](int w, uint32_t slot, int half, bool accumulate, bool free) {
                const uint64_t vd = operand_desc(
                    ring_at + slot * S::kTileBytes + half * (kTile / 2) * 128, S::kHalfBytes);
                if (elected) {
#pragma unroll
                    for (int k = 0; k < kTile / 32; ++k)
                        mma_tmem(tmem + w * S::kGroupColumns + S::kOut,
                                 tmem + w * S::kGroupColumns + half * (kTile / 4) + k * 8,
                                 vd + (k * 16 * 128 >> 4), kOutWord, accumulate || k != 0);
                    if (half == 1) mma_commit(&pv_done[w]);
                    if (free) mma_commit(&empty[slot]);
                }
                __syncwarp();
            };
            // both halves, each behind its weights: the first runs while the second's
            // weights are computed
            auto product = [&](int w, uint32_t slot, bool accumulate, bool free) -> bool {
                const uint32_t parity = p_count[w]++ & 1;
                if (!mbar_wait(&p_low[w], parity, failed)) return false;
                tmem_fence_after();
                values(w, slot, 0, accumulate, false);
                if (!mbar_wait(&p_high[w], parity, failed)) return false;
                tmem_fence_after();
                values(w, slot, 1, true, free);
                return true;
            };
            while (walk.next(args, s)) {
                const int n = s.k1 - s.k0;
                // Values past the request's tokens, and drafted ones that are not
                // finite, are cleared before the product reads them.  Eight pieces a
                // lane are looked at together: one by one, behind each other's
                // stores, a tile took some 5000 clocks and was what long drafts waited
                // for (512 nodes for each of 8 requests over 512 slots: 187 us, 126 with
                // this and the masks' words fetched ahead; 142 behind other calls' memory)
                auto clean = [&](int j, uint32_t slot) {
                    const int first = (s.k0 + j) * kTile;
                    if (first + kTile <= s.q.ctx) return;
                    const int from = max(s.q.ctx - first, 0), upto = min(s.q.length - first, kTile);
                    // an exponent of ones carries into its element's sign bit
                    constexpr uint32_t kExp = kBf16 ? 0x7F807F80u : 0x7C007C00u;
                    constexpr uint32_t kOne = kBf16 ? 0x00800080u : 0x04000400u;
                    auto flags = [](uint32_t x) { return ((x & kExp) + kOne) & 0x80008000u; };
                    bool bad = false;
#pragma unroll
                    for (int h = 0; h < S::kHalves; ++h) {
                        uint4* tile = reinterpret_cast<uint4*>(ring + slot * S::kTileBytes +
                                                               h * S::kHalfBytes);
                        constexpr int kAhead = 8;
                        for (int i = from * 8 + lane; i < upto * 8; i += 32 * kAhead) {
                            uint4 v[kAhead];
                            uint32_t any = 0;
#pragma unroll
                            for (int k = 0; k < kAhead; ++k)
                                v[k] = i + 32 * k < upto * 8 ? tile[i + 32 * k]
                                                             : make_uint4(0, 0, 0, 0);
#pragma unroll
                            for (int k = 0; k < kAhead; ++k)
                                any |= flags(v[k].x) | flags(v[k].y) | flags(v[k].z) |
                                       flags(v[k].w);
                            if (any == 0) continue;
                            bad = true;
#pragma unroll
                            for (int k = 0; k < kAhead; ++k) {
                                auto cleared = [&](uint32_t x) {
                                    return x & ~((flags(x) >> 15) * 0xFFFFu);
                                };
                                if (i + 32 * k < upto * 8)
                                    tile[i + 32 * k] = make_uint4(cleared(v[k].x), cleared(v[k].y),
                                                                  cleared(v[k].z), cleared(v[k].w));
                            }
                        }
                        for (int i = max(upto, 0) * 8 + lane; i < kTile * 8; i += 32)
                            tile[i] = make_uint4(0, 0, 0, 0);
                    }
                    if (bad) bad_s[seg & 1] = 1;
                    __threadfence_block();
                    fence_async_proxy();
                    __syncwarp();
                };

                mbar_wait(&q_full[0], seg & 1, failed);
                if (s.pair) mbar_wait(&q_full[1], pairs++ & 1, failed);
                tmem_fence_after();
                if (S::kParts == 2) {
                    uint32_t k = wait_item(items), k2 = wait_item(items + 1);
                    scores(0, k, k2, 0, false);
                    scores(1, k, k2, 0, true);
                    for (int j = 0; j < n; ++j) {
                        const bool more = j + 1 < n;
                        const uint32_t at = items + value_item<S::kParts>(j, n);
                        const uint32_t v = wait_item(at), v2 = wait_item(at + 1);
                        clean(j, v);
                        clean(j, v2);
                        if (!product(0, v, j > 0, true)) break;
                        if (more) {
                            const uint32_t next = items + key_item<S::kParts>(j + 1);
                            k = wait_item(next);
                            k2 = wait_item(next + 1);
                            scores(0, k, k2, 0, false);
                        }
                        if (!product(1, v2, j > 0, true)) break;
                        if (more) scores(1, k, k2, 0, true);
                    }
                } else if (s.pair) {
                    uint32_t k = wait_item(items);
                    scores(0, k, 0, 0, false);
                    scores(1, k, 0, 1, true);
                    for (int j = 0; j < n; ++j) {
                        const bool more = j + 1 < n;
                        // the next keys were copied before these values: both are
                        // at hand before the weights are
                        const uint32_t v = wait_item(items + value_item<S::kParts>(j, n));
                        if (more) k = wait_item(items + key_item<S::kParts>(j + 1));
                        clean(j, v);
                        if (!product(0, v, j > 0, false)) break;
                        if (more) scores(0, k, 0, 0, false);
                        if (!product(1, v, j > 0, true)) break;
                        if (more) scores(1, k, 0, 1, true);
                    }
                } else {
                    for (int w = 0; w < min(2, n); ++w)
                        scores(w, wait_item(items + key_item<S::kParts>(w)), 0, 0, true);
                    for (int j = 0; j < n; ++j) {
                        const int w = j & 1;
                        const uint32_t v = wait_item(items + value_item<S::kParts>(j, n));
                        clean(j, v);
                        if (!product(w, v, j > 1, true)) break;
                        if (j + 2 < n)
                            scores(w, wait_item(items + key_item<S::kParts>(j + 2)), 0, 0, true);
                    }
                }
                if (elected) mma_commit(&q_empty);
                __syncwarp();
                items += 2 * S::kParts * n;
                ++seg;
            }
            // everything issued is done before the block ends, also after a failure
            if (elected) mma_commit(&last);
            __syncwarp();
            const long long start = clock64();
            while (!mbar_try(&last, 0) && clock64() - start < kWaitClocks) {
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------- softmax
        const int w = warp >> 2;
        const int row = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + w * S::kGroupColumns + lanes;
        const uint32_t o_at = s_at + S::kOut;
        const float c = args.c;
        uint32_t seg = 0, count = 0;
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
            const bool active = (warp & 3) * 32 < rows;   // a warp with no row only keeps step
            const bool here = row < rows;
            const int node = (first_row + row) / group;
            const int64_t token = s.q.begin + node;
            const int64_t head = (int64_t)s.head * group + (first_row + row) - node * group;
            const unsigned long long* mask =
                reinterpret_cast<const unsigned long long*>(a.tree_mask) +
                (here ? token : 0) * a.mask_words;
            // asked for long before the tiles that need it
            const uint64_t mask_word = here ? __ldg(mask) : 0;

            // this group's queries, rows of the unit, into swizzled shared memory, or
            // its part of all of them
            if (s.pair || w == 0) {
                if (seg > 0) mbar_wait(&q_empty, (seg - 1) & 1, failed);
                if (w == 0 && row == 0) bad_s[seg & 1] = 0;
                uint8_t* tile = q_tiles + (s.pair ? w : 0) * S::kTileBytes;
                // 16-byte pieces copied without a register, all in flight at once
                constexpr int kPer = S::kWidth / 8;
                const int ch = row % kPer;
                const uint32_t to = smem_addr(tile) + (ch / 8) * S::kHalfBytes;
                const unsigned short* from =
                    static_cast<const unsigned short*>(a.q) + column0 + ch * 8;
#pragma unroll 4
                for (int r = row / kPer; r < rows; r += 128 / kPer) {
                    const uint32_t dst = to + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
                    if (column0 + ch * 8 < a.head_dim)
                        copy16(dst, from + query_row(args, s, first_row + r));
                    else  // columns past a narrower head's
                        zero16(dst);
                }
                copy16_wait();
                if (args.flip != 0) {
                    for (int r = row / kPer; r < rows; r += 128 / kPer) {
                        uint4* at = reinterpret_cast<uint4*>(tile + (ch / 8) * S::kHalfBytes +
                                                             r * 128 + (((ch & 7) ^ (r & 7)) << 4));
                        const uint4 x = *at;
                        *at = make_uint4(x.x ^ args.flip, x.y ^ args.flip, x.z ^ args.flip,
                                         x.w ^ args.flip);
                    }
                }
                fence_async_proxy();
                mbar_arrive(&q_full[w]);
            }

            float top = -INFINITY, sum = 0.f;
            const int step = s.pair ? 1 : 2;
            bool begun = false;
            for (int j = s.pair ? 0 : w; j < n; j += step) {
                const int first = (s.k0 + j) * kTile;
                const bool masked = first + kTile > s.q.ctx;
                MaskWindow window;
                if (masked && here)
                    window = mask_window(mask, mask_word, a.mask_words, s.q.ctx, first);
                if (!mbar_wait(&s_full[w], count & 1, failed)) break;
                tmem_fence_after();
                if (active) {
                    // The row's scores are walked twice, 64 columns at a time: the
                    // upper half and then the lower for the maximum, the lower, still in
                    // registers, and the upper again for the weights.  All 128 would
                    // not leave registers for the rest.
                    uint32_t bits[4];
                    if (masked) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            bits[q] = here ? seen_bits(window, a.mask_words, s.q.ctx, s.q.length,
                                                       first + 32 * q)
                                           : 0u;
                        __syncwarp();
                    }
                    auto hide = [&](uint32_t (&x)[32], int q) {
                        if (masked) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(bits[q] >> i & 1)) x[i] = 0xFF800000u;  // -infinity
                        }
                    };
                    uint32_t v[2][32];
                    float m = -INFINITY;
#pragma unroll
                    for (int h = 1; h >= 0; --h) {
                        float m0, m1;
                        tmem_load_max(s_at + 64 * h, v[0], m0);
                        tmem_load_max(s_at + 64 * h + 32, v[1], m1);
                        tmem_wait_load(v[0]);
                        tmem_settle(v[0], m0);
                        tmem_settle(v[1], m1);
                        if (masked) {
                            hide(v[0], 2 * h);
                            hide(v[1], 2 * h + 1);
                            m0 = m1 = -INFINITY;
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                m0 = max3(m0, as_float(v[0][i]), as_float(v[0][i + 1]));
                                m1 = max3(m1, as_float(v[1][i]), as_float(v[1][i + 1]));
                            }
                        }
                        m = max3(m, m0, m1);
                    }
                    // a new reference only where the tile's maximum is far from it
                    const bool grow = here && (m - top) * c > R::kRise;
                    const bool set = here && top == -INFINITY && m > -INFINITY;
                    bool move = grow || set;
                    if constexpr (!kBf16) {
                        const float fall = (top - m) * c;
                        move |= here && fall > R::kFall && sum * exp2_fast(fall) < kMostSum;
                    }
                    if (__any_sync(0xffffffffu, move)) {
                        const float f = move ? (set ? 0.f : exp2_fast((top - m) * c)) : 1.f;
                        if (move) top = m;
                        sum *= f;
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
                    // rows that have seen nothing yet have only -infinities:
                    // exponents relative to 0 make zeros of them
                    const float shift = top == -INFINITY ? 0.f : fmaf(top, c, -R::kBias);
                    const uint64_t c2 = pack_f32(c, c), shift2 = pack_f32(-shift, -shift);
                    uint64_t part[2] = {0, 0};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t(&x)[32] = v[q & 1];
                        if (q > 1) {
                            tmem_wait_load(x);
                            hide(x, q);
                        }
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float x0, x1;
                            const uint64_t two =
                                pack_f32(as_float(x[2 * i]), as_float(x[2 * i + 1]));
                            unpack_f32(fma_f32x2(two, c2, shift2), x0, x1);
                            x0 = exp2_fast(x0);
                            x1 = exp2_fast(x1);
                            part[i & 1] = add_f32x2(part[i & 1], pack_f32(x0, x1));
                            p[i] = round_pair<kBf16>(x0, x1);
                        }
                        if (q < 2) tmem_load(s_at + 32 * (q + 2), x);
                        // over columns whose scores have been read
                        tmem_store(s_at + 16 * q, p);
                        if (q == 1) {
                            tmem_wait_store();
                            tmem_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&p_low[w]);
                        }
                    }
                    float p0, p1;
                    unpack_f32(add_f32x2(part[0], part[1]), p0, p1);
                    sum += p0 + p1;
                    tmem_wait_store();
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (!active) mbar_arrive(&p_low[w]);
                    mbar_arrive(&p_high[w]);
                }
                begun = true;
                ++count;
            }
            if (begun) mbar_wait(&pv_done[w], (count - 1) & 1, failed);
            tmem_fence_after();

            // ------------------------------------ the segment's rows go out
            const bool join = !s.pair && n > 1;   // both groups hold states of the same rows
            float4* exchange = reinterpret_cast<float4*>(q_tiles);
            if (join && w == 1) {
                mbar_wait(&q_empty, seg & 1, failed);   // the queries have been read
                if (active) {
#pragma unroll 1
                    for (int q = 0; q < S::kWidth / 32; ++q) {
                        uint32_t o[32];
                        tmem_load(o_at + 32 * q, o);
                        tmem_wait_load(o);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            exchange[(q * 8 + i) * kTile + row] = make_float4(
                                __uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                    }
                    join_s[row][0] = top;
                    join_s[row][1] = sum;
                }
            }
            if (join) named_barrier<256>(1);
            if (s.pair || w == 0) {
                float f0 = 1.f, f1 = 0.f;
                if (join && here) {
                    const float other = join_s[row][0];
                    const float m = fmaxf(top, other);
                    const float base = m == -INFINITY ? 0.f : m;
                    f0 = exp2_fast((top - base) * c);
                    f1 = exp2_fast((other - base) * c);
                    if (top == -INFINITY) f0 = 0.f;
                    if (other == -INFINITY) f1 = 0.f;
                    sum = sum * f0 + join_s[row][1] * f1;
                    top = m;
                }
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
                const bool bad = bad_s[seg & 1] != 0;
                const int64_t o_row = token * a.q_heads + head;
                float* state = static_cast<float*>(a.workspace) +
                               state_at(blockIdx.x, s.k0 == 0 ? 1 : 0, args.rows_cap, D);
                const int state_row = row0 + row;
                float* pairs = state + 2 * state_row;
                float* acc = state + (2 + column0) * args.rows_cap + 8 * state_row;
                const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
                if (active) {
#pragma unroll 1
                    for (int q = 0; q < S::kWidth / 32; ++q) {
                        const int column = column0 + 32 * q;
                        uint32_t o[32];
                        if (begun) {
                            tmem_load(o_at + 32 * q, o);
                            tmem_wait_load(o);
                        }
                        float x[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(o[i]);
                        if (kSplit && spoiled) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = __int_as_float(0x7FC00000);
                        }
                        if (join) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float4 y = exchange[(q * 8 + i) * kTile + row];
                                x[4 * i] = x[4 * i] * f0 + y.x * f1;
                                x[4 * i + 1] = x[4 * i + 1] * f0 + y.y * f1;
                                x[4 * i + 2] = x[4 * i + 2] * f0 + y.z * f1;
                                x[4 * i + 3] = x[4 * i + 3] * f0 + y.w * f1;
                            }
                        }
                        if (bad && here) {
                            // the drafted values that were cleared, to the rows
                            // that see them: infinities and NaN
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
                                const unsigned short* vrow =
                                    static_cast<const unsigned short*>(a.v_cache) + at +
                                    s.head * a.head_stride + column;
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    if (column + i >= a.head_dim) break;
                                    const float e = widen16<kBf16>(vrow[i]);
                                    if (!isfinite(e)) x[i] += e;
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
                    if (here && column0 == 0) {
                        if (!whole) {
                            pairs[0] = fmaf(top, c, -R::kBias);
                            pairs[1] = sum;
                        } else if (a.lse != nullptr) {
                            a.lse[o_row] = sum == 0.f
                                               ? -INFINITY
                                               : fmaf(top, c, -R::kBias) * 0.69314718055994531f +
                                                     logf(sum);
                        }
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

// A cache as a map of (element, slot, head, page); boxes of 64 elements by the
// slots of page_box.  Pages outside read as zeros, and so do elements past a head
// narrower than the tile.
bool encode_cache(CUtensorMap* map, const ple_tree_attention_args& a, const void* cache) {
    const EncodeTiled fn = encode_tiled();
    if (fn == nullptr) return false;
    auto stride = [](int64_t elements, int64_t n) {
        return (cuuint64_t)(n == 1 ? 16 : elements * 2);
    };
    const cuuint64_t sizes[4] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.page_size,
                                 (cuuint64_t)a.kv_heads, (cuuint64_t)a.num_pages};
    const cuuint64_t strides[3] = {stride(a.slot_stride, a.page_size),
                                   stride(a.head_stride, a.kv_heads),
                                   stride(a.page_stride, a.num_pages)};
    const cuuint32_t box[4] = {64, (cuuint32_t)page_box(a.page_size), 1, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return fn(map,
              a.dtype == PLE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                  : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
              4, const_cast<void*>(cache), sizes, strides, box, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kBf16>
cudaError_t launch_tc(const TcArgs& args, const CUtensorMap& k, const CUtensorMap& v,
                      cudaStream_t stream) {
    auto* fn = tree_attention_tc_kernel<D, kBf16>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Shape<D>::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_kernel(fn, dim3((unsigned)args.blocks), dim3(kThreads), Shape<D>::kSmem, stream,
                      programmatic_launch(), args, k, v);
    if (e != cudaSuccess) return e;
    return launch_kernel(
        tree_attention_join_kernel<D, kBf16>,
        dim3((unsigned)args.blocks, (unsigned)((args.rows_cap + kJoinRows - 1) / kJoinRows)),
        dim3(kJoinThreads), 0, stream, programmatic_launch(), args);
}

}  // namespace

int64_t tree_attention_tc_workspace(int64_t T, int32_t q_heads, int32_t kv_heads, int32_t D,
                                    const DeviceFacts& dev) {
    return 4 * state_at(tc_blocks(dev), 0, tc_rows_cap(T, q_heads, kv_heads, D), padded_width(D));
}

// Pages that boxes of whole swizzle atoms (8 slots) cut evenly, and tiles whose
// ends stay within 31 bits.
bool tree_attention_tc_fits(const ple_tree_attention_args& a) {
    return a.page_size % 8 == 0 && (int64_t)a.max_pages * a.page_size <= INT32_MAX - kTile;
}

// *taken: whether the tensor maps take the caches' strides (else nothing ran).
cudaError_t launch_tree_attention_tc(const ple_tree_attention_args& a, const DeviceFacts& dev,
                                     cudaStream_t stream, bool* taken) {
    CUtensorMap k, v;
    *taken = encode_cache(&k, a, a.k_cache) && encode_cache(&v, a, a.v_cache);
    if (!*taken) return cudaSuccess;
    TcArgs args;
    args.a = a;
    args.blocks = tc_blocks(dev);
    args.group = a.q_heads / a.kv_heads;
    args.rows_cap = tc_rows_cap(a.num_tokens, a.q_heads, a.kv_heads, a.head_dim);
    args.unit_rows = unit_rows(padded_width(a.head_dim));
    // a scale of 0 as the least normal number: every exponent still rounds to 0,
    // and a hidden score stays -infinity
    args.c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1.17549435e-38f);
    args.flip = a.scale < 0 ? 0x80008000u : 0u;
    const bool bf16 = a.dtype == PLE_BF16;
    switch (padded_width(a.head_dim)) {
        case 64:
            return bf16 ? launch_tc<64, true>(args, k, v, stream)
                        : launch_tc<64, false>(args, k, v, stream);
        case 128:
            return bf16 ? launch_tc<128, true>(args, k, v, stream)
                        : launch_tc<128, false>(args, k, v, stream);
        default:
            return bf16 ? launch_tc<256, true>(args, k, v, stream)
                        : launch_tc<256, false>(args, k, v, stream);
    }
}

}  // namespace ple
