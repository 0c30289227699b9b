// Tensor-core and asynchronous-copy primitives of sm_103a used by this
// library's kernels: mbarriers with bounded waits, tiled bulk copies, and the
// fifth-generation matrix instructions with their tensor memory.
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace ple {
namespace {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count));
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// About a second: far beyond any wait inside one block, and an end to a wait
// that a mistake would make endless.
constexpr long long kWaitClocks = 2000000000ll;

// A whole warp waits for the phase of the given parity.  Where it does not come
// within kWaitClocks the block's `failed` is set and every later wait of the
// block that is not met at once returns false, to all lanes.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, volatile int* failed) {
    if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
    const long long start = clock64();
    bool over = false;
    while (!mbar_try(bar, parity) && !over) {
        if (clock64() - start > kWaitClocks) *failed = 1;
        over = *failed != 0;
    }
    return !__any_sync(0xffffffffu, over);
}

// The same for one lane.
__device__ __forceinline__ bool lane_wait(uint64_t* bar, uint32_t parity, volatile int* failed) {
    if (mbar_try(bar, parity)) return true;
    const long long start = clock64();
    while (!mbar_try(bar, parity)) {
        if (clock64() - start > kWaitClocks) *failed = 1;
        if (*failed) return false;
    }
    return true;
}

// A whole warp waits until *count has come to `least`, as mbar_wait does.
__device__ __forceinline__ void count_wait(const volatile uint32_t* count, uint32_t least,
                                           volatile int* failed) {
    if ((int32_t)(*count - least) < 0) {
        const long long start = clock64();
        while ((int32_t)(*count - least) < 0 && !*failed) {
            if (clock64() - start > kWaitClocks) *failed = 1;
        }
    }
    __syncwarp();
}

__device__ __forceinline__ void fence_barrier_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// Plain writes to shared memory before it become visible to copies and matrix
// instructions after it.
__device__ __forceinline__ void fence_async_proxy() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// One lane of a whole warp, the same one every time, known as one to the
// compiler (so operands of single-thread instructions stay uniform).
__device__ __forceinline__ bool elect_lane() {
    uint32_t chosen;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(chosen));
    return chosen != 0;
}

// A warpgroup's registers a thread, fewer or more than at launch: the sum over the
// block's warpgroups may not pass what it was launched with.
template <int kCount>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCount));
}
template <int kCount>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kCount));
}

template <int kThreads>
__device__ __forceinline__ void named_barrier(int id) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kThreads) : "memory");
}

// One box of a four-dimensional tensor map into shared memory.
__device__ __forceinline__ void copy_box(const CUtensorMap* map, uint32_t dst, uint64_t* bar, int x,
                                         int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// Sixteen bytes to shared memory behind the thread's back, and all of them there.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void zero16(uint32_t dst) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
}
__device__ __forceinline__ void copy16_wait() {
    asm volatile("cp.async.wait_all;" ::: "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Tensor memory of a whole SM, allocated and freed by one warp.
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(where)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}

__device__ __forceinline__ void tmem_wait_store() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tmem_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Thirty-two accumulator columns of a lane's row, and their writing back.  The
// loaded registers may be used only behind tmem_wait_load on them.
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&v)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
                 "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
                 "%29, %30, %31}, [%32];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                   "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]),
                   "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]),
                   "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
                   "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]),
                   "=r"(v[30]), "=r"(v[31])
                 : "r"(at));
}

// The same with the largest of the row's thirty-two (NaN aside) beside them.
__device__ __forceinline__ void tmem_load_max(uint32_t at, uint32_t (&v)[32], float& most) {
    asm volatile("tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
                 "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
                 "%29, %30, %31}, %32, [%33];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                   "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]),
                   "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
                   "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]),
                   "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]),
                   "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]),
                   "=f"(most)
                 : "r"(at));
}

// Sixteen columns with their largest, into v[at..at + 15].
__device__ __forceinline__ void tmem_load_max16(uint32_t from, uint32_t (&v)[32], const int at,
                                                float& most) {
    asm volatile("tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
                 "%15}, %16, [%17];"
                 : "=r"(v[at]), "=r"(v[at + 1]), "=r"(v[at + 2]), "=r"(v[at + 3]),
                   "=r"(v[at + 4]), "=r"(v[at + 5]), "=r"(v[at + 6]), "=r"(v[at + 7]),
                   "=r"(v[at + 8]), "=r"(v[at + 9]), "=r"(v[at + 10]), "=r"(v[at + 11]),
                   "=r"(v[at + 12]), "=r"(v[at + 13]), "=r"(v[at + 14]), "=r"(v[at + 15]),
                   "=f"(most)
                 : "r"(from));
}

// What was loaded before a tmem_wait_load of something later.
__device__ __forceinline__ void tmem_settle(uint32_t (&v)[32], float& most) {
    asm volatile(""
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                   "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                   "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]),
                   "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                   "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]),
                   "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31]),
                   "+f"(most));
}

__device__ __forceinline__ void tmem_wait_load(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                   "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                   "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]),
                   "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                   "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&v)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
                 "%30, %31, %32};"
                 :
                 : "r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
                   "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]),
                   "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
                   "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
                   "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]),
                   "r"(v[31])
                 : "memory");
}

__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16};"
                 :
                 : "r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
                   "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
                   "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}

// A shared-memory operand in the 128-byte swizzled layout: 8 rows of 128 bytes
// make an atom of 1024, atoms of consecutive rows follow each other (stride
// offset 1024).  lead: bytes from one block of 64 elements to the next along
// the rows, read for operands whose rows are the reduction (else unused).
__device__ __forceinline__ uint64_t operand_desc(uint32_t at, uint32_t lead) {
    return (uint64_t)((at >> 4) & 0x3FFF) | (uint64_t)((lead >> 4) & 0x3FFF) << 16 |
           (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Descriptors as a low word, to which steps add, and a constant high one.  Of a tile of
// halves whose rows are the reduction (as operand_desc), and of a tile of 8-bit elements
// whose rows are the swizzle's span: atoms of 8 rows, kAtom bytes (1024 with the 128-byte
// swizzle, 512 with that of 64).
__device__ __forceinline__ uint32_t half_desc_low(uint32_t at, uint32_t lead) {
    return ((at >> 4) & 0x3FFF) | ((lead >> 4) & 0x3FFF) << 16;
}
__host__ __device__ constexpr uint32_t half_desc_high() { return 1024 >> 4 | 1u << 14 | 2u << 29; }
__device__ __forceinline__ uint32_t element_desc_low(uint32_t at) {
    return ((at >> 4) & 0x3FFF) | 1u << 16;
}
template <uint32_t kAtom>
__host__ __device__ constexpr uint32_t element_desc_high() {
    static_assert(kAtom == 1024 || kAtom == 512, "");
    return kAtom >> 4 | 1u << 14 | (kAtom == 1024 ? 2u : 4u) << 29;
}

// The instruction word of kind::f16: 32-bit accumulator, both operands f16 or
// both bf16, A with the reduction along its rows; kAcross: B's rows are the
// reduction.
__host__ __device__ constexpr uint32_t mma_word(bool bf16, bool across, int m, int n) {
    return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (across ? 1u << 16 : 0u) |
           (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

__device__ __forceinline__ void mma_smem(uint32_t d, uint64_t a, uint64_t b, uint32_t word,
                                         bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(word), "r"((uint32_t)accumulate)
        : "memory");
}

// The same as mma_smem with A in tensor memory, two elements to a column.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t word,
                                         bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(word), "r"((uint32_t)accumulate)
        : "memory");
}

// With descriptors in words.  8-bit elements (kind::f8f6f4; both e4m3 with the word of
// f16), 32 a step, and A of halves in tensor memory.
template <uint32_t kWord, uint32_t kHigh>
__device__ __forceinline__ void mma_elements_at(uint32_t d, uint32_t a, uint32_t b,
                                                bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "n"(kWord), "r"((uint32_t)accumulate), "n"(kHigh)
        : "memory");
}
template <uint32_t kWord, uint32_t kHigh>
__device__ __forceinline__ void mma_tmem_at(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "n"(kWord), "r"((uint32_t)accumulate), "n"(kHigh)
        : "memory");
}

// Arrive on a barrier when every matrix instruction this thread issued before
// is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_addr(bar))
        : "memory");
}

}  // namespace
}  // namespace ple
