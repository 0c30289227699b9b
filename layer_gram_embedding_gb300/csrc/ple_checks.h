// Host checks that the entry points share.
#pragma once

#include <stdint.h>

#include "ple_tree_internal.h"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
inline bool mult8(int64_t s) { return s % 8 == 0; }

inline ple_status finish(cudaError_t e) {
    return e == cudaSuccess ? PLE_OK : (ple_status)ple::record_cuda_failure(e);
}

inline ple_status with_device(ple::DeviceFacts* dev) { return finish(ple::device_facts(dev)); }

inline bool head_dim_ok(int32_t d) { return d >= 8 && d <= PLE_MAX_HEAD_DIM && d % 8 == 0; }
inline bool dtype_ok(int32_t t) { return t == PLE_BF16 || t == PLE_F16; }

// A paged cache's geometry: sizes that keep every element offset in 63 bits.
inline bool cache_sizes_ok(int64_t num_pages, int64_t page_stride, int64_t head_stride,
                           int64_t slot_stride, int32_t heads, int32_t page_size,
                           int32_t max_pages, int32_t head_dim) {
    if (num_pages < 1 || num_pages > INT32_MAX || page_size < 1 || max_pages < 1 || heads < 1 ||
        heads > 65535)
        return false;
    if (page_stride < 0 || head_stride < 0 || slot_stride < 0) return false;
    const __int128 span = (__int128)(num_pages - 1) * page_stride +
                          (__int128)(heads - 1) * head_stride +
                          (__int128)(page_size - 1) * slot_stride + head_dim;
    return span <= INT64_MAX / 8 && (int64_t)max_pages * page_size <= INT32_MAX;
}

// Whether [a, a + n) and [b, b + m), in bytes, share one.
inline bool overlap(const void* a, __int128 n, const void* b, __int128 m) {
    const __int128 x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && n > 0 && m > 0 && x < y + m && y < x + n;
}

inline bool rows_ok(int64_t T, int64_t token, int32_t heads, int64_t head, int32_t dim) {
    if (token < 0 || head < 0) return false;
    return heads == 0 || (__int128)(T - 1) * token + (__int128)(heads - 1) * head + dim <=
                             INT64_MAX / 8;
}

inline bool attention_heads_ok(int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    return T >= 0 && T <= INT32_MAX && kv_heads >= 1 && q_heads >= 1 && q_heads <= 65535 &&
           q_heads % kv_heads == 0 && head_dim_ok(head_dim);
}

inline bool commit_outputs_overlap(const ple_tree_commit_args& a) {
    // a request's blocks, one a layer and cache, run in any order: what one of them
    // writes for the next step may be nothing that another still reads
    const int id_bytes = a.id_dtype == PLE_I32 ? 4 : 8;
    const __int128 B = a.num_requests;
    const __int128 context = a.ngram_context ? B * a.ctx_len * id_bytes : 0;
    const struct {
        const void* at;
        __int128 bytes;
    } out[] = {{a.next_ctx_lens, 4 * B}, {a.next_context, context}},
      in[] = {{a.input_ids, context ? (__int128)a.num_tokens * id_bytes : 0},
              {a.path, 4 * B * a.path_len},
              {a.accepted, 4 * B},
              {a.cu_seqlens, 4 * (B + 1)},
              {a.ngram_context, context},
              {a.ctx_lens, 4 * B},
              {a.page_table, 4 * B * a.max_pages}};
    if (overlap(out[0].at, out[0].bytes, out[1].at, out[1].bytes)) return true;
    for (const auto& o : out)
        for (const auto& i : in)
            if (overlap(o.at, o.bytes, i.at, i.bytes)) return true;
    return false;
}

}  // namespace
