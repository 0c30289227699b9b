// C ABI of the entry points for caches in 8 bits and for pages (declared in
// include/ple.h): host checks of scalar arguments and pointer values, then the
// launches on the caller's stream.  Nothing is allocated, read back or kept.
#include <stdint.h>

#include <cmath>

#include "ple_checks.h"
#include "ple_tree_fp8_internal.h"

namespace {

bool mult16(int64_t s) { return s % 16 == 0; }

bool dim8_ok(int32_t d) { return d >= 16 && d <= PLE_MAX_HEAD_DIM && d % 16 == 0; }

// Blocks that pages hold a whole number of, and strides that keep every scale's offset in
// 63 bits.
bool scales_ok(const ple_cache_scales& s, int64_t num_pages, int32_t heads, int32_t page_size) {
    if ((s.block != 16 && s.block != 32 && s.block != 64 && s.block != 128) ||
        page_size % s.block != 0 || s.page_stride < 0 || s.head_stride < 0)
        return false;
    const __int128 span = (__int128)(num_pages - 1) * s.page_stride +
                          (__int128)(heads - 1) * s.head_stride + page_size / s.block;
    return span <= INT64_MAX / 8;
}

bool scales_aligned(const ple_cache_scales& s) { return aligned(s.k, 2) && aligned(s.v, 2); }

}  // namespace

extern "C" ple_status ple_qk_norm_rope_fp8(const ple_qk_norm_rope_fp8_args* args, void* stream) {
    if (!args) return PLE_ERR_NULL;
    const ple_qk_norm_rope_args& a = args->base;
    const ple_cache_scales& s = args->scales;
    if (a.num_tokens < 0 || a.num_tokens > INT32_MAX || a.q_heads < 0 || a.q_heads > 65535 ||
        a.kv_heads < 1 || a.kv_heads > 65535 || a.q_heads + a.kv_heads > 65535 ||
        !dim8_ok(a.head_dim) || a.rotary_dim < 0 || a.rotary_dim > a.head_dim ||
        a.rotary_dim % 2 != 0 || !(a.eps >= 0.0f) || !std::isfinite(a.eps) ||
        !std::isfinite(a.rope_scale))
        return PLE_ERR_SIZE;
    if (!dtype_ok(a.dtype)) return PLE_ERR_ELEMENT;
    if (a.num_tokens == 0) return PLE_OK;
    const int64_t T = a.num_tokens;
    if (a.num_requests < 1 || !rows_ok(T, a.q_token, a.q_heads, a.q_head, a.head_dim) ||
        !rows_ok(T, a.q_out_token, a.q_heads, a.q_out_head, a.head_dim) ||
        !rows_ok(T, a.k_token, a.kv_heads, a.k_head, a.head_dim) ||
        !rows_ok(T, a.v_token, a.kv_heads, a.v_head, a.head_dim) ||
        !cache_sizes_ok(a.num_pages, a.page_stride, a.head_stride, a.slot_stride, a.kv_heads,
                        a.page_size, a.max_pages, a.head_dim) ||
        !scales_ok(s, a.num_pages, a.kv_heads, a.page_size))
        return PLE_ERR_SIZE;
    if ((a.q_heads && (!a.q || !a.q_out)) || !a.k || !a.v || !a.k_cache || !a.v_cache || !s.k ||
        !s.v || !a.page_table || !a.ctx_lens || !a.cu_seqlens ||
        (a.rotary_dim && (!a.rope || !a.positions)))
        return PLE_ERR_NULL;
    if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.q_out, 16) ||
        !aligned(a.q_weight, 16) || !aligned(a.k_weight, 16) || !aligned(a.positions, 4) ||
        !aligned(a.rope, 8) || !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) ||
        !aligned(a.page_table, 4) || !aligned(a.ctx_lens, 4) || !aligned(a.cu_seqlens, 4) ||
        !scales_aligned(s) || !mult8(a.q_token) || !mult8(a.q_head) || !mult8(a.k_token) ||
        !mult8(a.k_head) || !mult8(a.v_token) || !mult8(a.v_head) || !mult8(a.q_out_token) ||
        !mult8(a.q_out_head) || !mult16(a.page_stride) || !mult16(a.head_stride) ||
        !mult16(a.slot_stride))
        return PLE_ERR_ALIGN;
    ple::DeviceFacts dev;
    if (ple_status st = with_device(&dev); st != PLE_OK) return st;
    return finish(ple::launch_qk_norm_rope_fp8(*args, dev, static_cast<cudaStream_t>(stream)));
}

extern "C" int64_t ple_tree_attention_fp8_workspace(int64_t num_tokens, int32_t q_heads,
                                                    int32_t kv_heads, int32_t head_dim) {
    if (!attention_heads_ok(num_tokens, q_heads, kv_heads, head_dim) || !dim8_ok(head_dim))
        return -1;
    ple::DeviceFacts dev;
    if (with_device(&dev) != PLE_OK) return -1;
    return ple::tree_attention_fp8_workspace(num_tokens, q_heads, kv_heads, head_dim, dev);
}

extern "C" ple_status ple_tree_attention_fp8(const ple_tree_attention_fp8_args* args,
                                             void* stream) {
    if (!args) return PLE_ERR_NULL;
    const ple_tree_attention_args& a = args->base;
    const ple_cache_scales& s = args->scales;
    if (!attention_heads_ok(a.num_tokens, a.q_heads, a.kv_heads, a.head_dim) ||
        !dim8_ok(a.head_dim) || a.mask_words < 1 || a.mask_words > PLE_MAX_TREE_WORDS ||
        !std::isfinite(a.scale))
        return PLE_ERR_SIZE;
    if (!dtype_ok(a.dtype)) return PLE_ERR_ELEMENT;
    if (a.num_tokens == 0) return PLE_OK;
    // a tile of 128 slots ends within 31 bits; strides of one element and more, as a
    // tensor map wants them
    if (a.num_requests < 1 ||
        !cache_sizes_ok(a.num_pages, a.page_stride, a.head_stride, a.slot_stride, a.kv_heads,
                        a.page_size, a.max_pages, a.head_dim) ||
        (int64_t)a.max_pages * a.page_size > INT32_MAX - 128 ||
        !scales_ok(s, a.num_pages, a.kv_heads, a.page_size) ||
        (a.num_pages > 1 && (a.page_stride < 1 || a.page_stride >> 40)) ||
        (a.kv_heads > 1 && (a.head_stride < 1 || a.head_stride >> 40)) || a.slot_stride < 1 ||
        a.slot_stride >> 40 || !rows_ok(a.num_tokens, a.q_token, a.q_heads, a.q_head, a.head_dim) ||
        a.num_tokens > INT64_MAX / 8 / ((int64_t)a.q_heads * a.head_dim))
        return PLE_ERR_SIZE;
    if (!a.q || !a.k_cache || !a.v_cache || !s.k || !s.v || !a.page_table || !a.ctx_lens ||
        !a.cu_seqlens || !a.tree_mask || !a.out || !a.workspace)
        return PLE_ERR_NULL;
    if (!aligned(a.q, 16) || !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) ||
        !aligned(a.page_table, 4) || !aligned(a.ctx_lens, 4) || !aligned(a.cu_seqlens, 4) ||
        !aligned(a.tree_mask, 8) || !aligned(a.out, 16) || !aligned(a.lse, 4) ||
        !aligned(a.workspace, 16) || !scales_aligned(s) || !mult8(a.q_token) ||
        !mult8(a.q_head) || !mult16(a.page_stride) || !mult16(a.head_stride) ||
        !mult16(a.slot_stride))
        return PLE_ERR_ALIGN;
    ple::DeviceFacts dev;
    if (ple_status st = with_device(&dev); st != PLE_OK) return st;
    if (a.workspace_bytes <
        ple::tree_attention_fp8_workspace(a.num_tokens, a.q_heads, a.kv_heads, a.head_dim, dev))
        return PLE_ERR_SIZE;
    return finish(ple::launch_tree_attention_fp8(*args, dev, static_cast<cudaStream_t>(stream)));
}

extern "C" ple_status ple_tree_commit_fp8(const ple_tree_commit_fp8_args* args, void* stream) {
    if (!args) return PLE_ERR_NULL;
    const ple_tree_commit_args& a = args->base;
    const ple_cache_scales& s = args->scales;
    if (a.num_tokens < 0 || a.num_tokens > INT32_MAX || a.num_requests < 0 || a.path_len < 0 ||
        (a.path_len == 0 && a.path) || a.num_layers < 1 || a.num_layers > 65535 ||
        !dim8_ok(a.head_dim) || a.layer_stride < 0 || s.layer_stride < 0 ||
        !cache_sizes_ok(a.num_pages, a.page_stride, a.head_stride, a.slot_stride, a.kv_heads,
                        a.page_size, a.max_pages, a.head_dim) ||
        !scales_ok(s, a.num_pages, a.kv_heads, a.page_size) ||
        (__int128)(a.num_layers - 1) * a.layer_stride > INT64_MAX / 16 ||
        (__int128)(a.num_layers - 1) * s.layer_stride > INT64_MAX / 16)
        return PLE_ERR_SIZE;
    if (a.ngram_context && (a.ctx_len < 1 || a.ctx_len >= PLE_MAX_NGRAM)) return PLE_ERR_SIZE;
    if (a.ngram_context && a.id_dtype != PLE_I32 && a.id_dtype != PLE_I64) return PLE_ERR_DTYPE;
    if (a.num_requests == 0) return PLE_OK;
    if ((!a.path && a.path_len) || !a.accepted || !a.cu_seqlens || !a.ctx_lens ||
        !a.next_ctx_lens || !a.page_table || !a.k_cache || !a.v_cache || !s.k || !s.v ||
        (a.ngram_context && ((!a.input_ids && a.num_tokens) || !a.next_context)))
        return PLE_ERR_NULL;
    const int id_bytes = a.id_dtype == PLE_I32 ? 4 : 8;
    if (!aligned(a.path, 4) || !aligned(a.accepted, 4) || !aligned(a.cu_seqlens, 4) ||
        !aligned(a.ctx_lens, 4) || !aligned(a.next_ctx_lens, 4) || !aligned(a.page_table, 4) ||
        !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) || !scales_aligned(s) ||
        !mult16(a.layer_stride) || !mult16(a.page_stride) || !mult16(a.head_stride) ||
        !mult16(a.slot_stride) ||
        (a.ngram_context && (!aligned(a.input_ids, id_bytes) ||
                             !aligned(a.ngram_context, id_bytes) ||
                             !aligned(a.next_context, id_bytes))))
        return PLE_ERR_ALIGN;
    if (commit_outputs_overlap(a)) return PLE_ERR_SIZE;
    ple::DeviceFacts dev;
    if (ple_status st = with_device(&dev); st != PLE_OK) return st;
    return finish(ple::launch_tree_commit_fp8(*args, dev, static_cast<cudaStream_t>(stream)));
}

extern "C" int64_t ple_plan_pages_workspace(int32_t num_rows, int32_t num_pages) {
    if (num_rows < 1 || num_pages < 1) return -1;
    return ple::plan_pages_workspace(num_rows, num_pages);
}

extern "C" ple_status ple_plan_pages(const ple_plan_pages_args* args, void* stream) {
    if (!args) return PLE_ERR_NULL;
    const ple_plan_pages_args& a = *args;
    if (a.num_requests < 0 || a.num_rows < 1 || a.max_pages < 1 || a.page_size < 1 ||
        (int64_t)a.max_pages * a.page_size > INT32_MAX || a.num_pages < 1 || a.page_limit < 0 ||
        a.page_limit > a.num_pages ||
        // ranks of new pages are counted in 32 bits
        (int64_t)a.num_rows * a.max_pages > INT32_MAX - a.num_pages ||
        a.workspace_bytes < ple::plan_pages_workspace(a.num_rows, a.num_pages))
        return PLE_ERR_SIZE;
    if ((a.num_requests && (!a.page_table || !a.ctx_lens)) || !a.source || !a.want ||
        !a.next_table || !a.next_ctx_lens || !a.copies || !a.counts || !a.workspace)
        return PLE_ERR_NULL;
    if (!aligned(a.page_table, 4) || !aligned(a.ctx_lens, 4) || !aligned(a.source, 4) ||
        !aligned(a.want, 4) || !aligned(a.next_table, 4) || !aligned(a.next_ctx_lens, 4) ||
        !aligned(a.copies, 4) || !aligned(a.counts, 4) || !aligned(a.workspace, 16))
        return PLE_ERR_ALIGN;
    // rows of the next tables are written while others of the old ones are read
    const __int128 B = a.num_requests, N = a.num_rows, M = a.max_pages;
    const struct {
        const void* at;
        __int128 bytes;
    } out[] = {{a.next_table, 4 * N * M},
               {a.next_ctx_lens, 4 * N},
               {a.copies, 8 * (N + a.num_pages - a.page_limit)},
               {a.counts, 12},
               {a.workspace, ple::plan_pages_workspace(a.num_rows, a.num_pages)}},
      in[] = {{a.page_table, 4 * B * M}, {a.ctx_lens, 4 * B}, {a.source, 4 * N}, {a.want, 4 * N}};
    for (int i = 0; i < 5; ++i) {
        for (const auto& x : in)
            if (overlap(out[i].at, out[i].bytes, x.at, x.bytes)) return PLE_ERR_SIZE;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].at, out[i].bytes, out[j].at, out[j].bytes)) return PLE_ERR_SIZE;
    }
    return finish(ple::launch_plan_pages(a, static_cast<cudaStream_t>(stream)));
}

extern "C" ple_status ple_copy_pages(const ple_copy_pages_args* args, void* stream) {
    if (!args) return PLE_ERR_NULL;
    const ple_copy_pages_args& a = *args;
    const ple_cache_scales& s = a.scales;
    if (a.num_copies < 0 || a.num_layers < 1 || a.num_layers > 65535 || a.layer_stride < 0 ||
        (a.element_bytes != 1 && a.element_bytes != 2) || a.head_dim < 1 ||
        a.head_dim > PLE_MAX_HEAD_DIM || a.head_dim * a.element_bytes % 16 != 0 ||
        !cache_sizes_ok(a.num_pages, a.page_stride, a.head_stride, a.slot_stride, a.kv_heads,
                        a.page_size, 1, a.head_dim) ||
        (__int128)(a.num_layers - 1) * a.layer_stride > INT64_MAX / 16 ||
        !ple::copy_page_ok(a) || (!s.k != !s.v))
        return PLE_ERR_SIZE;
    if (s.k && (a.element_bytes != 1 || s.layer_stride < 0 ||
                !scales_ok(s, a.num_pages, a.kv_heads, a.page_size) ||
                (__int128)(a.num_layers - 1) * s.layer_stride > INT64_MAX / 16))
        return PLE_ERR_SIZE;
    if (a.num_copies == 0) return PLE_OK;
    if (!a.copies || !a.k_cache || !a.v_cache) return PLE_ERR_NULL;
    const int64_t whole = 16 / a.element_bytes;
    if (!aligned(a.copies, 8) || !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) ||
        a.layer_stride % whole || a.page_stride % whole || a.head_stride % whole ||
        a.slot_stride % whole || !scales_aligned(s))
        return PLE_ERR_ALIGN;
    ple::DeviceFacts dev;
    if (ple_status st = with_device(&dev); st != PLE_OK) return st;
    return finish(ple::launch_copy_pages(a, dev, static_cast<cudaStream_t>(stream)));
}
