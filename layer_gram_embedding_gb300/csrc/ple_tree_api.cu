// C ABI of the tree-verification entry points (declared in include/ple.h):
// host checks of scalar arguments and pointer values, then the launches on
// the caller's stream.  As in ple_api.cu nothing is allocated, read back or
// kept.
#include <stdint.h>

#include <cmath>

#include "ple_tree_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
bool mult8(int64_t s) { return s % 8 == 0; }

ple_status finish(cudaError_t e) {
    return e == cudaSuccess ? PLE_OK : (ple_status)ple::record_cuda_failure(e);
}

ple_status with_device(ple::DeviceFacts* dev) { return finish(ple::device_facts(dev)); }

bool head_dim_ok(int32_t d) { return d >= 8 && d <= PLE_MAX_HEAD_DIM && d % 8 == 0; }
bool dtype_ok(int32_t t) { return t == PLE_BF16 || t == PLE_F16; }

// A paged cache's geometry: sizes that keep every element offset in 63 bits.
bool cache_sizes_ok(int64_t num_pages, int64_t page_stride, int64_t head_stride,
                    int64_t slot_stride, int32_t heads, int32_t page_size, int32_t max_pages,
                    int32_t head_dim) {
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
bool overlap(const void* a, __int128 n, const void* b, __int128 m) {
    const __int128 x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && n > 0 && m > 0 && x < y + m && y < x + n;
}

bool rows_ok(int64_t T, int64_t token, int32_t heads, int64_t head, int32_t dim) {
    if (token < 0 || head < 0) return false;
    return heads == 0 || (__int128)(T - 1) * token + (__int128)(heads - 1) * head + dim <=
                             INT64_MAX / 8;
}

}  // namespace

extern "C" ple_status ple_build_tree_index(const int32_t* parent, const int32_t* cu_seqlens,
                                           const int32_t* ctx_lens, int32_t num_requests,
                                           int64_t num_tokens, int32_t mask_words,
                                           int32_t* positions, uint64_t* tree_mask, void* stream) {
    if (num_tokens < 0 || num_tokens > INT32_MAX || mask_words < 1 ||
        mask_words > PLE_MAX_TREE_WORDS)
        return PLE_ERR_SIZE;
    if (num_tokens == 0) return PLE_OK;
    if (num_requests < 1) return PLE_ERR_SIZE;
    if (!parent || !cu_seqlens || !ctx_lens || !positions || !tree_mask) return PLE_ERR_NULL;
    if (!aligned(parent, 4) || !aligned(cu_seqlens, 4) || !aligned(ctx_lens, 4) ||
        !aligned(positions, 4) || !aligned(tree_mask, 8))
        return PLE_ERR_ALIGN;
    return finish(ple::launch_tree_index(parent, cu_seqlens, ctx_lens, num_requests, num_tokens,
                                         mask_words, positions, tree_mask,
                                         static_cast<cudaStream_t>(stream)));
}

extern "C" ple_status ple_tree_row_ids(const void* input_ids, int32_t id_dtype,
                                       int64_t num_tokens, const int32_t* parent,
                                       const int32_t* cu_seqlens, const void* ngram_context,
                                       int32_t num_requests, int32_t ctx_len,
                                       const int64_t* layer_multipliers,
                                       const int64_t* vocab_sizes, const int64_t* offsets,
                                       int32_t num_heads, int32_t ngram_size,
                                       int32_t heads_per_ngram, int32_t num_layers,
                                       int64_t boundary_id, void* out, int32_t out_dtype,
                                       const void* heads, void* stream) {
    if (ngram_size < 2 || ngram_size > PLE_MAX_NGRAM || heads_per_ngram < 1 || num_layers < 1 ||
        num_tokens < 0 || num_tokens > INT32_MAX)
        return PLE_ERR_SIZE;
    if (ctx_len != ngram_size - 1) return PLE_ERR_GEOMETRY_CTX;
    if ((int64_t)num_heads != (int64_t)(ngram_size - 1) * heads_per_ngram)
        return PLE_ERR_GEOMETRY_HEADS;
    if (num_heads > PLE_MAX_HEADS || num_layers > 65535) return PLE_ERR_SIZE;
    if ((int64_t)num_layers * num_tokens > (INT64_MAX / 8) / num_heads) return PLE_ERR_SIZE;
    if (out_dtype != PLE_I32 && out_dtype != PLE_I64) return PLE_ERR_DTYPE;
    if (num_tokens == 0) return PLE_OK;
    if (num_requests < 1) return PLE_ERR_SIZE;
    if (!input_ids || !parent || !cu_seqlens || !ngram_context || !layer_multipliers || !out ||
        (!heads && (!vocab_sizes || !offsets)))
        return PLE_ERR_NULL;
    if (id_dtype != PLE_I32 && id_dtype != PLE_I64) return PLE_ERR_DTYPE;
    const int id_bytes = id_dtype == PLE_I32 ? 4 : 8;
    const int out_bytes = out_dtype == PLE_I32 ? 4 : 8;
    if (!aligned(input_ids, id_bytes) || !aligned(ngram_context, id_bytes) ||
        !aligned(parent, 4) || !aligned(cu_seqlens, 4) || !aligned(layer_multipliers, 8) ||
        !aligned(vocab_sizes, 8) || !aligned(offsets, 8) || !aligned(heads, 16) ||
        !aligned(out, out_bytes))
        return PLE_ERR_ALIGN;
    ple::DeviceFacts dev;
    if (ple_status st = with_device(&dev); st != PLE_OK) return st;
    ple::RowIdsParams p = {};
    p.ids = input_ids;
    p.ctx = ngram_context;
    p.mult = layer_multipliers;
    p.vocab = vocab_sizes;
    p.offsets = offsets;
    p.out = out;
    p.T = num_tokens;
    p.boundary = boundary_id;
    p.B = num_requests;
    p.N = ngram_size;
    p.hpn = heads_per_ngram;
    p.H = num_heads;
    p.L = num_layers;
    p.index_mode = ple::kIdxCu;
    p.out_bytes = out_bytes;
    p.cu = cu_seqlens;
    p.heads = heads;
    p.ones = 0xFFFFFFFFu;
    return finish(ple::launch_tree_row_ids(p, parent, id_bytes, dev,
                                           static_cast<cudaStream_t>(stream)));
}

extern "C" ple_status ple_prepare_rope(int32_t rotary_dim, double base, int32_t scaling,
                                       double factor, double trained_positions, double beta_fast,
                                       double beta_slow, int64_t* rope, void* stream) {
    if (rotary_dim < 2 || rotary_dim > PLE_MAX_HEAD_DIM || rotary_dim % 2 != 0 ||
        !(base >= 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor) ||
        scaling < PLE_ROPE_PLAIN || scaling > PLE_ROPE_PARTS)
        return PLE_ERR_SIZE;
    if (scaling == PLE_ROPE_PARTS &&
        (!(trained_positions > 0.0) || !std::isfinite(trained_positions) || !(beta_slow >= 0.0) ||
         !(beta_fast > beta_slow) || !std::isfinite(beta_fast)))
        return PLE_ERR_SIZE;
    if (!rope) return PLE_ERR_NULL;
    if (!aligned(rope, 8)) return PLE_ERR_ALIGN;
    return finish(ple::launch_prepare_rope(rotary_dim, base, scaling, factor, trained_positions,
                                           beta_fast, beta_slow, rope,
                                           static_cast<cudaStream_t>(stream)));
}

extern "C" ple_status ple_qk_norm_rope(const ple_qk_norm_rope_args* args, void* stream) {
    if (!args) return PLE_ERR_NULL;
    const ple_qk_norm_rope_args& a = *args;
    const bool cache = a.k_cache || a.v_cache;
    if (a.num_tokens < 0 || a.num_tokens > INT32_MAX || a.q_heads < 0 || a.kv_heads < 0 ||
        a.q_heads > 65535 || a.kv_heads > 65535 || a.q_heads + a.kv_heads < 1 ||
        a.q_heads + a.kv_heads > 65535 || !head_dim_ok(a.head_dim) || a.rotary_dim < 0 ||
        a.rotary_dim > a.head_dim || a.rotary_dim % 2 != 0 || !(a.eps >= 0.0f) ||
        !std::isfinite(a.eps) || !std::isfinite(a.rope_scale))
        return PLE_ERR_SIZE;
    if (!dtype_ok(a.dtype)) return PLE_ERR_ELEMENT;
    if (a.num_tokens == 0) return PLE_OK;
    const int64_t T = a.num_tokens;
    if (!rows_ok(T, a.q_token, a.q_heads, a.q_head, a.head_dim) ||
        !rows_ok(T, a.q_out_token, a.q_heads, a.q_out_head, a.head_dim) ||
        !rows_ok(T, a.k_token, a.kv_heads, a.k_head, a.head_dim))
        return PLE_ERR_SIZE;
    if (cache) {
        if (a.num_requests < 1 || a.kv_heads < 1 ||
            !cache_sizes_ok(a.num_pages, a.page_stride, a.head_stride, a.slot_stride, a.kv_heads,
                            a.page_size, a.max_pages, a.head_dim) ||
            !rows_ok(T, a.v_token, a.kv_heads, a.v_head, a.head_dim))
            return PLE_ERR_SIZE;
    } else if (!rows_ok(T, a.k_out_token, a.kv_heads, a.k_out_head, a.head_dim)) {
        return PLE_ERR_SIZE;
    }
    if ((a.q_heads && (!a.q || !a.q_out)) || (a.kv_heads && !a.k) ||
        (a.rotary_dim && (!a.rope || !a.positions)))
        return PLE_ERR_NULL;
    if (cache ? (!a.k_cache || !a.v_cache || !a.v || !a.page_table || !a.ctx_lens || !a.cu_seqlens)
              : (a.kv_heads && !a.k_out))
        return PLE_ERR_NULL;
    if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.q_out, 16) ||
        !aligned(a.q_weight, 16) || !aligned(a.k_weight, 16) || !aligned(a.positions, 4) ||
        !aligned(a.rope, 8) || !mult8(a.q_token) || !mult8(a.q_head) || !mult8(a.k_token) ||
        !mult8(a.k_head) || !mult8(a.q_out_token) || !mult8(a.q_out_head))
        return PLE_ERR_ALIGN;
    if (cache ? (!aligned(a.v, 16) || !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) ||
                 !aligned(a.page_table, 4) || !aligned(a.ctx_lens, 4) ||
                 !aligned(a.cu_seqlens, 4) || !mult8(a.v_token) || !mult8(a.v_head) ||
                 !mult8(a.page_stride) || !mult8(a.head_stride) || !mult8(a.slot_stride))
              : (!aligned(a.k_out, 16) || !mult8(a.k_out_token) || !mult8(a.k_out_head)))
        return PLE_ERR_ALIGN;
    ple::DeviceFacts dev;
    if (ple_status st = with_device(&dev); st != PLE_OK) return st;
    return finish(ple::launch_qk_norm_rope(a, dev, static_cast<cudaStream_t>(stream)));
}

namespace {

bool attention_heads_ok(int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    return T >= 0 && T <= INT32_MAX && kv_heads >= 1 && q_heads >= 1 && q_heads <= 65535 &&
           q_heads % kv_heads == 0 && head_dim_ok(head_dim);
}

}  // namespace

extern "C" int64_t ple_tree_attention_workspace(int64_t num_tokens, int32_t q_heads,
                                                int32_t kv_heads, int32_t head_dim) {
    if (!attention_heads_ok(num_tokens, q_heads, kv_heads, head_dim)) return -1;
    ple::DeviceFacts dev;
    if (with_device(&dev) != PLE_OK) return -1;
    return ple::tree_attention_workspace(num_tokens, q_heads, kv_heads, head_dim, dev);
}

extern "C" ple_status ple_tree_attention(const ple_tree_attention_args* args, void* stream) {
    if (!args) return PLE_ERR_NULL;
    const ple_tree_attention_args& a = *args;
    if (!attention_heads_ok(a.num_tokens, a.q_heads, a.kv_heads, a.head_dim) ||
        a.mask_words < 1 || a.mask_words > PLE_MAX_TREE_WORDS || !std::isfinite(a.scale))
        return PLE_ERR_SIZE;
    if (!dtype_ok(a.dtype)) return PLE_ERR_ELEMENT;
    if (a.num_tokens == 0) return PLE_OK;
    if (a.num_requests < 1 ||
        !cache_sizes_ok(a.num_pages, a.page_stride, a.head_stride, a.slot_stride, a.kv_heads,
                        a.page_size, a.max_pages, a.head_dim) ||
        !rows_ok(a.num_tokens, a.q_token, a.q_heads, a.q_head, a.head_dim) ||
        a.num_tokens > INT64_MAX / 8 / ((int64_t)a.q_heads * a.head_dim))
        return PLE_ERR_SIZE;
    if (!a.q || !a.k_cache || !a.v_cache || !a.page_table || !a.ctx_lens || !a.cu_seqlens ||
        !a.tree_mask || !a.out || !a.workspace)
        return PLE_ERR_NULL;
    if (!aligned(a.q, 16) || !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) ||
        !aligned(a.page_table, 4) || !aligned(a.ctx_lens, 4) || !aligned(a.cu_seqlens, 4) ||
        !aligned(a.tree_mask, 8) || !aligned(a.out, 16) || !aligned(a.lse, 4) ||
        !aligned(a.workspace, 16) || !mult8(a.q_token) || !mult8(a.q_head) ||
        !mult8(a.page_stride) || !mult8(a.head_stride) || !mult8(a.slot_stride))
        return PLE_ERR_ALIGN;
    ple::DeviceFacts dev;
    if (ple_status st = with_device(&dev); st != PLE_OK) return st;
    if (a.workspace_bytes <
        ple::tree_attention_workspace(a.num_tokens, a.q_heads, a.kv_heads, a.head_dim, dev))
        return PLE_ERR_SIZE;
    return finish(ple::launch_tree_attention(a, dev, static_cast<cudaStream_t>(stream)));
}

extern "C" ple_status ple_tree_commit(const ple_tree_commit_args* args, void* stream) {
    if (!args) return PLE_ERR_NULL;
    const ple_tree_commit_args& a = *args;
    if (a.num_tokens < 0 || a.num_tokens > INT32_MAX || a.num_requests < 0 || a.path_len < 0 ||
        (a.path_len == 0 && a.path) || a.num_layers < 1 || a.num_layers > 65535 ||
        !head_dim_ok(a.head_dim) || a.layer_stride < 0 ||
        !cache_sizes_ok(a.num_pages, a.page_stride, a.head_stride, a.slot_stride, a.kv_heads,
                        a.page_size, a.max_pages, a.head_dim) ||
        (__int128)(a.num_layers - 1) * a.layer_stride > INT64_MAX / 16)
        return PLE_ERR_SIZE;
    if (a.ngram_context && (a.ctx_len < 1 || a.ctx_len >= PLE_MAX_NGRAM)) return PLE_ERR_SIZE;
    if (a.ngram_context && a.id_dtype != PLE_I32 && a.id_dtype != PLE_I64) return PLE_ERR_DTYPE;
    if (!dtype_ok(a.dtype)) return PLE_ERR_ELEMENT;
    if (a.num_requests == 0) return PLE_OK;
    if ((!a.path && a.path_len) || !a.accepted || !a.cu_seqlens || !a.ctx_lens ||
        !a.next_ctx_lens || !a.page_table || !a.k_cache || !a.v_cache ||
        (a.ngram_context && ((!a.input_ids && a.num_tokens) || !a.next_context)))
        return PLE_ERR_NULL;
    const int id_bytes = a.id_dtype == PLE_I32 ? 4 : 8;
    if (!aligned(a.path, 4) || !aligned(a.accepted, 4) || !aligned(a.cu_seqlens, 4) ||
        !aligned(a.ctx_lens, 4) || !aligned(a.next_ctx_lens, 4) || !aligned(a.page_table, 4) ||
        !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) || !mult8(a.layer_stride) ||
        !mult8(a.page_stride) || !mult8(a.head_stride) || !mult8(a.slot_stride) ||
        (a.ngram_context && (!aligned(a.input_ids, id_bytes) ||
                             !aligned(a.ngram_context, id_bytes) ||
                             !aligned(a.next_context, id_bytes))))
        return PLE_ERR_ALIGN;
    // a request's blocks, one a layer and cache, run in any order: what one of them
    // writes for the next step may be nothing that another still reads
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
    if (overlap(out[0].at, out[0].bytes, out[1].at, out[1].bytes)) return PLE_ERR_SIZE;
    for (const auto& o : out)
        for (const auto& i : in)
            if (overlap(o.at, o.bytes, i.at, i.bytes)) return PLE_ERR_SIZE;
    ple::DeviceFacts dev;
    if (ple_status st = with_device(&dev); st != PLE_OK) return st;
    return finish(ple::launch_tree_commit(a, dev, static_cast<cudaStream_t>(stream)));
}
