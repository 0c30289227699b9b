// Internal launch interface of the entry points for caches in 8 bits and for
// pages (ple_cache_api.cu), next to ple_tree_internal.h.
#pragma once

#include <cuda.h>

#include "ple_tree_internal.h"

namespace ple {

cudaError_t launch_qk_norm_rope_fp8(const ple_qk_norm_rope_fp8_args& a, const DeviceFacts& dev,
                                    cudaStream_t stream);

int64_t tree_attention_fp8_workspace(int64_t T, int32_t q_heads, int32_t kv_heads,
                                     int32_t head_dim, const DeviceFacts& dev);
cudaError_t launch_tree_attention_fp8(const ple_tree_attention_fp8_args& a,
                                      const DeviceFacts& dev, cudaStream_t stream);

// Its kernel for many rows a key head (ple_tree_attention_fp8_tc.cu), on the caches' tensor
// maps.
int64_t tree_attention_fp8_tc_workspace(int64_t T, int32_t q_heads, int32_t kv_heads,
                                        int32_t head_dim, const DeviceFacts& dev);
cudaError_t launch_tree_attention_fp8_tc(const ple_tree_attention_fp8_args& a,
                                         const CUtensorMap& k, const CUtensorMap& v,
                                         const DeviceFacts& dev, cudaStream_t stream);

cudaError_t launch_tree_commit_fp8(const ple_tree_commit_fp8_args& a, const DeviceFacts& dev,
                                   cudaStream_t stream);

int64_t plan_pages_workspace(int32_t num_rows, int32_t num_pages);
cudaError_t launch_plan_pages(const ple_plan_pages_args& a, cudaStream_t stream);

// Whether a page's shares fit a grid.
bool copy_page_ok(const ple_copy_pages_args& a);
cudaError_t launch_copy_pages(const ple_copy_pages_args& a, const DeviceFacts& dev,
                              cudaStream_t stream);

}  // namespace ple
