// Internal launch interface of the tree-verification entry points
// (ple_tree_api.cu) and their kernels, next to ple_internal.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ple.h"
#include "ple_internal.h"

namespace ple {

// Notes a CUDA error for ple_last_cuda_error and returns PLE_ERR_CUDA.
int32_t record_cuda_failure(cudaError_t e);

cudaError_t launch_tree_index(const int32_t* parent, const int32_t* cu, const int32_t* ctx_lens,
                              int32_t B, int64_t T, int32_t words, int32_t* positions,
                              uint64_t* mask, cudaStream_t stream);

// The tree's row ids: the row-id parameters (cu set, req and local unused)
// and each node's parent.
cudaError_t launch_tree_row_ids(RowIdsParams p, const int32_t* parent, int id_bytes,
                                const DeviceFacts& dev, cudaStream_t stream);

cudaError_t launch_prepare_rope(int32_t rotary_dim, double base, int32_t scaling, double factor,
                                double trained, double beta_fast, double beta_slow,
                                int64_t* rope, cudaStream_t stream);

cudaError_t launch_qk_norm_rope(const ple_qk_norm_rope_args& a, const DeviceFacts& dev,
                                cudaStream_t stream);

cudaError_t launch_tree_commit(const ple_tree_commit_args& a, const DeviceFacts& dev,
                               cudaStream_t stream);

int64_t tree_attention_workspace(int64_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                 const DeviceFacts& dev);
cudaError_t launch_tree_attention(const ple_tree_attention_args& a, const DeviceFacts& dev,
                                  cudaStream_t stream);
// The tensor-core kernel (ple_tree_attention_tc.cu): which shapes it takes, the
// states of split rows, its launches.
bool tree_attention_tc_fits(const ple_tree_attention_args& a);
int64_t tree_attention_tc_workspace(int64_t T, int32_t q_heads, int32_t kv_heads,
                                    int32_t head_dim, const DeviceFacts& dev);
cudaError_t launch_tree_attention_tc(const ple_tree_attention_args& a, const DeviceFacts& dev,
                                     cudaStream_t stream, bool* taken);

}  // namespace ple
