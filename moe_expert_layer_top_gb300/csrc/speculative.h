// speculative.h — arguments and launchers of the kernels of a step with trees of drafted tokens.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

constexpr int kMaxTree = MOE_MAX_TREE_ROWS;  // rows of a tree
constexpr int kMaxCaches = 64;               // caches of one commit launch

int64_t attend_tree_workspace(const moe_attend_tree_io_t &io, const moe_kv_cache_t &c, int num_sms);
cudaError_t launch_attend_tree(const moe_attend_tree_io_t &io, const moe_kv_cache_t &c, void *workspace,
                               int64_t workspace_bytes, int32_t *status, int num_sms, cudaStream_t st);
int64_t tree_tiles_workspace(const moe_kv_cache_t &c, int num_sms);
cudaError_t launch_tree_tiles(const moe_attend_tree_io_t &io, const moe_kv_cache_t &c, int usual_rows, void *workspace,
                              int32_t *status, int num_sms, cudaStream_t st);
cudaError_t launch_verify_drafts(const moe_verify_drafts_io_t &io, int32_t *status, int num_sms, cudaStream_t st);
cudaError_t launch_commit_drafts(const moe_commit_drafts_io_t &io, const moe_kv_cache_t *caches, int32_t *status,
                                 cudaStream_t st);

}  // namespace moe
