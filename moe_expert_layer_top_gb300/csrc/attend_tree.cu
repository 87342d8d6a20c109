// attend_tree.cu — attention of trees of drafted tokens over the paged MXFP4 cache.
//
// The mathematics and the kernels are those of attend_paged.cu (paged.cuh); a row
// sees the keys in front of the tree and, of the tree's own keys, its ancestors'
// and its own.
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.cuh"

namespace moe {

int64_t attend_tree_workspace(const moe_attend_tree_io_t &io, const moe_kv_cache_t &c, int num_sms) {
  return workspace_of<true>(io.rows, c, num_sms);
}

cudaError_t launch_attend_tree(const moe_attend_tree_io_t &io, const moe_kv_cache_t &c, void *workspace,
                               int64_t workspace_bytes, int32_t *status, int num_sms, cudaStream_t st) {
  return launch_paged<true>(io.rows, io.parents, c, workspace, workspace_bytes, status, num_sms, st);
}

}  // namespace moe
