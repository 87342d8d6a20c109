// attend_tree.cu — attention of trees of drafted tokens over the paged MXFP4 cache.
//
// A row sees the keys in front of the tree and, of the tree's own keys, its
// ancestors' and its own. Small trees take the kernels of attend_paged.cu
// (paged.cuh), large ones those of tree_tiles.cu.
#include <cuda_runtime.h>
#include <stdint.h>

#include "paged.cuh"

namespace moe {

namespace {

// The kernels of paged.cuh decode keys and values once for every 32 rows of a kv head, those of tree_tiles.cu once for 128
// or 256.
constexpr int kTileRows = 33;  // rows of a kv head from which on tiles are taken

bool tiles(const moe_attend_tree_io_t &io, const moe_kv_cache_t &c) { return usual_rows(io.rows, c) >= kTileRows; }

}  // namespace

int64_t attend_tree_workspace(const moe_attend_tree_io_t &io, const moe_kv_cache_t &c, int num_sms) {
  return tiles(io, c) ? tree_tiles_workspace(c, num_sms) : workspace_of<true>(io.rows, c, num_sms);
}

cudaError_t launch_attend_tree(const moe_attend_tree_io_t &io, const moe_kv_cache_t &c, void *workspace,
                               int64_t workspace_bytes, int32_t *status, int num_sms, cudaStream_t st) {
  if (tiles(io, c))
    return launch_tree_tiles(io, c, usual_rows(io.rows, c), workspace, workspace_bytes, status, num_sms, st);
  return launch_paged<true>(io.rows, io.parents, c, workspace, workspace_bytes, status, num_sms, st);
}

}  // namespace moe
