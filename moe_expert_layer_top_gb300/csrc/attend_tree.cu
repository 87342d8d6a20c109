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

// The kernels of paged.cuh decode keys and values once for every 32 rows of a kv head (up to 48: every 24), those of
// tree_tiles.cu once for 128 or 256, with more to fill and to drain. Measured, device us, paged.cuh / tree_tiles.cu (8 kv
// heads):
//   rows of a kv head             24           32           36           48           64           96
//   D = 128
//   64 sequences of 2,048   74.4 / 116   98.0 / 118    133 / 118    136 / 119    180 / 121    263 / 126
//   16 of 4,096            38.8 / 57.4  51.1 / 56.9  67.2 / 57.5  67.6 / 57.2  89.7 / 59.2   127 / 60.4
//   4 of 4,096             18.8 / 26.9  23.1 / 27.2  25.5 / 27.2  25.8 / 27.9  32.7 / 28.2  43.4 / 29.5
//   1 of 32,768            26.9 / 36.2  33.6 / 36.4  37.8 / 36.7  38.2 / 37.2  49.1 / 37.6  66.1 / 39.0
//   1 of 4,096             14.1 / 19.8  17.6 / 19.9  16.3 / 20.2  16.6 / 20.6  20.0 / 21.1  22.7 / 22.4
//   1 of 500               11.8 / 16.0  13.7 / 16.4  11.8 / 16.6  11.7 / 16.6  14.6 / 17.2  15.9 / 18.3
//   D = 64
//   64 of 2,048            48.5 / 87.6  63.5 / 88.6  81.9 / 89.2  82.6 / 90.0   111 / 89.8   159 / 91.7
//   16 of 4,096            27.0 / 46.5  34.8 / 46.9  43.9 / 46.8  44.1 / 47.0  58.6 / 47.2  81.4 / 47.9
//   1 of 32,768            21.8 / 29.1  26.1 / 29.4  27.6 / 29.5  27.9 / 29.7  34.0 / 30.1  44.6 / 30.1
// How long the contexts are is not known here.
constexpr int kTileRows = 49;      // rows of a kv head from which on tiles are taken
constexpr int kTileRowsMany = 33;  // the same for D = 128 with more than
constexpr int kFewItems = 32;      // (sequence, kv head) pairs

bool tiles(const moe_attend_tree_io_t &io, const moe_kv_cache_t &c) {
  const bool many = c.head_dim == 128 && int64_t(io.rows.num_seqs) * c.num_kv_heads > kFewItems;
  return usual_rows(io.rows, c) >= (many ? kTileRowsMany : kTileRows);
}

}  // namespace

int64_t attend_tree_workspace(const moe_attend_tree_io_t &io, const moe_kv_cache_t &c, int num_sms) {
  return tiles(io, c) ? tree_tiles_workspace(c, num_sms) : workspace_of<true>(io.rows, c, num_sms);
}

cudaError_t launch_attend_tree(const moe_attend_tree_io_t &io, const moe_kv_cache_t &c, void *workspace,
                               int64_t workspace_bytes, int32_t *status, int num_sms, cudaStream_t st) {
  if (tiles(io, c))
    return launch_tree_tiles(io, c, usual_rows(io.rows, c), workspace, status, num_sms, st);
  return launch_paged<true>(io.rows, io.parents, c, workspace, workspace_bytes, status, num_sms, st);
}

}  // namespace moe
