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

// The kernels of paged.cuh decode keys and values once for every 32 rows of a kv head (up to 48: every 24), those of tree_tiles.cu once for 128
// or 256, with more to fill and to drain. Measured, device us, paged.cuh / tree_tiles.cu (8 kv heads, D = 128):
//   rows of a kv head              24           32           36           48           64           96
//   64 sequences of 2,048     79.9 / 118.8  105 / 120    140 / 123    142 / 124    189 / 128    270 / 131
//   16 of 4,096               42.5 / 63.0  55.4 / 62.7  72.0 / 65.5  71.7 / 65.4  94.5 / 67.4   131 / 69.6
//   4 of 4,096                21.1 / 28.8  26.6 / 29.0  28.8 / 30.2  29.3 / 31.8  36.9 / 32.1  47.7 / 36.0
//   1 of 32,768               31.0 / 38.7  39.4 / 39.3  41.5 / 41.0  41.7 / 42.8  52.9 / 43.7  68.9 / 46.5
//   1 of 4,096                18.1 / 22.1  22.4 / 22.8  19.5 / 23.9  20.1 / 24.4  24.2 / 25.2  25.9 / 28.1
//   1 of 500                  13.7 / 17.0  16.3 / 17.4  13.8 / 17.6  13.8 / 19.3  17.2 / 20.0  18.9 / 21.9
// D = 64 crosses at the same places. How long the contexts are is not known here.
constexpr int kTileRows = 33;      // rows of a kv head from which on tiles are taken
constexpr int kTileRowsFew = 49;   // the same with few items,
constexpr int kFewItems = 32;      // (sequence, kv head) pairs

bool tiles(const moe_attend_tree_io_t &io, const moe_kv_cache_t &c) {
  const int64_t items = int64_t(io.rows.num_seqs) * c.num_kv_heads;
  return usual_rows(io.rows, c) >= (items > kFewItems ? kTileRows : kTileRowsFew);
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
