// speculative_abi.cu — the C ABI of the calls of a step with trees of drafted tokens: checks of every host argument,
// then one launcher each. Nothing here allocates or synchronises.
#include <cuda_runtime.h>
#include <stdint.h>

#include "attention.h"
#include "checks.h"
#include "moe.h"
#include "speculative.h"

using namespace moe;

extern "C" {

moe_status_t moe_attend_tree_workspace(const moe_attend_tree_io_t *io, const moe_kv_cache_t *cache, int64_t *bytes_out) {
  if (!io || !cache || !bytes_out) return MOE_ERR_INVALID_ARG;
  moe_status_t s = paged_sizes_ok(io->rows, *cache);
  if (s != MOE_OK) return s;
  int sms = 0;
  s = device_sms(&sms);
  if (s != MOE_OK) return s;
  *bytes_out = attend_tree_workspace(*io, *cache, sms);
  return MOE_OK;
}

moe_status_t moe_attend_tree(const moe_attend_tree_io_t *io, const moe_kv_cache_t *cache, void *workspace,
                             int64_t workspace_bytes, int32_t *d_status, void *cuda_stream) {
  const NvtxRange nvtx_range("moe_attend_tree");
  if (!io || !cache) return MOE_ERR_INVALID_ARG;
  const moe_attend_paged_io_t &r = io->rows;
  moe_status_t s = paged_sizes_ok(r, *cache);
  if (s == MOE_OK) s = cache_ok(*cache);
  if (s != MOE_OK) return s;
  if (!finite(r.scale) || !aligned(d_status, 4) || !aligned(r.lse, 4)) return MOE_ERR_INVALID_ARG;
  if (r.flags & ~(MOE_FLAG_TEST_SKIP_READY | MOE_FLAG_TEST_BOUNDS)) return MOE_ERR_INVALID_ARG;
  if (r.num_rows == 0 || r.num_seqs == 0) return MOE_OK;
  const int64_t width = int64_t(r.num_heads) * cache->head_dim;
  if (!good(r.q, 16) || !good(r.out, 16) || !stride_ok(r.q_stride, width) || !stride_ok(r.out_stride, width))
    return MOE_ERR_INVALID_ARG;
  if (!good(r.lengths, 4) || !good(r.cu_rows, 4) || !good(io->parents, 4) || (r.max_pages && !good(r.page_table, 4)))
    return MOE_ERR_INVALID_ARG;
  int sms = 0;
  s = device_sms(&sms);
  if (s != MOE_OK) return s;
  const int64_t need = attend_tree_workspace(*io, *cache, sms);
  if (workspace_bytes < need || (need && !good(workspace, 16))) return MOE_ERR_INVALID_ARG;
  return launch_attend_tree(*io, *cache, workspace, workspace_bytes, d_status, sms,
                            static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status_t moe_verify_drafts(const moe_verify_drafts_io_t *io, int32_t *d_status, void *cuda_stream) {
  const NvtxRange nvtx_range("moe_verify_drafts");
  if (!io || io->flags) return MOE_ERR_INVALID_ARG;
  if (io->dtype != MOE_DTYPE_BF16 && io->dtype != MOE_DTYPE_F16 && io->dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  if (io->num_seqs < 0 || io->num_rows < 0 || io->max_rows < 1 || io->vocab < 1) return MOE_ERR_INVALID_ARG;
  if (io->num_seqs > 65535 || io->max_rows > MOE_MAX_TREE_ROWS || io->vocab > 1 << 24) return MOE_ERR_UNSUPPORTED;
  if (!aligned(d_status, 4)) return MOE_ERR_INVALID_ARG;
  if (io->num_seqs == 0) return MOE_OK;
  if (!good(io->cu_rows, 4) || !good(io->sample_u, 4) || !aligned(io->temperature, 4) || !good(io->out_tokens, 4) ||
      !good(io->path, 4) || !good(io->accepted, 4))
    return MOE_ERR_INVALID_ARG;
  if (io->num_rows) {
    if (!good(io->logits, io->dtype == MOE_DTYPE_F32 ? 4 : 2) || io->logits_stride < io->vocab) return MOE_ERR_INVALID_ARG;
    if (!aligned(io->draft_probs, 4) || (io->draft_probs && io->draft_stride < io->vocab)) return MOE_ERR_INVALID_ARG;
    if (!good(io->tokens, 4) || !aligned(io->parents, 4) || !good(io->accept_u, 4)) return MOE_ERR_INVALID_ARG;
  }
  int sms = 0;
  const moe_status_t s = device_sms(&sms);
  if (s != MOE_OK) return s;
  return launch_verify_drafts(*io, d_status, sms, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? MOE_OK
                                                                                                         : MOE_ERR_CUDA;
}

moe_status_t moe_commit_drafts(const moe_commit_drafts_io_t *io, const moe_kv_cache_t *caches, int32_t *d_status,
                               void *cuda_stream) {
  const NvtxRange nvtx_range("moe_commit_drafts");
  if (!io || !caches || io->flags & ~MOE_FLAG_TEST_BOUNDS) return MOE_ERR_INVALID_ARG;
  if (io->num_seqs < 0 || io->max_pages < 0 || io->path_stride < 1 || io->num_caches < 1) return MOE_ERR_INVALID_ARG;
  if (io->num_seqs > 65535 || io->num_caches > 4096) return MOE_ERR_UNSUPPORTED;
  for (int i = 0; i < io->num_caches; ++i) {
    const moe_kv_cache_t &c = caches[i], &first = caches[0];
    const moe_status_t s = cache_ok(c);
    if (s != MOE_OK) return s;
    if (c.page_size != first.page_size || c.num_kv_heads != first.num_kv_heads || c.head_dim != first.head_dim)
      return MOE_ERR_INVALID_ARG;
  }
  if (int64_t(io->max_pages) * caches[0].page_size > 1 << 30) return MOE_ERR_UNSUPPORTED;
  if (!aligned(d_status, 4)) return MOE_ERR_INVALID_ARG;
  if (io->num_seqs == 0) return MOE_OK;
  if (!good(io->lengths, 4) || !good(io->cu_rows, 4) || !good(io->path, 4) || !good(io->accepted, 4) ||
      !good(io->new_lengths, 4) || (io->max_pages && !good(io->page_table, 4)))
    return MOE_ERR_INVALID_ARG;
  int sms = 0;
  const moe_status_t s = device_sms(&sms);
  if (s != MOE_OK) return s;
  return launch_commit_drafts(*io, caches, d_status, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? MOE_OK
                                                                                                            : MOE_ERR_CUDA;
}

}  // extern "C"
