// attention_abi.cu — the C ABI of the attention calls: checks of every host
// argument, then one launcher each. Nothing here allocates or synchronises.
#include <cuda_runtime.h>
#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

#include "attention.h"
#include "moe.h"

using namespace moe;

namespace {

struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A required pointer, n-byte aligned.
bool good(const void *p, uintptr_t n) { return p && aligned(p, n); }

bool finite(float v) { return v - v == 0.0f; }

moe_status_t heads_ok(int32_t heads, int32_t kv_heads, int32_t dim, uint32_t dtype) {
  if (heads <= 0 || kv_heads <= 0 || dim <= 0 || heads % kv_heads) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return MOE_ERR_INVALID_ARG;
  if ((dim != 64 && dim != 128) || heads > 1024) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Rows of `width` contiguous elements, `stride` elements apart.
bool stride_ok(int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0; }

moe_status_t cache_sizes_ok(const moe_kv_cache_t &c) {
  if (c.num_pages < 0 || c.page_size <= 0 || c.num_kv_heads <= 0 || c.head_dim <= 0) return MOE_ERR_INVALID_ARG;
  if (c.page_size % 16 || c.page_size > 1024 || (c.head_dim != 64 && c.head_dim != 128) || c.num_kv_heads > 1024)
    return MOE_ERR_UNSUPPORTED;
  // cached rows are counted in 32 bits: more of them than a device's memory holds
  if (int64_t(c.num_pages) * c.page_size > int64_t(0xFFFFFFFFu) / c.num_kv_heads - 1) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status_t cache_ok(const moe_kv_cache_t &c) {
  const moe_status_t s = cache_sizes_ok(c);
  if (s != MOE_OK) return s;
  if (c.num_pages == 0) return MOE_OK;  // an empty cache: no pointer is used
  if (!good(c.k_codes, 16) || !good(c.k_scales, 16) || !good(c.v_codes, 16) || !good(c.v_scales, 16))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Multiprocessors of the current device, or 0 when it is not one the kernels are built for.
moe_status_t device_sms(int *sms) {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  return major == 10 && minor == 3 ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

moe_status_t paged_sizes_ok(const moe_attend_paged_io_t &io, const moe_kv_cache_t &c) {
  moe_status_t s = cache_sizes_ok(c);
  if (s == MOE_OK) s = heads_ok(io.num_heads, c.num_kv_heads, c.head_dim, io.dtype);
  if (s != MOE_OK) return s;
  if (io.num_seqs < 0 || io.num_rows < 0 || io.max_pages < 0 || io.max_rows < 1) return MOE_ERR_INVALID_ARG;
  if (io.num_seqs > kMaxSeqs) return MOE_ERR_UNSUPPORTED;
  if (int64_t(io.max_pages) * c.page_size > 1 << 30) return MOE_ERR_UNSUPPORTED;  // keys are counted in 32 bits
  if (int64_t(io.num_rows) * io.num_heads > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status_t prompt_sizes_ok(const moe_attend_prompt_io_t &io) {
  const moe_status_t s = heads_ok(io.num_heads, io.num_kv_heads, io.head_dim, io.dtype);
  if (s != MOE_OK) return s;
  if (io.num_seqs < 0 || io.num_rows < 0 || io.num_keys < 0) return MOE_ERR_INVALID_ARG;
  if (io.num_seqs > kMaxSeqs || int64_t(io.num_rows) * io.num_heads > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_qkv_append(const moe_qkv_append_io_t *io, const moe_kv_cache_t *cache, int32_t *d_status,
                            void *cuda_stream) {
  const NvtxRange nvtx_range("moe_qkv_append");
  if (!io || io->num_tokens < 0 || io->flags & ~MOE_FLAG_TEST_BOUNDS) return MOE_ERR_INVALID_ARG;
  moe_status_t s = heads_ok(io->num_heads, io->num_kv_heads, io->head_dim, io->dtype);
  if (s != MOE_OK) return s;
  const int64_t D = io->head_dim;
  if (io->rotary_dim < 0 || io->rotary_dim > D || io->rotary_dim % 2) return MOE_ERR_INVALID_ARG;
  if (io->rotary_dim % 16) return MOE_ERR_UNSUPPORTED;
  if (!finite(io->norm_eps) || io->norm_eps < 0.0f) return MOE_ERR_INVALID_ARG;
  if (cache) {
    s = cache_ok(*cache);
    if (s != MOE_OK) return s;
    if (cache->num_kv_heads != io->num_kv_heads || cache->head_dim != io->head_dim) return MOE_ERR_INVALID_ARG;
  }
  if (io->num_tokens == 0) return MOE_OK;
  if (!good(io->q, 16) || !good(io->k, 16) || !good(io->v, 16) || !good(io->q_out, 16)) return MOE_ERR_INVALID_ARG;
  if (!stride_ok(io->q_stride, io->num_heads * D) || !stride_ok(io->k_stride, io->num_kv_heads * D) ||
      !stride_ok(io->v_stride, io->num_kv_heads * D))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(io->k_out, 16) || !aligned(io->k_cached, 16) || !aligned(io->v_cached, 16) ||
      !aligned(io->q_norm, 16) || !aligned(io->k_norm, 16))
    return MOE_ERR_INVALID_ARG;
  if (io->rotary_dim &&
      (!good(io->rope, 16) || !good(io->positions, 4) || io->rope_positions <= 0))
    return MOE_ERR_INVALID_ARG;
  if (cache && !good(io->slots, 8)) return MOE_ERR_INVALID_ARG;
  if (!aligned(d_status, 4)) return MOE_ERR_INVALID_ARG;
  int sms = 0;
  s = device_sms(&sms);
  if (s != MOE_OK) return s;
  return launch_qkv_append(*io, cache, d_status, sms, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status_t moe_attend_paged_workspace(const moe_attend_paged_io_t *io, const moe_kv_cache_t *cache,
                                        int64_t *bytes_out) {
  if (!io || !cache || !bytes_out) return MOE_ERR_INVALID_ARG;
  moe_status_t s = paged_sizes_ok(*io, *cache);
  if (s != MOE_OK) return s;
  int sms = 0;
  s = device_sms(&sms);
  if (s != MOE_OK) return s;
  *bytes_out = attend_paged_workspace(*io, *cache, sms);
  return MOE_OK;
}

moe_status_t moe_attend_paged(const moe_attend_paged_io_t *io, const moe_kv_cache_t *cache, void *workspace,
                              int64_t workspace_bytes, int32_t *d_status, void *cuda_stream) {
  const NvtxRange nvtx_range("moe_attend_paged");
  if (!io || !cache) return MOE_ERR_INVALID_ARG;
  moe_status_t s = paged_sizes_ok(*io, *cache);
  if (s == MOE_OK) s = cache_ok(*cache);
  if (s != MOE_OK) return s;
  if (!finite(io->scale) || !aligned(d_status, 4) || !aligned(io->lse, 4)) return MOE_ERR_INVALID_ARG;
  if (io->flags & ~MOE_FLAG_TEST_BOUNDS) return MOE_ERR_INVALID_ARG;
  if (io->num_rows == 0 || io->num_seqs == 0) return MOE_OK;
  const int64_t width = int64_t(io->num_heads) * cache->head_dim;
  if (!good(io->q, 16) || !good(io->out, 16) || !stride_ok(io->q_stride, width) || !stride_ok(io->out_stride, width))
    return MOE_ERR_INVALID_ARG;
  if (!good(io->lengths, 4) || !good(io->cu_rows, 4) || (io->max_pages && !good(io->page_table, 4)))
    return MOE_ERR_INVALID_ARG;
  int sms = 0;
  s = device_sms(&sms);
  if (s != MOE_OK) return s;
  const int64_t need = attend_paged_workspace(*io, *cache, sms);
  if (workspace_bytes < need || (need && !good(workspace, 16))) return MOE_ERR_INVALID_ARG;
  return launch_attend_paged(*io, *cache, workspace, workspace_bytes, d_status, sms,
                             static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status_t moe_attend_prompt_workspace(const moe_attend_prompt_io_t *io, int64_t *bytes_out) {
  if (!io || !bytes_out) return MOE_ERR_INVALID_ARG;
  moe_status_t s = prompt_sizes_ok(*io);
  if (s != MOE_OK) return s;
  int sms = 0;
  s = device_sms(&sms);
  if (s != MOE_OK) return s;
  *bytes_out = attend_prompt_workspace(*io, sms);
  return MOE_OK;
}

moe_status_t moe_attend_prompt(const moe_attend_prompt_io_t *io, int32_t *d_status, void *cuda_stream) {
  const NvtxRange nvtx_range("moe_attend_prompt");
  if (!io) return MOE_ERR_INVALID_ARG;
  moe_status_t s = prompt_sizes_ok(*io);
  if (s != MOE_OK) return s;
  if ((io->causal != 0 && io->causal != 1) || io->flags & ~(MOE_FLAG_TEST_SKIP_READY | MOE_FLAG_TEST_BOUNDS))
    return MOE_ERR_INVALID_ARG;
  if (!finite(io->scale) || !aligned(d_status, 4) || !aligned(io->lse, 4)) return MOE_ERR_INVALID_ARG;
  if (io->num_rows == 0 || io->num_seqs == 0) return MOE_OK;
  const int64_t D = io->head_dim;
  if (!good(io->q, 16) || !good(io->out, 16) || !stride_ok(io->q_stride, io->num_heads * D) ||
      !stride_ok(io->out_stride, io->num_heads * D))
    return MOE_ERR_INVALID_ARG;
  if (io->num_keys && (!good(io->k, 16) || !good(io->v, 16) || !stride_ok(io->k_stride, io->num_kv_heads * D) ||
                       !stride_ok(io->v_stride, io->num_kv_heads * D)))
    return MOE_ERR_INVALID_ARG;
  if (!good(io->cu_rows, 4) || !good(io->cu_keys, 4)) return MOE_ERR_INVALID_ARG;
  int sms = 0;
  s = device_sms(&sms);
  if (s != MOE_OK) return s;
  if (io->workspace && (!aligned(io->workspace, 16) || io->workspace_bytes < attend_prompt_workspace(*io, sms)))
    return MOE_ERR_INVALID_ARG;
  return launch_attend_prompt(*io, d_status, sms, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // extern "C"
