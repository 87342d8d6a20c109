// checks.h — checks of host arguments that the attention calls share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <nvtx3/nvToolsExt.h>

#include "attention.h"
#include "moe.h"

namespace moe {

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

}  // namespace

}  // namespace moe
