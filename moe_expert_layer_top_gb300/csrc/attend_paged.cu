// attend_paged.cu — attention of the newest rows of each sequence over the paged MXFP4 cache.
#include <cuda_runtime.h>
#include <stdint.h>

#include "attend_simple.cuh"

namespace moe {

namespace {

struct PagedSource {
  const int32_t *page_table, *lengths, *cu_rows;
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int num_pages, page_size, max_pages, num_kv_heads;

  __device__ int keys(int b, int n, int num_keys, int32_t *status, int *first) const {
    *first = 0;
    int len = __ldg(lengths + b);
    if (len < 0 || len > max_pages * page_size) {
      out_of_range(status);
      len = len < 0 ? 0 : max_pages * page_size;
    }
    return len;
  }

  // One element pair (2i, 2i + 1) of key j; false where the page is out of range.
  template <int D>
  __device__ bool load(bool value, int b, int kv, int j, int i, float2 *out, int32_t *status) const {
    const int page = __ldg(page_table + int64_t(b) * max_pages + j / page_size);
    if (page < 0 || page >= num_pages) {
      out_of_range(status);
      *out = make_float2(0.0f, 0.0f);
      return false;
    }
    const int64_t at = (int64_t(page) * num_kv_heads + kv) * page_size + j % page_size;
    const uint32_t c = (value ? v_codes : k_codes)[at * (D / 2) + i];
    const float s = ue8m0_to_float((value ? v_scales : k_scales)[at * (D / 32) + i / 16]);
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(c), __NV_E2M1);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    *out = make_float2(f.x * s, f.y * s);
    return true;
  }
};

}  // namespace

int64_t attend_paged_workspace(const moe_attend_paged_io_t &io, const moe_kv_cache_t &c, int num_sms) { return 0; }

cudaError_t launch_attend_paged(const moe_attend_paged_io_t &io, const moe_kv_cache_t &c, void *workspace,
                                int32_t *status, int num_sms, cudaStream_t st) {
  SimpleArgs a = {};
  a.q = static_cast<const uint16_t *>(io.q);
  a.q_stride = io.q_stride;
  a.out = static_cast<uint16_t *>(io.out);
  a.out_stride = io.out_stride;
  a.lse = io.lse;
  a.cu_rows = io.cu_rows;
  a.num_seqs = io.num_seqs;
  a.num_rows = io.num_rows;
  a.num_heads = io.num_heads;
  a.num_kv_heads = c.num_kv_heads;
  a.causal = 1;
  a.scale = io.scale;
  a.status = status;
  const PagedSource src = {io.page_table, io.lengths, io.cu_rows, c.k_codes, c.k_scales, c.v_codes, c.v_scales,
                           c.num_pages, c.page_size, io.max_pages, c.num_kv_heads};
  return launch_simple(a, src, c.head_dim, io.dtype, st);
}

}  // namespace moe
