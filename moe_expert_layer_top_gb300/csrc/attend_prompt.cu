// attend_prompt.cu — causal attention over packed prompts with grouped heads.
#include <cuda_runtime.h>
#include <stdint.h>

#include "attend_simple.cuh"

namespace moe {

namespace {

template <class T>
struct PromptSource {
  const uint16_t *k, *v;
  int64_t k_stride, v_stride;
  const int32_t *cu_keys;
  int num_keys;

  __device__ int keys(int b, int n, int, int32_t *status, int *first) const {
    const Span s = seq_span(cu_keys, b, num_keys, status);
    *first = s.first;
    return s.n;
  }

  template <int D>
  __device__ bool load(bool value, int, int kv, int j, int i, float2 *out, int32_t *) const {
    const uint32_t w = *reinterpret_cast<const uint32_t *>((value ? v + j * v_stride : k + j * k_stride) + kv * D + 2 * i);
    *out = make_float2(T::lo(w), T::hi(w));
    return true;
  }
};

}  // namespace

cudaError_t launch_attend_prompt(const moe_attend_prompt_io_t &io, int32_t *status, int num_sms, cudaStream_t st) {
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
  a.num_kv_heads = io.num_kv_heads;
  a.causal = io.causal;
  a.scale = io.scale;
  a.status = status;
  const auto *k = static_cast<const uint16_t *>(io.k), *v = static_cast<const uint16_t *>(io.v);
  if (io.dtype == MOE_DTYPE_F16) {
    const PromptSource<F16> src = {k, v, io.k_stride, io.v_stride, io.cu_keys, io.num_keys};
    return launch_simple(a, src, io.head_dim, io.dtype, st);
  }
  const PromptSource<Bf16> src = {k, v, io.k_stride, io.v_stride, io.cu_keys, io.num_keys};
  return launch_simple(a, src, io.head_dim, io.dtype, st);
}

}  // namespace moe
