// attention.cuh — device-side building blocks shared by the attention kernels:
// 16-bit element types, checked sequence bounds, and the search for the
// sequence that a tile belongs to.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "attention.h"
#include "device.cuh"

namespace moe {

// An index from device memory is out of range: the first such error stays in *status.
__device__ __forceinline__ void out_of_range(int32_t *status) {
  if (status) report_error(status, MOE_ERR_DEVICE_BOUNDS);
}

// ------------------------------------------------------------------ 16-bit types

struct Bf16 {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float lo(uint32_t v) { return __uint_as_float(v << 16); }
  static __device__ __forceinline__ float hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {  // a in the low half
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
  }
};

struct F16 {
  using T = __half;
  static __device__ __forceinline__ float lo(uint32_t v) {
    return __low2float(*reinterpret_cast<const __half2 *>(&v));
  }
  static __device__ __forceinline__ float hi(uint32_t v) {
    return __high2float(*reinterpret_cast<const __half2 *>(&v));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
  }
};

// ------------------------------------------------------------------ sequences

// Entries [first, first + n) of a packed array of `total` rows.
struct Span {
  int first, n;
};

// Rows of sequence b by cu; an offset out of range empties the sequence and is reported.
__device__ __forceinline__ Span seq_span(const int32_t *cu, int b, int total, int32_t *status) {
  const int lo = __ldg(cu + b), hi = __ldg(cu + b + 1);
  if (lo < 0 || hi < lo || hi > total) {
    out_of_range(status);
    return {0, 0};
  }
  return {lo, hi - lo};
}

__device__ __forceinline__ int warp_inclusive_sum(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += u;
  }
  return v;
}

}  // namespace moe
