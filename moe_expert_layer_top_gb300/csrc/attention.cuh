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

// In the bounds-checked build (see in_bounds): whether 0 <= i < n. If not, that is reported and the caller skips the
// access. Constantly true in the normal build.
__device__ __forceinline__ bool index_ok(int32_t *status, int64_t i, int64_t n) {
  if constexpr (kBoundsChecked) {
    if (i < 0 || i >= n) {
      out_of_range(status);
      return false;
    }
  }
  return true;
}

// An item that several blocks share, as the first of them leaves it to the kernel that joins them; no parts: there is none.
struct alignas(16) Joint {
  int32_t parts, slot;         // which of the first block's two parts; of the later blocks it is the first
  int32_t row0, kv, r0, rows;  // first row of the sequence, kv head, first (token, head) pair, pairs
  int32_t unused[2];
};

// ------------------------------------------------------------------ 16-bit types

struct Bf16 {
  static constexpr uint32_t kMmaType = 1;  // operand type of the tensor-core instruction descriptor
  static constexpr float kWeightUp = 0.0f;
  static __device__ __forceinline__ float lo(uint32_t v) { return __uint_as_float(v << 16); }
  static __device__ __forceinline__ float hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {  // a in the low half
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
  }
};

struct F16 {
  static constexpr uint32_t kMmaType = 0;
  // Softmax weights are held times 2^kWeightUp (sum and product alike, so it drops out): with the reference up to 2^8
  // behind they reach 2^15, and the smallest step of f16, 2^-24, is 2^-31 of the reference's weight. Without it, of 65,536
  // keys with 2^-26 of the largest weight each (2^-10 in all) nothing is left in the product but all in the sum.
  static constexpr float kWeightUp = 7.0f;
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

// Rows of sequence b by cu; an offset out of range is reported and gives n = -1.
__device__ __forceinline__ Span seq_span(const int32_t *cu, int b, int total, int32_t *status) {
  const int lo = __ldg(cu + b), hi = __ldg(cu + b + 1);
  if (lo < 0 || hi < lo || hi > total) {
    out_of_range(status);
    return {0, -1};
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

// The sequence that tile number `tile` falls into, when sequence b has
// ceil(n_b / rows) tiles of `rows` rows. Called by a whole warp; seq = -1: past the last tile.
// Sequences that overlap (cu decreases, which is reported) may have more tiles than the grid, whose size follows from
// the number of rows: those are not computed. Leaving such sequences out takes the largest end of all before them; any
// form of that here, run or not, made the kernel around it slower (16,384 tokens 1.49 -> 1.53 to 1.58 ms, chunks with
// D = 64 141 -> 149 to 153 us).
struct TileAt {
  int seq, local, tiles;  // sequence, tile within it, its tiles
  Span rows, keys;        // of the sequence
};

// Where a search may begin: `base` tiles lie before sequence b0. A search that goes on where the last one ended makes
// all searches of a block one pass over the sequences (4,096 prompts of 30 tokens: 1.12 ms; 11.4 with searches from the
// start and without taking over the blocks past the last tile).
struct TileCursor {
  int b0 = 0;
  int64_t base = 0;
};

__device__ __forceinline__ TileAt find_tile(TileCursor &from, const int32_t *cu_rows, int num_rows, const int32_t *cu_keys,
                                            int num_keys, int num_seqs, int rows, int64_t tile, int32_t *status) {
  const int lane = threadIdx.x & 31;
  if (tile < from.base) from = TileCursor();
  while (from.b0 < num_seqs) {
    const int b = from.b0 + lane;
    Span r = {0, 0}, k = {0, 0};
    if (b < num_seqs) {
      r = seq_span(cu_rows, b, num_rows, status);
      k = seq_span(cu_keys, b, num_keys, status);
    }
    if (r.n < 0 || k.n < 0) r.n = 0;  // no result
    const int tiles = (r.n + rows - 1) / rows;
    const int64_t end = from.base + warp_inclusive_sum(tiles);
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, tile < end);
    if (hit) {
      const int w = __ffs(hit) - 1;
      TileAt at;
      at.seq = from.b0 + w;
      at.tiles = __shfl_sync(0xFFFFFFFFu, tiles, w);
      at.local = int(tile - (__shfl_sync(0xFFFFFFFFu, end, w) - at.tiles));
      at.rows = {__shfl_sync(0xFFFFFFFFu, r.first, w), __shfl_sync(0xFFFFFFFFu, r.n, w)};
      at.keys = {__shfl_sync(0xFFFFFFFFu, k.first, w), __shfl_sync(0xFFFFFFFFu, k.n, w)};
      return at;
    }
    from.base = __shfl_sync(0xFFFFFFFFu, end, 31);
    from.b0 += 32;
  }
  return {-1, 0, 0, {0, 0}, {0, 0}};
}

}  // namespace moe
