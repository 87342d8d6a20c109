// attend_simple.cuh — one-pass attention on the CUDA cores.
//
// A block takes 16 query rows of one kv head (a "row" here is one token and one
// of the group's heads) and walks the keys in tiles of 32 held in shared memory
// as binary32. Per tile and row: m' = max(m, max s), p = exp(s - m'),
// l = l exp(m - m') + sum p, o = o exp(m - m') + sum p V. Everything is binary32.
#pragma once

#include "attention.cuh"

namespace moe {

struct SimpleArgs {
  const uint16_t *q;
  int64_t q_stride;
  uint16_t *out;
  int64_t out_stride;
  float *lse;
  const int32_t *cu_rows;
  int num_seqs, num_rows, num_heads, num_kv_heads, causal;
  float scale;
  int32_t *status;
};

namespace {

constexpr int kRowTile = 16, kKeyTile = 32, kSimpleThreads = 128;

template <class T, int D, class Source>
__global__ void __launch_bounds__(kSimpleThreads) attend_simple_kernel(const SimpleArgs a, const Source src) {
  __shared__ float qs[kRowTile][D + 1], ks[kKeyTile][D + 1], ps[kRowTile][kKeyTile + 1], fix[kRowTile], sum[kRowTile];
  __shared__ int found[2];
  const int G = a.num_heads / a.num_kv_heads, kv = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  if (tid < 32) {  // the sequence and the tile within it
    int base = 0, fb = -1, ft = 0;
    for (int b0 = 0; b0 < a.num_seqs && fb < 0; b0 += 32) {
      const int b = b0 + lane;
      const int n = b < a.num_seqs ? seq_span(a.cu_rows, b, a.num_rows, a.status).n : 0;
      const int tiles = int((int64_t(n) * G + kRowTile - 1) / kRowTile);
      const int end = warp_inclusive_sum(tiles) + base;
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, int(blockIdx.x) < end);
      if (hit) {
        const int w = __ffs(hit) - 1;
        fb = b0 + w;
        ft = int(blockIdx.x) - (__shfl_sync(0xFFFFFFFFu, end, w) - __shfl_sync(0xFFFFFFFFu, tiles, w));
      }
      base = __shfl_sync(0xFFFFFFFFu, end, 31);
    }
    if (lane == 0) {
      found[0] = fb;
      found[1] = ft;
    }
  }
  __syncthreads();
  const int b = found[0];
  if (b < 0) return;
  const Span rows = seq_span(a.cu_rows, b, a.num_rows, a.status);
  int key0;
  const int m = src.keys(b, rows.n, 0, a.status, &key0);
  const int r0 = found[1] * kRowTile, R = rows.n * G;
  for (int i = tid; i < kRowTile * D; i += kSimpleThreads) {
    const int r = r0 + i / D, d = i % D;
    float x = 0.0f;
    if (r < R) {
      const uint32_t w = a.q[(rows.first + r / G) * a.q_stride + (kv * G + r % G) * D + d];
      x = T::lo(w) * a.scale;
    }
    qs[i / D][d] = x;
  }
  const int row = tid / 8, part = tid % 8;  // 8 threads a row
  const int r = r0 + row;
  int limit = m;
  if (a.causal) limit = min(m, m - rows.n + r / G + 1);
  if (r >= R) limit = 0;
  int last = m;
  if (a.causal) last = min(m, m - rows.n + min(r0 + kRowTile - 1, R - 1) / G + 1);
  float top = -INFINITY, total = 0.0f, o[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i] = 0.0f;
  for (int j0 = 0; j0 < last; j0 += kKeyTile) {
    __syncthreads();
    for (int i = tid; i < kKeyTile * D / 2; i += kSimpleThreads) {
      const int j = i / (D / 2), d = i % (D / 2);
      float2 x = make_float2(0.0f, 0.0f);
      if (j0 + j < m) src.template load<D>(false, b, kv, key0 + j0 + j, d, &x, a.status);
      ks[j][2 * d] = x.x;
      ks[j][2 * d + 1] = x.y;
    }
    __syncthreads();
    float s[kKeyTile / 8];
    float mx = top;
#pragma unroll
    for (int c = 0; c < kKeyTile / 8; ++c) {
      const int j = part + 8 * c;
      float acc = 0.0f;
      for (int d = 0; d < D; ++d) acc = fmaf(qs[row][d], ks[j][d], acc);
      s[c] = j0 + j < limit ? acc : -INFINITY;
      mx = fmaxf(mx, s[c]);
    }
#pragma unroll
    for (int d = 1; d < 8; d *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
    const float ref = mx == -INFINITY ? 0.0f : mx, f = expf(top - ref);
    float add = 0.0f;
#pragma unroll
    for (int c = 0; c < kKeyTile / 8; ++c) {
      const float p = expf(s[c] - ref);
      ps[row][part + 8 * c] = p;
      add += p;
    }
#pragma unroll
    for (int d = 1; d < 8; d *= 2) add += __shfl_xor_sync(0xFFFFFFFFu, add, d);
    total = total * f + add;
    top = mx;
    __syncthreads();
    for (int i = tid; i < kKeyTile * D / 2; i += kSimpleThreads) {
      const int j = i / (D / 2), d = i % (D / 2);
      float2 x = make_float2(0.0f, 0.0f);
      if (j0 + j < m) src.template load<D>(true, b, kv, key0 + j0 + j, d, &x, a.status);
      ks[j][2 * d] = x.x;
      ks[j][2 * d + 1] = x.y;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i] *= f;
    for (int j = 0; j < kKeyTile; ++j) {
      const float p = ps[row][j];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i] = fmaf(p, ks[j][part + 8 * i], o[i]);
    }
  }
  if (r >= R) return;
  const int64_t t = rows.first + r / G;
  const int h = kv * G + r % G;
  const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) a.out[t * a.out_stride + h * D + part + 8 * i] = uint16_t(T::pack(o[i] * inv, 0.0f));
  if (a.lse && part == 0) a.lse[t * a.num_heads + h] = total > 0.0f ? top + logf(total) : -INFINITY;
}

template <class Source>
cudaError_t launch_simple(const SimpleArgs &a, const Source &src, int dim, uint32_t dtype, cudaStream_t st) {
  const int G = a.num_heads / a.num_kv_heads;
  const int64_t tiles = int64_t(a.num_rows) * G / kRowTile + a.num_seqs;
  const dim3 grid(unsigned(tiles), a.num_kv_heads);
  if (dim == 64) {
    if (dtype == MOE_DTYPE_F16)
      attend_simple_kernel<F16, 64><<<grid, kSimpleThreads, 0, st>>>(a, src);
    else
      attend_simple_kernel<Bf16, 64><<<grid, kSimpleThreads, 0, st>>>(a, src);
  } else {
    if (dtype == MOE_DTYPE_F16)
      attend_simple_kernel<F16, 128><<<grid, kSimpleThreads, 0, st>>>(a, src);
    else
      attend_simple_kernel<Bf16, 128><<<grid, kSimpleThreads, 0, st>>>(a, src);
  }
  return cudaGetLastError();
}

}  // namespace

}  // namespace moe
