// commit_drafts.cu — the accepted rows of a tree moved to follow the context, in the caches of all layers.
//
// A move of bytes: token base + path[j] to base + j. With a few accepted rows a
// sequence it is bound by its chain of loads (offsets, path, pages, bytes), so a
// block takes one sequence and several layers at once: the places are looked up once, and all of the
// block's bytes are on their way before the first is written.
//
// A path rises, so path[j] >= j: rows moved in turn never overwrite one that is
// still to move. Rows are moved in batches in the order of the path, and within a batch every
// byte is read before any is written.
//
// Two caches a block and four pieces a thread: one cache a block starts too many blocks (64 sequences x 32 caches, five
// rows: 9.3 us against 7.4), four leave too few of them (the same 7.7; 32 sequences x 2 caches, D = 64: 4.2 against
// 3.6), eight pieces a thread cost registers (10.3). One sequence with two caches takes 3.2 us, a launch and four loads
// that wait for one another. Measured device times, calls in a graph.
#include <cuda_runtime.h>
#include <stdint.h>

#include "attention.cuh"
#include "speculative.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kHold = 4;  // pieces that a thread holds between its reads and its writes

struct Cache {
  uint8_t *part[4];  // K codes, V codes, K scales, V scales
};

struct CommitArgs {
  const int32_t *page_table, *lengths, *cu_rows, *path, *accepted;
  int32_t *new_lengths;
  int max_pages, path_stride, num_caches, num_pages, page_size, num_kv_heads;
  int64_t cached_rows;  // for the checks
  int32_t *status;
  Cache caches[kMaxCaches];
};

// A block for a sequence and every gridDim.y-th of the caches.
template <int D>
__global__ void __launch_bounds__(kThreads) commit_drafts_kernel(const __grid_constant__ CommitArgs a) {
  // of a (row, kv head): 16-byte pieces of codes, then the scales, D / 32 bytes of each
  constexpr int kCodes = D / 32, kPieces = 2 * kCodes + 2;
  constexpr uint32_t kNowhere = 0xFFFFFFFFu;
  __shared__ uint32_t from[MOE_MAX_TREE_ROWS], to[MOE_MAX_TREE_ROWS];  // cached rows of kv head 0
  __shared__ int bad;
  const int b = blockIdx.x, tid = threadIdx.x;
  int32_t *const status = blockIdx.y == 0 ? a.status : nullptr;  // what is out of range is reported once
  const int first = __ldg(a.cu_rows + b), end = __ldg(a.cu_rows + b + 1), length = __ldg(a.lengths + b);
  const int accepted = __ldg(a.accepted + b), n = end - first;
  const int64_t cap = int64_t(a.max_pages) * a.page_size;
  const bool wrong = first < 0 || end < first || length < 0 || length > cap || (n > 0 && length < n) ||
                     (n == 0 ? accepted != 0 : accepted < 0 || accepted >= n) || accepted >= MOE_MAX_TREE_ROWS ||
                     accepted >= a.path_stride;
  if (tid == 0) bad = wrong;
  __syncthreads();
  const int base = length - n;
  if (!wrong && n > 0) {
    for (int j = tid; j <= accepted; j += kThreads) {
      const int32_t *path = a.path + int64_t(b) * a.path_stride + j;
      const int p = __ldg(path), before = j ? __ldg(path - 1) : -1;
      if (j == 0 ? p != 0 : p <= before || p >= n) bad = 1;
      from[j] = to[j] = kNowhere;
      if (p == j || p < 0 || p >= n) continue;
      const int32_t *table = a.page_table + int64_t(b) * a.max_pages;
      const int s = base + p, t = base + j, ps = __ldg(table + s / a.page_size), pt = __ldg(table + t / a.page_size);
      if (ps < 0 || ps >= a.num_pages || pt < 0 || pt >= a.num_pages) {
        out_of_range(status);
        continue;
      }
      from[j] = uint32_t(ps) * a.num_kv_heads * a.page_size + s % a.page_size;
      to[j] = uint32_t(pt) * a.num_kv_heads * a.page_size + t % a.page_size;
    }
  }
  __syncthreads();
  if (bad) {
    if (tid == 0) out_of_range(status);
    if (blockIdx.y == 0 && tid == 0) a.new_lengths[b] = max(length, 0);
    return;
  }
  if (blockIdx.y == 0 && tid == 0) a.new_lengths[b] = n ? base + 1 + accepted : length;
  // A move is a row in one cache; groups of threads take moves in turn, a thread one piece of one kv head of each.
  const int caches = (a.num_caches - int(blockIdx.y) + int(gridDim.y) - 1) / int(gridDim.y), moves = accepted * caches;
  const int pieces = a.num_kv_heads * kPieces, groups = max(1, kThreads / pieces);
  const int group = pieces < kThreads ? tid / pieces : 0;
  for (int part = 0; part < pieces; part += kThreads) {
    const int mine = pieces < kThreads ? tid - group * pieces : part + tid;
    const int kv = mine / kPieces, piece = mine - kv * kPieces;
    const bool works = group < groups && mine < pieces;
    for (int batch = 0; batch < moves; batch += groups * kHold) {
      uint4 held[kHold];
      uint8_t *dst[kHold];
#pragma unroll
      for (int h = 0; h < kHold; ++h) {
        const int m = batch + h * groups + group;
        dst[h] = nullptr;
        if (!works || m >= moves) continue;
        const int j = m / caches, c = m - j * caches;
        if (to[j + 1] == kNowhere) continue;
        const int64_t at = int64_t(from[j + 1]) + kv * a.page_size, into = int64_t(to[j + 1]) + kv * a.page_size;
        if (!index_ok(a.status, at, a.cached_rows) || !index_ok(a.status, into, a.cached_rows)) continue;
        const Cache &cache = a.caches[blockIdx.y + c * gridDim.y];
        if (piece < 2 * kCodes) {
          uint8_t *const codes = cache.part[piece / kCodes] + (piece % kCodes) * 16;
          held[h] = *reinterpret_cast<const uint4 *>(codes + at * (D / 2));
          dst[h] = codes + into * (D / 2);
        } else {
          uint8_t *const scales = cache.part[piece - 2 * kCodes + 2];
          held[h].x = D == 128 ? *reinterpret_cast<const uint32_t *>(scales + at * 4)
                               : *reinterpret_cast<const uint16_t *>(scales + at * 2);
          dst[h] = scales + into * (D / 32);
        }
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < kHold; ++h) {
        if (!dst[h]) continue;
        if (piece < 2 * kCodes)
          *reinterpret_cast<uint4 *>(dst[h]) = held[h];
        else if (D == 128)
          *reinterpret_cast<uint32_t *>(dst[h]) = held[h].x;
        else
          *reinterpret_cast<uint16_t *>(dst[h]) = uint16_t(held[h].x);
      }
      __syncthreads();
    }
  }
}

}  // namespace

cudaError_t launch_commit_drafts(const moe_commit_drafts_io_t &io, const moe_kv_cache_t *caches, int32_t *status,
                                 cudaStream_t st) {
  for (int first = 0; first < io.num_caches; first += kMaxCaches) {
    CommitArgs a = {};
    a.page_table = io.page_table;
    a.lengths = io.lengths;
    a.cu_rows = io.cu_rows;
    a.path = io.path;
    a.accepted = io.accepted;
    a.new_lengths = io.new_lengths;
    a.max_pages = io.max_pages;
    a.path_stride = io.path_stride;
    a.num_caches = io.num_caches - first < kMaxCaches ? io.num_caches - first : kMaxCaches;
    a.status = status;
    const moe_kv_cache_t &c0 = caches[0];
    a.num_pages = c0.num_pages;
    for (int i = 1; i < io.num_caches; ++i) a.num_pages = a.num_pages < caches[i].num_pages ? a.num_pages : caches[i].num_pages;
    a.page_size = c0.page_size;
    a.num_kv_heads = c0.num_kv_heads;
    a.cached_rows = checked_capacity(int64_t(a.num_pages) * c0.page_size * c0.num_kv_heads, io.flags);
    for (int i = 0; i < a.num_caches; ++i) {
      const moe_kv_cache_t &c = caches[first + i];
      a.caches[i] = {{c.k_codes, c.v_codes, c.k_scales, c.v_scales}};
    }
    // two caches a block
    const dim3 grid(unsigned(io.num_seqs), unsigned(a.num_caches + 1) / 2);
    if (c0.head_dim == 64)
      commit_drafts_kernel<64><<<grid, kThreads, 0, st>>>(a);
    else
      commit_drafts_kernel<128><<<grid, kThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
