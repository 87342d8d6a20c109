// attend_paged.cu — attention of the newest rows of each sequence over the paged MXFP4 cache.
//
// Mathematics. For a row: s_j = scale q . K_j, o = sum_j exp(s_j - m) V_j /
// sum_j exp(s_j - m), one pass over the keys with a reference m and the two
// sums (see attend_prompt.cu). K_j = 2^(a - 127) k with E2M1 codes k and one
// scale code a per 32 dimensions; V likewise.
//   Keys: each code becomes an f16 value (exact), times 2^(a - a_max) with
//   a_max the largest of the key's scale codes; the score is multiplied by
//   2^(a_max - 127) after the product. Queries become f16 times a power of two
//   per row. Both are exact but for parts 2^-24 below the key's (row's) largest.
//   Values: codes times 2^(b - b_ref) in f16, with b_ref the largest scale code
//   seen so far in the group of 32 dimensions; like m it moves as the pass goes
//   on, and the accumulators of the group are rescaled when it does.
//   Probabilities: f16, at most 2^8 (the lazy reference of attend_prompt.cu).
// All sums are binary32, on the tensor cores (mma.sync m16n8k16, f16 operands).
//
// Bound. A cached token and kv head is D + D/16 bytes against 4 D flops per row
// and head: HBM for single tokens. Decoding the 4-bit codes is CUDA-core work
// whatever multiplies them (2 D conversions a token), and keeps the
// conversion pipe about 3/4 busy at the HBM rate. The codes go from shared
// memory straight into the registers that the MMA reads: tcgen05 would need K
// and V in 16 bits in shared memory first, and writing and reading those (for
// D = 128: 48 KB per 128 tokens beside 17 KB of codes in and out) would make
// shared memory the bound.
//
// Layout. Keys are the MMA's M (scores transposed: 16 keys x 8 rows), so a step
// of 8 rows wastes nothing on padding. The order of a product's inner dimension
// is free when both operands share it, so a lane's operand registers are decoded
// from whole 16-byte (K) and 8-byte (V) pieces of a cached row:
//   S^T = K Q^T   lane (g, t) = (lane / 4, lane % 4) decodes dimensions
//                 [t D/4, (t + 1) D/4) of keys g and g + 8
//   O^T = V^T P^T lane (g, t) decodes dimensions [g D/8, (g + 1) D/8) of keys
//                 2t, 2t + 1, 2t + 8, 2t + 9, two keys' codes interleaved
// P moves from the first product's result layout to the second's operand
// layout by movmatrix. Rows are (token, head) pairs of one kv head's group.
//
// Schedule. The work is a list of stages of 32 keys: sequence by sequence, kv head
// by kv head, row block by row block. Every block takes an equal, contiguous
// share of the list, so one long sequence spreads over all SMs and a batch of
// ragged ones stays balanced. One warp copies stages into a ring of shared
// memory (plain bulk copies; a page is contiguous per kv head); the other warps
// take stages in turn and meet only where a (sequence, kv head, row block) ends.
// What a block holds of an item it shares with other blocks goes to the
// workspace; a second kernel, launched with programmatic dependent launch, joins
// these in a fixed order. Results do not depend on timing.
#include <cuda_runtime.h>
#include <stdint.h>

#include "attention.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kStageKeys = 32;
constexpr int64_t kWaitNs = 1000000000;  // bound of every wait
constexpr float kLazy = 8.0f;            // the reference moves when the maximum is 2^kLazy beyond it
constexpr float kNone = 1e30f;           // minus the reference of a row that has seen no key
constexpr int kCombineThreads = 256;

struct PagedArgs {
  const uint16_t *q;
  int64_t q_stride;
  uint16_t *out;
  int64_t out_stride;
  float *lse;
  const int32_t *page_table, *lengths, *cu_rows;
  int num_seqs, num_rows, max_pages, num_heads, num_kv_heads, group;
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int num_pages, page_size;
  float scale2;    // |scale| log2 e, at least 2^-100
  uint32_t flip;   // 0x80008000 with a negative scale
  float *parts;    // workspace: two partial results a block
  int32_t *status;
};

// A variant: head size, n-tiles of 8 rows, warps (one loads), blocks per SM, ring stages.
template <int D_, int NT_, int WARPS_, int BLOCKS_, int STAGES_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, W = WARPS_ - 1, BLOCKS = BLOCKS_, STAGES = STAGES_;
  static constexpr int THREADS = WARPS_ * 32;
  static constexpr int ROWS = 8 * NT;           // (token, head) pairs of a row block
  static constexpr int KS = D / 16;             // k-steps of the score product
  static constexpr int MT = D / 16;             // m-tiles of the value product
  static constexpr int CODES = kStageKeys * D / 2, SCALES = kStageKeys * D / 32;
  static constexpr int STAGE_BYTES = 2 * (CODES + SCALES);
  static constexpr int SLAB = D + 4;            // row stride of the joined accumulators (floats)
  static constexpr int PART = ROWS * (D + 2);   // floats of one partial result
  struct Smem {
    alignas(128) uint8_t ring[STAGES][STAGE_BYTES];  // K codes, V codes, K scales, V scales
    float slab[W][8][SLAB];   // accumulators of one n-tile of every warp
    uint2 q[NT][KS][32];      // query operand registers
    float mul[ROWS];          // score units to exponents of two
    int limit[ROWS];          // keys that a row sees
    float ref[W][ROWS], sum[W][ROWS];
    int64_t before[kMaxSeqs / 32 + 1];  // stages of each 32 sequences, then summed
    uint64_t full[STAGES], empty[STAGES];
  };
};

// ------------------------------------------------------------------ the list of stages

struct Seq {
  int b, row0, n, len;  // sequence, first row, rows, keys
  int items, steps;     // kv heads x row blocks; stages of each
};

template <class C>
__device__ __forceinline__ Seq load_seq(const PagedArgs &a, int b, int32_t *status) {
  Seq s = {b, 0, 0, 0, 0, 0};
  if (b >= a.num_seqs) return s;
  const Span r = seq_span(a.cu_rows, b, a.num_rows, status);
  s.row0 = r.first;
  s.n = r.n;
  if (r.n == 0) return s;
  const int cap = a.max_pages * a.page_size;
  int len = __ldg(a.lengths + b);
  if (len < 0 || len > cap) {
    out_of_range(status);
    len = len < 0 ? 0 : cap;
  }
  s.len = len;
  s.items = a.num_kv_heads * ((s.n * a.group + C::ROWS - 1) / C::ROWS);
  s.steps = max(1, (len + kStageKeys - 1) / kStageKeys);  // a sequence without keys still writes its rows
  return s;
}

// Fills before[] with the stages ahead of every 32 sequences; returns all stages. Whole block.
template <class C>
__device__ int64_t count_stages(const PagedArgs &a, int64_t *before, int64_t *total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (a.num_seqs + 31) / 32;
  for (int c = warp; c < chunks; c += blockDim.x / 32) {
    const Seq s = load_seq<C>(a, c * 32 + lane, nullptr);
    int64_t v = int64_t(s.items) * s.steps;
#pragma unroll
    for (int d = 16; d; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if (lane == 0) before[c] = v;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t base = 0;
    for (int c0 = 0; c0 < chunks; c0 += 32) {
      const int64_t v = c0 + lane < chunks ? before[c0 + lane] : 0;
      int64_t s = v;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, s, d);
        if (lane >= d) s += u;
      }
      if (c0 + lane < chunks) before[c0 + lane] = base + s - v;
      base += __shfl_sync(0xFFFFFFFFu, s, 31);
    }
    if (lane == 0) *total = base;
  }
  __syncthreads();
  return *total;
}

// A place in the list: a sequence, and a stage of its items x steps.
struct Place {
  Seq s;
  int item, step;
};

// The place of stage p (0 <= p < all). Whole warp; the same for every lane.
template <class C>
__device__ Place find_stage(const PagedArgs &a, const int64_t *before, int64_t p) {
  const int lane = threadIdx.x & 31;
  const int chunks = (a.num_seqs + 31) / 32;
  int c = 0;
  for (int lo = 0, hi = chunks; lo < hi;) {  // the last chunk with before <= p
    const int mid = (lo + hi) / 2;
    if (before[mid] <= p) {
      c = mid;
      lo = mid + 1;
    } else {
      hi = mid;
    }
  }
  // chunks without stages share their start with the next one: the last is the one with stages
  const Seq mine = load_seq<C>(a, c * 32 + lane, nullptr);
  const int64_t own = int64_t(mine.items) * mine.steps;
  int64_t end = own;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, end, d);
    if (lane >= d) end += u;
  }
  const int64_t rest = p - before[c];
  const unsigned hit = __ballot_sync(0xFFFFFFFFu, rest < end);
  const int w = hit ? __ffs(hit) - 1 : 31;
  const int64_t in = rest - (__shfl_sync(0xFFFFFFFFu, end, w) - __shfl_sync(0xFFFFFFFFu, own, w));
  Place pl;
  pl.s = load_seq<C>(a, c * 32 + w, nullptr);
  pl.item = int(in / pl.s.steps);
  pl.step = int(in - int64_t(pl.item) * pl.s.steps);
  return pl;
}

// A run of stages of one item that a block computes.
struct Segment {
  Seq s;
  int kv, r0;       // kv head, first (token, head) pair
  int first, count; // stages
  bool whole;       // all of the item's stages
};

// Cuts the next segment off a block's share; `left` stages remain after it.
template <class C>
__device__ __forceinline__ Segment next_segment(const PagedArgs &a, Place &p, int64_t &left) {
  Segment g;
  g.s = p.s;
  const int blocks = p.s.items / a.num_kv_heads;
  g.kv = p.item / blocks;
  g.r0 = (p.item - g.kv * blocks) * C::ROWS;
  g.first = p.step;
  const int64_t room = p.s.steps - p.step;
  g.count = int(room < left ? room : left);
  g.whole = g.count == p.s.steps;
  left -= g.count;
  p.step = 0;
  ++p.item;
  if (left > 0) {
    while (p.item >= p.s.items) {  // the next sequence with rows
      p.s = load_seq<C>(a, p.s.b + 1, nullptr);
      p.item = 0;
      if (p.s.b >= a.num_seqs) {
        left = 0;
        break;
      }
    }
  }
  return g;
}

// Blocks that share the list: enough stages for each warp of a block to have one.
template <class C>
__device__ __forceinline__ int64_t active_blocks(int64_t stages, int64_t grid) {
  const int64_t n = (stages + C::W - 1) / C::W;
  return n < grid ? n : grid;
}

// ------------------------------------------------------------------ copies (the last warp)

template <class C>
__device__ void load_warp(const PagedArgs &a, typename C::Smem &sm, Place p, int64_t left) {
  const int lane = threadIdx.x & 31;
  const uint64_t policy = l2_evict_first_policy();
  int64_t g = 0;
  bool ok = true;
  while (ok && left > 0) {
    const Segment seg = next_segment<C>(a, p, left);
    const int32_t *table = a.page_table + int64_t(seg.s.b) * a.max_pages;
    for (int s0 = 0; ok && s0 < seg.count; s0 += 16) {
      // lane 2 i + u looks up granule u (16 keys) of stage s0 + i
      const int key = (seg.first + s0) * kStageKeys + lane * 16;
      int64_t at = -1;  // first cached row of the granule
      if (s0 + lane / 2 < seg.count && key < seg.s.len) {
        const int pi = key / a.page_size, page = __ldg(table + pi);
        if (page < 0 || page >= a.num_pages)
          out_of_range(a.status);
        else
          at = (int64_t(page) * a.num_kv_heads + seg.kv) * a.page_size + (key - pi * a.page_size);
      }
      const int batch = min(16, seg.count - s0);
      for (int i = 0; i < batch; ++i, ++g) {
        const int slot = int(g % C::STAGES);
        ok = mbar_wait(&sm.empty[slot], uint32_t((g / C::STAGES) & 1) ^ 1u, kWaitNs);
        if (!ok) break;
        // lanes 0-7: (part, granule); both granules carry their own address
        const int64_t row = __shfl_sync(0xFFFFFFFFu, at, 2 * i + (lane & 1));
        const unsigned have = __ballot_sync(0xFFFFFFFFu, row >= 0) & 3u;
        if (lane == 0) mbar_arrive_expect_tx(&sm.full[slot], uint32_t(__popc(have)) * (C::STAGE_BYTES / 2));
        __syncwarp();
        if (lane < 8 && row >= 0) {
          const int u = lane & 1, part = lane >> 1;
          const bool scales = part >= 2, value = part & 1;
          const int bytes = scales ? C::SCALES / 2 : C::CODES / 2;
          const int64_t width = scales ? C::D / 32 : C::D / 2;
          const uint8_t *src = (scales ? (value ? a.v_scales : a.k_scales) : (value ? a.v_codes : a.k_codes)) + row * width;
          uint8_t *dst = sm.ring[slot] + (scales ? 2 * C::CODES + (value ? C::SCALES : 0) : (value ? C::CODES : 0)) +
                         u * bytes;
          bulk_g2s(dst, src, uint32_t(bytes), &sm.full[slot], policy);
        }
      }
    }
  }
  if (!ok && a.status && lane == 0) report_error(a.status, MOE_ERR_TIMEOUT);
  // no copy may be in flight when the block exits
  for (int64_t j = 1; j <= C::STAGES && j <= g; ++j)
    mbar_wait(&sm.full[(g - j) % C::STAGES], uint32_t(((g - j) / C::STAGES) & 1), kWaitNs);
}

// ------------------------------------------------------------------ arithmetic

// Codes of byte B of w (low nibble first) as two f16.
template <int B>
__device__ __forceinline__ uint32_t decode2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b%2;\n\t}"
      : "=r"(r)
      : "r"(w), "n"(B));
  return r;
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^-e as binary32, e >= 0 (0 below 2^-126).
__device__ __forceinline__ float pow2_neg(int e) { return __uint_as_float(uint32_t(max(127 - e, 0)) << 23); }

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) { return F16::pack(lo, hi); }

__device__ __forceinline__ int max4(uint32_t w) {  // the largest of four bytes
  uint32_t m;
  asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(w & 0x00FF00FFu), "r"((w >> 8) & 0x00FF00FFu));
  return max(int(m & 0xFFFFu), int(m >> 16));
}

template <class C>
struct State {
  float o[C::MT][C::NT][4];      // [m-tile][n-tile]: dimension pair x row pair
  float ref[C::NT][2];           // minus the reference of rows 2t, 2t + 1 (exponents of two)
  float sum[C::NT][2];           // this lane's keys only
  int vref;                      // scale code that this lane's accumulators are relative to
};

// One stage of 32 keys. key0: its first key; len: keys of the sequence; masked: some row may not see all of it.
template <class C, int D = C::D>
__device__ __forceinline__ void stage(const PagedArgs &a, const typename C::Smem &sm, const uint8_t *ring, State<C> &st,
                                      const uint2 (&qreg)[C::NT <= 2 ? C::NT : 1][C::NT <= 2 ? C::KS : 1], int key0, int len,
                                      bool masked) {
  constexpr int NT = C::NT;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint8_t *kc = ring, *vc = ring + C::CODES, *ks = ring + 2 * C::CODES, *vs = ks + C::SCALES;

  // ---- scores: keys 16 u + g + 8 v
  constexpr int QW = D / 32;  // 32-bit words of a lane's quarter row
  uint32_t kw[2][2][QW], kf[2][2];
  float kmul[2][2];
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int key = 16 * u + 8 * v + g;
      if constexpr (D == 128) {
        const uint4 w = *reinterpret_cast<const uint4 *>(kc + key * (D / 2) + 16 * t);
        kw[u][v][0] = w.x, kw[u][v][1] = w.y, kw[u][v][2] = w.z, kw[u][v][3] = w.w;
      } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(kc + key * (D / 2) + 8 * t);
        kw[u][v][0] = w.x, kw[u][v][1] = w.y;
      }
      int mine, top;
      if constexpr (D == 128) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(ks + key * 4);
        top = max4(w);
        mine = int((w >> (8 * t)) & 0xFFu);
      } else {
        const uint32_t w = *reinterpret_cast<const uint16_t *>(ks + key * 2);
        const int lo = int(w & 0xFFu), hi = int(w >> 8);
        top = max(lo, hi);
        mine = t < 2 ? lo : hi;
      }
      const float f = pow2_neg(top - mine);
      kf[u][v] = f16x2(f, f);
      kmul[u][v] = ue8m0_to_float(uint32_t(top));
    }
  float s[2][NT][4];
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[u][n][c] = 0.0f;
#pragma unroll
  for (int k = 0; k < C::KS; ++k) {
    uint2 b[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (NT <= 2)
        b[n] = qreg[n][k];
      else
        b[n] = sm.q[n][k][lane];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t r[2][2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint32_t w = kw[u][v][k / 2];
        r[v][0] = mul2(k & 1 ? decode2<2>(w) : decode2<0>(w), kf[u][v]);
        r[v][1] = mul2(k & 1 ? decode2<3>(w) : decode2<1>(w), kf[u][v]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(s[u][n], r[0][0], r[1][0], r[0][1], r[1][1], b[n].x, b[n].y);
    }
  }
  // to score units; hidden keys to -inf
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[u][n][c] *= kmul[u][c >> 1];
  if (masked) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int limit = sm.limit[8 * n + 2 * t + e] - key0 - g;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v)
            if (16 * u + 8 * v >= limit) s[u][n][2 * v + e] = -INFINITY;
      }
  }
  // ---- reference
  float top[NT][2], mul[NT][2];
  bool move = false;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float2 m = *reinterpret_cast<const float2 *>(&sm.mul[8 * n + 2 * t]);
    mul[n][0] = m.x, mul[n][1] = m.y;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      top[n][e] = fmaxf(fmaxf(s[0][n][e], s[0][n][2 + e]), fmaxf(s[1][n][e], s[1][n][2 + e])) * mul[n][e];
      move |= top[n][e] + st.ref[n][e] > kLazy;
    }
  }
  if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = top[n][e];
#pragma unroll
        for (int d = 4; d < 32; d *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        const float next = m + st.ref[n][e] > 0.0f ? -m : st.ref[n][e];
        const float f = exp2_approx(next - st.ref[n][e]);
        st.ref[n][e] = next;
        st.sum[n][e] *= f;
#pragma unroll
        for (int i = 0; i < C::MT; ++i) {
          st.o[i][n][e] *= f;
          st.o[i][n][2 + e] *= f;
        }
      }
  }
  // ---- probabilities, in the operand layout of the second product
  uint32_t p[2][NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float x = exp2_approx(fmaf(s[u][n][2 * v], mul[n][0], st.ref[n][0]));
        const float y = exp2_approx(fmaf(s[u][n][2 * v + 1], mul[n][1], st.ref[n][1]));
        st.sum[n][0] += x;
        st.sum[n][1] += y;
        p[u][n][v] = transpose8x8(f16x2(x, y));
      }
  // ---- values: keys 16 u + 8 v + 2 t + e
  constexpr int VW = D / 64;  // 32-bit words of a lane's eighth of a row
  int code[2][2][2], vtop = 0;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = 16 * u + 8 * v + 2 * t + e;
        code[u][v][e] = key0 + key < len ? int(vs[key * (D / 32) + g / (256 / D)]) : 0;  // past the end: anything
        vtop = max(vtop, code[u][v][e]);
      }
  vtop = max(vtop, __shfl_xor_sync(0xFFFFFFFFu, vtop, 1));
  vtop = max(vtop, __shfl_xor_sync(0xFFFFFFFFu, vtop, 2));
  if (__any_sync(0xFFFFFFFFu, vtop > st.vref)) {
    const int next = max(vtop, st.vref);
    const float f = pow2_neg(next - st.vref);
    st.vref = next;
#pragma unroll
    for (int i = 0; i < C::MT; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) st.o[i][n][c] *= f;
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint32_t lo[2][VW], hi[2][VW], vf[2];  // even and odd dimensions of two keys, interleaved
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const uint8_t *row = vc + (16 * u + 8 * v + 2 * t) * (D / 2) + g * (D / 16);
      uint32_t x[VW], y[VW];
      if constexpr (VW == 2) {
        const uint2 xx = *reinterpret_cast<const uint2 *>(row), yy = *reinterpret_cast<const uint2 *>(row + D / 2);
        x[0] = xx.x, x[1] = xx.y, y[0] = yy.x, y[1] = yy.y;
      } else {
        x[0] = *reinterpret_cast<const uint32_t *>(row);
        y[0] = *reinterpret_cast<const uint32_t *>(row + D / 2);
      }
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        lo[v][w] = (x[w] & 0x0F0F0F0Fu) | ((y[w] << 4) & 0xF0F0F0F0u);
        hi[v][w] = ((x[w] >> 4) & 0x0F0F0F0Fu) | (y[w] & 0xF0F0F0F0u);
      }
      vf[v] = f16x2(pow2_neg(st.vref - code[u][v][0]), pow2_neg(st.vref - code[u][v][1]));
    }
#pragma unroll
    for (int i = 0; i < C::MT; ++i) {
      uint32_t r[2][2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint32_t l = lo[v][i / 4], h = hi[v][i / 4];
        r[v][0] = mul2((i & 3) == 0   ? decode2<0>(l)
                       : (i & 3) == 1 ? decode2<1>(l)
                       : (i & 3) == 2 ? decode2<2>(l)
                                      : decode2<3>(l),
                       vf[v]);
        r[v][1] = mul2((i & 3) == 0   ? decode2<0>(h)
                       : (i & 3) == 1 ? decode2<1>(h)
                       : (i & 3) == 2 ? decode2<2>(h)
                                      : decode2<3>(h),
                       vf[v]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(st.o[i][n], r[0][0], r[0][1], r[1][0], r[1][1], p[u][n][0], p[u][n][1]);
    }
  }
}

// Writes row (token, head) pair r of an item: 4 dimensions from d on, or (d < 0) its log sum exp.
template <class T>
__device__ __forceinline__ void store4(const PagedArgs &a, const Seq &s, int kv, int r, int dims, int d, float4 v) {
  const int tok = r / a.group, h = kv * a.group + r - tok * a.group;
  uint16_t *dst = a.out + int64_t(s.row0 + tok) * a.out_stride + int64_t(h) * dims + d;
  *reinterpret_cast<uint2 *>(dst) = make_uint2(T::pack(v.x, v.y), T::pack(v.z, v.w));
}

__device__ __forceinline__ void store_lse(const PagedArgs &a, const Seq &s, int kv, int r, float ref, float sum) {
  if (!a.lse) return;
  const int tok = r / a.group, h = kv * a.group + r - tok * a.group;
  a.lse[int64_t(s.row0 + tok) * a.num_heads + h] = sum > 0.0f ? (log2f(sum) + ref) * 0.6931471805599453f : -INFINITY;
}

// ------------------------------------------------------------------ main kernel

constexpr int kBarWarps = 1;

__device__ __forceinline__ int bar_and_warps(int threads, int v) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(v), "n"(kBarWarps), "r"(threads)
      : "memory");
  return r;
}

// The queries of a row block, as operand registers, with their limits and multipliers.
template <class T, class C>
__device__ void load_queries(const PagedArgs &a, typename C::Smem &sm, const Segment &seg, int warp) {
  constexpr int D = C::D, E = D / 4;  // a lane's dimensions
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  for (int n = warp; n < C::NT; n += C::W) {
    const int r = seg.r0 + 8 * n + g;
    const bool real = r < seg.s.n * a.group;
    const int tok = r / a.group, h = seg.kv * a.group + r - tok * a.group;
    uint4 raw[E / 8];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < E / 8; ++i) {
      raw[i] = make_uint4(0, 0, 0, 0);
      if (real)
        raw[i] = __ldg(reinterpret_cast<const uint4 *>(a.q + int64_t(seg.s.row0 + tok) * a.q_stride + int64_t(h) * D + E * t) + i);
      raw[i].x ^= a.flip, raw[i].y ^= a.flip, raw[i].z ^= a.flip, raw[i].w ^= a.flip;
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) amax = fmaxf(amax, fmaxf(fabsf(T::lo(w[c])), fabsf(T::hi(w[c]))));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    // times 2^(14 - e): the largest lies in [2^14, 2^15), parts down to 2^-28 of it keep all their bits
    const int e = min(max(int(__float_as_uint(amax) >> 23) - 127, -100), 126);
    const float up = __uint_as_float(uint32_t(127 + 14 - e > 254 ? 254 : 127 + 14 - e) << 23);
#pragma unroll
    for (int i = 0; i < E / 8; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int c = 0; c < 2; ++c)
        sm.q[n][2 * i + c][lane] = make_uint2(f16x2(T::lo(w[2 * c]) * up, T::hi(w[2 * c]) * up),
                                              f16x2(T::lo(w[2 * c + 1]) * up, T::hi(w[2 * c + 1]) * up));
    }
    if (t == 0) {
      sm.mul[8 * n + g] = a.scale2 / up;
      sm.limit[8 * n + g] = real ? min(seg.s.len, max(0, seg.s.len - seg.s.n + tok + 1)) : 0;
    }
  }
}

template <class T, class C>
__device__ void compute_warps(const PagedArgs &a, typename C::Smem &sm, Place p, int64_t left, int warp) {
  constexpr int D = C::D, NT = C::NT, kSync = C::W * 32;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int tid = warp * 32 + lane;
  int64_t base = 0;  // stages of the block before this segment
  bool first = true;
  int ok = 1;
  while (left > 0) {
    const Segment seg = next_segment<C>(a, p, left);
    load_queries<T, C>(a, sm, seg, warp);
    if (!bar_and_warps(kSync, ok)) break;
    State<C> st;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        st.ref[n][e] = kNone;
        st.sum[n][e] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < C::MT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) st.o[i][n][c] = 0.0f;
    }
    st.vref = 0;
    uint2 qreg[NT <= 2 ? NT : 1][NT <= 2 ? C::KS : 1];
    if constexpr (NT <= 2) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < C::KS; ++k) qreg[n][k] = sm.q[n][k][lane];
    }
    const int clear = max(0, seg.s.len - seg.s.n + 1 + seg.r0 / a.group);  // keys that every row sees
    // stage g of the block belongs to warp g mod W
    int i = int((warp - base % C::W + C::W) % C::W);
    for (; ok && i < seg.count; i += C::W) {
      const int64_t gs = base + i;
      const int slot = int(gs % C::STAGES);
      ok = mbar_wait(&sm.full[slot], uint32_t((gs / C::STAGES) & 1), kWaitNs) ? 1 : 0;
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) {
        if (a.status && lane == 0) report_error(a.status, MOE_ERR_TIMEOUT);
        break;
      }
      const int key0 = (seg.first + i) * kStageKeys;
      stage<C>(a, sm, sm.ring[slot], st, qreg, key0, seg.s.len, key0 + kStageKeys > min(clear, seg.s.len));
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[slot]);
    }
    base += seg.count;
    // ---- join the warps: reference and sum of each row, then the accumulators n-tile by n-tile
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = st.sum[n][e];
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
        if (g == 0) {
          sm.ref[warp][8 * n + 2 * t + e] = -st.ref[n][e];
          sm.sum[warp][8 * n + 2 * t + e] = l;
        }
      }
    if (!bar_and_warps(kSync, ok)) break;
    const float unit = ue8m0_to_float(uint32_t(st.vref));
    const int rows = seg.s.n * a.group - seg.r0;  // real rows of the block
    float *part = a.parts + (int64_t(blockIdx.x) * 2 + (first ? 0 : 1)) * C::PART;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = sm.ref[0][8 * n + 2 * t + e];
        for (int w = 1; w < C::W; ++w) m = fmaxf(m, sm.ref[w][8 * n + 2 * t + e]);
        f[e] = exp2_approx(-st.ref[n][e] - m);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < C::MT; i += 2)  // dimensions g D/8 + 2 i .. + 3
          *reinterpret_cast<float4 *>(&sm.slab[warp][2 * t + e][g * (D / 8) + 2 * i]) =
              make_float4(st.o[i][n][e] * f[e] * unit, st.o[i][n][2 + e] * f[e] * unit, st.o[i + 1][n][e] * f[e] * unit,
                          st.o[i + 1][n][2 + e] * f[e] * unit);
      bar_and_warps(kSync, 1);
      for (int idx = tid; idx < 8 * (D / 4); idx += kSync) {
        const int row = idx / (D / 4), d = 4 * (idx % (D / 4)), rr = 8 * n + row;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float m = sm.ref[0][rr], l = 0.0f;
        for (int w = 1; w < C::W; ++w) m = fmaxf(m, sm.ref[w][rr]);
#pragma unroll
        for (int w = 0; w < C::W; ++w) {
          const float4 x = *reinterpret_cast<const float4 *>(&sm.slab[w][row][d]);
          v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
          l += sm.sum[w][rr] * exp2_approx(sm.ref[w][rr] - m);
        }
        if (seg.whole) {
          if (rr < rows) {
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
            const bool any = l != 0.0f;
            store4<T>(a, seg.s, seg.kv, seg.r0 + rr, D, d,
                      any ? make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv) : make_float4(0, 0, 0, 0));
            if (d == 0) store_lse(a, seg.s, seg.kv, seg.r0 + rr, m, l);
          }
        } else {
          *reinterpret_cast<float4 *>(part + rr * D + d) = v;
          if (d == 0) {
            part[C::ROWS * D + rr] = m;
            part[C::ROWS * D + C::ROWS + rr] = l;
          }
        }
      }
      bar_and_warps(kSync, 1);
    }
    first = false;
  }
}

template <class T, class C>
__global__ void __launch_bounds__(C::THREADS, C::BLOCKS) attend_paged_kernel(const PagedArgs a) {
  extern __shared__ unsigned char paged_smem_raw[];
  typename C::Smem &sm =
      *reinterpret_cast<typename C::Smem *>((reinterpret_cast<uintptr_t>(paged_smem_raw) + 127) & ~uintptr_t(127));
  __shared__ int64_t total;
  const int warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    fence_mbar_init();
  }
  if (blockIdx.x == 0)  // what is out of range is reported once
    for (int b = threadIdx.x; b < a.num_seqs; b += C::THREADS) load_seq<C>(a, b, a.status);
  const int64_t all = count_stages<C>(a, sm.before, &total);
  const int64_t blocks = active_blocks<C>(all, gridDim.x);
  if (int64_t(blockIdx.x) >= blocks) return;
  const int64_t begin = int64_t(blockIdx.x) * all / blocks, end = (int64_t(blockIdx.x) + 1) * all / blocks;
  const Place p = find_stage<C>(a, sm.before, begin);
  if (warp == C::W)
    load_warp<C>(a, sm, p, end - begin);
  else
    compute_warps<T, C>(a, sm, p, end - begin, warp);
}

// ------------------------------------------------------------------ joining the blocks
// Block c joins the item that block c of the main kernel began last, if that
// item went on into later blocks.

template <class T, class C>
__global__ void __launch_bounds__(kCombineThreads) combine_paged_kernel(const PagedArgs a) {
  __shared__ int64_t before[kMaxSeqs / 32 + 1], total;
  const int64_t all = count_stages<C>(a, before, &total);
  const int64_t blocks = active_blocks<C>(all, gridDim.x);
  const int64_t c = blockIdx.x;
  Place p;
  int64_t begin = 0, end = 0, item0 = 0, item1 = 0;  // the block's stages, the item's
  if (c + 1 < blocks) {
    begin = c * all / blocks;
    end = (c + 1) * all / blocks;
    p = find_stage<C>(a, before, end - 1);
    item0 = end - 1 - p.step;
    item1 = item0 + p.s.steps;
  }
  pdl_wait_primary();  // every block: this kernel must not end before the main one
  if (item0 < begin || item1 <= end) return;  // begun by an earlier block, or complete
  // the blocks that hold parts of it: c, whose part is its last segment, and those after it, whose first it is
  int64_t last = c + 1;
  while ((last + 1) * all / blocks < item1) ++last;
  const float *part0 = a.parts + (c * 2 + (item0 == begin ? 0 : 1)) * C::PART;
  const auto part = [&](int64_t b) { return b == c ? part0 : a.parts + b * 2 * C::PART; };
  const int per = p.s.items / a.num_kv_heads, kv = p.item / per, r0 = (p.item - kv * per) * C::ROWS;
  const int rows = min(C::ROWS, p.s.n * a.group - r0);
  constexpr int D = C::D;
  for (int idx = threadIdx.x; idx < rows * (D / 4); idx += kCombineThreads) {
    const int row = idx / (D / 4), d = 4 * (idx % (D / 4));
    float m = -kNone;
    for (int64_t b = c; b <= last; ++b) m = fmaxf(m, part(b)[C::ROWS * D + row]);
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
    for (int64_t b = c; b <= last; ++b) {
      const float *x = part(b);
      const float f = exp2_approx(x[C::ROWS * D + row] - m);
      const float4 o = *reinterpret_cast<const float4 *>(x + row * D + d);
      v.x = fmaf(o.x, f, v.x), v.y = fmaf(o.y, f, v.y), v.z = fmaf(o.z, f, v.z), v.w = fmaf(o.w, f, v.w);
      l = fmaf(x[C::ROWS * D + C::ROWS + row], f, l);
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    store4<T>(a, p.s, kv, r0 + row, D, d,
              l != 0.0f ? make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv) : make_float4(0, 0, 0, 0));
    if (d == 0) store_lse(a, p.s, kv, r0 + row, m, l);
  }
}

// ------------------------------------------------------------------ host

template <class C>
constexpr size_t smem_bytes() {
  static_assert(C::BLOCKS * (sizeof(typename C::Smem) + 128 + 2048) <= 227 * 1024, "shared memory budget");
  return sizeof(typename C::Smem) + 128;
}

template <class T, class C>
cudaError_t launch(const PagedArgs &a, int num_sms, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(attend_paged_kernel<T, C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       int(smem_bytes<C>()));
  if (e != cudaSuccess) return e;
  const unsigned grid = unsigned(num_sms * C::BLOCKS);
  attend_paged_kernel<T, C><<<grid, C::THREADS, smem_bytes<C>(), st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kCombineThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_paged_kernel<T, C>, a);
}

// The variants: as few row blocks of at most 32 rows as the usual rows of a
// sequence need, and as few n-tiles a block as those leave.
template <int D, class F>
auto pick(int rows, F f) {
  const int blocks = (rows + 31) / 32, tiles = ((rows + blocks - 1) / blocks + 7) / 8;
  switch (tiles) {
    case 1: return f(Cfg<D, 1, 8, 2, D == 128 ? 16 : 32>());
    case 2: return f(Cfg<D, 2, 8, 2, D == 128 ? 16 : 32>());
    case 3: return f(Cfg<D, 3, 12, 1, 32>());
    default: return f(Cfg<D, 4, 8, 1, 32>());
  }
}

int usual_rows(const moe_attend_paged_io_t &io, const moe_kv_cache_t &c) {
  const int64_t rows = int64_t(io.max_rows < io.num_rows ? io.max_rows : io.num_rows) * (io.num_heads / c.num_kv_heads);
  return int(rows < 1 ? 1 : rows);
}

}  // namespace

int64_t attend_paged_workspace(const moe_attend_paged_io_t &io, const moe_kv_cache_t &c, int num_sms) {
  const auto bytes = [&](auto cfg) {
    using C = decltype(cfg);
    return int64_t(num_sms) * C::BLOCKS * 2 * C::PART * 4;
  };
  const int rows = usual_rows(io, c);
  return c.head_dim == 64 ? pick<64>(rows, bytes) : pick<128>(rows, bytes);
}

cudaError_t launch_attend_paged(const moe_attend_paged_io_t &io, const moe_kv_cache_t &c, void *workspace,
                                int32_t *status, int num_sms, cudaStream_t st) {
  PagedArgs a = {};
  a.q = static_cast<const uint16_t *>(io.q);
  a.q_stride = io.q_stride;
  a.out = static_cast<uint16_t *>(io.out);
  a.out_stride = io.out_stride;
  a.lse = io.lse;
  a.page_table = io.page_table;
  a.lengths = io.lengths;
  a.cu_rows = io.cu_rows;
  a.num_seqs = io.num_seqs;
  a.num_rows = io.num_rows;
  a.max_pages = io.max_pages;
  a.num_heads = io.num_heads;
  a.num_kv_heads = c.num_kv_heads;
  a.group = io.num_heads / c.num_kv_heads;
  a.k_codes = c.k_codes;
  a.k_scales = c.k_scales;
  a.v_codes = c.v_codes;
  a.v_scales = c.v_scales;
  a.num_pages = c.num_pages;
  a.page_size = c.page_size;
  a.scale2 = fmaxf(fabsf(io.scale) * 1.4426950408889634f, 0x1p-100f);
  a.flip = io.scale < 0.0f ? 0x80008000u : 0u;
  a.parts = static_cast<float *>(workspace);
  a.status = status;
  const bool h = io.dtype == MOE_DTYPE_F16;
  const auto go = [&](auto cfg) {
    using C = decltype(cfg);
    return h ? launch<F16, C>(a, num_sms, st) : launch<Bf16, C>(a, num_sms, st);
  };
  const int rows = usual_rows(io, c);
  return c.head_dim == 64 ? pick<64>(rows, go) : pick<128>(rows, go);
}

}  // namespace moe
