// attend_paged.cu — attention of the newest rows of each sequence over the paged MXFP4 cache.
//
// Mathematics. For a row: s_j = scale q . K_j, o = sum_j exp(s_j - m) V_j /
// sum_j exp(s_j - m), one pass over the keys with a reference m and the two
// sums (see attend_prompt.cu). K_j = 2^(a - 127) k with E2M1 codes k and one
// scale code a per 32 dimensions; V likewise.
//   Keys: codes as f16 (exact); the partial score of each group of 32
//   dimensions is multiplied by its 2^(a - 127) in binary32. Queries become f16
//   times a power of two per row: exact but for parts 2^-28 below the row's
//   largest and smaller.
//   Values: codes times 2^(b - b_ref) in f16, with b_ref the largest scale code
//   that the warp has seen; like m it moves as the pass goes on, and the
//   accumulators are rescaled when it does. Exact down to 2^-23 of the largest.
//   Probabilities: f16, at most 2^15 (the lazy reference of attend_prompt.cu, less
//   2^7 so that small ones keep their bits: exact to 2^-32 of the row's largest).
// All sums are binary32, on the tensor cores (mma.sync m16n8k16, f16 operands).
//
// Bound. A cached token and kv head is D + D/16 bytes against 4 D flops per row
// and head: HBM for single tokens. Decoding the 4-bit codes is CUDA-core work
// whatever multiplies them (2 D conversions a token, at half rate). 128 single
// tokens of 4,000 to 16,000 (D = 128, 32 + 8 heads) take 243 us, 4.83 TB/s or 71 %
// of the copy bandwidth: issue slots are 63 % busy, the ALU pipe 56 %. With 24
// rows of a kv head (steps of six rows, 64 sequences of 1,024 to 5,120, 82 us) it
// is neither: two warps a scheduler (the accumulators take the registers) wait on
// fixed latencies; tensor pipe 36 %, issue 44 %, HBM 30 %. One token over 4,096:
// 10.7 us, launches and the chain lookup - load - join.
// The codes go from shared memory straight into the registers that the MMA
// reads. tcgen05 would need V in 16 bits in shared memory first, since V's scale
// groups do not lie along the product's inner dimension (the keys). K's do: its
// codes and scales could be the operands of a block-scaled MMA as they are, with the
// queries split into 8-bit terms. That has not been built.
//
// Layout. Keys are the MMA's M (scores transposed: 16 keys x 8 rows), so a step
// of 8 rows wastes nothing on padding. The order of a product's inner dimension
// is free when both operands share it, so a lane's operand registers are decoded
// from whole 4-byte (K) and 8-byte (V) pieces of a cached row:
//   S^T = K Q^T   lane (g, t) = (lane / 4, lane % 4) decodes dimensions
//                 32 j + 8 t .. + 7 of keys g and g + 8, for each group j
//   O^T = V^T P^T lane (g, t) decodes dimensions [g D/8, (g + 1) D/8) of keys
//                 2t, 2t + 1, 2t + 8, 2t + 9, two keys' codes interleaved
// P moves from the first product's result layout to the second's operand
// layout by movmatrix. Rows are (token, head) pairs of one kv head's group.
//
// Schedule. The work is a list of items (sequence, kv head, row block), each of
// kOver units for its queries and its join and one for each stage of 32 keys.
// Every block takes an equal, contiguous share of the units, so one long sequence
// spreads over all SMs and a batch of ragged ones stays balanced. Within its share
// of an item a block's warps take the stages in turn. Each copies its own ahead of
// time into a ring of its own (cp.async), so they meet only where an item ends:
// there the accumulators of all warps are joined through shared memory, which the
// drained rings leave free. What a block holds of an item that it shares with
// other blocks goes to the workspace; a second kernel, launched with programmatic
// dependent launch, joins these in a fixed order. Results do not depend on timing.
// Tried and slower: one copying warp with bulk copies (128 tokens 479 us against
// 244), the next granule's scores between this one's exponentials and products
// (six rows 94 us against 82), whose registers cost more than the wait.
#include <cuda_runtime.h>
#include <stdint.h>

#include "attention.cuh"

namespace moe {

namespace {

constexpr int kStageKeys = 32;
// What an item costs beside its stages, in units of one stage. 24 ragged sequences with D = 64: 25.5 us with 16, 41 with
// 1; 64 steps of six rows 82 against 91. 10 and 24 are no better than 16.
constexpr int kOver = 16;
constexpr float kLazy = 8.0f;            // the reference moves when the maximum is 2^kLazy beyond it
constexpr float kNone = 3e38f;           // minus the reference of a row that has seen no key: below any score
constexpr int kCombineThreads = 256;
constexpr int kMaxBlocks = 1024;         // blocks of the main kernel, at most

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
  int64_t part_cap, cached_rows;  // partial results that it holds, rows of the cache: for the checks
  int32_t *status;
};

// A variant: head size, n-tiles of 8 rows, warps, blocks per SM, stages of each
// warp's ring, granules of 16 keys computed at a time.
template <int D_, int NT_, int W_, int BLOCKS_, int DEPTH_, int U_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, W = W_, BLOCKS = BLOCKS_, DEPTH = DEPTH_, U = U_;
  static constexpr int THREADS = W * 32;
  static constexpr int ROWS = 8 * NT;           // (token, head) pairs of a row block
  static constexpr int KS = D / 16;             // k-steps of the score product
  static constexpr int MT = D / 16;             // m-tiles of the value product
  static constexpr bool QREG = NT == 1;         // query operands stay in registers
  static constexpr int CODES = kStageKeys * D / 2, SCALES = kStageKeys * D / 32;
  static constexpr int STAGE_BYTES = 2 * (CODES + SCALES);
  static constexpr int SLAB = D + 4;            // row stride of the joined accumulators (floats)
  static constexpr int PART = ROWS * (D + 2);   // floats of one partial result
  struct Smem {
    union {
      alignas(128) uint8_t ring[W][DEPTH][STAGE_BYTES];  // K codes, V codes, K scales, V scales
      float slab[W][8][SLAB];  // accumulators of one n-tile of every warp, once the rings are drained
    };
    uint2 q[NT][KS][32];       // query operand registers
    float mul[ROWS];           // score units to exponents of two
    int limit[ROWS];           // keys that a row sees
    float ref[W][ROWS], sum[W][ROWS];
    int64_t before[kMaxSeqs / 32 + 1];  // units of each 32 sequences, then summed
  };
};

// ------------------------------------------------------------------ the list of work
// In units: an item (sequence, kv head, row block) is kOver units for its
// queries and its join, then one unit for each of its stages of 32 keys.

struct Seq {
  int b, row0, n, len;  // sequence, first row, rows, keys
  int items, steps;     // kv heads x row blocks; stages of each

  __device__ __forceinline__ int64_t units() const { return int64_t(items) * (steps + kOver); }
};

template <class C>
__device__ __forceinline__ Seq load_seq(const PagedArgs &a, int b, int32_t *status) {
  Seq s = {b, 0, 0, 0, 0, 0};
  if (b >= a.num_seqs) return s;
  const Span r = seq_span(a.cu_rows, b, a.num_rows, status);
  if (r.n <= 0) return s;
  s.row0 = r.first;
  s.n = r.n;
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

// A place in the list: a unit of an item of a sequence.
struct Place {
  Seq s;
  int item, unit;
};

// a / b for 0 <= a, 0 < b; in 32 bits where that is enough (a 64-bit division is about 100 instructions).
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return uint64_t(a | b) >> 32 ? a / b : int64_t(uint32_t(a) / uint32_t(b));
}

__device__ __forceinline__ int64_t warp_sums(int64_t v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += u;
  }
  return v;
}

// The list of all work, as a warp sees it: the 32 sequences of a chunk, one a
// lane, and (more than 32 sequences) the units ahead of each chunk in shared memory.
template <class C>
struct List {
  const PagedArgs &a;
  int64_t *before;
  int64_t all;    // units of all sequences
  Seq mine;       // sequence of this lane in chunk 0 (up to 32 sequences)
  int64_t end;    // units up to and with it

  // Whole block.
  __device__ List(const PagedArgs &args, int64_t *shared, int64_t *total) : a(args), before(shared) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunks = (a.num_seqs + 31) / 32;
    if (chunks <= 1) {  // every warp for itself: one round of loads, no barrier
      mine = load_seq<C>(a, lane, nullptr);
      end = warp_sums(mine.units());
      all = __shfl_sync(0xFFFFFFFFu, end, 31);
      return;
    }
    for (int c = warp; c < chunks; c += blockDim.x / 32) {
      const int64_t v = warp_sums(load_seq<C>(a, c * 32 + lane, nullptr).units());
      if (lane == 31 && index_ok(a.status, c, kMaxSeqs / 32 + 1)) before[c] = v;
    }
    __syncthreads();
    if (warp == 0) {
      int64_t base = 0;
      for (int c0 = 0; c0 < chunks; c0 += 32) {
        const int64_t v = c0 + lane < chunks ? before[c0 + lane] : 0, s = warp_sums(v);
        if (c0 + lane < chunks) before[c0 + lane] = base + s - v;
        base += __shfl_sync(0xFFFFFFFFu, s, 31);
      }
      if (lane == 0) *total = base;
    }
    __syncthreads();
    all = *total;
  }

  // The place of unit p (0 <= p < all). Whole warp; the same for every lane.
  __device__ Place find(int64_t p) const {
    const int lane = threadIdx.x & 31;
    const int chunks = (a.num_seqs + 31) / 32;
    int c = 0;
    Seq s = mine;
    int64_t stop = end, rest = p;
    if (chunks > 1) {
      for (int lo = 0, hi = chunks; lo < hi;) {  // the last chunk with before <= p: earlier ones with that start are empty
        const int mid = (lo + hi) / 2;
        if (before[mid] <= p) {
          c = mid;
          lo = mid + 1;
        } else {
          hi = mid;
        }
      }
      s = load_seq<C>(a, c * 32 + lane, nullptr);
      stop = warp_sums(s.units());
      rest = p - before[c];
    }
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, rest < stop);
    const int w = hit ? __ffs(hit) - 1 : 31;
    const int64_t in = rest - (__shfl_sync(0xFFFFFFFFu, stop, w) - __shfl_sync(0xFFFFFFFFu, s.units(), w));
    Place pl;
    pl.s.b = c * 32 + w;
    pl.s.row0 = __shfl_sync(0xFFFFFFFFu, s.row0, w);
    pl.s.n = __shfl_sync(0xFFFFFFFFu, s.n, w);
    pl.s.len = __shfl_sync(0xFFFFFFFFu, s.len, w);
    pl.s.items = __shfl_sync(0xFFFFFFFFu, s.items, w);
    pl.s.steps = __shfl_sync(0xFFFFFFFFu, s.steps, w);
    pl.item = int(divide(in, pl.s.steps + kOver));
    pl.unit = int(in - int64_t(pl.item) * (pl.s.steps + kOver));
    return pl;
  }
};

// A run of stages of one item that a block computes (count may be 0).
struct Segment {
  Seq s;
  int kv, r0;       // kv head, first (token, head) pair
  int first, count; // stages
};

// Cuts the next segment off a block's share; `left` units remain after it.
template <class C>
__device__ __forceinline__ Segment next_segment(const PagedArgs &a, Place &p, int64_t &left) {
  Segment g;
  g.s = p.s;
  const int blocks = p.s.items / a.num_kv_heads;
  g.kv = p.item / blocks;
  g.r0 = (p.item - g.kv * blocks) * C::ROWS;
  const int64_t room = p.s.steps + kOver - p.unit;
  const int take = int(room < left ? room : left);
  g.first = max(0, p.unit - kOver);
  g.count = max(0, p.unit + take - kOver) - g.first;
  left -= take;
  p.unit = 0;
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

// The blocks' shares of the list: about a stage for each warp at least, and equal to one unit.
struct Shares {
  int64_t blocks, each, more;  // the first `more` blocks have each + 1 units

  __device__ __forceinline__ int64_t begin(int64_t b) const { return b * each + (b < more ? b : more); }
};

template <class C>
__device__ __forceinline__ Shares make_shares(int64_t units, int64_t grid) {
  Shares s;
  s.blocks = units < grid * C::W ? (units + C::W - 1) / C::W : grid;
  s.each = s.blocks ? divide(units, s.blocks) : 0;
  s.more = units - s.each * s.blocks;
  return s;
}

// ------------------------------------------------------------------ copies
// Every warp copies its own stages (stage i of a segment is warp i mod W's)
// with cp.async, DEPTH - 1 of them ahead of the one it computes.

__device__ __forceinline__ void copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Codes lie in shared memory as [key][D/2 bytes], with the 16-byte groups of a
// key exchanged by key: a lane reads 4 bytes of a group (K) or 8 of a key (V),
// and the keys that a warp reads at once then fall into different banks.
template <int D>
__device__ __forceinline__ int swizzle(int key) {
  return D == 128 ? (key >> 1) & 3 : (key >> 2) & 1;
}

template <class C>
struct Copier {
  const int32_t *table;
  uint32_t at;    // lane 2 j + u: first cached row of granule u (16 keys) of the j-th stage of the batch
  int batch;      // stages copied of the batch (16 are looked up at a time)
  static constexpr uint32_t kNoRow = 0xFFFFFFFFu;

  __device__ __forceinline__ void start(const PagedArgs &a, const Segment &seg) {
    table = a.page_table + int64_t(seg.s.b) * a.max_pages;
    batch = 16;
  }

  // Copies stage i of the segment; the next call's is stage i + W.
  __device__ __forceinline__ void copy(const PagedArgs &a, const Segment &seg, int i, uint8_t *slot) {
    const int lane = threadIdx.x & 31;
    if (i < seg.count) {
      if (batch == 16) {
        batch = 0;
        const int step = i + (lane >> 1) * C::W, key = (seg.first + step) * kStageKeys + (lane & 1) * 16;
        at = kNoRow;
        if (step < seg.count && key < seg.s.len) {
          const int pi = key / a.page_size;
          const int page = index_ok(a.status, pi, a.max_pages) ? __ldg(table + pi) : 0;
          if (page < 0 || page >= a.num_pages)
            out_of_range(a.status);
          else
            at = (uint32_t(page) * a.num_kv_heads + seg.kv) * a.page_size + (key - pi * a.page_size);
          if (at != kNoRow && !index_ok(a.status, int64_t(at) + 15, a.cached_rows)) at = kNoRow;
        }
      }
      constexpr int kPer = C::CODES / 512;  // copies of 16 bytes a lane, of the codes of K (and of V)
      // 16 bytes are a key's group of 32 codes; see swizzle() for its place
      constexpr int kGroups = C::D / 32;
      const int to = (lane / kGroups) * (C::D / 2) + (((lane % kGroups) ^ swizzle<C::D>(lane / kGroups)) << 4);
      const uint32_t r0 = __shfl_sync(0xFFFFFFFFu, at, 2 * batch), r1 = __shfl_sync(0xFFFFFFFFu, at, 2 * batch + 1);
      ++batch;
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        const uint32_t r = 2 * c < kPer ? r0 : r1;
        const int in = (c % (kPer / 2)) * 512 + lane * 16;  // byte within the granule's codes
        if (r != kNoRow) {
          copy16(slot + c * 512 + to, a.k_codes + in + uint64_t(r) * (C::D / 2));
          copy16(slot + C::CODES + c * 512 + to, a.v_codes + in + uint64_t(r) * (C::D / 2));
        }
      }
      constexpr int kLanes = C::SCALES / 32;  // lanes that carry one granule's scales
      if (lane < 4 * kLanes) {
        const bool value = lane >= 2 * kLanes;
        const int l = lane & (2 * kLanes - 1);
        const uint32_t r = l < kLanes ? r0 : r1;
        if (r != kNoRow)
          copy16(slot + 2 * C::CODES + lane * 16,
                 (value ? a.v_scales : a.k_scales) + (l & (kLanes - 1)) * 16 + uint64_t(r) * (C::D / 32));
      }
    }
    copy_commit();
  }
};

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

// The same on accumulators that start at zero.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
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

// 2^(code - ref) as binary32 (code <= ref); a scale code of 0 (2^-127) counts as zero.
__device__ __forceinline__ float pow2_rel(uint32_t code, float unit) { return __uint_as_float(code << 23) * unit; }
// its unit: 2^(127 - ref)
__device__ __forceinline__ float pow2_unit(int ref) { return ue8m0_to_float(uint32_t(254 - ref)); }

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) { return F16::pack(lo, hi); }

template <class C>
struct State {
  float o[C::MT][C::NT][4];      // [m-tile][n-tile]: dimension pair x row pair
  float ref[C::NT][2];           // F16::kWeightUp minus the maximum that rows 2t, 2t + 1 refer to (exponents of two)
  float sum[C::NT][2];           // this lane's keys only
  int vref;                      // scale code that the accumulators are relative to
};

// U granules (16 U keys) of a stage, the first of them granule u0. key0: the
// stage's first key; len: keys of the sequence; masked: some row may not see all.
template <class C, int D = C::D>
__device__ __forceinline__ void granules(const typename C::Smem &sm, const uint8_t *ring, State<C> &st,
                                         const uint2 (&qreg)[C::QREG ? C::NT : 1][C::QREG ? C::KS : 1], int u0, int key0,
                                         int len, bool masked) {
  constexpr int NT = C::NT, U = C::U;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint8_t *kc = ring + u0 * 16 * (D / 2), *vc = kc + C::CODES;
  const uint8_t *ks = ring + 2 * C::CODES + u0 * 16 * (D / 32), *vs = ks + C::SCALES;
  key0 += 16 * u0;

  // ---- scale codes of V: keys 16 u + 8 v + 2 t + e
  uint32_t vcode[U][2][2], vtop = 0;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int e = 0; e < 2; ++e) vcode[u][v][e] = vs[(16 * u + 8 * v + 2 * t + e) * (D / 32) + g / (256 / D)];
  if (masked) {  // past the end there may be anything
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (key0 + 16 * u + 8 * v + 2 * t + e >= len) vcode[u][v][e] = 0;
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int v = 0; v < 2; ++v) vtop = max(vtop, max(vcode[u][v][0], vcode[u][v][1]));
  if (__any_sync(0xFFFFFFFFu, int(vtop) > st.vref)) {
    const int next = max(st.vref, int(__reduce_max_sync(0xFFFFFFFFu, vtop)));
    const float f = __uint_as_float(uint32_t(max(127 - (next - st.vref), 0)) << 23);
    st.vref = next;
#pragma unroll
    for (int i = 0; i < C::MT; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) st.o[i][n][c] *= f;
  }

  // ---- scores: keys 16 u + g + 8 v. A lane's word t of each group: two k-steps of a
  // group, then the group's partial score times its scale, 2^(code - 127), in binary32.
  constexpr int GR = D / 32;  // groups
  uint32_t kw[U][2][GR], kscale[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int key = 16 * u + 8 * v + g;
#pragma unroll
      for (int j = 0; j < GR; ++j)
        kw[u][v][j] = *reinterpret_cast<const uint32_t *>(kc + key * (D / 2) + ((j ^ swizzle<D>(g)) << 4) + 4 * t);
      if constexpr (D == 128)
        kscale[u][v] = *reinterpret_cast<const uint32_t *>(ks + key * 4);
      else
        kscale[u][v] = *reinterpret_cast<const uint16_t *>(ks + key * 2);
    }
  float s[U][NT][4];
#pragma unroll
  for (int j = 0; j < GR; ++j) {
    uint2 b[2][NT];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (C::QREG)
          b[h][n] = qreg[n][2 * j + h];
        else
          b[h][n] = sm.q[n][2 * j + h][lane];
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t x = kw[u][0][j], y = kw[u][1][j];
      float f[2];
#pragma unroll
      for (int v = 0; v < 2; ++v)
        f[v] = __uint_as_float((j == 0   ? kscale[u][v] << 23
                                : j == 1 ? kscale[u][v] << 15
                                : j == 2 ? kscale[u][v] << 7
                                         : kscale[u][v] >> 1) &
                               0x7F800000u);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float d[4];
        mma_f16_first(d, decode2<0>(x), decode2<0>(y), decode2<1>(x), decode2<1>(y), b[0][n].x, b[0][n].y);
        mma_f16(d, decode2<2>(x), decode2<2>(y), decode2<3>(x), decode2<3>(y), b[1][n].x, b[1][n].y);
#pragma unroll
        for (int c = 0; c < 4; ++c) s[u][n][c] = j == 0 ? d[c] * f[c >> 1] : fmaf(d[c], f[c >> 1], s[u][n][c]);
      }
    }
  }
  if (masked) {  // hidden keys to -inf
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int limit = sm.limit[8 * n + 2 * t + e] - key0 - g;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v)
            if (16 * u + 8 * v >= limit) s[u][n][2 * v + e] = -INFINITY;
      }
  }
  // ---- reference
  float mul[NT][2];
  bool move = false;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float2 m = *reinterpret_cast<const float2 *>(&sm.mul[8 * n + 2 * t]);
    mul[n][0] = m.x, mul[n][1] = m.y;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = fmaxf(s[0][n][e], s[0][n][2 + e]);
#pragma unroll
      for (int u = 1; u < U; ++u) x = fmaxf(x, fmaxf(s[u][n][e], s[u][n][2 + e]));
      move |= fmaf(x, mul[n][e], st.ref[n][e]) > kLazy + F16::kWeightUp;
    }
  }
  if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = s[0][n][e];
#pragma unroll
        for (int u = 0; u < U; ++u) m = fmaxf(m, fmaxf(s[u][n][e], s[u][n][2 + e]));
#pragma unroll
        for (int d = 4; d < 32; d *= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        m *= mul[n][e];
        const float next = m + st.ref[n][e] > F16::kWeightUp ? F16::kWeightUp - m : st.ref[n][e];
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
  uint32_t p[U][NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float x = exp2_approx(fmaf(s[u][n][2 * v], mul[n][0], st.ref[n][0]));
        const float y = exp2_approx(fmaf(s[u][n][2 * v + 1], mul[n][1], st.ref[n][1]));
        st.sum[n][0] += x;
        st.sum[n][1] += y;
        p[u][n][v] = transpose8x8(f16x2(x, y));
      }
  // ---- values: even and odd dimensions of two keys, interleaved
  constexpr int VW = D / 64;  // 32-bit words of a lane's eighth of a row
  const float vunit = pow2_unit(st.vref);
  uint32_t vlo[U][2][VW], vhi[U][2][VW], vf[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const uint8_t *row = vc + (16 * u + 8 * v + 2 * t) * (D / 2) + (((g / (256 / D)) ^ swizzle<D>(2 * t)) << 4) +
                           g * (D / 16) % 16;
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
        vlo[u][v][w] = (x[w] & 0x0F0F0F0Fu) | ((y[w] << 4) & 0xF0F0F0F0u);
        vhi[u][v][w] = ((x[w] >> 4) & 0x0F0F0F0Fu) | (y[w] & 0xF0F0F0F0u);
      }
      vf[u][v] = f16x2(pow2_rel(vcode[u][v][0], vunit), pow2_rel(vcode[u][v][1], vunit));
    }

#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < C::MT; ++i) {
      uint32_t r[2][2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint32_t l = vlo[u][v][i / 4], h = vhi[u][v][i / 4];
        r[v][0] = mul2((i & 3) == 0   ? decode2<0>(l)
                       : (i & 3) == 1 ? decode2<1>(l)
                       : (i & 3) == 2 ? decode2<2>(l)
                                      : decode2<3>(l),
                       vf[u][v]);
        r[v][1] = mul2((i & 3) == 0   ? decode2<0>(h)
                       : (i & 3) == 1 ? decode2<1>(h)
                       : (i & 3) == 2 ? decode2<2>(h)
                                      : decode2<3>(h),
                       vf[u][v]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(st.o[i][n], r[0][0], r[0][1], r[1][0], r[1][1], p[u][n][0], p[u][n][1]);
    }
  }
}

__device__ __forceinline__ bool row_ok(const PagedArgs &a, int row, int head) {
  return index_ok(a.status, row, a.num_rows) && index_ok(a.status, head, a.num_heads);
}

// Writes row (token, head) pair r of an item: 4 dimensions from d on, or (d < 0) its log sum exp.
template <class T>
__device__ __forceinline__ void store4(const PagedArgs &a, const Seq &s, int kv, int r, int dims, int d, float4 v) {
  const int tok = r / a.group, h = kv * a.group + r - tok * a.group;
  if (!row_ok(a, s.row0 + tok, h)) return;
  uint16_t *dst = a.out + int64_t(s.row0 + tok) * a.out_stride + int64_t(h) * dims + d;
  *reinterpret_cast<uint2 *>(dst) = make_uint2(T::pack(v.x, v.y), T::pack(v.z, v.w));
}

__device__ __forceinline__ void store_lse(const PagedArgs &a, const Seq &s, int kv, int r, float ref, float sum) {
  if (!a.lse) return;
  const int tok = r / a.group, h = kv * a.group + r - tok * a.group;
  if (!row_ok(a, s.row0 + tok, h)) return;
  a.lse[int64_t(s.row0 + tok) * a.num_heads + h] = sum != 0.0f ? (log2f(sum) + ref) * 0.6931471805599453f : -INFINITY;
}

// ------------------------------------------------------------------ main kernel

// The queries of a row block: loaded first, made into operand registers (with their limits and multipliers) when
// the copies of keys are on their way.
template <class T, class C>
struct Queries {
  static constexpr int D = C::D, GR = D / 32, PER = (C::NT + C::W - 1) / C::W;  // n-tiles of a warp
  uint4 raw[PER][GR];  // dimensions 32 i + 8 t .. + 7 of row g

  __device__ __forceinline__ void load(const PagedArgs &a, const Segment &seg, int warp) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int n = warp + k * C::W, r = seg.r0 + 8 * n + g;
      const int tok = r / a.group, h = seg.kv * a.group + r - tok * a.group;
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        raw[k][i] = make_uint4(0, 0, 0, 0);
        if (n < C::NT && r < seg.s.n * a.group && row_ok(a, seg.s.row0 + tok, h))
          raw[k][i] = __ldg(reinterpret_cast<const uint4 *>(a.q + int64_t(seg.s.row0 + tok) * a.q_stride +
                                                            int64_t(h) * D + 32 * i + 8 * t));
      }
    }
  }

  __device__ __forceinline__ void store(const PagedArgs &a, typename C::Smem &sm, const Segment &seg, int warp) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int n = warp + k * C::W, r = seg.r0 + 8 * n + g;
      if (n >= C::NT) break;
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        uint4 &v = raw[k][i];
        v.x ^= a.flip, v.y ^= a.flip, v.z ^= a.flip, v.w ^= a.flip;
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) amax = fmaxf(amax, fmaxf(fabsf(T::lo(w[c])), fabsf(T::hi(w[c]))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      // times 2^(14 - e): the largest lies in [2^14, 2^15), parts down to 2^-28 of it keep all their bits
      const int e = min(max(int(__float_as_uint(amax) >> 23) - 127, -100), 126);
      const float up = __uint_as_float(uint32_t(127 + 14 - e) << 23);
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        const uint32_t w[4] = {raw[k][i].x, raw[k][i].y, raw[k][i].z, raw[k][i].w};
#pragma unroll
        for (int c = 0; c < 2; ++c)
          sm.q[n][2 * i + c][lane] = make_uint2(f16x2(T::lo(w[2 * c]) * up, T::hi(w[2 * c]) * up),
                                                f16x2(T::lo(w[2 * c + 1]) * up, T::hi(w[2 * c + 1]) * up));
      }
      if (t == 0) {
        const bool real = r < seg.s.n * a.group;
        sm.mul[8 * n + g] = fmaxf(a.scale2 / up, 0x1p-126f);  // not 0: -inf must stay -inf
        sm.limit[8 * n + g] = real ? min(seg.s.len, max(0, seg.s.len - seg.s.n + r / a.group + 1)) : 0;
      }
    }
  }
};

template <class T, class C>
__global__ void __launch_bounds__(C::THREADS, C::BLOCKS) attend_paged_kernel(const PagedArgs a) {
  constexpr int D = C::D, NT = C::NT;
  extern __shared__ unsigned char paged_smem_raw[];
  typename C::Smem &sm =
      *reinterpret_cast<typename C::Smem *>((reinterpret_cast<uintptr_t>(paged_smem_raw) + 127) & ~uintptr_t(127));
  __shared__ int64_t total;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  pdl_launch_dependents();
  if (blockIdx.x == 0)  // what is out of range is reported once
    for (int b = tid; b < a.num_seqs; b += C::THREADS) load_seq<C>(a, b, a.status);
  const List<C> list(a, sm.before, &total);
  const Shares shares = make_shares<C>(list.all, gridDim.x);
  if (int64_t(blockIdx.x) >= shares.blocks) return;
  const int64_t begin = shares.begin(blockIdx.x), end = shares.begin(int64_t(blockIdx.x) + 1);
  Place place = list.find(begin);
  int64_t left = end - begin;
  bool first = true;
  while (left > 0) {
    const Segment seg = next_segment<C>(a, place, left);
    if (seg.count == 0) continue;
    Queries<T, C> queries;
    queries.load(a, seg, warp);
    Copier<C> copier;
    copier.start(a, seg);
#pragma unroll
    for (int c = 0; c < C::DEPTH - 1; ++c) copier.copy(a, seg, warp + c * C::W, sm.ring[warp][c]);
    queries.store(a, sm, seg, warp);
    __syncthreads();
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
    uint2 qreg[C::QREG ? NT : 1][C::QREG ? C::KS : 1];
    if constexpr (C::QREG) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < C::KS; ++k) qreg[n][k] = sm.q[n][k][lane];
    }
    const int clear = min(seg.s.len, max(0, seg.s.len - seg.s.n + 1 + seg.r0 / a.group));  // keys that every row sees
    int slot = 0;
    for (int i = warp; i < seg.count; i += C::W) {
      copy_wait<C::DEPTH - 2>();
      __syncwarp();  // every lane's copies of this stage are there, and nobody reads the slot that is filled next
      copier.copy(a, seg, i + (C::DEPTH - 1) * C::W, sm.ring[warp][slot == 0 ? C::DEPTH - 1 : slot - 1]);
      const int key0 = (seg.first + i) * kStageKeys;
      const bool masked = key0 + kStageKeys > clear;
#pragma unroll 1
      for (int u = 0; u < 2; u += C::U)
        granules<C>(sm, sm.ring[warp][slot], st, qreg, u, key0, seg.s.len, masked);
      slot = slot == C::DEPTH - 1 ? 0 : slot + 1;
    }
    copy_wait<0>();
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
    __syncthreads();  // the rings are drained: the slab takes their place
    const float unit = ue8m0_to_float(uint32_t(st.vref));
    const bool whole = seg.count == seg.s.steps;
    const int rows = seg.s.n * a.group - seg.r0;  // real rows of the block
    const int64_t slot_of = int64_t(blockIdx.x) * 2 + (first ? 0 : 1);
    float *part = a.parts + slot_of * C::PART;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = sm.ref[0][8 * n + 2 * t + e];
        for (int w = 1; w < C::W; ++w) m = fmaxf(m, sm.ref[w][8 * n + 2 * t + e]);
        f[e] = exp2_approx(-st.ref[n][e] - m) * unit;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < C::MT; i += 2)  // dimensions g D/8 + 2 i .. + 3
          *reinterpret_cast<float4 *>(&sm.slab[warp][2 * t + e][g * (D / 8) + 2 * i]) =
              make_float4(st.o[i][n][e] * f[e], st.o[i][n][2 + e] * f[e], st.o[i + 1][n][e] * f[e],
                          st.o[i + 1][n][2 + e] * f[e]);
      __syncthreads();
      for (int idx = tid; idx < 8 * (D / 4); idx += C::THREADS) {
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
        if (whole) {
          if (rr < rows) {
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;
            store4<T>(a, seg.s, seg.kv, seg.r0 + rr, D, d,
                      l != 0.0f ? make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv) : make_float4(0, 0, 0, 0));
            if (d == 0) store_lse(a, seg.s, seg.kv, seg.r0 + rr, m, l);
          }
        } else if (index_ok(a.status, slot_of, a.part_cap)) {
          *reinterpret_cast<float4 *>(part + rr * D + d) = v;
          if (d == 0) {
            part[C::ROWS * D + rr] = m;
            part[C::ROWS * D + C::ROWS + rr] = l;
          }
        }
      }
      __syncthreads();
    }
    first = false;
  }
}

// ------------------------------------------------------------------ joining the blocks
// Block c joins the item that block c of the main kernel began last, if that
// item went on into later blocks.

template <class T, class C>
__global__ void __launch_bounds__(kCombineThreads) combine_paged_kernel(const PagedArgs a) {
  __shared__ int64_t before[kMaxSeqs / 32 + 1], total;
  __shared__ float weight[8][kMaxBlocks], top[8], sum[8];  // by row
  static_assert(kCombineThreads == 8 * 32, "a warp for each row's weights");
  const List<C> list(a, before, &total);
  const Shares shares = make_shares<C>(list.all, gridDim.x);
  const int64_t c = blockIdx.x;
  Place p;
  int64_t begin = 0, end = 0, item0 = 0, item1 = 0, last = c + 1;  // the block's units, the item's, its last block
  if (c + 1 < shares.blocks) {
    begin = shares.begin(c);
    end = shares.begin(c + 1);
    p = list.find(end - 1);
    item0 = end - 1 - p.unit;
    item1 = item0 + kOver + p.s.steps;
    while (shares.begin(last + 1) < item1) ++last;
  }
  // the item's first stage is in a later block, or in an earlier one, or all of them are in this block: nothing to join
  const bool none = end <= item0 + kOver || begin > item0 + kOver || item1 <= end;
  pdl_wait_primary();  // every block: this kernel must not end before the main one
  if (none) return;
  // the blocks that hold parts of it: c, whose part is its last segment, and those after it, whose first it is
  constexpr int D = C::D, kAhead = 16;
  static_assert(8 * (D / 4) <= kCombineThreads, "one thread for four dimensions of a row");
  const int parts = int(last - c) + 1;
  if (!index_ok(a.status, parts - 1, kMaxBlocks) || !index_ok(a.status, 2 * last + 1, a.part_cap)) return;
  const int row0 = 8 * int(blockIdx.y);  // this block's 8 rows of the item
  const float *part0 = a.parts + (c * 2 + (item0 <= begin ? 0 : 1)) * C::PART;
  const float *part1 = a.parts + c * 2 * C::PART;  // the others: part b is 2 b slots on
  const auto part = [&](int b) { return b ? part1 + int64_t(b) * 2 * C::PART : part0; };
  const int row = threadIdx.x / (D / 4), d = 4 * (threadIdx.x % (D / 4)), at = (row0 + row) * D + d;
  const bool mine = row < 8;
  float4 v[kAhead];  // the first parts are on their way while the weights are made
#pragma unroll
  for (int b = 0; b < kAhead; ++b) {
    v[b] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (mine && b < parts) v[b] = *reinterpret_cast<const float4 *>(part(b) + at);
  }
  // weights of the parts: 2^(reference - largest), a warp for each row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  {
    const int head = C::ROWS * D + row0 + warp;
    float m0 = -kNone, l0 = 0.0f;
    if (lane < parts) {
      m0 = part(lane)[head];
      l0 = part(lane)[head + C::ROWS];
    }
    float m = m0;
    for (int b = lane + 32; b < parts; b += 32) m = fmaxf(m, part(b)[head]);
#pragma unroll
    for (int k = 16; k; k /= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, k));
    float l = 0.0f;
    for (int b = lane; b < parts; b += 32) {
      const float f = exp2_approx((b == lane ? m0 : part(b)[head]) - m);
      weight[warp][b] = f;
      l = fmaf(b == lane ? l0 : part(b)[head + C::ROWS], f, l);
    }
#pragma unroll
    for (int k = 16; k; k /= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, k);
    if (lane == 0) {
      top[warp] = m;
      sum[warp] = l;
    }
  }
  __syncthreads();
  const int per = p.s.items / a.num_kv_heads, kv = p.item / per, r0 = (p.item - kv * per) * C::ROWS;
  if (!mine || r0 + row0 + row >= p.s.n * a.group) return;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const auto add = [&](const float4 &x, float w) {
    o.x = fmaf(x.x, w, o.x), o.y = fmaf(x.y, w, o.y), o.z = fmaf(x.z, w, o.z), o.w = fmaf(x.w, w, o.w);
  };
#pragma unroll
  for (int b = 0; b < kAhead; ++b)
    if (b < parts) add(v[b], weight[row][b]);
#pragma unroll 8
  for (int b = kAhead; b < parts; ++b) add(*reinterpret_cast<const float4 *>(part(b) + at), weight[row][b]);
  const float l = sum[row], inv = l != 0.0f ? 1.0f / l : 0.0f;
  store4<T>(a, p.s, kv, r0 + row0 + row, D, d,
            l != 0.0f ? make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv) : make_float4(0, 0, 0, 0));
  if (d == 0) store_lse(a, p.s, kv, r0 + row0 + row, top[row], l);
}

// ------------------------------------------------------------------ host

template <class C>
constexpr size_t smem_bytes() {
  static_assert(C::BLOCKS * (sizeof(typename C::Smem) + 128 + 2048) <= 227 * 1024, "shared memory budget");
  return sizeof(typename C::Smem) + 128;
}

template <class C>
int blocks_of(int num_sms) {
  const int n = num_sms * C::BLOCKS;
  return n < kMaxBlocks ? n : kMaxBlocks;
}

template <class T, class C>
cudaError_t launch(const PagedArgs &a, int num_sms, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(attend_paged_kernel<T, C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       int(smem_bytes<C>()));
  if (e != cudaSuccess) return e;
  const unsigned grid = unsigned(blocks_of<C>(num_sms));
  attend_paged_kernel<T, C><<<grid, C::THREADS, smem_bytes<C>(), st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, C::NT);
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
// sequence need, and as few n-tiles a block as those leave. 64 sequences of 1,024
// to 5,120 (D = 128, groups of 4): 1 to 2 rows of a sequence take 49 us, 4 rows
// 67 (109 in the variant of 32), 6 rows 82 (110 there), 8 rows 112.
// Warps and blocks follow the registers: 16, 12 and 8 warps an SM with 128, 168
// and 255 (D = 64: 12). 8 rows: blocks of 4 warps instead of 8 gain 3 % with 128
// sequences (236 us against 243) and lose 7 % with one (11.4 against 10.7), whose
// parts to join are then twice as many. 24 rows: 12 or 10 warps an SM spill or halve
// the granules computed at once, 88 to 114 us against 65 (one long sequence) and 82.
template <int D, class F>
auto pick(int rows, F f) {
  const int blocks = (rows + 31) / 32, tiles = ((rows + blocks - 1) / blocks + 7) / 8;
  switch (tiles) {
    case 1: return f(Cfg<D, 1, 8, 2, D == 128 ? 3 : 5, 2>());
    case 2: return f(Cfg<D, 2, 4, 3, D == 128 ? 3 : 5, 2>());
    case 3: return f(Cfg<D, 3, 4, D == 128 ? 2 : 3, 5, 2>());
    default: return f(Cfg<D, 4, 4, D == 128 ? 2 : 3, 5, 1>());
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
    return int64_t(blocks_of<C>(num_sms)) * 2 * C::PART * 4;
  };
  const int rows = usual_rows(io, c);
  return c.head_dim == 64 ? pick<64>(rows, bytes) : pick<128>(rows, bytes);
}

cudaError_t launch_attend_paged(const moe_attend_paged_io_t &io, const moe_kv_cache_t &c, void *workspace,
                                int64_t workspace_bytes, int32_t *status, int num_sms, cudaStream_t st) {
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
  a.cached_rows = int64_t(c.num_pages) * c.page_size * c.num_kv_heads;
  a.scale2 = fmaxf(fabsf(io.scale) * 1.4426950408889634f, 0x1p-100f);
  a.flip = io.scale < 0.0f ? 0x80008000u : 0u;
  a.parts = static_cast<float *>(workspace);
  a.status = status;
  const bool h = io.dtype == MOE_DTYPE_F16;
  const auto go = [&](auto cfg) {
    using C = decltype(cfg);
    a.part_cap = checked_capacity(workspace_bytes / (C::PART * 4), io.flags);
    return h ? launch<F16, C>(a, num_sms, st) : launch<Bf16, C>(a, num_sms, st);
  };
  const int rows = usual_rows(io, c);
  return c.head_dim == 64 ? pick<64>(rows, go) : pick<128>(rows, go);
}

}  // namespace moe
