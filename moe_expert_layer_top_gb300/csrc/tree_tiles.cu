// tree_tiles.cu — attention of large trees over the paged MXFP4 cache, on the 5th-generation tensor cores.
//
// Mathematics. As in attend_paged.cu: s_j = scale q . K_j, o = sum_j softmax(s)_j V_j
// in one pass over the keys with a lazy reference, K_j = 2^(a - 127) k with
// codes k and one scale code a per 32 dimensions, V likewise. Rows are (token,
// head) pairs of one kv head's group; a row sees the keys in front of the tree,
// its ancestors' and its own.
//   Keys and values become f16 in shared memory: code times 2^(a - a_ref + 13). Of keys a_ref is the largest scale
//   code of 32; what it takes off goes into the factor of their scores, without an operation per score. Of values it
//   is the scale code that the accumulators are relative to: 3 above the largest of 16 tiles where it moves, and it
//   moves up when values beyond it are among the next 16. Exact down to 2^-33 of the largest seen. (With values
//   relative to those of 32 keys, and the rest in the exponents of their weights, the weights next to a far larger
//   value lost their bits in f16.)
//   Queries become f16 times a power of two per row, probabilities f16 as in attend_paged.cu. All sums are binary32.
//
// Bound. 4 D flops per (row, head, key) on the tensor cores; a decoded key tile serves 128 or 256 rows, so decoding
// (2 D conversions a key) is a small part of it, unlike with the 8 to 32 rows of a verify step.
//   Measured (32 + 8 heads of 128, 152 SMs, device time in a graph): 16 trees of 64 rows over 8,000 to 32,000 tokens
// 316 us, 985 TFLOP/s or half of a library product's rate; one of 64 rows over 131,071 tokens 149 us (925); one of 16
// rows over 4,096 20.6; 24 ragged ones (64 + 8 heads of 64, f16) 64. A step of a stream, 128 keys, takes 4,700
// clocks: 2,250 for the softmax (1,500 of them exponentials), 1,850 until its MMAs are issued and done, which at 128
// x 128 take all of the shared memory's bandwidth, the rest waits and mask. The streams overlap to 44 % of the tensor
// pipe's time and 42 % of the issue slots. Leaving out single parts (exponentials, decoding, its stores) gains 5 % at
// most each: what is left is the chain of latencies.
//   Tried and slower (16 trees of 64 rows): steps of 64 keys, so that one half's MMAs run under the other's softmax,
// 382 us; the same with two warps that only issue, 352 (96 registers a thread at launch, and their code falls out of
// the instruction cache); a thread for half a row 341 to 349; loads of S in front of the wait for the scales 339;
// waits that spin 396.
//
// Layout. A block has two streams of 128 rows (MMA M, TMEM lanes), whose softmax runs in turn with the other's MMAs:
//   wide items (more than 128 rows of a kv head): two row tiles over the same key tiles;
//   narrow ones: the same rows over alternate key tiles, joined at the item's end through shared memory.
//   warps 0-3   softmax of stream 0, a row a thread; warps 4-7 of stream 1; they also make the queries' tiles, and
//               one lane of each four issues the stream's MMAs: S = Q K^T, then O += P V with P from TMEM, where the
//               softmax wrote it over S (the stream has to wait for them anyway)
//   warps 8-11  keys, warps 12-15 values: codes and scales of 128 at a time, the next tile's by cp.async into places
//               of each thread's own, conversion into tiles (K-major and N-major, 128-byte swizzle) of a ring
// A stream's next S is issued behind P V of its step, by the same lane, so the S of a step that is complete also says
// that the stream's accumulators are.
//
// Schedule. As in attend_paged.cu: the items' key tiles in units, equal contiguous shares for one block on each SM, parts
// of items that several blocks share in a workspace, joined in a fixed order by a second kernel. Every warp finds its
// block's share by itself, and goes from item to item without a queue.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "attention.cuh"
#include "pairs.cuh"
#include "speculative.h"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kRows = 128;     // rows of a stream
constexpr int kKeys = 128;     // keys of a tile
constexpr int kThreads = 512;  // four warpgroups
// Registers: 128 a thread at launch; the softmax takes 24 more from the decoders.
constexpr int kRegsLaunch = 128, kRegsSoftmax = 152, kRegsDecode = 104;
static_assert(2 * kRegsSoftmax + 2 * kRegsDecode <= 4 * kRegsLaunch, "register split");
constexpr int kWarpDecode = 8;
constexpr uint32_t kTmemCols = 512;
constexpr int64_t kWaitNs = 1000000000;
constexpr float kLazy = 8.0f;       // the reference moves when the maximum is 2^kLazy beyond it
constexpr float kUp = 7.0f;         // weights are held times 2^kUp (F16::kWeightUp)
constexpr float kLowest = -3e38f;   // reference of a row without a weight
constexpr int kTop = 13;            // the largest scale of 32 keys becomes 2^kTop
constexpr int kBias = 127 + kTop;   // a value is its f16 times 2^(a_ref - kBias)
constexpr int kHeadroom = 3;        // the accumulators' scale code lies that far above the largest seen
// What an item costs beside its tiles, in units of a narrow tile.
constexpr int kOver = 8;
constexpr int kMinShare = 2;  // units of a share, at least: each block between an item's first and last has a tile of it
constexpr int kJoinThreads = 256;
constexpr int kMaxBlocks = 1024;

struct TileArgs {
  const uint16_t *q;
  int64_t q_stride;
  uint16_t *out;
  int64_t out_stride;
  float *lse;
  const int32_t *page_table, *lengths, *cu_rows, *parents;
  int num_seqs, num_rows, max_pages, num_heads, num_kv_heads, group;
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int num_pages, page_size;
  float scale2;   // |scale| log2 e, at least 2^-100
  uint32_t flip;  // 0x80008000 with a negative scale
  float *parts;
  Joint *joints;  // of each block
  int64_t part_cap, joint_cap, cached_rows;
  bool skip;  // the first decoding warp does nothing: every wait runs out
  int32_t *status;
};

// ------------------------------------------------------------------ the list of work
// An item is a (sequence, kv head, block of 256 rows): kOver units, then one (sequences of up to 128 rows) or two for
// each of its key tiles. A tile belongs to the block that has its first unit.

struct Seq {
  int b, row0, n, len;
  int items, blocks, tiles, weight;

  __device__ __forceinline__ int item_units() const { return tiles * weight + kOver; }
  __device__ __forceinline__ int64_t units() const { return int64_t(items) * item_units(); }
};

__device__ __forceinline__ Seq load_seq(const TileArgs &a, int b, int32_t *status) {
  Seq s = {b, 0, 0, 0, 0, 1, 0, 1};
  if (b >= a.num_seqs) return s;
  const Span r = seq_span(a.cu_rows, b, a.num_rows, status);
  if (r.n <= 0) return s;
  if (r.n > kMaxTree) {
    out_of_range(status);
    return s;
  }
  s.row0 = r.first;
  s.n = r.n;
  const int cap = a.max_pages * a.page_size;
  int len = __ldg(a.lengths + b);
  if (len < 0 || len > cap) {
    out_of_range(status);
    len = len < 0 ? 0 : cap;
  }
  s.len = len;
  const int rows = s.n * a.group;
  s.blocks = (rows + 2 * kRows - 1) / (2 * kRows);
  s.items = a.num_kv_heads * s.blocks;
  s.weight = rows > kRows ? 2 : 1;
  s.tiles = max(1, (len + kKeys - 1) / kKeys);  // a sequence without keys still writes its rows
  return s;
}

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

struct Place {
  Seq s;
  int item, unit;
};

// Units in front of each 32 sequences, summed by the whole block; then every warp looks places up by itself.
struct List {
  const TileArgs &a;
  const int64_t *before;
  int64_t all;

  __device__ List(const TileArgs &args, int64_t *shared, int64_t *total) : a(args), before(shared) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int chunks = (a.num_seqs + 31) / 32;
    for (int c = warp; c < chunks; c += blockDim.x / 32) {
      const int64_t v = warp_sums(load_seq(a, c * 32 + lane, nullptr).units());
      if (lane == 31 && index_ok(a.status, c, kMaxSeqs / 32 + 1)) shared[c] = v;
    }
    __syncthreads();
    if (warp == 0) {
      int64_t base = 0;
      for (int c0 = 0; c0 < chunks; c0 += 32) {
        const int64_t v = c0 + lane < chunks ? shared[c0 + lane] : 0, s = warp_sums(v);
        if (c0 + lane < chunks) shared[c0 + lane] = base + s - v;
        base += __shfl_sync(0xFFFFFFFFu, s, 31);
      }
      if (lane == 0) *total = base;
    }
    __syncthreads();
    all = *total;
  }

  // The sums are there.
  __device__ __forceinline__ List(const TileArgs &args, const int64_t *shared, int64_t total)
      : a(args), before(shared), all(total) {}

  // The place of unit p (0 <= p < all). Whole warp.
  __device__ Place find(int64_t p) const {
    const int lane = threadIdx.x & 31;
    int c = 0;
    for (int lo = 0, hi = (a.num_seqs + 31) / 32; lo < hi;) {  // the last chunk with before <= p
      const int mid = (lo + hi) / 2;
      if (before[mid] <= p) {
        c = mid;
        lo = mid + 1;
      } else {
        hi = mid;
      }
    }
    const Seq s = load_seq(a, c * 32 + lane, nullptr);
    const int64_t stop = warp_sums(s.units()), rest = p - before[c];
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, rest < stop);
    const int w = hit ? __ffs(hit) - 1 : 31;
    const int64_t in = rest - (__shfl_sync(0xFFFFFFFFu, stop, w) - __shfl_sync(0xFFFFFFFFu, s.units(), w));
    Place pl;
    pl.s = load_seq(a, c * 32 + w, nullptr);
    pl.item = int(divide(in, pl.s.item_units()));
    pl.unit = int(in - int64_t(pl.item) * pl.s.item_units());
    return pl;
  }
};

// A run of tiles of one item that a block computes (count may be 0).
struct Segment {
  Seq s;
  int kv, r0;        // kv head, first (token, head) pair
  int first, count;  // tiles
  bool wide;         // two row tiles

};

// Cuts the next segment off a block's share; `left` units remain after it.
__device__ __forceinline__ Segment next_segment(const TileArgs &a, Place &p, int64_t &left) {
  Segment g;
  g.s = p.s;
  g.kv = p.item / p.s.blocks;
  g.r0 = (p.item - g.kv * p.s.blocks) * 2 * kRows;
  g.wide = p.s.n * a.group - g.r0 > kRows;
  const int64_t room = p.s.item_units() - p.unit;
  const int take = int(room < left ? room : left), w = p.s.weight;
  g.first = (max(0, p.unit - kOver) + w - 1) / w;
  g.count = (max(0, p.unit + take - kOver) + w - 1) / w - g.first;
  left -= take;
  p.unit = 0;
  ++p.item;
  if (left > 0) {
    while (p.item >= p.s.items) {  // the next sequence with rows
      p.s = load_seq(a, p.s.b + 1, nullptr);
      p.item = 0;
      if (p.s.b >= a.num_seqs) {
        left = 0;
        break;
      }
    }
  }
  return g;
}

struct Shares {
  int64_t blocks, each, more;  // the first `more` blocks have each + 1 units

  __device__ __forceinline__ int64_t begin(int64_t b) const { return b * each + (b < more ? b : more); }
};

__device__ __forceinline__ Shares make_shares(int64_t units, int64_t grid) {
  Shares s;
  s.blocks = units < grid * kMinShare ? units / kMinShare : grid;  // an item alone has more units than that
  s.each = s.blocks ? divide(units, s.blocks) : 0;
  s.more = units - s.each * s.blocks;
  return s;
}

// What the block leaves to be joined: its last item, if it has the item's first tile and later blocks have others.
// Whole warp.
__device__ __forceinline__ void tell_joint(const TileArgs &a, const List &list) {
  const Shares shares = make_shares(list.all, gridDim.x);
  const int64_t c = blockIdx.x;
  Joint j = {};
  if (c + 1 < shares.blocks) {
    const int64_t begin = shares.begin(c), end = shares.begin(c + 1);
    const Place p = list.find(end - 1);
    const int64_t item0 = end - 1 - p.unit, tile0 = item0 + kOver;
    const int64_t tile1 = tile0 + int64_t(p.s.tiles - 1) * p.s.weight;  // the first and last tile's units
    if (tile0 >= begin && tile0 < end && tile1 >= end) {
      int64_t last = c + 1;
      while (shares.begin(last + 1) <= tile1) ++last;
      j.parts = int(last - c) + 1;
      j.slot = item0 <= begin ? 0 : 1;
      j.row0 = p.s.row0;
      j.kv = p.item / p.s.blocks;
      j.r0 = (p.item - j.kv * p.s.blocks) * 2 * kRows;
      j.rows = min(2 * kRows, p.s.n * a.group - j.r0);
    }
  }
  if ((threadIdx.x & 31) == 0 && index_ok(a.status, c, a.joint_cap)) a.joints[c] = j;
}

// ------------------------------------------------------------------ shared memory

template <int D>
struct Smem {
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kTileBytes = 128 * D * 2;  // 128 rows of Q, K or V in f16: D/64 parts of 128 rows x 128 bytes
  // Largest scales are kept for 8 tiles. Those of K tile j + 8 are written when K of tile j + 7 is there, for which S of
  // tile j + 7 - kStages / 2 >= j + 3 was done; that was issued behind P V of the tile before (or two before) in its
  // stream, and so were those before it: the softmax has read those of tile j. What V's are relative to likewise, by the P V
  // that V's entry of the ring was waited for.
  static constexpr int kExps = 8;
  static_assert(kExps >= kStages / 2 + 4, "largest scales");
  static constexpr int kRawBytes = kKeys * D / 2;
  static constexpr uint32_t kColO = 2 * kKeys;
  static_assert(kColO + 2 * D <= kTmemCols, "TMEM budget");
  uint8_t q[2][kTileBytes];
  uint8_t kv[kStages][kTileBytes];
  uint8_t raw[2][kRawBytes];                   // codes of K and V of the next tile as each thread copied them
  uint8_t join[D == 128 ? 16 : kRows * 64 * 4];  // D = 128: the second stream's query tile serves
  int exps[kExps][4];                          // by tile mod kExps: largest scale codes of 32 keys,
  int values[kExps];                           // and the scale code that the tile's values are relative to
  int tops[2][4];                              // of 16 tiles, by turns: the values' largest scale code, by warp
  uint8_t parent[kMaxTree];                    // place of the parent plus one
  int64_t before[kMaxSeqs / 32 + 1], total;    // of the list of work
  uint64_t q_full[2];      // the query tile is there (4 warps)
  uint64_t full[kStages];  // a K or V tile is there (4 warps)
  uint64_t empty[kStages]; // the MMAs that read it are done (2 commits: one of each stream, or two of one)
  uint64_t exps_full[kExps];  // a tile's exps and what its values are relative to are there (8 warps)
  uint64_t tops_full[2];   // 16 tiles' tops are there (4 warps)
  uint64_t s_full[2];      // S of a step complete, and everything issued before it
  uint64_t p_full[2];      // P of a step written (4 warps)
  uint64_t o_full[2];      // the stream's last P V is in O, and every MMA of the stream is done
  uint64_t met;            // the softmax warps among themselves (8 warps)
  uint64_t mma_done[2];    // the stream's MMAs are done, where it gave up
  uint32_t tmem_base;

  __device__ __forceinline__ uint8_t *exchange() { return D == 128 ? q[1] : join; }
  static constexpr size_t bytes() { return sizeof(Smem) + 1024; }
};

// ------------------------------------------------------------------ PTX wrappers

// D (+)= A B^T for K = 16 values of 16 bits, A and B in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same with A in TMEM (two values per 32-bit column).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One lane of the (whole) warp, known to the compiler as such.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Descriptor of V as the N-major B operand (see attend_prompt.cu).
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr) {
  return (sw128_desc(saddr) & ~(uint64_t(0x3FFFu) << 16)) | (uint64_t(kKeys * 128 >> 4) << 16);
}

// 32 consecutive columns of the warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// The same, and the largest of the row's values (NaN aside).
__device__ __forceinline__ void tmem_ld32_max(uint32_t taddr, uint32_t *r, float &top) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(top)
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Every load of this thread has its values; the registers pass through, so that no use moves ahead of the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}

__device__ __forceinline__ void tmem_wait_ld(uint32_t *r, float &top) {
  tmem_wait_ld(r);
  asm volatile("" : "+f"(top)::"memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ bool test(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, int32_t *status) {
  if (test(bar, parity) || mbar_wait(bar, parity, kWaitNs)) return true;
  if (status) report_error(status, MOE_ERR_TIMEOUT);
  return false;
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

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

// 2^e as binary32, e from -126 on (up to 127).
__device__ __forceinline__ float pow2(int e) { return __int_as_float((max(e, -126) + 127) << 23); }
// The same down to the smallest of all, 2^-149.
__device__ __forceinline__ float pow2_small(int e) { return e >= -126 ? pow2(e) : __int_as_float(1 << max(149 + e, 0)); }

__device__ __forceinline__ bool row_ok(const TileArgs &a, int row, int head) {
  return index_ok(a.status, row, a.num_rows) && index_ok(a.status, head, a.num_heads);
}

// ------------------------------------------------------------------ keys (warps 8-11) and values (warps 12-15)
// A warp takes 32 keys of each tile, a lane one group of 32 dimensions of every 8th (D = 128) or 16th key: 16 bytes of
// codes. Its lanes then store the 16-byte pieces of eight keys at a time, which the swizzle puts into different banks.

template <int D>
struct Decoder {
  using S = Smem<D>;
  static constexpr int kGroups = D / 32, kSpan = 32 / kGroups, kPer = 32 / kSpan;  // keys a pass, passes
  static constexpr uint32_t kNoRow = 0xFFFFFFFFu;
  const TileArgs &a;
  S &sm;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, v = (threadIdx.x >> 7) & 1;  // v: values
  const uint8_t *const codes, *const scales;
  const int group = lane / kSpan, in = lane % kSpan;
  const int32_t *table;
  uint32_t at;  // lane 2 j + u: cached row of granule u (16 keys) of the warp's keys in the j-th tile of the batch
  int looked;   // the batch's first tile: 16 of the segment are looked up at a time
  uint32_t batches = 0;  // of values, that the warps have agreed on
  uint32_t scale[kPer] = {};  // scale codes of the tile on its way

  __device__ __forceinline__ Decoder(const TileArgs &args, S &smem)
      : a(args), sm(smem), codes(v ? a.v_codes : a.k_codes), scales(v ? a.v_scales : a.k_scales) {}

  __device__ __forceinline__ void start(const Segment &seg) {
    table = a.page_table + int64_t(seg.s.b) * a.max_pages;
    looked = 0;
  }

  __device__ __forceinline__ static void copy16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  }

  // A scale code, or 0. In assembly, so that no selection behind the load waits for it here.
  __device__ __forceinline__ static uint32_t load_scale(const uint8_t *p, bool some) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %2, 0;\n\t"
        "mov.u32 %0, 0;\n\t"
        "@p ld.global.nc.u8 %0, [%1];\n\t}"
        : "=r"(r)
        : "l"(p), "r"(uint32_t(some)));
    return r;
  }

  // Codes and scales of tile i of the segment on their way. (Two tiles ahead measured the same, 331 and 75.7 us against
  // 329 and 74.5 with 16 trees of 64 rows and ragged ones of D = 64.)
  __device__ __forceinline__ void fetch(const Segment &seg, int i) {
    if (i < seg.count) {
      uint4 of[kGroups] = {};  // values: the scale codes of the lane's granule, and how many bytes of them are there
      int bytes = -1;
      if (i == looked || i - looked == 16) {
        looked = i;
        const int step = i + (lane >> 1), key = (seg.first + step) * kKeys + warp * 32 + (lane & 1) * 16;
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
        if (v) {
          bytes = at == kNoRow ? 0 : min(16, seg.s.len - key) * kGroups;
          if (bytes) {
#pragma unroll
            for (int k = 0; k < kGroups; ++k)
              of[k] = __ldg(reinterpret_cast<const uint4 *>(scales + uint64_t(at) * kGroups) + k);
          }
        }
      }
      const int from = 2 * (i - looked), rest = seg.s.len - (seg.first + i) * kKeys - warp * 32;  // of the warp's 32 keys
      uint32_t r[2] = {__shfl_sync(0xFFFFFFFFu, at, from), __shfl_sync(0xFFFFFFFFu, at, from + 1)};
      int end[2];  // keys that are there
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        end[u] = r[u] == kNoRow ? 0 : rest;
        if (r[u] == kNoRow) r[u] = 0;
      }
      const uint32_t to = smem_u32(sm.raw[v]) + (threadIdx.x & 127) * 16;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t *const c = codes + (uint64_t(r[u]) * (D / 2) + (in * (D / 2) + group * 16));
        const uint8_t *const q = scales + (uint64_t(r[u]) * kGroups + (in * kGroups + group));
#pragma unroll
        for (int h = 0; h < kPer / 2; ++h) {
          const int p = u * (kPer / 2) + h;
          const bool some = p * kSpan + in < end[u];
          copy16(to + p * 2048, c + h * (kSpan * D / 2), some ? 16 : 0);
          scale[p] = load_scale(q + h * (kSpan * kGroups), some);
        }
      }
      if (bytes >= 0) tell(of, bytes);  // the whole warp
    }
  }

  // The largest of the warp's scale codes of the batch, for the other warps of the values. Short, since most items come here
  // once and its code has to be fetched (byte by byte 24 ragged trees of D = 128 took 69 us in place of 62).
  __device__ __forceinline__ void tell(const uint4 (&of)[kGroups], int bytes) {
    uint32_t even = 0, odd = 0;  // of the bytes plus one, 255 (no scale) being 0
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const uint32_t w[4] = {of[k].x, of[k].y, of[k].z, of[k].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        // the word's bytes that are there: a shift by 32 and more leaves none
        const uint32_t x = w[c] & __funnelshift_rc(0xFFFFFFFFu, 0u, max(8 * (16 * k + 4 * c + 4 - bytes), 0));
        even = __vmaxu2(even, ((x & 0x00FF00FFu) + 0x00010001u) & 0x00FF00FFu);
        odd = __vmaxu2(odd, ((x >> 8 & 0x00FF00FFu) + 0x00010001u) & 0x00FF00FFu);
      }
    }
    even = __vmaxu2(even, odd);
    const int most = max(int(__reduce_max_sync(0xFFFFFFFFu, max(even & 0xFFFFu, even >> 16))) - 1, 0);
    if (lane == 0) {
      sm.tops[batches & 1][warp] = most;
      mbar_arrive(&sm.tops_full[batches & 1]);
    }
  }

  static __device__ __forceinline__ int largest(const uint32_t (&s)[kPer]) {
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < kPer; ++p) m = max(m, s[p] == 255 ? 0u : s[p]);
    return int(__reduce_max_sync(0xFFFFFFFFu, m));
  }

  // This thread's codes of a tile as f16 into their places.
  __device__ __forceinline__ void convert(uint8_t *tile, const uint8_t *raw, const uint32_t (&s)[kPer], int top) const {
    uint4 codes[kPer];
#pragma unroll
    for (int p = 0; p < kPer; ++p) codes[p] = *reinterpret_cast<const uint4 *>(raw + (threadIdx.x & 127) * 16 + p * 2048);
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
      const uint4 c = codes[p];
      const float f = s[p] == 255 ? INFINITY : __int_as_float(max(int(s[p]) - top + kBias, 0) << 23);
      const uint32_t f2 = F16::pack(f, f);
      const int key = warp * 32 + p * kSpan + in;
      uint8_t *const row = tile + (group / 2) * (kKeys * 128) + key * 128;
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = make_uint4(mul2(decode2<0>(w[i]), f2), mul2(decode2<1>(w[i]), f2), mul2(decode2<2>(w[i]), f2),
                                   mul2(decode2<3>(w[i]), f2));
        *reinterpret_cast<uint4 *>(row + ((((group & 1) * 4 + i) ^ (key & 7)) << 4)) = v;
      }
    }
  }

  __device__ __forceinline__ bool ready(uint32_t e) const {  // the ring's entry e may be filled
    return e < S::kStages || __all_sync(0xFFFFFFFFu, wait(&sm.empty[e % S::kStages], (e / S::kStages & 1) ^ 1, a.status));
  }

  // t: tiles of the block in front of the segment's. One copy of the code for K, V and every tile: see the softmax.
  __device__ __forceinline__ bool segment(const Segment &seg, uint32_t t) {
    start(seg);
    // What values are relative to. Their four warps agree on it, for 16 tiles at a time. (For each tile, so that all waited
    // for the slowest load, 24 ragged trees of D = 64 took 66 us in place of 64, with a cold L2 81 in place of 75; with tiles
    // converted first and once more where the scale moves D = 128 took 4 to 13 % more.)
    int relative = 0;
#pragma unroll 1
    for (int i = -1; i < seg.count; ++i) {
      if (i >= 0) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        const uint32_t n = t + i, e = 2 * n + v, slot = e % S::kStages;
        int top;
        if (v) {
          if (i == looked) {  // with a batch
            const int(&tops)[4] = sm.tops[batches & 1];
            if (!__all_sync(0xFFFFFFFFu, wait(&sm.tops_full[batches & 1], batches >> 1 & 1, a.status))) return false;
            ++batches;
            top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
            if (i == 0 || top > relative) relative = top + kHeadroom;
          }
          top = relative;
          if (warp == 0 && lane == 0) sm.values[n % S::kExps] = top;
        } else {
          top = largest(scale);
          if (lane == 0) sm.exps[n % S::kExps][warp] = top;
        }
        if (lane == 0) mbar_arrive(&sm.exps_full[n % S::kExps]);
        if (!ready(e)) return false;
        convert(sm.kv[slot], sm.raw[v], scale, top);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[slot]);
      }
      fetch(seg, i + 1);
    }
    return true;
  }
};

// ------------------------------------------------------------------ MMAs (one lane of a stream's first softmax warp)

template <int D>
struct Issuer {
  using S = Smem<D>;
  static constexpr uint32_t kBase = (1u << 4) | (uint32_t(kRows >> 4) << 24);  // f16 operands, binary32 sums
  static constexpr uint32_t kDescS = kBase | (uint32_t(kKeys >> 3) << 17);
  static constexpr uint32_t kDescO = kBase | (uint32_t(D >> 3) << 17) | (1u << 16);  // B is N-major
  const TileArgs &a;
  S &sm;
  const int x;
  const uint32_t tmem;

  __device__ __forceinline__ Issuer(const TileArgs &args, S &smem, int stream, uint32_t t)
      : a(args), sm(smem), x(stream), tmem(t) {}

  __device__ __forceinline__ bool full(uint32_t e) const {
    return wait(&sm.full[e % S::kStages], e / S::kStages & 1, a.status);
  }

  // The ring's entry e is no longer needed by this stream when what was issued is done.
  __device__ __forceinline__ void release(uint32_t e, bool wide) const {
    mma_commit(&sm.empty[e % S::kStages]);
    if (!wide) mma_commit(&sm.empty[e % S::kStages]);
  }

  // S of the block's tile t with query tile y.
  __device__ __forceinline__ bool scores(int y, uint32_t t, bool wide) const {
    const uint32_t e = 2 * t;
    if (!full(e)) return false;
    tmem_fence_after();
    const uint64_t qd = sw128_desc(smem_u32(sm.q[y])), kd = sw128_desc(smem_u32(sm.kv[e % S::kStages]));
    const uint32_t d = tmem + x * kKeys;
#pragma unroll
    for (int p = 0; p < D / 64; ++p)
#pragma unroll
      for (int c = 0; c < 4; ++c)  // 16 values are 32 bytes: 2 in the address field
        mma_ss(d, qd + p * (kRows * 128 >> 4) + 2 * c, kd + p * (kKeys * 128 >> 4) + 2 * c, kDescS, (p | c) != 0);
    mma_commit(&sm.s_full[x]);
    release(e, wide);
    return true;
  }

  // O of the stream with P and V of tile t.
  __device__ __forceinline__ bool values(uint32_t t, bool first, uint32_t parity, bool wide) const {
    const uint32_t e = 2 * t + 1;
    if (!full(e) || !wait(&sm.p_full[x], parity, a.status)) return false;
    tmem_fence_after();
    const uint64_t vd = v_desc(smem_u32(sm.kv[e % S::kStages]));
    const uint32_t pa = tmem + x * kKeys, d = tmem + S::kColO + x * D;
#pragma unroll
    for (int c = 0; c < kKeys / 16; ++c)  // 16 keys: 8 columns of P, 2048 bytes of V
      mma_ts(d, pa + 8 * c, vd + c * (2048 >> 4), kDescO, !first || c != 0);
    release(e, wide);
    return true;
  }
};

// ------------------------------------------------------------------ softmax (warps 0-7)

template <class T, int D>
struct Softmax {
  using S = Smem<D>;
  const TileArgs &a;
  S &sm;
  const int x = threadIdx.x >> 7, row = threadIdx.x & 127;
  const uint32_t lanes, ts, to;  // TMEM addresses of the warp's S and O
  const Issuer<D> issue;
  const bool issues = (threadIdx.x & 127) < 32;
  uint32_t scored = 0, ended = 0, meetings = 0, asked = 0;  // phases of s_full and p_full, o_full, met; bit y: of q_full[y]

  __device__ __forceinline__ Softmax(const TileArgs &args, S &smem, uint32_t tmem)
      : a(args), sm(smem), lanes(uint32_t((threadIdx.x >> 5 & 3) * 32) << 16), ts(tmem + lanes + x * kKeys),
        to(tmem + lanes + S::kColO + x * D),
        issue(args, smem, threadIdx.x >> 7, tmem) {}

  // No MMA may be in flight when TMEM is freed.
  __device__ __forceinline__ void give_up() const {
    if (issues && elect_one()) {
      mma_commit(&sm.mma_done[x]);
      mbar_wait(&sm.mma_done[x], 0, kWaitNs);
    }
  }

  // All softmax warps have come here. A barrier with a limit: a warp that gave up elsewhere does not come.
  __device__ __forceinline__ bool meet() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.met);
    return __all_sync(0xFFFFFFFFu, wait(&sm.met, meetings++ & 1, a.status));
  }

  // The thread's query as f16 into the stream's tile; the factor from products with f16 keys to exponents of two.
  __device__ __forceinline__ float load_query(const Segment &seg, int token, int head, bool store) {
    const uint4 *src = reinterpret_cast<const uint4 *>(a.q + int64_t(seg.s.row0 + token) * a.q_stride + int64_t(head) * D);
    float amax = 0.0f;
#pragma unroll 1
    for (int i = 0; i < D / 8; i += 8) {
      uint4 raw[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) raw[j] = __ldg(src + i + j);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) amax = fmaxf(amax, fmaxf(fabsf(T::lo(w[c])), fabsf(T::hi(w[c]))));
      }
    }
    // times 2^(14 - e): the largest lies in [2^14, 2^15), parts down to 2^-28 of it keep all their bits
    const int e = min(max(int(__float_as_uint(amax) >> 23) - 127, -100), 126);
    const float up = __uint_as_float(uint32_t(127 + 14 - e) << 23);
    if (store) {
#pragma unroll 1
      for (int i = 0; i < D / 8; i += 8) {  // once more, now near
        uint4 raw[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) raw[j] = __ldg(src + i + j);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t w[4] = {raw[j].x ^ a.flip, raw[j].y ^ a.flip, raw[j].z ^ a.flip, raw[j].w ^ a.flip};
          uint32_t f[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) f[c] = F16::pack(T::lo(w[c]) * up, T::hi(w[c]) * up);
          *reinterpret_cast<uint4 *>(sm.q[seg.wide ? x : 0] + (i / 8) * (kRows * 128) + row * 128 + ((j ^ (row & 7)) << 4)) =
              make_uint4(f[0], f[1], f[2], f[3]);
        }
      }
      fence_proxy_async();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.q_full[seg.wide ? x : 0]);
    }
    return a.scale2 / up;
  }

  // Which of 128 keys, the first `ahead` places behind the tree's first, the row of a token sees.
  __device__ __forceinline__ void visible(int token, int ahead, uint32_t (&see)[4]) const {
    uint32_t m[kMaxTree / 32];
#pragma unroll
    for (int w = 0; w < kMaxTree / 32; ++w) m[w] = 0;
    for (int j = token; j >= 0; j = int(sm.parent[j]) - 1) {
#pragma unroll
      for (int w = 0; w < kMaxTree / 32; ++w)
        if (j >> 5 == w) m[w] |= 1u << (j & 31);
    }
    const auto word = [&](int i) {  // bits 32 i .. of the tree, all set in front of it
      uint32_t r = i < 0 ? 0xFFFFFFFFu : 0u;
#pragma unroll
      for (int w = 0; w < kMaxTree / 32; ++w)
        if (i == w) r = m[w];
      return r;
    };
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int first = ahead + 32 * c;
      see[c] = __funnelshift_r(word(first >> 5), word((first >> 5) + 1), first & 31);
    }
  }

  // 32 of the row's scores as far as it sees the keys, and the largest of them.
  static __device__ __forceinline__ float hide(uint32_t see, uint32_t (&s)[32]) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (!(see >> i & 1)) s[i] = 0xFF800000u;  // -inf
      top = fmaxf(top, __uint_as_float(s[i]));
    }
    return top;
  }

  // P = 2^(s mul + base) of 32 scores in f16 into its place, and the sum.
  __device__ __forceinline__ float exponentials(int c, const uint32_t (&s)[32], float mul, float base) const {
    uint32_t p[16];
    uint64_t add[2] = {0, 0};
    const uint64_t m = pair(mul, mul), b = pair(base, base);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float2 e = unpair(fma_pair(pair(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), m, b));
      const float u = exp2_approx(e.x), v = exp2_approx(e.y);
      add[(j >> 1) & 1] = add_pair(add[(j >> 1) & 1], pair(u, v));
      p[j / 2] = F16::pack(u, v);
    }
    tmem_st16(ts + 16 * c, p);
    const float2 sum = unpair(add_pair(add[0], add[1]));
    return sum.x + sum.y;
  }

  // Factor from the products with 32 keys to exponents of two; not 0: -inf must stay -inf.
  __device__ __forceinline__ float factor(float unit, int code) const { return fmaxf(unit * pow2(code - kBias), 0x1p-126f); }

  __device__ __forceinline__ void scale_accumulators(float f) const {
#pragma unroll 1
    for (int i = 0; i < D / 32; ++i) {
      uint32_t o[32];
      tmem_ld32(to + 32 * i, o);
      tmem_wait_ld(o);
#pragma unroll
      for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
      tmem_st32(to + 32 * i, o);
    }
  }

  // 32 dimensions of the row's accumulators.
  __device__ __forceinline__ void load_out(int first, float f, float (&v)[32]) const {
    uint32_t o[32];
    tmem_ld32(to + first, o);
    tmem_wait_ld(o);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o[i]) * f;
  }

  // The row's result: 32 dimensions from `first` on, whole or as a part (four dimensions of all rows, then the next four).
  __device__ __forceinline__ void store_out(const Segment &seg, float *part, int part_row, int token, int head, int first,
                                            float inv, const float (&v)[32]) const {
    if (part) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<float4 *>(part + ((first / 4 + c) * (2 * kRows) + part_row) * 4) =
            make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    } else {
      uint16_t *out = a.out + int64_t(seg.s.row0 + token) * a.out_stride + int64_t(head) * D + first;
      const bool some = inv != 0.0f;  // a NaN counts
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = some ? T::pack(v[8 * c + 2 * i] * inv, v[8 * c + 2 * i + 1] * inv) : 0u;
        *reinterpret_cast<uint4 *>(out + 8 * c) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }

  __device__ __forceinline__ bool segment(const Segment &seg, uint32_t t, int slot) {
    // The thread's row; those behind the last compute what it does, and write nothing.
    const int wanted = seg.r0 + (seg.wide ? x * kRows : 0) + row, r = min(wanted, seg.s.n * a.group - 1);
    const int token = r / a.group, head = seg.kv * a.group + r - token * a.group;
    bool real = r == wanted;
    if (!row_ok(a, seg.s.row0 + token, head)) return false;
    const float unit = load_query(seg, token, head, seg.wide || x == 0);
    const int before = seg.s.len - seg.s.n;  // keys in front of the tree
    if ((seg.first + seg.count) * kKeys > before) {
      const int i = threadIdx.x;
      if (i < seg.s.n) {
        int p = index_ok(a.status, seg.s.row0 + i, a.num_rows) ? __ldg(a.parents + seg.s.row0 + i) : -1;
        if (p >= i) {
          out_of_range(a.status);
          p = -1;
        }
        sm.parent[i] = uint8_t(p < 0 ? 0 : p + 1);
      }
      if (!meet()) return false;
    }
    float ref = kLowest, total = 0.0f;
    int scale = 0;  // of the accumulators
    // the stream's tiles of the segment: every one, or every second
    const int start = seg.wide ? 0 : x, stride = seg.wide ? 1 : 2;
    const int y = seg.wide ? x : 0;  // its query tile
    if (start < seg.count && issues) {
      bool ok = true;
      if (elect_one()) ok = wait(&sm.q_full[y], asked >> y & 1, a.status) && issue.scores(y, t + start, seg.wide);
      if (!__all_sync(0xFFFFFFFFu, ok)) return false;
    }
    asked ^= seg.wide ? 3 : 1;
    for (int i = start; i < seg.count; i += stride) {
      const int key0 = (seg.first + i) * kKeys;
      const bool opening = i == start;
      const uint32_t n = t + i;
      if (!__all_sync(0xFFFFFFFFu, wait(&sm.exps_full[n % S::kExps], n / S::kExps & 1, a.status))) return false;
      const int(&exps)[4] = sm.exps[n % S::kExps];
      const int values = sm.values[n % S::kExps];
      const bool masked = key0 + kKeys > before;  // some key of the tile may be hidden
      uint32_t see[4] = {0, 0, 0, 0};
      if (masked) visible(token, key0 - before, see);
      if (!__all_sync(0xFFFFFFFFu, wait(&sm.s_full[x], scored & 1, a.status))) return false;
      tmem_fence_after();
      // The row's largest score. Of the four times 32 the first two stay, in s1 and s0.
      uint32_t s0[32], s1[32];
      float t0, t1, top;
      tmem_ld32_max(ts + 96, s1, t1);
      tmem_ld32_max(ts + 64, s0, t0);
      tmem_wait_ld(s1, t1);
      tmem_wait_ld(s0, t0);
      if (masked) t1 = hide(see[3], s1), t0 = hide(see[2], s0);
      top = fmaxf(t1 * factor(unit, exps[3]), t0 * factor(unit, exps[2]));
      tmem_ld32_max(ts + 32, s1, t1);
      tmem_ld32_max(ts, s0, t0);
      tmem_wait_ld(s1, t1);
      tmem_wait_ld(s0, t0);
      if (masked) t1 = hide(see[1], s1), t0 = hide(see[0], s0);
      top = fmaxf(top, fmaxf(t1 * factor(unit, exps[1]), t0 * factor(unit, exps[0])));
      if (opening) {
        ref = fmaxf(top, kLowest);
        scale = values;
      } else if (__any_sync(0xFFFFFFFFu, top - ref > kLazy) || values > scale) {
        // the accumulators hold every tile before this one (see the order of issue)
        float f = 1.0f;
        if (top - ref > kLazy) {
          f = exp2_approx(ref - top);
          ref = top;
        }
        total *= f;
        if (values > scale) {
          f *= pow2(scale - values);
          scale = values;
        }
        scale_accumulators(f);
      }
      // P = 2^(s - ref) in f16, and the sum. A loop: its code has to share the instruction cache with the decoders' (with
      // four times 32 exponentials one after another, twice, and four copies of the decoding the warps waited for
      // instructions a third of the time: 16 trees of 64 rows 520 us).
#pragma unroll 1
      for (int c = 0; c < 4; c += 2) {
        if (c) {
          tmem_wait_ld(s0);
          tmem_wait_ld(s1);
          if (masked) hide(see[2], s0), hide(see[3], s1);
        }
        total += exponentials(c, s0, factor(unit, exps[c]), kUp - ref);
        if (c == 0) tmem_ld32(ts + 64, s0);
        total += exponentials(c + 1, s1, factor(unit, exps[c + 1]), kUp - ref);
        if (c == 0) tmem_ld32(ts + 96, s1);
      }
      tmem_wait_st();
      tmem_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.p_full[x]);
      if (issues) {
        bool ok = true;
        if (elect_one()) {
          ok = issue.values(t + i, opening, scored & 1, seg.wide);
          if (i + stride < seg.count)
            ok = ok && issue.scores(y, t + i + stride, seg.wide);
          else
            mma_commit(&sm.o_full[x]);
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) return false;
      }
      ++scored;
    }
    if (start < seg.count) {
      if (!__all_sync(0xFFFFFFFFu, wait(&sm.o_full[x], ended & 1, a.status))) return false;
      ++ended;
      tmem_fence_after();
    }
    // ---- results
    const bool whole = seg.count == seg.s.tiles;
    float *part = nullptr;
    if (!whole) {
      if (!index_ok(a.status, slot, a.part_cap)) real = false;
      part = a.parts + int64_t(slot) * 2 * kRows * (D + 2);
    }
    const bool both = !seg.wide && seg.count > 1;  // two streams of the same rows
    float f = pow2_small(scale - kBias);
    if (both) {
      float2 *const rows = reinterpret_cast<float2 *>(sm.exchange());  // reference and sum, by stream
      rows[x * kRows + row] = make_float2(ref, total);
      if (!meet()) return false;
      const float2 u = rows[row], v = rows[kRows + row];
      if (!meet()) return false;
      const float m = fmaxf(u.x, v.x);
      total = u.y * exp2_approx(u.x - m) + v.y * exp2_approx(v.x - m);
      f *= exp2_approx(ref - m);
      ref = m;
    }
    const float inv = total != 0.0f ? 1.0f / total : 0.0f;  // a NaN stays one
    const int part_row = (seg.wide ? x * kRows : 0) + row;
    const bool writes = seg.wide || x == 0;
    if (real && writes) {
      if (part) {
        part[2 * kRows * D + part_row] = ref;
        part[2 * kRows * D + 2 * kRows + part_row] = total;
      } else if (a.lse) {
        a.lse[int64_t(seg.s.row0 + token) * a.num_heads + head] =
            total != 0.0f ? (log2f(total) + (ref - kUp)) * 0.6931471805599453f : -INFINITY;
      }
    }
#pragma unroll 1
    for (int half = 0; half < D / 64; ++half) {
      uint8_t *const place = sm.exchange() + row * 256;  // 64 floats of the row, 16-byte pieces exchanged by row
      if (both && x == 1) {
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          float v[32];
          load_out(64 * half + 32 * i, f, v);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<float4 *>(place + (((8 * i + c) ^ (row & 15)) << 4)) =
                make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
        }
      }
      if (both && !meet()) return false;
      if (writes) {
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          float v[32];
          load_out(64 * half + 32 * i, f, v);
          if (both) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float4 o = *reinterpret_cast<const float4 *>(place + (((8 * i + c) ^ (row & 15)) << 4));
              v[4 * c] += o.x, v[4 * c + 1] += o.y, v[4 * c + 2] += o.z, v[4 * c + 3] += o.w;
            }
          }
          if (real) store_out(seg, part, part_row, token, head, 64 * half + 32 * i, inv, v);
        }
      }
      if (both && !meet()) return false;
    }
    tmem_fence_before();
    return meet();  // parents and sums of this segment have been read
  }
};

// ------------------------------------------------------------------ kernel

template <class T, int D>
__global__ void __launch_bounds__(kThreads, 1) tree_tiles_kernel(const TileArgs a) {
  extern __shared__ unsigned char tiles_smem_raw[];
  using S = Smem<D>;
  static_assert(S::bytes() <= 227 * 1024, "shared memory budget");
  S &sm = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(tiles_smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  if (warp == kWarpDecode) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == kWarpDecode + 1 && elect_one()) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&sm.full[i], 4);
      mbar_init(&sm.empty[i], 2);
    }
    for (int i = 0; i < S::kExps; ++i) mbar_init(&sm.exps_full[i], 8);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sm.tops_full[x], 4);
      mbar_init(&sm.q_full[x], 4);
      mbar_init(&sm.s_full[x], 1);
      mbar_init(&sm.p_full[x], 4);
      mbar_init(&sm.o_full[x], 1);
      mbar_init(&sm.mma_done[x], 1);
    }
    mbar_init(&sm.met, 8);
    fence_mbar_init();
  }
  if (blockIdx.x == 0)  // what is out of range is reported once
    for (int b = threadIdx.x; b < a.num_seqs; b += kThreads) load_seq(a, b, a.status);
  const List list(a, sm.before, &sm.total);
  const Shares shares = make_shares(list.all, gridDim.x);
  const bool any = int64_t(blockIdx.x) < shares.blocks;
  const int64_t begin = any ? shares.begin(blockIdx.x) : 0, end = any ? shares.begin(int64_t(blockIdx.x) + 1) : 0;
  Place place;
  if (any) place = list.find(begin);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = sm.tmem_base;
  int64_t left = end - begin;
  uint32_t t = 0;  // tiles of the block so far
  if (warp < kWarpDecode) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    Softmax<T, D> role(a, sm, tmem);
    for (int i = 0; left > 0; ++i) {
      const Segment seg = next_segment(a, place, left);
      if (seg.count == 0) continue;
      if (!role.segment(seg, t, int(blockIdx.x) * 2 + (i ? 1 : 0))) {
        role.give_up();
        break;
      }
      t += seg.count;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsDecode));
    Decoder<D> role(a, sm);
    if (a.skip && warp == kWarpDecode) left = 0;
    while (left > 0) {
      const Segment seg = next_segment(a, place, left);
      if (seg.count == 0) continue;
      if (!role.segment(seg, t)) break;
      t += seg.count;
    }
  }
  if (warp == kThreads / 32 - 1) tell_joint(a, List(a, sm.before, sm.total));  // in the shadow of the last softmax
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == kWarpDecode)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ------------------------------------------------------------------ joining the blocks
// Block c joins the item whose first tile is the main kernel's block c's, if later blocks have tiles of it too. What
// there is to join the main kernel has left: the blocks without work, most of them, end at once (with the list of work
// looked through again by each block the joins took 10 to 23 us).

template <int D>
constexpr int kJoinRows = kJoinThreads / (D / 4);  // rows at a time: a thread has four dimensions of one

template <class T, int D>
__global__ void __launch_bounds__(kJoinThreads) join_tiles_kernel(const TileArgs a) {
  const int c = int(blockIdx.x);
  pdl_wait_primary();  // every block: this kernel must not end before the main one
  const Joint p = a.joints[c];
  const int parts = p.parts;
  if (parts == 0) return;
  if (!index_ok(a.status, parts - 1, kMaxBlocks) || !index_ok(a.status, 2 * (c + parts - 1), a.part_cap)) return;
  constexpr int64_t kPart = 2 * kRows * (D + 2);
  const float *const part0 = a.parts + int64_t(c * 2 + p.slot) * kPart, *const part1 = a.parts + int64_t(c) * 2 * kPart;
  const auto part = [&](int b) { return b ? part1 + int64_t(b) * 2 * kPart : part0; };
  const int kv = p.kv, r0 = p.r0, rows = p.rows;
  const int row = threadIdx.x % kJoinRows<D>, d = 4 * (threadIdx.x / kJoinRows<D>);
  constexpr int kAtOnce = 2;  // parts (with 8 of them 16 trees of 64 rows take 326 us in place of 315)
  for (int i = int(blockIdx.y) * kJoinRows<D> + row; i < rows; i += int(gridDim.y) * kJoinRows<D>) {
    float m = kLowest, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int b0 = 0; b0 < parts; b0 += kAtOnce) {
      float mb[kAtOnce], lb[kAtOnce];
      float4 v[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const bool some = b0 + k < parts;
        const float *const from = part(some ? b0 + k : b0);
        mb[k] = some ? from[2 * kRows * D + i] : kLowest;
        lb[k] = some ? from[2 * kRows * (D + 1) + i] : 0.0f;
        v[k] = *reinterpret_cast<const float4 *>(from + d * (2 * kRows) + i * 4);
        if (!some) v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) top = fmaxf(top, mb[k]);
      const float f = exp2_approx(m - top);
      m = top;
      l *= f, o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const float w = exp2_approx(mb[k] - top);
        l = fmaf(lb[k], w, l);
        o.x = fmaf(v[k].x, w, o.x), o.y = fmaf(v[k].y, w, o.y), o.z = fmaf(v[k].z, w, o.z), o.w = fmaf(v[k].w, w, o.w);
      }
    }
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    const int r = r0 + i, token = r / a.group, h = kv * a.group + r - token * a.group;
    if (!row_ok(a, p.row0 + token, h)) continue;
    *reinterpret_cast<uint2 *>(a.out + int64_t(p.row0 + token) * a.out_stride + int64_t(h) * D + d) =
        l != 0.0f ? make_uint2(T::pack(o.x * inv, o.y * inv), T::pack(o.z * inv, o.w * inv)) : make_uint2(0, 0);
    if (d == 0 && a.lse)
      a.lse[int64_t(p.row0 + token) * a.num_heads + h] = l != 0.0f ? (log2f(l) + (m - kUp)) * 0.6931471805599453f : -INFINITY;
  }
}

// ------------------------------------------------------------------ host

int blocks_of(int num_sms) { return num_sms < kMaxBlocks ? num_sms : kMaxBlocks; }
int64_t part_bytes(const moe_kv_cache_t &c) { return int64_t(2) * kRows * (c.head_dim + 2) * 4; }

template <class T, int D>
cudaError_t launch(const TileArgs &a, int usual_rows, int num_sms, cudaStream_t st) {
  // The register split assumes the launch's share: a build that gave the kernel less must not run. Only the answer is
  // remembered, not a query that failed.
  static std::atomic<int> regs{0};
  if (!regs.load(std::memory_order_relaxed)) {
    cudaFuncAttributes at;
    const cudaError_t asked = cudaFuncGetAttributes(&at, tree_tiles_kernel<T, D>);
    if (asked != cudaSuccess) return asked;
    regs.store(at.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != kRegsLaunch) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaFuncSetAttribute(tree_tiles_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       int(Smem<D>::bytes()));
  if (e != cudaSuccess) return e;
  const unsigned grid = unsigned(blocks_of(num_sms));
  tree_tiles_kernel<T, D><<<grid, kThreads, Smem<D>::bytes(), st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // As many blocks of an item as the usual rows need. (With fewer, each with several runs of rows, 16 trees of 64 rows
  // took 324 and 327 us in place of 321, 24 ragged ones 72 and 81 in place of 70.)
  const int most = usual_rows < 2 * kRows ? usual_rows : 2 * kRows;
  cfg.gridDim = dim3(grid, unsigned((most + kJoinRows<D> - 1) / kJoinRows<D>));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_tiles_kernel<T, D>, a);
}

}  // namespace

int64_t tree_tiles_workspace(const moe_kv_cache_t &c, int num_sms) {
  return int64_t(blocks_of(num_sms)) * (2 * part_bytes(c) + int64_t(sizeof(Joint)));
}

cudaError_t launch_tree_tiles(const moe_attend_tree_io_t &io, const moe_kv_cache_t &c, int usual_rows, void *workspace,
                              int32_t *status, int num_sms, cudaStream_t st) {
  const moe_attend_paged_io_t &r = io.rows;
  TileArgs a = {};
  a.q = static_cast<const uint16_t *>(r.q);
  a.q_stride = r.q_stride;
  a.out = static_cast<uint16_t *>(r.out);
  a.out_stride = r.out_stride;
  a.lse = r.lse;
  a.page_table = r.page_table;
  a.lengths = r.lengths;
  a.cu_rows = r.cu_rows;
  a.parents = io.parents;
  a.num_seqs = r.num_seqs;
  a.num_rows = r.num_rows;
  a.max_pages = r.max_pages;
  a.num_heads = r.num_heads;
  a.num_kv_heads = c.num_kv_heads;
  a.group = r.num_heads / c.num_kv_heads;
  a.k_codes = c.k_codes;
  a.k_scales = c.k_scales;
  a.v_codes = c.v_codes;
  a.v_scales = c.v_scales;
  a.num_pages = c.num_pages;
  a.page_size = c.page_size;
  a.cached_rows = int64_t(c.num_pages) * c.page_size * c.num_kv_heads;
  a.scale2 = fmaxf(fabsf(r.scale) * 1.4426950408889634f, 0x1p-100f);
  a.flip = r.scale < 0.0f ? 0x80008000u : 0u;
  a.parts = static_cast<float *>(workspace);
  const int blocks = blocks_of(num_sms);
  a.joints = reinterpret_cast<Joint *>(static_cast<char *>(workspace) + 2 * blocks * part_bytes(c));
  a.part_cap = checked_capacity(int64_t(2) * blocks, r.flags);
  a.joint_cap = blocks;
  a.skip = r.flags & MOE_FLAG_TEST_SKIP_READY;
  a.status = status;
  const bool h = r.dtype == MOE_DTYPE_F16;
  if (c.head_dim == 64) return h ? launch<F16, 64>(a, usual_rows, num_sms, st) : launch<Bf16, 64>(a, usual_rows, num_sms, st);
  return h ? launch<F16, 128>(a, usual_rows, num_sms, st) : launch<Bf16, 128>(a, usual_rows, num_sms, st);
}

}  // namespace moe
