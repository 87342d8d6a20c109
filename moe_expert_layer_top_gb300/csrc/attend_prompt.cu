// attend_prompt.cu — causal attention over packed prompts, on the 5th-generation tensor cores.
//
// Mathematics. For each row: s_j = scale q . k_j over the keys it sees,
// o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m). One pass over the keys in
// tiles of 128 keeps a reference m and the two sums. The reference only moves
// when the running maximum has grown by more than 2^8 in the exponent: until
// then the terms are at most 2^8 (2^15 in f16, which holds them times 2^7), which
// neither binary32 sums nor 16-bit P can overflow, so the accumulator is rarely
// rescaled. P is rounded to the inputs' type for the second product (half a step,
// 2^-9 or 2^-12 in the root mean square of a row: what the output's own rounding
// costs; in f16 absolutely 2^-32 of the row's largest where that is more); sums are
// binary32.
//
// Bound. 4 D flops per (row, head, key) against 16-bit inputs read once: the
// tensor pipe, for all but the shortest prompts. 16,384 tokens (32 + 8 heads of
// 128) take 1.40 ms alone and 1.47 to 1.52 call after call (1.57 and 1.45 to 1.50
// PFLOP/s, 83 and 76 to 79 % of the measured bf16 rate; the clock falls then). A
// pair of row tiles costs 1.5 us for a key tile (1.06 of MMAs) and 4.4 us beside
// them (first loads, the first and last softmax, output), so 16 packed prompts with
// few key tiles each take 79 us where their MMAs need 35. D = 64: an MMA with N = 64
// takes as long as one with 128, so the value product has half the rate: three
// chunks behind 4,000 tokens 139 us, of which 88 for the MMAs. 257 tokens: 11.3.
//
// Layout. A row of the tile is a (token, head) pair: the G heads of a kv head's
// group are packed, r = token * G + head, so one key tile serves all of them and
// short prompts still fill the 128 rows of an MMA (floor(128 / G) G of them; a
// group of more than 128 heads is cut into equal parts). A block takes two such row
// tiles A and B. While the tensor cores work for one, the softmax of the other
// runs on the CUDA cores:
//   warps 0-3   softmax of tile A, one row (TMEM lane) a thread
//   warps 4-7   softmax of tile B
//   warp 8      TMA: Q, then K and V tiles of 128 keys into a ring of shared memory;
//               at the end it zeroes the rows of the last V tile that lie past
//               the sequence (they belong to the next one, and 0 * NaN is NaN),
//               and asks for the block's next work
//   warp 9      MMA issuer: S = Q K^T (both operands from shared memory), then
//               O += P V with P from TMEM, where the softmax wrote it over S
// The work is a list of steps (row tile, key tile): A0 B0 A1 B1 ..., then what
// one of the two has left. TMEM holds O of both and a ring of S: step q has S
// buffer q mod kBufs, so S of the next steps is computed while the softmax of
// this one runs (D = 64: three buffers; D = 128 leaves room for two). The MMAs of
// one thread run in the order of issue: S(q + kBufs) goes after P V of q, which
// reads the same columns.
//
// Where the works are few and the keys many, a work's keys are split: each part is a
// work of its own, which leaves O, reference and sum of its rows in the workspace, and
// a second kernel joins the parts in their order.
//
// A block goes from work to work without stopping: its barriers and TMEM stay, and
// the next Q, K and V are loaded while the last softmax and the output of this work
// run. With a block for each work these cost 6.5 us in place of 4.4 (16 packed
// prompts 90 us, 4,096 prompts of 30 tokens 11.4 ms against 1.12, 257 tokens 10.3).
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "attention.cuh"
#include "tcgen05.cuh"

namespace moe {

namespace {

constexpr int kRows = 128;     // rows of a tile (MMA M, TMEM lanes)
constexpr int kKeys = 128;     // keys of a tile
constexpr int kThreads = 384;  // three warpgroups; two warps of the last have no work
// Registers: 168 a thread at launch (384 x 168 = 64,512). The softmax keeps a
// row of 128 scores, so the last warpgroup hands most of its share to the other
// two: 2 x 128 x 224 + 128 x 56 = 64,512.
constexpr int kRegsLaunch = 168, kRegsSoftmax = 224, kRegsOther = 56;
static_assert(2 * kRegsSoftmax + kRegsOther <= 3 * kRegsLaunch, "register split");
constexpr int kWarpLoad = 8, kWarpMma = 9;
constexpr uint32_t kTmemCols = 512;
// Bound of every wait. A constant: with one from the caller 16,384 tokens took 1.54 ms in place of 1.50, 16 packed prompts
// 82.2 us in place of 80.9.
constexpr int64_t kWaitNs = 1000000000;
constexpr float kLazy = 8.0f;            // the reference moves when the maximum is 2^kLazy beyond it
// Key tiles of a part, at least. 64 rows over 4,096 keys: 29 us with 4 (or 2), 32 with 8, 43 with 16, 58 in one part.
constexpr int kSplitTiles = 4;
constexpr int kMaxSplits = 16;

struct PromptArgs {
  uint16_t *out;
  int64_t out_stride;
  float *lse;
  const int32_t *cu_rows, *cu_keys;
  int num_seqs, num_rows, num_keys, num_heads, causal;
  int group;       // heads packed into a row tile
  int groups;      // such groups of a kv head
  int all_groups;  // and of all heads
  int tokens;      // tokens of a row tile
  float up;        // T::kWeightUp in score units: the reference stands that far below (added to the exponent instead, the
                   // same number of operations, chunks with D = 64 took 149 us in place of 141.6)
  float scale2;    // |scale| log2 e, at least 2^-100: scores times this are exponents of two
  float lowest;    // reference of a row without a weight yet: below any score
  bool negative;   // the scale is: scores change sign
  int32_t *status;
  bool skip_tail;  // test hook: the mark of a zeroed last V tile is never set
  int splits;    // parts that a work's keys may be split into
  float *parts;  // workspace: of each part, O and (reference, sum) of its 256 rows
  int64_t part_cap;  // row tiles of parts that it holds, for the checks
};

// What a block does at a time: two row tiles of a sequence, for the heads of a group.
struct Work {
  int row0, n;       // the sequence's first row, its rows
  int key0, keys;    // its first key, its keys
  int t0;            // the block's first row within the sequence
  int kv, head0;     // kv head, the first of the block's heads
  int tiles0, tiles1;  // key tiles of row tiles A and B
  int valid;           // 0: there is no further work
  // where the barriers stand when it begins: steps, S of each row tile, entries of the ring (each modulo twice its
  // ring), and the phases of o_full
  int step0, s0, s1, entry0, o0, o1;
  int skip, parts, slot;  // keys of the sequence before key0; parts of this tile, and where this one goes

  __device__ __forceinline__ int tiles(int x) const { return x ? tiles1 : tiles0; }
  __device__ __forceinline__ int both() const { return min(tiles0, tiles1); }  // key tiles that both have
  __device__ __forceinline__ int all() const { return max(tiles0, tiles1); }
};

template <int D>
struct Smem {
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kTileBytes = 128 * D * 2;  // 128 rows of Q, K or V: D/64 parts of 128 rows x 128 bytes
  static constexpr int kBufs = D == 128 ? 2 : 3;  // S tiles in TMEM
  static constexpr uint32_t kColO = kBufs * kKeys;
  static_assert(kColO + 2 * D <= kTmemCols && kBufs <= 3, "TMEM budget");
  uint8_t q[2][kTileBytes];
  uint8_t kv[kStages][kTileBytes];
  uint8_t out[D == 128 ? 8 : 1][32 * 128];  // D = 128: 64 values of 32 rows of each softmax warp, on their way out
  uint4 next;                // the launch control's answer
  Work work[2];
  uint64_t next_full;        // the answer is there
  uint64_t work_full[2], work_empty[2];  // a Work is there; all have read it (8 softmax warps, the MMA lane)
  uint64_t q_full[2];        // Q of a row tile landed
  uint64_t q_empty[2];       // every S of the row tile is done
  uint64_t full[kStages];    // a K or V tile landed
  uint64_t empty[kStages];   // the MMAs that read it are done
  uint64_t tail[4];          // the last V tile of a work is zeroed past the sequence's end, by work mod 4: the loads
                             // are up to two works ahead of the MMAs
  uint64_t s_full[2][kBufs]; // S of (row tile, key tile j) complete, by j mod kBufs: no phase ends unseen
  uint64_t p_full[kBufs];    // P of a step written (4 warps)
  uint64_t o_full[2];        // the row tile's last P V is in O
  uint64_t mma_done;
  uint32_t tmem_base;
  static constexpr size_t kBytes = 2 * kTileBytes + kStages * kTileBytes + 8 * 32 * 128 + 1024 + 1024;
};

// ------------------------------------------------------------------ PTX wrappers

__device__ __forceinline__ void tma_load(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

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

// One lane of the (whole) warp. The compiler knows that code under this
// predicate runs in a single lane; under lane == 0 it would loop over lanes
// around every instruction that takes uniform registers (each MMA).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Descriptor of V as the N-major B operand: 64 values of N (128 bytes) by 8
// keys is one swizzled block of 1024 bytes; blocks of the next 8 keys follow
// (stride offset), the next 64 values of N lie a part (128 keys) further
// (leading offset).
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

// Every load of this thread has its values. The registers pass through, so
// that no use of them moves ahead of the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------------ the block's work

// Keys that row t of the sequence sees.
__device__ __forceinline__ int key_limit(const PromptArgs &a, int keys, int n, int t) {
  return a.causal ? min(keys, max(0, keys - n + t + 1)) : keys;
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

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, int32_t *status, int64_t ns = kWaitNs) {
  if (test(bar, parity) || mbar_wait(bar, parity, ns)) return true;
  if (status) report_error(status, MOE_ERR_TIMEOUT);
  return false;
}

// ------------------------------------------------------------------ the list of work
// The grid has a block for every Work. A running block takes over those that have not started yet, one by one, through
// the hardware's launch control; the others run as blocks of their own. (Heads run fastest: the heads of a sequence's
// long tiles come before its short ones.) Whole warp.
template <bool SPLIT>
__device__ __forceinline__ Work find_work(const PromptArgs &a, TileCursor &cursor, uint32_t block, int32_t *status) {
  int part = 0;
  const int slot = int(block);
  if constexpr (SPLIT) {
    part = int(block % uint32_t(a.splits));
    block /= uint32_t(a.splits);
  }
  const uint32_t tile = block / a.all_groups, head = block - tile * a.all_groups;
  const TileAt at =
      find_tile(cursor, a.cu_rows, a.num_rows, a.cu_keys, a.num_keys, a.num_seqs, 2 * a.tokens, tile, status);
  Work w;
  w.valid = at.seq >= 0;
  w.row0 = at.rows.first;
  w.n = at.rows.n;
  w.key0 = at.keys.first;
  w.keys = at.keys.n;
  w.kv = head / a.groups;
  w.head0 = head * a.group;
  w.t0 = (at.tiles - 1 - at.local) * (2 * a.tokens);  // the last rows see the most keys: they start first
  const auto key_tiles = [&](int first) {
    return first < w.n ? (key_limit(a, w.keys, w.n, min(first + a.tokens, w.n) - 1) + kKeys - 1) / kKeys : 0;
  };
  w.tiles0 = key_tiles(w.t0);
  w.tiles1 = key_tiles(w.t0 + a.tokens);
  w.step0 = w.s0 = w.s1 = w.entry0 = w.o0 = w.o1 = 0;
  if constexpr (SPLIT) {  // equal parts, of kSplitTiles key tiles at least
    const int all = w.all(), most = min(a.splits, max(1, all / kSplitTiles)), per = max(1, (all + most - 1) / most);
    w.slot = slot;
    w.parts = max(1, (all + per - 1) / per);
    if (part >= w.parts) w.valid = 0;
    w.skip = part * per * kKeys;
    w.key0 += w.skip;
    w.keys -= w.skip;
    w.tiles0 = min(max(w.tiles0 - part * per, 0), per);
    w.tiles1 = min(max(w.tiles1 - part * per, 0), per);
  }
  return w;
}

// Asks for the index of a block that has not started, which then never will.
__device__ __forceinline__ void ask_next(uint4 *answer, uint64_t *bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}

// The answer: whether there was one, and its index.
__device__ __forceinline__ bool read_next(const uint4 *answer, uint32_t &block) {
  uint32_t got;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n\t}"
      : "=r"(got), "=r"(block)
      : "r"(smem_u32(answer))
      : "memory");
  return got != 0;
}

// ------------------------------------------------------------------ TMA (warp 8)

__device__ __forceinline__ bool row_ok(const PromptArgs &a, int row, int head) {
  return index_ok(a.status, row, a.num_rows) && index_ok(a.status, head, a.num_heads);
}

// Entry i of the list K 0, V 0, K 1, V 1, ... of w into the ring, as its entry number base + i (one lane).
template <int D>
__device__ __forceinline__ void load_tile(const CUtensorMap *kmap, const CUtensorMap *vmap, const PromptArgs &a, Smem<D> &sm,
                                          const Work &w, uint32_t base, int i) {
  using S = Smem<D>;
  const uint32_t s = (base + i) % S::kStages;
  if (!index_ok(a.status, w.key0 + (i >> 1) * kKeys, a.num_keys) || !index_ok(a.status, w.kv, a.all_groups / a.groups))
    return;  // who waits for it reports that too
  mbar_arrive_expect_tx(&sm.full[s], S::kTileBytes);
  const CUtensorMap *map = i & 1 ? vmap : kmap;
#pragma unroll
  for (int p = 0; p < D / 64; ++p)
    tma_load(sm.kv[s] + p * (kKeys * 128), map, 64 * p, w.kv, w.key0 + (i >> 1) * kKeys, &sm.full[s]);
}

// Q of row tile x (one lane). Rows past the sequence are another one's, or zeros past the last: their scores are hidden.
template <int D>
__device__ __forceinline__ void load_queries(const CUtensorMap *qmap, const PromptArgs &a, Smem<D> &sm, const Work &w, int x) {
  if (!row_ok(a, w.row0 + w.t0 + x * a.tokens, w.head0 + a.group - 1)) return;
  mbar_arrive_expect_tx(&sm.q_full[x], uint32_t(a.tokens * a.group * D * 2));
#pragma unroll
  for (int p = 0; p < D / 64; ++p)
    tma_load(sm.q[x] + p * (kRows * 128), qmap, 64 * p, w.head0, w.row0 + w.t0 + x * a.tokens, &sm.q_full[x]);
}

// Q and the first entries of the block's first work, as many as the ring has slots, went out with the barriers'
// initialisation.
template <int D, bool SPLIT>
__device__ void load_warp(const CUtensorMap *qmap, const CUtensorMap *kmap, const CUtensorMap *vmap, const PromptArgs &a,
                          Smem<D> &sm, Work w) {
  using S = Smem<D>;
  const int lane = threadIdx.x & 31;
  TileCursor cursor;
  uint32_t base = 0, asked = 0;  // entries of the ring so far; questions for further work
  int queries[2] = {w.tiles0 > 0, w.tiles1 > 0}, issued = min(2 * w.all(), S::kStages);
  for (uint32_t t = 0;; ++t) {
    const int n = w.all();
    bool ok = true;
    if (elect_one()) {
      for (int i = issued; i < 2 * n; ++i) {
        const uint32_t e = base + i;
        if (e >= S::kStages && !wait(&sm.empty[e % S::kStages], (e / S::kStages & 1) ^ 1, a.status)) {
          ok = false;
          break;
        }
        load_tile<D>(kmap, vmap, a, sm, w, base, i);
        ++issued;
        if (t > 0 && i == 0) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (!ok || w.tiles(x) == 0) continue;
            ok = queries[x] == 0 || wait(&sm.q_empty[x], (queries[x] - 1) & 1, a.status);
            if (!ok) continue;
            load_queries<D>(qmap, a, sm, w, x);
            ++queries[x];
          }
          if (!ok) break;
        }
      }
    }
    const auto ask = [&] {
      if (elect_one()) {
        mbar_arrive_expect_tx(&sm.next_full, 16);
        ask_next(&sm.next, &sm.next_full);
      }
      ++asked;
    };
    ask();
    // one lane issued: the others follow
    issued = __reduce_max_sync(0xFFFFFFFFu, unsigned(issued));
    queries[0] = __reduce_max_sync(0xFFFFFFFFu, unsigned(queries[0]));
    queries[1] = __reduce_max_sync(0xFFFFFFFFu, unsigned(queries[1]));
    ok = __all_sync(0xFFFFFFFFu, ok);
    const int cut = w.keys - (n - 1) * kKeys;  // keys of the last tile
    if (ok && n > 0 && cut < kKeys) {
      const uint32_t e = base + 2 * n - 1, s = e % S::kStages;
      ok = __all_sync(0xFFFFFFFFu, wait(&sm.full[s], e / S::kStages & 1, a.status));
      if (ok) {
        for (int p = 0; p < D / 64; ++p)
          for (int c = cut * 8 + lane; c < kKeys * 8; c += 32)
            *reinterpret_cast<uint4 *>(sm.kv[s] + p * (kKeys * 128) + c * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async();
      }
    }
    __syncwarp();
    if (ok && lane == 0 && !a.skip_tail) mbar_arrive(&sm.tail[t & 3]);
    base += issued;
    const Work was = w;
    w.valid = 0;
    for (uint32_t block; __all_sync(0xFFFFFFFFu, wait(&sm.next_full, (asked - 1) & 1, a.status)) && read_next(&sm.next, block);) {
      if (ok) w = find_work<SPLIT>(a, cursor, block, a.status);
      if (w.valid || !ok) break;
      fence_proxy_async();
      __syncwarp();
      ask();  // the grid is as large as it can be for these sizes: blocks past the last tile are taken over for nothing
    }
    w.step0 = (was.step0 + was.tiles0 + was.tiles1) % S::kBufs;
    w.s0 = (was.s0 + was.tiles0) % (2 * S::kBufs);
    w.s1 = (was.s1 + was.tiles1) % (2 * S::kBufs);
    w.entry0 = (was.entry0 + 2 * n) % (2 * S::kStages);
    w.o0 = was.o0 ^ (was.tiles0 > 0);
    w.o1 = was.o1 ^ (was.tiles1 > 0);
    const uint32_t slot = (t + 1) & 1;
    if (ok && t > 0) ok = __all_sync(0xFFFFFFFFu, wait(&sm.work_empty[slot], ((t + 1) / 2 - 1) & 1, a.status));
    if (!ok) w.valid = 0;
    fence_proxy_async();  // the answer has been read before another is asked for
    __syncwarp();
    if (ok && lane == 0) {
      sm.work[slot] = w;
      mbar_arrive(&sm.work_full[slot]);
    }
    if (!w.valid) break;
    issued = 0;
  }
  // no copy may be in flight when the block exits
#pragma unroll
  for (int x = 0; x < 2; ++x)
    if (queries[x] > 0) mbar_wait(&sm.q_full[x], (queries[x] - 1) & 1, kWaitNs);
  for (uint32_t j = 1; j <= S::kStages && j <= base; ++j) {
    const uint32_t e = base - j;
    mbar_wait(&sm.full[e % S::kStages], e / S::kStages & 1, kWaitNs);
  }
}

// ------------------------------------------------------------------ MMA issuer (one lane of warp 9)

template <class T, int D>
__device__ void mma_lane(const PromptArgs &a, Smem<D> &sm, uint32_t tmem) {
  using S = Smem<D>;
  constexpr uint32_t kType = T::kMmaType;
  constexpr uint32_t kBase = (1u << 4) | (kType << 7) | (kType << 10) | (uint32_t(kRows >> 4) << 24);
  constexpr uint32_t kDescS = kBase | (uint32_t(kKeys >> 3) << 17);
  constexpr uint32_t kDescO = kBase | (uint32_t(D >> 3) << 17) | (1u << 16);  // B is N-major
  constexpr uint32_t kTile = S::kTileBytes >> 4;                              // in a descriptor's address field
  const uint64_t qd0 = sw128_desc(smem_u32(sm.q[0])), kd0 = sw128_desc(smem_u32(sm.kv[0])), vd0 = v_desc(smem_u32(sm.kv[0]));
  // Two places in the list of a work's steps, the next S to issue (k...) and the next P V (v...): row tile, key tile, the
  // ring slot and phase of its K or V tile, the S buffer. Kept by increments, in registers: this lane's own latency is on
  // the critical path. (S of the next work under the last steps of this one was slower: a second place to issue S from
  // cost every step more than the works' ends gained.)
  int kslot = 0, kbuf = 0, kc0 = 0, kc1 = 0, vslot = 1, vbuf = 0;
  uint32_t kphase = 0, vphase = 0, pphase = 0;  // pphase: of the P buffers, flips when their ring starts over
  uint32_t qphase = 0;                          // bit x: of q_full[x]
  bool ok = true;
  for (uint32_t t = 0; ok; ++t) {
    if (!wait(&sm.work_full[t & 1], t >> 1 & 1, a.status)) break;
    const Work &w = sm.work[t & 1];
    if (!w.valid) break;
    const int tiles0 = w.tiles0, tiles1 = w.tiles1;
    const int n = max(tiles0, tiles1), m = min(tiles0, tiles1), longer = tiles1 > tiles0 ? 1 : 0, steps = tiles0 + tiles1;
    const bool cut = w.keys < n * kKeys;
    mbar_arrive(&sm.work_empty[t & 1]);
    int kx = m > 0 ? 0 : longer, kj = 0, vx = kx, vj = 0, issued = 0;
    bool kfresh = true, vfresh = true;  // the first step of its key tile
    const auto scores = [&] {           // S of the next step into its buffer
      if (kfresh && !wait(&sm.full[kslot], kphase, a.status)) return false;
      tmem_fence_after();
      const uint64_t qd = qd0 + (kx ? kTile : 0u), kd = kd0 + uint32_t(kslot) * kTile;
      const uint32_t d = tmem + kbuf * kKeys;
#pragma unroll
      for (int p = 0; p < D / 64; ++p)
#pragma unroll
        for (int c = 0; c < 4; ++c)  // 16 values are 32 bytes: 2 in the address field
          mma_ss(d, qd + p * (kRows * 128 >> 4) + 2 * c, kd + p * (kKeys * 128 >> 4) + 2 * c, kDescS, (p | c) != 0);
      mma_commit(&sm.s_full[kx][kx ? kc1 : kc0]);
      if (kx) {
        kc1 = kc1 + 1 == S::kBufs ? 0 : kc1 + 1;
      } else {
        kc0 = kc0 + 1 == S::kBufs ? 0 : kc0 + 1;
      }
      if (kj + 1 == (kx ? tiles1 : tiles0)) mma_commit(&sm.q_empty[kx]);
      kfresh = kx == 1 || kj >= m;  // the last step that reads this K tile
      if (kfresh) {
        mma_commit(&sm.empty[kslot]);
        ++kj;
        kx = kj < m ? 0 : longer;
        kslot += 2;
        if (kslot >= S::kStages) {
          kslot -= S::kStages;
          kphase ^= 1;
        }
      } else {
        kx = 1;
      }
      kbuf = kbuf + 1 == S::kBufs ? 0 : kbuf + 1;
      ++issued;
      return true;
    };
    while (ok && issued < S::kBufs && issued < steps) {
      if (kj == 0) {  // the first S of both row tiles are among these
        ok = wait(&sm.q_full[kx], qphase >> kx & 1, a.status);
        qphase ^= 1u << kx;
      }
      ok = ok && scores();
    }
    for (int q = 0; ok && q < steps; ++q) {
      if (vfresh)
        ok = wait(&sm.full[vslot], vphase, a.status) &&
             (!cut || vj + 1 < n || wait(&sm.tail[t & 3], t >> 2 & 1, a.status));
      ok = ok && wait(&sm.p_full[vbuf], pphase, a.status);
      if (!ok) break;
      tmem_fence_after();
      const uint64_t vd = vd0 + uint32_t(vslot) * kTile;
      const uint32_t pa = tmem + vbuf * kKeys, d = tmem + S::kColO + (vx ? D : 0);
#pragma unroll
      for (int c = 0; c < kKeys / 16; ++c)  // 16 keys: 8 columns of P, 2048 bytes of V
        mma_ts(d, pa + 8 * c, vd + c * (2048 >> 4), kDescO, (vj | c) != 0);
      if (issued < steps) ok = scores();
      if (vj + 1 == (vx ? tiles1 : tiles0)) mma_commit(&sm.o_full[vx]);
      vfresh = vx == 1 || vj >= m;
      if (vfresh) {
        mma_commit(&sm.empty[vslot]);
        ++vj;
        vx = vj < m ? 0 : longer;
        vslot += 2;
        if (vslot >= S::kStages) {
          vslot -= S::kStages;
          vphase ^= 1;
        }
      } else {
        vx = 1;
      }
      vbuf = vbuf + 1 == S::kBufs ? 0 : vbuf + 1;
      if (vbuf == 0) pphase ^= 1;
    }
  }
  mma_commit(&sm.mma_done);  // every MMA is done before TMEM is freed
  mbar_wait(&sm.mma_done, 0, kWaitNs);
}

// ------------------------------------------------------------------ softmax (warps 0-7)

// A row's scores of one key tile; keys from lim on are hidden.
__device__ __forceinline__ void load_scores(uint32_t ts, int lim, bool negative, uint32_t (&s)[kKeys]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, s + 32 * i);
#pragma unroll
  for (int i = 0; i < 4; ++i) tmem_wait_ld(s + 32 * i);
  if (negative) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) s[i] ^= 0x80000000u;
  }
  if (__any_sync(0xFFFFFFFFu, lim < kKeys)) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i)
      if (i >= lim) s[i] = 0xFF800000u;  // -inf
  }
}

// P = 2^(s scale2 + base) in 16 bits, the row's largest score, and the sum of P before its rounding.
template <class T>
__device__ __forceinline__ void exponentials(const uint32_t (&s)[kKeys], uint32_t (&p)[kKeys / 2], float scale2,
                                             float base, float &top, float &sum) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, add[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kKeys; i += 2) {
    const float x = __uint_as_float(s[i]), y = __uint_as_float(s[i + 1]);
    const int c = (i >> 1) & 3;
    mx[c] = fmaxf(mx[c], fmaxf(x, y));
    const float u = exp2_approx(fmaf(x, scale2, base)), v = exp2_approx(fmaf(y, scale2, base));
    add[c] += u + v;
    p[i / 2] = T::pack(u, v);
  }
  top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
  sum = (add[0] + add[1]) + (add[2] + add[3]);
}

template <class T, int D, bool SPLIT>
__device__ __forceinline__ bool softmax_work(const PromptArgs &a, Smem<D> &sm, const Work &w, uint32_t tmem) {
  using S = Smem<D>;
  const int x = threadIdx.x >> 7, row = threadIdx.x & 127, warp = row >> 5;
  // the thread's row of the sequence and its head; rows past the tile's tokens or the sequence see nothing
  const int t = w.t0 + x * a.tokens + row / a.group, h = w.head0 + row % a.group;
  bool real = row < a.tokens * a.group && t < w.n;
  if (real) real = row_ok(a, w.row0 + t, h);
  const int skip = SPLIT ? w.skip : 0;
  const int limit = real ? key_limit(a, w.keys + skip, w.n, t) - skip : 0;
  const uint32_t lanes = uint32_t(warp * 32) << 16;
  const uint32_t to = tmem + lanes + S::kColO + x * D;
  float ref = 0.0f, total = 0.0f;  // the reference in score units, a.up below the score that it stands for
  bool ok = true;
  const int tiles = w.tiles(x), both = w.both(), step0 = w.step0, s0 = x ? w.s1 : w.s0;
  for (int j = 0; j < tiles; ++j) {
    const int b = (step0 + (j < both ? 2 * j + x : both + j)) % S::kBufs, c = s0 + j;
    const uint32_t ts = tmem + lanes + b * kKeys;
    ok = __all_sync(0xFFFFFFFFu, wait(&sm.s_full[x][c % S::kBufs], (c / S::kBufs) & 1, a.status));
    if (!ok) return false;
    tmem_fence_after();
    const int lim = limit - j * kKeys;
    uint32_t s[kKeys], p[kKeys / 2];
    float top, sum;
    load_scores(ts, lim, a.negative, s);
    bool redo = true;
    if (j > 0) {  // with the reference as it is; the maximum only says whether that was good enough
      exponentials<T>(s, p, a.scale2, -ref * a.scale2, top, sum);
      redo = __any_sync(0xFFFFFFFFu, (top - ref) * a.scale2 > kLazy + T::kWeightUp);
      if (redo) load_scores(ts, lim, a.negative, s);  // P is not stored yet: S is still there
    }
    if (redo) {
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < kKeys; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(s[i]));
      top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (j == 0) {
        ref = fmaxf(T::kWeightUp != 0.0f ? top - a.up : top, a.lowest);
      } else {
        // O has to hold every tile before this one: then V of key tile j - 1 has been released. (Its slot is not
        // released again before this step is done, and was not in an older phase when S of this step was issued.)
        const int i = w.entry0 + 2 * j - 1;
        ok = __all_sync(0xFFFFFFFFu, wait(&sm.empty[i % S::kStages], (i / S::kStages) & 1, a.status));
        if (!ok) return false;
        tmem_fence_after();
        const bool move = (top - ref) * a.scale2 > kLazy + T::kWeightUp;
        if constexpr (T::kWeightUp != 0.0f) top -= a.up;
        const float f = move ? exp2_approx((ref - top) * a.scale2) : 1.0f;
        if (move) ref = top;
        total *= f;
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
      exponentials<T>(s, p, a.scale2, -ref * a.scale2, top, sum);
    }
    total += sum;
    tmem_st32(ts, p);
    tmem_st32(ts + 32, p + 32);
    tmem_wait_st();
    tmem_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.p_full[b]);
  }
  if (w.tiles(x) > 0) {
    if (!__all_sync(0xFFFFFFFFu, wait(&sm.o_full[x], x ? w.o1 : w.o0, a.status))) return false;
    tmem_fence_after();
  }
  if constexpr (SPLIT) {
    if (w.parts > 1) {  // as it is, for the join
      if (real) real = index_ok(a.status, int64_t(w.slot) * 2 + x, a.part_cap);
      float *const part = a.parts + (int64_t(w.slot) * 2 + x) * kRows * (D + 2);
      if (real) {
        part[kRows * D + row] = total != 0.0f ? ref * a.scale2 : -INFINITY;
        part[kRows * D + kRows + row] = total;
      }
      if (tiles > 0) {
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          uint32_t o[32];
          tmem_ld32(to + 32 * i, o);
          tmem_wait_ld(o);
          if (real) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint4 *>(part + row * D + 32 * i + 4 * c) =
                  make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          }
        }
      }
      return true;
    }
  }
  // O / sum. Rows of 256 bytes go through the warp's own shared memory, 64 values of 32 rows at a time, and out by whole
  // pieces of rows (16-byte pieces exchanged by row, against bank conflicts); rows of 128 straight from their threads.
  // 16 packed prompts with D = 128: 77 us, 81 straight; chunks with D = 64: 140 us straight, 145 through shared memory.
  const float inv = total != 0.0f ? 1.0f / total : 0.0f;  // a NaN stays one
  const bool any = limit > 0;  // a row without keys has no accumulator of its own
  const auto load_out = [&](int first, uint32_t (&v)[16]) {  // 32 values of the row from the first on
    uint32_t o[32];
    if (w.tiles(x) > 0) {
      tmem_ld32(to + first, o);
      tmem_wait_ld(o);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      v[i] = any ? T::pack(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv) : 0u;
  };
  if constexpr (D == 64) {
    uint16_t *out = a.out + int64_t(w.row0 + t) * a.out_stride + int64_t(h) * D;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t v[16];
      load_out(32 * i, v);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (real)
          *reinterpret_cast<uint4 *>(out + 32 * i + 8 * c) = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    }
  } else {
    uint8_t *stage = sm.out[threadIdx.x >> 5];
    const int lane = threadIdx.x & 31;
    constexpr int kStep = 4;  // rows that a warp stores at once, 8 lanes each
    const int c8 = lane % 8, l8 = lane / 8, dt = kStep / a.group, dh = kStep - dt * a.group;
    const int64_t step = dt * a.out_stride + dh * D, wrap = a.out_stride - a.group * D;
    const int rows = a.tokens * a.group;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t v[16];
        load_out(64 * half + 32 * i, v);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4 *>(stage + lane * 128 + (((4 * i + c) ^ (lane & 7)) << 4)) =
              make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
      }
      __syncwarp();
      int rr = warp * 32 + l8, tt = w.t0 + x * a.tokens + rr / a.group, hh = rr % a.group;
      uint16_t *out = a.out + int64_t(w.row0 + tt) * a.out_stride + int64_t(w.head0 + hh) * D + 64 * half + 8 * c8;
#pragma unroll
      for (int i = 0; i < 32; i += kStep) {
        if (rr < rows && tt < w.n && row_ok(a, w.row0 + tt, w.head0 + hh))
          *reinterpret_cast<uint4 *>(out) =
              *reinterpret_cast<const uint4 *>(stage + (l8 + i) * 128 + ((c8 ^ ((l8 + i) & 7)) << 4));
        rr += kStep;
        tt += dt;
        hh += dh;
        out += step;
        if (hh >= a.group) {
          hh -= a.group;
          ++tt;
          out += wrap;
        }
      }
      __syncwarp();
    }
  }
  if (real && a.lse)
    a.lse[int64_t(w.row0 + t) * a.num_heads + h] =
        total != 0.0f ? (log2f(total) + ref * a.scale2) * 0.6931471805599453f : -INFINITY;
  return true;
}

template <class T, int D, bool SPLIT>
__device__ void softmax_warps(const PromptArgs &a, Smem<D> &sm, uint32_t tmem) {
  using S = Smem<D>;
  int64_t ns = kWaitNs;
  for (uint32_t t = 0;; ++t) {
    if (!__all_sync(0xFFFFFFFFu, wait(&sm.work_full[t & 1], t >> 1 & 1, a.status, ns))) return;
    const Work &w = sm.work[t & 1];
    if (!w.valid) return;
    if (!softmax_work<T, D, SPLIT>(a, sm, w, tmem)) return;
    // the next work comes when the loads of this one are out; a warp whose own row tile is short waits for the other's
    ns = kWaitNs + int64_t(w.all()) * 100000;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.work_empty[t & 1]);
  }
}

// ------------------------------------------------------------------ kernel

template <class T, int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) attend_prompt_kernel(const __grid_constant__ CUtensorMap qmap,
                                                                    const __grid_constant__ CUtensorMap kmap,
                                                                    const __grid_constant__ CUtensorMap vmap,
                                                                    const PromptArgs a) {
  extern __shared__ unsigned char prompt_smem_raw[];
  using S = Smem<D>;
  static_assert(sizeof(S) + 1024 <= S::kBytes && S::kBytes <= 227 * 1024, "shared memory budget");
  S &sm = *reinterpret_cast<S *>((reinterpret_cast<uintptr_t>(prompt_smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  // every warp finds the block's first work for itself: nothing to wait for
  TileCursor cursor;
  const Work w = find_work<SPLIT>(a, cursor, blockIdx.x, warp == kWarpLoad ? a.status : nullptr);
  if (!w.valid) return;  // past the last tile: the whole block
  if (warp == kWarpLoad) {
    if (elect_one()) {
      mbar_init(&sm.next_full, 1);
      for (int i = 0; i < S::kStages; ++i) {
        mbar_init(&sm.full[i], 1);
        mbar_init(&sm.empty[i], 1);
      }
      for (int i = 0; i < 4; ++i) mbar_init(&sm.tail[i], 1);
      for (int i = 0; i < S::kBufs; ++i) mbar_init(&sm.p_full[i], 4);
      for (int x = 0; x < 2; ++x) {
        mbar_init(&sm.work_full[x], 1);
        mbar_init(&sm.work_empty[x], 9);
        mbar_init(&sm.q_full[x], 1);
        mbar_init(&sm.q_empty[x], 1);
        for (int i = 0; i < S::kBufs; ++i) mbar_init(&sm.s_full[x][i], 1);
        mbar_init(&sm.o_full[x], 1);
      }
      mbar_init(&sm.mma_done, 1);
      fence_mbar_init();
      fence_proxy_async();  // the copies' completions go to these barriers
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (w.tiles(x) > 0) load_queries<D>(&qmap, a, sm, w, x);
      for (int i = 0; i < S::kStages && i < 2 * w.all(); ++i) load_tile<D>(&kmap, &vmap, a, sm, w, 0, i);
      sm.work[0] = w;
      mbar_arrive(&sm.work_full[0]);
    }
  } else if (warp == kWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = sm.tmem_base;
  if (warp < kWarpLoad) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    softmax_warps<T, D, SPLIT>(a, sm, tmem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kWarpLoad) load_warp<D, SPLIT>(&qmap, &kmap, &vmap, a, sm, w);
    if (warp == kWarpMma && elect_one()) mma_lane<T, D>(a, sm, tmem);
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == kWarpMma)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ------------------------------------------------------------------ joining the parts of split keys
// A block for 32 rows of a tile, a warp for a row at a time: the parts' references and sums a lane each, then O.
constexpr int kJoinThreads = 256, kJoinRows = 32;

template <class T, int D>
__global__ void __launch_bounds__(kJoinThreads) join_prompt_kernel(const PromptArgs a) {
  static_assert(kMaxSplits <= 32, "a lane for each part");
  TileCursor cursor;
  const Work w = find_work<true>(a, cursor, blockIdx.x * uint32_t(a.splits), nullptr);
  if (!w.valid || w.parts == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int64_t kPart = 2 * kRows * (D + 2);
  for (int i = 0; i < kJoinRows / (kJoinThreads / 32); ++i) {
    const int r = int(blockIdx.y) * kJoinRows + i * (kJoinThreads / 32) + warp, x = r / kRows, row = r % kRows;
    const int t = w.t0 + x * a.tokens + row / a.group, h = w.head0 + row % a.group;
    if (row >= a.tokens * a.group || t >= w.n) continue;
    if (!row_ok(a, w.row0 + t, h) || !index_ok(a.status, w.parts - 1, kMaxSplits) ||
        !index_ok(a.status, int64_t(w.slot + w.parts - 1) * 2 + x, a.part_cap))
      continue;
    const float *const from = a.parts + w.slot * kPart + int64_t(x) * kRows * (D + 2);
    float ref = -INFINITY, sum = 0.0f;  // a part without a weight for the row has no say in the reference
    if (lane < w.parts) {
      ref = from[lane * kPart + kRows * D + row];
      sum = from[lane * kPart + kRows * D + kRows + row];
    }
    float top = ref;
#pragma unroll
    for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const float weight = sum != 0.0f ? exp2_approx(ref - top) : 0.0f;  // a part in which the row sees no key has no O
    float total = weight * sum;
#pragma unroll
    for (int d = 16; d; d /= 2) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p = 0; p < w.parts; ++p) {
      const float f = __shfl_sync(0xFFFFFFFFu, weight, p);
      if (f == 0.0f || lane >= D / 4) continue;
      const float4 v = *reinterpret_cast<const float4 *>(from + p * kPart + row * D + 4 * lane);
      o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
    }
    const float inv = total > 0.0f ? 1.0f / total : total;  // 0, or a NaN: also of a part whose O has no weight
    if (lane < D / 4)
      *reinterpret_cast<uint2 *>(a.out + int64_t(w.row0 + t) * a.out_stride + int64_t(h) * D + 4 * lane) =
          total != 0.0f ? make_uint2(T::pack(o.x * inv, o.y * inv), T::pack(o.z * inv, o.w * inv)) : make_uint2(0, 0);
    if (lane == 0 && a.lse)
      a.lse[int64_t(w.row0 + t) * a.num_heads + h] =
          total != 0.0f ? (log2f(total) + top) * 0.6931471805599453f : -INFINITY;
  }
}

// ------------------------------------------------------------------ host

// Boxes of 64 values x `heads` heads x `rows` rows, 128-byte swizzle, over [total][all_heads][dim] with the caller's row stride.
bool encode(CUtensorMap *map, const void *base, int dim, int all_heads, int64_t total, int64_t stride, int heads, int rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {cuuint64_t(dim), cuuint64_t(all_heads), cuuint64_t(total)};
  const cuuint64_t strides[2] = {cuuint64_t(dim) * 2, cuuint64_t(stride) * 2};
  const cuuint32_t box[3] = {64, cuuint32_t(heads), cuuint32_t(rows)}, estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
  CUtensorMap q, k, v;
};

// The most works that these sizes can have.
int64_t works_bound(const PromptArgs &a) { return (int64_t(a.num_rows) / (2 * a.tokens) + a.num_seqs) * a.all_groups; }

// Heads that share a row tile, and what follows from them.
void set_groups(const moe_attend_prompt_io_t &io, PromptArgs &a) {
  const int group = io.num_heads / io.num_kv_heads;
  a.group = group < kRows ? group : kRows;
  while (group % a.group) --a.group;
  a.groups = group / a.group;
  a.all_groups = io.num_heads / a.group;
  a.tokens = kRows / a.group;
  a.num_rows = io.num_rows;
  a.num_seqs = io.num_seqs;
}

// The keys are split where the works alone leave half of the GPU idle and the keys suffice for three parts (the join is
// a kernel of its own: 64 rows over 1,024 keys take 25 us in two parts, 21 in one). 32 + 8 heads of 128, 32,768 keys:
// one row 40 us (364 in one part), 64 rows 71 (395), 512 rows 231 (399).
int splits_of(const PromptArgs &a, int num_keys, int num_sms) {
  const int64_t works = works_bound(a);
  if (works < 1 || num_keys < 3 * kSplitTiles * kKeys) return 1;
  int64_t s = num_sms / works;
  s = s < kMaxSplits ? s : kMaxSplits;
  s = s < num_keys / (kSplitTiles * kKeys) ? s : num_keys / (kSplitTiles * kKeys);
  return s < 1 ? 1 : int(s);
}

template <class T, int D, bool SPLIT>
cudaError_t launch(const Maps &maps, const PromptArgs &a, cudaStream_t st) {
  const int64_t works = works_bound(a), blocks = works * (SPLIT ? a.splits : 1);
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  // The register split above assumes the launch's share: a build that gave the kernel less must not run. Only the answer
  // is remembered, not a query that failed.
  static std::atomic<int> regs{0};
  if (!regs.load(std::memory_order_relaxed)) {
    cudaFuncAttributes at;
    const cudaError_t asked = cudaFuncGetAttributes(&at, attend_prompt_kernel<T, D, SPLIT>);
    if (asked != cudaSuccess) return asked;
    regs.store(at.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != kRegsLaunch) return cudaErrorInvalidConfiguration;
  const cudaError_t e = cudaFuncSetAttribute(attend_prompt_kernel<T, D, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(Smem<D>::kBytes));
  if (e != cudaSuccess) return e;
  attend_prompt_kernel<T, D, SPLIT><<<unsigned(blocks), kThreads, Smem<D>::kBytes, st>>>(
      maps.q, maps.k, maps.v, a);
  if constexpr (SPLIT) {
    const cudaError_t launched = cudaGetLastError();
    if (launched != cudaSuccess) return launched;
    join_prompt_kernel<T, D><<<dim3(unsigned(works), 2 * kRows / kJoinRows), kJoinThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

int64_t attend_prompt_workspace(const moe_attend_prompt_io_t &io, int num_sms) {
  if (io.num_rows == 0 || io.num_seqs == 0) return 0;
  PromptArgs a = {};
  set_groups(io, a);
  const int splits = splits_of(a, io.num_keys, num_sms);
  return splits > 1 ? works_bound(a) * splits * 2 * kRows * (io.head_dim + 2) * 4 : 0;
}

cudaError_t launch_attend_prompt(const moe_attend_prompt_io_t &io, int32_t *status, int num_sms, cudaStream_t st) {
  PromptArgs a = {};
  a.out = static_cast<uint16_t *>(io.out);
  a.out_stride = io.out_stride;
  a.lse = io.lse;
  a.cu_rows = io.cu_rows;
  a.cu_keys = io.cu_keys;
  a.num_seqs = io.num_seqs;
  a.num_rows = io.num_rows;
  a.num_keys = io.num_keys;
  a.num_heads = io.num_heads;
  set_groups(io, a);
  a.splits = io.workspace ? splits_of(a, io.num_keys, num_sms) : 1;
  a.parts = static_cast<float *>(io.workspace);
  a.part_cap = checked_capacity(io.workspace ? io.workspace_bytes / (int64_t(kRows) * (io.head_dim + 2) * 4) : 0, io.flags);
  a.causal = io.causal;
  a.skip_tail = io.flags & MOE_FLAG_TEST_SKIP_READY;
  a.scale2 = fmaxf(fabsf(io.scale) * 1.4426950408889634f, 0x1p-100f);
  a.up = io.dtype == MOE_DTYPE_F16 ? F16::kWeightUp / a.scale2 : 0.0f;
  a.lowest = -3e38f / fmaxf(a.scale2, 1.0f);  // times scale2 it is finite
  a.negative = io.scale < 0.0f;
  a.status = status;
  const int D = io.head_dim;
  Maps maps;
  memset(&maps, 0, sizeof maps);
  if (!encode(&maps.q, io.q, D, io.num_heads, io.num_rows, io.q_stride, a.group, a.tokens)) return cudaErrorInvalidValue;
  if (io.num_keys && (!encode(&maps.k, io.k, D, io.num_kv_heads, io.num_keys, io.k_stride, 1, kKeys) ||
                      !encode(&maps.v, io.v, D, io.num_kv_heads, io.num_keys, io.v_stride, 1, kKeys)))
    return cudaErrorInvalidValue;
  const bool h = io.dtype == MOE_DTYPE_F16;
  if (a.splits > 1) {
    if (D == 64) return h ? launch<F16, 64, true>(maps, a, st) : launch<Bf16, 64, true>(maps, a, st);
    return h ? launch<F16, 128, true>(maps, a, st) : launch<Bf16, 128, true>(maps, a, st);
  }
  if (D == 64) return h ? launch<F16, 64, false>(maps, a, st) : launch<Bf16, 64, false>(maps, a, st);
  return h ? launch<F16, 128, false>(maps, a, st) : launch<Bf16, 128, false>(maps, a, st);
}

}  // namespace moe
