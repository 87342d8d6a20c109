// verify_drafts.cu — drafted tokens against the target's probabilities, and the token behind them.
//
// Mathematics. p = softmax(x / t) over the vocabulary, x the logits behind a row.
// A row's children are asked in their order. With the probabilities q that they
// were drawn from, what is left after k rejections is p_k = max(p_(k-1) - q, 0) /
// sum; by induction max(p - c_k q, 0) / N_k with c_0 = 0, N_0 = 1, c_(k+1) = c_k + N_k
// and N_k the sum, so a rejection costs one pass over the vocabulary and one
// number. Without q a rejected token's p becomes 0 and no pass is needed: N is 1
// minus what was taken off. The new token is the first whose running sum exceeds u times the whole.
//
// Accuracy. A decision compares numbers of relative error 2^-20: it is the
// formula's unless u lies that close to the border. The new token has a border for each
// token: with 2^17 tokens sums off by 2^-24 of the whole (one rounding of a large
// weight) would give another token once in some hundred draws. So the weights
// that a token is chosen from are computed in two binary32 each (a table of 2^(k/32) and a
// polynomial, about 2^-36 relative), and their sums are kept in two as well; binary64 runs at a
// hundredth of the rate here.
//
// Bound. Only the rows on the way are read: with one accepted child after another
// the rows come one after another, each a pass over the vocabulary that ends in a barrier. A cluster of
// blocks takes a sequence, and each block a part of the vocabulary.
//
// Layout. A block's warps have consecutive parts of its part, in units of 8
// tokens, a unit a lane. What every warp finds goes to a slot of its own in every block of the cluster
// (distributed shared memory), and every warp of every block joins all slots in the same order: all hold the
// same numbers, and walk the tree alike without telling one another. The slots lie in the order of
// the vocabulary, so they also say which warp's part holds the new token.
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "attention.cuh"
#include "speculative.h"

namespace moe {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kUnit = 8;  // tokens that a lane takes at a time

struct VerifyArgs {
  const void *logits;
  int64_t logits_stride;
  const float *draft;
  int64_t draft_stride;
  const int32_t *tokens, *parents, *cu_rows;
  const float *temperature, *accept_u, *sample_u;
  int32_t *out_tokens, *path, *accepted;
  int num_rows, max_rows, vocab;
  int32_t *status;
  float2 powers[32];  // 2^(k/32) in two binary32
};

// ------------------------------------------------------------------ numbers in two binary32

struct Two {
  float hi, lo;
};

__device__ __forceinline__ Two add(Two a, float hi, float lo) {
  const float s = a.hi + hi, b = s - a.hi;
  return {s, a.lo + ((a.hi - (s - b)) + (hi - b)) + lo};
}

// Symmetric in a and b to the last bit.
__device__ __forceinline__ Two add(Two a, Two b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo);
  const float hi = s + e;
  return {hi, e - (hi - s)};
}

__device__ __forceinline__ bool less(Two a, Two b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }

__device__ __forceinline__ Two times(Two a, float f) {
  const float p = a.hi * f, e = fmaf(a.hi, f, -p) + a.lo * f, hi = p + e;
  return {hi, e - (hi - p)};
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log2(e) / t in two.
__device__ __forceinline__ Two exponent_unit(float t) {
  constexpr float kHi = 1.44269502f, kLo = float(1.4426950408889634074 - double(1.44269502f));
  const float hi = kHi / t;
  return {hi, (fmaf(-hi, t, kHi) + kLo) / t};
}

// 2^(d c) for d <= 0. With y = d c = n + k/32 + r, |r| <= 1/64: 2^y = 2^n 2^(k/32) (1 + z), z = 2^r - 1 by its series, the
// first term in two. Below 2^-126: 0.
__device__ __forceinline__ Two power(float d, Two c, const float2 *powers) {
  constexpr float kHi = 0.693147182f, kLo = float(0.69314718055994530942 - double(0.693147182f));  // ln 2
  constexpr float k2 = 0.240226507f, k3 = 0.0555041087f, k4 = 0.00961812911f;                      // ln 2^i / i!
  constexpr float kRound = 12582912.0f;                                                           // 1.5 2^23
  const float yh = d * c.hi, yl = fmaf(d, c.lo, fmaf(d, c.hi, -yh));
  const float at = fmaf(yh, 32.0f, kRound), r = fmaf(at - kRound, -0x1p-5f, yh);
  const int i = __float_as_int(at) - 0x4B400000;
  const float2 p = powers[i & 31];
  const float zh = r * kHi, both = r + yl;
  float zl = fmaf(yl, kHi, fmaf(r, kLo, fmaf(r, kHi, -zh)));
  zl = fmaf(both * both, fmaf(both, fmaf(both, k4, k3), k2), zl);
  const float sh = __fmul_rn(p.x, zh), hi = p.x + sh;
  const float lo = ((p.x - hi) + sh) + fmaf(p.x, zl, fmaf(p.x, zh, -sh)) + fmaf(p.y, zh, p.y);
  const float scale = __int_as_float(((i >> 5) + 127) << 23);
  const bool none = yh < -126.0f;
  return {none ? 0.0f : hi * scale, none ? 0.0f : lo * scale};
}

// ------------------------------------------------------------------ rows of the vocabulary

__device__ __forceinline__ float value(const float *p) { return __ldg(p); }
__device__ __forceinline__ float value(const __nv_bfloat16 *p) { return __bfloat162float(__ldg(p)); }
__device__ __forceinline__ float value(const __half *p) { return __half2float(__ldg(p)); }

__device__ __forceinline__ void unpack(uint4 v, float *x, const __nv_bfloat16 *) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = Bf16::lo(w[i]), x[2 * i + 1] = Bf16::hi(w[i]);
}
__device__ __forceinline__ void unpack(uint4 v, float *x, const __half *) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[2 * i] = F16::lo(w[i]), x[2 * i + 1] = F16::hi(w[i]);
}
__device__ __forceinline__ void unpack(uint4 v, float *x, const float *) {
  x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
}

// A row in units of 8 tokens that begin on 16-byte boundaries: the first and the last may be cut by the row's ends.
template <class E>
struct Row {
  const E *p;
  int shift, vocab;  // the first unit begins `shift` tokens in front of the row

  __device__ __forceinline__ Row(const void *base, int64_t stride, int64_t row, int v)
      : p(static_cast<const E *>(base) + row * stride), vocab(v) {
    shift = int((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(E));
  }
  __device__ __forceinline__ int units() const { return (vocab + shift + kUnit - 1) / kUnit; }
  __device__ __forceinline__ int first(int u) const { return u * kUnit - shift; }

  // The unit's logits; -inf past the row's ends.
  __device__ __forceinline__ void load(int u, float (&x)[kUnit]) const {
    const int e = first(u);
    if (e >= 0 && e + kUnit <= vocab) {
      constexpr int kPer = 16 / sizeof(E);
#pragma unroll
      for (int i = 0; i < kUnit / kPer; ++i)
        unpack(__ldg(reinterpret_cast<const uint4 *>(p + e) + i), x + i * kPer, static_cast<const E *>(nullptr));
    } else {
#pragma unroll
      for (int i = 0; i < kUnit; ++i) x[i] = e + i >= 0 && e + i < vocab ? value(p + e + i) : -INFINITY;
    }
  }
};

// Eight of the draft's probabilities from token e on, 0 past the row's ends.
__device__ __forceinline__ void load_draft(const float *p, int e, int vocab, float (&q)[kUnit]) {
  if (e >= 0 && e + kUnit <= vocab && (reinterpret_cast<uintptr_t>(p + e) & 15) == 0) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p + e)), b = __ldg(reinterpret_cast<const float4 *>(p + e) + 1);
    q[0] = a.x, q[1] = a.y, q[2] = a.z, q[3] = a.w, q[4] = b.x, q[5] = b.y, q[6] = b.z, q[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) q[i] = e + i >= 0 && e + i < vocab ? __ldg(p + e + i) : 0.0f;
  }
}

// ------------------------------------------------------------------ the cluster

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void store_remote(float4 *dst, uint32_t rank, float4 v) {
  asm volatile(
      "{\n\t.reg .u32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.v4.f32 [a], {%2, %3, %4, %5};\n\t}" ::"r"(smem_u32(dst)),
      "r"(rank), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
      : "memory");
}

struct Smem {
  float4 slots[2][kMaxCluster * kWarps];  // by block of the cluster and warp; two sets in turn
  float2 powers[32];
  float x[kMaxTree], q[kMaxTree], u[kMaxTree];  // of each row: its logit, its draft probability (both in its parent's row)
  int token[kMaxTree];
  int parent[kMaxTree];    // kNever: not asked
  int rejected[kMaxTree];  // tokens of the rejected children of the row
  int way[kMaxTree];       // accepted rows, the root first
};
constexpr int kNever = -2;

// Largest logit (and the first token that has it), and the sum of 2^((x - max) c).
struct Peak {
  float top, sum;
  int token;

  __device__ __forceinline__ void join(const Peak &o, float c) {
    const float t = fmaxf(top, o.top), ref = t == -INFINITY ? 0.0f : t;
    sum = sum * exp2_approx((top - ref) * c) + o.sum * exp2_approx((o.top - ref) * c);
    if (o.top > top || (o.top == top && o.token < token)) token = o.token;
    top = t;
  }
};

template <class E, bool DRAFT>
struct Walker {
  const VerifyArgs &a;
  Smem &sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank(), size = cluster_size();
  int set = 0;
  Two unit = {0.0f, 0.0f};  // log2(e) / temperature
  int count = 0;            // rejected tokens

  __device__ Walker(const VerifyArgs &args, Smem &smem) : a(args), sm(smem) {}

  // The warp's units of a row.
  __device__ __forceinline__ void part(const Row<E> &row, int &begin, int &end) const {
    const int units = row.units(), each = (units + int(size) * kWarps - 1) / (int(size) * kWarps);
    begin = min(units, (int(rank) * kWarps + warp) * each);
    end = min(units, begin + each);
  }

  // This warp's value into its slot everywhere; then all slots are there.
  __device__ __forceinline__ const float4 *exchange(float4 v) {
    float4 *slots = sm.slots[set];
    set ^= 1;
    if (lane < int(size)) store_remote(&slots[rank * kWarps + warp], lane, v);
    cluster_sync();
    return slots;
  }

  __device__ __forceinline__ Peak peak(const Row<E> &row) {
    int begin, end;
    part(row, begin, end);
    Peak k = {-INFINITY, 0.0f, INT32_MAX};
    const float c = unit.hi;
#pragma unroll 4
    for (int u = begin + lane; u < end; u += 32) {
      float x[kUnit];
      row.load(u, x);
      float t = x[0];
#pragma unroll
      for (int i = 1; i < kUnit; ++i) t = fmaxf(t, x[i]);
      if (t > k.top) {
        k.sum *= exp2_approx((k.top - t) * c);
        k.top = t;
#pragma unroll
        for (int i = kUnit - 1; i >= 0; --i)
          if (x[i] == t) k.token = row.first(u) + i;
      }
      const float ref = k.top == -INFINITY ? 0.0f : k.top;
#pragma unroll
      for (int i = 0; i < kUnit; ++i) k.sum += exp2_approx((x[i] - ref) * c);
    }
#pragma unroll
    for (int d = 16; d; d /= 2)
      k.join({__shfl_xor_sync(0xFFFFFFFFu, k.top, d), __shfl_xor_sync(0xFFFFFFFFu, k.sum, d),
              __shfl_xor_sync(0xFFFFFFFFu, k.token, d)},
             c);
    const float4 *slots = exchange(make_float4(k.top, k.sum, __int_as_float(k.token), 0.0f));
    k = {-INFINITY, 0.0f, INT32_MAX};
    for (int i = lane; i < int(size) * kWarps; i += 32) k.join({slots[i].x, slots[i].y, __float_as_int(slots[i].z)}, c);
#pragma unroll
    for (int d = 16; d; d /= 2)
      k.join({__shfl_xor_sync(0xFFFFFFFFu, k.top, d), __shfl_xor_sync(0xFFFFFFFFu, k.sum, d),
              __shfl_xor_sync(0xFFFFFFFFu, k.token, d)},
             c);
    return k;
  }

  // What is left of the unit's tokens: 2^((x - top) c) less taken q, or without the rejected tokens.
  __device__ __forceinline__ void left(const Row<E> &row, const float *draft, int u, float top, Two taken, Two (&w)[kUnit]) const {
    float x[kUnit], q[kUnit];
    row.load(u, x);
    const int e = row.first(u);
    if (DRAFT && taken.hi != 0.0f) load_draft(draft, e, row.vocab, q);
    if (!DRAFT) {
      for (int j = 0; j < count; ++j) {
        const int at = sm.rejected[j] - e;
#pragma unroll
        for (int i = 0; i < kUnit; ++i)
          if (at == i) x[i] = -INFINITY;
      }
    }
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      w[i] = power(x[i] - top, unit, sm.powers);
      if (DRAFT && taken.hi != 0.0f) {
        const float g = __fmul_rn(taken.hi, q[i]), gl = fmaf(taken.lo, q[i], fmaf(taken.hi, q[i], -g));
        const float s = w[i].hi - g, b = s - w[i].hi;
        const float lo = ((w[i].hi - (s - b)) - (g + b)) + (w[i].lo - gl), hi = s + lo;
        w[i] = hi > 0.0f ? Two{hi, lo - (hi - s)} : Two{0.0f, 0.0f};
      }
    }
  }

  // The warps' sums of what is left, in their slots.
  __device__ __forceinline__ const float4 *sums(const Row<E> &row, const float *draft, float top, Two taken) {
    int begin, end;
    part(row, begin, end);
    Two s = {0.0f, 0.0f};
    for (int u = begin + lane; u < end; u += 32) {
      Two w[kUnit];
      left(row, draft, u, top, taken, w);
#pragma unroll
      for (int i = 0; i < kUnit; ++i) s = add(s, w[i].hi, w[i].lo);
    }
    s = add(s, Two{0.0f, 0.0f});
#pragma unroll
    for (int d = 16; d; d /= 2)
      s = add(s, Two{__shfl_xor_sync(0xFFFFFFFFu, s.hi, d), __shfl_xor_sync(0xFFFFFFFFu, s.lo, d)});
    return exchange(make_float4(s.hi, s.lo, 0.0f, 0.0f));
  }

  // Sum of all of them.
  __device__ __forceinline__ Two whole(const float4 *slots) const {
    Two s = {0.0f, 0.0f};
    for (int i = lane; i < int(size) * kWarps; i += 32) s = add(s, Two{slots[i].x, slots[i].y});
#pragma unroll
    for (int d = 16; d; d /= 2)
      s = add(s, Two{__shfl_xor_sync(0xFFFFFFFFu, s.hi, d), __shfl_xor_sync(0xFFFFFFFFu, s.lo, d)});
    return s;
  }

  static __device__ __forceinline__ Two scan(Two s, int lane) {  // inclusive
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const Two o = {__shfl_up_sync(0xFFFFFFFFu, s.hi, d), __shfl_up_sync(0xFFFFFFFFu, s.lo, d)};
      if (lane >= d) s = add(o, s);
    }
    return s;
  }

  static __device__ __forceinline__ Two from_lane(Two s, int l) {
    return {__shfl_sync(0xFFFFFFFFu, s.hi, l), __shfl_sync(0xFFFFFFFFu, s.lo, l)};
  }

  // The new token, on one lane of the warp whose part holds it; -1 elsewhere. `total`: whether there was anything to choose from.
  __device__ int choose(const Row<E> &row, const float *draft, float top, Two taken, float u, bool &any) {
    const float4 *slots = sums(row, draft, top, taken);
    // running sums over the slots, consecutive ones a lane
    const int n = int(size) * kWarps, per = (n + 31) / 32;
    Two mine = {0.0f, 0.0f};
    for (int i = lane * per; i < min(n, lane * per + per); ++i) mine = add(mine, Two{slots[i].x, slots[i].y});
    const Two upto = scan(mine, lane), all = from_lane(upto, 31);
    any = all.hi > 0.0f;
    if (!any) return -1;
    const Two border = times(all, fminf(fmaxf(u, 0.0f), 1.0f));
    // the first slot whose running sum exceeds the border; by a rounding, or with u = 1, there may be none: the last that has
    // a weight
    Two run = {__shfl_up_sync(0xFFFFFFFFu, upto.hi, 1), __shfl_up_sync(0xFFFFFFFFu, upto.lo, 1)};
    if (lane == 0) run = {0.0f, 0.0f};
    int hit = INT32_MAX, last = -1;
    Two before = run, before_last = run;
    for (int i = lane * per; i < min(n, lane * per + per); ++i) {
      if (slots[i].x > 0.0f) {
        const Two next = add(run, Two{slots[i].x, slots[i].y});
        if (hit == INT32_MAX && less(border, next)) hit = i, before = run;
        last = i, before_last = run;
        run = next;
      }
    }
    const int first = __reduce_min_sync(0xFFFFFFFFu, hit);
    int owner = first;
    if (first == INT32_MAX) {
      owner = __reduce_max_sync(0xFFFFFFFFu, last);
      before = before_last;
    }
    before = from_lane(before, owner / per);
    if (owner != int(rank) * kWarps + warp) return -1;
    // this warp's part once more, 32 units at a time
    int begin, end;
    part(row, begin, end);
    int found = -1, positive = -1;
    for (int u0 = begin; u0 < end && found < 0; u0 += 32) {
      Two w[kUnit], s = {0.0f, 0.0f};
      const int unit_at = u0 + lane;
      if (unit_at < end) {
        left(row, draft, unit_at, top, taken, w);
      } else {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) w[i] = {0.0f, 0.0f};
      }
#pragma unroll
      for (int i = 0; i < kUnit; ++i) s = add(s, w[i].hi, w[i].lo);
      s = add(s, Two{0.0f, 0.0f});
      const Two to = scan(s, lane);
      const unsigned over = __ballot_sync(0xFFFFFFFFu, s.hi > 0.0f && less(border, add(before, to)));
      Two from = {__shfl_up_sync(0xFFFFFFFFu, to.hi, 1), __shfl_up_sync(0xFFFFFFFFu, to.lo, 1)};
      from = lane ? add(before, from) : before;
      int mine_found = -1;
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        if (w[i].hi > 0.0f) {
          positive = row.first(unit_at) + i;
          from = add(from, Two{w[i].hi, w[i].lo});
          if (mine_found < 0 && less(border, from)) mine_found = positive;
        }
      }
      if (mine_found < 0) mine_found = positive;
      if (over) found = __shfl_sync(0xFFFFFFFFu, mine_found, __ffs(over) - 1);
      before = add(before, from_lane(to, 31));
    }
    if (found < 0) found = __reduce_max_sync(0xFFFFFFFFu, positive);
    return lane == 0 ? found : -1;
  }
};

// A block of a cluster of one sequence.
template <class E, bool DRAFT>
__global__ void __launch_bounds__(kThreads) verify_drafts_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ Smem sm;
  Walker<E, DRAFT> w(a, sm);
  const int tid = threadIdx.x, lane = w.lane, b = int(blockIdx.x / w.size);
  int32_t *const status = w.rank == 0 ? a.status : nullptr;  // what is out of range is reported once
  int32_t *const out = a.out_tokens + int64_t(b) * a.max_rows, *const path = a.path + int64_t(b) * a.max_rows;
  Span rows = seq_span(a.cu_rows, b, a.num_rows, tid == 0 ? status : nullptr);
  if (rows.n > a.max_rows) {
    if (tid == 0) out_of_range(status);
    rows.n = -1;
  }
  if (rows.n <= 0) {  // the whole cluster
    if (w.rank == 0) {
      for (int j = tid; j < a.max_rows; j += kThreads) out[j] = path[j] = -1;
      if (tid == 0) a.accepted[b] = 0;
    }
    return;
  }
  const int n = rows.n;
  for (int i = tid; i < n; i += kThreads) {
    const int at = rows.first + i, token = __ldg(a.tokens + at);
    int parent = a.parents ? __ldg(a.parents + at) : i - 1;
    if (parent >= i) out_of_range(status);
    const bool good = token >= 0 && token < a.vocab;
    if (i > 0 && !good) out_of_range(status);
    if (i == 0 || parent < 0 || parent >= i || !good) parent = kNever;
    sm.parent[i] = parent;
    sm.token[i] = token;
    sm.u[i] = __ldg(a.accept_u + at);
    if (parent >= 0) {
      const int64_t row = rows.first + parent;
      sm.x[i] = value(static_cast<const E *>(a.logits) + row * a.logits_stride + token);
      sm.q[i] = DRAFT ? __ldg(a.draft + row * a.draft_stride + token) : 1.0f;
    }
  }
  if (tid < 32) sm.powers[tid] = a.powers[tid];
  if (tid == 0) sm.way[0] = 0;
  float t = a.temperature ? __ldg(a.temperature + b) : 1.0f;
  if (!(t >= 0.0f && t < INFINITY)) {
    if (tid == 0) out_of_range(status);
    t = 1.0f;
  }
  const bool greedy = t == 0.0f;
  w.unit = exponent_unit(greedy ? 1.0f : fmaxf(t, 0x1p-100f));
  __syncthreads();

  int node = 0, accepted = 0;
  Peak k;
  Two taken;   // c times the sum of all weights
  bool valid;  // there is a distribution
  while (true) {
    const Row<E> row(a.logits, a.logits_stride, rows.first + node, a.vocab);
    const float *draft = DRAFT ? a.draft + int64_t(rows.first + node) * a.draft_stride : nullptr;
    k = w.peak(row);
    valid = k.sum > 0.0f && k.sum < INFINITY && k.top > -INFINITY;
    if (!valid) break;
    taken = {0.0f, 0.0f};
    w.count = 0;
    float mass = 1.0f;  // N
    Two all = {0.0f, 0.0f}, rest = {0.0f, 0.0f};  // the sum of all weights, and N times it
    bool stale = false;  // N is to be computed
    int next = -1;
    for (int base = 0; base < n && next < 0; base += 32) {
      const int i0 = base + lane;
      unsigned asked = __ballot_sync(0xFFFFFFFFu, i0 < n && sm.parent[min(i0, n - 1)] == node);
      while (asked) {
        const int i = base + __ffs(asked) - 1;
        asked &= asked - 1;
        const int y = sm.token[i];
        bool yes;
        float p = exp2_approx((sm.x[i] - k.top) * w.unit.hi) / k.sum;
        if (greedy) {
          yes = y == k.token;
        } else if constexpr (DRAFT) {
          if (stale) {
            rest = w.whole(w.sums(row, draft, k.top, taken));
            mass = rest.hi / all.hi;
            stale = false;
          }
          yes = sm.u[i] * mass * sm.q[i] < p - taken.hi / k.sum * sm.q[i];
        } else {
          for (int j = 0; j < w.count; ++j)
            if (sm.rejected[j] == y) p = 0.0f;
          yes = sm.u[i] * mass < p;
        }
        if (yes) {
          next = i;
          break;
        }
        if (greedy) continue;
        if constexpr (DRAFT) {
          if (all.hi == 0.0f) all = rest = w.whole(w.sums(row, draft, k.top, taken));
          taken = add(taken, rest);
          stale = true;
        } else {
          mass = fmaxf(mass - p, 0.0f);
          __syncthreads();  // nobody reads the list
          if (tid == 0) sm.rejected[w.count] = y;
          ++w.count;
          __syncthreads();
        }
      }
    }
    if (next < 0) break;
    node = next;
    ++accepted;
    if (tid == 0) sm.way[accepted] = node;
  }
  __syncthreads();
  if (w.rank == 0) {
    for (int j = tid; j < a.max_rows; j += kThreads) {
      path[j] = j <= accepted ? sm.way[j] : -1;
      if (j != accepted) out[j] = j < accepted ? sm.token[sm.way[j + 1]] : -1;
    }
    if (tid == 0) {
      a.accepted[b] = accepted;
      if (!valid) out[accepted] = -1;
      if (valid && greedy) out[accepted] = k.token;
    }
  }
  if (!valid || greedy) return;
  const Row<E> row(a.logits, a.logits_stride, rows.first + node, a.vocab);
  const float *draft = DRAFT ? a.draft + int64_t(rows.first + node) * a.draft_stride : nullptr;
  const float u = __ldg(a.sample_u + b);
  bool any;
  int token = w.choose(row, draft, k.top, taken, u, any);
  if (!any) {  // nothing is left: the target's own probabilities
    w.count = 0;
    token = w.choose(row, draft, k.top, {0.0f, 0.0f}, u, any);
  }
  if (token >= 0) out[accepted] = token;
}

// ------------------------------------------------------------------ host

template <class E, bool DRAFT>
cudaError_t launch(const VerifyArgs &a, int num_seqs, int cluster, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(num_seqs) * unsigned(cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<E, DRAFT>, a);
}

struct Powers {
  float2 v[32];
  Powers() {
    for (int i = 0; i < 32; ++i) {
      const double p = std::exp2(i / 32.0);
      v[i].x = float(p);
      v[i].y = float(p - double(v[i].x));
    }
  }
};

}  // namespace

cudaError_t launch_verify_drafts(const moe_verify_drafts_io_t &io, int32_t *status, int num_sms, cudaStream_t st) {
  static const Powers powers;
  VerifyArgs a = {};
  a.logits = io.logits;
  a.logits_stride = io.logits_stride;
  a.draft = io.draft_probs;
  a.draft_stride = io.draft_stride;
  a.tokens = io.tokens;
  a.parents = io.parents;
  a.cu_rows = io.cu_rows;
  a.temperature = io.temperature;
  a.accept_u = io.accept_u;
  a.sample_u = io.sample_u;
  a.out_tokens = io.out_tokens;
  a.path = io.path;
  a.accepted = io.accepted;
  a.num_rows = io.num_rows;
  a.max_rows = io.max_rows;
  a.vocab = io.vocab;
  a.status = status;
  for (int i = 0; i < 32; ++i) a.powers[i] = powers.v[i];
  // blocks of a sequence: as many as fill the GPU twice, of 4096 tokens at least
  int cluster = 1;
  while (cluster < kMaxCluster && int64_t(io.num_seqs) * cluster < 2 * num_sms && io.vocab / (2 * cluster) >= 4096) cluster *= 2;
  const bool draft = io.draft_probs != nullptr;
  if (io.dtype == MOE_DTYPE_F32)
    return draft ? launch<float, true>(a, io.num_seqs, cluster, st) : launch<float, false>(a, io.num_seqs, cluster, st);
  if (io.dtype == MOE_DTYPE_F16)
    return draft ? launch<__half, true>(a, io.num_seqs, cluster, st) : launch<__half, false>(a, io.num_seqs, cluster, st);
  return draft ? launch<__nv_bfloat16, true>(a, io.num_seqs, cluster, st)
               : launch<__nv_bfloat16, false>(a, io.num_seqs, cluster, st);
}

}  // namespace moe
