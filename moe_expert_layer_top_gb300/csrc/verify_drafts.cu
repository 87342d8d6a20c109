// verify_drafts.cu — drafted tokens against the target's probabilities, and the token behind them.
//
// Mathematics. p = softmax(x / t) over the vocabulary, x the logits behind a row.
// A row's children are asked in their order. With the probabilities q that they
// were drawn from, what is left after k rejections is p_k = max(p_(k-1) - q, 0) /
// sum; by induction max(p - c_k q, 0) / N_k with c_0 = 0, N_0 = 1, c_(k+1) = c_k + N_k
// and N_k the sum, so a rejection costs one pass over the vocabulary and one
// number. Without q a rejected token's p becomes 0 and N is 1 minus what was taken off,
// without a pass until little is left. The new token is the first whose running sum exceeds u times the whole.
//
// Accuracy. A decision compares numbers of relative error 2^-20: it is the formula's unless u lies that close to the
// border. To keep that behind rejections, where both sides are what is left of larger numbers, the child's weight and the
// sums are held in two binary32. The new token has a border for each token: with 2^17 tokens sums off by 2^-24 of the
// whole (one rounding of a large weight) would give another token once in some hundred draws. So the weights that a token
// is chosen from are computed in two binary32 each where they are large (a table of 2^(k/32) and a polynomial, about 2^-36
// relative) or next to what the draft takes of them, in one without a bias where they are not, and their sums are kept in
// two; binary64 runs at a hundredth of the rate here.
//
// Bound. Only the rows on the way are read: with one accepted child after another the rows come one after another, each a
// pass over the vocabulary that ends in a barrier. A cluster of blocks takes a sequence, and each block a part of the
// vocabulary.
//   Measured (131,072 tokens, device time in a graph): one chain of six in bf16 13 us, of a single row 6; 64 chains of
// six with a draft, fp32, 71 us, of single rows 11 to 15; 16 trees of 64 rows 23 to 30; 24 of up to 16 rows with a draft over
// 50,021 tokens 37 to 42. Issue slots are 20 to 30 % busy, HBM 4 to 23 %: rows one after another, each a chain of latencies.
//
// Layout. A block's warps have consecutive parts of its part, in units of 8 tokens, a unit a lane. What every warp finds
// goes to a slot of its own in every block of the cluster (distributed shared memory), and every warp of every block
// joins all slots in the same order (peak.h): all hold the same numbers, and walk the tree alike without telling one
// another. The slots lie in the order of the vocabulary, so they also say which warp's part holds the new token.
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "attention.cuh"
#include "peak.h"
#include "speculative.h"

namespace moe {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kBatch = 4;  // units of a lane on their way at once
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

// a - b in two, without an error.
__device__ __forceinline__ Two minus(float a, float b) {
  const float s = a - b, c = s - a;
  return {s, (a - (s - c)) - (b + c)};
}

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
// first term in two. Below 2^-126: 0. The low part reaches 2^-14 of the high one.
__device__ __forceinline__ Two power(Two d, Two c, const float2 *powers) {
  constexpr float kHi = 0.693147182f, kLo = float(0.69314718055994530942 - double(0.693147182f));  // ln 2
  constexpr float k2 = 0.240226507f, k3 = 0.0555041087f, k4 = 0.00961812911f;                      // ln 2^i / i!
  constexpr float kRound = 12582912.0f;                                                           // 1.5 2^23
  const float yh = d.hi * c.hi, yl = fmaf(d.lo, c.hi, fmaf(d.hi, c.lo, fmaf(d.hi, c.hi, -yh)));
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

// The same with 2^-22 relative, by the exponential instruction.
__device__ __forceinline__ float power_approx(Two d, Two c) {
  const float y = d.hi * c.hi, yl = fmaf(d.lo, c.hi, fmaf(d.hi, c.lo, fmaf(d.hi, c.hi, -y))), p = exp2_approx(y);
  return y < -126.0f ? 0.0f : fmaf(p * 0.693147182f, yl, p);
}

// In one binary32: 2^-23 relative, from roundings without a common sign (the series leaves 2^-28 off at its
// ends, 2^-31 on the whole). d >= -126 / c. With y = n - g: n from y's rounding, g exact but for one rounding. (Two at a
// time with the packed instructions took more, for the constants, which those cannot take from the instruction.)
__device__ __forceinline__ float power_short(float d, float lo, Two c) {
  constexpr float k1 = 0.693147182f, k2 = 0.240226507f, k3 = 0.0555041087f, k4 = 0.00961812911f, k5 = 0.00133335581f,
                  k6 = 0.000154035304f, k7 = 1.52527338e-05f;  // ln 2^i / i!
  const float at = fmaf(d, c.hi, 12582912.0f);  // 1.5 2^23 + n
  const float f = fmaf(lo, c.hi, fmaf(d, c.lo, fmaf(d, c.hi, 12582912.0f - at)));
  const float q = fmaf(f, fmaf(f, fmaf(f, fmaf(f, fmaf(f, fmaf(f, k7, k6), k5), k4), k3), k2), k1);
  return fmaf(f, q, 1.0f) * __int_as_float((__float_as_int(at) << 23) + 0x3F800000);  // the low bits of `at` into the exponent
}

// Weights of this part of the largest and more are computed in two binary32, the others in one. With 2^16 tokens, a fifth
// of the whole below it, the running sums are then off by 2^-34 of the whole; with 2^-12 by 2^-33, with 2^-16 by 2^-35.
constexpr float kShort = 0x1p-13f;
// Weights below 2^-126 of the largest are computed as that: what is less than kNothing is no weight, and no sum of them
// either.
constexpr float kNothing = 0x1p-100f;

// With a draft: tokens of which less than this part of c q is left or missing are computed in two binary32 as well. In one
// they would have the rounding of the weight, 2^-23 of it, cut off below 0: where the draft is nearly the target, all that
// is left would be that (a part of 2^-26 of the weights, next to a true residual of any size).
constexpr float kNear = 0x1p-18f;
// What is left behind rejections of less than this part of all weights is nothing: it is of the size of the sums' errors.
constexpr float kRest = 0x1p-30f;

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

// Values from p[e] on, `none` in front of the row and behind it. Out of line, as all that is rare or called in several
// places: a call runs most of this code once, from a cold instruction cache (with everything inline the kernels had 125
// and 180 KB; one chain took 12.7 us).
template <class E>
__device__ __noinline__ void load_cut(const E *p, int e, int vocab, float none, float *x) {
#pragma unroll 1
  for (int i = 0; i < kUnit; ++i) x[i] = e + i >= 0 && e + i < vocab ? value(p + e + i) : none;
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

  // Units [a, b) lie in the row as a whole.
  __device__ __forceinline__ bool whole(int a, int b) const { return first(a) >= 0 && first(b) <= vocab; }

  // The logits of a unit that does.
  static constexpr int kPer = 16 / sizeof(E), kPieces = kUnit / kPer;  // of a 16-byte piece; pieces
  __device__ __forceinline__ void ask(int u, uint4 (&v)[kPieces]) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(p + first(u)) + i);
  }
  static __device__ __forceinline__ void take(const uint4 (&v)[kPieces], float (&x)[kUnit]) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) unpack(v[i], x + i * kPer, static_cast<const E *>(nullptr));
  }

  // The unit's logits; -inf past the row's ends.
  __device__ __forceinline__ void load(int u, float (&x)[kUnit]) const {
    const int e = first(u);
    if (whole(u, u + 1)) {
      uint4 v[kPieces];
      ask(u, v);
      take(v, x);
    } else {
      float c[kUnit];
      load_cut(p, e, vocab, -INFINITY, c);
#pragma unroll
      for (int i = 0; i < kUnit; ++i) x[i] = c[i];
    }
  }
};

// Eight of the draft's probabilities from token e on, 0 past the row's ends.
__device__ __forceinline__ void load_draft(const float *p, int e, int vocab, float (&q)[kUnit]) {
  if (e >= 0 && e + kUnit <= vocab && (reinterpret_cast<uintptr_t>(p + e) & 15) == 0) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p + e)), b = __ldg(reinterpret_cast<const float4 *>(p + e) + 1);
    q[0] = a.x, q[1] = a.y, q[2] = a.z, q[3] = a.w, q[4] = b.x, q[5] = b.y, q[6] = b.z, q[7] = b.w;
  } else {
    float c[kUnit];
    load_cut(p, e, vocab, 0.0f, c);
#pragma unroll
    for (int i = 0; i < kUnit; ++i) q[i] = c[i];
  }
}

// ------------------------------------------------------------------ the cluster

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
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
  float2 large[kWarps][32 * kUnit + 32];  // logits (and draft probabilities) of weights to be in two, until there are 32
  Two part[kWarps];        // sums of the warps where the new token is looked for, and what they found
  int found[kWarps];
};
constexpr int kNever = -2;

template <class E, bool DRAFT>
struct Walker {
  const VerifyArgs &a;
  Smem &sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank(), size = cluster_size();
  int set = 0;
  Two unit = {0.0f, 0.0f};  // log2(e) / temperature
  float least = 0.0f;       // -126 of it
  int count = 0;            // rejected tokens

  __device__ Walker(const VerifyArgs &args, Smem &smem) : a(args), sm(smem) {}

  // The warp's units of a row.
  __device__ __forceinline__ void part(const Row<E> &row, int &begin, int &end) const {
    const int units = row.units(), each = (units + int(size) * kWarps - 1) / (int(size) * kWarps);
    begin = min(units, (int(rank) * kWarps + warp) * each);
    end = min(units, begin + each);
  }

  // This warp's value (its first lane's: every block gets the same) into its slot everywhere; then all slots are there.
  __device__ __forceinline__ const float4 *exchange(float4 v) {
    v = make_float4(__shfl_sync(0xFFFFFFFFu, v.x, 0), __shfl_sync(0xFFFFFFFFu, v.y, 0), __shfl_sync(0xFFFFFFFFu, v.z, 0),
                    __shfl_sync(0xFFFFFFFFu, v.w, 0));
    float4 *slots = sm.slots[set];
    set ^= 1;
    if (lane < int(size)) store_remote(&slots[rank * kWarps + warp], lane, v);
    cluster_sync();
    return slots;
  }

  // Joined over the warp's lanes; the first lane's result everywhere.
  __device__ __forceinline__ Peak join_lanes(Peak k) const {
#pragma unroll
    for (int d = 16; d; d /= 2)
      k.join({__shfl_xor_sync(0xFFFFFFFFu, k.top, d), __shfl_xor_sync(0xFFFFFFFFu, k.sum, d),
              __shfl_xor_sync(0xFFFFFFFFu, k.token, d)},
             unit.hi, exp2_approx);
    return {__shfl_sync(0xFFFFFFFFu, k.top, 0), __shfl_sync(0xFFFFFFFFu, k.sum, 0), __shfl_sync(0xFFFFFFFFu, k.token, 0)};
  }

  // The same numbers on every thread of the cluster: the walk goes by them, and no thread may take another way.
  // behind: what else is to be done before all warps meet.
  template <class F>
  __device__ __forceinline__ Peak peak(const Row<E> &row, F behind) {
    int begin, end;
    part(row, begin, end);
    Peak k = {-INFINITY, 0.0f, INT32_MAX};
    float low = 0.0f, batch = 0.0f;  // of k.sum (a lane may add up thousands of units); what it is to grow by
    const float c = unit.hi;
    const auto look = [&](int u, const float (&x)[kUnit]) {
      float t = x[0];
#pragma unroll
      for (int i = 1; i < kUnit; ++i) t = fmaxf(t, x[i]);
      if (t > k.top) {
        const float f = exp2_approx((k.top - t) * c);
        k.sum *= f, low *= f, batch *= f;
        k.top = t;
#pragma unroll
        for (int i = kUnit - 1; i >= 0; --i)
          if (x[i] == t) k.token = row.first(u) + i;
      }
      const float ref = k.top == -INFINITY ? 0.0f : k.top;
      float e[kUnit];
#pragma unroll
      for (int i = 0; i < kUnit; ++i) e[i] = exp2_approx((x[i] - ref) * c);
      batch += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    };
#pragma unroll 1
    for (int u0 = begin; u0 < end; u0 += 32 * kBatch) {
      if (u0 + 32 * kBatch <= end && row.whole(u0, u0 + 32 * kBatch)) {
        uint4 v[kBatch][Row<E>::kPieces];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) row.ask(u0 + 32 * j + lane, v[j]);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          float x[kUnit];
          row.take(v[j], x);
          look(u0 + 32 * j + lane, x);
        }
      } else {
#pragma unroll 1
        for (int u = u0 + lane; u < min(end, u0 + 32 * kBatch); u += 32) {
          float x[kUnit];
          row.load(u, x);
          look(u, x);
        }
      }
      const Two s = add(Two{k.sum, low}, batch, 0.0f);
      k.sum = s.hi, low = s.lo, batch = 0.0f;
    }
    k.sum += low;
    k = join_lanes(k);
    behind();
    const float4 *slots = exchange(make_float4(k.top, k.sum, __int_as_float(k.token), 0.0f));
    k = {-INFINITY, 0.0f, INT32_MAX};
    for (int i = lane; i < int(size) * kWarps; i += 32)
      k.join({slots[i].x, slots[i].y, __float_as_int(slots[i].z)}, c, exp2_approx);
    return join_lanes(k);
  }

  // What is left of a weight less taken q: nothing below 0.
  static __device__ __forceinline__ Two left_long(Two w, float q, Two taken) {
    if (DRAFT && taken.hi != 0.0f) {
      const float g = __fmul_rn(taken.hi, q), gl = fmaf(taken.lo, q, fmaf(taken.hi, q, -g));
      const float s = w.hi - g, b = s - w.hi;
      const float lo = ((w.hi - (s - b)) - (g + b)) + (w.lo - gl), hi = s + lo;
      w = hi > 0.0f ? Two{hi, lo - (hi - s)} : Two{0.0f, 0.0f};
    }
    return w;
  }

  // The rejected tokens among the 8 from e on have no weight.
  __device__ __forceinline__ void reject(int e, float (&x)[kUnit]) const {
#pragma unroll 1
    for (int j = 0; j < count; ++j) {
      const int at = sm.rejected[j] - e;
      if (uint32_t(at) >= kUnit) continue;
#pragma unroll
      for (int i = 0; i < kUnit; ++i)
        if (at == i) x[i] = -INFINITY;
    }
  }

  // The weights of 8 tokens in one binary32; the large ones as a mask, and 0 in their place. Whole warp.
  __device__ __forceinline__ uint32_t weights_short(const float (&x)[kUnit], float top, float (&w)[kUnit]) const {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      // 32-bit logits: the difference's rounding would be 2^-20 of a small weight
      const Two d = sizeof(E) == 4 ? minus(x[i], top) : Two{x[i] - top, 0.0f};
      w[i] = power_short(fmaxf(d.hi, least), d.hi > least ? d.lo : 0.0f, unit);
    }
    uint32_t large = 0;
    const float most = fmaxf(fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])), fmaxf(fmaxf(w[4], w[5]), fmaxf(w[6], w[7])));
    if (__any_sync(0xFFFFFFFFu, most > kShort)) {
#pragma unroll
      for (int i = 0; i < kUnit; ++i)
        if (w[i] > kShort) {
          w[i] = 0.0f;
          large |= 1u << i;
        }
    }
    return large;
  }

  // What is left of them less taken q; those next to it as a mask, and 0 in their place, in w too. Whole warp.
  static __device__ __forceinline__ uint32_t less_draft(Two taken, const float (&q)[kUnit], float (&w)[kUnit],
                                                        float (&left)[kUnit]) {
    const float near = taken.hi * kNear;
    bool some = false;
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      left[i] = fmaf(-taken.lo, q[i], fmaf(-taken.hi, q[i], w[i]));
      some |= fabsf(left[i]) < near * q[i];
    }
    uint32_t mask = 0;
    if (__any_sync(0xFFFFFFFFu, some)) {
#pragma unroll
      for (int i = 0; i < kUnit; ++i)
        if (fabsf(left[i]) < near * q[i]) {
          left[i] = w[i] = 0.0f;
          mask |= 1u << i;
        }
    }
#pragma unroll
    for (int i = 0; i < kUnit; ++i) left[i] = fmaxf(left[i], 0.0f);
    return mask;
  }

  // f(i, what is left of token i) for the large ones of a unit. Whole warp; a lane's one after another.
  template <class F>
  __device__ __forceinline__ void each_large(uint32_t large, const float (&x)[kUnit], const float (&q)[kUnit], float top, Two taken,
                                             F f) const {
    while (__any_sync(0xFFFFFFFFu, large != 0)) {
      const int i = large ? __ffs(large) - 1 : 0;
      float xi = x[0], qi = q[0];
#pragma unroll
      for (int j = 1; j < kUnit; ++j) {
        if (i == j) xi = x[j];
        if (i == j) qi = q[j];
      }
      const Two w = left_long(power(minus(xi, top), unit, sm.powers), qi, taken);
      if (large) f(i, w);
      large &= large - 1;
    }
  }

  struct Sums {
    const float4 *slots;  // of the warps, of what is left
    Two all;              // of all weights
  };

  // Sums of what is left with c = taken / (sum of all weights), or, without a draft, of all tokens but the rejected ones.
  // fresh (with a draft): c = 1, with a guess at the sum of all weights, which is computed in the same pass. The sums are
  // corrected for what the guess was off by, d: what is left of w - guess q becomes less by d q, where it is positive.
  // Where it changes its sign that is not so: these tokens are among those next to c q as long as d is within kNear, and
  // if they are of any weight, the sums are computed again with the sum of all weights.
  __device__ __forceinline__ Sums sums(const Row<E> &row, const float *draft, float top, Two taken, bool fresh) {
    int begin, end;
    part(row, begin, end);
    Two s, all = {0.0f, 0.0f};
#pragma unroll 1
    while (true) {
      s = {0.0f, 0.0f};
      float share = 0.0f;  // the draft's probabilities where something is left
      float close = 0.0f;  // and next to c q
      const bool drafted = DRAFT && taken.hi != 0.0f;
      int kept = 0;        // weights that wait to be computed in two
      const auto long_sum = [&](float2 l) {
        const Two w = power(minus(l.x, top), unit, sm.powers), r = left_long(w, l.y, taken);
        s = add(s, r.hi, r.lo);
        if (DRAFT && fresh) {
          all = add(all, w.hi, w.lo);
          if (r.hi > 0.0f) share += l.y;
          if (fabsf(fmaf(-taken.hi, l.y, w.hi + w.lo)) < taken.hi * kNear * l.y) close += l.y;
        }
      };
      float x[kUnit], q[kUnit] = {}, nq[kUnit] = {};  // of this unit, and the next
      uint4 nx[Row<E>::kPieces];                      // logits of the next, as they come
      const auto ask = [&](int u) {
        if (u >= end) return;
        if (row.whole(u, u + 1)) row.ask(u, nx);
        if (drafted) load_draft(draft, row.first(u), row.vocab, nq);
      };
      const auto take = [&](int u) {
        if (u >= end) {
#pragma unroll
          for (int i = 0; i < kUnit; ++i) x[i] = -INFINITY;
        } else if (row.whole(u, u + 1)) {
          row.take(nx, x);
        } else {
          load_cut(row.p, row.first(u), row.vocab, -INFINITY, x);
        }
      };
      ask(begin + lane);
#pragma unroll 1
      for (int u0 = begin; u0 < end; u0 += 32) {
        const int u = u0 + lane;
        take(u);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) q[i] = nq[i];
        ask(u + 32);
        if (!DRAFT) reject(row.first(u), x);
        float w[kUnit], left[kUnit];
        uint32_t longer = weights_short(x, top, w);
        if (drafted) {
          longer |= less_draft(taken, q, w, left);
          if (fresh) {
            all = add(all, (w[0] + w[1]) + (w[2] + w[3]), 0.0f);
            all = add(all, (w[4] + w[5]) + (w[6] + w[7]), 0.0f);
#pragma unroll
            for (int i = 0; i < kUnit; ++i) share += left[i] > 0.0f ? q[i] : 0.0f;
          }
        } else {
#pragma unroll
          for (int i = 0; i < kUnit; ++i) left[i] = w[i];
        }
        s = add(s, (left[0] + left[1]) + (left[2] + left[3]), 0.0f);
        s = add(s, (left[4] + left[5]) + (left[6] + left[7]), 0.0f);
        if (__any_sync(0xFFFFFFFFu, longer != 0)) {  // 32 of them at a time
          const int mine = __popc(longer);
          int at = kept + warp_inclusive_sum(mine) - mine;
          kept = __shfl_sync(0xFFFFFFFFu, at + mine, 31);
#pragma unroll
          for (int i = 0; i < kUnit; ++i)
            if (longer >> i & 1) sm.large[warp][at++] = make_float2(x[i], q[i]);
          __syncwarp();
#pragma unroll 1
          for (; kept >= 32; kept -= 32) long_sum(sm.large[warp][kept - 32 + lane]);
          __syncwarp();
        }
      }
      if (lane < kept) long_sum(sm.large[warp][lane]);
      s = add(s, Two{0.0f, 0.0f});
      all = add(all, Two{0.0f, 0.0f});
#pragma unroll
      for (int d = 16; d; d /= 2) {
        s = add(s, Two{__shfl_xor_sync(0xFFFFFFFFu, s.hi, d), __shfl_xor_sync(0xFFFFFFFFu, s.lo, d)});
        if (DRAFT && fresh) {
          all = add(all, Two{__shfl_xor_sync(0xFFFFFFFFu, all.hi, d), __shfl_xor_sync(0xFFFFFFFFu, all.lo, d)});
          share += __shfl_xor_sync(0xFFFFFFFFu, share, d);
          close += __shfl_xor_sync(0xFFFFFFFFu, close, d);
        }
      }
      if (!DRAFT || !fresh) break;
      const float4 *const slots = exchange(make_float4(all.hi, all.lo, close, 0.0f));
      all = whole(slots);
      close = 0.0f;
      for (int i = lane; i < int(size) * kWarps; i += 32) close += slots[i].z;
#pragma unroll
      for (int d = 16; d; d /= 2) close += __shfl_xor_sync(0xFFFFFFFFu, close, d);
      close = __shfl_sync(0xFFFFFFFFu, close, 0);
      const float off = (all.hi - taken.hi) + all.lo;
      if (close <= 0x1p-14f && fabsf(off) <= taken.hi * (kNear / 2)) {
        s = add(s, Two{-off * share, 0.0f});
        if (s.hi < 0.0f) s = {0.0f, 0.0f};
        break;
      }
      taken = all;
      fresh = false;
    }
    return {exchange(make_float4(s.hi, s.lo, 0.0f, 0.0f)), all};
  }

  // Sum of all of them.
  __device__ __forceinline__ Two whole(const float4 *slots) const {
    Two s = {0.0f, 0.0f};
    for (int i = lane; i < int(size) * kWarps; i += 32) s = add(s, Two{slots[i].x, slots[i].y});
#pragma unroll
    for (int d = 16; d; d /= 2)
      s = add(s, Two{__shfl_xor_sync(0xFFFFFFFFu, s.hi, d), __shfl_xor_sync(0xFFFFFFFFu, s.lo, d)});
    return from_lane(s, 0);
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

  // The new token, on one thread of the block that has it; -1 elsewhere. any: whether there was anything to choose from.
  // weights: their sum, where something is taken; fresh (it is not known yet): see sums().
  __device__ int choose(const Row<E> &row, const float *draft, float top, Two taken, Two weights, bool fresh, float u,
                        bool &any) {
    const Sums found_sums = sums(row, draft, top, taken, fresh);
    const float4 *slots = found_sums.slots;
    if (DRAFT && fresh) taken = weights = found_sums.all;
    // running sums over the slots, consecutive ones a lane
    constexpr int kPerLane = (kMaxCluster * kWarps + 31) / 32;
    const int n = int(size) * kWarps, per = (n + 31) / 32;
    Two slot[kPerLane], upto[kPerLane];
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const int i = lane * per + j;
      const bool some = j < per && i < n;
      slot[j] = {some ? slots[i].x : 0.0f, some ? slots[i].y : 0.0f};
      upto[j] = j ? add(upto[j - 1], slot[j]) : slot[j];
    }
    const Two to_lane = scan(upto[kPerLane - 1], lane), all = from_lane(to_lane, 31);
    any = all.hi > (DRAFT && taken.hi != 0.0f ? fmaxf(kNothing, kRest * weights.hi) : kNothing);
    if (!any) return -1;
    const Two border = times(all, fminf(fmaxf(u, 0.0f), 1.0f));
    // the first slot whose running sum exceeds the border; by a rounding, or with u = 1, there may be none: the last that has
    // a weight
    Two run = {__shfl_up_sync(0xFFFFFFFFu, to_lane.hi, 1), __shfl_up_sync(0xFFFFFFFFu, to_lane.lo, 1)};
    if (lane == 0) run = {0.0f, 0.0f};
    int hit = INT32_MAX, last = -1;
    Two before = run, before_last = run;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      if (slot[j].hi > kNothing) {
        const Two in_front = j ? add(run, upto[j - 1]) : run;
        if (hit == INT32_MAX && less(border, add(run, upto[j]))) hit = lane * per + j, before = in_front;
        last = lane * per + j, before_last = in_front;
      }
    }
    int owner = __reduce_min_sync(0xFFFFFFFFu, hit);
    if (owner == INT32_MAX) {
      owner = __reduce_max_sync(0xFFFFFFFFu, last);
      before = before_last;
    }
    before = from_lane(before, owner / per);
    if (owner / kWarps != int(rank)) return -1;  // the whole block
    // the owner's part once more, by all warps: 32 units each, one a lane
    const int units = row.units(), each = (units + n - 1) / n, begin = min(units, owner * each), end = min(units, begin + each);
    int positive = -1;  // the last token with a weight
    for (int u0 = begin; u0 < end; u0 += 32 * kWarps) {
      const int at = u0 + 32 * warp + lane;
      float x[kUnit], q[kUnit] = {}, v[kUnit];
      if (at < end) {
        row.load(at, x);
        if (DRAFT && taken.hi != 0.0f) load_draft(draft, row.first(at), row.vocab, q);
      } else {
#pragma unroll
        for (int i = 0; i < kUnit; ++i) x[i] = -INFINITY;
      }
      if (!DRAFT) reject(row.first(at), x);
      uint32_t large = weights_short(x, top, v);
      if (DRAFT && taken.hi != 0.0f) {
        float left[kUnit];
        large |= less_draft(taken, q, v, left);
#pragma unroll
        for (int i = 0; i < kUnit; ++i) v[i] = left[i];
      }
      Two w[kUnit], s = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kUnit; ++i) w[i] = {v[i], 0.0f};
      each_large(large, x, q, top, taken, [&](int k, Two l) {
#pragma unroll
        for (int i = 0; i < kUnit; ++i)
          if (i == k) w[i] = l;
      });
#pragma unroll
      for (int i = 0; i < kUnit; ++i) s = add(s, w[i].hi, w[i].lo);
      s = add(s, Two{0.0f, 0.0f});
      const Two to = scan(s, lane);
      __syncthreads();  // the last round's sums have been read
      if (lane == 31) sm.part[warp] = to;
      __syncthreads();
      Two parts = scan(lane < kWarps ? sm.part[lane] : Two{0.0f, 0.0f}, lane);
      Two from = from_lane(parts, max(warp - 1, 0));
      from = warp ? add(before, from) : before;
      before = add(before, from_lane(parts, kWarps - 1));
      const Two above = {__shfl_up_sync(0xFFFFFFFFu, to.hi, 1), __shfl_up_sync(0xFFFFFFFFu, to.lo, 1)};
      if (lane) from = add(from, above);
      // the first token of the lane's whose running sum exceeds the border, if the one in front of the lane does not
      int found = INT32_MAX;
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        if (w[i].hi > kNothing) {
          positive = row.first(at) + i;
          from = add(from, w[i]);
          if (found == INT32_MAX && less(border, from)) found = positive;
        }
      }
      found = __reduce_min_sync(0xFFFFFFFFu, found);
      if (lane == 0) sm.found[warp] = found;
      __syncthreads();
      found = __reduce_min_sync(0xFFFFFFFFu, lane < kWarps ? sm.found[lane] : INT32_MAX);
      if (found != INT32_MAX) return threadIdx.x == 0 ? found : -1;
    }
    positive = __reduce_max_sync(0xFFFFFFFFu, positive);
    __syncthreads();
    if (lane == 0) sm.found[warp] = positive;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) positive = max(positive, sm.found[i]);
    return threadIdx.x == 0 ? positive : -1;
  }
};

// A block of a cluster of one sequence.
template <class E, bool DRAFT>
__global__ void __launch_bounds__(kThreads, 2) verify_drafts_kernel(const __grid_constant__ VerifyArgs a) {
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
  // No block may store into another one's shared memory before that one has begun: each says so here, and waits for the
  // others in front of its first exchange, when the root's row has been read.
  cluster_arrive();
  const int n = rows.n;
  // A row's logit and draft probability lie in its parent's row: they come while the root's row is read.
  static_assert(kThreads >= kMaxTree, "a thread for each row");
  float row_x = 0.0f, row_q = 1.0f;
  if (tid < n) {
    const int at = rows.first + tid, token = __ldg(a.tokens + at);
    int parent = a.parents ? __ldg(a.parents + at) : tid - 1;
    if (parent >= tid) out_of_range(status);
    const bool good = token >= 0 && token < a.vocab;
    if (tid > 0 && !good) out_of_range(status);
    if (tid == 0 || parent < 0 || parent >= tid || !good) parent = kNever;
    sm.parent[tid] = parent;
    sm.token[tid] = token;
    sm.u[tid] = __ldg(a.accept_u + at);
    if (parent >= 0) {
      const int64_t row = rows.first + parent;
      row_x = value(static_cast<const E *>(a.logits) + row * a.logits_stride + token);
      if (DRAFT) row_q = __ldg(a.draft + row * a.draft_stride + token);
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
  // Beyond these ends all that is computed from it would not stay in range: `least` of a temperature of 2^122 is -inf, and
  // then a logit of -inf gets a NaN as its weight.
  w.unit = exponent_unit(greedy ? 1.0f : fminf(fmaxf(t, 0x1p-100f), 0x1p100f));
  w.least = -126.0f / w.unit.hi;
  __syncthreads();

  int node = 0, accepted = 0;
  Peak k;
  Two taken;   // c times the sum of all weights
  Two all;     // that sum, if it is known
  bool valid;  // there is a distribution
  while (true) {
    const Row<E> row(a.logits, a.logits_stride, rows.first + node, a.vocab);
    const float *draft = DRAFT ? a.draft + int64_t(rows.first + node) * a.draft_stride : nullptr;
    k = w.peak(row, [&] {
      if (node != 0) return;  // once
      if (tid < n) sm.x[tid] = row_x, sm.q[tid] = row_q;
      cluster_wait();
    });
    valid = k.sum > 0.0f && k.sum < INFINITY && k.top > -INFINITY;
    if (!valid) break;
    taken = {0.0f, 0.0f};
    w.count = 0;
    all = {0.0f, 0.0f};
    Two rest = {0.0f, 0.0f};  // N times the sum of all weights, where it was summed
    float mass = 1.0f;        // without a draft, before that: N
    float summed = 0.0f;      // and what the sum was
    bool stale = false;       // with a draft: N is to be computed
    bool nothing = false;     // and nothing is left
    int next = -1;
    for (int base = 0; base < n && next < 0; base += 32) {
      const int i0 = base + lane;
      unsigned asked = __ballot_sync(0xFFFFFFFFu, i0 < n && sm.parent[min(i0, n - 1)] == node);
      while (asked) {
        const int i = base + __ffs(asked) - 1;
        asked &= asked - 1;
        const int y = sm.token[i];
        bool yes;
        const Two d = minus(sm.x[i], k.top);
        const auto exactly = [&] {
          const Two e = power(d, w.unit, sm.powers);
          return e.hi > kNothing ? add(e, Two{0.0f, 0.0f}) : Two{0.0f, 0.0f};
        };
        Two p = {power_approx(d, w.unit), 0.0f};  // the child's weight
        if (p.hi <= kNothing) p.hi = 0.0f;
        if (greedy) {
          yes = y == k.token;
        } else if constexpr (DRAFT) {
          if (stale && !nothing) {
            const auto sums = w.sums(row, draft, k.top, taken, all.hi == 0.0f);
            rest = w.whole(sums.slots);
            if (all.hi == 0.0f) all = taken = sums.all;
            nothing = rest.hi <= kRest * all.hi;
            stale = false;
          }
          if (taken.hi != 0.0f) p = w.left_long(exactly(), sm.q[i], taken);
          yes = !nothing && sm.u[i] * (taken.hi == 0.0f ? k.sum : rest.hi) * sm.q[i] < p.hi;
        } else {
          // Taken off 1, N loses as many bits as the rejected tokens took of it (its terms are good to 2^-22): once less than
          // a quarter is left, the others are summed, and again where less than 2^-10 of that sum is left. (Already with a
          // half left: 16 trees of 64, the mean of 24 draws, 31.0 us, with an eighth 29.4. What this second place for sums
          // costs calls that never come here, in registers and instructions to fetch: one chain 12.5 -> 12.9 us; out of line,
          // with a walker of its own or this one, it was no better.)
          if (summed == 0.0f ? mass < 0.25f : rest.hi < 0x1p-10f * summed) {
            rest = w.whole(w.sums(row, draft, k.top, taken, false).slots);
            summed = rest.hi;
            if (rest.hi <= kNothing) rest = {0.0f, 0.0f}, summed = -1.0f;  // and so it stays
          }
          if (summed != 0.0f) p = exactly();
          for (int j = 0; j < w.count; ++j)
            if (sm.rejected[j] == y) p = {0.0f, 0.0f};
          yes = sm.u[i] * (summed == 0.0f ? mass * k.sum : rest.hi) < p.hi;
        }
        if (yes) {
          next = i;
          break;
        }
        if (greedy) continue;
        if constexpr (DRAFT) {
          // c becomes 1, for now with the sum that the walk has; then it grows by N
          if (!nothing) taken = taken.hi == 0.0f ? Two{k.sum, 0.0f} : add(taken, rest);
          stale = true;
        } else {
          mass = fmaxf(mass - p.hi / k.sum, 0.0f);
          if (summed != 0.0f) {
            rest = add(rest, Two{-p.hi, -p.lo});
            if (rest.hi < 0.0f) rest = {0.0f, 0.0f};
          }
          __syncthreads();  // nobody reads the list
          if (tid == 0) sm.rejected[w.count] = y;
          ++w.count;
          __syncthreads();
        }
      }
    }
    if (nothing) taken = {0.0f, 0.0f};  // the new token is p's own
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
      // Also where one is to be chosen: should the sums find a place and the tokens there, by their rounding, none, it
      // stays. The block that finds one writes it behind the cluster's barriers, and so after this.
      out[accepted] = valid ? k.token : -1;
    }
  }
  if (!valid || greedy) return;
  const Row<E> row(a.logits, a.logits_stride, rows.first + node, a.vocab);
  const float *draft = DRAFT ? a.draft + int64_t(rows.first + node) * a.draft_stride : nullptr;
  const float u = __ldg(a.sample_u + b);
  bool any = false;
  int token = -1;
#pragma unroll 1
  for (int again = 0; again < 2 && !any; ++again) {
    token = w.choose(row, draft, k.top, taken, all, DRAFT && taken.hi != 0.0f && all.hi == 0.0f, u, any);
    w.count = 0;  // if nothing is left: the target's own probabilities
    taken = {0.0f, 0.0f};
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
  if (cluster > 8) {
    const cudaError_t e = cudaFuncSetAttribute(verify_drafts_kernel<E, DRAFT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
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
  // Blocks of a sequence: of 2,048 tokens at least, and in all at most 1.7 an SM in clusters of 16, 2.6 in smaller ones (the
  // kernel holds two an SM: what is more waits for the sequences that end first). Measured, device us by blocks of a cluster:
  //                                        sequences     1     2     4     8    16
  //   chains of 6, 131,072 tokens, drafted       14   149    88    52    34    30
  //                                              16   161    91    54    37    40
  //                                              20   141    79    48    37    39
  //                                              24   155    82    52    39    48
  //                                              48   167    95    67    64    83
  //                                              56   175    97    71    72    98
  //                                              96   184   116   105   110   159
  //                                             128   182   122   118   133   200
  //   trees of 16, 131,072 tokens                14   120    69    41    27    23
  //                                              16   130    73    42    29    31
  //                                              20   114    63    37    27    31
  //   trees of 64, a quarter greedy              16     -     -    43    30    27
  //   chains of 6, 50,021 tokens                 14    51    35    27    21    20
  //                                              24    45    30    23    20    25
  //                                              96    54    40    40    48    79
  //                                             160    60    51    56    76   130
  //                                             256    79    74    91   126   215
  //                                             512   120   122   159   238   422
  const auto fits = [&](int n) {
    return int64_t(io.num_seqs) * n * 10 <= (n == kMaxCluster ? 17 : 26) * num_sms && io.vocab / n >= 2048;
  };
  int cluster = 1;
  while (cluster < kMaxCluster && fits(2 * cluster)) cluster *= 2;
  const bool draft = io.draft_probs != nullptr;
  if (io.dtype == MOE_DTYPE_F32)
    return draft ? launch<float, true>(a, io.num_seqs, cluster, st) : launch<float, false>(a, io.num_seqs, cluster, st);
  if (io.dtype == MOE_DTYPE_F16)
    return draft ? launch<__half, true>(a, io.num_seqs, cluster, st) : launch<__half, false>(a, io.num_seqs, cluster, st);
  return draft ? launch<__nv_bfloat16, true>(a, io.num_seqs, cluster, st)
               : launch<__nv_bfloat16, false>(a, io.num_seqs, cluster, st);
}

}  // namespace moe
