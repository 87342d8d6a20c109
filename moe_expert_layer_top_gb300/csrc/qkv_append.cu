// qkv_append.cu — per-head RMSNorm of queries and keys, rotary positions, and
// the MXFP4 append of keys and values to the paged cache, in one pass.
//
// A group of D/8 lanes holds one head of one token, 8 elements a lane in two
// runs of 4. For a rotation of pairs (i, i + R/2) the runs are the two halves of
// the lane's 4 pairs, for pairs (2i, 2i + 1) they are neighbours: either way a
// pair never leaves its lane. Per head: r = 1 / sqrt(mean(x^2) + eps), n = x w r,
// (a, b) -> (a cos - b sin, b cos + a sin). A rotated key passes through shared
// memory once, to lie 8 contiguous elements a lane: an MX group of 32 is then 4
// lanes, its largest magnitude two shuffles away, its codes one 4-byte store a lane.
//
// Keys are computed in two-float arithmetic. A key is rounded to 16 bits and
// then to one of 16 codes; in plain binary32 (relative error 1e-7) about one
// code in 3 million would fall on the other side of a border, so caches made
// by two programs from the same keys would differ. With about 2^-45 they do not,
// short of ties nobody meets. Queries are rounded once from binary32.
//
// Bound. Few tokens: latency (6 tokens 3.6 us, 384 tokens with 64 + 8 heads of 64
// 6.7 us). Many: HBM on paper, 26 KB a token with the values returned (D = 128,
// 32 + 8 heads); in fact instructions, about 6,900 warp instructions a token, the
// two-float keys a third of them. 4,096 tokens take 35 us, 3.1 TB/s or 45 % of the
// copy bandwidth, with issue slots 71 % busy. Keys in binary32 with two-float
// arithmetic only near a border were slower: a warp takes the slow path if one lane does.
#include <cuda_runtime.h>
#include <stdint.h>

#include "attention.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kNoPlace = 0xFFFFFFFFu;  // cached rows are counted in 32 bits (the ABI refuses larger caches)

struct AppendArgs {
  moe_qkv_append_io_t io;
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  const int64_t *slots;                              // NULL: no cache
  int64_t slots_total;                               // num_pages * page_size
  int page_size;
  int parts;  // warps per token
  int64_t cached_rows;  // of all pages and kv heads, for the checks
  int32_t *status;
};

// ------------------------------------------------------------------ two-float arithmetic
// A value is hi + lo. The sums and products are the error-free transformations
// of Knuth and of Dekker (with a fused multiply-add for the product's error).
struct Two {
  float hi, lo;
};

__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}

__device__ __forceinline__ Two two_mul(Two a, float b) {
  const float p = __fmul_rn(a.hi, b);
  return {p, __fmaf_rn(a.hi, b, -p) + a.lo * b};
}

__device__ __forceinline__ Two two_add(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi);
  return two_sum(s.hi, s.lo + (a.lo + b.lo));
}

// 1 / sqrt(a): the hardware's approximation (2 ulp) and one step of the series
// y (1 + r/2 + 3 r^2 / 8), r = 1 - a y^2, with r in two-float arithmetic.
__device__ __forceinline__ Two two_rsqrt(Two a) {
  const float y = rsqrtf(a.hi);
  const Two y2 = two_mul({y, 0.0f}, y);
  const Two ay2 = two_mul(y2, a.hi);
  const float r = (1.0f - ay2.hi) - (ay2.lo + a.lo * y2.hi);
  return {y, y * r * (0.5f + 0.375f * r)};
}

// a + b as one binary32 that rounds to 16 bits as the sum itself would:
// truncated, with the last bit set when anything was cut off (round to odd).
__device__ __forceinline__ float two_add_odd(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi);
  const float lo = s.lo + (a.lo + b.lo);
  const float hi = lo != 0.0f ? __fadd_rn(s.hi, lo) : s.hi;  // an exact zero keeps its sign
  const float rest = __fsub_rn(lo, __fsub_rn(hi, s.hi));
  const uint32_t h = __float_as_uint(hi);
  const uint32_t inward = (h ^ __float_as_uint(rest)) >> 31;  // the sum lies between hi and zero
  return rest != 0.0f ? __uint_as_float((h - inward) | 1u) : hi;
}

// ------------------------------------------------------------------ one head

template <class T>
__device__ __forceinline__ void unpack4(const uint2 &r, float *x) {
  x[0] = T::lo(r.x), x[1] = T::hi(r.x), x[2] = T::lo(r.y), x[3] = T::hi(r.y);
}

template <class T>
__device__ __forceinline__ void unpack8(const uint4 &r, float (&x)[8]) {
  unpack4<T>(make_uint2(r.x, r.y), x);
  unpack4<T>(make_uint2(r.z, r.w), x + 4);
}

template <class T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(T::pack(x[0], x[1]), T::pack(x[2], x[3]), T::pack(x[4], x[5]), T::pack(x[6], x[7]));
}

// What a lane holds of a head: elements a .. a + 3 and b .. b + 3, and the
// angles of its four pairs. Pair i is elements (first(i), second(i)) of the 8.
struct Lane {
  int a, b;
  bool turned;         // its elements are rotated
  bool interleaved;
  float c[4], s[4];
};

__device__ __forceinline__ Lane make_lane(const moe_qkv_append_io_t &io, int64_t position, int l) {
  Lane t;
  const int R = io.rotary_dim, D = io.head_dim, p = 4 * l;  // pairs p .. p + 3
  t.interleaved = io.interleaved;
  t.turned = 2 * p < R;
  if (t.interleaved) {
    t.a = 2 * p;
    t.b = 2 * p + 4;
  } else if (t.turned) {
    t.a = p;
    t.b = p + R / 2;
  } else {  // the rest, as pairs too
    t.a = R + (p - R / 2);
    t.b = t.a + (D - R) / 2;
  }
  float4 c = make_float4(1.0f, 1.0f, 1.0f, 1.0f), s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (t.turned) {
    const float *row = io.rope + position * R;
    c = __ldg(reinterpret_cast<const float4 *>(row + p));
    s = __ldg(reinterpret_cast<const float4 *>(row + R / 2 + p));
  }
  t.c[0] = c.x, t.c[1] = c.y, t.c[2] = c.z, t.c[3] = c.w;
  t.s[0] = s.x, t.s[1] = s.y, t.s[2] = s.z, t.s[3] = s.w;
  return t;
}

// Both runs of the lane, of a head.
__device__ __forceinline__ uint4 load_runs(const uint16_t *head, const Lane &t) {
  const uint2 a = *reinterpret_cast<const uint2 *>(head + t.a), b = *reinterpret_cast<const uint2 *>(head + t.b);
  return make_uint4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ void store_runs(uint16_t *head, const Lane &t, const uint4 &y) {
  *reinterpret_cast<uint2 *>(head + t.a) = make_uint2(y.x, y.y);
  *reinterpret_cast<uint2 *>(head + t.b) = make_uint2(y.z, y.w);
}

// y = the rotated x; the two orders of the pairs differ in which elements they are.
__device__ __forceinline__ void rotate(const Lane &t, const float (&x)[8], float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i];
  if (!t.turned) return;
  if (t.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = fmaf(-x[2 * i + 1], t.s[i], x[2 * i] * t.c[i]);
      y[2 * i + 1] = fmaf(x[2 * i], t.s[i], x[2 * i + 1] * t.c[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = fmaf(-x[i + 4], t.s[i], x[i] * t.c[i]);
      y[i + 4] = fmaf(x[i], t.s[i], x[i + 4] * t.c[i]);
    }
  }
}

// w: the norm's weights of the lane's elements (not used without a norm).
template <int D>
__device__ __forceinline__ void query_head(const moe_qkv_append_io_t &io, const Lane &t, const float (&w)[8],
                                           float (&x)[8], float (&y)[8]) {
  if (io.q_norm) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int d = D / 16; d; d /= 2) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
    const float r = rsqrtf(fmaf(ss, 1.0f / D, io.norm_eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= w[i] * r;
  }
  rotate(t, x, y);
}

template <int D>
__device__ __forceinline__ void key_head(const moe_qkv_append_io_t &io, const Lane &t, const float (&w)[8],
                                         const float (&x)[8], float (&y)[8]) {
  Two n[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) n[i] = {x[i], 0.0f};
  if (io.k_norm) {
    Two ss = {x[0] * x[0], 0.0f};  // squares of 16-bit values are exact
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      const Two s = two_sum(ss.hi, x[i] * x[i]);
      ss = {s.hi, ss.lo + s.lo};
    }
#pragma unroll
    for (int d = D / 16; d; d /= 2) {
      const Two o = {__shfl_xor_sync(0xFFFFFFFFu, ss.hi, d), __shfl_xor_sync(0xFFFFFFFFu, ss.lo, d)};
      ss = two_add(ss, o);
    }
    const Two r = two_rsqrt(two_add({ss.hi * (1.0f / D), ss.lo * (1.0f / D)}, {io.norm_eps, 0.0f}));
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = two_mul(r, x[i] * w[i]);  // x w is exact: 2 x 11 bits at most
  }
  bool odd = false;  // infinities and NaN: the error terms make them NaN, the plain formula is theirs
  if (t.turned) {
    if (t.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = two_add_odd(two_mul(n[2 * i], t.c[i]), two_mul(n[2 * i + 1], -t.s[i]));
        y[2 * i + 1] = two_add_odd(two_mul(n[2 * i + 1], t.c[i]), two_mul(n[2 * i], t.s[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = two_add_odd(two_mul(n[i], t.c[i]), two_mul(n[i + 4], -t.s[i]));
        y[i + 4] = two_add_odd(two_mul(n[i + 4], t.c[i]), two_mul(n[i], t.s[i]));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = two_add_odd(n[i], {0.0f * n[i].hi, 0.0f});
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) odd |= !(fabsf(y[i]) <= 3.402823466e38f);
  if (odd) {
    float plain[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) plain[i] = n[i].hi;
    rotate(t, plain, y);
  }
}

// MXFP4 of a head held 8 elements a lane: the lane's 8 codes, the group's scale
// code, and (if wanted) the values they stand for. The arithmetic is moe_quantize_mxfp4's.
template <class T>
__device__ __forceinline__ void quantize_head(const uint4 &raw, uint32_t &codes, uint32_t &scale, uint4 *values) {
  float x[8];
  unpack8<T>(raw, x);
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
  scale = mx_scale_code_emax(amax, 2);
  const float down = ue8m0_to_float(254 - scale);  // 2^(127 - scale): exact products, as mx_unscale's
  codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) codes |= uint32_t(float2_to_e2m1x2(x[2 * i] * down, x[2 * i + 1] * down)) << (8 * i);
  if (values) {
    const float up = ue8m0_to_float(scale);
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(codes >> (8 * i)), __NV_E2M1);
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
      y[2 * i] = f.x * up;
      y[2 * i + 1] = f.y * up;
    }
    *values = pack8<T>(y);
  }
}

// ------------------------------------------------------------------ kernel
// A unit is what a warp's groups take at once: as many k heads, q heads or v
// heads as the warp has groups. `parts` warps share a token and take its units
// in turn, k first (they cost most); each loads the angles once.
template <class T, int D>
__global__ void __launch_bounds__(kThreads) qkv_append_kernel(const AppendArgs a) {
  constexpr int L = D / 8, kHeads = 32 / L, kWarps = kThreads / 32;
  __shared__ uint4 turned[kWarps][32];  // rotated keys on their way to 8 contiguous elements a lane
  const moe_qkv_append_io_t &io = a.io;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % L, sub = lane / L;
  const uint32_t id = blockIdx.x * kWarps + warp;  // of the warp
  const uint32_t token = id / a.parts, part = id - token * a.parts;
  if (token >= uint32_t(io.num_tokens)) return;
  const int64_t t = token;
  int64_t position = 0;
  if (io.rotary_dim) {
    position = __ldg(io.positions + t);
    if (position < 0 || position >= io.rope_positions) {
      if (lane == 0) out_of_range(a.status);
      return;  // every warp of the token
    }
  }
  uint32_t place = kNoPlace;  // first cached row of the token's kv heads
  if (a.slots) {
    const int64_t slot = __ldg(a.slots + t);
    if (slot >= a.slots_total) {
      if (lane == 0) out_of_range(a.status);
    } else if (slot >= 0) {
      const uint32_t page = uint32_t(slot) / uint32_t(a.page_size);
      place = page * io.num_kv_heads * a.page_size + (uint32_t(slot) - page * a.page_size);
    }
  }
  const Lane hold = make_lane(io, position, l);
  const int nq = io.num_heads, nk = io.num_kv_heads;
  const int uk = (nk + kHeads - 1) / kHeads, uq = (nq + kHeads - 1) / kHeads, units = 2 * uk + uq;
  const auto *q = static_cast<const uint16_t *>(io.q) + t * io.q_stride;
  const auto *k = static_cast<const uint16_t *>(io.k) + t * io.k_stride;
  const auto *v = static_cast<const uint16_t *>(io.v) + t * io.v_stride;
  // The next unit's elements are on their way while one is computed.
  const auto load = [&](int u) {
    const bool is_k = u < uk, is_q = !is_k && u < uk + uq;
    const int h = (is_k ? u : is_q ? u - uk : u - uk - uq) * kHeads + sub;
    uint4 r = make_uint4(0, 0, 0, 0);
    if (u < units && h < (is_q ? nq : nk)) {
      if (is_q || is_k)
        r = load_runs((is_q ? q : k) + int64_t(h) * D, hold);
      else
        r = reinterpret_cast<const uint4 *>(v + int64_t(h) * D)[l];
    }
    return r;
  };
  uint4 next = load(part);
  for (int u = part; u < units; u += a.parts) {
    const bool is_k = u < uk, is_q = !is_k && u < uk + uq;
    const int h = (is_k ? u : is_q ? u - uk : u - uk - uq) * kHeads + sub;
    const bool real = h < (is_q ? nq : nk);
    uint4 raw = next;
    next = load(u + a.parts);
    if (is_q) {
      float x[8], y[8], w[8] = {};
      if (io.q_norm) unpack8<T>(load_runs(static_cast<const uint16_t *>(io.q_norm), hold), w);
      unpack8<T>(raw, x);
      query_head<D>(io, hold, w, x, y);
      if (real && index_ok(a.status, t * nq + h, int64_t(io.num_tokens) * nq))
        store_runs(static_cast<uint16_t *>(io.q_out) + (t * nq + h) * D, hold, pack8<T>(y));
      continue;
    }
    const int64_t row = (t * nk + h) * D;
    const bool inside = index_ok(a.status, real ? t * nk + h : 0, int64_t(io.num_tokens) * nk);
    if (is_k) {
      float x[8], y[8], w[8] = {};
      if (io.k_norm) unpack8<T>(load_runs(static_cast<const uint16_t *>(io.k_norm), hold), w);
      unpack8<T>(raw, x);
      key_head<D>(io, hold, w, x, y);
      __syncwarp();  // the last unit's keys have been read
      store_runs(reinterpret_cast<uint16_t *>(turned[warp]) + sub * D, hold, pack8<T>(y));
      __syncwarp();
      raw = turned[warp][lane];
      if (io.k_out && real && inside) reinterpret_cast<uint4 *>(static_cast<uint16_t *>(io.k_out) + row)[l] = raw;
    }
    uint32_t codes, scale;
    uint4 values;
    void *kept = is_k ? io.k_cached : io.v_cached;
    quantize_head<T>(raw, codes, scale, kept ? &values : nullptr);
    if (!real) continue;
    if (kept && inside) reinterpret_cast<uint4 *>(static_cast<uint16_t *>(kept) + row)[l] = values;
    if (place != kNoPlace) {
      const uint64_t at = place + uint32_t(h) * a.page_size;
      if (!index_ok(a.status, at, a.cached_rows)) continue;
      reinterpret_cast<uint32_t *>((is_k ? a.k_codes : a.v_codes) + at * (D / 2))[l] = codes;
      if ((l & 3) == 0) ((is_k ? a.k_scales : a.v_scales) + at * (D / 32))[l >> 2] = uint8_t(scale);
    }
  }
}

template <class T, int D>
cudaError_t launch(const AppendArgs &a, cudaStream_t st) {
  const int64_t blocks = (int64_t(a.io.num_tokens) * a.parts + kThreads / 32 - 1) / (kThreads / 32);
  if (int64_t(a.io.num_tokens) * a.parts > INT32_MAX) return cudaErrorInvalidConfiguration;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  qkv_append_kernel<T, D><<<unsigned(blocks), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qkv_append(const moe_qkv_append_io_t &io, const moe_kv_cache_t *cache, int32_t *status,
                              int num_sms, cudaStream_t st) {
  AppendArgs a = {};
  a.io = io;
  a.status = status;
  if (cache) {
    a.slots = io.slots;
    a.k_codes = cache->k_codes;
    a.k_scales = cache->k_scales;
    a.v_codes = cache->v_codes;
    a.v_scales = cache->v_scales;
    a.page_size = cache->page_size;
    a.slots_total = int64_t(cache->num_pages) * cache->page_size;
    a.cached_rows = checked_capacity(a.slots_total * cache->num_kv_heads, io.flags);
  }
  const int heads = 256 / io.head_dim;  // of a unit
  const int units = 2 * ((io.num_kv_heads + heads - 1) / heads) + (io.num_heads + heads - 1) / heads;
  // Few tokens: a warp for each unit. Many: about 96 warps for each SM (three times what it holds), so that a
  // warp's share of the token's own work (place, angles, addresses) is spread over several units. 4,096 tokens: 35 us,
  // 60 with a warp for each unit, 40 with one a token; 384 tokens: 6.7 us, 13.5 with one a token.
  const int64_t want = (int64_t(96) * num_sms + io.num_tokens - 1) / io.num_tokens;
  a.parts = int(want < units ? want : units);
  const bool h = io.dtype == MOE_DTYPE_F16;
  if (io.head_dim == 64) return h ? launch<F16, 64>(a, st) : launch<Bf16, 64>(a, st);
  return h ? launch<F16, 128>(a, st) : launch<Bf16, 128>(a, st);
}

}  // namespace moe
