// qkv_append.cu — per-head RMSNorm of queries and keys, rotary positions, and
// the MXFP4 append of keys and values to the paged cache, in one pass.
//
// A group of D/8 lanes holds one head of one token, 8 elements (16 bytes) a
// lane. Per head: r = 1 / sqrt(mean(x^2) + eps); n = x w r; the rotation of
// pairs (i, i + R/2) reads the partner lane by shuffle, that of pairs
// (2i, 2i + 1) stays in the lane. An MX group of 32 elements is 4 lanes: its
// largest magnitude is two shuffles away, its codes are one 4-byte store a lane.
//
// Keys are computed in two-float arithmetic. A key is rounded to 16 bits and
// then to one of 16 codes; in plain binary32 (relative error 1e-7) about one
// code in 3 million would fall on the other side of a border, so caches made
// by two programs from the same keys would differ. With about 2^-45 they do not,
// short of ties nobody meets. Queries are rounded once from binary32.
#include <cuda_runtime.h>
#include <stdint.h>

#include "attention.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

struct AppendArgs {
  moe_qkv_append_io_t io;
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  const int64_t *slots;                              // NULL: no cache
  int64_t slots_total;                               // num_pages * page_size
  int page_size;
  int parts;  // blocks per token
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

__device__ __forceinline__ Two two_neg(Two a) { return {-a.hi, -a.lo}; }

// 1 / sqrt(a): the hardware's approximation (2 ulp) and one step of the series
// y (1 + r/2 + 3 r^2 / 8), r = 1 - a y^2, with r in two-float arithmetic.
__device__ __forceinline__ Two two_rsqrt(Two a) {
  const float y = rsqrtf(a.hi);
  const Two y2 = two_mul({y, 0.0f}, y);
  const Two ay2 = two_mul(y2, a.hi);
  const float r = (1.0f - ay2.hi) - (ay2.lo + a.lo * y2.hi);
  return {y, y * r * (0.5f + 0.375f * r)};
}

// hi + lo as one binary32 that rounds to 16 bits as the sum itself would:
// truncated, with the last bit set when anything was cut off (round to odd).
__device__ __forceinline__ float two_to_odd(Two a) {
  const Two s = two_sum(a.hi, a.lo);
  uint32_t b = __float_as_uint(s.hi);
  if (s.lo != 0.0f) {
    if ((s.lo < 0.0f) != (s.hi < 0.0f)) b -= 1;  // the sum lies between hi and zero
    b |= 1u;
  }
  return __uint_as_float(b);
}

// ------------------------------------------------------------------ one head

template <class T>
__device__ __forceinline__ void unpack(const uint4 &r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = T::lo(w[i]);
    x[2 * i + 1] = T::hi(w[i]);
  }
}

template <class T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(T::pack(x[0], x[1]), T::pack(x[2], x[3]), T::pack(x[4], x[5]), T::pack(x[6], x[7]));
}

// cos and sin of the lane's 8 elements (1 and 0 past the rotated dimensions),
// the sine with the sign that its element takes: out = x cos + partner sin.
struct Turn {
  float c[8], s[8];
};

template <int D>
__device__ __forceinline__ Turn load_turn(const moe_qkv_append_io_t &io, int64_t position, int l) {
  Turn t;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t.c[i] = 1.0f;
    t.s[i] = 0.0f;
  }
  const int R = io.rotary_dim;
  if (8 * l >= R) return t;
  const float *row = io.rope + position * R;
  if (io.interleaved) {  // the lane's pairs are 4 l .. 4 l + 3
    const float4 c = __ldg(reinterpret_cast<const float4 *>(row + 4 * l));
    const float4 s = __ldg(reinterpret_cast<const float4 *>(row + R / 2 + 4 * l));
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.c[2 * i] = t.c[2 * i + 1] = cc[i];
      t.s[2 * i] = -ss[i];
      t.s[2 * i + 1] = ss[i];
    }
  } else {
    const bool second = 16 * l >= R;  // elements R/2 .. R - 1
    const int i0 = 8 * l - (second ? R / 2 : 0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float4 c = __ldg(reinterpret_cast<const float4 *>(row + i0 + 4 * j));
      const float4 s = __ldg(reinterpret_cast<const float4 *>(row + R / 2 + i0 + 4 * j));
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t.c[4 * j + i] = cc[i];
        t.s[4 * j + i] = second ? ss[i] : -ss[i];
      }
    }
  }
  return t;
}

// The lane (within the group) that holds the partners of this lane's elements.
__device__ __forceinline__ int partner_lane(const moe_qkv_append_io_t &io, int l) {
  const int h = io.rotary_dim / 16;  // lanes of half the rotated dimensions
  if (io.interleaved || l >= 2 * h) return l;
  return l < h ? l + h : l - h;
}

template <class T, int D>
__device__ __forceinline__ uint4 query_head(const moe_qkv_append_io_t &io, const uint4 &raw, const Turn &t, int l,
                                            int partner) {
  constexpr int L = D / 8;
  float x[8];
  unpack<T>(raw, x);
  if (io.q_norm) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int d = L / 2; d; d /= 2) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
    const float r = rsqrtf(ss * (1.0f / D) + io.norm_eps);
    float w[8];
    unpack<T>(__ldg(reinterpret_cast<const uint4 *>(io.q_norm) + l), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= w[i] * r;
  }
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float mine = x[i ^ 1], far = __shfl_sync(0xFFFFFFFFu, x[i], partner, L);
    y[i] = 8 * l < io.rotary_dim ? fmaf(io.interleaved ? mine : far, t.s[i], x[i] * t.c[i]) : x[i];
  }
  return pack8<T>(y);
}

template <class T, int D>
__device__ __forceinline__ uint4 key_head(const moe_qkv_append_io_t &io, const uint4 &raw, const Turn &t, int l,
                                          int partner) {
  constexpr int L = D / 8;
  float x[8];
  unpack<T>(raw, x);
  Two n[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) n[i] = {x[i], 0.0f};
  if (io.k_norm) {
    Two ss = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // squares of 16-bit values are exact
      const Two s = two_sum(ss.hi, x[i] * x[i]);
      ss = {s.hi, ss.lo + s.lo};
    }
#pragma unroll
    for (int d = L / 2; d; d /= 2) {
      const Two o = {__shfl_xor_sync(0xFFFFFFFFu, ss.hi, d), __shfl_xor_sync(0xFFFFFFFFu, ss.lo, d)};
      ss = two_add(ss, o);
    }
    const Two r = two_rsqrt(two_add({ss.hi * (1.0f / D), ss.lo * (1.0f / D)}, {io.norm_eps, 0.0f}));
    float w[8];
    unpack<T>(__ldg(reinterpret_cast<const uint4 *>(io.k_norm) + l), w);
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = two_mul(r, x[i] * w[i]);  // x w is exact: 2 x 11 bits at most
  }
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    Two far = {__shfl_sync(0xFFFFFFFFu, n[i].hi, partner, L), __shfl_sync(0xFFFFFFFFu, n[i].lo, partner, L)};
    if (io.interleaved) far = n[i ^ 1];
    const bool turned = 8 * l < io.rotary_dim;
    const Two r = turned ? two_add(two_mul(n[i], t.c[i]), two_mul(far, t.s[i])) : n[i];
    y[i] = two_to_odd(r);
    // the error terms know neither signed zeros nor infinities: those are the plain formula's
    const float plain = turned ? n[i].hi * t.c[i] + far.hi * t.s[i] : n[i].hi;
    if (y[i] == 0.0f || !(fabsf(plain) <= 3.402823466e38f)) y[i] = plain;
  }
  return pack8<T>(y);
}

// MXFP4 of a head held 8 elements a lane: the lane's 8 codes, the group's scale
// code, and (if wanted) the values they stand for.
template <class T>
__device__ __forceinline__ void quantize_head(const uint4 &raw, uint32_t &codes, uint32_t &scale, uint4 *values) {
  float x[8];
  unpack<T>(raw, x);
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
  scale = mx_scale_code_emax(amax, 2);
  codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    codes |= uint32_t(float2_to_e2m1x2(mx_unscale(x[2 * i], scale), mx_unscale(x[2 * i + 1], scale))) << (8 * i);
  if (values) {
    const float s = ue8m0_to_float(scale);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c = codes >> (4 * i);
      const uint32_t e = (c >> 1) & 3u, m = c & 1u;
      // E2M1: (2 + m) 2^(e - 2) for e > 0, m / 2 for e = 0
      const float a = e ? float((2u + m) << e) * 0.25f : float(m) * 0.5f;
      y[i] = ((c & 8u) ? -a : a) * s;
    }
    *values = pack8<T>(y);
  }
}

// ------------------------------------------------------------------ kernel
// Block (token, part): its groups take the token's q heads, then k, then v,
// one in every parts * groups. The table row is loaded once per lane.
template <class T, int D>
__global__ void __launch_bounds__(kThreads) qkv_append_kernel(const AppendArgs a) {
  constexpr int L = D / 8, kGroups = kThreads / L;
  const moe_qkv_append_io_t &io = a.io;
  const int64_t t = blockIdx.x / a.parts;
  const int part = blockIdx.x % a.parts;
  const int l = threadIdx.x % L;
  int64_t position = 0;
  if (io.rotary_dim) {
    position = __ldg(io.positions + t);
    if (position < 0 || position >= io.rope_positions) {
      if (threadIdx.x == 0) out_of_range(a.status);
      return;  // the whole block
    }
  }
  int64_t page = -1;
  int offset = 0;
  if (a.slots) {
    const int64_t slot = __ldg(a.slots + t);
    if (slot >= a.slots_total) {
      if (threadIdx.x == 0) out_of_range(a.status);
    } else if (slot >= 0) {
      page = slot / a.page_size;
      offset = int(slot - page * a.page_size);
    }
  }
  const Turn turn = load_turn<D>(io, position, l);
  const int partner = partner_lane(io, l);
  const int nq = io.num_heads, nk = io.num_kv_heads, total = nq + 2 * nk;
  const auto *q = static_cast<const uint16_t *>(io.q) + t * io.q_stride;
  const auto *k = static_cast<const uint16_t *>(io.k) + t * io.k_stride;
  const auto *v = static_cast<const uint16_t *>(io.v) + t * io.v_stride;
  const int stride = a.parts * kGroups;
  // Shuffles involve whole warps: every group runs the same number of rounds,
  // and in a round the warps of mixed kinds take each kind in turn.
  for (int base = part * kGroups; base < total; base += stride) {
    const int h = base + threadIdx.x / L;
    const bool is_q = h < nq, is_k = !is_q && h < nq + nk, is_v = !is_q && !is_k && h < total;
    const int kv = is_q ? 0 : (is_k ? h - nq : h - nq - nk);
    const uint16_t *src = is_q ? q + int64_t(h) * D : (is_k ? k : v) + int64_t(kv) * D;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (h < total) raw = reinterpret_cast<const uint4 *>(src)[l];  // not the read-only path: q_out may be q
    if (__any_sync(0xFFFFFFFFu, is_q)) {
      const uint4 y = query_head<T, D>(io, raw, turn, l, partner);
      if (is_q) reinterpret_cast<uint4 *>(static_cast<uint16_t *>(io.q_out) + (t * nq + h) * D)[l] = y;
    }
    if (!__any_sync(0xFFFFFFFFu, is_k || is_v)) continue;
    const int64_t row = (t * nk + kv) * D;
    if (__any_sync(0xFFFFFFFFu, is_k)) {
      const uint4 y = key_head<T, D>(io, raw, turn, l, partner);
      if (is_k) {
        raw = y;
        if (io.k_out) reinterpret_cast<uint4 *>(static_cast<uint16_t *>(io.k_out) + row)[l] = y;
      }
    }
    uint32_t codes, scale;
    uint4 values;
    void *kept = is_k ? io.k_cached : io.v_cached;
    quantize_head<T>(raw, codes, scale, (io.k_cached || io.v_cached) ? &values : nullptr);
    if (!is_k && !is_v) continue;
    if (kept) reinterpret_cast<uint4 *>(static_cast<uint16_t *>(kept) + row)[l] = values;
    if (page >= 0) {
      const int64_t at = (page * nk + kv) * a.page_size + offset;
      reinterpret_cast<uint32_t *>((is_k ? a.k_codes : a.v_codes) + at * (D / 2))[l] = codes;
      if ((l & 3) == 0) ((is_k ? a.k_scales : a.v_scales) + at * (D / 32))[l >> 2] = uint8_t(scale);
    }
  }
}

template <class T, int D>
cudaError_t launch(const AppendArgs &a, cudaStream_t st) {
  const int64_t blocks = int64_t(a.io.num_tokens) * a.parts;
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
  }
  const int groups = kThreads / (io.head_dim / 8);
  const int rounds = (io.num_heads + 2 * io.num_kv_heads + groups - 1) / groups;
  // Few tokens: one round a block, so that the heads of a token run side by side.
  a.parts = int64_t(io.num_tokens) * rounds <= 4 * num_sms ? rounds : 1;
  const bool h = io.dtype == MOE_DTYPE_F16;
  if (io.head_dim == 64) return h ? launch<F16, 64>(a, st) : launch<Bf16, 64>(a, st);
  return h ? launch<F16, 128>(a, st) : launch<Bf16, 128>(a, st);
}

}  // namespace moe
