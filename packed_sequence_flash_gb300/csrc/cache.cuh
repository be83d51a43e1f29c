// cache.cuh -- the 8-bit paged key/value cache as the kernels see it, and the
// arithmetic of its blocks.
//
// A page holds `page` tokens (16, 32, 64 or 128) of every KV head: e4m3 codes
// k [pages][Hkv][page][Dqk] and v [pages][Hkv][page][Dv] (any strides, the row
// contiguous) with one fp32 scale per (page, head) for K and one for V; a code c
// stands for c * scale. Token j of sequence b is row j % page of page
// table[b][j / page]. weight [pages][Hkv][page] is the attention weight that
// the token has received so far.
#pragma once

#include <math_constants.h>
#include <stdint.h>

#include "common.cuh"

namespace psf {

struct CacheView {
  uint8_t *k, *v;
  float *k_scale, *v_scale;  // [pages][Hkv]
  float* weight;             // [pages][Hkv][page], nullable
  int64_t k_sp, k_sh, k_sr, v_sp, v_sh, v_sr;  // strides (page, head, row) in bytes
  int pages, page, page_lg, Hkv, Dqk, Dv;
};

// The sequences of a call. cu (nullable): exclusive prefix sums of the rows
// (query rows, or new tokens) that each sequence has in a packed tensor of T
// rows; without it every sequence has `each` rows.
struct SeqView {
  const int32_t* table;  // [B][max_pages]
  const int32_t* lens;   // [B] tokens in the cache
  const int32_t* cu;
  int B, max_pages, T, each;
  int max_rows;  // most rows of a sequence
};

// Sequence b: n tokens in the cache, m rows of the packed tensor from row q0.
// A description that cannot be right (lengths past the page table, rows outside
// the tensor) sets bad and leaves the sequence without tokens (and rows).
struct Seq {
  int n, m, q0;
  bool bad;
};
__device__ __forceinline__ Seq seq_at(const SeqView& s, int page, int b) {
  Seq r;
  r.n = s.lens[b];
  r.q0 = s.cu ? s.cu[b] : b * s.each;
  r.m = s.cu ? s.cu[b + 1] - r.q0 : s.each;
  const bool rows_bad = r.q0 < 0 || r.m < 0 || r.m > s.max_rows || (int64_t)r.q0 + r.m > s.T;
  r.bad = rows_bad || r.n < 0 || (int64_t)r.n > (int64_t)s.max_pages * page;
  if (r.bad) r.n = 0;
  if (rows_bad) r.m = 0;
  return r;
}

// Whether the prefix sums do not begin at 0 (rows in front of the first sequence would belong to none).
__device__ __forceinline__ bool cu_bad(const SeqView& s) { return s.cu && s.cu[0] != 0; }

// Scale of a block whose largest magnitude is a (finite, >= 0): the smallest
// power of two s >= 2^-126 with a <= 448 s (448 = 1.75 * 2^8 is the largest e4m3
// value). A power of two costs no precision in a floating format and keeps a
// later change of scale exact down to the format's subnormals.
__device__ __forceinline__ float block_scale(float a) {
  const int bits = __float_as_int(a);
  const int e = (bits >> 23) - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  return __int_as_float(min(max(e, 1), 254) << 23);
}

// Two fp32 values -> two e4m3 codes (round to nearest even), lo in the low byte.
// |x| never exceeds 448 by more than a rounding here; what is not finite becomes NaN.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes -> two fp16 values (exact), low byte in the low half.
__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t pair) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)pair));
  return d;
}
__device__ __forceinline__ float2 e4m3_to_float2(uint32_t pair) {
  const uint32_t h = e4m3_to_half2(pair);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// q = a value rounded to fp32, rest = that value minus q: q with an odd last bit
// where it is not exact, so that rounding it again, to fewer bits, is the value's
// own rounding (65 / 1.3f is 50 in fp32, a tie of e4m3 that the quotient is not).
__device__ __forceinline__ float round_to_odd(float q, float rest) {
  const int bits = __float_as_int(q);
  const bool move = fabsf(rest) > 0.f && !(bits & 1) && fabsf(q) > 0.f;
  return move ? __int_as_float((rest > 0.f) == (q > 0.f) ? bits + 1 : bits - 1) : q;
}
__device__ __forceinline__ float divide_to_odd(float x, float y) {
  const float q = x / y;
  return round_to_odd(q, fmaf(-q, y, x));
}
__device__ __forceinline__ float multiply_to_odd(float x, float y) {
  const float p = x * y;
  return round_to_odd(p, fmaf(x, y, -p));
}
// Codes times r <= 1, rounded to e4m3 again. For a power of two the products are
// made in fp16: exact wherever the result is not 0 (codes have 4 significant
// bits and results below 2^-10 become 0; fp16 reaches down to 2^-24).
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float r) {
  const float2 a = e4m3_to_float2(codes & 0xffff), b = e4m3_to_float2(codes >> 16);
  return e4m3_pair(multiply_to_odd(a.x, r), multiply_to_odd(a.y, r)) |
         (e4m3_pair(multiply_to_odd(b.x, r), multiply_to_odd(b.y, r)) << 16);
}
__device__ __forceinline__ uint32_t rescale4_half(uint32_t codes, __half2 r) {
  uint32_t lo = e4m3_to_half2(codes & 0xffff), hi = e4m3_to_half2(codes >> 16);
  const __half2 a = __hmul2(*reinterpret_cast<__half2*>(&lo), r), b = __hmul2(*reinterpret_cast<__half2*>(&hi), r);
  uint16_t x, y;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(x) : "r"(*reinterpret_cast<const uint32_t*>(&a)));
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(y) : "r"(*reinterpret_cast<const uint32_t*>(&b)));
  return x | ((uint32_t)y << 16);
}
__device__ __forceinline__ uint4 rescale16(uint4 x, float r) {
  if ((__float_as_int(r) & 0x7fffff) == 0 && r <= 1.f && r >= 0.f) {
    const __half2 h = __float2half2_rn(r);
    return make_uint4(rescale4_half(x.x, h), rescale4_half(x.y, h), rescale4_half(x.z, h), rescale4_half(x.w, h));
  }
  return make_uint4(rescale4(x.x, r), rescale4(x.y, r), rescale4(x.z, r), rescale4(x.w, r));
}
__device__ __forceinline__ float finite_or_nan(float x) { return fabsf(x) <= 3.402823466e38f ? x : CUDART_NAN_F; }

// Largest b in [0, B) with start(b) <= x, start increasing with start(0) <= x;
// every lane of the warp returns it. 32 probes a step: two dependent loads up
// to 1024 sequences.
template <typename F>
__device__ __forceinline__ int warp_find(int B, int64_t x, F start) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int probe = lo + (int)(threadIdx.x & 31) * step;
    const bool in = probe < hi && start(probe) <= x;
    // (at least one, whatever a caller's array holds: b stays in range)
    const int c = max(__popc(__ballot_sync(0xffffffffu, in)), 1);
    lo += (c - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

}  // namespace psf
