// cache.cu -- the memory-bound kernels of the 8-bit paged cache: append
// (quantise new rows into their pages), gather (pages back to packed 16-bit
// rows) and eviction (selection of the tokens to keep, compaction in place).
#include "cache.cuh"
#include "launch.h"
#include "launch_cache.h"

namespace psf {

namespace {

// ---------------------------------------------------------------- append
// One CTA per (sequence, page it enters, head, K or V): the largest new
// magnitude, the block's scale, the older codes of the page if the scale grew,
// the new codes. Bound by memory: 2 bytes read and 1 written per element. The
// largest magnitude is taken on packed 16-bit patterns (their order without the
// sign is that of the values) and codes are made with a product by the scale's
// reciprocal, exact for a power of two: with a division and a test of every
// element for being finite, 10 Ki prompt tokens of 8 heads of 128 took 30 us, now
// 18 (floor 9.4; the rest is the chain of loads from cu to the page). Sequence
// b's pages are tasks start(b) .. in an index space that leaves floor(cu / page) +
// 2 b tasks before it, room enough for the floor((n - 2) / page) + 2 pages that n
// rows can touch, so a CTA finds its page from cu alone.
constexpr int kAppendThreads = 128;
constexpr float kMaxFloat = 3.402823466e38f;
constexpr int kAppendHeld = 8;  // 16-byte vectors a thread keeps between its two looks at the rows

template <typename T>
__global__ void __launch_bounds__(kAppendThreads, 8)
    append_kernel(CacheView c, SeqView s, const T* kin, int64_t k_ss, int64_t k_sh, const T* vin, int64_t v_ss,
                  int64_t v_sh, int* status) {
  __shared__ float warp_top[kAppendThreads / 32];
  const int tid = threadIdx.x, h = blockIdx.y;
  const bool is_v = blockIdx.z;
  auto start = [&](int b) -> int64_t { return (s.cu ? s.cu[b] : b * s.each) / c.page + 2 * (int64_t)b; };
  after_previous_kernel();
  if (first_block()) {
    bool bad = cu_bad(s);
    for (int i = tid; i < s.B; i += kAppendThreads) {
      const Seq x = seq_at(s, c.page, i);
      bad |= x.bad || x.m > x.n;
    }
    if (bad) record_status(status, kStatusDeviceArgs);
  }
  const int b = warp_find(s.B, blockIdx.x, start);
  const Seq q = seq_at(s, c.page, b);
  if (q.bad || q.m > q.n) return;
  const int64_t nth = (int64_t)blockIdx.x - start(b);
  const int first = q.n - q.m;  // position of the first new token
  const int64_t pi = (first >> c.page_lg) + nth;
  if (nth < 0 || q.m == 0 || pi > (q.n - 1) >> c.page_lg) return;
  const int pg = s.table[(int64_t)b * s.max_pages + pi];
  if (pg < 0 || pg >= c.pages) {
    if (tid == 0) record_status(status, kStatusDeviceArgs);
    return;
  }
  const int base = (int)pi << c.page_lg;
  const int r0 = max(first - base, 0), r1 = min(q.n - base, c.page);  // new rows of the page
  const int D = is_v ? c.Dv : c.Dqk;
  const int lg = D == 192 ? 0 : 31 - __clz(D >> 3);
  const int vecs = D >> 3;  // 8-element vectors of a row
  const T* in = is_v ? vin : kin;
  const int64_t ss = is_v ? v_ss : k_ss;
  in += (is_v ? v_sh : k_sh) * h + ss * (base + r0 - first + q.q0);
  uint8_t* out = is_v ? c.v + c.v_sp * pg + c.v_sh * h : c.k + c.k_sp * pg + c.k_sh * h;
  const int64_t sr = is_v ? c.v_sr : c.k_sr;
  float* scale_at = (is_v ? c.v_scale : c.k_scale) + (int64_t)pg * c.Hkv + h;
  const int items = (r1 - r0) * vecs;
  auto row_of = [&](int i) { return D == 192 ? i / 24 : i >> lg; };

  uint4 held[kAppendHeld];
  uint32_t most = 0;  // largest patterns without sign, of the low and of the high halves
  auto look = [&](const uint4& x) {
    most = __vmaxu2(most, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                   __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
  };
  auto load = [&](int i) {
    const int r = row_of(i);
    return *reinterpret_cast<const uint4*>(in + ss * r + (i - r * vecs) * 8);
  };
#pragma unroll
  for (int u = 0; u < kAppendHeld; ++u) {
    const int i = u * kAppendThreads + tid;
    held[u] = i < items ? load(i) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < kAppendHeld; ++u) look(held[u]);
#pragma unroll 2
  for (int i = kAppendHeld * kAppendThreads + tid; i < items; i += kAppendThreads) look(load(i));
  const float2 pair = unpack2<T>(most);
  const bool odd = __syncthreads_or(!(pair.x <= kMaxFloat) || !(pair.y <= kMaxFloat));  // inf or NaN among the rows
  float top = fmaxf(pair.x, pair.y);
  if (odd) {  // once more, over the finite values alone
    top = 0.f;
#pragma unroll 1
    for (int i = tid; i < items; i += kAppendThreads) {
      const uint4 x = load(i);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack2<T>(w[j]);
        if (fabsf(f.x) <= kMaxFloat) top = fmaxf(top, fabsf(f.x));
        if (fabsf(f.y) <= kMaxFloat) top = fmaxf(top, fabsf(f.y));
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) warp_top[tid >> 5] = top;
  const float old = *scale_at;
  __syncthreads();  // also: every thread has read the old scale
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) top = fmaxf(top, warp_top[w]);
  const float fresh = block_scale(top);
  const float scale = r0 > 0 ? fmaxf(fresh, old) : fresh;
  if (tid == 0 && (r0 == 0 || scale != old)) *scale_at = scale;

  if (r0 > 0 && scale != old) {
    const float r = old / scale;
    for (int i = tid; i < r0 * (D >> 4); i += kAppendThreads) {
      const int row = i / (D >> 4);
      uint4* at = reinterpret_cast<uint4*>(out + sr * row + (i - row * (D >> 4)) * 16);
      *at = rescale16(*at, r);
    }
  }
  auto store = [&](int i, const uint32_t (&e)[4]) {
    const int row = row_of(i);
    *reinterpret_cast<uint2*>(out + sr * (r0 + row) + (i - row * vecs) * 8) =
        make_uint2(e[0] | (e[1] << 16), e[2] | (e[3] << 16));
  };
  // A scale that the append chose is a power of two; one that was there may not be.
  if (!odd && (__float_as_int(scale) & 0x7fffff) == 0 && scale > 0.f) {
    const float inv = 1.f / scale;
    auto put = [&](int i, const uint4& x) {
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t e[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack2<T>(w[j]);
        e[j] = e4m3_pair(f.x * inv, f.y * inv);
      }
      store(i, e);
    };
#pragma unroll
    for (int u = 0; u < kAppendHeld; ++u) {
      const int i = u * kAppendThreads + tid;
      if (i < items) put(i, held[u]);
    }
    for (int i = kAppendHeld * kAppendThreads + tid; i < items; i += kAppendThreads) put(i, load(i));
  } else {
#pragma unroll 1
    for (int i = tid; i < items; i += kAppendThreads) {
      const uint4 x = load(i);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t e[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack2<T>(w[j]);
        e[j] = e4m3_pair(divide_to_odd(finite_or_nan(f.x), scale), divide_to_odd(finite_or_nan(f.y), scale));
      }
      store(i, e);
    }
  }
  if (!is_v && c.weight)
    for (int r = r0 + tid; r < r1; r += kAppendThreads) c.weight[((int64_t)pg * c.Hkv + h) * c.page + r] = 0.f;
}

// One new row per sequence (a decode step): a warp per (sequence, K or V, head).
// Latency bounds it: length -> page -> old scale, the row's largest magnitude in
// a warp, at most a page of older codes when the scale grew. 64 sequences of 8
// heads: 3.7 us; 4096: 30 us. With a CTA each, as above, 6.6 and 252 us.
template <typename T>
__global__ void __launch_bounds__(kAppendThreads)
    append_one_kernel(CacheView c, SeqView s, const T* kin, int64_t k_ss, int64_t k_sh, const T* vin, int64_t v_ss,
                      int64_t v_sh, int* status) {
  const int lane = threadIdx.x & 31;
  const int64_t task = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int b = (int)(task / (2 * c.Hkv)), y = (int)(task - (int64_t)b * 2 * c.Hkv);
  const bool is_v = y >= c.Hkv;
  const int h = is_v ? y - c.Hkv : y;
  after_previous_kernel();
  if (b >= s.B) return;
  const int D = is_v ? c.Dv : c.Dqk, words = D >> 6;  // pairs of elements per lane: 1, 2, 3 or 8
  const uint32_t* in = reinterpret_cast<const uint32_t*>(is_v ? vin + v_ss * b + v_sh * h : kin + k_ss * b + k_sh * h);
  uint32_t w[8], most = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = j < words ? in[lane * words + j] : 0;
  const int n = s.lens[b];
  bool ok = n >= 1 && (int64_t)n <= (int64_t)s.max_pages * c.page;
  const int row = (n - 1) & (c.page - 1);
  const int pg = ok ? s.table[(int64_t)b * s.max_pages + ((n - 1) >> c.page_lg)] : -1;
  ok = pg >= 0 && pg < c.pages;
  if (!ok) {
    if (lane == 0) record_status(status, kStatusDeviceArgs);
    return;
  }
  float* scale_at = (is_v ? c.v_scale : c.k_scale) + (int64_t)pg * c.Hkv + h;
  const float old = *scale_at;
#pragma unroll
  for (int j = 0; j < 8; ++j) most = __vmaxu2(most, w[j] & 0x7fff7fffu);
  const float2 pair = unpack2<T>(most);
  float top = fmaxf(pair.x, pair.y);
  const bool odd = __any_sync(0xffffffffu, !(pair.x <= kMaxFloat) || !(pair.y <= kMaxFloat));
  if (odd) {  // inf or NaN in the row: over the finite values alone
    top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 f = unpack2<T>(w[j]);
      if (fabsf(f.x) <= kMaxFloat) top = fmaxf(top, fabsf(f.x));
      if (fabsf(f.y) <= kMaxFloat) top = fmaxf(top, fabsf(f.y));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float fresh = block_scale(top), scale = row > 0 ? fmaxf(fresh, old) : fresh;
  uint8_t* out = is_v ? c.v + c.v_sp * pg + c.v_sh * h : c.k + c.k_sp * pg + c.k_sh * h;
  const int64_t sr = is_v ? c.v_sr : c.k_sr;
  if (row > 0 && scale != old) {
    const float r = old / scale;
    const int vecs = D >> 4;
#pragma unroll 4
    for (int i = lane; i < row * vecs; i += 32) {
      const int at = i / vecs;
      uint4* x = reinterpret_cast<uint4*>(out + sr * at + (i - at * vecs) * 16);
      *x = rescale16(*x, r);
    }
  }
  const bool plain = !odd && (__float_as_int(scale) & 0x7fffff) == 0 && scale > 0.f;
  const float inv = 1.f / scale;
  uint16_t* to = reinterpret_cast<uint16_t*>(out + sr * row) + lane * words;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < words) {
      const float2 f = unpack2<T>(w[j]);
      to[j] = (uint16_t)(plain ? e4m3_pair(f.x * inv, f.y * inv)
                               : e4m3_pair(divide_to_odd(finite_or_nan(f.x), scale),
                                           divide_to_odd(finite_or_nan(f.y), scale)));
    }
  if (lane == 0) {
    if (row == 0 || scale != old) *scale_at = scale;
    if (!is_v && c.weight) c.weight[((int64_t)pg * c.Hkv + h) * c.page + row] = 0.f;
  }
}

// ---------------------------------------------------------------- gather
// cu_k = prefix sums of the lengths (one CTA).
constexpr int kPrefixThreads = 1024;
__global__ void __launch_bounds__(kPrefixThreads)
    gather_prefix_kernel(SeqView s, int page, int32_t* cu_k, int64_t total_k, int* status) {
  __shared__ int64_t tot[32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  after_previous_kernel();
  let_next_kernel_start();
  int64_t carry = 0;
  for (int base = 0; base < s.B; base += kPrefixThreads) {
    const int b = base + tid;
    int64_t x = 0;
    if (b < s.B) {
      const int n = s.lens[b];
      if (n < 0 || (int64_t)n > (int64_t)s.max_pages * page)
        record_status(status, kStatusDeviceArgs);
      else
        x = n;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) tot[wid] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
      before += w < wid ? tot[w] : 0;
      all += tot[w];
    }
    const int64_t sum = carry + before + x;
    if (b < s.B) cu_k[b + 1] = (int32_t)min(sum, (int64_t)0x7fffffff);
    carry += all;
    __syncthreads();
  }
  if (tid == 0) {
    cu_k[0] = 0;
    if (carry > total_k) record_status(status, kStatusDeviceArgs);
  }
}

// One CTA per (sequence, page, head, K or V). Bound by memory: 1 byte read and 2
// written per element (82,859 tokens of 8 heads of 128: 85 us, 0.88 of a copy's
// rate). Sequence b's pages are tasks floor(cu_k / page) + b onwards (a sequence
// of n tokens has at most floor(n / page) + 1 pages). Rows at or past total_k are not written.
constexpr int kGatherThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kGatherThreads)
    gather_kernel(CacheView c, SeqView s, const int32_t* cu_k, T* ko, T* vo, int64_t total_k, int* status) {
  const int tid = threadIdx.x, h = blockIdx.y;
  const bool is_v = blockIdx.z;
  auto start = [&](int b) -> int64_t { return cu_k[b] / c.page + (int64_t)b; };
  after_previous_kernel();
  const int b = warp_find(s.B, blockIdx.x, start);
  const int64_t pi = (int64_t)blockIdx.x - start(b);
  const int row0 = cu_k[b], n = cu_k[b + 1] - row0;
  if (pi < 0 || (pi << c.page_lg) >= n) return;
  const int pg = s.table[(int64_t)b * s.max_pages + pi];
  if (pg < 0 || pg >= c.pages) {
    if (tid == 0) record_status(status, kStatusDeviceArgs);
    return;
  }
  const int D = is_v ? c.Dv : c.Dqk;
  const int64_t at = row0 + (pi << c.page_lg);
  const int rows = (int)min((int64_t)min(n - (int)(pi << c.page_lg), c.page), total_k - at);
  const uint8_t* in = is_v ? c.v + c.v_sp * pg + c.v_sh * h : c.k + c.k_sp * pg + c.k_sh * h;
  const int64_t sr = is_v ? c.v_sr : c.k_sr;
  const float scale = (is_v ? c.v_scale : c.k_scale)[(int64_t)pg * c.Hkv + h];
  T* out = (is_v ? vo : ko) + (at * c.Hkv + h) * D;
  const int vecs = D >> 4;
  for (int i = tid; i < rows * vecs; i += kGatherThreads) {
    const int r = i / vecs, col = (i - r * vecs) * 16;
    const uint4 x = *reinterpret_cast<const uint4*>(in + sr * r + col);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = e4m3_to_float2(w[j] & 0xffff), d = e4m3_to_float2(w[j] >> 16);
      o[2 * j] = pack2<T>(a.x * scale, a.y * scale);
      o[2 * j + 1] = pack2<T>(d.x * scale, d.y * scale);
    }
    uint4* to = reinterpret_cast<uint4*>(out + (int64_t)r * c.Hkv * D + col);
    to[0] = make_uint4(o[0], o[1], o[2], o[3]);
    to[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// ---------------------------------------------------------------- eviction
// Order of the weights as unsigned integers: NaN above all, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_weight(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

constexpr int kSelectThreads = 512;

// Exclusive block-wide prefix sum.
__device__ int select_scan(int v, int* warp_tot) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_tot[wid] = x;
  __syncthreads();
  const int before = __reduce_add_sync(0xffffffffu, lane < wid ? warp_tot[lane] : 0);
  __syncthreads();
  return before + x - v;
}

constexpr int kSelectBins = 2048;

// One CTA per (head, sequence). The smallest kept weight is found digit by digit
// (11, 11 and 10 bits of its key) from histograms in shared memory (integer
// counts: their order does not matter). Then the kept tokens
// are listed in their order, the new blocks' scales set and the weights written.
// Latency bounds it: a few passes over one head's weights, which stay in shared
// memory (in the workspace when they are too many). Halving the interval of keys
// instead, two bits a pass, took 16 passes: 96 us against 44 for 384 heads of 11 Ki tokens.
__global__ void __launch_bounds__(kSelectThreads, 2)
    evict_select_kernel(CacheView c, SeqView s, int budget, int recent, int32_t* new_lens, EvictWorkspace ws,
                        int smem_keys, int smem_kept, int* status) {
  extern __shared__ uint32_t dyn_smem[];  // keys, then the list of kept tokens
  __shared__ int hist[kSelectBins];
  __shared__ int warp_tot[32], found_bin, found_above;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int h = blockIdx.x, b = blockIdx.y;
  after_previous_kernel();
  let_next_kernel_start();
  const int n = s.lens[b];
  const int32_t* table = s.table + (int64_t)b * s.max_pages;
  const int64_t unit = (int64_t)b * c.Hkv + h;
  bool bad = n < 0 || (int64_t)n > (int64_t)s.max_pages * c.page;
  if (!bad && n > budget)
    for (int i = tid; i < (n + c.page - 1) >> c.page_lg; i += kSelectThreads)
      bad |= table[i] < 0 || table[i] >= c.pages;
  bad = __syncthreads_or(bad);
  const bool skip = bad || n <= budget;
  if (tid == 0) {
    if (bad) record_status(status, kStatusDeviceArgs);
    if (h == 0) new_lens[b] = skip ? n : budget;
    ws.live[unit] = skip ? 0 : 1;
  }
  if (skip) return;

  const int old = n - recent, need = budget - recent;
  uint32_t* keys = n <= smem_keys ? dyn_smem : ws.keys + unit * ws.cap;
  int4* items = ws.items + unit * budget;
  int* kept = reinterpret_cast<int*>(dyn_smem + smem_keys);  // when budget <= smem_kept
  const bool in_smem = budget <= smem_kept;
  auto weight_at = [&](int j) -> float* {
    return c.weight + ((int64_t)table[j >> c.page_lg] * c.Hkv + h) * c.page + (j & (c.page - 1));
  };
  // Four tokens at a time (of one page, whose rows all exist).
#pragma unroll 4
  for (int j = tid * 4; j < n; j += kSelectThreads * 4) {
    const float4 w = *reinterpret_cast<const float4*>(weight_at(j));
    *reinterpret_cast<uint4*>(keys + j) =
        make_uint4(weight_key(w.x), weight_key(w.y), weight_key(w.z), weight_key(w.w));
  }
  uint32_t thr = 0xffffffffu;  // key of the smallest kept weight
  int all_above = 0;           // older tokens with a larger key
  if (need > 0) {
    thr = 0;
    int shift = 21;
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? 11 : 10;
      for (int i = tid; i < kSelectBins; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
#pragma unroll 2
      for (int j = tid * 4; j < old; j += kSelectThreads * 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(keys + j);
        const uint32_t k[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < old && (pass == 0 || (k[e] >> (shift + bits)) == (thr >> (shift + bits))))
            atomicAdd(&hist[(k[e] >> shift) & ((1 << bits) - 1)], 1);
      }
      __syncthreads();
      // Bins from the top, a few per thread: the one in which the count reaches `need`.
      constexpr int PER = kSelectBins / kSelectThreads;
      const int hi = kSelectBins - 1 - PER * tid;
      int sum = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) sum += hist[hi - i];
      int before = all_above + select_scan(sum, warp_tot);
      if (before < need && before + sum >= need) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int count = hist[hi - i];
          if (before < need && before + count >= need) {
            found_bin = hi - i;
            found_above = before;
          }
          before += count;
        }
      }
      __syncthreads();
      thr |= (uint32_t)found_bin << shift;
      all_above = found_above;
      shift -= pass == 0 ? 11 : 10;
    }
  } else {
    __syncthreads();
  }
  // Thread t lists tokens [t per, (t + 1) per); an odd `per` spreads the shared-memory reads.
  const int per = ((n + kSelectThreads - 1) / kSelectThreads) | 1;
  const int j0 = min(tid * per, n), j1 = min(j0 + per, n);
  int above = 0, equal = 0;
  for (int j = j0; j < min(j1, old); ++j) {
    above += keys[j] > thr;
    equal += keys[j] == thr;
  }
  const int quota = need - all_above;  // tokens with exactly the smallest kept weight: the first ones
  const int eq_before = select_scan(equal, warp_tot);
  const int eq_kept = min(max(quota - eq_before, 0), equal);
  const int mine = above + eq_kept + max(j1 - max(j0, old), 0);
  int at = select_scan(mine, warp_tot);
  for (int j = j0, left = eq_kept; j < j1; ++j) {
    bool keep = j >= old || keys[j] > thr;
    if (!keep && keys[j] == thr && left > 0) {
      keep = true;
      --left;
    }
    if (keep) {
      if (in_smem)
        kept[at] = j;
      else
        items[at].x = j;
      ++at;
    }
  }
  __syncthreads();

  // Blocks: a warp takes 128 kept tokens, four per lane. A new block's scale is
  // the largest of its tokens' scales; where each token comes from and the
  // ratios of the scales go to the kernel that moves the codes.
  const int blocks = (budget + c.page - 1) >> c.page_lg;
  for (int base = wid * 128; base < budget; base += kSelectThreads / 32 * 128) {
    int from[4], pg[4];
    float sk[4], sv[4], tk[4], tv[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = base + u * 32 + lane;
      from[u] = j < budget ? (in_smem ? kept[j] : items[j].x) : -1;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) pg[u] = from[u] >= 0 ? table[from[u] >> c.page_lg] : 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t a = (int64_t)pg[u] * c.Hkv + h;
      tk[u] = sk[u] = from[u] >= 0 ? c.k_scale[a] : 0.f;
      tv[u] = sv[u] = from[u] >= 0 ? c.v_scale[a] : 0.f;
    }
    const int width = min(c.page, 32);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      for (int o = 1; o < width; o <<= 1) {
        tk[u] = fmaxf(tk[u], __shfl_xor_sync(0xffffffffu, tk[u], o));
        tv[u] = fmaxf(tv[u], __shfl_xor_sync(0xffffffffu, tv[u], o));
      }
    if (c.page >= 64) {
      tk[0] = tk[1] = fmaxf(tk[0], tk[1]);
      tk[2] = tk[3] = fmaxf(tk[2], tk[3]);
      tv[0] = tv[1] = fmaxf(tv[0], tv[1]);
      tv[2] = tv[3] = fmaxf(tv[2], tv[3]);
    }
    if (c.page == 128) {
      tk[0] = tk[1] = tk[2] = tk[3] = fmaxf(tk[0], tk[2]);
      tv[0] = tv[1] = tv[2] = tv[3] = fmaxf(tv[0], tv[2]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = base + u * 32 + lane;
      if (j < budget) {
        const float rk = tk[u] > 0.f ? sk[u] / tk[u] : 1.f, rv = tv[u] > 0.f ? sv[u] / tv[u] : 1.f;
        items[j] = make_int4(pg[u], from[u] & (c.page - 1), __float_as_int(rk), __float_as_int(rv));
        *weight_at(j) = key_weight(keys[from[u]]);
        if ((j & (c.page - 1)) == 0) ws.scale[unit * blocks + (j >> c.page_lg)] = make_float2(tk[u], tv[u]);
      }
    }
  }
  __syncthreads();  // every old scale has been read
  for (int blk = tid; blk < blocks; blk += kSelectThreads) {
    const float2 t = ws.scale[unit * blocks + blk];
    const int64_t a = (int64_t)table[blk] * c.Hkv + h;
    c.k_scale[a] = t.x;
    c.v_scale[a] = t.y;
  }
}

// Moves the codes: one CTA per (head, sequence, K or V, column slice), the kept
// tokens in order and in batches. A token never moves up, so a batch's writes
// touch nothing that a later batch still has to read: the next batch is on its
// way while one is written, which waits only until all of its own rows are read.
// Slices of a row go to CTAs of their own when (head, sequence) pairs alone
// would not fill the device. Bound by memory: every kept code is read and written
// once, in rows of 128 bytes scattered over the old pages; 384 heads x 4096 of
// 11 Ki tokens of head dim 128 move 786 MB in 136 us, 0.85 of a copy's rate (156 us
// with a batch read only after the one before was written).
constexpr int kMoveThreads = 256;
constexpr int kMoveVecs = 2;  // of a batch per thread; with 3 or 4 fewer CTAs fit an SM (4: 227 us for 183 in all)
__global__ void __launch_bounds__(kMoveThreads, 6)
    evict_move_kernel(CacheView c, SeqView s, int budget, EvictWorkspace ws, int slices) {
  const int tid = threadIdx.x, h = blockIdx.x, b = blockIdx.y;
  const bool is_v = blockIdx.z & 1;
  const int slice = blockIdx.z >> 1;
  const int64_t unit = (int64_t)b * c.Hkv + h;
  const int vecs = ((is_v ? c.Dv : c.Dqk) >> 4) / slices;  // 16-byte vectors of this CTA's part of a row
  const int32_t* table = s.table + (int64_t)b * s.max_pages;
  const int rows = kMoveThreads / vecs, mine = tid / vecs;  // rows a pass, and this thread's of them
  const int64_t sp = is_v ? c.v_sp : c.k_sp, sr = is_v ? c.v_sr : c.k_sr;
  uint8_t* base = (is_v ? c.v + c.v_sh * h : c.k + c.k_sh * h) + (slice * vecs + tid - mine * vecs) * 16;
  const int4* items = ws.items + unit * budget;
  const int last = mine < rows ? budget : 0;  // threads past the rows of a pass have none
  after_previous_kernel();
  if (!ws.live[unit]) return;
  uint4 x[kMoveVecs], next[kMoveVecs];
  float r[kMoveVecs], r_next[kMoveVecs];
  int2 at[kMoveVecs];  // page and row of the next batch's tokens
  auto look = [&](int j0) {
#pragma unroll
    for (int u = 0; u < kMoveVecs; ++u) {
      const int j = j0 + u * rows;
      if (j < last) {
        const int4 from = items[j];
        at[u] = make_int2(from.x, from.y);
        r_next[u] = __int_as_float(is_v ? from.w : from.z);
      }
    }
  };
  auto load = [&](int j0) {
#pragma unroll
    for (int u = 0; u < kMoveVecs; ++u)
      if (j0 + u * rows < last) next[u] = *reinterpret_cast<const uint4*>(base + sp * at[u].x + sr * at[u].y);
  };
  const int step = rows * kMoveVecs;
  look(mine);
  load(mine);
  for (int j0 = mine; j0 - mine < budget; j0 += step) {
#pragma unroll
    for (int u = 0; u < kMoveVecs; ++u) {
      x[u] = next[u];
      r[u] = r_next[u];
    }
    look(j0 + step);
    __syncthreads();  // the batch is read
    load(j0 + step);
#pragma unroll
    for (int u = 0; u < kMoveVecs; ++u) {
      const int j = j0 + u * rows;
      if (j < last) {
        if (r[u] != 1.f) x[u] = rescale16(x[u], r[u]);
        *reinterpret_cast<uint4*>(base + sp * table[j >> c.page_lg] + sr * (j & (c.page - 1))) = x[u];
      }
    }
  }
}

}  // namespace

cudaError_t launch_cache_append(const CacheView& c, const SeqView& s, const void* k, int64_t k_ss, int64_t k_sh,
                                const void* v, int64_t v_ss, int64_t v_sh, int f16, int* status, cudaStream_t st) {
  // One row per sequence: a warp per row and head. Else a CTA per page and head.
  const bool one = !s.cu && s.each == 1;
  const int warps = kAppendThreads / 32;
  const dim3 grid = one ? dim3((unsigned)(((int64_t)s.B * 2 * c.Hkv + warps - 1) / warps))
                        : dim3((unsigned)(s.T / c.page + 2 * (int64_t)s.B), c.Hkv, 2);
  if (f16)
    return launch_early(one ? append_one_kernel<__half> : append_kernel<__half>, grid, kAppendThreads, 0, st, c, s,
                        static_cast<const __half*>(k), k_ss, k_sh, static_cast<const __half*>(v), v_ss, v_sh, status);
  return launch_early(one ? append_one_kernel<__nv_bfloat16> : append_kernel<__nv_bfloat16>, grid, kAppendThreads, 0, st,
                      c, s, static_cast<const __nv_bfloat16*>(k), k_ss, k_sh, static_cast<const __nv_bfloat16*>(v),
                      v_ss, v_sh, status);
}

cudaError_t launch_cache_gather(const CacheView& c, const SeqView& s, void* k, void* v, int32_t* cu_k,
                                int64_t total_k, int f16, int* status, cudaStream_t st) {
  cudaError_t e = launch_early(gather_prefix_kernel, dim3(1), kPrefixThreads, 0, st, s, c.page, cu_k, total_k, status);
  if (e != cudaSuccess || total_k == 0) return e;
  const dim3 grid((unsigned)(total_k / c.page + s.B), c.Hkv, 2);
  if (f16)
    return launch_early(gather_kernel<__half>, grid, kGatherThreads, 0, st, c, s, (const int32_t*)cu_k,
                        static_cast<__half*>(k), static_cast<__half*>(v), total_k, status);
  return launch_early(gather_kernel<__nv_bfloat16>, grid, kGatherThreads, 0, st, c, s, (const int32_t*)cu_k,
                      static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v), total_k, status);
}

cudaError_t launch_cache_evict(const CacheView& c, const SeqView& s, int budget, int recent, int32_t* new_lens,
                               const EvictWorkspace& ws, int sms, int* status, cudaStream_t st) {
  static std::atomic<uint64_t> select_set{0};
  cudaError_t e = kernel_setup(evict_select_kernel, kEvictSmemKeys * 4, false, select_set);
  if (e != cudaSuccess) return e;
  const int smem_keys = (int)(ws.cap < kEvictSmemKeys ? ws.cap : kEvictSmemKeys);
  const int smem_kept = smem_keys + (int64_t)budget <= kEvictSmemKeys ? budget : 0;
  e = launch_early(evict_select_kernel, dim3(c.Hkv, s.B), kSelectThreads, (smem_keys + smem_kept) * 4, st, c, s, budget,
                   recent, new_lens, ws, smem_keys, smem_kept, status);
  if (e != cudaSuccess) return e;
  // Two CTAs per SM if the rows can be cut that far: parts of 32 bytes (a memory sector) or more.
  const int least = (c.Dqk < c.Dv ? c.Dqk : c.Dv) / 32;
  int slices = 1;
  while (slices * 2 <= least && slices < 4 && (int64_t)c.Hkv * s.B * 2 * slices < 2 * sms) slices *= 2;
  return launch_early(evict_move_kernel, dim3(c.Hkv, s.B, 2 * slices), kMoveThreads, 0, st, c, s, budget, ws, slices);
}

}  // namespace psf
