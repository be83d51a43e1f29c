// cache_attn.cu -- attention of a few query rows per sequence over the 8-bit
// paged cache.
#include "cache.cuh"
#include "launch_cache.h"

namespace psf {

namespace {

// Keys [lo, hi) that row i of a sequence with m rows and n cached tokens sees
// (the last row sits at the last token).
__device__ __forceinline__ void row_keys(const CacheAttnParams& p, int n, int m, int i, int& lo, int& hi) {
  const int at = i + n - m;
  hi = p.causal ? min(n, at + 1) : n;
  lo = p.window > 0 ? max(0, at - p.window + 1) : 0;
  if (hi < lo) hi = lo;
}

__device__ __forceinline__ float logit(const CacheAttnParams& p, float dot) {
  const float z = dot * p.scale;
  return p.softcap > 0.f ? p.softcap * tanhf(z / p.softcap) : z;
}

// One CTA per (query row, query head): the scores of all keys in two passes
// (maximum and sum, then the weighted values), all in fp32.
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
template <typename T>
__global__ void __launch_bounds__(kThreads) cache_attn_kernel(const CacheAttnParams p) {
  __shared__ float qs[512], red[2][kWarps], acc[512];
  const CacheView& c = p.c;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int t = blockIdx.x, hq = blockIdx.y, h = hq / p.G;
  T* out = static_cast<T*>(p.out) + p.o_ss * t + p.o_sh * hq;
  float* lse = p.lse + (int64_t)hq * p.s.T + t;
  int b = 0;
  if (p.s.cu)
    b = warp_find(p.s.B, t, [&](int x) -> int64_t { return p.s.cu[x]; });
  else
    b = p.s.each ? t / p.s.each : 0;
  Seq q = seq_at(p.s, c.page, b);
  if (q.bad && tid == 0) record_status(p.status, kStatusDeviceArgs);
  int lo = 0, hi = 0;
  if (t >= q.q0 && t < q.q0 + q.m) row_keys(p, q.n, q.m, t - q.q0, lo, hi);
  const T* qr = static_cast<const T*>(p.q) + p.q_ss * t + p.q_sh * hq;
  for (int d = tid; d < c.Dqk; d += kThreads) qs[d] = (float)qr[d];
  for (int d = tid; d < 512; d += kThreads) acc[d] = 0.f;
  __syncthreads();
  const int32_t* table = p.s.table + (int64_t)b * p.s.max_pages;
  auto page_of = [&](int j) {
    int pg = table[j >> c.page_lg];
    if (pg < 0 || pg >= c.pages) {
      record_status(p.status, kStatusDeviceArgs);
      pg = 0;
    }
    return pg;
  };
  auto score = [&](int j) {
    const int pg = page_of(j);
    const uint8_t* k = c.k + c.k_sp * pg + c.k_sh * h + c.k_sr * (j & (c.page - 1));
    float dot = 0.f;
    for (int d = lane * 2; d < c.Dqk; d += 64) {
      const float2 x = e4m3_to_float2(*reinterpret_cast<const uint16_t*>(k + d));
      dot = fmaf(x.x, qs[d], fmaf(x.y, qs[d + 1], dot));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    return logit(p, dot * c.k_scale[(int64_t)pg * c.Hkv + h]);
  };
  float top = -CUDART_INF_F, sum = 0.f;
  for (int j = lo + wid; j < hi; j += kWarps) {
    const float z = score(j), m = fmaxf(top, z);
    sum = sum * __expf(top - m) + expf(z - m);
    top = m;
  }
  if (lane == 0) {
    red[0][wid] = top;
    red[1][wid] = sum;
  }
  __syncthreads();
  float all = -CUDART_INF_F, total = 0.f;
  for (int w = 0; w < kWarps; ++w) all = fmaxf(all, red[0][w]);
  for (int w = 0; w < kWarps; ++w)
    if (red[1][w] > 0.f || red[1][w] != red[1][w]) total += red[1][w] * expf(red[0][w] - all);
  const float l = hi > lo ? all + logf(total) : -CUDART_INF_F;
  float o[16];
  for (int u = 0; u < 16; ++u) o[u] = 0.f;
  for (int j = lo + wid; j < hi; j += kWarps) {
    const float w = expf(score(j) - l);
    const int pg = page_of(j);
    const uint8_t* v = c.v + c.v_sp * pg + c.v_sh * h + c.v_sr * (j & (c.page - 1));
    const float wv = w * c.v_scale[(int64_t)pg * c.Hkv + h];
    for (int u = 0, d = lane * 2; d < c.Dv; d += 64, u += 2) {
      const float2 x = e4m3_to_float2(*reinterpret_cast<const uint16_t*>(v + d));
      o[u] = fmaf(x.x, wv, o[u]);
      o[u + 1] = fmaf(x.y, wv, o[u + 1]);
    }
  }
  for (int w = 0; w < kWarps; ++w) {
    if (wid == w)
      for (int u = 0, d = lane * 2; d < c.Dv; d += 64, u += 2) {
        acc[d] += o[u];
        acc[d + 1] += o[u + 1];
      }
    __syncthreads();
  }
  for (int d = tid * 2; d < c.Dv; d += kThreads * 2)
    *reinterpret_cast<uint32_t*>(out + d) = pack2<T>(acc[d], acc[d + 1]);
  if (tid == 0) *lse = l;
}

// Weights of the keys, from the finished lse: a warp per (sequence, KV head,
// key) sums exp(z - lse) over the rows and heads that see the key, in their order,
// and adds the sum once (atomically: another sequence may share the page).
template <typename T>
__global__ void __launch_bounds__(kThreads) cache_weight_kernel(const CacheAttnParams p) {
  const CacheView& c = p.c;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.z, h = blockIdx.y;
  const Seq q = seq_at(p.s, c.page, b);
  for (int j = blockIdx.x * kWarps + (threadIdx.x >> 5); j < q.n; j += gridDim.x * kWarps) {
    const int pg = p.s.table[(int64_t)b * p.s.max_pages + (j >> c.page_lg)];
    if (pg < 0 || pg >= c.pages) continue;
    const uint8_t* k = c.k + c.k_sp * pg + c.k_sh * h + c.k_sr * (j & (c.page - 1));
    const float ks = c.k_scale[(int64_t)pg * c.Hkv + h];
    float sum = 0.f;
    for (int i = 0; i < q.m; ++i) {
      int lo, hi;
      row_keys(p, q.n, q.m, i, lo, hi);
      if (j < lo || j >= hi) continue;
      for (int g = 0; g < p.G; ++g) {
        const T* qr = static_cast<const T*>(p.q) + p.q_ss * (q.q0 + i) + p.q_sh * (h * p.G + g);
        float dot = 0.f;
        for (int d = lane * 2; d < c.Dqk; d += 64) {
          const float2 x = e4m3_to_float2(*reinterpret_cast<const uint16_t*>(k + d));
          dot = fmaf(x.x, (float)qr[d], fmaf(x.y, (float)qr[d + 1], dot));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        sum += expf(logit(p, dot * ks) - p.lse[(int64_t)(h * p.G + g) * p.s.T + q.q0 + i]);
      }
    }
    if (lane == 0) atomicAdd(c.weight + ((int64_t)pg * c.Hkv + h) * c.page + (j & (c.page - 1)), sum);
  }
}

}  // namespace

cudaError_t launch_cache_attn(const CacheAttnParams& p, int sms, cudaStream_t st) {
  const dim3 grid(p.s.T, p.Hq);
  if (p.f16)
    cache_attn_kernel<__half><<<grid, kThreads, 0, st>>>(p);
  else
    cache_attn_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.accumulate) return e;
  const int keys = p.s.max_pages << p.c.page_lg;
  const dim3 wgrid((unsigned)(keys + kWarps - 1) / kWarps < 256 ? (keys + kWarps - 1) / kWarps : 256, p.c.Hkv, p.s.B);
  if (p.f16)
    cache_weight_kernel<__half><<<wgrid, kThreads, 0, st>>>(p);
  else
    cache_weight_kernel<__nv_bfloat16><<<wgrid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace psf
