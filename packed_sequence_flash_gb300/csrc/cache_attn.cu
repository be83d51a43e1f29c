// cache_attn.cu -- launches of the cache attention: the main kernel, the join of
// partial results, and the weights.
#include "cache_attn.cuh"

namespace psf {

namespace {

// Weights of the keys, from the stored scores and the finished lse: a thread
// sums exp2(score - lse) of four keys over the rows that see them, in their
// order, and adds the sums once (atomically: another sequence may share the page).
constexpr int kWeightThreads = 128;
constexpr int kWeightKeys = 4 * kWeightThreads;
__global__ void __launch_bounds__(kWeightThreads) cache_weight_kernel(const __grid_constant__ CacheAttnParams p) {
  const CacheView& c = p.c;
  const int b = blockIdx.z, h = blockIdx.y, j = blockIdx.x * kWeightKeys + threadIdx.x * 4;
  const Seq q = seq_at(p.s, c.page, b);
  const int pg = j < q.n ? p.s.table[(int64_t)b * p.s.max_pages + (j >> c.page_lg)] : -1;
  const bool none = pg < 0 || pg >= c.pages;
  if (none && !first_block()) return;
  after_previous_kernel();
  if (none) return;
  float* weight = c.weight + ((int64_t)pg * c.Hkv + h) * c.page + (j & (c.page - 1));
  const float* s = p.scores + (((int64_t)b * c.Hkv + h) * p.score_rows) * p.score_cap + j;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < q.m; ++i) {
    int lo, hi;
    ca_row_keys(p, q.n, q.m, i, lo, hi);
    if (j + 4 <= lo || j >= hi) continue;
#pragma unroll 4
    for (int g = 0; g < p.G; ++g) {
      const float4 z = *reinterpret_cast<const float4*>(s + (int64_t)(i * p.G + g) * p.score_cap);
      const float l = p.lse[(int64_t)(h * p.G + g) * p.s.T + q.q0 + i] * 1.4426950408889634f;
      const float e[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j + k >= lo && j + k < hi) sum[k] += ex2_approx(e[k] - l);  // scores past these were never written
    }
  }
  if (j + 4 <= q.n) {
    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(weight), "f"(sum[0]), "f"(sum[1]), "f"(sum[2]),
                 "f"(sum[3])
                 : "memory");
  } else {
    for (int k = 0; j + k < q.n; ++k) atomicAdd(weight + k, sum[k]);
  }
}

template <int DQK, int DV, int NT, bool EXTRA>
cudaError_t run(CacheAttnParams& p, int max_q, int sms, cudaStream_t st) {
  using C = CaCfg<DQK, DV, NT>;
  static std::atomic<uint64_t> main_set{0}, unit_set{0}, share_set{0};
  cudaError_t e = kernel_setup(cache_attn_kernel<DQK, DV, NT, EXTRA>, C::SMEM, true, main_set);
  if (e == cudaSuccess) e = kernel_setup(cache_join_kernel<DV, true>, 0, true, unit_set);
  if (e == cudaSuccess) e = kernel_setup(cache_join_kernel<DV, false>, 0, true, share_set);
  if (e != cudaSuccess) return e;
  const int grid = sms * C::CTAS;
  p.tile_lg = NT == 1 ? 3 : 4;
  p.row_tiles = max(1, (int)(((int64_t)min(max_q, p.s.T) * p.G + C::R - 1) / C::R));
  e = launch_early(cache_attn_kernel<DQK, DV, NT, EXTRA>, dim3(grid), kCaThreads, C::SMEM, st, p);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)p.c.Hkv * p.row_tiles * p.s.B;
  if (units > 2 * grid)  // fewer shares than units: a CTA per share
    return launch_early(cache_join_kernel<DV, false>, dim3(grid), kJoinThreads, 0, st, p, grid);
  int parts = 1;
  while (parts < C::R && units * parts * 2 <= 2 * sms) parts *= 2;
  return launch_early(cache_join_kernel<DV, true>, dim3(p.c.Hkv * p.row_tiles, p.s.B + (p.s.cu ? 1 : 0), parts),
                      kJoinThreads, 0, st, p, grid);
}

template <int DQK, int DV, int NT>
cudaError_t run(CacheAttnParams& p, int max_q, int sms, cudaStream_t st) {
  return p.accumulate || p.softcap > 0.f ? run<DQK, DV, NT, true>(p, max_q, sms, st)
                                         : run<DQK, DV, NT, false>(p, max_q, sms, st);
}

}  // namespace

cudaError_t launch_cache_attn(CacheAttnParams& p, int max_q, int sms, cudaStream_t st) {
  const bool one = cache_attn_nt(p.c.Dqk, (int64_t)max_q * p.G) == 1;
  cudaError_t e;
  if (p.c.Dqk == 64)
    e = one ? run<64, 64, 1>(p, max_q, sms, st) : run<64, 64, 2>(p, max_q, sms, st);
  else if (p.c.Dqk == 128)
    e = one ? run<128, 128, 1>(p, max_q, sms, st) : run<128, 128, 2>(p, max_q, sms, st);
  else if (p.c.Dqk == 192)
    e = one ? run<192, 128, 1>(p, max_q, sms, st) : run<192, 128, 2>(p, max_q, sms, st);
  else
    e = run<512, 512, 1>(p, max_q, sms, st);
  if (e != cudaSuccess || !p.accumulate) return e;
  static std::atomic<uint64_t> weight_set{0};
  if ((e = kernel_setup(cache_weight_kernel, 0, true, weight_set)) != cudaSuccess) return e;
  const unsigned chunks = (unsigned)((p.score_cap + kWeightKeys - 1) / kWeightKeys);
  return launch_early(cache_weight_kernel, dim3(chunks, p.c.Hkv, p.s.B), kWeightThreads, 0, st, p);
}

}  // namespace psf
