// cache_attn.cu -- launches of the cache attention: the main kernel, the join of
// partial results, and the weights.
#include "cache_attn.cuh"

namespace psf {

namespace {

// Weights of the keys, from the stored scores and the finished lse: a thread per
// key sums exp2(score - lse) over the rows that see it, in their order, and
// adds the sum once (atomically: another sequence may share the page).
constexpr int kWeightThreads = 256;
__global__ void __launch_bounds__(kWeightThreads) cache_weight_kernel(const __grid_constant__ CacheAttnParams p) {
  const CacheView& c = p.c;
  const int b = blockIdx.z, h = blockIdx.y, j = blockIdx.x * kWeightThreads + threadIdx.x;
  const Seq q = seq_at(p.s, c.page, b);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (j >= q.n) return;
  const int pg = p.s.table[(int64_t)b * p.s.max_pages + (j >> c.page_lg)];
  if (pg < 0 || pg >= c.pages) return;
  const float* s = p.scores + (((int64_t)b * c.Hkv + h) * p.score_rows) * p.score_cap + j;
  float sum = 0.f;
  for (int i = 0; i < q.m; ++i) {
    int lo, hi;
    ca_row_keys(p, q.n, q.m, i, lo, hi);
    if (j < lo || j >= hi) continue;
    for (int g = 0; g < p.G; ++g)
      sum += ex2_approx(s[(int64_t)(i * p.G + g) * p.score_cap] -
                        p.lse[(int64_t)(h * p.G + g) * p.s.T + q.q0 + i] * 1.4426950408889634f);
  }
  atomicAdd(c.weight + ((int64_t)pg * c.Hkv + h) * c.page + (j & (c.page - 1)), sum);
}

// A kernel that may start while the one before it still runs (it waits with griddepcontrol.wait).
template <typename... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, int threads, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int DQK, int DV, int NT>
cudaError_t run(CacheAttnParams& p, int max_q, int sms, cudaStream_t st) {
  using C = CaCfg<DQK, DV, NT>;
  cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<DQK, DV, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::SMEM);
  if (e != cudaSuccess) return e;
  const int grid = sms * C::CTAS;
  p.row_tiles = max(1, (int)(((int64_t)max_q * p.G + C::R - 1) / C::R));
  cache_attn_kernel<DQK, DV, NT><<<grid, kCaThreads, C::SMEM, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_after(cache_join_kernel<DQK, DV, NT>, dim3(p.c.Hkv * p.row_tiles, p.s.B + (p.s.cu ? 1 : 0)),
                      kJoinThreads, st, (const CacheAttnParams)p, grid);
}

}  // namespace

// Row tiles of 8 rows for one group of heads and one token, of 16 and 32 rows
// where there are more rows; 8 at head dim 512, where O takes 128 registers.
int cache_attn_nt(int Dqk, int64_t rows) { return Dqk == 512 || rows <= 8 ? 1 : (rows <= 16 ? 2 : 4); }

cudaError_t launch_cache_attn(CacheAttnParams& p, int max_q, int sms, cudaStream_t st) {
  const int nt = cache_attn_nt(p.c.Dqk, (int64_t)max_q * p.G);
  cudaError_t e;
#define PSF_RUN(DQK, DV)                                              \
  e = nt == 1 ? run<DQK, DV, 1>(p, max_q, sms, st)                    \
              : (nt == 2 ? run<DQK, DV, 2>(p, max_q, sms, st) : run<DQK, DV, 4>(p, max_q, sms, st))
  if (p.c.Dqk == 64)
    PSF_RUN(64, 64);
  else if (p.c.Dqk == 128)
    PSF_RUN(128, 128);
  else if (p.c.Dqk == 192)
    PSF_RUN(192, 128);
  else
    e = run<512, 512, 1>(p, max_q, sms, st);
#undef PSF_RUN
  if (e != cudaSuccess || !p.accumulate) return e;
  const unsigned chunks = (unsigned)((p.score_cap + kWeightThreads - 1) / kWeightThreads);
  return launch_after(cache_weight_kernel, dim3(chunks, p.c.Hkv, p.s.B), kWeightThreads, st,
                      (const CacheAttnParams)p);
}

}  // namespace psf
