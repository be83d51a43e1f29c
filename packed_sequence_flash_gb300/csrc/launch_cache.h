// launch_cache.h -- host-side launchers of the 8-bit cache's kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "cache.cuh"

namespace psf {

// Once per device (done: a bit per device index): a kernel's dynamic shared
// memory limit and, for the attention's kernels, all of an SM's memory to shared
// memory rather than L1. A kernel that starts early shares SMs with the one
// before it, whose split stays while they run: behind a kernel with a small share
// the attention had room for two of its three CTAs per SM, and the third waited
// for one of them to end. The copying kernels need the L1 (the gather took 98 us
// for 84 without it), so they keep it and let nothing start before they are done.
template <typename K>
inline cudaError_t kernel_setup(K kernel, int smem_bytes, bool all_shared, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  if (all_shared)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && smem_bytes > 0)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// For kernels launched by launch_early: waits until the kernel before this one in
// the stream is done, and lets the one after it start (it waits in the same way).
__device__ __forceinline__ void after_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The kernel that comes next waits for this one alone, so this one must not be
// over before the one in front of it: its first block always waits, whatever the others do.
__device__ __forceinline__ bool first_block() { return blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0; }

// A launch that may begin while the kernel before it in the stream still runs;
// its kernel waits with griddepcontrol.wait before it touches memory.
template <typename... A>
inline cudaError_t launch_early(void (*kernel)(A...), dim3 grid, int threads, int smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Eviction workspace: per (sequence, head) whether it is evicted from, the kept
// tokens in order (page and row they come from, old / new scale of K and of V),
// the new blocks' scales (K, V) and, for sequences too long for shared memory,
// the keys of their weights.
constexpr int kEvictSmemKeys = 48 * 1024;
struct EvictWorkspace {
  int* live;       // [B][Hkv]
  int4* items;     // [B][Hkv][budget]
  float2* scale;   // [B][Hkv][blocks]
  uint32_t* keys;  // [B][Hkv][cap], used when cap > kEvictSmemKeys
  int64_t cap;     // tokens a page table row can hold
};

// New rows k, v (strides in elements: row, head) into the cache.
cudaError_t launch_cache_append(const CacheView& c, const SeqView& s, const void* k, int64_t k_ss, int64_t k_sh,
                                const void* v, int64_t v_ss, int64_t v_sh, int f16, int* status, cudaStream_t st);
// Cached rows as packed 16-bit [total_k, Hkv, D], and their prefix sums.
cudaError_t launch_cache_gather(const CacheView& c, const SeqView& s, void* k, void* v, int32_t* cu_k,
                                int64_t total_k, int f16, int* status, cudaStream_t st);
// Selection of the kept tokens, then compaction in place.
cudaError_t launch_cache_evict(const CacheView& c, const SeqView& s, int budget, int recent, int32_t* new_lens,
                               const EvictWorkspace& ws, int sms, int* status, cudaStream_t st);

struct CacheAttnParams {
  CUtensorMap tm_k, tm_v;  // (d, row, head, page) of the codes
  CacheView c;
  SeqView s;
  const void* q;
  int64_t q_ss, q_sh;  // strides in elements (row, head)
  void* out;
  int64_t o_ss, o_sh;
  float* lse;  // [Hq][T]
  int G;  // query heads of a KV head
  uint32_t g_mul;  // x / G = (mulhi(x, g_mul) + x) >> g_shift
  int g_shift;
  float scale, softcap;
  int causal, window;  // window > 0: left window counting the current token
  int accumulate;      // add each key's probabilities to c.weight
  int f16;
  int min_share;  // a CTA's share is at least this many key tiles
  int row_tiles;  // of a sequence with the most rows
  int tile_lg;    // log2 of the rows of a tile
  // Workspace: partial results [CTA][2][R][Dv] and their lse in log2 units
  // [CTA][2][R]; scores [B * Hkv][score_rows][score_cap] in log2 units.
  float *part_o, *part_l, *scores;
  int64_t score_rows, score_cap;
  int* status;
  uint64_t limit_ns;
};
// Groups of 8 query rows in a row tile, for the most rows a KV head has in a
// sequence. Two share what the codes cost to expand: 16 rows over 32 x 32 Ki keys
// took 361 us as one tile and 627 us as two; with up to 8 rows half of the tile
// would be empty. One at head dim 512, whose state fills the registers.
constexpr int cache_attn_nt(int Dqk, int64_t rows) { return Dqk == 512 || rows <= 8 ? 1 : 2; }
// CTAs per SM: as many as shared memory and registers hold.
constexpr int cache_attn_ctas(int Dqk, int nt) { return Dqk == 512 ? 1 : (Dqk == 192 || nt == 2 ? 2 : 3); }
cudaError_t launch_cache_attn(CacheAttnParams& p, int max_q, int sms, cudaStream_t st);

}  // namespace psf
