// launch_rotary.h -- host-side launchers of the position rotation and of the
// cache's append with it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "cache.cuh"
#include "rotary.cuh"

namespace psf {

// The tensors of a rotation: up to two (queries and keys) of the same rows, H[i] heads each (0: none); strides in
// elements (batch, row, head); S rows in a batch row.
struct RotaryRows {
  const void* x[2];
  void* y[2];
  int64_t xb[2], xs[2], xh[2], yb[2], ys[2], yh[2];
  int H[2];
  int D, S;
  int64_t rows;
  // Where positions are not given: a row's place in its segment (cu: prefix sums of
  // nseg segments, or of dev_meta[0] of them), aligned to the end of the segment's keys (cu_k, nullable), or in its batch row.
  const int32_t* cu;
  const int32_t* cu_k;
  const int32_t* dev_meta;
  int nseg;
};
cudaError_t launch_rotary(const RotaryView& r, const PlaceView& place, const RotaryRows& a, int f16, int sms, int* status,
                          cudaStream_t st);

// New rows k (rotated), v into the cache as launch_cache_append does it, and q.x[0] rotated into q.y[0] (q.H[0] heads;
// 0: none). Positions not given are the rows' places in the cache.
cudaError_t launch_cache_append_rotary(const CacheView& c, const SeqView& s, const RotaryView& r, const PlaceView& place,
                                       const void* k, int64_t k_ss, int64_t k_sh, const void* v, int64_t v_ss,
                                       int64_t v_sh, const RotaryRows& q, int f16, int sms, int* status, cudaStream_t st);

}  // namespace psf
