// cache_prompt.cuh -- attention of prompt chunks over the 8-bit paged cache (sm_103a).
//
//   out_i = sum_j p_ij V_j,  p_ij = exp(z_ij - lse_i),  z_ij = scale q_i . K_j (capped)
//
// What bounds it: with many query rows every cached byte is used hundreds of
// times, so the tensor cores do (2 (Dqk + Dv) flop per pair), and the codes have
// to reach them as 16-bit operands. One CTA per SM takes 256 rows of a KV head's
// queries (its G query heads together, token-major) over 128 keys at a time, in
// two halves of 128 rows with a score tile and an accumulator each in tensor memory:
//   S_X = Q_X K^T  ->  softmax  ->  O_X += P_X V
// so that one half's softmax runs beside the other half's products, and the
// expansion of a key tile serves 256 rows. The halves' products take turns.
// Measured: two chunks of 2048 tokens over 32 Ki keys (32 / 8 heads of 128) 1.70 ms,
// 1255 TF/s, 0.67 of a large product's rate; two windowed prompts of 8001 at 192/128 552 us. A tile's 32 products fill the tensor pipe
// for 2048 cycles (64 each, timed alone) of some 4000 that the tile takes: each half
// goes round scores - softmax - P V, with the issue slots half full, and the softmax's
// loop is faster the fewer registers and instructions it has (two threads a row, 88
// registers each; 2.10 ms without the turns, 1.90 with what the loop no longer keeps).
// Scores of one chunk begin 13 K cycles after the kernel (schedule, table, codes).
//
//   warps 0, 2     MMA issuers of half A (and TMEM allocator) and half B
//   warp 1         which rows and tiles come next, where their pages are, scales
//   warps 4-11     softmax of half A, two threads a row; 12-19 of half B
//   warps 20-23, 24-27  expansion of K, of V: codes from global memory, a tile ahead
//                  in registers, to fp16 tiles in shared memory (128-byte swizzle)
//
// Numbers: codes are exact in fp16, queries are scaled by a power of two per row
// into fp16's range (exact for what lies within 28 octaves of the row's largest).
// Scores, sums and O are fp32. The scale of a K page multiplies the scores of its
// 16-key blocks; that of a V page goes into P, which is rounded to fp16 and kept
// below 2^15 by a reference of its own, set so that the row's largest is 2^3 and
// moved when one would pass 2^15; the row sum has a reference without it. P is off
// by 2^-11 of itself or 2^-28 (half of fp16's last step, 2^-25, over 2^3) of the
// row's largest. (bf16 would round P 8 times as coarsely.)
//
// Work: (KV head, sequence, 256-row tile) units in that order, a unit's key tiles
// in a row; each CTA takes an equal run of all of them, so one chunk over a long
// cache fills the device as a batch does. What a run cuts is left as a partial
// result (o / l, lse) and joined in the order of the runs by the kernel after it.
// Nothing depends on the order of execution.
#pragma once

#include "cache.cuh"
#include "cache_attn.cuh"
#include "launch_prompt.h"

namespace psf {

constexpr int kPpRows = 256;    // query rows of a unit
constexpr int kPpKeys = 128;    // keys of a tile
constexpr int kPpThreads = 896;
constexpr int kPpUnits = 3;     // units announced and not yet done with
constexpr int kPpDescs = 8;     // tiles described ahead (and still read by the softmax)
// References of a row's probabilities: with the V scales (P is at most 2^kPpTop of it, 2^kPpHead when it is set) and
// without (the row sum's, at most 2^kPpLazyM below a score). A move costs a pass over O. With 2^3 it takes 12 octaves to
// cause one; with 2^7, 8 octaves, and 16 mixed prompts take 3 % longer, where P would go on 4 octaves further down.
constexpr float kPpHead = 3.f, kPpTop = 15.f, kPpLazyM = 24.f, kPpNone = kPpLazyM + 26.f;
constexpr int kPpSnap = 8;      // places from a unit's end that a share's is moved to it
constexpr int kPpUnitCost = 4;  // of a unit, in half-tiles: queries in, last product and result out

template <int DQK, int DV>
struct PpCfg {
  static constexpr int QCH = DQK / 64, VCH = DV / 64;  // 64-column chunks
  static constexpr int K_BYTES = QCH * kChunkBytes, V_BYTES = VCH * kChunkBytes;
  static constexpr int NK = DQK == 64 ? 4 : DQK == 128 ? 2 : 1, NV = DQK == 64 ? 4 : 2;  // tiles in shared memory
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = 2 * K_BYTES;
  static constexpr int V_OFF = K_OFF + NK * K_BYTES;
  static constexpr int STG_COLS = 16;  // columns of a result staged at a time, per warp
  static constexpr int STG_BYTES = 32 * STG_COLS * 2;
  static constexpr int STG_OFF = V_OFF + NV * V_BYTES;
  static constexpr bool SERIES = DQK != 192;  // caps of small scores by a series (see the softmax)
  static constexpr bool STAGED = DQK != 192;  // else there is no room, and rows are written as they lie
  static constexpr int SMEM = STG_OFF + (STAGED ? 16 * STG_BYTES : 0) + 1024;
  static constexpr int T_S = 0;    // half X's scores at 128 X; P over columns 0-31 and 64-95 of them
  static constexpr int T_O = 256;  // accumulators at [256, 256 + DV) and [384, 384 + DV)
  // Registers of a thread after the split: 4 softmax warpgroups, K, V, the rest; 7 * 72 in all (launched with 72 each).
  static constexpr int R_SOFT = DQK == 192 ? 80 : 88, R_K = DQK == 192 ? 72 : 48, R_V = DQK == 192 ? 56 : 48, R_REST = 56;
  static_assert(4 * R_SOFT + R_K + R_V + R_REST <= 7 * 72, "registers of the block");
  static_assert(NV + 4 <= kPpDescs, "tiles described ahead");
};

struct PpUnit {
  int b, h, n, m, q0;  // b < 0: no more units
  int r0, rows;        // rows of the (sequence, head), token-major, from r0
  int t0, nt;          // key tiles of this share
  int lo, hi;          // keys that some row sees
  int in_lo, in_hi;    // keys that every row sees
  int slot;            // -1: the share holds all key tiles; else the partial result's place: 1 begins here, 0 continues
  int ends;            // the unit's last tile is in this share
};

// Row tile rt of a sequence: its rows, the keys they see and the tiles of those.
struct PpTiles {
  int r0, rows, lo, hi, t0, kt;
};
__device__ __forceinline__ PpTiles pp_tiles(const PromptParams& p, int n, int m, int rt) {
  PpTiles t;
  t.r0 = rt * kPpRows;
  t.rows = min(kPpRows, m * p.a.G - t.r0);
  const int i0 = ca_token(p.a, t.r0), i1 = ca_token(p.a, t.r0 + t.rows - 1);
  int unused;
  ca_row_keys(p.a, n, m, i0, t.lo, unused);
  ca_row_keys(p.a, n, m, i1, unused, t.hi);
  t.lo = min(t.lo, t.hi);  // (a row that sees nothing has hi = lo)
  if (p.a.window <= 0) t.lo = 0;
  t.t0 = t.lo / kPpKeys;
  t.kt = t.hi > t.lo ? (t.hi + kPpKeys - 1) / kPpKeys - t.t0 : 0;
  return t;
}
// Half-tiles that a key tile costs: half B is idle where there are no rows for it.
__device__ __forceinline__ int pp_weight(int rows) { return rows > kPpRows / 2 ? 2 : 1; }
__device__ __forceinline__ int pp_cost(const PpTiles& t) { return kPpUnitCost + pp_weight(t.rows) * t.kt; }
// Row tiles of up to 2^31 - 1 rows (rounding up by a sum passes 32 bits in the last 255 of them).
__host__ __device__ constexpr int pp_tiles_of(int rows) { return rows / kPpRows + (rows % kPpRows != 0); }
static_assert(pp_tiles_of(0) == 0 && pp_tiles_of(1) == 1 && pp_tiles_of(256) == 1 && pp_tiles_of(257) == 2 &&
              pp_tiles_of(0x7fffffff) == 1 << 23, "row tiles");
__device__ __forceinline__ int pp_row_tiles(const PromptParams& p, const Seq& q) { return pp_tiles_of(q.m * p.a.G); }

// By a whole warp: the cost of one head's units of sequence first + lane (0 past `last`).
__device__ __forceinline__ int64_t pp_costs(const PromptParams& p, int first, int last, bool record) {
  const int lane = threadIdx.x & 31, b = first + lane;
  Seq q = {0, 0, 0, false};
  if (b < last) q = seq_at(p.a.s, p.a.c.page, b);
  if (record && q.bad) record_status(p.a.status, kStatusDeviceArgs);
  const int rt = pp_row_tiles(p, q);
  int64_t mine = 0;
  if (rt > 0) mine = pp_cost(pp_tiles(p, q.n, q.m, 0));
  for (uint32_t more = __ballot_sync(0xffffffffu, rt > 1); more; more &= more - 1) {
    const int from = __ffs(more) - 1;
    const int n = __shfl_sync(0xffffffffu, q.n, from), m = __shfl_sync(0xffffffffu, q.m, from);
    const int tiles = __shfl_sync(0xffffffffu, rt, from);
    int64_t sum = 0;
    for (int i = 1 + lane; i < tiles; i += 32) sum += pp_cost(pp_tiles(p, n, m, i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == from) mine += sum;
  }
  return mine;
}

// Where a run of places begins: head, sequence, row tile and how far into its places.
struct PpStart {
  int h, b, rt, off;
  int64_t places;  // of the run; 0: none
};
__device__ __forceinline__ int64_t warp_inclusive(int64_t x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if ((int)(threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

// The walk over a share's units, by a whole warp.
struct PpWalk {
  int64_t left;
  int h, b, rt, off, tiles;
  Seq q;
  __device__ __forceinline__ void start(const PromptParams& p, const PpStart& s) {
    left = s.places;
    h = s.h;
    b = s.b;
    rt = s.rt;
    off = s.off;
    q = seq_at(p.a.s, p.a.c.page, b);
    tiles = pp_row_tiles(p, q);
  }
  // The next unit with tiles (or with rows and no keys at all) of this share.
  __device__ __forceinline__ bool next(const PromptParams& p, PpUnit& u) {
    while (left > 0) {
      if (rt >= tiles) {
        rt = 0;
        if (++b >= p.a.s.B) {
          b = 0;
          if (++h >= p.a.c.Hkv) return false;
        }
        q = seq_at(p.a.s, p.a.c.page, b);
        tiles = pp_row_tiles(p, q);
        continue;
      }
      const PpTiles t = pp_tiles(p, q.n, q.m, rt);
      const int w = pp_weight(t.rows), cost = pp_cost(t);
      int stop = (int)min((int64_t)cost, off + left);
      if (stop < cost) {
        if (cost - stop <= kPpSnap) {
          stop = cost;
          left = stop - off;
        } else if (stop <= kPpSnap) {
          return false;
        }
      }
      // A tile belongs to the share that its first place lies in.
      const int k0 = max(off - kPpUnitCost + w - 1, 0) / w, k1 = max(stop - kPpUnitCost + w - 1, 0) / w;
      const bool begins = off == 0;
      left -= stop - off;
      off = 0;
      ++rt;
      if (t.kt > 0 ? k1 <= k0 : !begins) continue;
      u.b = b;
      u.h = h;
      u.n = q.n;
      u.m = q.m;
      u.q0 = q.q0;
      u.r0 = t.r0;
      u.rows = t.rows;
      u.t0 = t.t0 + k0;
      u.nt = t.kt > 0 ? k1 - k0 : 0;
      u.lo = t.lo;
      u.hi = t.hi;
      int lo, hi;
      ca_row_keys(p.a, q.n, q.m, ca_token(p.a, t.r0), lo, hi);
      u.in_hi = hi;
      ca_row_keys(p.a, q.n, q.m, ca_token(p.a, t.r0 + t.rows - 1), lo, hi);
      u.in_lo = lo;
      u.slot = k0 == 0 && k1 >= t.kt ? -1 : k0 == 0 ? 1 : 0;
      u.ends = k1 >= t.kt;
      return true;
    }
    return false;
  }
};

// Whether this is the lane of a converged warp that issues for it (always the same one).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}
// The thread's number, read anew.
__device__ __forceinline__ int thread_now() {
  int t;
  asm volatile("mov.u32 %0, %tid.x;" : "=r"(t));
  return t;
}
template <int V>
struct VecTag {
  static constexpr int value = V;
};
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }

// Four codes as fp16.
__device__ __forceinline__ void pp_expand4(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
// Sixteen codes as fp16 (two 16-byte granules).
__device__ __forceinline__ void pp_expand(const uint4& x, uint4& a, uint4& b) {
  pp_expand4(x.x, a.x, a.y);
  pp_expand4(x.y, a.z, a.w);
  pp_expand4(x.z, b.x, b.y);
  pp_expand4(x.w, b.z, b.w);
}
// 0x80 in every byte of x that is a NaN code.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t without_nan(uint32_t x) { return x & ~((nan_bytes(x) >> 7) * 0xffu); }

// CAP: logits softcapped (p.a.softcap > 0). SPAN: keys that share their scales, 16 or 64 (pages of 64 and more).
template <int DQK, int DV, bool CAP, int SPAN>
__global__ void __launch_bounds__(kPpThreads, 1) cache_prompt_kernel(const __grid_constant__ PromptParams p) {
  using C = PpCfg<DQK, DV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t q_full[2], k_full[C::NK], k_empty[C::NK], v_full[C::NV], v_empty[C::NV];
  __shared__ uint64_t s_full[2], p_full[2], pv_done[2], o_free[2], drain[2], turn[2];
  __shared__ uint64_t unit_full[kPpUnits], unit_empty[kPpUnits], desc_full[kPpDescs], desc_empty[kPpDescs];
  __shared__ PpUnit unit_at[kPpUnits];
  // Of the 16-key blocks of a tile: offsets of their first rows' codes (< 0: no row sees any), scales.
  __shared__ int64_t desc_k[kPpDescs][8], desc_v[kPpDescs][8];
  __shared__ __align__(16) float2 desc_scale[kPpDescs][8];  // K scale and log2 of the V scale
  __shared__ uint32_t desc_nan[kPpDescs][4];             // keys that some row sees with NaN codes in V (edge tiles)
  __shared__ float2 row_top[2][2][kPpRows];              // what the two threads of a row tell each other, by the tile's parity
  __shared__ int2 row_keys[2][kPpRows];                  // keys that a row sees, by the unit's parity
  __shared__ float row_fac[kPpRows];                     // query scale times the logit scale
  __shared__ PpStart begin_at;
  __shared__ uint32_t tmem_base_smem;
  __shared__ int abort_flag;

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < C::NK; ++i) {
      mbar_init(&k_full[i], 4);
      mbar_init(&k_empty[i], 2);  // both MMA issuers
    }
    for (int i = 0; i < C::NV; ++i) {
      mbar_init(&v_full[i], 4);
      mbar_init(&v_empty[i], 2);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 8);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 8);
      mbar_init(&pv_done[x], 1);
      mbar_init(&drain[x], 1);
      mbar_init(&turn[x], 1);
      mbar_init(&o_free[x], 8);
    }
    for (int i = 0; i < kPpUnits; ++i) {
      mbar_init(&unit_full[i], 1);
      mbar_init(&unit_empty[i], 26);  // softmax and expansion warps, the MMA issuers
    }
    for (int i = 0; i < kPpDescs; ++i) {
      mbar_init(&desc_full[i], 1);
      mbar_init(&desc_empty[i], 4);  // the V warps
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  // Nothing above touches memory that the kernel before this one may still write.
  after_previous_kernel();
  let_next_kernel_start();

  // The places of all units, and where this share begins. One warp counts them, 32 sequences at a time, and then looks for
  // the place (its code is short: what every warp runs once costs more to fetch than to run).
  if (warp == 0) {
    tmem_alloc(&tmem_base_smem, 512);
    tmem_relinquish();
  } else if (warp == 1) {
    if (lane == 0 && blockIdx.x == 0 && cu_bad(p.a.s)) record_status(p.a.status, kStatusDeviceArgs);
    int64_t cost = 0, at = 0, rem = 0, places = 0;
    int h = 0, b = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      at = 0;
#pragma unroll 1
      for (b = 0; b < p.a.s.B; b += 32) {
        if (pass == 0 || p.a.s.B > 32) cost = pp_costs(p, b, p.a.s.B, pass == 0 && blockIdx.x == 0);
        const int64_t end = at + warp_inclusive(cost);
        const uint32_t past = __ballot_sync(0xffffffffu, pass == 1 && end > rem);
        if (past) {
          at = __shfl_sync(0xffffffffu, end - cost, __ffs(past) - 1);
          b += __ffs(past) - 1;
          break;
        }
        at = __shfl_sync(0xffffffffu, end, 31);
      }
      if (pass == 0) {
        const int64_t total = at * p.a.c.Hkv;
        const int parts = (int)min(quotient(total + p.a.min_share - 1, p.a.min_share), (int64_t)gridDim.x);
        if ((int)blockIdx.x >= parts) break;
        const CaShares shares(total, parts);
        const int64_t pos = shares.first(blockIdx.x);
        places = shares.first(blockIdx.x + 1) - pos;
        h = (int)quotient(pos, at);
        rem = pos - at * h;
      }
    }
    if (places == 0) {
      if (lane == 0) {
        begin_at.places = 0;
        p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
      }
    } else {
      const Seq q = seq_at(p.a.s, p.a.c.page, b);
      const int tiles = pp_row_tiles(p, q);
#pragma unroll 1
      for (int r = 0; r < tiles; r += 32) {
        const int mine = r + lane < tiles ? pp_cost(pp_tiles(p, q.n, q.m, r + lane)) : 0;
        const int64_t to = at + warp_inclusive(mine);
        const uint32_t in = __ballot_sync(0xffffffffu, to > rem);
        if (in) {
          if (lane == __ffs(in) - 1) {
            PpStart start = {h, b, r + lane, (int)(rem - (to - mine)), places};
            // A cut next to a unit's end, or its beginning, is moved there: both shares see it so.
            if (start.off > 0 && mine - start.off <= kPpSnap) {
              start.places -= mine - start.off;
              start.off = 0;
              ++start.rt;
            } else if (start.off <= kPpSnap) {
              start.places += start.off;
              start.off = 0;
            }
            begin_at = start;
            if (start.places <= 0) p.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
          }
          break;
        }
        at = __shfl_sync(0xffffffffu, to, 31);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_smem;
  if (begin_at.places <= 0) {
    if (warp == 0) tmem_dealloc(tmem, 512);
    return;
  }
  const Ctl ctl{p.a.status, p.a.limit_ns, &abort_flag};

  uint32_t nunit = 0;  // units that this role has seen

  if (warp < 4) {
    setmaxnreg_dec<C::R_REST>();
    if (warp == 1) {
      // ---------------------------------------------------------- what comes next
      PpWalk walk;
      walk.start(p, begin_at);
      int4 join = make_int4(0, 0, 0, 0);  // 1: a unit begins here and goes on (head, sequence, row tile); 2: one that continues ends here
      uint32_t it = 0;
      bool ok = true;
      while (ok) {
        PpUnit u;
        const bool more = walk.next(p, u);
        if (!more) u.b = -1;
        if (more && u.nt == 0) {
          // Rows without keys are written here: the other warps get units with tiles alone. (The expansion looks for the
          // next unit in the middle of one; a run of empty ones would fill the ring in front of it.)
          for (int e = lane; e < u.rows * (DV / 8); e += 32) {
            const int r = e / (DV / 8), col = e - r * (DV / 8), z = u.r0 + r, i = ca_token(p.a, z), hq = u.h * p.a.G + z - i * p.a.G;
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.out) + p.a.o_ss * (u.q0 + i) + p.a.o_sh * hq + col * 8) =
                make_uint4(0, 0, 0, 0);
            if (col == 0) p.a.lse[(int64_t)hq * p.a.s.T + u.q0 + i] = -CUDART_INF_F;
          }
          continue;
        }
        if (more && u.slot == 0 && u.ends) join.x |= 2;
        if (more && u.slot == 1) join = make_int4(join.x | 1, u.h, u.b, u.r0 / kPpRows);
        const int us = nunit % kPpUnits;
        if (!wait_bar_warp(&unit_empty[us], ((nunit / kPpUnits) & 1) ^ 1, ctl)) break;
        if (lane == 0) {
          unit_at[us] = u;
          mbar_arrive(&unit_full[us]);
        }
        ++nunit;
        if (!more) break;
        // Four tiles at a time, a 16-key block per lane.
        for (int t = 0; t < u.nt && ok; t += 4) {
          const int mine = t + (lane >> 3), key = (u.t0 + mine) * kPpKeys + (lane & 7) * 16;
          int64_t k_off = -1, v_off = -1;
          float2 sc = make_float2(0.f, 1.f);
          // (All blocks of SPAN keys of which some row sees one: they share the first block's scales.)
          if (mine < u.nt && (key & -SPAN) < u.hi && (key & -SPAN) + SPAN > u.lo) {
            int pg = p.a.s.table[(int64_t)u.b * p.a.s.max_pages + (key >> p.a.c.page_lg)];
            if (pg < 0 || pg >= p.a.c.pages) {
              record_status(p.a.status, kStatusDeviceArgs);
              pg = 0;
            }
            const int64_t at = (int64_t)pg * p.a.c.Hkv + u.h;
            sc = make_float2(p.a.c.k_scale[at], p.a.c.v_scale[at]);
            const int row = key & (p.a.c.page - 1);
            k_off = p.a.c.k_sp * pg + p.a.c.k_sh * u.h + p.a.c.k_sr * row;
            v_off = p.a.c.v_sp * pg + p.a.c.v_sh * u.h + p.a.c.v_sr * row;
          }
          for (int i = 0; i < 4 && t + i < u.nt; ++i) {
            const int ds = it % kPpDescs;
            if (!wait_bar_warp(&desc_empty[ds], ((it / kPpDescs) & 1) ^ 1, ctl)) {
              ok = false;
              break;
            }
            if ((lane >> 3) == i) {
              desc_k[ds][lane & 7] = k_off;
              desc_v[ds][lane & 7] = v_off;
              desc_scale[ds][lane & 7] = make_float2(sc.x, log2f(sc.y));
              if ((lane & 7) < 4) desc_nan[ds][lane & 7] = 0;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&desc_full[ds]);
            ++it;
          }
        }
      }
      if (lane == 0) p.joins[blockIdx.x] = join;
    } else if (warp != 3) {
      // ---------------------------------------------------------- MMA issuer of a half
      // The warp stays together and what it computes with is the same in all lanes, in a way that the compiler sees (votes
      // and broadcasts): descriptors are then made in the uniform registers that the products take them from. One lane issues.
      constexpr uint32_t id_qk = idesc_f32acc<__half>(128, 128, 0, 0);
      constexpr uint32_t id_pv = idesc_f32acc<__half>(128, DV, 0, 1);
      auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
      auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_bar_warp(bar, parity, ctl); };
      const int x = same(warp >> 1);
      const uint32_t tm = same(tmem), t_s = tm + C::T_S + x * 128, t_o = tm + C::T_O + x * 128;
      const uint64_t q_d = sdesc_sw128(smem_u32(smem + C::Q_OFF) + x * C::K_BYTES, 16, 1024);
      const uint64_t k_d = sdesc_sw128(smem_u32(smem + C::K_OFF), 16, 1024);
      const uint64_t v_d = sdesc_sw128(smem_u32(smem + C::V_OFF), kChunkBytes, 1024);
      uint32_t it = 0, un = 0, up = 0, ks = 0, kp = 0, vs = 0, vp = 0, kv = 0, nhalf = 0;  // slots and phases; counts
      bool ok = true;
      // The halves' products take turns, a tile's P V and the next scores at a time: left to themselves they come at the same
      // moments, each takes twice as long, and the softmaxes that wait for them then run at the same moments, too.
      uint32_t nturn = 0;
      auto my_turn = [&] {
        ++nturn;
        return wait(&turn[x], (nturn & 1) ^ x);
      };
      auto pass_turn = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(&turn[x ^ 1]);
      };
      auto scores = [&] {
        const uint64_t b = k_d + (uint64_t)(ks * (C::K_BYTES >> 4));
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < C::QCH; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss(t_s, q_d + (c * kChunkBytes + kk * 32) / 16, b + (c * kChunkBytes + kk * 32) / 16, id_qk, (c | kk) != 0);
          mma_commit(&s_full[x]);
          mma_commit(&k_empty[ks]);
        }
        if (++ks == C::NK) {
          ks = 0;
          kp ^= 1;
        }
      };
      while (ok) {
        if (!wait(&unit_full[un], up)) break;
        const volatile PpUnit& u = unit_at[un];
        const int nt = same(u.nt);
        const bool none = same(u.b) < 0, idle = x == 1 && same(u.rows) <= kPpRows / 2;
        const bool edge = same(u.t0 * kPpKeys < u.in_lo || (u.t0 + 1) * kPpKeys > u.in_hi) != 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&unit_empty[un]);
        if (++un == kPpUnits) {
          un = 0;
          up ^= 1;
        }
        if (none) break;
        if ((!idle && !wait(&q_full[x], nhalf & 1)) || !wait(&k_full[ks], kp) || !my_turn()) break;
        tc_fence_after();
        if (idle) {  // half B has no rows: its shares of the releases, as the tiles come
          pass_turn();
          for (int jj = 0; jj < nt && ok; ++jj, ++it) {
            if (!wait(&k_full[ks], kp) || !wait(&v_full[vs], vp)) {
              ok = false;
              break;
            }
            __syncwarp();
            if (lane == 0) {  // (before the turn: half A waits for the tile that comes into this one's place)
              mbar_arrive(&k_empty[ks]);
              mbar_arrive(&v_empty[vs]);
            }
            if (!my_turn()) {
              ok = false;
              break;
            }
            pass_turn();
            if (++ks == C::NK) {
              ks = 0;
              kp ^= 1;
            }
            if (++vs == C::NV) {
              vs = 0;
              vp ^= 1;
            }
          }
          continue;
        }
        scores();
        pass_turn();
#pragma unroll 1
        for (int jj = 0; jj < nt; ++jj, ++it) {
          const bool more = jj + 1 < nt;
          if (!wait(&v_full[vs], vp) || (jj == 0 && nhalf > 0 && !wait(&o_free[x], (nhalf - 1) & 1)) ||
              (more && !wait(&k_full[ks], kp))) {
            ok = false;
            break;
          }
          uint32_t kept = jj > 0;
          if (!kept && edge) {
            const uint32_t* nan = desc_nan[it % kPpDescs];
            kept = same((nan[0] | nan[1] | nan[2] | nan[3]) != 0);
          }
          const uint64_t b = v_d + (uint64_t)(vs * (C::V_BYTES >> 4));
          if (!wait(&p_full[x], kv & 1) || !my_turn()) {
            ok = false;
            break;
          }
          ++kv;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(t_o, t_s + (kk >> 2) * 64 + (kk & 3) * 8, b + kk * 128, id_pv, kk > 0 ? 1 : kept);
            mma_commit(&v_empty[vs]);
            if (!more) mma_commit(&pv_done[x]);
          }
          if (++vs == C::NV) {
            vs = 0;
            vp ^= 1;
          }
          if (more) scores();
          pass_turn();
        }
        ++nhalf;
      }
      // Wind down: wait until every MMA this thread issued has finished.
      if (elect_one()) mma_commit(&drain[x]);
      wait_bar_drain(&drain[x], 0, p.a.limit_ns);
    }
  } else if (warp >= 20) {
    // ------------------------------------------------------------ expansion
    const int ew = warp - 20;
    auto ready = [&](uint64_t* bar) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // V 16-code vectors of a tile per thread: row 8 (4 (i / CH) + w) + lane / 4 of warp w, vector lane % 4 of chunk i % CH
    // (64 components). Eight lanes that write together then have two rows, whose swizzles keep them out of each other's banks.
    auto expand = [&](auto vecs_tag, const bool is_v) {
      constexpr int V = decltype(vecs_tag)::value, CH = V / 4;
      const int w = ew & 3, rr = lane >> 2, vq = lane & 3;
      const uint8_t* base =
          (is_v ? p.a.c.v : p.a.c.k) + (is_v ? p.a.c.v_sr : p.a.c.k_sr) * ((w & 1) * 8 + rr) + vq * 16;
      const int64_t (*descs)[8] = is_v ? desc_v : desc_k;
      uint64_t* full = is_v ? v_full : k_full;
      uint64_t* empty = is_v ? v_empty : k_empty;
      uint8_t* tiles = smem + (is_v ? C::V_OFF : C::K_OFF) + (w * 8 + rr) * 128 + (((2 * vq) ^ rr) << 4);
      const int second = ((2 * vq) ^ rr) & 1 ? -16 : 16;  // from a vector's first granule to its second
      const uint32_t depth = is_v ? C::NV : C::NK, bytes = is_v ? C::V_BYTES : C::K_BYTES;
      uint4 x[V];
      uint32_t it = 0, slot = 0, phase = 1;
      bool ok = true;
      // A unit is read from shared memory whenever it is needed, and given back when the one after it is begun. -1: none left.
      auto take_unit = [&]() -> int {
        const int us = nunit % kPpUnits;
        if (!wait_bar_warp(&unit_full[us], (nunit / kPpUnits) & 1, ctl) || unit_at[us].b < 0) return -1;
        ++nunit;
        return us;
      };
      auto load = [&](uint32_t j) -> bool {  // the codes of the j-th tile of this CTA
        if (!wait_bar_warp(&desc_full[j % kPpDescs], (j / kPpDescs) & 1, ctl)) return false;
        const int64_t* at = descs[j % kPpDescs] + (w >> 1);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int64_t off = at[2 * g];
          const uint8_t* row = base + off;
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            x[g * CH + c] = make_uint4(0, 0, 0, 0);
            if (off >= 0) x[g * CH + c] = *reinterpret_cast<const uint4*>(row + c * 64);
          }
        }
        return true;
      };
      int us = take_unit();
      if (us >= 0) ok = load(0);
      while (us >= 0 && ok) {
        const volatile PpUnit& u = unit_at[us];
        int after = -1;
        const int nt = u.nt;
#pragma unroll 1
        for (int jj = 0; jj < nt; ++jj, ++it) {
          if (!wait_bar_warp(&empty[slot], phase, ctl)) {
            ok = false;
            break;
          }
          if (is_v) {
            // Every product with the tile NV back is done, and so is its softmax.
            if (it >= C::NV && lane == 0) mbar_arrive(&desc_empty[(it - C::NV) % kPpDescs]);
            const int key0 = (u.t0 + jj) * kPpKeys;
            if (key0 < u.in_lo || key0 + kPpKeys > u.in_hi) {
              // A row's probability is 0 for a key that it does not see, which keeps out any code but NaN. NaN codes
              // (stale ones may be) become 0 here; the softmax puts one in for the rows that see it.
#pragma unroll
              for (int i = 0; i < V; ++i)
                if (nan_bytes(x[i].x) | nan_bytes(x[i].y) | nan_bytes(x[i].z) | nan_bytes(x[i].w)) {
                  const int r = (i / CH) * 32 + w * 8 + rr;
                  x[i] = make_uint4(without_nan(x[i].x), without_nan(x[i].y), without_nan(x[i].z), without_nan(x[i].w));
                  if (key0 + r >= u.lo && key0 + r < u.hi) atomicOr(&desc_nan[it % kPpDescs][r >> 5], 1u << (r & 31));
                }
            }
          }
          uint8_t* to = tiles + slot * bytes;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            uint4 a, b;
            pp_expand(x[i], a, b);
            uint8_t* at = to + (i % CH) * kChunkBytes + (i / CH) * 4096;
            *reinterpret_cast<uint4*>(at) = a;
            *reinterpret_cast<uint4*>(at + second) = b;
          }
          ready(&full[slot]);
          if (++slot == depth) {
            slot = 0;
            phase ^= 1;
          }
          // The tile after it (of the next unit, too) on its way.
          const bool more = jj + 1 < nt;
          if (!more) after = take_unit();
          if (more || after >= 0) {
            if (!load(it + 1)) {
              ok = false;
              break;
            }
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&unit_empty[us]);
        us = after;
      }
    };
    if (ew < 4) {
      if constexpr (C::R_K != 72) setmaxnreg_dec<C::R_K>();  // (what it was launched with)
    } else {
      setmaxnreg_dec<C::R_V>();
    }
    // (The same code for both where they have one size: it has to be fetched, too.)
    if constexpr (DQK == DV) {
      expand(VecTag<DQK / 16>(), ew >= 4);
    } else {
      if (ew < 4)
        expand(VecTag<DQK / 16>(), false);
      else
        expand(VecTag<DV / 16>(), true);
    }
  } else {
    // ------------------------------------------------------------ softmax of a half
    setmaxnreg_inc<C::R_SOFT>();
    // Warps 4-7 and 8-11 have half A, 12-15 and 16-19 half B; two threads share a row, the first has keys 0-63 of a tile (and
    // columns 0 to DV / 2 - 1 of O), the second the others. P lies over the first half of a thread's own scores.
    const int sw = warp - 4, x = sw >> 3, y = (sw >> 2) & 1, row = x * 128 + (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lane_base + C::T_S + x * 128 + y * 64, to = tmem + lane_base + C::T_O + x * 128 + y * (DV / 2);
    const float2 zero2 = make_float2(0.f, 0.f);
    auto pair_sync = [&] { asm volatile("bar.sync %0, 64;" ::"r"(1 + x * 4 + (warp & 3)) : "memory"); };
    uint32_t it = 0, kv = 0, nhalf = 0;
    bool ok = true;
    // Capped logits in log2 units, cap2 tanh(a). tanh a = 1 - 2 / (e^(2a) + 1) is off by some 2^-22 however small a is:
    // 2^-16 of a logit for caps up to 64. For larger ones ca_tanh, which takes three times the instructions. Where all
    // scores of a warp are below a quarter of the cap, the series of ca_tanh, on the multipliers alone (a chunk of 512 over 32
    // Ki keys under a cap of 30: 353 us, 12 % less; 16 mixed prompts 632, 5 % less, but 4 % more under a cap of 5). With 192
    // key components the registers it takes cost more than it saves (4 % of a windowed prompt). The vote makes a score's last
    // bits depend on those beside it in the tile.
    const float cap2 = p.a.softcap * 1.4426950408889634f;
    const bool cap_near = p.a.softcap <= 64.f;
    // A warp's 16 rows of a unit's queries, 8 lanes a row and four rows at a time: into registers, and to shared memory as
    // fp16 scaled by a power of two per row.
    constexpr int QV = DQK / 64;
    // (What follows from the thread alone is made again where it is needed: kept, it would take registers from the scores.)
    auto q_row_of = [&](int t) { return x * 128 + ((t >> 5) & 3) * 32 + y * 16 + ((t & 31) >> 3); };
    uint4 qx[4][QV];
    auto load_q = [&](const volatile PpUnit& u) {
      const int rows = u.rows, r0 = u.r0, q0 = u.q0, h = u.h, t = thread_now(), q_row = q_row_of(t), l8 = t & 7;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = q_row + 4 * k, z = r0 + r, i = ca_token(p.a, z);
        const uint16_t* from = static_cast<const uint16_t*>(p.a.q) + p.a.q_ss * (q0 + i) + p.a.q_sh * (h * p.a.G + z - i * p.a.G) +
                               l8 * 8;
#pragma unroll
        for (int c = 0; c < QV; ++c) {
          qx[k][c] = make_uint4(0, 0, 0, 0);
          if (r < rows) qx[k][c] = *reinterpret_cast<const uint4*>(from + c * 64);
        }
      }
    };
    auto store_as = [&](auto type) {
      using T = decltype(type);
      const int t = thread_now(), q_row = q_row_of(t), l8 = t & 7;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = q_row + 4 * k;
        uint32_t most = 0;  // largest patterns without sign, of the low and of the high halves
#pragma unroll
        for (int c = 0; c < QV; ++c)
          most = __vmaxu2(most, __vmaxu2(__vmaxu2(qx[k][c].x & 0x7fff7fffu, qx[k][c].y & 0x7fff7fffu),
                                         __vmaxu2(qx[k][c].z & 0x7fff7fffu, qx[k][c].w & 0x7fff7fffu)));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, o));
        const float2 ends = unpack2<T>(most);
        const float top = fmaxf(ends.x, ends.y);
        const int field = min(268 - (__float_as_int(top) >> 23), 253);  // 2^14 <= top * 2^(field - 127) < 2^15
        const float up = __int_as_float(field << 23), down = __int_as_float((254 - field) << 23);
        uint8_t* at = smem + C::Q_OFF + x * C::K_BYTES + sw128_offset(r & 127, l8);
#pragma unroll
        for (int c = 0; c < QV; ++c) {
          const uint32_t w[4] = {qx[k][c].x, qx[k][c].y, qx[k][c].z, qx[k][c].w};
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = mul2(unpack2<T>(w[e]), make_float2(up, up));
            h[e] = pack2<__half>(f.x, f.y);
          }
          *reinterpret_cast<uint4*>(at + c * kChunkBytes) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        if (l8 == 0) row_fac[r] = down * (CAP ? p.a.scale / p.a.softcap : p.a.scale * 1.4426950408889634f);
      }
    };
    auto store_q = [&] {
      if (p.a.f16)
        store_as(__half());
      else
        store_as(__nv_bfloat16());
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[x]);
    };
    auto idle_in = [&](const volatile PpUnit& u) { return x == 1 && u.rows <= kPpRows / 2; };
    bool have_q = false;
    // The unit is read from shared memory whenever it is needed: the scores fill the registers.
    for (; ok; ++nunit) {
      const int us = nunit % kPpUnits;
      // (Both threads of a row go on or neither does: they meet at a barrier.)
      auto both = [&](bool mine) -> bool {
        uint32_t r;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %1, 0;\n\t"
            "barrier.cta.red.and.pred q, %2, 64, p;\n\t"
            "selp.u32 %0, 1, 0, q;\n\t}"
            : "=r"(r)
            : "r"((uint32_t)mine), "r"(1 + x * 4 + (warp & 3))
            : "memory");
        return r != 0;
      };
      if (!both(wait_bar(&unit_full[us], (nunit / kPpUnits) & 1, ctl))) break;
      const volatile PpUnit& u = unit_at[us];
      if (u.b < 0) break;
      auto done = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(&unit_empty[us]);
      };
      const bool valid = row < u.rows;
      // Element offset of this thread's row in out, and its place in lse.
      auto out_at = [&](int64_t& lse_at) -> int64_t {
        const int z = u.r0 + (valid ? row : 0), i = ca_token(p.a, z), hq = u.h * p.a.G + z - i * p.a.G;
        lse_at = (int64_t)hq * p.a.s.T + u.q0 + i;
        return p.a.o_ss * (u.q0 + i) + p.a.o_sh * hq;
      };
      if (idle_in(u)) {
        it += u.nt;
        done();
        continue;
      }
      if (!have_q) {
        load_q(u);
        store_q();
      }
      have_q = false;
      if (y == 0) {
        int key_lo = 0, key_hi = 0x7fffffff;
        if (valid) ca_row_keys(p.a, u.n, u.m, ca_token(p.a, u.r0 + row), key_lo, key_hi);
        row_keys[nunit & 1][row] = make_int2(key_lo, key_hi);
      }
      pair_sync();
      float fac = 0.f, m = kCaFloor, ro = kCaFloor, l = 0.f;
      const int nt = u.nt;
#pragma unroll 1
      for (int jj = 0; jj < nt; ++jj, ++it) {
        const int c0 = (u.t0 + jj) * kPpKeys + y * 64;
        const bool edge = c0 - y * 64 < u.in_lo || c0 - y * 64 + kPpKeys > u.in_hi;
        // Of this thread's 64 keys it sees [lo_c, hi_c).
        int lo_c = 0, hi_c = 64;
        if (edge) {
          const int2 keys = row_keys[nunit & 1][row];
          lo_c = keys.x - c0;
          hi_c = min(keys.y - c0, 64);
        }
        const bool masked = edge && __any_sync(0xffffffffu, lo_c > 0 || hi_c < 64);
        const bool up = wait_bar(&s_full[x], kv & 1, ctl);
        tc_fence_after();
        if (jj == 0) fac = row_fac[row];
        const float2* sc = desc_scale[it % kPpDescs] + y * 4;
        // The factor of a block's 16 scores: not 0, so that -inf stays -inf (2^-100 of any score is next to 0).
        auto factor = [&](float k_scale) { return CAP ? 1.f : fmaxf(fac * k_scale, 0x1p-100f); };
        float mx = -CUDART_INF_F, yx = -CUDART_INF_F;  // largest score, and largest with what the V scale adds
        uint32_t s[32];
        // Scores c .. c + 31: capped, masked (and put back where they are read again), their largest.
        auto look = [&](int c) {
          tmem_ld32(ts + c, s);
          if constexpr (CAP && C::SERIES) {
            float most = 0.f;  // largest magnitude of a = score / cap
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float k1 = fac * sc[(c + e) / SPAN * (SPAN / 16)].x;
              const float2 a = mul2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), make_float2(k1, k1));
              most = fmax3(most, fabsf(a.x), fabsf(a.y));
              s[e] = __float_as_uint(a.x);
              s[e + 1] = __float_as_uint(a.y);
            }
            if (__all_sync(0xffffffffu, most < 0.25f)) {
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float2 a = make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), b = mul2(a, a);
                float2 t = fma2(b, make_float2(62.f / 2835.f, 62.f / 2835.f), make_float2(-17.f / 315.f, -17.f / 315.f));
                t = fma2(b, t, make_float2(2.f / 15.f, 2.f / 15.f));
                t = fma2(b, t, make_float2(-1.f / 3.f, -1.f / 3.f));
                t = fma2(b, t, make_float2(1.f, 1.f));
                t = mul2(mul2(a, make_float2(cap2, cap2)), t);
                s[e] = __float_as_uint(t.x);
                s[e + 1] = __float_as_uint(t.y);
              }
            } else if (cap_near) {
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float2 t = mul2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])),
                                      make_float2(2.8853900817779268f, 2.8853900817779268f));
                const float2 d = add2(make_float2(ex2_approx(t.x), ex2_approx(t.y)), make_float2(1.f, 1.f));
                const float2 z = fma2(make_float2(rcp_approx(d.x), rcp_approx(d.y)), make_float2(-2.f * cap2, -2.f * cap2),
                                      make_float2(cap2, cap2));
                s[e] = __float_as_uint(z.x);
                s[e + 1] = __float_as_uint(z.y);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) s[e] = __float_as_uint(cap2 * ca_tanh(__uint_as_float(s[e])));
            }
          } else if constexpr (CAP) {
            if (cap_near) {
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float k1 = 2.f * 1.4426950408889634f * fac * sc[(c + e) / SPAN * (SPAN / 16)].x;
                const float2 t = mul2(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), make_float2(k1, k1));
                const float2 d = add2(make_float2(ex2_approx(t.x), ex2_approx(t.y)), make_float2(1.f, 1.f));
                const float2 z = fma2(make_float2(rcp_approx(d.x), rcp_approx(d.y)), make_float2(-2.f * cap2, -2.f * cap2),
                                      make_float2(cap2, cap2));
                s[e] = __float_as_uint(z.x);
                s[e + 1] = __float_as_uint(z.y);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                s[e] = __float_as_uint(cap2 * ca_tanh(__uint_as_float(s[e]) * (fac * sc[(c + e) / SPAN * (SPAN / 16)].x)));
            }
          }
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c + e < lo_c || c + e >= hi_c) s[e] = 0xff800000u;  // -inf
          }
          if ((CAP || masked) && c > 0) tmem_st32(ts + c, s);
#pragma unroll
          for (int k = 0; k < 32; k += 16) {
            float a[5];
#pragma unroll
            for (int e = 0; e < 5; ++e)
              a[e] = fmax3(__uint_as_float(s[k + 3 * e]), __uint_as_float(s[k + 3 * e + 1]), __uint_as_float(s[k + 3 * e + 2]));
            const float t = fmaxf(fmax3(a[0], a[1], a[2]), fmax3(a[3], a[4], __uint_as_float(s[k + 15])));
            if constexpr (SPAN == 16) {
              const float2 sv = sc[(c + k) >> 4];
              const float z = t * factor(sv.x);
              mx = fmaxf(mx, z);
              yx = fmaxf(yx, z + sv.y);
            } else {
              mx = fmaxf(mx, t);
            }
          }
        };
        look(32);
        look(0);
        const float2 sc0 = sc[0];
        const float f64 = factor(sc0.x);
        if constexpr (SPAN == 64) {
          mx *= f64;
          yx = mx + sc0.y;
        }
        row_top[kv & 1][y][row] = make_float2(mx, yx);
        if (!both(up)) {
          ok = false;
          break;
        }
        {
          const float2 other = row_top[kv & 1][y ^ 1][row];
          mx = fmaxf(mx, other.x);
          yx = fmaxf(yx, other.y);
        }
        ++kv;
        const float m_new = mx > m + kPpLazyM ? mx : m, ro_new = yx > ro + kPpTop ? yx - kPpHead : ro;
        const float alpha = m_new == m ? 1.f : ex2_approx(m - m_new), beta = ro_new == ro ? 1.f : ex2_approx(ro - ro_new);
        // P = 2^(score + log2 of the V scale - ro), over the scores' first columns. A block's part of the row sum is that
        // without the V scale: its sum times 2^(ro - m - log2 of the V scale). Where that is above 2^kPpNone, P is below
        // 2^-26 (scores are at most kPpLazyM above m) and 0 in fp16; with the exponent held there it stays 0, and the row
        // sum in range.
        float rs = 0.f;
        float2 sum[2] = {zero2, zero2};
        float base = fmaxf(sc0.y - ro_new, -kPpNone - m_new);
        float2 f2 = make_float2(f64, f64), b2 = make_float2(base, base);
        auto add_up = [&] {
          const float2 all = add2(sum[0], sum[1]);
          rs = fmaf(all.x + all.y, ex2_approx(-m_new - base), rs);
          sum[0] = sum[1] = zero2;
        };
        auto weigh = [&](int c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            if (SPAN == 16 && (e & 7) == 0 && c + e > 0) {
              add_up();
              const float2 sv = sc[(c + 2 * e) >> 4];
              const float f = factor(sv.x);
              base = fmaxf(sv.y - ro_new, -kPpNone - m_new);
              f2 = make_float2(f, f);
              b2 = make_float2(base, base);
            }
            const float2 z = fma2(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), f2, b2);
            const float2 ex = make_float2(ex2_approx(z.x), ex2_approx(z.y));
            sum[e & 1] = add2(sum[e & 1], ex);
            pk[e] = pack2<__half>(ex.x, ex.y);
          }
          tmem_st16_async(ts + (c >> 1), pk);
        };
        weigh(0);
        tmem_ld32(ts + 32, s);
        weigh(32);
        add_up();
        uint32_t nan = 0;
        if (edge) {
          if (!both(wait_bar(&v_full[it % C::NV], (it / C::NV) & 1, ctl))) {
            ok = false;
            break;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) nan |= desc_nan[it % kPpDescs][k];
        }
        tmem_wait_st();
        if (nan != 0 || (jj > 0 && __any_sync(0xffffffffu, beta != 1.f))) {
          // O (this thread's columns) moved to the new reference: it holds the products up to the tile before, which the
          // commit of the scores covers.
#pragma unroll 1
          for (int c = 0; c < DV / 2; c += 16) {
            uint32_t r[16];
            tmem_ld16(to + c, r);
            // (0 on a unit's first tile, whose product then adds to it.)
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = jj == 0 ? 0u : __float_as_uint(__uint_as_float(r[e]) * beta);
            if (nan != 0) {  // NaN where a NaN code is seen
#pragma unroll 1
              for (int key = 0; key < kPpKeys; ++key) {
                if (!(desc_nan[it % kPpDescs][key >> 5] >> (key & 31) & 1)) continue;
                const uint4 q = *reinterpret_cast<const uint4*>(p.a.c.v + desc_v[it % kPpDescs][key >> 4] +
                                                                p.a.c.v_sr * (key & 15) + y * (DV / 2) + c);
                const uint32_t codes[4] = {q.x, q.y, q.z, q.w};
                const bool sees = key - y * 64 >= lo_c && key + c0 - y * 64 < row_keys[nunit & 1][row].y;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (sees && (nan_bytes(codes[e >> 2]) >> (8 * (e & 3) + 7) & 1)) r[e] = 0x7fffffffu;
              }
            }
            tmem_st16(to + c, r);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
        l = l * alpha + rs;
        m = m_new;
        ro = ro_new;
      }
      if (!ok) break;
      // The next unit's queries, whose place is free once the last scores are made: on their way while the last product is,
      // in place before this unit's results are written.
      {
        const int next = (nunit + 1) % kPpUnits;
        if (!both(wait_bar(&unit_full[next], ((nunit + 1) / kPpUnits) & 1, ctl))) break;
        have_q = unit_at[next].b >= 0 && !idle_in(unit_at[next]);
        if (have_q) load_q(unit_at[next]);
      }
      // The row's sum, in the order of the threads.
      row_top[kv & 1][y][row].x = l;
      if (!both(wait_bar(&pv_done[x], nhalf & 1, ctl))) break;
      ++nhalf;
      l = row_top[kv & 1][0][row].x + row_top[kv & 1][1][row].x;
      pair_sync();
      tc_fence_after();
      if (have_q) store_q();
      // out = O 2^(ro - m) / l, the power in two steps: V scales may be as small as fp32 goes.
      const float half_up = ex2_approx(0.5f * (ro - m)), inv = l == 0.f ? 0.f : half_up / l;
      const float lg = l == 0.f ? -CUDART_INF_F : m + log2f(l);
      int64_t lse_at;
      const int64_t o_at = out_at(lse_at);
      if (u.slot < 0) {
        constexpr int G16 = C::STG_COLS / 8;  // 16-byte granules of a staged row
        uint8_t* stg = smem + C::STG_OFF + ((thread_now() >> 5) - 4) * C::STG_BYTES;
#pragma unroll 1
        for (int c = 0; c < DV / 2 / C::STG_COLS; ++c) {
          uint32_t r[C::STG_COLS], pk[C::STG_COLS / 2];
          tmem_ld_cols(to + c * C::STG_COLS, r);
#pragma unroll
          for (int e = 0; e < C::STG_COLS / 2; ++e) {
            const float lo = __uint_as_float(r[2 * e]) * half_up * inv, hi = __uint_as_float(r[2 * e + 1]) * half_up * inv;
            pk[e] = p.a.f16 ? pack2<__half>(lo, hi) : pack2<__nv_bfloat16>(lo, hi);
          }
          if constexpr (!C::STAGED) {
            if (valid) {
              uint4* at = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.out) + o_at + y * (DV / 2) + c * C::STG_COLS);
#pragma unroll
              for (int q = 0; q < G16; ++q) at[q] = make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
            }
            continue;
          }
          __syncwarp();
#pragma unroll
          for (int q = 0; q < G16; ++q)
            *reinterpret_cast<uint4*>(stg + lane * (G16 * 16) + ((q ^ (G16 == 4 ? (lane >> 1) & 3 : (lane >> 2) & 1)) << 4)) =
                make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < G16; ++k) {
            const int rr = k * (32 / G16) + lane / G16, q = lane % G16;
            const int64_t at = __shfl_sync(0xffffffffu, o_at, rr);
            const bool live = __shfl_sync(0xffffffffu, (int)valid, rr);
            const uint4 t = *reinterpret_cast<const uint4*>(
                stg + rr * (G16 * 16) + ((q ^ (G16 == 4 ? (rr >> 1) & 3 : (rr >> 2) & 1)) << 4));
            if (live) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.out) + at + y * (DV / 2) + c * C::STG_COLS + q * 8) = t;
          }
        }
        if (valid && y == 0) p.a.lse[lse_at] = lg * 0.69314718055994531f;
      } else {
        // Partial results lie as [column / 4][row]: a warp writes 512 bytes in a row.
        const int64_t slot = (int64_t)blockIdx.x * 2 + u.slot;
        float4* part = reinterpret_cast<float4*>(p.a.part_o) + (slot * (DV / 4) + y * (DV / 8)) * kPpRows + row;
#pragma unroll 1
        for (int c = 0; c < DV / 2; c += 16) {
          uint32_t r[16];
          tmem_ld16(to + c, r);
          if (valid) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              part[(c / 4 + q) * kPpRows] = make_float4(
                  __uint_as_float(r[4 * q]) * half_up * inv, __uint_as_float(r[4 * q + 1]) * half_up * inv,
                  __uint_as_float(r[4 * q + 2]) * half_up * inv, __uint_as_float(r[4 * q + 3]) * half_up * inv);
          }
        }
        if (valid && y == 0) p.a.part_l[slot * kPpRows + row] = lg;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[x]);
      done();
    }
    tmem_wait_st();  // (a wait that ran out can come between a store and its own)
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partial results of the unit that begins in share blockIdx.x and goes
// on in the next ones, in the order of the shares: 32 of its rows per CTA
// (blockIdx.y). The last row of CTAs writes the rows past the last sequence.
constexpr int kPpJoinRows = 32;
constexpr int kPpJoinThreads = 256;
template <int DV>
__global__ void __launch_bounds__(kPpJoinThreads) cache_prompt_join_kernel(const __grid_constant__ PromptParams p, int grid) {
  constexpr int VEC = DV / 4, COLS = kPpJoinThreads / 32;  // columns of four at a time
  __shared__ __align__(16) float stage[kPpJoinRows][DV + 4];
  static_assert(__alignof__(stage) >= alignof(float4) && (DV + 4) % 4 == 0, "rows are written by fours");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_next_kernel_start();
  after_previous_kernel();
  if (blockIdx.y == kPpRows / kPpJoinRows) {
    int first = p.a.s.cu ? min(max(p.a.s.cu[p.a.s.B], 0), p.a.s.T) : p.a.s.T;
    if (first >= p.a.s.T) return;
    // Prefix sums that fall can end in front of rows that a sequence has: those are its own.
    __shared__ int ends;
    if (tid == 0) ends = first;
    __syncthreads();
    for (int b = tid; b < p.a.s.B; b += kPpJoinThreads) {
      const Seq q = seq_at(p.a.s, p.a.c.page, b);
      if (q.m > 0) first = max(first, q.q0 + q.m);
    }
    atomicMax(&ends, first);
    __syncthreads();
    const int Hq = p.a.c.Hkv * p.a.G;
    const int64_t rest = (int64_t)(p.a.s.T - ends) * Hq * (DV / 8);
    for (int64_t e = (int64_t)blockIdx.x * kPpJoinThreads + tid; e < rest; e += (int64_t)gridDim.x * kPpJoinThreads) {
      const int64_t rh = e / (DV / 8);
      const int col = (int)(e - rh * (DV / 8)), t = ends + (int)(rh / Hq), h = (int)(rh % Hq);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.out) + p.a.o_ss * t + p.a.o_sh * h + col * 8) =
          make_uint4(0, 0, 0, 0);
      if (col == 0) p.a.lse[(int64_t)h * p.a.s.T + t] = -CUDART_INF_F;
    }
    return;
  }
  const int4 join = p.joins[blockIdx.x];
  if (!(join.x & 1)) return;
  const int h = join.y, at0 = blockIdx.y * kPpJoinRows;
  const Seq q = seq_at(p.a.s, p.a.c.page, join.z);
  const int n0 = join.w * kPpRows + at0, live = min(kPpJoinRows, q.m * p.a.G - n0);
  if (live <= 0) return;
  __shared__ int parts;
  if (tid == 0) {
    int c = blockIdx.x + 1;
    while (c < grid && !(p.joins[c].x & 2)) ++c;
    parts = min(c, grid - 1) - (int)blockIdx.x + 1;
  }
  __syncthreads();
  const int np = parts, r = min(lane, live - 1);
  auto slot_at = [&](int i) -> int64_t { return (int64_t)(blockIdx.x + i) * 2 + (i == 0); };
  float top = kCaFloor, sum = 0.f;
  for (int i = 0; i < np; ++i) top = fmaxf(top, p.a.part_l[slot_at(i) * kPpRows + at0 + r]);
  for (int i = 0; i < np; ++i) sum += ex2_approx(p.a.part_l[slot_at(i) * kPpRows + at0 + r] - top);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int v = warp; v < VEC; v += COLS) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < np; ++i) {
      const float w = ex2_approx(p.a.part_l[slot_at(i) * kPpRows + at0 + r] - top) * inv;
      const float4 a = reinterpret_cast<const float4*>(p.a.part_o)[(slot_at(i) * VEC + v) * kPpRows + at0 + r];
      acc.x = fmaf(a.x, w, acc.x);
      acc.y = fmaf(a.y, w, acc.y);
      acc.z = fmaf(a.z, w, acc.z);
      acc.w = fmaf(a.w, w, acc.w);
    }
    *reinterpret_cast<float4*>(&stage[lane][v * 4]) = acc;
  }
  __syncthreads();
  for (int e = tid; e < live * (DV / 8); e += kPpJoinThreads) {
    const int rr = e / (DV / 8), col = (e - rr * (DV / 8)) * 8, z = n0 + rr, i = ca_token(p.a, z);
    const float* s = &stage[rr][col];
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = p.a.f16 ? pack2<__half>(s[2 * k], s[2 * k + 1]) : pack2<__nv_bfloat16>(s[2 * k], s[2 * k + 1]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.a.out) + p.a.o_ss * (q.q0 + i) +
                              p.a.o_sh * (h * p.a.G + z - i * p.a.G) + col) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (warp == 0 && lane < live) {
    const int z = n0 + lane, i = ca_token(p.a, z);
    p.a.lse[(int64_t)(h * p.a.G + z - i * p.a.G) * p.a.s.T + q.q0 + i] =
        sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * 0.69314718055994531f;
  }
}

}  // namespace psf
