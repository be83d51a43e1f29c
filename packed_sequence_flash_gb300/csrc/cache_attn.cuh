// cache_attn.cuh -- attention of a few query rows per sequence over the 8-bit
// paged cache (sm_103a).
//
//   out_i = sum_j p_ij V_j,  p_ij = exp(z_ij - lse_i),  z_ij = scale q_i . K_j (capped)
//
// What bounds it: every key and value byte is read once per group of query
// heads and used for 8 or 16 rows, 2 flop per byte and row, so the kernel is a
// stream of the cache: the floor is bytes / HBM bandwidth. A 128-row tensor
// tile (tcgen05) would be nearly empty and would need the codes as 16-bit
// operands in shared memory, that is every byte expanded and written back
// once; warp-level products take their operands from registers, where the
// codes are expanded in place, so that instruction is the fitting one.
// Measured (bf16, head dim 128, 32 query and 8 KV heads; GB300): 64 sequences of
// 16 to 32 Ki tokens 480 us for 3.27 GB, the rate of a plain copy; 32 of 64 to
// 8192 tokens 59.4 us for 307 MB (floor 45.2: 5 us until the first tile, 4 us of
// join and some 4 us in which the CTAs end); one of 32 Ki tokens 22 us (floor
// 9.9); one of 777 tokens with 16 / 4 heads 10 us, all latency; 1024 of 10 to 200
// tokens 102 us (floor 35: every unit runs through all of the code once, and
// fetching it is what limits there). Out of L2 a tile of
// 64 keys takes an SM 515 cycles for 8 rows and 790 for 16 (the expansion, two
// cycles of the integer pipe for two codes, is most of it); from memory 690.
//
// Rows: the query rows of one KV head (m rows x G heads, token-major) in tiles
// of R = 8 NT rows: 8 where a KV head has no more, else 16. Keys: tiles of 64. A
// CTA takes an equal share of all (sequence, KV head, row tile, key tile) in
// that order, wherever it begins and ends, so ragged batches and a single long
// sequence alike fill the device. A share that covers all tiles of a (sequence,
// head, row tile) writes its result; otherwise it leaves a partial result (o / l,
// lse) that the join kernel adds up in the order of the CTAs. Nothing depends on
// the order of execution.
//
//   warp 4     producer: the next unit and its queries ahead of time, page
//              numbers and scales one batch ahead, K and V pages by TMA into a
//              ring of stages (128-byte rows, 128-byte swizzle; 64-byte rows
//              for head dim 64)
//   warps 0-3  16 keys of each tile each, with a softmax state of their own
//              (nothing but the ring's barriers between them); joined at the
//              end of the unit
//
// S^T = K Q^T: 16 keys are the rows of the product, 8 query rows its columns,
// so a group of up to 8 heads wastes nothing. The order in which the head dim
// is contracted is free, so a lane reads 16 consecutive codes of its two key
// rows and its Q operand is arranged to match. O^T += V^T P^T likewise: a lane
// reads 16 consecutive codes of four keys, pairs up keys with byte permutes,
// and owns those 16 head-dim rows of O^T. P^T is S^T's accumulator transposed
// in registers (movmatrix). The map from a position in the product to a key
// row is chosen so that neither kind of read has a bank conflict under the swizzle.
//
// Numbers: codes are exact in fp16. Q rows are scaled by a power of two into
// fp16's range (exact for what matters: 28 octaves below the row's largest).
// Scores, sums and O are fp32. P enters the product with V in fp16, scaled to at
// most 2^15 by a reference that includes the block's V scale, so that blocks of
// very different scales stay in range; the row sum has a reference without it.
// Both references move only when a score exceeds them by 2^8, which a warp vote
// finds. bf16 would round P 8 times as coarsely for no gain in range.
#pragma once

#include "cache.cuh"
#include "launch_cache.h"

namespace psf {

constexpr int kCaKeys = 64;       // keys per tile
constexpr int kCaWarps = 4;       // consumer warps, 16 keys of a tile each
constexpr int kCaConsumers = 32 * kCaWarps;
constexpr int kCaThreads = kCaConsumers + 32;
constexpr int kCaUnits = 3;       // units under way: finishing, current, next
constexpr float kCaLazy = 8.f;    // a reference moves when a score is 2^8 above it
constexpr float kCaHead = 7.f;    // the P reference sits 2^7 below the largest value
constexpr float kCaFloor = -3e38f;  // references before the first score (finite: no inf - inf)

template <int DQK, int DV, int NT>
struct CaCfg {
  static constexpr int R = 8 * NT;
  static constexpr int KP = DQK <= 128 ? 1 : (DQK + 127) / 128;  // 128-byte planes of a K row
  static constexpr int VP = DV <= 128 ? 1 : (DV + 127) / 128;
  static constexpr int ROWB = DQK == 64 ? 64 : 128;  // bytes of a row in a plane
  static constexpr int PLANE = kCaKeys * ROWB;
  static constexpr int STAGE = (KP + VP) * PLANE;
  static constexpr int CTAS = cache_attn_ctas(DQK, NT);
  static constexpr int RAW = R * DQK * 2;        // queries as they come, one of kCaUnits buffers
  static constexpr int QPITCH = DQK + 8;         // fp16 elements of a query row
  static constexpr int OPITCH = DV + 4;          // fp32 elements
  static constexpr int OBYTES = kCaWarps * R * OPITCH * 4;
  static constexpr int FIXED = kCaUnits * RAW + OBYTES + 1024;
  // As many stages as fit beside 2 KB of static and 1 KB of reserved shared
  // memory: 64 KB or more of the cache in flight per SM.
  static constexpr int FIT = (233472 / CTAS - 3 * 1024 - FIXED) / STAGE;
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int RAW_OFF = STAGES * STAGE;
  static constexpr int O_OFF = RAW_OFF + kCaUnits * RAW;
  static constexpr int Q_OFF = O_OFF;  // the queries are done with before O is written
  static constexpr int SMEM = STAGES * STAGE + FIXED;
  static_assert(STAGES >= 2 && CTAS * STAGES * STAGE >= 64 * 1024, "bytes in flight");
  static_assert(R * QPITCH * 2 <= OBYTES, "queries fit where O goes");
};

// a / b, in 32 bits when both fit (most of the time).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// Share of the work. A unit is a (sequence, head, row tile); it costs its key
// tiles and kCaUnit more (queries in, four warps' states into one, result out),
// laid out as kCaUnit places and then a place per tile. Each CTA takes an equal
// run of the places of the units in order. Without the unit's cost a
// share of many short sequences took five times as long as one of a long one
// (16 sequences of 5 to 4099 tokens: 148 us).
constexpr int kCaUnit = 6;
struct CaSeq {
  Seq q;
  int rt, kt, t0;  // row tiles, key tiles, first key tile
  __device__ __forceinline__ int cost() const { return kt + kCaUnit; }
  __device__ __forceinline__ int64_t places(int Hkv) const { return kt ? (int64_t)Hkv * rt * cost() : 0; }
};
template <typename P>  // CacheAttnParams or what ca_seq needs of it
__device__ __forceinline__ CaSeq ca_seq(const P& p, int b) {
  CaSeq s;
  s.q = seq_at(p.s, p.c.page, b);
  const int lo = p.window > 0 ? max(0, s.q.n - s.q.m - p.window + 1) : 0;
  s.t0 = lo / kCaKeys;
  s.kt = s.q.m > 0 ? max(0, (s.q.n + kCaKeys - 1) / kCaKeys - s.t0) : 0;
  s.rt = (s.q.m * p.G + (1 << p.tile_lg) - 1) >> p.tile_lg;
  return s;
}
// CTAs that share `total` places, and how they do.
__device__ __forceinline__ int ca_parts(int64_t total, int grid, int min_share) {
  const int64_t most = (total + min_share - 1) / min_share;
  return (int)(most < grid ? most : grid);
}
struct CaShares {
  int64_t each, more;  // the first `more` CTAs take each + 1 places, the others each
  __device__ __forceinline__ CaShares(int64_t total, int parts) {
    each = parts ? quotient(total, parts) : 0;
    more = total - each * parts;
  }
  __device__ __forceinline__ int64_t first(int c) const { return each * c + min((int64_t)c, more); }
  // The CTA that place x belongs to.
  __device__ __forceinline__ int owner(int64_t x) const {
    const int64_t cut = more * (each + 1);
    return (int)(x < cut ? quotient(x, each + 1) : more + quotient(x - cut, each));
  }
};

// x / G for a row x of the tile order (token-major), 0 <= x < 2^31, G's reciprocal rounded up to 33 bits: exact.
__device__ __forceinline__ int ca_token(const CacheAttnParams& p, int x) {
  return (int)((__umulhi((uint32_t)x, p.g_mul) + (uint32_t)x) >> p.g_shift);
}

// tanh(a). 1 - 2 / (e^(2a) + 1) is off by some 2^-22 however small a is, so alone
// it drowns logits far below the cap (a cap of 10^6 made an lse of 7 wrong by 0.04).
// Below 1/4 its Taylor series up to a^9: the next term is 2^-26 of the value, the
// rest fp32's roundings. From there on 2^-22 is at most 2^-20 of the value.
__device__ __forceinline__ float ca_tanh(float a) {
  const float b = a * a;
  const float series = fmaf(fmaf(fmaf(fmaf(62.f / 2835.f, b, -17.f / 315.f), b, 2.f / 15.f), b, -1.f / 3.f), b, 1.f) * a;
  const float whole = fmaf(-2.f, rcp_approx(ex2_approx(a * 2.8853900817779268f) + 1.f), 1.f);
  return fabsf(a) < 0.25f ? series : whole;
}

// Keys [lo, hi) that row i of m sees of n cached tokens (the last row sits at the last token).
__device__ __forceinline__ void ca_row_keys(const CacheAttnParams& p, int n, int m, int i, int& lo, int& hi) {
  const int at = i + n - m;
  hi = p.causal ? min(n, at + 1) : n;
  lo = p.window > 0 ? max(0, at - p.window + 1) : 0;
  if (hi < lo) hi = lo;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint4 lds128(const uint8_t* a) { return *reinterpret_cast<const uint4*>(a); }
__device__ __forceinline__ uint2 lds64(const uint8_t* a) { return *reinterpret_cast<const uint2*>(a); }
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// Whether x holds for all consumer threads.
__device__ __forceinline__ bool consumers_all(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
// Contiguous copy of `bytes` (a multiple of 16) into shared memory, counted on bar.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// By all threads of a block: the places of all sequences, and those before and in
// this thread's run of `per` neighbouring sequences. A run's loads do not wait
// for one another; with a scan per THREADS sequences, 4096 of them took 45 us.
struct CaCount {
  int64_t total, before, mine;
  int first, per;
};
// (Calls of their own, with the parameters in registers: as part of the kernels
// these loops made one sequence of 777 keys 0.5 us slower, which takes neither.)
struct CaFew {
  SeqView s;
  struct {
    int page, Hkv;
  } c;
  int window, G, tile_lg;
  __device__ __forceinline__ explicit CaFew(const CacheAttnParams& p)
      : s(p.s), c{p.c.page, p.c.Hkv}, window(p.window), G(p.G), tile_lg(p.tile_lg) {}
};
__device__ __noinline__ int64_t ca_run_places(const CacheAttnParams& params, int first, int per, bool record) {
  const CaFew p(params);
  int64_t n = 0;
  bool bad = false;
#pragma unroll 8
  for (int i = 0; i < per; ++i)
    if (first + i < p.s.B) {
      const CaSeq s = ca_seq(p, first + i);
      bad |= s.q.bad;
      n += s.places(p.c.Hkv);
    }
  if (record && bad) record_status(params.status, kStatusDeviceArgs);
  return n;
}
// The sequence of a run that place `pos` lies in; *base: the places before the run, and then those before the sequence.
__device__ __noinline__ int ca_run_find(const CacheAttnParams& params, int first, int per, int64_t pos, int64_t* base) {
  const CaFew p(params);
  int b = first;
  int64_t end = *base, at = end;
#pragma unroll 8
  for (int i = 0; i < per; ++i) {
    const int x = min(first + i, p.s.B - 1);  // (more than once the last: `end` is above `pos` by then)
    end += ca_seq(p, x).places(p.c.Hkv);
    if (end <= pos) {
      b = x + 1;
      at = end;
    }
  }
  *base = at;
  return b;
}
template <int THREADS>
__device__ __forceinline__ CaCount ca_count(const CacheAttnParams& p, int64_t* scan, bool record) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  CaCount r = {0, 0, 0, tid, 1};
  if (p.s.B <= THREADS) {
    if (tid < p.s.B) {
      const CaSeq s = ca_seq(p, tid);
      if (record && s.q.bad) record_status(p.status, kStatusDeviceArgs);
      r.mine = s.places(p.c.Hkv);
    }
  } else {
    r.per = (p.s.B + THREADS - 1) / THREADS;
    r.first = tid * r.per;
    r.mine = ca_run_places(p, r.first, r.per, record);
  }
  int64_t x = r.mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scan[warp] = x;
  __syncthreads();
  r.before = x - r.mine;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) r.before += scan[w];
    r.total += scan[w];
  }
  return r;
}
// The sequence that place `pos` (< total) lies in, and the places before it, for all threads of the block.
__device__ __forceinline__ void ca_locate(const CacheAttnParams& p, const CaCount& count, int64_t pos, int* found_b,
                                          int64_t* found_base) {
  if (pos >= count.before && pos < count.before + count.mine) {
    int64_t base = count.before;
    *found_b = count.per == 1 ? count.first : ca_run_find(p, count.first, count.per, pos, &base);
    *found_base = base;
  }
  __syncthreads();
}

// The same without a search: the places of all sequences, and those before
// sequence `b`, for all threads of the block. (Two sums over the warps; the scan
// above cost the join of one long sequence 0.6 us more.)
template <int THREADS>
__device__ int64_t ca_before(const CacheAttnParams& p, longlong2* sums, int b, int64_t* total) {
  int64_t all = 0, before = 0;
  for (int i = threadIdx.x; i < p.s.B; i += THREADS) {
    const int64_t n = ca_seq(p, i).places(p.c.Hkv);
    all += n;
    before += i < b ? n : 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = make_longlong2(all, before);
  __syncthreads();
  all = before = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    all += sums[w].x;
    before += sums[w].y;
  }
  *total = all;
  return before;
}

// One unit of a share, and the keys and tiles it concerns.
struct CaUnit {
  int b, h, rt, n, m, q0;
  int t0, t1;        // key tiles of this share
  int whole;         // the share holds all key tiles of the unit
  int slot;          // partial result: 1 = the unit begins in this share, 0 = it continues
  int lo, hi;        // keys that some row of the row tile sees
  int in_lo, in_hi;  // keys that every row sees: tiles inside need no mask
  int ta, tb;        // key tiles of the share with keys in [lo, hi)
  float* scores;     // where the tile's first row keeps its scores
};
struct CaWalk {
  int64_t left;       // places still to come
  int b, h, rt, off;  // the unit they begin in, and how far into it
  CaSeq s;
  __device__ __forceinline__ void start(const CacheAttnParams& p, int64_t pos, int64_t end, int seq, int64_t base) {
    left = end - pos;
    b = seq;
    s = ca_seq(p, b);
    const int64_t x = quotient(pos - base, s.cost());
    off = (int)(pos - base - x * s.cost());
    h = (int)quotient(x, s.rt);
    rt = (int)(x - (int64_t)h * s.rt);
  }
  __device__ __forceinline__ bool next(const CacheAttnParams& p, CaUnit& u) {
    while (left > 0) {
      if (h == p.c.Hkv || s.kt == 0) {
        if (++b >= p.s.B) return false;
        s = ca_seq(p, b);
        h = rt = off = 0;
        continue;
      }
      const int stop = (int)min((int64_t)s.cost(), off + left);
      const int k0 = max(off - kCaUnit, 0), k1 = stop - kCaUnit;
      u.h = h;
      u.rt = rt;
      left -= stop - off;
      off = 0;
      if (++rt == s.rt) {
        rt = 0;
        ++h;
      }
      if (k1 <= k0) continue;  // nothing but the places in front of the tiles
      u.b = b;
      u.n = s.q.n;
      u.m = s.q.m;
      u.q0 = s.q.q0;
      u.t0 = s.t0 + k0;
      u.t1 = s.t0 + k1;
      u.whole = k1 - k0 == s.kt;
      u.slot = k0 == 0;
      const int i0 = ca_token(p, u.rt << p.tile_lg), i1 = ca_token(p, min((u.rt + 1) << p.tile_lg, u.m * p.G) - 1);
      ca_row_keys(p, u.n, u.m, i0, u.lo, u.in_hi);
      ca_row_keys(p, u.n, u.m, i1, u.in_lo, u.hi);
      u.scores = p.scores + (((int64_t)b * p.c.Hkv + u.h) * p.score_rows + (u.rt << p.tile_lg)) * p.score_cap;
      u.ta = max(u.t0, u.lo / kCaKeys);
      u.tb = min(u.t1, (u.hi + kCaKeys - 1) / kCaKeys);
      return true;
    }
    return false;
  }
};

// EXTRA: logits are capped or scores kept (p.softcap, p.accumulate).
template <int DQK, int DV, int NT, bool EXTRA>
__global__ void __launch_bounds__(kCaThreads, CaCfg<DQK, DV, NT>::CTAS)
    cache_attn_kernel(const __grid_constant__ CacheAttnParams p) {
  using C = CaCfg<DQK, DV, NT>;
  constexpr bool QREGS = NT * DQK <= (EXTRA ? 64 : 256);  // Q operand kept in registers
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[C::STAGES], empty[C::STAGES];
  __shared__ float2 meta[C::STAGES][kCaWarps];  // K scale and log2 of the V scale of 16 keys
  __shared__ uint64_t q_full[kCaUnits], q_empty[kCaUnits];
  __shared__ CaUnit unit_at[kCaUnits];  // b < 0: no more units
  __shared__ float row_fac[C::R];  // query scale times the logit scale
  __shared__ int2 row_lim[C::R];   // keys that a row sees
  __shared__ float st_mu[kCaWarps][C::R], st_l[kCaWarps][C::R], fin_l[C::R];
  __shared__ int64_t scan[kCaThreads / 32], found_base;
  __shared__ int found_b, abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kCaWarps);
    }
    for (int i = 0; i < kCaUnits; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], kCaWarps);
    }
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  // Nothing above touches memory that the kernel before this one may still
  // write; the join may start once every CTA is past this point.
  after_previous_kernel();
  let_next_kernel_start();

  // The whole work, and the sequence that this share begins in.
  if (tid == 0 && blockIdx.x == 0 && cu_bad(p.s)) record_status(p.status, kStatusDeviceArgs);
  const CaCount count = ca_count<kCaThreads>(p, scan, blockIdx.x == 0);
  const int parts = ca_parts(count.total, gridDim.x, p.min_share);
  if ((int)blockIdx.x >= parts) return;
  const CaShares shares(count.total, parts);
  const int64_t pos = shares.first(blockIdx.x);
  ca_locate(p, count, pos, &found_b, &found_base);
  const Ctl ctl{p.status, p.limit_ns, &abort_flag};

  if (warp == kCaWarps) {
    // ------------------------------------------------------------ producer
    CaWalk walk;
    walk.start(p, pos, shares.first(blockIdx.x + 1), found_b, found_base);
    const int box_lg = min(p.c.page_lg, 6), box = 1 << box_lg, per_box = box / 16, boxes = kCaKeys >> box_lg;
    uint32_t it = 0, nu = 0;
    bool ok = true;
    // Lane l looks after 16-key slice l of the next eight tiles.
    auto page_at = [&](const CaUnit& u, int tile0) {
      const int key = tile0 * kCaKeys + lane * 16, first = key & -box;
      if (first >= u.hi || first + box <= u.lo || tile0 * 4 + lane >= u.tb * 4) return -1;
      int pg = p.s.table[(int64_t)u.b * p.s.max_pages + (key >> p.c.page_lg)];
      if (pg < 0 || pg >= p.c.pages) {
        record_status(p.status, kStatusDeviceArgs);
        pg = 0;
      }
      return pg;
    };
    auto scales_at = [&](int h, int pg) {
      const int64_t a = (int64_t)pg * p.c.Hkv + h;
      return pg < 0 ? make_float2(0.f, 1.f) : make_float2(p.c.k_scale[a], p.c.v_scale[a]);
    };
    // Hands the next unit to the consumers with its queries, as they are: a row
    // each of the first eight lanes. Without one, tells them so.
    auto announce = [&](bool more, const CaUnit& u) {
      const int qb = nu % kCaUnits;
      if (nu >= kCaUnits && !wait_bar(&q_empty[qb], (nu / kCaUnits - 1) & 1, ctl)) return false;
      const int n0 = u.rt * C::R, rows = more ? min(u.m * p.G - n0, C::R) : 0;
      if (lane == 0) {
        if (more)
          unit_at[qb] = u;
        else
          unit_at[qb].b = -1;
        mbar_arrive_expect_tx(&q_full[qb], (uint32_t)rows * DQK * 2);
      }
      __syncwarp();
      if (lane < rows) {
        const int x = n0 + lane, i = ca_token(p, x), hq = u.h * p.G + (x - i * p.G);
        bulk_load(smem + C::RAW_OFF + qb * C::RAW + lane * DQK * 2,
                  static_cast<const uint16_t*>(p.q) + p.q_ss * (u.q0 + i) + p.q_sh * hq, DQK * 2, &q_full[qb]);
      }
      ++nu;
      return true;
    };
    // The first unit is an empty one, which only looks for the next: the code for
    // that stands here once (instructions are fetched anew for every short unit).
    CaUnit u, next;
    u.b = u.h = u.lo = u.hi = u.ta = u.tb = 0;
    int pg = -1;
    bool more = true;
    while (ok && more) {
      float2 sc = scales_at(u.h, pg);
      int pg_next = page_at(u, u.ta + 8), pg_unit = -1;
      bool first = true;
      for (int t8 = u.ta; ok && (first || t8 < u.tb); t8 += 8) {
        float2 sc_next = make_float2(0.f, 1.f);
        int pg_after = -1;
#pragma unroll 1
        for (int i = 0; i < 8 && (first || t8 + i < u.tb); ++i) {
          if (t8 + i < u.tb) {
            const int st = it % C::STAGES;
            if (it >= C::STAGES && !wait_bar(&empty[st], ((it / C::STAGES) - 1) & 1, ctl)) {
              ok = false;
              break;
            }
            const int key0 = (t8 + i) * kCaKeys;
            uint8_t* dst = smem + st * C::STAGE;
            const int b0 = max(u.lo - key0, 0) >> box_lg, b1 = min((u.hi - key0 + box - 1) >> box_lg, boxes);
            if (lane == 0) mbar_expect_tx(&full[st], (uint32_t)(b1 - b0) * box * C::ROWB * (C::KP + C::VP));
            for (int x = b0; x < b1; ++x) {
              const int use = __shfl_sync(0xffffffffu, pg, i * 4 + x * per_box);
              if (lane == 0) {
                const int row = (key0 + x * box) & (p.c.page - 1);
#pragma unroll
                for (int k = 0; k < C::KP; ++k)
                  tma_load_4d(dst + k * C::PLANE + x * box * C::ROWB, &p.tm_k, &full[st], k * 128, row, u.h, use);
#pragma unroll
                for (int k = 0; k < C::VP; ++k)
                  tma_load_4d(dst + (C::KP + k) * C::PLANE + x * box * C::ROWB, &p.tm_v, &full[st], k * 128, row, u.h,
                              use);
              }
            }
            // The scales are waited for only here, with the codes on their way.
            if ((lane >> 2) == i) meta[st][lane & 3] = make_float2(sc.x, log2f(sc.y));
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
            ++it;
          }
          if (i == 0) {
            sc_next = scales_at(u.h, pg_next);
            pg_after = page_at(u, t8 + 16);
            if (first) {
              // With the first tile out: which unit comes next, its queries and first pages.
              first = false;
              more = walk.next(p, next);
              if (more) pg_unit = page_at(next, next.ta);
              if (!announce(more, next)) ok = false;
            }
          }
        }
        pg = pg_next;
        sc = sc_next;
        pg_next = pg_after;
      }
      u = next;
      pg = pg_unit;
    }
    // The CTA does not end before its copies have landed (the wait has a limit of
    // its own: the consumers may give up and end first).
    {
      const uint64_t limit = p.limit_ns > 100000000ull ? p.limit_ns : 100000000ull;
      for (uint32_t k = it > C::STAGES ? it - C::STAGES : 0; k < it; ++k)
        wait_bar_drain(&full[k % C::STAGES], (k / C::STAGES) & 1, limit);
      for (uint32_t k = nu > kCaUnits ? nu - kCaUnits : 0; k < nu; ++k)
        wait_bar_drain(&q_full[k % kCaUnits], (k / kCaUnits) & 1, limit);
    }
    return;
  }

  // ------------------------------------------------------------ consumers
  const int g = lane >> 2, t = lane & 3;
  // Position in a product -> key row of the warp's 16 (bits 0-2; bit 3 stays).
  auto row_at = [](int x) {
    return DQK == 64 ? ((x & 1) * 3) ^ ((x >> 1) & 1) ^ (x & 4) : ((x & 1) * 5) ^ (x & 2) ^ (x & 4);
  };
  const int ka = warp * 16 + row_at(g);  // key rows of this lane's scores: ka, ka + 8
  const int va = warp * 16 + row_at(2 * t), vb = warp * 16 + row_at(2 * t + 1);  // V rows: va, vb, + 8 each
  float* ob = reinterpret_cast<float*>(smem + C::O_OFF);
  auto k_off = [&](int row, int j) -> uint32_t {
    if (DQK == 64) return row * 64 + ((t ^ ((row >> 1) & 3)) << 4);
    return (j >> 1) * C::PLANE + row * 128 + ((((j & 1) * 4 + t) ^ (row & 7)) << 4);
  };
  auto v_off = [&](int row, int j) -> uint32_t {
    if (DV == 64) return C::PLANE + row * 64 + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8;
    return (C::KP + j) * C::PLANE + row * 128 + ((g ^ (row & 7)) << 4);
  };
  const uint8_t* qs = smem + C::Q_OFF + g * C::QPITCH * 2 + t * 32;  // Q operand: 16 fp16 of each 64
  constexpr int MT = DV / 16;           // products along the head dim of V
  constexpr int VW = DV == 64 ? 2 : 4;  // 4-code words a lane reads of a key row and plane
  int st = 0;         // stage of the ring
  uint32_t ring = 0;  // its phase
  bool ok = true;
  for (uint32_t nu = 0;; ++nu) {
    const int qb = nu % kCaUnits;
    // All warps go on or none does: a wait that ran out in one of them must not
    // leave the others at a barrier.
    if (!consumers_all(wait_bar(&q_full[qb], (nu / kCaUnits) & 1, ctl))) break;
    const CaUnit& u = unit_at[qb];
    if (u.b < 0) break;
    const int rows = u.m * p.G, n0 = u.rt * C::R, lo = u.lo, hi = u.hi;
    // Queries to fp16, each row scaled by a power of two: a warp two rows.
#pragma unroll
    for (int e2 = 0; e2 < 2 * NT; ++e2) {
      constexpr int E = DQK / 32;  // elements per lane and row
      const int r = warp + e2 * kCaWarps;
      const uint32_t* from =
          reinterpret_cast<const uint32_t*>(smem + C::RAW_OFF + qb * C::RAW + r * DQK * 2) + lane * (E / 2);
      float v[E], top = 0.f;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const uint32_t w = n0 + r < rows ? from[e / 2] : 0u;
        const float2 f = p.f16 ? unpack2<__half>(w) : unpack2<__nv_bfloat16>(w);
        v[e] = f.x;
        v[e + 1] = f.y;
        top = fmax3(top, fabsf(f.x), fabsf(f.y));
      }
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const int field = min(268 - (__float_as_int(top) >> 23), 253);  // 2^14 <= top * 2^(field - 127) < 2^15
      const float up = __int_as_float(field << 23), down = __int_as_float((254 - field) << 23);
      uint32_t* to = reinterpret_cast<uint32_t*>(smem + C::Q_OFF + r * C::QPITCH * 2) + lane * (E / 2);
#pragma unroll
      for (int e = 0; e < E; e += 2) to[e / 2] = pack2<__half>(v[e] * up, v[e + 1] * up);
      if (lane == 0) {
        int2 lim = make_int2(0, 0);
        if (n0 + r < rows) ca_row_keys(p, u.n, u.m, ca_token(p, n0 + r), lim.x, lim.y);
        row_lim[r] = lim;
        row_fac[r] = down * (p.softcap > 0.f ? p.scale / p.softcap : p.scale * 1.4426950408889634f);
      }
    }
    consumers_sync();
    uint32_t qf[NT][QREGS ? DQK / 8 : 1];
    if constexpr (QREGS) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < DQK / 64; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint4 a = lds128(qs + nt * 8 * C::QPITCH * 2 + j * 128 + x * 16);
            qf[nt][j * 8 + x * 4] = a.x;
            qf[nt][j * 8 + x * 4 + 1] = a.y;
            qf[nt][j * 8 + x * 4 + 2] = a.z;
            qf[nt][j * 8 + x * 4 + 3] = a.w;
          }
    }
    float fac[NT][2], mu[NT][2], ro[NT][2], l[NT][2];
    float o[MT][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        fac[nt][c] = row_fac[nt * 8 + 2 * t + c];
        mu[nt][c] = ro[nt][c] = kCaFloor;
        l[nt][c] = 0.f;
      }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[m][nt][c] = 0.f;

    auto tile_step = [&](auto mask_tag, int tile) {
      constexpr bool MASK = decltype(mask_tag)::value;
      const uint8_t* sb = smem + st * C::STAGE;
      const int key = tile * kCaKeys + ka;
      float s[NT][4], s2[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[nt][c] = s2[nt][c] = 0.f;
#pragma unroll
      for (int j = 0; j < DQK / 64; ++j) {
        const uint4 xa = lds128(sb + k_off(ka, j)), xb = lds128(sb + k_off(ka + 8, j));
        const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
        uint32_t qv[NT][8];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          if constexpr (QREGS) {
#pragma unroll
            for (int e = 0; e < 8; ++e) qv[nt][e] = qf[nt][j * 8 + e];
          } else {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint4 a = lds128(qs + nt * 8 * C::QPITCH * 2 + j * 128 + x * 16);
              qv[nt][x * 4] = a.x;
              qv[nt][x * 4 + 1] = a.y;
              qv[nt][x * 4 + 2] = a.z;
              qv[nt][x * 4 + 3] = a.w;
            }
          }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t a0 = e4m3_to_half2(wa[w] & 0xffff), a2 = e4m3_to_half2(wa[w] >> 16);
          const uint32_t a1 = e4m3_to_half2(wb[w] & 0xffff), a3 = e4m3_to_half2(wb[w] >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816((w & 1) ? s2[nt] : s[nt], a0, a1, a2, a3, qv[nt][2 * w], qv[nt][2 * w + 1]);
        }
      }
      // Exponents of the row sum's terms (x) and of P (y) against the references:
      // x = z - mu, y = z + log2 v_scale - ro, z the score in log2 units.
      const float2 sc = meta[st][warp];
      float x[NT][4], y[NT][4], f[NT][2];
      bool move = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f[nt][0] = fac[nt][0] * sc.x;
        f[nt][1] = fac[nt][1] * sc.x;
#pragma unroll
        for (int c = 0; c < 4; ++c) s[nt][c] += s2[nt][c];
        if (EXTRA && p.softcap > 0.f) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            s[nt][c] = p.softcap * 1.4426950408889634f * ca_tanh(s[nt][c] * f[nt][c & 1]);
          f[nt][0] = f[nt][1] = 1.f;
        }
        if (EXTRA && p.accumulate) {
          float* at = u.scores + (int64_t)(nt * 8 + 2 * t) * (int)p.score_cap + key;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (n0 + nt * 8 + 2 * t + (c & 1) < rows && key + (c >> 1) * 8 < hi)
              at[(c & 1) * p.score_cap + (c >> 1) * 8] = s[nt][c] * f[nt][c & 1];
        }
        const float dy[2] = {sc.y - ro[nt][0], sc.y - ro[nt][1]};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[nt][c] = fmaf(s[nt][c], f[nt][c & 1], -mu[nt][c & 1]);
          y[nt][c] = fmaf(s[nt][c], f[nt][c & 1], dy[c & 1]);
          if constexpr (MASK) {
            const int2 lim = row_lim[nt * 8 + 2 * t + (c & 1)];
            const int k = key + (c >> 1) * 8;
            if (k < lim.x || k >= lim.y) s[nt][c] = x[nt][c] = y[nt][c] = -CUDART_INF_F;
          }
        }
        move |= fmaxf(fmax3(x[nt][0], x[nt][1], x[nt][2]), x[nt][3]) > kCaLazy ||
                fmaxf(fmax3(y[nt][0], y[nt][1], y[nt][2]), y[nt][3]) > kCaHead + kCaLazy;
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float of[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float z[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
              z[e] = MASK && s[nt][c + 2 * e] == -CUDART_INF_F ? -CUDART_INF_F : s[nt][c + 2 * e] * f[nt][c];
            float top = fmaxf(z[0], z[1]);
#pragma unroll
            for (int e = 4; e < 32; e <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, e));
            const float m1 = fmaxf(mu[nt][c], top), r1 = fmaxf(ro[nt][c], top + sc.y - kCaHead);
            l[nt][c] *= ex2_approx(mu[nt][c] - m1);
            of[c] = ex2_approx(ro[nt][c] - r1);
            mu[nt][c] = m1;
            ro[nt][c] = r1;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              x[nt][c + 2 * e] = z[e] - m1;
              y[nt][c + 2 * e] = z[e] + (sc.y - r1);
            }
          }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[m][nt][c] *= of[c & 1];
        }
      }
      uint32_t p0[NT], p1[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          l[nt][c & 1] += ex2_approx(x[nt][c]);
          w[c] = ex2_approx(y[nt][c]);
        }
        p0[nt] = transpose8x8(pack2<__half>(w[0], w[1]));
        p1[nt] = transpose8x8(pack2<__half>(w[2], w[3]));
      }
      bool nan_seen = false;  // the same for all lanes
#pragma unroll
      for (int j = 0; j < C::VP; ++j) {
        uint32_t v[4][4];
        const int rows4[4] = {va, vb, va + 8, vb + 8};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (DV == 64) {
            const uint2 a = lds64(sb + v_off(rows4[r], j));
            v[r][0] = a.x;
            v[r][1] = a.y;
          } else {
            const uint4 a = lds128(sb + v_off(rows4[r], j));
            v[r][0] = a.x;
            v[r][1] = a.y;
            v[r][2] = a.z;
            v[r][3] = a.w;
          }
        }
        if constexpr (MASK) {
          // A row's probability is 0 for a key that it does not see, which keeps out
          // any code but NaN. NaN codes (stale ones may be) become 0 here; one
          // that some row sees is put in below, for that row alone.
          uint32_t nan = 0;
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < VW; ++e) nan |= (v[r][e] & 0x7f7f7f7fu) + 0x01010101u;
          if (__any_sync(0xffffffffu, nan & 0x80808080u)) {
            uint32_t seen = 0;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int k = tile * kCaKeys + rows4[r];
#pragma unroll
              for (int e = 0; e < VW; ++e) {
                const uint32_t x = ((v[r][e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                if (k >= lo && k < hi) seen |= x;
                v[r][e] &= ~((x >> 7) * 0xffu);
              }
            }
            nan_seen |= __any_sync(0xffffffffu, seen) != 0;
          }
        }
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          const uint32_t y0 = __byte_perm(v[0][e], v[1][e], 0x5140), y1 = __byte_perm(v[0][e], v[1][e], 0x7362);
          const uint32_t z0 = __byte_perm(v[2][e], v[3][e], 0x5140), z1 = __byte_perm(v[2][e], v[3][e], 0x7362);
          const int m = j * 8 + e * 2;
          const uint32_t a0 = e4m3_to_half2(y0 & 0xffff), a1 = e4m3_to_half2(y0 >> 16);
          const uint32_t a2 = e4m3_to_half2(z0 & 0xffff), a3 = e4m3_to_half2(z0 >> 16);
          const uint32_t b0 = e4m3_to_half2(y1 & 0xffff), b1 = e4m3_to_half2(y1 >> 16);
          const uint32_t b2 = e4m3_to_half2(z1 & 0xffff), b3 = e4m3_to_half2(z1 >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(o[m][nt], a0, a1, a2, a3, p0[nt], p1[nt]);
            mma16816(o[m + 1][nt], b0, b1, b2, b3, p0[nt], p1[nt]);
          }
        }
      }
      if constexpr (MASK) {
        if (nan_seen) {
#pragma unroll 1
          for (int r = 0; r < 16; ++r) {
            const int row = warp * 16 + r, k = tile * kCaKeys + row;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t code = sb[v_off(row, m >> 3) + (m & 7) * 2 + e];
                if ((code & 0x7f) == 0x7f)
#pragma unroll
                  for (int c = 0; c < 2 * NT; ++c) {
                    const int2 lim = row_lim[(c >> 1) * 8 + 2 * t + (c & 1)];
                    if (k >= lim.x && k < lim.y) o[m][c >> 1][2 * e + (c & 1)] = CUDART_NAN_F;
                  }
              }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    };

    const int ta = u.ta, tb = u.tb, in_lo = u.in_lo, in_hi = u.in_hi;
    for (int tile = ta; tile < tb; ++tile) {
      if (ok && !wait_bar(&full[st], ring, ctl)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) continue;
      if (tile * kCaKeys >= in_lo && (tile + 1) * kCaKeys <= in_hi)
        tile_step(MaskTag<false>(), tile);
      else
        tile_step(MaskTag<true>(), tile);
      if (++st == C::STAGES) {
        st = 0;
        ring ^= 1;
      }
    }

    // ---------------------------------------------------------- end of the unit: four states into one
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
        if (g == 0) {
          st_mu[warp][nt * 8 + 2 * t + c] = mu[nt][c];
          st_l[warp][nt * 8 + 2 * t + c] = l[nt][c];
        }
      }
    consumers_sync();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = nt * 8 + 2 * t + c;
        float top = kCaFloor, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kCaWarps; ++w) top = fmaxf(top, st_mu[w][r]);
#pragma unroll
        for (int w = 0; w < kCaWarps; ++w) sum += st_l[w][r] * ex2_approx(st_mu[w][r] - top);
        f[c] = sum == 0.f ? 0.f : ex2_approx(ro[nt][c] - top) / sum;
        if (warp == 0 && g == 0) fin_l[r] = sum == 0.f ? -CUDART_INF_F : top + log2f(sum);
      }
#pragma unroll
      for (int m = 0; m < MT; m += 2) {
        const int d = DV == 64 ? g * 8 + m * 2 : (m >> 3) * 128 + g * 16 + (m & 7) * 2;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          *reinterpret_cast<float4*>(ob + (warp * C::R + nt * 8 + 2 * t + c) * C::OPITCH + d) =
              make_float4(o[m][nt][c] * f[c], o[m][nt][2 + c] * f[c], o[m + 1][nt][c] * f[c],
                          o[m + 1][nt][2 + c] * f[c]);
      }
    }
    consumers_sync();
    const int live = min(C::R, rows - n0);
    const int64_t slot = (int64_t)blockIdx.x * 2 + u.slot;
    for (int x = tid; x < live * (DV / 4); x += kCaConsumers) {
      const int r = x / (DV / 4), d = (x - r * (DV / 4)) * 4, z = n0 + r, i = ca_token(p, z);
      float4 a = *reinterpret_cast<const float4*>(ob + r * C::OPITCH + d);
#pragma unroll
      for (int w = 1; w < kCaWarps; ++w) {
        const float4 b = *reinterpret_cast<const float4*>(ob + (w * C::R + r) * C::OPITCH + d);
        a.x += b.x;
        a.y += b.y;
        a.z += b.z;
        a.w += b.w;
      }
      if (u.whole) {
        const uint2 w = p.f16 ? make_uint2(pack2<__half>(a.x, a.y), pack2<__half>(a.z, a.w))
                              : make_uint2(pack2<__nv_bfloat16>(a.x, a.y), pack2<__nv_bfloat16>(a.z, a.w));
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + p.o_ss * (u.q0 + i) +
                                  p.o_sh * (u.h * p.G + z - i * p.G) + d) = w;
      } else {
        *reinterpret_cast<float4*>(p.part_o + (slot * C::R + r) * DV + d) = a;
      }
    }
    if (tid < live) {
      const int z = n0 + tid, i = ca_token(p, z);
      if (u.whole)
        p.lse[(int64_t)(u.h * p.G + z - i * p.G) * p.s.T + u.q0 + i] = fin_l[tid] * 0.69314718055994531f;
      else
        p.part_l[slot * C::R + tid] = fin_l[tid];
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_empty[qb]);
  }
}

// Joins the partial results of units that several CTAs share, in the order of
// the CTAs, and writes the rows that no CTA wrote: sequences without keys and
// rows past the last sequence.
// BY_UNIT: one CTA per (head, row tile), sequence and part of the row tile: rows
// go to CTAs of their own when there are few units, whose partial results are
// then many (57 per unit for one sequence of 32 Ki keys and 8 heads: 15 us with
// one CTA each). blockIdx.y = B: rows past the last sequence.
// Otherwise (more units than CTAs could share) one CTA per share, for the unit
// that begins in it and goes on in the next one.
constexpr int kJoinThreads = 512;
template <int DV, bool BY_UNIT>
__global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(const __grid_constant__ CacheAttnParams p, int grid) {
  __shared__ float4 sums[kJoinThreads];
  __shared__ float2 tops[kJoinThreads];
  const int tid = threadIdx.x;
  let_next_kernel_start();
  auto zero_rows = [&](const Seq& q, int h, int n0, int count) {  // `count` rows of head h from row n0 of the tile order
    // (Vectors in 64 bits: 2^27 rows of head dim 128 have 2^31.)
    for (int64_t x = tid; x < (int64_t)count * (DV / 8); x += kJoinThreads) {
      const int r = (int)(x / (DV / 8)), col = (int)(x % (DV / 8)), y = n0 + r, i = ca_token(p, y);
      const int hq = h * p.G + y - i * p.G;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + p.o_ss * (q.q0 + i) + p.o_sh * hq + col * 8) =
          make_uint4(0, 0, 0, 0);
      if (col == 0) p.lse[(int64_t)hq * p.s.T + q.q0 + i] = -CUDART_INF_F;
    }
  };
  // Until the attention kernel is done: which unit this CTA joins, and where its
  // partial results are.
  const bool tail = BY_UNIT && blockIdx.y == p.s.B;
  CaSeq s = {};
  int h = 0, n0 = 0, live = 0, c0 = 0, c1 = 0;  // rows [n0, n0 + live) of head h; shares c0 .. c1
  const int part = BY_UNIT ? (1 << p.tile_lg) / gridDim.z : 1 << p.tile_lg;
  if constexpr (BY_UNIT) {
    if (!tail) s = ca_seq(p, blockIdx.y);
    h = blockIdx.x / p.row_tiles;
    const int rt = blockIdx.x % p.row_tiles;
    n0 = (rt << p.tile_lg) + blockIdx.z * part;
    live = tail || rt >= s.rt ? 0 : min(part, s.q.m * p.G - n0);
    if (!tail && live <= 0 && !first_block()) return;
    __shared__ longlong2 counts[kJoinThreads / 32];
    int64_t total;
    const int64_t before = ca_before<kJoinThreads>(p, counts, blockIdx.y, &total);
    if (live > 0 && s.kt > 0) {
      const CaShares shares(total, ca_parts(total, grid, p.min_share));
      const int64_t x0 = before + ((int64_t)h * s.rt + rt) * s.cost() + kCaUnit;  // the unit's first tile
      c0 = shares.owner(x0);
      c1 = shares.owner(x0 + s.kt - 1);
      if (c0 == c1 && !first_block()) return;  // one CTA had it all and wrote it
    }
  } else {
    __shared__ int64_t scan[kJoinThreads / 32], found_base;
    __shared__ int found_b;
    const CaCount count = ca_count<kJoinThreads>(p, scan, false);
    const int parts = ca_parts(count.total, grid, p.min_share);
    if ((int)blockIdx.x + 1 < parts) {
      const CaShares shares(count.total, parts);
      const int64_t cut = shares.first(blockIdx.x + 1);
      ca_locate(p, count, cut, &found_b, &found_base);
      s = ca_seq(p, found_b);
      const int64_t unit = quotient(cut - found_base, s.cost()), x0 = found_base + unit * s.cost() + kCaUnit;
      c0 = shares.owner(x0);
      c1 = shares.owner(x0 + s.kt - 1);
      h = (int)(unit / s.rt);
      n0 = (int)(unit - (int64_t)h * s.rt) << p.tile_lg;
      live = c0 == (int)blockIdx.x ? min(part, s.q.m * p.G - n0) : 0;
    }
  }
  after_previous_kernel();
  if (tail || !BY_UNIT) {  // rows past the last sequence
    int first = p.s.cu ? min(max(p.s.cu[p.s.B], 0), p.s.T) : p.s.T;
    if (first < p.s.T) {
      // Prefix sums that fall can end in front of rows that a sequence has: those are its own.
      __shared__ int ends;
      if (tid == 0) ends = first;
      __syncthreads();
      for (int b = tid; b < p.s.B; b += kJoinThreads) {
        const Seq x = seq_at(p.s, p.c.page, b);
        if (x.m > 0) first = max(first, x.q0 + x.m);
      }
      atomicMax(&ends, first);
      __syncthreads();
      first = ends;
    }
    const Seq rest = {0, p.s.T - first, first, false};
    if (rest.m > 0 && blockIdx.z == 0)
      for (int64_t x = blockIdx.x; x < (int64_t)rest.m * p.c.Hkv; x += gridDim.x)
        zero_rows(rest, (int)(x % p.c.Hkv), (int)(x / p.c.Hkv) * p.G, p.G);
  }
  if constexpr (BY_UNIT) {
    if (live > 0 && s.kt == 0) zero_rows(s.q, h, n0, live);  // a sequence without keys
  } else {
    for (int b = blockIdx.x; b < p.s.B; b += gridDim.x) {
      const CaSeq e = ca_seq(p, b);
      if (e.kt == 0 && e.q.m > 0)
        for (int x = 0; x < p.c.Hkv; ++x) zero_rows(e.q, x, 0, e.q.m * p.G);
    }
  }
  if (live <= 0 || c0 == c1) return;
  const int np = c1 - c0 + 1, at0 = BY_UNIT ? blockIdx.z * part : 0;
  auto row_at = [&](int i, int r) -> int64_t { return (((int64_t)(c0 + i) * 2 + (i == 0)) << p.tile_lg) + at0 + r; };
  // A thread takes four columns of a row over every groups-th partial result, with
  // a running maximum and sum of its own; the groups are added in their order.
  constexpr int VEC = DV / 4;
  const int wide = min(part, kJoinThreads / VEC), groups = kJoinThreads / (VEC * wide);  // rows at a time
  const int gr = tid / (VEC * wide), rr = tid / VEC % wide, d = (tid % VEC) * 4;
  for (int r0 = 0; r0 < live; r0 += wide) {
    const int r = min(r0 + rr, live - 1);
    float top = kCaFloor, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = gr; k0 < np; k0 += groups * 4) {
      float l[4];
      float4 a[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = k0 + u * groups;
        l[u] = -CUDART_INF_F;
        a[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < np) {
          l[u] = p.part_l[row_at(k, r)];
          a[u] = *reinterpret_cast<const float4*>(p.part_o + row_at(k, r) * DV + d);
        }
      }
      float m = top;
#pragma unroll
      for (int u = 0; u < 4; ++u) m = fmaxf(m, l[u]);
      const float f = ex2_approx(top - m);
      acc.x *= f;
      acc.y *= f;
      acc.z *= f;
      acc.w *= f;
      sum *= f;
      top = m;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float w = ex2_approx(l[u] - m);
        sum += w;
        acc.x = fmaf(a[u].x, w, acc.x);
        acc.y = fmaf(a[u].y, w, acc.y);
        acc.z = fmaf(a[u].z, w, acc.z);
        acc.w = fmaf(a[u].w, w, acc.w);
      }
    }
    __syncthreads();
    sums[tid] = acc;
    tops[tid] = make_float2(top, sum);
    __syncthreads();
    if (gr == 0 && r0 + rr < live) {
      float m = top;
      for (int k = 1; k < groups; ++k) m = fmaxf(m, tops[tid + k * VEC * wide].x);
      float f = ex2_approx(top - m);
      acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
      sum *= f;
      for (int k = 1; k < groups; ++k) {
        const float2 ts = tops[tid + k * VEC * wide];
        const float4 a = sums[tid + k * VEC * wide];
        f = ex2_approx(ts.x - m);
        sum = fmaf(ts.y, f, sum);
        acc.x = fmaf(a.x, f, acc.x);
        acc.y = fmaf(a.y, f, acc.y);
        acc.z = fmaf(a.z, f, acc.z);
        acc.w = fmaf(a.w, f, acc.w);
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int y = n0 + r, i = ca_token(p, y);
      acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      const uint2 w = p.f16 ? make_uint2(pack2<__half>(acc.x, acc.y), pack2<__half>(acc.z, acc.w))
                            : make_uint2(pack2<__nv_bfloat16>(acc.x, acc.y), pack2<__nv_bfloat16>(acc.z, acc.w));
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + p.o_ss * (s.q.q0 + i) +
                                p.o_sh * (h * p.G + y - i * p.G) + d) = w;
      if (d == 0)
        p.lse[(int64_t)(h * p.G + y - i * p.G) * p.s.T + s.q.q0 + i] =
            sum == 0.f ? -CUDART_INF_F : (m + log2f(sum)) * 0.69314718055994531f;
    }
  }
}

}  // namespace psf
