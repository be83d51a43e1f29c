// rotary.cu -- the position rotation of queries and keys (forward and backward),
// and the cache's append with it.
#include "launch_cache.h"
#include "launch_rotary.h"

namespace psf {

namespace {

// ---------------------------------------------------------------- rows
// Bytes: 2 read and 2 written per element. A CTA takes up to kRowTokens tokens
// with all heads of both tensors, so that the angles, the costly part (some 100
// instructions each), are made once per token and pair and lie in shared memory
// for every head, as the tokens' addresses do. A thread keeps one unit of 16
// components (rotary.cuh) and walks over (token, head), kRowBatch loads ahead of
// the stores; then the CTA goes on to other tokens.
// Many rows are bound by memory: 65536 tokens of 32 + 8 heads of 128 take 198 us,
// 198 at the copy rate. Fewer are bound by latency, loads - places - angles -
// stores, over 32 warps an SM: 20011 tokens of 12 + 12 heads of 128 take 44 us for
// 36, 8192 tokens of 16 + 4 heads 16 to 18 us for 12.4 (issue slots 61 to 64 % busy
// from cold). A row needs heads: 65536 tokens of 1 + 1 heads of 64 give 32 of a CTA's
// threads a unit and take 60 us for 5. Measured
// beside it, from cold: 1, 2, 4, 8 tokens a CTA 90, 63, 51, 53 us for the 20011
// tokens and 342, 238, 209, 223 for the 65536; 2 loads ahead and 6 CTAs an SM for 4
// and 4: 57 and 244; pairs' products by twos, whose operands' places cost what the
// products save: 213 for the 65536.
constexpr int kRowThreads = 256;
constexpr int kRowTokens = 4;
constexpr int kRowBatch = 4;

struct RowsShared {
  alignas(16) float2 cs[kRowTokens][kRotaryPairs];  // scale * (cos, sin), read two pairs at a time
  int place[kRowTokens];
  uint64_t turns[kRotaryPairs];
  bool odd[kRotaryPairs];  // the frequency has no angle
  // Where head 0 of a token's row would lie, were all heads in tensor 0, or in tensor 1; of the next tokens, too.
  const char* x[2][kRowTokens][2];
  char* y[2][kRowTokens][2];
};

static_assert(alignof(RowsShared) >= alignof(float4), "pairs are read by twos");

// What the frequencies stand for, for rows_tables, by all threads (without a barrier behind it).
__device__ __forceinline__ void rows_turns(RowsShared& sh, const RotaryView& r) {
  for (int i = threadIdx.x; i < r.half; i += kRowThreads) {
    const float f = r.inv_freq[i];
    sh.turns[i] = turns_per_position(f);
    sh.odd[i] = no_angle(f);
  }
}

// Element offset of a row in tensor i of the arguments, or in its result.
__device__ __forceinline__ int64_t row_at(const RotaryRows& a, int64_t row, const int64_t (&batch)[2], const int64_t (&step)[2],
                                          int i) {
  if (a.S == a.rows) return row * step[i];
  const uint32_t b = (uint32_t)row / (uint32_t)a.S;
  return b * batch[i] + ((uint32_t)row - b * (uint32_t)a.S) * step[i];
}

// Places and tables of tokens [row0, row0 + n), by all threads. base(row): a row's
// place where positions are not given, by a whole warp. The pairs of unit u lie as
// float4 (q, u), q = 0..3, so that neighbouring units' reads do not meet in a bank;
// PLAIN: in their order.
template <bool PLAIN, typename F>
__device__ __forceinline__ void rows_tables(RowsShared& sh, const RotaryView& r, const PlaceView& p, int64_t row0, int n,
                                            F base) {
  const int tid = threadIdx.x, warp = tid >> 5;
  if (!p.pos) {
    if (warp < n) {
      const int place = base(row0 + warp);
      if ((tid & 31) == 0) sh.place[warp] = place;
    }
    __syncthreads();
  }
  const int units = r.half >> 3;
  for (int e = tid; e < n * r.half; e += kRowThreads) {
    const int t = over_half(r, e), i = e - t * r.half;
    const int place = p.pos ? p.pos[p.axis_stride * r.axis[i] + row0 + t] : sh.place[t];
    float2 cs = rotary_pair(r, sh.turns[i], place);
    if (sh.odd[i]) cs = make_float2(CUDART_NAN_F, CUDART_NAN_F);
    sh.cs[t][PLAIN ? i : (((i >> 1) & 3) * units + (i >> 3)) * 2 + (i & 1)] = cs;
  }
  __syncthreads();
}

// Tokens [g * tokens, ...) for g = blockIdx.x, blockIdx.x + gridDim.x, .... tables(row0, n): makes sh.cs; the first loads are
// on their way meanwhile.
template <typename T, typename F>
__device__ __forceinline__ void rotate_rows(RowsShared& sh, const RotaryView& r, const RotaryRows& a, int tokens, F tables) {
  // (Whole quotients of numbers up to 256 by up to 64 in fp32: with the half added none lies within a rounding of a whole one.)
  const int units = a.D >> 4, turning = r.half >> 3;
  const float per = __frcp_rn((float)units);
  const int slots = (int)((kRowThreads + 0.5f) * per), slot = (int)((threadIdx.x + 0.5f) * per), u = threadIdx.x - slot * units;
  const RotaryUnit un = rotary_unit(r, u);
  const int heads = a.H[0] + a.H[1];
  // Addresses of the tokens' rows once per CTA, not for every row and head.
  auto addresses = [&](int64_t row0, int par) {
    const int tk = threadIdx.x >> 2, i = threadIdx.x & 1;
    if (tk >= tokens || row0 + tk >= a.rows) return;
    const int64_t back = i ? a.H[0] : 0;
    if (threadIdx.x & 2)
      sh.y[par][tk][i] = static_cast<char*>(a.y[i]) + sizeof(T) * (row_at(a, row0 + tk, a.yb, a.ys, i) - a.yh[i] * back);
    else
      sh.x[par][tk][i] = static_cast<const char*>(a.x[i]) + sizeof(T) * (row_at(a, row0 + tk, a.xb, a.xs, i) - a.xh[i] * back);
  };
  const int c0 = un.c0 * (int)sizeof(T), c1 = un.c1 * (int)sizeof(T);
  int64_t row0 = (int64_t)blockIdx.x * tokens;
  int n = (int)min((int64_t)tokens, a.rows - row0), par = 0;
  int t, h;
  auto settle = [&] {
    while (h >= heads && t < n) {
      h -= heads;
      ++t;
    }
  };
  uint4 v0[kRowBatch], v1[kRowBatch];
  uint32_t at[kRowBatch];  // head << 3 | token
  static_assert(kRowTokens < 8, "three bits");
  auto load = [&] {
#pragma unroll
    for (int k = 0; k < kRowBatch; ++k) {
      at[k] = (uint32_t)h << 3 | t;
      if (t < n) {
        const int i = h >= a.H[0];
        const char* x = sh.x[par][t][i] + (i ? a.xh[1] : a.xh[0]) * (int)sizeof(T) * h;
        v0[k] = *reinterpret_cast<const uint4*>(x + c0);
        v1[k] = *reinterpret_cast<const uint4*>(x + c1);
        h += slots;
        settle();
      }
    }
  };
  addresses(row0, 0);
  rows_turns(sh, r);
  for (;;) {
    __syncthreads();
    t = slot < slots ? 0 : n;
    h = slot;
    settle();
    load();
    const int64_t next = row0 + (int64_t)gridDim.x * tokens;
    if (next < a.rows) addresses(next, par ^ 1);
    tables(row0, n);
    while ((int)(at[0] & 7) < n) {
#pragma unroll
      for (int k = 0; k < kRowBatch; ++k) {
        const int tk = at[k] & 7, hk = at[k] >> 3;
        if (tk >= n) break;
        const int i = hk >= a.H[0];
        char* y = sh.y[par][tk][i] + (i ? a.yh[1] : a.yh[0]) * (int)sizeof(T) * hk;
        if (un.pair >= 0) {
          float val[16];
          unpack8<T>(v0[k], val, 0);
          unpack8<T>(v1[k], val, 8);
          const float4* cs = reinterpret_cast<const float4*>(sh.cs[tk]) + u;
          turn_unit(val, r.interleaved, [&](int e) {
            const float4 two = cs[(e >> 1) * turning];
            return e & 1 ? make_float2(two.z, two.w) : make_float2(two.x, two.y);
          });
          v0[k] = pack8<T>(val, 0);
          v1[k] = pack8<T>(val, 8);
        } else if ((i ? a.x[1] : a.x[0]) == (i ? a.y[1] : a.y[0])) {
          continue;
        }
        *reinterpret_cast<uint4*>(y + c0) = v0[k];
        *reinterpret_cast<uint4*>(y + c1) = v1[k];
      }
      load();
    }
    if (next >= a.rows) break;
    row0 = next;
    n = (int)min((int64_t)tokens, a.rows - row0);
    par ^= 1;
  }
}

// The same for any layout: a pair, or a component that passes, at a time. Bound by its instructions (two divisions and two rows'
// addresses for each): 65536 tokens of 16 + 4 heads of 72, all of it turned, take 221 us for 56 at the copy rate, of 128 with 50
// turned 558 for 99.
template <typename T>
__device__ __forceinline__ void rotate_rows_any(RowsShared& sh, const RotaryView& r, const RotaryRows& a, int64_t row0,
                                                int n) {
  const uint32_t heads = a.H[0] + a.H[1], items = a.D - r.half;
  for (uint32_t e = threadIdx.x; e < n * heads * items; e += kRowThreads) {  // (at most 4 * 131070 * 1023)
    const uint32_t th = e / items;
    const int x = (int)(e - th * items), t = (int)(th / heads), h = (int)(th - t * heads);
    const int i = h >= a.H[0];
    const T* from =
        static_cast<const T*>(a.x[i]) + row_at(a, row0 + t, a.xb, a.xs, i) + a.xh[i] * (h - (i ? a.H[0] : 0));
    T* to = static_cast<T*>(a.y[i]) + row_at(a, row0 + t, a.yb, a.ys, i) + a.yh[i] * (h - (i ? a.H[0] : 0));
    if (x < r.half) {
      const int c0 = r.start + (r.interleaved ? 2 * x : x), c1 = c0 + (r.interleaved ? 1 : r.half);
      const float2 y = turned((float)from[c0], (float)from[c1], sh.cs[t][x]);
      to[c0] = (T)y.x;
      to[c1] = (T)y.y;
    } else if (a.x[i] != a.y[i]) {
      const int c = x - r.half < r.start ? x - r.half : x + r.half;
      to[c] = from[c];
    }
  }
}

template <typename T, bool ANY>
__global__ void __launch_bounds__(kRowThreads, 4)
    rotary_kernel(const __grid_constant__ RotaryView r, const PlaceView p, const __grid_constant__ RotaryRows a, int tokens,
                  int* status) {
  __shared__ RowsShared sh;
  after_previous_kernel();
  int nseg = a.nseg;
  if (a.cu) {
    if (a.dev_meta) nseg = min(max(a.dev_meta[0], 0), nseg);
    if (blockIdx.x == 0) {
      bool bad = a.cu[0] != 0 || a.cu[nseg] > a.rows || (a.cu_k && a.cu_k[0] != 0);
      for (int i = threadIdx.x; i < nseg; i += kRowThreads)
        bad |= a.cu[i + 1] < a.cu[i] || (a.cu_k && a.cu_k[i + 1] < a.cu_k[i]);
      if (bad) record_status(status, kStatusDeviceArgs);
    }
  }
  auto base = [&](int64_t row) -> int {
    if (!a.cu) return (int)(row % a.S);
    if (nseg == 0 || row >= a.cu[nseg]) return 0;
    const int s = warp_find(nseg, row, [&](int i) { return a.cu[i]; });
    return a.cu_k ? (int)row - a.cu[s + 1] + (a.cu_k[s + 1] - a.cu_k[s]) : (int)row - a.cu[s];
  };
  auto tables = [&](int64_t row0, int n) { rows_tables<ANY>(sh, r, p, row0, n, base); };
  if constexpr (ANY) {
    const int64_t row0 = (int64_t)blockIdx.x * tokens;
    const int n = (int)min((int64_t)tokens, a.rows - row0);
    rows_turns(sh, r);
    __syncthreads();
    tables(row0, n);
    rotate_rows_any<T>(sh, r, a, row0, n);
  } else {
    rotate_rows<T>(sh, r, a, tokens, tables);
  }
}

// ---------------------------------------------------------------- append
// Many new rows: a CTA per (sequence, page it enters, K or V, up to 8 heads), 128
// threads to a head at a time, and CTAs of a few tokens for the queries, which run
// beside them. A key is turned in fp32 and never rounded to 16 bits in between: the
// block's scale and codes are those of the turned values. The angles of a page's
// new rows are made once, in shared memory, for all of its heads: made for every
// head anew they were most of the work (17 Ki tokens with 8 KV heads of 128 and 32
// query heads took 118 us in all; now 87, 63 at the copy rate: the pages' kernel
// alone 45 us and the queries' 52, with issue slots 63 % busy in both). Rows are kept as they came between the look for
// the largest magnitude and the codes, and turned twice: kept as fp32 they took
// twice the registers. Where a page's angles have no room in shared memory (128
// rows of more than 208 pairs) a thread makes its own.
constexpr int kPageThreads = 128;  // of a head
constexpr int kPageGroups = 4;     // heads at a time
constexpr int kPageHeads = 8;
constexpr int kPageHeld = 4;       // units of a thread kept between the two looks at the rows
constexpr int kTableBytes = 208 * 1024;
constexpr float kMaxFinite = 3.402823466e38f;

struct AppendArgs {
  CacheView c;
  SeqView s;
  PlaceView p;
  RotaryRows q;
  const void *k, *v;
  int64_t k_ss, k_sh, v_ss, v_sh;
  int tokens;      // of a CTA of query rows
  int* status;
};

// Row's place in the cache, by a whole warp: 0 for rows of no sequence, or of one that takes none.
__device__ __forceinline__ int cache_place(const SeqView& s, int page, int64_t row) {
  const int b = s.cu ? warp_find(s.B, row, [&](int i) { return s.cu[i]; }) : (int)(row / max(s.each, 1));
  const Seq x = seq_at(s, page, min(b, s.B - 1));
  const int64_t i = row - x.q0;
  return x.bad || x.m > x.n || i < 0 || i >= x.m ? 0 : (int)(x.n - x.m + i);
}

// Barriers of the threads of a head.
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); }
__device__ __forceinline__ bool group_or(int g, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(1 + g)
      : "memory");
  return r != 0;
}

// TABLE: angles from shared memory. UNITS: rows come in units of 16 components, else a component at a time.
template <typename T, bool TABLE, bool UNITS>
__global__ void __launch_bounds__(kPageThreads* kPageGroups, 2)
    append_rotary_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ RotaryView r) {
  extern __shared__ __align__(16) float2 table[];  // [row][half]: a row as in rows_tables, PLAIN without UNITS
  static_assert(__alignof__(table) >= alignof(float4), "pairs are read by twos");
  __shared__ uint64_t turns[kRotaryPairs];
  __shared__ float warp_top[kPageGroups][kPageThreads / 32];
  const CacheView& c = a.c;
  const SeqView& s = a.s;
  const int tid = threadIdx.x & (kPageThreads - 1), g = threadIdx.x / kPageThreads;
  const bool is_v = blockIdx.z;
  after_previous_kernel();
  let_next_kernel_start();  // the queries' kernel, which waits for nothing of this one
  if (first_block()) {
    bool bad = cu_bad(s);
    for (int i = threadIdx.x; i < s.B; i += kPageThreads * kPageGroups) {
      const Seq x = seq_at(s, c.page, i);
      bad |= x.bad || x.m > x.n;
    }
    if (bad) record_status(a.status, kStatusDeviceArgs);
  }
  const int64_t task = blockIdx.x;
  auto start = [&](int b) -> int64_t { return (s.cu ? s.cu[b] : b * s.each) / c.page + 2 * (int64_t)b; };
  const int b = warp_find(s.B, task, start);
  const Seq q = seq_at(s, c.page, b);
  if (q.bad || q.m > q.n) return;
  const int64_t nth = task - start(b);
  const int first = q.n - q.m;  // place of the first new token
  const int64_t pi = (first >> c.page_lg) + nth;
  if (nth < 0 || q.m == 0 || pi > (q.n - 1) >> c.page_lg) return;
  const int pg = s.table[(int64_t)b * s.max_pages + pi];
  if (pg < 0 || pg >= c.pages) {
    if (threadIdx.x == 0) record_status(a.status, kStatusDeviceArgs);
    return;
  }
  const int at0 = (int)pi << c.page_lg;
  const int r0 = max(first - at0, 0), r1 = min(q.n - at0, c.page);  // new rows of the page
  const int D = is_v ? c.Dv : c.Dqk, units = D >> 4, items = (r1 - r0) * units, turning = r.half >> 3;
  const int64_t ss = is_v ? a.v_ss : a.k_ss, sr = is_v ? c.v_sr : c.k_sr;
  const int64_t token0 = (int64_t)q.q0 + at0 + r0 - first;  // packed row of the page's first new one
  // Head dims of 64, 128 and 512 have 4, 8 and 32 units, 192 has 12.
  const int lg = 31 - __clz(units);
  auto row_of = [&](int e) { return units == 12 ? (int)((uint32_t)e / 12u) : e >> lg; };
  const int head0 = blockIdx.y * kPageHeads, heads = min(c.Hkv - head0, kPageHeads);
  const T* in = nullptr;
  auto unit_of = [&](int u) { return UNITS && !is_v ? rotary_unit(r, u) : RotaryUnit{u * 16, u * 16 + 8, -1}; };
  auto fetch = [&](int e, uint4& v0, uint4& v1) {
    const int row = row_of(e);
    const RotaryUnit un = unit_of(e - row * units);
    v0 = *reinterpret_cast<const uint4*>(in + ss * row + un.c0);
    v1 = *reinterpret_cast<const uint4*>(in + ss * row + un.c1);
  };
  uint4 v0[kPageHeld], v1[kPageHeld];
  auto fetch_held = [&](int h) {
    in = static_cast<const T*>(is_v ? a.v : a.k) + (is_v ? a.v_sh : a.k_sh) * h + ss * token0;
#pragma unroll
    for (int k = 0; k < kPageHeld; ++k)
      if (k * kPageThreads + tid < items) fetch(k * kPageThreads + tid, v0[k], v1[k]);
  };
  if (g < heads) fetch_held(head0 + g);

  auto place_of = [&](int row, int pair) {
    return a.p.pos ? a.p.pos[a.p.axis_stride * r.axis[pair] + token0 + row] : at0 + r0 + row;
  };
  auto angle = [&](int row, int pair) {
    const float2 cs = rotary_pair(r, turns[pair], place_of(row, pair));
    return no_angle(r.inv_freq[pair]) ? make_float2(CUDART_NAN_F, CUDART_NAN_F) : cs;
  };
  if (!is_v) {
    for (int i = threadIdx.x; i < r.half; i += kPageThreads * kPageGroups) turns[i] = turns_per_position(r.inv_freq[i]);
    __syncthreads();
    if constexpr (TABLE) {
      for (int e = threadIdx.x; e < (r1 - r0) * r.half; e += kPageThreads * kPageGroups) {
        const int row = over_half(r, e), i = e - row * r.half;
        table[row * r.half + (UNITS ? (((i >> 1) & 3) * turning + (i >> 3)) * 2 + (i & 1) : i)] = angle(row, i);
      }
      __syncthreads();
    }
  }
  // The 16 values of unit e of the new rows.
  auto values = [&](int e, const uint4& w0, const uint4& w1, float (&y)[16]) {
    unpack8<T>(w0, y, 0);
    unpack8<T>(w1, y, 8);
    if (is_v) return;
    const int row = row_of(e), u = e - row * units;
    if constexpr (UNITS) {
      if (u < turning) {
        const float4* cs = reinterpret_cast<const float4*>(table + row * r.half) + u;
        turn_unit(y, r.interleaved, [&](int i) {
          if constexpr (TABLE) {
            const float4 two = cs[(i >> 1) * turning];
            return i & 1 ? make_float2(two.z, two.w) : make_float2(two.x, two.y);
          } else {
            return angle(row, u * 8 + i);
          }
        });
      }
    } else {
      const T* x = in + ss * row;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const RotaryComponent z = rotary_component(r, u * 16 + i);
        if (z.pair >= 0) {
          const float2 cs = TABLE ? table[row * r.half + z.pair] : angle(row, z.pair);
          const float other = (float)x[z.other];
          y[i] = z.first ? turned(y[i], other, cs).x : turned(other, y[i], cs).y;
        }
      }
    }
  };
  for (int hh = g; hh < heads; hh += kPageGroups) {
    const int h = head0 + hh;
    uint8_t* out = is_v ? c.v + c.v_sp * pg + c.v_sh * h : c.k + c.k_sp * pg + c.k_sh * h;
    float* scale_at = (is_v ? c.v_scale : c.k_scale) + (int64_t)pg * c.Hkv + h;
    const float old = *scale_at;
    float top = 0.f;
    auto all_units = [&](auto f) {  // f(unit, its values)
#pragma unroll
      for (int k = 0; k < kPageHeld; ++k)
        if (k * kPageThreads + tid < items) {
          float y[16];
          values(k * kPageThreads + tid, v0[k], v1[k], y);
          f(k * kPageThreads + tid, y);
        }
#pragma unroll 1
      for (int e = kPageHeld * kPageThreads + tid; e < items; e += kPageThreads) {
        float y[16];
        uint4 w0, w1;
        fetch(e, w0, w1);
        values(e, w0, w1, y);
        f(e, y);
      }
    };
    all_units([&](int, const float (&y)[16]) {
#pragma unroll
      for (int i = 0; i < 16; i += 2) top = fmax3(top, fabsf(y[i]), fabsf(y[i + 1]));
    });
    // (NaN does not show in a maximum and becomes the code NaN by itself; infinities do and have to be told.)
    const bool odd = group_or(g, !(top <= kMaxFinite));
    if (odd) {  // once more, over the finite values alone
      top = 0.f;
#pragma unroll 1
      for (int e = tid; e < items; e += kPageThreads) {
        float y[16];
        uint4 w0, w1;
        fetch(e, w0, w1);
        values(e, w0, w1, y);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (fabsf(y[i]) <= kMaxFinite) top = fmaxf(top, fabsf(y[i]));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 31) == 0) warp_top[g][tid >> 5] = top;
    group_sync(g);  // also: every thread has read the old scale
#pragma unroll
    for (int w = 0; w < kPageThreads / 32; ++w) top = fmaxf(top, warp_top[g][w]);
    const float fresh = block_scale(top);
    const float scale = r0 > 0 ? fmaxf(fresh, old) : fresh;
    if (tid == 0 && (r0 == 0 || scale != old)) *scale_at = scale;
    if (r0 > 0 && scale != old) {
      const float ratio = old / scale;
      for (int i = tid; i < r0 * units; i += kPageThreads) {
        const int row = i / units;
        uint4* to = reinterpret_cast<uint4*>(out + sr * row + (i - row * units) * 16);
        *to = rescale16(*to, ratio);
      }
    }
    // A scale that the append chose is a power of two; one that was there may not be.
    const bool plain = !odd && (__float_as_int(scale) & 0x7fffff) == 0 && scale > 0.f;
    const float inv = plain ? 1.f / scale : 0.f;
    all_units([&](int e, const float (&y)[16]) {
      const int row = row_of(e);
      const RotaryUnit un = unit_of(e - row * units);
      uint32_t w[8];
      if (plain) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = e4m3_pair(y[2 * i] * inv, y[2 * i + 1] * inv);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          w[i] = e4m3_pair(divide_to_odd(finite_or_nan(y[2 * i]), scale), divide_to_odd(finite_or_nan(y[2 * i + 1]), scale));
      }
      uint8_t* to = out + sr * (r0 + row);
      *reinterpret_cast<uint2*>(to + un.c0) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
      *reinterpret_cast<uint2*>(to + un.c1) = make_uint2(w[4] | (w[5] << 16), w[6] | (w[7] << 16));
    });
    if (!is_v && c.weight)
      for (int row = r0 + tid; row < r1; row += kPageThreads) c.weight[((int64_t)pg * c.Hkv + h) * c.page + row] = 0.f;
    if (hh + kPageGroups < heads) fetch_held(h + kPageGroups);
    group_sync(g);  // warp_top is read
  }
}

// The query rows of an append: as rotary_kernel, with places in the cache, and a CTA per group of tokens. (Resident CTAs that walk
// over the groups, as there, have not been measured beside the pages' kernel, whose CTAs they would share the SMs with.)
template <typename T, bool ANY>
__global__ void __launch_bounds__(kRowThreads, 4)
    append_queries_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ RotaryView r) {
  __shared__ RowsShared sh;
  // The pages' kernel lets this one start once everything before it is done, and touches nothing that is read or written
  // here. (What comes next waits for this kernel alone, so one block waits for that one.)
  if (first_block()) after_previous_kernel();
  let_next_kernel_start();
  auto tables = [&](int64_t row0, int n) {
    rows_tables<ANY>(sh, r, a.p, row0, n, [&](int64_t row) { return cache_place(a.s, a.c.page, row); });
  };
  if constexpr (ANY) {
    const int64_t row0 = (int64_t)blockIdx.x * a.tokens;
    const int n = (int)min((int64_t)a.tokens, a.q.rows - row0);
    rows_turns(sh, r);
    __syncthreads();
    tables(row0, n);
    rotate_rows_any<T>(sh, r, a.q, row0, n);
  } else {
    rotate_rows<T>(sh, r, a.q, a.tokens, tables);
  }
}

// One new row per sequence (a decode step): a warp per (sequence, K or V or query
// head). Latency bounds it, as in the append without rotation: the row lies in
// shared memory as fp32, so that a lane reaches the other half of its pairs. 64
// sequences of 8 KV and 32 query heads of 128: 4.4 us a replayed step (2.3 without
// rotation and queries); each warp makes its sequence's angles for itself.
template <typename T>
__global__ void __launch_bounds__(kPageThreads)
    append_rotary_one_kernel(const __grid_constant__ AppendArgs a, const __grid_constant__ RotaryView r) {
  __shared__ __align__(8) float row_at[kPageThreads / 32][512];
  static_assert(__alignof__(row_at) >= alignof(float2), "components are written by twos");
  __shared__ float2 cs_at[kPageThreads / 32][kRotaryPairs];
  const CacheView& c = a.c;
  const SeqView& s = a.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t task = (int64_t)blockIdx.x * (kPageThreads / 32) + warp;
  const int kinds = 2 * c.Hkv + a.q.H[0];
  const int b = (int)(task / kinds), kind = (int)(task - (int64_t)b * kinds);
  const bool is_v = kind >= c.Hkv && kind < 2 * c.Hkv, is_q = kind >= 2 * c.Hkv;
  const int h = is_q ? kind - 2 * c.Hkv : is_v ? kind - c.Hkv : kind;
  after_previous_kernel();
  if (b >= s.B) return;
  const int D = is_v ? c.Dv : c.Dqk, words = D >> 6;  // pairs of components per lane: 1, 2, 3 or 8
  const T* in = is_q ? static_cast<const T*>(a.q.x[0]) + a.q.xs[0] * b + a.q.xh[0] * h
                     : static_cast<const T*>(is_v ? a.v : a.k) + (is_v ? a.v_ss : a.k_ss) * b + (is_v ? a.v_sh : a.k_sh) * h;
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = j < words ? reinterpret_cast<const uint32_t*>(in)[lane * words + j] : 0;
  const int n = s.lens[b];
  const bool length_ok = n >= 1 && (int64_t)n <= (int64_t)s.max_pages * c.page;
  float y[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = unpack2<T>(w[j]);
    y[2 * j] = f.x;
    y[2 * j + 1] = f.y;
  }
  if (!is_v) {
    float* row = row_at[warp];
    float2* cs = cs_at[warp];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < words) *reinterpret_cast<float2*>(row + (lane * words + j) * 2) = make_float2(y[2 * j], y[2 * j + 1]);
    for (int i = lane; i < r.half; i += 32) {
      const float f = r.inv_freq[i];
      const int place = a.p.pos ? a.p.pos[a.p.axis_stride * r.axis[i] + b] : length_ok ? n - 1 : 0;
      const float2 x = rotary_pair(r, turns_per_position(f), place);
      cs[i] = no_angle(f) ? make_float2(CUDART_NAN_F, CUDART_NAN_F) : x;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < 2 * words) {
        const RotaryComponent z = rotary_component(r, lane * words * 2 + j);
        if (z.pair >= 0) {
          const float other = row[z.other];
          y[j] = z.first ? turned(y[j], other, cs[z.pair]).x : turned(other, y[j], cs[z.pair]).y;
        }
      }
  }
  if (is_q) {
    uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<T*>(a.q.y[0]) + a.q.ys[0] * b + a.q.yh[0] * h) + lane * words;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < words) to[j] = pack2<T>(y[2 * j], y[2 * j + 1]);
    return;
  }
  const int row = (n - 1) & (c.page - 1);
  const int pg = length_ok ? s.table[(int64_t)b * s.max_pages + ((n - 1) >> c.page_lg)] : -1;
  if (pg < 0 || pg >= c.pages) {
    if (lane == 0) record_status(a.status, kStatusDeviceArgs);
    return;
  }
  float* scale_at = (is_v ? c.v_scale : c.k_scale) + (int64_t)pg * c.Hkv + h;
  const float old = *scale_at;
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (fabsf(y[j]) <= kMaxFinite) top = fmaxf(top, fabsf(y[j]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float fresh = block_scale(top), scale = row > 0 ? fmaxf(fresh, old) : fresh;
  uint8_t* out = is_v ? c.v + c.v_sp * pg + c.v_sh * h : c.k + c.k_sp * pg + c.k_sh * h;
  const int64_t sr = is_v ? c.v_sr : c.k_sr;
  if (row > 0 && scale != old) {
    const float ratio = old / scale;
    const int vecs = D >> 4;
#pragma unroll 4
    for (int i = lane; i < row * vecs; i += 32) {
      const int at = i / vecs;
      uint4* x = reinterpret_cast<uint4*>(out + sr * at + (i - at * vecs) * 16);
      *x = rescale16(*x, ratio);
    }
  }
  const bool plain = (__float_as_int(scale) & 0x7fffff) == 0 && scale > 0.f;
  const float inv = plain ? 1.f / scale : 0.f;
  uint16_t* to = reinterpret_cast<uint16_t*>(out + sr * row) + lane * words;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < words) {
      const float lo = finite_or_nan(y[2 * j]), hi = finite_or_nan(y[2 * j + 1]);
      to[j] = (uint16_t)(plain ? e4m3_pair(lo * inv, hi * inv) : e4m3_pair(divide_to_odd(lo, scale), divide_to_odd(hi, scale)));
    }
  if (lane == 0) {
    if (row == 0 || scale != old) *scale_at = scale;
    if (!is_v && c.weight) c.weight[((int64_t)pg * c.Hkv + h) * c.page + row] = 0.f;
  }
}

// Tokens that a CTA of rows takes at a time: one where there are few, to fill the device, up to four from two CTAs an SM on
// (20 heads of 128, 150 tokens: 3.7 us with one, 4.1 with two, 4.4 with four; 700: 5.4, 4.5, 4.7; 4000: 15.5, 11.8, 10.1).
int row_tokens(int64_t rows, int sms) { return (int)min(max(rows / (2 * sms), (int64_t)1), (int64_t)kRowTokens); }

template <typename T>
cudaError_t run_rotary(const RotaryView& r, const PlaceView& p, const RotaryRows& a, int sms, int* status,
                       cudaStream_t st) {
  const int tokens = row_tokens(a.rows, sms);
  const bool units = rotary_units(r, a.D);
  const int64_t groups = (a.rows + tokens - 1) / tokens;
  // Up to ten groups of tokens per resident CTA, as many CTAs as are resident walk over them (20011 tokens of 24 heads: 43.8 us for
  // 45.8 with two groups a CTA, 8192 of 20: 15.8 for 16.9). More of them drift apart, which the memory takes ill (65536 tokens
  // of 40 heads: 215 us for 198).
  const int64_t resident = (int64_t)4 * sms;
  const dim3 grid((unsigned)(!units ? groups : groups <= 10 * resident ? min(groups, resident) : (groups + 1) / 2));
  return launch_early(units ? rotary_kernel<T, false> : rotary_kernel<T, true>, grid, kRowThreads, 0, st, r,
                      p, a, tokens, status);
}

template <typename T>
cudaError_t run_append(AppendArgs& a, const RotaryView& r, int sms, cudaStream_t st) {
  const int warps = kPageThreads / 32;
  if (!a.s.cu && a.s.each == 1) {
    const int64_t tasks = (int64_t)a.s.B * (2 * a.c.Hkv + a.q.H[0]);
    return launch_early(append_rotary_one_kernel<T>, dim3((unsigned)((tasks + warps - 1) / warps)), kPageThreads, 0, st, a,
                        r);
  }
  const bool units = rotary_units(r, a.c.Dqk);
  const int bytes = a.c.page * r.half * (int)sizeof(float2);
  const bool table = bytes <= kTableBytes;
  const dim3 grid((unsigned)(a.s.T / a.c.page + 2 * (int64_t)a.s.B), (a.c.Hkv + kPageHeads - 1) / kPageHeads, 2);
  static std::atomic<uint64_t> units_set{0}, any_set{0};
  cudaError_t e = kernel_setup(append_rotary_kernel<T, true, true>, kTableBytes, false, units_set);
  if (e == cudaSuccess) e = kernel_setup(append_rotary_kernel<T, true, false>, kTableBytes, false, any_set);
  if (e == cudaSuccess) {
    auto kernel = units ? (table ? append_rotary_kernel<T, true, true> : append_rotary_kernel<T, false, true>)
                        : (table ? append_rotary_kernel<T, true, false> : append_rotary_kernel<T, false, false>);
    e = launch_early(kernel, grid, kPageThreads * kPageGroups, table ? bytes : 0, st, a, r);
  }
  if (e != cudaSuccess || a.q.H[0] == 0) return e;
  a.tokens = row_tokens(a.q.rows, sms);
  return launch_early(units ? append_queries_kernel<T, false> : append_queries_kernel<T, true>,
                      dim3((unsigned)((a.q.rows + a.tokens - 1) / a.tokens)), kRowThreads, 0, st, a, r);
}

}  // namespace

cudaError_t launch_rotary(const RotaryView& r, const PlaceView& place, const RotaryRows& a, int f16, int sms, int* status,
                          cudaStream_t st) {
  return f16 ? run_rotary<__half>(r, place, a, sms, status, st) : run_rotary<__nv_bfloat16>(r, place, a, sms, status, st);
}

cudaError_t launch_cache_append_rotary(const CacheView& c, const SeqView& s, const RotaryView& r, const PlaceView& place,
                                       const void* k, int64_t k_ss, int64_t k_sh, const void* v, int64_t v_ss,
                                       int64_t v_sh, const RotaryRows& q, int f16, int sms, int* status, cudaStream_t st) {
  AppendArgs a = {c, s, place, q, k, v, k_ss, k_sh, v_ss, v_sh, 0, status};
  return f16 ? run_append<__half>(a, r, sms, st) : run_append<__nv_bfloat16>(a, r, sms, st);
}

}  // namespace psf
