// kv_split.cuh - how attention over the paged cache is divided among the
// thread blocks of a launch, and how their parts are joined.
//
// An entry is a group of ROWS query rows of one sequence (rows in the order
// (token, head of the key head's group)); an item is an entry and a key head.
// The tokens that an item's rows see are cut into tiles, and the tiles of all
// items, in the order (entry, head, tile), are cut into as many equal ranges as
// there are thread blocks: a ragged batch, or one long sequence, keeps every
// SM busy to the end.  An item counts as OVER tiles more than it has, for what
// it costs by itself (its queries, its output): these come before its first
// tile, and a range that ends or begins among them has none or all of its tiles.
// The lengths are on the device, so every thread block finds its range itself.
// An item that falls into several ranges leaves the running maximum, the sum and
// the unnormalised output of each part in the workspace; kv_combine_kernel joins
// them, in the order of the tokens.  The division follows from the lengths alone,
// so results do not depend on timing.
#pragma once

#include "kv_cache.cuh"

namespace sta {

struct AttendParams {
  KvLayout c;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;                     // [B][hq][S] or null
  RowStrides qs, os;
  int window;                     // tokens, 0: unlimited
  int group;                      // query heads per key head
  int row_groups;                 // groups of ROWS query rows per (sequence, key head)
  int entries;                    // B * row_groups
  float scale_log2;
  int4* meta;                     // per thread block: the item that it leaves unfinished
  float* part_ml;                 // [2 grid][rows][2]: M, l
  float* part_o;                  // [2 grid][rows][d]
};

// log2 of the weight that the running maximum gets.  f16 weights (e4m3 cache)
// end at 2^-25: with the lift a weight is lost only below 2^-32 of the largest,
// so that 2^17 lost ones still add up to less than a bf16 rounding.  bf16
// weights have fp32's range and need none.
template <bool F8>
constexpr float kLift = F8 ? 7.f : 0.f;

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float bf16x2_max_abs(uint32_t w) {
  return fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u)));
}

__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float times) {
  return pack_f16x2(__uint_as_float(w << 16) * times, __uint_as_float(w & 0xffff0000u) * times);
}

// For products of narrower numbers a query row with largest magnitude m is first
// multiplied by `down`, the power of two that takes m to [2^TOP, 2^(TOP + 1)), and
// its scores by `up`.  Both, and `up` times the scale of the scores, stay normal
// numbers: m from 2^127 on (TOP = 0) gets to [2, 4), and rows below 2^(TOP - 120)
// stay smaller than the others and keep fewer bits.  f16 (TOP = 0): what becomes
// subnormal is off by 2^-25 of the largest at most.  A row with an infinity becomes
// NaN as a whole, as its softmax is: e4m3 has no infinity, and scores that are all
// -inf would look like masked ones.
struct QueryScale {
  float down, up;
};

template <int TOP>
__device__ __forceinline__ QueryScale query_scale(float m) {
  int e = static_cast<int>(__float_as_uint(m) >> 23) - 127 - TOP;
  e = e < -120 ? -120 : (e > 126 ? 126 : e);
  return {m < INFINITY ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23)
                       : __int_as_float(0x7fffffff),
          __uint_as_float(static_cast<uint32_t>(127 + e) << 23)};
}

// Queries that are taken as they are: NaN in the place of infinities.
__device__ __forceinline__ uint32_t bf16x2_inf_to_nan(uint32_t w) {
  return w | (__vcmpeq2(w & 0x7fff7fffu, 0x7f807f80u) & 0x00400040u);
}

// Scales of a block of an e4m3 cache as the softmax uses them.  A value scale
// of 0 (a block never written) counts as 2^-100.  (Both approximations are good to
// 2^-22 for scales below 2^126.)
struct KvScale {
  float k, log2_v, inv_v;
};

__device__ __forceinline__ KvScale kv_scale(float k, float v) {
  const float vs = fmaxf(v, 7.888609052210118e-31f);
  return {k, __log2f(vs), __fdividef(1.f, vs)};
}

// Four (e4m3) or two (bf16) values of a word without its infinities and NaN:
// where some rows of a tile do not see a token, its values must not meet their
// zero weights in the product (0 * NaN); the rows that do see it get them back
// when the item is joined.
template <bool F8>
__device__ __forceinline__ uint32_t drop_nonfinite(uint32_t w, bool& any) {
  const uint32_t mask = F8 ? 0x7f7f7f7fu : 0x7f807f80u;
  const uint32_t hit = F8 ? __vcmpeq4(w & mask, mask) : __vcmpeq2(w & mask, mask);
  any = any || hit != 0;
  return w & ~hit;
}

// Tokens that the rows of one row group see: [lo, hi), and the valid rows.
struct ItemRange {
  int lo, hi;       // positions; hi <= lo: nothing
  int rows;         // valid rows of the group (0: none)
  int fresh, pos0, len;
};

template <int ROWS>
__device__ __forceinline__ ItemRange item_range(const AttendParams& p, int entry) {
  ItemRange r;
  const int b = entry / p.row_groups, rg = entry - b * p.row_groups;
  const KvSeqLen sl = kv_seq(p.c, b);
  r.fresh = sl.fresh;
  r.pos0 = sl.pos0;
  r.len = sl.len;
  const int row0 = rg * ROWS;
  const int left = sl.fresh * p.group - row0;
  r.rows = left < 0 ? 0 : (left > ROWS ? ROWS : left);
  r.lo = r.hi = 0;
  if (r.rows > 0) {
    const int s0 = row0 / p.group, s1 = (row0 + r.rows - 1) / p.group;
    const int top = sl.pos0 + s1 + 1;
    r.hi = top < sl.len ? top : sl.len;
    if (p.window > 0) {
      const int low = sl.pos0 + s0 - p.window + 1;
      r.lo = low > 0 ? low : 0;
    }
  }
  return r;
}

template <int TILE>
__device__ __forceinline__ int item_tiles(const ItemRange& r) {
  return r.hi <= r.lo ? 0 : (r.hi + TILE - 1) / TILE - r.lo / TILE;
}

// What an item counts.
template <int TILE, int OVER>
__device__ __forceinline__ int item_units(const ItemRange& r) {
  return r.hi <= r.lo ? 0 : (r.hi + TILE - 1) / TILE - r.lo / TILE + OVER;
}

// The sum of a row's weights when all of its tokens are counted.  A row that has a
// position sees at least its own token: if it has no weight all the same, its
// scores are all -inf (an infinite key), and its softmax is NaN.  0 is left for
// rows that see nothing.
__device__ __forceinline__ float final_sum(float l, int pos) {
  return l == 0.f && pos >= 0 ? __int_as_float(0x7fffffff) : l;
}

template <int D>
__device__ __forceinline__ void write_row4(const AttendParams& p, int b, int h, int row, int d0,
                                           float4 o) {
  const int s = row / p.group, g = row - s * p.group;
  __nv_bfloat16* dst = p.out + b * p.os.b + (static_cast<long long>(h) * p.group + g) * p.os.h +
                       s * p.os.s + d0;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
}

__device__ __forceinline__ void write_lse(const AttendParams& p, int b, int h, int row, float m,
                                          float l, float lift) {
  if (p.lse == nullptr) return;
  const int s = row / p.group, g = row - s * p.group;
  // m is -inf and l 0 for a row that sees nothing: -inf
  p.lse[(static_cast<long long>(b) * p.c.hq + static_cast<long long>(h) * p.group + g) * p.c.S +
        s] = l > 0.f || l != l ? (m - lift + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// Tokens [lo, hi) that all query rows from first to last of an item see.
struct SeenByAll {
  int lo, hi;
};

__device__ __forceinline__ SeenByAll seen_by_all(const AttendParams& p, const ItemRange& r,
                                                 int first, int last) {
  SeenByAll a;
  a.hi = min(r.pos0 + first / p.group + 1, r.len);
  a.lo = p.window > 0 ? r.pos0 + last / p.group - p.window + 1 : 0;
  return a;
}

// The units [u0, u1) of a thread block, counted over all items; `entry` holds
// the first of them, and the entry's first unit is `base`.
struct KvRange {
  long long u0, u1, total, base;
  int ncta;                         // thread blocks that have a range
  int entry;
};

// The joining kernel is launched while the attention kernel runs (programmatic
// dependent launch), so that its launch costs nothing at the end; it waits here
// until that kernel is complete and its writes are visible.
__device__ __forceinline__ void wait_for_parts() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_kernel_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// a b / c, in 32 bits where they do: that division takes a fraction of the time,
// and every thread block waits for these.
__device__ __forceinline__ long long mul_div(long long a, long long b, long long c) {
  const long long x = a * b;
  if (x < 0x100000000ll)
    return static_cast<uint32_t>(x) / static_cast<uint32_t>(c);
  return x / c;
}

// Rows that see no token at all belong to no range: zeros, -inf.  By all threads
// of all thread blocks.
template <int D, int ROWS, int THREADS>
__device__ __forceinline__ void kv_empty_rows(const AttendParams& p) {
  for (int e = blockIdx.x; e < p.entries; e += gridDim.x) {
    const ItemRange r = item_range<ROWS>(p, e);
    if (r.hi > r.lo || r.rows == 0) continue;
    const int b = e / p.row_groups, row0 = (e - b * p.row_groups) * ROWS;
    for (int i = threadIdx.x; i < r.rows * p.c.hkv * (D / 4); i += THREADS) {
      const int d4 = i % (D / 4), rr = (i / (D / 4)) % r.rows, h = i / (D / 4) / r.rows;
      write_row4<D>(p, b, h, row0 + rr, 4 * d4, make_float4(0.f, 0.f, 0.f, 0.f));
      if (d4 == 0) write_lse(p, b, h, row0 + rr, -INFINITY, 0.f, 0.f);
    }
  }
}

// Called by all threads of a thread block of kv_..._kernel<..., ROWS, TILE>.
template <int D, int ROWS, int TILE, int OVER, int THREADS>
__device__ __forceinline__ KvRange kv_range(const AttendParams& p) {
  __shared__ long long s_start[2];
  __shared__ long long s_warp[THREADS / 32];
  const KvLayout& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  KvRange g;
  const int chunk = (p.entries + THREADS - 1) / THREADS;
  const int e0 = min(p.entries, static_cast<int>(threadIdx.x) * chunk);
  const int e1 = min(p.entries, e0 + chunk);
  long long mine = 0;
  for (int e = e0; e < e1; ++e) mine += item_units<TILE, OVER>(item_range<ROWS>(p, e));
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_warp[warp] = incl;
  if (threadIdx.x == 0) s_start[0] = -1;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  before *= c.hkv;
  total *= c.hkv;
  // with fewer units than thread blocks one each
  g.ncta = total < gridDim.x ? static_cast<int>(total) : static_cast<int>(gridDim.x);
  g.total = total;
  g.u0 = cta < g.ncta ? mul_div(total, cta, g.ncta) : total;
  g.u1 = cta < g.ncta ? mul_div(total, cta + 1, g.ncta) : total;
  if (g.u0 < g.u1 && before <= g.u0 && g.u0 < before + mine * c.hkv) {
    long long at = before;
    if (e1 - e0 == 1) {
      s_start[0] = e0;
      s_start[1] = at;
    }
    for (int e = e0; e1 - e0 > 1 && e < e1; ++e) {
      const long long n =
          static_cast<long long>(item_units<TILE, OVER>(item_range<ROWS>(p, e))) * c.hkv;
      if (g.u0 < at + n) {
        s_start[0] = e;
        s_start[1] = at;
        break;
      }
      at += n;
    }
  }
  if (threadIdx.x == 0) p.meta[cta] = make_int4(-1, 0, 0, 0);
  __syncthreads();
  let_next_kernel_start();
  g.entry = static_cast<int>(s_start[0]);
  g.base = s_start[1];
  if (g.entry < 0) g.u1 = g.u0;                     // no range
  return g;
}

// Runs through the pieces of a range: tiles [t0, t1) of one item each.
struct KvPiece {
  ItemRange r;
  long long u, base, head0;         // next unit; first unit of the entry, of the item
  int entry, b, h, row0;
  int t0, t1, tiles;                // tiles of the piece, and all of the item
  __device__ __forceinline__ void start(const KvRange& g) {
    u = g.u0;
    entry = g.entry;
    base = g.base;
  }
  template <int ROWS, int TILE, int OVER>
  __device__ __forceinline__ bool next(const AttendParams& p, const KvRange& g) {
    for (;;) {
      if (u >= g.u1) return false;
      r = item_range<ROWS>(p, entry);
      const int units = item_units<TILE, OVER>(r);
      const long long all = static_cast<long long>(units) * p.c.hkv;
      if (u >= base + all) {
        base += all;
        if (++entry >= p.entries) return false;     // cannot be: u < total
        continue;
      }
      h = static_cast<int>(mul_div(u - base, 1, units));
      head0 = base + static_cast<long long>(h) * units;
      tiles = units - OVER;
      t0 = max(0, static_cast<int>(u - head0) - OVER);
      const long long end = min(head0 + units, g.u1);
      t1 = max(0, static_cast<int>(end - head0) - OVER);
      u = end;
      if (t1 > t0) break;
    }
    b = entry / p.row_groups;
    row0 = (entry - b * p.row_groups) * ROWS;
    return true;
  }
  template <int TILE>
  __device__ __forceinline__ int tok0() const { return (r.lo / TILE + t0) * TILE; }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
  // where a part is left in the workspace: a thread block leaves two at most,
  // the rest of an item that others began, and the beginning of another
  __device__ __forceinline__ long long slot() const {
    return 2ll * blockIdx.x + (t0 > 0 ? 0 : 1);
  }
  // One thread: notes an item that goes on in the next thread blocks, up to the
  // owner of its last unit, the one whose range [total i / n, total (i + 1) / n)
  // holds it.
  template <int OVER>
  __device__ __forceinline__ void leave(const AttendParams& p, const KvRange& g) const {
    if (whole() || t0 != 0) return;
    const long long end = head0 + tiles + OVER - 1;
    long long c1 = end * g.ncta / g.total;
    while (c1 + 1 < g.ncta && mul_div(g.total, c1 + 1, g.ncta) <= end) ++c1;
    while (c1 > 0 && mul_div(g.total, c1, g.ncta) > end) --c1;
    p.meta[blockIdx.x] = make_int4(entry, h, r.rows, static_cast<int>(c1));
  }
};

// Values that are infinite or NaN, of tokens that some rows of a tile see and
// others do not, must not meet the zero weights of the others in the product
// (0 * NaN): they are left out of it, and afterwards the rows that do see them
// get them back here.  Adds to columns d0 .. d0 + 3 of query row `row` those
// of tokens [from, from + count) that lie in steps of TOK tokens outside those
// that all rows of its tile see.  Only called when something was left out.
struct MendItem {
  int b, h, pos0, len;
};

template <int D, bool F8, int TOK>
__device__ __noinline__ float4 mend_row(const AttendParams& p, const MendItem& it,
                                        const SeenByAll& all, int row, int from, int count,
                                        int d0, float4 acc) {
  const int pos = it.pos0 + row / p.group;
  const int lo = max(from, p.window > 0 ? max(0, pos - p.window + 1) : 0);
  const int hi = min(min(from + count, it.len), pos + 1);
  float a[4] = {acc.x, acc.y, acc.z, acc.w};
  for (int j = lo; j < hi; ++j) {
    const int t = j & ~(TOK - 1);
    if (t >= all.lo && t + TOK <= all.hi) {         // nothing was left out of this step
      j = t + TOK - 1;
      continue;
    }
    const int id = p.c.table[static_cast<long long>(it.b) * p.c.width + (j >> p.c.shift)];
    if (id < 0 || id >= p.c.num_blocks) continue;
    const uint8_t* src = p.c.v + id * p.c.v_block + it.h * p.c.v_head +
                         static_cast<long long>(j & ((1 << p.c.shift) - 1)) * D * (F8 ? 1 : 2);
    for (int e = 0; e < 4; ++e) {
      if constexpr (F8) {
        if ((src[d0 + e] & 0x7f) == 0x7f) a[e] = __int_as_float(0x7fffffff);
      } else {
        const uint32_t w = reinterpret_cast<const uint16_t*>(src)[d0 + e];
        if ((w & 0x7f80u) == 0x7f80u) a[e] += __uint_as_float(w << 16);
      }
    }
  }
  return make_float4(a[0], a[1], a[2], a[3]);
}

// Joins the parts of the item that thread block blockIdx.x of the attention
// kernel left unfinished, in the order of its tokens: the first part is in its
// second place, the others in the first places of the thread blocks after it.
// Latency is all that counts here.  SPLIT = 4: the block's four warps share a
// query row, each with every fourth part, since a long item of few rows has as
// many parts as there are thread blocks.  SPLIT = 1: a warp takes four rows at
// once, of items of many rows and few parts.
template <int D, int ROWS, int SPLIT>
__global__ void __launch_bounds__(128) kv_combine_kernel(const AttendParams p, float lift) {
  constexpr int kF = D / 32;                        // floats per lane
  constexpr int kR = SPLIT == 1 ? 4 : 1;            // rows of a warp
  constexpr int kAhead = 8 / kR;                    // parts on their way at once
  __shared__ float s_acc[SPLIT == 1 ? 1 : 4][D];
  __shared__ float s_l[4];
  const int cta = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp % SPLIT;
  wait_for_parts();
  const int4 it = p.meta[cta];                      // entry, head, rows, last thread block
  const int row_at = (blockIdx.y * (4 / SPLIT) + warp / SPLIT) * kR;
  if (it.x < 0 || row_at >= it.z) return;           // the same for the warps of a row
  const int n = it.w - cta + 1, live = min(kR, it.z - row_at);
  auto at = [&](int i) { return (2ll * (cta + i) + (i == 0 ? 1 : 0)) * ROWS + row_at; };
  float m[kR], l[kR], f[kR], acc[kR][kF];
#pragma unroll
  for (int k = 0; k < kR; ++k) {
    m[k] = -INFINITY;
    l[k] = 0.f;
#pragma unroll
    for (int e = 0; e < kF; ++e) acc[k][e] = 0.f;
  }
  // the first parts are on their way before the maxima are known
  float x[kAhead][kR][kF];
  auto load = [&](int i0, int j, int count) {
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      if (j + e >= count) break;
      const float* src = p.part_o + at(i0 + (j + e) * SPLIT) * D + lane * kF;
#pragma unroll
      for (int k = 0; k < kR; ++k) {
        if (k >= live) break;
        if constexpr (kF == 4)
          *reinterpret_cast<float4*>(x[e][k]) = *reinterpret_cast<const float4*>(src + k * D);
        else
          *reinterpret_cast<float2*>(x[e][k]) = *reinterpret_cast<const float2*>(src + k * D);
      }
    }
  };
  auto parts = [&](int i0) { return min(32, (n - i0 + SPLIT - 1) / SPLIT); };
  if (w < n) load(w, 0, parts(w));
  for (int i = lane; i < n; i += 32)
#pragma unroll
    for (int k = 0; k < kR; ++k)
      if (k < live) m[k] = fmaxf(m[k], p.part_ml[(at(i) + k) * 2]);
#pragma unroll
  for (int k = 0; k < kR; ++k)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m[k] = fmaxf(m[k], __shfl_xor_sync(0xffffffffu, m[k], o));
  for (int i0 = w; i0 < n; i0 += 32 * SPLIT) {      // own parts i0, i0 + SPLIT, ...
    const int count = parts(i0);
#pragma unroll
    for (int k = 0; k < kR; ++k) {
      f[k] = 0.f;
      if (lane < count && k < live) {
        const float2 ml =
            *reinterpret_cast<const float2*>(p.part_ml + (at(i0 + lane * SPLIT) + k) * 2);
        f[k] = ml.y == 0.f ? 0.f : fast_exp2(ml.x - m[k]);    // 0: saw nothing
        l[k] = fmaf(ml.y, f[k], l[k]);
      }
    }
    for (int j = 0; j < count; j += kAhead) {
      if (i0 > w || j > 0) load(i0, j, count);
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        if (j + e >= count) break;
#pragma unroll
        for (int k = 0; k < kR; ++k) {
          const float fi = __shfl_sync(0xffffffffu, f[k], j + e);
#pragma unroll
          for (int c = 0; c < kF; ++c)
            acc[k][c] = fi == 0.f ? acc[k][c] : fmaf(x[e][k][c], fi, acc[k][c]);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kR; ++k)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], o);
  if constexpr (SPLIT > 1) {
    static_assert(SPLIT == 4, "the block's warps share one row");
#pragma unroll
    for (int e = 0; e < kF; ++e) s_acc[warp][lane * kF + e] = acc[0][e];
    if (lane == 0) s_l[warp] = l[0];
    __syncthreads();
    if (warp > 0) return;
    l[0] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) l[0] += s_l[k];
#pragma unroll
    for (int e = 0; e < kF; ++e)
      acc[0][e] = s_acc[0][lane * kF + e] + s_acc[1][lane * kF + e] + s_acc[2][lane * kF + e] +
                  s_acc[3][lane * kF + e];
  }
  const int b = it.x / p.row_groups, row0 = (it.x - b * p.row_groups) * ROWS + row_at;
#pragma unroll
  for (int k = 0; k < kR; ++k) {
    if (k >= live) break;
    const int s = (row0 + k) / p.group, g = row0 + k - s * p.group;
    __nv_bfloat16* dst = p.out + b * p.os.b +
                         (static_cast<long long>(it.y) * p.group + g) * p.os.h + s * p.os.s +
                         lane * kF;
    if (l[k] == 0.f) l[k] = final_sum(0.f, kv_seq(p.c, b).pos0 + s);
    const float inv = l[k] == 0.f ? 0.f : 1.f / l[k];
#pragma unroll
    for (int e = 0; e < kF; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[k][e] * inv, acc[k][e + 1] * inv);
    if (lane == 0) write_lse(p, b, it.y, row0 + k, m[k], l[k], lift);
  }
}

}  // namespace sta
