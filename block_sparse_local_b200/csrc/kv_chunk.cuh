// kv_chunk.cuh - attention of many new tokens per sequence (pieces of prompts)
// over the paged key/value cache (kv_cache.cuh).
//
// The mathematics is kv_decode.cuh's; with many query rows per key head the
// bound is arithmetic, 4 d flops per (row, key) pair, so the products run on
// tcgen05 with the pipeline of attn_fwd.cuh: two slots of 128 query rows whose
// softmax (16 warps, two threads per row) and matrix products alternate, scores
// and outputs in TMEM, P written back to TMEM as the A operand of P V.
// Rows are (token, head of the group), the heads fastest, so that a tile of
// keys serves 256 / group tokens of all heads of its group.
//
// A tile of 128 tokens is 1 to 8 blocks, those of an e4m3 cache have to become
// 16-bit operands first, and what lies behind a sequence's end must become
// zeros.  A producer warp copies a tile's blocks: bf16 rows by TMA straight into
// the swizzled operand tiles, e4m3 rows by bulk copies into a staging tile, from
// where two converter warps take them through registers.  The converter warps
// also clean the values of tiles that not all rows see (mend_row).
// e4m3 numbers become f16, exactly (cvt: one instruction for two, where the
// bits of a bf16 with the scale in them took five), and the products are those
// of the plain numbers; queries are f16 too, scaled by a power of two per row,
// and the blocks' scales are constants of the exponent, 16 tokens at a time
// (kv_decode.cuh).
//
// The work is divided as in kv_split.cuh, one thread block per SM.
//
// Measured (d = 128, 32 query and 8 key heads): 2048 new tokens over 32768, e4m3,
// 1.16 to 1.19 ms (900 to 915 TFLOP/s; attn_fwd.cuh reaches 1,110 to 1,275 on plain
// tensors), from a bf16 cache 1.13 to 1.17 ms.  A tile takes about 4,550 cycles
// (difference of 16384 and 32768 tokens times the clocks seen), from a bf16 cache
// 3,700, but at 1.5 GHz under the power cap where e4m3 runs at 1.8; the products of
// both slots are some 2,050 of them.  The rest is waiting: a slot's softmax for its
// scores, the next scores for its P, which lies on their columns.
#pragma once

#include "attn_fwd.cuh"
#include "kv_split.cuh"

namespace sta {

template <int D, bool F8>
struct ChunkCfg {
  static constexpr int kRows = 2 * kBM;
  static constexpr int kTile = kBN;
  static constexpr int kOver = 4;                     // see kv_split.cuh
  static constexpr int kSoftWarps = 16;
  static constexpr int kWarpMma = 16;
  static constexpr int kWarpProd = 17;
  static constexpr int kWarpConv0 = 18;               // and 19
  // 20 warps, five per scheduler: 96 registers a thread, as attn_fwd.cuh has
  static constexpr int kThreads = 32 * 20;
  // e4m3 rows of a tile of keys and one of values, as they are in the cache
  static constexpr int kStageOff = FwdCfg<D>::kBarOff;
  static constexpr int kStageBytes = F8 ? kBN * D : 0;
  static constexpr int kScaleOff = kStageOff + 2 * kStageBytes;
  // Per tile: 8 groups of 16 tokens, {k scale, log2 and inverse of the v scale}.
  // Those of tile J are read until both slots' products of tile J are issued,
  // which the producer has waited for when it writes those of tile J + ring
  // depth + 1.
  static constexpr int kScaleRing = D == 128 ? 4 : 8;
  static constexpr int kMaskOff = kScaleOff + (F8 ? kScaleRing * 128 : 0);
  // pieces of the range, as the producer finds them; the other roles are fewer
  // pieces behind it than the ring is deep (each has a tile at least, and the
  // producer has waited for the scores of the tile ring depth before its last)
  static constexpr int kPieceRing = 8;
  static constexpr int kPieceOff = kMaskOff + kScaleRing * 4;   // masks: groups that were loaded
  static constexpr int kBarOff = kPieceOff + kPieceRing * 64;
  static constexpr int kSmemBytes = kBarOff + 512 + 1024;     // + 1024-byte alignment
};

// A piece of the range, in shared memory (64 bytes).
struct alignas(16) ChunkPiece {
  int n, t0;                // tiles (0: there is no further piece), first token
  int b, h;
  int row0, rows;           // first row of the item, rows
  int pos0, len;            // of the sequence
  int lo, hi;               // tokens that the item's rows see
  SeenByAll all[2];         // those that all rows of a slot see
  int whole, slot;          // the whole item; else its place in the workspace
};

// Byte offset of 16-byte chunk ch (8 columns) of row t in a [128][D] bf16
// operand tile: panels of 64 columns, 128-byte swizzle.
template <int D>
__device__ __forceinline__ uint32_t tile_chunk(int t, int ch) {
  return (ch >> 3) * FwdCfg<D>::kPanelBytes + t * 128 + (((ch & 7) ^ (t & 7)) << 4);
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z,
                                       uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

__device__ __forceinline__ uint4 lds128_at(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Box {x .., y .., z, w} of a (d, slot, head, block) view of the cache.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z, int w, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_"
      "tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w),
      "l"(policy)
      : "memory");
}

// Not all rows of the item see the whole tile at t0.
__device__ __forceinline__ bool to_clean(const SeenByAll& all, int t0) {
  return t0 < all.lo || t0 + kBN > all.hi;
}

// Generic-proxy writes of this thread become visible to the tensor core's reads.
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// max(a, b, c), NaN if one of them is.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Instruction descriptor, kind::f16 with f16 (F16) or bf16 operands, fp32 D.
template <bool F16>
__host__ __device__ constexpr uint32_t idesc_of(int M, int N, bool b_mn_major) {
  return idesc_bf16(M, N, b_mn_major) & (F16 ? ~((1u << 7) | (1u << 10)) : ~0u);
}

// S_slot = Q_slot K^T and O_slot (+)= P_slot V as in attn_fwd.cuh (whose P
// layout these share), the slot's scores at column 128 slot.
template <int D, bool F16>
__device__ __forceinline__ void chunk_issue_s(uint32_t tm, uint64_t dq, uint64_t dk, int ks,
                                              int slot) {
  using F = FwdCfg<D>;
  constexpr uint32_t kIdesc = idesc_of<F16>(kBM, kBN, false);
  const uint64_t qa = dq + ((static_cast<uint32_t>(slot) * F::kBlockBytes) >> 4);
  const uint64_t ka = dk + ((static_cast<uint32_t>(ks) * F::kBlockBytes) >> 4);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * F::kPanelBytes + (kk & 3) * 32) >> 4;
    umma_ss(tm + slot * 128, qa + off, ka + off, kIdesc, kk > 0 ? 1u : 0u);
  }
}

template <int D, bool F16, bool ACC>
__device__ __forceinline__ void chunk_issue_pv(uint32_t tm, uint64_t dv, int vs, int slot) {
  using F = FwdCfg<D>;
  constexpr uint32_t kIdesc = idesc_of<F16>(kBM, D, true);
  constexpr int G = (kBN / 16) / kSplit;
  const uint64_t va = dv + ((static_cast<uint32_t>(vs) * F::kBlockBytes) >> 4);
#pragma unroll
  for (int kk = 0; kk < kBN / 16; ++kk) {
    const uint32_t acol = (kk / G) * (kBN / kSplit) + (kk % G) * 8;
    umma_ts(tm + F::kOCol + slot * D, tm + slot * 128 + acol, va + ((kk * 16 * 128) >> 4), kIdesc,
            (ACC || kk > 0) ? 1u : 0u);
  }
}

// GROUPS: how many groups of tokens in a half tile (64) may have scales of their
// own: one with blocks of 64 tokens or more, else four.  2048 new tokens over
// 32768, d = 128: 1.16 to 1.19 ms with one (blocks of 64), 1.28 to 1.29 ms with four
// (blocks of 16 or 32; 5,280 cycles a tile).
template <int D, bool F8, int GROUPS>
__global__ void __launch_bounds__(ChunkCfg<D, F8>::kThreads, 1)
    kv_chunk_kernel(const __grid_constant__ CUtensorMap tmap_k,
                    const __grid_constant__ CUtensorMap tmap_v, const AttendParams p) {
  using C = ChunkCfg<D, F8>;
  using F = FwdCfg<D>;
  constexpr int KST = F::kKStages, VST = F::kVStages;
  static_assert(KST == VST && VST <= 4, "one ring depth for both operands");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* q_full = bars;            // [2] a slot's query rows are in shared memory
  uint64_t* k_full = q_full + 2;
  uint64_t* k_empty = k_full + KST;
  uint64_t* v_full = k_empty + KST;
  uint64_t* v_empty = v_full + VST;
  uint64_t* s_full = v_empty + VST;   // [2] scores of a slot's tile in TMEM
  uint64_t* p_full = s_full + 2;      // [2] its P in TMEM
  uint64_t* o_full = p_full + 2;      // [2] all products of a slot's piece
  uint64_t* sc_full = o_full + 2;     // [ring] scales of a tile
  uint64_t* pc_full = sc_full + C::kScaleRing;   // [ring] a piece
  uint64_t* raw_full = pc_full + C::kPieceRing;   // e4m3: [2] staged keys, values
  uint64_t* raw_empty = raw_full + 2;
  uint64_t* land = raw_full;          // bf16: [VST] values that are to be cleaned
  uint64_t* mma_done = raw_full + 4;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* dropped = abort_flag + 1;   // infinities or NaN left out of a product

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < KST; ++i) {
      mbar_init(&k_full[i], F8 ? 2 : 1);              // converters, or the producer's copies
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 2);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], C::kSoftWarps / 2);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], C::kSoftWarps / 2);
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < C::kScaleRing; ++i) mbar_init(&sc_full[i], 1);
    for (int i = 0; i < C::kPieceRing; ++i) mbar_init(&pc_full[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&raw_full[i], F8 && i >= 2 ? 2 : 1);
    mbar_init(mma_done, 1);
    *abort_flag = error_raised() ? 1 : 0;
    *dropped = 0;
    fence_mbar_init();
  }
  if (warp == C::kWarpMma) tmem_alloc(tmem_holder, F::kTmemCols);
  tc_fence_before();
  const KvRange range = kv_range<D, C::kRows, C::kTile, C::kOver, C::kThreads>(p);   // synchronises
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const bool skip = *abort_flag != 0;
  const uint32_t smem_q = smem_u32(smem + F::kQOff);
  const uint32_t smem_k = smem_u32(smem + F::kKOff);
  const uint32_t smem_v = smem_u32(smem + F::kVOff);
  const ChunkPiece* pieces = reinterpret_cast<const ChunkPiece*>(smem + C::kPieceOff);
  // the np-th piece, or null when a wait gave up
  auto wait_piece = [&](int np) -> const ChunkPiece* {
    const int i = np % C::kPieceRing;
    return mbar_wait_warp(&pc_full[i], (np / C::kPieceRing) & 1, abort_flag) ? pieces + i : nullptr;
  };

  if (skip) {
    // a wait gave up earlier: nothing is computed
  } else if (warp == C::kWarpProd) {
    // ------------------------------------------------------------ producer
    // Lane l < 128 / block has the tile's block l.
    const KvLayout& c = p.c;
    const int block = 1 << c.shift, blocks = kBN >> c.shift;
    const uint32_t gmask = (1u << (block >> 4)) - 1u; // a block's groups
    volatile uint32_t* masks = reinterpret_cast<volatile uint32_t*>(smem + C::kMaskOff);
    const uint64_t pol = policy_evict_last();         // other items read the same keys
    int jt = 0;                                       // tiles so far: ring positions
    bool ok = true;
    KvPiece pc;
    pc.start(range);
    for (int np = 0; ok; ++np) {
      const bool more = pc.next<C::kRows, C::kTile, C::kOver>(p, range);
      const ItemRange& r = pc.r;
      const int n = more ? pc.t1 - pc.t0 : 0, base = more ? pc.tok0<C::kTile>() : 0;
      const int last_row = pc.row0 + r.rows - 1;
      if (lane == 0) {
        ChunkPiece w;
        w.n = n;
        if (more) {
          w.t0 = base;
          w.b = pc.b;
          w.h = pc.h;
          w.row0 = pc.row0;
          w.rows = r.rows;
          w.pos0 = r.pos0;
          w.len = r.len;
          w.lo = r.lo;
          w.hi = r.hi;
          for (int i = 0; i < 2; ++i)
            w.all[i] = seen_by_all(p, r, min(pc.row0 + i * kBM, last_row),
                                   min(pc.row0 + i * kBM + kBM - 1, last_row));
          w.whole = pc.whole();
          w.slot = static_cast<int>(pc.slot());
          pc.leave<C::kOver>(p, range);
        }
        *reinterpret_cast<ChunkPiece*>(smem + C::kPieceOff + np % C::kPieceRing * 64) = w;
        mbar_arrive(&pc_full[np % C::kPieceRing]);
      }
      __syncwarp();
      if (!more) break;
      const int* table = c.table + static_cast<long long>(pc.b) * c.width;
      // those of both slots: the later rows' lower end, the earlier ones' upper end
      const SeenByAll all = seen_by_all(p, r, pc.row0, last_row);
      auto fetch_id = [&](int j) {                    // -2: nothing to load
        const int t = base + j * kBN + (lane << c.shift);
        return lane < blocks && j < n && t < r.hi && t + block > r.lo
                   ? __ldg(table + (t >> c.shift)) : -2;
      };
      int id_next = fetch_id(0);
      for (int j = 0; ok && j < n; ++j) {
        const int J = jt + j, st = J % KST, ring = J % C::kScaleRing;
        const int id = id_next;
        id_next = fetch_id(j + 1);
        const bool good = id >= 0 && id < c.num_blocks;
        if (!good && id != -2) kv_bad_index();
        const uint32_t count = __popc(__ballot_sync(0xffffffffu, good));
        const uint32_t here =
            __reduce_or_sync(0xffffffffu, good ? gmask << (lane * (block >> 4)) : 0u);
        const uint8_t* ksrc = c.k + static_cast<long long>(good ? id : 0) * c.k_block +
                              pc.h * c.k_head;
        const uint8_t* vsrc = c.v + static_cast<long long>(good ? id : 0) * c.v_block +
                              pc.h * c.v_head;
        if constexpr (F8) {
          const long long at = static_cast<long long>(good ? id : 0) * c.hkv + pc.h;
          const float sk = __ldg(c.k_scale + at), sv = __ldg(c.v_scale + at);
          const uint32_t bytes = D << c.shift;
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            if (J > 0 && !mbar_wait_warp(&raw_empty[o], (J - 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            if (lane == 0) {
              if (o == 0) masks[ring] = here;
              mbar_arrive_expect_tx(&raw_full[o], count * bytes);
            }
            __syncwarp();
            if (good)
              bulk_load(smem + C::kStageOff + o * C::kStageBytes + lane * bytes, o ? vsrc : ksrc,
                        bytes, &raw_full[o]);
          }
          const KvScale x = kv_scale(good ? sk : 1.f, good ? sv : 1.f);
          if (lane < blocks) {
            const uint32_t to = smem_u32(smem + C::kScaleOff) + ring * 128 + lane * block;
            for (int g = 0; g < block >> 4; ++g)
              sts128(to + g * 16, __float_as_uint(x.k), __float_as_uint(x.log2_v),
                     __float_as_uint(x.inv_v), 0u);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[ring]);
        } else {
          auto issue = [&](int o, uint64_t* bar) {
            if (lane == 0) mbar_arrive_expect_tx(bar, count * (D * 2u << c.shift));
            __syncwarp();
            if (good) {
              uint8_t* dst = smem + (o ? F::kVOff : F::kKOff) + st * F::kBlockBytes +
                             lane * block * 128;
#pragma unroll
              for (int pn = 0; pn < F::kPanels; ++pn)
                tma_load_4d(dst + pn * F::kPanelBytes, o ? &tmap_v : &tmap_k, bar, pn * 64, 0,
                            pc.h, id, pol);
            }
          };
          ok = J < KST || mbar_wait_warp(&k_empty[st], ((J / KST) - 1) & 1, abort_flag);
          if (!ok) break;
          issue(0, &k_full[st]);
          ok = J < VST || mbar_wait_warp(&v_empty[st], ((J / VST) - 1) & 1, abort_flag);
          if (!ok) break;
          if (lane == 0) masks[ring] = here;
          if (to_clean(all, base + j * kBN)) {
            issue(1, &land[st]);
          } else {
            issue(1, &v_full[st]);
            if (lane == 0) mbar_arrive(&v_full[st]);
          }
        }
      }
      jt += n;
    }
    if (!ok) {
      // a wait gave up: no copy may be in flight when the block ends
      const uint64_t t = globaltimer_ns();
      while (globaltimer_ns() - t < 1000000ull) {
      }
    }
  } else if (warp >= C::kWarpConv0) {
    // ------------------------------------------------------------ converters
    const int half = warp - C::kWarpConv0;            // tokens 64 half .. of a tile
    volatile uint32_t* masks = reinterpret_cast<volatile uint32_t*>(smem + C::kMaskOff);
    int jt = 0;
    uint32_t dirty = 0;                               // bf16: phase of each land barrier
    bool ok = true;
    for (int np = 0; ok; ++np) {
      const ChunkPiece* w = wait_piece(np);
      if (w == nullptr || w->n == 0) break;
      const int n = w->n, base = w->t0, lo = w->lo, hi = w->hi;
      const SeenByAll all{w->all[1].lo, w->all[0].hi};
      if constexpr (F8) {
        // A lane has 16 numbers of a row.  At d = 128 lanes 4 .. 7 of every eight
        // have the other row of a pair: their 16-byte stores then fall on other
        // chunk positions than those of lanes 0 .. 3, whose panel they do not share.
        constexpr int kLanes = D / 16;
        constexpr int kRowsPer = 32 / kLanes, kSteps = 16 / kRowsPer;
        const int ch = lane % kLanes;
        const int lrow = D == 128 ? (lane / kLanes) ^ ((lane >> 2) & 1) : lane / kLanes;
        const uint32_t src0 = smem_u32(smem + C::kStageOff) + (64 * half + lrow) * D + ch * 16;
        // chunk positions repeat every 8 rows
        uint32_t to[kSteps < 2 ? 1 : 2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (i < (kSteps < 2 ? 1 : 2))
              to[i][e] = tile_chunk<D>(64 * half + (i * kRowsPer + lrow) % 8, 2 * ch + e);
        for (int j = 0; ok && j < n; ++j) {
          const int J = jt + j, st = J % KST;
          const int t0 = base + j * kBN;
#pragma unroll
          for (int o = 0; o < 2; ++o) {               // keys, values
            ok = mbar_wait_warp(&raw_full[o], J & 1, abort_flag) &&
                 (J < KST || mbar_wait_warp(o ? &v_empty[st] : &k_empty[st], ((J / KST) - 1) & 1,
                                            abort_flag));
            if (!ok) break;
            const uint32_t here = masks[J % C::kScaleRing];
            const bool check = here != 0xffu || t0 < lo || t0 + kBN > hi ||
                               (o == 1 && to_clean(all, t0));
            const uint32_t src = src0 + o * C::kStageBytes;
            const uint32_t dst = (o ? smem_v : smem_k) + st * F::kBlockBytes;
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
              uint4 raw[kSteps];
#pragma unroll
              for (int i = 0; i < kSteps; ++i) raw[i] = lds128_at(src + (16 * g + i * kRowsPer) * D);
              if (check) {
                // tokens outside the sequence, and NaN among values that some
                // rows do not see
                bool any = false;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                  const int t = t0 + 64 * half + 16 * g + i * kRowsPer + lrow;
                  const bool in = ((here >> (4 * half + g)) & 1) && t >= lo && t < hi;
                  if (!in) raw[i] = make_uint4(0u, 0u, 0u, 0u);
                  if (o == 1) {
                    raw[i].x = drop_nonfinite<true>(raw[i].x, any);
                    raw[i].y = drop_nonfinite<true>(raw[i].y, any);
                    raw[i].z = drop_nonfinite<true>(raw[i].z, any);
                    raw[i].w = drop_nonfinite<true>(raw[i].w, any);
                  }
                }
                if (any) *dropped = 1;
              }
#pragma unroll
              for (int i = 0; i < kSteps; ++i) {
                const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                uint32_t y[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  y[2 * e] = e4m3x2_to_f16x2(w[e] & 0xffffu);
                  y[2 * e + 1] = e4m3x2_to_f16x2(w[e] >> 16);
                }
                const uint32_t at = dst + (16 * g + (i * kRowsPer) / 8 * 8) * 128;
                const int x = kSteps < 2 ? 0 : (kRowsPer < 8 ? i % 2 : 0);
                sts128(at + to[x][0], y[0], y[1], y[2], y[3]);
                sts128(at + to[x][1], y[4], y[5], y[6], y[7]);
              }
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(o ? &v_full[st] : &k_full[st]);
              mbar_arrive(&raw_empty[o]);
            }
          }
        }
      } else {
        for (int j = 0; ok && j < n; ++j) {
          // A tile that some rows do not see, or not all of it: its values
          // without infinities and NaN, and zeros where there is no token.
          const int J = jt + j, st = J % VST;
          const int t0 = base + j * kBN;
          if (!to_clean(all, t0)) continue;
          ok = mbar_wait_warp(&land[st], (dirty >> st) & 1, abort_flag);
          if (!ok) break;
          dirty ^= 1u << st;
          const uint32_t here = masks[J % C::kScaleRing];
          bool any = false;
#pragma unroll 4
          for (int i = lane; i < 64 * D / 8; i += 32) {
            const int row = 64 * half + i / (D / 8);
            const uint32_t at = smem_v + st * F::kBlockBytes + tile_chunk<D>(row, i % (D / 8));
            const bool in = ((here >> (row >> 4)) & 1) && t0 + row >= lo && t0 + row < hi;
            const uint4 x = lds128_at(at);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            uint32_t y[4];
            bool hit = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = drop_nonfinite<false>(w[e], hit);
            any = any || (hit && in);
            if (!in) sts128(at, 0u, 0u, 0u, 0u);
            else if (hit) sts128(at, y[0], y[1], y[2], y[3]);
          }
          if (any) *dropped = 1;
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_full[st]);
        }
      }
      jt += n;
    }
  } else if (warp == C::kWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t tm = warp_uniform(tmem);
    const uint64_t dq = sdesc_sw128(warp_uniform(smem_q), 16, 1024);
    const uint64_t dk = sdesc_sw128(warp_uniform(smem_k), 16, 1024);
    const uint64_t dv = sdesc_sw128(warp_uniform(smem_v), F::kPanelBytes, 1024);
    int jt = 0;
    bool ok = true;
    for (int np = 0; ok; ++np) {
      const ChunkPiece* w = wait_piece(np);
      const int n = w != nullptr ? w->n : 0;
      if (n == 0) break;
      ok = mbar_wait_warp(&k_full[jt % KST], (jt / KST) & 1, abort_flag) &&
           mbar_wait_warp(&q_full[0], np & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        chunk_issue_s<D, F8>(tm, dq, dk, jt % KST, 0);
        umma_commit(&s_full[0]);
      }
      __syncwarp();
      ok = mbar_wait_warp(&q_full[1], np & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        chunk_issue_s<D, F8>(tm, dq, dk, jt % KST, 1);
        umma_commit(&s_full[1]);
        umma_commit(&k_empty[jt % KST]);
      }
      __syncwarp();
      for (int j = 0; j < n; ++j) {
        const int J = jt + j, vs = J % VST, ksn = (J + 1) % KST;
        ok = mbar_wait_warp(&v_full[vs], (J / VST) & 1, abort_flag) &&
             mbar_wait_warp(&p_full[0], J & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          if (j > 0) chunk_issue_pv<D, F8, true>(tm, dv, vs, 0);
          else chunk_issue_pv<D, F8, false>(tm, dv, vs, 0);
        }
        __syncwarp();
        if (j + 1 < n) {
          ok = mbar_wait_warp(&k_full[ksn], ((J + 1) / KST) & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            chunk_issue_s<D, F8>(tm, dq, dk, ksn, 0);
            umma_commit(&s_full[0]);
          }
        } else if (elect_one()) {
          umma_commit(&o_full[0]);
        }
        __syncwarp();
        ok = mbar_wait_warp(&p_full[1], J & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          if (j > 0) chunk_issue_pv<D, F8, true>(tm, dv, vs, 1);
          else chunk_issue_pv<D, F8, false>(tm, dv, vs, 1);
          if (j + 1 < n) {
            chunk_issue_s<D, F8>(tm, dq, dk, ksn, 1);
            umma_commit(&s_full[1]);
            umma_commit(&k_empty[ksn]);
          } else {
            umma_commit(&o_full[1]);
          }
          umma_commit(&v_empty[vs]);
        }
        __syncwarp();
      }
      jt += n;
    }
    // No MMA may still run when TMEM is released.
    if (elect_one()) umma_commit(mma_done);
    __syncwarp();
    mbar_wait_drain(mma_done, 0);
  } else {
    // ------------------------------------------------------------ softmax
    // Warp w serves slot w / 8, TMEM lane quarter w % 4 and, in it, 16 rows;
    // lanes t and t + 16 share a row, each with half of its columns.
    constexpr int kCols = kBN / kSplit;
    constexpr int kOCols = D / kSplit;
    const int slot = warp / 8;
    const int half = lane >> 4;
    const int lr = (warp & 3) * 32 + ((warp / 4) & 1) * 16 + (lane & 15);   // row in the slot
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32 + ((warp / 4) & 1) * 16) << 16;
    const uint32_t t_s = tmem + lane_off + (slot ? 128u : 0u);
    const uint32_t t_o = tmem + lane_off + F::kOCol + (slot ? D : 0);
    float sl2 = p.scale_log2;  // e4m3: times what the row's queries were divided by
    int jt = 0;
    // Loads the row's half of the queries of a piece.  Rows past the last one
    // are zeros that see what the last row sees.
    auto load_q = [&](const ChunkPiece& w, uint4 x[kOCols / 8]) {
      const bool live = slot * kBM + lr < w.rows;
      const int row = w.row0 + (live ? slot * kBM + lr : w.rows - 1);
      const int t = row / p.group, g = row - t * p.group;
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + w.b * p.qs.b + (static_cast<long long>(w.h) * p.group + g) * p.qs.h + t * p.qs.s +
          half * kOCols);
#pragma unroll
      for (int e = 0; e < kOCols / 8; ++e) x[e] = live ? src[e] : make_uint4(0u, 0u, 0u, 0u);
    };
    // ... and hands them to the tensor core.
    auto store_q = [&](uint4 x[kOCols / 8]) {
      if constexpr (F8) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < kOCols / 8; ++e)
          m = fmaxf(m, fmaxf(fmaxf(bf16x2_max_abs(x[e].x), bf16x2_max_abs(x[e].y)),
                             fmaxf(bf16x2_max_abs(x[e].z), bf16x2_max_abs(x[e].w))));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        const QueryScale qs = query_scale<0>(m);
        sl2 = p.scale_log2 * qs.up;
#pragma unroll
        for (int e = 0; e < kOCols / 8; ++e)
          x[e] = make_uint4(bf16x2_to_f16x2(x[e].x, qs.down), bf16x2_to_f16x2(x[e].y, qs.down),
                            bf16x2_to_f16x2(x[e].z, qs.down), bf16x2_to_f16x2(x[e].w, qs.down));
      } else {
#pragma unroll
        for (int e = 0; e < kOCols / 8; ++e)
          x[e] = make_uint4(bf16x2_inf_to_nan(x[e].x), bf16x2_inf_to_nan(x[e].y),
                            bf16x2_inf_to_nan(x[e].z), bf16x2_inf_to_nan(x[e].w));
      }
#pragma unroll
      for (int e = 0; e < kOCols / 8; ++e)
        sts128(smem_q + slot * F::kBlockBytes + tile_chunk<D>(lr, half * (kOCols / 8) + e), x[e].x,
               x[e].y, x[e].z, x[e].w);
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[slot]);
    };
    const ChunkPiece* w = wait_piece(0);
    bool ok = w != nullptr;
    int n = ok ? w->n : 0;
    if (n > 0) {
      uint4 x[kOCols / 8];
      load_q(*w, x);
      store_q(x);
    }
    for (int np = 0; n > 0; ++np) {
      const int rr = slot * kBM + lr;                 // row of the item
      const int pos = w->pos0 + (w->row0 + min(rr, w->rows - 1)) / p.group;
      int t0 = w->t0;
      float m_run = -INFINITY;   // running max, log2 units of the scaled scores
      float l_run = 0.f;         // this thread's part of the row sum
      for (int j = 0; j < n; ++j, t0 += kBN) {
        uint32_t sc_at = 0;
        KvScale one{sl2, 0.f, 1.f};
        // What multiplies a score: the key scale and the row's factor.  Masked scores
        // are -inf already, so it must not be 0 where both are small (keys of zeros
        // have the scale 2^-64, a row of zeros the factor 2^-123): at the smallest
        // normal number it still makes nothing of any score.
        auto scale_of = [&](const uint4& x) {
          return KvScale{fmaxf(__uint_as_float(x.x) * sl2, 1.1754943508222875e-38f),
                         __uint_as_float(x.y), __uint_as_float(x.z)};
        };
        if constexpr (F8) {
          const int ring = (jt + j) % C::kScaleRing;
          if (!mbar_wait_warp(&sc_full[ring], ((jt + j) / C::kScaleRing) & 1, abort_flag)) {
            ok = false;
            break;
          }
          sc_at = smem_u32(smem + C::kScaleOff) + ring * 128 + half * 64;
          if constexpr (GROUPS == 1) {
            one = scale_of(lds128_at(sc_at));
          }
        }
        if (!mbar_wait_warp(&s_full[slot], (jt + j) & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        float s[kCols];
        auto load_scores = [&]() {
          uint32_t sr[kCols];
#pragma unroll
          for (int cc = 0; cc < kCols / 32; ++cc) tmem_ld_half32<kCols>(t_s + cc * 32, sr + cc * 32);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < kCols; ++c) s[c] = __uint_as_float(sr[c]);
          if (to_clean(w->all[slot], t0)) {
            const int hi = pos + 1 - t0 - half * kCols;
            const int lo = p.window > 0 ? hi - p.window : -kBN;
#pragma unroll
            for (int c = 0; c < kCols; ++c)
              if (c < lo || c >= hi) s[c] = -INFINITY;
          }
        };
        load_scores();
        // group g of 16 columns: x = s mul + add, without the reference
        constexpr int kGroups = GROUPS, kPerGroup = kCols / kGroups;
        auto group = [&](int g) {
          if constexpr (GROUPS == 1) {
            return one;
          } else {
            return scale_of(lds128_at(sc_at + g * 16));
          }
        };
        uint32_t pk[kCols / 2];
        auto exp_pack = [&](float ref, auto with_max, float& mx) {
          const float neg = (ref == -INFINITY) ? 0.f : kLift<F8> - ref;
          float sum = 0.f;
          mx = -INFINITY;
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const KvScale k = group(g);
            const float2 mul = make_float2(k.k, k.k);
            const float2 add = make_float2(neg + k.log2_v, neg + k.log2_v);
            float2 ls = make_float2(0.f, 0.f);
            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
            for (int c = g * kPerGroup; c < (g + 1) * kPerGroup; c += 2) {
              if constexpr (decltype(with_max)::value) {
                if ((c & 2) == 0) m0 = fmax3_nan(m0, s[c], s[c + 1]);
                else m1 = fmax3_nan(m1, s[c], s[c + 1]);
              }
              const float2 x = __ffma2_rn(make_float2(s[c], s[c + 1]), mul, add);
              float2 e;
              if (exp2_on_fma(c / 2)) e = exp2_fma2(x);
              else e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
              ls = __fadd2_rn(ls, e);
              pk[c / 2] = F8 ? pack_f16x2(e.x, e.y) : pack_bf16x2(e.x, e.y);
            }
            sum = F8 ? fmaf(ls.x + ls.y, k.inv_v, sum) : ls.x + ls.y;
            if constexpr (decltype(with_max)::value) {
              const float m = fmax3_nan(m0, m1, m1);
              mx = F8 ? fmax3_nan(mx, fmaf(m, k.k, k.log2_v), mx) : m * k.k;
            }
          }
          return sum;
        };
        auto own_max = [&]() {
          float mx = -INFINITY;
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            const KvScale k = group(g);
            float mq[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int c = g * kPerGroup; c < (g + 1) * kPerGroup; c += 2)
              mq[(c >> 1) & 1] = fmax3_nan(mq[(c >> 1) & 1], s[c], s[c + 1]);
            const float m = fmax3_nan(mq[0], mq[1], mq[1]);
            mx = F8 ? fmax3_nan(mx, fmaf(m, k.k, k.log2_v), mx) : m * k.k;
          }
          return mx;
        };
        // reference of the exponent: see attn_fwd.cuh
        using kNoMax = std::integral_constant<bool, false>;
        using kWithMax = std::integral_constant<bool, true>;
        float mx = -INFINITY;
        float lsum;
        float alpha = 1.f;
        bool resc;
        auto raise_ref = [&]() {
          const float other = __shfl_xor_sync(0xffffffffu, mx, 16);
          mx = fmax3_nan(mx, other, other);
          // a score that is NaN or +inf: the row is NaN (not every exponential
          // above would say so)
          if (!(mx < INFINITY)) l_run = __int_as_float(0x7fffffff);
          resc = mx > m_run + 8.0f;
          if (resc) {
            alpha = fast_exp2(m_run - mx);
            m_run = mx;
            l_run *= alpha;
          }
        };
        if (__any_sync(0xffffffffu, m_run == -INFINITY)) {
          mx = own_max();
          raise_ref();
          lsum = exp_pack(m_run, kNoMax{}, mx);
        } else {
          lsum = exp_pack(m_run, kWithMax{}, mx);
          raise_ref();
          if (__any_sync(0xffffffffu, resc)) {
            load_scores();
            lsum = exp_pack(m_run, kNoMax{}, mx);
          }
        }
#pragma unroll
        for (int cc = 0; cc < kCols / 32; ++cc) tmem_st_half16<kCols>(t_s + cc * 16, pk + cc * 16);
        l_run += lsum;
        if (j > 0 && __any_sync(0xffffffffu, resc)) {
#pragma unroll
          for (int cc = 0; cc < kOCols / 32; ++cc) {
            uint32_t o[32];
            tmem_ld_half32<kOCols>(t_o + cc * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st_half32<kOCols>(t_o + cc * 32, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[slot]);
      }
      jt += n;
      if (!ok) break;
      // The next piece's queries are loaded before the last product is there
      // and handed over as soon as this piece's products no longer read the
      // old ones: its first scores are computed while O is written out.
      const ChunkPiece* next = wait_piece(np + 1);
      const int n_next = next != nullptr ? next->n : 0;
      uint4 qx[kOCols / 8];
      if (n_next > 0) load_q(*next, qx);
      if (next == nullptr || !mbar_wait_warp(&o_full[slot], np & 1, abort_flag)) break;
      tc_fence_after();
      if (n_next > 0) store_q(qx);
      l_run += __shfl_xor_sync(0xffffffffu, l_run, 16);
      const bool live = rr < w->rows, whole = w->whole != 0;
      if (whole) l_run = final_sum(l_run, pos);
      const long long at = static_cast<long long>(w->slot) * C::kRows + rr;
      const float inv = whole ? (l_run == 0.f ? 0.f : 1.f / l_run) : 1.f;
      const int row = w->row0 + rr, t = row / p.group, g = row - t * p.group;
      __nv_bfloat16* out = p.out + w->b * p.os.b +
                           (static_cast<long long>(w->h) * p.group + g) * p.os.h + t * p.os.s +
                           half * kOCols;
      float* part = p.part_o + at * D + half * kOCols;
      if (*dropped == 0) {
#pragma unroll
        for (int cc = 0; cc < kOCols / 32; ++cc) {
          uint32_t o[32];
          tmem_ld_half32<kOCols>(t_o + cc * 32, o);
          tmem_wait_ld();
          if (live && whole) {
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16x2(__uint_as_float(o[8 * v4 + 2 * e]) * inv,
                                   __uint_as_float(o[8 * v4 + 2 * e + 1]) * inv);
              reinterpret_cast<uint4*>(out)[cc * 4 + v4] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (live) {
#pragma unroll
            for (int v4 = 0; v4 < 8; ++v4)
              reinterpret_cast<uint4*>(part)[cc * 8 + v4] =
                  make_uint4(o[4 * v4], o[4 * v4 + 1], o[4 * v4 + 2], o[4 * v4 + 3]);
          }
        }
      } else {
        // the same with what was left out of the products (for any piece of
        // this thread block), through local memory: rare
        float o[kOCols];
        for (int cc = 0; cc < kOCols / 32; ++cc) {
          uint32_t x[32];
          tmem_ld_half32<kOCols>(t_o + cc * 32, x);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[cc * 32 + e] = __uint_as_float(x[e]);
        }
        for (int e = 0; live && e < kOCols; e += 4) {
          float4 x = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          x = mend_row<D, F8, C::kTile>(p, MendItem{w->b, w->h, w->pos0, w->len},
                                        SeenByAll{w->all[1].lo, w->all[0].hi}, row, w->t0,
                                        n * kBN, half * kOCols + e, x);
          if (whole)
            *reinterpret_cast<uint2*>(out + e) =
                make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
          else
            *reinterpret_cast<float4*>(part + e) = x;
        }
      }
      if (live && half == 0) {
        if (whole) write_lse(p, w->b, w->h, row, m_run, l_run, kLift<F8>);
        else *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m_run, l_run);
      }
      // the next piece's first product overwrites O only after this slot's next P
      tc_fence_before();
      w = next;
      n = n_next;
    }
  }

  if (!skip) kv_empty_rows<D, C::kRows, C::kThreads>(p);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == C::kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, F::kTmemCols);
  }
}

}  // namespace sta
