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
// zeros.  Three loader warps do all of that, 16 tokens at a time: bf16 rows by
// TMA straight into the swizzled operand tiles, e4m3 rows by bulk copies into a
// staging tile and from there through registers.
// e4m3 numbers become f16, exactly (cvt: one instruction for two, where the
// bits of a bf16 with the scale in them took five), and the products are those
// of the plain numbers; queries are f16 too, scaled by a power of two per row,
// and the blocks' scales are constants of the exponent, 16 tokens at a time
// (kv_decode.cuh).
//
// The work is divided as in kv_split.cuh, one thread block per SM.
#pragma once

#include "attn_fwd.cuh"
#include "kv_split.cuh"

namespace sta {

template <int D, bool F8>
struct ChunkCfg {
  static constexpr int kRows = 2 * kBM;
  static constexpr int kTile = kBN;
  static constexpr int kSoftWarps = 16;
  static constexpr int kWarpMma = 16;
  static constexpr int kLoadWarps = 3;
  static constexpr int kWarpLoad0 = 17;
  // 20 warps, five per scheduler: 96 registers a thread, as attn_fwd.cuh has
  static constexpr int kThreads = 32 * (kSoftWarps + 1 + kLoadWarps);
  // e4m3 rows of a tile of keys and one of values, as they are in the cache
  static constexpr int kStageOff = FwdCfg<D>::kBarOff;
  static constexpr int kStageBytes = F8 ? kBN * D : 0;
  static constexpr int kScaleOff = kStageOff + 2 * kStageBytes;
  // scales of the tiles that some softmax warp may still need: those of tile J
  // are read until both slots' products of tile J are issued, which a loader
  // that writes those of tile J + ring depth + 1 has waited for
  static constexpr int kScaleRing = F8 ? 8 : 0;
  static constexpr int kBarOff = kScaleOff + kScaleRing * 128;
  static constexpr int kSmemBytes = kBarOff + 512 + 1024;     // + 1024-byte alignment
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

template <int D, bool F8>
__global__ void __launch_bounds__(ChunkCfg<D, F8>::kThreads, 1)
    kv_chunk_kernel(const __grid_constant__ CUtensorMap tmap_k,
                    const __grid_constant__ CUtensorMap tmap_v, const AttendParams p) {
  using C = ChunkCfg<D, F8>;
  using F = FwdCfg<D>;
  constexpr int KST = F::kKStages, VST = F::kVStages;
  static_assert(KST == VST, "one ring depth for both operands");
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
  uint64_t* land = o_full + 2;        // [2][3] a loader warp's own copies: keys, values
  uint64_t* sc_full = land + 6;       // [ring] scales of a tile
  uint64_t* mma_done = sc_full + C::kScaleRing;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* dropped = abort_flag + 1;   // infinities or NaN left out of a product

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < KST; ++i) {
      mbar_init(&k_full[i], C::kLoadWarps);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], C::kLoadWarps);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], C::kSoftWarps / 2);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], C::kSoftWarps / 2);
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < 6; ++i) mbar_init(&land[i], 1);
    for (int i = 0; i < C::kScaleRing; ++i) mbar_init(&sc_full[i], 1);
    mbar_init(mma_done, 1);
    *abort_flag = error_raised() ? 1 : 0;
    *dropped = 0;
    fence_mbar_init();
  }
  if (warp == C::kWarpMma) tmem_alloc(tmem_holder, F::kTmemCols);
  tc_fence_before();
  const KvRange range = kv_range<D, C::kRows, C::kTile, C::kThreads>(p);   // synchronises
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const bool skip = *abort_flag != 0;
  const uint32_t smem_q = smem_u32(smem + F::kQOff);
  const uint32_t smem_k = smem_u32(smem + F::kKOff);
  const uint32_t smem_v = smem_u32(smem + F::kVOff);
  KvPiece pc;
  pc.start(range);

  if (skip) {
    // a wait gave up earlier: nothing is computed
  } else if (warp >= C::kWarpLoad0) {
    // ------------------------------------------------------------ loaders
    // A tile is 8 groups of 16 tokens, each inside one block.  Every loader
    // warp has every third group of a tile, for the values shifted by one: 6, 5
    // and 5 of a tile's 16.  Lane g < 8 holds what is known of group g.
    const int lw = warp - C::kWarpLoad0;
    const KvLayout& c = p.c;
    const int block_mask = (1 << c.shift) - 1;
    int jt = 0;                                       // tiles so far: ring positions
    uint32_t cleaned = 0;                             // phase of this warp's land barrier
    bool ok = true;
    while (ok && pc.next<C::kRows, C::kTile>(p, range)) {
      const ItemRange& r = pc.r;
      const int n = pc.t1 - pc.t0, base = pc.tok0<C::kTile>();
      const int* table = c.table + static_cast<long long>(pc.b) * c.width;
      const SeenByAll all = seen_by_all(p, r, pc.row0, pc.row0 + r.rows - 1);
      auto fetch_id = [&](int j) {                    // -2: nothing to load
        const int t = base + j * kBN + 16 * lane;
        return lane < 8 && j < n && t < r.hi && t + 16 > r.lo ? __ldg(table + (t >> c.shift)) : -2;
      };
      auto check_id = [&](int id) {
        const bool good = id >= 0 && id < c.num_blocks;
        if (!good && id != -2) kv_bad_index();
        return good;
      };
      int id = fetch_id(0);
      if constexpr (F8) {
        constexpr int kGroup = 16 * D;                // bytes of a group in the cache
        constexpr int kLanes = D / 16;                // lanes per row
        constexpr int kRowsPer = 32 / kLanes;         // rows of a warp's access
        const int lrow = lane / kLanes, ch = lane % kLanes;
        // copies this warp's groups of operand o into its place in the staging tile
        auto issue = [&](int o, int j, bool good) {
          const bool mine = good && lane < 8 && lane % 3 == (lw + o) % 3;
          const int count = __popc(__ballot_sync(0xffffffffu, mine));
          if (lane == 0) mbar_arrive_expect_tx(&land[o * 3 + lw], count * kGroup);
          __syncwarp();
          if (mine) {
            const int in = (base + j * kBN + 16 * lane) & block_mask;
            const uint8_t* src = (o ? c.v + id * c.v_block + pc.h * c.v_head
                                    : c.k + id * c.k_block + pc.h * c.k_head) +
                                 static_cast<long long>(in) * D;
            bulk_load(smem + C::kStageOff + o * C::kStageBytes + lane * kGroup, src, kGroup,
                      &land[o * 3 + lw]);
          }
        };
        bool good = check_id(id);
        float sk = 1.f, sv = 1.f;
        auto fetch_scale = [&]() {
          sk = good ? __ldg(c.k_scale + static_cast<long long>(id) * c.hkv + pc.h) : 1.f;
          sv = good ? __ldg(c.v_scale + static_cast<long long>(id) * c.hkv + pc.h) : 1.f;
        };
        issue(0, 0, good);
        issue(1, 0, good);
        fetch_scale();
        for (int j = 0; ok && j < n; ++j) {
          const int J = jt + j, st = J % KST;
          const int t0 = base + j * kBN;
          const bool part = t0 < all.lo || t0 + kBN > all.hi;
          const bool edge = t0 < r.lo || t0 + kBN > r.hi;
          const uint32_t here = __ballot_sync(0xffffffffu, good);
          const int id_next = fetch_id(j + 1);
#pragma unroll
          for (int o = 0; o < 2; ++o) {               // keys, values
            if (!mbar_wait_warp(&land[o * 3 + lw], J & 1, abort_flag) ||
                (J >= KST &&
                 !mbar_wait_warp(o ? &v_empty[st] : &k_empty[st], ((J / KST) - 1) & 1,
                                 abort_flag))) {
              ok = false;
              break;
            }
            if (o == 0 && lw == 0) {
              const uint32_t at = smem_u32(smem + C::kScaleOff) + (J % C::kScaleRing) * 128;
              const KvScale x = kv_scale(sk, sv);
              if (lane < 8)
                sts128(at + lane * 16, __float_as_uint(x.k), __float_as_uint(x.log2_v),
                       __float_as_uint(x.inv_v), 0u);
              __syncwarp();
              if (lane == 0) mbar_arrive(&sc_full[J % C::kScaleRing]);
            }
            const uint32_t dst = (o ? smem_v : smem_k) + st * F::kBlockBytes;
            const uint32_t src = smem_u32(smem + C::kStageOff + o * C::kStageBytes);
            for (int g = (lw + o) % 3; g < 8; g += 3) {
              const bool there = (here >> g) & 1;
              uint4 raw[16 / kRowsPer];
#pragma unroll
              for (int i = 0; i < 16 / kRowsPer; ++i) {
                const int row = 16 * g + i * kRowsPer + lrow;
                raw[i] = lds128_at(src + row * D + ch * 16);
                if (!there || (edge && (t0 + row < r.lo || t0 + row >= r.hi)))
                  raw[i] = make_uint4(0u, 0u, 0u, 0u);
              }
#pragma unroll
              for (int i = 0; i < 16 / kRowsPer; ++i) {
                const int row = 16 * g + i * kRowsPer + lrow;
                uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w}, y[8];
                if (o == 1 && part) {
                  bool any = false;
#pragma unroll
                  for (int e = 0; e < 4; ++e) w[e] = drop_nonfinite<true>(w[e], any);
                  if (any) *dropped = 1;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  y[2 * e] = e4m3x2_to_f16x2(w[e] & 0xffffu);
                  y[2 * e + 1] = e4m3x2_to_f16x2(w[e] >> 16);
                }
                // the lanes of the second panel store their odd chunk first: the
                // eight lanes of a phase then touch eight chunk positions (at
                // d = 64 they are two rows, whose swizzles differ already)
                const int sw = D == 128 ? (ch >> 2) & 1 : 0;
                const uint32_t a0 = dst + tile_chunk<D>(row, 2 * ch + sw);
                const uint32_t a1 = dst + tile_chunk<D>(row, 2 * ch + 1 - sw);
                sts128(a0, sw ? y[4] : y[0], sw ? y[5] : y[1], sw ? y[6] : y[2],
                       sw ? y[7] : y[3]);
                sts128(a1, sw ? y[0] : y[4], sw ? y[1] : y[5], sw ? y[2] : y[6],
                       sw ? y[3] : y[7]);
              }
            }
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(o ? &v_full[st] : &k_full[st]);
            // the next tile's rows over the ones just read
            if (o == 0) {
              id = id_next;
              good = check_id(id);
            }
            if (j + 1 < n) issue(o, j + 1, good);
            if (o == 1) fetch_scale();
          }
        }
      } else {
        constexpr int kGroup = 16 * D * 2;
        const uint64_t pol = policy_evict_last();     // other items read the same keys
        for (int j = 0; ok && j < n; ++j) {
          const int J = jt + j, st = J % KST;
          const int t0 = base + j * kBN;
          const bool good = check_id(id);
          const int blk = id;
          id = fetch_id(j + 1);
          auto issue = [&](int o, uint64_t* bar) {
            const bool mine = good && lane < 8 && lane % 3 == (lw + o) % 3;
            const int count = __popc(__ballot_sync(0xffffffffu, mine));
            if (lane == 0) mbar_arrive_expect_tx(bar, count * kGroup);
            __syncwarp();
            if (mine) {
              const int in = (t0 + 16 * lane) & block_mask;
              uint8_t* dst = smem + (o ? F::kVOff : F::kKOff) + st * F::kBlockBytes + lane * 16 * 128;
#pragma unroll
              for (int pn = 0; pn < F::kPanels; ++pn)
                tma_load_4d(dst + pn * F::kPanelBytes, o ? &tmap_v : &tmap_k, bar, pn * 64, in,
                            pc.h, blk, pol);
            }
          };
          if (J >= KST && !mbar_wait_warp(&k_empty[st], ((J / KST) - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          issue(0, &k_full[st]);
          if (J >= KST && !mbar_wait_warp(&v_empty[st], ((J / KST) - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t here = __ballot_sync(0xffffffffu, good);
          if (t0 >= all.lo && t0 + kBN <= all.hi && (here & 0xffu) == 0xffu) {
            issue(1, &v_full[st]);
            continue;
          }
          // a tile that some rows do not see, or not all of it: its values
          // without infinities and NaN, and zeros where there is no token
          issue(1, &land[lw]);
          if (!mbar_wait_warp(&land[lw], cleaned++ & 1, abort_flag)) {
            ok = false;
            break;
          }
          bool any = false;
          for (int g = (lw + 1) % 3; g < 8; g += 3) {
            for (int i = lane; i < 16 * D / 8; i += 32) {
              const int row = 16 * g + i / (D / 8);
              const uint32_t at = smem_v + st * F::kBlockBytes + tile_chunk<D>(row, i % (D / 8));
              const bool in = ((here >> g) & 1) && t0 + row >= r.lo && t0 + row < r.hi;
              const uint4 x = in ? lds128_at(at) : make_uint4(0u, 0u, 0u, 0u);
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
              uint32_t y[4];
              bool hit = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = drop_nonfinite<false>(w[e], hit);
              any = any || hit;
              if (!in || hit) sts128(at, y[0], y[1], y[2], y[3]);
            }
          }
          if (any) *dropped = 1;
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_full[st]);
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
  } else if (warp == C::kWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t tm = warp_uniform(tmem);
    const uint64_t dq = sdesc_sw128(warp_uniform(smem_q), 16, 1024);
    const uint64_t dk = sdesc_sw128(warp_uniform(smem_k), 16, 1024);
    const uint64_t dv = sdesc_sw128(warp_uniform(smem_v), F::kPanelBytes, 1024);
    int jt = 0, np = 0;
    bool ok = true;
    for (; ok && pc.next<C::kRows, C::kTile>(p, range); ++np) {
      const int n = pc.t1 - pc.t0;
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
    bool ok = true;
    for (int np = 0; ok && pc.next<C::kRows, C::kTile>(p, range); ++np) {
      const int n = pc.t1 - pc.t0;
      const int rr = slot * kBM + lr;                 // row of the item
      const bool live = rr < pc.r.rows;
      int pos;
      {
        // rows past the last one are zeros that see what the last row sees
        const int row = pc.row0 + (live ? rr : pc.r.rows - 1);
        const int s = row / p.group, g = row - s * p.group;
        pos = pc.r.pos0 + s;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + pc.b * p.qs.b + (static_cast<long long>(pc.h) * p.group + g) * p.qs.h +
            s * p.qs.s + half * kOCols);
        uint4 x[kOCols / 8];
#pragma unroll
        for (int e = 0; e < kOCols / 8; ++e) x[e] = live ? src[e] : make_uint4(0u, 0u, 0u, 0u);
        if constexpr (F8) {
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < kOCols / 8; ++e)
            m = fmaxf(m, fmaxf(fmaxf(bf16x2_max_abs(x[e].x), bf16x2_max_abs(x[e].y)),
                               fmaxf(bf16x2_max_abs(x[e].z), bf16x2_max_abs(x[e].w))));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          const QueryScale qs = query_scale(m);
          sl2 = p.scale_log2 * qs.up;
#pragma unroll
          for (int e = 0; e < kOCols / 8; ++e)
            x[e] = make_uint4(bf16x2_to_f16x2(x[e].x, qs.down), bf16x2_to_f16x2(x[e].y, qs.down),
                              bf16x2_to_f16x2(x[e].z, qs.down), bf16x2_to_f16x2(x[e].w, qs.down));
        }
#pragma unroll
        for (int e = 0; e < kOCols / 8; ++e)
          sts128(smem_q + slot * F::kBlockBytes + tile_chunk<D>(lr, half * (kOCols / 8) + e),
                 x[e].x, x[e].y, x[e].z, x[e].w);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[slot]);
      }
      // the slot's rows all see [all.lo, all.hi)
      const int last_row = pc.row0 + pc.r.rows - 1;
      const SeenByAll all = seen_by_all(p, pc.r, min(pc.row0 + slot * kBM, last_row),
                                        min(pc.row0 + slot * kBM + kBM - 1, last_row));
      int t0 = pc.tok0<C::kTile>();
      float m_run = -INFINITY;   // running max, log2 units of the scaled scores
      float l_run = 0.f;         // this thread's part of the row sum
      for (int j = 0; j < n; ++j, t0 += kBN) {
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
          if (t0 < all.lo || t0 + kBN > all.hi) {
            const int hi = pos + 1 - t0 - half * kCols;
            const int lo = p.window > 0 ? hi - p.window : -kBN;
#pragma unroll
            for (int c = 0; c < kCols; ++c)
              if (c < lo || c >= hi) s[c] = -INFINITY;
          }
        };
        load_scores();
        // group g of 16 columns: x = s mul + add, without the reference
        constexpr int kGroups = F8 ? kCols / 16 : 1, kPerGroup = kCols / kGroups;
        uint32_t sc_at = 0;
        if constexpr (F8) {
          const int ring = (jt + j) % C::kScaleRing;
          if (!mbar_wait_warp(&sc_full[ring], ((jt + j) / C::kScaleRing) & 1, abort_flag)) {
            ok = false;
            break;
          }
          sc_at = smem_u32(smem + C::kScaleOff) + ring * 128 + half * (kGroups * 16);
        }
        auto group = [&](int g) {
          if constexpr (F8) {
            const uint4 w = lds128_at(sc_at + g * 16);
            return KvScale{__uint_as_float(w.x) * sl2, __uint_as_float(w.y),
                           __uint_as_float(w.z)};
          } else {
            return KvScale{sl2, 0.f, 1.f};
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
      if (!ok || !mbar_wait_warp(&o_full[slot], np & 1, abort_flag)) { ok = false; break; }
      tc_fence_after();
      l_run += __shfl_xor_sync(0xffffffffu, l_run, 16);
      const bool whole = pc.whole();
      const bool mend = *dropped != 0;
      const long long at = pc.slot(range) * C::kRows + rr;
      const float inv = whole ? (l_run == 0.f ? 0.f : 1.f / l_run) : 1.f;
#pragma unroll
      for (int cc = 0; cc < kOCols / 32; ++cc) {
        uint32_t o[32];
        tmem_ld_half32<kOCols>(t_o + cc * 32, o);
        tmem_wait_ld();
        if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float4 x = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                   __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
            const int d0 = half * kOCols + cc * 32 + e;
            if (mend)
              x = mend_row<D, F8, C::kTile>(p, pc, pc.row0 + rr, pc.row0, last_row,
                                            pc.tok0<C::kTile>(), n * kBN, d0, x);
            o[e] = __float_as_uint(x.x * inv);
            o[e + 1] = __float_as_uint(x.y * inv);
            o[e + 2] = __float_as_uint(x.z * inv);
            o[e + 3] = __float_as_uint(x.w * inv);
          }
          if (whole) {
            const int row = pc.row0 + rr, s = row / p.group, g = row - s * p.group;
            uint4* dst = reinterpret_cast<uint4*>(
                p.out + pc.b * p.os.b + (static_cast<long long>(pc.h) * p.group + g) * p.os.h +
                s * p.os.s + half * kOCols + cc * 32);
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16x2(__uint_as_float(o[8 * v4 + 2 * e]),
                                   __uint_as_float(o[8 * v4 + 2 * e + 1]));
              dst[v4] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            uint4* dst = reinterpret_cast<uint4*>(p.part_o + at * D + half * kOCols + cc * 32);
#pragma unroll
            for (int v4 = 0; v4 < 8; ++v4)
              dst[v4] = make_uint4(o[4 * v4], o[4 * v4 + 1], o[4 * v4 + 2], o[4 * v4 + 3]);
          }
        }
      }
      if (live && half == 0) {
        if (whole) write_lse(p, pc.b, pc.h, pc.row0 + rr, m_run, l_run, kLift<F8>);
        else *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m_run, l_run);
      }
      if (threadIdx.x == 0) pc.leave(p, range);
      // the next piece's first product overwrites O only after this slot's next P
      tc_fence_before();
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == C::kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, F::kTmemCols);
  }
}

}  // namespace sta
