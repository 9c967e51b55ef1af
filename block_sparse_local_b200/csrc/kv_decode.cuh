// kv_decode.cuh - attention of a few new tokens per sequence over the paged
// key/value cache (kv_cache.cuh).
//
// For query row r = (token s, head g of the key head's group), position
// p = seq_len - new_len + s:
//   out_r = sum_j w_rj V_j / sum_j w_rj,  w_rj = exp(q_r . K_j / sqrt(d)),
// j over the cached positions in (p - window, p].  With an 8-bit cache K_j and
// V_j are e4m3 numbers times a scale per (block, head).  The scales never
// touch the numbers: with x_j = log2(e)/sqrt(d) * ks_j * (q . k_j) and M a
// running maximum of x_j + log2 vs_j, the kernel accumulates
//   O = sum_j e_j v_j,  l = sum_j e_j / vs_j,  e_j = 2^(x_j + log2 vs_j - M),
// so that O / l is the result: one more constant in the multiply-add that the
// exponent needs anyway, and the same matrix product on the plain numbers.
//
// What bounds it: the cache is read once, 2 d bytes (e4m3) per token and key
// head against 4 d flops for each of the (few) query rows, so HBM.  Hence the
// split: the tokens of all (sequence, key head) items are laid end to end and
// cut into as many equal ranges as there are thread blocks (two per SM), so
// that a batch of ragged lengths, or one long sequence, keeps every SM loading
// until the end.  An item that falls into several ranges leaves (M, l, O) of
// each in the workspace and kv_combine_kernel joins them, in order (kv_split.cuh).
//
// A warp takes 16 query rows and its own tokens: copies (cp.async) into its own
// ring of shared-memory stages, m16n8k16 products, softmax in fp32 registers;
// no barrier in the loop.  Up to 64 rows per item: kRT row tiles, one warp
// each, share a ring.  The operands never go through a transposition: the
// order of d inside Q K^T, and the order of the output columns of P V, are
// free, so that a lane's fragments are 16 consecutive bytes of a cached row,
// for keys and values alike; e4m3 becomes f16 in registers, which is exact.
// Shared-memory chunks of 16 bytes are permuted within their 128-byte line so
// that both access patterns are free of bank conflicts.
#pragma once

#include "kv_split.cuh"

namespace sta {

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// D += A B, 16 x 8 x 16, f16 (F8: the cache's numbers as f16) or bf16 operands.
template <bool F8>
__device__ __forceinline__ void mma16816(float d[4], const uint32_t a[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F8)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, bool F8, int RT>
struct DecodeCfg {
  static constexpr int kElem = F8 ? 1 : 2;
  static constexpr int kRow = D * kElem;                    // bytes of a cached row
  static constexpr int kTok = (!F8 && D == 128) ? 16 : 32;  // tokens of a warp's step
  static constexpr int kTW = RT == 4 ? 2 : 4;               // token groups (rings)
  static constexpr int kWarps = RT * kTW;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kTile = kTW * kTok;                  // tokens of a thread block's step
  static constexpr int kRows = 16 * RT;
  static constexpr int kOver = 1;                           // see kv_split.cuh
  static constexpr int kStage = 2 * kTok * kRow;            // K and V bytes of a ring stage
  // two thread blocks per SM share its shared memory with one row tile, else one
  static constexpr int kCtas = RT == 1 ? 2 : 1;
  static constexpr int kStages =
      (96 * 1024 * (RT == 1 ? 1 : 2)) / (kTW * kStage) < 6
          ? (96 * 1024 * (RT == 1 ? 1 : 2)) / (kTW * kStage) : 6;
  static constexpr int kScaleOff = kTW * kStages * kStage;  // 16 bytes per stage
  static constexpr int kLoopBytes = kScaleOff + kTW * kStages * 16;
  static constexpr int kMergeRow = D + 4;                   // floats, padded against conflicts
  static constexpr int kMergeBytes = kWarps * 16 * (kMergeRow + 2) * 4;
  static constexpr int kSmemBytes = kLoopBytes > kMergeBytes ? kLoopBytes : kMergeBytes;
};

// Byte offset of 16-byte chunk ch of row t in a K or V stage: chunks move
// within their 128-byte line (two 64-byte rows share one) so that the eight
// lanes of a shared-memory phase touch eight different chunk positions, both
// when they read 4 chunks of 2 neighbouring rows (keys) and 2 chunks of 4 rows
// two apart (values).
template <int ROW>
__device__ __forceinline__ uint32_t stage_chunk(int t, int ch) {
  if constexpr (ROW == 64)
    return (t >> 1) * 128 + ((((((t & 1) << 2) | ch)) ^ (((t >> 1) & 3) << 1)) << 4);
  else
    return t * ROW + ((ch ^ ((t & 6) ^ ((t & 1) << 2))) << 4);
}

template <int D, bool F8, int RT>
__global__ void __launch_bounds__(DecodeCfg<D, F8, RT>::kThreads, DecodeCfg<D, F8, RT>::kCtas)
    kv_decode_kernel(const AttendParams p) {
  using C = DecodeCfg<D, F8, RT>;
  constexpr int kTok = C::kTok, kRow = C::kRow, kNS = C::kStages;
  constexpr int kChunks = kRow / 16;                // 16-byte chunks of a row
  constexpr int kHalves = kTok / 16;                // 16-token parts, each inside one block
  constexpr int kNT = kTok / 8;                     // score tiles of a step
  constexpr int kOT = D / 8;                        // output tiles
  constexpr int kPer = 16 / C::kElem;               // elements of a chunk
  constexpr int kKL = D / (4 * kPer);               // key chunks per lane and score tile
  extern __shared__ __align__(128) uint8_t smem[];

  const KvLayout& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tw = warp % C::kTW, rt = warp / C::kTW;
  const int g = lane >> 2, cq = lane & 3;

  const KvRange range = kv_range<D, C::kRows, C::kTile, C::kOver, C::kThreads>(p);
  if (range.u0 >= range.u1) return;

  const uint32_t ring = smem_u32(smem) + tw * kNS * C::kStage;
  const uint32_t ring_scale = smem_u32(smem) + C::kScaleOff + tw * kNS * 16;
  const int block_mask = (1 << c.shift) - 1;

  KvPiece pc;
  pc.start(range);
  while (pc.next<C::kRows, C::kTile, C::kOver>(p, range)) {
    const ItemRange& r = pc.r;
    const int h = pc.h, b = pc.b, row0 = pc.row0, t0 = pc.t0, t1 = pc.t1;

    // --------------------------------------------------------------- query rows
    // Lane (g, cq) holds of rows g and g + 8 the elements of chunk 4 l + cq,
    // the ones that it holds of every key.  With an f16 product a row is first
    // scaled by a power of two to below 2, so that no bf16 value overflows f16.
    const int rbase = row0 + 16 * rt;
    uint32_t qf[D / 16][4];
    float cr[2];
    int pos[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = rbase + g + 8 * i;
      const int last = row0 + r.rows - 1;
      const bool ok = row <= last;
      const int rr = ok ? row : last;               // padding rows see what the last row sees
      const int s = rr / p.group, gg = rr - s * p.group;
      pos[i] = r.pos0 + s;
      const __nv_bfloat16* src = p.q + b * p.qs.b +
                                 (static_cast<long long>(h) * p.group + gg) * p.qs.h + s * p.qs.s;
      uint32_t w[D / 8];                            // d / 4 bf16 of the row
#pragma unroll
      for (int l = 0; l < kKL; ++l) {
#pragma unroll
        for (int v = 0; v < kPer / 8; ++v) {
          const uint4 x = ok ? *reinterpret_cast<const uint4*>(src + (4 * l + cq) * kPer + 8 * v)
                             : make_uint4(0u, 0u, 0u, 0u);
          w[(l * kPer / 8 + v) * 4 + 0] = x.x;
          w[(l * kPer / 8 + v) * 4 + 1] = x.y;
          w[(l * kPer / 8 + v) * 4 + 2] = x.z;
          w[(l * kPer / 8 + v) * 4 + 3] = x.w;
        }
      }
      cr[i] = p.scale_log2;
      if constexpr (F8) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < D / 8; ++e) m = fmaxf(m, bf16x2_max_abs(w[e]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const QueryScale qs = query_scale(m);
        cr[i] *= qs.up;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) w[k] = bf16x2_to_f16x2(w[k], qs.down);
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[k][i] = w[2 * k];
        qf[k][i + 2] = w[2 * k + 1];
      }
    }
    // the tile's rows all see [all_lo, all_hi): no mask needed inside
    const int last_row = row0 + r.rows - 1;
    const SeenByAll all = seen_by_all(p, r, min(rbase, last_row), min(rbase + 15, last_row));

    // --------------------------------------------------------------- the loop
    const int steps = t1 - t0;
    const int tok_base = pc.tok0<C::kTile>() + tw * kTok;
    const int* table = c.table + static_cast<long long>(b) * c.width;
    int ids[kHalves];                               // blocks of the next step to be issued
    auto fetch_ids = [&](int k) {
#pragma unroll
      for (int x = 0; x < kHalves; ++x) {
        const int t = tok_base + k * C::kTile + 16 * x;
        ids[x] = (k < steps && t < r.hi && t + 16 > r.lo) ? __ldg(table + (t >> c.shift)) : -2;
      }
    };
    auto issue = [&](int k) {
      const uint32_t st = ring + (k % kNS) * C::kStage;
      const int t = tok_base + k * C::kTile;
      const uint8_t *kb[kHalves], *vb[kHalves];
      bool ok[kHalves];
#pragma unroll
      for (int x = 0; x < kHalves; ++x) {
        ok[x] = ids[x] >= 0 && ids[x] < c.num_blocks;
        if (!ok[x] && ids[x] != -2 && lane == 0) kv_bad_index();
        const long long id = ok[x] ? ids[x] : 0;
        const long long in = static_cast<long long>((t + 16 * x) & block_mask) * kRow;
        kb[x] = c.k + id * c.k_block + h * c.k_head + in;
        vb[x] = c.v + id * c.v_block + h * c.v_head + in;
        if constexpr (F8) {
          if (rt == 0 && lane < 2) {
            const float* sp = (lane == 0 ? c.k_scale : c.v_scale) + id * c.hkv + h;
            cp_async4(ring_scale + (k % kNS) * 16 + x * 8 + lane * 4, sp, ok[x]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kTok * kChunks / 32; ++i) {
        if (i % RT != rt && RT > 1) continue;
        constexpr int kRowsPer = 32 / kChunks > 0 ? 32 / kChunks : 1;
        const int row = i * kRowsPer + lane / kChunks, ch = lane % kChunks;
        const int x = (i * kRowsPer) / 16;
        const bool in = ok[x] && t + row >= r.lo && t + row < r.hi;
        const long long off = static_cast<long long>(row - 16 * x) * kRow + ch * 16;
        const uint32_t dst = st + stage_chunk<kRow>(row, ch);
        cp_async16(dst, in ? kb[x] + off : c.k, in);
        cp_async16(dst + kTok * kRow, in ? vb[x] + off : c.v, in);
      }
      cp_async_commit();
    };
    float o[kOT][4];
#pragma unroll
    for (int j = 0; j < kOT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    bool dropped = false;                           // infinities or NaN left out of a product

    fetch_ids(0);
#pragma unroll
    for (int k = 0; k < kNS - 1; ++k) {
      if (k < steps) issue(k); else cp_async_commit();
      fetch_ids(k + 1);
    }
    for (int k = 0; k < steps; ++k) {
      cp_async_wait<kNS - 2>();
      if constexpr (RT > 1)                         // the ring's warps: their copies have landed
        asm volatile("bar.sync %0, %1;" ::"r"(1 + tw), "n"(32 * RT) : "memory");
      else
        __syncwarp();
      if (k + kNS - 1 < steps) issue(k + kNS - 1); else cp_async_commit();
      fetch_ids(k + kNS);
      const int t = tok_base + k * C::kTile;
      if (t >= r.hi || t + kTok <= r.lo) continue;  // the same for the whole warp
      const uint32_t sk = ring + (k % kNS) * C::kStage;
      const uint32_t sv = sk + kTok * kRow;
      float ksc[kHalves], lv[kHalves], iv[kHalves];
#pragma unroll
      for (int x = 0; x < kHalves; ++x) {
        ksc[x] = 1.f;
        lv[x] = 0.f;
        iv[x] = 1.f;
        if constexpr (F8) {
          const uint2 w = lds64(ring_scale + (k % kNS) * 16 + x * 8);
          ksc[x] = __uint_as_float(w.x);
          const KvScale sc = kv_scale(ksc[x], __uint_as_float(w.y));
          lv[x] = sc.log2_v;
          iv[x] = sc.inv_v;
        }
      }
      // scores
      float s[kNT][4];
#pragma unroll
      for (int j = 0; j < kNT; ++j) {
        s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
        for (int l = 0; l < kKL; ++l) {
          const uint4 w = lds128(sk + stage_chunk<kRow>(8 * j + g, 4 * l + cq));
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
          if constexpr (F8) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mma16816<true>(s[j], qf[4 * l + e], e4m3x2_to_f16x2(ww[e] & 0xffffu),
                             e4m3x2_to_f16x2(ww[e] >> 16));
          } else {
            mma16816<false>(s[j], qf[2 * l], ww[0], ww[1]);
            mma16816<false>(s[j], qf[2 * l + 1], ww[2], ww[3]);
          }
        }
      }
      const bool masked = t < all.lo || t + kTok > all.hi;
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < kNT; ++j) {
        const int x = j / 2;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = e >> 1;
          float y = fmaf(s[j][e], cr[i] * ksc[x], lv[x]);
          if (masked) {
            const int tok = t + 8 * j + 2 * cq + (e & 1);
            const bool see = tok <= pos[i] && tok < r.len && tok >= 0 &&
                             (p.window <= 0 || tok > pos[i] - p.window);
            if (!see) y = -INFINITY;
          }
          s[j][e] = y;
          mx[i] = fmaxf(mx[i], y);
        }
      }
      float alpha[2];
      bool up = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
        // the reference moves only when the maximum grew by more than 2^8, which
        // with the lift leaves weights up to 2^15, inside f16's range
        alpha[i] = 1.f;
        if (mx[i] > m_run[i] + 8.f || m_run[i] == -INFINITY) {
          alpha[i] = mx[i] == -INFINITY ? 1.f : fast_exp2(m_run[i] - mx[i]);
          up = up || mx[i] > m_run[i];
          m_run[i] = fmaxf(m_run[i], mx[i]);
        }
      }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int j = 0; j < kOT; ++j) {
          o[j][0] *= alpha[0];
          o[j][1] *= alpha[0];
          o[j][2] *= alpha[1];
          o[j][3] *= alpha[1];
        }
        l_run[0] *= alpha[0];
        l_run[1] *= alpha[1];
      }
      const float ref[2] = {m_run[0] == -INFINITY ? 0.f : m_run[0] - kLift<F8>,
                            m_run[1] == -INFINITY ? 0.f : m_run[1] - kLift<F8>};
      // P and O += P V, 16 tokens at a time
#pragma unroll
      for (int x = 0; x < kHalves; ++x) {
        uint32_t pf[4];
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float* sj = s[2 * x + y];
          float e4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            e4[e] = fast_exp2(sj[e] - ref[e >> 1]);
            sum[e >> 1] += e4[e];
          }
          pf[2 * y] = F8 ? pack_f16x2(e4[0], e4[1]) : pack_bf16x2(e4[0], e4[1]);
          pf[2 * y + 1] = F8 ? pack_f16x2(e4[2], e4[3]) : pack_bf16x2(e4[2], e4[3]);
        }
        l_run[0] = fmaf(sum[0], iv[x], l_run[0]);
        l_run[1] = fmaf(sum[1], iv[x], l_run[1]);
        const int tr = 16 * x + 2 * cq;             // this lane's tokens tr, +1, +8, +9
        if constexpr (F8) {
          uint32_t a[4][4];                         // 16 (d = 128) or 8 bytes of each
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int row = tr + (y & 1) + (y >> 1) * 8;
            if constexpr (D == 128) {
              const uint4 w = lds128(sv + stage_chunk<kRow>(row, g));
              a[y][0] = w.x; a[y][1] = w.y; a[y][2] = w.z; a[y][3] = w.w;
            } else {
              const uint2 w = lds64(sv + stage_chunk<kRow>(row, g >> 1) + (g & 1) * 8);
              a[y][0] = w.x; a[y][1] = w.y; a[y][2] = 0; a[y][3] = 0;
            }
          }
          if (masked && p.c.S > 1) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
              for (int w = 0; w < D / 32; ++w) a[y][w] = drop_nonfinite<true>(a[y][w], dropped);
          }
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {
            const uint32_t lo0 = __byte_perm(a[0][w], a[1][w], 0x5140);
            const uint32_t hi0 = __byte_perm(a[0][w], a[1][w], 0x7362);
            const uint32_t lo1 = __byte_perm(a[2][w], a[3][w], 0x5140);
            const uint32_t hi1 = __byte_perm(a[2][w], a[3][w], 0x7362);
            mma16816<true>(o[4 * w], pf, e4m3x2_to_f16x2(lo0 & 0xffffu),
                           e4m3x2_to_f16x2(lo1 & 0xffffu));
            mma16816<true>(o[4 * w + 1], pf, e4m3x2_to_f16x2(lo0 >> 16),
                           e4m3x2_to_f16x2(lo1 >> 16));
            mma16816<true>(o[4 * w + 2], pf, e4m3x2_to_f16x2(hi0 & 0xffffu),
                           e4m3x2_to_f16x2(hi1 & 0xffffu));
            mma16816<true>(o[4 * w + 3], pf, e4m3x2_to_f16x2(hi0 >> 16),
                           e4m3x2_to_f16x2(hi1 >> 16));
          }
        } else {
#pragma unroll
          for (int ch = 0; ch < D / 64; ++ch) {
            uint32_t a[4][4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint4 w = lds128(sv + stage_chunk<kRow>(tr + (y & 1) + (y >> 1) * 8,
                                                            g + 8 * ch));
              a[y][0] = w.x; a[y][1] = w.y; a[y][2] = w.z; a[y][3] = w.w;
            }
            if (masked && p.c.S > 1) {
#pragma unroll
              for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int w = 0; w < 4; ++w)
                  a[y][w] = drop_nonfinite<false>(a[y][w], dropped);
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              mma16816<false>(o[8 * ch + 2 * w], pf, __byte_perm(a[0][w], a[1][w], 0x5410),
                              __byte_perm(a[2][w], a[3][w], 0x5410));
              mma16816<false>(o[8 * ch + 2 * w + 1], pf, __byte_perm(a[0][w], a[1][w], 0x7632),
                              __byte_perm(a[2][w], a[3][w], 0x7632));
            }
          }
        }
      }
    }
    // ------------------------------------------------- join the warps' tokens
    cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 1);
      l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 2);
    }
    __syncthreads();                                // the rings are free
    float* mo = reinterpret_cast<float*>(smem);     // [warp][16][kMergeRow]
    float* mml = mo + C::kWarps * 16 * C::kMergeRow;  // [warp][16][2]
    {
      // output tile j, columns 2 cq and 2 cq + 1: the kPer-element chunks (8
      // bytes of one at d = 64, e4m3) that the lanes g = 2 cq, 2 cq + 1 read
      constexpr int kRun = F8 ? D / 8 : 8;          // consecutive d of a lane's V chunk
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float* row = mo + (warp * 16 + g + 8 * i) * C::kMergeRow;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
          for (int j = 0; j < kOT; j += 4) {
            const int d0 = (2 * cq + q) * kRun + (j % kRun) + (j / kRun) * 8 * kRun;
            *reinterpret_cast<float4*>(row + d0) =
                make_float4(o[j][2 * i + q], o[j + 1][2 * i + q], o[j + 2][2 * i + q],
                            o[j + 3][2 * i + q]);
          }
        }
        if (cq == 0) {
          mml[(warp * 16 + g + 8 * i) * 2] = m_run[i];
          mml[(warp * 16 + g + 8 * i) * 2 + 1] = l_run[i];
        }
      }
    }
    const bool mend = __syncthreads_or(dropped) != 0;
    const bool whole = pc.whole();
    const long long slot = pc.slot();
    for (int i = threadIdx.x; i < r.rows * (D / 4); i += C::kThreads) {
      const int d4 = i % (D / 4), rr = i / (D / 4);
      const int w0 = (rr / 16) * C::kTW;
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < C::kTW; ++w) m = fmaxf(m, mml[((w0 + w) * 16 + rr % 16) * 2]);
      float l = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::kTW; ++w) {
        const float* ml = mml + ((w0 + w) * 16 + rr % 16) * 2;
        const float f = ml[1] == 0.f ? 0.f : fast_exp2(ml[0] - m);   // 0: saw nothing
        const float4 x = *reinterpret_cast<const float4*>(
            mo + ((w0 + w) * 16 + rr % 16) * C::kMergeRow + 4 * d4);
        l = fmaf(ml[1], f, l);
        acc.x = fmaf(x.x, f, acc.x);
        acc.y = fmaf(x.y, f, acc.y);
        acc.z = fmaf(x.z, f, acc.z);
        acc.w = fmaf(x.w, f, acc.w);
      }
      if (mend) {
        const int tile0 = row0 + rr / 16 * 16;
        acc = mend_row<D, F8, kTok>(p, MendItem{b, h, r.pos0, r.len},
                                    seen_by_all(p, r, tile0, min(tile0 + 15, row0 + r.rows - 1)),
                                    row0 + rr, pc.tok0<C::kTile>(), (t1 - t0) * C::kTile, 4 * d4,
                                    acc);
      }
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        write_row4<D>(p, b, h, row0 + rr, 4 * d4,
                      make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        if (d4 == 0) write_lse(p, b, h, row0 + rr, m, l, kLift<F8>);
      } else {
        *reinterpret_cast<float4*>(p.part_o + (slot * C::kRows + rr) * D + 4 * d4) = acc;
        if (d4 == 0)
          *reinterpret_cast<float2*>(p.part_ml + (slot * C::kRows + rr) * 2) = make_float2(m, l);
      }
    }
    if (threadIdx.x == 0) pc.leave<C::kOver>(p, range);
    __syncthreads();                                // before the next piece's copies
  }
}

}  // namespace sta
