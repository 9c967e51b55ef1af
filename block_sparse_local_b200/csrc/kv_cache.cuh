// kv_cache.cuh - the paged key/value cache: what its kernels share, and the
// kernel that appends tokens to it.
//
// Layout.  k_cache and v_cache hold blocks of `block` tokens, [num_blocks][hkv]
// [block][d], the last two dimensions contiguous; block_table[b][i] is the
// block of positions i*block .. i*block + block - 1 of sequence b.  The cache
// is bf16, or e4m3 with one fp32 scale per (block, head) and operand: a value
// is its e4m3 number times the scale.  Scales are powers of two, so that
// raising a block's scale because a larger token arrives moves the numbers
// already there by whole exponents: exact, but for those that leave the
// normal range of e4m3 downwards.
//
// seq_lens[b] counts the tokens of sequence b in the cache, the new ones
// included; the new ones are the last new_lens[b] (all S when new_lens is
// null), so token s of the call has position seq_lens[b] - new_lens[b] + s.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "device_ptx.cuh"

namespace sta {

// A block index outside the cache, or a length beyond the block table: the
// access is skipped.
__device__ __forceinline__ void kv_bad_index() { atomicOr(&g_status[1], 1u); }

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 5.421010862427522e-20f;   // 2^-64, the scale of a block of zeros

struct KvLayout {
  uint8_t* k;                    // caches, [num_blocks][hkv][block][d]
  uint8_t* v;
  float* k_scale;                // [num_blocks][hkv]; null: bf16 cache
  float* v_scale;
  long long k_block, k_head;     // strides in bytes
  long long v_block, v_head;
  const int* table;              // [B][width]
  const int* seq_lens;           // [B]
  const int* new_lens;           // [B] or null
  int width;
  int num_blocks;
  int shift;                     // log2(block)
  int B, S, hq, hkv;
};

struct RowStrides {              // in elements: batch, head, token
  long long b, h, s;
};

// Lengths of sequence b: tokens that the block table can hold, new tokens of
// this call, and the position of the first of them.
struct KvSeqLen {
  int len;     // readable tokens
  int fresh;   // new tokens, 0 .. S
  int pos0;    // position of the first new token (negative: not in the cache)
};

__device__ __forceinline__ KvSeqLen kv_seq(const KvLayout& c, int b) {
  KvSeqLen r;
  const int n = c.seq_lens[b];
  const long long cap = static_cast<long long>(c.width) << c.shift;
  r.len = n < 0 ? 0 : (n > cap ? static_cast<int>(cap) : n);
  if (n > cap) kv_bad_index();
  int f = c.new_lens != nullptr ? c.new_lens[b] : c.S;
  r.fresh = f < 0 ? 0 : (f > c.S ? c.S : f);
  // a padded slot of the batch (length 0) has all its tokens before position 0
  r.pos0 = (n < 0 ? 0 : n) - r.fresh;
  return r;
}

struct AppendParams {
  KvLayout c;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* q;        // null: no queries to rotate
  __nv_bfloat16* q_out;
  RowStrides ks, vs, qs, os;
  const float* rope;             // [rows][d]: d/2 cosines, d/2 sines; null: no rotation
  int interleaved;               // pairs (2i, 2i + 1) instead of (i, i + d/2)
  int pages;                     // blocks that S tokens can touch, at most
  int kv_blocks;                 // thread blocks that store e4m3 keys and values
  int q_groups, kv_groups;       // heads by kHeadGroup; e4m3 cache: no kv_groups
  unsigned int units;            // B * S * (q_groups + 2 kv_groups) * d / 16
};

// Heads of a token that one thread turns, one unit each: they share the angles,
// and their loads are on the way together.
constexpr int kHeadGroup = 4;

// One unit of work is 16 elements of a token's row, a vector of 8 pairs: the
// pairs (i, i + d/2) of 8 consecutive i, or 8 consecutive pairs (2i, 2i + 1).
// So the two 16-byte loads of a unit hold whole pairs in either layout.
__device__ __forceinline__ void unit_unpack(uint4 a, uint4 b, float x[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

template <int D>
__device__ __forceinline__ void unit_load(const __nv_bfloat16* row, int c, bool interleaved,
                                          float x[16]) {
  const int e0 = interleaved ? 16 * c : 8 * c;
  const int e1 = interleaved ? 16 * c + 8 : D / 2 + 8 * c;
  unit_unpack(*reinterpret_cast<const uint4*>(row + e0), *reinterpret_cast<const uint4*>(row + e1),
              x);
}

// Cosines and sines of a unit's 8 pairs at a position.
struct UnitAngles {
  float co[8], si[8];
};

template <int D>
__device__ __forceinline__ UnitAngles unit_angles(const float* rope, long long pos, int c) {
  const float4* cs = reinterpret_cast<const float4*>(rope + pos * D + 8 * c);
  const float4* sn = reinterpret_cast<const float4*>(rope + pos * D + D / 2 + 8 * c);
  UnitAngles r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 a = __ldg(cs + h), b = __ldg(sn + h);
    r.co[4 * h] = a.x; r.co[4 * h + 1] = a.y; r.co[4 * h + 2] = a.z; r.co[4 * h + 3] = a.w;
    r.si[4 * h] = b.x; r.si[4 * h + 1] = b.y; r.si[4 * h + 2] = b.z; r.si[4 * h + 3] = b.w;
  }
  return r;
}

// Rotates the unit's pairs by the angles of one position: (a, b) becomes
// (a cos - b sin, b cos + a sin), in fp32 from the fp32 table.  Products and
// sums are rounded one by one (no multiply-add), as elementary operations
// round them elsewhere: the kernel waits for memory, and a token gets the same
// e4m3 number whichever program stored it.
__device__ __forceinline__ void unit_rotate(const UnitAngles& w, bool interleaved, float x[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    if (interleaved) { a = x[2 * i]; b = x[2 * i + 1]; }
    else { a = x[i]; b = x[8 + i]; }
    const float y0 = __fsub_rn(__fmul_rn(a, w.co[i]), __fmul_rn(b, w.si[i]));
    const float y1 = __fadd_rn(__fmul_rn(b, w.co[i]), __fmul_rn(a, w.si[i]));
    if (interleaved) { x[2 * i] = y0; x[2 * i + 1] = y1; }
    else { x[i] = y0; x[8 + i] = y1; }
  }
}

template <int D>
__device__ __forceinline__ void unit_store_bf16(__nv_bfloat16* row, int c, bool interleaved,
                                                const float x[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  const int e0 = interleaved ? 16 * c : 8 * c;
  const int e1 = interleaved ? 16 * c + 8 : D / 2 + 8 * c;
  *reinterpret_cast<uint4*>(row + e0) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(row + e1) = make_uint4(w[4], w[5], w[6], w[7]);
}

// Two fp32 -> two e4m3 (nearest even, finite overflow saturates, NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 -> f16x2, exact (every e4m3 value is an f16 value; NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
      : "=r"(r) : "r"(two));
  return r;
}

// The smallest power of two s with amax <= 448 s = 1.75 * 2^8 s, at least
// 2^-64; amax is finite.
__device__ __forceinline__ float e4m3_scale(float amax) {
  if (amax <= kE4m3Max * kMinScale) return kMinScale;
  const uint32_t u = __float_as_uint(amax);        // normal: amax > 2^-56
  int e = static_cast<int>(u >> 23) - 8;           // biased exponent of 2^(x - 8)
  if ((u & 0x7fffffu) > 0x600000u) e += 1;         // mantissa above 1.75
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.4028234663852886e38f ? a : 0.f;    // inf and NaN do not set a scale
}

// Moves the e4m3 numbers of 16 bytes to another scale: rn(number * ratio).
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float ratio) {
  uint32_t out = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t f = e4m3x2_to_f16x2((w >> (16 * h)) & 0xffffu);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f));
    out |= pack_e4m3x2(x.x * ratio, x.y * ratio) << (16 * h);
  }
  return out;
}

// Queries, and keys and values of a bf16 cache: thread `u` of the launch has one
// unit of up to kHeadGroup heads of one token (heads fastest, then tokens).
template <int D>
__device__ __forceinline__ void append_units(const AppendParams& p, unsigned int u) {
  constexpr int kUnits = D / 16;
  const KvLayout& c = p.c;
  if (u >= p.units) return;
  const bool inter = p.interleaved != 0;
  const int cu = static_cast<int>(u % kUnits);
  const unsigned int groups = p.q_groups + 2 * p.kv_groups;
  const unsigned int r = u / kUnits, tok = r / groups;
  int g = static_cast<int>(r - tok * groups);
  const int b = static_cast<int>(tok / static_cast<unsigned int>(c.S));
  const int s = static_cast<int>(tok - static_cast<unsigned int>(b) * c.S);
  const KvSeqLen sl = kv_seq(c, b);
  const int pos = sl.pos0 + s;
  if (s >= sl.fresh || pos < 0 || pos >= sl.len) return;
  const int kind = g < p.q_groups ? 0 : g < p.q_groups + p.kv_groups ? 1 : 2;   // q, k, v
  if (kind > 0) g -= p.q_groups + (kind - 1) * p.kv_groups;
  const int h0 = g * kHeadGroup, heads = min(kHeadGroup, (kind == 0 ? c.hq : c.hkv) - h0);
  const RowStrides& st = kind == 0 ? p.qs : kind == 1 ? p.ks : p.vs;
  const __nv_bfloat16* src = (kind == 0 ? p.q : kind == 1 ? p.k : p.v) + b * st.b + h0 * st.h +
                             s * st.s;
  __nv_bfloat16* dst;
  long long step;
  if (kind == 0) {
    dst = p.q_out + b * p.os.b + h0 * p.os.h + s * p.os.s;
    step = p.os.h;
  } else {
    const int id = c.table[static_cast<long long>(b) * c.width + (pos >> c.shift)];
    if (id < 0 || id >= c.num_blocks) {
      kv_bad_index();
      return;
    }
    step = (kind == 1 ? c.k_head : c.v_head) / 2;
    dst = reinterpret_cast<__nv_bfloat16*>(kind == 1 ? c.k + id * c.k_block
                                                     : c.v + id * c.v_block) +
          h0 * step + (pos & ((1 << c.shift) - 1)) * D;
  }
  const int e0 = inter ? 16 * cu : 8 * cu, e1 = inter ? 16 * cu + 8 : D / 2 + 8 * cu;
  uint4 in[kHeadGroup][2];
#pragma unroll
  for (int i = 0; i < kHeadGroup; ++i) {
    if (i < heads) {
      in[i][0] = *reinterpret_cast<const uint4*>(src + i * st.h + e0);
      in[i][1] = *reinterpret_cast<const uint4*>(src + i * st.h + e1);
    }
  }
  if (kind < 2 && p.rope != nullptr) {
    const UnitAngles w = unit_angles<D>(p.rope, pos, cu);
#pragma unroll
    for (int i = 0; i < kHeadGroup; ++i) {
      if (i >= heads) break;
      float x[16];
      unit_unpack(in[i][0], in[i][1], x);
      unit_rotate(w, inter, x);
      unit_store_bf16<D>(dst + i * step, cu, inter, x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kHeadGroup; ++i) {
      if (i >= heads) break;
      *reinterpret_cast<uint4*>(dst + i * step + e0) = in[i][0];
      *reinterpret_cast<uint4*>(dst + i * step + e1) = in[i][1];
    }
  }
}

// kv_append_kernel: the first kv_blocks thread blocks store keys and values of
// an e4m3 cache, one (sequence, touched cache block, head, K or V) each; the
// others what is rounded to bf16 (append_units).
//
// Memory-bound: every input is read once and every output written once.  One
// thread block owns a whole (cache block, head), so the block's amax, its
// scale and the numbers that the scale covers meet in registers and shared
// memory, with one read of the tokens, no second pass and no atomics.  A prompt of
// 32768 tokens (32 and 8 heads of 128) takes 146 to 149 us with an e4m3 cache (755
// MB, 5.1 TB/s), 130 us with a bf16 cache (822 MB, 6.3 TB/s, what a copy reaches).
// NT threads with U units each hold up to NT * U / (D/16) tokens.
// With an e4m3 cache (F8) the registers are kept to 64, for half of the SM's
// warps: that prompt, repeated, takes 144 us, 154 with the 74 that the compiler
// would take; two heads per thread instead of spilling a few: 150.  For a bf16 cache
// the spilling costs more than the warps gain (seven pieces of up to 777 tokens, 16
// heads of 64, repeated: 10.3 us without, 12.5 with; among other calls 12.4).
template <int D, bool F8, int NT, int U>
__global__ void __launch_bounds__(NT, F8 && U <= 2 ? 1024 / NT : 1)
    kv_append_kernel(const AppendParams p) {
  constexpr int kUnits = D / 16;                    // units of a row
  const bool inter = p.interleaved != 0;
  const KvLayout& c = p.c;
  if (static_cast<int>(blockIdx.x) >= p.kv_blocks) {
    append_units<D>(p, (blockIdx.x - p.kv_blocks) * NT + threadIdx.x);
    return;
  }
  // ------------------------------------------------------------ keys, values
  unsigned int t = blockIdx.x;
  const bool is_v = (t & 1u) != 0;
  t >>= 1;
  const int h = static_cast<int>(t % static_cast<unsigned int>(c.hkv));
  t /= static_cast<unsigned int>(c.hkv);
  const int pg = static_cast<int>(t % static_cast<unsigned int>(p.pages));
  const int b = static_cast<int>(t / static_cast<unsigned int>(p.pages));
  const KvSeqLen sl = kv_seq(c, b);
  const int block = 1 << c.shift;
  const int first = sl.pos0 < 0 ? 0 : sl.pos0;      // first position to store
  const int end = min(sl.pos0 + sl.fresh, sl.len);  // one past the last
  const int entry = (first >> c.shift) + pg;
  const int lo = max(first, entry << c.shift);
  const int hi = min(end, (entry + 1) << c.shift);
  if (lo >= hi) return;
  const int id = c.table[static_cast<long long>(b) * c.width + entry];
  if (id < 0 || id >= c.num_blocks) {
    if (threadIdx.x == 0) kv_bad_index();
    return;
  }
  const int slot0 = lo & (block - 1);
  const int n = hi - lo;
  const __nv_bfloat16* src = is_v
      ? p.v + b * p.vs.b + h * p.vs.h + static_cast<long long>(lo - sl.pos0) * p.vs.s
      : p.k + b * p.ks.b + h * p.ks.h + static_cast<long long>(lo - sl.pos0) * p.ks.s;
  const long long src_s = is_v ? p.vs.s : p.ks.s;
  uint8_t* dst = is_v ? c.v + id * c.v_block + h * c.v_head : c.k + id * c.k_block + h * c.k_head;
  const bool turn = !is_v && p.rope != nullptr;
  float x[U][16];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int u = static_cast<int>(threadIdx.x) + i * NT;
    const int tok = u / kUnits, cu = u % kUnits;
    if (tok < n) {
      unit_load<D>(src + tok * src_s, cu, inter, x[i]);
      if (turn) unit_rotate(unit_angles<D>(p.rope, lo + tok, cu), inter, x[i]);
#pragma unroll
      for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[i][e]));   // not NaN
    }
  }
  if (amax > 3.4028234663852886e38f) {              // an infinity: what else there is
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if ((static_cast<int>(threadIdx.x) + i * NT) / kUnits < n) {
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, finite_abs(x[i][e]));
      }
    }
  }
  {
    __shared__ float part[NT / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float* sp = (is_v ? c.v_scale : c.k_scale) + static_cast<long long>(id) * c.hkv + h;
    const float was = *sp;                          // every thread reads it before it changes
    if constexpr (NT > 32) {
      if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < NT / 32; ++w) amax = fmaxf(amax, part[w]);
    } else {
      __syncwarp();
    }
    float scale = e4m3_scale(amax);
    if (slot0 > 0) scale = fmaxf(scale, was);
    if (threadIdx.x == 0) *sp = scale;
    if (slot0 > 0 && was < scale) {                 // earlier tokens of the block move along
      const float ratio = was / scale;
      uint4* old = reinterpret_cast<uint4*>(dst);
      for (int i = threadIdx.x; i < slot0 * (D / 16); i += NT) {
        uint4 w = old[i];
        w.x = rescale_e4m3x4(w.x, ratio);
        w.y = rescale_e4m3x4(w.y, ratio);
        w.z = rescale_e4m3x4(w.z, ratio);
        w.w = rescale_e4m3x4(w.w, ratio);
        old[i] = w;
      }
    }
    const float inv = 1.f / scale;                  // exact: a power of two
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int u = static_cast<int>(threadIdx.x) + i * NT;
      const int tok = u / kUnits, cu = u % kUnits;
      if (tok < n) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = pack_e4m3x2(x[i][4 * e] * inv, x[i][4 * e + 1] * inv) |
                 (pack_e4m3x2(x[i][4 * e + 2] * inv, x[i][4 * e + 3] * inv) << 16);
        uint8_t* row = dst + (slot0 + tok) * D;
        if (inter) {
          *reinterpret_cast<uint4*>(row + 16 * cu) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          *reinterpret_cast<uint2*>(row + 8 * cu) = make_uint2(w[0], w[1]);
          *reinterpret_cast<uint2*>(row + D / 2 + 8 * cu) = make_uint2(w[2], w[3]);
        }
      }
    }
  }
}

}  // namespace sta
