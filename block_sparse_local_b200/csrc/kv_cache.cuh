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

// Set when a kernel met a block index outside the cache, or a length beyond
// the block table: the access was skipped.  Read and cleared by
// sta_device_status(); no kernel looks at it, so later calls are not affected.
__device__ unsigned int g_kv_bounds = 0;

__device__ __forceinline__ void kv_bad_index() { atomicOr(&g_kv_bounds, 1u); }

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
  int rope_rows;
  int interleaved;               // pairs (2i, 2i + 1) instead of (i, i + d/2)
  int pages;                     // blocks that S tokens can touch, at most
  int kv_blocks;                 // thread blocks of the key/value part
};

// One unit of work is 16 elements of a token's row, a vector of 8 pairs: the
// pairs (i, i + d/2) of 8 consecutive i, or 8 consecutive pairs (2i, 2i + 1).
// So the two 16-byte loads of a unit hold whole pairs in either layout.
template <int D>
__device__ __forceinline__ void unit_load(const __nv_bfloat16* row, int c, bool interleaved,
                                          float x[16]) {
  const int e0 = interleaved ? 16 * c : 8 * c;
  const int e1 = interleaved ? 16 * c + 8 : D / 2 + 8 * c;
  const uint4 a = *reinterpret_cast<const uint4*>(row + e0);
  const uint4 b = *reinterpret_cast<const uint4*>(row + e1);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Rotates the unit's pairs by the angles of one position: (a, b) becomes
// (a cos - b sin, b cos + a sin), in fp32 from the fp32 table.  Products and
// sums are rounded one by one (no multiply-add), as elementary operations
// round them elsewhere: the kernel waits for memory, and a token gets the same
// e4m3 number whichever program stored it.
template <int D>
__device__ __forceinline__ void unit_rotate(const float* rope, long long pos, int c,
                                            bool interleaved, float x[16]) {
  const float4* cs = reinterpret_cast<const float4*>(rope + pos * D + 8 * c);
  const float4* sn = reinterpret_cast<const float4*>(rope + pos * D + D / 2 + 8 * c);
  float co[8], si[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 a = __ldg(cs + h), b = __ldg(sn + h);
    co[4 * h] = a.x; co[4 * h + 1] = a.y; co[4 * h + 2] = a.z; co[4 * h + 3] = a.w;
    si[4 * h] = b.x; si[4 * h + 1] = b.y; si[4 * h + 2] = b.z; si[4 * h + 3] = b.w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    if (interleaved) { a = x[2 * i]; b = x[2 * i + 1]; }
    else { a = x[i]; b = x[8 + i]; }
    const float y0 = __fsub_rn(__fmul_rn(a, co[i]), __fmul_rn(b, si[i]));
    const float y1 = __fadd_rn(__fmul_rn(b, co[i]), __fmul_rn(a, si[i]));
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

// kv_append_kernel: the first kv_blocks thread blocks store keys and values,
// one (sequence, touched cache block, head, K or V) each; the others rotate
// queries, one unit per thread.
//
// Memory-bound: every input is read once and every output written once.  One
// thread block owns a whole (cache block, head), so the block's amax, its
// scale and the numbers that the scale covers meet in registers and shared
// memory, with one read of the tokens, no second pass and no atomics.
// NT threads with U units each hold up to NT * U / (D/16) tokens.
template <int D, bool F8, int NT, int U>
__global__ void __launch_bounds__(NT) kv_append_kernel(const AppendParams p) {
  constexpr int kUnits = D / 16;                    // units of a row
  const bool inter = p.interleaved != 0;
  const KvLayout& c = p.c;
  if (static_cast<int>(blockIdx.x) >= p.kv_blocks) {
    // ---------------------------------------------------------------- queries
    const long long u = static_cast<long long>(blockIdx.x - p.kv_blocks) * NT + threadIdx.x;
    const int cu = static_cast<int>(u % kUnits);
    const long long row = u / kUnits;               // (b, s, h), heads fastest
    const unsigned int hq = static_cast<unsigned int>(c.hq);
    const unsigned int bs = static_cast<unsigned int>(row / hq);
    const int h = static_cast<int>(row - static_cast<long long>(bs) * hq);
    const int b = static_cast<int>(bs / static_cast<unsigned int>(c.S));
    const int s = static_cast<int>(bs % static_cast<unsigned int>(c.S));
    if (b >= c.B) return;
    const KvSeqLen sl = kv_seq(c, b);
    const int pos = sl.pos0 + s;
    if (s >= sl.fresh || pos < 0 || pos >= p.rope_rows) return;
    float x[16];
    unit_load<D>(p.q + b * p.qs.b + h * p.qs.h + s * p.qs.s, cu, inter, x);
    unit_rotate<D>(p.rope, pos, cu, inter, x);
    unit_store_bf16<D>(p.q_out + b * p.os.b + h * p.os.h + s * p.os.s, cu, inter, x);
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
      if (turn) unit_rotate<D>(p.rope, lo + tok, cu, inter, x[i]);
      if constexpr (F8) {
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, finite_abs(x[i][e]));
      } else {
        unit_store_bf16<D>(reinterpret_cast<__nv_bfloat16*>(dst) + (slot0 + tok) * D, cu, inter,
                           x[i]);
      }
    }
  }
  if constexpr (F8) {
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
