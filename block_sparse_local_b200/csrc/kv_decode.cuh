// kv_decode.cuh - attention of a few new tokens per sequence over the paged
// key/value cache (kv_cache.cuh).
//
// For query row r = (token s, head g of the key head's group), position
// p = seq_len - new_len + s:
//   out_r = sum_j w_rj V_j / sum_j w_rj,  w_rj = exp(q_r . K_j / sqrt(d)),
// j over the cached positions in (p - window, p].  With an 8-bit cache K_j and
// V_j are e4m3 numbers times a scale per (block, head).  The scales never
// touch the numbers: with x_j = log2(e)/sqrt(d) * ks_j * (q . k_j) and a
// reference M near the maximum of x_j + log2 vs_j, the kernel accumulates
//   O = sum_j e_j v_j,  l = sum_j e_j / vs_j,  e_j = 2^(x_j + log2 vs_j - M),
// so that O / l is the result.
//
// What bounds it: the cache is read once, 2 d bytes (e4m3) per token and key
// head against 4 d flops for each of the (few) query rows, so HBM.  So nothing
// may be done to the cached numbers on the way: they go by TMA into swizzled
// shared memory and from there into tcgen05 products as they are.  The products
// are transposed, S^T = K Q^T and O^T += V^T P^T, so that the 128 rows of an
// MMA are tokens (and then columns of V), and the few queries are its N:
//  * e4m3 keys want 8-bit queries.  A row, scaled by a power of two to below
//    448, is the sum of two e4m3 numbers per element, hi + lo: exact for bf16's 8
//    bits down to 2^-10 of the row's largest element, and off by at most 2^-17 of
//    that below (the largest is above 2^7, and half of the last step is 2^-10).
//  * e4m3 values want 8-bit weights.  A weight is the sum of three e5m2 numbers,
//    each what the ones before it left: 2^-9 relative (a bf16 weight has 2^-8),
//    and e5m2 has f16's exponents, so that weights down to 2^-27 of the largest
//    count (kDecodeLift).
//  * a bf16 cache takes bf16 queries, and a weight is the sum of two bf16 numbers
//    (one, for lack of shared memory, with more than 32 rows).
// The terms of a row are rows of their own in N (with 64 query rows, whose
// accumulators would not fit, the two products of a query go into one): an MMA
// this narrow costs what reading its 128 rows from shared memory costs, about 48
// cycles, whatever its N.
// A thread of the softmax has one token and up to 32 query rows: the scales are
// constants of the thread, no maximum is exchanged as long as no score passes
// the reference by much (a vote), and l is summed up at the end of an item.
//
// Two groups of one or two warpgroups: softmax of even and odd tiles, each with
// its own reference, sums and accumulator, so that one's exponentials run beside
// the other's products; at the end of an item the group that had its last tile
// joins the two parts, while the other goes on.  With more than 16 rows
// a group's two warpgroups share the rows.  One more warp issues the products,
// one prepares the queries of the next item, one copies keys and one values (a
// copy takes a warp about 65 cycles to issue, and with short blocks there are
// many).  The work is divided as
// in kv_split.cuh, a thread block per SM.
//
// Measured (e4m3, d = 128, 32 query and 8 key heads, joining included, among other
// calls): 64 sequences of up to 8192 tokens 107 to 113 us, box to box (5.3 to 5.5
// TB/s; a copy runs at 6.5), two of 131071 93 to 95 us (5.6 to 5.7 TB/s), one of 4096
// 16.4 us (launches and the latency of one tile: 2 us until the division is known, 2
// to the first scores, 4 to the end).
// An item costs about 4 us besides its tiles, which the copies of the next item
// hide only in part; that is what short contexts pay.
#pragma once

#include "kv_chunk.cuh"
#include "kv_split.cuh"

namespace sta {

// log2 of what the weight of the reference is, and how far (log2) a score may
// pass the reference before that moves: weights stay below 2^15, inside e5m2's
// and f16's range, and e4m3 weights are lost below 2^-17 only, 2^-27 of the
// reference's, so that 2^17 lost ones add up to less than a bf16 rounding.
constexpr float kDecodeLift = 10.f;
constexpr float kDecodeLag = 5.f;

// A reference M is kept as what is added to a score, kDecodeLift - M; a row that
// has seen nothing yet has one that any score passes, and -inf does not.
constexpr float kNoRef = 1e30f;
__device__ __forceinline__ float ref_of(float add) {
  return add == kNoRef ? -INFINITY : kDecodeLift - add;
}
__device__ __forceinline__ float add_of(float ref) {
  return ref == -INFINITY ? kNoRef : kDecodeLift - ref;
}

template <int D, bool F8, int ROWS>
struct DecodeCfg {
  static constexpr int kRows = ROWS;                        // query rows of an item: 8, 16, 32, 64
  static constexpr int kTile = 128;                         // tokens
  static constexpr int kElem = F8 ? 1 : 2;
  static constexpr int kRowBytes = D * kElem;
  static constexpr int kSwizzle = kRowBytes < 128 ? kRowBytes : 128;   // 64 or 128 bytes
  static constexpr int kPanels = kRowBytes / kSwizzle;
  static constexpr int kPanelBytes = kTile * kSwizzle;
  static constexpr int kTileBytes = kPanels * kPanelBytes;
  static constexpr int kStageBytes = 2 * kTileBytes;        // keys and values
  // See kv_split.cuh: an item costs about 4 us by itself, a tile 0.6 us for every
  // 32 KB (solved from the times of thread blocks with 2 to 10 items).
  static constexpr int kOver = kStageBytes >= 65536 ? 3 : kStageBytes >= 32768 ? 7 : 10;
  static constexpr int kK = F8 ? 32 : 16;                   // K of an MMA

  static constexpr int kSplitRows = ROWS <= 16 ? 1 : 2;     // warpgroups of a group
  static constexpr int kWgRows = ROWS / kSplitRows;         // rows of a warpgroup
  static constexpr int kPart = ROWS < 16 ? ROWS : 16;       // rows whose terms lie together
  static constexpr int kParts = ROWS / kPart;

  // scores: per part the rows' hi terms, then the lo terms
  static constexpr bool kQCat = F8 && ROWS < 64;
  static constexpr int kQTerms = F8 ? 2 : 1;
  static constexpr int kQProds = F8 && !kQCat ? 2 : 1;
  static constexpr int kSPart = kPart * (kQCat ? 2 : 1);    // columns of a part
  static constexpr int kSN = kParts * kSPart < 16 ? 16 : kParts * kSPart;
  static constexpr int kQBytes = kQProds * kSN * kRowBytes;
  static constexpr int kSBufs = ROWS < 64 ? 2 : 1;          // per group
  // outputs: per part the rows of each term; weights in shared memory with the
  // rows contiguous, [chunk of 16 bytes of rows][token]
  static constexpr int kPTerms = F8 ? 3 : ROWS <= 32 ? 2 : 1;
  static constexpr int kOPart = kPart * kPTerms;
  static constexpr int kON = (kParts * kOPart + 15) / 16 * 16;
  static constexpr int kPChunk = kTile * 16;
  static constexpr int kPBytes = kON * kElem / 16 * kPChunk;
  static constexpr int kPBufs = ROWS <= (F8 ? 16 : 8) ? 2 : 1;   // per group

  static constexpr int kMisc = 3 * 1024 + ROWS * 128;
  static constexpr int kFit = (227 * 1024 - 2048 - kMisc - 2 * kQBytes - 2 * kPBufs * kPBytes) /
                              kStageBytes;
  static constexpr int kStages = kFit < 12 ? kFit : 12;
  static constexpr int kQOff = kStages * kStageBytes;       // [2] by piece
  static constexpr int kPOff = kQOff + 2 * kQBytes;         // [2 groups][kPBufs]
  static constexpr int kScaleOff = kPOff + 2 * kPBufs * kPBytes;    // [stage][8 blocks] {k, v}
  static constexpr int kRowOff = kScaleOff + kStages * 64;  // [2 pieces][rows] factor of a score
  static constexpr int kPosOff = kRowOff + 2 * kRows * 4;   // [2 pieces][rows] position
  static constexpr int kRefOff = kPosOff + 2 * kRows * 4;   // [4 pieces][2 groups][rows]
  static constexpr int kSumOff = kRefOff + 8 * kRows * 4;   // [2 pieces][2 groups][4 warps][rows]
  static constexpr int kEndOff = kSumOff + 16 * kRows * 4;  // [2 pieces][rows] {two factors}
  static constexpr int kPieceRing = 16;
  static constexpr int kAlphaOff = kEndOff + 2 * kRows * 8;    // [2 groups][rows]
  static constexpr int kPieceOff = kAlphaOff + 2 * kRows * 4;
  static constexpr int kBarOff = kPieceOff + kPieceRing * 64;
  static constexpr int kSmemBytes = kBarOff + 704 + 1024;   // + alignment
  static constexpr int kSoftWarps = 8 * kSplitRows;
  static constexpr int kWarpMma = kSoftWarps;
  static constexpr int kWarpKeys = kSoftWarps + 1;
  static constexpr int kWarpValues = kSoftWarps + 2;
  static constexpr int kWarpQuery = kSoftWarps + 3;
  static constexpr int kThreads = 32 * (kSoftWarps + 4);
  // columns: score tiles of group 0, of group 1, then O0 and O1, of even and of
  // odd pieces where there is room
  static constexpr uint32_t kOCol = 2 * kSBufs * kSN;
  static constexpr int kOBufs = kOCol + 4 * kON <= 512 ? 2 : 1;
  static constexpr uint32_t kCols = kOCol + 2 * kOBufs * kON;
  static constexpr uint32_t kTmemCols = kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512 && kBarOff - kScaleOff <= kMisc - 704 && kStages >= 2, "");
};

// Matrix descriptor with 128- or 64-byte swizzle.
template <int SWIZZLE>
__device__ __forceinline__ uint64_t sdesc_sw(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  const uint64_t d = sdesc_sw128(saddr, lbo, sbo);
  return SWIZZLE == 128 ? d : (d & ~(7ull << 61)) | (4ull << 61);
}

// Matrix descriptor without swizzle, for an operand whose M or N dimension is
// contiguous: 8 rows (of K) of 16 bytes are 128 consecutive bytes; `kstep` bytes
// to the next 8 rows, `nstep` to the next 16 bytes of M or N.
__device__ __forceinline__ uint64_t sdesc_plain_mn(uint32_t saddr, uint32_t kstep,
                                                   uint32_t nstep) {
  return sdesc_sw128(saddr, kstep, nstep) & ~(7ull << 61);
}

// Instruction descriptor: fp32 accumulators; F8: kind::f8f6f4 with A e4m3 and B
// e4m3, else kind::f16 with bf16 operands.  Of the product with the values both
// operands have K as the outer dimension, and F8 weights are e5m2.
template <bool F8>
__host__ __device__ constexpr uint32_t idesc_few(int M, int N, bool values) {
  return (1u << 4) | (F8 ? (values ? 1u << 10 : 0u) : (1u << 7) | (1u << 10)) |
         (values ? (1u << 15) | (1u << 16) : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

template <bool F8>
__device__ __forceinline__ void umma_few(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  if constexpr (F8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a),
        "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    umma_ss(d, a, b, idesc, accumulate);
}

// N consecutive columns of this thread's TMEM lane, N = 8 or 16.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float* x) {
  static_assert(N == 8 || N == 16, "");
  uint32_t r[N];
  if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  else
    STA_TMEM_LD16(taddr, r);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = __uint_as_float(r[i]);
}

// Twice 8 columns of this thread's lane, one wait.
__device__ __forceinline__ void tmem_ld_2x8(uint32_t ta, uint32_t tb, float* a, float* b) {
  uint32_t r[16];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(ta));
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
                 "=r"(r[14]), "=r"(r[15])
               : "r"(tb));
  // (the registers hold the values after the wait only: tied to it)
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = __uint_as_float(r[i]);
    b[i] = __uint_as_float(r[8 + i]);
  }
}

template <int N>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const float* x) {
  uint32_t r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = __float_as_uint(x[i]);
  if constexpr (N == 8) STA_TMEM_ST8(taddr, r);
  else STA_TMEM_ST16(taddr, r);
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

// 4 bytes to shared memory, 0 where nothing is to be read.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
// One of the arrivals that `bar` counts on, once this thread's cp.async copies
// so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// Block numbers of a piece, 32 at a time and as many ahead: lane l of tile j
// asks for the tile's block l.
struct BlockIds {
  const int* table;
  int lo, hi, first, shift;          // of the piece: tokens; first token; log2(block)
  int chunk, now, ahead;
  __device__ __forceinline__ int fetch(int c) const {     // -2: nothing to load
    const int t = first + ((32 * c + static_cast<int>(threadIdx.x & 31)) << shift);
    return t < hi && t + (1 << shift) > lo ? __ldg(table + (t >> shift)) : -2;
  }
  __device__ __forceinline__ void start(const int* tab, int l, int h, int t0, int sh) {
    table = tab;
    lo = l;
    hi = h;
    first = t0;
    shift = sh;
    chunk = 0;
    now = fetch(0);
    ahead = fetch(1);
  }
  __device__ __forceinline__ int at(int j, int blocks) {  // all lanes, j ascending
    const int lane = threadIdx.x & 31, i = j * blocks;
    if ((i >> 5) != chunk) {
      ++chunk;
      now = ahead;
      ahead = fetch(chunk + 1);
    }
    const int id = __shfl_sync(0xffffffffu, now, (i + lane) & 31);
    return lane < blocks ? id : -2;
  }
};

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// Sums of N <= 32 values over a warp's lanes by halves: every lane whose number
// is i modulo N gets the sum of value i.  x is overwritten.
template <int N>
__device__ __forceinline__ float warp_sums(float* x, int lane) {
#pragma unroll
  for (int k = N / 2; k >= 1; k /= 2) {
    const bool up = (lane & k) != 0;
#pragma unroll
    for (int i = 0; i < k; ++i) {
      const float send = up ? x[i] : x[i + k];
      const float keep = up ? x[i + k] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, send, k);
    }
  }
  float s = x[0];
#pragma unroll
  for (int o = N; o < 32; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <int D, bool F8, int ROWS>
__global__ void __launch_bounds__(DecodeCfg<D, F8, ROWS>::kThreads, 1)
    kv_decode_kernel(const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const AttendParams p) {
  using C = DecodeCfg<D, F8, ROWS>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* v_full = k_full + NS;
  uint64_t* empty = v_full + NS;
  uint64_t* s_full = empty + NS;      // [2][2] by group: scores in TMEM
  uint64_t* p_full = s_full + 4;      // [2][2] by group and buffer: weights in shared memory
  uint64_t* pv_done = p_full + 4;     // [2][2] their product is in O
  uint64_t* q_full = pv_done + 4;     // [2] by piece
  uint64_t* q_empty = q_full + 2;     // [2] all products of a piece done
  uint64_t* pc_full = q_empty + 2;    // [ring]
  uint64_t* w_sync = pc_full + C::kPieceRing;   // [4] a warpgroup's warps
  uint64_t* ended = w_sync + 4;       // [2] by piece: all softmax warps are through it
  uint64_t* joined = ended + 2;       // [2] its parts have been joined
  uint64_t* q_first = joined + 2;     // queries of the first piece
  uint64_t* mma_done = q_first + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* dropped = abort_flag + 1;   // infinities or NaN left out of a product
  volatile int* votes = dropped + 1;  // [4][2] the warpgroup's last tile that passed a reference
  static_assert((3 * NS + 16 + C::kPieceRing + 10) * 8 + 44 <= 704, "barriers");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // barriers, a thread each, and how many arrive on them
  for (int i = threadIdx.x; &k_full[i] <= mma_done; i += C::kThreads) {
    uint64_t* bar = &k_full[i];
    int count = 1;
    if (i < NS) count = F8 ? 33 : 1;                  // keys: with the 32 lanes' scales
    else if (bar >= p_full && bar < pv_done) count = 4 * C::kSplitRows;
    else if (bar >= w_sync && bar < ended) count = 4;
    else if (bar >= ended && bar < joined) count = C::kSoftWarps;
    else if (bar >= joined && bar < q_first) count = 4 * C::kSplitRows;
    else if (bar == q_first) count = C::kSoftWarps;
    mbar_init(bar, count);
  }
  if (threadIdx.x < 8) votes[threadIdx.x] = 0;
  if (threadIdx.x == 32) *abort_flag = error_raised() ? 1 : 0;
  if (threadIdx.x == 0) *dropped = 0;
  fence_mbar_init();
  if (warp == C::kWarpMma) tmem_alloc(tmem_holder, C::kTmemCols);
  tc_fence_before();
  const KvRange range = kv_range<D, C::kRows, C::kTile, C::kOver, C::kThreads>(p);  // synchronises
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const bool skip = *abort_flag != 0;
  const ChunkPiece* pieces = reinterpret_cast<const ChunkPiece*>(smem + C::kPieceOff);
  auto wait_piece = [&](int np) -> const ChunkPiece* {
    const int i = np % C::kPieceRing;
    return mbar_wait_warp(&pc_full[i], (np / C::kPieceRing) & 1, abort_flag) ? pieces + i : nullptr;
  };

  // The queries of piece np into their buffer, by `threads` threads, D / 8 per row,
  // and for every row the factor of its scores and its position; no references
  // yet (of four sets: the earlier pieces' are read until their parts are joined).
  auto prepare = [&](int np, const ChunkPiece* w, int thread, auto threads) {
    constexpr int PT = C::kPart, kBy = decltype(threads)::value;
    constexpr int kLanes = D / 8, kStep = kBy / kLanes;       // threads per row; rows at once
    constexpr int kTurns = (ROWS + kStep - 1) / kStep, kAhead = kTurns < 8 ? kTurns : 8;
    const int qb = np & 1;
    const int e = thread % kLanes;
    const int rows = w->rows, row0 = w->row0, pos0 = w->pos0;
    const __nv_bfloat16* base = p.q + w->b * p.qs.b +
                                static_cast<long long>(w->h) * p.group * p.qs.h + 8 * e;
    const uint32_t to = sbase + C::kQOff + qb * C::kQBytes;
    for (int k0 = 0; k0 < kTurns; k0 += kAhead) {
      uint4 x[kAhead];                                // loads first, all on their way
      int pos[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = (k0 + k) * kStep + thread / kLanes;
        const bool live = r < rows;
        const int row = row0 + (live ? r : rows - 1);
        const int t = row / p.group, g = row - t * p.group;
        pos[k] = pos0 + t;
        x[k] = live ? *reinterpret_cast<const uint4*>(base + g * p.qs.h + t * p.qs.s)
                    : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int r = (k0 + k) * kStep + thread / kLanes;
        float factor = p.scale_log2;
        if constexpr (F8) {
          float m = fmaxf(fmaxf(bf16x2_max_abs(x[k].x), bf16x2_max_abs(x[k].y)),
                          fmaxf(bf16x2_max_abs(x[k].z), bf16x2_max_abs(x[k].w)));
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          // to [2^7, 2^8): both terms inside e4m3's range
          const QueryScale qs = query_scale<7>(m);
          const float down = qs.down;
          factor *= qs.up;
          const uint32_t w4[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
          uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = __uint_as_float(w4[i] << 16) * down;
            const float b = __uint_as_float(w4[i] & 0xffff0000u) * down;
            const uint32_t h = pack_e4m3x2(a, b);
            const uint32_t back = e4m3x2_to_f16x2(h);
            const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&back));
            const uint32_t l = pack_e4m3x2(a - hf.x, b - hf.y);
            hi[i >> 1] |= h << (16 * (i & 1));
            lo[i >> 1] |= l << (16 * (i & 1));
          }
          // row of the operand; 16-byte chunk e / 2 of it, its half e % 2
          const int qr = C::kQCat ? r / PT * C::kSPart + r % PT : r;
          constexpr int kLo = (C::kQCat ? PT : C::kSN) * C::kSwizzle;
          const int sw = C::kSwizzle == 128 ? (qr & 7) : ((qr >> 1) & 3);
          const uint32_t at = to + qr * C::kSwizzle + (((e >> 1) ^ sw) << 4) + (e & 1) * 8;
          if (r < ROWS) {
            sts64(at, hi[0], hi[1]);
            sts64(at + kLo, lo[0], lo[1]);
          }
        } else if (r < ROWS) {
          const uint32_t at = to + (e >> 3) * (C::kSN * 128) + r * 128 +
                              (((e & 7) ^ (r & 7)) << 4);
          sts128(at, bf16x2_inf_to_nan(x[k].x), bf16x2_inf_to_nan(x[k].y),
                 bf16x2_inf_to_nan(x[k].z), bf16x2_inf_to_nan(x[k].w));
        }
        if (e == 0 && r < ROWS) {
          sts32(sbase + C::kRowOff + (qb * ROWS + r) * 4, __float_as_uint(factor));
          sts32(sbase + C::kPosOff + (qb * ROWS + r) * 4, static_cast<uint32_t>(pos[k]));
        }
      }
    }
    for (int i = thread; i < 2 * ROWS; i += kBy)
      sts32(sbase + C::kRefOff + (np % 4 * 2 * ROWS + i) * 4, __float_as_uint(kNoRef));
    fence_async_shared();
    __syncwarp();
  };
  // the first piece's come from all softmax warps, the others' from one warp
  auto wait_queries = [&](int np) {
    return np == 0 ? mbar_wait_warp(q_first, 0, abort_flag)
                   : mbar_wait_warp(&q_full[np & 1], ((np >> 1) + (np & 1) + 1) & 1, abort_flag);
  };

  if (skip) {
    // a wait gave up earlier: nothing is computed
  } else if (warp == C::kWarpKeys || warp == C::kWarpValues) {
    // ------------------------------------------------------------ copies
    // Lane l < 128 / block has the tile's block l.
    const bool values = warp == C::kWarpValues;
    const KvLayout& c = p.c;
    const int block = 1 << c.shift, blocks = C::kTile >> c.shift;
    const uint64_t pol = policy_evict_first();
    int jt = 0;
    bool ok = true;
    KvPiece pc;
    pc.start(range);
    for (int np = 0; ok; ++np) {
      if (!values) {
        // the warp that copies keys also finds the pieces; the ring holds more of
        // them than there are stages: none is overwritten before its last tile's
        // stage is free
        const bool more = pc.next<C::kRows, C::kTile, C::kOver>(p, range);
        if (lane == 0) {
          const ItemRange& r = pc.r;
          ChunkPiece w;
          w.n = more ? pc.t1 - pc.t0 : 0;
          if (more) {
            w.t0 = pc.tok0<C::kTile>();
            w.b = pc.b;
            w.h = pc.h;
            w.row0 = pc.row0;
            w.rows = r.rows;
            w.pos0 = r.pos0;
            w.len = r.len;
            w.lo = r.lo;
            w.hi = r.hi;
            w.all[0] = w.all[1] = seen_by_all(p, r, pc.row0, pc.row0 + r.rows - 1);
            w.whole = pc.whole();
            w.slot = static_cast<int>(pc.slot());
            pc.leave<C::kOver>(p, range);
          }
          *reinterpret_cast<ChunkPiece*>(smem + C::kPieceOff + np % C::kPieceRing * 64) = w;
          mbar_arrive(&pc_full[np % C::kPieceRing]);
        }
        __syncwarp();
      }
      const ChunkPiece* w = wait_piece(np);
      const int n = w != nullptr ? w->n : 0;
      if (n == 0) break;
      const int h = w->h;
      BlockIds ids;
      ids.start(c.table + static_cast<long long>(w->b) * c.width, w->lo, w->hi, w->t0, c.shift);
      for (int j = 0; j < n; ++j) {
        const int J = jt + j, st = J % NS;
        const int id = ids.at(j, blocks);
        const bool good = id >= 0 && id < c.num_blocks;
        if (!good && id != -2) kv_bad_index();
        const uint32_t count = __popc(__ballot_sync(0xffffffffu, good));
        const uint32_t bytes = count * (C::kRowBytes << c.shift);
        if (J >= NS && !mbar_wait_warp(&empty[st], ((J / NS) - 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        uint64_t* bar = values ? &v_full[st] : &k_full[st];
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        uint8_t* dst = smem + st * C::kStageBytes + (values ? C::kTileBytes : 0) +
                       lane * block * C::kSwizzle;
        if (good) {
#pragma unroll
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_4d(dst + pn * C::kPanelBytes, values ? &tmap_v : &tmap_k, bar,
                        pn * (C::kSwizzle / C::kElem), 0, h, id, pol);
        }
        if constexpr (F8) {
          if (!values) {
            const long long at = static_cast<long long>(good ? id : 0) * c.hkv + h;
            if (lane < blocks) {
              const uint32_t to = sbase + C::kScaleOff + st * 64 + lane * 8;
              cp_async4(to, c.k_scale + at, good);
              cp_async4(to + 4, c.v_scale + at, good);
            }
            cp_async_arrive(bar);
          }
        }
      }
      jt += n;
    }
    if (!ok) {
      // a wait gave up: no copy may be in flight when the block ends
      asm volatile("cp.async.wait_all;" ::: "memory");
      const uint64_t t = globaltimer_ns();
      while (globaltimer_ns() - t < 1000000ull) {
      }
    }
  } else if (warp == C::kWarpQuery) {
    // ------------------------------------------------------------ queries
    // of the next piece, as soon as the one before the last has no products
    // outstanding
    for (int np = 0;; ++np) {
      const ChunkPiece* w = wait_piece(np);
      if (w == nullptr || w->n == 0) break;
      if (np == 0) continue;
      if (np >= 2 && !mbar_wait_warp(&q_empty[np & 1], ((np >> 1) - 1) & 1, abort_flag)) break;
      prepare(np, w, lane, std::integral_constant<int, 32>{});
      if (lane == 0) mbar_arrive(&q_full[np & 1]);
    }
  } else if (warp == C::kWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t tm = warp_uniform(tmem);
    const uint32_t sb = warp_uniform(sbase);
    constexpr uint32_t kAtom = 8 * C::kSwizzle;       // 8 rows of a panel
    constexpr uint32_t kIdescS = idesc_few<F8>(128, C::kSN, false);
    constexpr uint32_t kIdescO = idesc_few<F8>(128, C::kON, true);
    // keys: rows of d; queries alike, with the keys' swizzle
    const uint64_t dk = sdesc_sw<C::kSwizzle>(sb, 16, kAtom);
    const uint64_t dq = sdesc_sw<C::kSwizzle>(sb + C::kQOff, 16, kAtom);
    // values: d along the rows.  With fewer than 128 columns (d = 64) the
    // second half of M repeats the first (bf16: panel stride 0; e4m3: 64-byte
    // rows, likewise)
    constexpr uint32_t kPanelStep = D == 128 ? C::kPanelBytes : 0;
    const uint64_t dv = sdesc_sw<C::kSwizzle>(sb + C::kTileBytes, kPanelStep, kAtom);
    const uint64_t dp = sdesc_plain_mn(sb + C::kPOff, 128, C::kPChunk);
    auto issue_s = [&](int st, int buf, int qb) {
      const uint64_t a = dk + ((st * C::kStageBytes) >> 4);
#pragma unroll
      for (int t = 0; t < C::kQProds; ++t) {
        const uint64_t b = dq + ((qb * C::kQBytes + t * C::kSN * C::kRowBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / C::kK; ++kk) {
          const int byte = kk * 32, pn = byte / C::kSwizzle, in = byte % C::kSwizzle;
          umma_few<F8>(tm + buf * C::kSN, a + ((pn * C::kPanelBytes + in) >> 4),
                       b + ((pn * C::kSN * C::kSwizzle + in) >> 4), kIdescS, t + kk > 0 ? 1u : 0u);
        }
      }
    };
    auto issue_pv = [&](int st, int ocol, int pbuf, bool first) {
      const uint64_t a = dv + ((st * C::kStageBytes) >> 4);
      const uint64_t b = dp + ((pbuf * C::kPBytes) >> 4);
#pragma unroll
      for (int kk = 0; kk < C::kTile / C::kK; ++kk)
        umma_few<F8>(tm + ocol, a + ((kk * C::kK * C::kSwizzle) >> 4),
                     b + ((kk * C::kK * 16) >> 4), kIdescO, kk > 0 ? 1u : (first ? 0u : 1u));
    };
    // Scores are issued up to two tiles (one of each group) ahead of the products
    // with the values, as far as there are stages and score buffers.  Tile J
    // belongs to group J % 2, its scores to the group's buffer (J / 2) % kSBufs,
    // last read for tile J - 2 kSBufs.
    constexpr int kLead = NS > 2 && C::kSBufs > 1 ? 2 : 1;
    int js = 0, jo = 0;                // tiles whose scores, whose products are issued
    // of the tiles in between, by the last bits of their numbers: a group's first
    // of a piece, the last of a piece, of an odd piece
    uint32_t first = 0, last = 0, odd = 0;
    int start = 0;                     // first tile of the piece before
    bool ok = true;
    auto finish = [&]() {
      const int st = jo % NS, g = jo & 1, pb = (jo >> 1) % C::kPBufs;
      const uint32_t bit = 1u << (jo & 31);
      if (!mbar_wait_warp(&v_full[st], (jo / NS) & 1, abort_flag) ||
          !mbar_wait_warp(&p_full[2 * g + pb], ((jo >> 1) / C::kPBufs) & 1, abort_flag))
        return false;
      tc_fence_after();
      const int par = (odd & bit) ? 1 : 0;
      if (elect_one()) {
        issue_pv(st, C::kOCol + (par % C::kOBufs * 2 + g) * C::kON, g * C::kPBufs + pb,
                 (first & bit) != 0);
        umma_commit(&pv_done[2 * g + pb]);
        umma_commit(&empty[st]);
        if (last & bit) umma_commit(&q_empty[par]);
      }
      __syncwarp();
      ++jo;
      return true;
    };
    for (int np = 0; ok; ++np) {
      const ChunkPiece* w = wait_piece(np);
      const int n = w != nullptr ? w->n : 0;
      if (n == 0) break;
      // these queries take the buffer of the last piece but one: its products first
      while (ok && jo < start) ok = finish();
      start = js;
      ok = ok && wait_queries(np);
      for (int j = 0; ok && j < n; ++j) {
        const int st = js % NS, buf = (js & 1) * C::kSBufs + ((js >> 1) % C::kSBufs);
        const uint32_t bit = 1u << (js & 31);
        first = j < 2 ? first | bit : first & ~bit;
        last = j == n - 1 ? last | bit : last & ~bit;
        odd = np & 1 ? odd | bit : odd & ~bit;
        ok = mbar_wait_warp(&k_full[st], (js / NS) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          issue_s(st, buf, np & 1);
          umma_commit(&s_full[buf]);
        }
        __syncwarp();
        ++js;
        if (js - jo > kLead) ok = finish();
      }
    }
    while (ok && jo < js) ok = finish();
    // No MMA may still run when TMEM is released.
    if (elect_one()) umma_commit(mma_done);
    __syncwarp();
    mbar_wait_drain(mma_done, 0);
  } else {
    // ------------------------------------------------------------ softmax
    const int wg = warp >> 2;                         // warpgroup
    const int grp = wg / C::kSplitRows;               // group: tiles of parity grp
    const int wrow = wg % C::kSplitRows * C::kWgRows; // first of its rows
    const int tid = threadIdx.x & 127;                // token of the tile; TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // lane quarter * 32 << 16
    // Barrier of the warpgroup's warps; bounded, as every wait.
    uint32_t w_phase = 0;
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&w_sync[wg]);
      return mbar_wait_warp(&w_sync[wg], w_phase++ & 1, abort_flag);
    };
    // rows are worked on 8 at a time, in a part of kPart that lie together
    constexpr int CH = 8, PT = C::kPart;
    constexpr bool kKeep = ROWS <= 16;                // scores stay in registers
    // first column of row r, a multiple of 8, in a score tile and in O
    auto s_col = [&](int r) { return r / PT * C::kSPart + r % PT; };
    auto o_col = [&](int r) { return r / PT * C::kOPart + r % PT; };

    // Waits until the group's product of its tile m is in O.  Called at the latest
    // kPBufs tiles later, so that the barrier cannot be a phase further.
    auto product = [&](int m) {
      return mbar_wait_warp(&pv_done[2 * grp + m % C::kPBufs], (m / C::kPBufs) & 1, abort_flag);
    };

    const ChunkPiece* w = wait_piece(0);
    int n = w != nullptr ? w->n : 0;
    bool ok = true;
    if (n > 0) {
      prepare(0, w, threadIdx.x, std::integral_constant<int, 32 * C::kSoftWarps>{});
      if (lane == 0) mbar_arrive(q_first);
    }
    int jt = 0;                                       // tiles so far
    int mine = 0;                                     // of this group
    for (int np = 0; n > 0; ++np) {
      const uint32_t rows_at = sbase + C::kRowOff + ((np & 1) * ROWS + wrow) * 4;
      const uint32_t pos_at = rows_at + (C::kPosOff - C::kRowOff);
      const SeenByAll all = w->all[0];
      float2 l[C::kWgRows / 2];
#pragma unroll
      for (int r = 0; r < C::kWgRows / 2; ++r) l[r] = make_float2(0.f, 0.f);
      const uint32_t t_o = tmem + lanes + C::kOCol + np % C::kOBufs * 2 * C::kON;   // O0, O1
      const uint32_t sums = sbase + C::kSumOff + (np & 1) * 8 * ROWS * 4;
      const uint32_t ends = sbase + C::kEndOff + (np & 1) * ROWS * 8;
      const uint32_t refs = sbase + C::kRefOff + np % 4 * 2 * ROWS * 4;     // of group 0
      const uint32_t my_refs = refs + (grp * ROWS + wrow) * 4;
      int done = 0;                                   // tiles of this piece that the group had
      // the accumulators and sums that it uses are free
      if (np >= C::kOBufs)
        ok = mbar_wait_warp(&joined[(np - C::kOBufs) & 1], ((np - C::kOBufs) >> 1) & 1, abort_flag);
      for (int j = 0; ok && j < n; ++j) {
        const int J = jt + j;
        if ((J & 1) != grp) continue;
        const int st = J % NS;
        const int t0 = w->t0 + j * C::kTile;
        const bool part = to_clean(all, t0);
        // the rows' factors, positions and references (a group without a tile does
        // not wait: the barrier may be a phase further by then)
        if (done == 0 && !wait_queries(np)) {
          ok = false;
          break;
        }
        if (!mbar_wait_warp(&k_full[st], (J / NS) & 1, abort_flag)) { ok = false; break; }
        KvScale sc{1.f, 0.f, 1.f};
        if constexpr (F8) {
          const uint2 x = lds64(sbase + C::kScaleOff + st * 64 + (tid >> p.c.shift) * 8);
          sc = kv_scale(__uint_as_float(x.x), __uint_as_float(x.y));
        }
        if (part && wrow == 0) {
          // Values of a token that not every row sees: zeros for the others'
          // weights to meet instead of infinities and NaN, and for what lies
          // outside the sequence.
          const int t = t0 + tid;
          if (t < all.lo || t >= all.hi) {
            if (!mbar_wait(&v_full[st], (J / NS) & 1, abort_flag)) ok = false;
            const bool in = t >= w->lo && t < w->hi;
            bool any = false;
#pragma unroll 1
            for (int ch = 0; ok && ch < C::kRowBytes / 16; ++ch) {
              const uint32_t at = sbase + st * C::kStageBytes + C::kTileBytes +
                                  (ch * 16 / C::kSwizzle) * C::kPanelBytes + tid * C::kSwizzle +
                                  ch * 16 % C::kSwizzle;
              uint4 x = lds128_at(at);
              bool hit = false;
              x.x = drop_nonfinite<F8>(x.x, hit);
              x.y = drop_nonfinite<F8>(x.y, hit);
              x.z = drop_nonfinite<F8>(x.z, hit);
              x.w = drop_nonfinite<F8>(x.w, hit);
              if (!in) sts128(at, 0u, 0u, 0u, 0u);
              else if (hit) sts128(at, x.x, x.y, x.z, x.w);
              any = any || (hit && in);
            }
            if (any) *dropped = 1;
          }
          ok = __all_sync(0xffffffffu, ok);
        }
        const int buf = grp * C::kSBufs + mine % C::kSBufs;
        const uint32_t t_s = tmem + lanes + buf * C::kSN;
        if (!ok || !mbar_wait_warp(&s_full[buf], (mine / C::kSBufs) & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();

        // x[r] = score of the warpgroup's row r0 + r in log2 units, plus log2 of the
        // value scale
        auto scores = [&](int r0, float2* x) {
          float* xs = reinterpret_cast<float*>(x);
          if constexpr (C::kQCat) {
            float lo[CH];
            tmem_ld_2x8(t_s + s_col(wrow + r0), t_s + s_col(wrow + r0) + PT, xs, lo);
#pragma unroll
            for (int r = 0; r < CH / 2; ++r)
              x[r] = __fadd2_rn(x[r], make_float2(lo[2 * r], lo[2 * r + 1]));
          } else {
            tmem_ld_cols<CH>(t_s + s_col(wrow + r0), xs);
          }
          const float2 k2 = make_float2(sc.k, sc.k), v2 = make_float2(sc.log2_v, sc.log2_v);
#pragma unroll
          for (int r = 0; r < CH; r += 4) {
            const uint4 f = lds128_at(rows_at + (r0 + r) * 4);
            const float2 fa = make_float2(__uint_as_float(f.x), __uint_as_float(f.y));
            const float2 fb = make_float2(__uint_as_float(f.z), __uint_as_float(f.w));
            x[r / 2] = __ffma2_rn(x[r / 2], __fmul2_rn(fa, k2), v2);
            x[r / 2 + 1] = __ffma2_rn(x[r / 2 + 1], __fmul2_rn(fb, k2), v2);
          }
          if (part) {
            const int t = t0 + tid;
#pragma unroll
            for (int r = 0; r < CH; r += 4) {
              const uint4 f = lds128_at(pos_at + (r0 + r) * 4);
              const uint32_t at[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int pos = static_cast<int>(at[k]);
                if (t > pos || (p.window > 0 && t <= pos - p.window)) xs[r + k] = -INFINITY;
              }
            }
          }
        };
        // ... relative to the rows' references, what 2^x is taken of
        auto shift = [&](int r0, float2* x) {
#pragma unroll
          for (int r = 0; r < CH; r += 4) {
            const uint4 f = lds128_at(my_refs + (r0 + r) * 4);
            x[r / 2] = __fadd2_rn(x[r / 2], make_float2(__uint_as_float(f.x),
                                                        __uint_as_float(f.y)));
            x[r / 2 + 1] = __fadd2_rn(x[r / 2 + 1], make_float2(__uint_as_float(f.z),
                                                                __uint_as_float(f.w)));
          }
        };
        float2 x[(kKeep ? C::kWgRows : CH) / 2];
        bool raise = done == 0;
        if (raise) {
          if constexpr (kKeep) {
#pragma unroll
            for (int r0 = 0; r0 < C::kWgRows; r0 += CH) scores(r0, x + r0 / 2);
          }
        } else {
          float top = -INFINITY;
#pragma unroll
          for (int r0 = 0; r0 < C::kWgRows; r0 += CH) {
            float2* y = kKeep ? x + r0 / 2 : x;
            scores(r0, y);
            shift(r0, y);
#pragma unroll
            for (int r = 0; r < CH / 2; ++r) top = fmax3(top, y[r].x, y[r].y);
          }
          // (a warp may vote on the next tile before another has read this vote: two
          // words; on the tile after that only once all have met again)
          volatile int* vote = votes + 2 * wg + (mine & 1);
          if (top > kDecodeLift + kDecodeLag) *vote = mine + 1;
          if (!meet()) { ok = false; break; }
          raise = *vote == mine + 1;
          if constexpr (kKeep) {
            if (raise) {
#pragma unroll
              for (int r0 = 0; r0 < C::kWgRows; r0 += CH) scores(r0, x + r0 / 2);
            }
          }
        }
        if (raise) {
          // The references rise to the tile's maxima (rare after the group's first
          // tile of an item), and what has been summed up is scaled; the group's last
          // product has to be in O by then.
          // The maxima are exchanged where the sums will be: they have been read when
          // the warps meet for the second time.  The factors are read after that, with
          // no barrier before a warp may leave its sums: they have a place of their own,
          // written again only after all warps have met in the group's next rise.  (With a
          // barrier instead: 39.0 us for 16 windows of 4096 tokens, 37.8 so.)
          const uint32_t exch = sums + (grp * 4 * ROWS + wrow) * 4;   // [4][rows]
          const uint32_t alphas = sbase + C::kAlphaOff + (grp * ROWS + wrow) * 4;
#pragma unroll
          for (int r0 = 0; r0 < C::kWgRows; r0 += CH) {
            float2* y = kKeep ? x + r0 / 2 : x;
            if constexpr (!kKeep) scores(r0, y);
#pragma unroll
            for (int r = 0; r < CH; ++r) {
              const float m = warp_max(r & 1 ? y[r / 2].y : y[r / 2].x);
              if (lane == 0) sts32(exch + ((warp & 3) * ROWS + r0 + r) * 4, __float_as_uint(m));
            }
          }
          ok = meet() && ok;
          if (tid < C::kWgRows) {
            const float old = ref_of(__uint_as_float(lds32(my_refs + tid * 4)));
            float m = old;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              m = fmaxf(m, __uint_as_float(lds32(exch + (k * ROWS + tid) * 4)));
            sts32(my_refs + tid * 4, __float_as_uint(add_of(m)));
            sts32(alphas + tid * 4, __float_as_uint(m > old ? fast_exp2(old - m) : 1.f));
          }
          ok = meet() && ok;
          if (done > 0) {
            ok = product(mine - 1) && ok;
            tc_fence_after();
#pragma unroll
            for (int r0 = 0; r0 < C::kWgRows; r0 += CH) {
              float alpha[CH];
#pragma unroll
              for (int r = 0; r < CH; r += 4) {
                const uint4 f = lds128_at(alphas + (r0 + r) * 4);
                alpha[r] = __uint_as_float(f.x);
                alpha[r + 1] = __uint_as_float(f.y);
                alpha[r + 2] = __uint_as_float(f.z);
                alpha[r + 3] = __uint_as_float(f.w);
              }
#pragma unroll
              for (int r = 0; r < CH; r += 2)
                l[(r0 + r) / 2] = __fmul2_rn(l[(r0 + r) / 2], make_float2(alpha[r], alpha[r + 1]));
#pragma unroll
              for (int t = 0; t < C::kPTerms; ++t) {
                const uint32_t at = t_o + grp * C::kON + o_col(wrow + r0) + t * PT;
                float o[CH];
                tmem_ld_cols<CH>(at, o);
#pragma unroll
                for (int r = 0; r < CH; ++r) o[r] *= alpha[r];
                tmem_st_cols<CH>(at, o);
              }
            }
            tmem_wait_st();
          }
          if (!ok) break;
          if constexpr (kKeep) {
#pragma unroll
            for (int r0 = 0; r0 < C::kWgRows; r0 += CH) shift(r0, x + r0 / 2);
          }
        }
        // weights, and their sums
        // (an earlier product of the group has read what was there)
        if (mine >= C::kPBufs && !product(mine - C::kPBufs)) { ok = false; break; }
        const uint32_t pbase = sbase + C::kPOff + tid * 16 +
                               (grp * C::kPBufs + mine % C::kPBufs) * C::kPBytes;
        const float2 inv2 = make_float2(sc.inv_v, sc.inv_v);
#pragma unroll
        for (int r0 = 0; r0 < C::kWgRows; r0 += CH) {
          float2* y = kKeep ? x + r0 / 2 : x;
          if constexpr (!kKeep) {
            scores(r0, y);
            shift(r0, y);
          }
          float e[CH];
#pragma unroll
          for (int r = 0; r < CH; r += 2) {
            const float2 v = make_float2(fast_exp2(y[r / 2].x), fast_exp2(y[r / 2].y));
            l[(r0 + r) / 2] = __ffma2_rn(v, inv2, l[(r0 + r) / 2]);
            e[r] = v.x;
            e[r + 1] = v.y;
          }
          // the token's weights: 16-byte chunks, from the first of the part
          const uint32_t to = pbase +
                              (wrow + r0) / PT * (C::kOPart * C::kElem / 16) * C::kPChunk;
          if constexpr (F8) {
            // three e5m2 terms of every weight: e5m2 is the upper byte of f16
            uint32_t w3[3][CH / 4];
#pragma unroll
            for (int r = 0; r < CH; r += 4) {
              uint32_t b[3][2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t h = pack_f16x2(e[r + 2 * k], e[r + 2 * k + 1]);
                b[0][k] = h & 0xff00ff00u;
                const __half2 d1 = __hsub2(*reinterpret_cast<const __half2*>(&h),
                                           *reinterpret_cast<const __half2*>(&b[0][k]));
                b[1][k] = *reinterpret_cast<const uint32_t*>(&d1) & 0xff00ff00u;
                const __half2 d2 = __hsub2(d1, *reinterpret_cast<const __half2*>(&b[1][k]));
                uint16_t t3;                          // rounded
                asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;"
                    : "=h"(t3) : "r"(*reinterpret_cast<const uint32_t*>(&d2)));
                b[2][k] = t3;
              }
              w3[0][r / 4] = __byte_perm(b[0][0], b[0][1], 0x7531);
              w3[1][r / 4] = __byte_perm(b[1][0], b[1][1], 0x7531);
              w3[2][r / 4] = __byte_perm(b[2][0], b[2][1], 0x5410);
            }
            if constexpr (PT == 16) {                 // a chunk per term
              const uint32_t in = to + (r0 % PT);
#pragma unroll
              for (int t = 0; t < 3; ++t) sts64(in + t * C::kPChunk, w3[t][0], w3[t][1]);
            } else {
              sts128(to, w3[0][0], w3[0][1], w3[1][0], w3[1][1]);
              sts64(to + C::kPChunk, w3[2][0], w3[2][1]);
            }
          } else {
            // Two bf16 terms.  The first is the next smaller bf16 number, so that
            // neither is 0 or negative unless the weight is 0: an infinite value
            // then stays what it is.
            uint32_t hi[CH / 2], lo[CH / 2];
#pragma unroll
            for (int r = 0; r < CH; r += 2) {
              if constexpr (C::kPTerms == 2) {
                const uint32_t a = (max(__float_as_uint(e[r]), 1u) - 1u) & 0xffff0000u;
                const uint32_t b = (max(__float_as_uint(e[r + 1]), 1u) - 1u) & 0xffff0000u;
                hi[r / 2] = (a >> 16) | b;
                lo[r / 2] = pack_bf16x2(e[r] - __uint_as_float(a), e[r + 1] - __uint_as_float(b));
              } else {
                hi[r / 2] = pack_bf16x2(e[r], e[r + 1]);
              }
            }
            const uint32_t in = to + r0 % PT / 8 * C::kPChunk;
            sts128(in, hi[0], hi[1], hi[2], hi[3]);
            if constexpr (C::kPTerms == 2)
              sts128(in + PT / 8 * C::kPChunk, lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_async_shared();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * grp + mine % C::kPBufs]);
        ++mine;
        ++done;
      }
      jt += n;
      // sums of the rows over the group's tokens
      {
        const uint32_t to = sums + ((grp * 4 + (warp & 3)) * ROWS + wrow) * 4;
        const float a = warp_sums<C::kWgRows>(reinterpret_cast<float*>(l), lane);
        if (lane < C::kWgRows) sts32(to + lane * 4, __float_as_uint(a));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ended[np & 1]);
      if (((jt - 1) & 1) == grp) {
        // The group of the last tile joins the parts, once all sums are there and
        // all products done; every warpgroup its rows.
        ok = ok && mbar_wait_warp(&ended[np & 1], (np >> 1) & 1, abort_flag);
        const bool whole = w->whole != 0;
        const int rows = w->rows;
        if (tid < C::kWgRows) {
          const int rr = wrow + tid;
          const float m0 = ref_of(__uint_as_float(lds32(refs + rr * 4)));
          const float m1 = ref_of(__uint_as_float(lds32(refs + (ROWS + rr) * 4)));
          float l0 = 0.f, l1 = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            l0 += __uint_as_float(lds32(sums + (k * ROWS + rr) * 4));
            l1 += __uint_as_float(lds32(sums + ((4 + k) * ROWS + rr) * 4));
          }
          const float m = fmaxf(m0, m1);
          float f0 = l0 == 0.f ? 0.f : fast_exp2(m0 - m);   // 0: saw nothing
          float f1 = l1 == 0.f ? 0.f : fast_exp2(m1 - m);
          float lt = l0 * f0 + l1 * f1;
          if (whole) lt = final_sum(lt, w->pos0 + (w->row0 + rr) / p.group);
          if (rr < rows) {
            if (whole) {
              write_lse(p, w->b, w->h, w->row0 + rr, m, lt, kDecodeLift);
            } else {
              const long long at = static_cast<long long>(w->slot) * ROWS + rr;
              *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m, lt);
            }
          }
          if (whole) {
            const float inv = lt == 0.f ? 0.f : 1.f / lt;
            f0 *= inv;
            f1 *= inv;
          }
          sts64(ends + rr * 8, __float_as_uint(f0), __float_as_uint(f1));
        }
        ok = meet() && ok;
        ok = ok && mbar_wait_warp(&q_empty[np & 1], (np >> 1) & 1, abort_flag);
        tc_fence_after();
        const bool mend = *dropped != 0;
        int t = (w->row0 + wrow) / p.group, g = w->row0 + wrow - t * p.group;
        const long long head = static_cast<long long>(w->h) * p.group;
        __nv_bfloat16* out = p.out + w->b * p.os.b + tid;
        float* part_o = p.part_o + (static_cast<long long>(w->slot) * ROWS + wrow) * D + tid;
#pragma unroll
        for (int q0 = 0; q0 < C::kWgRows; q0 += 8) {
          if (wrow + q0 >= rows) break;
          float o[2][8];
          const uint32_t at = t_o + o_col(wrow + q0);
          tmem_ld_2x8(at, at + C::kON, o[0], o[1]);
#pragma unroll
          for (int term = 1; term < C::kPTerms; ++term) {
            float x2[2][8];
            tmem_ld_2x8(at + term * PT, at + C::kON + term * PT, x2[0], x2[1]);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              o[0][r] += x2[0][r];
              o[1][r] += x2[1][r];
            }
          }
#pragma unroll
          for (int r = 0; r < 8; ++r, part_o += D, g = g + 1 == p.group ? (++t, 0) : g + 1) {
            const int rr = wrow + q0 + r;
            if (rr >= rows || tid >= D) continue;
            const uint2 f = lds64(ends + rr * 8);
            const float f0 = __uint_as_float(f.x), f1 = __uint_as_float(f.y);
            // a group without a tile has an accumulator that is none
            float v = (f0 == 0.f ? 0.f : o[0][r] * f0) + (f1 == 0.f ? 0.f : o[1][r] * f1);
            if (mend) {
              const float4 y = mend_row<D, F8, 1>(p, MendItem{w->b, w->h, w->pos0, w->len}, all,
                                                  w->row0 + rr, w->t0, n * C::kTile, tid & ~3,
                                                  make_float4(0.f, 0.f, 0.f, 0.f));
              v += (tid & 3) == 0 ? y.x : (tid & 3) == 1 ? y.y : (tid & 3) == 2 ? y.z : y.w;
            }
            if (whole) out[(head + g) * p.os.h + t * p.os.s] = __float2bfloat16_rn(v);
            else *part_o = v;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&joined[np & 1]);
      }
      const ChunkPiece* next = ok ? wait_piece(np + 1) : nullptr;
      const int n_next = next != nullptr ? next->n : 0;
      if (next == nullptr) ok = false;
      if (!ok) break;
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
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace sta
