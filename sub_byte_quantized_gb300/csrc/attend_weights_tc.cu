// Attention weight of every cached token for many query rows (more than eight per kv head: an observation
// window at the end of a prompt), head_dim 128, on the fifth-generation tensor cores. The formula, the
// definition of the scores and the window are those of attend_weights.cu.
//
//   S^T = K . Q^T   M 128 tokens x N rows x K 128 dims (tcgen05.mma kind::f16, f32 accumulators in TMEM)
//
// The tokens are the M side: TMEM lane = token, column = query row, so a thread sums the weights of its
// token over the columns it reads and nothing crosses lanes. Operands are exact in f16: Hadamard codes and
// int8 query codes (S is the exact integer dot), or, for the block layouts, code x scale as hi + lo parts
// (an f16 scale times an at most 8-bit code has 19 bits: the f16 product and the fma's remainder hold it
// exactly; asymmetric values are rounded to f32 first), scaled by a power of two per token, times the query
// scaled by a power of two per row (f32 queries as hi + lo too, three products).
//
// Bound by the exponentials: 32 query heads x 32 rows over 32749 tokens, 8 kv heads, take 33.5 M of them,
// 7 us at 16 per clock and SM; the products take 2 us, the packed keys 3. One CTA per SM:
//   warps 0-15  weights: four groups of four (TMEM lane quarters); accumulators go to the groups in turn (with
//               two groups, a scheduler's two warps left every latency open: 28 instead of 19 us)
//   warps 16-19 unpack: one token row per thread, packed row -> swizzled f16 tile (two buffers); rows of the
//               tiles to come are prefetched into L2
//   warp  20    one lane issues the MMAs; the warp owns the TMEM allocation (four accumulators of 128 rows)
// Query rows beyond 256 (128 with f32 queries) are taken in further groups over the same tokens, whose sums
// stay in shared memory. Every wait is bounded; a CTA whose wait gives up writes NaN scores.
#include "attend_weights.cuh"

namespace kvq {
namespace {
using namespace weights;

constexpr int kD = 128, kTile = 128;     // head_dim; tokens per tile = TMEM lanes
constexpr int kBlk = 128;                // query rows per accumulator
constexpr int kMaxTiles = 16;            // tiles per CTA (sums in shared memory)
constexpr int kEpiWarps = 16, kUnpWarp = 16, kUnpThreads = 128, kMmaWarp = 20, kWarps = 21, kThreads = 32 * kWarps;
constexpr int kAhead = 3;                // tiles that the unpack warps prefetch ahead
constexpr int kAcc = 4, kTmemCols = kAcc * kBlk;
constexpr int kOperand = kTile * kD * 2; // bytes of one f16 operand of 128 rows: two 64-dim column blocks

constexpr int kWinRowsTc = 4 * kWarps;   // query rows at a time in a window CTA

// HILO: the key values enter as hi + lo. QLO: so do the queries.
template <bool HILO, bool QLO>
struct Smem {
  static constexpr int A = kOperand * (HILO ? 2 : 1);             // per buffer
  static constexpr int GROUP = QLO ? kBlk : 2 * kBlk;             // query rows at a time
  static constexpr int OFF_B = 2 * A, B = 2 * kOperand;
  static constexpr int OFF_ROW = OFF_B + B;                       // float2 (factor, lse) per row, then limits
  static constexpr int OFF_SUM = OFF_ROW + 2 * kBlk * 12;         // [accumulator of the group][tiles][128]
  static constexpr int OFF_BAR = OFF_SUM + 2 * kMaxTiles * kTile * 4;
  static constexpr int TOTAL = OFF_BAR + 128;
  static_assert(TOTAL <= 227 * 1024, "one CTA per SM");
};
// mbarriers: tiles full / empty, accumulators full / empty, drain
enum { B_AF = 0, B_AE = 2, B_DF = 4, B_DE = 4 + kAcc, B_DR = 4 + 2 * kAcc, N_BAR };

__device__ __forceinline__ uint64_t sdesc(uint32_t addr) {        // 128-byte swizzle, 8-row groups 1 KB apart
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t da, uint64_t db, uint32_t id, uint32_t accumulate) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
               ::"r"(d), "l"(da), "l"(db), "r"(id), "r"(accumulate));
}
__device__ __forceinline__ void mma_commit(uint64_t *b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(b)));
}
__device__ __forceinline__ uint32_t sw128(int row, int byte) {
  return (uint32_t)((row >> 3) * 1024 + (row & 7) * 128 + ((((byte >> 4) ^ (row & 7))) << 4) + (byte & 15));
}
// Byte offset of 8-dim group gi of a row in an operand.
__device__ __forceinline__ uint32_t group_at(int row, int gi) { return (uint32_t)(gi >> 3) * (kOperand / 2) + sw128(row, 16 * (gi & 7)); }

// 32 TMEM columns of this warp's lanes: the load is issued by one call and waited for by the other, which
// names the registers so that no use of them moves above it.
__device__ __forceinline__ void tm_issue32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tm_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// One token's packed row and scales in registers.
template <int KL>
struct TokenRow {
  static constexpr int RB = KL == KVQ_Q8_0 ? 128 : KL == KVQ_Q6_0 ? 96 : KL == KVQ_HAD_INT2 ? 32 : 64;
  uint4 w[RB / 16];
  uint2 scale, zero;
};
__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
template <int KL>
__device__ __forceinline__ void prefetch_row(const CacheView &cv, size_t row) {
  prefetch_l2(cv.payload[0] + row * TokenRow<KL>::RB);
  prefetch_l2(static_cast<const uint8_t *>(cv.scale[0]) + row * (is_hadamard(KL) ? 4 : 8));
  if constexpr (KL == KVQ_ASYM4_G32) prefetch_l2(reinterpret_cast<const uint8_t *>(cv.zero[0]) + row * 8);
}
template <int KL>
__device__ __forceinline__ void load_row(const CacheView &cv, size_t row, TokenRow<KL> &t) {
  const uint4 *p = reinterpret_cast<const uint4 *>(cv.payload[0] + row * TokenRow<KL>::RB);
#pragma unroll
  for (int i = 0; i < TokenRow<KL>::RB / 16; ++i) t.w[i] = __ldg(p + i);
  if constexpr (!is_hadamard(KL)) t.scale = __ldg(static_cast<const uint2 *>(cv.scale[0]) + row);
  if constexpr (KL == KVQ_ASYM4_G32) t.zero = __ldg(reinterpret_cast<const uint2 *>(cv.zero[0]) + row);
}
// The power of two that a block-layout token's values are divided by: its largest scale (or zero-point)
// comes into [2^5, 2^6), so that 8-bit codes times it stay inside f16.
__device__ __forceinline__ float token_unit(uint2 scale, uint2 zero, bool zeros) {
  const float2 a = __half22float2(u32_as_h2(scale.x)), b = __half22float2(u32_as_h2(scale.y));
  float m = fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y)));
  if (zeros) {
    const float2 c = __half22float2(u32_as_h2(zero.x)), d = __half22float2(u32_as_h2(zero.y));
    m = fmaxf(m, fmaxf(fmaxf(fabsf(c.x), fabsf(c.y)), fmaxf(fabsf(d.x), fabsf(d.y))));
  }
  const int e = ((__float_as_int(m) >> 23) & 0xFF) - 127 - 5;       // f16 range: -29 .. 10 (m = 0: no matter)
  return __int_as_float((min(max(e, -60), 60) + 127) << 23);
}
// Eight codes' words -> (hi, lo) operand groups; pairs (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ void scale_codes(const uint32_t (&code)[4], uint32_t s2, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    hi[k] = hmul2(code[k], s2);
    lo[k] = hfma2(code[k], s2, hi[k] ^ 0x80008000u);     // the product's exact remainder
  }
}
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// The thread's token row as operand rows `row` of the tile at `tile` (lo parts kOperand behind).
template <int KL>
__device__ __forceinline__ void unpack_token(const TokenRow<KL> &t, uint8_t *tile, int row) {
  float inv = 1.0f;
  if constexpr (!is_hadamard(KL)) inv = 1.0f / token_unit(t.scale, t.zero, KL == KVQ_ASYM4_G32);   // a power of two
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    float s = 0.0f, z = 0.0f;
    uint32_t s2 = 0;
    if constexpr (!is_hadamard(KL)) {
      const float2 sp = __half22float2(u32_as_h2(b < 2 ? t.scale.x : t.scale.y));
      s = ((b & 1) ? sp.y : sp.x) * inv;
      s2 = pack_f16x2(s, s);
      if constexpr (KL == KVQ_ASYM4_G32) {
        const float2 zp = __half22float2(u32_as_h2(b < 2 ? t.zero.x : t.zero.y));
        z = ((b & 1) ? zp.y : zp.x) * inv;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int gi = 4 * b + k;                          // dims 8 gi .. 8 gi + 7
      uint32_t c[4];
      if constexpr (KL == KVQ_Q8_0) {
        unpack8_s8(word_of(t.w[gi >> 1], 2 * (gi & 1)), word_of(t.w[gi >> 1], 2 * (gi & 1) + 1), c);
      } else if constexpr (KL == KVQ_Q6_0) {
        // block b: 24 bytes from 24 b = words 6 b ..: four words of low nibbles, two of high fields
        const int lw = 6 * b + k, hw = 6 * b + 4 + (k >> 1);
        const uint32_t h = word_of(t.w[hw >> 2], hw & 3);
        unpack8_s6(word_of(t.w[lw >> 2], lw & 3), (k & 1) ? h >> 16 : h & 0xFFFFu, c);
      } else if constexpr (KL == KVQ_HAD_INT2) {
        const uint32_t h = word_of(t.w[gi >> 3], (gi >> 1) & 3);
        unpack8_s2((gi & 1) ? h >> 16 : h & 0xFFFFu, c);
      } else if constexpr (KL == KVQ_ASYM4_G32) {
        unpack8_u4(word_of(t.w[gi >> 2], gi & 3), c);
      } else {
        unpack8_q4(word_of(t.w[gi >> 2], gi & 3), c);
      }
      uint8_t *o = tile + group_at(row, gi);
      if constexpr (is_hadamard(KL)) {
        *reinterpret_cast<uint4 *>(o) = make_uint4(c[0], c[1], c[2], c[3]);
      } else {
        uint32_t hi[4], lo[4];
        if constexpr (KL == KVQ_ASYM4_G32) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(u32_as_h2(c[i]));
            const float x = fmaf(f.x, s, z), y = fmaf(f.y, s, z);
            hi[i] = pack_f16x2(x, y);
            const float2 g = __half22float2(u32_as_h2(hi[i]));
            lo[i] = pack_f16x2(x - g.x, y - g.y);
          }
        } else {
          scale_codes(c, s2, hi, lo);
        }
        *reinterpret_cast<uint4 *>(o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(o + kOperand) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
  }
}

// Query rows [r0, r0 + n) of the kv head as operand rows (zero up to a multiple of 32), and their factors.
template <int KL, bool QLO>
__device__ __forceinline__ void query_operand(const AttendArgs &a, int bb, int kvh, int r0, int n, uint8_t *sb, float2 *par) {
  const int rows = a.gqa * a.n_q, n32 = (n + 31) / 32 * 32, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto put = [&](int i, int gi, const float (&v)[8]) {
    uint8_t *o = sb + (i >> 7) * kOperand + group_at(i & 127, gi);
    *reinterpret_cast<uint4 *>(o) = make_uint4(pack_f16x2(v[0], v[4]), pack_f16x2(v[1], v[5]), pack_f16x2(v[2], v[6]), pack_f16x2(v[3], v[7]));
    if constexpr (QLO) {
      float l[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) l[k] = v[k] - __half2float(__float2half_rn(v[k]));
      *reinterpret_cast<uint4 *>(o + kOperand) =
          make_uint4(pack_f16x2(l[0], l[4]), pack_f16x2(l[1], l[5]), pack_f16x2(l[2], l[6]), pack_f16x2(l[3], l[7]));
    }
  };
  if constexpr (is_hadamard(KL)) {
    // the attention's query preparation has left the codes in the workspace on the tcgen05 path
    const bool ready = tc_prefill_shape(a.cache.layout, a.cache.v_layout, kD, rows);
    if (ready) {
      for (int u = threadIdx.x; u < n32 * 16; u += kThreads) {
        const int i = u >> 4, gi = u & 15, r = r0 + i;
        float v[8] = {};
        if (i < n) {
          const size_t row = query_row_index(a, bb, kvh, r);
          const uint2 c8 = *reinterpret_cast<const uint2 *>(a.q8 + row * kD + 8 * gi);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = (float)(int8_t)(((k < 4 ? c8.x : c8.y) >> (8 * (k & 3))) & 0xFFu);
          if (gi == 0) par[i].x = a.scale * a.s_q[row] * kLog2e;
        }
        put(i, gi, v);
      }
    } else {
      for (int i = warp; i < n32; i += kWarps) {           // a warp per row: four dims per lane, then eight in lanes 0-15
        float x[4] = {}, v[8];
        int q8[4] = {};
        float s = 0.0f;
        if (i < n) load4_f32(a.q, a.q_dtype, query_row_index(a, bb, kvh, r0 + i) * kD + 4 * lane, x);
        s = had_query_row<4>(x, q8, lane);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = (float)__shfl_sync(0xffffffffu, q8[k & 3], (2 * lane + (k >> 2)) & 31);
        if (lane < 16) put(i, lane, v);
        if (lane == 0 && i < n) par[i].x = a.scale * s * kLog2e;
      }
    }
  } else {
    for (int u = threadIdx.x; u < n32 * 16; u += kThreads) {   // sixteen lanes per row (n32 * 16 is a multiple of 32)
      const int i = u >> 4, gi = u & 15;
      float v[8] = {}, m = 0.0f;
      if (i < n) load8_f32(a.q, a.q_dtype, query_row_index(a, bb, kvh, r0 + i) * kD + 8 * gi, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(v[k]));
#pragma unroll
      for (int k = 1; k < 16; k <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
      int e = 0;                                          // the largest |q| into [2^10, 2^11)
      if (m > 0.0f) e = min(max(((__float_as_int(m) >> 23) & 0xFF) - 127 - 10, -100), 100);
      const float pre = __int_as_float((127 - e) << 23);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= pre;
      put(i, gi, v);
      if (gi == 0 && i < n) par[i].x = a.scale * __int_as_float((127 + e) << 23) * kLog2e;
    }
  }
}

template <int KL, bool QLO>
__global__ void __launch_bounds__(kThreads, 1) attend_weights_tc_kernel(WeightArgs wa) {
  constexpr bool HILO = !is_hadamard(KL);
  using S = Smem<HILO, QLO>;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ uint32_t tmem_base;
  const AttendArgs &a = wa.a;
  const CacheView &cv = a.cache;
  const int bh = blockIdx.y, bb = bh / cv.H, kvh = bh - bb * cv.H;
  const SeqLen sl = seq_of(a, bb);
  if (is_hadamard(KL) && (int)blockIdx.x >= wa.n_ctas) {
    const int j = (int)blockIdx.x - wa.n_ctas;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (sl.n_body + j * kWinTokens < sl.kv_len) window_tokens<kD, kWarps, kWinRowsTc>(wa, sl, bb, kvh, j, reinterpret_cast<float *>(sm));
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int first = (int)blockIdx.x * wa.units;            // this CTA's first tile
  const int n_tiles = min((sl.n_body + kTile - 1) / kTile - first, wa.units);
  if (n_tiles <= 0) {
    if (blockIdx.x == 0 && blockIdx.y == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int rows = a.gqa * a.n_q;
  uint64_t *bar = reinterpret_cast<uint64_t *>(sm + S::OFF_BAR);
  float2 *par = reinterpret_cast<float2 *>(sm + S::OFF_ROW);
  int *lim = reinterpret_cast<int *>(par + 2 * kBlk);
  float *sums = reinterpret_cast<float *>(sm + S::OFF_SUM);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(bar + B_AF + i, kUnpThreads);
      bar_init(bar + B_AE + i, 1);
    }
    for (int i = 0; i < kAcc; ++i) {
      bar_init(bar + B_DF + i, 1);
      bar_init(bar + B_DE + i, 128);                      // the four warps that read it
    }
    bar_init(bar + B_DR, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int i = tid; i < 2 * kMaxTiles * kTile; i += kThreads) sums[i] = 0.0f;
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_base)), "n"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;");
  const uint32_t tmem = tmem_base;
  const int t_last = sl.n_body - 1, min_lim = row_limit(a, sl, 0);   // limits grow with the query index
  // plane row of token t (past the body: its last token)
  auto token_row = [&](int t) { return cache_row(cv, bb, kvh, min(t, t_last)); };
  bool ok = true;
  int tile_n = 0, item_n = 0, drains = 0;                  // tiles and accumulators before this group

  for (int r0 = 0; r0 < rows && ok; r0 += S::GROUP) {
    const int n = min(rows - r0, S::GROUP), nblk = (n + kBlk - 1) / kBlk;
    query_operand<KL, QLO>(a, bb, kvh, r0, n, sm + S::OFF_B, par);
    if (r0 == 0) asm volatile("griddepcontrol.wait;" ::: "memory");   // the rows' log-sum-exp come from phase 2
    __syncthreads();
    for (int i = tid; i < nblk * kBlk; i += kThreads) {
      float lse2 = INFINITY;
      int l = -1;
      if (i < n) row_result(a, sl, bb, kvh, r0 + i, lse2, l);
      par[i] = make_float2(lse2 == INFINITY ? 0.0f : par[i].x, lse2);   // a row that sees nothing may hold any score
      lim[i] = l;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // generic writes -> tensor-core reads
    __syncthreads();

    if (warp < kEpiWarps) {
      // ---------------- weights: group g takes every fourth accumulator
      const int g = warp >> 2, lr = 32 * (warp & 3) + lane, items = n_tiles * nblk;
      const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
      auto tile_of = [&](int i) { return nblk == 2 ? i >> 1 : i; };
      // what the scores of item i's token are multiplied by
      auto unit_of = [&](int i) -> float {
        const size_t row = token_row((first + tile_of(i)) * kTile + lr);
        if constexpr (is_hadamard(KL)) return __ldg(static_cast<const float *>(cv.scale[0]) + row);
        const uint2 s = __ldg(static_cast<const uint2 *>(cv.scale[0]) + row);
        uint2 z = make_uint2(0u, 0u);
        if constexpr (KL == KVQ_ASYM4_G32) z = __ldg(reinterpret_cast<const uint2 *>(cv.zero[0]) + row);
        return token_unit(s, z, KL == KVQ_ASYM4_G32);
      };
      float f = g < items ? unit_of(g) : 0.0f;
      for (int i = g; i < items && ok; i += 4) {
        const int tile = tile_of(i), blk = nblk == 2 ? i & 1 : 0, it = item_n + i;
        const int t0 = (first + tile) * kTile, t = t0 + lr;
        const float f_next = i + 4 < items ? unit_of(i + 4) : 0.0f;   // in flight while this item is summed
        const int cols = (min(n - blk * kBlk, kBlk) + 31) / 32 * 32;
        const float2 *pr = par + blk * kBlk;
        const bool masked = t0 + kTile - 1 > min_lim;
        ok = __all_sync(0xffffffffu, bar_wait(bar + B_DF + (it & (kAcc - 1)), (it / kAcc) & 1));
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;");
        const uint32_t acc = tmem + lanes + (uint32_t)(it & (kAcc - 1)) * kBlk;
        float w[4] = {0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < cols; c += 32) {
          uint32_t d[32];
          tm_issue32(acc + c, d);
          tm_wait32(d);
          if (!masked) {
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const float4 p = *reinterpret_cast<const float4 *>(pr + c + k);
              w[k & 3] += ex2(fmaf(__uint_as_float(d[k]) * f, p.x, -p.y));
              w[(k & 3) + 1] += ex2(fmaf(__uint_as_float(d[k + 1]) * f, p.z, -p.w));
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float2 p = pr[c + k];
              const float e = ex2(fmaf(__uint_as_float(d[k]) * f, p.x, -p.y));
              w[k & 3] += t <= lim[blk * kBlk + c + k] ? e : 0.0f;
            }
          }
        }
        asm volatile("tcgen05.fence::before_thread_sync;");   // the reads above precede the next MMAs
        bar_arrive(bar + B_DE + (it & (kAcc - 1)));
        // an accumulator's rows of a tile belong to one thread at a time
        sums[(blk * kMaxTiles + tile) * kTile + lr] += (w[0] + w[1]) + (w[2] + w[3]);
        f = f_next;
      }
    } else if (warp >= kUnpWarp && warp < kMmaWarp) {
      // ---------------- unpack: one token row per thread
      const int lr = tid - 32 * kUnpWarp;
#pragma unroll
      for (int k = 1; k < kAhead; ++k)
        if (k < n_tiles) prefetch_row<KL>(cv, token_row((first + k) * kTile + lr));
      TokenRow<KL> t;
      for (int j = 0; j < n_tiles && ok; ++j) {
        const int tn = tile_n + j, buf = tn & 1;
        load_row<KL>(cv, token_row((first + j) * kTile + lr), t);
        if (j + kAhead < n_tiles) prefetch_row<KL>(cv, token_row((first + j + kAhead) * kTile + lr));
        if (tn >= 2) ok = __all_sync(0xffffffffu, bar_wait(bar + B_AE + buf, ((tn >> 1) - 1) & 1));
        if (!ok) break;
        unpack_token<KL>(t, sm + buf * S::A, lr);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        bar_arrive(bar + B_AF + buf);
      }
    } else if (warp == kMmaWarp && lane == 0) {
      // ---------------- MMA issue (one thread)
      for (int j = 0; j < n_tiles && ok; ++j) {
        const int tn = tile_n + j, buf = tn & 1;
        ok = bar_wait(bar + B_AF + buf, (tn >> 1) & 1);
        if (!ok) break;
        asm volatile("tcgen05.fence::after_thread_sync;");
        const uint32_t at = smem_addr(sm + buf * S::A);
        for (int blk = 0; blk < nblk && ok; ++blk) {
          const int it = item_n + j * nblk + blk, ab = it & (kAcc - 1);
          if (it >= kAcc) ok = bar_wait(bar + B_DE + ab, (it / kAcc - 1) & 1);
          if (!ok) break;
          asm volatile("tcgen05.fence::after_thread_sync;");
          const uint32_t bt = smem_addr(sm + S::OFF_B + blk * kOperand), d = tmem + ab * kBlk;
          const uint32_t cols = (uint32_t)(min(n - blk * kBlk, kBlk) + 31) / 32 * 32;
          const uint32_t id = (1u << 4) | ((cols >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);   // f16, f32 accumulate, K-major
#pragma unroll
          for (int pass = HILO ? 0 : 2; pass < 3; ++pass) {
            // lo hi, hi lo, hi hi: the small products first, while there is little that their sum's truncation
            // can cost (f32 queries: the weights' error 1.6e-6 -> 3e-7)
            if (!QLO && pass == 1) continue;
            // a k-step is 32 bytes, four to a column block: the start addresses differ by constants
            const uint64_t da = sdesc(at + (pass == 0 ? kOperand : 0)), db = sdesc(bt + (pass == 1 ? kOperand : 0));
#pragma unroll
            for (int ks = 0; ks < kD / 16; ++ks) {
              const uint64_t o = ((ks >> 2) * (kOperand / 2) + 32 * (ks & 3)) >> 4;
              mma_f16(d, da + o, db + o, id, pass > (HILO ? 0 : 2) || ks > 0 ? 1u : 0u);
            }
          }
          mma_commit(bar + B_DF + ab);
        }
        if (ok) mma_commit(bar + B_AE + buf);
      }
      mma_commit(bar + B_DR);                             // every MMA issued above completes before the next group
      if (!bar_wait(bar + B_DR, drains & 1)) ok = false;
    }
    ++drains;
    tile_n += n_tiles;
    item_n += n_tiles * nblk;
    ok = !__syncthreads_or(!ok);
  }
  const float *in = wa.scores_in ? wa.scores_in + (size_t)bh * wa.stride : nullptr;
  float *out = wa.scores_out + (size_t)bh * wa.stride;
  for (int i = tid; i < n_tiles * kTile; i += kThreads) {
    const int t = first * kTile + i;
    const float v = ok ? sums[i] + sums[kMaxTiles * kTile + i] : __int_as_float(0x7fc00000);
    if (t < sl.n_body) out[t] = in ? fmaf(wa.decay, in[t], v) : v;
  }
  asm volatile("tcgen05.fence::before_thread_sync;");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;");
  if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
}

template <int KL, bool QLO>
cudaError_t launch_tc(WeightArgs &wa, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  constexpr int body = Smem<!is_hadamard(KL), QLO>::TOTAL;
  constexpr int smem = is_hadamard(KL) ? max_of(body, window_smem<kD, kWarps, kWinRowsTc>()) : body;
  cudaError_t e = set_smem_once(done, attend_weights_tc_kernel<KL, QLO>, smem);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // one CTA per SM: a head's tiles shared out over what its window leaves of one wave, at most kMaxTiles each
  const int heads = wa.a.cache.B * wa.a.cache.H, n_tiles = (wa.a.n_body + kTile - 1) / kTile;
  const int n_win = is_hadamard(KL) ? (wa.a.n_win + kWinTokens - 1) / kWinTokens : 0;
  const int wave = max(1, sms / heads - n_win);
  wa.units = max(1, min((n_tiles + wave - 1) / wave, kMaxTiles));
  wa.n_ctas = (n_tiles + wa.units - 1) / wa.units;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(wa.n_ctas + n_win), (unsigned)heads);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_weights_tc_kernel<KL, QLO>, wa);
}
template <int KL>
cudaError_t launch_queries(WeightArgs &wa, cudaStream_t st) {
  return wa.a.q_dtype == KVQ_F32 ? launch_tc<KL, true>(wa, st) : launch_tc<KL, false>(wa, st);
}

}  // namespace

cudaError_t launch_attend_weights_tc(WeightArgs &wa, cudaStream_t st) {
  switch (wa.a.cache.layout) {
    case KVQ_Q4_0: return launch_queries<KVQ_Q4_0>(wa, st);
    case KVQ_Q6_0: return launch_queries<KVQ_Q6_0>(wa, st);
    case KVQ_Q8_0: return launch_queries<KVQ_Q8_0>(wa, st);
    case KVQ_ASYM4_G32: return launch_queries<KVQ_ASYM4_G32>(wa, st);
    case KVQ_HAD_INT4: return launch_tc<KVQ_HAD_INT4, false>(wa, st);   // int8 query codes are exact
    default: return launch_tc<KVQ_HAD_INT2, false>(wa, st);
  }
}

}  // namespace kvq
