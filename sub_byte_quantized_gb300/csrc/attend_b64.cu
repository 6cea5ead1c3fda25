// Phase 1 of the split-K attention over the 8-bit block layouts (int8 or e4m3 codes, one f32 scale per 64 tokens, head
// and plane), head_dim 128 or 256, in groups of eight query rows of a kv head.
//
//   x_rt = alpha log2(e) s_k(block) sum_d q_rd c_td,  m_r = max_t x_rt,  p = 2^(x - m)
//   o_r += s_v(block) sum_t p_rt v_td   (v: the codes)
// with mma.sync.m16n8k16 (f16 in, f32 accumulate), tokens (QK) and dims (PV) on the M side, the eight rows on the N side:
//   S^T[16 tokens][8 rows] = C[16 tokens][16 dims] . q^T,   O^T[16 dims][8 rows] = V^T[16 dims][16 tokens] . P^T
// Exactness: both code types are exact in f16; bf16 and f16 queries are after a power-of-two factor per row, f32 ones
// are split into two f16 parts (22 bits). One scale per block means that no scale touches the operands: s_k goes into
// the row's factor, and every stage's PV product starts from zero and joins the output as o = o corr + s_v acc in f32,
// which also keeps the tensor cores' truncated additions short. The probabilities are taken 2^12 times larger, so that
// both f16 parts of p (p = hi + lo, 22 bits) stay above f16's subnormals for tokens of little weight.
//
// Work: a unit is one block of 64 tokens of one (sequence, kv head, group of eight rows); the call's units stand in one row,
// heads one after the other. From the lengths, each CTA finds the units of its own. Where every head can be cut into
// equal pieces of few more units than an even share, so that all pieces fit the CTAs, a CTA has one piece of one head;
// else every CTA takes the same number of neighbouring units, and one whose units pass from a head to the next finishes the
// one (a partial each: running maximum, sum, output) and goes on with the other. So ragged batches, short lists and few
// heads leave as much to do to every CTA, without a plan from the host. Head `i` in CTA `c` has partial c + i: a head's
// partials are neighbours, and the last kernel joins them.
//
// Data movement: a CTA's four warps take the stages of its units in turn (32 tokens at head_dim 128, 16 at 256: 8 KB for
// both planes), each through its own ring with 16-byte cp.async; rows are placed with an XOR swizzle of their 16-byte
// columns, so that ldmatrix (plain for K: 4 codes of a token per lane; transposed for V: 2 dims of 2 tokens) is free of
// bank conflicts. At a head's end the warps' states are combined in shared memory.
//
// Bound: the packed cache's bytes from HBM. 128K tokens of 8 kv heads (268 MB) 55 to 57 us by the GPU with the join, where the
// bytes alone take 41 in a kernel that only reads; 16 ragged paged sequences (285 MB) 58 to 59. 16-token stages, three in flight and four
// CTAs per SM 58.8 (57.3 in the same run), four in flight and three CTAs 57.8 (dealt out as here; an
// earlier kernel, with such stages interleaved over a head's CTAs, took 51.9, and 97.9 for ragged: not tried on this one).
#include "attend_b64.cuh"

namespace kvq {
namespace {
using namespace mma;
using namespace b64;

constexpr int kWarps = 4;

template <int D>
struct Cfg {
  static constexpr int STAGE = D == 128 ? 32 : 16;       // tokens
  static constexpr int RING = D == 128 ? 2 : 3;
  static constexpr int PLANE = STAGE * D;                // bytes of one plane's rows
  static constexpr int BYTES = 2 * PLANE + 16;           // both planes, and the block's two scales
  static constexpr int SMEM = kWarps * RING * BYTES;
  static constexpr int PITCH = D + 4;                     // floats of a row of a warp's state: free of bank conflicts
  static_assert(kWarps * 8 * (PITCH + 2) * 4 <= SMEM, "the warps' states reuse the stages");
};

// 16-byte column j of row `row`.
template <int D>
__device__ __forceinline__ uint32_t swz(int row, int j) {
  return (uint32_t)(row * D + ((j ^ (row & 7)) << 4));
}
template <int D, bool E4M3, bool QSPLIT, bool PAGED>
__global__ void __maxnreg__(D == 128 ? 152 : 224) attend_b64_kernel(AttendArgs a) {
  using C = Cfg<D>;
  constexpr int KS = D / 16, TILES = C::STAGE / 16, CPR = D / 16;
  extern __shared__ __align__(1024) uint8_t smem[];
#if defined(__CUDA_ARCH__) && __CUDA_ARCH__ >= 900
  asm volatile("griddepcontrol.launch_dependents;");
#endif
  const CacheView &cv = a.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, mi = lane >> 3;
  const int R = a.gqa * a.n_q, groups = (R + 7) / 8, heads = cv.H * groups;
#if defined(__CUDA_ARCH__) && __CUDA_ARCH__ >= 900
  // lengths that the kernel before may have written (this call's own append does not)
  if (PAGED && a.fresh_tail == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
#endif
  const Deal deal = deal_of<PAGED>(a, heads, lane);
  Walk<PAGED> walk(a, deal, heads, lane);
  Span &sp = walk.sp;
  if (sp.n == 0) {                                       // more CTAs than work
    pdl_wait_if(false);
    return;
  }
  walk.wait_for_append(a);

  uint8_t *ring = smem + warp * C::RING * C::BYTES;
  float *sm = reinterpret_cast<float *>(smem), *so = sm + kWarps * 16;
  for (; sp.n > 0; walk.advance(a, heads)) {
  const int kvh = sp.hd / groups, row0 = 8 * (sp.hd - kvh * groups), rows = min(8, R - row0);
  const int t_first = 64 * sp.blk, t_end = min(sp.len, t_first + 64 * sp.n);
  SeqLen sl;
  sl.kv_len = sp.len;
  sl.q_pos0 = PAGED ? sp.len - a.n_q : a.q_pos0;
  // the warp's stages: tokens t_first + (4 i + warp) STAGE
  const int n_stages = (t_end - t_first + C::STAGE - 1) / C::STAGE, n_mine = (n_stages - warp + kWarps - 1) / kWarps;
  const size_t head_row0 = ((size_t)sp.b * cv.H + kvh) * cv.cap;
  auto issue = [&](int i) {
    if (i < n_mine) {
      const int ts = t_first + (kWarps * i + warp) * C::STAGE;
      const size_t r = cache_row_t<PAGED>(cv, sp.b, kvh, head_row0, ts);   // a stage lies in one block
      const uint8_t *kp = cv.payload[0] + r * D + 16 * lane, *vp = cv.payload[1] + r * D + 16 * lane;
      const uint32_t sK = smem_addr(ring + (i % C::RING) * C::BYTES), sV = sK + C::PLANE;
      const int live = (t_end - ts) * CPR;               // 16-byte pieces of rows in the piece; the rest is zero-filled
      if (live >= C::STAGE * CPR) {
#pragma unroll
        for (int k = 0; k < C::STAGE * CPR / 32; ++k) {
          const uint32_t at = swz<D>((lane + 32 * k) / CPR, (lane + 32 * k) % CPR);
          cp_async16(sK + at, kp + 512 * k, 16);
          cp_async16(sV + at, vp + 512 * k, 16);
        }
      } else {
#pragma unroll
        for (int k = 0; k < C::STAGE * CPR / 32; ++k) {
          const uint32_t at = swz<D>((lane + 32 * k) / CPR, (lane + 32 * k) % CPR);
          const bool ok = lane + 32 * k < live;
          cp_async16(sK + at, ok ? kp + 512 * k : cv.payload[0], ok ? 16 : 0);
          cp_async16(sV + at, ok ? vp + 512 * k : cv.payload[1], ok ? 16 : 0);
        }
      }
      if (lane < 2) cp_async4(sK + 2 * C::PLANE + 4 * lane, static_cast<const float *>(lane ? cv.scale[1] : cv.scale[0]) + (r >> 6), 4);
    }
    cp_async_commit();
  };
  // Query fragments: row g, dims 16 j + 4 c + 0..3 (the k order in which ldmatrix hands out K's codes). They are asked for in
  // front of the first stages: behind those of all CTAs they would arrive microseconds later.
  uint32_t bq[KS][2], bl[QSPLIT ? KS : 1][2];
  float row_alpha = 0.0f;
  {
    uint2 raw[KS][QSPLIT ? 2 : 1];                       // four values each
    const size_t qr = query_row_index(a, sp.b, kvh, row0 + min(g, rows - 1)) * D + 4 * c;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      if constexpr (QSPLIT) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const float *>(a.q) + qr + 16 * j));
        raw[j][0] = make_uint2(w.x, w.y);
        raw[j][1] = make_uint2(w.z, w.w);
      } else {
        raw[j][0] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.q) + qr + 16 * j));
      }
    }
#pragma unroll
    for (int i = 0; i < C::RING; ++i) issue(i);
    float x[KS][4], mx = 0.0f;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      if constexpr (QSPLIT) {
        x[j][0] = __uint_as_float(raw[j][0].x); x[j][1] = __uint_as_float(raw[j][0].y);
        x[j][2] = __uint_as_float(raw[j][1].x); x[j][3] = __uint_as_float(raw[j][1].y);
      } else if (a.q_dtype == KVQ_BF16) {
        x[j][0] = bf16_bits_to_f32(raw[j][0].x & 0xFFFFu); x[j][1] = bf16_bits_to_f32(raw[j][0].x >> 16);
        x[j][2] = bf16_bits_to_f32(raw[j][0].y & 0xFFFFu); x[j][3] = bf16_bits_to_f32(raw[j][0].y >> 16);
      } else {
        const float2 lo = __half22float2(u32_as_h2(raw[j][0].x)), hi = __half22float2(u32_as_h2(raw[j][0].y));
        x[j][0] = lo.x; x[j][1] = lo.y; x[j][2] = hi.x; x[j][3] = hi.y;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (g >= rows) x[j][i] = 0.0f;
        mx = fmaxf(mx, fabsf(x[j][i]));
      }
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    int e = 0;                                           // the row's largest |q| goes to [2^13, 2^14)
    if (mx > 0.0f) e = min(max(((__float_as_int(mx) >> 23) & 0xFF) - 127 - 13, -100), 100);
    const float pre = ldexpf(1.0f, -e);
    row_alpha = a.scale * ldexpf(1.0f, e) * kLog2e;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      float h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[j][i] *= pre;
        h[i] = __half2float(__float2half_rn(x[j][i]));
      }
      bq[j][0] = pack_f16x2(h[0], h[1]);
      bq[j][1] = pack_f16x2(h[2], h[3]);
      if constexpr (QSPLIT) {
        bl[j][0] = pack_f16x2(x[j][0] - h[0], x[j][1] - h[1]);
        bl[j][1] = pack_f16x2(x[j][2] - h[2], x[j][3] - h[3]);
      }
    }
  }
  // the lane's two columns of S^T and O^T are rows 2c and 2c + 1
  const float alpha[2] = {__shfl_sync(0xffffffffu, row_alpha, 8 * c), __shfl_sync(0xffffffffu, row_alpha, 8 * c + 4)};
  int lim[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) lim[k] = 2 * c + k < rows ? row_limit(a, sl, (row0 + 2 * c + k) % a.n_q) : -1;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  float O[KS][4];
#pragma unroll
  for (int j = 0; j < KS; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) O[j][k] = 0.0f;

  for (int i = 0; i < n_mine; ++i) {
    cp_async_wait<C::RING - 1>();
    __syncwarp();
    const uint8_t *sb = ring + (i % C::RING) * C::BYTES;
    const uint32_t sK = smem_addr(sb), sV = sK + C::PLANE;
    const float2 sc = *reinterpret_cast<const float2 *>(sb + 2 * C::PLANE);
    const int ts = t_first + (kWarps * i + warp) * C::STAGE;
    const float f[2] = {alpha[0] * sc.x, alpha[1] * sc.x};

    // scores in base 2: x[t][k] is token ts + 16 t + g + 8 (k >> 1), row 2c + (k & 1)
    float x[TILES][4];
    bool rise = false;
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      float s2[2][4] = {};                               // two chains of dependent products
#pragma unroll
      for (int j = 0; j < KS; j += 2) {
        uint32_t w[4];
        ldsm_x4(sK + swz<D>(16 * t + (mi & 1) * 8 + (lane & 7), j + (mi >> 1)), w);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t A[4];
          codes_f16<E4M3, false>(w[2 * u], A[0], A[2]);
          codes_f16<E4M3, false>(w[2 * u + 1], A[1], A[3]);
          mma16816(s2[u], A, bq[j + u][0], bq[j + u][1]);
          if constexpr (QSPLIT) mma16816(s2[u], A, bl[j + u][0], bl[j + u][1]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[t][k] = ts + 16 * t + g + 8 * (k >> 1) <= lim[k & 1] ? (s2[0][k] + s2[1][k]) * f[k & 1] : -INFINITY;
        rise = rise || x[t][k] > m[k & 1] + kRise;
      }
    }
    // The reference m follows the maximum only where a score passes it by kRise: then 2^12 p still fits f16, and most
    // stages have no reduction over lanes and nothing to rescale.
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float mx = m[k];
#pragma unroll
        for (int t = 0; t < TILES; ++t) mx = fmaxf(mx, fmaxf(x[t][k], x[t][k + 2]));
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
        const float corr = m[k] == -INFINITY ? 0.0f : ex2(m[k] - mx);
        m[k] = mx;
        l[k] *= corr;
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          O[j][k] *= corr;
          O[j][k + 2] *= corr;
        }
      }
    }
    const float sv = sc.y * 0x1p-12f;
    const float base[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};    // nothing seen yet: p = 2^-inf
    uint32_t ph[TILES][2], pl[TILES][2];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      float p[4], h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        p[k] = ex2(x[t][k] - base[k & 1]);
        l[k & 1] += p[k];
        p[k] *= 4096.0f;
        h[k] = __half2float(__float2half_rn(p[k]));
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        ph[t][k] = movm_t(pack_f16x2(h[2 * k], h[2 * k + 1]));
        pl[t][k] = movm_t(pack_f16x2(p[2 * k] - h[2 * k], p[2 * k + 1] - h[2 * k + 1]));
      }
    }
#pragma unroll
    for (int j = 0; j < KS; j += 2) {
      float acc[2][4] = {};
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        uint32_t w[4];
        ldsm_x4_t(sV + swz<D>(16 * t + (mi & 1) * 8 + (lane & 7), j + (mi >> 1)), w);
#pragma unroll
        for (int u = 0; u < 2; ++u) {                    // M rows g / g + 8: dims 16 (j + u) + 2g / + 2g + 1
          uint32_t A[4];
          codes_f16<E4M3, true>(w[2 * u], A[0], A[1]);
          codes_f16<E4M3, true>(w[2 * u + 1], A[2], A[3]);
          mma16816(acc[u], A, ph[t][0], ph[t][1]);
          mma16816(acc[u], A, pl[t][0], pl[t][1]);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) O[j + u][k] = fmaf(acc[u][k], sv, O[j + u][k]);
    }
    __syncwarp();                                        // the stage is read: its place is free
    issue(i + C::RING);
  }
  cp_async_wait<0>();
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], x);
  __syncthreads();
  // the warps' states: [warp][row]: m, l; then [warp][row][D]
  if (lane < 4) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      sm[(warp * 8 + 2 * c + k) * 2] = m[k];
      sm[(warp * 8 + 2 * c + k) * 2 + 1] = l[k];
    }
  }
#pragma unroll
  for (int j = 0; j < KS; ++j)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      *reinterpret_cast<float2 *>(so + (warp * 8 + 2 * c + k) * C::PITCH + 16 * j + 2 * g) = make_float2(O[j][k], O[j][2 + k]);
  __syncthreads();
  const int head = sp.b * heads + sp.hd;
  const size_t part = (size_t)blockIdx.x + head;
  for (int r = warp; r < rows; r += kWarps) {
    float M = -INFINITY, w[kWarps], L = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) M = fmaxf(M, sm[(k * 8 + r) * 2]);
    const float ref = M == -INFINITY ? 0.0f : M;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      w[k] = ex2(sm[(k * 8 + r) * 2] - ref);
      L = fmaf(sm[(k * 8 + r) * 2 + 1], w[k], L);
    }
#pragma unroll
    for (int d = 0; d < D; d += 128) {
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float4 x = *reinterpret_cast<const float4 *>(so + (k * 8 + r) * C::PITCH + d + 4 * lane);
        o.x = fmaf(x.x, w[k], o.x);
        o.y = fmaf(x.y, w[k], o.y);
        o.z = fmaf(x.z, w[k], o.z);
        o.w = fmaf(x.w, w[k], o.w);
      }
      *reinterpret_cast<float4 *>(a.part_o + (part * 8 + r) * D + d + 4 * lane) = o;
    }
    if (lane == 0) {
      a.part_m[part * 8 + r] = M;                        // (base 2)
      a.part_l[part * 8 + r] = L;
    }
  }
  if (sp.blk == 0 && threadIdx.x == 0) a.spans[head] = walk.ctas_of_head(deal);
  __syncthreads();                                       // the ring is free again
  }
}

// Joins the partials of every row: M = max m, out = sum o 2^(m - M) / sum l 2^(m - M). SPLIT: a CTA per row, whose warps
// split the partials; else a warp per row. Zeros only where the sum is 0 (a row that sees nothing): a sum that is not a number,
// as scores that are none or a wait that gave up leave it, stays one.
constexpr int kJoinWarps = 4, kBatch = 4;
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kJoinWarps * 32) join_b64_kernel(AttendArgs a, unsigned n_rows) {
  constexpr int V = D / 128;                             // float4 per lane
  __shared__ float sm_m[kJoinWarps], sm_l[kJoinWarps];
  __shared__ __align__(16) float sm_o[SPLIT ? kJoinWarps : 1][SPLIT ? D : 4];
#if defined(__CUDA_ARCH__) && __CUDA_ARCH__ >= 900
  asm volatile("griddepcontrol.wait;" ::: "memory");
#endif
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t row = SPLIT ? (size_t)blockIdx.x : (size_t)blockIdx.x * kJoinWarps + warp;
  if (row >= n_rows) return;
  const int R = a.gqa * a.n_q, groups = (R + a.group - 1) / a.group;
  const size_t bh = row / R;
  const int r = (int)(row - bh * R), b = (int)(bh / a.cache.H);
  const int len = a.seq_lens ? min(max(__ldg(a.seq_lens + b), 0), a.kv_len) : a.kv_len;
  float M = -INFINITY, L = 0.0f;
  float4 O[V];
#pragma unroll
  for (int v = 0; v < V; ++v) O[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (len > 0) {
    const size_t head = bh * groups + r / a.group;
    const int2 span = a.spans[head];
    const size_t p0 = (head + span.x) * a.group + r % a.group;
    const int n = span.y - span.x + 1;
    for (int i0 = SPLIT ? warp : 0; i0 < n; i0 += kBatch * (SPLIT ? kJoinWarps : 1)) {
      float mc[kBatch], lc[kBatch], bm = M;
      float4 oc[kBatch][V];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * (SPLIT ? kJoinWarps : 1);
        const bool ok = i < n;
        const size_t p = p0 + (size_t)a.group * (ok ? i : 0);
        mc[u] = ok ? a.part_m[p] : -INFINITY;
        lc[u] = ok ? a.part_l[p] : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
          oc[u][v] = ok ? *reinterpret_cast<const float4 *>(a.part_o + p * D + 128 * v + 4 * lane) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        bm = fmaxf(bm, mc[u]);
      }
      if (bm == -INFINITY) {                             // pieces that the row does not see: sums of 0, or no numbers
#pragma unroll
        for (int u = 0; u < kBatch; ++u) L += lc[u];
        continue;
      }
      const float corr = exp2f(M - bm);
      L *= corr;
#pragma unroll
      for (int v = 0; v < V; ++v) O[v].x *= corr, O[v].y *= corr, O[v].z *= corr, O[v].w *= corr;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const float w = exp2f(mc[u] - bm);
        L = fmaf(lc[u], w, L);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          O[v].x = fmaf(oc[u][v].x, w, O[v].x);
          O[v].y = fmaf(oc[u][v].y, w, O[v].y);
          O[v].z = fmaf(oc[u][v].z, w, O[v].z);
          O[v].w = fmaf(oc[u][v].w, w, O[v].w);
        }
      }
      M = bm;
    }
  }
  if constexpr (SPLIT) {
    if (lane == 0) sm_m[warp] = M, sm_l[warp] = L;
#pragma unroll
    for (int v = 0; v < V; ++v) *reinterpret_cast<float4 *>(&sm_o[warp][128 * v + 4 * lane]) = O[v];
    __syncthreads();
    float Mt = sm_m[0];
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) Mt = fmaxf(Mt, sm_m[w]);
    for (int d = threadIdx.x; d < D; d += kJoinWarps * 32) {
      float Lt = 0.0f, x = 0.0f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) {
        const float f = sm_m[w] == -INFINITY ? 0.0f : exp2f(sm_m[w] - Mt);
        Lt = fmaf(sm_l[w], f, Lt);
        x = fmaf(sm_o[w][d], f, x);
      }
      a.out[out_row(a, row) * D + d] = Lt == 0.0f ? 0.0f : x / Lt;
    }
  } else {
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int v = 0; v < V; ++v)
      *reinterpret_cast<float4 *>(a.out + out_row(a, row) * D + 128 * v + 4 * lane) = make_float4(O[v].x * inv, O[v].y * inv, O[v].z * inv, O[v].w * inv);
  }
}

template <int D, bool E4M3, bool QSPLIT, bool PAGED>
cudaError_t launch_t(const AttendArgs &a, cudaStream_t st) {
  static std::atomic<bool> configured[kMaxDevices];
  auto kernel = attend_b64_kernel<D, E4M3, QSPLIT, PAGED>;
  const cudaError_t e = set_smem_once(configured, kernel, Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  chained(cfg, attr, a.grid, kWarps * 32, Cfg<D>::SMEM, st);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int D, bool E4M3>
cudaError_t launch_de(const AttendArgs &a, cudaStream_t st) {
  const bool paged = a.cache.page_shift >= 0;
  if (a.q_dtype == KVQ_F32) return paged ? launch_t<D, E4M3, true, true>(a, st) : launch_t<D, E4M3, true, false>(a, st);
  return paged ? launch_t<D, E4M3, false, true>(a, st) : launch_t<D, E4M3, false, false>(a, st);
}

}  // namespace

cudaError_t launch_join_b64(const AttendArgs &a, cudaStream_t st) {
  const unsigned rows = (unsigned)((size_t)a.cache.B * a.Hq * a.n_q);
  const int sms = sm_count();
  // Few rows have many partials each: a CTA for a row, else a warp (64 rows, 128K tokens: 57.3 / 63.3 us with phase 1; 512 rows
  // 59.3 / 60.3; 640 rows 98.3 / 98.3; 1024 rows 97.3 / 97.4, of 32 blocks 36.1 / 35.7; 2048 rows 100.1 / 98.9, of 32 blocks
  // 39.4 / 37.5; 32768 rows 330 / 299)
  const bool split = rows <= 8u * (unsigned)sms;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  chained(cfg, attr, split ? rows : (rows + kJoinWarps - 1) / kJoinWarps, kJoinWarps * 32, 0, st);
  if (a.cache.D == 128)
    return split ? cudaLaunchKernelEx(&cfg, join_b64_kernel<128, true>, a, rows) : cudaLaunchKernelEx(&cfg, join_b64_kernel<128, false>, a, rows);
  return split ? cudaLaunchKernelEx(&cfg, join_b64_kernel<256, true>, a, rows) : cudaLaunchKernelEx(&cfg, join_b64_kernel<256, false>, a, rows);
}

cudaError_t launch_attend_b64(const AttendArgs &a, cudaStream_t st) {
  if (a.group != 8) return launch_attend_b64_rows(a, st);
  if (a.cache.layout == KVQ_E4M3_B64) return a.cache.D == 128 ? launch_de<128, true>(a, st) : launch_de<256, true>(a, st);
  return a.cache.D == 128 ? launch_de<128, false>(a, st) : launch_de<256, false>(a, st);
}

}  // namespace kvq
