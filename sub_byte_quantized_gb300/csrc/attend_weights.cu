// Attention weight of every cached token, after an attention call has left each query row's log-sum-exp
//   lse_r = log sum_t exp(alpha q_r . k_t)   (over the tokens row r sees):
//   scores_out[t] = decay scores_in[t] + sum_r exp(alpha q_r . k_t - lse_r),
// r over the gqa * n_q query rows of the token's kv head. One more pass over the K plane alone: every
// token belongs to one warp, which sums its rows in a fixed order, so nothing is added atomically and
// equal calls give equal bits.
//
// The dot products are the attention's own: mma.sync m16n8k16, 16 tokens by 8 query rows, on exact f16
// codes (4-, 6-, 8- and 2-bit) and queries that are exact in f16 after a power-of-two prescale (f32
// queries as hi + lo parts); block layouts scale every 32-dim block's f32 partial by the token's f16
// scale (asymmetric: plus zero-point times the block's query sum), Hadamard layouts give the exact
// integer dot with the int8 query codes. Window tokens (Hadamard) are scored in f32 from the ring by
// CTAs of their own behind the body's.
//
// Eight warps per CTA. The query rows sit in shared memory in operand order, 64 at a time; a warp loads
// a tile's packed rows straight into registers, where the words are already the fragment's (lane c of a
// quad holds dims 8c .. 8c+7 of every block).
#include "kvq_internal.cuh"
#include "mma_util.cuh"

namespace kvq {
namespace {
using namespace mma;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kPassRows = 64;            // query rows in shared memory at a time
constexpr int kManyTiles = 4;            // tiles per warp when several passes over the rows are needed
constexpr int kWinTokens = 32;           // window tokens per CTA
constexpr int kWinRows = 16;             // query rows of a window pass: two per warp
constexpr float kLog2e = 1.4426950408889634f;

template <int D, bool SPLIT>
__host__ __device__ constexpr int frag_bytes() { return kPassRows * D * 2 * (SPLIT ? 2 : 1); }
// operand fragments, per-block query sums, alpha, lse and limit per row, a row buffer per warp
template <int D, bool SPLIT>
__host__ __device__ constexpr int body_smem() {
  return frag_bytes<D, SPLIT>() + kPassRows * (D / 32 + 3) * 4 + kWarps * D * 4;
}
template <int D>
__host__ __device__ constexpr int window_smem() { return (kWinTokens * (D + 4) + kWinRows * D + kWarps * kWinTokens + 2 * kWinRows) * 4; }
template <int KL, int D, bool SPLIT>
__host__ __device__ constexpr int smem_bytes() {
  return is_hadamard(KL) && window_smem<D>() > body_smem<D, SPLIT>() ? window_smem<D>() : body_smem<D, SPLIT>();
}

// The packed codes of the 8 dims 32b + 8c .. of one token, for every block b: what one lane holds.
template <int KL, int NB>
struct RowWords {
  static constexpr int N = KL == KVQ_Q8_0 || KL == KVQ_Q6_0 ? 2 : 1;
  uint32_t w[NB][N];
};
template <int KL, int NB>
__device__ __forceinline__ void load_words(const uint8_t *row, int c, RowWords<KL, NB> &r) {
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if constexpr (KL == KVQ_Q8_0) {
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(row + 32 * b + 8 * c));
      r.w[b][0] = v.x;
      r.w[b][1] = v.y;
    } else if constexpr (KL == KVQ_Q6_0) {
      r.w[b][0] = __ldg(reinterpret_cast<const uint32_t *>(row + 24 * b + 4 * c));
      r.w[b][1] = __ldg(reinterpret_cast<const uint16_t *>(row + 24 * b + 16 + 2 * c));
    } else if constexpr (KL == KVQ_HAD_INT2) {
      r.w[b][0] = __ldg(reinterpret_cast<const uint16_t *>(row + 8 * b + 2 * c));
    } else {
      r.w[b][0] = __ldg(reinterpret_cast<const uint32_t *>(row + 16 * b + 4 * c));
    }
  }
}
// -> four exact f16 pairs of the codes: values (0,4), (1,5), (2,6), (3,7)
template <int KL, int NB>
__device__ __forceinline__ void unpack_words(const RowWords<KL, NB> &r, int b, uint32_t (&o)[4]) {
  if constexpr (KL == KVQ_Q8_0) unpack8_s8(r.w[b][0], r.w[b][1], o);
  else if constexpr (KL == KVQ_Q6_0) unpack8_s6(r.w[b][0], r.w[b][1], o);
  else if constexpr (KL == KVQ_HAD_INT2) unpack8_s2(r.w[b][0], o);
  else if constexpr (KL == KVQ_ASYM4_G32) unpack8_u4(r.w[b][0], o);
  else unpack8_q4(r.w[b][0], o);
}

// One token tile as a lane holds it: rows g and g + 8.
template <int KL, int D>
struct Tile {
  static constexpr int NB = D / 32, NS = is_hadamard(KL) ? 1 : NB / 2;   // scale words (f16 pairs, or one f32)
  RowWords<KL, NB> k[2];
  uint32_t scale[2][NS];
  uint32_t zero[2][KL == KVQ_ASYM4_G32 ? NB / 2 : 1];
};
template <int KL, int D>
__device__ __forceinline__ void load_tile(const CacheView &cv, int bb, int kvh, int t0, int t_last, int g, int c, Tile<KL, D> &t) {
  constexpr int NB = D / 32;
  const size_t row0 = cache_row(cv, bb, kvh, t0);        // 16 aligned tokens are consecutive rows
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const size_t row = row0 + min(g + 8 * h, t_last - t0);   // rows past the body repeat its last token
    load_words<KL, NB>(cv.payload[0] + row * cv.row_bytes, c, t.k[h]);
    if constexpr (is_hadamard(KL)) {
      t.scale[h][0] = __ldg(static_cast<const uint32_t *>(cv.scale[0]) + row);
    } else {
      const uint32_t *s = static_cast<const uint32_t *>(cv.scale[0]) + row * (NB / 2);
#pragma unroll
      for (int i = 0; i < NB / 2; i += 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(s + i));
        t.scale[h][i] = v.x;
        t.scale[h][i + 1] = v.y;
      }
      if constexpr (KL == KVQ_ASYM4_G32) {
        const uint32_t *z = reinterpret_cast<const uint32_t *>(cv.zero[0]) + row * (NB / 2);
#pragma unroll
        for (int i = 0; i < NB / 2; i += 2) {
          const uint2 v = __ldg(reinterpret_cast<const uint2 *>(z + i));
          t.zero[h][i] = v.x;
          t.zero[h][i + 1] = v.y;
        }
      }
    }
  }
}

struct RowParams {
  float *alpha, *lse2;         // score factor and log-sum-exp in base 2 (+infinity: the row adds nothing)
  int *limit;                  // last token the row sees
};

// One query row r of the kv head into shared memory: operand fragments of its prescaled values (or int8
// codes), block sums, factor, log-sum-exp. A whole warp; rows past the last are zero and add nothing.
template <int KL, int D, bool SPLIT>
__device__ __forceinline__ void prepare_row(const AttendArgs &a, const SeqLen &sl, int bb, int kvh, int r, int slot, int lane,
                                            float *buf, uint2 *frag, float *qsum, const RowParams &p) {
  constexpr int V = D / 32, KS = D / 16;
  const bool live = r < a.gqa * a.n_q;
  const size_t row = live ? query_row_index(a, bb, kvh, r) : 0;
  float x[V];
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = 0.0f;
  if (live) {
    if constexpr (V == 4) load4_f32(a.q, a.q_dtype, row * D + lane * V, x);
    else load8_f32(a.q, a.q_dtype, row * D + lane * V, x);
  }
  float alpha;
  if constexpr (is_hadamard(KL)) {
    int q8[V];
    const float s = had_query_row<V>(x, q8, lane);
    alpha = a.scale * s * kLog2e;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = (float)q8[i];
  } else {
    // power-of-two prescale: the row's largest |q| in [2^13, 2^14), exact and inside f16
    float mx = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) mx = fmaxf(mx, fabsf(x[i]));
#pragma unroll
    for (int m = 16; m; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
    int e = 0;
    if (mx > 0.0f) e = min(max(((__float_as_int(mx) >> 23) & 0xFF) - 127 - 13, -100), 100);
    const float pre = ldexpf(1.0f, -e);
    alpha = a.scale * ldexpf(1.0f, e) * kLog2e;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] *= pre;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) buf[lane * V + i] = x[i];
  __syncwarp();
  const bool mine = lane < D / 8;                        // lane = 4 * block + c: dims 8 * lane .. + 7
  float v[8], s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = mine ? buf[8 * lane + i] : 0.0f;
    s += v[i];
  }
  if (mine) {
    const int b = lane >> 2, c = lane & 3;
    uint2 *f = frag + ((size_t)(slot >> 3) * KS + 2 * b) * 32 + (slot & 7) * 4 + c;
    f[0] = make_uint2(pack_f16x2(v[0], v[4]), pack_f16x2(v[1], v[5]));
    f[32] = make_uint2(pack_f16x2(v[2], v[6]), pack_f16x2(v[3], v[7]));
    if constexpr (SPLIT) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] -= __half2float(__float2half_rn(v[i]));
      f += kPassRows / 8 * KS * 32;
      f[0] = make_uint2(pack_f16x2(v[0], v[4]), pack_f16x2(v[1], v[5]));
      f[32] = make_uint2(pack_f16x2(v[2], v[6]), pack_f16x2(v[3], v[7]));
    }
  }
  if constexpr (KL == KVQ_ASYM4_G32) {
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if (mine && (lane & 3) == 0) qsum[slot * (D / 32) + (lane >> 2)] = s;
  }
  if (lane == 0) {
    const float lse = live ? a.lse[row] : -INFINITY;
    const bool seen = lse > -INFINITY;
    p.alpha[slot] = seen ? alpha : 0.0f;
    p.lse2[slot] = seen ? lse * kLog2e : INFINITY;
    p.limit[slot] = live ? row_limit(a, sl, r % a.n_q) : -1;
  }
  __syncwarp();
}

// Adds to w[0] / w[1] (tokens g and g + 8 of the tile at t0) the weights of eight query rows.
// f: the rows' operand fragments (this lane's), sums their block sums, p their parameters.
template <int KL, int D, bool SPLIT, class F>
__device__ __forceinline__ void add_rows(const Tile<KL, D> &t, const uint32_t (&A)[D / 16][4], F frag, const float *sums,
                                         const RowParams &p, int t0, bool masked, int g, int c, float (&w)[2]) {
  constexpr int NB = D / 32;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if constexpr (is_hadamard(KL)) {
    float d[2][4] = {};                                  // two chains of the exact integer dot
#pragma unroll
    for (int ks = 0; ks < 2 * NB; ++ks) {
      const uint2 b = frag(ks);
      mma16816(d[ks & 1], A[ks], b.x, b.y);
    }
    const float s0 = __uint_as_float(t.scale[0][0]), s1 = __uint_as_float(t.scale[1][0]);
    x[0] = (d[0][0] + d[1][0]) * s0;
    x[1] = (d[0][1] + d[1][1]) * s0;
    x[2] = (d[0][2] + d[1][2]) * s1;
    x[3] = (d[0][3] + d[1][3]) * s1;
  } else {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float d[4];
      const uint2 f0 = frag(2 * b), f1 = frag(2 * b + 1);
      mma16816_c(d, A[2 * b], f0.x, f0.y, 0.f, 0.f, 0.f, 0.f);
      mma16816(d, A[2 * b + 1], f1.x, f1.y);
      if constexpr (SPLIT) {
        const uint2 l0 = frag(2 * NB + 2 * b), l1 = frag(2 * NB + 2 * b + 1);
        mma16816(d, A[2 * b], l0.x, l0.y);
        mma16816(d, A[2 * b + 1], l1.x, l1.y);
      }
      const float2 sa = __half22float2(u32_as_h2(t.scale[0][b >> 1])), sb = __half22float2(u32_as_h2(t.scale[1][b >> 1]));
      const float s0 = (b & 1) ? sa.y : sa.x, s1 = (b & 1) ? sb.y : sb.x;
      x[0] = fmaf(s0, d[0], x[0]);
      x[1] = fmaf(s0, d[1], x[1]);
      x[2] = fmaf(s1, d[2], x[2]);
      x[3] = fmaf(s1, d[3], x[3]);
      if constexpr (KL == KVQ_ASYM4_G32) {
        const float2 za = __half22float2(u32_as_h2(t.zero[0][b >> 1])), zb = __half22float2(u32_as_h2(t.zero[1][b >> 1]));
        const float z0 = (b & 1) ? za.y : za.x, z1 = (b & 1) ? zb.y : zb.x;
        const float q0 = sums[2 * c * NB + b], q1 = sums[(2 * c + 1) * NB + b];
        x[0] = fmaf(z0, q0, x[0]);
        x[1] = fmaf(z0, q1, x[1]);
        x[2] = fmaf(z1, q0, x[2]);
        x[3] = fmaf(z1, q1, x[3]);
      }
    }
  }
  const float2 al = *reinterpret_cast<const float2 *>(p.alpha + 2 * c), ls = *reinterpret_cast<const float2 *>(p.lse2 + 2 * c);
  float e[4] = {ex2(fmaf(x[0], al.x, -ls.x)), ex2(fmaf(x[1], al.y, -ls.y)), ex2(fmaf(x[2], al.x, -ls.x)),
                ex2(fmaf(x[3], al.y, -ls.y))};
  if (masked) {
    const int2 lim = *reinterpret_cast<const int2 *>(p.limit + 2 * c);
    if (t0 + g > lim.x) e[0] = 0.0f;
    if (t0 + g > lim.y) e[1] = 0.0f;
    if (t0 + g + 8 > lim.x) e[2] = 0.0f;
    if (t0 + g + 8 > lim.y) e[3] = 0.0f;
  }
  w[0] += e[0] + e[1];
  w[1] += e[2] + e[3];
}

// The sum over a quad's query rows, then scores_out of the tile's sixteen tokens.
__device__ __forceinline__ void write_tile(const WeightArgs &wa, size_t head, int t0, int n_body, int g, int c, float (&w)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] += __shfl_xor_sync(0xffffffffu, w[h], 1);
    w[h] += __shfl_xor_sync(0xffffffffu, w[h], 2);
  }
  const int t = t0 + g + 8 * c;
  if (c < 2 && t < n_body) {
    const size_t at = head * (size_t)wa.stride + t;
    const float v = c ? w[1] : w[0];
    wa.scores_out[at] = wa.scores_in ? fmaf(wa.decay, wa.scores_in[at], v) : v;
  }
}

// Window tokens [n_body + 32 j, ..) of one kv head: lanes are tokens, warps are query rows.
template <int D>
__device__ __forceinline__ void window_tokens(const WeightArgs &wa, const SeqLen &sl, int bb, int kvh, int j, float *sm) {
  const AttendArgs &a = wa.a;
  constexpr int V = D / 32, KST = D + 4;                  // row stride: 16-byte reads of 8 rows hit all banks
  float *ks = sm, *qs = ks + kWinTokens * KST, *part = qs + kWinRows * D, *lse2 = part + kWarps * kWinTokens;
  int *lim = reinterpret_cast<int *>(lse2 + kWinRows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rows = a.gqa * a.n_q;
  const int t0 = sl.n_body + j * kWinTokens, n = min(kWinTokens, sl.kv_len - t0);
  const size_t head = (size_t)bb * a.cache.H + kvh;
  const float *ring = a.cache.ring[0] + head * a.cache.n_recent * D;
  for (int i = threadIdx.x; i < kWinTokens * (D / 4); i += kThreads) {
    const int t = i / (D / 4), d = i % (D / 4) * 4;
    const float *src = ring + (size_t)((t0 + min(t, n - 1)) % a.cache.n_recent) * D + d;
    *reinterpret_cast<float4 *>(ks + t * KST + d) = *reinterpret_cast<const float4 *>(src);
  }
  float w = 0.0f;
  for (int r0 = 0; r0 < rows; r0 += kWinRows) {
    __syncthreads();                                     // the last pass's rows are read; the keys are there
    for (int s = warp; s < kWinRows; s += kWarps) {
      const int r = r0 + s;
      const bool live = r < rows;
      const size_t row = live ? query_row_index(a, bb, kvh, r) : 0;
      float x[V];
      int q8[V];
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = 0.0f;
      if (live) {
        if constexpr (V == 4) load4_f32(a.q, a.q_dtype, row * D + lane * V, x);
        else load8_f32(a.q, a.q_dtype, row * D + lane * V, x);
      }
      had_query_row<V>(x, q8, lane);                      // x: the rotated f32 row
#pragma unroll
      for (int i = 0; i < V; ++i) qs[s * D + lane * V + i] = x[i];
      if (lane == 0) {
        const float lse = live ? a.lse[row] : -INFINITY;
        lse2[s] = lse > -INFINITY ? lse * kLog2e : INFINITY;
        lim[s] = live ? row_limit(a, sl, r % a.n_q) : -1;
      }
    }
    __syncthreads();
    const float *q0 = qs + (2 * warp) * D, *q1 = q0 + D;
    float d0 = 0.0f, d1 = 0.0f;
#pragma unroll 8
    for (int d = 0; d < D; d += 4) {
      const float4 k = *reinterpret_cast<const float4 *>(ks + lane * KST + d);
      const float4 x = *reinterpret_cast<const float4 *>(q0 + d), y = *reinterpret_cast<const float4 *>(q1 + d);
      d0 = fmaf(x.x, k.x, fmaf(x.y, k.y, fmaf(x.z, k.z, fmaf(x.w, k.w, d0))));
      d1 = fmaf(y.x, k.x, fmaf(y.y, k.y, fmaf(y.z, k.z, fmaf(y.w, k.w, d1))));
    }
    const float f = a.scale * kLog2e;
    const int t = t0 + lane;
    if (t <= lim[2 * warp]) w += ex2(fmaf(d0, f, -lse2[2 * warp]));
    if (t <= lim[2 * warp + 1]) w += ex2(fmaf(d1, f, -lse2[2 * warp + 1]));
  }
  part[warp * kWinTokens + lane] = w;
  __syncthreads();
  if (warp == 0 && lane < n) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v += part[k * kWinTokens + lane];
    const size_t at = head * (size_t)wa.stride + t0 + lane;
    wa.scores_out[at] = wa.scores_in ? fmaf(wa.decay, wa.scores_in[at], v) : v;
  }
}

// MANY: more query rows than one pass holds (every warp then keeps kManyTiles tiles' sums across the
// passes and reads their packed rows again from the cache); else any number of tiles per warp.
template <int KL, int D, bool SPLIT, bool MANY>
__global__ void __launch_bounds__(kThreads, D == 128 && !SPLIT ? 3 : 2) attend_weights_kernel(WeightArgs wa) {
  constexpr int KS = D / 16;
  extern __shared__ __align__(16) uint8_t smem[];
#if defined(__CUDA_ARCH__) && __CUDA_ARCH__ >= 900
  asm volatile("griddepcontrol.wait;" ::: "memory");     // the rows' log-sum-exp come from phase 2
#endif
  const AttendArgs &a = wa.a;
  const CacheView &cv = a.cache;
  const int bh = blockIdx.y, bb = bh / cv.H, kvh = bh - bb * cv.H;
  const SeqLen sl = seq_of(a, bb);
  if (is_hadamard(KL) && (int)blockIdx.x >= wa.n_ctas) {
    const int j = (int)blockIdx.x - wa.n_ctas;
    if (sl.n_body + j * kWinTokens < sl.kv_len)
      window_tokens<D>(wa, sl, bb, kvh, j, reinterpret_cast<float *>(smem));
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int n_tiles = (sl.n_body + 15) / 16;
  // the CTA's tiles, dealt to the warps in turn
  const int first = (int)blockIdx.x * wa.tiles * kWarps;
  if (first >= n_tiles) return;
  const int rows = a.gqa * a.n_q;
  uint2 *frag = reinterpret_cast<uint2 *>(smem);
  float *qsum = reinterpret_cast<float *>(smem + frag_bytes<D, SPLIT>());
  RowParams p;
  p.alpha = qsum + kPassRows * (D / 32);
  p.lse2 = p.alpha + kPassRows;
  p.limit = reinterpret_cast<int *>(p.lse2 + kPassRows);
  float *buf = p.lse2 + 2 * kPassRows + warp * D;
  // tokens behind the first row's limit need the per-row test (limits grow with the query index)
  const int min_lim = row_limit(a, sl, 0);
  const int t_last = sl.n_body - 1;
  float w[MANY ? kManyTiles : 1][2] = {};
  for (int r0 = 0; r0 < rows; r0 += kPassRows) {
    const int n_rows = min(rows - r0, kPassRows), n_slots = (n_rows + 7) / 8 * 8;
    if (MANY && r0 > 0) __syncthreads();
    for (int s = warp; s < n_slots; s += kWarps)
      prepare_row<KL, D, SPLIT>(a, sl, bb, kvh, r0 + s, s, lane, buf, frag, qsum, p);
    __syncthreads();
    for (int i = 0; i < (MANY ? kManyTiles : wa.tiles); ++i) {
      const int tile = first + i * kWarps + warp;
      if (tile >= n_tiles) break;
      const int t0 = 16 * tile;
      Tile<KL, D> t;
      load_tile<KL, D>(cv, bb, kvh, t0, t_last, g, c, t);
      uint32_t A[KS][4];
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        uint32_t lo[4], hi[4];
        unpack_words<KL, D / 32>(t.k[0], b, lo);
        unpack_words<KL, D / 32>(t.k[1], b, hi);
        A[2 * b][0] = lo[0]; A[2 * b][1] = hi[0]; A[2 * b][2] = lo[1]; A[2 * b][3] = hi[1];
        A[2 * b + 1][0] = lo[2]; A[2 * b + 1][1] = hi[2]; A[2 * b + 1][2] = lo[3]; A[2 * b + 1][3] = hi[3];
      }
      float sum[2] = {0.f, 0.f};
      const bool masked = t0 + 15 > min_lim;
      for (int nt = 0; nt < n_slots / 8; ++nt) {
        const uint2 *f = frag + (size_t)nt * KS * 32 + lane;
        auto get = [&](int ks) { return ks < KS ? f[ks * 32] : f[(kPassRows / 8 * KS + ks - KS) * 32]; };
        const RowParams q = {p.alpha + 8 * nt, p.lse2 + 8 * nt, p.limit + 8 * nt};
        add_rows<KL, D, SPLIT>(t, A, get, qsum + 8 * nt * (D / 32), q, t0, masked, g, c, sum);
      }
      if constexpr (MANY) {
#pragma unroll
        for (int k = 0; k < kManyTiles; ++k)
          if (k == i) {
            w[k][0] += sum[0];
            w[k][1] += sum[1];
          }
      } else {
        write_tile(wa, bh, t0, sl.n_body, g, c, sum);
      }
    }
  }
  if constexpr (MANY) {
#pragma unroll
    for (int k = 0; k < kManyTiles; ++k) {
      const int tile = first + k * kWarps + warp;
      if (tile < n_tiles) write_tile(wa, bh, 16 * tile, sl.n_body, g, c, w[k]);
    }
  }
}

template <int KL, int D, bool SPLIT, bool MANY>
cudaError_t launch_one(WeightArgs &wa, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  constexpr int smem = smem_bytes<KL, D, SPLIT>();
  cudaError_t e = set_smem_once(done, attend_weights_kernel<KL, D, SPLIT, MANY>, smem);
  if (e != cudaSuccess) return e;
  const AttendArgs &a = wa.a;
  cudaLaunchConfig_t cfg = {};
  const int n_win = is_hadamard(KL) ? (a.n_win + kWinTokens - 1) / kWinTokens : 0;
  // a paged sequence shorter than its window still has none of it in the body: the body is sized for
  // the longest sequence, whose body is kv_len - n_win
  wa.n_ctas = (a.n_body + 16 * kWarps * wa.tiles - 1) / (16 * kWarps * wa.tiles);
  cfg.gridDim = dim3((unsigned)(wa.n_ctas + n_win), (unsigned)(a.cache.B * a.cache.H));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_weights_kernel<KL, D, SPLIT, MANY>, wa);
}

template <int KL, int D>
cudaError_t launch_layout(WeightArgs &wa, cudaStream_t st) {
  const bool many = wa.a.gqa * wa.a.n_q > kPassRows;
  wa.tiles = kManyTiles;
  if constexpr (is_hadamard(KL)) {
    return many ? launch_one<KL, D, false, true>(wa, st) : launch_one<KL, D, false, false>(wa, st);
  } else {
    if (wa.a.q_dtype == KVQ_F32) return many ? launch_one<KL, D, true, true>(wa, st) : launch_one<KL, D, true, false>(wa, st);
    return many ? launch_one<KL, D, false, true>(wa, st) : launch_one<KL, D, false, false>(wa, st);
  }
}

template <int D>
cudaError_t launch_dim(WeightArgs &wa, cudaStream_t st) {
  switch (wa.a.cache.layout) {
    case KVQ_Q4_0: return launch_layout<KVQ_Q4_0, D>(wa, st);
    case KVQ_Q6_0: return launch_layout<KVQ_Q6_0, D>(wa, st);
    case KVQ_Q8_0: return launch_layout<KVQ_Q8_0, D>(wa, st);
    case KVQ_ASYM4_G32: return launch_layout<KVQ_ASYM4_G32, D>(wa, st);
    case KVQ_HAD_INT4: return launch_layout<KVQ_HAD_INT4, D>(wa, st);
    default: return launch_layout<KVQ_HAD_INT2, D>(wa, st);
  }
}

}  // namespace

cudaError_t launch_attend_weights(const AttendArgs &a, const float *scores_in, float *scores_out, long long stride,
                                  float decay, cudaStream_t st) {
  WeightArgs wa;
  wa.a = a;
  wa.scores_in = decay == 0.0f ? nullptr : scores_in;
  wa.scores_out = scores_out;
  wa.stride = stride;
  wa.decay = decay;
  return a.cache.D == 128 ? launch_dim<128>(wa, st) : launch_dim<256>(wa, st);
}

}  // namespace kvq
