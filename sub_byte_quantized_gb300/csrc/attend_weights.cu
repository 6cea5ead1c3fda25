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
// Decode calls need no second pass over K: their phase 1 leaves its masked scores behind (4 bytes per query
// row and token, against 72 to 136 for a packed K row, and mostly still in L2), and one small kernel turns
// them into weights. The others score K again:
//   up to eight query rows per kv head   bound by the K plane's bytes: each warp streams 32-token stages
//       through a private cp.async ring, with the rows' operand fragments in registers
//   more rows, head_dim 128              attend_weights_tc.cu
//   more rows, head_dim 256              bound by the tensor pipe and the exponentials: the rows' fragments sit
//       in shared memory, 64 rows at a time, and a warp applies them to 16 tokens that it holds in registers
#include "attend_weights.cuh"

namespace kvq {
namespace {
using namespace weights;

constexpr int kFewWarps = 4;             // warps per CTA, up to eight rows
constexpr int kManyWarps = 8;            // warps per CTA, more rows
constexpr int kStage = 32;               // tokens of a stage or of a warp's unit
constexpr int kRing = 3;                 // stages per warp in shared memory

constexpr int kPassRows = 64;             // query rows in shared memory at a time, more rows
// The rows' operand fragments (hi, then lo), block sums, alpha, lse and limit, and a row buffer per warp.
template <int D, bool SPLIT, int ROWS, int WARPS>
__host__ __device__ constexpr int rows_smem() { return ROWS * D * 2 * (SPLIT ? 2 : 1) + ROWS * (D / 32 + 3) * 4 + WARPS * D * 4; }

// A plane of one layout: bytes of a row, and of its scales (and zero-points).
template <int KL, int D>
__host__ __device__ constexpr int row_bytes() {
  return KL == KVQ_Q8_0 ? D : KL == KVQ_Q6_0 ? D / 32 * 24 : KL == KVQ_HAD_INT2 ? D / 4 : D / 2;
}
template <int KL, int D>
__host__ __device__ constexpr int scale_bytes() { return is_hadamard(KL) ? 4 : D / 16; }
// A stage: rows padded by 16 bytes (an odd number of 16-byte columns: the fragment reads of eight rows
// fall in different banks), then scales, then zero-points.
template <int KL, int D>
__host__ __device__ constexpr int stage_bytes() {
  return kStage * (row_bytes<KL, D>() + 16 + scale_bytes<KL, D>() * (KL == KVQ_ASYM4_G32 ? 2 : 1));
}

// Operand order. A row's bytes are read in 16-byte columns; lane c of a quad holds the 4-byte word c of
// every column (what ldmatrix gives), except Q6_0, whose 24-byte blocks are read word by word:
//   4-bit codes   column = block b, dims 32b + 8c + 0..7:  k-steps 2b, 2b+1 take (0,4) (1,5) and (2,6) (3,7)
//   8-bit codes   columns 2b, 2b+1, dims 32b + 4c + 0..3 and 32b + 16 + 4c + 0..3: (0,1) (2,3) each
//   2-bit codes   column = 64 dims, 16c + 0..15: k-step k takes (k, 8 + k) (4 + k, 12 + k)
//   Q6_0          dims 32b + 8c + 0..7, as the 4-bit codes
// Hadamard codes stay where they are in their f16 lane, as exact subnormals u 16^j 2^-24 or u 4^k 2^-24 of the
// offset code u = code + 8 or code + 2: one lop3 per pair. The query entries facing a shifted field are divided by
// it, the 2^-24 goes into the row's factor and the offset times the query's sum into the accumulator's initial
// value; all of it is exact in integers. The other layouts' codes become exact signed values (asymmetric: code - 8,
// and the zero-point z + 8 s), since offsets would cost the scores' precision.
template <int KL, int D>
struct Words {
  static constexpr int NB = D / 32, N = KL == KVQ_Q6_0 ? 2 * NB : row_bytes<KL, D>() / 16;
};
// Words of one row from global memory.
template <int KL, int D>
__device__ __forceinline__ void load_words(const uint8_t *row, int c, uint32_t (&w)[Words<KL, D>::N]) {
  if constexpr (KL == KVQ_Q6_0) {
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
      w[2 * b] = __ldg(reinterpret_cast<const uint32_t *>(row + 24 * b + 4 * c));
      w[2 * b + 1] = __ldg(reinterpret_cast<const uint16_t *>(row + 24 * b + 16 + 2 * c));
    }
  } else {
#pragma unroll
    for (int j = 0; j < Words<KL, D>::N; ++j) w[j] = __ldg(reinterpret_cast<const uint32_t *>(row + 16 * j + 4 * c));
  }
}
// One row's words -> its half h of the A fragments (0: token g, 1: token g + 8).
template <int KL, int D>
__device__ __forceinline__ void unpack_row(const uint32_t (&w)[Words<KL, D>::N], int h, uint32_t (&A)[D / 16][4]) {
  if constexpr (KL == KVQ_HAD_INT2) {
#pragma unroll
    for (int ch = 0; ch < D / 64; ++ch) {
      const uint32_t lo = prmt(w[ch], 0u, 0x4240u), hi = prmt(w[ch], 0u, 0x4341u);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t m = 0x00030003u << (2 * k), x = 0x00020002u << (2 * k);
        A[4 * ch + k][h] = lop3<0x6a>(lo, m, x);
        A[4 * ch + k][2 + h] = lop3<0x6a>(hi, m, x);
      }
    }
  } else {
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
      uint32_t o[4];
      if constexpr (KL == KVQ_Q8_0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t x = w[2 * b + i] ^ 0x80808080u;   // code + 128 under the exponent of 1024, then - 1152
          o[2 * i] = hadd2(prmt(x, 0x64646464u, 0x4140u), 0xE480E480u);
          o[2 * i + 1] = hadd2(prmt(x, 0x64646464u, 0x4342u), 0xE480E480u);
        }
      } else if constexpr (KL == KVQ_Q6_0) {
        unpack8_s6(w[2 * b], w[2 * b + 1], o);
      } else {
        if constexpr (is_hadamard(KL)) unpack8_sub<false>(w[b], o);
        else if constexpr (KL == KVQ_ASYM4_G32) unpack8_u4m8(w[b], o);
        else unpack8_q4(w[b], o);
      }
      A[2 * b][h] = o[0];
      A[2 * b][2 + h] = o[1];
      A[2 * b + 1][h] = o[2];
      A[2 * b + 1][2 + h] = o[3];
    }
  }
}

// One 16-token tile as a lane holds it (tokens g and g + 8): operand fragments of its codes, scales and
// zero-points in f32.
template <int KL, int D>
struct Tile {
  static constexpr int NB = D / 32, NS = is_hadamard(KL) ? 1 : NB;
  uint32_t A[2 * NB][4];
  float scale[2][NS], zero[2][KL == KVQ_ASYM4_G32 ? NB : 1];
};
// SMEM: the scales lie in shared memory (else global, read-only).
template <bool SMEM, class T>
__device__ __forceinline__ T load_of(const uint8_t *p) {
  if constexpr (SMEM) return *reinterpret_cast<const T *>(p);
  else return __ldg(reinterpret_cast<const T *>(p));
}
template <bool SMEM, int N>
__device__ __forceinline__ void f16_scales(const uint8_t *p, float (&out)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const uint2 v = load_of<SMEM, uint2>(p + 2 * i);
    const float2 f = __half22float2(u32_as_h2(v.x)), e = __half22float2(u32_as_h2(v.y));
    out[i] = f.x; out[i + 1] = f.y; out[i + 2] = e.x; out[i + 3] = e.y;
  }
}
template <bool SMEM, int KL, int D>
__device__ __forceinline__ void load_scales(const uint8_t *scale, const uint8_t *zero, int h, Tile<KL, D> &t) {
  if constexpr (is_hadamard(KL)) t.scale[h][0] = load_of<SMEM, float>(scale);
  else f16_scales<SMEM>(scale, t.scale[h]);
  if constexpr (KL == KVQ_ASYM4_G32) {
    f16_scales<SMEM>(zero, t.zero[h]);
#pragma unroll
    for (int b = 0; b < D / 32; ++b) t.zero[h][b] = fmaf(8.0f, t.scale[h][b], t.zero[h][b]);
  }
}

struct RowParams {
  float *alpha, *lse2;         // score factor and log-sum-exp in base 2 (+infinity: the row adds nothing)
  int *limit;                  // last token the row sees
};

// One query row r of the kv head into shared memory: operand fragments of its prescaled values (or int8
// codes), two k-steps to 16 bytes (lo parts lo_at entries behind), the accumulator's block terms, and the
// row's factor. A whole warp; rows past the last are zero.
template <int KL, int D, bool SPLIT>
__device__ __forceinline__ void prepare_row(const AttendArgs &a, int bb, int kvh, int r, int slot, int lane, float *buf,
                                            uint4 *frag, int lo_at, float *qsum, float *alpha_out) {
  constexpr int V = D / 32, KP = D / 32;                 // values per lane; pairs of k-steps
  constexpr bool SUB = is_hadamard(KL);                  // codes enter as subnormals
  const bool live = r < a.gqa * a.n_q;
  const size_t row = live ? query_row_index(a, bb, kvh, r) : 0;
  float x[V];
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = 0.0f;
  if (live) {
    if constexpr (V == 4) load4_f32(a.q, a.q_dtype, row * D + lane * V, x);
    else load8_f32(a.q, a.q_dtype, row * D + lane * V, x);
  }
  float alpha = a.scale * kLog2e * (SUB ? 16777216.0f : 1.0f);
  if constexpr (is_hadamard(KL)) {
    int q8[V];
    alpha *= had_query_row<V>(x, q8, lane);
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
    const float pre = __int_as_float((127 - e) << 23);
    alpha *= __int_as_float((127 + e) << 23);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] *= pre;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) buf[lane * V + i] = x[i];
  __syncwarp();
  // lane 4 b + c: pair b of k-steps, quad lane c
  const int b = lane >> 2, c = lane & 3;
  float v[8], s = 0.0f;                                  // the eight entries of its fragment, in order
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    int d;
    float f = 1.0f;
    if constexpr (KL == KVQ_HAD_INT2) {
      // k-steps 2b, 2b + 1 are k = 2 (b % 2) and the next of column b / 2
      const int k = 2 * (b & 1) + (i >> 2);
      d = 64 * (b >> 1) + 16 * c + k + ((i & 1) ? 8 : 0) + ((i & 2) ? 4 : 0);
      f = 1.0f / (float)(1 << (2 * k));
    } else if constexpr (KL == KVQ_Q8_0) {
      d = 32 * b + 4 * c + (i & 3) + 16 * (i >> 2);
    } else {
      d = 32 * b + 8 * c + 2 * (i >> 2) + ((i & 2) >> 1) + 4 * (i & 1);
      if (SUB && (i & 2)) f = 0.0625f;
    }
    const float y = lane < D / 8 ? buf[d] : 0.0f;
    s += y;
    v[i] = y * f;
  }
  if (lane < D / 8) {
    uint4 *f = frag + ((slot >> 3) * KP + b) * 32 + (slot & 7) * 4 + c;
    f[0] = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
    if constexpr (SPLIT) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] -= __half2float(__float2half_rn(v[i]));
      f[lo_at] = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
    }
  }
  if constexpr (SUB || KL == KVQ_ASYM4_G32) {
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if constexpr (is_hadamard(KL)) {                     // one accumulator: the whole row's sum in block 0
#pragma unroll
      for (int m = 4; m < 32; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    }
    constexpr float kTerm = !SUB ? 1.0f : (KL == KVQ_HAD_INT2 ? -2.0f : -8.0f) * 5.9604644775390625e-8f;
    if (lane < D / 8 && c == 0) qsum[slot * KP + b] = s * kTerm;
  }
  if (lane == 0) alpha_out[slot] = alpha;
  __syncwarp();
}
// Adds to w[0] / w[1] (tokens t0 + g and t0 + g + 8) the weights of eight query rows, of which this
// lane's accumulator columns are rows 2c and 2c + 1: factors al, log-sum-exp ls, limits lim, and block
// terms q0 / q1. frag(b): the rows' operand fragments of k-steps 2b and 2b + 1 (lo parts from D / 32 on).
template <int KL, int D, bool SPLIT, class F>
__device__ __forceinline__ void add_rows(const Tile<KL, D> &t, F frag, float2 al, float2 ls, int2 lim, const float *q0,
                                         const float *q1, int t0, bool masked, int g, float (&w)[2]) {
  constexpr int NB = D / 32;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if constexpr (is_hadamard(KL)) {
    float d[2][4];                                       // two chains of the exact integer dot x 2^-24
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint4 f = frag(b);
      if (b == 0) {
        mma16816_c(d[0], t.A[0], f.x, f.y, q0[0], q1[0], q0[0], q1[0]);
        mma16816_c(d[1], t.A[1], f.z, f.w, 0.f, 0.f, 0.f, 0.f);
      } else {
        mma16816(d[0], t.A[2 * b], f.x, f.y);
        mma16816(d[1], t.A[2 * b + 1], f.z, f.w);
      }
    }
    x[0] = (d[0][0] + d[1][0]) * t.scale[0][0];
    x[1] = (d[0][1] + d[1][1]) * t.scale[0][0];
    x[2] = (d[0][2] + d[1][2]) * t.scale[1][0];
    x[3] = (d[0][3] + d[1][3]) * t.scale[1][0];
  } else {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float d[4];
      const uint4 f = frag(b);
      mma16816_c(d, t.A[2 * b], f.x, f.y, 0.f, 0.f, 0.f, 0.f);
      mma16816(d, t.A[2 * b + 1], f.z, f.w);
      if constexpr (SPLIT) {
        const uint4 l = frag(NB + b);
        mma16816(d, t.A[2 * b], l.x, l.y);
        mma16816(d, t.A[2 * b + 1], l.z, l.w);
      }
      const float s0 = t.scale[0][b], s1 = t.scale[1][b];
      x[0] = fmaf(s0, d[0], x[0]);
      x[1] = fmaf(s0, d[1], x[1]);
      x[2] = fmaf(s1, d[2], x[2]);
      x[3] = fmaf(s1, d[3], x[3]);
      if constexpr (KL == KVQ_ASYM4_G32) {
        const float z0 = t.zero[0][b], z1 = t.zero[1][b];
        x[0] = fmaf(z0, q0[b], x[0]);
        x[1] = fmaf(z0, q1[b], x[1]);
        x[2] = fmaf(z1, q0[b], x[2]);
        x[3] = fmaf(z1, q1[b], x[3]);
      }
    }
  }
  float e[4] = {ex2(fmaf(x[0], al.x, -ls.x)), ex2(fmaf(x[1], al.y, -ls.y)), ex2(fmaf(x[2], al.x, -ls.x)),
                ex2(fmaf(x[3], al.y, -ls.y))};
  if (masked) {
    if (t0 + g > lim.x) e[0] = 0.0f;
    if (t0 + g > lim.y) e[1] = 0.0f;
    if (t0 + g + 8 > lim.x) e[2] = 0.0f;
    if (t0 + g + 8 > lim.y) e[3] = 0.0f;
  }
  w[0] += e[0] + e[1];
  w[1] += e[2] + e[3];
}

// The weights of 32 tokens, two tiles' w[0], w[1] summed over the quad: lane (g, c) gets token g + 8 c.
// Each exchange sends the half that the partner keeps.
__device__ __forceinline__ float quad_total(const float (&w)[4], int c) {
  const bool odd = c & 1;
  float lo = odd ? w[1] : w[0], hi = odd ? w[3] : w[2];
  lo += __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1);
  hi += __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
  const bool up = c & 2;
  return (up ? hi : lo) + __shfl_xor_sync(0xffffffffu, up ? lo : hi, 2);
}

// This lane's token rows g and g + 8 of the tile at token t0, from the cache.
template <int KL, int D>
__device__ __forceinline__ void load_global_tile(const CacheView &cv, int bb, int kvh, int t0, int t_last, int g, int c,
                                                 Tile<KL, D> &t) {
  const size_t row0 = cache_row(cv, bb, kvh, t0);        // 16 aligned tokens are consecutive rows
  uint32_t w[2][Words<KL, D>::N];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const size_t r = row0 + max(min(g + 8 * h, t_last - t0), 0);   // rows past the body repeat its last token
    load_words<KL, D>(cv.payload[0] + r * row_bytes<KL, D>(), c, w[h]);
    load_scales<false>(static_cast<const uint8_t *>(cv.scale[0]) + r * scale_bytes<KL, D>(),
                       KL == KVQ_ASYM4_G32 ? reinterpret_cast<const uint8_t *>(cv.zero[0]) + r * scale_bytes<KL, D>() : nullptr, h, t);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) unpack_row<KL, D>(w[h], h, t.A);
}
// The same from a stage in shared memory: token row `row` of the stage at sb.
template <int KL, int D>
__device__ __forceinline__ void load_stage_tile(const uint8_t *sb, int row, int lane, Tile<KL, D> &t) {
  constexpr int RB = row_bytes<KL, D>(), SB = scale_bytes<KL, D>(), PITCH = RB + 16, N = Words<KL, D>::N;
  const int g = lane >> 2, c = lane & 3;
  uint32_t w[2][N];
  if constexpr (KL == KVQ_Q6_0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t *p = sb + (row + g + 8 * h) * PITCH;
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        w[h][2 * b] = *reinterpret_cast<const uint32_t *>(p + 24 * b + 4 * c);
        w[h][2 * b + 1] = *reinterpret_cast<const uint16_t *>(p + 24 * b + 16 + 2 * c);
      }
    }
  } else {
    // matrices of an ldmatrix: tokens 0-7 and 8-15 of columns j and j + 1
    const uint32_t at = smem_addr(sb + (row + (lane & 7) + 8 * ((lane >> 3) & 1)) * PITCH + 16 * (lane >> 4));
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      uint32_t m[4];
      ldsm_x4(at + 16 * j, m);
      w[0][j] = m[0];
      w[1][j] = m[1];
      w[0][j + 1] = m[2];
      w[1][j + 1] = m[3];
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint8_t *s = sb + kStage * PITCH + (row + g + 8 * h) * SB;
    load_scales<true>(s, s + kStage * SB, h, t);
    unpack_row<KL, D>(w[h], h, t.A);
  }
}

// Scores that phase 1 has left behind (a.part_s, base 2, RP rows per token): lanes read consecutive 16-byte
// pieces, RP / 4 lanes (at least one) hold a token.
constexpr int kScoreThreads = 256, kScoreTokens = 1024;
template <int RP, int D, bool HAD>
__global__ void __launch_bounds__(kScoreThreads) attend_weights_scores_kernel(WeightArgs wa) {
  constexpr int V = RP < 4 ? RP : 4, LPT = RP / V;       // values per lane, lanes per token
  constexpr int PER = kScoreTokens * LPT / kScoreThreads;
  extern __shared__ __align__(16) uint8_t smem[];
  const AttendArgs &a = wa.a;
  const int bh = blockIdx.y, bb = bh / a.cache.H, kvh = bh - bb * a.cache.H;
  const SeqLen sl = seq_of(a, bb);
  if (HAD && (int)blockIdx.x >= wa.n_ctas) {
    const int j = (int)blockIdx.x - wa.n_ctas;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (sl.n_body + j * kWinTokens < sl.kv_len)
      window_tokens<D, kScoreThreads / 32>(wa, sl, bb, kvh, j, reinterpret_cast<float *>(smem));
    return;
  }
  const int t0 = (int)blockIdx.x * kScoreTokens;
  if (t0 >= sl.n_body) {
    if (blockIdx.x == 0 && blockIdx.y == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  // tokens up to the widest limit (the last query index) have scores; the others have no weight
  const int end = min(sl.n_body, row_limit(a, sl, a.n_q - 1) + 1);
  const float *ps = a.part_s + (size_t)bh * a.s_tokens * RP;
  const float *in = wa.scores_in ? wa.scores_in + (size_t)bh * wa.stride : nullptr;
  float *out = wa.scores_out + (size_t)bh * wa.stride;
  float x[PER][V], old[PER];
  uint64_t last;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(last));
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int i = k * kScoreThreads + (int)threadIdx.x, t = t0 + i / LPT;
    if (t < end) {
      const float *p = ps + (size_t)t * RP + (i % LPT) * V;
      if constexpr (V == 4) asm volatile("ld.global.L2::cache_hint.v4.f32 {%0, %1, %2, %3}, [%4], %5;" : "=f"(x[k][0]), "=f"(x[k][1]), "=f"(x[k][2]), "=f"(x[k][3]) : "l"(p), "l"(last) : "memory");
      else asm volatile("ld.global.L2::cache_hint.v2.f32 {%0, %1}, [%2], %3;" : "=f"(x[k][0]), "=f"(x[k][1]) : "l"(p), "l"(last) : "memory");
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) x[k][v] = -INFINITY;
    }
    old[k] = in && t < sl.n_body ? in[t] : 0.0f;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");     // the rows' log-sum-exp come from phase 2
  float lse2[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    int limit;
    row_result(a, sl, bb, kvh, ((int)threadIdx.x % LPT) * V + v, lse2[v], limit);
  }
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int i = k * kScoreThreads + (int)threadIdx.x, t = t0 + i / LPT;
    float w = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) w += ex2(x[k][v] - lse2[v]);   // a row that adds nothing has lse2 = +infinity
    if (t >= end) w = 0.0f;                              // (a failed row's lse2 is NaN)
    if constexpr (LPT == 2) w += __shfl_xor_sync(0xffffffffu, w, 1);
    if (i % LPT == 0 && t < sl.n_body) out[t] = in ? fmaf(wa.decay, old[k], w) : w;
  }
}

// Up to eight query rows. CTA x of a (batch, kv head) takes every gridDim-th group of four stages.
template <int KL, int D, bool SPLIT>
__global__ void __launch_bounds__(32 * kFewWarps, D == 128 && !SPLIT ? 5 : 1) attend_weights_few_kernel(WeightArgs wa) {
  constexpr int NB = D / 32, RB = row_bytes<KL, D>(), SB = scale_bytes<KL, D>();
  constexpr int STAGE = stage_bytes<KL, D>(), PITCH = RB + 16, OFF_S = kStage * PITCH, OFF_Z = OFF_S + kStage * SB;
  // the rows' operands pass through the ring's last slots, which the first stages leave free
  static_assert(rows_smem<D, SPLIT, 8, kFewWarps>() <= kFewWarps * STAGE, "the query rows fit the last slots");
  extern __shared__ __align__(16) uint8_t smem[];
  const AttendArgs &a = wa.a;
  const CacheView &cv = a.cache;
  const int bh = blockIdx.y, bb = bh / cv.H, kvh = bh - bb * cv.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const SeqLen sl = seq_of(a, bb);
  if (is_hadamard(KL) && (int)blockIdx.x >= wa.n_ctas) {
    const int j = (int)blockIdx.x - wa.n_ctas;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (sl.n_body + j * kWinTokens < sl.kv_len)
      window_tokens<D, kFewWarps>(wa, sl, bb, kvh, j, reinterpret_cast<float *>(smem));
    return;
  }
  const int n_stages = (sl.n_body + kStage - 1) / kStage, step = wa.n_ctas * kFewWarps;
  const int s_first = (int)blockIdx.x * kFewWarps + warp;
  uint8_t *ring = smem + warp * STAGE;                    // slot i of the warp: + i * kFewWarps * STAGE
  // stage s into slot i of the warp's ring; tokens past the body repeat its last one
  auto issue = [&](int s, int i) {
    if (s < n_stages) {
      const int t0 = s * kStage, last = min(kStage, sl.n_body - t0) - 1;
      const size_t row0 = cache_row(cv, bb, kvh, t0);    // 32 aligned tokens are consecutive rows
      uint8_t *sb = ring + i * kFewWarps * STAGE;
      const uint8_t *kp = cv.payload[0] + row0 * RB;
      constexpr int CPR = RB / 16;
      if (last == kStage - 1) {
        // a whole stage is one run of bytes; where 32 pieces are whole rows, every address is a constant
        // away from the lane's first
        const uint8_t *src = kp + 16 * lane;
        const uint32_t dst = smem_addr(sb + (lane / CPR) * PITCH + 16 * (lane % CPR));
#pragma unroll
        for (int k = 0; k < CPR; ++k) {
          if constexpr (32 % CPR == 0) {
            cp_async16(dst + k * (32 / CPR) * PITCH, src + 512 * k, 16);
          } else {
            const int q = lane + 32 * k;
            cp_async16(smem_addr(sb + (q / CPR) * PITCH + 16 * (q % CPR)), src + 512 * k, 16);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < CPR; ++k) {
          const int q = lane + 32 * k, row = q / CPR, j = q % CPR;
          cp_async16(smem_addr(sb + row * PITCH + 16 * j), kp + (size_t)min(row, last) * RB + 16 * j, 16);
        }
      }
      const uint8_t *sp = static_cast<const uint8_t *>(cv.scale[0]) + (row0 + min(lane, last)) * SB;
      if constexpr (SB == 16) cp_async16(smem_addr(sb + OFF_S + lane * SB), sp, 16);
      else cp_async_scale<SB>(smem_addr(sb + OFF_S + lane * SB), sp, SB);
      if constexpr (KL == KVQ_ASYM4_G32) {
        const uint8_t *zp = reinterpret_cast<const uint8_t *>(cv.zero[0]) + (row0 + min(lane, last)) * SB;
        if constexpr (SB == 16) cp_async16(smem_addr(sb + OFF_Z + lane * SB), zp, 16);
        else cp_async_scale<SB>(smem_addr(sb + OFF_Z + lane * SB), zp, SB);
      }
    }
    cp_async_commit();                                   // always one group per call
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) issue(s_first + i * step, i);

  // the query rows: operand fragments to registers by way of shared memory
  uint8_t *qmem = smem + (kRing - 1) * kFewWarps * STAGE;
  uint4 *frag = reinterpret_cast<uint4 *>(qmem);
  float *qsum = reinterpret_cast<float *>(qmem + 8 * D * 2 * (SPLIT ? 2 : 1)), *alpha = qsum + 8 * NB;
  float *lse2 = alpha + 8;
  int *limit = reinterpret_cast<int *>(lse2 + 8);
  float *buf = lse2 + 16 + warp * D;
  for (int r = warp; r < 8; r += kFewWarps) prepare_row<KL, D, SPLIT>(a, bb, kvh, r, r, lane, buf, frag, NB * 32, qsum, alpha);
  asm volatile("griddepcontrol.wait;" ::: "memory");     // the rows' log-sum-exp come from phase 2
  if (threadIdx.x < 8) row_result(a, sl, bb, kvh, threadIdx.x, lse2[threadIdx.x], limit[threadIdx.x]);
  __syncthreads();
  uint4 B[(SPLIT ? 2 : 1) * NB];
#pragma unroll
  for (int b = 0; b < (SPLIT ? 2 : 1) * NB; ++b) B[b] = frag[b * 32 + lane];
  const float2 ls = *reinterpret_cast<const float2 *>(lse2 + 2 * c);
  float2 al = *reinterpret_cast<const float2 *>(alpha + 2 * c);
  if (ls.x == INFINITY) al.x = 0.0f;                      // a row that sees nothing may hold any score
  if (ls.y == INFINITY) al.y = 0.0f;
  const int2 lim = *reinterpret_cast<const int2 *>(limit + 2 * c);
  constexpr bool TERMS = is_hadamard(KL) || KL == KVQ_ASYM4_G32;
  float q0[NB], q1[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    q0[b] = TERMS ? qsum[2 * c * NB + b] : 0.0f;
    q1[b] = TERMS ? qsum[(2 * c + 1) * NB + b] : 0.0f;
  }
  __syncthreads();                                       // the last slots may be filled
  const int min_lim = row_limit(a, sl, 0);                // limits grow with the query index
  const float *in = wa.scores_in ? wa.scores_in + (size_t)bh * wa.stride : nullptr;
  float *out = wa.scores_out + (size_t)bh * wa.stride;
  auto get = [&](int b) { return B[b]; };

  int slot = 0;
  for (int s = s_first; s < n_stages; s += step) {
    const int t0 = s * kStage, t = t0 + lane / 4 + 8 * c;
    const float old = in && t < sl.n_body ? in[t] : 0.0f;
    issue(s + (kRing - 1) * step, slot == 0 ? kRing - 1 : slot - 1);
    cp_async_wait<kRing - 1>();
    __syncwarp();
    const uint8_t *sb = ring + slot * kFewWarps * STAGE;
    float w[4];
    const bool masked = t0 + kStage - 1 > min_lim;
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      Tile<KL, D> tl;
      load_stage_tile<KL, D>(sb, 16 * tile, lane, tl);
      float sum[2] = {0.f, 0.f};
      add_rows<KL, D, SPLIT>(tl, get, al, ls, lim, q0, q1, t0 + 16 * tile, masked, g, sum);
      w[2 * tile] = sum[0];
      w[2 * tile + 1] = sum[1];
    }
    __syncwarp();                                        // the slot is free for the next issue
    const float v = quad_total(w, c);
    if (t < sl.n_body) out[t] = in ? fmaf(wa.decay, old, v) : v;
    slot = slot + 1 == kRing ? 0 : slot + 1;
  }
  asm volatile("cp.async.wait_group 0;\n" ::: "memory");
}

// More than eight query rows, head_dim 256. A CTA takes `units` groups of 32 tokens, dealt to its warps in turn.
// PASSES: more rows than shared memory holds at a time; a warp then keeps the sums of its kManyUnits units
// across the passes (and reads their packed rows again from the cache).
constexpr int kManyUnits = 4;
template <int KL, bool SPLIT, bool PASSES>
__global__ void __launch_bounds__(32 * kManyWarps, 2) attend_weights_many_kernel(WeightArgs wa) {
  constexpr int D = 256, NB = D / 32, ROWS = kPassRows;
  extern __shared__ __align__(16) uint8_t smem[];
  const AttendArgs &a = wa.a;
  const CacheView &cv = a.cache;
  const int bh = blockIdx.y, bb = bh / cv.H, kvh = bh - bb * cv.H;
  const SeqLen sl = seq_of(a, bb);
  if (is_hadamard(KL) && (int)blockIdx.x >= wa.n_ctas) {
    const int j = (int)blockIdx.x - wa.n_ctas;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (sl.n_body + j * kWinTokens < sl.kv_len)
      window_tokens<D, kManyWarps>(wa, sl, bb, kvh, j, reinterpret_cast<float *>(smem));
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int n_units = (sl.n_body + kStage - 1) / kStage, first = (int)blockIdx.x * wa.units;
  const int mine = min(n_units - first, wa.units);
  if (mine <= 0) {
    if (blockIdx.x == 0 && blockIdx.y == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int rows = a.gqa * a.n_q;
  uint4 *frag = reinterpret_cast<uint4 *>(smem);
  float *qsum = reinterpret_cast<float *>(smem + ROWS * D * 2 * (SPLIT ? 2 : 1));
  RowParams p;
  p.alpha = qsum + ROWS * NB;
  p.lse2 = p.alpha + ROWS;
  p.limit = reinterpret_cast<int *>(p.lse2 + ROWS);
  float *buf = p.lse2 + 2 * ROWS + warp * D;
  const int min_lim = row_limit(a, sl, 0);                // limits grow with the query index
  const int t_last = sl.n_body - 1;
  float keep[PASSES ? kManyUnits : 1][4] = {};
  const float *in = wa.scores_in ? wa.scores_in + (size_t)bh * wa.stride : nullptr;
  float *out = wa.scores_out + (size_t)bh * wa.stride;
  auto write = [&](int u, float (&w)[4]) {
    const int t = (first + u) * kStage + g + 8 * c;
    const float v = quad_total(w, c);
    if (t < sl.n_body) out[t] = in ? fmaf(wa.decay, in[t], v) : v;
  };
  for (int r0 = 0; r0 < rows; r0 += ROWS) {
    const int n_tiles = (min(rows - r0, ROWS) + 7) / 8;
    if (PASSES && r0 > 0) __syncthreads();
    for (int s = warp; s < 8 * n_tiles; s += kManyWarps)
      prepare_row<KL, D, SPLIT>(a, bb, kvh, r0 + s, s, lane, buf, frag, ROWS / 8 * NB * 32, qsum, p.alpha);
    if (r0 == 0) asm volatile("griddepcontrol.wait;" ::: "memory");   // the rows' log-sum-exp come from phase 2
    __syncthreads();
    for (int s = threadIdx.x; s < 8 * n_tiles; s += 32 * kManyWarps) {
      row_result(a, sl, bb, kvh, r0 + s, p.lse2[s], p.limit[s]);
      if (p.lse2[s] == INFINITY) p.alpha[s] = 0.0f;       // a row that sees nothing may hold any score
    }
    __syncthreads();
#pragma unroll 1
    for (int i = 0, u = warp; u < mine; ++i, u += kManyWarps) {
      const int t0 = (first + u) * kStage;
      float w[4] = {0.f, 0.f, 0.f, 0.f};
      const bool masked = t0 + kStage - 1 > min_lim;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {              // the fragments of 16 tokens fit the registers
        Tile<KL, D> tl;
        // a unit's second tile may lie behind the body: it then repeats the last token of the first
        const int tt = t0 + 16 * half;
        load_global_tile<KL, D>(cv, bb, kvh, tt <= t_last ? tt : t0, t_last, g, c, tl);
        float sum[2] = {};
#pragma unroll 1
        for (int nt = 0; nt < n_tiles; ++nt) {
          const uint4 *f = frag + nt * NB * 32 + lane;
          const float2 al = *reinterpret_cast<const float2 *>(p.alpha + 8 * nt + 2 * c);
          const float2 ls = *reinterpret_cast<const float2 *>(p.lse2 + 8 * nt + 2 * c);
          int2 lim = make_int2(0, 0);
          if (masked) lim = *reinterpret_cast<const int2 *>(p.limit + 8 * nt + 2 * c);
          const float *q0 = qsum + (8 * nt + 2 * c) * NB;
          auto get = [&](int b) { return b < NB ? f[b * 32] : f[(ROWS / 8 * NB + b - NB) * 32]; };
          add_rows<KL, D, SPLIT>(tl, get, al, ls, lim, q0, q0 + NB, tt, masked, g, sum);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          w[k] = half == 0 ? sum[k] : w[k];
          w[2 + k] = half == 1 ? sum[k] : w[2 + k];
        }
      }
      if constexpr (PASSES) {
#pragma unroll
        for (int k = 0; k < kManyUnits; ++k)
          if (k == i)
#pragma unroll
            for (int j = 0; j < 4; ++j) keep[k][j] += w[j];
      } else {
        write(u, w);
      }
    }
  }
  if constexpr (PASSES) {
#pragma unroll
    for (int k = 0; k < kManyUnits; ++k)
      if (warp + k * kManyWarps < mine) write(warp + k * kManyWarps, keep[k]);
  }
}

int device_sms() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <int KL, int D, class K>
cudaError_t launch_one(K *kernel, WeightArgs &wa, int warps, int smem, std::atomic<bool> (&done)[kMaxDevices], cudaStream_t st) {
  cudaError_t e = set_smem_once(done, kernel, smem);
  if (e != cudaSuccess) return e;
  const int n_win = is_hadamard(KL) ? (wa.a.n_win + kWinTokens - 1) / kWinTokens : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(wa.n_ctas + n_win), (unsigned)(wa.a.cache.B * wa.a.cache.H));
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, wa);
}

// Resident CTAs of a kernel per SM on the current device, asked once.
template <class K>
int resident_ctas(K *kernel, int threads, int smem, std::atomic<int> (&known)[kMaxDevices]) {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 1;
  n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n < 1) n = 1;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

template <int KL, int D, bool SPLIT>
cudaError_t launch_few(WeightArgs &wa, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  static std::atomic<int> known[kMaxDevices];
  constexpr int stages = kFewWarps * kRing * stage_bytes<KL, D>();
  constexpr int smem = is_hadamard(KL) ? max_of(stages, window_smem<D, kFewWarps>()) : stages;
  // one wave of resident CTAs over all (batch, kv head); sequences of their own lengths are cut finer (at
  // most eight stages per warp), so that the long ones do not end alone
  cudaError_t e = set_smem_once(done, attend_weights_few_kernel<KL, D, SPLIT>, smem);
  if (e != cudaSuccess) return e;
  const int per_sm = resident_ctas(attend_weights_few_kernel<KL, D, SPLIT>, 32 * kFewWarps, smem, known);
  const int heads = wa.a.cache.B * wa.a.cache.H, n_stages = (wa.a.n_body + kStage - 1) / kStage;
  const int wave = max(1, device_sms() * per_sm / heads);
  const int most = (n_stages + kFewWarps - 1) / kFewWarps;
  wa.n_ctas = min(wa.a.seq_lens ? max(wave, (most + 7) / 8) : wave, most);
  return launch_one<KL, D>(attend_weights_few_kernel<KL, D, SPLIT>, wa, kFewWarps, smem, done, st);
}

template <int RP, int D, bool HAD>
cudaError_t launch_scores(WeightArgs &wa, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  constexpr int smem = HAD ? window_smem<D, kScoreThreads / 32>() : 0;
  wa.n_ctas = (wa.a.n_body + kScoreTokens - 1) / kScoreTokens;
  return launch_one<HAD ? KVQ_HAD_INT4 : KVQ_Q4_0, D>(attend_weights_scores_kernel<RP, D, HAD>, wa, kScoreThreads / 32, smem, done, st);
}
template <int D, bool HAD>
cudaError_t launch_scores_rows(WeightArgs &wa, cudaStream_t st) {
  if (wa.a.s_rows == 2) return launch_scores<2, D, HAD>(wa, st);
  return wa.a.s_rows == 4 ? launch_scores<4, D, HAD>(wa, st) : launch_scores<8, D, HAD>(wa, st);
}

template <int KL, bool SPLIT, bool PASSES>
cudaError_t launch_many(WeightArgs &wa, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  constexpr int D = 256, rows = rows_smem<D, SPLIT, kPassRows, kManyWarps>();
  constexpr int smem = is_hadamard(KL) ? max_of(rows, window_smem<D, kManyWarps>()) : rows;
  // two CTAs per SM: the units of a head shared out over one wave (a warp keeps at most kManyUnits
  // across passes)
  const int heads = wa.a.cache.B * wa.a.cache.H, n_units = (wa.a.n_body + kStage - 1) / kStage;
  const int wave = max(1, device_sms() * 2 / heads);
  wa.units = (n_units + wave - 1) / wave;
  wa.units = (wa.units + kManyWarps - 1) / kManyWarps * kManyWarps;
  if (PASSES) wa.units = min(wa.units, kManyUnits * kManyWarps);
  wa.units = max(wa.units, kManyWarps);
  wa.n_ctas = (n_units + wa.units - 1) / wa.units;
  return launch_one<KL, D>(attend_weights_many_kernel<KL, SPLIT, PASSES>, wa, kManyWarps, smem, done, st);
}

template <int KL, int D, bool SPLIT>
cudaError_t launch_rows(WeightArgs &wa, cudaStream_t st) {
  const int rows = wa.a.gqa * wa.a.n_q;
  if (rows <= 8) return launch_few<KL, D, SPLIT>(wa, st);
  if constexpr (D == 128) return launch_attend_weights_tc(wa, st);
  else return rows <= kPassRows ? launch_many<KL, SPLIT, false>(wa, st) : launch_many<KL, SPLIT, true>(wa, st);
}

template <int KL, int D>
cudaError_t launch_layout(WeightArgs &wa, cudaStream_t st) {
  if constexpr (!is_hadamard(KL))
    if (wa.a.q_dtype == KVQ_F32) return launch_rows<KL, D, true>(wa, st);
  return launch_rows<KL, D, false>(wa, st);
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
  wa.units = 0;
  // the lengths were there before phase 1 of this call began: reading them needs no wait for phase 2
  wa.a.fresh_tail = 1;
  if (a.part_s) {
    if (is_hadamard(a.cache.layout)) return launch_scores_rows<128, true>(wa, st);
    return a.cache.D == 128 ? launch_scores_rows<128, false>(wa, st) : launch_scores_rows<256, false>(wa, st);
  }
  return a.cache.D == 128 ? launch_dim<128>(wa, st) : launch_dim<256>(wa, st);
}

}  // namespace kvq
