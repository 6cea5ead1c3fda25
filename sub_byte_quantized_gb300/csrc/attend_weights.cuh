// Shared by the kernels that turn attention scores into per-token weights: what phase 2 left for a query
// row, and the exact-f32 window's tokens.
#pragma once

#include "kvq_internal.cuh"
#include "mma_util.cuh"

namespace kvq {
namespace weights {
using namespace mma;

constexpr int kWinTokens = 32;           // window tokens per CTA
constexpr float kLog2e = 1.4426950408889634f;
__host__ __device__ constexpr int max_of(int a, int b) { return a > b ? a : b; }

// Window CTA: keys, ROWS query rows (two or four per warp), partial sums, lse and limits.
template <int D, int WARPS, int ROWS = 2 * WARPS>
__host__ __device__ constexpr int window_smem() { return (kWinTokens * (D + 4) + ROWS * D + WARPS * kWinTokens + 2 * ROWS) * 4; }

// What the attention's second phase left for query row r; rows past the last and rows that see nothing add nothing.
// NaN (a phase 1 whose wait gave up) goes on into the weights of the tokens the row sees.
__device__ __forceinline__ void row_result(const AttendArgs &a, const SeqLen &sl, int bb, int kvh, int r, float &lse2, int &limit) {
  const bool live = r < a.gqa * a.n_q;
  const float lse = live ? a.lse[query_row_index(a, bb, kvh, r)] : -INFINITY;
  lse2 = lse == -INFINITY ? INFINITY : lse * kLog2e;
  limit = lse == -INFINITY ? -1 : row_limit(a, sl, r % a.n_q);
}

// Window tokens [n_body + 32 j, ..) of one kv head: lanes are tokens, warps are query rows (PW of them at a
// time). The rotated f32 rows come from the attention's query preparation where its kernel leaves them in the
// workspace, and are formed here otherwise.
template <int D, int kWarps, int ROWS = 2 * kWarps>
__device__ __forceinline__ void window_tokens(const WeightArgs &wa, const SeqLen &sl, int bb, int kvh, int j, float *sm) {
  const AttendArgs &a = wa.a;
  constexpr int kThreads = 32 * kWarps, PW = ROWS / kWarps;
  constexpr int V = D / 32, KST = D + 4;                  // row stride: 16-byte reads of 8 rows hit all banks
  float *ks = sm, *qs = ks + kWinTokens * KST, *part = qs + ROWS * D, *lse2 = part + kWarps * kWinTokens;
  int *lim = reinterpret_cast<int *>(lse2 + ROWS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rows = a.gqa * a.n_q;
  const int t0 = sl.n_body + j * kWinTokens, n = min(kWinTokens, sl.kv_len - t0);
  const size_t head = (size_t)bb * a.cache.H + kvh;
  const float *ring = a.cache.ring[0] + head * a.cache.n_recent * D;
  const bool ready = tc_prefill_shape(a.cache.layout, a.cache.v_layout, D, rows);
  for (int i = threadIdx.x; i < kWinTokens * (D / 4); i += kThreads) {
    const int t = i / (D / 4), d = i % (D / 4) * 4;
    cp_async16(smem_addr(ks + t * KST + d), ring + (size_t)((t0 + min(t, n - 1)) % a.cache.n_recent) * D + d, 16);
  }
  float w = 0.0f;
  for (int r0 = 0; r0 < rows; r0 += ROWS) {
    __syncthreads();                                     // the last pass's rows are read
    if (ready) {
      for (int i = threadIdx.x; i < ROWS * (D / 4); i += kThreads) {
        const int s = i / (D / 4), d = i % (D / 4) * 4;
        cp_async16(smem_addr(qs + s * D + d), a.q_rot + query_row_index(a, bb, kvh, min(r0 + s, rows - 1)) * D + d, 16);
      }
    } else {
#pragma unroll
      for (int u = 0; u < PW; ++u) {
        const int s = u * kWarps + warp, r = r0 + s;
        float x[V];
        int q8[V];
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = 0.0f;
        if (r < rows) {
          if constexpr (V == 4) load4_f32(a.q, a.q_dtype, query_row_index(a, bb, kvh, r) * D + lane * V, x);
          else load8_f32(a.q, a.q_dtype, query_row_index(a, bb, kvh, r) * D + lane * V, x);
        }
        had_query_row<V>(x, q8, lane);                    // x: the rotated f32 row
#pragma unroll
        for (int i = 0; i < V; ++i) qs[s * D + lane * V + i] = x[i];
      }
    }
    for (int s = threadIdx.x; s < ROWS; s += kThreads) row_result(a, sl, bb, kvh, r0 + s, lse2[s], lim[s]);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    const float *q = qs + PW * warp * D;
    float d[PW] = {};
#pragma unroll 4
    for (int i = 0; i < D; i += 4) {
      const float4 k = *reinterpret_cast<const float4 *>(ks + lane * KST + i);
#pragma unroll
      for (int u = 0; u < PW; ++u) {
        const float4 x = *reinterpret_cast<const float4 *>(q + u * D + i);
        d[u] = fmaf(x.x, k.x, fmaf(x.y, k.y, fmaf(x.z, k.z, fmaf(x.w, k.w, d[u]))));
      }
    }
    const float f = a.scale * kLog2e;
#pragma unroll
    for (int u = 0; u < PW; ++u) {
      const int s = PW * warp + u;
      if (t0 + lane <= lim[s]) w += ex2(fmaf(d[u], f, -lse2[s]));
    }
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

}  // namespace weights

// More than eight query rows per kv head, head_dim 128, on the fifth-generation tensor cores.
cudaError_t launch_attend_weights_tc(WeightArgs &wa, cudaStream_t st);

}  // namespace kvq
