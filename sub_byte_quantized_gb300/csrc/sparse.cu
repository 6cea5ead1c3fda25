// Attention over blocks of 64 tokens that a cheap score selects for each query.
//
// Bounds, per block, kv head and channel: lo_d = min_t k_td and hi_d = max_t k_td over the block's tokens (the values the
// packed rows stand for; Hadamard layouts: in the rotated basis), in int8 by one scale per block, s = max(|lo|, |hi|) / 127:
// floor(lo / s) and ceil(hi / s), so that the bounds stay bounds.
// Score of a block for one query row: sum_d max(q8_d lo_d, q8_d hi_d) s_q s, with the row in int8 (s_q = amax / 127), which
// no q8 . k of the block exceeds. q8 >= 0 takes hi and q8 < 0 takes lo, so with q+ = max(q8, 0) and q- = min(q8, 0) it is
// q+ . hi + q- . lo: dp4a, exact integers (below 2^24), then two rounded products: the same bits whatever the order. The
// query heads of a kv head read one cache, so they share a list: the largest of their scores counts.
// Lists: the blocks with the highest scores, by the radix selection that the budget's calls use.
// Attention: each (query, kv head) is a sequence of its own of one kv head, whose table names the selected blocks in the
// same pool: a page of one head is a contiguous run of rows, so a pool [n_pages][H][page] is a pool of n_pages * H * page / 64
// pages of one head and 64 tokens, and a contiguous cache [B][H][cap] one of B * H * cap / 64. The attention kernels read it
// as it is.
//
// Bound: the bounds pass by the packed keys' bytes (a decode step renews one block per head: latency); scores and selection
// by latency; the attention by the selected rows' bytes, a few of them by latency too.
#include "kvq_internal.cuh"
#include "unpack.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// Block index (in the plane of bounds or scales) of block `blk` of (b, h).
__device__ __forceinline__ size_t block_index(const CacheView &c, int b, int h, int blk) {
  return cache_row(c, b, h, blk << 6) >> 6;
}
__device__ __forceinline__ int clamped_len(const int32_t *seq_lens, int b, int kv_len) {
  return seq_lens ? min(max(__ldg(seq_lens + b), 0), kv_len) : kv_len;
}

// One CTA per (block, head): threads hold 8 channels each and split the tokens.
template <int LAYOUT, int D>
__global__ void __launch_bounds__(kThreads) block_bounds_kernel(BoundsArgs a) {
  constexpr int GROUPS = D / 8, LANES = kThreads / GROUPS, LEN = 64 / LANES;   // LANES threads share a channel group
  __shared__ float lo_s[kWarps][D], hi_s[kWarps][D], top_s[kWarps];
  const CacheView &c = a.cache;
  const int b = blockIdx.y / c.H, h = blockIdx.y - b * c.H, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int end = clamped_len(a.seq_lens, b, a.kv_len), first = a.seq_lens ? max(end - a.n_fresh, 0) : a.first;
  const int blk = (first >> 6) + blockIdx.x;
  if (first >= end || (blk << 6) >= end) return;
  const int gi = tid % GROUPS, t0 = (blk << 6) + tid / GROUPS;
  const size_t row0 = cache_row(c, b, h, blk << 6);
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) lo[i] = INFINITY, hi[i] = -INFINITY;
#pragma unroll
  for (int j = 0; j < LEN; ++j) {
    const int t = t0 + j * LANES;
    if (t < end) {
      const size_t row = row0 + (t & 63);
      float x[8];
      unpack8(LAYOUT, c, 0, row, gi, x);
      const float s = is_b64(LAYOUT) ? static_cast<const float *>(c.scale[0])[row >> 6]
                      : is_hadamard(LAYOUT) ? static_cast<const float *>(c.scale[0])[row] : 1.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (is_b64(LAYOUT) || is_hadamard(LAYOUT)) x[i] = __fmul_rn(x[i], s);
        lo[i] = fminf(lo[i], x[i]);
        hi[i] = fmaxf(hi[i], x[i]);
      }
    }
  }
  if constexpr (GROUPS == 16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = fminf(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], 16));
      hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], 16));
    }
  }
  if (lane < GROUPS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo_s[warp][8 * gi + i] = lo[i];
      hi_s[warp][8 * gi + i] = hi[i];
    }
  }
  __syncthreads();
  // thread: D * 2 / 256 bounds, those of dims d = tid % D
  constexpr int OWN = 2 * D / kThreads;
  float v[OWN], top = 0.0f;
#pragma unroll
  for (int k = 0; k < OWN; ++k) {
    const int e = tid + k * kThreads, d = e % D;
    const bool up = e >= D;
    v[k] = up ? hi_s[0][d] : lo_s[0][d];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v[k] = up ? fmaxf(v[k], hi_s[w][d]) : fminf(v[k], lo_s[w][d]);
    top = fmaxf(top, fabsf(v[k]));
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
  if (lane == 0) top_s[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, top_s[w]);
  const float s = __fdiv_rn(top, 127.0f);
  const size_t at = row0 >> 6;
  if (tid == 0) a.scale[at] = s;
#pragma unroll
  for (int k = 0; k < OWN; ++k) {
    const int e = tid + k * kThreads;
    const float x = s > 0.0f ? __fdiv_rn(v[k], s) : 0.0f;
    a.codes[at * 2 * D + e] = (int8_t)fminf(fmaxf(e >= D ? ceilf(x) : floorf(x), -127.0f), 127.0f);
  }
}

// Scores of kTile blocks for one (query, kv head): the heads' rows in int8 in shared memory, four threads per block.
constexpr int kTile = 64;
constexpr int kRows = 8;                                 // query heads at a time
template <int D>
__global__ void __launch_bounds__(kThreads) block_scores_kernel(BlockSelectArgs a) {
  constexpr int V = D / 32;
  __shared__ __align__(16) int8_t q_neg[kRows][D], q_pos[kRows][D];
  __shared__ float q_step[kRows];
  const CacheView &c = a.cache;
  const int vb = blockIdx.y, bh = vb / a.n_q, i = vb - bh * a.n_q, b = bh / c.H, h = bh - b * c.H;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = clamped_len(a.seq_lens, b, a.kv_len);
  const int limit = a.causal ? min(len - 1, (a.seq_lens ? len - a.n_q : a.q_pos0) + i) : len - 1;
  const int n = limit < 0 ? 0 : (limit >> 6) + 1;        // blocks that the row sees
  if (blockIdx.x == 0 && tid == 0) a.counts[vb] = n;
  const int blk = blockIdx.x * kTile + (tid >> 2);
  if (blockIdx.x * kTile >= n || n <= a.n_sel) return;   // (few blocks: all are kept, and no score is read)
  uint4 lo[D / 64], hi[D / 64];                          // the thread's quarter of the block's bounds
  float scale = 0.0f;
  const bool live = blk < n;
  if (live) {
    const size_t at = block_index(c, b, h, blk);
    const uint4 *p = reinterpret_cast<const uint4 *>(a.codes + at * 2 * D) + (tid & 3) * (D / 64);
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      lo[k] = __ldg(p + k);
      hi[k] = __ldg(p + D / 16 + k);
    }
    scale = __ldg(a.scale + at);
  }
  float best = -INFINITY;
  for (int r0 = 0; r0 < a.gqa; r0 += kRows) {
    __syncthreads();
    if (r0 + warp < a.gqa) {
      const size_t row = ((size_t)bh * a.gqa + r0 + warp) * a.n_q + i;
      float x[V];
      int q8[V];
      if (V == 4) load4_f32(a.q, a.q_dtype, row * D + lane * 4, x);
      else load8_f32(a.q, a.q_dtype, row * D + lane * 8, x);
      float s;
      if (a.rotated) {
        s = had_query_row<V>(x, q8, lane);
      } else {
        float top = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) top = fmaxf(top, fabsf(x[k]));
#pragma unroll
        for (int m = 16; m; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        s = __fdiv_rn(top, 127.0f);
#pragma unroll
        for (int k = 0; k < V; ++k) q8[k] = s > 0.0f ? (int)fminf(fmaxf(rintf(__fdiv_rn(x[k], s)), -127.0f), 127.0f) : 0;
      }
#pragma unroll
      for (int k = 0; k < V; ++k) {
        q_neg[warp][lane * V + k] = (int8_t)min(q8[k], 0);
        q_pos[warp][lane * V + k] = (int8_t)max(q8[k], 0);
      }
      if (lane == 0) q_step[warp] = s;
    }
    __syncthreads();
    const int rows = min(kRows, a.gqa - r0);
    for (int r = 0; r < rows; ++r) {
      int dot = 0;
#pragma unroll
      for (int k = 0; k < D / 64; ++k) {
        const uint4 n4 = *reinterpret_cast<const uint4 *>(&q_neg[r][((tid & 3) * (D / 64) + k) * 16]);
        const uint4 p4 = *reinterpret_cast<const uint4 *>(&q_pos[r][((tid & 3) * (D / 64) + k) * 16]);
        if (live) {
          dot = __dp4a((int)n4.x, (int)lo[k].x, dot);
          dot = __dp4a((int)n4.y, (int)lo[k].y, dot);
          dot = __dp4a((int)n4.z, (int)lo[k].z, dot);
          dot = __dp4a((int)n4.w, (int)lo[k].w, dot);
          dot = __dp4a((int)p4.x, (int)hi[k].x, dot);
          dot = __dp4a((int)p4.y, (int)hi[k].y, dot);
          dot = __dp4a((int)p4.z, (int)hi[k].z, dot);
          dot = __dp4a((int)p4.w, (int)hi[k].w, dot);
        }
      }
      dot += __shfl_xor_sync(0xffffffffu, dot, 1);
      dot += __shfl_xor_sync(0xffffffffu, dot, 2);
      best = fmaxf(best, __fmul_rn((float)dot, q_step[r]));
    }
  }
  if (live && (tid & 3) == 0) a.scores[(size_t)vb * a.stride + blk] = __fmul_rn(best, scale);
}

// One warp per list: the selected blocks as pages of one head, and the sequence's length. A list ends at the first
// entry that is not above the one before it or that its row does not see.
__global__ void __launch_bounds__(kThreads) sparse_table_kernel(SparseArgs a) {
  const int vb = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const CacheView &c = a.cache;
  if (vb >= c.B * c.H * a.n_q) return;
  const int bh = vb / a.n_q, i = vb - bh * a.n_q, b = bh / c.H, h = bh - b * c.H;
  const int len = clamped_len(a.seq_lens, b, a.kv_len);
  const int limit = a.causal ? min(len - 1, (a.seq_lens ? len - a.n_q : a.q_pos0) + i) : len - 1;
  const int32_t *sel = a.sel + (size_t)vb * a.n_sel;
  int count = 0, last = -1;
  for (int j0 = 0; j0 < a.n_sel; j0 += 32) {
    const int j = j0 + lane;
    const int e = j < a.n_sel ? __ldg(sel + j) : -1;
    int before = __shfl_up_sync(0xffffffffu, e, 1);
    if (lane == 0) before = last;
    const bool ok = e > before && e >= 0 && e <= (limit >> 6) && limit >= 0;
    const unsigned bad = ~__ballot_sync(0xffffffffu, ok);
    const int n = bad ? __ffs((int)bad) - 1 : 32;
    if (lane < n) a.table[(size_t)vb * a.n_sel + j] = (int)block_index(c, b, h, e);
    if (n > 0) last = __shfl_sync(0xffffffffu, e, n - 1);
    count += n;
    if (n < 32) break;
  }
  if (lane == 0) a.lens[vb] = count > 0 ? 64 * (count - 1) + min(64, limit + 1 - 64 * last) : 0;
}

// q [B][Hq][n_q][D] -> [B * H * n_q][gqa][D], 16 bytes per thread.
__global__ void __launch_bounds__(kThreads) sparse_queries_kernel(SparseArgs a, int per_row, long long total) {
  const long long e = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (e >= total) return;
  const long long row = e / per_row, vb = row / a.gqa, bh = vb / a.n_q;
  const long long src = (bh * a.gqa + (row - vb * a.gqa)) * a.n_q + (vb - bh * a.n_q);
  a.q_out[e] = __ldg(static_cast<const uint4 *>(a.q) + src * per_row + (e - row * per_row));
}

template <int LAYOUT>
cudaError_t launch_bounds_t(const BoundsArgs &a, dim3 grid, cudaStream_t st) {
  if (a.cache.D == 128) block_bounds_kernel<LAYOUT, 128><<<grid, kThreads, 0, st>>>(a);
  else block_bounds_kernel<LAYOUT, 256><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_bounds(const BoundsArgs &a, cudaStream_t st) {
  const long long blocks = a.seq_lens ? ((long long)min(a.n_fresh, a.kv_len) + 62) / 64 + 1 : ((long long)a.kv_len + 63) / 64 - a.first / 64;
  const dim3 grid((unsigned)blocks, (unsigned)(a.cache.B * a.cache.H));
  switch (a.cache.layout) {
    case KVQ_Q4_0: return launch_bounds_t<KVQ_Q4_0>(a, grid, st);
    case KVQ_Q6_0: return launch_bounds_t<KVQ_Q6_0>(a, grid, st);
    case KVQ_Q8_0: return launch_bounds_t<KVQ_Q8_0>(a, grid, st);
    case KVQ_ASYM4_G32: return launch_bounds_t<KVQ_ASYM4_G32>(a, grid, st);
    case KVQ_HAD_INT4: return launch_bounds_t<KVQ_HAD_INT4>(a, grid, st);
    case KVQ_HAD_INT2: return launch_bounds_t<KVQ_HAD_INT2>(a, grid, st);
    case KVQ_INT8_B64: return launch_bounds_t<KVQ_INT8_B64>(a, grid, st);
    default: return launch_bounds_t<KVQ_E4M3_B64>(a, grid, st);
  }
}

cudaError_t launch_block_select(const BlockSelectArgs &a, cudaStream_t st) {
  const int lists = a.cache.B * a.cache.H * a.n_q, blocks = (int)(((long long)a.kv_len + 63) / 64);
  const dim3 grid((unsigned)((blocks + kTile - 1) / kTile), (unsigned)lists);
  if (a.cache.D == 128) block_scores_kernel<128><<<grid, kThreads, 0, st>>>(a);
  else block_scores_kernel<256><<<grid, kThreads, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  SelectArgs s = {lists, 1, blocks, a.n_sel, a.n_sink, a.n_recent, a.stride, a.scores, a.counts, a.sel, nullptr};
  return launch_evict_select(s, st);
}

cudaError_t launch_sparse_prepare(const SparseArgs &a, cudaStream_t st) {
  const int lists = a.cache.B * a.cache.H * a.n_q;
  if (a.n_q > 1) {                                       // (a kernel of its own: what follows the table's may read q before that has ended)
    const int per_row = a.cache.D * (a.q_dtype == KVQ_F32 ? 4 : 2) / 16;
    const long long total = (long long)lists * a.gqa * per_row;
    sparse_queries_kernel<<<(unsigned)((total + kThreads - 1) / kThreads), kThreads, 0, st>>>(a, per_row, total);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  sparse_table_kernel<<<(unsigned)((lists + kWarps - 1) / kWarps), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
