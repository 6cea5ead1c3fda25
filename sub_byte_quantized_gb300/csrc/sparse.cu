// Attention over blocks of 64 tokens that a cheap score selects for each query.
//
// Bounds, per block, kv head and channel: lo_d = min_t k_td and hi_d = max_t k_td over the block's tokens (the values the
// packed rows stand for; Hadamard layouts: in the rotated basis), in int8 by one scale per block, s = max(|lo|, |hi|) / 127:
// floor(lo / s) and ceil(hi / s), so that the bounds stay bounds.
// Score of a block for one query row: sum_d max(q8_d lo_d, q8_d hi_d) s_q s, with the row in int8 (s_q = amax / 127), which
// no q8 . k of the block exceeds but by rounding (each division before its floor or ceil, and at 127 the scale's own). q8 >= 0 takes hi and q8 < 0 takes lo, so with q+ = max(q8, 0) and q- = min(q8, 0) it is
// q+ . hi + q- . lo: dp4a, exact integers (below 2^24), then two rounded products: the same bits whatever the order. The
// query heads of a kv head read one cache, so they share a list: the largest of their scores counts.
// Lists: the blocks with the highest scores, by the radix selection that the budget's calls use, whose kernel scores them too.
// Attention: each (query, kv head) is a sequence of its own of one kv head, whose table names the selected blocks in the
// same pool: a page of one head is a contiguous run of rows, so a pool [n_pages][H][page] is a pool of n_pages * H * page / 64
// pages of one head and 64 tokens, and a contiguous cache [B][H][cap] one of B * H * cap / 64. The attention kernels read it
// as it is.
//
// Bound: the bounds pass by the packed keys' bytes (a decode step renews one block per head: latency); scores and selection
// by latency; the attention by the selected rows' bytes, a few of them by latency too.
// Bounds of 128K tokens of 8 kv heads in Q4_0: 46 us, bound by their instructions (issue 65 %, DRAM 21 %); with the selection 57.5.
#include <cuda_fp8.h>

#include "kvq_internal.cuh"

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

// Codes of 32 consecutive channels of a row, as they were read and as floats (value = code * scale [+ zero]). Integer fields
// become floats under the exponent of 2^23 (and an addition that takes the offset away): the conversion instructions run at a
// quarter of the rate.
template <int LAYOUT>
struct Raw32 {
  static constexpr int WORDS = LAYOUT == KVQ_HAD_INT2 ? 2 : LAYOUT == KVQ_Q6_0 ? 6 : LAYOUT == KVQ_Q8_0 || is_b64(LAYOUT) ? 8 : 4;
  uint32_t w[WORDS];
  float scale, zero;
  __device__ __forceinline__ void load(const CacheView &c, size_t row, int blk) {
    const uint8_t *p = c.payload[0] + row * (size_t)c.row_bytes + blk * 4 * WORDS;
    if constexpr (WORDS % 4 == 0) {
#pragma unroll
      for (int i = 0; i < WORDS; i += 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i / 4);
        w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < WORDS; i += 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p) + i / 2);
        w[i] = v.x; w[i + 1] = v.y;
      }
    }
    if constexpr (is_b64(LAYOUT)) scale = 1.0f;          // one scale per block: it joins the bounds
    else if constexpr (is_hadamard(LAYOUT)) scale = __ldg(static_cast<const float *>(c.scale[0]) + row);
    else scale = __half2float(static_cast<const __half *>(c.scale[0])[row * (c.D / kBlock) + blk]);
    zero = LAYOUT == KVQ_ASYM4_G32 ? __half2float(c.zero[0][row * (c.D / kBlock) + blk]) : 0.0f;
  }
  static __device__ __forceinline__ float offset_code(uint32_t u, float offset) {   // u < 2^23
    return __uint_as_float(0x4B000000u | u) - (8388608.0f + offset);
  }
  __device__ __forceinline__ float value(int i) const {
    float x;
    if constexpr (LAYOUT == KVQ_Q4_0 || LAYOUT == KVQ_ASYM4_G32) {
      // The field stays where it is: code 2^p under 2^23, and the scale is divided by 2^p (f16 scales: exact).
      const int p = 4 * (i & 3);
      const uint32_t word = (i & 4) ? w[i >> 3] >> 16 : w[i >> 3], flip = LAYOUT == KVQ_Q4_0 ? 8u << p : 0u;
      x = __uint_as_float((word & (0xFu << p)) ^ (0x4B000000u | flip)) - (8388608.0f + (float)flip);
      const float s = scale * (1.0f / (float)(1 << p));
      return LAYOUT == KVQ_Q4_0 ? __fmul_rn(x, s) : fmaf(x, s, zero);
    } else if constexpr (LAYOUT == KVQ_HAD_INT4) {
      x = offset_code(((w[i >> 3] >> (4 * (i & 7))) & 0xFu) ^ 8u, 8.0f);
    } else if constexpr (LAYOUT == KVQ_HAD_INT2) {
      x = offset_code(((w[i >> 4] >> (2 * (i & 15))) & 3u) ^ 2u, 2.0f);
    } else if constexpr (LAYOUT == KVQ_Q6_0) {
      x = offset_code((((w[i >> 3] >> (4 * (i & 7))) & 0xFu) | (((w[4 + (i >> 4)] >> (2 * (i & 15))) & 3u) << 4)) ^ 32u, 32.0f);
    } else if constexpr (LAYOUT == KVQ_E4M3_B64) {
      const uint32_t two = (w[i >> 2] >> (16 * ((i >> 1) & 1))) & 0xFFFFu;
      const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3)));
      return (i & 1) ? f.y : f.x;
    } else {
      x = offset_code(((w[i >> 2] >> (8 * (i & 3))) & 0xFFu) ^ 0x80u, 128.0f);
    }
    return is_b64(LAYOUT) ? x : __fmul_rn(x, scale);
  }
};

// One warp per (block, head): lane = (token lane, 32 channels); each passes over its tokens, then the token lanes halve their
// channels with each other until every lane has the bounds of a few.
template <int LAYOUT, int D>
__global__ void __launch_bounds__(kThreads) block_bounds_kernel(BoundsArgs a) {
  constexpr int PARTS = D / 32, TL = 32 / PARTS, EACH = 64 / TL, OWN = 32 / TL;   // token lanes, tokens each, channels in the end
  const CacheView &c = a.cache;
  const int b = blockIdx.y / c.H, h = blockIdx.y - b * c.H, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int end = clamped_len(a.seq_lens, b, a.kv_len), first = a.seq_lens ? max(end - a.n_fresh, 0) : a.first;
  const long long blk64 = (long long)(first >> 6) + (long long)blockIdx.x * kWarps + warp;
  if (first >= end || blk64 * 64 >= end) return;         // whole warps
  const int blk = (int)blk64, part = lane % PARTS, tl = lane / PARTS, n = min(64, end - 64 * blk);
  const size_t row0 = cache_row(c, b, h, 64 * blk);
  float lo[32], hi[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) lo[i] = INFINITY, hi[i] = -INFINITY;
  constexpr int AT_ONCE = Raw32<LAYOUT>::WORDS > 4 ? 2 : 4;
#pragma unroll 1
  for (int j0 = 0; j0 < EACH; j0 += AT_ONCE) {
    Raw32<LAYOUT> raw[AT_ONCE];
    // tokens behind the end read the block's first row again: what they bring is there already
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      const int t = tl + (j0 + j) * TL;
      raw[j].load(c, row0 + (t < n ? t : 0), part);
    }
#pragma unroll
    for (int i = 0; i < 32; ++i)
#pragma unroll
      for (int j = 0; j < AT_ONCE; j += 2) {
        const float x = raw[j].value(i), y = raw[j + 1].value(i);
        lo[i] = fminf(fminf(lo[i], x), y);
        hi[i] = fmaxf(fmaxf(hi[i], x), y);
      }
  }
  int mine = 32 * part;                                  // the first channel of the lane's
#pragma unroll
  for (int half = 16, m = 16; half >= OWN; half >>= 1, m >>= 1) {
    const bool up = lane & m;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float l = __shfl_xor_sync(0xffffffffu, up ? lo[i] : lo[i + half], m);
      const float g = __shfl_xor_sync(0xffffffffu, up ? hi[i] : hi[i + half], m);
      lo[i] = fminf(up ? lo[i + half] : lo[i], l);
      hi[i] = fmaxf(up ? hi[i + half] : hi[i], g);
    }
    if (up) mine += half;
  }
  const float each = is_b64(LAYOUT) ? __ldg(static_cast<const float *>(c.scale[0]) + (row0 >> 6)) : 1.0f;
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < OWN; ++i) {
    if (is_b64(LAYOUT)) {                                // (a rounded product keeps the order)
      lo[i] = __fmul_rn(lo[i], each);
      hi[i] = __fmul_rn(hi[i], each);
    }
    top = fmaxf(top, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
  const float s = __fdiv_rn(top, 127.0f);
  const size_t at = row0 >> 6;
  if (lane == 0) a.scale[at] = s;
  uint32_t code[2][OWN / 4];
#pragma unroll
  for (int i = 0; i < OWN; ++i) {
    const float l = s > 0.0f ? floorf(__fdiv_rn(lo[i], s)) : 0.0f, g = s > 0.0f ? ceilf(__fdiv_rn(hi[i], s)) : 0.0f;
    const uint32_t cl = (uint32_t)(int)fminf(fmaxf(l, -127.0f), 127.0f) & 0xFFu, cg = (uint32_t)(int)fminf(fmaxf(g, -127.0f), 127.0f) & 0xFFu;
    code[0][i >> 2] = (i & 3) ? code[0][i >> 2] | cl << (8 * (i & 3)) : cl;
    code[1][i >> 2] = (i & 3) ? code[1][i >> 2] | cg << (8 * (i & 3)) : cg;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < OWN / 4; ++i) *reinterpret_cast<uint32_t *>(a.codes + (at * 2 + k) * D + mine + 4 * i) = code[k][i];
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
  const dim3 grid((unsigned)((blocks + kWarps - 1) / kWarps), (unsigned)(a.cache.B * a.cache.H));
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
