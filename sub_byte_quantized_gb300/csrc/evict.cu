// Keeping a cache inside a budget: which tokens stay (selection by running attention weight), and
// moving their packed rows together (compaction).
//
// Selection, per (batch, kv head): of L tokens the first n_sink and the last n_recent stay; among the
// others the k with the highest scores, ties going to the lowest index. That set is {score > T} and the
// first few of {score == T}, T being the k-th highest score: a radix selection over order-preserving
// 32-bit keys finds T in three digits (11, 11 and 10 bits), then one ordered pass writes the list in
// ascending order. One cluster works on one (batch, kv head): every CTA keeps its slice of the keys in
// shared memory, so the scores are read from memory once; the digits' histograms and the slices' counts
// are summed over distributed shared memory. Bound by latency (load, three histogram rounds, the
// ordered pass), not by its bytes.
//
// Compaction: row keep[i] of every plane moves to row i. keep ascends, so keep[i] >= i: a round reads
// the sources of the next block of target rows, everyone waits until all of the cluster's reads have
// arrived, then writes. Reads of later rounds lie behind what this round writes, so they are issued
// before the wait and stay in flight across it. One cluster per (batch, kv head, plane); into another
// cache nothing can be overwritten too early, and the rounds need no barrier. Bound by memory.
#include <cooperative_groups.h>

#include "kvq_internal.cuh"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------------------------ selection
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kSelFixed = (3 * kBins + 2 * kSelWarps + 8) * 4;      // histograms, per-warp counts, results
constexpr int kSelMaxKeys = (227 * 1024 - kSelFixed) / 4 / 4 * 4;   // keys one CTA can hold

// Keys compare like the scores: NaN counts as -infinity, -0 as +0.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// RESIDENT: the slice's keys fit shared memory (else every pass reads the scores again).
template <bool RESIDENT>
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(SelectArgs a) {
  extern __shared__ __align__(16) uint32_t sm[];
  uint32_t *hist = sm;                                   // [3][kBins]
  uint32_t *wcount = sm + 3 * kBins;                     // [2][kSelWarps]: greater, equal
  uint32_t *res = wcount + 2 * kSelWarps;                // digit, remaining, slice's greater and equal
  uint32_t *keys = res + 8;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), ranks = (int)cl.num_blocks();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.x / ranks, b = bh / a.H;
  const int L = a.seq_lens ? min(max(__ldg(a.seq_lens + b), 0), a.kv_len) : a.kv_len;
  int32_t *keep = a.keep + (size_t)bh * a.n_keep;
  if (a.new_lens && bh % a.H == 0 && rank == 0 && tid == 0) a.new_lens[b] = min(L, a.n_keep);
  if (L <= a.n_keep) {                                   // everything stays (the whole cluster takes this branch)
    for (int i = rank * kSelThreads + tid; i < a.n_keep; i += ranks * kSelThreads) keep[i] = i < L ? i : -1;
    return;
  }
  const int lo = a.n_sink, hi = L - a.n_recent;          // the tokens that compete; lo < hi since L > n_keep
  for (int i = rank * kSelThreads + tid; i < a.n_sink + a.n_recent; i += ranks * kSelThreads) {
    if (i < a.n_sink) keep[i] = i;
    else keep[a.n_keep - a.n_recent + (i - a.n_sink)] = hi + (i - a.n_sink);
  }
  const int k = a.n_keep - a.n_sink - a.n_recent;
  if (k == 0) return;                                    // the same for every CTA
  const int per = ((hi - lo + ranks - 1) / ranks + 31) / 32 * 32;
  const int s0 = (int)min((long long)hi, lo + (long long)rank * per);   // this CTA's slice [s0, s0 + n)
  const int n = min(per, hi - s0);
  const float *score = a.scores + (size_t)bh * a.stride + s0;
  auto key_at = [&](int i) { return RESIDENT ? keys[i] : score_key(__ldg(score + i)); };

  for (int i = tid; i < 3 * kBins; i += kSelThreads) hist[i] = 0;
  __syncthreads();
  uint32_t prefix = 0, mask = 0, want = (uint32_t)k;      // T's digits so far, and the rank inside them
#pragma unroll
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0);
    const uint32_t width = d == 2 ? 1024u : 2048u;
    uint32_t *h = hist + d * kBins;
    for (int i0 = warp * 32; i0 < n; i0 += kSelThreads) {   // whole warps: the votes below need all lanes
      const int i = i0 + lane;
      uint32_t key = 0;
      bool in = i < n;
      if (in) {
        key = d == 0 || !RESIDENT ? score_key(__ldg(score + i)) : keys[i];
        if (RESIDENT && d == 0) keys[i] = key;
        in = (key & mask) == prefix;
      }
      const uint32_t digit = (key >> shift) & (width - 1);
      // long runs of one score (zeros) would serialise on one counter: count such a warp at once
      const unsigned who = __ballot_sync(0xffffffffu, in);
      if (who == 0) continue;
      const uint32_t first = __shfl_sync(0xffffffffu, digit, __ffs(who) - 1);
      if (__all_sync(0xffffffffu, !in || digit == first)) {
        if (lane == 0) atomicAdd(h + first, (uint32_t)__popc(who));
      } else if (in) {
        atomicAdd(h + digit, 1u);
      }
    }
    cl.sync();                                           // every slice is counted
    // thread t owns bins 2t and 2t + 1; counts above them by a suffix scan over warps
    uint32_t c0 = 0, c1 = 0;
    for (int r = 0; r < ranks; ++r) {
      const uint2 v = *reinterpret_cast<const uint2 *>(cl.map_shared_rank(h, r) + 2 * tid);
      c0 += v.x;
      c1 += v.y;
    }
    uint32_t suf = c0 + c1;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint32_t o = __shfl_down_sync(0xffffffffu, suf, m);
      if (lane + m < 32) suf += o;
    }
    if (lane == 0) wcount[warp] = suf;
    __syncthreads();
    uint32_t above = 0;                                  // in the warps of higher bins
    {
      uint32_t w = lane > warp ? wcount[lane] : 0;
#pragma unroll
      for (int m = 16; m; m >>= 1) w += __shfl_xor_sync(0xffffffffu, w, m);
      above = w;
    }
    const uint32_t above1 = above + suf - c0 - c1, above0 = above1 + c1;   // keys in bins over 2t + 1 / over 2t
    if (above1 < want && want <= above1 + c1) { res[0] = 2 * tid + 1; res[1] = want - above1; }
    if (above0 < want && want <= above0 + c0) { res[0] = 2 * tid; res[1] = want - above0; }
    __syncthreads();
    prefix |= res[0] << shift;
    mask |= (width - 1) << shift;
    want = res[1];
    __syncthreads();                                     // res and wcount are written again
  }
  // `want` of the keys equal to T stay. Count this slice's greater and equal keys by warp sub-slice.
  const int sub = ((n + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int w0 = min(n, warp * sub), w1 = min(n, w0 + sub);
  uint32_t ng = 0, ne = 0;
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t key = key_at(i);
    ng += key > prefix;
    ne += key == prefix;
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    ng += __shfl_xor_sync(0xffffffffu, ng, m);
    ne += __shfl_xor_sync(0xffffffffu, ne, m);
  }
  if (lane == 0) {
    wcount[warp] = ng;
    wcount[kSelWarps + warp] = ne;
  }
  __syncthreads();
  uint32_t gt = lane < warp ? wcount[lane] : 0, eq = lane < warp ? wcount[kSelWarps + lane] : 0;
  uint32_t gt_all = wcount[lane], eq_all = wcount[kSelWarps + lane];
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, m);
    eq += __shfl_xor_sync(0xffffffffu, eq, m);
    gt_all += __shfl_xor_sync(0xffffffffu, gt_all, m);
    eq_all += __shfl_xor_sync(0xffffffffu, eq_all, m);
  }
  if (tid == 0) {
    res[2] = gt_all;
    res[3] = eq_all;
  }
  cl.sync();
  for (int r = 0; r < rank; ++r) {
    const uint32_t *o = cl.map_shared_rank(res, r);
    gt += o[2];
    eq += o[3];
  }
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < w1 ? key_at(i) : 0;
    const bool g = i < w1 && key > prefix, e = i < w1 && key == prefix;
    const unsigned mg = __ballot_sync(0xffffffffu, g), me = __ballot_sync(0xffffffffu, e);
    const unsigned below = (1u << lane) - 1u;
    const uint32_t eq_rank = eq + __popc(me & below);
    if (g || (e && eq_rank < want))
      keep[a.n_sink + gt + __popc(mg & below) + min(eq_rank, want)] = s0 + i;
    gt += __popc(mg);
    eq += __popc(me);
  }
  cl.sync();                                             // no CTA leaves while another reads its counts
}

// ------------------------------------------------------------------------------------ compaction
constexpr int kMoveThreads = 512;
constexpr int kMoveUnits = 4;                            // units in flight per thread and round

template <class U>
__device__ __forceinline__ U load_unit(const uint8_t *p) { return __ldcg(reinterpret_cast<const U *>(p)); }

// One plane of one (batch, kv head): target rows [0, n_rows) in rounds of the whole cluster (IN_PLACE)
// or of the CTAs of one grid row. U: the unit moved at once; a row is `upr` units.
template <class U, bool IN_PLACE>
__device__ __forceinline__ void move_rows(const CompactArgs &a, const MovePart &p, int b, int kvh, int new_len, int n_rows,
                                          int L, int rank, int ranks) {
  const int upr = p.row_bytes / (int)sizeof(U);
  const int32_t *keep = a.keep + ((size_t)b * a.src.H + kvh) * a.n_keep;
  const size_t head = (size_t)b * a.src.H + kvh;
  const unsigned total = (unsigned)n_rows * upr;         // at most 2^31 (the host checks)
  const unsigned round = (unsigned)ranks * kMoveThreads * kMoveUnits;
  auto src_row = [&](int t) -> const uint8_t * {
    const size_t r = p.is_scores ? head * (size_t)a.scores_stride + t : cache_row(a.src, b, kvh, t);
    return p.src + r * p.row_bytes;
  };
  auto dst_row = [&](int t) -> uint8_t * {
    const size_t r = p.is_scores ? head * (size_t)a.out_stride + t : cache_row(a.dst, b, kvh, t);
    return p.dst + r * p.row_bytes;
  };
  // unit u of the round that starts at `base`
  auto unit_of = [&](unsigned base, int u) { return base + ((unsigned)u * ranks + rank) * kMoveThreads + threadIdx.x; };
  // the source token of a unit: -1 = leave the target as it is, -2 = zero (scores behind the kept ones)
  auto source = [&](unsigned id) -> int {
    if (id >= total) return -1;
    const int row = (int)(id / upr);
    if (row >= new_len) return -2;
    const int t = __ldg(keep + row);
    if (t < 0 || t >= L || (IN_PLACE && t == row)) return -1;
    return t;
  };
  U cur[kMoveUnits], nxt[kMoveUnits];
  int st[kMoveUnits], sn[kMoveUnits];
  auto gather = [&](unsigned base, int (&s)[kMoveUnits], U (&v)[kMoveUnits]) {
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u) s[u] = source(unit_of(base, u));
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u) {
      v[u] = U{};
      if (s[u] >= 0) v[u] = load_unit<U>(src_row(s[u]) + (size_t)(unit_of(base, u) % upr) * sizeof(U));
    }
  };
  gather(0, st, cur);
  for (unsigned base = 0; base < total; base += round) {
    if constexpr (IN_PLACE) {
      // this round's values have arrived (the register reads below wait for the loads) before any CTA
      // of the cluster writes over their rows
#pragma unroll
      for (int u = 0; u < kMoveUnits; ++u) asm volatile("" ::"r"(reinterpret_cast<const uint32_t *>(&cur[u])[0]) : "memory");
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    if (round < total - base) gather(base + round, sn, nxt);
    if constexpr (IN_PLACE) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u) {
      const unsigned id = unit_of(base, u);
      if (st[u] != -1) *reinterpret_cast<U *>(dst_row((int)(id / upr)) + (size_t)(id % upr) * sizeof(U)) = cur[u];
      cur[u] = nxt[u];
      st[u] = sn[u];
    }
  }
}

template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(CompactArgs a) {
  const int bh = blockIdx.x / a.ranks, b = bh / a.src.H, kvh = bh - b * a.src.H;
  const MovePart &p = a.part[blockIdx.y];
  const int L = a.seq_lens ? min(max(__ldg(a.seq_lens + b), 0), a.kv_len) : a.kv_len;
  const int new_len = min(L, a.n_keep);
  // the scores behind the kept ones become zero, ready for the tokens appended next
  const int n_rows = p.is_scores ? (int)min((long long)a.kv_len, a.out_stride) : new_len;
  const int ranks = a.ranks, rank = blockIdx.x - bh * ranks;   // IN_PLACE: these CTAs are one cluster
  switch (p.unit) {
    case 16: move_rows<uint4, IN_PLACE>(a, p, b, kvh, new_len, n_rows, L, rank, ranks); break;
    case 8: move_rows<uint2, IN_PLACE>(a, p, b, kvh, new_len, n_rows, L, rank, ranks); break;
    default: move_rows<uint32_t, IN_PLACE>(a, p, b, kvh, new_len, n_rows, L, rank, ranks); break;
  }
}

// The exact window: slot of token t is t mod R, and every kept window token moves back by the number of
// tokens cut, so the ring turns left by that number. Into another cache a copy; in place three
// reversals (of the first e rows, of the rest, of all), each one swap per pair of rows. One CTA per
// (batch, kv head, plane, 32 dims).
constexpr int kRingThreads = 256;
__global__ void __launch_bounds__(kRingThreads) evict_ring_kernel(CompactArgs a, int in_place) {
  const int bh = blockIdx.x, b = bh / a.src.H, R = a.src.n_recent, D = a.src.D;
  const int L = a.seq_lens ? min(max(__ldg(a.seq_lens + b), 0), a.kv_len) : a.kv_len;
  const int e = (L - min(L, a.n_keep)) % R;
  const size_t at = (size_t)bh * R * D + 32 * blockIdx.z;
  const float *src = a.src.ring[blockIdx.y] + at;
  float *dst = a.dst.ring[blockIdx.y] + at;
  const int col = 4 * (threadIdx.x & 7), r0 = threadIdx.x >> 3;
  constexpr int kRows = kRingThreads / 8;
  if (!in_place) {
    for (int j = r0; j < R; j += kRows)
      *reinterpret_cast<float4 *>(dst + (size_t)j * D + col) =
          *reinterpret_cast<const float4 *>(src + (size_t)((j + e) % R) * D + col);
    return;
  }
  if (e == 0) return;
  const int first[3] = {0, e, 0}, last[3] = {e, R, R};
  for (int s = 0; s < 3; ++s) {
    const int m = last[s] - first[s];
    for (int j = r0; j < m / 2; j += kRows) {
      float4 *x = reinterpret_cast<float4 *>(dst + (size_t)(first[s] + j) * D + col);
      float4 *y = reinterpret_cast<float4 *>(dst + (size_t)(last[s] - 1 - j) * D + col);
      const float4 t = *x;
      *x = *y;
      *y = t;
    }
    __syncthreads();
  }
}

int device_sms() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <bool RESIDENT>
cudaError_t launch_select(const SelectArgs &a, int ranks, int smem, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = set_smem_once(done, evict_select_kernel<RESIDENT>, 227 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ranks * a.B * a.H);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<RESIDENT>, a);
}

}  // namespace

cudaError_t launch_evict_select(const SelectArgs &a, cudaStream_t st) {
  // CTAs per (batch, kv head): one per 8192 tokens, at most the portable cluster size of 8
  int ranks = 1;
  while (ranks < 8 && (long long)ranks * 8192 < a.kv_len) ranks *= 2;
  const int per = (a.kv_len + ranks - 1) / ranks + 32;
  if (per <= kSelMaxKeys) return launch_select<true>(a, ranks, kSelFixed + 4 * per, st);
  return launch_select<false>(a, ranks, kSelFixed, st);
}

cudaError_t launch_evict_compact(CompactArgs a, bool in_place, cudaStream_t st) {
  const int heads = a.src.B * a.src.H;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = st;
  cudaError_t e;
  // CTAs per plane of one (batch, kv head): about two per SM over the two payload planes; in place one
  // cluster (at most the portable 8)
  const int want = max(1, device_sms() / heads);
  if (in_place) {
    a.ranks = 1;
    while (a.ranks < 8 && a.ranks < want) a.ranks *= 2;
    cfg.gridDim = dim3((unsigned)a.ranks * heads, a.n_parts);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, evict_move_kernel<true>, a);
  } else {
    a.ranks = want;
    cfg.gridDim = dim3((unsigned)want * heads, a.n_parts);
    e = cudaLaunchKernelEx(&cfg, evict_move_kernel<false>, a);
  }
  if (e != cudaSuccess || a.src.n_recent == 0) return e;
  evict_ring_kernel<<<dim3(heads, 2, a.src.D / 32), kRingThreads, 0, st>>>(a, in_place ? 1 : 0);
  return cudaGetLastError();
}

}  // namespace kvq
