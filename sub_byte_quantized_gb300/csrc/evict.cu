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
constexpr int kBins = 2048;
template <int THREADS>
__host__ __device__ constexpr int select_fixed() { return (3 * kBins + 2 * (THREADS / 32) + 4) * 4; }   // histograms, per-warp counts, results
constexpr int kSelMaxKeys = (227 * 1024 - select_fixed<1024>()) / 4 / 128 * 128;   // keys one CTA can hold

// Keys compare like the scores: NaN counts as -infinity, -0 as +0.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// RESIDENT: the slice's keys fit shared memory (else every pass reads the scores again).
template <int THREADS, bool RESIDENT>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) evict_select_kernel(SelectArgs a) {
  constexpr int WARPS = THREADS / 32, OWN = kBins / THREADS;   // bins per thread, neighbouring
  extern __shared__ __align__(16) uint32_t sm[];
  uint32_t *hist = sm;                                   // [3][kBins]
  uint32_t *wcount = sm + 3 * kBins;                     // [2][WARPS]
  uint32_t *res = wcount + 2 * WARPS;                    // digit, rank inside it
  uint32_t *keys = res + 4;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), ranks = (int)cl.num_blocks();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.x / ranks, b = bh / a.H;
  const int L = a.seq_lens ? min(max(__ldg(a.seq_lens + b), 0), a.kv_len) : a.kv_len;
  int32_t *keep = a.keep + (size_t)bh * a.n_keep;
  if (a.new_lens && bh % a.H == 0 && rank == 0 && tid == 0) a.new_lens[b] = min(L, a.n_keep);
  if (L <= a.n_keep) {                                   // everything stays (the whole cluster takes this branch)
    for (int i = rank * THREADS + tid; i < a.n_keep; i += ranks * THREADS) keep[i] = i < L ? i : -1;
    return;
  }
  const int lo = a.n_sink, hi = L - a.n_recent;          // the tokens that compete; lo < hi since L > n_keep
  for (int i = rank * THREADS + tid; i < a.n_sink + a.n_recent; i += ranks * THREADS) {
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
  if constexpr (RESIDENT) {
#pragma unroll 8
    for (int i = tid; i < n; i += THREADS) keys[i] = score_key(__ldg(score + i));
  }
  for (int i = tid; i < 3 * kBins; i += THREADS) hist[i] = 0;
  __syncthreads();
  uint32_t prefix = 0, mask = 0, want = (uint32_t)k;      // T's digits so far, and the rank inside them
  uint32_t gt = 0, eq = 0;                               // keys over / equal to T in the slices before this one
#pragma unroll
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0);
    const uint32_t width = d == 2 ? 1024u : 2048u;
    uint32_t *h = hist + d * kBins;
    for (int i0 = warp * 128; i0 < n; i0 += 4 * THREADS) {  // whole warps: the votes below need all lanes
      const int i = i0 + 4 * lane;                          // four keys per lane
      uint32_t key[4];
      if constexpr (RESIDENT) {
        const uint4 v = *reinterpret_cast<const uint4 *>(keys + i);   // (the keys' space is a multiple of 128)
        key[0] = v.x; key[1] = v.y; key[2] = v.z; key[3] = v.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) key[j] = i + j < n ? key_at(i + j) : 0;
      }
      bool in[4], any = false;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        in[j] = i + j < n && (key[j] & mask) == prefix;
        any |= in[j];
      }
      if (!__any_sync(0xffffffffu, any)) continue;
      // long runs of one score (zeros) would serialise on one counter: count such a group at once
      const uint32_t first = __shfl_sync(0xffffffffu, (key[0] >> shift) & (width - 1), 0);
      bool same = true;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        key[j] = (key[j] >> shift) & (width - 1);
        same &= in[j] && key[j] == first;
      }
      if (__all_sync(0xffffffffu, same)) {
        if (lane == 0) atomicAdd(h + first, 128u);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (in[j]) atomicAdd(h + key[j], 1u);
      }
    }
    cl.sync();                                           // every slice is counted
    // thread t owns bins OWN t .. OWN t + OWN - 1; the counts above them by a suffix scan over warps
    uint32_t c[OWN] = {}, before[OWN] = {};              // all slices; the slices before this one
    for (int r = 0; r < ranks; ++r) {
      const uint32_t *o = cl.map_shared_rank(h, r) + OWN * tid;
#pragma unroll
      for (int j = 0; j < OWN; j += 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(o + j);
        c[j] += v.x;
        c[j + 1] += v.y;
        before[j] += r < rank ? v.x : 0;
        before[j + 1] += r < rank ? v.y : 0;
      }
    }
    if (d == 2) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // the last remote reads
    uint32_t own = 0;
#pragma unroll
    for (int j = 0; j < OWN; ++j) own += c[j];
    uint32_t suf = own;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint32_t o = __shfl_down_sync(0xffffffffu, suf, m);
      if (lane + m < 32) suf += o;
    }
    if (lane == 0) wcount[warp] = suf;
    __syncthreads();
    uint32_t above = lane > warp && lane < WARPS ? wcount[lane] : 0;   // in the warps of higher bins
#pragma unroll
    for (int m = 16; m; m >>= 1) above += __shfl_xor_sync(0xffffffffu, above, m);
    above += suf - own;
#pragma unroll
    for (int j = OWN - 1; j >= 0; --j) {                 // above = keys in the bins over bin j
      if (above < want && want <= above + c[j]) {
        res[0] = OWN * tid + j;
        res[1] = want - above;
      }
      above += c[j];
    }
    __syncthreads();
    const uint32_t digit = res[0];
    want = res[1];
    prefix |= digit << shift;
    mask |= (width - 1) << shift;
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
      const uint32_t bin = OWN * tid + j;
      if (bin > digit) gt += before[j];
      if (d == 2 && bin == digit) eq += before[j];
    }
    __syncthreads();                                     // res and wcount are written again
  }
  // block sums of gt and eq (each key counted by one thread)
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, m);
    eq += __shfl_xor_sync(0xffffffffu, eq, m);
  }
  if (lane == 0) {
    wcount[warp] = gt;
    wcount[WARPS + warp] = eq;
  }
  __syncthreads();
  gt = lane < WARPS ? wcount[lane] : 0;
  eq = lane < WARPS ? wcount[WARPS + lane] : 0;
  __syncthreads();
  // `want` of the keys equal to T stay. This slice's greater and equal keys by warp sub-slice.
  const int sub = ((n + WARPS - 1) / WARPS + 31) / 32 * 32;
  const int w0 = min(n, warp * sub), w1 = min(n, w0 + sub);
  uint32_t ng = 0, ne = 0;
#pragma unroll 4
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
    wcount[WARPS + warp] = ne;
  }
  __syncthreads();
  gt += lane < warp ? wcount[lane] : 0;
  eq += lane < warp ? wcount[WARPS + lane] : 0;
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, m);
    eq += __shfl_xor_sync(0xffffffffu, eq, m);
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
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // no CTA leaves while another reads its counts
}

// ------------------------------------------------------------------------------------ compaction
constexpr int kMoveThreads = 512;
constexpr int kMoveUnits = 4;                            // units in flight per thread and round

// The rows of one plane (or of the scores) of one (batch, kv head), a column of each for this thread.
template <bool PAGED>
struct PlaneRows {
  uint8_t *base;
  int row_bytes;
  const CacheView *c;
  int b, kvh;
  __device__ __forceinline__ uint8_t *at(int t) const {
    if constexpr (PAGED) return base + (unsigned long long)cache_row_paged(*c, b, kvh, t) * (unsigned)row_bytes;
    else return base + (unsigned long long)(unsigned)t * (unsigned)row_bytes;
  }
};
template <bool PAGED>
__device__ __forceinline__ PlaneRows<PAGED> rows_of(const CacheView &c, uint8_t *plane, int row_bytes, long long scores_stride,
                                                    int b, int kvh, int col) {
  PlaneRows<PAGED> r = {plane + col, row_bytes, &c, b, kvh};
  if constexpr (!PAGED) {
    const size_t head = (size_t)b * c.H + kvh;
    r.base += head * (size_t)(scores_stride >= 0 ? scores_stride : c.cap) * row_bytes;
  }
  return r;
}

// Source token of target row `row`: -1 = leave the row as it is, -2 = zero (scores behind the kept ones).
template <bool IN_PLACE>
__device__ __forceinline__ int source_of(const int32_t *keep, int row, int new_len, int n_rows, int L) {
  if (row >= new_len) return row < n_rows ? -2 : -1;
  const int t = __ldg(keep + row);
  return (unsigned)t >= (unsigned)L || (IN_PLACE && t == row) ? -1 : t;
}

// Target rows [0, n_rows). A thread keeps its column of the row (row_bytes / sizeof(U) threads hold a row)
// and steps through rows; U: the unit moved at once. Into another cache every CTA moves its own rounds. In
// place the ranks' CTAs are one cluster whose rounds are ordered by its barrier; the sources of the round
// after next are looked up, and the rows of the next one read, while this one waits.
template <class U, bool IN_PLACE, bool PAGED>
__device__ __forceinline__ void move_rows(const CompactArgs &a, const MovePart &p, int b, int kvh, int new_len, int n_rows,
                                          int L, int rank) {
  const int upr = p.row_bytes / (int)sizeof(U), rpp = kMoveThreads / upr;   // threads per row, rows per pass
  const int own = (int)threadIdx.x / upr, col = ((int)threadIdx.x - own * upr) * (int)sizeof(U);
  const int32_t *keep = a.keep + ((size_t)b * a.src.H + kvh) * a.n_keep;
  const auto src = rows_of<PAGED>(a.src, const_cast<uint8_t *>(p.src), p.row_bytes, p.is_scores ? a.scores_stride : -1, b, kvh, col);
  const auto dst = rows_of<PAGED>(a.dst, p.dst, p.row_bytes, p.is_scores ? a.out_stride : -1, b, kvh, col);
  const int step = a.ranks * rpp, round = step * kMoveUnits;   // rows between a thread's units, rows per round
  const int row0 = own < rpp ? rank * rpp + own : n_rows;      // (threads beyond the last whole row idle)
  if constexpr (!IN_PLACE) {
    for (int base = row0; base < n_rows; base += round) {
      int st[kMoveUnits];
      U v[kMoveUnits];
#pragma unroll
      for (int u = 0; u < kMoveUnits; ++u) st[u] = source_of<false>(keep, base + u * step, new_len, n_rows, L);
#pragma unroll
      for (int u = 0; u < kMoveUnits; ++u) {
        v[u] = U{};
        if (st[u] >= 0) v[u] = __ldcg(reinterpret_cast<const U *>(src.at(st[u])));
      }
#pragma unroll
      for (int u = 0; u < kMoveUnits; ++u)
        if (st[u] != -1) *reinterpret_cast<U *>(dst.at(base + u * step)) = v[u];
    }
  } else {
    U cur[kMoveUnits], nxt[kMoveUnits];
    int st[kMoveUnits], sn[kMoveUnits];                  // sources of this round and the next
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u) {
      st[u] = source_of<true>(keep, row0 + u * step, new_len, n_rows, L);
      sn[u] = source_of<true>(keep, row0 + round + u * step, new_len, n_rows, L);
    }
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u) {
      cur[u] = U{};
      if (st[u] >= 0) cur[u] = __ldcg(reinterpret_cast<const U *>(src.at(st[u])));
    }
    for (int base = 0; base < n_rows; base += round) {
      // This round's values have arrived (the register reads below wait for the loads) before any CTA of the
      // cluster writes over their rows. That is all the barrier orders: nothing written before it is read
      // after it, so the arrive needs no release of this thread's earlier stores.
#pragma unroll
      for (int u = 0; u < kMoveUnits; ++u) asm volatile("" ::"r"(reinterpret_cast<const uint32_t *>(&cur[u])[0]) : "memory");
      asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
      const bool more = n_rows - base > round;
      if (more) {
#pragma unroll
        for (int u = 0; u < kMoveUnits; ++u) {
          nxt[u] = U{};
          if (sn[u] >= 0) nxt[u] = __ldcg(reinterpret_cast<const U *>(src.at(sn[u])));
        }
      }
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
      for (int u = 0; u < kMoveUnits; ++u)
        if (st[u] != -1) *reinterpret_cast<U *>(dst.at(row0 + base + u * step)) = cur[u];
      if (more) {
#pragma unroll
        for (int u = 0; u < kMoveUnits; ++u) {
          cur[u] = nxt[u];
          st[u] = sn[u];
          sn[u] = source_of<true>(keep, row0 + base + 2 * round + u * step, new_len, n_rows, L);
        }
      }
    }
  }
}

template <bool IN_PLACE, bool PAGED>
__device__ __forceinline__ void move_part(const CompactArgs &a, const MovePart &p, int b, int kvh, int new_len, int n_rows, int L,
                                          int rank) {
  switch (p.unit) {
    case 16: move_rows<uint4, IN_PLACE, PAGED>(a, p, b, kvh, new_len, n_rows, L, rank); break;
    case 8: move_rows<uint2, IN_PLACE, PAGED>(a, p, b, kvh, new_len, n_rows, L, rank); break;
    default: move_rows<uint32_t, IN_PLACE, PAGED>(a, p, b, kvh, new_len, n_rows, L, rank); break;
  }
}

template <bool IN_PLACE, bool PAGED>
__global__ void __launch_bounds__(kMoveThreads, 2) evict_move_kernel(CompactArgs a) {
  const int bh = blockIdx.x / a.ranks, b = bh / a.src.H, kvh = bh - b * a.src.H, rank = blockIdx.x - bh * a.ranks;
  const MovePart &p = a.part[blockIdx.y];
  const int L = a.seq_lens ? min(max(__ldg(a.seq_lens + b), 0), a.kv_len) : a.kv_len;
  const int new_len = min(L, a.n_keep);
  // the scores behind the kept ones become zero, ready for the tokens appended next; they are not paged
  if (p.is_scores) move_rows<uint32_t, IN_PLACE, false>(a, p, b, kvh, new_len, (int)min((long long)a.kv_len, a.out_stride), L, rank);
  else move_part<IN_PLACE, PAGED>(a, p, b, kvh, new_len, new_len, L, rank);
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

template <int THREADS, bool RESIDENT>
cudaError_t launch_select(const SelectArgs &a, int ranks, int keys, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = set_smem_once(done, evict_select_kernel<THREADS, RESIDENT>, 227 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ranks * a.B * a.H);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = select_fixed<THREADS>() + 4 * keys;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<THREADS, RESIDENT>, a);
}

}  // namespace

cudaError_t launch_evict_select(const SelectArgs &a, cudaStream_t st) {
  // CTAs per (batch, kv head): one per 8192 tokens, at most the portable cluster size of 8
  int ranks = 1;
  while (ranks < 8 && (long long)ranks * 8192 < a.kv_len) ranks *= 2;
  const int keys = ((a.kv_len + ranks - 1) / ranks + 31 + 127) / 128 * 128;
  if (keys > kSelMaxKeys) return launch_select<1024, false>(a, ranks, 0, st);
  // rows of one CTA: half the threads, two CTAs per SM
  return ranks == 1 ? launch_select<512, true>(a, ranks, keys, st) : launch_select<1024, true>(a, ranks, keys, st);
}

cudaError_t launch_evict_compact(CompactArgs a, bool in_place, cudaStream_t st) {
  const int heads = a.src.B * a.src.H;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = st;
  cudaError_t e;
  const int most = a.n_keep < a.kv_len ? a.n_keep : a.kv_len;
  if (in_place) {
    // one cluster per plane of a (batch, kv head), at most the portable 8 CTAs: enough for two waves of two
    // CTAs per SM over the two payload planes
    const int want = (2 * device_sms() + heads - 1) / heads;
    a.ranks = 1;
    while (a.ranks < 8 && a.ranks < want) a.ranks *= 2;
    cfg.gridDim = dim3((unsigned)a.ranks * heads, a.n_parts);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = a.src.page_shift >= 0 ? cudaLaunchKernelEx(&cfg, evict_move_kernel<true, true>, a)
                              : cudaLaunchKernelEx(&cfg, evict_move_kernel<true, false>, a);
  } else {
    // nothing waits: one round per CTA for the widest rows, the scheduler overlaps them
    const int upr = (a.src.row_bytes > a.src.v_row_bytes ? a.src.row_bytes : a.src.v_row_bytes) / 16;
    const int round = kMoveThreads / upr * kMoveUnits;
    a.ranks = min((most + round - 1) / round, max(1, (1 << 16) / heads));
    cfg.gridDim = dim3((unsigned)a.ranks * heads, a.n_parts);
    e = cudaLaunchKernelEx(&cfg, evict_move_kernel<false, false>, a);
  }
  if (e != cudaSuccess || a.src.n_recent == 0) return e;
  evict_ring_kernel<<<dim3(heads, 2, a.src.D / 32), kRingThreads, 0, st>>>(a, in_place ? 1 : 0);
  return cudaGetLastError();
}

}  // namespace kvq
