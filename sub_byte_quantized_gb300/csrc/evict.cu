// Keeping a cache inside a budget: which tokens stay (selection by running attention weight), and
// moving their packed rows together (compaction).
//
// Selection, per (batch, kv head): of L tokens the first n_sink and the last n_recent stay; among the
// others the k with the highest scores, ties going to the lowest index. That set is {score > T} and the
// first few of {score == T}, T being the k-th highest score: a radix selection over order-preserving
// 32-bit keys finds T in three digits (12, 10 and 10 bits), then one ordered pass writes the list in
// ascending order. One cluster works on one (batch, kv head): every CTA keeps its slice of the keys in
// shared memory, so the scores are read from memory once; the digits' counts are summed over distributed
// shared memory. Bound by latency (load, three histogram rounds, the ordered pass), not by its bytes: 13.6
// us for 32K of 128K tokens in 8 heads, 8.2 for 1021 of up to 4099 in 256 heads.
//
// Compaction: row keep[i] of every plane moves to row i. keep ascends, so keep[i] >= i: a round reads
// the sources of the next block of target rows, everyone waits until all of the cluster's reads have
// arrived, then writes; reads of later rounds lie behind what it writes. One cluster per (batch, kv head,
// plane); into another cache nothing can be overwritten too early, and the rounds need no barrier. Bound
// by memory: scattered rows of 64 bytes and scales of 8 cost whole DRAM bursts (128K to 32K tokens in Q4_0,
// 8 heads: 81 MB read for 41 that are needed, 22.3 us; 16 ragged sequences in Q8_0 in place 53.5 us). Before the
// barrier's arrival the loads must have returned: a relaxed arrival does not wait for them (and took 46.7 us, now and
// then with rows that another CTA had already written over).
#include <cooperative_groups.h>

#include "kvq_internal.cuh"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------------------------ selection
// Digits of 12, 10 and 10 bits: the first one's histogram takes every key, and at 12 bits (sign, exponent and three
// bits of the fraction) fewer of a warp's keys meet in one counter.
__host__ __device__ constexpr int digit_shift(int d) { return d == 0 ? 20 : d == 1 ? 10 : 0; }
__host__ __device__ constexpr int digit_bins(int d) { return d == 0 ? 4096 : 1024; }
__host__ __device__ constexpr int digit_at(int d) { return d == 0 ? 0 : 4096 + 1024 * (d - 1); }   // its first counter
constexpr int kBins = digit_at(3), kGroups = kBins / 32;   // counters; their sums in groups of 32
template <int THREADS>                   // histograms, their groups' sums, per-warp counts, results
__host__ __device__ constexpr int select_fixed() { return (kBins + kGroups + 2 * (THREADS / 32) + 4) * 4; }
constexpr int kBlockSelectSmem = (kMaxSelectBlocks / 8 + 256) * 4 + select_fixed<512>();   // of the longest lists
static_assert(kBlockSelectSmem <= 200 * 1024, "the longest lists' scores fit");
constexpr int kSelMaxKeys = (227 * 1024 - select_fixed<1024>()) / 4 / 128 * 128;   // keys one CTA can hold

// Keys compare like the scores: NaN counts as -infinity, -0 as +0. No score has a key below 2^22: key 0 stands for
// "no token", and what it adds to the lowest counter is never reached.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One warp: among the bins of which each lane holds OWN neighbouring ones (`c`: their counts, all slices; `before`:
// in the slices before this one), the bin of the key that has `want` - 1 keys over it, `above` of them in bins
// over all of these. Sets `above` to what lies over that bin, adds the earlier slices' keys over it to `gt`, and
// returns its index; `at` its earlier slices' count.
template <int OWN>
__device__ __forceinline__ int find_bin(const uint32_t (&c)[OWN], const uint32_t (&before)[OWN], uint32_t want, int lane,
                                        uint32_t &above, uint32_t &gt, uint32_t &at) {
  uint32_t own = 0;
#pragma unroll
  for (int j = 0; j < OWN; ++j) own += c[j];
  uint32_t over = own;                                   // suffix sums: the counts of this lane and those above
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const uint32_t o = __shfl_down_sync(0xffffffffu, over, m);
    if (lane + m < 32) over += o;
  }
  over += above - own;
  int hit = -1;
  uint32_t hit_over = 0;
#pragma unroll
  for (int j = OWN - 1; j >= 0; --j) {
    if (over < want && want <= over + c[j]) hit = j, hit_over = over;
    over += c[j];
  }
  const int from = __ffs(__ballot_sync(0xffffffffu, hit >= 0)) - 1;
  const int bin = OWN * from + __shfl_sync(0xffffffffu, hit, from);
  above = __shfl_sync(0xffffffffu, hit_over, from);
  uint32_t more = 0, here = 0;
#pragma unroll
  for (int j = 0; j < OWN; ++j) {
    if (OWN * lane + j > bin) more += before[j];
    if (OWN * lane + j == bin) here = before[j];
  }
  gt += __reduce_add_sync(0xffffffffu, more);
  at = __shfl_sync(0xffffffffu, here, from);
  return bin;
}

// Where the scores come from: memory, or (the blocks that a query selects) the bounds of the keys.
struct ScoresInMemory {
  static constexpr int D = 0;
};
template <int DIM>
struct ScoresOfBlocks {
  static constexpr int D = DIM;
  BlockSelectArgs s;
};
// The blocks that list `vb` = (sequence, kv head, query) sees.
__device__ __forceinline__ int blocks_seen(const BlockSelectArgs &s, int vb) {
  const int bh = vb / s.n_q, i = vb - bh * s.n_q, b = bh / s.cache.H;
  const int len = s.seq_lens ? min(max(__ldg(s.seq_lens + b), 0), s.kv_len) : s.kv_len;
  const int limit = s.causal ? min(len - 1, (s.seq_lens ? len - s.n_q : s.q_pos0) + i) : len - 1;
  return limit < 0 ? 0 : (limit >> 6) + 1;
}
// Scores of the blocks [s0, s0 + n) of list vb into `score`: the query heads' rows in int8 (their negative and positive parts
// apart, eight heads at a time), four threads per block.
constexpr int kRowsAtOnce = 8;
template <int THREADS, int D>
__device__ __forceinline__ void score_blocks(const BlockSelectArgs &a, int vb, int s0, int n, float *score) {
  constexpr int V = D / 32;
  __shared__ __align__(16) int8_t q_neg[kRowsAtOnce][D], q_pos[kRowsAtOnce][D];
  __shared__ float q_step[kRowsAtOnce];
  const CacheView &c = a.cache;
  const int bh = vb / a.n_q, i = vb - bh * a.n_q, b = bh / c.H, h = bh - b * c.H;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, part = tid & 3;
  for (int r0 = 0; r0 < a.gqa; r0 += kRowsAtOnce) {
    if (r0 > 0) __syncthreads();
    if (warp < kRowsAtOnce && r0 + warp < a.gqa) {
      const size_t row = ((size_t)bh * a.gqa + r0 + warp) * a.n_q + i;
      float x[V], s;
      int q8[V];
      if (V == 4) load4_f32(a.q, a.q_dtype, row * D + lane * 4, x);
      else load8_f32(a.q, a.q_dtype, row * D + lane * 8, x);
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
    const int rows = min(kRowsAtOnce, a.gqa - r0);
    for (int i0 = 0; i0 < n; i0 += THREADS / 4) {        // whole warps: the sums below need all lanes
      const int j = i0 + (tid >> 2);
      const bool live = j < n;
      uint4 lo[D / 64], hi[D / 64];                      // the thread's quarter of the block's bounds
      float scale = 0.0f;
      if (live) {
        const size_t at = cache_row(c, b, h, (s0 + j) << 6) >> 6;
        const uint4 *p = reinterpret_cast<const uint4 *>(a.codes + at * 2 * D) + part * (D / 64);
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          lo[k] = __ldg(p + k);
          hi[k] = __ldg(p + D / 16 + k);
        }
        scale = __ldg(a.scale + at);
      } else {
#pragma unroll
        for (int k = 0; k < D / 64; ++k) lo[k] = hi[k] = make_uint4(0u, 0u, 0u, 0u);
      }
      float best = -INFINITY;
      for (int r = 0; r < rows; ++r) {
        int dot = 0;
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          const uint4 x = *reinterpret_cast<const uint4 *>(&q_neg[r][(part * (D / 64) + k) * 16]);
          const uint4 y = *reinterpret_cast<const uint4 *>(&q_pos[r][(part * (D / 64) + k) * 16]);
          dot = __dp4a((int)x.x, (int)lo[k].x, dot);
          dot = __dp4a((int)x.y, (int)lo[k].y, dot);
          dot = __dp4a((int)x.z, (int)lo[k].z, dot);
          dot = __dp4a((int)x.w, (int)lo[k].w, dot);
          dot = __dp4a((int)y.x, (int)hi[k].x, dot);
          dot = __dp4a((int)y.y, (int)hi[k].y, dot);
          dot = __dp4a((int)y.z, (int)hi[k].z, dot);
          dot = __dp4a((int)y.w, (int)hi[k].w, dot);
        }
        dot += __shfl_xor_sync(0xffffffffu, dot, 1);
        dot += __shfl_xor_sync(0xffffffffu, dot, 2);
        best = fmaxf(best, __fmul_rn((float)dot, q_step[r]));
      }
      best = __fmul_rn(best, scale);                     // (its rounding keeps the order: as if the largest were taken after it)
      if (live && part == 0) score[j] = r0 > 0 ? fmaxf(score[j], best) : best;
    }
  }
  __syncthreads();
}

// RESIDENT: the slice's keys fit shared memory (else every pass reads the scores again). RANKS: CTAs of a cluster, at most.
template <int THREADS, int RANKS, bool RESIDENT, class Source>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) evict_select_kernel(SelectArgs a, Source src) {
  constexpr int WARPS = THREADS / 32;
  extern __shared__ __align__(16) uint32_t sm[];
  uint32_t *hist = sm, *group = hist + kBins;
  uint32_t *wcount = group + kGroups;                    // [2][WARPS]
  uint32_t *res = wcount + 2 * WARPS;                    // digit, rank inside it; earlier slices' keys over T, equal to T
  uint32_t *keys = res + 4;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), ranks = (int)cl.num_blocks();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bh = blockIdx.x / ranks, b = bh / a.H;
  int L;
  if constexpr (Source::D > 0) L = blocks_seen(src.s, bh);
  else L = a.seq_lens ? min(max(__ldg(a.seq_lens + b), 0), a.kv_len) : a.kv_len;
  int32_t *keep = a.keep + (size_t)bh * a.n_keep;
  if (a.new_lens && bh % a.H == 0 && rank == 0 && tid == 0) a.new_lens[b] = min(L, a.n_keep);
  if (L <= a.n_keep) {                                   // everything stays (the whole cluster takes this branch)
    for (long long i = rank * THREADS + tid; i < a.n_keep; i += ranks * THREADS) keep[i] = i < L ? (int)i : -1;   // (n_keep up to 2^31 - 1)
    return;
  }
  const int lo = a.n_sink, hi = L - a.n_recent;          // the tokens that compete; lo < hi since L > n_keep
  for (int i = rank * THREADS + tid; i < a.n_sink + a.n_recent; i += ranks * THREADS) {
    if (i < a.n_sink) keep[i] = i;
    else keep[a.n_keep - a.n_recent + (i - a.n_sink)] = hi + (i - a.n_sink);
  }
  const int k = a.n_keep - a.n_sink - a.n_recent;
  if (k == 0) return;                                    // the same for every CTA
  // this CTA's slice [s0, s0 + n), from a multiple of four on; in shared memory np keys, a multiple of 128
  const int lo4 = lo & ~3, per = ((hi - lo4 + ranks - 1) / ranks + 31) / 32 * 32;
  const int s0 = (int)min((long long)hi, lo4 + (long long)rank * per);
  const int n = min(per, hi - s0), np = (n + 127) / 128 * 128;
  const float *score = nullptr;
  if constexpr (Source::D == 0) score = a.scores + (size_t)bh * a.stride + s0;
  auto key_of = [&](int i, float x) { return i < n && s0 + i >= lo ? score_key(x) : 0u; };
  auto four = [&](int i, uint32_t (&key)[4]) {
    if constexpr (RESIDENT) {
      const uint4 v = *reinterpret_cast<const uint4 *>(keys + i);
      key[0] = v.x; key[1] = v.y; key[2] = v.z; key[3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) key[j] = key_of(i + j, i + j < n ? __ldg(score + i + j) : 0.0f);
    }
  };
  if constexpr (Source::D > 0) {
    float *fresh = reinterpret_cast<float *>(keys);
    score_blocks<THREADS, Source::D>(src.s, bh, s0, max(n, 0), fresh);
    for (int i = tid; i < np; i += THREADS) keys[i] = key_of(i, i < n ? fresh[i] : 0.0f);
  } else if constexpr (RESIDENT) {
    if (a.stride % 4 == 0) {                             // rows and slices begin at 16-byte boundaries
#pragma unroll 1
      for (int i0 = 4 * tid; i0 < np; i0 += 16 * THREADS) {   // four loads in flight
        float4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + 4 * THREADS * u;
          v[u] = i < n ? __ldg(reinterpret_cast<const float4 *>(score + i)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + 4 * THREADS * u;
          if (i < np)
            *reinterpret_cast<uint4 *>(keys + i) = make_uint4(key_of(i, v[u].x), key_of(i + 1, v[u].y), key_of(i + 2, v[u].z), key_of(i + 3, v[u].w));
        }
      }
    } else {
#pragma unroll 4
      for (int i = tid; i < np; i += THREADS) keys[i] = key_of(i, i < n ? __ldg(score + i) : 0.0f);
    }
  }
  for (int i = tid; i < kBins; i += THREADS) hist[i] = 0;
  __syncthreads();
  uint32_t prefix = 0, want = (uint32_t)k;               // T's digits so far, and the rank inside them
  uint32_t gt = 0, eq = 0;                               // keys over / equal to T in the slices before this one
#pragma unroll
  for (int d = 0; d < 3; ++d) {
    const int shift = digit_shift(d), bins = digit_bins(d);
    uint32_t *h = hist + digit_at(d), *gr = group + digit_at(d) / 32;
    for (int i0 = warp * 128; i0 < np; i0 += 4 * THREADS) { // whole warps: the votes below need all lanes
      uint32_t key[4];
      four(i0 + 4 * lane, key);
      bool in[4] = {true, true, true, true};
      if (d > 0) {                                       // keys whose higher digits are T's
#pragma unroll
        for (int j = 0; j < 4; ++j) in[j] = key[j] >> digit_shift(d - 1) == prefix;
        if (!__any_sync(0xffffffffu, in[0] || in[1] || in[2] || in[3])) continue;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) key[j] = (key[j] >> shift) & (bins - 1);
      // long runs of one score (zeros) would serialise on one counter: count such a group at once
      if (d == 0 || __all_sync(0xffffffffu, in[0] && in[1] && in[2] && in[3])) {
        const uint32_t first = __shfl_sync(0xffffffffu, key[0], 0);
        const uint32_t other = (key[0] ^ first) | (key[1] ^ first) | (key[2] ^ first) | (key[3] ^ first);
        if (__all_sync(0xffffffffu, other == 0)) {
          if (lane == 0) atomicAdd(h + first, 128u);
          continue;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (in[j]) atomicAdd(h + key[j], 1u);
    }
    __syncthreads();
    // sums of the groups of 32 bins: the search below reads these and then 32 bins from every slice, not the
    // whole histograms (8 KB from each of eight CTAs and digit over the cluster's network: 3 to 5 thousand cycles)
    {
      const int own = bins / THREADS;                    // neighbouring bins of a thread, a power of two
      uint32_t c = 0;
      for (int j = 0; j < own; ++j) c += h[own * tid + j];
      for (int m = 1; m < 32 / own; m <<= 1) c += __shfl_xor_sync(0xffffffffu, c, m);
      if (own * tid % 32 == 0) gr[own * tid / 32] = c;
    }
    cl.sync();                                           // every slice is counted
    if (warp == 0) {
      uint32_t above = 0, at;
      int g;
      // (the slices' words are asked for together: one latency, not eight)
      if (d == 0) {
        uint32_t c[4] = {}, b[4] = {};                   // 128 groups, else 32
        uint4 v[RANKS];
#pragma unroll
        for (int r = 0; r < RANKS; ++r) v[r] = reinterpret_cast<const uint4 *>(cl.map_shared_rank(gr, min(r, ranks - 1)))[lane];
#pragma unroll
        for (int r = 0; r < RANKS; ++r) {
          const uint32_t w[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            c[j] += r < ranks ? w[j] : 0;
            b[j] += r < rank ? w[j] : 0;
          }
        }
        g = find_bin(c, b, want, lane, above, gt, at);
      } else {
        uint32_t c[1] = {}, b[1] = {}, v[RANKS];
#pragma unroll
        for (int r = 0; r < RANKS; ++r) v[r] = cl.map_shared_rank(gr, min(r, ranks - 1))[lane];
#pragma unroll
        for (int r = 0; r < RANKS; ++r) {
          c[0] += r < ranks ? v[r] : 0;
          b[0] += r < rank ? v[r] : 0;
        }
        g = find_bin(c, b, want, lane, above, gt, at);
      }
      uint32_t c[1] = {}, b[1] = {}, v[RANKS];
#pragma unroll
      for (int r = 0; r < RANKS; ++r) v[r] = cl.map_shared_rank(h, min(r, ranks - 1))[32 * g + lane];
#pragma unroll
      for (int r = 0; r < RANKS; ++r) {
        c[0] += r < ranks ? v[r] : 0;
        b[0] += r < rank ? v[r] : 0;
      }
      const int bin = 32 * g + find_bin(c, b, want, lane, above, gt, at);
      if (lane == 0) {
        res[0] = bin;
        res[1] = want - above;
        res[2] = gt;
        res[3] = at;
      }
    }
    __syncthreads();
    if (d == 2) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // the last remote reads
    prefix = d == 0 ? res[0] : prefix * bins + res[0];
    want = res[1];
  }
  gt = res[2];
  eq = res[3];
  // `want` of the keys equal to T stay, in order. Mostly a slice keeps all of its own or none: then what it keeps
  // are its keys from a bound on. Warps take sub-slices in order: each counts what it keeps, and writes behind those
  // before it.
  const int sub = ((n + WARPS - 1) / WARPS + 127) / 128 * 128;
  const int w0 = min(np, warp * sub), w1 = min(np, w0 + sub);
  const uint32_t own = hist[digit_at(2) + (prefix & (digit_bins(2) - 1))];   // the slice's keys equal to T
  const uint32_t stay = eq >= want ? 0 : min(own, want - eq);
  const uint32_t bound = stay == 0 ? prefix + 1 : prefix;
  const bool some = stay > 0 && stay < own;              // (the same for the whole CTA)
  uint32_t ng = 0, ne = 0;
#pragma unroll 2
  for (int i = w0 + 4 * lane; i < w1; i += 128) {
    uint32_t key[4];
    four(i, key);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ng += key[j] >= bound;
      if (some) ne += key[j] == prefix;
    }
  }
  ng = __reduce_add_sync(0xffffffffu, ng);
  ne = __reduce_add_sync(0xffffffffu, ne);
  if (lane == 0) {
    wcount[warp] = ng;
    wcount[WARPS + warp] = ne;
  }
  __syncthreads();
  keep += a.n_sink;
  uint32_t at = gt + min(eq, want) + __reduce_add_sync(0xffffffffu, lane < warp ? wcount[lane] : 0);
  auto key_at = [&](int i) -> uint32_t {
    if constexpr (RESIDENT) return keys[i];
    else return key_of(i, i < n ? __ldg(score + i) : 0.0f);
  };
  const unsigned below = (1u << lane) - 1u;
  if (!some) {
#pragma unroll 4
    for (int i = w0 + lane; i < w1; i += 32) {
      const bool in = key_at(i) >= bound;
      const unsigned m = __ballot_sync(0xffffffffu, in);
      if (in) keep[at + __popc(m & below)] = s0 + i;
      at += __popc(m);
    }
  } else {                                               // the first `stay` of the keys equal to T
    uint32_t rank_eq = __reduce_add_sync(0xffffffffu, lane < warp ? wcount[WARPS + lane] : 0);
    at -= rank_eq - min(rank_eq, stay);                   // (the counts took all of them)
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint32_t key = key_at(i);
      const unsigned me = __ballot_sync(0xffffffffu, key == prefix);
      const bool in = key > prefix || (key == prefix && rank_eq + __popc(me & below) < stay);
      const unsigned m = __ballot_sync(0xffffffffu, in);
      if (in) keep[at + __popc(m & below)] = s0 + i;
      at += __popc(m);
      rank_eq += __popc(me);
    }
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // no CTA leaves while another reads its counts
}

// ------------------------------------------------------------------------------------ compaction
constexpr int kMoveThreads = 512;
constexpr int kMoveUnits = 4;                            // 16-byte units of the payload per thread and round

// Rows of one plane of one (batch, kv head).
template <bool PAGED>
struct PlaneRows {
  uint8_t *base;                                         // contiguous: row 0 of the (batch, kv head); else the pool
  int row_bytes;
  template <class U>
  __device__ __forceinline__ U *at(size_t row, int byte) const {
    return reinterpret_cast<U *>(base + (unsigned long long)row * (unsigned)row_bytes + byte);
  }
};
template <bool PAGED>
__device__ __forceinline__ PlaneRows<PAGED> plane_rows(const CacheView &c, void *plane, int row_bytes, int b, int kvh) {
  uint8_t *p = static_cast<uint8_t *>(plane);
  if constexpr (!PAGED) p += ((size_t)b * c.H + kvh) * c.cap * row_bytes;
  return {p, row_bytes};
}
// Row of token t in those planes.
template <bool PAGED>
__device__ __forceinline__ size_t plane_row(const CacheView &c, int b, int kvh, int t) {
  if constexpr (PAGED) return cache_row_paged(c, b, kvh, t);
  else return (unsigned)t;
}

// Source token of target row `row`, or -1: leave the row as it is.
template <bool IN_PLACE>
__device__ __forceinline__ int source_of(const int32_t *keep, int row, int new_len, int L) {
  if (row >= new_len) return -1;
  const int t = __ldg(keep + row);
  return (unsigned)t >= (unsigned)L || (IN_PLACE && t == row) ? -1 : t;
}

// What one thread moves in a round: up to four 16-byte units of the payload (its column of four rows, `step`
// rows apart) and the scales and zero-points (U) of up to two whole rows of the same block.
template <class U>
struct Moved {
  uint4 v[kMoveUnits];
  U scale[2], zero[2];
};

// Target rows [0, new_len) of one plane. Rounds cover `step` * 4 rows of all the ranks' CTAs. Into another
// cache every CTA moves its own rounds. In place the ranks' CTAs are one cluster whose rounds are ordered by
// its barrier.
template <class U, bool IN_PLACE, bool PAGED>
__device__ __forceinline__ void move_plane(const CompactArgs &a, int plane, int b, int kvh, int new_len, int L, int rank) {
  const int bytes = plane ? a.src.v_row_bytes : a.src.row_bytes;
  const int upr = bytes / 16, rpp = kMoveThreads / upr;  // threads per row, rows per pass
  const int own = (int)threadIdx.x / upr, col = 16 * ((int)threadIdx.x - own * upr);
  const int32_t *keep = a.keep + ((size_t)b * a.src.H + kvh) * a.n_keep;
  const auto src = plane_rows<PAGED>(a.src, a.src.payload[plane], bytes, b, kvh);
  const auto dst = plane_rows<PAGED>(a.dst, a.dst.payload[plane], bytes, b, kvh);
  const auto src_s = plane_rows<PAGED>(a.src, a.src.scale[plane], sizeof(U), b, kvh);
  const auto dst_s = plane_rows<PAGED>(a.dst, a.dst.scale[plane], sizeof(U), b, kvh);
  const bool zeros = (plane ? a.src.v_layout : a.src.layout) == KVQ_ASYM4_G32;
  const auto src_z = plane_rows<PAGED>(a.src, zeros ? a.src.zero[plane] : nullptr, sizeof(U), b, kvh);
  const auto dst_z = plane_rows<PAGED>(a.dst, zeros ? a.dst.zero[plane] : nullptr, sizeof(U), b, kvh);
  const int step = a.ranks * rpp, round = step * kMoveUnits;
  constexpr int kFar = 1 << 30;                          // no such row
  const int row0 = own < rpp ? rank * rpp + own : kFar;  // (threads beyond the last whole row idle)
  // scale row k of this thread: row (tid + 512 k) of the CTA's rpp * 4 rows of a round
  int srow[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = (int)threadIdx.x + kMoveThreads * k, pass = i / rpp;
    srow[k] = pass < kMoveUnits ? pass * step + rank * rpp + (i - pass * rpp) : kFar;
  }
  auto look = [&](int base, int (&st)[kMoveUnits], int (&ss)[2]) {
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u) st[u] = source_of<IN_PLACE>(keep, row0 + base + u * step, new_len, L);
#pragma unroll
    for (int k = 0; k < 2; ++k) ss[k] = source_of<IN_PLACE>(keep, srow[k] + base, new_len, L);
  };
  auto read = [&](const int (&st)[kMoveUnits], const int (&ss)[2], Moved<U> &m) {
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u)
      if (st[u] >= 0) m.v[u] = __ldcg(src.template at<uint4>(plane_row<PAGED>(a.src, b, kvh, st[u]), col));
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (ss[k] >= 0) {
        const size_t r = plane_row<PAGED>(a.src, b, kvh, ss[k]);
        m.scale[k] = __ldcg(src_s.template at<U>(r, 0));
        if (zeros) m.zero[k] = __ldcg(src_z.template at<U>(r, 0));
      }
  };
  auto write = [&](int base, const int (&st)[kMoveUnits], const int (&ss)[2], const Moved<U> &m) {
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u)
      if (st[u] >= 0) *dst.template at<uint4>(plane_row<PAGED>(a.dst, b, kvh, row0 + base + u * step), col) = m.v[u];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (ss[k] >= 0) {
        const size_t r = plane_row<PAGED>(a.dst, b, kvh, srow[k] + base);
        *dst_s.template at<U>(r, 0) = m.scale[k];
        if (zeros) *dst_z.template at<U>(r, 0) = m.zero[k];
      }
  };
  if constexpr (!IN_PLACE) {
    for (int base = 0; base < new_len; base += round) {
      int st[kMoveUnits], ss[2];
      Moved<U> m;
      look(base, st, ss);
      read(st, ss, m);
      write(base, st, ss, m);
    }
  } else {
    int st[kMoveUnits], ss[2];
    Moved<U> m = {};
    look(0, st, ss);
    for (int base = 0; base < new_len; base += round) {
      read(st, ss, m);
      // This round's values have been read before any CTA of the cluster writes over their rows.
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      write(base, st, ss, m);
      look(base + round, st, ss);
    }
  }
}

// The scores: moved likewise, and zero behind the kept ones, ready for the tokens appended next.
template <bool IN_PLACE>
__device__ __forceinline__ void move_scores(const CompactArgs &a, int b, int kvh, int new_len, int L, int rank) {
  const size_t head = (size_t)b * a.src.H + kvh;
  const int32_t *keep = a.keep + head * a.n_keep;
  const float *src = a.scores + head * (size_t)a.scores_stride;
  float *dst = a.scores_out + head * (size_t)a.out_stride;
  const int n = (int)min((long long)a.kv_len, a.out_stride), step = a.ranks * kMoveThreads, round = step * kMoveUnits;
  for (int base = 0; base < n; base += round) {
    float v[kMoveUnits];
    int st[kMoveUnits];
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u) {
      st[u] = source_of<IN_PLACE>(keep, base + u * step + rank * kMoveThreads + (int)threadIdx.x, new_len, L);
      v[u] = 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u)
      if (st[u] >= 0) v[u] = __ldcg(src + st[u]);
    if constexpr (IN_PLACE) {                            // as in move_plane
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
#pragma unroll
    for (int u = 0; u < kMoveUnits; ++u) {
      const int row = base + u * step + rank * kMoveThreads + (int)threadIdx.x;
      if (st[u] >= 0 || (row >= new_len && row < n)) dst[row] = v[u];
    }
  }
}

// Grid: (ranks * heads, K plane, V plane and scores).
template <class U, bool IN_PLACE, bool PAGED>
__global__ void __launch_bounds__(kMoveThreads, 2) evict_move_kernel(CompactArgs a) {
  const int bh = blockIdx.x / a.ranks, b = bh / a.src.H, kvh = bh - b * a.src.H, rank = blockIdx.x - bh * a.ranks;
  const int L = a.seq_lens ? min(max(__ldg(a.seq_lens + b), 0), a.kv_len) : a.kv_len;
  const int new_len = min(L, a.n_keep);
  if (blockIdx.y == 2) move_scores<IN_PLACE>(a, b, kvh, new_len, L, rank);
  else move_plane<U, IN_PLACE, PAGED>(a, blockIdx.y, b, kvh, new_len, L, rank);
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

template <int THREADS, int RANKS, bool RESIDENT, class Source>
cudaError_t launch_select(const SelectArgs &a, const Source &src, int ranks, int keys, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  auto kernel = evict_select_kernel<THREADS, RANKS, RESIDENT, Source>;
  cudaError_t e = set_smem_once(done, kernel, Source::D > 0 ? kBlockSelectSmem : 227 * 1024);
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
  return cudaLaunchKernelEx(&cfg, kernel, a, src);
}

}  // namespace

cudaError_t launch_evict_select(const SelectArgs &a, cudaStream_t st) {
  // CTAs per (batch, kv head): one per 8192 tokens, at most the portable cluster size of 8
  int ranks = 1;
  while (ranks < 8 && (long long)ranks * 8192 < a.kv_len) ranks *= 2;
  const int keys = ((a.kv_len + ranks - 1) / ranks + 31 + 127) / 128 * 128;
  if (keys > kSelMaxKeys) return launch_select<1024, 8, false>(a, ScoresInMemory{}, ranks, 0, st);
  // rows of one CTA: half the threads, two CTAs per SM
  return ranks == 1 ? launch_select<512, 1, true>(a, ScoresInMemory{}, ranks, keys, st)
                    : launch_select<1024, 8, true>(a, ScoresInMemory{}, ranks, keys, st);
}

cudaError_t launch_block_select(const BlockSelectArgs &b, cudaStream_t st) {
  const int lists = b.cache.B * b.cache.H * b.n_q, blocks = (int)(((long long)b.kv_len + 63) / 64);
  // CTAs per list: one per 128 blocks (the scores of as many are one pass of its threads) where all are resident at once (two
  // per SM), and at most 8192 blocks each (2048 blocks, 8 lists, with the bounds in front: 57.5 us with eight CTAs, 78.2 with one)
  int ranks = 1;
  while (ranks < 8 && (ranks * 8192LL < blocks || (ranks * 128 < blocks && ranks * lists <= sm_count()))) ranks *= 2;
  const int keys = ((blocks + ranks - 1) / ranks + 31 + 127) / 128 * 128;
  const SelectArgs a = {lists, 1, blocks, b.n_sel, b.n_sink, b.n_recent, 0, nullptr, nullptr, b.sel, nullptr};
  return b.cache.D == 128 ? launch_select<512, 8, true>(a, ScoresOfBlocks<128>{b}, ranks, keys, st)
                          : launch_select<512, 8, true>(a, ScoresOfBlocks<256>{b}, ranks, keys, st);
}

namespace {

template <class U>
cudaError_t launch_move(CompactArgs &a, bool in_place, cudaStream_t st) {
  const int heads = a.src.B * a.src.H, most = a.n_keep < a.kv_len ? a.n_keep : a.kv_len;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = st;
  const unsigned parts = a.scores ? 3 : 2;
  if (!in_place) {
    // nothing waits: one round per CTA for the widest rows, the scheduler overlaps them
    const int upr = (a.src.row_bytes > a.src.v_row_bytes ? a.src.row_bytes : a.src.v_row_bytes) / 16;
    const int round = kMoveThreads / upr * kMoveUnits;
    a.ranks = min((most + round - 1) / round, max(1, (1 << 16) / heads));
    cfg.gridDim = dim3((unsigned)a.ranks * heads, parts);
    return cudaLaunchKernelEx(&cfg, evict_move_kernel<U, false, false>, a);
  }
  // one cluster per plane of a (batch, kv head), at most the portable 8 CTAs, as many as are resident at once
  // (two per SM over the two planes): a CTA's rounds overlap better than CTAs that follow one another
  const int want = max(1, device_sms() / heads);
  a.ranks = 1;
  while (a.ranks < 8 && 2 * a.ranks <= want) a.ranks *= 2;
  cfg.gridDim = dim3((unsigned)a.ranks * heads, parts);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.src.page_shift >= 0 ? cudaLaunchKernelEx(&cfg, evict_move_kernel<U, true, true>, a)
                               : cudaLaunchKernelEx(&cfg, evict_move_kernel<U, true, false>, a);
}

}  // namespace

cudaError_t launch_evict_compact(CompactArgs a, bool in_place, cudaStream_t st) {
  // the scales of a row: one f32, or D / 32 f16
  const cudaError_t e = is_hadamard(a.src.layout) ? launch_move<uint32_t>(a, in_place, st)
                        : a.src.D == 128          ? launch_move<uint2>(a, in_place, st)
                                                  : launch_move<uint4>(a, in_place, st);
  if (e != cudaSuccess || a.src.n_recent == 0) return e;
  evict_ring_kernel<<<dim3(a.src.B * a.src.H, 2, a.src.D / 32), kRingThreads, 0, st>>>(a, in_place ? 1 : 0);
  return cudaGetLastError();
}

}  // namespace kvq
