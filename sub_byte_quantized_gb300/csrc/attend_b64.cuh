// What the attention kernels over the 8-bit block layouts share: how a call's blocks are dealt out to the CTAs, and codes as f16.
#pragma once

#include "kvq_internal.cuh"
#include "mma_util.cuh"

namespace kvq {
namespace b64 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRise = 3.9f;            // 2^(12 + 3.9) < 65504
// What a CTA pays for a second head, in units: a piece may be so much longer than an even share.
constexpr int kSlack = 5;

// Two codes each -> exact f16 pairs. K: bytes (0, 1) and (2, 3) of a word; V: bytes (0, 2) and (1, 3).
template <bool E4M3, bool V>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t &a, uint32_t &b) {
  if constexpr (E4M3) {
    if (V) w = mma::prmt(w, 0u, 0x3120u);
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}\n" : "=r"(a), "=r"(b) : "r"(w));
  } else {                                               // the code plus 128 under the exponent of 1024, less 1152
    const uint32_t x = w ^ 0x80808080u;
    a = mma::hadd2(mma::prmt(x, 0x64646464u, V ? 0x4240u : 0x4140u), 0xE480E480u);
    b = mma::hadd2(mma::prmt(x, 0x64646464u, V ? 0x4341u : 0x4342u), 0xE480E480u);
  }
}

// Where a run of units stands: sequence b, head `hd` of it (kv head * groups + group), its blocks [blk, blk + n).
struct Span {
  int b, hd, blk, n, len;      // len: tokens of the sequence that some row sees
};
// Tokens of sequence b that the call looks at.
template <bool PAGED>
__device__ __forceinline__ int seen_len(const AttendArgs &a, int b) {
  if constexpr (PAGED) return min(max(__ldg(a.seq_lens + b), 0), a.kv_len);
  else return a.causal ? min(a.kv_len, a.q_pos0 + a.n_q) : a.kv_len;
}
__device__ __forceinline__ int blocks_of(int len) { return (int)(((long long)len + 63) >> 6); }
__device__ __forceinline__ int pieces_of(int blocks, int per) { return (blocks + per - 1) / per; }
__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// How a call's units are dealt out (by one warp).
struct Deal {
  long long per;               // units a CTA
  bool pieces;                 // a CTA has one piece of one head
};
template <bool PAGED>
__device__ __forceinline__ Deal deal_of(const AttendArgs &a, int heads, int lane) {
  if (a.per > 0) return {a.per, true};                   // the caller's chunk: its grid holds every piece
  const int B = a.cache.B;
  long long total = 0;
  if constexpr (PAGED) {
    for (int b = lane; b < B; b += 32) total += (long long)heads * blocks_of(seen_len<PAGED>(a, b));
    total = warp_sum(total);
  } else {
    total = (long long)B * heads * blocks_of(seen_len<PAGED>(a, 0));
  }
  const long long per = max(1LL, (total + gridDim.x - 1) / gridDim.x);
  if (per > INT_MAX - kSlack) return {per, false};
  long long n[kSlack] = {};                              // pieces of at most per + j units
  if constexpr (PAGED) {
    for (int b = lane; b < B; b += 32) {
      const int nb = blocks_of(seen_len<PAGED>(a, b));
#pragma unroll
      for (int j = 0; j < kSlack; ++j) n[j] += pieces_of(nb, (int)per + j);
    }
#pragma unroll
    for (int j = 0; j < kSlack; ++j) n[j] = warp_sum(n[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kSlack; ++j) n[j] = (long long)B * pieces_of(blocks_of(seen_len<PAGED>(a, 0)), (int)per + j);
  }
#pragma unroll
  for (int j = 0; j < kSlack; ++j)
    if (n[j] * heads <= gridDim.x) return {per + j, true};
  return {per, false};
}
// Weight of sequence b in the row of what is dealt out: its heads' pieces, or their units.
template <bool PAGED>
__device__ __forceinline__ long long share_of(const AttendArgs &a, const Deal &d, int heads, int b) {
  if (b >= a.cache.B) return 0;
  const int nb = blocks_of(seen_len<PAGED>(a, b));
  return (long long)heads * (d.pieces ? pieces_of(nb, (int)d.per) : nb);
}


// A CTA's way through its units: the first span, and the ones that follow it.
template <bool PAGED>
struct Walk {
  Span sp;
  long long u0, left;          // the first unit (or piece), and the units from the present span on
  __device__ __forceinline__ Walk(const AttendArgs &a, const Deal &deal, int heads, int lane) : sp{0, 0, 0, 0, 0}, left(0) {
    u0 = deal.pieces ? (long long)blockIdx.x : deal.per * blockIdx.x;
    long long before = 0;                                // what the sequences in front of sp.b weigh
    if constexpr (PAGED) {
      for (;; sp.b += 32) {
        const long long own = share_of<PAGED>(a, deal, heads, sp.b + lane);
        long long upto = own;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const long long o = __shfl_up_sync(0xffffffffu, upto, m);
          if (lane >= m) upto += o;
        }
        const unsigned over = __ballot_sync(0xffffffffu, before + upto > u0);
        if (over) {
          const int at = __ffs((int)over) - 1;
          before += __shfl_sync(0xffffffffu, upto - own, at);
          sp.b += at;
          break;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
        if (sp.b + 32 >= a.cache.B) return;              // nothing is left for this CTA
      }
    } else {
      const long long each = share_of<PAGED>(a, deal, heads, 0);
      if (u0 >= each * a.cache.B) return;
      sp.b = (int)(u0 / each);
      before = each * sp.b;
    }
    sp.len = seen_len<PAGED>(a, sp.b);
    const int nb = blocks_of(sp.len);
    if (deal.pieces) {                                   // a head in equal pieces
      const int n = pieces_of(nb, (int)deal.per), at = (int)(u0 - before), size = (nb + n - 1) / n;
      sp.hd = at / n;
      sp.blk = (at - sp.hd * n) * size;
      sp.n = max(0, min(size, nb - sp.blk));
      left = sp.n;
    } else {
      sp.hd = (int)((u0 - before) / nb);
      sp.blk = (int)((u0 - before) - (long long)sp.hd * nb);
      sp.n = (int)min(deal.per, (long long)nb - sp.blk);
      left = deal.per;                                   // (the last CTA's may end earlier: there is no head behind it)
    }
  }
  // the next head with tokens
  __device__ __forceinline__ void advance(const AttendArgs &a, int heads) {
    left -= sp.n;
    sp.n = 0;
    if (left <= 0) return;
    if (++sp.hd == heads) {
      sp.hd = 0;
      do {
        if (++sp.b == a.cache.B) return;
        sp.len = seen_len<PAGED>(a, sp.b);
      } while (sp.len <= 0);
    }
    sp.blk = 0;
    sp.n = (int)min(left, (long long)blocks_of(sp.len));
  }
  // Rows that the kernel before appends: CTAs that read them wait for it. (A CTA looks at its first head only where it has
  // one alone.)
  __device__ __forceinline__ void wait_for_append(const AttendArgs &a) const {
    int lo = a.fresh_lo, hi = a.fresh_hi;
    if (PAGED && a.fresh_tail > 0) lo = sp.len - a.fresh_tail, hi = sp.len;
    pdl_wait_if(left > sp.n || (64 * sp.blk < hi && lo < 64 * (sp.blk + sp.n)));
  }
  // First and last CTA of the head that begins with the present span.
  __device__ __forceinline__ int2 ctas_of_head(const Deal &deal) const {
    const int nb = blocks_of(sp.len);
    int last = (int)blockIdx.x;
    if (deal.pieces) {
      const int n = pieces_of(nb, (int)deal.per), size = (nb + n - 1) / n;
      last += pieces_of(nb, size) - 1;                   // (equal sizes may need fewer pieces than there is room for)
    } else {
      last = (int)((u0 + (deal.per - left) + nb - 1) / deal.per);
    }
    return make_int2((int)blockIdx.x, last);
  }
};

// A launch that may begin while the kernel before it still runs.
inline void chained(cudaLaunchConfig_t &cfg, cudaLaunchAttribute &attr, unsigned ctas, int threads, int smem, cudaStream_t st) {
  cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
}

}  // namespace b64
}  // namespace kvq
