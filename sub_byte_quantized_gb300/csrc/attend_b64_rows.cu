// Phase 1 of the attention over the 8-bit block layouts for many query rows of a kv head (prompts, long speculative runs),
// head_dim 128: 128 rows per CTA, 16 for each of eight warps, over blocks of 64 tokens.
//
//   x = alpha log2(e) s_k (q . c),  p = 2^(x - m),  o += s_v (p . v)     as in attend_b64.cu, with the same exactness
// Here the rows are on the M side of mma.sync.m16n8k16 and a warp holds its rows' queries, scores and outputs in registers: a
// score's accumulator is the A operand of the product with V as it stands. A block's codes become f16 once for all 128 rows,
// in shared memory: each thread turns the codes that it read a block ahead into the next of three buffers, whose barriers let
// warps run up to a block apart, so that one's softmax meets another's products. Rows of 256 bytes with an XOR swizzle of their 16-byte columns, so that ldmatrix (plain for K, transposed for V) is free of
// bank conflicts. No warp needs another's state: partials are written from registers.
//
// Work is dealt out as in attend_b64.cu, with groups of 128 rows.
//
// Bound: the tensor cores' rate for mma.sync and its operands from shared memory (per 64 tokens and warp 64 products for the
// scores, 128 for both parts of p, 64 ldmatrix of 512 bytes).
// 256 rows x 8 sequences over 4096 tokens, 8 kv heads: 301 us with the join (298 where a wait that gave up marked its own warp alone),
// the tensor pipe 61 % busy.
#include "attend_b64.cuh"

namespace kvq {
namespace {
using namespace mma;
using namespace b64;

constexpr int kThreads = 256, kRows = kB64ManyRows;
constexpr int kD = 128, kKS = kD / 16;
constexpr int kTile = 64 * kD * 2;                       // bytes of one plane of a block in f16
constexpr int kBuffers = 3;
constexpr int kSmem = 2 * kBuffers * kTile + 64;       // and a barrier pair per buffer

// 16-byte column j of token row `row` of a tile.
__device__ __forceinline__ uint32_t swz(int row, int j) { return (uint32_t)(row * 256 + ((j ^ (row & 7)) << 4)); }

template <bool E4M3, bool QSPLIT, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) attend_b64_rows_kernel(AttendArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
#if defined(__CUDA_ARCH__) && __CUDA_ARCH__ >= 900
  asm volatile("griddepcontrol.launch_dependents;");
#endif
  const CacheView &cv = a.cache;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3, mi = lane >> 3;
  const int R = a.gqa * a.n_q, groups = (R + kRows - 1) / kRows, heads = cv.H * groups;
#if defined(__CUDA_ARCH__) && __CUDA_ARCH__ >= 900
  if (PAGED && a.fresh_tail == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
#endif
  const Deal deal = deal_of<PAGED>(a, heads, lane);
  Walk<PAGED> walk(a, deal, heads, lane);
  Span &sp = walk.sp;
  if (sp.n == 0) {
    pdl_wait_if(false);
    return;
  }
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + 2 * kBuffers * kTile), *empty = full + kBuffers;
  volatile int *gave_up = reinterpret_cast<int *>(empty + kBuffers);
  if (tid == 0) {
    *gave_up = 0;
#pragma unroll
    for (int k = 0; k < 2 * kBuffers; ++k) bar_init(full + k, kThreads / 32);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  walk.wait_for_append(a);
  // Block number `it` of the CTA lies in buffer it % kBuffers, for the (it / kBuffers)-th time. Waits are bounded: a warp whose wait
  // gives up goes on without waiting, and may then write over a block that another warp still reads. It says so before it writes
  // anything more, so a warp that has read such bytes finds `gave_up` set when it leaves its rows behind: they are NaN, as
  // are all that the CTA leaves from then on. Rows left before were read from whole blocks.
  int it = 0;
  bool failed = false;
  auto wait = [&](uint64_t *bar, int times) {
    if (!failed && !bar_wait(bar, (uint32_t)(times & 1))) failed = true;
  };
  auto arrive = [&](uint64_t *bar) {
    __syncwarp();
    if (lane == 0) bar_arrive(bar);
  };

  for (; sp.n > 0; walk.advance(a, heads)) {
    const int kvh = sp.hd / groups, row0 = kRows * (sp.hd - kvh * groups), wrow = row0 + 16 * warp;   // the warp's first row
    SeqLen sl;
    sl.kv_len = sp.len;
    sl.q_pos0 = PAGED ? sp.len - a.n_q : a.q_pos0;
    // blocks that some row of the CTA sees
    const int seen = max_row_limit(a, sl, row0, min(R, row0 + kRows));
    const int n = seen < 0 ? 0 : min(sp.n, (seen >> 6) - sp.blk + 1);
    const size_t head_row0 = ((size_t)sp.b * cv.H + kvh) * cv.cap;

    // (Plain loads: the append in front of this grid may write while it is already running, a scale next to one that another
    // CTA has read. The read-only path is for what nobody writes.)
    // A thread's codes: 16-byte pieces tid and tid + 256 of each plane (token p / 8, column p % 8), and the block's scales.
    uint4 raw[4];
    float2 sc = make_float2(0.0f, 0.0f), sc_next = sc;   // scales of the block computed from, and of the codes at hand
    auto fetch = [&](int i) {
      if (i >= n) return;
      const int t0 = 64 * (sp.blk + i);
      const size_t r = cache_row_t<PAGED>(cv, sp.b, kvh, head_row0, t0);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int p = tid + kThreads * k;
        const bool ok = t0 + p / 8 < sp.len;             // rows behind the sequence: codes 0
        raw[k] = ok ? reinterpret_cast<const uint4 *>(cv.payload[0] + r * kD)[p] : make_uint4(0u, 0u, 0u, 0u);
        raw[2 + k] = ok ? reinterpret_cast<const uint4 *>(cv.payload[1] + r * kD)[p] : make_uint4(0u, 0u, 0u, 0u);
      }
      sc_next = make_float2(static_cast<const float *>(cv.scale[0])[r >> 6], static_cast<const float *>(cv.scale[1])[r >> 6]);
    };
    auto convert = [&](int buffer) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int p = tid + kThreads * (k & 1), row = p >> 3, j = 2 * (p & 7);
        uint8_t *tile = smem + (2 * buffer + (k >> 1)) * kTile;
        uint32_t f[8];
        codes_f16<E4M3, false>(raw[k].x, f[0], f[1]);
        codes_f16<E4M3, false>(raw[k].y, f[2], f[3]);
        codes_f16<E4M3, false>(raw[k].z, f[4], f[5]);
        codes_f16<E4M3, false>(raw[k].w, f[6], f[7]);
        *reinterpret_cast<uint4 *>(tile + swz(row, j)) = make_uint4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<uint4 *>(tile + swz(row, j + 1)) = make_uint4(f[4], f[5], f[6], f[7]);
      }
    };
    fetch(0);

    // the warp's queries: rows wrow + g and wrow + g + 8, dims 16 j + 2c, + 1 and + 8, + 9; a power of two per row
    uint32_t qh[kKS][4], ql[QSPLIT ? kKS : 1][4];
    float alpha[2];
    int lim[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = wrow + g + 8 * k;
      const bool live = r < R && r < row0 + kRows;
      const size_t at = query_row_index(a, sp.b, kvh, live ? r : row0) * kD + 2 * c;
      lim[k] = live ? row_limit(a, sl, r % a.n_q) : -1;
      float x[kKS][4], mx = 0.0f;
#pragma unroll
      for (int j = 0; j < kKS; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const size_t e = at + 16 * j + 8 * h;
          float2 v;
          if constexpr (QSPLIT) {
            v = __ldg(reinterpret_cast<const float2 *>(static_cast<const float *>(a.q) + e));
          } else {
            const uint32_t u = __ldg(reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(a.q) + e));
            v = a.q_dtype == KVQ_BF16 ? make_float2(bf16_bits_to_f32(u & 0xFFFFu), bf16_bits_to_f32(u >> 16)) : __half22float2(u32_as_h2(u));
          }
          x[j][2 * h] = live ? v.x : 0.0f;
          x[j][2 * h + 1] = live ? v.y : 0.0f;
          mx = fmaxf(mx, fmaxf(fabsf(x[j][2 * h]), fabsf(x[j][2 * h + 1])));
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      int e = 0;                                         // the row's largest |q| goes to [2^13, 2^14)
      if (mx > 0.0f) e = min(max(((__float_as_int(mx) >> 23) & 0xFF) - 127 - 13, -100), 100);
      const float pre = ldexpf(1.0f, -e);
      alpha[k] = a.scale * ldexpf(1.0f, e) * kLog2e;
#pragma unroll
      for (int j = 0; j < kKS; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float u = x[j][2 * h] * pre, v = x[j][2 * h + 1] * pre;
          const float uh = __half2float(__float2half_rn(u)), vh = __half2float(__float2half_rn(v));
          qh[j][k + 2 * h] = pack_f16x2(uh, vh);
          if constexpr (QSPLIT) ql[j][k + 2 * h] = pack_f16x2(u - uh, v - vh);
        }
    }
    const bool work = wrow < R;                          // (the same for the warp)
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, O[kKS * 2][4];
#pragma unroll
    for (int j = 0; j < 2 * kKS; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) O[j][k] = 0.0f;

    float2 sc_then = sc;
    auto prepare = [&](int i) {                          // block i of the span, whose codes have been read, and the read of the next
      const int at = it + i, buffer = at % kBuffers;
      if (at >= kBuffers) wait(empty + buffer, at / kBuffers - 1);
      if (failed) {
        *gave_up = 1;
        __threadfence_block();
      }
      convert(buffer);
      arrive(full + buffer);
      sc_then = sc_next;
      fetch(i + 1);
    };
    if (n > 0) prepare(0);
    for (int i = 0; i < n; ++i) {
      sc = sc_then;
      if (i + 1 < n) prepare(i + 1);
      const int buffer = (it + i) % kBuffers;
      wait(full + buffer, (it + i) / kBuffers);
      if (work) {
        const uint32_t sK = smem_addr(smem + 2 * buffer * kTile), sV = sK + kTile;
        const int t0 = 64 * (sp.blk + i);
        const float f[2] = {alpha[0] * sc.x, alpha[1] * sc.x};
        // scores: s[t][k] is token t0 + 8 t + 2c + (k & 1), row g + 8 (k >> 1)
        float s[8][4] = {};
        bool rise = false;
#pragma unroll
        for (int j = 0; j < kKS; ++j)                    // eight chains of products
#pragma unroll
          for (int t = 0; t < 8; t += 2) {               // matrices: tokens 8t .. (dims 16j, + 8), tokens 8(t + 1) .. (the same)
            uint32_t b[4];
            ldsm_x4(sK + swz(8 * t + 8 * (mi >> 1) + (lane & 7), 2 * j + (mi & 1)), b);
            mma16816(s[t], qh[j], b[0], b[1]);
            mma16816(s[t + 1], qh[j], b[2], b[3]);
            if constexpr (QSPLIT) {
              mma16816(s[t], ql[j], b[0], b[1]);
              mma16816(s[t + 1], ql[j], b[2], b[3]);
            }
          }
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int tok = t0 + 8 * t + 2 * c + (k & 1);
            s[t][k] = tok <= lim[k >> 1] ? s[t][k] * f[k >> 1] : -INFINITY;
            rise = rise || s[t][k] > m[k >> 1] + kRise;
          }
        // the reference follows the maximum only where a score passes it by kRise (attend_b64.cu)
        if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float mx = m[k];
#pragma unroll
            for (int t = 0; t < 8; ++t) mx = fmaxf(mx, fmaxf(s[t][2 * k], s[t][2 * k + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float corr = m[k] == -INFINITY ? 0.0f : ex2(m[k] - mx);
            m[k] = mx;
            l[k] *= corr;
#pragma unroll
            for (int j = 0; j < 2 * kKS; ++j) {
              O[j][2 * k] *= corr;
              O[j][2 * k + 1] *= corr;
            }
          }
        }
        const float base[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
        uint32_t ph[4][4], pl[4][4];                     // A operands of 16 tokens each
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float u = ex2(s[t][2 * k] - base[k]), v = ex2(s[t][2 * k + 1] - base[k]);
            l[k] += u + v;
            const float uh = __half2float(__float2half_rn(u * 4096.0f)), vh = __half2float(__float2half_rn(v * 4096.0f));
            ph[t >> 1][k + 2 * (t & 1)] = pack_f16x2(uh, vh);
            pl[t >> 1][k + 2 * (t & 1)] = pack_f16x2(fmaf(u, 4096.0f, -uh), fmaf(v, 4096.0f, -vh));
          }
        const float sv = sc.y * 0x1p-12f;
#pragma unroll
        for (int j = 0; j < 2 * kKS; j += 4) {           // dims 8 j .. 8 (j + 4)
          float acc[4][4] = {};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            uint32_t b[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) ldsm_x4_t(sV + swz(16 * t + 8 * (mi & 1) + (lane & 7), j + 2 * u + (mi >> 1)), b[u]);
#pragma unroll
            for (int u = 0; u < 4; ++u) mma16816(acc[u], ph[t], b[u >> 1][2 * (u & 1)], b[u >> 1][2 * (u & 1) + 1]);
#pragma unroll
            for (int u = 0; u < 4; ++u) mma16816(acc[u], pl[t], b[u >> 1][2 * (u & 1)], b[u >> 1][2 * (u & 1) + 1]);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) O[j + u][k] = fmaf(acc[u][k], sv, O[j + u][k]);
        }
      }
      arrive(empty + buffer);
    }
    it += max(n, 0);
    const size_t head = (size_t)sp.b * heads + sp.hd, part = (size_t)blockIdx.x + head;
    if (work) {
      const bool lost = failed || *gave_up;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
        const int r = wrow + g + 8 * k;
        if (r < R) {
          const size_t p = part * kRows + (r - row0);
#pragma unroll
          for (int j = 0; j < 2 * kKS; ++j)
            *reinterpret_cast<float2 *>(a.part_o + p * kD + 8 * j + 2 * c) = make_float2(O[j][2 * k], O[j][2 * k + 1]);
          if (c == 0) {
            a.part_m[p] = m[k];
            a.part_l[p] = lost ? __int_as_float(0x7FC00000) : l[k];
          }
        }
      }
    }
    if (sp.blk == 0 && tid == 0) a.spans[head] = walk.ctas_of_head(deal);
  }
}

template <bool E4M3, bool QSPLIT, bool PAGED>
cudaError_t launch_t(const AttendArgs &a, cudaStream_t st) {
  static std::atomic<bool> configured[kMaxDevices];
  auto kernel = attend_b64_rows_kernel<E4M3, QSPLIT, PAGED>;
  const cudaError_t e = set_smem_once(configured, kernel, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  chained(cfg, attr, a.grid, kThreads, kSmem, st);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}
template <bool E4M3>
cudaError_t launch_e(const AttendArgs &a, cudaStream_t st) {
  const bool paged = a.cache.page_shift >= 0;
  if (a.q_dtype == KVQ_F32) return paged ? launch_t<E4M3, true, true>(a, st) : launch_t<E4M3, true, false>(a, st);
  return paged ? launch_t<E4M3, false, true>(a, st) : launch_t<E4M3, false, false>(a, st);
}

}  // namespace

cudaError_t launch_attend_b64_rows(const AttendArgs &a, cudaStream_t st) {
  return a.cache.layout == KVQ_E4M3_B64 ? launch_e<true>(a, st) : launch_e<false>(a, st);
}

}  // namespace kvq
