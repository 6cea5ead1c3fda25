// Phase 1 of the split-K attention over the 8-bit block layouts (int8 or e4m3 codes, one f32 scale per 64 tokens, head
// and plane), head_dim 128 or 256, in groups of eight query rows of a kv head.
//
//   x_rt = alpha log2(e) s_k(block) sum_d q_rd c_td,  m_r = max_t x_rt,  p = 2^(x - m)
//   o_r += s_v(block) sum_t p_rt v_td   (v: the codes)
// with mma.sync.m16n8k16 (f16 in, f32 accumulate), tokens (QK) and dims (PV) on the M side, the eight rows on the N side:
//   S^T[16 tokens][8 rows] = C[16 tokens][16 dims] . q^T,   O^T[16 dims][8 rows] = V^T[16 dims][16 tokens] . P^T
// Exactness: both code types are exact in f16; bf16 and f16 queries are after a power-of-two factor per row, f32 ones
// are split into two f16 parts (22 bits). One scale per block means that no scale touches the operands: s_k goes into
// the row's factor, and every stage's PV product starts from zero and joins the output as o = o corr + s_v acc in f32,
// which also keeps the tensor cores' truncated additions short. The probabilities are taken 2^12 times larger, so that
// both f16 parts of p (p = hi + lo, 22 bits) stay above f16's subnormals for tokens of little weight.
//
// Data movement: each of a CTA's four warps streams a contiguous quarter of the chunk's stages (32 tokens at head_dim
// 128, 16 at 256: 8 KB for both planes) through its own ring with 16-byte cp.async; rows are placed with an XOR swizzle
// of their 16-byte columns, so that ldmatrix (plain for K: 4 codes of a token per lane; transposed for V: 2 dims of 2
// tokens) is free of bank conflicts. The warps' states are combined in shared memory, one partial per row and chunk.
//
// Bound: the packed cache's bytes from HBM.
#include <cfloat>

#include "kvq_internal.cuh"
#include "mma_util.cuh"

namespace kvq {
namespace {
using namespace mma;

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Cfg {
  static constexpr int STAGE = D == 128 ? 32 : 16;       // tokens
  static constexpr int RING = 2;
  static constexpr int PLANE = STAGE * D;                // bytes of one plane's rows
  static constexpr int BYTES = 2 * PLANE + 16;           // both planes, and the block's two scales
  static constexpr int CTAS = kB64CtasPerSm(D);
  static constexpr int SMEM = kWarps * RING * BYTES;
  static_assert(kWarps * 8 * (D + 2) * 4 <= SMEM, "the warps' states reuse the stages");
};

// 16-byte column j of row `row`.
template <int D>
__device__ __forceinline__ uint32_t swz(int row, int j) {
  return (uint32_t)(row * D + ((j ^ (row & 7)) << 4));
}
// Two codes each -> exact f16 pairs. K: bytes (0, 1) and (2, 3) of a word; V: bytes (0, 2) and (1, 3).
template <bool E4M3, bool V>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t &a, uint32_t &b) {
  if constexpr (E4M3) {
    if (V) w = prmt(w, 0u, 0x3120u);
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}\n" : "=r"(a), "=r"(b) : "r"(w));
  } else {                                               // the code plus 128 under the exponent of 1024, less 1152
    const uint32_t x = w ^ 0x80808080u;
    a = hadd2(prmt(x, 0x64646464u, V ? 0x4240u : 0x4140u), 0xE480E480u);
    b = hadd2(prmt(x, 0x64646464u, V ? 0x4341u : 0x4342u), 0xE480E480u);
  }
}

template <int D, bool E4M3, bool QSPLIT, bool PAGED>
__global__ void __launch_bounds__(kWarps * 32, Cfg<D>::CTAS) attend_b64_kernel(AttendArgs a) {
  using C = Cfg<D>;
  constexpr int KS = D / 16, TILES = C::STAGE / 16, CPR = D / 16;
  extern __shared__ __align__(1024) uint8_t smem[];
#if defined(__CUDA_ARCH__) && __CUDA_ARCH__ >= 900
  asm volatile("griddepcontrol.launch_dependents;");
#endif
  const CacheView &cv = a.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, mi = lane >> 3;
  const int bh = blockIdx.y, bb = bh / cv.H, kvh = bh - bb * cv.H;
  const SeqLen sl = seq_of_t<PAGED>(a, bb);
  const int row0 = blockIdx.z * 8, R = min(8, a.gqa * a.n_q - row0);
  const int t0 = blockIdx.x * sl.chunk, t1 = min(sl.n_body, t0 + sl.chunk);
  const int w_lim = max_row_limit(a, sl, row0, row0 + R);
  pdl_wait_if(t0 <= w_lim && t0 < sl.fresh_hi && sl.fresh_lo < min(t1, w_lim + 1));
  if (t0 > w_lim || t0 >= t1) return;                    // no row sees this chunk (phase 2 skips it)
  const int t_end = min(t1, w_lim + 1);
  const int n_stages = (t_end - t0 + C::STAGE - 1) / C::STAGE, spw = (n_stages + kWarps - 1) / kWarps;
  const int s_first = min(n_stages, warp * spw), n_mine = min(n_stages, s_first + spw) - s_first;
  const int tw0 = t0 + s_first * C::STAGE;

  uint8_t *ring = smem + warp * C::RING * C::BYTES;
  const size_t head_row0 = (size_t)bh * cv.cap;
  auto issue = [&](int i) {
    if (i < n_mine) {
      const int ts = tw0 + i * C::STAGE;
      const size_t r = cache_row_t<PAGED>(cv, bb, kvh, head_row0, ts);   // a stage lies in one block
      const uint8_t *kp = cv.payload[0] + r * D, *vp = cv.payload[1] + r * D;
      uint8_t *sb = ring + (i % C::RING) * C::BYTES;
      const uint32_t sK = smem_addr(sb), sV = sK + C::PLANE;
      const int live = (t_end - ts) * CPR;               // 16-byte pieces of rows in the chunk; the rest is zero-filled
#pragma unroll
      for (int k = 0; k < C::STAGE * CPR / 32; ++k) {
        const int q = lane + 32 * k, row = q / CPR, j = q % CPR;
        const bool ok = q < live;
        cp_async16(sK + swz<D>(row, j), kp + (ok ? 16 * q : 0), ok ? 16 : 0);
        cp_async16(sV + swz<D>(row, j), vp + (ok ? 16 * q : 0), ok ? 16 : 0);
      }
      if (lane < 2) cp_async4(sK + 2 * C::PLANE + 4 * lane, static_cast<const float *>(cv.scale[lane]) + (r >> 6), 4);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < C::RING; ++i) issue(i);

  // query fragments: row g, dims 16 j + 4 c + 0..3 (the k order in which ldmatrix hands out K's codes)
  uint32_t bq[KS][2], bl[QSPLIT ? KS : 1][2];
  float row_alpha = 0.0f;
  {
    float x[KS][4], mx = 0.0f;
    const size_t qr = g < R ? query_row_index(a, bb, kvh, row0 + g) * D : 0;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j][i] = 0.0f;
      if (g < R) load4_f32(a.q, a.q_dtype, qr + 16 * j + 4 * c, x[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(x[j][i]));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    int e = 0;                                           // the row's largest |q| goes to [2^13, 2^14)
    if (mx > 0.0f) e = min(max(((__float_as_int(mx) >> 23) & 0xFF) - 127 - 13, -100), 100);
    const float pre = ldexpf(1.0f, -e);
    row_alpha = a.scale * ldexpf(1.0f, e) * kLog2e;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      float h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[j][i] *= pre;
        h[i] = __half2float(__float2half_rn(x[j][i]));
      }
      bq[j][0] = pack_f16x2(h[0], h[1]);
      bq[j][1] = pack_f16x2(h[2], h[3]);
      if constexpr (QSPLIT) {
        bl[j][0] = pack_f16x2(x[j][0] - h[0], x[j][1] - h[1]);
        bl[j][1] = pack_f16x2(x[j][2] - h[2], x[j][3] - h[3]);
      }
    }
  }
  // the lane's two columns of S^T and O^T are rows 2c and 2c + 1
  const float alpha[2] = {__shfl_sync(0xffffffffu, row_alpha, 8 * c), __shfl_sync(0xffffffffu, row_alpha, 8 * c + 4)};
  int lim[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) lim[k] = 2 * c + k < R ? min(t_end - 1, row_limit(a, sl, (row0 + 2 * c + k) % a.n_q)) : -1;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  float O[KS][4];
#pragma unroll
  for (int j = 0; j < KS; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) O[j][k] = 0.0f;

  for (int i = 0; i < n_mine; ++i) {
    cp_async_wait<C::RING - 1>();
    __syncwarp();
    const uint8_t *sb = ring + (i % C::RING) * C::BYTES;
    const uint32_t sK = smem_addr(sb), sV = sK + C::PLANE;
    const float2 sc = *reinterpret_cast<const float2 *>(sb + 2 * C::PLANE);
    const int ts = tw0 + i * C::STAGE;

    float s[TILES][4];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s[t][k] = 0.0f;
#pragma unroll
      for (int j = 0; j < KS; j += 2) {
        uint32_t w[4];
        ldsm_x4(sK + swz<D>(16 * t + (mi & 1) * 8 + (lane & 7), j + (mi >> 1)), w);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t A[4];
          codes_f16<E4M3, false>(w[2 * u], A[0], A[2]);
          codes_f16<E4M3, false>(w[2 * u + 1], A[1], A[3]);
          mma16816(s[t], A, bq[j + u][0], bq[j + u][1]);
          if constexpr (QSPLIT) mma16816(s[t], A, bl[j + u][0], bl[j + u][1]);
        }
      }
    }
    // token of s[t][k]: ts + 16 t + g + 8 (k >> 1), row 2c + (k & 1)
    const float f[2] = {alpha[0] * sc.x, alpha[1] * sc.x};
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s[t][k] = ts + 16 * t + g + 8 * (k >> 1) <= lim[k & 1] ? s[t][k] * f[k & 1] : -INFINITY;
        mx[k & 1] = fmaxf(mx[k & 1], s[t][k]);
      }
    float corr[2], base[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], x));
      const float mn = fmaxf(m[k], mx[k]);
      base[k] = mn == -INFINITY ? 0.0f : mn;             // a row that has seen nothing yet: p = 2^-inf = 0
      corr[k] = ex2(m[k] - base[k]);
      m[k] = mn;
      l[k] *= corr[k];
    }
    uint32_t ph[TILES][2], pl[TILES][2];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      float p[4], h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        p[k] = ex2(s[t][k] - base[k & 1]);
        l[k & 1] += p[k];
        p[k] *= 4096.0f;
        h[k] = __half2float(__float2half_rn(p[k]));
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        ph[t][k] = movm_t(pack_f16x2(h[2 * k], h[2 * k + 1]));
        pl[t][k] = movm_t(pack_f16x2(p[2 * k] - h[2 * k], p[2 * k + 1] - h[2 * k + 1]));
      }
    }
    const float sv = sc.y * 0x1p-12f;
#pragma unroll
    for (int j = 0; j < KS; j += 2) {
      float acc[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[u][k] = 0.0f;
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        uint32_t w[4];
        ldsm_x4_t(sV + swz<D>(16 * t + (mi & 1) * 8 + (lane & 7), j + (mi >> 1)), w);
#pragma unroll
        for (int u = 0; u < 2; ++u) {                    // M rows g / g + 8: dims 16 (j + u) + 2g / + 2g + 1
          uint32_t A[4];
          codes_f16<E4M3, true>(w[2 * u], A[0], A[1]);
          codes_f16<E4M3, true>(w[2 * u + 1], A[2], A[3]);
          mma16816(acc[u], A, ph[t][0], ph[t][1]);
          mma16816(acc[u], A, pl[t][0], pl[t][1]);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) O[j + u][k] = fmaf(acc[u][k], sv, O[j + u][k] * corr[k & 1]);
    }
    __syncwarp();                                        // the stage is read: its place is free
    issue(i + C::RING);
  }
  cp_async_wait<0>();
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], x);
  __syncthreads();
  // the warps' states: [warp][row]: m, l; then [warp][row][D]
  float *sm = reinterpret_cast<float *>(smem), *so = sm + kWarps * 16;
  if (lane < 4) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      sm[(warp * 8 + 2 * c + k) * 2] = m[k];
      sm[(warp * 8 + 2 * c + k) * 2 + 1] = l[k];
    }
  }
#pragma unroll
  for (int j = 0; j < KS; ++j)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      *reinterpret_cast<float2 *>(so + (size_t)(warp * 8 + 2 * c + k) * D + 16 * j + 2 * g) = make_float2(O[j][k], O[j][2 + k]);
  __syncthreads();
  for (int r = warp; r < R; r += kWarps) {
    if (t0 > row_limit(a, sl, (row0 + r) % a.n_q)) continue;             // this row does not see the chunk
    float M = -INFINITY, w[kWarps], L = 0.0f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) M = fmaxf(M, sm[(k * 8 + r) * 2]);
    const float ref = M == -INFINITY ? 0.0f : M;         // (NaN states)
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      w[k] = ex2(sm[(k * 8 + r) * 2] - ref);
      L = fmaf(sm[(k * 8 + r) * 2 + 1], w[k], L);
    }
    const size_t pi = query_row_index(a, bb, kvh, row0 + r) * a.C + blockIdx.x;
#pragma unroll
    for (int d = 0; d < D; d += 128) {
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float4 x = *reinterpret_cast<const float4 *>(so + (size_t)(k * 8 + r) * D + d + 4 * lane);
        o.x = fmaf(x.x, w[k], o.x);
        o.y = fmaf(x.y, w[k], o.y);
        o.z = fmaf(x.z, w[k], o.z);
        o.w = fmaf(x.w, w[k], o.w);
      }
      *reinterpret_cast<float4 *>(a.part_o + pi * D + d + 4 * lane) = o;
    }
    if (lane == 0) {
      a.part_m[pi] = M * kLn2;
      a.part_l[pi] = L;
    }
  }
}

template <int D, bool E4M3, bool QSPLIT, bool PAGED>
cudaError_t launch_t(const AttendArgs &a, cudaStream_t st) {
  static std::atomic<bool> configured[kMaxDevices];
  auto kernel = attend_b64_kernel<D, E4M3, QSPLIT, PAGED>;
  const cudaError_t e = set_smem_once(configured, kernel, Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.n_chunks, a.cache.B * a.cache.H, (a.gqa * a.n_q + 7) / 8);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = Cfg<D>::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int D, bool E4M3>
cudaError_t launch_de(const AttendArgs &a, cudaStream_t st) {
  const bool paged = a.cache.page_shift >= 0;
  if (a.q_dtype == KVQ_F32) return paged ? launch_t<D, E4M3, true, true>(a, st) : launch_t<D, E4M3, true, false>(a, st);
  return paged ? launch_t<D, E4M3, false, true>(a, st) : launch_t<D, E4M3, false, false>(a, st);
}

}  // namespace

cudaError_t launch_attend_b64(const AttendArgs &a, cudaStream_t st) {
  if (a.cache.layout == KVQ_E4M3_B64) return a.cache.D == 128 ? launch_de<128, true>(a, st) : launch_de<256, true>(a, st);
  return a.cache.D == 128 ? launch_de<128, false>(a, st) : launch_de<256, false>(a, st);
}

}  // namespace kvq
