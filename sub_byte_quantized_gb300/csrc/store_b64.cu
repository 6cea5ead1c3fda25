// Appends into the 8-bit block layouts: one f32 scale for the 64 tokens of a block, per head and plane.
//
//   need = amax(new rows of the block) / T,  T = 127 (int8) or 448 (e4m3)
//   s'   = need                    where the block's first new row is its row 0 (or it has no scale yet)
//        = s                       where need <= s
//        = s 2^k                   else, with the smallest k >= 1 that s 2^k >= need; kept codes become round(c 2^-k)
//   new codes = round(x / s'), one correctly rounded division each
// A power of two makes a kept row's second rounding exact to state (an integer shift, or an exponent's), and since a
// scale that grows at least doubles, the roundings of a row that is kept through all of them sum to less than one
// step of the last scale.
//
// One unit is the run of new rows of one block, head and plane. A warp takes it where a run is at most 8 rows (a
// decode step: one row), a CTA of 8 warps else (a whole block: 16 KB of bf16 at head_dim 128); either way the rows stay in
// registers between the pass over their maximum and the codes. This file is compiled with -fmad=false.
//
// Bound: the rows read and the codes written, once each; small appends by latency (load, reduce, divide, store).
#include <cfloat>
#include <cuda_fp8.h>
#include <type_traits>

#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kFewRows = 8;          // longest run that a warp takes

template <bool E4M3>
__device__ __forceinline__ uint2 encode8(const float (&y)[8]) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    uint32_t two;
    if constexpr (E4M3) {
      two = __nv_cvt_float2_to_fp8x2(make_float2(y[i], y[i + 1]), __NV_SATFINITE, __NV_E4M3);
    } else {
      const int a = (int)fminf(fmaxf(rintf(y[i]), -127.0f), 127.0f), b = (int)fminf(fmaxf(rintf(y[i + 1]), -127.0f), 127.0f);
      two = (uint32_t)(a & 0xFF) | ((uint32_t)(b & 0xFF) << 8);
    }
    w[i >> 2] |= two << (8 * (i & 2));
  }
  return make_uint2(w[0], w[1]);
}
template <bool E4M3>
__device__ __forceinline__ void decode8(uint2 p, float (&y)[8]) {
  const uint32_t w[2] = {p.x, p.y};
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint32_t two = (w[i >> 2] >> (8 * (i & 2))) & 0xFFFFu;
    if constexpr (E4M3) {
      const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
      y[i] = __low2float(h);
      y[i + 1] = __high2float(h);
    } else {
      y[i] = (float)(int8_t)(two & 0xFFu);
      y[i + 1] = (float)(int8_t)(two >> 8);
    }
  }
}

struct Run {
  const void *src;
  size_t elem;                 // element of the first new row
  long long stride;            // elements between new rows
  int m, o;                    // new rows, and the block row of the first
  uint8_t *rows;               // the block's payload
  float *scale;
};

// One run, by the NT threads of a warp or a CTA.
template <int D, bool E4M3, int NT>
__device__ __forceinline__ void store_run(const Run &u, int dtype, int tid, float *sm) {
  constexpr int TPR = D / 8, RP = NT / TPR;              // threads per row, rows per pass
  constexpr int P = (NT == 32 ? kFewRows : 64) / RP;
  constexpr float kTop = E4M3 ? 448.0f : 127.0f;
  const int r0 = tid / TPR, col = 8 * (tid % TPR);
  float v[P][8], amax = 0.0f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int r = p * RP + r0;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
    if (r < u.m) load8_f32(u.src, dtype, u.elem + (size_t)r * u.stride + col, v[p]);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[p][i]));
  }
  if constexpr (NT == 32) {                              // a longer run behind a unit's first: read again below
    for (int r = P * RP + r0; r < u.m; r += RP) {
      float x[8];
      load8_f32(u.src, dtype, u.elem + (size_t)r * u.stride + col, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
    }
  }
  float old = *u.scale;
#pragma unroll
  for (int k = 16; k; k >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, k));
  if constexpr (NT > 32) {
    if ((tid & 31) == 0) sm[tid >> 5] = amax;
    __syncthreads();                                     // every thread has read the old scale too
    amax = sm[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) amax = fmaxf(amax, sm[w]);
    __syncthreads();
  } else {
    __syncwarp();
  }
  if (u.o == 0 || !(old > 0.0f)) old = 0.0f;
  const float need = __fdiv_rn(fminf(amax, FLT_MAX), kTop);   // an infinity counts as the largest value: scales stay finite
  float s = old;
  int k = 0;
  if (need > old) {
    s = need;
    if (old > 0.0f) {
      int eo, en;
      const float mo = frexpf(old, &eo), mn = frexpf(need, &en);
      k = en - eo + (mn > mo ? 1 : 0);
      s = ldexpf(old, k);
    }
  }
  if (tid == 0) *u.scale = s;
  if (k > 0) {
    const float f = ldexpf(1.0f, -min(k, 64));
    for (int r = r0; r < u.o; r += RP) {
      uint2 *p = reinterpret_cast<uint2 *>(u.rows + r * D + col);
      float y[8];
      decode8<E4M3>(*p, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= f;
      *p = encode8<E4M3>(y);
    }
  }
  auto put = [&](int r, const float (&x)[8]) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = s > 0.0f ? __fdiv_rn(x[i], s) : 0.0f;
    *reinterpret_cast<uint2 *>(u.rows + (u.o + r) * D + col) = encode8<E4M3>(y);
  };
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (p * RP + r0 < u.m) put(p * RP + r0, v[p]);
  if constexpr (NT == 32) {
    for (int r = P * RP + r0; r < u.m; r += RP) {
      float x[8];
      load8_f32(u.src, dtype, u.elem + (size_t)r * u.stride + col, x);
      put(r, x);
    }
  }
}

struct BlockGeom {
  int n_new, pos0, pos_offset, blocks;     // blocks: per sequence, at most
  const int32_t *seq_pos;
  long long units;                         // 2 * B * H * blocks
};

// Equal numbers of rows for every (sequence, head): unit u is block u % blocks of head u / blocks.
template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kThreads) store_b64_kernel(CacheView c, const void *__restrict__ k_new, const void *__restrict__ v_new,
                                                             int dtype, BlockGeom g) {
#if defined(__CUDA_ARCH__) && __CUDA_ARCH__ >= 900
  asm volatile("griddepcontrol.launch_dependents;");   // attention may launch and wait on us
#endif
  __shared__ float sm[kThreads / 32];
  const long long unit = (long long)blockIdx.x * (kThreads / NT) + threadIdx.x / NT;
  if (unit >= g.units) return;                           // whole warps, or the whole CTA
  const long long head = unit / g.blocks, bh = head % ((long long)c.B * c.H);
  const int kv = head >= (long long)c.B * c.H, bb = (int)(bh / c.H), h = (int)(bh - (long long)bb * c.H);
  const long long start = (long long)(g.seq_pos ? __ldg(g.seq_pos + bb) : g.pos0) + g.pos_offset;
  const long long lo = max(start, 0LL), hi = min(start + g.n_new, (long long)c.cap);
  const long long b0 = ((lo >> 6) + (unit - head * g.blocks)) << 6;        // the block's first token
  const long long t0 = max(lo, b0), t1 = min(hi, b0 + 64);
  if (t0 >= t1) return;
  const size_t row = cache_row(c, bb, h, (int)b0);
  const Run u = {kv ? v_new : k_new, (size_t)(bh * g.n_new + (t0 - start)) * D, D, (int)(t1 - t0), (int)(t0 - b0),
                 (kv ? c.payload[1] : c.payload[0]) + row * D, static_cast<float *>(kv ? c.scale[1] : c.scale[0]) + (row >> 6)};
  store_run<D, E4M3, NT>(u, dtype, threadIdx.x % NT, sm);
}

// A ragged run of tokens. Consecutive pool rows of one block are a run; the runs of a block that follow each other in
// the call (up to kGap tokens without a slot between them) are appended one after the other by the one unit that begins at
// the first of them, so that no two units share a scale. CTA (w, h, plane) takes the units that begin at its kWindow
// tokens: those whose first run is long with all its warps, the others a warp each.
constexpr int kWindow = 16, kGap = 64;

struct Slots {
  const long long *slots;
  long long pool;
  int n;
  // pool row of token t, -1 where it has none
  __device__ __forceinline__ long long at(long long t) const {
    const long long s = t >= 0 && t < n ? __ldg(slots + t) : -1;
    return s < pool ? s : -1;
  }
  // whether token t, with pool row s >= 0, begins a unit
  __device__ __forceinline__ bool begins(int t, long long s) const {
    for (int k = 1; k <= kGap + 1 && k <= t; ++k) {
      const long long before = at(t - k);
      if (before >= 0) return (before >> 6) != (s >> 6);
    }
    return true;
  }
  // length of the run that begins at token t with pool row s (a warp's work)
  __device__ __forceinline__ int run(int t, long long s) const {
    const int lane = threadIdx.x & 31, most = 64 - (int)(s & 63);
    const unsigned a = __ballot_sync(0xffffffffu, lane < most && at((long long)t + lane) == s + lane);
    const unsigned b = __ballot_sync(0xffffffffu, lane + 32 < most && at((long long)t + lane + 32) == s + lane + 32);
    return ~a ? __ffs((int)~a) - 1 : ~b ? 31 + __ffs((int)~b) : 64;
  }
  // the token behind t (exclusive) that goes on with the block of pool row s; -1 where none does
  __device__ __forceinline__ int next(int t, long long s) const {
    for (int k = 0; k <= kGap && t + k < n; ++k) {
      const long long r = at(t + k);
      if (r >= 0) return (r >> 6) == (s >> 6) ? t + k : -1;
    }
    return -1;
  }
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) store_b64_slots_kernel(CacheView c, SlotRows g) {
  __shared__ float sm[kThreads / 32];
  __shared__ int len[kWindow];                           // of the first run of the unit that begins at each token; 0: none
  const int t0 = blockIdx.x * kWindow, h = blockIdx.y, kv = blockIdx.z, tid = threadIdx.x;
  const Slots sl = {g.slots, (long long)c.n_pages << c.page_shift, g.n_tokens};
  for (int i = tid >> 5; i < kWindow; i += kThreads / 32) {
    const long long s = sl.at((long long)t0 + i);
    const int n = s >= 0 && sl.begins(t0 + i, s) ? sl.run(t0 + i, s) : 0;
    if ((tid & 31) == 0) len[i] = n;
  }
  __syncthreads();
  const RowsIn in = {kv ? g.v.data : g.k.data, 0, kv ? g.v.head : g.k.head, kv ? g.v.token : g.k.token};
  auto unit = [&](int i, auto threads) {
    constexpr int NT = decltype(threads)::value;
    for (int t = t0 + i, m = len[i]; t >= 0;) {
      const long long s = sl.at(t), b0 = s & ~63LL;
      if (m == 0) m = sl.run(t, s);
      const size_t row = (size_t)((((b0 >> c.page_shift) * c.H + h) << c.page_shift) + (b0 & ((1LL << c.page_shift) - 1)));
      const Run u = {in.data, (size_t)(t * in.token + h * in.head), in.token, m, (int)(s - b0),
                     (kv ? c.payload[1] : c.payload[0]) + row * D, static_cast<float *>(kv ? c.scale[1] : c.scale[0]) + (row >> 6)};
      store_run<D, E4M3, NT>(u, g.dtype, NT == 32 ? tid & 31 : tid, sm);
      t = sl.next(t + m, s);
      m = 0;
      if (NT > 32) __syncthreads();                      // its bytes and scale are the next run's to read
      else __syncwarp();
    }
  };
  for (int i = 0; i < kWindow; ++i)
    if (len[i] > kFewRows) unit(i, std::integral_constant<int, kThreads>{});
  for (int i = tid >> 5; i < kWindow; i += kThreads / 32)
    if (len[i] > 0 && len[i] <= kFewRows) unit(i, std::integral_constant<int, 32>{});
}

template <int D, bool E4M3>
cudaError_t launch_dt(const CacheView &c, const void *k_new, const void *v_new, int dtype, const BlockGeom &g, cudaStream_t st) {
  if (g.n_new <= kFewRows)
    store_b64_kernel<D, E4M3, 32><<<(unsigned)((g.units + 7) / 8), kThreads, 0, st>>>(c, k_new, v_new, dtype, g);
  else
    store_b64_kernel<D, E4M3, kThreads><<<(unsigned)g.units, kThreads, 0, st>>>(c, k_new, v_new, dtype, g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_store_b64(const CacheView &c, const void *k_new, const void *v_new, int dtype, int n_new, int pos0,
                             cudaStream_t st, const int32_t *seq_pos, int pos_offset) {
  BlockGeom g = {n_new, pos0, pos_offset, (int)(((long long)n_new + 62) / 64) + 1, seq_pos, 0};
  g.units = 2LL * c.B * c.H * g.blocks;
  const bool e4m3 = c.layout == KVQ_E4M3_B64;
  if (c.D == 128)
    return e4m3 ? launch_dt<128, true>(c, k_new, v_new, dtype, g, st) : launch_dt<128, false>(c, k_new, v_new, dtype, g, st);
  return e4m3 ? launch_dt<256, true>(c, k_new, v_new, dtype, g, st) : launch_dt<256, false>(c, k_new, v_new, dtype, g, st);
}

cudaError_t launch_store_b64_slots(const CacheView &c, const SlotRows &g, cudaStream_t st) {
  const dim3 grid((unsigned)(((long long)g.n_tokens + kWindow - 1) / kWindow), (unsigned)c.H, 2);
  const bool e4m3 = c.layout == KVQ_E4M3_B64;
  if (c.D == 128) {
    if (e4m3) store_b64_slots_kernel<128, true><<<grid, kThreads, 0, st>>>(c, g);
    else store_b64_slots_kernel<128, false><<<grid, kThreads, 0, st>>>(c, g);
  } else {
    if (e4m3) store_b64_slots_kernel<256, true><<<grid, kThreads, 0, st>>>(c, g);
    else store_b64_slots_kernel<256, false><<<grid, kThreads, 0, st>>>(c, g);
  }
  return cudaGetLastError();
}

}  // namespace kvq
