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
// Bound: the rows read and the codes written, once each; small appends by latency (load, reduce, divide, store). One token of 64
// sequences, 8 kv heads, e4m3: 4.2 us, 5.3 where scales grow (the kept rows of a block are read eight at a time); 12200 tokens of 16 prompts by
// slots 35.1 us: one unit after the other in a CTA, with the barrier of each unit's maximum between its loads and its codes (first
// of the stalls; issue slots 54 % busy, DRAM 10 %).
#include <cfloat>
#include <cuda_fp8.h>
#include <type_traits>

#include "kvq_internal.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;
constexpr int kFewRows = 8;          // longest run that a warp takes

// Codes of eight values given in steps (int8: half to even; e4m3: to nearest even, saturating).
template <bool E4M3>
__device__ __forceinline__ uint2 encode8(const float (&y)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if constexpr (E4M3) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * k], y[4 * k + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * k + 2], y[4 * k + 3]), __NV_SATFINITE, __NV_E4M3);
      w[k] = lo | (hi << 16);
    } else {                                             // 1.5 * 2^23 + y: the sum's rounding is rint, its low byte the code
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(fminf(fmaxf(y[4 * k + i], -127.0f), 127.0f) + 12582912.0f);
      w[k] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    }
  }
  return make_uint2(w[0], w[1]);
}
// encode8(x / s), the divisions correctly rounded. inv = 1 / s, 0 where the products are not to be trusted.
template <bool E4M3>
__device__ __forceinline__ uint2 encode8_of(const float (&x)[8], float s, float inv) {
  // x inv is within 2^-22 of the quotient and of its rounding (2^-24 each for inv, the product and the quotient)
  if (inv > 0.0f) {
    if constexpr (E4M3) {                                // the codes of values that far to both sides, if they agree
      float lo[8], hi[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __fmul_rn(x[i], inv);
        lo[i] = __fmul_rn(y, 1.0f - 0x1p-22f);
        hi[i] = __fmul_rn(y, 1.0f + 0x1p-22f);
      }
      const uint2 a = encode8<E4M3>(lo), b = encode8<E4M3>(hi);
      if (a.x == b.x && a.y == b.y) return a;
    } else {                                             // (at most 127.001, so off by less than 2^-14: no half-way quotient is nearer)
      uint32_t c[8];
      float far = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __fmul_rn(x[i], inv), t = __fadd_rn(y, 12582912.0f);
        c[i] = __float_as_uint(t);
        far = fmaxf(far, fabsf(__fsub_rn(y, __fsub_rn(t, 12582912.0f))));
      }
      if (far < 0.5f - 0x1p-14f)
        return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                          __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
    }
  }
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = s > 0.0f ? __fdiv_rn(x[i], s) : 0.0f;
  return encode8<E4M3>(y);
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

// Eight values as they were read, and as floats.
template <bool F32>
struct Raw8 {
  uint4 w[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void *src, size_t e) {
    if constexpr (F32) {
      const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(src) + e);
      w[0] = __ldg(p);
      w[1] = __ldg(p + 1);
    } else {
      w[0] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(src) + e));
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  // max with the magnitudes: of 16-bit types their bits, two at a time (they are ordered like the values)
  __device__ __forceinline__ void amax(uint32_t &m) const {
    if constexpr (F32) {
      const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, u[i] & 0x7FFFFFFFu);
    } else {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __vmaxu2(m, u[i] & 0x7FFF7FFFu);
    }
  }
  static __device__ __forceinline__ float amax_value(bool bf16, uint32_t m) {
    if constexpr (F32) return __uint_as_float(m);
    m = max(m & 0xFFFFu, m >> 16);
    return bf16 ? __uint_as_float(m << 16) : __half2float(__ushort_as_half((unsigned short)m));
  }
  // max with the magnitudes of the values that are numbers (the bits of the others lie above infinity's)
  __device__ void amax_of_numbers(bool bf16, float &m) const {
    float v[8];
    get(bf16, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  }
  __device__ __forceinline__ void get(bool bf16, float (&v)[8]) const {
    if constexpr (F32) {
      const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
    } else {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (bf16) {
          v[2 * i] = __uint_as_float(u[i] << 16);
          v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
          v[2 * i] = f.x;
          v[2 * i + 1] = f.y;
        }
      }
    }
  }
};

// One run, by the NT threads of a warp or a CTA.
template <int D, bool E4M3, int NT, bool F32>
__device__ __forceinline__ void store_run(const Run &u, int dtype, int tid, float *sm) {
  constexpr int TPR = D / 8, RP = NT / TPR;              // threads per row, rows per pass
  constexpr int P = (NT == 32 ? kFewRows : 64) / RP;
  constexpr float kTop = E4M3 ? 448.0f : 127.0f;
  const int r0 = tid / TPR, col = 8 * (tid % TPR);
  const bool bf16 = dtype == KVQ_BF16;
  Raw8<F32> raw[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int r = p * RP + r0;
    if (r < u.m) raw[p].load(u.src, u.elem + (size_t)r * u.stride + col);
    else raw[p].zero();
  }
  float old = *u.scale;
  uint32_t bits = 0;
#pragma unroll
  for (int p = 0; p < P; ++p) raw[p].amax(bits);
  if constexpr (NT == 32) {                              // a longer run behind a unit's first: read again below
    for (int r = P * RP + r0; r < u.m; r += RP) {
      Raw8<F32> more;
      more.load(u.src, u.elem + (size_t)r * u.stride + col);
      more.amax(bits);
    }
  }
  float amax = Raw8<F32>::amax_value(bf16, bits);
  if (amax != amax) {                                    // values that are no numbers do not count
    amax = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) raw[p].amax_of_numbers(bf16, amax);
    if constexpr (NT == 32) {
      for (int r = P * RP + r0; r < u.m; r += RP) {
        Raw8<F32> more;
        more.load(u.src, u.elem + (size_t)r * u.stride + col);
        more.amax_of_numbers(bf16, amax);
      }
    }
  }
#pragma unroll
  for (int k = 16; k; k >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, k));
  if constexpr (NT > 32) {                               // (two buffers in turn: the next run's maxima do not meet this one's)
    if ((tid & 31) == 0) sm[tid >> 5] = amax;
    __syncthreads();                                     // every thread has read the old scale too
    amax = sm[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) amax = fmaxf(amax, sm[w]);
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
    constexpr int AT_ONCE = 8;                           // rows read together: a decode step's warp has up to 63 of them
    for (int r = r0; r < u.o; r += AT_ONCE * RP) {
      uint2 was[AT_ONCE];
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j)
        was[j] = r + j * RP < u.o ? *reinterpret_cast<const uint2 *>(u.rows + (r + j * RP) * D + col) : make_uint2(0u, 0u);
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) {
        if (r + j * RP >= u.o) break;
        float y[8];
        decode8<E4M3>(was[j], y);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= f;
        *reinterpret_cast<uint2 *>(u.rows + (r + j * RP) * D + col) = encode8<E4M3>(y);
      }
    }
  }
  const float inv = s > 0x1p-100f && s < 0x1p100f && amax <= FLT_MAX ? __frcp_rn(s) : 0.0f;
  auto put = [&](int r, const Raw8<F32> &x) {
    float v[8];
    x.get(bf16, v);
    *reinterpret_cast<uint2 *>(u.rows + (u.o + r) * D + col) = encode8_of<E4M3>(v, s, inv);
  };
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (p * RP + r0 < u.m) put(p * RP + r0, raw[p]);
  if constexpr (NT == 32) {
    for (int r = P * RP + r0; r < u.m; r += RP) {
      Raw8<F32> more;
      more.load(u.src, u.elem + (size_t)r * u.stride + col);
      put(r, more);
    }
  }
}

struct BlockGeom {
  int n_new, pos0, pos_offset, blocks;     // blocks: per sequence, at most
  const int32_t *seq_pos;
  long long units;                         // 2 * B * H * blocks
};

// Equal numbers of rows for every (sequence, head): unit u is block u % blocks of head u / blocks.
template <int D, bool E4M3, int NT, bool F32>
__global__ void __launch_bounds__(kThreads) store_b64_kernel(CacheView c, const void *__restrict__ k_new, const void *__restrict__ v_new,
                                                             int dtype, BlockGeom g) {
#if defined(__CUDA_ARCH__) && __CUDA_ARCH__ >= 900
  asm volatile("griddepcontrol.launch_dependents;");   // attention may launch and wait on us
#endif
  __shared__ float sm[kThreads / 32];
  const long long unit = (long long)blockIdx.x * (kThreads / NT) + threadIdx.x / NT;
  if (unit >= g.units) return;                           // whole warps, or the whole CTA
  long long head, bh;
  int kv, bb, h;
  if (g.units <= 0x7FFFFFFFLL) {                         // 32-bit index arithmetic (every realistic call)
    const unsigned u = (unsigned)unit, uh = u / (unsigned)g.blocks, per = (unsigned)(c.B * c.H);
    kv = uh >= per;
    const unsigned ubh = kv ? uh - per : uh;
    bb = (int)(ubh / (unsigned)c.H);
    h = (int)(ubh - (unsigned)bb * (unsigned)c.H);
    head = uh;
    bh = ubh;
  } else {
    head = unit / g.blocks;
    bh = head % ((long long)c.B * c.H);
    kv = head >= (long long)c.B * c.H;
    bb = (int)(bh / c.H);
    h = (int)(bh - (long long)bb * c.H);
  }
  const long long start = (long long)(g.seq_pos ? __ldg(g.seq_pos + bb) : g.pos0) + g.pos_offset;
  const long long lo = max(start, 0LL), hi = min(start + g.n_new, (long long)c.cap);
  const long long b0 = ((lo >> 6) + (unit - head * g.blocks)) << 6;        // the block's first token
  const long long t0 = max(lo, b0), t1 = min(hi, b0 + 64);
  if (t0 >= t1) return;
  const size_t row = cache_row(c, bb, h, (int)b0);
  const Run u = {kv ? v_new : k_new, (size_t)(bh * g.n_new + (t0 - start)) * D, D, (int)(t1 - t0), (int)(t0 - b0),
                 (kv ? c.payload[1] : c.payload[0]) + row * D, static_cast<float *>(kv ? c.scale[1] : c.scale[0]) + (row >> 6)};
  store_run<D, E4M3, NT, F32>(u, dtype, threadIdx.x % NT, sm);
}

// A ragged run of tokens. Consecutive pool rows of one block are a run; the runs of a block that follow each other in
// the call (up to kGap tokens without a slot between them) are appended one after the other by the one unit that begins at
// the first of them, so that no two units share a scale. CTA (w, y, plane) takes the units that begin at its W tokens, for
// every gridDim.y-th head: those whose first run is long with all its warps, the others a warp each.
constexpr int kGap = 64;

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

template <int D, bool E4M3, int W, bool F32>
__global__ void __launch_bounds__(kThreads) store_b64_slots_kernel(CacheView c, SlotRows g) {
  __shared__ float sm[2][kThreads / 32];
  __shared__ int begin[W], len[W], count;                // the units: first token, and length of the first run
  const int t0 = blockIdx.x * W, kv = blockIdx.z, tid = threadIdx.x;
  const Slots sl = {g.slots, (long long)c.n_pages << c.page_shift, g.n_tokens};
  if (tid < 32) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < W; i += 32) {
      const long long s = i + tid < W ? sl.at((long long)t0 + i + tid) : -1;
      const bool first = s >= 0 && sl.begins(t0 + i + tid, s);
      const unsigned m = __ballot_sync(0xffffffffu, first);
      if (first) begin[n + __popc(m & ((1u << tid) - 1u))] = t0 + i + tid;
      n += __popc(m);
    }
    if (tid == 0) count = n;
  }
  __syncthreads();
  const int units = count;
  if (units == 0) return;                                // (most CTAs of a prompt's tokens)
  for (int i = tid >> 5; i < units; i += kThreads / 32) {
    const int n = sl.run(begin[i], sl.at(begin[i]));
    if ((tid & 31) == 0) len[i] = n;
  }
  __syncthreads();
  const RowsIn in = {kv ? g.v.data : g.k.data, 0, kv ? g.v.head : g.k.head, kv ? g.v.token : g.k.token};
  int turn = 0;
  auto unit = [&](int i, int h, auto threads) {
    constexpr int NT = decltype(threads)::value;
    for (int t = begin[i], m = len[i]; t >= 0;) {
      const long long s = sl.at(t), b0 = s & ~63LL;
      if (m == 0) m = sl.run(t, s);
      const size_t row = (size_t)((((b0 >> c.page_shift) * c.H + h) << c.page_shift) + (b0 & ((1LL << c.page_shift) - 1)));
      const Run u = {in.data, (size_t)(t * in.token + h * in.head), in.token, m, (int)(s - b0),
                     (kv ? c.payload[1] : c.payload[0]) + row * D, static_cast<float *>(kv ? c.scale[1] : c.scale[0]) + (row >> 6)};
      store_run<D, E4M3, NT, F32>(u, g.dtype, NT == 32 ? tid & 31 : tid, sm[turn]);
      turn ^= 1;
      t = sl.next(t + m, s);
      m = 0;
      if (t >= 0) {                                      // its bytes and scale are the next run's to read
        if (NT > 32) __syncthreads();
        else __syncwarp();
      }
    }
  };
  for (int i = 0; i < units; ++i)
    if (len[i] > kFewRows)
      for (int h = blockIdx.y; h < c.H; h += gridDim.y) unit(i, h, std::integral_constant<int, kThreads>{});
  for (int i = tid >> 5; i < units; i += kThreads / 32)
    if (len[i] <= kFewRows)
      for (int h = blockIdx.y; h < c.H; h += gridDim.y) unit(i, h, std::integral_constant<int, 32>{});
}

template <int D, bool E4M3, bool F32>
cudaError_t launch_dt(const CacheView &c, const void *k_new, const void *v_new, int dtype, const BlockGeom &g, cudaStream_t st) {
  // a warp or a CTA for each run (64 sequences, 8 kv heads: one row 2.9 / 5.1 us, 8 rows 4.6 / 6.7)
  if (g.n_new <= kFewRows)
    store_b64_kernel<D, E4M3, 32, F32><<<(unsigned)((g.units + 7) / 8), kThreads, 0, st>>>(c, k_new, v_new, dtype, g);
  else
    store_b64_kernel<D, E4M3, kThreads, F32><<<(unsigned)g.units, kThreads, 0, st>>>(c, k_new, v_new, dtype, g);
  return cudaGetLastError();
}
template <int D, bool E4M3>
cudaError_t launch_de(const CacheView &c, const void *k_new, const void *v_new, int dtype, const BlockGeom &g, cudaStream_t st) {
  return dtype == KVQ_F32 ? launch_dt<D, E4M3, true>(c, k_new, v_new, dtype, g, st) : launch_dt<D, E4M3, false>(c, k_new, v_new, dtype, g, st);
}

}  // namespace

cudaError_t launch_store_b64(const CacheView &c, const void *k_new, const void *v_new, int dtype, int n_new, int pos0,
                             cudaStream_t st, const int32_t *seq_pos, int pos_offset) {
  BlockGeom g = {n_new, pos0, pos_offset, (int)(((long long)n_new + 62) / 64) + 1, seq_pos, 0};
  g.units = 2LL * c.B * c.H * g.blocks;
  const bool e4m3 = c.layout == KVQ_E4M3_B64;
  if (c.D == 128)
    return e4m3 ? launch_de<128, true>(c, k_new, v_new, dtype, g, st) : launch_de<128, false>(c, k_new, v_new, dtype, g, st);
  return e4m3 ? launch_de<256, true>(c, k_new, v_new, dtype, g, st) : launch_de<256, false>(c, k_new, v_new, dtype, g, st);
}

namespace {

template <int D, bool E4M3, bool F32>
cudaError_t launch_slots_t(const CacheView &c, const SlotRows &g, cudaStream_t st) {
  // Many tokens (prompts): 64 of them and several heads per CTA, about sixteen CTAs per SM, so that few CTAs look at the map for
  // each unit; few tokens, which may all begin units of their own: 16, and a CTA for each head. (12200 tokens of 16 prompts, 8
  // kv heads: 35.8 us, with eight CTAs per SM 39.2, with 16 tokens and one head 46.4)
  if (g.n_tokens > 2048) {
    const long long windows = ((long long)g.n_tokens + 63) / 64, want = 16 * (long long)sm_count() / (2 * windows);
    const dim3 grid((unsigned)windows, (unsigned)(want < 1 ? 1 : want > c.H ? c.H : want), 2);
    store_b64_slots_kernel<D, E4M3, 64, F32><<<grid, kThreads, 0, st>>>(c, g);
  } else {
    const dim3 grid((unsigned)((g.n_tokens + 15) / 16), (unsigned)c.H, 2);
    store_b64_slots_kernel<D, E4M3, 16, F32><<<grid, kThreads, 0, st>>>(c, g);
  }
  return cudaGetLastError();
}
template <int D, bool E4M3>
cudaError_t launch_slots_dt(const CacheView &c, const SlotRows &g, cudaStream_t st) {
  return g.dtype == KVQ_F32 ? launch_slots_t<D, E4M3, true>(c, g, st) : launch_slots_t<D, E4M3, false>(c, g, st);
}

}  // namespace

cudaError_t launch_store_b64_slots(const CacheView &c, const SlotRows &g, cudaStream_t st) {
  const bool e4m3 = c.layout == KVQ_E4M3_B64;
  if (c.D == 128) return e4m3 ? launch_slots_dt<128, true>(c, g, st) : launch_slots_dt<128, false>(c, g, st);
  return e4m3 ? launch_slots_dt<256, true>(c, g, st) : launch_slots_dt<256, false>(c, g, st);
}

}  // namespace kvq
