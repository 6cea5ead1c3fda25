// Quantisation of one token row into a packed plane, shared by the append kernels (plain and with
// rotary positions). Translation units that include this are compiled with -fmad=false: every value
// is one IEEE float32 operation at a time (__fdiv_rn / __fsub_rn / __fmul_rn, rintf = round half to
// even, __float2half_rn), so the bytes match the definition exactly.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

constexpr float kF16Max = 65504.0f;

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_min(float v) {
  v = fminf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fminf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

__device__ __forceinline__ __half f16_sat(float x) {
  return __float2half_rn(fminf(fmaxf(x, -kF16Max), kF16Max));
}

// Codes clamp(rint(x / s), LO, HI) of N values (0 when s == 0), x / s the correctly rounded quotient: as
// bit fields of an unsigned word each, two's complement (the caller masks them).
//
// The quotient is taken as r = x * fl(1 / s), off by less than 2^-22 of itself, i.e. by less than 7e-5 for
// |x / s| <= 256 (beyond, both clamp alike). It rounds like the correct quotient unless a half-integer lies
// between the two, and then r is within 1e-4 of one: those rare threads divide. Rounding is the addition of
// 1.5 * 2^23 (nearest even), whose low mantissa bits are the code. A scale below 2^-100 divides throughout
// (its reciprocal could overflow).
template <int LO, int HI, int N>
__device__ __forceinline__ void round_codes(const float (&x)[N], float s, uint32_t (&code)[N]) {
  constexpr float kMagic = 12582912.0f;
  if (!(s > 0.0f)) {
#pragma unroll
    for (int i = 0; i < N; ++i) code[i] = 0;
    return;
  }
  const float inv = __frcp_rn(s);
  bool divide = s < 0x1p-100f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float r = fminf(fmaxf(__fmul_rn(x[i], inv), -300.0f), 300.0f), m = __fadd_rn(r, kMagic);
    divide |= fabsf(__fsub_rn(r, __fsub_rn(m, kMagic))) > 0.4999f;
    code[i] = __float_as_uint(fminf(fmaxf(m, kMagic + LO), kMagic + HI));
  }
  if (divide) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      code[i] = (uint32_t)(int)fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), (float)LO), (float)HI);
  }
}

// Eight values (dims 32 blk + 8 lb + 0..7) of a row, in a thread whose three neighbours in the aligned
// group of four hold the rest of the block. LAYOUT: KVQ_Q4_0, KVQ_Q6_0, KVQ_Q8_0 or KVQ_ASYM4_G32.
// Every lane of the warp calls it (full-warp shuffles); one with valid == false stores nothing.
template <int LAYOUT>
__device__ __forceinline__ void quant_block(const CacheView &c, int kv, long long crow, int row_bytes, int nb, int blk,
                                            int lb, const float (&v)[8], bool valid) {
  uint8_t *prow = (kv ? c.payload[1] : c.payload[0]) + (size_t)crow * row_bytes;
  __half *srow = static_cast<__half *>((kv ? c.scale[1] : c.scale[0])) + (size_t)crow * nb;

  if (LAYOUT == KVQ_ASYM4_G32) {
    float mn = v[0], mx = v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) { mn = fminf(mn, v[i]); mx = fmaxf(mx, v[i]); }
    mn = quad_min(mn);
    mx = quad_max(mx);
    const __half sh = f16_sat(__fdiv_rn(__fsub_rn(mx, mn), 15.0f));
    const __half zh = f16_sat(mn);
    const float s = __half2float(sh), z = __half2float(zh);
    float x[8];
    uint32_t q[8], w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fsub_rn(v[i], z);
    round_codes<0, 15>(x, s, q);
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= (q[i] & 0xFu) << (4 * i);
    if (!valid) return;
    *reinterpret_cast<uint32_t *>(prow + blk * 16 + lb * 4) = w;
    if (lb == 0) {
      srow[blk] = sh;
      (kv ? c.zero[1] : c.zero[0])[(size_t)crow * nb + blk] = zh;
    }
    return;
  }

  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
  amax = quad_max(amax);
  if (LAYOUT == KVQ_Q4_0) {
    const __half sh = f16_sat(__fdiv_rn(amax, 8.0f));
    const float s = __half2float(sh);
    uint32_t q[8], w = 0;
    round_codes<-8, 7>(v, s, q);
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= (q[i] & 0xFu) << (4 * i);
    if (!valid) return;
    *reinterpret_cast<uint32_t *>(prow + blk * 16 + lb * 4) = w;
    if (lb == 0) srow[blk] = sh;
  } else if (LAYOUT == KVQ_Q8_0) {
    const __half sh = f16_sat(__fdiv_rn(amax, 128.0f));
    const float s = __half2float(sh);
    uint32_t q[8], w0 = 0, w1 = 0;             // byte i = value i (two's complement)
    round_codes<-128, 127>(v, s, q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w0 |= (q[i] & 0xFFu) << (8 * i);
      w1 |= (q[4 + i] & 0xFFu) << (8 * i);
    }
    if (!valid) return;
    *reinterpret_cast<uint2 *>(prow + blk * 32 + lb * 8) = make_uint2(w0, w1);
    if (lb == 0) srow[blk] = sh;
  } else {  // Q6_0
    const __half sh = f16_sat(__fdiv_rn(amax, 32.0f));
    const float s = __half2float(sh);
    uint32_t q[8], lo = 0, hi = 0;
    round_codes<-32, 31>(v, s, q);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo |= (q[i] & 0xFu) << (4 * i);
      hi |= ((q[i] >> 4) & 0x3u) << (2 * i);   // values 4k..4k+3 -> byte k, bits 0,2,4,6
    }
    if (!valid) return;
    uint8_t *bp = prow + blk * 24;
    *reinterpret_cast<uint32_t *>(bp + lb * 4) = lo;
    *reinterpret_cast<uint16_t *>(bp + 16 + lb * 2) = (uint16_t)hi;
    if (lb == 0) srow[blk] = sh;
  }
}

// A whole row in one warp, V = D/32 consecutive values per lane, rotated here: BITS 4 (scale
// amax / 7, codes [-7, 7], two per byte) or 2 (scale amax, codes [-1, 1], four per byte). in_ring:
// the rotated float32 row also goes to slot pos mod n_recent of the window.
template <int V, int BITS>
__device__ __forceinline__ void quant_had(const CacheView &c, int kv, long long crow, int row_bytes, int lane,
                                          float (&x)[V], bool in_ring, long long bh, int pos) {
  warp_fwht<V>(x, lane);
  const float cD = inv_sqrt_dim(32 * V);
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i] = __fmul_rn(x[i], cD);
    amax = fmaxf(amax, fabsf(x[i]));
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  constexpr int QMAX = BITS == 4 ? 7 : 1;
  const float s = __fdiv_rn(amax, (float)QMAX);
  uint32_t q[V], w = 0;                                     // field i of the lane at bits BITS*i
  round_codes<-QMAX, QMAX>(x, s, q);
#pragma unroll
  for (int i = 0; i < V; ++i) w |= (q[i] & ((1u << BITS) - 1u)) << (BITS * i);
  uint8_t *prow = (kv ? c.payload[1] : c.payload[0]) + (size_t)crow * row_bytes;
  if (V * BITS == 8) {
    prow[lane] = (uint8_t)w;
  } else if (V * BITS == 16) {
    *reinterpret_cast<uint16_t *>(prow + lane * 2) = (uint16_t)w;
  } else {
    *reinterpret_cast<uint32_t *>(prow + lane * 4) = w;
  }
  if (lane == 0) static_cast<float *>((kv ? c.scale[1] : c.scale[0]))[crow] = s;
  if (in_ring) {
    float *dst = (kv ? c.ring[1] : c.ring[0]) + ((size_t)bh * c.n_recent + (size_t)(pos % c.n_recent)) * (32 * V) + lane * V;
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4 *>(dst + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  }
}

}  // namespace kvq
