// Quantisation of one token row into a packed plane, shared by the append kernels (plain and with
// rotary positions). Translation units that include this are compiled with -fmad=false: every value
// is one IEEE float32 operation at a time (__fdiv_rn / __fsub_rn / __fmul_rn, rintf = round half to
// even, __float2half_rn), so the bytes match the definition exactly.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

constexpr float kF16Max = 65504.0f;

__device__ __forceinline__ __half f16_sat(float x) {
  return __float2half_rn(fminf(fmaxf(x, -kF16Max), kF16Max));
}

// Codes clamp(rint(x / s), LEAST, HI) of N values (0 when s == 0), x / s the correctly rounded quotient, each
// as the float 1.5 * 2^23 + code - LO, whose bits are kCodeBase + (code - LO).
//
// fl(1 / s) is off by at most 2^-24 of itself and the correctly rounded quotient by 2^-24 of its own, so both
// lie between the products of x with fl(1 / s) made smaller and larger by 2^-22; where the two round to one
// integer, so does the quotient. Rounding is the addition of 1.5 * 2^23 - LO in one fma (nearest even). A thread
// with a value whose products round apart divides (of random values about one warp of 512 in a thousand for 4-bit
// codes, in a hundred for 8-bit ones). `fast`: 1 / s is finite and normal, no x is NaN, and no quotient lies half a step or
// more below LEAST or (TOP_CLAMP: it may round to HI + 1 there) above HI; else every thread divides.
constexpr uint32_t kCodeBase = 0x4B400000u;              // the bits of 1.5 * 2^23
template <int LO, int HI, int LEAST, bool TOP_CLAMP, int N>
__device__ __forceinline__ void round_codes(const float (&x)[N], float s, bool fast, uint32_t (&code)[N]) {
  constexpr float kBase = 12582912.0f, kZero = kBase - LO;
  if (!(s > 0.0f)) {
#pragma unroll
    for (int i = 0; i < N; ++i) code[i] = kCodeBase + (uint32_t)(-LO);
    return;
  }
  const float inv = __frcp_rn(s), less = __fmul_rn(inv, 1.0f - 0x1p-22f), more = __fmul_rn(inv, 1.0f + 0x1p-22f);
  uint32_t apart = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float m = __fmaf_rn(x[i], less, kZero);
    apart |= __float_as_uint(m) ^ __float_as_uint(__fmaf_rn(x[i], more, kZero));
    code[i] = __float_as_uint(TOP_CLAMP ? fminf(m, kBase + (HI - LO)) : m);
  }
  if (!fast || apart) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      code[i] = kCodeBase + (uint32_t)(-LO) + (uint32_t)(int)fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), (float)LEAST), (float)HI);
  }
}
// N = 32 / BITS fields of BITS bits, field i at BITS * i: the two's complement codes of a signed layout
// (LO = -2^(BITS - 1)), or the codes of an unsigned one. One shift-add per code; what the base's bits add up
// to is taken off at the end, and the offset -LO comes out of the fields' top bits.
template <int BITS, bool SIGNED, int N>
__device__ __forceinline__ uint32_t pack_codes(const uint32_t *code) {
  static_assert(BITS * N <= 32, "one word");
  uint32_t w = 0, base = 0, flip = 0;
#pragma unroll
  for (int i = N - 1; i >= 0; --i) {
    w = (w << BITS) + code[i];
    base = (base << BITS) + kCodeBase;
    flip = (flip << BITS) | (1u << (BITS - 1));
  }
  w -= base;
  return SIGNED ? w ^ flip : w;
}
// The larger of two values, NaN if one is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Maximum of value(0 .. N - 1) and `start` over aligned groups of 32 / N neighbouring lanes (the lanes of a 32-value
// block). NaN takes no part in it but clears `numbers`: it is looked for by a maximum that keeps it, and the
// warp that has met one takes its maxima again.
template <int N, class F>
__device__ __forceinline__ float block_max(float start, F value, bool &numbers) {
  float v = start;
#pragma unroll
  for (int i = 0; i < N; ++i) v = max_nan(v, value(i));
#pragma unroll
  for (int m = 1; m < 32 / N; m <<= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, m));
  numbers = v == v;
  if (__any_sync(0xffffffffu, !numbers)) {
    v = start;
#pragma unroll
    for (int i = 0; i < N; ++i) v = fmaxf(v, value(i));
#pragma unroll
    for (int m = 1; m < 32 / N; m <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, m));
  }
  return v;
}

// N = 8 or 16 values (dims 32 blk + N lb + 0 ..) of a row, in a thread whose neighbours in the aligned
// group of 32 / N hold the rest of the block. LAYOUT: KVQ_Q4_0, KVQ_Q6_0, KVQ_Q8_0 or KVQ_ASYM4_G32.
// Every lane of the warp calls it (full-warp shuffles); one with valid == false stores nothing.
template <int LAYOUT, int N>
__device__ __forceinline__ void quant_block(const CacheView &c, int kv, long long crow, int row_bytes, int nb, int blk,
                                            int lb, const float (&v)[N], bool valid) {
  uint8_t *prow = (kv ? c.payload[1] : c.payload[0]) + (size_t)crow * row_bytes;
  __half *srow = static_cast<__half *>((kv ? c.scale[1] : c.scale[0])) + (size_t)crow * nb;
  uint32_t q[N];

  if (LAYOUT == KVQ_ASYM4_G32) {
    bool numbers;
    const float mn = -block_max<N>(-v[0], [&](int i) { return -v[i]; }, numbers);
    const float mx = block_max<N>(v[0], [&](int i) { return v[i]; }, numbers);
    const float span = __fsub_rn(mx, mn);
    const __half sh = f16_sat(__fdiv_rn(span, 15.0f));
    const __half zh = f16_sat(mn);
    const float s = __half2float(sh), z = __half2float(zh);
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __fsub_rn(v[i], z);
    // the quotients' ends: half a step beyond the codes only where z or s are coarse beside the block's span
    const bool fast = numbers && __fsub_rn(mx, z) <= __fmul_rn(s, 15.4375f) && __fsub_rn(mn, z) >= __fmul_rn(s, -0.4375f);
    round_codes<0, 15, 0, false>(x, s, fast, q);
    if (!valid) return;
    uint32_t *o = reinterpret_cast<uint32_t *>(prow + blk * 16 + lb * (N / 2));
    if constexpr (N == 16) *reinterpret_cast<uint2 *>(o) = make_uint2(pack_codes<4, false, 8>(q), pack_codes<4, false, 8>(q + 8));
    else *o = pack_codes<4, false, 8>(q);
    if (lb == 0) {
      srow[blk] = sh;
      (kv ? c.zero[1] : c.zero[0])[(size_t)crow * nb + blk] = zh;
    }
    return;
  }

  bool numbers;
  const float amax = block_max<N>(0.0f, [&](int i) { return fabsf(v[i]); }, numbers);
  constexpr int TOP = LAYOUT == KVQ_Q4_0 ? 8 : (LAYOUT == KVQ_Q8_0 ? 128 : 32);
  const __half sh = f16_sat(__fdiv_rn(amax, (float)TOP));
  const float s = __half2float(sh);
  round_codes<-TOP, TOP - 1, -TOP, true>(v, s, numbers && amax <= __fmul_rn(s, TOP + 0.4375f), q);
  if (!valid) return;
  if (lb == 0) srow[blk] = sh;
  if (LAYOUT == KVQ_Q4_0) {
    uint32_t *o = reinterpret_cast<uint32_t *>(prow + blk * 16 + lb * (N / 2));
    if constexpr (N == 16) *reinterpret_cast<uint2 *>(o) = make_uint2(pack_codes<4, true, 8>(q), pack_codes<4, true, 8>(q + 8));
    else *o = pack_codes<4, true, 8>(q);
  } else if (LAYOUT == KVQ_Q8_0) {             // byte i = value i
    uint8_t *o = prow + blk * 32 + lb * N;
    if constexpr (N == 16)
      *reinterpret_cast<uint4 *>(o) = make_uint4(pack_codes<8, true, 4>(q), pack_codes<8, true, 4>(q + 4), pack_codes<8, true, 4>(q + 8), pack_codes<8, true, 4>(q + 12));
    else
      *reinterpret_cast<uint2 *>(o) = make_uint2(pack_codes<8, true, 4>(q), pack_codes<8, true, 4>(q + 4));
  } else {                                     // Q6_0: low nibbles, then values 4k .. 4k + 3 -> high byte k
    // u = code + 32 = (its low four bits) + 16 * (the high field with its sign bit flipped)
    uint32_t lo[N], hi[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t u = q[i] - kCodeBase;
      lo[i] = kCodeBase + (u & 15u);
      hi[i] = kCodeBase + (u >> 4);
    }
    uint32_t *o = reinterpret_cast<uint32_t *>(prow + blk * 24 + lb * (N / 2));   // (24-byte blocks: 8-byte aligned)
    if constexpr (N == 16) {
      *reinterpret_cast<uint2 *>(o) = make_uint2(pack_codes<4, false, 8>(lo), pack_codes<4, false, 8>(lo + 8));
      *reinterpret_cast<uint32_t *>(prow + blk * 24 + 16 + lb * 4) = pack_codes<2, true, 16>(hi);
    } else {
      *o = pack_codes<4, false, 8>(lo);
      *reinterpret_cast<uint16_t *>(prow + blk * 24 + 16 + lb * 2) = (uint16_t)pack_codes<2, true, 8>(hi);
    }
  }
}

// A whole row in LANES neighbouring lanes (a warp, or the half of one), V consecutive values per lane,
// rotated here: BITS 4 (scale amax / 7, codes [-7, 7], two per byte) or 2 (scale amax, codes [-1, 1], four
// per byte). in_ring: the rotated float32 row also goes to slot pos mod n_recent of the window. Every lane
// of the warp calls it; those with valid == false store nothing.
//
// The rotation is the butterfly of warp_fwht in the same order: half-spans inside the lane, then lane bits;
// a lane's partner value o gives o + x or o - x as one fma with the factor 1 or -1 (rounded once, like the
// sum itself).
template <int V, int LANES, int BITS>
__device__ __forceinline__ void quant_had(const CacheView &c, int kv, long long crow, int row_bytes, int lane,
                                          float (&x)[V], bool in_ring, long long bh, int pos, bool valid) {
#pragma unroll
  for (int h = 1; h < V; h <<= 1)
#pragma unroll
    for (int i = 0; i < V; ++i)
      if ((i & h) == 0) {
        const float a = x[i], b = x[i + h];
        x[i] = __fadd_rn(a, b);
        x[i + h] = __fsub_rn(a, b);
      }
#pragma unroll
  for (int m = 1; m < LANES; m <<= 1) {
    const float sign = (lane & m) ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = __fmaf_rn(x[i], sign, __shfl_xor_sync(0xffffffffu, x[i], m));
  }
  const float cD = inv_sqrt_dim(LANES * V);
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i] = __fmul_rn(x[i], cD);
    amax = fmaxf(amax, fabsf(x[i]));
  }
#pragma unroll
  for (int m = LANES / 2; m; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  constexpr int QMAX = BITS == 4 ? 7 : 1;
  const float s = __fdiv_rn(amax, (float)QMAX);
  uint32_t q[V];
  // codes as offsets from -QMAX - 1, the fields' own offset; the ends are QMAX s to a rounding of s (a NaN in the
  // row makes every value NaN and s 0)
  round_codes<-QMAX - 1, QMAX, -QMAX, false>(x, s, s >= 0x1p-100f && s <= 0x1p100f, q);
  if (!valid) return;
  const uint32_t w = pack_codes<BITS, true, V>(q);
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
    float *dst = (kv ? c.ring[1] : c.ring[0]) + ((size_t)bh * c.n_recent + (size_t)(pos % c.n_recent)) * (LANES * V) + lane * V;
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4 *>(dst + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  }
}

}  // namespace kvq
