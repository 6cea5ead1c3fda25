// Eight values of a packed row, by layout (compiled out where the layout is a constant).
#pragma once

#include <cuda_fp8.h>

#include "kvq_internal.cuh"

namespace kvq {

// Unpack 8 values (group gi of a token row) of a packed row of plane kv, in that plane's `layout`, into f32 (value = code *
// scale [+ zero]). For the layouts with one scale per token or block (Hadamard, 8-bit blocks) the raw codes are produced
// (the scale is applied by the caller).
__device__ __forceinline__ void unpack8(int layout, const CacheView &c, int kv, size_t row, int gi, float out[8]) {
  const uint8_t *p = (kv ? c.payload[1] : c.payload[0]) + row * (size_t)(kv ? c.v_row_bytes : c.row_bytes);
  const int blk = gi >> 2, sub = gi & 3;
  if (layout == KVQ_HAD_INT4) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p + gi * 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = (float)((int)((w >> (4 * i)) & 0xFu ^ 0x8u) - 8);
    return;
  }
  if (layout == KVQ_HAD_INT2) {                       // four 2-bit fields per byte, (v ^ 2) - 2
    const uint32_t w = *reinterpret_cast<const uint16_t *>(p + gi * 2);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = (float)((int)((w >> (2 * i)) & 0x3u ^ 0x2u) - 2);
    return;
  }
  if (layout == KVQ_INT8_B64 || layout == KVQ_E4M3_B64) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p + gi * 8);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint32_t two = ((i < 4 ? w.x : w.y) >> (8 * (i & 2))) & 0xFFFFu;
      if (layout == KVQ_E4M3_B64) {
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3)));
        out[i] = f.x;
        out[i + 1] = f.y;
      } else {
        out[i] = (float)(int8_t)(two & 0xFFu);
        out[i + 1] = (float)(int8_t)(two >> 8);
      }
    }
    return;
  }
  const float s = __half2float(static_cast<const __half *>((kv ? c.scale[1] : c.scale[0]))[row * (c.D / kBlock) + blk]);
  if (layout == KVQ_Q4_0) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p + blk * 16 + sub * 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = (float)((int)((w >> (4 * i)) & 0xFu ^ 0x8u) - 8) * s;
  } else if (layout == KVQ_Q6_0) {
    const uint32_t lo = *reinterpret_cast<const uint32_t *>(p + blk * 24 + sub * 4);
    const uint32_t hi = *reinterpret_cast<const uint16_t *>(p + blk * 24 + 16 + sub * 2);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t v = ((lo >> (4 * i)) & 0xFu) | (((hi >> (2 * i)) & 0x3u) << 4);
      out[i] = (float)((int)(v ^ 0x20u) - 0x20) * s;
    }
  } else if (layout == KVQ_Q8_0) {                    // byte i = value i, (v ^ 0x80) - 0x80
    const uint2 w = *reinterpret_cast<const uint2 *>(p + blk * 32 + sub * 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = ((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xFFu;
      out[i] = (float)((int)(b ^ 0x80u) - 0x80) * s;
    }
  } else {  // ASYM4_G32
    const float z = __half2float((kv ? c.zero[1] : c.zero[0])[row * (c.D / kBlock) + blk]);
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p + blk * 16 + sub * 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = fmaf((float)((w >> (4 * i)) & 0xFu), s, z);
  }
}

}  // namespace kvq
