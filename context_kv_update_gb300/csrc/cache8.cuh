// cache8.cuh -- device helpers of the cache held in 8 bits: e4m3 codes, and a power of two for
// every block of tokens and head.
#pragma once

#include <cuda_fp16.h>

#include "dflash_internal.cuh"

namespace dflash {

constexpr int kLeastExp8 = -124;  // below it a bf16 number no longer holds every code's value

// Two fp32 values (at most 448 in magnitude) as e4m3 codes, `lo` in the low byte: nearest, ties
// to even; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The values of two codes.
__device__ __forceinline__ float2 e4m3_values(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(pair)));
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// 2^e for e from -149 to 128 (infinite there).
__device__ __forceinline__ float exp2_int(int e) {
  return e >= -126 ? __int_as_float((e + 127) << 23) : __int_as_float(1 << (e + 149));
}
// A scale byte's factor; 255 is NaN.
__device__ __forceinline__ float scale8_value(uint32_t byte) {
  return byte == 255u ? __int_as_float(0x7fffffff) : exp2_int(static_cast<int>(byte) - 127);
}
// The least exponent e with a <= 448 2^e, of those that are written; a finite, >= 0.
__device__ __forceinline__ int scale8_exponent(float a) {
  const int bits = __float_as_int(a);
  return max((bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0), kLeastExp8);
}

// The exponent of a positive number's leading bit (2^e <= x < 2^(e + 1)); 128 of NaN.
__device__ __forceinline__ int leading_exponent(float x) {
  return static_cast<int>(__float_as_uint(x) >> 23 & 255u) - 127;
}

// Byte offset of a (page, K|V, head) of a layer in the codes, and place of its first scale.
struct Cache8 {
  uint8_t *codes, *scales;
  int block, P, NP, nkv, hd, layer;
  __device__ __forceinline__ int64_t head(int page, int kv, int h) const {
    return ((static_cast<int64_t>(layer) * NP + page) * 2 + kv) * nkv + h;
  }
  __device__ __forceinline__ uint8_t *code(int page, int kv, int h, int slot) const {
    return codes + (head(page, kv, h) * P + slot) * hd;
  }
  __device__ __forceinline__ uint8_t *scale(int page, int kv, int h, int slot) const {
    return scales + head(page, kv, h) * (P / block) + slot / block;
  }
};
inline Cache8 cache8_of(const dflash_geom &g, const dflash_cache8 &c, int layer) {
  return {static_cast<uint8_t *>(c.codes), static_cast<uint8_t *>(c.scales), c.block, g.page_size,
          g.num_pool_pages, g.nkv, g.head_dim, layer};
}

}  // namespace dflash
