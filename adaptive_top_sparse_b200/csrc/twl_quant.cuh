// INT4 of one token row, shared by the cache kernels and the 4-bit attention.
#pragma once

#include "twl_common.cuh"

namespace twl {

struct Half4 {
  uint32_t lo, hi;  // channels (4l, 4l+1) and (4l+2, 4l+3)
};

__device__ __forceinline__ Half4 load_half4(const uint16_t* p) {
  uint2 v = *reinterpret_cast<const uint2*>(p);
  return Half4{v.x, v.y};
}

// One code: n = min(L, rint_even(fp32(x - z) / s)); x - z >= 0 because z is the row minimum.
__device__ __forceinline__ uint32_t code_of(uint32_t xbits, float z, float s, float levels) {
  float x = __half2float(__ushort_as_half((unsigned short)(xbits & 0xFFFFu)));
  float r = rintf(__fdiv_rn(__fsub_rn(x, z), s));
  r = fminf(fmaxf(r, 0.f), levels);
  return (uint32_t)r;
}
__device__ __forceinline__ uint32_t nibble(uint32_t xbits, float z, float s) {
  return code_of(xbits, z, s, 15.f);
}

// INT4 of one token row held by a warp (lane l: channels 4l .. 4l+3): returns the lane's 4
// nibbles (channel 2j in the low nibble of byte j) and, in *sz, fp16 scale | fp16 zero << 16.
__device__ __forceinline__ uint16_t quantize_row_warp(const Half4& v, uint32_t* sz) {
  int k0 = f16_key(v.lo), k1 = f16_key(v.lo >> 16), k2 = f16_key(v.hi), k3 = f16_key(v.hi >> 16);
  int kmn = min(min(k0, k1), min(k2, k3));
  int kmx = max(max(k0, k1), max(k2, k3));
  kmn = __reduce_min_sync(0xffffffffu, kmn);
  kmx = __reduce_max_sync(0xffffffffu, kmx);
  const uint32_t mn_bits = f16_from_key(kmn), mx_bits = f16_from_key(kmx);
  const float mn = __half2float(__ushort_as_half((unsigned short)mn_bits));
  const float mx = __half2float(__ushort_as_half((unsigned short)mx_bits));
  const __half s16 = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 15.f));
  const float s = __half2float(s16);
  uint32_t packed = 0;
  if (s != 0.f) {
    uint32_t n0 = nibble(v.lo, mn, s), n1 = nibble(v.lo >> 16, mn, s);
    uint32_t n2 = nibble(v.hi, mn, s), n3 = nibble(v.hi >> 16, mn, s);
    packed = n0 | (n1 << 4) | (n2 << 8) | (n3 << 12);
  }
  *sz = uint32_t(__half_as_ushort(s16)) | (mn_bits << 16);
  return (uint16_t)packed;
}

}  // namespace twl
