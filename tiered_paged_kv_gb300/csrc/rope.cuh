// The angles of rotary positions, for the kernels that rotate (see kv_rope.cu).
#pragma once
#include "paged.cuh"

namespace tpk {

// frac(f / (2 pi)) in units of 2^-64 turns, |f| < 2^32.
__device__ __forceinline__ uint64_t turns64(float f) {
  const uint32_t w = __float_as_uint(f);
  const int e = (w >> 23) & 0xff;
  const uint32_t m = (w & 0x7fffff) | (e ? 0x800000u : 0);
  // 1 / (2 pi) * 2^96
  const unsigned __int128 c = ((unsigned __int128)0x28be60dbu << 64) | 0x9391054a7f09d5f4ull;
  const int shift = 182 - (e ? e : 1);  // f = m 2^(e - 150), so F = m c 2^(e - 150) 2^(64 - 96)
  const unsigned __int128 x = m * c;
  const uint64_t t = shift < 128 ? (uint64_t)(x >> shift) : 0;  // at least 24
  return (w >> 31) ? 0 - t : t;
}

// (cos, sin) of pos * f.
__device__ __forceinline__ float2 turned_by(float f, int64_t pos) {
  const uint64_t angle = turns64(f) * (uint64_t)pos;
  float s, c;
  sincospif((float)(int32_t)((angle + 0x80000000u) >> 32) * 0x1p-31f, &s, &c);  // of pi * (2 * turns)
  if (!(fabsf(f) < 0x1p32f)) s = c = __int_as_float(0x7fffffff);
  return make_float2(c, s);
}

}  // namespace tpk
