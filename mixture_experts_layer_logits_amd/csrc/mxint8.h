// MXINT8 encoding of one block of 32 consecutive row elements on the device: the values of the
// 8-bit activation checkpoints (shared by the row kernels and by the GEMM epilogues).
//
// Value = q 2^(s - 6) with a whole q in [-127, 127] and one byte s + 127 per block.  2^s is the
// smallest power of two with amax <= 127/64 2^s, not below 2^-120 (the factor 2^(6 - s) stays a
// normal number) and not above 2^127 (the last byte); q = round(v 2^(6 - s)), ties to even, held at
// 127 in the one case where it would pass it, amax above 127/64 2^127.  A value is off by at most
// half a step, 2^(s - 7): that is max(amax / 127, 2^-127), since amax > 127/128 2^s above the lowest
// s, and a held one by less than 2^128 - 127 2^121 = 2^121 < amax / 127.  A block that holds an
// infinity or NaN gets the byte 255 and comes back as NaN in all its elements.  Whole 8-bit steps
// instead of E4M3's three mantissa bits: a gradient formed from the checkpoint sees 0.6% noise (rms
// over normal data) instead of 2.6%.
#pragma once
#include "common.h"

namespace moe {

constexpr int kCk8Block = 32;

// Scale byte of a block whose largest magnitude is amax (bits compared, so an infinity or NaN among
// the block's magnitudes has to arrive as such: see ck8_max).
__device__ __forceinline__ int ck8_scale_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int eb = (int)(u >> 23);
  if (eb == 255) return 255;
  const int b = eb + ((u & 0x7fffffu) > 0x7e0000u ? 1 : 0);  // amax = (1 + man / 2^23) 2^(eb - 127)
  return b < 7 ? 7 : (b > 254 ? 254 : b);
}

// Larger of two magnitudes by their bits: as fmaxf for numbers, and NaN wins over everything.
__device__ __forceinline__ float ck8_max(float m, float v) {
  const uint32_t a = __float_as_uint(m), b = __float_as_uint(v) & 0x7fffffffu;
  return __uint_as_float(a > b ? a : b);
}

// 2^(6 - s), exact
__device__ __forceinline__ float ck8_inv_scale(int byte) {
  return __uint_as_float((uint32_t)(byte == 255 ? 127 : 260 - byte) << 23);
}

// Four values of one block -> four codes (bytes 0..3).  v inv + 1.5 2^23 rounds once, to a whole
// number in the low mantissa bits (two's complement).  The one value that can round to 128 (an
// amax above 127/64 2^127, whose scale byte stops at 254) is held at 127.
__device__ __forceinline__ uint32_t ck8_codes4(float a, float b, float c, float d, float inv) {
  constexpr float kMagic = 12582912.f;
  const float hi = kMagic + 127.f, lo = kMagic - 127.f;
  const uint32_t x = __float_as_uint(fminf(fmaxf(fmaf(a, inv, kMagic), lo), hi));
  const uint32_t y = __float_as_uint(fminf(fmaxf(fmaf(b, inv, kMagic), lo), hi));
  const uint32_t z = __float_as_uint(fminf(fmaxf(fmaf(c, inv, kMagic), lo), hi));
  const uint32_t w = __float_as_uint(fminf(fmaxf(fmaf(d, inv, kMagic), lo), hi));
  const uint32_t xy = __builtin_amdgcn_perm(y, x, 0x0c0c0400u), zw = __builtin_amdgcn_perm(w, z, 0x0c0c0400u);
  return xy | (zw << 16);
}

// 2^(s - 6), NaN for the byte 255 (any other byte is taken as it is; the smallest factor, 2^-133, is a subnormal)
__device__ __forceinline__ float ck8_scale(int byte) {
  const float f = __builtin_ldexpf(1.f, byte - 133);
  return byte == 255 ? __uint_as_float(0x7fc00000u) : f;
}

// Code i (0..3) of a word as a float, times the block's factor (exact)
__device__ __forceinline__ void ck8_values4(uint32_t w, float scale, float (&v)[4]) {
  v[0] = (float)(int8_t)(w) * scale;
  v[1] = (float)(int8_t)(w >> 8) * scale;
  v[2] = (float)(int8_t)(w >> 16) * scale;
  v[3] = (float)((int32_t)w >> 24) * scale;
}

}  // namespace moe
