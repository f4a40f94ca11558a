// Device pieces of the block-128 FP8 format (see fp8.hip for the definition).
#pragma once

#include "ft_internal.hpp"

namespace ft {

constexpr int kFp8Block = 128;  // elements of the contraction axis that share a scale

struct Fp8Scale {
  float scale, inv;  // 2^e and 2^-e (NaN and 0 for a block with a NaN or an infinity)
};

// The block scale from the largest magnitude's fp32 bits: 448 = 1.75 * 2^8, so
// e is the maximum's exponent - 8, one more if its fraction is above 1.75.
__device__ __forceinline__ Fp8Scale fp8_scale(uint32_t amax) {
  int e = int(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased exponent of the scale
  e = max(e, 1);
  Fp8Scale s;
  const bool bad = amax >= 0x7f800000u;
  s.scale = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(uint32_t(e) << 23);
  s.inv = bad ? 0.f : __uint_as_float(uint32_t(254 - e) << 23);
  return s;
}

__device__ __forceinline__ void fp8_load8(const uint16_t *p, float (&v)[8]) {
  const u32x4 d = ld16(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = d[i];
    v[2 * i] = __uint_as_float(w << 16);
    v[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
  }
}
__device__ __forceinline__ void fp8_load8(const float *p, float (&v)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}

// Largest magnitude of 8 values as bits: unsigned order is the order of
// magnitudes, with infinity and every NaN above the finite ones.
__device__ __forceinline__ uint32_t abs_max8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// Maximum over the 16 lanes of a wave's row, in each of them.
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t x) {
  x = max(x, dpp_u32<0xB1>(x, x));
  x = max(x, dpp_u32<0x4E>(x, x));
  x = max(x, dpp_u32<0x141>(x, x));
  x = max(x, dpp_u32<0x140>(x, x));
  return x;
}

// Four scaled values -> four E4M3 codes.  A block with a NaN or an infinity
// has inv = 0: its NaN * 0 is kept out of the codes.
__device__ __forceinline__ uint32_t fp8_codes4(float a, float b, float c, float d, float inv) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, r, true);
  return inv == 0.f ? 0u : uint32_t(r);
}
__device__ __forceinline__ u32x2 fp8_codes8(const float (&v)[8], float inv) {
  return u32x2{fp8_codes4(v[0], v[1], v[2], v[3], inv), fp8_codes4(v[4], v[5], v[6], v[7], inv)};
}

// Eight E4M3 codes (two dwords) -> eight bf16, in order.  Exact: an E4M3 value
// has 4 significant bits and an exponent that bf16 holds.
__device__ __forceinline__ bf16x8 fp8x8_to_bf16x8(uint32_t lo, uint32_t hi) {
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  bf16x8 r;
  r[0] = p0[0]; r[1] = p0[1]; r[2] = p1[0]; r[3] = p1[1];
  r[4] = p2[0]; r[5] = p2[1]; r[6] = p3[0]; r[7] = p3[1];
  return r;
}

}  // namespace ft
