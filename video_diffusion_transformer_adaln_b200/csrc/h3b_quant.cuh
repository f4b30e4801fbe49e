// Warp reductions and the per-row int8 quantizer's decision, shared by the row
// kernels (k_rowops.cu, k_resnorm.cu).
#pragma once

#include "h3b_common.cuh"

namespace h3b {

// ---------------------------------------------------------------------------
// Warp / block reductions
// ---------------------------------------------------------------------------
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// A row's largest magnitude is NaN where a value is, so that its scale is, and its products do not pass for finite ones.
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// The quantizer decision, in binary32 exactly as the method states it:
// scale = absmax / 127, code = round-half-even(v / scale) clamped to [-127, 127];
// absmax == 0 gives code 0.
__device__ __forceinline__ int quant_code(float v, float scale, float absmax) {
  if (absmax == 0.0f) return 0;
  int c = __float2int_rn(__fdiv_rn(v, scale));
  return max(-127, min(127, c));
}
// The same decision without a division per element: t = v * RN(1/scale)
// differs from RN(v / scale) by less than 2^-15.4 for |t| <= 127.5, so when t
// is farther than 2^-14 from a half-integer both round to the same integer;
// only then-near ties take the correctly rounded division. Bit-identical to
// quant_code for every input (absmax > 0).
constexpr float kTieGuard = 0.5f - 1.0f / 16384.0f;
__device__ __forceinline__ int quant_code_fast(float v, float scale, float rcp) {
  float t = v * rcp;
  float c = rintf(t);
  if (fabsf(t - c) > kTieGuard) c = rintf(__fdiv_rn(v, scale));
  return max(-127, min(127, (int)c));
}
// Eight codes of one 16-byte bf16 vector without a branch per element:
// a = fma(v, RN(1/scale), 1.5 * 2^23) rounds the exact product p = v * RN(1/scale)
// to the nearest integer c (ties to even) in the low mantissa bits, whose low
// byte is the int8 code (|p| <= 127.5 never yields -128), and
// dd = fma(v, RN(1/scale), -c) is p - c to within 2^-25. p differs from v / scale
// by at most 127.5 * 2^-24 = 2^-17 and RN(v / scale) from v / scale by at most
// 2^-18, so where |dd| <= 0.5 - 2^-14 the binary32 decision rint(RN(v / scale))
// is c. The largest |dd| is tracked and the dd are returned; if an element lies
// closer to a half-integer the caller patches those elements with quant8_slow.
__device__ __forceinline__ uint2 quant8_fast(uint4 v, float rcp, float& worst, float2 (&dds)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const float2 r2 = make_float2(rcp, rcp), M2 = make_float2(12582912.0f, 12582912.0f);
  const float2 nM2 = make_float2(-12582912.0f, -12582912.0f);
  uint32_t b[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
    const float2 a = __ffma2_rn(x, r2, M2);
    const float2 c = __fadd2_rn(a, nM2);  // exact
    const float2 dd = __ffma2_rn(x, r2, make_float2(-c.x, -c.y));
    worst = fmaxf(worst, fmaxf(fabsf(dd.x), fabsf(dd.y)));
    dds[e] = dd;
    b[2 * e] = __float_as_uint(a.x);
    b[2 * e + 1] = __float_as_uint(a.y);
  }
  const uint32_t lo = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  const uint32_t hi = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  return make_uint2(lo, hi);
}
__device__ __forceinline__ uint32_t pack4_i8(int a, int b, int c, int d) {
  return (uint32_t)(a & 0xFF) | ((uint32_t)(b & 0xFF) << 8) | ((uint32_t)(c & 0xFF) << 16) |
         ((uint32_t)(d & 0xFF) << 24);
}
// Scales below this take the division for every element (quant8_slow); at or
// above it RN(1/scale) is finite and every quantity below is a normal number.
constexpr float kMinFastScale = 0x1p-100f;
// The codes of a vector whose fast path saw a near tie, patched element by
// element. On bf16 rows a few elements in a thousand have v * RN(1/scale) within
// 2^-14 of a half-integer (bf16 values over a bf16 absmax put many quotients on
// or next to one, most of them exactly), so only those elements, found from the
// fast path's distances dd, are decided again, without a division: with h the
// half-integer next to the product and r = v - h * scale,
//   r is exact in binary32 (one fma): v and h * scale are multiples of
//     ulp(scale) / 2, and |r| < 2^-13 scale (|v / scale - h| < 2^-14 + 2^-17)
//     needs fewer than 13 bits of them;
//   RN(v / scale) == h exactly when |r| <= scale * ulp(h) / 2 (h has at most 9
//     significant bits, so a quotient midway to h's neighbour rounds to h; the
//     smaller spacing just below |h| = 0.5 changes no code), and then the code
//     is the even integer next to h (rint(h));
//   otherwise the code is h + 0.5 when r > 0 and h - 0.5 when r < 0.
// A zero, subnormal or tiny scale (the whole row) takes the division itself.
// kGivenDd: the fast path's dd are passed in (d0..d3); otherwise they are
// recomputed here, which keeps the caller's live registers down.
template <bool kGivenDd>
__device__ __noinline__ uint2 quant8_slow(uint4 v, float scale, float rcp, float absmax, uint2 code, float2 d0,
                                         float2 d1, float2 d2, float2 d3) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (!(scale >= kMinFastScale)) {
    int c[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[2 * e] = quant_code(bf16_lo(w[e]), scale, absmax);
      c[2 * e + 1] = quant_code(bf16_hi(w[e]), scale, absmax);
    }
    return make_uint2(pack4_i8(c[0], c[1], c[2], c[3]), pack4_i8(c[4], c[5], c[6], c[7]));
  }
  uint32_t word[2] = {code.x, code.y};
  const float given[8] = {d0.x, d0.y, d1.x, d1.y, d2.x, d2.y, d3.x, d3.y};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
    const float c0 = fmaf(x, rcp, 12582912.0f) - 12582912.0f;  // as quant8_fast
    const float dd = kGivenDd ? given[e] : fmaf(x, rcp, -c0);
    if (fabsf(dd) > kTieGuard) {
      const float h = c0 + copysignf(0.5f, dd);
      const float r = fmaf(-h, scale, x);
      const float us = __uint_as_float((__float_as_uint(h) & 0x7F800000u) - (24u << 23)) * scale;
      const float c = fabsf(r) <= us ? rintf(h) : (r > 0.0f ? h + 0.5f : h - 0.5f);
      const uint32_t byte = (uint32_t)max(-127, min(127, (int)c)) & 0xFFu;
      const int k = e >> 2, sh = 8 * (e & 3);
      word[k] = (word[k] & ~(0xFFu << sh)) | (byte << sh);
    }
  }
  return make_uint2(word[0], word[1]);
}
// Eight codes of one bf16 vector, bit-identical to quant_code on each element.
template <bool kGivenDd>
__device__ __forceinline__ uint2 quant8(uint4 v, float scale, float rcp, float absmax) {
  float worst = scale >= kMinFastScale ? 0.0f : 1.0f;  // zero, tiny or NaN scale: the slow path decides
  float2 dd[4];
  uint2 code = quant8_fast(v, rcp, worst, dd);
  if (worst > kTieGuard) code = quant8_slow<kGivenDd>(v, scale, rcp, absmax, code, dd[0], dd[1], dd[2], dd[3]);
  return code;
}

}  // namespace h3b
