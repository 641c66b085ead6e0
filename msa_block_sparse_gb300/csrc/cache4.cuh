// The 4-bit cache format on the device: e2m1 codes with one e4m3 scale per 16
// channels (msa.h, "Paged cache held in 4 bits").
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "kernels.cuh"

namespace msa {

constexpr int kCodeBytes = kD / 2;                       // one token's codes
constexpr int kScaleBytes = kD / 16;                     // and its scales
constexpr int kSlabCodes = kBlock * kCodeBytes;          // 8192: codes of a page of one head
constexpr int kSlab = kSlabCodes + kBlock * kScaleBytes; // 9216

// Byte offsets inside a slab
__device__ __forceinline__ int slab_code(int slot) { return slot * kCodeBytes; }
__device__ __forceinline__ int slab_scale(int slot) { return kSlabCodes + slot * kScaleBytes; }

// Scale byte of 16 channels from their largest magnitude (after the gain).
// Both roundings are the format's: /6 in fp32 (correctly rounded), then e4m3
// to nearest even with saturation.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  return __nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.0f), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3)));
}

// e2m1 codes of two values divided by a scale s > 0 (rs = 1 / s rounded); low
// nibble = a.  The quotient is formed as x rs and corrected once by its exact
// residual: a quotient on the border of two codes has few bits, so the
// corrected value hits it exactly and the tie goes to the even code, as in the
// definition.  Magnitudes are bounded first so that no step overflows.
__device__ __forceinline__ uint32_t code_pair(float a, float b, float s, float rs) {
  a = fminf(fmaxf(a, -1e30f), 1e30f);
  b = fminf(fmaxf(b, -1e30f), 1e30f);
  float qa = a * rs, qb = b * rs;
  qa = copysignf(fmaf(fmaf(-qa, s, a), rs, qa), a);   // -0 keeps its sign
  qb = copysignf(fmaf(fmaf(-qb, s, b), rs, qb), b);
  return __nv_cvt_float2_to_fp4x2(make_float2(qa, qb), __NV_E2M1, cudaRoundNearest);
}

__device__ __forceinline__ float2 word_f2(uint32_t u) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}

// Codes (8 bytes) and scale byte of 16 bf16 channels (8 packed words).
__device__ __forceinline__ uint2 quantise16(const uint32_t (&x)[8], float inv_gain,
                                            uint32_t* scale) {
  uint32_t m = 0;                                  // largest magnitude as bf16 bits
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, x[i] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);
  if (m >= 0x7F80u) {                              // an infinity or NaN
    *scale = 0x7Fu;
    return make_uint2(0u, 0u);
  }
  const uint32_t sb = scale_byte(__uint_as_float(m << 16) * inv_gain);
  *scale = sb;
  if (sb == 0u) return make_uint2(0u, 0u);
  const float s = scale_value(sb), rs = __frcp_rn(s);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = word_f2(x[i]);
    w[i >> 2] |= code_pair(f.x * inv_gain, f.y * inv_gain, s, rs) << (8 * (i & 3));
  }
  return make_uint2(w[0], w[1]);
}

// 8 codes (one word, channel order) as four packed fp16 pairs, exact.  The
// bytes are unpacked in the conversion's own block: taken out by shifts and masks
// they cost two more instructions each, and this unpacking bounds the score kernel.
__device__ __forceinline__ void codes_half2(uint32_t w, __half2 (&h)[4]) {
  uint32_t r[4];
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<__half2*>(&r[i]);
}

}  // namespace msa
