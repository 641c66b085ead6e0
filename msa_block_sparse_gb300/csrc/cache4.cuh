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
// Both roundings are the format's: /6 in fp32, then e4m3 to nearest even with
// saturation.  The quotient is a times the rounded 1/6, corrected by its exact
// residual a - 6 q, which rounds it correctly (Markstein 1990) unless it underflows, far
// below the smallest scale; what is cut off saturates all the same.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  constexpr float kSixth = 1.0f / 6.0f;
  const float a = fminf(amax, 0x1p100f), q = a * kSixth;
  return __nv_cvt_float_to_fp8(fmaf(fmaf(-6.0f, q, a), kSixth, q), __NV_SATFINITE, __NV_E4M3);
}

// 1 / x to 2^-22 or so, for normal x
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3)));
}

__device__ __forceinline__ float2 word_f2(uint32_t u) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}

// e2m1 codes of the pair x divided by a scale s > 0, from nx = -x and nrs near -1 / s;
// low nibble = x.x.  The quotient q = nx nrs, good to 2^-21, is corrected once by its exact
// residual q s - x and is then off by 2^-40 before its last rounding: a quotient on the
// border of two codes has few bits, so the corrected value hits it exactly and the tie
// goes to the even code, as in the definition; any other is 2^-12 or more away (8 bits over
// 4).  -0 stays -0.
__device__ __forceinline__ uint32_t code_pair(float2 nx, float s, float nrs) {
  const float2 r2 = make_float2(nrs, nrs);
  const float2 q = __fmul2_rn(nx, r2);
  const float2 e = __ffma2_rn(q, make_float2(s, s), nx);
  return __nv_cvt_float2_to_fp4x2(__ffma2_rn(e, r2, q), __NV_E2M1, cudaRoundNearest);
}

// The negatives of two packed bf16: an integer addition flips a float's sign bit
__device__ __forceinline__ float2 neg_word_f2(uint32_t u) {
  return make_float2(__uint_as_float(u * 0x10000u + 0x80000000u),
                     __uint_as_float((u & 0xFFFF0000u) ^ 0x80000000u));
}

// Scale of 16 channels from their largest magnitude m (bf16 bits): the byte, and
// in *s what the values are divided by (scale times gain; 0: all codes are 0).
// Values that could overflow the quotient's residual (only past 2^100 times the
// largest held value) are to be cut to +-*cut first.
struct Scale16 {
  uint32_t byte;
  float s, nrs, cut;     // nrs: near -1 / s; cut: 0 = no need
};

__device__ __forceinline__ Scale16 scale16(uint32_t m, float gain, float inv_gain) {
  Scale16 r;
  r.cut = 0.f;
  if (m >= 0x7F80u) {                              // an infinity or NaN
    r.byte = 0x7Fu;
    r.s = r.nrs = 0.f;
    return r;
  }
  const float amax = __uint_as_float(m << 16);
  r.byte = scale_byte(amax * inv_gain);
  r.s = scale_value(r.byte) * gain;
  r.nrs = r.byte ? -rcp(r.s) : 0.f;
  if (amax * 0x1p-30f > r.s && r.byte) r.cut = 8.f * r.s;   // saturated: any cut above 6 scales
  return r;
}

// x (packed bf16) cut to +-sc.cut
__device__ __forceinline__ uint32_t cut_word(const Scale16& sc, uint32_t x) {
  const float2 f = word_f2(x);
  return pack_bf16x2(fminf(fmaxf(f.x, -sc.cut), sc.cut), fminf(fmaxf(f.y, -sc.cut), sc.cut));
}

__device__ __forceinline__ uint32_t code_word(const Scale16& sc, uint32_t x) {
  return code_pair(neg_word_f2(x), sc.s, sc.nrs);
}

// Codes (8 bytes) and scale byte of 16 bf16 channels (8 packed words).
__device__ __forceinline__ uint2 quantise16(uint32_t (&x)[8], float gain, float inv_gain,
                                            uint32_t* scale) {
  uint32_t m = 0;                                  // largest magnitude as bf16 bits
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, x[i] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);
  const Scale16 sc = scale16(m, gain, inv_gain);
  *scale = sc.byte;
  if (sc.cut != 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = cut_word(sc, x[i]);
  }
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = code_word(sc, x[i]);
  if (sc.s == 0.f) return make_uint2(0u, 0u);
  return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
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
