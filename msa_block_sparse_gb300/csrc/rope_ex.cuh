// Rotation of a head's channels held in registers: a row of D channels belongs to D / 8
// threads with 8 channels each, both halves of every pair in one thread.  Shared by the
// prologue (rope_ex.cu) and the append to 16-bit pages (cache16.cu).
#pragma once
#include "kernels.cuh"

namespace msa {

constexpr int kRxMaxPairs = 128;

// Angle per position of each pair as the 64-bit fixed-point fraction of a turn
struct RxTurns {
  unsigned long long f[kRxMaxPairs];
};

RxTurns rx_turns(const msa_rope_t& rope);

// cos and sin of position * turn
__device__ __forceinline__ float2 rx_cos_sin(int pos, unsigned long long turn) {
  const long long ang = static_cast<long long>(
      static_cast<unsigned long long>(static_cast<long long>(pos)) * turn);
  float2 r;
  sincospif(static_cast<float>(ang) * 1.0842021724855044e-19f, &r.y, &r.x);   // * 2^-63
  return r;
}

__device__ __forceinline__ float2 bf2(uint32_t u) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}

// The 8 channels of a thread: pieces [off0, off0 + 4) and [off1, off1 + 4).  In
// the rotated part of the "half" layout the pieces are partners (off1 = off0 + R/2);
// elsewhere they are 8 consecutive channels.
struct RxLane {
  int off0, off1, pair;   // pair: first frequency
  bool rot;
};

template <bool kHalf>
__device__ __forceinline__ RxLane rx_lane(int c, int R) {
  RxLane l;
  l.rot = 8 * c < R;
  l.off0 = kHalf && l.rot ? 4 * c : 8 * c;
  l.off1 = kHalf && l.rot ? 4 * c + (R >> 1) : 8 * c + 4;
  l.pair = 4 * c;
  return l;
}

struct RxRow {
  uint2 a, b;
};

template <bool kHalf>
__device__ __forceinline__ RxRow rx_load(const __nv_bfloat16* row, const RxLane& l) {
  RxRow r;
  if (kHalf) {
    r.a = __ldcs(reinterpret_cast<const uint2*>(row + l.off0));
    r.b = __ldcs(reinterpret_cast<const uint2*>(row + l.off1));
  } else {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(row + l.off0));
    r.a = make_uint2(u.x, u.y);
    r.b = make_uint2(u.z, u.w);
  }
  return r;
}

// The same from shared memory
template <bool kHalf>
__device__ __forceinline__ RxRow rx_read(const __nv_bfloat16* row, const RxLane& l) {
  RxRow r;
  if (kHalf) {
    r.a = *reinterpret_cast<const uint2*>(row + l.off0);
    r.b = *reinterpret_cast<const uint2*>(row + l.off1);
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(row + l.off0);
    r.a = make_uint2(u.x, u.y);
    r.b = make_uint2(u.z, u.w);
  }
  return r;
}

// The 8 channels as four packed values: v[0], v[1] the first channels of the thread's
// pairs 0, 1 and 2, 3, v[2], v[3] their second channels, for either layout.
template <bool kHalf>
__device__ __forceinline__ void rx_unpack(const RxRow& r, float2 (&v)[4]) {
  const float2 a = bf2(r.a.x), b = bf2(r.a.y), c = bf2(r.b.x), d = bf2(r.b.y);
  if (kHalf) {
    v[0] = a;
    v[1] = b;
    v[2] = c;
    v[3] = d;
  } else {
    v[0] = make_float2(a.x, b.x);
    v[1] = make_float2(c.x, d.x);
    v[2] = make_float2(a.y, b.y);
    v[3] = make_float2(c.y, d.y);
  }
}

template <bool kHalf>
__device__ __forceinline__ RxRow rx_pack(const float2 (&v)[4]) {
  RxRow r;
  if (kHalf) {
    r.a = make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y));
    r.b = make_uint2(pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
  } else {
    r.a = make_uint2(pack_bf16x2(v[0].x, v[2].x), pack_bf16x2(v[0].y, v[2].y));
    r.b = make_uint2(pack_bf16x2(v[1].x, v[3].x), pack_bf16x2(v[1].y, v[3].y));
  }
  return r;
}

template <bool kHalf>
__device__ __forceinline__ void rx_store(__nv_bfloat16* row, const RxLane& l, const RxRow& r) {
  if (kHalf) {
    *reinterpret_cast<uint2*>(row + l.off0) = r.a;
    *reinterpret_cast<uint2*>(row + l.off1) = r.b;
  } else {
    *reinterpret_cast<uint4*>(row + l.off0) = make_uint4(r.a.x, r.a.y, r.b.x, r.b.y);
  }
}

// Turns the 8 channels: v[p] = v[p] * c[p] + v[p ^ 2] * s[p]; signs and any factors
// are in the coefficients.  Channels that are not rotated (`rot` false) take no part of
// another one: their sines of 0 would make a NaN of an infinity there.
__device__ __forceinline__ void rx_turn(float2 (&v)[4], const float2 (&c)[4], const float2 (&s)[4], bool rot) {
  float2 o[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 t = __fmul2_rn(v[p ^ 2], s[p]);
    o[p] = __ffma2_rn(v[p], c[p], make_float2(rot ? t.x : 0.f, rot ? t.y : 0.f));
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) v[p] = o[p];
}

// Coefficients of one token: cos and +-sin (dir = 1 forward, -1 back), each times
// the factor w of the value it multiplies (w = 1 + weight, or all ones).
__device__ __forceinline__ void rx_coefficients(const float* tab, int half, const RxLane& l,
                                                const float2 (&w)[4], float dir, float2 (&c)[4],
                                                float2 (&s)[4]) {
  float4 cv = make_float4(1.f, 1.f, 1.f, 1.f), sv = make_float4(0.f, 0.f, 0.f, 0.f);
  if (l.rot) {
    cv = *reinterpret_cast<const float4*>(tab + l.pair);
    sv = *reinterpret_cast<const float4*>(tab + half + l.pair);
  }
  const float2 c2[2] = {make_float2(cv.x, cv.y), make_float2(cv.z, cv.w)};
  const float2 s2[2] = {make_float2(dir * sv.x, dir * sv.y), make_float2(dir * sv.z, dir * sv.w)};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    c[p] = __fmul2_rn(w[p], c2[p & 1]);
    const float2 t = __fmul2_rn(w[p ^ 2], s2[p & 1]);
    s[p] = p < 2 ? make_float2(-t.x, -t.y) : t;
  }
}

}  // namespace msa
