// Beam search's selection: of all W * V continuations of a prompt's W beams the K with the
// best score s_w + log softmax(x_w)_v.
//
// Bound by memory in the limit: the logits are read once (the only large input).  Measured: 32
// prompts x 8 beams x 131,072 bf16 logits (67 MB) 24 us; alone and with cold caches the scan takes
// 22 (3.1 TB/s; an exponential per value and its end fill half of the issue slots) and the merge
// 9, of which about 7 are launch and latency.  4 beams x 32,000 fp32 7.5 us, latency.
//
//   beam_scan_kernel   CTA = a slice of one beam's vocabulary.  One pass: every thread sums
//                      the exponentials of its values (2^(x log2 e - ref), ref a whole
//                      number) and keeps the maximum of each 16 or so of them.  The maxima
//                      give a bound that the slice's K best values reach; the few pieces that
//                      hold any such value are read again (from L2) and ranked.  Within
//                      a beam the order of the scores is that of the values, so that nothing
//                      else of the slice can be chosen.
//   beam_merge_kernel  CTA = a prompt.  Log-sum-exp of its beams from the slices, scores of
//                      the slices' candidates in 64 bits, the best K in order; equal scores
//                      by the beam, then by the values, as the slices had them.
//
// K best of n values without sorting: the values are dealt into groups, and the K-th
// largest of the groups' maxima is a bound that at least K values reach; of values in no
// particular order about 1.4 K do.  These few are ranked by counting.  Where far more reach
// it (equal values at the border), the slice is taken tile by tile with unique keys (value,
// then the lower index): at most the K best threads hold anything above the bound then.
#include "kernels.cuh"

namespace msa {

namespace {

constexpr int kBmThreads = 256;
constexpr int kBmMaxK = 64;
constexpr int kBmMaxW = 64;
constexpr int kBmValues = 16;                          // of a thread and tile
constexpr int kBmTile = kBmThreads * kBmValues;
constexpr int kBmCap = kBmMaxK * kBmValues + kBmThreads;   // keys of the buffer
constexpr int kBmPieces = 32;                          // maxima that a thread keeps
constexpr int kBmList = 1024;                          // pieces read again
constexpr int kBmCandidates = 16384;                   // of a prompt, at most
constexpr int kBmMergeThreads = 512;
constexpr float kBmLog2e = 1.4426950216293335f;        // log2 e in fp32, 1.33e-8 of it too small
constexpr double kBmLn2 = 0.69314718055994530942, kBmRef = kBmLn2 * (1.4426950408889634 / 1.4426950216293335);
constexpr float kBmHuge = 0x1p28f;                     // beyond: |x log2 e - ref| could overflow 2^127
constexpr float kBmLow = -0x1p29f;                     // reference of values below -2^28 alone: below any other

// Order of floats as order of unsigned integers (0: below -infinity, used for "nothing")
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ unsigned long long ordered(double x) {
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
  return u >> 63 ? ~u : u | (1ull << 63);
}

// A value and its place in the vocabulary: larger is better, no two are equal
__device__ __forceinline__ unsigned long long key_of(float x, uint32_t idx) {
  return (static_cast<unsigned long long>(ordered(x)) << 32) | (0xFFFFFFFFu - idx);
}

// Sum of e^x of a slice: sum * 2^ref, ref a whole number (-infinity: the sum is 0), so that
// joining two sums rounds nothing but the addition.  Exponents are x times fp32's log2 e, whose
// 1.33e-8 is put right for x = ref ln 2, from which the terms that count are a few away:
// ref ln 2 (1 + 1.33e-8) stands for ref.  ref = kBmLow: nothing above -2^28, sum is a count.
struct BeamScan {
  float ref, sum;
};

template <typename T>
struct Vec;      // 16 bytes of logits
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float* x) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 part(const float* p, int lo, int hi) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = i >= lo && i < hi ? p[i] : -INFINITY;
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ uint4 nothing() {
    return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 part(const __nv_bfloat16* p, int lo, int hi) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = 2 * i >= lo && 2 * i < hi ? __bfloat16_as_ushort(p[2 * i]) : 0xFF80u;
      const uint32_t b =
          2 * i + 1 >= lo && 2 * i + 1 < hi ? __bfloat16_as_ushort(p[2 * i + 1]) : 0xFF80u;
      w[i] = a | b << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ uint4 nothing() {
    return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
  }
};

__device__ __forceinline__ float bm_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^d of a whole number d <= 0
__device__ __forceinline__ float bm_scale(float d) {
  return d < -126.f ? 0.f : __int_as_float((static_cast<int>(d) + 127) << 23);
}

// NaN counts as -infinity, what lies above 2^28 as 2^28, -0 as 0: keys go by the bits
__device__ __forceinline__ float plain(float x) {
  return x != x ? -INFINITY : x == 0.f ? 0.f : fminf(x, kBmHuge);
}

struct ScanSmem {
  unsigned long long key[kBmCap];
  unsigned long long best[kBmMaxK];
  alignas(16) float group[128];
  union {
    float piece[kBmPieces][kBmThreads];                // maxima of the pass
    unsigned long long gkey[kBmThreads];               // later: the threads' best keys
  };
  int list[kBmList];
  float sum[kBmThreads / 32], ref[kBmThreads / 32];
  float bound;
  unsigned long long bound_key;
  int count, pieces;
};

// The K best of the sm.count keys in sm.key, in order, into sm.best; count <= kBmCap.
// All threads; sm.count becomes what is kept.  Ranks by counting; more than kBmThreads keys
// (rare) are first cut by the bound of their groups.
__device__ __forceinline__ void bm_rank(ScanSmem& sm, int K) {
  __syncthreads();
  int n = sm.count;
  const int tid = threadIdx.x;
  while (n > kBmThreads) {
    // groups: the keys i, i + 256, ... of a thread
    unsigned long long mine[(kBmCap + kBmThreads - 1) / kBmThreads], top = 0;
#pragma unroll
    for (int k = 0; k < (kBmCap + kBmThreads - 1) / kBmThreads; ++k) {
      const int i = tid + k * kBmThreads;
      mine[k] = i < n ? sm.key[i] : 0;
      top = mine[k] > top ? mine[k] : top;
    }
    sm.gkey[tid] = top;
    __syncthreads();
    int above = 0;
#pragma unroll 8
    for (int i = 0; i < kBmThreads; ++i) above += sm.gkey[i] > top;
    if (above == K - 1) sm.bound_key = top;      // n > 256 >= K: there is a K-th group
    if (tid == 0) sm.count = 0;
    __syncthreads();
    const unsigned long long bound = sm.bound_key;
#pragma unroll
    for (int k = 0; k < (kBmCap + kBmThreads - 1) / kBmThreads; ++k)
      if (mine[k] >= bound) sm.key[atomicAdd(&sm.count, 1)] = mine[k];
    __syncthreads();
    n = sm.count;
  }
  if (tid < n) {
    const unsigned long long mine = sm.key[tid];
    int above = 0;
#pragma unroll 8
    for (int i = 0; i < n; ++i) above += sm.key[i] > mine;
    if (above < K) sm.best[above] = mine;
  }
  __syncthreads();
  n = min(n, K);
  if (tid < n) sm.key[tid] = sm.best[tid];
  if (tid == 0) sm.count = n;
  __syncthreads();
}

}  // namespace

// grid (slices, rows)
template <typename T>
__global__ void __launch_bounds__(kBmThreads, 4) beam_scan_kernel(
    const T* __restrict__ logits, long long ld, int V, int K, const uint8_t* __restrict__ finished,
    BeamScan* __restrict__ stats, unsigned long long* __restrict__ keys) {
  pdl_enter();
  using L = Vec<T>;
  constexpr int kVecs = kBmValues / L::kN;
  __shared__ ScanSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slices = gridDim.x, row = blockIdx.y;
  if (finished && finished[row]) return;                 // goes on by the pad token alone
  const T* x = logits + static_cast<long long>(row) * ld;
  // vectors of 16 aligned bytes; the row begins `skew` values into the first one
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const T* xa = x - skew;
  const int nvec = (skew + V + L::kN - 1) / L::kN;
  const int v0 = static_cast<int>(static_cast<long long>(nvec) * blockIdx.x / slices);
  const int v1 = static_cast<int>(static_cast<long long>(nvec) * (blockIdx.x + 1) / slices);
  auto load = [&](int v) -> uint4 {
    if (v >= v1) return L::nothing();
    const int lo = v * L::kN;
    if (lo >= skew && lo + L::kN <= skew + V)
      return __ldcs(reinterpret_cast<const uint4*>(xa + lo));
    return L::part(xa + lo, skew - lo, skew + V - lo);
  };
  // this thread's sum is (sum - less) * 2^ref: `less` is what rounding added, as a slice of the largest
  // vocabulary has 4,096 tiles, whose errors can all go one way (equal logits)
  float ref = -INFINITY, sum = 0.f, less = 0.f;
  constexpr int kTile = kVecs * kBmThreads;              // vectors of a tile
  const int tiles = (v1 - v0 + kTile - 1) / kTile, per = (tiles + kBmPieces - 1) / kBmPieces;
  float top = -INFINITY, piece = -INFINITY;              // maxima: of all, of `per` tiles
  if (tid == 0) sm.count = sm.pieces = 0;
  uint4 raw[kVecs];
  // tiles that lie within the slice and the row, but for the vectors at the row's ends
  const int whole_lo = skew > 0 ? 1 : 0, whole_hi = min(v1, (skew + V) / L::kN);
  auto load_tile = [&](int t) {
    const int v = v0 + t * kTile;
    if (v >= whole_lo && v + kTile <= whole_hi) {
      const uint4* p = reinterpret_cast<const uint4*>(xa + static_cast<size_t>(v) * L::kN) + tid;
#pragma unroll
      for (int u = 0; u < kVecs; ++u) raw[u] = __ldcs(p + u * kBmThreads);
    } else {
#pragma unroll
      for (int u = 0; u < kVecs; ++u) raw[u] = load(v + u * kBmThreads + tid);
    }
  };
  auto place = [&](int t, int i) -> uint32_t {           // value i of this thread and tile t
    return static_cast<uint32_t>((v0 + t * kTile + (i / L::kN) * kBmThreads + tid) * L::kN + i % L::kN - skew);
  };
  load_tile(0);
  float* mine = &sm.piece[0][tid];                       // where the next maximum goes
  for (int t = 0, left = per; t < tiles; ++t) {
    float val[kBmValues];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) L::unpack(raw[u], val + u * L::kN);
    if (t + 1 < tiles) load_tile(t + 1);
    // ---- maximum and sum of exponentials of this thread's values.  x log2 e - ref with ref
    // whole is rounded relative to itself, however large x is.
    float best = -INFINITY, part = 0.f, to = ref;
    auto scan = [&]() {
      best = fmaxf(val[0], val[1]);
#pragma unroll
      for (int i = 2; i < kBmValues; i += 2) best = max3f(best, val[i], val[i + 1]);
      to = fmaxf(ref, rintf(best * kBmLog2e));
      const float2 hi = make_float2(kBmLog2e, kBmLog2e);
      const float2 r = make_float2(-to, -to);
      float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < kBmValues; i += 2) {
        const float2 y = __ffma2_rn(make_float2(val[i], val[i + 1]), hi, r);
        acc[(i >> 1) & 1] = __fadd2_rn(acc[(i >> 1) & 1], make_float2(bm_ex2(y.x), bm_ex2(y.y)));
      }
      const float2 a = __fadd2_rn(acc[0], acc[1]);
      part = a.x + a.y;
    };
    scan();
    if (best > -INFINITY && !(part < INFINITY && fabsf(best) < kBmHuge)) {   // NaN, +infinity, huge
#pragma unroll
      for (int i = 0; i < kBmValues; ++i) val[i] = plain(val[i]);
      scan();
      if (best < -kBmHuge) {                             // they count where the beam has nothing else, and alike
        to = fmaxf(ref, kBmLow);
        part = 0.f;
#pragma unroll
        for (int i = 0; i < kBmValues; ++i) part += val[i] > -INFINITY && to == kBmLow ? 1.f : 0.f;
      }
    }
    if (best > -INFINITY) {
      if (to != ref) {
        const float f = ref > -INFINITY ? bm_scale(ref - to) : 0.f;
        sum *= f;
        less *= f;
      }
      const float y = part - less, all = sum + y;
      less = (all - sum) - y;
      sum = all;
      ref = to;
    }
    piece = fmaxf(piece, best);
    if (--left == 0 || t + 1 == tiles) {
      *mine = piece;
      mine += kBmThreads;
      top = fmaxf(top, piece);
      piece = -INFINITY;
      left = per;
    }
  }
  // ---- bound: the K-th largest of the maxima of 64 or 128 groups of threads
  float bound;
  {
    const int groups = K <= 32 ? 64 : 128, share_of = kBmThreads / groups;
    float g = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    if (share_of == 4) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
    if (tid % share_of == 0) sm.group[tid / share_of] = g;
    __syncthreads();
    // the threads of a group compare its maximum with a share of the others each
    int above = 0, level = 0;
#pragma unroll 4
    for (int i = tid % share_of * 4; i < groups; i += 4 * share_of) {   // side by side: no bank twice
      const float4 o = *reinterpret_cast<const float4*>(&sm.group[i]);
      above += (o.x > g) + (o.y > g) + (o.z > g) + (o.w > g);
      level += (o.x >= g) + (o.y >= g) + (o.z >= g) + (o.w >= g);
    }
    above += __shfl_xor_sync(0xffffffffu, above, 1);
    level += __shfl_xor_sync(0xffffffffu, level, 1);
    if (share_of == 4) {
      above += __shfl_xor_sync(0xffffffffu, above, 2);
      level += __shfl_xor_sync(0xffffffffu, level, 2);
    }
    if (above < K && level >= K) sm.bound = g;           // one value, whoever writes it
    __syncthreads();
    bound = sm.bound;
  }
  // ---- the pieces that reach it, and their values
  if (top >= bound && top > -INFINITY)
#pragma unroll 4
    for (int p = 0; p * per < tiles; ++p) {
      const float m = sm.piece[p][tid];
      if (m >= bound && m > -INFINITY) {
        const int at = atomicAdd(&sm.pieces, 1);
        if (at < kBmList) sm.list[at] = p << 8 | tid;
      }
    }
  __syncthreads();
  const int pieces = sm.pieces;
  if (pieces <= kBmList) {
    const int each = per * kBmValues;
    for (int e = tid; e < pieces * each; e += kBmThreads) {
      const int k = e / each, i = e - k * each, u = i / L::kN;
      const int v = v0 + ((sm.list[k] >> 8) * per * kVecs + u) * kBmThreads + (sm.list[k] & 255);
      const int idx = v * L::kN + i % L::kN - skew;
      if (v >= v1 || idx < 0 || idx >= V) continue;
      const float z = plain(static_cast<float>(x[idx]));
      if (z >= bound && z > -INFINITY) {
        const int at = atomicAdd(&sm.count, 1);
        if (at < kBmCap) sm.key[at] = key_of(z, idx);
      }
    }
    __syncthreads();
  }
  if (pieces > kBmList || sm.count > kBmCap) {
    // equal values at the border, or the best ones close together: tile by tile, the threads
    // are the groups, and at most K threads hold keys above the bound of their best keys
    int kept = 0;                                        // keys of the tiles before
    __syncthreads();
    for (int t = 0; t < tiles; ++t) {
      load_tile(t);
      float val[kBmValues];
#pragma unroll
      for (int u = 0; u < kVecs; ++u) L::unpack(raw[u], val + u * L::kN);
      unsigned long long mine = 0;
#pragma unroll
      for (int i = 0; i < kBmValues; ++i) {
        val[i] = plain(val[i]);
        const unsigned long long k = val[i] > -INFINITY ? key_of(val[i], place(t, i)) : 0;
        mine = k > mine ? k : mine;
      }
      // K keys are kept: only better ones matter
      const unsigned long long floor_key = kept == K ? sm.key[K - 1] : 0;
      if (!__syncthreads_or(mine > floor_key)) continue;
      sm.gkey[tid] = mine;
      if (tid == 0) {
        sm.bound_key = 1;                                // fewer than K threads hold anything
        sm.count = kept;
      }
      __syncthreads();
      int above = 0;
#pragma unroll 8
      for (int i = 0; i < kBmThreads; ++i) above += sm.gkey[i] > mine;
      if (above == K - 1 && mine > 0) sm.bound_key = mine;
      __syncthreads();
      const unsigned long long bk = sm.bound_key > floor_key ? sm.bound_key : floor_key + 1;
#pragma unroll
      for (int i = 0; i < kBmValues; ++i) {
        const unsigned long long k = val[i] > -INFINITY ? key_of(val[i], place(t, i)) : 0;
        if (k >= bk) sm.key[atomicAdd(&sm.count, 1)] = k;
      }
      bm_rank(sm, K);
      kept = sm.count;
    }
  }
  bm_rank(sm, K);
  unsigned long long* out = keys + (static_cast<size_t>(row) * slices + blockIdx.x) * K;
  if (tid < K) out[tid] = tid < sm.count ? sm.key[tid] : 0;
  // ---- the slice's sum: references first, then the sums, the last of them in 64 bits
  float most = ref;
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
  sum = most > -INFINITY ? sum * bm_scale(ref - most) : 0.f;
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  if (lane == 0) {
    sm.ref[warp] = most;
    sm.sum[warp] = sum;
  }
  __syncthreads();
  if (tid == 0) {
    float r[kBmThreads / 32], v[kBmThreads / 32];
#pragma unroll
    for (int i = 0; i < kBmThreads / 32; ++i) {
      r[i] = sm.ref[i];
      v[i] = sm.sum[i];
      most = fmaxf(most, r[i]);
    }
    double total = 0.0;
    if (most > -INFINITY) {
#pragma unroll
      for (int i = 0; i < kBmThreads / 32; ++i) total += v[i] * bm_scale(r[i] - most);
    }
    stats[static_cast<size_t>(row) * slices + blockIdx.x] = {most, static_cast<float>(total)};
  }
}

// ---------------------------------------------------------------- merge

namespace {

constexpr int kBmGroups = 128;
constexpr int kBmPer = kBmMergeThreads / kBmGroups;
constexpr int kBmMine = kBmCandidates / kBmMergeThreads;            // candidates of a thread
constexpr int kBmSurvivors = kBmMaxK * kBmPer * kBmMine;            // at most after the first cut

// A candidate: score (ordered; 0: none) and what decides where scores are equal: the lower beam, then
// the larger logit, then the lower token.  Larger wins.  (Scores of a beam are ordered as its
// logits, by which its slices chose; rounded to 64 bits, near ones or those of a beam far below 0 are equal.)
struct Cand {
  unsigned long long s, tie;
};
__device__ __forceinline__ bool beats(const Cand& a, const Cand& b) {
  return a.s > b.s || (a.s == b.s && a.tie > b.tie);
}
__device__ __forceinline__ unsigned long long tie_of(int w, uint32_t logit, uint32_t token) {
  return static_cast<unsigned long long>(kBmMaxW - 1 - w) << 56 | static_cast<unsigned long long>(logit) << 24 |
         (0xFFFFFFu - token);                          // V <= 2^24
}

struct MergeSmem {
  union {
    Cand group[kBmGroups];
    unsigned long long group_s[kBmGroups];
  };
  double lse[kBmMaxW], score[kBmMaxW];
  int low[kBmMaxW];                    // nothing above -2^28: so many values, which count as -2^28
  int found[8][kBmMergeThreads / 32];  // among them: of a warp's pieces
  Cand bound;
  int count;
  unsigned long long left[2];          // scores of as many candidates as merge_room says, then their ties
};

// Candidates left after the first cut: K groups of kBmPer threads at most, each with its share of `total`
constexpr int merge_room(int total, int K) { return K * kBmPer * ((total + kBmMergeThreads - 1) / kBmMergeThreads); }

// ln(hi + lo) + n ln 2 (see BeamScan), hi >= 0 the larger part, to 5e-9: with hi = 2^e m, m from
// sqrt(1/2) to sqrt(2), and s = (m - 1) / (m + 1), ln m = 2 s + 2 s^3 / 3 + 2 s^5 / 5 + ...  s is kept as
// a sum of two fp32, so that only the last steps need 64 bits (a log in 64 bits takes 1.5 us here).
__device__ __forceinline__ double bm_log(float hi, float lo, float n) {
  int e = static_cast<int>(__float_as_uint(hi) >> 23) - 127;
  float m = __uint_as_float((__float_as_uint(hi) & 0x007FFFFFu) | 0x3F800000u);
  if (m > 1.41421354f) {
    m *= 0.5f;
    ++e;
  }
  lo *= __int_as_float((127 - e) << 23);                // e from -1 to 60 or so here
  const float f = m - 1.f, g = m + 1.f, g1 = (m - (g - 1.f)) + lo;   // f exact, m + 1 + lo = g + g1
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(g));
  const float s = f * r;
  const float s1 = (fmaf(-s, g, f) + lo - s * g1) * r;
  const float q = s * s;
  const float c = q * s * fmaf(q, fmaf(q, fmaf(q, fmaf(q, fmaf(q, 2.f / 13, 2.f / 11), 2.f / 9), 2.f / 7), 2.f / 5), 2.f / 3);
  return n * kBmRef + e * kBmLn2 + (static_cast<double>(2.f * s) + fmaf(2.f, s1, c));
}

// Bound that at least K candidates reach, from the best candidate of every thread.  At most
// the K best groups (of 4 threads) hold anything at or above it.
__device__ __forceinline__ void bm_bound(MergeSmem& sm, Cand top, int K) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int m = 1; m < kBmPer; m <<= 1) {
    const Cand o = {__shfl_xor_sync(0xffffffffu, top.s, m), __shfl_xor_sync(0xffffffffu, top.tie, m)};
    if (beats(o, top)) top = o;
  }
  if (tid % kBmPer == 0) sm.group[tid / kBmPer] = top;
  if (tid == 0) {
    sm.bound = {1, 0};                  // fewer than K groups hold anything
    sm.count = 0;
  }
  __syncthreads();
  int above = 0;
#pragma unroll 8
  for (int i = tid % kBmPer; i < kBmGroups; i += kBmPer)      // side by side: no bank twice
    above += beats(sm.group[i], top);
#pragma unroll
  for (int m = 1; m < kBmPer; m <<= 1) above += __shfl_xor_sync(0xffffffffu, above, m);
  if (above == K - 1 && top.s > 0 && tid % kBmPer == 0) sm.bound = top;
  __syncthreads();
}

// The same by scores alone: at least K candidates reach sm.bound.s, and with equal scores at the
// border any number.
__device__ __forceinline__ void bm_bound_score(MergeSmem& sm, unsigned long long top, int K) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int m = 1; m < kBmPer; m <<= 1) {
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, top, m);
    top = o > top ? o : top;
  }
  if (tid % kBmPer == 0) sm.group_s[tid / kBmPer] = top;
  if (tid == 0) sm.count = 0;
  __syncthreads();
  int above = 0, level = 0;
#pragma unroll 8
  for (int i = tid % kBmPer; i < kBmGroups; i += kBmPer) {
    above += sm.group_s[i] > top;
    level += sm.group_s[i] >= top;
  }
#pragma unroll
  for (int m = 1; m < kBmPer; m <<= 1) {
    above += __shfl_xor_sync(0xffffffffu, above, m);
    level += __shfl_xor_sync(0xffffffffu, level, m);
  }
  if (above < K && level >= K) sm.bound.s = top > 0 ? top : 1;   // one value, whoever writes it
  __syncthreads();
}

// Candidates of a beam that has nothing above -2^28 (rare): its values count alike, so that the
// K best are those at the lowest places, which the slices, who rank by size, need not have kept.
// `left` values are there; out: the beam's keys in place of its slices'.
template <typename T>
__device__ __forceinline__ void bm_lowest(MergeSmem& sm, const T* x, int V, int K, int left, unsigned long long* out,
                                       int room) {
  constexpr int kDeep = 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int want = left < K ? left : K;
  int have = 0;
  for (int v0 = 0; v0 < V && have < want; v0 += kDeep * kBmMergeThreads) {
    uint32_t there[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int v = v0 + u * kBmMergeThreads + tid;
      there[u] = v < V && static_cast<float>(x[v]) > -INFINITY;
    }
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      there[u] = __ballot_sync(0xffffffffu, there[u] != 0);
      if (lane == 0) sm.found[u][warp] = __popc(there[u]);
    }
    __syncthreads();
    for (int u = 0; u < kDeep && have < want; ++u) {
      int before = have;
      for (int w = 0; w < kBmMergeThreads / 32; ++w) {
        have += sm.found[u][w];
        before += w < warp ? sm.found[u][w] : 0;
      }
      before += __popc(there[u] & ((1u << lane) - 1u));
      if ((there[u] >> lane & 1) && before < want)
        out[before] = key_of(-kBmHuge, v0 + u * kBmMergeThreads + tid);
    }
    __syncthreads();                                   // read before the next pieces are counted
  }
  for (int i = want + tid; i < room; i += kBmMergeThreads) out[i] = 0;
}

}  // namespace

// grid (prompts)
__global__ void __launch_bounds__(kBmMergeThreads, 2) beam_merge_kernel(
    const BeamScan* __restrict__ stats, unsigned long long* keys, const void* __restrict__ logits, int dtype,
    long long ld, const float* scores, const uint8_t* __restrict__ finished, int W, int V, int K,
    int slices, int pad_token, float* scores_out, int32_t* __restrict__ parents,
    int32_t* __restrict__ tokens) {
  pdl_enter();
  extern __shared__ __align__(16) uint8_t smem_raw[];
  MergeSmem& sm = *reinterpret_cast<MergeSmem*>(smem_raw);
  const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // candidate i = (beam, slice, rank); the first key is asked for before it is needed
  const int per_row = slices * K, total = W * per_row;
  keys += static_cast<size_t>(n) * total;
  unsigned long long key0 = tid < total ? keys[tid] : 0;
  int any_low = 0;
  // ---- log-sum-exp of every beam, a warp each; NaN as score: the beam is dead
  for (int w = warp; w < W; w += kBmMergeThreads / 32) {
    const int row = n * W + w;
    const BeamScan* st = stats + static_cast<size_t>(row) * slices;
    const BeamScan mine = lane < slices ? st[lane] : BeamScan{-INFINITY, 0.f};
    const float s = scores[row];
    const bool live = s > -INFINITY;
    const bool ended = finished && finished[row];
    float ref = mine.ref, hi = 0.f, lo = 0.f;           // sum: hi + lo, times 2^ref
    auto join = [&](float x, float x1) {
      const float t = hi + x, d = t - hi;
      lo += x1 + ((hi - (t - d)) + (x - d));
      hi = t;
    };
    if (live && !ended) {
      for (int i = lane + 32; i < slices; i += 32) ref = fmaxf(ref, st[i].ref);
#pragma unroll
      for (int m = 16; m >= 1; m >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, m));
      if (ref > -INFINITY) {
        hi = mine.sum * bm_scale(mine.ref - ref);
        for (int i = lane + 32; i < slices; i += 32) join(st[i].sum * bm_scale(st[i].ref - ref), 0.f);
      }
#pragma unroll
      for (int m = 16; m >= 1; m >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, hi, m);
        join(x, __shfl_xor_sync(0xffffffffu, lo, m));
      }
    }
    if (lane == 0) {
      sm.score[w] = live ? static_cast<double>(s == 0.f ? 0.f : s) : -INFINITY;   // -0 is 0
      sm.lse[w] = ended || ref == -INFINITY ? 0.0 : bm_log(hi, lo, ref);   // no candidates: no matter
      sm.low[w] = 0;
      if (live && !ended && ref == kBmLow) {
        sm.lse[w] = bm_log(hi, lo, 0.f) - kBmHuge;
        sm.low[w] = static_cast<int>(hi + lo);             // at most 2^24: exact
        any_low = 1;
      }
    }
  }
  if (__syncthreads_or(any_low)) {
    for (int w = 0; w < W; ++w) {
      const int left = sm.low[w];
      if (left == 0) continue;
      const long long at = (static_cast<long long>(n) * W + w) * ld;
      if (dtype == MSA_F32)
        bm_lowest(sm, static_cast<const float*>(logits) + at, V, K, left, keys + w * per_row, per_row);
      else
        bm_lowest(sm, static_cast<const __nv_bfloat16*>(logits) + at, V, K, left, keys + w * per_row, per_row);
    }
    __syncthreads();
    if (tid < total) key0 = keys[tid];
  }
  auto score = [&](int i) -> unsigned long long {        // ordered; 0: none
    const int w = i / per_row, row = n * W + w;
    const double s = sm.score[w];
    if (!(s > -INFINITY)) return 0;
    if (finished && finished[row]) return i - w * per_row == 0 ? ordered(s) : 0;
    const unsigned long long key = i < kBmMergeThreads ? key0 : keys[i];
    if (key == 0) return 0;
    const float x = sm.low[w] ? -kBmHuge : unordered(static_cast<uint32_t>(key >> 32));
    return ordered(s + (static_cast<double>(x) - sm.lse[w]));
  };
  auto tie = [&](int i) -> unsigned long long {
    const int w = i / per_row;
    if (finished && finished[n * W + w]) return tie_of(w, 0u, pad_token);
    const unsigned long long key = i < kBmMergeThreads ? key0 : keys[i];
    return tie_of(w, static_cast<uint32_t>(key >> 32), 0xFFFFFFFFu - static_cast<uint32_t>(key));
  };
  const int room = merge_room(total, K);
  unsigned long long *left_s = sm.left, *left_tie = sm.left + room;
  auto keep = [&](int at, const Cand& c) {
    left_s[at] = c.s;
    left_tie[at] = c.tie;
  };
  const unsigned long long one = tid < total ? score(tid) : 0;
  {
    unsigned long long top = one;
    for (int i = tid + kBmMergeThreads; i < total; i += kBmMergeThreads) {
      const unsigned long long s = score(i);
      top = s > top ? s : top;
    }
    bm_bound_score(sm, top, K);
    const unsigned long long bound = sm.bound.s;
    if (top >= bound)
      for (int i = tid; i < total; i += kBmMergeThreads) {
        const unsigned long long s = i == tid ? one : score(i);
        if (s < bound) continue;
        const int at = atomicAdd(&sm.count, 1);
        if (at < room) keep(at, {s, tie(i)});
      }
  }
  __syncthreads();
  int left = sm.count;
  __syncthreads();
  if (left > room) {                                   // rare: equal scores at the border
    Cand top = {0, 0};
    for (int i = tid; i < total; i += kBmMergeThreads) {
      const Cand c = {score(i), tie(i)};
      if (beats(c, top)) top = c;
    }
    bm_bound(sm, top, K);
    const Cand bound = sm.bound;
    for (int i = tid; i < total; i += kBmMergeThreads) {
      const Cand c = {score(i), tie(i)};
      if (!beats(bound, c)) keep(atomicAdd(&sm.count, 1), c);
    }
    __syncthreads();
    left = sm.count;
    __syncthreads();
  }
  while (left > kBmMergeThreads) {                     // rare: the best ones lie in few threads
    Cand top = {0, 0};
    for (int i = tid; i < left; i += kBmMergeThreads) {
      const Cand c = {left_s[i], left_tie[i]};
      if (beats(c, top)) top = c;
    }
    bm_bound(sm, top, K);
    const Cand bound = sm.bound;
    for (int i0 = 0; i0 < left; i0 += kBmMergeThreads) {   // what is kept moves down, among what has been read
      const Cand c = i0 + tid < left ? Cand{left_s[i0 + tid], left_tie[i0 + tid]} : Cand{0, 0};
      __syncthreads();
      if (!beats(bound, c)) keep(atomicAdd(&sm.count, 1), c);
    }
    __syncthreads();
    left = sm.count;
    __syncthreads();                                   // read before the next round clears it
  }
  // ---- in order
  float* so = scores_out + static_cast<size_t>(n) * K;
  int32_t *po = parents + static_cast<size_t>(n) * K, *to = tokens + static_cast<size_t>(n) * K;
  if (tid < left) {
    const Cand mine = {left_s[tid], left_tie[tid]};
    int above = 0;
#pragma unroll 8
    for (int i = 0; i < left; ++i) above += left_s[i] > mine.s;
    if (above < K)                                     // few: equal scores
#pragma unroll 8
      for (int i = 0; i < left; ++i) above += left_s[i] == mine.s && left_tie[i] > mine.tie;
    if (above < K) {
      const unsigned long long u = mine.s >> 63 ? mine.s & ~(1ull << 63) : ~mine.s;
      so[above] = static_cast<float>(__longlong_as_double(static_cast<long long>(u)));
      po[above] = n * W + kBmMaxW - 1 - static_cast<int>(mine.tie >> 56);
      to[above] = static_cast<int>(0xFFFFFFu - static_cast<uint32_t>(mine.tie & 0xFFFFFFu));
    }
  }
  if (tid >= left && tid < K) {                        // fewer continuations than places
    so[tid] = -INFINITY;
    po[tid] = -1;
    to[tid] = -1;
  }
}

// ---------------------------------------------------------------- host

namespace {

struct BeamWorkspace {
  BeamScan* stats;
  unsigned long long* keys;
};

// Slices of a row: the number that makes the time least.  A thread spends about 7 instructions on
// a value and 700 on the CTA's start, bound and ranking; with c CTAs on an SM the pass over the
// values, which waits for memory, takes 0.3 c times as long and the rest 0.8 c (not less than once).  A slice
// costs the merge about as much as 4 values, and a candidate beyond one per thread half an
// instruction of each (its score in 64 bits).  Measured against counting rounds of 4 CTAs per SM alone, candidates
// for free, on the same logits again and again: 16 prompts x 4 x 50,000 10.5 us and 10.7, 19 x 5 x 50,001 10.9 and
// 11.9, 4 x 16 x 50,000 (K = 16) 13.3 and 17.2, 1 x 32 x 100,000 (K = 32) 28 and 57, 64 x 4 x 32,000 13.6 and 13.4.
// On several sets of logits in turn: 12.5 and 10.9, 12.7 and 12.5, 15.3 and 17.4, 30 and 57, 15.5 and 14.9.  No slice
// under 1024 values, and a prompt's candidates within what the merge takes.
int beam_slices(long long rows, int W, int V, int K) {
  const long long sms = device_sm_count();
  long long most = V / 1024;
  if (most > kBmCandidates / (W * K)) most = kBmCandidates / (W * K);
  if (most > 64 * sms / rows) most = 64 * sms / rows;        // more even nothing out
  long long best = 1, least = 0;
  for (long long s = 1; s <= most || s == 1; ++s) {
    const long long c = (rows * s + sms - 1) / sms, scan = c > 3 ? 3 * c : 10, rest = c > 1 ? 8 * c : 10;
    const long long tiles = (V + kBmTile * s - 1) / (kBmTile * s);
    const long long more = W * K * s - kBmMergeThreads;
    const long long time = (scan * tiles * kBmValues * 7 + rest * 700) / 10 + 26 * s + (more > 0 ? more / 2 : 0);
    if (s == 1 || time < least) {
      least = time;
      best = s;
    }
  }
  return static_cast<int>(best);
}

BeamWorkspace carve_beam_workspace(WsCursor& ws, long long rows, int slices, int K) {
  BeamWorkspace w;
  w.stats = ws.take<BeamScan>(static_cast<size_t>(rows) * slices);
  w.keys = ws.take<unsigned long long>(static_cast<size_t>(rows) * slices * K);
  return w;
}

size_t beam_bytes(long long rows, int slices, int K) {
  WsCursor ws(nullptr);
  carve_beam_workspace(ws, rows, slices, K);
  return ws.used + 256;
}

bool beam_sizes_ok(int N, int W, int V, int K) {
  return N >= 1 && W >= 1 && W <= kBmMaxW && V >= 1 && V <= (1 << 24) && K >= 1 && K <= kBmMaxK &&
         static_cast<long long>(K) <= static_cast<long long>(W) * V &&
         static_cast<long long>(N) * W <= 65535;
}

}  // namespace

}  // namespace msa

using namespace msa;

extern "C" {

size_t msa_beam_select_workspace_size(int N, int W, int V, int K) {
  if (!beam_sizes_ok(N, W, V, K)) return 0;
  const long long rows = static_cast<long long>(N) * W;
  return beam_bytes(rows, beam_slices(rows, W, V, K), K);
}

msa_status_t msa_beam_select(const void* logits, int dtype, int64_t row_stride, const float* scores,
                             const uint8_t* finished, int N, int W, int V, int K, int pad_token,
                             float* scores_out, int32_t* parents, int32_t* tokens,
                             void* workspace, size_t workspace_bytes, msa_stream_t stream) {
  const size_t size = dtype == MSA_F32 ? 4 : 2;
  if (dtype != MSA_F32 && dtype != MSA_BF16)
    return fail(MSA_ERR_INVALID_ARG, "dtype %d is neither MSA_F32 nor MSA_BF16", dtype);
  if (!logits || reinterpret_cast<uintptr_t>(logits) % size != 0)
    return fail(MSA_ERR_INVALID_ARG, "logits is null or not aligned to its type");
  MSA_REQUIRE_PTR(scores_out);
  MSA_REQUIRE_PTR(parents);
  MSA_REQUIRE_PTR(tokens);
  MSA_REQUIRE_PTR(workspace);
  if (!scores || reinterpret_cast<uintptr_t>(scores) % 4 != 0)
    return fail(MSA_ERR_INVALID_ARG, "scores is null or not 4-byte aligned");
  if (N < 1 || W < 1 || V < 1 || K < 1)
    return fail(MSA_ERR_INVALID_ARG, "N, W, V and K must be >= 1 (got %d, %d, %d, %d)", N, W, V, K);
  if (W > kBmMaxW || K > kBmMaxK || V > (1 << 24) || static_cast<long long>(N) * W > 65535)
    return fail(MSA_ERR_UNSUPPORTED,
                "at most %d beams, %d continuations, 2^24 tokens and 65535 rows (got %d, %d, %d, %lld)",
                kBmMaxW, kBmMaxK, W, K, V, static_cast<long long>(N) * W);
  if (static_cast<long long>(K) > static_cast<long long>(W) * V)
    return fail(MSA_ERR_INVALID_ARG, "K = %d of only %lld continuations", K, static_cast<long long>(W) * V);
  if (row_stride < V) return fail(MSA_ERR_INVALID_ARG, "row_stride is below V");
  if (pad_token < 0 || pad_token >= V)
    return fail(MSA_ERR_INVALID_ARG, "pad_token %d outside [0, %d)", pad_token, V);
  // a prompt's CTA writes its K places while others' scores and flags are still to be read; its own W scores
  // it has read before: in place where they are the same
  const struct {
    const void* at;
    const char* name;
  } out[3] = {{scores_out, "scores_out"}, {parents, "parents"}, {tokens, "tokens"}};
  const size_t places = 4ull * N * K, rows_in = static_cast<size_t>(N) * W;
  for (int i = 0; i < 3; ++i) {
    if (overlap(out[i].at, places, scores, 4 * rows_in) && !(i == 0 && scores_out == scores && K == W))
      return fail(MSA_ERR_INVALID_ARG, "%s overlaps scores (scores_out may be scores where K = W)", out[i].name);
    if (finished && overlap(out[i].at, places, finished, rows_in))
      return fail(MSA_ERR_INVALID_ARG, "%s overlaps finished", out[i].name);
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].at, places, out[j].at, places))
        return fail(MSA_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[j].name);
  }
  const long long rows = static_cast<long long>(N) * W;
  const int slices = beam_slices(rows, W, V, K);
  if (workspace_bytes < beam_bytes(rows, slices, K)) return fail(MSA_ERR_INVALID_ARG, "workspace too small");
  WsCursor ws(workspace);
  const BeamWorkspace w = carve_beam_workspace(ws, rows, slices, K);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope trace_("beam_scan_kernel", st);
    const dim3 grid(slices, static_cast<unsigned>(rows));
    if (dtype == MSA_F32)
      launch_pdl(beam_scan_kernel<float>, grid, kBmThreads, 0, st, static_cast<const float*>(logits),
                 row_stride, V, K, finished, w.stats, w.keys);
    else
      launch_pdl(beam_scan_kernel<__nv_bfloat16>, grid, kBmThreads, 0, st,
                 static_cast<const __nv_bfloat16*>(logits), row_stride, V, K, finished, w.stats, w.keys);
  }
  MSA_TRY(check_launch("beam_scan_kernel"));
  MSA_TRY(ensure_smem(beam_merge_kernel, sizeof(MergeSmem) + kBmSurvivors * sizeof(Cand), "beam_merge_kernel"));
  {
    TraceScope trace_("beam_merge_kernel", st);
    const size_t smem = sizeof(MergeSmem) + merge_room(W * slices * K, K) * sizeof(Cand);
    launch_pdl(beam_merge_kernel, static_cast<unsigned>(N), kBmMergeThreads, smem, st,
               w.stats, w.keys, logits, dtype, static_cast<long long>(row_stride), scores, finished, W, V, K, slices,
               pad_token, scores_out, parents, tokens);
  }
  return check_launch("beam_merge_kernel");
}

}  // extern "C"
