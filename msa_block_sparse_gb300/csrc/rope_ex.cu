// Prologue for any rotary layout: per-head Gemma RMSNorm (optional) and the
// rotation of the first R channels, in one pass, with its backward.
//   z = x rsqrt(mean(x^2) + eps) (1 + w)      (z = x without weights)
//   y = z with its pairs (a, b) turned: a' = gain (a cos - b sin),
//       b' = gain (b cos + a sin), angle = position * f_i;
//       pair i = channels (i, i + R/2) ("half") or (2i, 2i + 1) ("interleaved")
//   dz = the pairs of dy turned back (times gain), g = dz (1 + w), xh = x r:
//   dx = r (g - xh mean(g xh)),  dw = sum over tokens and heads of dz xh
// Bound by memory: 4 bytes per value forward, 6 backward (4 without weights).  Measured:
// 16,384 tokens x 64 heads x 128 (537 MB) forward 89 us, 6.0 TB/s; gradients of 16,384 x
// 12 x 256 (302 MB) 57 us, 5.3 TB/s; 32 tokens x 64 heads 2.8 us; the first without weights
// (64 channels rotated) 90 us forward and 92 us back.
//
// Work: the [T * H, D] rows are cut into runs of consecutive rows, one run per
// CTA (grid-stride in the backward).  A row belongs to D / 8 threads with 8
// channels each, chosen so that the two halves of every pair sit in one thread: two
// pieces of 4 channels R / 2 apart in the rotated part of the "half" layout, 8
// consecutive channels elsewhere.  The angles of the run's tokens are computed once per
// CTA into shared memory.
//
// Angles: the host turns each frequency into the 64-bit fixed-point fraction of
// a turn F_i = f_i / (2 pi) * 2^64, so position * F_i mod 2^64 is the angle in
// turns without a large fp32 argument (F_i has a double's 53 bits: positions below
// 2^31 keep their angle to 2^-24 of a turn).
#include <cmath>
#include "rope_ex.cuh"

namespace msa {

namespace {

constexpr int kRxThreads = 128;
constexpr int kRxMaxAngles = 2048;   // (token, pair) entries of a CTA's table: 16 KB
constexpr int kRxMaxH = 256;
struct RxArgs {
  const __nv_bfloat16* x;
  const __nv_bfloat16* dy;        // backward: upstream gradient
  __nv_bfloat16* y;               // forward: y, backward: dx
  const __nv_bfloat16* w;         // null: no norm
  const int32_t* positions;       // null: position within cu's sequence
  const int32_t* cu;
  float* dw_part;                 // backward: [gridDim.x, D]
  long long rows;                 // T * H
  int T, H, S, R, run;            // run: rows per CTA
  uint32_t inv;                   // ceil(2^20 / H): i / H == (i * inv) >> 20 for i < 4096
  uint32_t inv_half;              // ceil(2^20 / (R / 2)), for k < 2048
  float eps, gain;
};

// cos and sin (times gain) of the tokens t0 .. t0 + ntok - 1 of the run:
// table[tok * R + i] = cos, [tok * R + R / 2 + i] = sin of pair i.  live[tok]: the token
// is one of cu's sequences (or has a position given).  Every thread of the CTA takes
// part; both may be read after the next barrier.
__device__ __forceinline__ void rx_angles(const RxArgs& a, const RxTurns& turns, int t0, int ntok,
                                          unsigned long long* freq, int* pos, bool* live, float* table) {
  const int half = a.R >> 1;
  // frequencies by way of shared memory: lanes that index the parameters apart are
  // served one at a time
  for (int i = threadIdx.x; i < half; i += blockDim.x) freq[i] = turns.f[i];
  for (int tok = threadIdx.x; tok < ntok; tok += blockDim.x) {
    const int t = t0 + tok;
    if (a.positions) {
      pos[tok] = __ldg(a.positions + t);
      live[tok] = true;
    } else {
      int lo = 0, hi = a.S;                  // largest s with cu[s] <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu + mid) <= t) lo = mid; else hi = mid;
      }
      const int first = __ldg(a.cu + lo), end = __ldg(a.cu + lo + 1);
      pos[tok] = t - first;
      live[tok] = t >= first && t < end;
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < ntok * half; k += blockDim.x) {
    const int tok = static_cast<int>((static_cast<uint32_t>(k) * a.inv_half) >> 20);
    const int i = k - tok * half;
    const float2 cs = rx_cos_sin(pos[tok], freq[i]);
    table[tok * a.R + i] = cs.x * a.gain;
    table[tok * a.R + half + i] = cs.y * a.gain;
  }
}

// Sums of four values over the D / 8 lanes of a row, in every lane: two exchanges
// halve what a lane carries, so that the four cost 10 shuffles and not 20 (32 lanes).
template <int kLpr>
__device__ __forceinline__ void rx_sum4(float& a, float& b, float& c, float& d) {
  const int lane = threadIdx.x & 31;
  const bool hi = lane & (kLpr / 2), odd = lane & (kLpr / 4);
  float x = hi ? c : a, y = hi ? d : b;            // what this lane keeps
  x += __shfl_xor_sync(0xffffffffu, hi ? a : c, kLpr / 2);
  y += __shfl_xor_sync(0xffffffffu, hi ? b : d, kLpr / 2);
  float z = odd ? y : x;
  z += __shfl_xor_sync(0xffffffffu, odd ? x : y, kLpr / 4);
#pragma unroll
  for (int m = kLpr / 8; m >= 1; m >>= 1) z += __shfl_xor_sync(0xffffffffu, z, m);
  const int base = lane & ~(kLpr - 1);
  a = __shfl_sync(0xffffffffu, z, base);
  b = __shfl_sync(0xffffffffu, z, base + kLpr / 4);
  c = __shfl_sync(0xffffffffu, z, base + kLpr / 2);
  d = __shfl_sync(0xffffffffu, z, base + 3 * kLpr / 4);
}

}  // namespace

// Rows of a thread come one after another, kSlots apart; three rows' loads are in
// flight while a fourth is normed, turned and stored.  The coefficients (1 + w) cos
// and (1 + w) sin stay in registers while the token stays the same.  Arithmetic runs on
// packed pairs of fp32: the kernel would be bound by instruction issue otherwise
// (162 instructions per warp and row took 112 us for 16,384 tokens x 64 heads).
template <int D, bool kNorm, bool kHalf>
__global__ void __launch_bounds__(kRxThreads, 8) rope_ex_kernel(const RxArgs a, const RxTurns turns) {
  pdl_enter();
  constexpr int kLpr = D / 8, kSlots = kRxThreads / kLpr;
  __shared__ __align__(16) float table[2 * kRxMaxAngles];
  __shared__ int pos[kRxMaxAngles / 8];
  __shared__ bool live[kRxMaxAngles / 8];
  __shared__ unsigned long long freq[kRxMaxPairs];
  const long long r0 = static_cast<long long>(blockIdx.x) * a.run;
  const int n = static_cast<int>(a.rows - r0 < a.run ? a.rows - r0 : a.run);
  const int t0 = static_cast<int>(r0 / a.H);
  const int h0 = static_cast<int>(r0 - static_cast<long long>(t0) * a.H);
  const int ntok = (h0 + n + a.H - 1) / a.H;
  const int c = threadIdx.x & (kLpr - 1), slot = threadIdx.x / kLpr;
  const RxLane l = rx_lane<kHalf>(c, a.R);
  const __nv_bfloat16* xb = a.x + r0 * D;
  __nv_bfloat16* yb = a.y + r0 * D;
  constexpr int kDeep = 4;
  RxRow raw[kDeep];
  auto fetch = [&](int i, RxRow& r) {
    r.a = r.b = make_uint2(0u, 0u);
    if (i < n) r = rx_load<kHalf>(xb + static_cast<size_t>(i) * D, l);
  };
#pragma unroll
  for (int k = 0; k < kDeep - 1; ++k) fetch(k * kSlots + slot, raw[k]);
  float2 w1[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) w1[p] = make_float2(1.f, 1.f);
  if (kNorm) {
    float2 wv[4];
    RxRow wr;
    wr.a = *reinterpret_cast<const uint2*>(a.w + l.off0);
    wr.b = *reinterpret_cast<const uint2*>(a.w + l.off1);
    rx_unpack<kHalf>(wr, wv);
#pragma unroll
    for (int p = 0; p < 4; ++p) w1[p] = __fadd2_rn(wv[p], w1[p]);
  }
  rx_angles(a, turns, t0, ntok, freq, pos, live, table);
  __syncthreads();
  int have = -1;
  float2 cc[4], ss[4];
  // the loop bounds are uniform over the CTA: every lane reaches the shuffles
  for (int base = 0; base < n; base += kDeep * kSlots) {
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      if (base + k * kSlots >= n) break;
      const int i = base + k * kSlots + slot;
      fetch(i + (kDeep - 1) * kSlots, raw[(k + kDeep - 1) % kDeep]);
      float2 v[4];
      rx_unpack<kHalf>(raw[k], v);
      float2 rr = make_float2(1.f, 1.f);
      if (kNorm) {
        float2 q = __fmul2_rn(v[0], v[0]);
#pragma unroll
        for (int p = 1; p < 4; ++p) q = __ffma2_rn(v[p], v[p], q);
        float sum = q.x + q.y;
#pragma unroll
        for (int m = kLpr / 2; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        rr.x = rr.y = rsqrtf(sum * (1.f / D) + a.eps);
      }
      if (i >= n) continue;
      const int tok = static_cast<int>((static_cast<uint32_t>(h0 + i) * a.inv) >> 20);
      if (tok != have) {
        if (!live[tok]) continue;                  // the token in `have` is a live one
        have = tok;
        rx_coefficients(table + tok * a.R, a.R >> 1, l, w1, 1.f, cc, ss);
      }
      rx_turn(v, cc, ss, !kNorm || l.rot);
      if (kNorm) {
#pragma unroll
        for (int p = 0; p < 4; ++p) v[p] = __fmul2_rn(v[p], rr);
      }
      // without the norm, what is not rotated keeps its bits
      rx_store<kHalf>(yb + static_cast<size_t>(i) * D, l, kNorm || l.rot ? rx_pack<kHalf>(v) : raw[k]);
    }
  }
}

// Two rows of a thread at a time: their reductions share shuffles and their chains
// overlap.  Rows come through a ring of bulk copies per warp (a stage holds the
// warp's next 1 KB of dy and of x) that runs ahead across runs.  16,384 x 12 x 256, with
// the sum of dw behind it: 57.2 us (1, 3, 4 stages: 62.2, 58.0, 59.0; loads to registers a
// pair of rows ahead 59.5; 5 CTAs per SM 64.5).
constexpr int kRxStages = 2;

struct RxBwdSmem {
  alignas(128) uint8_t ring[kRxThreads / 32][kRxStages][2][1024];
  alignas(16) float table[2 * kRxMaxAngles];
  unsigned long long freq[kRxMaxPairs];
  uint64_t full[kRxThreads / 32][kRxStages];
  int pos[kRxMaxAngles / 8];
  bool live[kRxMaxAngles / 8];
};

template <int D, bool kNorm, bool kHalf>
__global__ void __launch_bounds__(kRxThreads, 4) rope_ex_bwd_kernel(const RxArgs a,
                                                                    const RxTurns turns,
                                                                    uint32_t* status) {
  pdl_enter();
  constexpr int kLpr = D / 8, kSlots = kRxThreads / kLpr;
  constexpr int kPass = 32 / kLpr;                 // rows of a warp side by side
  constexpr int kWarpRows = 2 * kPass, kCtaRows = 2 * kSlots;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  RxBwdSmem& sm = *reinterpret_cast<RxBwdSmem*>(smem_raw);
  float* table = sm.table;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = threadIdx.x & (kLpr - 1), slot = threadIdx.x / kLpr;
  const RxLane l = rx_lane<kHalf>(c, a.R);
  if (lane == 0) {
    for (int i = 0; i < kRxStages; ++i) mbar_init(&sm.full[warp][i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  const long long stride = static_cast<long long>(gridDim.x) * a.run;
  auto rows_of = [&](long long r0) {
    return static_cast<int>(a.rows - r0 < a.run ? a.rows - r0 : a.run);
  };
  // ---- loads: the warp's part of chunk after chunk, run after run
  long long load_r0 = static_cast<long long>(blockIdx.x) * a.run;
  int load_base = 0;
  uint32_t nload = 0, nuse = 0;
  bool dead = false;                               // a wait ran out
  auto load = [&]() {
    if (load_r0 >= a.rows) return;
    const int n = rows_of(load_r0);
    if (lane == 0) {
      const int st = nload % kRxStages, i = load_base + warp * kWarpRows;
      const int rows = n - i < kWarpRows ? n - i : kWarpRows;
      if (rows > 0) {
        const uint32_t bytes = rows * D * sizeof(__nv_bfloat16);
        const size_t at = static_cast<size_t>(load_r0 + i) * D;
        mbar_arrive_expect_tx(&sm.full[warp][st], kNorm ? 2 * bytes : bytes);
        bulk_load(sm.ring[warp][st][0], a.dy + at, bytes, &sm.full[warp][st]);
        if (kNorm) bulk_load(sm.ring[warp][st][1], a.x + at, bytes, &sm.full[warp][st]);
      } else {
        mbar_arrive(&sm.full[warp][st]);           // no rows of this chunk are the warp's
      }
    }
    ++nload;
    load_base += kCtaRows;
    if (load_base >= n) {
      load_base = 0;
      load_r0 += stride;
    }
  };
  for (int i = 0; i < kRxStages; ++i) load();
  float2 one[4], w1[4], aw[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    one[p] = make_float2(1.f, 1.f);
    aw[p] = make_float2(0.f, 0.f);
  }
  if (kNorm) {
    RxRow wr;
    wr.a = *reinterpret_cast<const uint2*>(a.w + l.off0);
    wr.b = *reinterpret_cast<const uint2*>(a.w + l.off1);
    rx_unpack<kHalf>(wr, w1);
#pragma unroll
    for (int p = 0; p < 4; ++p) w1[p] = __fadd2_rn(w1[p], one[p]);
  }
  for (long long r0 = static_cast<long long>(blockIdx.x) * a.run; r0 < a.rows; r0 += stride) {
    const int n = rows_of(r0);
    const int t0 = static_cast<int>(r0 / a.H);
    const int h0 = static_cast<int>(r0 - static_cast<long long>(t0) * a.H);
    const int ntok = (h0 + n + a.H - 1) / a.H;
    __nv_bfloat16* ob = a.y + r0 * D;
    __syncthreads();                              // the previous run's angles are consumed
    rx_angles(a, turns, t0, ntok, sm.freq, sm.pos, sm.live, table);
    __syncthreads();
    int have = -1;
    bool on = false;
    float2 cc[4], ss[4];
    for (int base = 0; base < n; base += kCtaRows) {   // uniform over the CTA
      const int st = nuse % kRxStages;
      if (!dead && !__all_sync(0xffffffffu, mbar_wait(&sm.full[warp][st], (nuse / kRxStages) & 1, status, 70))) {
        for (uint32_t k = nuse + 1; k < nload; ++k)    // wait (bounded) for what is on its way
          (void)mbar_wait(&sm.full[warp][k % kRxStages], (k / kRxStages) & 1, status, 71);
        dead = true;
      }
      if (dead) continue;
      ++nuse;
      // rows i and i + kPass; behind the run's end the ring holds old rows, which are
      // read but not used
      const int i = base + warp * kWarpRows + lane / kLpr;
      RxRow raw[2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int x = 0; x < (kNorm ? 2 : 1); ++x)
          raw[k][x] = rx_read<kHalf>(reinterpret_cast<const __nv_bfloat16*>(sm.ring[warp][st][x]) +
                                         (lane / kLpr + k * kPass) * D, l);
      __syncwarp();
      load();
      float2 dz[2][4], xv[2][4], g[2][4];
      float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
      bool put[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        rx_unpack<kHalf>(raw[k][0], dz[k]);
        const int ik = i + k * kPass < n ? i + k * kPass : n - 1;
        const int tok = static_cast<int>((static_cast<uint32_t>(h0 + ik) * a.inv) >> 20);
        if (tok != have) {
          have = tok;
          on = sm.live[tok];
          rx_coefficients(table + tok * a.R, a.R >> 1, l, one, -1.f, cc, ss);
        }
        put[k] = on && i + k * kPass < n;
        if (!kNorm || l.rot) {                     // a branch: selects took 59.0 us for 57.2
          rx_turn(dz[k], cc, ss, true);
        } else {
#pragma unroll
          for (int p = 0; p < 4; ++p) dz[k][p] = __fmul2_rn(dz[k][p], cc[p]);
        }
        if (kNorm) {
          rx_unpack<kHalf>(raw[k][1], xv[k]);
          float2 q = make_float2(0.f, 0.f), d = q;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            g[k][p] = __fmul2_rn(dz[k][p], w1[p]);
            q = __ffma2_rn(xv[k][p], xv[k][p], q);
            d = __ffma2_rn(g[k][p], xv[k][p], d);
          }
          sum[k][0] = q.x + q.y;
          sum[k][1] = d.x + d.y;
        }
      }
      if (kNorm) rx_sum4<kLpr>(sum[0][0], sum[0][1], sum[1][0], sum[1][1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (!put[k]) continue;
        if (kNorm) {
          // r = rsqrt(mean(x^2) + eps), dot = sum(g x):
          // dx = r g - x (r^3 dot / D), dw += dz x r
          const float r = rsqrtf(sum[k][0] * (1.f / D) + a.eps);
          const float k2 = -(r * r) * (r * (sum[k][1] * (1.f / D)));
          const float2 rr = make_float2(r, r), kk = make_float2(k2, k2);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            aw[p] = __ffma2_rn(__fmul2_rn(dz[k][p], rr), xv[k][p], aw[p]);
            dz[k][p] = __ffma2_rn(xv[k][p], kk, __fmul2_rn(g[k][p], rr));
          }
        }
        rx_store<kHalf>(ob + static_cast<size_t>(i + k * kPass) * D, l,
                        kNorm || l.rot ? rx_pack<kHalf>(dz[k]) : raw[k][0]);
      }
    }
  }
  if (kNorm) {
    // the CTA's row slots, added in slot order -> one partial row
    __syncthreads();
    float* red = table;                            // [kSlots][D]: 4 KB
    const float av[8] = {aw[0].x, aw[0].y, aw[1].x, aw[1].y, aw[2].x, aw[2].y, aw[3].x, aw[3].y};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // channel of the thread's e-th value (rx_unpack)
      const int ch = kHalf ? (e < 4 ? l.off0 + e : l.off1 + e - 4) : l.off0 + 2 * (e & 3) + (e >> 2);
      red[slot * D + ch] = av[e];
    }
    __syncthreads();
    for (int ch = threadIdx.x; ch < D; ch += kRxThreads) {
      float acc = 0.f;
      for (int sl = 0; sl < kSlots; ++sl) acc += red[sl * D + ch];
      a.dw_part[static_cast<size_t>(blockIdx.x) * D + ch] = acc;
    }
  }
}

// dw[ch] = the partial rows in a fixed order: thread (k, ch) adds rows k,
// k + 128, ... (all its loads in flight), then a pairwise tree over k.
constexpr int kRxSumCh = 8, kRxSumWays = 128;
constexpr int kRxBwdCtas = 608;                    // 4 per SM, all resident
constexpr int kRxSumRows = (kRxBwdCtas + kRxSumWays - 1) / kRxSumWays;
__global__ void __launch_bounds__(kRxSumCh * kRxSumWays)
    rope_ex_dw_kernel(const float* __restrict__ part, int nparts, int D, float* __restrict__ dw) {
  pdl_enter();
  __shared__ float red[kRxSumWays][kRxSumCh];
  const int cl = threadIdx.x % kRxSumCh, k = threadIdx.x / kRxSumCh;
  const int ch = blockIdx.x * kRxSumCh + cl;
  float v[kRxSumRows];
#pragma unroll
  for (int j = 0; j < kRxSumRows; ++j) {
    const int p = k + j * kRxSumWays;
    v[j] = p < nparts ? part[static_cast<size_t>(p) * D + ch] : 0.f;
  }
  float acc = 0.f;
#pragma unroll
  for (int j = 0; j < kRxSumRows; ++j) acc += v[j];
  red[k][cl] = acc;
  __syncthreads();
#pragma unroll
  for (int s = kRxSumWays / 2; s >= 1; s >>= 1) {
    if (k < s) red[k][cl] += red[k + s][cl];
    __syncthreads();
  }
  if (k == 0) dw[ch] = red[0][cl];
}

// ---------------------------------------------------------------- host

// Rows per run: about `target`, whole tokens where they fit (a token cut in two has
// its angles computed twice), fewer when the run's tokens would not fit the angle
// table.  A run of n rows touches at most (n + 2 H - 2) / H tokens.
static int rx_run(int H, int R, long long target) {
  const int cap_tok = kRxMaxAngles / (R / 2);            // >= 16
  const long long cap = static_cast<long long>(cap_tok - 1) * H;
  if (target > cap) target = cap;
  if (target > 512) target = 512;
  return static_cast<int>(target > H ? target / H * H : target);
}

constexpr int kRxRun = 128;         // backward
constexpr int kRxFwdRun = 64;       // forward, when there are rows enough

// Forward: 64 rows per CTA (128 cost small calls 1.4 us and gain nothing), fewer
// when that would leave SMs without a CTA, 16 at least.
static int rx_fwd_run(long long rows, int H, int R) {
  long long run = rows / (2 * device_sm_count());
  run = run < 16 ? 16 : (run > kRxFwdRun ? kRxFwdRun : run);
  return rx_run(H, R, run);
}

// Backward: the resident CTAs share the rows evenly, each in runs of at most 128
// rows or so.
static int rx_bwd_run(long long rows, int H, int R) {
  const long long share = (rows + kRxBwdCtas - 1) / kRxBwdCtas;
  const long long parts = (share + kRxRun - 1) / kRxRun;
  long long run = (share + parts - 1) / parts;
  if (run > H) run = (run + H - 1) / H * H;              // whole tokens, rounded up
  return rx_run(H, R, run);
}

static int rx_bwd_ctas(long long rows, int run) {
  const long long n = (rows + run - 1) / run;
  return static_cast<int>(n < kRxBwdCtas ? n : kRxBwdCtas);
}

size_t rope_ex_bwd_workspace_floats(int T, int H, int D) {
  (void)T;
  (void)H;
  return static_cast<size_t>(kRxBwdCtas) * D;
}

unsigned long long rope_turn(double freq) {
  const double turn = freq / 6.283185307179586476925286766559;
  const double frac = turn - std::floor(turn);
  return frac >= 1.0 ? 0 : static_cast<unsigned long long>(frac * 18446744073709551616.0);
}

RxTurns rx_turns(const msa_rope_t& rope) {
  RxTurns t;
  for (int i = 0; i < kRxMaxPairs; ++i)
    t.f[i] = i < rope.dim / 2 ? rope_turn(rope.freqs[i]) : 0;
  return t;
}

static RxArgs rx_args(const RopeExJob& j, const msa_rope_t& rope) {
  RxArgs a{};
  a.x = j.x;
  a.dy = j.dy;
  a.y = j.y;
  a.w = j.w;
  a.positions = j.positions;
  a.cu = j.cu;
  a.rows = static_cast<long long>(j.T) * j.H;
  a.T = j.T;
  a.H = j.H;
  a.S = j.S;
  a.R = rope.dim;
  a.inv = ((1u << 20) + j.H - 1) / j.H;
  a.inv_half = ((1u << 20) + rope.dim / 2 - 1) / (rope.dim / 2);
  a.eps = j.eps;
  a.gain = rope.gain;
  return a;
}

template <int D>
static msa_status_t rx_forward(const RopeExJob& j, const msa_rope_t& rope, cudaStream_t stream) {
  RxArgs a = rx_args(j, rope);
  a.run = rx_fwd_run(a.rows, j.H, rope.dim);
  const RxTurns turns = rx_turns(rope);
  const unsigned grid = static_cast<unsigned>((a.rows + a.run - 1) / a.run);
  TraceScope trace_("rope_ex_kernel", stream);
  const bool half = rope.layout == MSA_ROPE_HALF;
  launch_pdl(j.w ? (half ? rope_ex_kernel<D, true, true> : rope_ex_kernel<D, true, false>)
                 : (half ? rope_ex_kernel<D, false, true> : rope_ex_kernel<D, false, false>),
             grid, kRxThreads, 0, stream, a, turns);
  return check_launch("rope_ex_kernel");
}

template <int D>
static msa_status_t rx_backward(const RopeExJob& j, const msa_rope_t& rope, float* dw,
                                float* dw_part, cudaStream_t stream) {
  RxArgs a = rx_args(j, rope);
  a.run = rx_bwd_run(a.rows, j.H, rope.dim);
  a.dw_part = dw_part;
  const RxTurns turns = rx_turns(rope);
  const int ctas = rx_bwd_ctas(a.rows, a.run);
  uint32_t* sw = nullptr;
  MSA_TRY(status_word(&sw));
  {
    TraceScope trace_("rope_ex_bwd_kernel", stream);
    const bool half = rope.layout == MSA_ROPE_HALF;
    auto kernel = j.w ? (half ? rope_ex_bwd_kernel<D, true, true> : rope_ex_bwd_kernel<D, true, false>)
                      : (half ? rope_ex_bwd_kernel<D, false, true> : rope_ex_bwd_kernel<D, false, false>);
    MSA_TRY(ensure_smem(kernel, sizeof(RxBwdSmem), "rope_ex_bwd_kernel"));
    launch_pdl(kernel, ctas, kRxThreads, sizeof(RxBwdSmem), stream, a, turns, sw);
  }
  msa_status_t e = check_launch("rope_ex_bwd_kernel");
  if (e != MSA_OK || !j.w) return e;
  {
    TraceScope trace_("rope_ex_dw_kernel", stream);
    launch_pdl(rope_ex_dw_kernel, D / kRxSumCh, kRxSumCh * kRxSumWays, 0, stream, dw_part, ctas, D,
               dw);
  }
  return check_launch("rope_ex_dw_kernel");
}

msa_status_t launch_rope_ex(const RopeExJob& j, const msa_rope_t& rope, cudaStream_t stream) {
  if (j.D == 64) return rx_forward<64>(j, rope, stream);
  if (j.D == 128) return rx_forward<128>(j, rope, stream);
  return rx_forward<256>(j, rope, stream);
}

msa_status_t launch_rope_ex_bwd(const RopeExJob& j, const msa_rope_t& rope, float* dw,
                                float* dw_part, cudaStream_t stream) {
  if (j.D == 64) return rx_backward<64>(j, rope, dw, dw_part, stream);
  if (j.D == 128) return rx_backward<128>(j, rope, dw, dw_part, stream);
  return rx_backward<256>(j, rope, dw, dw_part, stream);
}

// ====================================================================== C ABI

msa_status_t check_rope_arg(const msa_rope_t* rope, int D) {
  if (!rope) return fail(MSA_ERR_INVALID_ARG, "rope is null");
  if (rope->dim < 16 || rope->dim % 16 != 0 || rope->dim > 2 * kRxMaxPairs)
    return fail(MSA_ERR_UNSUPPORTED, "rope dim %d is not a multiple of 16 in [16, %d]", rope->dim,
                2 * kRxMaxPairs);
  if (rope->dim > D)
    return fail(MSA_ERR_INVALID_ARG, "rope dim %d above the head dim %d", rope->dim, D);
  if (rope->layout != MSA_ROPE_HALF && rope->layout != MSA_ROPE_INTERLEAVED)
    return fail(MSA_ERR_INVALID_ARG, "rope layout %d unknown", rope->layout);
  if (!(rope->gain > 0.0f) || !std::isfinite(rope->gain))
    return fail(MSA_ERR_INVALID_ARG, "rope gain must be finite and > 0");
  for (int i = 0; i < rope->dim / 2; ++i)
    if (!std::isfinite(rope->freqs[i]))
      return fail(MSA_ERR_INVALID_ARG, "rope frequency %d is not finite", i);
  return MSA_OK;
}

static msa_status_t check_rope_ex(const void* x, const void* w, const int32_t* positions,
                                  const int32_t* cu, int S, int T, int H, int D, float eps,
                                  const msa_rope_t* rope) {
  (void)x;
  if (w && !aligned16(w)) return fail(MSA_ERR_INVALID_ARG, "w is not 16-byte aligned");
  if (T < 1 || H < 1) return fail(MSA_ERR_INVALID_ARG, "T and H must be >= 1 (got %d, %d)", T, H);
  if (H > kRxMaxH)
    return fail(MSA_ERR_UNSUPPORTED, "at most %d heads per tensor (got %d)", kRxMaxH, H);
  if (D != 64 && D != 128 && D != 256)
    return fail(MSA_ERR_UNSUPPORTED, "head dim must be 64, 128 or 256 (got %d)", D);
  if (positions) {
    if (!aligned16(positions)) return fail(MSA_ERR_INVALID_ARG, "positions is not 16-byte aligned");
  } else {
    if (!cu || !aligned16(cu))
      return fail(MSA_ERR_INVALID_ARG, "neither positions nor (16-byte aligned) cu_seqlens given");
    if (S < 1) return fail(MSA_ERR_INVALID_ARG, "S must be >= 1 (got %d)", S);
  }
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(MSA_ERR_INVALID_ARG, "eps must be >= 0");
  return check_rope_arg(rope, D);
}

}  // namespace msa

using namespace msa;

extern "C" {

msa_status_t msa_rope_init(msa_rope_t* rope, int dim, double base, int layout, int scaling,
                           double factor, double orig_len, double beta_fast, double beta_slow,
                           double gain) {
  if (!rope) return fail(MSA_ERR_INVALID_ARG, "rope is null");
  if (dim < 16 || dim % 16 != 0 || dim > 2 * kRxMaxPairs)
    return fail(MSA_ERR_UNSUPPORTED, "rope dim %d is not a multiple of 16 in [16, %d]", dim,
                2 * kRxMaxPairs);
  if (layout != MSA_ROPE_HALF && layout != MSA_ROPE_INTERLEAVED)
    return fail(MSA_ERR_INVALID_ARG, "rope layout %d unknown", layout);
  if (scaling < MSA_ROPE_PLAIN || scaling > MSA_ROPE_YARN)
    return fail(MSA_ERR_INVALID_ARG, "rope scaling %d unknown", scaling);
  if (!(base > 1.0) || !std::isfinite(base))
    return fail(MSA_ERR_INVALID_ARG, "rope base must be finite and > 1");
  if (scaling != MSA_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(MSA_ERR_INVALID_ARG, "rope factor must be finite and >= 1");
  if (scaling == MSA_ROPE_YARN) {
    if (!(orig_len >= 1.0) || !std::isfinite(orig_len))
      return fail(MSA_ERR_INVALID_ARG, "orig_len must be finite and >= 1");
    if (!(beta_fast > beta_slow) || !(beta_slow >= 0.0) || !std::isfinite(beta_fast))
      return fail(MSA_ERR_INVALID_ARG, "beta_fast > beta_slow >= 0 is needed");
  }
  if (!std::isfinite(gain) || gain < 0.0)
    return fail(MSA_ERR_INVALID_ARG, "gain must be finite and >= 0 (0: the scaling's own)");
  const double two_pi = 6.283185307179586476925286766559;
  const double b = scaling == MSA_ROPE_NTK
                       ? base * std::pow(factor, static_cast<double>(dim) / (dim - 2)) : base;
  if (!std::isfinite(b)) return fail(MSA_ERR_INVALID_ARG, "rope base overflows");
  rope->dim = dim;
  rope->layout = layout;
  rope->reserved = 0.0f;
  for (int i = 0; i < kRxMaxPairs; ++i) {
    rope->freqs[i] = 0.0;
    if (i >= dim / 2) continue;
    double f = std::pow(b, -2.0 * i / dim);
    if (scaling == MSA_ROPE_LINEAR) f /= factor;
    if (scaling == MSA_ROPE_YARN) {
      // pairs with more than beta_fast turns over the trained length keep their
      // angle, those below beta_slow are stretched, a linear ramp between
      double keep = (orig_len * f / two_pi - beta_slow) / (beta_fast - beta_slow);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      f = f / factor * (1.0 - keep) + f * keep;
    }
    rope->freqs[i] = f;
  }
  const double own = scaling == MSA_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  rope->gain = static_cast<float>(gain > 0.0 ? gain : own);
  return MSA_OK;
}

msa_status_t msa_qk_norm_rope_ex(const void* x, void* y, int T, int H, int D, const void* w,
                                 const int32_t* positions, const int32_t* cu_seqlens, int S,
                                 const msa_rope_t* rope, float eps, msa_stream_t stream) {
  MSA_REQUIRE_PTR(x);
  MSA_REQUIRE_PTR(y);
  MSA_TRY(check_rope_ex(x, w, positions, cu_seqlens, S, T, H, D, eps, rope));
  RopeExJob j{};
  j.x = static_cast<const __nv_bfloat16*>(x);
  j.y = static_cast<__nv_bfloat16*>(y);
  j.w = static_cast<const __nv_bfloat16*>(w);
  j.positions = positions;
  j.cu = cu_seqlens;
  j.T = T;
  j.H = H;
  j.D = D;
  j.S = S;
  j.eps = eps;
  return launch_rope_ex(j, *rope, static_cast<cudaStream_t>(stream));
}

size_t msa_qk_norm_rope_bwd_ex_workspace_size(int T, int H, int D) {
  if (T < 1 || H < 1 || D < 1) return 0;
  return rope_ex_bwd_workspace_floats(T, H, D) * sizeof(float);
}

msa_status_t msa_qk_norm_rope_bwd_ex(const void* x, const void* dy, void* dx, float* dw, int T,
                                     int H, int D, const void* w, const int32_t* positions,
                                     const int32_t* cu_seqlens, int S, const msa_rope_t* rope,
                                     float eps, void* workspace, size_t workspace_bytes,
                                     msa_stream_t stream) {
  MSA_REQUIRE_PTR(dy);
  MSA_REQUIRE_PTR(dx);
  if (w) {
    MSA_REQUIRE_PTR(x);
    MSA_REQUIRE_PTR(dw);
    MSA_REQUIRE_PTR(workspace);
  }
  MSA_TRY(check_rope_ex(x, w, positions, cu_seqlens, S, T, H, D, eps, rope));
  if (w && workspace_bytes < msa_qk_norm_rope_bwd_ex_workspace_size(T, H, D))
    return fail(MSA_ERR_INVALID_ARG, "workspace too small");
  RopeExJob j{};
  j.x = static_cast<const __nv_bfloat16*>(x);
  j.dy = static_cast<const __nv_bfloat16*>(dy);
  j.y = static_cast<__nv_bfloat16*>(dx);
  j.w = static_cast<const __nv_bfloat16*>(w);
  j.positions = positions;
  j.cu = cu_seqlens;
  j.T = T;
  j.H = H;
  j.D = D;
  j.S = S;
  j.eps = eps;
  return launch_rope_ex_bwd(j, *rope, dw, static_cast<float*>(workspace),
                            static_cast<cudaStream_t>(stream));
}

}  // extern "C"
