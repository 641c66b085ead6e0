// Decode step over the 4-bit paged cache: the rule of msa_decode_step (block
// scores by the largest index logit, own block + best 15 earlier ones, softmax
// attention over their keys) on values held as e2m1 codes with one e4m3 scale per
// 16 channels.  Two launches:
//
//   decode4_score_kernel   streams the index-key slabs (72 bytes per key, the bulk
//                          of the bytes) and writes one score per (sequence, head,
//                          block); not launched when no sequence can have more
//                          than 16 blocks
//   decode4_attend_kernel  one cluster per (sequence, KV head): its CTAs rank the
//                          scores, take the selected blocks in turn, attend to them
//                          and merge through distributed shared memory
//
// Both run on mma.sync m16n8k16 with fp16 operands: one query row (scores) or at
// most 16 (attention) is far below the tensor core's 128-row tiles.  Codes are exact
// in fp16, code * scale is too (6 significant bits, [2^-10, 2688]), and q's 8
// significant bits are, after a power of two per row brings its largest magnitude to
// [2^14, 2^15) (what falls below fp16's range then is < 2^-38 of that largest).
//
// Scores: a tile is 16 keys x 128 channels.  Thread (g, c) = (lane / 4, lane % 4)
// loads 16 bytes of key g and of key g + 8: the 32 channels 32c .. 32c + 31, scale
// blocks 2c and 2c + 1.  k-step t takes channels 32c + 4t .. + 3 of every thread, and
// the B operand has q of those channels in the column of their scale block, zeros
// elsewhere: the product's 8 columns are the 8 scale blocks' partial sums, so the
// scales are applied to fp32 sums, 2 per thread and key, and nothing is rounded
// before that.
#include <atomic>
#include <cmath>
#include "cache4.cuh"

namespace msa {

namespace {

constexpr double kLog2e = 1.4426950408889634;

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// Blocks of sequence b: 0 for padding (length 0) and for lengths out of range.
__device__ __forceinline__ int d4_len(int L, int max_pages, uint32_t* status) {
  if (L < 0 || L > max_pages * kBlock) {
    atomicOr(status, kStatusBounds);
    return 0;
  }
  return L;
}

// Exponent e such that 2^e times a row's largest magnitude (bf16 bits m) lies
// in [2^14, 2^15); bounded so that 2^e is a normal fp32
__device__ __forceinline__ int row_shift(uint32_t m) {
  const int e = 14 - (static_cast<int>(m >> 7) - 127);
  return e > 120 ? 120 : e;
}

__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// two packed bf16 times f (a power of two) as packed fp16
__device__ __forceinline__ uint32_t bf2_to_h2(uint32_t u, float f) {
  const float2 x = word_f2(u);
  return h2u(__floats2half2_rn(x.x * f, x.y * f));
}

// two e4m3 bytes of a 16-bit word as fp32
__device__ __forceinline__ float2 scales_f2(uint32_t two) {
  return __half22float2(__half2(
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3)));
}

}  // namespace

// ---------------------------------------------------------------- scores

constexpr int kScWarps = 9;
constexpr int kScThreads = 32 * kScWarps;
constexpr int kScStages = 2;
constexpr int kScUnroll = 8;    // tiles of 16 keys whose products overlap
constexpr int kScMaxB = 1024;   // rows whose unit counts are summed at a time

struct Score4Smem {
  alignas(128) uint8_t slab[kScWarps][kScStages][kSlab];
  uint64_t full[kScWarps][kScStages];
  int start[kScMaxB + 1];       // first unit of each row
  int bh[kScThreads];           // units of the pass: row * Hkv + head,
  int blk[kScThreads];          // block,
  int page[kScThreads];         // page (-1: none)
  int at[kScWarps][kScStages];  // unit of each buffer
  int warp_sums[kScWarps];
  int claim;                    // next unit of the pass
};
static_assert(sizeof(Score4Smem) <= 232448, "score shared memory above the 227 KB limit");

// Persistent CTAs, one per SM, each with an equal run of the units (row, head,
// block to score), counted from the lengths by every CTA for itself.  A CTA looks up
// 288 units at a time, one per thread; then its warps claim units and stream their
// slabs, each through its own two buffers with bulk copies.  Bound by memory: 64 rows of
// 8k - 32k tokens x 4 heads, 379 MB, 64 us, 5.9 TB/s.  166 KB in flight per SM: 12 warps
// (221 KB) took 67 us and left no room for a CTA of the attention to start beside them (the
// whole step 91.2 us, with 9 warps 88.1), 6 warps 76.  Loads straight to registers took 91 us,
// claims across SMs from a counter in global memory 69.
__global__ void __launch_bounds__(kScThreads, 1) decode4_score_kernel(
    const __nv_bfloat16* __restrict__ q_idx, const uint8_t* __restrict__ kidx,
    const int32_t* __restrict__ table, const int32_t* __restrict__ lens, int B, int Hkv,
    int num_pages, int max_pages, int n_init, float* __restrict__ scores, uint32_t* status) {
  // the wait has to stay ahead of the trigger, and no launch may come between this kernel and
  // decode4_attend_kernel, which reads q and the lengths before it waits for this one
  pdl_enter();
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Score4Smem& sm = *reinterpret_cast<Score4Smem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  if (lane == 0) {
    for (int i = 0; i < kScStages; ++i) mbar_init(&sm.full[warp][i], 1);
    fence_mbar_init();
  }
  uint32_t nload = 0, nuse = 0;                    // slabs asked for and used by this warp
  bool dead = false;                               // a wait ran out
  for (int b0 = 0; b0 < B; b0 += kScMaxB) {
    const int nb = min(kScMaxB, B - b0);
    // ---- start[i] = units of the rows before i; none where all blocks are kept
    __syncthreads();
    int total = 0;
    for (int i0 = 0; i0 < nb; i0 += kScThreads) {
      const int i = i0 + tid;
      int v = 0;
      if (i < nb) {
        const int own = (d4_len(lens[b0 + i], max_pages, status) + kBlock - 1) / kBlock - 1;
        v = own >= kTopK ? (own - n_init) * Hkv : 0;
      }
      int x = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      if (lane == 31) sm.warp_sums[warp] = x;
      __syncthreads();
      int before = total;
#pragma unroll
      for (int w = 0; w < kScWarps; ++w) {
        if (w < warp) before += sm.warp_sums[w];
        total += sm.warp_sums[w];
      }
      if (i < nb) sm.start[i] = before + x - v;
      __syncthreads();
    }
    if (tid == 0) sm.start[nb] = total;
    __syncthreads();
    const int u0 = static_cast<int>(static_cast<long long>(total) * blockIdx.x / gridDim.x);
    const int u1 = static_cast<int>(static_cast<long long>(total) * (blockIdx.x + 1) / gridDim.x);
    for (int base = u0; base < u1; base += kScThreads) {
      const int n = min(kScThreads, u1 - base);
      __syncthreads();                             // the previous pass is done
      if (tid < n) {
        const int u = base + tid;
        int lo = 0, hi = nb;                       // largest i with start[i] <= u
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (sm.start[mid] <= u) lo = mid; else hi = mid;
        }
        const int r = u - sm.start[lo];
        const int per = (sm.start[lo + 1] - sm.start[lo]) / Hkv;   // blocks of one head
        const int h = r / per, bh = (b0 + lo) * Hkv + h, blk = n_init + r - h * per;
        int pg = table[static_cast<size_t>(b0 + lo) * max_pages + blk];
        if (pg < 0 || pg >= num_pages) {
          atomicOr(status, kStatusBounds);
          scores[static_cast<size_t>(bh) * max_pages + blk] = -INFINITY;
          pg = -1;
        }
        sm.bh[tid] = bh;
        sm.blk[tid] = blk;
        sm.page[tid] = pg;
      }
      if (tid == 0) sm.claim = 0;
      __syncthreads();
      if (dead) continue;
      auto load = [&]() {                          // claim a unit and ask for its slab
        int i = n;
        if (lane == 0) {
          do {
            i = atomicAdd(&sm.claim, 1);
          } while (i < n && sm.page[i] < 0);
          if (i < n) {
            const int st = nload % kScStages;
            sm.at[warp][st] = i;
            mbar_arrive_expect_tx(&sm.full[warp][st], kSlab);
            bulk_load(sm.slab[warp][st],
                      kidx + (static_cast<size_t>(sm.page[i]) * Hkv + sm.bh[i] % Hkv) * kSlab, kSlab,
                      &sm.full[warp][st]);
          }
        }
        nload += __shfl_sync(0xffffffffu, i, 0) < n ? 1u : 0u;
      };
      int have_bh = -1;
      uint32_t bq[2][4][2];                        // B operand of the k-steps
      for (int i = 0; i < kScStages; ++i) load();
      while (nuse < nload) {
        const int st = nuse % kScStages;
        __syncwarp();                              // lane 0's entry of the unit
        // the row's q, while the slab is on its way
        const int unit = sm.at[warp][st], bh = sm.bh[unit];
        if (bh != have_bh) {
          have_bh = bh;
          // lane l looks at channels 4l .. 4l + 3 for the row's largest magnitude
          const __nv_bfloat16* qr = q_idx + static_cast<size_t>(bh) * kD;
          const uint2 mine = *reinterpret_cast<const uint2*>(qr + 4 * lane);
          uint32_t m = __vmaxu2(mine.x & 0x7FFF7FFFu, mine.y & 0x7FFF7FFFu);
          m = max(m & 0xFFFFu, m >> 16);
          m = __reduce_max_sync(0xffffffffu, m);
          const float f = exp2i(row_shift(m));
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint2 w = *reinterpret_cast<const uint2*>(qr + 32 * c + 16 * hf + 4 * t);
              const bool col = g == 2 * c + hf;    // this thread's column is the block's
              bq[hf][t][0] = col ? bf2_to_h2(w.x, f) : 0u;
              bq[hf][t][1] = col ? bf2_to_h2(w.y, f) : 0u;
            }
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.full[warp][st], (nuse / kScStages) & 1, status, 81))) {
          for (++nuse; nuse < nload; ++nuse)       // wait (bounded) for what is on its way
            (void)mbar_wait(&sm.full[warp][nuse % kScStages], (nuse / kScStages) & 1, status, 82);
          dead = true;
          break;
        }
        ++nuse;
        const uint8_t* slab = sm.slab[warp][st];
        float best = -INFINITY;
#pragma unroll kScUnroll
        for (int r0 = 0; r0 < kBlock; r0 += 16) {
          const uint4 ka = *(reinterpret_cast<const uint4*>(slab + slab_code(r0 + g)) + c);
          const uint4 kb = *(reinterpret_cast<const uint4*>(slab + slab_code(r0 + g + 8)) + c);
          const uint32_t sa = *(reinterpret_cast<const uint16_t*>(slab + slab_scale(r0 + g)) + c);
          const uint32_t sb = *(reinterpret_cast<const uint16_t*>(slab + slab_scale(r0 + g + 8)) + c);
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {            // 8 channels: two k-steps
            __half2 ha[4], hb[4];
            codes_half2(wa[w], ha);
            codes_half2(wb[w], hb);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int t = (2 * w + k) & 3, hf = w >> 1;
              mma_f16_16816(acc, h2u(ha[2 * k]), h2u(hb[2 * k]), h2u(ha[2 * k + 1]),
                            h2u(hb[2 * k + 1]), bq[hf][t][0], bq[hf][t][1]);
            }
          }
          const float2 fa = scales_f2(sa), fb = scales_f2(sb);
          float za = fmaf(acc[0], fa.x, acc[1] * fa.y), zb = fmaf(acc[2], fb.x, acc[3] * fb.y);
          za += __shfl_xor_sync(0xffffffffu, za, 1);
          zb += __shfl_xor_sync(0xffffffffu, zb, 1);
          za += __shfl_xor_sync(0xffffffffu, za, 2);
          zb += __shfl_xor_sync(0xffffffffu, zb, 2);
          best = fmaxf(best, fmaxf(za, zb));
        }
        const int blk = sm.blk[unit];
        __syncwarp();                              // every lane has read the buffer
        load();
#pragma unroll
        for (int m = 4; m <= 16; m <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, m));
        if (lane == 0) scores[static_cast<size_t>(bh) * max_pages + blk] = best;
      }
    }
  }
}

// ---------------------------------------------------------------- attention

constexpr int kAtWarps = 4;
constexpr int kAtThreads = 32 * kAtWarps;
constexpr int kKeysPerWarp = kBlock / kAtWarps;
constexpr int kAtPer = kMaxSeqlen / kBlock / kAtThreads;   // scores per thread
constexpr int kMaxDevices = 64;
constexpr float kAtRescale = 8.0f;  // log2 of the largest weight before a rescale (fp16: below 2^16)

// A warp's 32 keys of a block, as they lie in the slabs
struct Attend4Keys {
  alignas(16) uint8_t k[kKeysPerWarp * kCodeBytes];
  alignas(16) uint8_t ks[kKeysPerWarp * kScaleBytes];
  alignas(16) uint8_t v[kKeysPerWarp * kCodeBytes];
  alignas(16) uint8_t vs[kKeysPerWarp * kScaleBytes];
};

// kWhole: the CTA's slabs all at once, asked for by warp 0 as soon as it knows the
// blocks; two (4 blocks) or three CTAs fit an SM.  Otherwise each warp streams its keys
// through two buffers of its own; four CTAs fit.
template <int NS, bool kWhole_>
struct Attend4Smem {
  static constexpr int kBlocks = kTopK / NS;       // blocks per CTA
  static constexpr bool kWhole = kWhole_;
  static constexpr int kStages = 2;
  union {
    struct {
      alignas(16) uint8_t k[kWhole ? kBlocks : 1][kSlab];
      alignas(16) uint8_t v[kWhole ? kBlocks : 1][kSlab];
    } whole;
    Attend4Keys s[kWhole ? 1 : kAtWarps][kStages];
    alignas(16) float o[kAtWarps][16][kD];         // per warp, once the keys are used
  };
  // sums (and maximum, weight) of this CTA's rows of the result, by sender: stored here
  // by the cluster's CTAs, which may be ahead of this one
  alignas(16) float part[NS][16 / NS][kD];
  alignas(16) float part_ml[NS][16 / NS][2];
  unsigned long long cand[4 * (kTopK - 1) * kAtPer];   // selection: keys left to be ranked
  alignas(16) uint4 qa[8][32];                     // A operand of the 8 k-steps, per lane
  float ml[kAtWarps][16][2];
  unsigned long long gmax[32];                     // selection: best key of each group of threads
  int list[kTopK];                                 // selected blocks, -1 behind
  int page[kBlocks];
  int ncand;
  uint64_t full[kAtWarps][kStages];                // whole slabs: the first kBlocks of them
  uint64_t joined;                                 // part, part_ml are complete
};

// Float4 `chunk` (channel / 4) of row r in a [16][128] array of sums: permuted so
// that the accumulator fragments' stores and the rows' loads meet no bank twice.
__device__ __forceinline__ int o_at(int r, int chunk) {
  return r * kD + 4 * (chunk ^ (chunk >> 3) ^ ((r & 1) << 2));
}

// Orders (score, block): a higher score first, then the lower block; 0 = none.
__device__ __forceinline__ unsigned long long rank_key(float score, int block) {
  const uint32_t u = __float_as_uint(score + 0.f);         // -0 equals 0
  const uint32_t k = u & 0x80000000u ? ~u : u | 0x80000000u;
  return static_cast<unsigned long long>(k) << 32 | static_cast<uint32_t>(0x7FFFFFFF - block);
}

__device__ __forceinline__ uint32_t cluster_map(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// Stores into a CTA of the cluster; `bar`, in the same CTA, counts the bytes.
__device__ __forceinline__ void st_async4(uint32_t a, const float4& v, uint32_t bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a),
      "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void st_async2(uint32_t a, float x, float y, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(a),
               "f"(x), "f"(y), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void cluster_arrive() {  // publishes barriers (after fence_mbar_init), no data
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// grid (NS, B * Hkv) in clusters of NS CTAs; CTA `split` attends to the selected
// blocks split, split + NS, ...  Each warp takes 32 keys of every block.  Bound by
// instruction issue and latency: 256 rows, 75 MB, 33 us with cold caches and 25 us
// behind the scores, 2.0 instructions per cycle and SM (a fifth of the time is the
// selection, a tenth the joining of the sums); 4 rows 3.8 us.  Slabs shared by the CTA's
// warps instead of a stream for each (8 times fewer copies) took 1.5 us more.
//
// The CTAs' sums are joined by asynchronous stores into the CTA that finishes a row,
// counted by its barrier; two cluster barriers around loads from the others took 1.2 us
// more (4 rows: 5.0 us), since their release waits for all earlier stores.
//
// Lengths, q and everything else but the scores were complete before the scores' kernel
// passed its own wait, so they are read while that kernel's last CTAs run.
//
// S = Q K^T: rows are heads; n-tile column g is key (g >> 1) + 4 (g & 1) of 8, so
// that the accumulator's column pair (2c, 2c + 1) is keys (c, c + 4), which is how
// the rows of V are then read (rows c, c + 4, c + 8, c + 12 of 16: both halves of
// the shared-memory banks).  Channels of a k-step as in the score kernel.
// O = P V: thread (g, c) reads 8 bytes of codes = scale block g of a key, column
// g of n-tile i is channel 16 g + i.  Keys behind the sequence's end have P = 0 and
// scale 0, whatever their slots hold.
template <int NS, bool kWhole>
__global__ void __launch_bounds__(kAtThreads, kWhole ? 3 : 4) decode4_attend_kernel(
    const __nv_bfloat16* __restrict__ q, const uint8_t* __restrict__ kc,
    const uint8_t* __restrict__ vc, const int32_t* __restrict__ table,
    const int32_t* __restrict__ lens, const float* __restrict__ scores, int G, int Hkv,
    int num_pages, int max_pages, int n_init, float sl2, int sl2_exp, float v_gain,
    __nv_bfloat16* __restrict__ o, int32_t* __restrict__ sel_out, uint32_t* status) {
  if (max_pages <= kTopK) pdl_wait();              // no scores' kernel stands in between
  extern __shared__ __align__(128) uint8_t smem_raw[];
  using Smem = Attend4Smem<NS, kWhole>;
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  constexpr int kBlocks = Smem::kBlocks, kRows = 16 / NS;
  const int split = blockIdx.x, bh = blockIdx.y, b = bh / Hkv, h = bh % Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  // ---- everything that depends on no other load is asked for at once
  const int my_rows = max(0, min(G - split * kRows, kRows));   // of the result, to finish here
  const int len = lens[b];
  // q as the A operand of the 8 k-steps: rows g and g + 8 in fp16, each with a power
  // of two; thread c of a row has channels 32 c .. 32 c + 31.  Each warp makes and
  // stores two k-steps.  f0, f1: factor of the rows' sums, scale * k_gain * log2(e) over
  // that power (sl2 in [1, 2] times 2^sl2_exp).  It is kept in [2^-126, 2^91]: the sums lie
  // below 2^34 and are multiples of 2^-34, so that 2^-126 makes all of them 0 for the
  // softmax, 2^91 tells any two of them apart and no product overflows.  With 0 a masked
  // key's -inf would become a NaN.
  float f0, f1;
  {
    uint4 a0, a1;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = g + 8 * half;
      uint4 x[4];
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < G)
          x[i] = *(reinterpret_cast<const uint4*>(
                       q + (static_cast<size_t>(b) * G * Hkv + static_cast<size_t>(h) * G + r) * kD +
                       32 * c) + i);
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu),
                                 __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu)));
      }
      m = max(m & 0xFFFFu, m >> 16);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = row_shift(m);
      const float f = exp2i(e);
      (half ? f1 : f0) = sl2 * exp2i(max(-126, min(90, sl2_exp - e)));
      const uint4 mine = warp == 0 ? x[0] : (warp == 1 ? x[1] : (warp == 2 ? x[2] : x[3]));
      (half ? a0.y : a0.x) = bf2_to_h2(mine.x, f);
      (half ? a0.w : a0.z) = bf2_to_h2(mine.y, f);
      (half ? a1.y : a1.x) = bf2_to_h2(mine.z, f);
      (half ? a1.w : a1.z) = bf2_to_h2(mine.w, f);
    }
    sm.qa[2 * warp][lane] = a0;
    sm.qa[2 * warp + 1][lane] = a1;
  }
  if (max_pages > kTopK) pdl_wait();
  pdl_launch();
  const float* sc = scores + static_cast<size_t>(bh) * max_pages;
  float score[kAtPer];                             // blocks tid + 128 r (behind the own block: anything)
  if (max_pages > kTopK) {
#pragma unroll
    for (int r = 0; r < kAtPer; ++r) {
      const int i = kAtThreads * r + tid;
      score[r] = i < max_pages ? __ldcg(sc + i) : 0.f;   // not to be moved before the wait
    }
  }
  const int L = d4_len(len, max_pages, status);
  const int nblk = (L + kBlock - 1) / kBlock;
  const int own = nblk - 1;
  // by the lanes of warp 0 that use them before the next barrier of the CTA
  if (tid < kAtWarps * Smem::kStages) {
    mbar_init(&sm.full[0][0] + tid, 1);
    if (tid == 0) mbar_init(&sm.joined, 1);
    fence_mbar_init();
    if (tid == 0 && my_rows > 0)
      mbar_arrive_expect_tx(&sm.joined, NS * my_rows * (kD + 2) * sizeof(float));
  }
  __syncwarp();                                    // the barrier wants whole warps
  cluster_arrive();
  if (tid == 0) sm.ncand = 0;
  if (own >= kTopK) {
    // ---- the 15 best earlier blocks.  The threads form 32 groups of 4; the 15th of
    // the groups' best keys bounds the 15th best key from below, so that few keys
    // (about 20; at most 15 groups' keys) are left to be ranked among each other.
    unsigned long long key[kAtPer], top = 0ull;
#pragma unroll
    for (int r = 0; r < kAtPer; ++r) {
      const int i = kAtThreads * r + tid;
      key[r] = 0ull;
      if (i < own)
        key[r] = i < n_init ? (0xFFFFFFFFull << 32 | static_cast<uint32_t>(0x7FFFFFFF - i))
                            : rank_key(score[r], i);
      top = key[r] > top ? key[r] : top;
    }
#pragma unroll
    for (int m = 8; m <= 16; m <<= 1) {            // lanes l, l + 8, l + 16, l + 24
      const unsigned long long x = __shfl_xor_sync(0xffffffffu, top, m);
      top = x > top ? x : top;
    }
    if (lane < 8) sm.gmax[8 * warp + lane] = top;
    __syncthreads();
    const unsigned long long mine = sm.gmax[lane];
    int before = 0;
#pragma unroll 8
    for (int j = 0; j < 32; ++j) before += sm.gmax[j] > mine ? 1 : 0;
    // fewer than 15 groups with keys: every key is a candidate
    const uint32_t at15 = __ballot_sync(0xffffffffu, mine != 0ull && before == kTopK - 2);
    const unsigned long long bar =
        at15 ? __shfl_sync(0xffffffffu, mine, __ffs(at15) - 1) : 1ull;
    int cnt = 0, at[kAtPer];                       // places among the warp's candidates
#pragma unroll
    for (int r = 0; r < kAtPer; ++r) {
      const uint32_t in = __ballot_sync(0xffffffffu, key[r] >= bar);
      at[r] = cnt + __popc(in & ((1u << lane) - 1u));
      cnt += __popc(in);
    }
    int from = 0;
    if (lane == 0 && cnt > 0) from = atomicAdd(&sm.ncand, cnt);
    from = __shfl_sync(0xffffffffu, from, 0);
#pragma unroll
    for (int r = 0; r < kAtPer; ++r)
      if (key[r] >= bar) sm.cand[from + at[r]] = key[r];
    __syncthreads();
    if (warp == 0) {
      const int nc = sm.ncand;
      for (int t = lane; t < nc; t += 32) {
        const unsigned long long me = sm.cand[t];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < nc; ++j) rank += sm.cand[j] > me ? 1 : 0;
        if (rank < kTopK - 1) sm.list[rank] = 0x7FFFFFFF - static_cast<int>(static_cast<uint32_t>(me));
      }
      if (lane == 31) sm.list[kTopK - 1] = own;
    }
  } else if (tid < kTopK) {
    sm.list[tid] = tid < nblk ? tid : -1;          // every block
  }
  __syncwarp();
  // ---- warp 0: this CTA's blocks
  if (warp == 0) {
    if (lane < kBlocks) {
      const int blk = sm.list[split + NS * lane];
      int pg = -1;
      if (blk >= 0) {
        pg = table[static_cast<size_t>(b) * max_pages + blk];
        if (pg < 0 || pg >= num_pages) {
          atomicOr(status, kStatusBounds);
          pg = -1;
        }
      }
      sm.page[lane] = pg;
      if (kWhole && pg >= 0) {
        const size_t off = (static_cast<size_t>(pg) * Hkv + h) * kSlab;
        mbar_arrive_expect_tx(&sm.full[0][0] + lane, 2 * kSlab);
        bulk_load(sm.whole.k[lane], kc + off, kSlab, &sm.full[0][0] + lane);
        bulk_load(sm.whole.v[lane], vc + off, kSlab, &sm.full[0][0] + lane);
      }
    }
    if (split == 0 && lane < kTopK && sel_out) {   // ascending, -1 last
      const uint32_t me = static_cast<uint32_t>(sm.list[lane]);
      int at = 0;
#pragma unroll
      for (int j = 0; j < kTopK; ++j) {
        const uint32_t x = static_cast<uint32_t>(sm.list[j]);
        at += x < me || (x == me && j < lane) ? 1 : 0;
      }
      sel_out[static_cast<size_t>(bh) * kTopK + at] = static_cast<int>(me);
    }
  }
  __syncthreads();                                 // blocks, pages and q are known to every warp
  // ---- each warp takes its 32 keys of the CTA's blocks
  const int kw = kKeysPerWarp * warp;              // this warp's first key
  int my_page = -1, my_keys = 0;                   // lane i: block i's page and its valid keys of mine
  if (lane < kBlocks) {
    my_page = sm.page[lane];
    const int n = (sm.list[split + NS * lane] == own ? L - own * kBlock : kBlock) - kw;
    my_keys = my_page < 0 ? 0 : max(0, min(n, kKeysPerWarp));
  }
  uint32_t todo = __ballot_sync(0xffffffffu, my_keys > 0), ask = todo;
  const size_t head = static_cast<size_t>(h) * kSlab, row = static_cast<size_t>(Hkv) * kSlab;
  uint32_t nload = 0, nuse = 0;
  bool dead = false;                               // a wait ran out
  auto load = [&]() {                              // the next block's keys, K and V
    if (kWhole || ask == 0u) return;
    const int pg = __shfl_sync(0xffffffffu, my_page, __ffs(ask) - 1);
    if (lane == 0) {
      const int st = nload % Smem::kStages;
      Attend4Keys& d = sm.s[warp][st];
      const size_t off = pg * row + head;
      mbar_arrive_expect_tx(&sm.full[warp][st], sizeof(Attend4Keys));
      bulk_load(d.k, kc + off + slab_code(kw), sizeof(d.k), &sm.full[warp][st]);
      bulk_load(d.ks, kc + off + slab_scale(kw), sizeof(d.ks), &sm.full[warp][st]);
      bulk_load(d.v, vc + off + slab_code(kw), sizeof(d.v), &sm.full[warp][st]);
      bulk_load(d.vs, vc + off + slab_scale(kw), sizeof(d.vs), &sm.full[warp][st]);
    }
    ++nload;
    ask &= ask - 1u;
  };
  for (int i = 0; i < Smem::kStages; ++i) load();
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  float acc[16][4];
#pragma unroll
  for (int nt = 0; nt < 16; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;

#pragma unroll 1
  for (; todo; todo &= todo - 1u) {                // uniform over the warp
    const int i = __ffs(todo) - 1;
    const int nvalid = __shfl_sync(0xffffffffu, my_keys, i);
    const int st = nuse % Smem::kStages;
    uint64_t* full = kWhole ? &sm.full[0][0] + i : &sm.full[warp][st];
    if (!__all_sync(0xffffffffu, mbar_wait(full, kWhole ? 0 : (nuse / Smem::kStages) & 1, status, 80))) {
      dead = true;
      break;
    }
    ++nuse;
    const uint8_t *dk, *dks, *dv, *dvs;            // this warp's keys
    if (kWhole) {
      dk = sm.whole.k[i] + slab_code(kw);
      dks = sm.whole.k[i] + slab_scale(kw);
      dv = sm.whole.v[i] + slab_code(kw);
      dvs = sm.whole.v[i] + slab_scale(kw);
    } else {
      const Attend4Keys& d = sm.s[warp][st];
      dk = d.k;
      dks = d.ks;
      dv = d.v;
      dvs = d.vs;
    }
    // ---- S: four n-tiles side by side, so that four chains of products overlap
    float s[4][4];
    uint4 w4[4];
    __half2 ksc[4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const int key = 8 * nt + (g >> 1) + 4 * (g & 1);
      w4[nt] = *(reinterpret_cast<const uint4*>(dk + kCodeBytes * key) + c);
      const uint32_t two = *(reinterpret_cast<const uint16_t*>(dks + kScaleBytes * key) + c);
      ksc[nt] = __half2(
          __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3));
      s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {                  // 8 channels: two k-steps
      const uint4 qa[2] = {sm.qa[2 * j][lane], sm.qa[2 * j + 1][lane]};
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const uint32_t w = j == 0 ? w4[nt].x : (j == 1 ? w4[nt].y : (j == 2 ? w4[nt].z : w4[nt].w));
        __half2 hh[4];
        codes_half2(w, hh);
        const __half2 s2 = j < 2 ? __low2half2(ksc[nt]) : __high2half2(ksc[nt]);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          mma_f16_16816(s[nt], qa[k].x, qa[k].y, qa[k].z, qa[k].w,
                        h2u(__hmul2(hh[2 * k], s2)), h2u(__hmul2(hh[2 * k + 1], s2)));
      }
    }
    // ---- mask and running softmax of this warp's keys
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      if (nvalid < kKeysPerWarp) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool ok = 8 * nt + c + 4 * e < nvalid;
          s[nt][e] = ok ? s[nt][e] : -INFINITY;
          s[nt][2 + e] = ok ? s[nt][2 + e] : -INFINITY;
        }
      }
      mx0 = fmaxf(mx0, fmaxf(s[nt][0], s[nt][1]));
      mx1 = fmaxf(mx1, fmaxf(s[nt][2], s[nt][3]));
    }
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, m));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, m));
    }
    // the maximum moves only when it grows by more than 2^8: weights stay below
    // 2^8, which fp16 holds as well as those below 1
    const bool up0 = (mx0 - m0) * f0 > kAtRescale || m0 == -INFINITY;
    const bool up1 = (mx1 - m1) * f1 > kAtRescale || m1 == -INFINITY;
    if (__any_sync(0xffffffffu, up0 || up1)) {
      const float n0 = up0 ? mx0 : m0, n1 = up1 ? mx1 : m1;
      const float a0 = m0 == -INFINITY ? 0.f : ex2((m0 - n0) * f0), a1 = m1 == -INFINITY ? 0.f : ex2((m1 - n1) * f1);
      m0 = n0;
      m1 = n1;
      l0 *= a0;
      l1 *= a1;
#pragma unroll
      for (int nt = 0; nt < 16; ++nt) {
        acc[nt][0] *= a0;
        acc[nt][1] *= a0;
        acc[nt][2] *= a1;
        acc[nt][3] *= a1;
      }
    }
    const float e0 = m0 == -INFINITY ? 0.f : -m0, e1 = m1 == -INFINITY ? 0.f : -m1;
    // P in fp16 (11 significant bits); the row sum takes the rounded values, so
    // rounding does not change the weights' total.  Exponents are (s - m) f, of which the
    // maximum's own is exactly 0: fma(s, f, -(m f)) is off by half a unit of m f, which passes 16
    // from logits of 2^29 on.
    auto weights = [](float x, float y, float e, float f) {
      const float2 z = __fmul2_rn(__fadd2_rn(make_float2(x, y), make_float2(e, e)), make_float2(f, f));
      return __floats2half2_rn(ex2(z.x), ex2(z.y));
    };
    uint32_t pa[2][4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const __half2 p0 = weights(s[nt][0], s[nt][1], e0, f0), p1 = weights(s[nt][2], s[nt][3], e1, f1);
      const float2 r0 = __half22float2(p0), r1 = __half22float2(p1);
      l0 += r0.x + r0.y;
      l1 += r1.x + r1.y;
      pa[nt >> 1][2 * (nt & 1)] = h2u(p0);
      pa[nt >> 1][2 * (nt & 1) + 1] = h2u(p1);
    }
    // ---- O += P V
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      // keys c + 4 r, r = 0 .. 3, channels 16 g ..; each conversion takes a byte with
      // one channel's codes of two keys, the pair that the B operand wants
      uint2 w[4];
      uint32_t sb[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int key = 16 * kk + c + 4 * r;
        w[r] = *reinterpret_cast<const uint2*>(dv + kCodeBytes * key + 8 * g);
        sb[r] = key < nvalid ? dvs[kScaleBytes * key + g] : 0u;
      }
      __half2 s2[2];
#pragma unroll
      for (int r = 0; r < 2; ++r)
        s2[r] = __half2(__nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>(sb[2 * r] | sb[2 * r + 1] << 8), __NV_E4M3));
#pragma unroll
      for (int q8 = 0; q8 < 2; ++q8) {             // 8 channels
        __half2 ev[2][4], od[2][4];                // even and odd channels, keys r = 0, 1 and 2, 3
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t x = q8 ? w[2 * r].y : w[2 * r].x, y = q8 ? w[2 * r + 1].y : w[2 * r + 1].x;
          codes_half2((x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u), ev[r]);
          codes_half2(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), od[r]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {              // channels 16 g + 8 q8 + 2 j and + 1
          const int nt = 8 * q8 + 2 * j;
          mma_f16_16816(acc[nt], pa[kk][0], pa[kk][1], pa[kk][2], pa[kk][3],
                        h2u(__hmul2(ev[0][j], s2[0])), h2u(__hmul2(ev[1][j], s2[1])));
          mma_f16_16816(acc[nt + 1], pa[kk][0], pa[kk][1], pa[kk][2], pa[kk][3],
                        h2u(__hmul2(od[0][j], s2[0])), h2u(__hmul2(od[1][j], s2[1])));
        }
      }
    }
    __syncwarp();                                  // every lane has read the buffer
    load();
  }
  // Wait (bounded) for whatever is still on its way: after a wait that ran out, and
  // for whole slabs in which this warp had no valid keys.
  if (kWhole) {
    if (warp == 0)
      for (int i = 0; i < kBlocks; ++i)
        if (sm.page[i] >= 0) (void)mbar_wait(&sm.full[0][0] + i, 0, status, 83);
  } else if (dead) {
    for (++nuse; nuse < nload; ++nuse)
      (void)mbar_wait(&sm.full[warp][nuse % Smem::kStages], (nuse / Smem::kStages) & 1, status, 83);
  }
  __syncthreads();                                 // the keys make room for the warps' sums
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  // ---- the CTA's warps, then the cluster's CTAs
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // columns 2c, 2c + 1 of n-tile i: channels 32 c + i and 32 c + 16 + i
    float* ow = &sm.o[warp][0][0];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<float4*>(ow + o_at(g + 8 * (e >> 1), 8 * c + 4 * (e & 1) + j)) =
          make_float4(acc[4 * j][e], acc[4 * j + 1][e], acc[4 * j + 2][e], acc[4 * j + 3][e]);
  }
  if (c == 0) {
    sm.ml[warp][g][0] = m0 * f0;                   // finite, or -inf without keys
    sm.ml[warp][g][1] = l0;
    sm.ml[warp][g + 8][0] = m1 * f1;
    sm.ml[warp][g + 8][1] = l1;
  }
  __syncthreads();
  cluster_wait();                                  // every CTA's barrier is initialised
  {
    const int r = tid >> 3;                        // 16 rows x 8 threads, float4s tid % 8 + 8 j
    float mm = -INFINITY, f[kAtWarps], l = 0.f;
#pragma unroll
    for (int w = 0; w < kAtWarps; ++w) mm = fmaxf(mm, sm.ml[w][r][0]);
#pragma unroll
    for (int w = 0; w < kAtWarps; ++w) {
      f[w] = sm.ml[w][r][0] == -INFINITY ? 0.f : ex2(sm.ml[w][r][0] - mm);
      l += f[w] * sm.ml[w][r][1];
    }
    // to the CTA that finishes the row
    const uint32_t to = r / kRows, bar = cluster_map(smem_u32(&sm.joined), to);
    const uint32_t row_at = cluster_map(smem_u32(sm.part[split][r % kRows]), to);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = o_at(r, (tid & 7) + 8 * j);
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][0][0] + at);
        t.x = fmaf(f[w], x.x, t.x);
        t.y = fmaf(f[w], x.y, t.y);
        t.z = fmaf(f[w], x.z, t.z);
        t.w = fmaf(f[w], x.w, t.w);
      }
      if (r < G) st_async4(row_at + 16 * ((tid & 7) + 8 * j), t, bar);
    }
    if ((tid & 7) == 0 && r < G) st_async2(cluster_map(smem_u32(sm.part_ml[split][r % kRows]), to), mm, l, bar);
  }
  // ---- this CTA's rows of the result, a warp each.  Every CTA stores its sums, also
  // after waits that ran out, a few limits later at most: none leaves while it is
  // stored to.
  if (warp >= my_rows) return;
  bool here = false;
  for (int t = 0; t < 8 && !here; ++t) here = mbar_wait<true>(&sm.joined, 0, status, 84);
  for (int w = warp; w < my_rows; w += kAtWarps) {
    const int r = split * kRows + w;
    float mm = -INFINITY, l = 0.f;
#pragma unroll
    for (int p = 0; p < NS; ++p) mm = fmaxf(mm, sm.part_ml[p][w][0]);
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < NS; ++p) {
      const float2 ml = *reinterpret_cast<const float2*>(sm.part_ml[p][w]);
      const float4 x = *reinterpret_cast<const float4*>(&sm.part[p][w][4 * lane]);
      const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - mm);
      l = fmaf(f, ml.y, l);
      t.x = fmaf(f, x.x, t.x);
      t.y = fmaf(f, x.y, t.y);
      t.z = fmaf(f, x.z, t.z);
      t.w = fmaf(f, x.w, t.w);
    }
    const float inv = l > 0.f ? v_gain / l : 0.f;
    uint2 out;
    out.x = pack_bf16x2(t.x * inv, t.y * inv);
    out.y = pack_bf16x2(t.z * inv, t.w * inv);
    *reinterpret_cast<uint2*>(o + (static_cast<size_t>(b) * G * Hkv + static_cast<size_t>(h) * G + r) * kD +
                              4 * lane) = out;
  }
}

// ---------------------------------------------------------------- host

namespace {

struct Decode4Workspace {
  float* scores;       // [B, Hkv, max_pages]
};

Decode4Workspace carve_decode4_workspace(WsCursor& ws, int B, int Hkv, int max_pages) {
  Decode4Workspace w;
  w.scores = ws.take<float>(static_cast<size_t>(B) * Hkv * max_pages);
  return w;
}

template <int NS, bool kWhole>
struct Attend4 {
  static constexpr size_t kSmem = sizeof(Attend4Smem<NS, kWhole>);

  // Launch attributes; the kernel's own, where they are not the default ones
  static msa_status_t prepare(cudaLaunchConfig_t* cfg, cudaLaunchAttribute (&attr)[2], int rows) {
    MSA_TRY(ensure_smem(decode4_attend_kernel<NS, kWhole>, kSmem, "decode4_attend_kernel"));
    if (NS > 8) {                                  // beyond the portable size of a cluster
      static std::atomic<bool> done[kMaxDevices];
      int dev = 0;
      if (cudaGetDevice(&dev) != cudaSuccess) return fail(MSA_ERR_CUDA, "cudaGetDevice failed");
      const bool known = dev >= 0 && dev < kMaxDevices;
      if (!known || !done[dev].load()) {
        const cudaError_t e = cudaFuncSetAttribute(decode4_attend_kernel<NS, kWhole>,
                                                   cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return fail(MSA_ERR_CUDA, "decode4_attend_kernel: %s", cudaGetErrorString(e));
        if (known) done[dev].store(true);
      }
    }
    cfg->gridDim = dim3(NS, static_cast<unsigned>(rows));
    cfg->blockDim = kAtThreads;
    cfg->dynamicSmemBytes = kSmem;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = NS;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg->attrs = attr;
    cfg->numAttrs = 1;
    return MSA_OK;
  }

  // Whether all the rows' clusters run side by side on the current device
  static bool fits(long long rows) {
    static std::atomic<int> most[kMaxDevices];     // clusters + 1, 0: not asked yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
    int n = most[dev].load();
    if (n == 0) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[2];
      int c = 0;
      if (prepare(&cfg, attr, 1) != MSA_OK ||
          cudaOccupancyMaxActiveClusters(&c, decode4_attend_kernel<NS, kWhole>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        c = 0;
      }
      n = c + 1;
      most[dev].store(n);
    }
    return rows < n;
  }

  static msa_status_t launch(const void* q, const void* kc, const void* vc, const int32_t* table,
                             const int32_t* lens, const float* scores, int B, int G, int Hkv,
                             int num_pages, int max_pages, int n_init, double logit_scale, float v_gain,
                             void* o, int32_t* sel_out, uint32_t* sw, cudaStream_t stream) {
    int e = 0;
    const float sl2 = static_cast<float>(2.0 * std::frexp(logit_scale, &e));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    MSA_TRY(prepare(&cfg, attr, B * Hkv));
    cfg.stream = stream;
    cfg.numAttrs = 2;
    TraceScope trace_("decode4_attend_kernel", stream);
    cudaLaunchKernelEx(&cfg, decode4_attend_kernel<NS, kWhole>, static_cast<const __nv_bfloat16*>(q),
                       static_cast<const uint8_t*>(kc), static_cast<const uint8_t*>(vc), table, lens,
                       scores, G, Hkv, num_pages, max_pages, n_init, sl2, e - 1, v_gain,
                       static_cast<__nv_bfloat16*>(o), sel_out, sw);
    return check_launch("decode4_attend_kernel");
  }
};

}  // namespace

}  // namespace msa

using namespace msa;

extern "C" {

size_t msa_decode4_step_workspace_size(int B, int Hq, int Hkv, int max_pages) {
  (void)Hq;
  if (B < 1 || Hkv < 1 || max_pages < 1) return 0;
  WsCursor ws(nullptr);
  carve_decode4_workspace(ws, B, Hkv, max_pages);
  return ws.used + 256;
}

msa_status_t msa_decode4_step(const void* q, const void* q_idx, const void* k_cache,
                              const void* v_cache, const void* kidx_cache,
                              const int32_t* block_table, const int32_t* cache_lens, int B, int Hq,
                              int Hkv, int num_pages, int max_pages, float scale, float k_gain,
                              float v_gain, int n_init, void* o, int32_t* sel_out, void* workspace,
                              size_t workspace_bytes, msa_stream_t stream) {
  MSA_REQUIRE_PTR(q);
  MSA_REQUIRE_PTR(q_idx);
  MSA_REQUIRE_PTR(k_cache);
  MSA_REQUIRE_PTR(v_cache);
  MSA_REQUIRE_PTR(kidx_cache);
  MSA_REQUIRE_PTR(block_table);
  MSA_REQUIRE_PTR(cache_lens);
  MSA_REQUIRE_PTR(o);
  MSA_REQUIRE_PTR(workspace);
  if (sel_out && !aligned16(sel_out))
    return fail(MSA_ERR_INVALID_ARG, "sel_out is not 16-byte aligned");
  if (B < 1) return fail(MSA_ERR_INVALID_ARG, "B must be >= 1");
  MSA_TRY(check_cache_sizes(Hkv, num_pages, max_pages));
  if (static_cast<long long>(B) * Hkv > 65535)
    return fail(MSA_ERR_UNSUPPORTED, "B * Hkv = %lld above 65535",
                static_cast<long long>(B) * Hkv);
  if (Hq < 1 || Hq % Hkv != 0)
    return fail(MSA_ERR_INVALID_ARG, "Hq (%d) must be a positive multiple of Hkv (%d)", Hq, Hkv);
  const int G = Hq / Hkv;
  if (G > 16) return fail(MSA_ERR_UNSUPPORTED, "at most 16 query heads per KV head (got %d)", G);
  if (!(scale > 0.0f) || !std::isfinite(scale))
    return fail(MSA_ERR_INVALID_ARG, "scale must be finite and > 0");
  MSA_TRY(check_gains(k_gain, v_gain, 1.0f));
  if (!std::isfinite(static_cast<float>(static_cast<double>(scale) * k_gain * kLog2e)))
    return fail(MSA_ERR_INVALID_ARG, "scale * k_gain overflows");
  if (n_init < 0 || n_init > kTopK - 1)
    return fail(MSA_ERR_INVALID_ARG, "n_init %d outside [0, %d]", n_init, kTopK - 1);
  if (workspace_bytes < msa_decode4_step_workspace_size(B, Hq, Hkv, max_pages))
    return fail(MSA_ERR_INVALID_ARG, "workspace too small");
  WsCursor ws(workspace);
  const Decode4Workspace w = carve_decode4_workspace(ws, B, Hkv, max_pages);
  uint32_t* sw = nullptr;
  MSA_TRY(status_word(&sw));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (max_pages > kTopK) {
    MSA_TRY(ensure_smem(decode4_score_kernel, sizeof(Score4Smem), "decode4_score_kernel"));
    {
      TraceScope trace_("decode4_score_kernel", st);
      launch_pdl(decode4_score_kernel, device_sm_count(), kScThreads, sizeof(Score4Smem), st,
                 static_cast<const __nv_bfloat16*>(q_idx), static_cast<const uint8_t*>(kidx_cache),
                 block_table, cache_lens, B, Hkv, num_pages, max_pages, n_init, w.scores, sw);
    }
    MSA_TRY(check_launch("decode4_score_kernel"));
  }
  // CTAs per row: as many as run side by side with all rows' (more of them shorten a
  // row's chain of blocks, a second wave costs more than that gains), with their slabs
  // whole while that fits too.  The whole step, rows of 4k - 8k tokens, 16 / 8 / 4 whole /
  // 4 / 2 / 1 CTAs: 20 rows 12.6 / 13.9 / 14.8 / 20.6 / 30.4 / 50.2 us, 40 rows 20.3 / 15.1 /
  // 15.9 / 21.8 / 31.6 / 51.3, 68 rows 36.6 / 26.7 / 19.7 / 24.7 / 34.1 / 53.4, 128 rows 64.9 /
  // 43.7 / 37.9 / 32.5 / 41.5 / 61.3, 304 rows 139 / 87 / 79 / 66 / 56 / 74; 1 CTA per row is
  // within 5 % of 2 from 480 rows on.
  const long long rows = static_cast<long long>(B) * Hkv;
  auto attend = Attend4<16, true>::fits(rows)  ? Attend4<16, true>::launch
                : Attend4<8, true>::fits(rows) ? Attend4<8, true>::launch
                : Attend4<4, true>::fits(rows) ? Attend4<4, true>::launch
                : Attend4<4, false>::fits(rows) ? Attend4<4, false>::launch
                                                : Attend4<2, false>::launch;
  return attend(q, k_cache, v_cache, block_table, cache_lens, w.scores, B, G, Hkv, num_pages,
                max_pages, n_init, static_cast<double>(scale) * k_gain * kLog2e, v_gain, o, sel_out, sw, st);
}

}  // extern "C"
