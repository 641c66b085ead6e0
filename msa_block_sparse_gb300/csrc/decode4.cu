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
#include <cmath>
#include "cache4.cuh"

namespace msa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kD4Threads = 128;

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

constexpr int kScWarps = 12;
constexpr int kScStages = 2;
constexpr int kScMaxB = 1024;   // rows whose unit counts are summed in shared memory

struct Score4Smem {
  alignas(128) uint8_t slab[kScWarps][kScStages][kSlab];
  uint64_t full[kScWarps][kScStages];
  int start[kScMaxB + 1];       // first unit of each sequence of the pass
  int warp_sums[kScWarps];
};
static_assert(sizeof(Score4Smem) <= 232448, "score shared memory above the 227 KB limit");

// Persistent CTAs, one per SM.  The units (sequence, head, block to score) are
// counted from the lengths by every CTA and cut into equal runs, one per warp of the
// grid; a warp streams its slabs through its own two buffers with bulk copies and
// shares nothing with the others.  Rows beyond 1024 are taken in further passes.
__global__ void __launch_bounds__(32 * kScWarps, 1) decode4_score_kernel(
    const __nv_bfloat16* __restrict__ q_idx, const uint8_t* __restrict__ kidx,
    const int32_t* __restrict__ table, const int32_t* __restrict__ lens, int B, int Hkv,
    int num_pages, int max_pages, int n_init, float* __restrict__ scores, uint32_t* status) {
  pdl_enter();
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Score4Smem& sm = *reinterpret_cast<Score4Smem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int gw = blockIdx.x * kScWarps + warp, nw = gridDim.x * kScWarps;
  if (lane == 0) {
    for (int i = 0; i < kScStages; ++i) mbar_init(&sm.full[warp][i], 1);
    fence_mbar_init();
  }
  uint32_t nload = 0, nuse = 0;                    // slabs asked for and used by this warp
  bool dead = false;                               // a wait ran out
  for (int b0 = 0; b0 < B; b0 += kScMaxB) {
    const int nb = min(kScMaxB, B - b0);
    // ---- start[i] = units of the sequences before i; none where all blocks are kept
    auto units_of = [&](int b) {
      const int L = d4_len(lens[b], max_pages, status);
      const int own = (L + kBlock - 1) / kBlock - 1;
      return own >= kTopK ? (own - n_init) * Hkv : 0;
    };
    __syncthreads();
    int carry = 0;
    for (int i0 = 0; i0 < nb; i0 += 32 * kScWarps) {
      const int i = i0 + tid;
      const int v = i < nb ? units_of(b0 + i) : 0;
      int x = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
      }
      if (lane == 31) sm.warp_sums[warp] = x;
      __syncthreads();
      int before = carry, total = carry;
#pragma unroll
      for (int w = 0; w < kScWarps; ++w) {
        if (w < warp) before += sm.warp_sums[w];
        total += sm.warp_sums[w];
      }
      if (i < nb) sm.start[i] = before + x - v;
      carry = total;
      __syncthreads();
    }
    if (tid == 0) sm.start[nb] = carry;
    __syncthreads();
    const int total = carry;
    // ---- this warp's run of units
    const int u0 = static_cast<int>(static_cast<long long>(total) * gw / nw);
    const int u1 = static_cast<int>(static_cast<long long>(total) * (gw + 1) / nw);
    if (u0 >= u1 || dead) continue;
    // lane l keeps (row, head, block, page) of unit base + l
    int my_bh = 0, my_blk = 0, my_pg = -1;
    auto look_up = [&](int base) {
      const int u = base + lane;
      my_pg = -1;
      if (u < u1) {
        int lo = 0, hi = nb;                       // largest i with start[i] <= u
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (sm.start[mid] <= u) lo = mid; else hi = mid;
        }
        const int b = b0 + lo, r = u - sm.start[lo];
        const int per = (sm.start[lo + 1] - sm.start[lo]) / Hkv;   // blocks of one head
        const int h = r / per;
        my_bh = b * Hkv + h;
        my_blk = n_init + r - h * per;
        my_pg = table[static_cast<size_t>(b) * max_pages + my_blk];
        if (my_pg < 0 || my_pg >= num_pages) {
          atomicOr(status, kStatusBounds);
          scores[static_cast<size_t>(my_bh) * max_pages + my_blk] = -INFINITY;
          my_pg = -1;
        }
      }
    };
    int have_bh = -1;
    uint32_t bq[2][4][2];                          // B operand of the k-steps
    bool ok = true;
    for (int base = u0; base < u1 && ok; base += 32) {
      look_up(base);
      // units of this group that have a page, in order
      uint32_t todo = __ballot_sync(0xffffffffu, my_pg >= 0), ask = todo;
      auto load = [&]() {
        if (!ask) return;
        const int j = __ffs(ask) - 1;
        ask &= ask - 1u;
        const int pg = __shfl_sync(0xffffffffu, my_pg, j), bh = __shfl_sync(0xffffffffu, my_bh, j);
        if (lane == 0) {
          const int st = nload % kScStages;
          mbar_arrive_expect_tx(&sm.full[warp][st], kSlab);
          bulk_load(sm.slab[warp][st], kidx + (static_cast<size_t>(pg) * Hkv + bh % Hkv) * kSlab, kSlab,
                    &sm.full[warp][st]);
        }
        ++nload;
      };
      for (int i = 0; i < kScStages; ++i) load();
      while (todo) {
        const int j = __ffs(todo) - 1;
        todo &= todo - 1u;
        const int bh = __shfl_sync(0xffffffffu, my_bh, j), blk = __shfl_sync(0xffffffffu, my_blk, j);
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
        const int st = nuse % kScStages;
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.full[warp][st], (nuse / kScStages) & 1, status, 81))) {
          ok = false;
          break;
        }
        ++nuse;
        const uint8_t* slab = sm.slab[warp][st];
        float best = -INFINITY;
#pragma unroll 2
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
        __syncwarp();                              // every lane has read the buffer
        load();
#pragma unroll
        for (int m = 4; m <= 16; m <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, m));
        if (lane == 0) scores[static_cast<size_t>(bh) * max_pages + blk] = best;
      }
    }
    if (!ok) {                                     // slabs still on their way: wait (bounded), leave
      for (; nuse < nload; ++nuse)
        (void)mbar_wait(&sm.full[warp][nuse % kScStages], (nuse / kScStages) & 1, status, 82);
      dead = true;
    }
  }
}

// ---------------------------------------------------------------- attention

constexpr int kAtWarps = kD4Threads / 32;
constexpr int kCand = kTopK;        // candidates per warp: 15 and one empty

template <int NS>
struct Attend4Smem {
  static constexpr int kBlocks = kTopK / NS;       // blocks per CTA
  alignas(16) uint8_t k[kBlocks][kSlab];
  alignas(16) uint8_t v[kBlocks][kSlab];
  alignas(16) float o[kAtWarps][16][kD];           // per warp, then [0] = the CTA's sum
  float ml[kAtWarps][16][2];
  float cta_ml[16][2];
  union {
    alignas(16) uint2 cand[kAtWarps * kCand];      // selection: (key, block)
    uint32_t qh[16 * kD / 2];                      // q rows, packed fp16
  };
  float qfac[16];                                  // per row: what undoes q's power of two
  uint32_t bits[kMaxSeqlen / kBlock / 32];         // kept blocks
  int list[kTopK];
  int page[kBlocks];
  uint64_t full[kBlocks];
};

__device__ __forceinline__ uint32_t cluster_map(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// grid (NS, B * Hkv) in clusters of NS CTAs; CTA `split` attends to the selected
// blocks split, split + NS, ...  Each warp takes 32 keys of every block.
//
// S = Q K^T: rows are heads; n-tile column g is key (g >> 1) + 4 (g & 1) of 8, so
// that the accumulator's column pair (2c, 2c + 1) is keys (c, c + 4), which is how
// the rows of V are then read (rows c, c + 4, c + 8, c + 12 of 16: both halves of
// the shared-memory banks).  Channels of a k-step as in the score kernel.
// O = P V: thread (g, c) reads 8 bytes of codes = scale block g of a key, column
// g of n-tile i is channel 16 g + i.  Keys behind the sequence's end have P = 0 and
// scale 0, whatever their slots hold.
template <int NS>
__global__ void __launch_bounds__(kD4Threads) decode4_attend_kernel(
    const __nv_bfloat16* __restrict__ q, const uint8_t* __restrict__ kc,
    const uint8_t* __restrict__ vc, const int32_t* __restrict__ table,
    const int32_t* __restrict__ lens, const float* __restrict__ scores, int G, int Hkv,
    int num_pages, int max_pages, int n_init, float sl2, float v_gain,
    __nv_bfloat16* __restrict__ o, int32_t* __restrict__ sel_out, uint32_t* status) {
  pdl_enter();
  extern __shared__ __align__(128) uint8_t smem_raw[];
  using Smem = Attend4Smem<NS>;
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  constexpr int kBlocks = Smem::kBlocks;
  const int split = blockIdx.x, bh = blockIdx.y, b = bh / Hkv, h = bh % Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int L = d4_len(lens[b], max_pages, status);
  const int nblk = (L + kBlock - 1) / kBlock;
  const int own = nblk - 1;
  if (tid == 0) {
    for (int i = 0; i < kBlocks; ++i) mbar_init(&sm.full[i], 1);
    fence_mbar_init();
  }
  // ---- selection (every CTA of the cluster for itself)
  if (tid < kMaxSeqlen / kBlock / 32) sm.bits[tid] = 0u;
  if (tid < kTopK) sm.list[tid] = -1;
  if (own >= kTopK) {
    // Block 128 r + 32 w + l is lane l's r-th of warp w.  Each warp takes out its
    // 15 best in turn (ties: lowest id), then the 60 candidates are ranked.
    const float* sc = scores + static_cast<size_t>(bh) * max_pages;
    constexpr int kPer = kMaxSeqlen / kBlock / kD4Threads;
    uint32_t key[kPer];                            // ordered as the scores are; 0: none
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      const int i = kD4Threads * r + tid;
      key[r] = 0u;
      if (i < own) {
        // + 0: a score of -0 equals one of 0
        const uint32_t u = i < n_init ? 0u : __float_as_uint(sc[i] + 0.f);
        key[r] = i < n_init ? 0xFFFFFFFFu : (u & 0x80000000u ? ~u : u | 0x80000000u);
      }
    }
    __syncthreads();                               // bits and list are set up
#pragma unroll 1
    for (int n = 0; n < kTopK - 1; ++n) {
      uint32_t top = key[0];
      int at = 0;
#pragma unroll
      for (int r = 1; r < kPer; ++r)
        if (key[r] > top) top = key[r], at = r;
      const uint32_t best = __reduce_max_sync(0xffffffffu, top);
      const uint32_t id = static_cast<uint32_t>(kD4Threads * at + tid);
      const uint32_t win = __reduce_min_sync(0xffffffffu, top == best ? id : 0xFFFFFFFFu);
      if (lane == 0) sm.cand[warp * kCand + n] = make_uint2(best, win);
      if (best == 0u) {                            // the warp has no more blocks
        for (int k = n + 1 + lane; k < kTopK - 1; k += 32) sm.cand[warp * kCand + k] = make_uint2(0u, 0u);
        break;
      }
#pragma unroll
      for (int r = 0; r < kPer; ++r)
        if (id == win && r == at) key[r] = 0u;
    }
    if (lane == 0) sm.cand[warp * kCand + kCand - 1] = make_uint2(0u, 0u);
    __syncthreads();
    if (tid < kAtWarps * kCand) {
      const uint2 me = sm.cand[tid];
      int before = 0;
#pragma unroll 16
      for (int j = 0; j < kAtWarps * kCand; ++j) {
        const uint2 x = sm.cand[j];
        before += (x.x > me.x || (x.x == me.x && x.y < me.y)) ? 1 : 0;
      }
      if (me.x != 0u && before < kTopK - 1) atomicOr(&sm.bits[me.y >> 5], 1u << (me.y & 31));
    }
    if (tid == kD4Threads - 1) atomicOr(&sm.bits[own >> 5], 1u << (own & 31));
    __syncthreads();
    if (warp == 0) {                               // set bits in ascending order
      uint32_t m = sm.bits[lane];
      int at = __popc(m);
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, at, d);
        if (lane >= d) at += x;
      }
      at -= __popc(m);
      while (m && at < kTopK) {
        sm.list[at++] = 32 * lane + __ffs(m) - 1;
        m &= m - 1u;
      }
    }
  } else {
    __syncthreads();
    if (tid < nblk) sm.list[tid] = tid;            // every block
  }
  __syncthreads();
  if (split == 0 && tid < kTopK && sel_out)
    sel_out[static_cast<size_t>(bh) * kTopK + tid] = sm.list[tid];
  // ---- this CTA's blocks: all K and V slabs on their way at once
  if (tid < kBlocks) {
    const int blk = sm.list[split + NS * tid];
    int pg = -1;
    if (blk >= 0) {
      pg = table[static_cast<size_t>(b) * max_pages + blk];
      if (pg < 0 || pg >= num_pages) {
        atomicOr(status, kStatusBounds);
        pg = -1;
      }
    }
    sm.page[tid] = pg;
    if (pg >= 0) {
      const size_t off = (static_cast<size_t>(pg) * Hkv + h) * kSlab;
      mbar_arrive_expect_tx(&sm.full[tid], 2 * kSlab);
      bulk_load(sm.k[tid], kc + off, kSlab, &sm.full[tid]);
      bulk_load(sm.v[tid], vc + off, kSlab, &sm.full[tid]);
    }
  }
  // ---- q rows as fp16 with a power of two per row; warp w rows 4w .. 4w + 3
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * warp + i;
    uint2 x = make_uint2(0u, 0u);
    if (r < G)
      x = *reinterpret_cast<const uint2*>(
          q + (static_cast<size_t>(b) * G * Hkv + static_cast<size_t>(h) * G + r) * kD + 4 * lane);
    uint32_t m = __vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu);
    m = max(m & 0xFFFFu, m >> 16);
    m = __reduce_max_sync(0xffffffffu, m);
    const int e = row_shift(m);
    const float f = exp2i(e);
    sm.qh[r * (kD / 2) + 2 * lane] = bf2_to_h2(x.x, f);
    sm.qh[r * (kD / 2) + 2 * lane + 1] = bf2_to_h2(x.y, f);
    if (lane == 0) sm.qfac[r] = exp2i(-e);
  }
  __syncthreads();
  uint32_t qa[8][4];                               // A operand of the 8 k-steps
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const uint2 r0 = *reinterpret_cast<const uint2*>(&sm.qh[g * (kD / 2) + 16 * c + 2 * t]);
    const uint2 r1 = *reinterpret_cast<const uint2*>(&sm.qh[(g + 8) * (kD / 2) + 16 * c + 2 * t]);
    qa[t][0] = r0.x;
    qa[t][1] = r1.x;
    qa[t][2] = r0.y;
    qa[t][3] = r1.y;
  }
  const float f0 = sl2 * sm.qfac[g], f1 = sl2 * sm.qfac[g + 8];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  float acc[16][4];
#pragma unroll
  for (int nt = 0; nt < 16; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;

#pragma unroll 1
  for (int i = 0; i < kBlocks; ++i) {
    if (sm.page[i] < 0) continue;                  // uniform over the CTA
    const int blk = sm.list[split + NS * i];
    const int nvalid = blk == own ? L - own * kBlock : kBlock;
    const int kw = 32 * warp;                      // this warp's first key
    if (!__all_sync(0xffffffffu, mbar_wait(&sm.full[i], 0, status, 80))) break;
    if (kw >= nvalid) continue;                    // uniform over the warp
    // ---- S
    float s[4][4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
      const int key = kw + 8 * nt + (g >> 1) + 4 * (g & 1);
      const uint4 w4 = *(reinterpret_cast<const uint4*>(sm.k[i] + slab_code(key)) + c);
      const uint32_t sc = *(reinterpret_cast<const uint16_t*>(sm.k[i] + slab_scale(key)) + c);
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
      const __half2 sh = __half2(
          __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(sc), __NV_E4M3));
#pragma unroll
      for (int j = 0; j < 4; ++j) {                // 8 channels: two k-steps
        __half2 hh[4];
        codes_half2(w[j], hh);
        const __half2 s2 = j < 2 ? __low2half2(sh) : __high2half2(sh);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int t = 2 * j + k;
          mma_f16_16816(s[nt], qa[t][0], qa[t][1], qa[t][2], qa[t][3],
                        h2u(__hmul2(hh[2 * k], s2)), h2u(__hmul2(hh[2 * k + 1], s2)));
        }
      }
    }
    // ---- mask and running softmax of this warp's keys
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool ok = kw + 8 * nt + c + 4 * e < nvalid;
        s[nt][e] = ok ? s[nt][e] * f0 : -INFINITY;
        s[nt][2 + e] = ok ? s[nt][2 + e] * f1 : -INFINITY;
        mx0 = fmaxf(mx0, s[nt][e]);
        mx1 = fmaxf(mx1, s[nt][2 + e]);
      }
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, m));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, m));
    }
    const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
    const float a0 = mn0 == -INFINITY ? 1.f : exp2f(m0 - mn0);
    const float a1 = mn1 == -INFINITY ? 1.f : exp2f(m1 - mn1);
    const float e0 = mn0 == -INFINITY ? 0.f : mn0, e1 = mn1 == -INFINITY ? 0.f : mn1;
    m0 = mn0;
    m1 = mn1;
    l0 *= a0;
    l1 *= a1;
#pragma unroll
    for (int nt = 0; nt < 16; ++nt) {
      acc[nt][0] *= a0;
      acc[nt][1] *= a0;
      acc[nt][2] *= a1;
      acc[nt][3] *= a1;
    }
    // P in fp16 (11 significant bits; the row's largest is 1): the row sum takes
    // the rounded values, so rounding does not change the weights' total
    uint32_t pa[2][4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const __half2 p0 = __floats2half2_rn(exp2f(s[nt][0] - e0), exp2f(s[nt][1] - e0));
      const __half2 p1 = __floats2half2_rn(exp2f(s[nt][2] - e1), exp2f(s[nt][3] - e1));
      const float2 r0 = __half22float2(p0), r1 = __half22float2(p1);
      l0 += r0.x + r0.y;
      l1 += r1.x + r1.y;
      pa[nt >> 1][2 * (nt & 1)] = h2u(p0);
      pa[nt >> 1][2 * (nt & 1) + 1] = h2u(p1);
    }
    // ---- O += P V
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      __half2 vv[4][8];                            // keys c, c + 4, c + 8, c + 12: channels 16 g ..
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int key = kw + 16 * kk + c + 4 * r;
        const uint2 w = *reinterpret_cast<const uint2*>(sm.v[i] + slab_code(key) + 8 * g);
        const uint32_t sb = key < nvalid ? sm.v[i][slab_scale(key) + g] : 0u;
        const __half2 s2 = __half2half2(__half(__nv_cvt_fp8_to_halfraw(
            static_cast<__nv_fp8_storage_t>(sb), __NV_E4M3)));
        __half2 t4[4];
        codes_half2(w.x, t4);
#pragma unroll
        for (int j = 0; j < 4; ++j) vv[r][j] = __hmul2(t4[j], s2);
        codes_half2(w.y, t4);
#pragma unroll
        for (int j = 0; j < 4; ++j) vv[r][4 + j] = __hmul2(t4[j], s2);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {                // channels 16 g + 2j and + 2j + 1
        const uint32_t lo0 = __byte_perm(h2u(vv[0][j]), h2u(vv[1][j]), 0x5410);
        const uint32_t lo1 = __byte_perm(h2u(vv[2][j]), h2u(vv[3][j]), 0x5410);
        const uint32_t hi0 = __byte_perm(h2u(vv[0][j]), h2u(vv[1][j]), 0x7632);
        const uint32_t hi1 = __byte_perm(h2u(vv[2][j]), h2u(vv[3][j]), 0x7632);
        mma_f16_16816(acc[2 * j], pa[kk][0], pa[kk][1], pa[kk][2], pa[kk][3], lo0, lo1);
        mma_f16_16816(acc[2 * j + 1], pa[kk][0], pa[kk][1], pa[kk][2], pa[kk][3], hi0, hi1);
      }
    }
  }
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  // ---- the CTA's warps, then the cluster's CTAs
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // columns 2c, 2c + 1 of n-tile i: channels 32 c + i and 32 c + 16 + i
    float* r0 = &sm.o[warp][g][32 * c + 4 * j];
    float* r1 = &sm.o[warp][g + 8][32 * c + 4 * j];
    *reinterpret_cast<float4*>(r0) = make_float4(acc[4 * j][0], acc[4 * j + 1][0], acc[4 * j + 2][0], acc[4 * j + 3][0]);
    *reinterpret_cast<float4*>(r0 + 16) = make_float4(acc[4 * j][1], acc[4 * j + 1][1], acc[4 * j + 2][1], acc[4 * j + 3][1]);
    *reinterpret_cast<float4*>(r1) = make_float4(acc[4 * j][2], acc[4 * j + 1][2], acc[4 * j + 2][2], acc[4 * j + 3][2]);
    *reinterpret_cast<float4*>(r1 + 16) = make_float4(acc[4 * j][3], acc[4 * j + 1][3], acc[4 * j + 2][3], acc[4 * j + 3][3]);
  }
  if (c == 0) {
    sm.ml[warp][g][0] = m0;
    sm.ml[warp][g][1] = l0;
    sm.ml[warp][g + 8][0] = m1;
    sm.ml[warp][g + 8][1] = l1;
  }
  __syncthreads();
  {
    const int r = tid >> 3, d0 = (tid & 7) * 16;   // 16 rows x 8 threads
    float mm = -INFINITY, f[kAtWarps], l = 0.f;
#pragma unroll
    for (int w = 0; w < kAtWarps; ++w) mm = fmaxf(mm, sm.ml[w][r][0]);
#pragma unroll
    for (int w = 0; w < kAtWarps; ++w) {
      f[w] = sm.ml[w][r][0] == -INFINITY ? 0.f : exp2f(sm.ml[w][r][0] - mm);
      l += f[w] * sm.ml[w][r][1];
    }
#pragma unroll
    for (int d = 0; d < 16; d += 4) {
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][r][d0 + d]);
        t.x = fmaf(f[w], x.x, t.x);
        t.y = fmaf(f[w], x.y, t.y);
        t.z = fmaf(f[w], x.z, t.z);
        t.w = fmaf(f[w], x.w, t.w);
      }
      *reinterpret_cast<float4*>(&sm.o[0][r][d0 + d]) = t;
    }
    if ((tid & 7) == 0) {
      sm.cta_ml[r][0] = mm;
      sm.cta_ml[r][1] = l;
    }
  }
  cluster_sync();
  {
    // CTA `split` finishes rows split * 16 / NS ..: 8 threads per row and 16
    // channels each (2 rows or more), 64 threads per row otherwise unused
    constexpr int kRows = 16 / NS;
    const int r = split * kRows + (tid >> 5), d0 = (tid & 31) * 4;
    if ((tid >> 5) < kRows && r < G) {
      const uint32_t mla = smem_u32(&sm.cta_ml[r][0]), oa = smem_u32(&sm.o[0][r][d0]);
      float2 ml[NS];
      float mm = -INFINITY, l = 0.f;
#pragma unroll
      for (int p = 0; p < NS; ++p) {
        ml[p] = ld_cluster2(cluster_map(mla, p));
        mm = fmaxf(mm, ml[p].x);
      }
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int p = 0; p < NS; ++p) {
        const float f = ml[p].x == -INFINITY ? 0.f : exp2f(ml[p].x - mm);
        const float4 x = ld_cluster4(cluster_map(oa, p));
        l = fmaf(f, ml[p].y, l);
        t.x = fmaf(f, x.x, t.x);
        t.y = fmaf(f, x.y, t.y);
        t.z = fmaf(f, x.z, t.z);
        t.w = fmaf(f, x.w, t.w);
      }
      const float inv = l > 0.f ? v_gain / l : 0.f;
      uint2 out;
      out.x = pack_bf16x2(t.x * inv, t.y * inv);
      out.y = pack_bf16x2(t.z * inv, t.w * inv);
      *reinterpret_cast<uint2*>(
          o + (static_cast<size_t>(b) * G * Hkv + static_cast<size_t>(h) * G + r) * kD + d0) = out;
    }
  }
  cluster_sync();                                  // no CTA leaves while it is read
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

template <int NS>
msa_status_t launch_attend4(const void* q, const void* kc, const void* vc, const int32_t* table,
                            const int32_t* lens, const float* scores, int B, int G, int Hkv,
                            int num_pages, int max_pages, int n_init, float sl2, float v_gain,
                            void* o, int32_t* sel_out, uint32_t* sw, cudaStream_t stream) {
  const size_t smem = sizeof(Attend4Smem<NS>);
  MSA_TRY(ensure_smem(decode4_attend_kernel<NS>, smem, "decode4_attend_kernel"));
  TraceScope trace_("decode4_attend_kernel", stream);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(NS, static_cast<unsigned>(B) * Hkv);
  cfg.blockDim = kD4Threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = NS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, decode4_attend_kernel<NS>, static_cast<const __nv_bfloat16*>(q),
                     static_cast<const uint8_t*>(kc), static_cast<const uint8_t*>(vc), table, lens,
                     scores, G, Hkv, num_pages, max_pages, n_init, sl2, v_gain,
                     static_cast<__nv_bfloat16*>(o), sel_out, sw);
  return check_launch("decode4_attend_kernel");
}

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
    TraceScope trace_("decode4_score_kernel", st);
    launch_pdl(decode4_score_kernel, device_sm_count(), 32 * kScWarps, sizeof(Score4Smem), st,
               static_cast<const __nv_bfloat16*>(q_idx), static_cast<const uint8_t*>(kidx_cache),
               block_table, cache_lens, B, Hkv, num_pages, max_pages, n_init, w.scores, sw);
    MSA_TRY(check_launch("decode4_score_kernel"));
  }
  return launch_attend4<4>(q, k_cache, v_cache, block_table, cache_lens, w.scores, B, G, Hkv,
                           num_pages, max_pages, n_init, scale * k_gain * kLog2e, v_gain, o,
                           sel_out, sw, st);
}

}  // extern "C"
