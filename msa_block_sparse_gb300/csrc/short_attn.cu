// Full attention of one new token per row over few pages (msa_decode_shared where a call's
// tables are small): one launch, in which every row is read by itself, instead of the plan, the
// items and their joining of shared_attn.cu.
//
// A cluster of up to 8 CTAs per (row, KV head); CTA `split` takes the row's pages split, split +
// NS, ..., each warp 32 keys of a page.  K and V come by TMA (128B-swizzled).  At most 16
// query heads per KV head make one m16 tile, so that the products are mma.sync m16n8k16 with
// operands straight from shared memory: a tcgen05 tile has 128 rows and would bring its
// round trips through TMEM.  The warps' sums are joined in the CTA, the CTAs' by
// asynchronous stores into the one that finishes a row.
//
// Bound by latency in the smallest calls (launch, lengths and table entries, K and V, the joining: 4
// rows of 1,500 tokens, 64 heads on 4, 5.8 us), by memory in the largest (8 rows of 8k tokens, 134 MB, 23
// us, 5.8 TB/s).  K and V each have one buffer, which refills while the other is in use: two of each
// leave room for one CTA per SM, and half of the clusters wait (4 rows x 13 pages 6.4 -> 10.1 us).
#include <cfloat>
#include "kernels.cuh"

namespace msa {

namespace {

constexpr int kShWarps = 4, kShThreads = 32 * kShWarps;
constexpr int kShHalf = 128 * 64 * 2;              // 64 channels of a page
constexpr int kShTile = 2 * kShHalf;               // K or V of a page

template <int NS>
struct ShortSmem {
  // sums (and maximum, weight) of this CTA's rows of the result, by sender
  alignas(16) float part[NS][16 / NS][kD];
  alignas(16) float part_ml[NS][16 / NS][2];
  float ml[kShWarps][16][2];
  uint64_t full_k, full_v;
  uint64_t joined;
};

__device__ __forceinline__ void sh_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void sh_ldmatrix_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ float sh_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t sh_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// Float4 `chunk` (channel / 4) of row r in a [16][128] array of sums: a fragment's stores (4
// rows x 2 chunks at a time) and the rows' loads (8 chunks) meet no bank twice
__device__ __forceinline__ int sh_at(int r, int chunk) { return r * kD + 4 * (chunk ^ ((r & 3) << 1)); }

}  // namespace

// grid (NS, rows x KV heads) in clusters of NS CTAs.  Column g of a tile of 8 keys is key
// (g >> 1) + 4 (g & 1), so that 16-byte loads of K meet no bank twice; the channels of
// two k-steps are a thread's 8 consecutive ones, for q and K alike.
template <int NS>
__global__ void __launch_bounds__(kShThreads, 3) short_attn_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const __nv_bfloat16* q, const int32_t* __restrict__ table, const int32_t* __restrict__ lens,
    int G, int Hkv, int num_pages, int max_pages, float sl2, __nv_bfloat16* o, float* __restrict__ lse,
    uint32_t* status) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ ShortSmem<NS> sm;
  // K, then V of a page; later the warps' sums
  uint8_t* kv = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  constexpr int kRows = 16 / NS;
  const int split = blockIdx.x, b = blockIdx.y / Hkv, h = blockIdx.y - b * Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int my_rows = max(0, min(G - split * kRows, kRows));   // of the result, to finish here
  if (tid == 0) {
    mbar_init(&sm.full_k, 1);
    mbar_init(&sm.full_v, 1);
    mbar_init(&sm.joined, 1);
    fence_mbar_init();
    if (my_rows > 0) mbar_arrive_expect_tx(&sm.joined, NS * my_rows * (kD + 2) * 4);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_enter();
  // ---- everything that depends on no other load is asked for at once
  const int L0 = lens[b], col = split + NS * lane;
  const int entry = col < max_pages ? table[static_cast<size_t>(b) * max_pages + col] : -1;
  const __nv_bfloat16* qr = q + (static_cast<size_t>(b) * Hkv + h) * G * kD;
  uint4 q0[4], q1[4];                              // rows g and g + 8, channels 8 (4 i + c) ..
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q0[i] = q1[i] = make_uint4(0u, 0u, 0u, 0u);
    if (g < G) q0[i] = reinterpret_cast<const uint4*>(qr + g * kD)[4 * i + c];
    if (g + 8 < G) q1[i] = reinterpret_cast<const uint4*>(qr + (g + 8) * kD)[4 * i + c];
  }
  const bool usable = L0 >= 0 && L0 <= max_pages * kBlock;
  const int L = usable ? L0 : 0, npages = (L + kBlock - 1) / kBlock;
  const bool there = col < npages, good = there && entry >= 0 && entry < num_pages;
  if (tid < 32 && ((there && !good) || !usable)) atomicOr(status, kStatusBounds);
  const uint32_t mask = __ballot_sync(0xffffffffu, good);   // pages that are none have no keys
  const int n = __popc(mask);
  uint32_t left[2] = {mask, mask}, to_do = mask;   // lanes of the pages that are left (K, V)
  auto load = [&](int v) {                         // the next page's K or V; whole warp 0
    const int at = __shfl_sync(0xffffffffu, entry, __ffs(left[v]) - 1) * Hkv + h;
    left[v] &= left[v] - 1;
    if (lane == 0) {
      uint8_t* dst = kv + v * kShTile;
      uint64_t* bar = v ? &sm.full_v : &sm.full_k;
      const CUtensorMap* tm = v ? &tm_v : &tm_k;
      mbar_arrive_expect_tx(bar, kShTile);
      tma_load_3d(dst, tm, bar, 0, 0, at);
      tma_load_3d(dst + kShHalf, tm, bar, 64, 0, at);
    }
  };
  if (warp == 0 && n > 0) {
    load(0);
    load(1);
  }
  __syncthreads();                                 // the barriers, for the other warps

  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // of rows g and g + 8, this thread's keys
  float acc[16][4];
#pragma unroll
  for (int nt = 0; nt < 16; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
  bool ok = true;
  for (int t = 0; t < n; ++t) {                    // the same for all threads
    const int at = split + NS * (__ffs(to_do) - 1);            // column
    to_do &= to_do - 1;
    const int tail = min(kBlock, L - at * kBlock) - 32 * warp;  // this warp's keys
    ok = ok && mbar_wait(&sm.full_k, t & 1, status, 140);
    ok = __all_sync(0xffffffffu, ok);
    float s[4][4];
    if (ok && tail > 0) {
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
        const int key = 32 * warp + 8 * nt + (g >> 1) + 4 * (g & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 k = *reinterpret_cast<const uint4*>(kv + (i >> 1) * kShHalf + sw128_offset(key, 4 * (i & 1) + c));
          const uint32_t lo[4] = {q0[i].x, q1[i].x, q0[i].y, q1[i].y}, hi[4] = {q0[i].z, q1[i].z, q0[i].w, q1[i].w};
          sh_mma(s[nt], lo, k.x, k.y);
          sh_mma(s[nt], hi, k.z, k.w);
        }
      }
    }
    if (t + 1 < n) {
      __syncthreads();                             // every warp is done with K
      if (warp == 0) {
        fence_proxy_async_smem();
        load(0);
      }
    }
    if (ok && tail > 0) {
      // ---- columns 2 c, 2 c + 1 of tile nt: keys 8 nt + c and 8 nt + c + 4
      float x0 = m0, x1 = m1;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (8 * nt + c + 4 * e >= tail) s[nt][e] = s[nt][2 + e] = -INFINITY;
          x0 = fmaxf(x0, s[nt][e]);
          x1 = fmaxf(x1, s[nt][2 + e]);
        }
      }
#pragma unroll
      for (int d = 1; d <= 2; d <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
      }
      // the maximum is subtracted before the factor; -infinity less itself would be NaN
      const float u0 = fmaxf(x0, -FLT_MAX), u1 = fmaxf(x1, -FLT_MAX);
      const float f0 = sh_ex2((m0 - u0) * sl2), f1 = sh_ex2((m1 - u1) * sl2);
      m0 = x0;
      m1 = x1;
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int nt = 0; nt < 16; ++nt) {
        acc[nt][0] *= f0;
        acc[nt][1] *= f0;
        acc[nt][2] *= f1;
        acc[nt][3] *= f1;
      }
      uint32_t p[2][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const float p00 = sh_ex2((s[nt][0] - u0) * sl2), p01 = sh_ex2((s[nt][1] - u0) * sl2);
        const float p10 = sh_ex2((s[nt][2] - u1) * sl2), p11 = sh_ex2((s[nt][3] - u1) * sl2);
        l0 += p00 + p01;
        l1 += p10 + p11;
        p[nt >> 1][2 * (nt & 1)] = pack_bf16x2(p00, p01);       // at most 2^-8 each
        p[nt >> 1][2 * (nt & 1) + 1] = pack_bf16x2(p10, p11);
      }
      ok = __all_sync(0xffffffffu, mbar_wait(&sm.full_v, t & 1, status, 141));
      if (ok) {
        uint8_t* vs = kv + kShTile;
        // what lies behind the row's end may be anything, and 0 times it has to be 0
        if (tail < 32) {
          if (lane >= tail) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              *reinterpret_cast<uint4*>(vs + (i >> 3) * kShHalf + (32 * warp + lane) * 128 + 16 * (i & 7)) =
                  make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          // row j of 16 of the product is key (j >> 3) 8 + (j & 7 >> 1) + 4 (j & 1), as in S
          const int j = lane & 15, key = 32 * warp + 16 * kk + (j & 8) + ((j & 7) >> 1) + 4 * (j & 1);
#pragma unroll
          for (int nt = 0; nt < 16; nt += 2) {
            const int ch = nt + (lane >> 4);       // 8 channels
            uint32_t v[4];
            sh_ldmatrix_t(v, smem_u32(vs) + (ch >> 3) * kShHalf + sw128_offset(key, ch & 7));
            sh_mma(acc[nt], p[kk], v[0], v[1]);
            sh_mma(acc[nt + 1], p[kk], v[2], v[3]);
          }
        }
      }
    }
    if (t + 1 < n) {
      __syncthreads();                             // and with V
      if (warp == 0) {
        fence_proxy_async_smem();
        load(1);
      }
    }
  }
  // a warp without keys, or after a wait that ran out, has not seen the copies land
  if (n > 0) {
    (void)mbar_wait(&sm.full_k, (n - 1) & 1, status, 142);
    (void)mbar_wait(&sm.full_v, (n - 1) & 1, status, 143);
  }
#pragma unroll
  for (int d = 1; d <= 2; d <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, d);
    l1 += __shfl_xor_sync(0xffffffffu, l1, d);
  }
  // keys, but no product that is a number: NaN, as the definition has it
  if (l0 != l0 && m0 == -INFINITY) m0 = 0.f;
  if (l1 != l1 && m1 == -INFINITY) m1 = 0.f;
  __syncthreads();                                 // the keys make room for the warps' sums
  float* sums = reinterpret_cast<float*>(kv);    // [warps][16][128]
#pragma unroll
  for (int nt = 0; nt < 16; ++nt) {
    // channels 8 nt + 2 c, + 1
    float* w = sums + warp * 16 * kD + 2 * (c & 1);
    *reinterpret_cast<float2*>(w + sh_at(g, 2 * nt + (c >> 1))) = make_float2(acc[nt][0], acc[nt][1]);
    *reinterpret_cast<float2*>(w + sh_at(g + 8, 2 * nt + (c >> 1))) = make_float2(acc[nt][2], acc[nt][3]);
  }
  if (c == 0) {
    sm.ml[warp][g][0] = m0;
    sm.ml[warp][g][1] = l0;
    sm.ml[warp][g + 8][0] = m1;
    sm.ml[warp][g + 8][1] = l1;
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // every CTA's barrier is there
  {
    const int r = tid >> 3;                        // 16 rows x 8 threads, float4s tid % 8 + 8 j
    float mm = -INFINITY, f[kShWarps], l = 0.f;
#pragma unroll
    for (int w = 0; w < kShWarps; ++w) mm = fmaxf(mm, sm.ml[w][r][0]);
#pragma unroll
    for (int w = 0; w < kShWarps; ++w) {
      f[w] = sm.ml[w][r][0] == -INFINITY ? 0.f : sh_ex2((sm.ml[w][r][0] - mm) * sl2);
      l += sm.ml[w][r][0] == -INFINITY ? 0.f : f[w] * sm.ml[w][r][1];
    }
    // to the CTA that finishes the row
    const uint32_t to = r / kRows, bar = sh_map(smem_u32(&sm.joined), to);
    const uint32_t row_at = sh_map(smem_u32(sm.part[split][r % kRows]), to);
    if (r < G) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int chunk = (tid & 7) + 8 * j;
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kShWarps; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(sums + w * 16 * kD + sh_at(r, chunk));
          if (f[w] == 0.f) continue;
          t.x = fmaf(f[w], x.x, t.x);
          t.y = fmaf(f[w], x.y, t.y);
          t.z = fmaf(f[w], x.z, t.z);
          t.w = fmaf(f[w], x.w, t.w);
        }
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                         row_at + 16 * chunk),
                     "f"(t.x), "f"(t.y), "f"(t.z), "f"(t.w), "r"(bar)
                     : "memory");
      }
      if ((tid & 7) == 0)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                         sh_map(smem_u32(sm.part_ml[split][r % kRows]), to)),
                     "f"(mm), "f"(l), "r"(bar)
                     : "memory");
    }
  }
  // ---- this CTA's rows of the result, a warp each.  Every CTA stores its sums, also after
  // waits that ran out, a few limits later at most: none leaves while it is stored to.
  if (warp >= my_rows) return;
  bool here = false;
  for (int t = 0; t < 8 && !here; ++t) here = mbar_wait<true>(&sm.joined, 0, status, 144);
  for (int w = warp; w < my_rows; w += kShWarps) {
    float mm = -INFINITY, l = 0.f;
#pragma unroll
    for (int p = 0; p < NS; ++p) mm = fmaxf(mm, sm.part_ml[p][w][0]);
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < NS; ++p) {
      const float2 ml = *reinterpret_cast<const float2*>(sm.part_ml[p][w]);
      const float4 x = *reinterpret_cast<const float4*>(&sm.part[p][w][4 * lane]);
      if (ml.x == -INFINITY) continue;
      const float f = sh_ex2((ml.x - mm) * sl2);
      l = fmaf(f, ml.y, l);
      t.x = fmaf(f, x.x, t.x);
      t.y = fmaf(f, x.y, t.y);
      t.z = fmaf(f, x.z, t.z);
      t.w = fmaf(f, x.w, t.w);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const size_t at = (static_cast<size_t>(b) * Hkv + h) * G + split * kRows + w;
    *reinterpret_cast<uint2*>(o + at * kD + 4 * lane) =
        make_uint2(pack_bf16x2(t.x * inv, t.y * inv), pack_bf16x2(t.z * inv, t.w * inv));
    if (lse && lane == 0) lse[at] = mm == -INFINITY ? -INFINITY : fmaf(mm, sl2, log2f(l)) * 0.6931471805599453f;
  }
}

// CTAs per (row, KV head), and how many of them an SM takes: two where all of them then run side by
// side (three would crowd some SMs: 16 x 4 rows of 8 pages 6.2 us and 7.7), else three.  Clusters leave
// gaps: of 304 places those of 4 CTAs fill about 285, those of 8 266.  More CTAs than run at two per SM
// pay where each keeps 4 pages or more (24 x 4 rows of 16 pages 11.3 us with 4 CTAs, 14.8 with 2; 76 rows of
// 8 7.8 and 7.5).
struct ShortPlan {
  int ctas, per_sm;
};
static ShortPlan short_plan(int rows, int max_pages) {
  const int sms = device_sm_count();
  auto places = [&](int n) { return n == 8 ? 7 * sms / 4 : n == 4 ? 15 * sms / 8 : 2 * sms; };
  for (int n = 8; n > 1; n /= 2) {
    if (max_pages <= n / 2) continue;
    if (n * rows <= places(n)) return {n, 2};
    if (2 * n * rows <= 3 * places(n) && max_pages >= 4 * n) return {n, 3};
  }
  return {1, rows <= places(1) ? 2 : 3};
}

namespace {

template <int NS>
msa_status_t launch_short(const ShortAttn& a, int per_sm, cudaStream_t st, uint32_t* sw) {
  // a third of an SM's shared memory; so much more that only two fit
  constexpr size_t kSmem = 2 * kShTile + 1024, kMore = 16384;
  MSA_TRY(ensure_smem(short_attn_kernel<NS>, kSmem + kMore, "short_attn_kernel"));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = NS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(NS, static_cast<unsigned>(a.B * a.Hkv));
  cfg.blockDim = kShThreads;
  cfg.dynamicSmemBytes = kSmem + (per_sm == 2 ? kMore : 0);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, short_attn_kernel<NS>, a.tm_k, a.tm_v, a.q, a.table, a.lens, a.G, a.Hkv, a.num_pages,
                     a.max_pages, a.sl2, a.o, a.lse, sw);
  return check_launch("short_attn_kernel");
}

}  // namespace

// Few pages in all, and few of a row, so that reading every row by itself, mostly from L2 where
// rows share, costs less than finding out what they share.  This kernel against the three of
// shared_attn.cu on the same tables (16 heads per KV head, 4 KV heads): 1 row x 4 pages 3.7 us against 13.0; 4 x 13,
// 11 of them shared, 6.0 against 15.9; 8 x 64 all different 23 against 38, all shared 14.9 against 22.5; 24 x 60
// up to 60 pages each 34 against 53, all 60 shared 29 against 35 (26.6 with 2 heads).  The borders are where rows that
// are full and share everything take as long in either form: 20 x 70 33.7 and 34.5, 16 x 80 30.9 and 29.9, 10 x 125
// 30.4 and 30.7; and where a CTA walks many pages alone: 1 x 128 20.6 and 22.0.
bool short_attn_fits(int B, int G, int Hkv, int max_pages) {
  const long long rows = static_cast<long long>(B) * Hkv;
  return G <= 16 && max_pages <= 128 && rows * max_pages <= 40LL * device_sm_count() &&
         max_pages <= 20 * short_plan(static_cast<int>(rows), max_pages).ctas;    // a lane per page of a CTA
}

msa_status_t launch_short_attn(const ShortAttn& a, cudaStream_t stream) {
  uint32_t* sw = nullptr;
  MSA_TRY(status_word(&sw));
  TraceScope trace_("short_attn_kernel", stream);
  const ShortPlan plan = short_plan(a.B * a.Hkv, a.max_pages);
  switch (plan.ctas) {
    case 8: return launch_short<8>(a, plan.per_sm, stream, sw);
    case 4: return launch_short<4>(a, plan.per_sm, stream, sw);
    case 2: return launch_short<2>(a, plan.per_sm, stream, sw);
    default: return launch_short<1>(a, plan.per_sm, stream, sw);
  }
}

}  // namespace msa
