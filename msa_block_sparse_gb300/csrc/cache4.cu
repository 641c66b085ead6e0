// Writing and reading the 4-bit paged cache: a pack (store, load) and the new
// token of a decode step (append).  Moves of 256 bytes of bf16 against 72 bytes
// of pages per (token, head): bound by memory for a pack, by latency for a step.
// Measured: 15,190 tokens x 4 heads x 3 tensors (60 MB each way) stored and loaded in
// 21.0 us together, 5.7 TB/s (25.5 with 32-byte stores that a pair of instructions filled
// and the heads of all tensors in one loop); 64 new tokens appended and read back in 6.0 us.
//
// Store and load: one thread per 16 channels (32 bytes of bf16, 8 bytes of codes,
// one scale byte), so that a scale needs no exchange between threads.  The 8 threads of
// a row sit side by side and a warp takes 4 consecutive tokens of one head: its
// codes are 256 consecutive bytes of the slab and its scales one 32-byte sector.  A CTA
// finds the places of its 16 tokens once and then takes them through its share of a
// tensor's heads, the next head's loads in flight.
#include <cmath>
#include "cache4.cuh"

namespace msa {

namespace {

constexpr int kC4Threads = 128;
constexpr int kC4Ctas = 12;                 // per SM
constexpr int kC4Tokens = kC4Threads / 8;   // tokens of one head that a CTA takes together

struct Cache4Args {
  const __nv_bfloat16* x[3];     // store: inputs [T, H, 128]
  __nv_bfloat16* y[3];           // load: outputs
  uint8_t* cache[3];             // [num_pages, H, 9216]
  const uint8_t* rcache[3];
  float gain[3], inv_gain[3];
  const int32_t* table;
  const int32_t* cu;
  const int32_t* start;
  int n, S, T, H, num_pages, max_pages;
};

// Page and slot of token t's position; page -1: out of range, -2: not a token of
// the pack.  Every lane of the warp calls it (8 lanes per token, tokens ascending).
// Up to 32 sequences are searched by one load and a vote per token, more by bisection.
__device__ __forceinline__ int2 c4_place(const Cache4Args& a, int t, uint32_t* status) {
  int lo = 0, first, from = 0;
  const int begin = __ldg(a.cu), end = __ldg(a.cu + a.S);
  if (a.S <= 32) {
    const int lane = threadIdx.x & 31;
    const int cu = lane < a.S ? __ldg(a.cu + lane) : 0;
    const int st = a.start && lane < a.S ? __ldg(a.start + lane) : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {                  // largest s with cu[s] <= the warp's k-th token
      const int tk = __shfl_sync(0xffffffffu, t, 8 * k);
      const uint32_t at = __ballot_sync(0xffffffffu, lane < a.S && cu <= tk);
      if (lane >> 3 == k) lo = at ? 31 - __clz(at) : 0;
    }
    first = __shfl_sync(0xffffffffu, cu, lo);
    from = __shfl_sync(0xffffffffu, st, lo);
  } else {
    int hi = a.S;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.cu + mid) <= t) lo = mid; else hi = mid;
    }
    first = __ldg(a.cu + lo);
    if (a.start) from = __ldg(a.start + lo);
  }
  if (t >= a.T || t < begin || t >= end) return make_int2(-2, 0);
  const long long pos = static_cast<long long>(t - first) + from;
  int page = -1;
  if (pos >= 0 && pos < static_cast<long long>(a.max_pages) * kBlock)
    page = __ldg(a.table + static_cast<size_t>(lo) * a.max_pages + pos / kBlock);
  if (page < 0 || page >= a.num_pages) {
    atomicOr(status, kStatusBounds);
    return make_int2(-1, 0);
  }
  return make_int2(page, static_cast<int>(pos % kBlock));
}

}  // namespace

// grid (token groups, shares of the heads, tensors)
__global__ void __launch_bounds__(kC4Threads) cache4_store_kernel(const Cache4Args a,
                                                                  uint32_t* status) {
  pdl_enter();
  const int c = threadIdx.x & 7;                   // 16 channels
  const int t = blockIdx.x * kC4Tokens + (threadIdx.x >> 3), n = blockIdx.z;
  int h = blockIdx.y;
  const uint4* src = reinterpret_cast<const uint4*>(
      a.x[n] + (static_cast<size_t>(t) * a.H + h) * kD + 16 * c);
  uint4 u = make_uint4(0u, 0u, 0u, 0u), v = u;
  if (t < a.T) {                                   // asked for while the place is looked up
    u = __ldcs(src);
    v = __ldcs(src + 1);
  }
  const int2 at = c4_place(a, t, status);
  if (at.x < 0) return;
  uint8_t* slab = a.cache[n] + (static_cast<size_t>(at.x) * a.H + h) * kSlab;
  const int code_at = slab_code(at.y) + 8 * c, scale_at = slab_scale(at.y) + c;
  const float gain = a.gain[n], inv_gain = a.inv_gain[n];
  while (true) {
    uint32_t x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    h += gridDim.y;
    src += gridDim.y * (kD / 8);
    if (h < a.H) {
      u = __ldcs(src);
      v = __ldcs(src + 1);
    }
    uint32_t sb;
    const uint2 codes = quantise16(x, gain, inv_gain, &sb);
    *reinterpret_cast<uint2*>(slab + code_at) = codes;
    slab[scale_at] = static_cast<uint8_t>(sb);
    if (h >= a.H) return;
    slab += static_cast<size_t>(gridDim.y) * kSlab;
  }
}

// A thread's 16 channels are 8 c .. and 64 + 8 c .., so that 8 threads store 128
// consecutive bytes at a time.
__global__ void __launch_bounds__(kC4Threads) cache4_load_kernel(const Cache4Args a,
                                                                 uint32_t* status) {
  pdl_enter();
  const int c = threadIdx.x & 7;
  const int t = blockIdx.x * kC4Tokens + (threadIdx.x >> 3), n = blockIdx.z;
  const int2 at = c4_place(a, t, status);
  if (at.x == -2) return;
  int h = blockIdx.y;
  uint4* dst = reinterpret_cast<uint4*>(
      a.y[n] + (static_cast<size_t>(t) * a.H + h) * kD + 8 * c);
  const uint8_t* slab = a.rcache[n] + (static_cast<size_t>(max(at.x, 0)) * a.H + h) * kSlab;
  const int code_at = slab_code(at.y) + 4 * c, scale_at = slab_scale(at.y) + (c >> 1);
  const float gain = a.gain[n];
  uint32_t w[2] = {0u, 0u}, sb[2] = {0u, 0u};
  auto fetch = [&]() {
    if (at.x < 0) return;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      w[p] = __ldcs(reinterpret_cast<const uint32_t*>(slab + code_at + 32 * p));
      sb[p] = __ldcs(slab + scale_at + 4 * p);
    }
  };
  fetch();
  while (true) {
    const uint32_t cw[2] = {w[0], w[1]}, cs[2] = {sb[0], sb[1]};
    h += gridDim.y;
    slab += static_cast<size_t>(gridDim.y) * kSlab;
    if (h < a.H) fetch();
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      // code * scale * gain has at most 6 significant bits: exact in fp32 and in bf16
      const float s = scale_value(cs[p]) * gain;
      const float2 s2 = make_float2(s, s);
      __half2 h4[4];
      codes_half2(cw[p], h4);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __fmul2_rn(__half22float2(h4[i]), s2);
        o[i] = pack_bf16x2(f.x, f.y);
      }
      __stcs(dst + 8 * p, make_uint4(o[0], o[1], o[2], o[3]));
    }
    if (h >= a.H) return;
    dst += gridDim.y * (kD / 8);
  }
}

// CTAs: one per token group and tensor while that fills the GPU; the heads are split
// among several when there are few groups.
static dim3 c4_grid(int T, int n, int H) {
  const int groups = (T + kC4Tokens - 1) / kC4Tokens;
  const int want = (kC4Ctas * device_sm_count() + groups * n - 1) / (groups * n);
  return dim3(groups, want < H ? want : H, n);
}

// ---------------------------------------------------------------- append
//
// One new token per sequence: grid (B, row groups), a warp per row of the
// (Hq + 4 Hkv) rows q, index q, k, index k, v.  Lane l holds channels 4l ..
// 4l + 3; the row's normed values pass through shared memory so that any pairing
// finds its partner; the 4 lanes of a 16-channel block share its scale.
namespace {

constexpr int kApWarps = 4;

struct Append4Args {
  const __nv_bfloat16* src[5];    // q, index q, k, index k, v
  const __nv_bfloat16* w[4];
  __nv_bfloat16* out[2];          // q_out, q_idx_out
  uint8_t* cache[3];              // k, index k, v
  float gain[3], inv_gain[3];
  const int32_t* table;
  const int32_t* lens;
  int Hq, H, num_pages, max_pages, R, layout;
  float eps, rope_gain;
};

struct Append4Turns {
  unsigned long long f[kD / 2];
};

}  // namespace

__global__ void __launch_bounds__(32 * kApWarps) decode4_append_kernel(const Append4Args a,
                                                                       const Append4Turns turns,
                                                                       uint32_t* status) {
  pdl_enter();
  __shared__ __align__(16) float cs[kD / 2], sn[kD / 2];
  __shared__ __align__(16) float z[kApWarps][kD];
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = a.lens[b];
  if (L == 0) return;                               // padding
  const bool in_range = L > 0 && L <= a.max_pages * kBlock;
  const int p = L - 1;
  const int page = in_range ? a.table[static_cast<size_t>(b) * a.max_pages + p / kBlock] : -1;
  if (page < 0 || page >= a.num_pages) {
    if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(status, kStatusBounds);
    return;
  }
  const int rows = a.Hq + 4 * a.H;
  const int r = blockIdx.y * kApWarps + warp;
  int job = 0, h = r;                               // 0 q, 1 index q, 2 k, 3 index k, 4 v
  if (r >= a.Hq) {
    job = 1 + (r - a.Hq) / a.H;
    h = (r - a.Hq) % a.H;
  }
  uint2 raw = make_uint2(0u, 0u);
  uint2 wr = raw;
  if (r < rows) {
    const int heads = job == 0 ? a.Hq : a.H;
    raw = *reinterpret_cast<const uint2*>(a.src[job] + (static_cast<size_t>(b) * heads + h) * kD +
                                          4 * lane);
    if (job < 4) wr = *reinterpret_cast<const uint2*>(a.w[job] + 4 * lane);
  }
  const int half = a.R >> 1;
  // 16 pairs per warp: lanes that index the parameters apart are served one at a time
  const int pr = 16 * warp + lane;
  if (lane < 16 && pr < half) {
    const long long ang = static_cast<long long>(static_cast<unsigned long long>(p) * turns.f[pr]);
    float s, c;
    sincospif(static_cast<float>(ang) * 1.0842021724855044e-19f, &s, &c);   // * 2^-63
    cs[pr] = c * a.rope_gain;
    sn[pr] = s * a.rope_gain;
  }
  __syncthreads();
  if (r >= rows) return;                            // whole warps
  uint32_t o[2] = {raw.x, raw.y};
  if (job < 4) {
    const float2 x0 = word_f2(raw.x), x1 = word_f2(raw.y), w0 = word_f2(wr.x), w1 = word_f2(wr.y);
    float v[4] = {x0.x, x0.y, x1.x, x1.y};
    float ss = fmaf(v[0], v[0], fmaf(v[1], v[1], fmaf(v[2], v[2], v[3] * v[3])));
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    const float rinv = rsqrtf(ss * (1.f / kD) + a.eps);
    v[0] *= rinv * (1.f + w0.x);
    v[1] *= rinv * (1.f + w0.y);
    v[2] *= rinv * (1.f + w1.x);
    v[3] *= rinv * (1.f + w1.y);
    *reinterpret_cast<float4*>(&z[warp][4 * lane]) = make_float4(v[0], v[1], v[2], v[3]);
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int ch = 4 * lane + e;
      if (ch < a.R) {
        const bool il = a.layout == MSA_ROPE_INTERLEAVED;
        const bool second = il ? (ch & 1) : ch >= half;
        const int pair = il ? ch >> 1 : (second ? ch - half : ch);
        const int other = il ? ch ^ 1 : (second ? ch - half : ch + half);
        const float t = z[warp][other] * sn[pair];
        v[e] = fmaf(v[e], cs[pair], second ? t : -t);
      }
    }
    o[0] = pack_bf16x2(v[0], v[1]);
    o[1] = pack_bf16x2(v[2], v[3]);
  }
  if (job < 2) {
    const int heads = job == 0 ? a.Hq : a.H;
    *reinterpret_cast<uint2*>(a.out[job] + (static_cast<size_t>(b) * heads + h) * kD + 4 * lane) =
        make_uint2(o[0], o[1]);
    return;
  }
  // ---- 4-bit store: largest magnitude of the block's 16 channels over 4 lanes
  const int n = job - 2;
  uint32_t m = __vmaxu2(o[0] & 0x7FFF7FFFu, o[1] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const Scale16 sc = scale16(m, a.gain[n], a.inv_gain[n]);
  uint32_t code = 0u;
  if (sc.cut != 0.f) {
    o[0] = cut_word(sc, o[0]);
    o[1] = cut_word(sc, o[1]);
  }
  if (sc.s != 0.f) code = code_word(sc, o[0]) | code_word(sc, o[1]) << 8;
  uint8_t* slab = a.cache[n] + (static_cast<size_t>(page) * a.H + h) * kSlab;
  const int slot = p % kBlock;
  *reinterpret_cast<uint16_t*>(slab + slab_code(slot) + 2 * lane) = static_cast<uint16_t>(code);
  if ((lane & 3) == 0) slab[slab_scale(slot) + (lane >> 2)] = static_cast<uint8_t>(sc.byte);
}

// ====================================================================== C ABI

// a finite power of two between 2^-64 and 2^64
bool good_gain(float g) {
  if (!(g > 0.0f) || !std::isfinite(g)) return false;
  int e = 0;
  return std::frexp(g, &e) == 0.5f && e >= -63 && e <= 65;
}

msa_status_t check_gains(float k_gain, float v_gain, float kidx_gain) {
  if (!good_gain(k_gain) || !good_gain(v_gain) || !good_gain(kidx_gain))
    return fail(MSA_ERR_INVALID_ARG, "gains must be powers of two from 2^-64 to 2^64");
  return MSA_OK;
}

msa_status_t check_cache_sizes(int Hkv, int num_pages, int max_pages) {
  if (Hkv < 1 || num_pages < 1 || max_pages < 1)
    return fail(MSA_ERR_INVALID_ARG, "Hkv, num_pages and max_pages must be >= 1");
  if (Hkv > 256) return fail(MSA_ERR_UNSUPPORTED, "at most 256 KV heads (got %d)", Hkv);
  if (max_pages > kMaxSeqlen / kBlock)
    return fail(MSA_ERR_UNSUPPORTED, "max_pages %d above the supported %d", max_pages,
                kMaxSeqlen / kBlock);
  return MSA_OK;
}

// The common part of store and load: pairs of (pack tensor, cache), each both
// given or both null.
static msa_status_t cache4_args(const void* const (&x)[3], const void* const (&cache)[3],
                                const float (&gain)[3], const int32_t* table, const int32_t* cu,
                                const int32_t* start, int S, int T, int Hkv, int num_pages,
                                int max_pages, Cache4Args* a, int (&which)[3]) {
  static const char* const names[3] = {"k", "v", "k_idx"};
  MSA_REQUIRE_PTR(table);
  MSA_REQUIRE_PTR(cu);
  if (start && !aligned16(start)) return fail(MSA_ERR_INVALID_ARG, "start is not 16-byte aligned");
  if (S < 1 || T < 1) return fail(MSA_ERR_INVALID_ARG, "S and T must be >= 1 (got %d, %d)", S, T);
  MSA_TRY(check_cache_sizes(Hkv, num_pages, max_pages));
  MSA_TRY(check_gains(gain[0], gain[1], gain[2]));
  a->n = 0;
  for (int i = 0; i < 3; ++i) {
    if (!x[i] && !cache[i]) continue;
    if (!x[i] || !cache[i])
      return fail(MSA_ERR_INVALID_ARG, "%s and its cache must be given together", names[i]);
    if (!aligned16(x[i]) || !aligned16(cache[i]))
      return fail(MSA_ERR_INVALID_ARG, "%s or its cache is not 16-byte aligned", names[i]);
    which[a->n++] = i;
  }
  if (a->n == 0) return fail(MSA_ERR_INVALID_ARG, "no tensor given");
  a->table = table;
  a->cu = cu;
  a->start = start;
  a->S = S;
  a->T = T;
  a->H = Hkv;
  a->num_pages = num_pages;
  a->max_pages = max_pages;
  return MSA_OK;
}

}  // namespace msa

using namespace msa;

extern "C" {

msa_status_t msa_cache4_store(const void* k, const void* v, const void* k_idx, void* k_cache,
                              void* v_cache, void* kidx_cache, const int32_t* block_table,
                              const int32_t* cu_seqlens, const int32_t* start, int S, int T,
                              int Hkv, int num_pages, int max_pages, float k_gain, float v_gain,
                              float kidx_gain, msa_stream_t stream) {
  const void* x[3] = {k, v, k_idx};
  const void* c[3] = {k_cache, v_cache, kidx_cache};
  const float g[3] = {k_gain, v_gain, kidx_gain};
  Cache4Args a{};
  int which[3] = {0, 0, 0};
  MSA_TRY(cache4_args(x, c, g, block_table, cu_seqlens, start, S, T, Hkv, num_pages, max_pages, &a,
                      which));
  for (int i = 0; i < a.n; ++i) {
    a.x[i] = static_cast<const __nv_bfloat16*>(x[which[i]]);
    a.cache[i] = static_cast<uint8_t*>(const_cast<void*>(c[which[i]]));
    a.gain[i] = g[which[i]];
    a.inv_gain[i] = 1.0f / g[which[i]];
  }
  uint32_t* sw = nullptr;
  MSA_TRY(status_word(&sw));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope trace_("cache4_store_kernel", st);
    launch_pdl(cache4_store_kernel, c4_grid(T, a.n, Hkv), kC4Threads, 0, st, a, sw);
  }
  return check_launch("cache4_store_kernel");
}

msa_status_t msa_cache4_load(const void* k_cache, const void* v_cache, const void* kidx_cache,
                             const int32_t* block_table, const int32_t* cu_seqlens,
                             const int32_t* start, int S, int T, int Hkv, int num_pages,
                             int max_pages, float k_gain, float v_gain, float kidx_gain, void* k,
                             void* v, void* k_idx, msa_stream_t stream) {
  const void* x[3] = {k, v, k_idx};
  const void* c[3] = {k_cache, v_cache, kidx_cache};
  const float g[3] = {k_gain, v_gain, kidx_gain};
  Cache4Args a{};
  int which[3] = {0, 0, 0};
  MSA_TRY(cache4_args(x, c, g, block_table, cu_seqlens, start, S, T, Hkv, num_pages, max_pages, &a,
                      which));
  for (int i = 0; i < a.n; ++i) {
    a.y[i] = static_cast<__nv_bfloat16*>(const_cast<void*>(x[which[i]]));
    a.rcache[i] = static_cast<const uint8_t*>(c[which[i]]);
    a.gain[i] = g[which[i]];
  }
  uint32_t* sw = nullptr;
  MSA_TRY(status_word(&sw));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope trace_("cache4_load_kernel", st);
    launch_pdl(cache4_load_kernel, c4_grid(T, a.n, Hkv), kC4Threads, 0, st, a, sw);
  }
  return check_launch("cache4_load_kernel");
}

msa_status_t msa_decode4_append(const void* q, const void* q_idx, const void* k, const void* v,
                                const void* k_idx, const void* w_q, const void* w_qi,
                                const void* w_k, const void* w_ki, void* k_cache, void* v_cache,
                                void* kidx_cache, const int32_t* block_table,
                                const int32_t* cache_lens, int B, int Hq, int Hkv, int num_pages,
                                int max_pages, const msa_rope_t* rope, float k_gain, float v_gain,
                                float kidx_gain, float eps, void* q_out, void* q_idx_out,
                                msa_stream_t stream) {
  MSA_REQUIRE_PTR(q);
  MSA_REQUIRE_PTR(q_idx);
  MSA_REQUIRE_PTR(k);
  MSA_REQUIRE_PTR(v);
  MSA_REQUIRE_PTR(k_idx);
  MSA_REQUIRE_PTR(w_q);
  MSA_REQUIRE_PTR(w_qi);
  MSA_REQUIRE_PTR(w_k);
  MSA_REQUIRE_PTR(w_ki);
  MSA_REQUIRE_PTR(k_cache);
  MSA_REQUIRE_PTR(v_cache);
  MSA_REQUIRE_PTR(kidx_cache);
  MSA_REQUIRE_PTR(block_table);
  MSA_REQUIRE_PTR(cache_lens);
  MSA_REQUIRE_PTR(q_out);
  MSA_REQUIRE_PTR(q_idx_out);
  if (B < 1) return fail(MSA_ERR_INVALID_ARG, "B must be >= 1");
  MSA_TRY(check_cache_sizes(Hkv, num_pages, max_pages));
  if (Hq < 1 || Hq % Hkv != 0)
    return fail(MSA_ERR_INVALID_ARG, "Hq (%d) must be a positive multiple of Hkv (%d)", Hq, Hkv);
  if (Hq > 256) return fail(MSA_ERR_UNSUPPORTED, "at most 256 query heads (got %d)", Hq);
  MSA_TRY(check_rope_arg(rope, kD));
  MSA_TRY(check_gains(k_gain, v_gain, kidx_gain));
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(MSA_ERR_INVALID_ARG, "eps must be >= 0");
  using bf = __nv_bfloat16;
  Append4Args a{};
  const void* src[5] = {q, q_idx, k, k_idx, v};
  const void* w[4] = {w_q, w_qi, w_k, w_ki};
  for (int i = 0; i < 5; ++i) a.src[i] = static_cast<const bf*>(src[i]);
  for (int i = 0; i < 4; ++i) a.w[i] = static_cast<const bf*>(w[i]);
  a.out[0] = static_cast<bf*>(q_out);
  a.out[1] = static_cast<bf*>(q_idx_out);
  a.cache[0] = static_cast<uint8_t*>(k_cache);
  a.cache[1] = static_cast<uint8_t*>(kidx_cache);
  a.cache[2] = static_cast<uint8_t*>(v_cache);
  const float gains[3] = {k_gain, kidx_gain, v_gain};
  for (int i = 0; i < 3; ++i) {
    a.gain[i] = gains[i];
    a.inv_gain[i] = 1.0f / gains[i];
  }
  a.table = block_table;
  a.lens = cache_lens;
  a.Hq = Hq;
  a.H = Hkv;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.R = rope->dim;
  a.layout = rope->layout;
  a.eps = eps;
  a.rope_gain = rope->gain;
  Append4Turns turns;
  for (int i = 0; i < kD / 2; ++i) turns.f[i] = i < rope->dim / 2 ? rope_turn(rope->freqs[i]) : 0;
  uint32_t* sw = nullptr;
  MSA_TRY(status_word(&sw));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope trace_("decode4_append_kernel", st);
    dim3 grid(B, (Hq + 4 * Hkv + kApWarps - 1) / kApWarps);
    launch_pdl(decode4_append_kernel, grid, 32 * kApWarps, 0, st, a, turns, sw);
  }
  return check_launch("decode4_append_kernel");
}

}  // extern "C"
