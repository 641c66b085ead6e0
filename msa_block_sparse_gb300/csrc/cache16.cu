// Appending new tokens to a 16-bit paged cache: the prologue of q and k (and of the index
// q and k), per head
//   y = R_p (x rsqrt(mean(x^2) + eps) (1 + w))      (without w: y = R_p x)
// with the rotation R_p of the token's position p, its k (and index k) and v put into the
// slot p % 128 of its page.  Several tokens per row: a prompt, a chunk of one, drafted
// tokens, or the one new token of a decode step.
//
// Bound by memory for a pack (each value read and written once), by latency for a step.
//
// Work: a CTA takes a run of tokens and either heads of q or heads of the smaller tensors
// (k, v, index q, index k: taken as one tensor of all their heads, since each by itself is a few
// rows per token).  It looks up the tokens' places and the angles once; a row of 128
// channels then belongs to 16 threads (rope_ex.cuh), three rows' loads in flight.
#include <cmath>
#include "rope_ex.cuh"

namespace msa {

namespace {

constexpr int kCaThreads = 128;
constexpr int kCaMaxTokens = 16;                 // of a CTA
constexpr int kCaSlots = kCaThreads / (kD / 8);  // rows side by side

struct CaJob {
  const __nv_bfloat16* x;       // [T, H, 128]
  const __nv_bfloat16* w;       // [128], null: no norm
  __nv_bfloat16* y;             // [T, H, 128] or (paged) [num_pages, H, 128, 128]
  int paged, turn;
};

struct CaArgs {
  CaJob q, small[4];            // small: k, v, index q, index k, each of Hkv heads
  int Hq, Hkv, smalls;
  const int32_t *table, *cu, *lens;
  int S, T, num_pages, max_pages, R, run;
  int q_shares;                 // blockIdx.y below: heads of q, the others: of the small ones
  float eps, gain;
  uint32_t inv_half;            // ceil(2^20 / (R / 2)), for k < 2048
};

struct CaSmem {
  alignas(16) float table[kCaMaxTokens * kD];
  alignas(16) float w1[4][kD];  // 1 + w of the small tensors
  unsigned long long freq[kD / 2];
  int pos[kCaMaxTokens];
  int page[kCaMaxTokens];       // -1: the token is left alone
};

// Rows (token, head h0 .. h0 + nh - 1); heads run fastest.  kQ: heads of q, whose factors
// (1 + w) cos and (1 + w) sin stay in registers while the token stays the same.  Otherwise
// head h is head h % Hkv of small tensor h / Hkv.  kNorm: the tensor (one of them) has weights.
template <bool kQ, bool kNorm, bool kHalf>
__device__ __forceinline__ void ca_rows(const CaArgs& a, const CaSmem& sm, int t0, int ntok, int h0,
                                        int nh) {
  const int c = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const RxLane l = rx_lane<kHalf>(c, a.R);
  const int n = ntok * nh;
  float2 w1[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) w1[p] = make_float2(1.f, 1.f);
  if (kQ && kNorm) {
    float2 wv[4];
    RxRow wr;
    wr.a = *reinterpret_cast<const uint2*>(a.q.w + l.off0);
    wr.b = *reinterpret_cast<const uint2*>(a.q.w + l.off1);
    rx_unpack<kHalf>(wr, wv);
#pragma unroll
    for (int p = 0; p < 4; ++p) w1[p] = __fadd2_rn(wv[p], w1[p]);
  }
  constexpr int kDeep = 4;
  RxRow raw[kDeep];
  // row i = (token f_tok, head h0 + f_h); both counters go up by kCaSlots rows at a time
  int f_tok = slot / nh, f_h = slot - f_tok * nh, c_tok = f_tok, c_h = f_h;
  const int d_tok = kCaSlots / nh, d_h = kCaSlots - d_tok * nh;
  auto step = [&](int& tok, int& h) {
    tok += d_tok;
    h += d_h;
    if (h >= nh) {
      h -= nh;
      ++tok;
    }
  };
  auto fetch = [&](RxRow& r) {
    r.a = r.b = make_uint2(0u, 0u);
    if (f_tok < ntok) {
      const __nv_bfloat16* x = a.q.x;
      int H = a.Hq, h = h0 + f_h;
      if (!kQ) {
        H = a.Hkv;
        const int j = h / H;
        h -= j * H;
        x = a.small[j].x;
      }
      r = rx_load<kHalf>(x + (static_cast<size_t>(t0 + f_tok) * H + h) * kD, l);
    }
    step(f_tok, f_h);
  };
#pragma unroll
  for (int k = 0; k < kDeep - 1; ++k) fetch(raw[k]);
  int have = -1;
  float2 cc[4], ss[4];
  for (int base = 0; base < n; base += kDeep * kCaSlots) {   // uniform: every lane reaches the shuffles
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      if (base + k * kCaSlots >= n) break;
      fetch(raw[(k + kDeep - 1) % kDeep]);
      float2 v[4];
      rx_unpack<kHalf>(raw[k], v);
      float2 rr = make_float2(1.f, 1.f);
      if (kNorm) {
        float2 q = __fmul2_rn(v[0], v[0]);
#pragma unroll
        for (int p = 1; p < 4; ++p) q = __ffma2_rn(v[p], v[p], q);
        float sum = q.x + q.y;
#pragma unroll
        for (int m = 8; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        rr.x = rr.y = rsqrtf(sum * (1.f / kD) + a.eps);
      }
      const int tok = c_tok;
      int h = h0 + c_h;
      step(c_tok, c_h);
      if (tok >= ntok || sm.page[tok] < 0) continue;
      __nv_bfloat16* row;
      RxRow out = raw[k];                                    // what is not turned keeps its bits
      if (kQ) {
        if (tok != have) {
          have = tok;
          rx_coefficients(sm.table + tok * a.R, a.R >> 1, l, w1, 1.f, cc, ss);
        }
        rx_turn(v, cc, ss, !kNorm || l.rot);
        if (kNorm) {
#pragma unroll
          for (int p = 0; p < 4; ++p) v[p] = __fmul2_rn(v[p], rr);
        }
        if (kNorm || l.rot) out = rx_pack<kHalf>(v);
        row = a.q.y + (static_cast<size_t>(t0 + tok) * a.Hq + h) * kD;
      } else {
        const int j = h / a.Hkv;
        h -= j * a.Hkv;
        const CaJob& job = a.small[j];
        if (job.turn) {
          const bool norm = kNorm && job.w;
          if (norm) {
            const float4 x = *reinterpret_cast<const float4*>(&sm.w1[j][l.off0]);
            const float4 y = *reinterpret_cast<const float4*>(&sm.w1[j][l.off1]);
            if (kHalf) {
              w1[0] = make_float2(x.x, x.y);
              w1[1] = make_float2(x.z, x.w);
              w1[2] = make_float2(y.x, y.y);
              w1[3] = make_float2(y.z, y.w);
            } else {
              w1[0] = make_float2(x.x, x.z);
              w1[1] = make_float2(y.x, y.z);
              w1[2] = make_float2(x.y, x.w);
              w1[3] = make_float2(y.y, y.w);
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) w1[p] = __fmul2_rn(w1[p], rr);
          } else {
#pragma unroll
            for (int p = 0; p < 4; ++p) w1[p] = make_float2(1.f, 1.f);
          }
          rx_coefficients(sm.table + tok * a.R, a.R >> 1, l, w1, 1.f, cc, ss);
          rx_turn(v, cc, ss, !norm || l.rot);
          if (norm || l.rot) out = rx_pack<kHalf>(v);
        }
        row = job.paged ? job.y + ((static_cast<size_t>(sm.page[tok]) * a.Hkv + h) * kBlock +
                                   (sm.pos[tok] & (kBlock - 1))) * kD
                        : job.y + (static_cast<size_t>(t0 + tok) * a.Hkv + h) * kD;
      }
      rx_store<kHalf>(row, l, out);
    }
  }
}

}  // namespace

// grid (runs of tokens, shares of q's heads and of the small tensors' heads)
template <bool kHalf>
__global__ void __launch_bounds__(kCaThreads, 6) cache_append_kernel(const __grid_constant__ CaArgs a,
                                                                     const __grid_constant__ RxTurns turns,
                                                                     uint32_t* status) {
  pdl_enter();
  __shared__ CaSmem sm;
  const int t0 = blockIdx.x * a.run, ntok = min(a.run, a.T - t0);
  const int half = a.R >> 1;
  const bool of_q = static_cast<int>(blockIdx.y) < a.q_shares;
  for (int i = threadIdx.x; i < half; i += kCaThreads) sm.freq[i] = turns.f[i];
  if (static_cast<int>(threadIdx.x) < ntok) {
    const int t = t0 + threadIdx.x;
    // as many tokens in every row: a first guess that one load confirms
    int s = static_cast<int>(static_cast<long long>(t) * a.S / a.T);
    int first = __ldg(a.cu + s), end = __ldg(a.cu + s + 1), L = __ldg(a.lens + s);
    if (t < first || t >= end) {
      int lo = 0, hi = a.S;                // largest s with cu[s] <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu + mid) <= t) lo = mid; else hi = mid;
      }
      s = lo;
      first = __ldg(a.cu + s);
      end = __ldg(a.cu + s + 1);
      L = __ldg(a.lens + s);
    }
    int pos = 0, page = -1;
    if (t >= first && t < end && L != 0) {     // length 0: padding
      const long long p = static_cast<long long>(L) - end + t;
      if (p >= 0 && p < static_cast<long long>(a.max_pages) * kBlock) {
        pos = static_cast<int>(p);
        page = __ldg(a.table + static_cast<size_t>(s) * a.max_pages + pos / kBlock);
      }
      if (page < 0 || page >= a.num_pages) {
        page = -1;
        atomicOr(status, kStatusBounds);
      }
    }
    sm.pos[threadIdx.x] = pos;
    sm.page[threadIdx.x] = page;
  }
  bool normed = false;                         // one of the small tensors is
  if (!of_q) {
    for (int j = 0; j < a.smalls; ++j) {
      if (!a.small[j].w) continue;
      normed = true;
      sm.w1[j][threadIdx.x] = 1.f + __bfloat162float(a.small[j].w[threadIdx.x]);
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < ntok * half; k += kCaThreads) {
    const int tok = static_cast<int>((static_cast<uint32_t>(k) * a.inv_half) >> 20);
    const int i = k - tok * half;
    const float2 cs = rx_cos_sin(sm.pos[tok], sm.freq[i]);
    sm.table[tok * a.R + i] = cs.x * a.gain;
    sm.table[tok * a.R + half + i] = cs.y * a.gain;
  }
  __syncthreads();
  const int heads = of_q ? a.Hq : a.smalls * a.Hkv;
  const int y = of_q ? blockIdx.y : blockIdx.y - a.q_shares;
  const int ny = of_q ? a.q_shares : gridDim.y - a.q_shares;
  const int h0 = heads * y / ny, nh = heads * (y + 1) / ny - h0;
  if (of_q) {
    if (a.q.w) ca_rows<true, true, kHalf>(a, sm, t0, ntok, h0, nh);
    else ca_rows<true, false, kHalf>(a, sm, t0, ntok, h0, nh);
  } else {
    if (normed) ca_rows<false, true, kHalf>(a, sm, t0, ntok, h0, nh);
    else ca_rows<false, false, kHalf>(a, sm, t0, ntok, h0, nh);
  }
}

}  // namespace msa

using namespace msa;

extern "C" {

msa_status_t msa_cache_append(const void* q, const void* k, const void* v, const void* q_idx,
                              const void* k_idx, const void* w_q, const void* w_k,
                              const void* w_qi, const void* w_ki, void* k_cache, void* v_cache,
                              void* kidx_cache, const int32_t* block_table,
                              const int32_t* cu_seqlens, const int32_t* cache_lens, int S, int T,
                              int Hq, int Hkv, int num_pages, int max_pages,
                              const msa_rope_t* rope, float eps, void* q_out, void* q_idx_out,
                              msa_stream_t stream) {
  MSA_REQUIRE_PTR(q);
  MSA_REQUIRE_PTR(k);
  MSA_REQUIRE_PTR(v);
  MSA_REQUIRE_PTR(k_cache);
  MSA_REQUIRE_PTR(v_cache);
  MSA_REQUIRE_PTR(q_out);
  MSA_REQUIRE_PTR(block_table);
  MSA_REQUIRE_PTR(cu_seqlens);
  MSA_REQUIRE_PTR(cache_lens);
  const bool index = q_idx || k_idx || kidx_cache || q_idx_out;
  if (index) {
    if (!q_idx || !k_idx || !kidx_cache || !q_idx_out)
      return fail(MSA_ERR_INVALID_ARG, "q_idx, k_idx, kidx_cache and q_idx_out must be given together");
    MSA_REQUIRE_PTR(q_idx);
    MSA_REQUIRE_PTR(k_idx);
    MSA_REQUIRE_PTR(kidx_cache);
    MSA_REQUIRE_PTR(q_idx_out);
  } else if (w_qi || w_ki) {
    return fail(MSA_ERR_INVALID_ARG, "w_qi and w_ki need q_idx and k_idx");
  }
  const void* w[4] = {w_q, w_k, w_qi, w_ki};
  for (int i = 0; i < 4; ++i)
    if (w[i] && !aligned16(w[i])) return fail(MSA_ERR_INVALID_ARG, "a weight is not 16-byte aligned");
  if (S < 1 || T < 1) return fail(MSA_ERR_INVALID_ARG, "S and T must be >= 1 (got %d, %d)", S, T);
  MSA_TRY(check_cache_sizes(Hkv, num_pages, max_pages));
  if (Hq < 1 || Hq % Hkv != 0)
    return fail(MSA_ERR_INVALID_ARG, "Hq (%d) must be a positive multiple of Hkv (%d)", Hq, Hkv);
  if (Hq > 256) return fail(MSA_ERR_UNSUPPORTED, "at most 256 query heads (got %d)", Hq);
  MSA_TRY(check_rope_arg(rope, kD));
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(MSA_ERR_INVALID_ARG, "eps must be >= 0");
  using bf = __nv_bfloat16;
  CaArgs a{};
  auto job = [](const void* x, const void* wx, void* y, bool paged, bool turn) {
    return CaJob{static_cast<const bf*>(x), static_cast<const bf*>(wx), static_cast<bf*>(y), paged, turn};
  };
  a.q = job(q, w_q, q_out, false, true);
  a.small[0] = job(k, w_k, k_cache, true, true);
  a.small[1] = job(v, nullptr, v_cache, true, false);
  a.smalls = 2;
  if (index) {
    a.small[2] = job(q_idx, w_qi, q_idx_out, false, true);
    a.small[3] = job(k_idx, w_ki, kidx_cache, true, true);
    a.smalls = 4;
  }
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.table = block_table;
  a.cu = cu_seqlens;
  a.lens = cache_lens;
  a.S = S;
  a.T = T;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.R = rope->dim;
  a.eps = eps;
  a.gain = rope->gain;
  a.inv_half = ((1u << 20) + rope->dim / 2 - 1) / (rope->dim / 2);
  // Tokens per CTA: about 256 rows of q (shorter runs repeat the places' and angles' work),
  // but enough CTAs for the GPU; heads are split when there are few tokens.
  const int small = a.smalls * Hkv, fill = 8 * device_sm_count();
  int run = 256 / Hq;
  if (run > T / fill) run = T / fill;
  a.run = run < 1 ? 1 : (run > kCaMaxTokens ? kCaMaxTokens : run);
  const int runs = (T + a.run - 1) / a.run;
  auto shares = [&](int heads) {               // no CTA with less than a pass of rows
    const int want = fill / runs, most = (heads * a.run + kCaSlots - 1) / kCaSlots;
    const int n = want < most ? want : most;
    return n < 1 ? 1 : n > heads ? heads : n;
  };
  a.q_shares = shares(Hq);
  const int y_ctas = a.q_shares + shares(small);
  const RxTurns turns = rx_turns(*rope);
  uint32_t* sw = nullptr;
  MSA_TRY(status_word(&sw));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope trace_("cache_append_kernel", st);
    launch_pdl(rope->layout == MSA_ROPE_HALF ? cache_append_kernel<true> : cache_append_kernel<false>,
               dim3(runs, y_ctas), kCaThreads, 0, st, a, turns, sw);
  }
  return check_launch("cache_append_kernel");
}

}  // extern "C"
