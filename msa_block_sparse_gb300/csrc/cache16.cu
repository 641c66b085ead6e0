// Appending new tokens to a 16-bit paged cache: the prologue of q and k (and of the index
// q and k), per head
//   y = R_p (x rsqrt(mean(x^2) + eps) (1 + w))      (without w: y = R_p x)
// with the rotation R_p of the token's position p, its k (and index k) and v put into the
// slot p % 128 of its page.  Several tokens per row: a prompt, a chunk of one, drafted
// tokens, or the one new token of a decode step.
//
// Bound by memory for a pack (each value read and written once): 22.5k tokens of 64 + 4 + 4 heads and
// index heads 159 us (922 MB, 5.8 TB/s); by latency for a step: 64 rows 3.5 us.
//
// Work, of two kinds of CTAs.  Those of q take a run of its [T Hq] rows, as in
// rope_ex.cu: a row of 128 channels belongs to 16 threads, which keep the factors
// (1 + w) cos and (1 + w) sin while the token stays the same.  k, v and the index heads are a
// few rows per token each: a CTA takes 8 tokens, 16 threads each, through a share of all
// these heads, tensor after tensor; the factors are formed once per tensor, and all threads
// change tensors at the same row, so that the loads (three rows are in flight) run on across
// the border.  A CTA looks its tokens' places and angles up once.
#include <cmath>
#include "rope_ex.cuh"

namespace msa {

namespace {

constexpr int kCaThreads = 128;
constexpr int kCaSlots = kCaThreads / (kD / 8);  // rows side by side
constexpr int kCaTokens = 16;                    // of a CTA at most
constexpr int kCaPerSm = 8;                      // CTAs of an SM
constexpr int kCaDeep = 4;                       // rows of a thread loaded or at work

struct CaJob {
  const __nv_bfloat16* x;       // [T, H, 128]
  const __nv_bfloat16* w;       // [128], null: no norm
  __nv_bfloat16* y;             // [T, H, 128] or (paged) [num_pages, H, 128, 128]
  int paged, turn;
};

struct CaArgs {
  CaJob q, small[4];            // small: k, v, index q, index k, each of H heads
  int Hq, H, rows;              // rows: heads of all small tensors
  int q_run, q_ctas;            // rows of q per CTA; CTAs of q, the others have small tensors,
  int shares;                   // the rows of a group of tokens in so many shares
  const int32_t *table, *cu, *lens;
  int S, T, num_pages, max_pages, R;
  float eps, gain;
  uint32_t inv_half;            // ceil(2^20 / (R / 2)), for k < 2048
  uint32_t inv_hq;              // ceil(2^20 / Hq), for i < 4096
};

struct CaSmem {
  alignas(16) float table[kCaTokens * kD];       // per token: cos, then sin, of its R / 2 pairs
  unsigned long long freq[kD / 2];
  int2 place[kCaTokens];                         // position, page (-1: the token is left alone)
};

// Places and angles of the tokens t0 .. t0 + ntok - 1
__device__ __forceinline__ void ca_tokens(const CaArgs& a, const RxTurns& turns, CaSmem& sm, int t0,
                                          int ntok, uint32_t* status) {
  const int half = a.R >> 1;
  for (int i = threadIdx.x; i < half; i += kCaThreads) sm.freq[i] = turns.f[i];
  if (static_cast<int>(threadIdx.x) < kCaTokens) {
    int pos = 0, page = -1;
    const int t = t0 + threadIdx.x;
    if (static_cast<int>(threadIdx.x) < ntok) {
      // as many tokens in every row: a first guess that one load confirms
      int s = static_cast<int>(static_cast<long long>(t) * a.S / a.T);
      int first = __ldg(a.cu + s), end = __ldg(a.cu + s + 1), L = __ldg(a.lens + s);
      if (t < first || t >= end) {
        int lo = 0, hi = a.S;                    // largest s with cu[s] <= t
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (__ldg(a.cu + mid) <= t) lo = mid; else hi = mid;
        }
        s = lo;
        first = __ldg(a.cu + s);
        end = __ldg(a.cu + s + 1);
        L = __ldg(a.lens + s);
      }
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
    }
    sm.place[threadIdx.x] = make_int2(pos, page);
  }
  __syncthreads();
  for (int k = threadIdx.x; k < ntok * half; k += kCaThreads) {
    const int tok = static_cast<int>((static_cast<uint32_t>(k) * a.inv_half) >> 20);
    const int i = k - tok * half;
    const float2 cs = rx_cos_sin(sm.place[tok].x, sm.freq[i]);
    sm.table[tok * a.R + i] = cs.x * a.gain;
    sm.table[tok * a.R + half + i] = cs.y * a.gain;
  }
  __syncthreads();
}

template <bool kHalf>
__device__ __forceinline__ void ca_weights(const __nv_bfloat16* w, const RxLane& l, float2 (&w1)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) w1[p] = make_float2(1.f, 1.f);
  if (!w) return;
  float2 wv[4];
  RxRow wr;
  wr.a = *reinterpret_cast<const uint2*>(w + l.off0);
  wr.b = *reinterpret_cast<const uint2*>(w + l.off1);
  rx_unpack<kHalf>(wr, wv);
#pragma unroll
  for (int p = 0; p < 4; ++p) w1[p] = __fadd2_rn(wv[p], w1[p]);
}

// Norm (of the 16 lanes' row) and rotation of a row; what is not turned keeps its bits
template <bool kNorm, bool kHalf>
__device__ __forceinline__ RxRow ca_row(const RxRow& raw, const float2 (&cc)[4], const float2 (&ss)[4],
                                        const RxLane& l, float eps) {
  float2 v[4];
  rx_unpack<kHalf>(raw, v);
  float2 rr = make_float2(1.f, 1.f);
  if (kNorm) {
    float2 q = __fmul2_rn(v[0], v[0]);
#pragma unroll
    for (int p = 1; p < 4; ++p) q = __ffma2_rn(v[p], v[p], q);
    float sum = q.x + q.y;
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    rr.x = rr.y = rsqrtf(sum * (1.f / kD) + eps);
  }
  rx_turn(v, cc, ss, !kNorm || l.rot);
  if (kNorm) {
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = __fmul2_rn(v[p], rr);
  }
  return kNorm || l.rot ? rx_pack<kHalf>(v) : raw;
}

// n consecutive rows of q from row r0 on, the first of token t0 and head h0
template <bool kNorm, bool kHalf>
__device__ __forceinline__ void ca_q(const CaArgs& a, const RxTurns& turns, CaSmem& sm, uint32_t* status) {
  const long long all = static_cast<long long>(a.T) * a.Hq, r0 = static_cast<long long>(blockIdx.x) * a.q_run;
  const int n = static_cast<int>(all - r0 < a.q_run ? all - r0 : a.q_run);
  const int t0 = static_cast<int>(r0 / a.Hq), h0 = static_cast<int>(r0 - static_cast<long long>(t0) * a.Hq);
  const int c = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const RxLane l = rx_lane<kHalf>(c, a.R);
  const __nv_bfloat16* xb = a.q.x + r0 * kD;
  __nv_bfloat16* yb = a.q.y + r0 * kD;
  RxRow raw[kCaDeep];
  auto fetch = [&](int i, RxRow& r) {
    r.a = r.b = make_uint2(0u, 0u);
    if (i < n) r = rx_load<kHalf>(xb + static_cast<size_t>(i) * kD, l);
  };
#pragma unroll
  for (int k = 0; k < kCaDeep - 1; ++k) fetch(k * kCaSlots + slot, raw[k]);
  float2 w1[4];
  ca_weights<kHalf>(kNorm ? a.q.w : nullptr, l, w1);
  ca_tokens(a, turns, sm, t0, (h0 + n + a.Hq - 1) / a.Hq, status);
  int have = -1;
  bool live = false;
  float2 cc[4], ss[4];
  for (int base = 0; base < n; base += kCaDeep * kCaSlots) {   // uniform: every lane reaches the shuffles
#pragma unroll
    for (int k = 0; k < kCaDeep; ++k) {
      if (base + k * kCaSlots >= n) break;
      const int i = base + k * kCaSlots + slot;
      fetch(i + (kCaDeep - 1) * kCaSlots, raw[(k + kCaDeep - 1) % kCaDeep]);
      const int tok = static_cast<int>((static_cast<uint32_t>(h0 + i) * a.inv_hq) >> 20);
      if (tok != have && i < n) {
        have = tok;
        live = sm.place[tok].y >= 0;
        rx_coefficients(sm.table + tok * a.R, a.R >> 1, l, w1, 1.f, cc, ss);
      }
      const RxRow out = ca_row<kNorm, kHalf>(raw[k], cc, ss, l, a.eps);
      if (i < n && live) rx_store<kHalf>(yb + static_cast<size_t>(i) * kD, l, out);
    }
  }
}

// The small tensors' heads r0 .. r1 - 1 of 8 tokens
template <bool kHalf>
__device__ __forceinline__ void ca_small(const CaArgs& a, const RxTurns& turns, CaSmem& sm, uint32_t* status) {
  const int cta = blockIdx.x - a.q_ctas, group = cta / a.shares, share = cta - group * a.shares;
  const int t0 = group * kCaSlots, ntok = min(kCaSlots, a.T - t0);
  const int r0 = a.rows * share / a.shares, r1 = a.rows * (share + 1) / a.shares;
  const int c = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const RxLane l = rx_lane<kHalf>(c, a.R);
  const size_t first = static_cast<size_t>(t0 + slot) * a.H;    // row of this token in any of them
  // loads
  int fr = r0, fj = r0 / a.H, fleft = a.H - (r0 - fj * a.H);
  const __nv_bfloat16* fp = a.small[fj].x + (first + a.H - fleft) * kD;
  RxRow raw[kCaDeep];
  auto fetch = [&](RxRow& r) {
    r.a = r.b = make_uint2(0u, 0u);
    if (fr >= r1) return;
    if (slot < ntok) r = rx_load<kHalf>(fp, l);
    fp += kD;
    if (--fleft == 0 && fr + 1 < r1) {
      fp = a.small[++fj].x + first * kD;
      fleft = a.H;
    }
    ++fr;
  };
#pragma unroll
  for (int k = 0; k < kCaDeep - 1; ++k) fetch(raw[k]);
  ca_tokens(a, turns, sm, t0, ntok, status);
  const int2 at = sm.place[slot];
  int r = r0, j = r0 / a.H, left = 0, ystep = kD;
  bool norm = false, turn = false;
  __nv_bfloat16* yp = nullptr;
  float2 cc[4], ss[4];
  auto enter = [&](int h) {                    // tensor j, from its head h on
    const CaJob& b = a.small[j];
    left = a.H - h;
    norm = b.w != nullptr;
    turn = b.turn != 0;
    ystep = b.paged ? kBlock * kD : kD;
    yp = b.y + (b.paged ? (static_cast<size_t>(max(at.y, 0)) * a.H + h) * kBlock + (at.x & (kBlock - 1))
                        : first + h) * kD;
    float2 w1[4];
    ca_weights<kHalf>(b.w, l, w1);
    rx_coefficients(sm.table + slot * a.R, a.R >> 1, l, w1, 1.f, cc, ss);
  };
  enter(r0 - j * a.H);
  while (r < r1) {                             // uniform over the CTA
#pragma unroll
    for (int k = 0; k < kCaDeep; ++k) {
      if (r >= r1) break;
      fetch(raw[(k + kCaDeep - 1) % kCaDeep]);
      RxRow out = raw[k];
      if (turn) out = norm ? ca_row<true, kHalf>(raw[k], cc, ss, l, a.eps) : ca_row<false, kHalf>(raw[k], cc, ss, l, a.eps);
      if (at.y >= 0) rx_store<kHalf>(yp, l, out);
      yp += ystep;
      if (++r < r1 && --left == 0) {
        ++j;
        enter(0);
      }
    }
  }
}

}  // namespace

template <bool kHalf>
__global__ void __launch_bounds__(kCaThreads, kCaPerSm) cache_append_kernel(const __grid_constant__ CaArgs a,
                                                                     const __grid_constant__ RxTurns turns,
                                                                     uint32_t* status) {
  pdl_enter();
  __shared__ CaSmem sm;
  if (static_cast<int>(blockIdx.x) >= a.q_ctas) ca_small<kHalf>(a, turns, sm, status);
  else if (a.q.w) ca_q<true, kHalf>(a, turns, sm, status);
  else ca_q<false, kHalf>(a, turns, sm, status);
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
  a.rows = 2 * Hkv;
  if (index) {
    a.small[2] = job(q_idx, w_qi, q_idx_out, false, true);
    a.small[3] = job(k_idx, w_ki, kidx_cache, true, true);
    a.rows = 4 * Hkv;
  }
  a.Hq = Hq;
  a.H = Hkv;
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
  a.inv_hq = ((1u << 20) + Hq - 1) / Hq;
  // q: 64 rows per CTA, fewer (a pass of rows at least) when that would leave SMs without one; more,
  // up to 256, as long as that leaves 4 rounds of CTAs (places and angles are looked up once per CTA:
  // 22.5k tokens of 64 heads 168 us with 64 rows, 163 with 128, 160 with 256 or 512); at most 16 tokens.
  // The others: shares of a token's heads while there are SMs for them.
  const int sms = device_sm_count();
  const long long q_rows = static_cast<long long>(T) * Hq;
  long long run = q_rows / (2 * sms);
  run = run < kCaSlots ? kCaSlots : (run > 64 ? 64 : run);
  const long long rounds = q_rows / (4 * kCaPerSm * sms);
  if (rounds > run) run = rounds > 256 ? 256 : rounds;
  if (run > static_cast<long long>(kCaTokens - 1) * Hq) run = static_cast<long long>(kCaTokens - 1) * Hq;
  a.q_run = static_cast<int>(run > Hq ? run / Hq * Hq : run);
  const long long q_ctas = (q_rows + a.q_run - 1) / a.q_run;
  const int groups = (T - 1) / kCaSlots + 1, fill = 4 * sms / groups;
  a.shares = fill < 1 ? 1 : (fill < a.rows ? fill : a.rows);
  const long long ctas = q_ctas + static_cast<long long>(groups) * a.shares;
  if (ctas > INT32_MAX) return fail(MSA_ERR_UNSUPPORTED, "T = %d tokens of %d heads are too many", T, Hq);
  a.q_ctas = static_cast<int>(q_ctas);
  // a row is read and written by the same threads, in place where the rows are the same; elsewhere other
  // CTAs have yet to read
  const size_t qb = static_cast<size_t>(T) * Hq * kD * sizeof(bf), kb = static_cast<size_t>(T) * Hkv * kD * sizeof(bf);
  const struct {
    const void* at;
    size_t bytes;
    const char* name;
  } out[2] = {{q_out, qb, "q_out"}, {q_idx_out, kb, "q_idx_out"}},
    in[5] = {{q, qb, "q"}, {k, kb, "k"}, {v, kb, "v"}, {q_idx, kb, "q_idx"}, {k_idx, kb, "k_idx"}};
  for (int i = 0; i < (index ? 2 : 1); ++i)
    for (int j = 0; j < (index ? 5 : 3); ++j)
      if (overlap(out[i].at, out[i].bytes, in[j].at, in[j].bytes) && !(j == 3 * i && out[i].at == in[j].at))
        return fail(MSA_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, in[j].name);
  if (index && overlap(q_out, qb, q_idx_out, kb)) return fail(MSA_ERR_INVALID_ARG, "q_out overlaps q_idx_out");
  const RxTurns turns = rx_turns(*rope);
  uint32_t* sw = nullptr;
  MSA_TRY(status_word(&sw));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope trace_("cache_append_kernel", st);
    launch_pdl(rope->layout == MSA_ROPE_HALF ? cache_append_kernel<true> : cache_append_kernel<false>,
               static_cast<unsigned>(ctas), kCaThreads, 0, st, a, turns, sw);
  }
  return check_launch("cache_append_kernel");
}

}  // extern "C"
