// Full attention of one new token per row over the 16-bit paged cache, with pages that
// neighbouring rows share read once for all of them.
//   o = softmax(scale q K^T) V,   lse = log sum exp(scale q K^T)
//
// Sharing.  With c_i the number of leading full pages that the rows i and i + 1 (of those
// with tokens) have in common, the rows that share a page at column c are the maximal
// runs with c_i > c: the runs form a tree, whose nodes are rectangles (rows i0 .. i0 + m - 1,
// columns v0 .. v1 - 1).  A row's keys are those of the nodes on its path and of its own
// leaf (one row, the columns behind).  Every node is cut into items (up to 256 query rows x a
// range of columns x a KV head) of about equal work; an item leaves a partial result
// (maximum, sum, unnormalised o in fp32) per query row, and the parts of a row are joined.
//
//   shared_plan_kernel     one CTA: c_i, tree, item length, items, each row's list of parts
//   shared_attn_kernel     persistent CTAs (one per SM) that claim items
//   shared_combine_kernel  joins the parts
//
// Attention of an item: tiles of 128 query rows (token rows x the G heads of a KV head),
// two streams of tensor-core work per CTA:
//   wide    two tiles over the same pages; stream s has tile s and all keys
//   narrow  one tile (a leaf's G rows, or up to 128 shared ones); stream s has the keys
//           64 s .. 64 s + 63 of every page; the halves' results are merged at the end
// so that a page in shared memory serves up to 256 query rows and either stream's softmax
// runs while the other's products do.  A stream takes 64 keys at a time, S (128 x 64) in two
// buffers, so that the next block's products are there when a softmax ends.  Roles: warp 0 claims items and streams K and V pages
// through a ring of 32 KB stages by TMA; warps 1 and 2 issue a stream's MMAs (P, in bf16, is
// read from TMEM as the A operand); warp 3 gathers q; warps 4-7 and 8-11 are the streams'
// softmax (a thread per query row).  P is rounded to bf16 (at most 2^-8 each, beside o's own
// rounding); maxima, sums and o stay in fp32.
//
// Bound by memory where little is shared: 64 rows of 8k to 32k tokens, 64 heads on 4, 380 us (2.5
// GB, 6.6 TB/s).  Prefixes of 8k to 32k shared by 8 rows each: 94 us (443 MB).  One of 16k shared
// by 64 rows with up to 4k of their own: 94 us (348 MB, 40 GFLOP), the plan about 9 of them.  4
// rows of 1,500 tokens: 15.4 us, latency (short_attn.cu takes such calls where the tables are small: 5.8).
#include <cfloat>
#include <cmath>
#include "kernels.cuh"

namespace msa {

namespace {

constexpr int kSaMaxRows = 2048;           // rows of a call
constexpr int kSaLevels = 6;               // levels of sharing above a leaf
constexpr int kSaMaxSegs = kSaLevels + 1;
constexpr int kSaThreads = 384;
constexpr int kSaStages = 5;
constexpr int kSaTile = 128 * 128 * 2;     // bytes of a 128 x 128 bf16 tile
constexpr int kSaHalf = kSaTile / 2;       // one 64-channel half
constexpr int kSaQWarp = 3;
constexpr uint32_t kSaIdescS = idesc_bf16(128, 64, false, false);        // S = Q K^T, 64 keys
constexpr uint32_t kSaIdescPV = idesc_bf16(128, 128, false, true);       // O += P V
constexpr float kSaLog2e = 1.4426950408889634f;
constexpr float kSaRescale = 8.0f;         // log2 of the largest P before o is rescaled (P < 256 fits bf16)
constexpr uint32_t kSaColO = 256;          // S of stream s at 128 s, O at 256 + 128 s

// Work of a CTA: rows i0 .. i0 + nr - 1 (of the live ones), columns c0 .. c1 - 1, KV head
// g.  Its parts are query rows ro * G .. of a block of m * G whose first is `base`.
struct alignas(16) SaItem {
  int i0, nr, c0, c1;
  int g, m, ro, base;
  int row, len;           // the first of the rows, and its tokens
  int side, pad;          // the rows are row, row + 1, ...: none between them is empty
};

// Parts of a row in one node: splits of (m G) query rows each, `ro` the row in the node
struct SaSeg {
  int base, m, ro, splits;
};

struct SaPlan {
  int* live;          // [B] rows with tokens, in order
  SaItem* items;
  int* counts;        // [0] items, [1] next to claim (behind the CTAs' first ones)
  SaSeg* segs;        // [B][kSaMaxSegs]
  int* n_segs;        // [B], 0 for rows without tokens
  float4* part_o;     // [blocks][32][m G]
  float2* part_ml;    // (reference for the exponentials among the products q k, sum)
  int max_items, max_parts;
};

__device__ __forceinline__ float sa_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes global -> shared, asynchronously
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void umma_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

}  // namespace

// ---------------------------------------------------------------- plan

namespace {

constexpr int kPlThreads = 1024;           // fewer for few rows, whose barriers then cost less
constexpr int kPlLengths = 32;
constexpr int kPlRowInts = 9, kPlNodeInts = 8;    // of the dynamic shared memory, per row and node
// Candidate item lengths in pages: of runs, and of rows alone, which are cut shorter (their
// items fill what the runs leave, and their parts are small).  The last ones always fit the
// workspace: one item per node and tile.
constexpr int kPlCuts = kPlLengths / 2;
constexpr int kPlAlones = 10;
__constant__ int kPlCut[kPlCuts] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128, 256, 1024};
__constant__ int kPlAlone[kPlAlones] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 1024};
// Candidate c: its runs' length is c / 2, its rows' is as long, but at most 8 or 24
__device__ __forceinline__ int pl_alone(int c) {
  return c >> 1 == kPlCuts - 1 ? kPlAlones - 1 : min(c >> 1, c & 1 ? 5 : 8);
}
__device__ __forceinline__ int2 pl_length(int c) { return make_int2(kPlCut[c >> 1], kPlAlone[pl_alone(c)]); }

// What runs, or rows alone, come to in items of a length
struct PlWeight {
  float sum, slowest, long_sum, memory;    // times of all items, the longest, the runs' long ones; of the memory
  int items, long_items;
  uint32_t parts;
};
// Times in us, from traces and from runs over item lengths: a page in a narrow and a wide item,
// an item's start and end as far as no page passes; of the whole GPU: a query row's part
// (written, joined), 64 KB of K and V from memory
constexpr float kPlNarrow = 1.07f, kPlWide = 1.7f;
constexpr float kPlStart = 2.2f, kPlWideStart = 4.5f;
constexpr float kPlPart = 0.00022f;
constexpr float kPlMemory = 0.0099f;
constexpr float kPlTail = 0.12f;         // of a row's longest item: what others wait for at the end
constexpr int kPlLong = 8;               // rows alone with as many pages come before the others

// Exclusive scans over the CTA's first `count` threads (the others' values are 0) of two values at
// a time; total = the sums.  Warps without a value only add up.  One barrier: a buffer is used
// again two scans later.
struct PlScan {
  int2 (*warp_sums)[kPlThreads / 32];
  int turn = 0;

  __device__ __forceinline__ int2 operator()(int2 v, int count, int2* total) {
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const bool busy = wp * 32 < count;
    int2* sums = warp_sums[turn];
    turn ^= 1;
    int2 x = v;
    if (busy) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, x.x, d), b = __shfl_up_sync(0xffffffffu, x.y, d);
        if (lane >= d) {
          x.x += a;
          x.y += b;
        }
      }
      if (lane == 31) sums[wp] = x;
    }
    __syncthreads();
    const int2 own = lane * 32 < count ? sums[lane] : make_int2(0, 0);
    *total = make_int2(__reduce_add_sync(0xffffffffu, own.x), __reduce_add_sync(0xffffffffu, own.y));
    if (busy) {
      x.x += __reduce_add_sync(0xffffffffu, lane < wp ? own.x : 0) - v.x;
      x.y += __reduce_add_sync(0xffffffffu, lane < wp ? own.y : 0) - v.y;
    }
    return x;
  }
};

// ceil(pages / L) with 1 / L, good to 2 units, at hand: (x + 1/2) / L stays 1 / (2 L) away from whole
// numbers, the product's error (x <= 2047: 2047 / L 2^-21) does not reach that far
__device__ __forceinline__ int pl_splits(int pages, int L, float inv) {
  return static_cast<int>((static_cast<float>(pages + L - 1) + 0.5f) * inv);
}

}  // namespace

// Runs of rows that share: boundary i, between the live rows i and i + 1, stands for the run
// of which it is the first boundary with the run's least value c_i (the run's rows share the
// columns below c_i, and only a part of the run's rows any behind).
__global__ void __launch_bounds__(kPlThreads) shared_plan_kernel(
    const int32_t* __restrict__ table, const int32_t* __restrict__ lens, int B, int G, int Hkv,
    int max_pages, int sms, SaPlan plan, uint32_t* status) {
  pdl_enter();
  extern __shared__ int smem_i[];
  __shared__ int2 warp_sums[2][kPlThreads / 32];
  __shared__ int longest_run, short_items, chosen;
  __shared__ PlWeight weight[kPlCuts + kPlAlones];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int threads = blockDim.x, warps = threads / 32;
  PlScan scan{warp_sums};
  int* row_of = smem_i;                    // live rows
  int* len_of = row_of + B;                // their lengths
  int* common = len_of + B;                // c_i
  int* rep = common + B;                   // first boundary of the run
  int* parent = rep + B;                   // boundary of the run above, -1: none
  int* first = parent + B;                 // first live row of the run
  int* rows = first + B;                   // its live rows; 0: the boundary stands for no run
  int* leaf_up = rows + B;                 // boundary of the run above a row alone, -1: none
  int* depth = leaf_up + B;
  int* nd_of = depth + B;                  // [2 B] node of boundary i, of live row i; -1: none
  int* nd_v0 = nd_of + 2 * B;              // nodes: first column,
  int* nd_pages = nd_v0 + 2 * B;           // columns,
  int* nd_i0 = nd_pages + 2 * B;           // first live row,
  int* nd_m = nd_i0 + 2 * B;               // rows,
  int* nd_tiles = nd_m + 2 * B;            // tiles of up to 256 query rows,
  int* nd_item = nd_tiles + 2 * B;         // first item
  int* nd_part = nd_item + 2 * B;          // and first part

  // Two units of what is compared below, asked for before the lengths are known: as if every row
  // had tokens
  struct Unit {
    int i, j0, most, x[8], y[8];
  };
  const int chunks = (max_pages + 255) / 256;
  auto place = [&](Unit& t, int u, int pairs) {
    const int chunk = chunks == 1 || pairs < 1 ? 0 : u / pairs;   // the first columns of all pairs first
    t.i = u - chunk * pairs;
    t.j0 = chunk * 256;
  };
  auto load = [&](Unit& t, int ra, int rb, int end) {
    const int32_t* a = table + static_cast<size_t>(ra) * max_pages;
    const int32_t* b = table + static_cast<size_t>(rb) * max_pages;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int j = t.j0 + 32 * k + lane;
      t.x[k] = j < end ? __ldg(a + j) : 0;
      t.y[k] = j < end ? __ldg(b + j) : 0;
    }
  };
  Unit p, q;
  place(p, warp, B - 1);
  place(q, warp + warps, B - 1);
  if (warp < (B - 1) * chunks) load(p, p.i, p.i + 1, max_pages);
  if (warp + warps < (B - 1) * chunks) load(q, q.i, q.i + 1, max_pages);
  // ---- rows with tokens
  int n = 0;
  for (int b0 = 0; b0 < B; b0 += threads) {
    const int b = b0 + tid;
    int L = 0;
    if (b < B) {
      L = lens[b];
      if (L < 0 || L > max_pages * kBlock) {
        atomicOr(status, kStatusBounds);
        L = 0;
      }
      if (L == 0) plan.n_segs[b] = 0;
    }
    int2 total;
    const int at = n + scan(make_int2(L > 0, 0), min(B - b0, threads), &total).x;
    if (L > 0) {
      row_of[at] = b;
      len_of[at] = L;
      plan.live[at] = b;
    }
    n += total.x;
  }
  if (tid == 0) longest_run = short_items = 0;
  __syncthreads();
  for (int i = tid; i < n; i += threads)
    common[i] = i + 1 < n ? min(len_of[i], len_of[i + 1]) / kBlock : 0;
  __syncthreads();
  // ---- full pages that neighbours have in common: a warp per pair and 256 columns, which
  // lowers the value to the first column that differs
  {
    const int units = (n - 1) * chunks;
    auto need = [&](Unit& t, int u) {
      t.most = u < units ? min(len_of[t.i], len_of[t.i + 1]) / kBlock : 0;
      return t.j0 < t.most;
    };
    auto look = [&](const Unit& t) {
      if (t.j0 >= t.most) return;
      int at = -1;
#pragma unroll
      for (int k = 7; k >= 0; --k) {
        const uint32_t differ =
            __ballot_sync(0xffffffffu, t.x[k] != t.y[k] && t.j0 + 32 * k + lane < t.most);
        if (differ) at = t.j0 + 32 * k + __ffs(differ) - 1;
      }
      if (at >= 0 && lane == 0) atomicMin(&common[t.i], at);
    };
    for (int u = warp; u < units; u += 2 * warps) {   // two units' loads in flight
      if (u != warp || n != B) {
        place(p, u, n - 1);
        place(q, u + warps, n - 1);
        if (need(p, u)) load(p, row_of[p.i], row_of[p.i + 1], p.most);
        if (need(q, u + warps)) load(q, row_of[q.i], row_of[q.i + 1], q.most);
      } else {
        need(p, u);
        need(q, u + warps);
      }
      look(p);
      look(q);
    }
  }
  __syncthreads();
  // ---- runs, a warp per boundary: the nearest boundaries with less on both sides; the
  // higher of the two values is where the run above ends
  for (int i = warp; i < n; i += warps) {
    const int v = common[i];               // the last row's is 0
    int l = -1, r = n - 1, rp = i, up = -1;
    if (v > 0) {
      for (int j0 = i - 1; j0 >= 0; j0 -= 32) {
        const int c = j0 - lane >= 0 ? common[j0 - lane] : -1;
        const uint32_t less = __ballot_sync(0xffffffffu, c < v);
        const uint32_t run = less ? (less & (0u - less)) - 1u : 0xffffffffu;   // lanes before the first
        const uint32_t same = __ballot_sync(0xffffffffu, c == v) & run;
        if (same) rp = j0 - (31 - __clz(same));
        if (less) {
          l = j0 - (__ffs(less) - 1);
          break;
        }
      }
      for (int j0 = i + 1; j0 < n - 1; j0 += 32) {
        const int c = j0 + lane < n - 1 ? common[j0 + lane] : -1;
        const uint32_t less = __ballot_sync(0xffffffffu, c < v);
        if (less) {
          r = min(j0 + __ffs(less) - 1, n - 1);
          break;
        }
      }
      l = max(l, -1);
      const int lv = l >= 0 ? common[l] : 0, rv = r < n - 1 ? common[r] : 0;
      if (lv > 0 || rv > 0) up = lv >= rv ? l : r;
    }
    if (lane == 0) {
      rep[i] = rp;
      parent[i] = up;
      first[i] = l + 1;
      rows[i] = v > 0 && rp == i ? r - l : 0;
    }
  }
  __syncthreads();
  for (int i = tid; i < n; i += threads) {
    const int lv = i > 0 ? common[i - 1] : 0, rv = common[i];
    leaf_up[i] = lv > 0 || rv > 0 ? rep[lv >= rv ? i - 1 : i] : -1;
    int p = parent[i];
    if (p >= 0) p = rep[p];
    parent[i] = p;
  }
  __syncthreads();
  for (int i = tid; i < n; i += threads) {
    int d = 0;
    if (rows[i] > 0)
      for (int p = parent[i]; p >= 0; p = parent[p]) ++d;
    depth[i] = d;
  }
  __syncthreads();
  // ---- nodes: the runs of the first levels (deeper ones are not shared), then the rows
  // alone with the columns that are left
  const int tile_rows = 128 / G;           // token rows of a tile
  int runs = 0, longs = 0, alone = 0;      // nodes: the runs, then rows alone, long ones first
  for (int k = tid; k < n; k += threads) {
    int p = leaf_up[k];
    while (p >= 0 && depth[p] >= kSaLevels) p = parent[p];
    leaf_up[k] = p;
  }
  for (int pass = 0; pass < 2; ++pass) {   // count the runs, then place both kinds
    if (pass == 0 && n <= threads) continue;          // one round: the scan tells it
    int at_run = 0, at_long = 0, at_alone = 0;
    for (int k0 = 0; k0 < n; k0 += threads) {
      const int k = k0 + tid;
      int v0 = 0, pages = 0, v1 = 0, pages1 = 0;
      if (k < n) {
        if (rows[k] > 0 && depth[k] < kSaLevels) {
          v0 = parent[k] >= 0 ? common[parent[k]] : 0;
          pages = common[k] - v0;
        }
        v1 = leaf_up[k] >= 0 ? common[leaf_up[k]] : 0;
        pages1 = (len_of[k] + kBlock - 1) / kBlock - v1;
      }
      int2 total;
      const bool is_long = pages1 >= kPlLong;
      const int2 sc = scan(make_int2((pages > 0) | (is_long << 16), pages1 > 0 && !is_long), min(n - k0, threads), &total);
      if (n <= threads) {
        runs = total.x & 0xFFFF;
        longs = total.x >> 16;
      }
      if (pass == 1 && k < n) {
        auto put = [&](int at, int first_col, int cols, int i0, int m) {
          nd_v0[at] = first_col;
          nd_pages[at] = cols;
          nd_i0[at] = i0;
          nd_m[at] = m;
          nd_tiles[at] = (m + 2 * tile_rows - 1) / (2 * tile_rows);
          atomicAdd(&short_items, cols * nd_tiles[at]);
        };
        nd_of[k] = nd_of[B + k] = -1;
        if (pages > 0) {
          nd_of[k] = at_run + (sc.x & 0xFFFF);
          put(nd_of[k], v0, pages, first[k], rows[k]);
          atomicMax(&longest_run, pages);
        }
        if (pages1 > 0) {
          nd_of[B + k] = is_long ? runs + at_long + (sc.x >> 16) : runs + longs + at_alone + sc.y;
          put(nd_of[B + k], v1, pages1, k, 1);
        }
      }
      at_run += total.x & 0xFFFF;
      at_long += total.x >> 16;
      at_alone += total.y;
    }
    runs = at_run;
    longs = at_long;
    alone = at_alone;
  }
  const int nodes = runs + longs + alone;
  __syncthreads();
  // ---- item lengths: a warp weighs a length of the runs, or of the rows alone.  The SMs' share of all items' times, or the
  // memory's, and a part of a row's item at the end; or the rounds that the runs' long items
  // take, whichever is more (in a round that is not full, items are 0.6 as long: the CTAs at
  // work have more of the memory's bandwidth each).  Where items of one page fit a round,
  // they are the shortest.
  const bool one_page = static_cast<long long>(short_items) * Hkv <= sms;
  for (int c = warp; c < kPlCuts + kPlAlones && !one_page; c += warps) {
    const bool shared = c < kPlCuts;       // of the runs, else of the rows alone
    const int L = shared ? kPlCut[c] : kPlAlone[c - kPlCuts], most = min(longest_run, L);
    const float inv = __fdividef(1.f, static_cast<float>(L));
    float sum = 0.f, slowest = 0.f, long_sum = 0.f, memory = 0.f;
    int items = 0, long_items = 0;
    long long parts = 0;
    for (int k = (shared ? 0 : runs) + lane; k < (shared ? runs : nodes); k += 32) {
      const int pages = nd_pages[k], m = nd_m[k];
      const int ns = pl_splits(pages, L, inv);
      const int each = nd_tiles[k] * ns * Hkv;
      const bool wide = min(m, 2 * tile_rows) > tile_rows;
      const float per = __fdividef((wide ? kPlWide : kPlNarrow) * pages, static_cast<float>(ns)) +
                        (wide ? kPlWideStart : kPlStart);
      sum += per * each;
      memory += static_cast<float>(pages * Hkv) * kPlMemory;
      items += each;
      parts += static_cast<long long>(m) * G * ns * Hkv;
      slowest = fmaxf(slowest, per);
      if (shared && 2 * pages > most * ns) {
        long_sum += per * each;
        long_items += each;
      }
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, d);
      memory += __shfl_xor_sync(0xffffffffu, memory, d);
      if (shared) long_sum += __shfl_xor_sync(0xffffffffu, long_sum, d);
    }
    // a maximum of numbers that are not negative, as integers; parts capped so that sums fit
    slowest = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(slowest)));
    items = __reduce_add_sync(0xffffffffu, items);
    long_items = __reduce_add_sync(0xffffffffu, long_items);
    const uint32_t all_parts =
        __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(parts < (1 << 25) ? parts : (1 << 25)));
    if (lane == 0) weight[c] = {sum, slowest, long_sum, memory, items, long_items, all_parts};
  }
  if (!one_page) __syncthreads();
  if (!one_page && warp == 0) {            // a lane per candidate
    int best = lane;
    const PlWeight a = weight[lane >> 1], b = weight[kPlCuts + pl_alone(lane)];
    const float run = a.slowest, single = b.slowest, all = static_cast<float>(sms);
    const int items = a.items + b.items;
    const uint32_t all_parts = a.parts + b.parts;
    float t = fmaxf(run, single);
    if (items > sms) {
      const float share = __fdividef(a.sum + b.sum, all);
      const float slow = fmaxf(1.f, __fdividef(a.memory + b.memory, share));
      float rounds_time = run;
      if (a.long_items > sms) {
        const float x = __fdividef(static_cast<float>(a.long_items), all), full = floorf(x);
        const float last = x > full ? fmaxf(x - full, 0.6f) : 0.f;
        rounds_time = __fdividef(a.long_sum, static_cast<float>(a.long_items)) * (full + last);
      }
      t = slow * fmaxf(share + kPlTail * single, rounds_time);
    }
    t += all_parts * kPlPart;
    if (items > plan.max_items || all_parts > static_cast<uint32_t>(plan.max_parts)) t = INFINITY;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
      const float ot = __shfl_xor_sync(0xffffffffu, t, d);
      const int ob = __shfl_xor_sync(0xffffffffu, best, d);
      if (ot < t || (ot == t && ob > best)) {
        t = ot;
        best = ob;
      }
    }
    if (lane == 0) chosen = best;
  }
  if (!one_page) __syncthreads();
  const int best = one_page ? 0 : chosen;
  const int L = pl_length(best).x, L1 = pl_length(best).y;
  const float inv = __fdividef(1.f, static_cast<float>(L)), inv1 = __fdividef(1.f, static_cast<float>(L1));
  auto splits = [&](int k) {
    return nd_m[k] > 1 ? pl_splits(nd_pages[k], L, inv) : pl_splits(nd_pages[k], L1, inv1);
  };
  // ---- first item and part of every node
  int n_items = 0, n_parts = 0;
  for (int k0 = 0; k0 < nodes; k0 += threads) {
    const int k = k0 + tid;
    int items = 0, parts = 0;
    if (k < nodes) {
      const int ns = splits(k);
      items = nd_tiles[k] * ns * Hkv;
      parts = nd_m[k] * G * ns * Hkv;
    }
    int2 total;
    const int2 at = scan(make_int2(items, parts), min(nodes - k0, threads), &total);
    if (k < nodes) {
      nd_item[k] = n_items + at.x;
      nd_part[k] = n_parts + at.y;
    }
    n_items += total.x;
    n_parts += total.y;
  }
  n_items = min(n_items, plan.max_items);
  if (tid == 0) {
    plan.counts[0] = n_items;
    plan.counts[1] = sms;                  // every CTA begins with the item of its own number
  }
  __syncthreads();
  // ---- items, a thread each; those of a node's tiles over the same pages side by side
  for (int e = tid; e < n_items; e += threads) {
    int lo = 0, hi = nodes;
    while (hi - lo > 1) {                  // last node whose first item is not behind e
      const int mid = (lo + hi) >> 1;
      if (nd_item[mid] <= e) lo = mid; else hi = mid;
    }
    const int pages = nd_pages[lo], m = nd_m[lo], tiles = nd_tiles[lo], ns = splits(lo);
    const uint32_t at = e - nd_item[lo];
    const uint32_t rest = tiles == 1 ? at : at / static_cast<uint32_t>(tiles);
    const int tile = at - rest * tiles;
    const int s = rest / static_cast<uint32_t>(Hkv), g = rest - s * Hkv;
    const float inv_ns = 1.f / static_cast<float>(ns);
    // pages s / ns, rounded down (the products stay below 2^21: see pl_splits)
    auto cut = [&](int k) { return static_cast<int>((static_cast<float>(pages * k) + 0.5f) * inv_ns); };
    const int ro = tile * 2 * tile_rows, i0 = nd_i0[lo] + ro, nr = min(2 * tile_rows, m - ro);
    int4* item = reinterpret_cast<int4*>(plan.items + e);
    item[0] = make_int4(i0, nr, nd_v0[lo] + cut(s), nd_v0[lo] + cut(s + 1));
    item[1] = make_int4(g, m, ro, nd_part[lo] + (s * Hkv + g) * m * G);
    const int last = row_of[i0 + nr - 1];
    item[2] = make_int4(row_of[i0], len_of[i0], last - row_of[i0] == nr - 1, 0);
  }
  // ---- every row's parts: its own node, then the runs above
  for (int i = tid; i < n; i += threads) {
    SaSeg* out = plan.segs + static_cast<size_t>(row_of[i]) * kSaMaxSegs;
    int k = 0;
    auto add = [&](int nd) {
      out[k++] = {nd_part[nd], nd_m[nd], i - nd_i0[nd], splits(nd)};
    };
    if (nd_of[B + i] >= 0) add(nd_of[B + i]);
    for (int p = leaf_up[i]; p >= 0; p = parent[p]) add(nd_of[p]);
    plan.n_segs[row_of[i]] = k;
  }
}

// ---------------------------------------------------------------- attention

namespace {

// What an item is for the warps other than the producer
struct SaSlot {
  int i0, nr, g, m;
  int ro, base;
  int pages;          // valid ones; -1: no items left
  int tail;           // keys of the last of them
  int wide;
  int row;            // the first of the rows where they lie side by side, else -1
  uint32_t ring;      // stages used before the item
  uint32_t qt;        // q tiles used before the item
};

struct SaSmem {
  uint8_t q[2][kSaTile];
  uint8_t ring[kSaStages][kSaTile];
  float2 ml[2][128];                           // narrow: (max, sum) of each half's rows
  SaSlot slot[2];
  uint64_t slot_full[2], slot_empty[2];
  uint64_t q_full[2], q_empty[2];
  uint64_t full[kSaStages], empty[kSaStages];
  // per stream and S buffer: a waiter is never more than one phase behind
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];
  uint64_t ml_full, o_free;
  uint32_t tmem_base;
};
static_assert(sizeof(SaSmem) <= 232448, "above the 227 KB of a CTA");

// 64 values of S as P: p = 2^((s - mu) sl2), packed; sums into acc.  The maximum is subtracted
// before the factor: rounded as a product, a large one would be off by whole units.
__device__ __forceinline__ void sa_exp64(const uint32_t (&sv)[64], float sl2, float mu, uint32_t* pk,
                                         float2 (&acc)[4]) {
  const float2 f = make_float2(sl2, sl2), nmu = make_float2(-mu, -mu);
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const float2 y = fmul2(fadd2(make_float2(__uint_as_float(sv[2 * j]), __uint_as_float(sv[2 * j + 1])), nmu), f);
    const float2 p = make_float2(sa_ex2(y.x), sa_ex2(y.y));
    acc[j & 3] = fadd2(acc[j & 3], p);
    pk[j] = pack_bf16x2(p.x, p.y);
  }
}

__device__ __forceinline__ float sa_max64(const uint32_t (&sv)[64]) {
  float mx[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(sv[8 * i + j]);
    mx[i] = fmaxf(max3f(max3f(max3f(x[0], x[1], x[2]), x[3], x[4]), x[5], x[6]), x[7]);
  }
  return max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
}

__device__ __forceinline__ void sa_load64(uint32_t addr, uint32_t (&sv)[64]) {
  tmem_ld32(addr, sv);
  tmem_ld32(addr + 32, sv + 32);
  tmem_ld_wait();
}

}  // namespace

__global__ void __launch_bounds__(kSaThreads, 1) shared_attn_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const __nv_bfloat16* __restrict__ q, const int32_t* __restrict__ table, int G, int Hkv, int num_pages, int max_pages, float sl2,
    float rescale, const SaPlan plan, uint32_t* status) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  SaSmem& sm = *reinterpret_cast<SaSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hq = G * Hkv, tile_rows = 128 / G;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.slot_full[i], 1);
      mbar_init(&sm.slot_empty[i], 2 + 1 + 8);
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 2);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&sm.s_full[i][b], 1);
        mbar_init(&sm.p_full[i][b], 4);
        mbar_init(&sm.pv_done[i][b], 1);
      }
    }
    for (int i = 0; i < kSaStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 2);
    }
    mbar_init(&sm.ml_full, 8);
    mbar_init(&sm.o_free, 8);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  // All that needed nothing of the plan: the kernel that makes it runs meanwhile (it uses no
  // TMEM, and what came before it has ended, so that no CTA waits for the columns taken here).
  pdl_enter();
  const bool aligned = (smem_u32(smem_raw) & 1023u) == 0;  // the tiles need it
  if (!aligned && tid == 0) atomicOr(status, kStatusBounds);
  // the first item is asked for together with their number (there is room for it in any case)
  SaItem it, nx;
  if (warp == 0) nx = plan.items[blockIdx.x];
  const int n_items = aligned ? plan.counts[0] : 0;
  // CTAs beyond the items have nothing to do: the others claim as many

  if (static_cast<int>(blockIdx.x) >= n_items) {
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer
    // The next item is claimed, read, checked and published in steps between the last pages
    // of the current one, so that their latencies (an atomic, the item, its table entries) pass
    // while pages are on the way, and q is there when the item's turn comes.  Not earlier:
    // an item claimed by a CTA that is still busy waits (claims at the first page: system
    // prompt 110 -> 125 us).
    uint32_t pos = 0, qt = 0, tc = 0;      // stages and q tiles used, items published
    bool alive = true;
    int id = 0, page = -1, nx_page = -1, valid = 0, step = 1;
    uint32_t ring_end = 0;                 // stages used when the published items are loaded
    auto entry = [&](const SaItem& t, int c) {
      return c < t.c1 ? __ldg(table + static_cast<size_t>(t.row) * max_pages + c) : -1;
    };
    auto prepare = [&]() {
      if (step == 0) {
        if (lane == 0) id = atomicAdd(plan.counts + 1, 1);
      } else if (step == 1) {
        id = tc > 0 ? __shfl_sync(0xffffffffu, id, 0) : static_cast<int>(blockIdx.x);
        if (tc > 0 && id < n_items) nx = plan.items[id];
      } else if (step == 2) {
        if (id < n_items) nx_page = entry(nx, nx.c0 + lane);
      } else if (step == 3) {
        // pages that are none have no keys
        const bool more = id < n_items;
        bool last_ok = true;
        valid = 0;
        if (more) {
          int pg = nx_page;
          for (int c = nx.c0;;) {
            const uint32_t oks = __ballot_sync(0xffffffffu, pg >= 0 && pg < num_pages);
            valid += __popc(oks);
            if (nx.c1 - c <= 32) {
              last_ok = (oks >> (nx.c1 - 1 - c)) & 1;
              break;
            }
            c += 32;
            pg = entry(nx, c + lane);
          }
        }
        const int tb = tc & 1;
        if (lane == 0) {
          alive = mbar_wait(&sm.slot_empty[tb], ((tc >> 1) & 1) ^ 1, status, 100);
          if (alive) {
            SaSlot& s = sm.slot[tb];
            s.pages = -1;
            if (more) {
              if (valid != nx.c1 - nx.c0) atomicOr(status, kStatusBounds);
              s.i0 = nx.i0;
              s.nr = nx.nr;
              s.g = nx.g;
              s.m = nx.m;
              s.ro = nx.ro;
              s.base = nx.base;
              s.pages = valid;
              s.tail = last_ok ? min(kBlock, nx.len - (nx.c1 - 1) * kBlock) : kBlock;
              s.wide = nx.nr > tile_rows;
              s.row = nx.side ? nx.row : -1;
              s.ring = ring_end;
              s.qt = qt;
            }
            mbar_arrive(&sm.slot_full[tb]);
          }
        }
        alive = __shfl_sync(0xffffffffu, alive ? 1 : 0, 0) != 0;
        if (more) {
          ring_end += 2 * valid;
          qt += nx.nr > tile_rows ? 2 : 1;
        }
        ++tc;
      }
      ++step;
    };
    while (true) {
      while (alive && step < 4) prepare();
      if (!alive || id >= n_items) break;
      it = nx;
      page = nx_page;
      step = 0;
      int left = valid;                    // pages of the item to come
      for (int c = it.c0; alive && c < it.c1; c += 32) {
        if (c > it.c0) page = entry(it, c + lane);
        uint32_t oks = __ballot_sync(0xffffffffu, page >= 0 && page < num_pages);
        for (; alive && oks; oks &= oks - 1) {
          const int pg = __shfl_sync(0xffffffffu, page, __ffs(oks) - 1);
          if (lane == 0) {
            const int at = pg * Hkv + it.g;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              const uint32_t st = pos % kSaStages;
              alive = mbar_wait(&sm.empty[st], ((pos / kSaStages) & 1) ^ 1, status, 101 + kv);
              if (!alive) break;
              mbar_arrive_expect_tx(&sm.full[st], kSaTile);
              const CUtensorMap* tm = kv ? &tm_v : &tm_k;
              tma_load_3d(sm.ring[st], tm, &sm.full[st], 0, 0, at);
              tma_load_3d(sm.ring[st] + kSaHalf, tm, &sm.full[st], 64, 0, at);
              ++pos;
            }
          }
          alive = __shfl_sync(0xffffffffu, alive ? 1 : 0, 0) != 0;
          if (alive && --left < 4 && step < 4) prepare();
        }
      }
    }
    if (!alive && lane == 0) {
      // a wait ran out: the copies in flight have to land before the CTA ends
      const uint32_t from = pos > kSaStages ? pos - kSaStages : 0;
      for (uint32_t p = from; p < pos; ++p)
        (void)mbar_wait(&sm.full[p % kSaStages], (p / kSaStages) & 1, status, 103);
    }
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------------------------------ MMA of stream s
    const int s = warp - 1;
    if (elect_one()) {
      uint32_t uses[2] = {0, 0};            // of the S buffers
      uint32_t tc = 0, items_with_o = 0;
      bool ok = true;
      auto pv_wait = [&](int b) {           // the last PV that read buffer b is done
        return uses[b] == 0 || mbar_wait(&sm.pv_done[s][b], (uses[b] - 1) & 1, status, 110);
      };
      while (ok) {
        const int tb = tc & 1;
        if (!(ok = mbar_wait(&sm.slot_full[tb], (tc >> 1) & 1, status, 111))) break;
        const SaSlot t = sm.slot[tb];
        if (t.pages < 0) break;
        const uint32_t qi = t.qt + (t.wide ? s : 0);
        const int qb = qi & 1;
        if (!(ok = mbar_wait(&sm.q_full[qb], (qi >> 1) & 1, status, 112))) break;
        tc_fence_after();
        const uint32_t qa = smem_u32(sm.q[qb]);
        const uint32_t d_s = tmem + 128 * s, d_o = tmem + kSaColO + 128 * s;
        // block j: 64 keys of page j (narrow) or half of page j / 2 (wide), in S buffer j & 1
        const int blocks = t.wide ? 2 * t.pages : t.pages;
        auto scores = [&](int j) -> bool {
          const uint32_t p = t.ring + 2 * (t.wide ? j >> 1 : j), st = p % kSaStages;
          const int b = j & 1, half = t.wide ? b : s;
          if (!mbar_wait(&sm.full[st], (p / kSaStages) & 1, status, 113) || !pv_wait(b)) return false;
          tc_fence_after();
          const uint32_t ka = smem_u32(sm.ring[st]) + half * 64 * 128;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = (kk >> 2) * kSaHalf + (kk & 3) * 32;
            umma_bf16(d_s + 64 * b, sdesc_sw128(qa + off, 16, 1024), sdesc_sw128(ka + off, 16, 1024),
                      kSaIdescS, kk > 0);
          }
          umma_commit(&sm.s_full[s][b]);
          if (!t.wide || b == 1) umma_commit(&sm.empty[st]);
          ++uses[b];
          return true;
        };
        if (blocks > 0) ok = scores(0);
        for (int j = 0; ok && j < blocks; ++j) {
          if (j + 1 < blocks && !(ok = scores(j + 1))) break;
          const int b = j & 1, half = t.wide ? b : s;
          const uint32_t p = t.ring + 2 * (t.wide ? j >> 1 : j) + 1, st = p % kSaStages;
          // uses of b so far: block j's (block j + 2 has not been issued)
          if (!(ok = mbar_wait(&sm.p_full[s][b], (uses[b] - 1) & 1, status, 114))) break;
          if (!(ok = mbar_wait(&sm.full[st], (p / kSaStages) & 1, status, 115))) break;
          // the item's first PV overwrites O: the item before must have been read
          if (j == 0 && items_with_o > 0 &&
              !(ok = mbar_wait(&sm.o_free, (items_with_o - 1) & 1, status, 116)))
            break;
          tc_fence_after();
          const uint32_t va = smem_u32(sm.ring[st]) + half * 64 * 128;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_tmem_a(d_o, d_s + 64 * b + 8 * kk, sdesc_sw128(va + kk * 2048, kSaHalf, 1024), kSaIdescPV,
                        j > 0 || kk > 0);
          umma_commit(&sm.pv_done[s][b]);
          if (!t.wide || b == 1) umma_commit(&sm.empty[st]);
        }
        if (!ok) break;
        ++items_with_o;
        mbar_arrive(&sm.slot_empty[tb]);
        if (t.wide) mbar_arrive(&sm.q_empty[qb]);    // the other stream reads the other tile
        umma_commit(&sm.q_empty[qb]);
        ++tc;
      }
    }
  } else if (warp == kSaQWarp) {
    // ------------------------------------------------------------ q
    uint32_t tc = 0;
    bool ok = true;
    while (ok) {
      const int tb = tc & 1;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.slot_full[tb], (tc >> 1) & 1, status, 120)))) break;
      const SaSlot t = sm.slot[tb];
      if (t.pages < 0) break;
      for (int w = 0; ok && w <= t.wide; ++w) {
        const uint32_t qi = t.qt + w;
        const int qb = qi & 1;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.q_empty[qb], ((qi >> 1) & 1) ^ 1, status, 121)))) break;
        // rows of the tile, 16 lanes each; all copies are in flight together, so that a tile takes
        // one latency, or two (which rows, then q)
        const int r0 = w * tile_rows, nr = min(tile_rows, t.nr - r0) * G;
        uint32_t from[4];                                // this lane's rows 32 k + lane, as rows of q
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = 32 * k + lane, tok = r / G;
          int row = 0;
          if (r < nr) row = t.row >= 0 ? t.row + r0 + tok : plan.live[t.i0 + r0 + tok];
          from[k] = row * Hq + t.g * G + (r - tok * G);
        }
        const int c = lane & 15, up = lane >> 4;
        uint8_t* dst = sm.q[qb] + (c >> 3) * kSaHalf;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (32 * k >= nr) break;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int r = 32 * k + 2 * j + up;
            const uint32_t f = __shfl_sync(0xffffffffu, from[k], 2 * j + up);
            if (r < nr)
              cp_async16(dst + sw128_offset(r, c & 7), q + static_cast<size_t>(f) * kD + 8 * c);
          }
        }
        cp_async_wait_all();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full[qb]);
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(&sm.slot_empty[tb]);
      ++tc;
    }
  } else {
    // ------------------------------------------------------------ softmax of stream s
    const int s = (warp - 4) >> 2, subp = warp & 3;
    const int r = subp * 32 + lane;                      // tile row = TMEM lane
    const uint32_t trow = static_cast<uint32_t>(subp * 32) << 16;
    const uint32_t d_s = tmem + 128 * s + trow, d_o = tmem + kSaColO + 128 * s + trow;
    uint32_t uses[2] = {0, 0}, tc = 0, merges = 0;
    bool ok = true;
    while (ok) {
      const int tb = tc & 1;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.slot_full[tb], (tc >> 1) & 1, status, 130)))) break;
      const SaSlot t = sm.slot[tb];
      if (t.pages < 0) break;
      const int r0 = t.wide ? s * tile_rows : 0;         // first token row of the tile
      const int nq = min(tile_rows, t.nr - r0) * G;      // its query rows
      const bool work = subp * 32 < nq;                  // the warp has any
      float m = -INFINITY, l = 0.f;
      const int blocks = t.wide ? 2 * t.pages : t.pages;
      for (int j = 0; ok && j < blocks; ++j) {
        const int b = j & 1;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.s_full[s][b], uses[b] & 1, status, 131)))) break;
        tc_fence_after();
        // keys of the block: a page that is not full is a leaf's last (narrow)
        const bool cut = j + 1 == blocks && t.tail < kBlock;
        const int lim = cut ? min(64, t.tail - 64 * s) : 64;
        const uint32_t sbuf = d_s + 64 * b;
        if (work) {
          uint32_t sv[64], pk[32];
          sa_load64(sbuf, sv);
          if (lim < 64) {
#pragma unroll
            for (int k = 0; k < 64; ++k) sv[k] = k < lim ? sv[k] : 0xFF800000u;
          }
          const bool any = lim > 0;
          const float mnew = any ? fmaxf(m, sa_max64(sv)) : m;
          const bool resc = mnew > m + rescale;
          // products of -infinity alone so far: they weigh nothing, and -infinity less itself would be NaN
          const float mu = resc ? mnew : fmaxf(m, -FLT_MAX);
          float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                           make_float2(0.f, 0.f)};
          if (any) {
            sa_exp64(sv, sl2, mu, pk, acc);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) pk[k] = 0u;
          }
          const bool need = resc && m != -INFINITY;
          if (__any_sync(0xffffffffu, need)) {
            // O stands still once the PV of the block before is done
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.pv_done[s][b ^ 1], (uses[b ^ 1] - 1) & 1, status, 132)))) break;
            tc_fence_after();
            const float alpha = need ? sa_ex2((m - mu) * sl2) : 1.f;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t v[32];
              __syncwarp();
              tmem_ld32(d_o + c * 32, v);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
              tmem_st16(d_o + c * 32, v);
              tmem_st16(d_o + c * 32 + 16, v + 16);
            }
          }
          if (any) {
            const float2 a = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
            const float rs = a.x + a.y;
            l = (need ? l * sa_ex2((m - mu) * sl2) : l) + rs;   // without `need` and with resc: 0 or NaN
            m = resc ? mnew : m;
          }
          __syncwarp();                        // the stores are the whole warp's
          tmem_st16(sbuf, pk);
          tmem_st16(sbuf + 16, pk + 16);
          tmem_st_wait();
        }
        if (cut) {
          // what lies behind the row's end may be anything, and 0 times it has to be 0
          // (either stream clears what it multiplies)
          const uint32_t p = t.ring + 2 * j + 1, st = p % kSaStages;
          if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[st], (p / kSaStages) & 1, status, 133)))) break;
          const int key = 64 * s + (r >> 1);
          if (key >= t.tail) {
            uint4* v = reinterpret_cast<uint4*>(sm.ring[st] + (r & 1) * kSaHalf + key * 128);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[s][b]);
        ++uses[b];
      }
      if (!ok) break;
      // ---- the item's parts
      const size_t rows = static_cast<size_t>(t.m) * G;
      const size_t at = static_cast<size_t>(t.ro + r0) * G + r;
      float4* po = plan.part_o + static_cast<size_t>(t.base) * 32 + at;
      const bool mine = r < nq;
      if (t.pages > 0) {
        const int b = (blocks - 1) & 1;
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.pv_done[s][b], (uses[b] - 1) & 1, status, 134)))) break;
      }
      float f0 = 1.f, f1 = 0.f;
      // keys, but no product that is a number: as the definition has it, NaN (a reference of
      // -infinity would stand for no keys)
      if (l != l && m == -INFINITY) m = 0.f;
      float2 ml = make_float2(m, l);
      if (!t.wide && t.pages > 0) {
        // both halves' maxima; either stream then writes half of the channels
        sm.ml[s][r] = ml;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.ml_full);
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.ml_full, merges & 1, status, 135)))) break;
        ++merges;
        const float2 a = sm.ml[0][r], c = sm.ml[1][r];
        const float M = fmaxf(a.x, c.x);
        f0 = a.x == -INFINITY ? 0.f : sa_ex2((a.x - M) * sl2);
        f1 = c.x == -INFINITY ? 0.f : sa_ex2((c.x - M) * sl2);
        ml = make_float2(M, a.y * f0 + c.y * f1);
      }
      tc_fence_after();
      if (t.pages == 0) {
        if (mine && (t.wide || s == 0)) {
          for (int d = 0; d < 32; ++d) po[d * rows] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      } else if (work) {
        const uint32_t o0 = tmem + kSaColO + trow;
#pragma unroll 1
        for (int c = 0; c < (t.wide ? 8 : 4); ++c) {
          const int col = t.wide ? 16 * c : 64 * s + 16 * c;
          uint32_t x[16], y[16];
          __syncwarp();                          // the loads are the whole warp's
          if (t.wide) {
            tmem_ld16(d_o + col, x);
          } else {
            tmem_ld16(o0 + col, x);
            tmem_ld16(o0 + 128 + col, y);
          }
          tmem_ld_wait();
          if (!t.wide) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float a = f0 > 0.f ? __uint_as_float(x[j]) * f0 : 0.f;
              x[j] = __float_as_uint(f1 > 0.f ? fmaf(__uint_as_float(y[j]), f1, a) : a);
            }
          }
          if (mine) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              po[(col / 4 + j) * rows] =
                  make_float4(__uint_as_float(x[4 * j]), __uint_as_float(x[4 * j + 1]),
                              __uint_as_float(x[4 * j + 2]), __uint_as_float(x[4 * j + 3]));
          }
        }
      }
      if (mine && (t.wide || s == 0)) plan.part_ml[t.base + at] = ml;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.o_free);
        mbar_arrive(&sm.slot_empty[tb]);
      }
      ++tc;
    }
  }
  __syncwarp();                              // the lanes of a role join
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- combine

// grid (rows, KV heads, shares of Gc heads); thread (way, d4, head): heads run fastest, as the
// parts lie in memory, and the ways take every so many-th part.  Bound by latency (the row's
// list, then its parts, 6 per thread in flight), so the list is read at once, by whoever
// is there first.
constexpr int kCbThreads = 512, kCbDeep = 6;

__global__ void __launch_bounds__(kCbThreads, 2) shared_combine_kernel(const SaPlan plan, int G, int Hkv, int Gc,
                                                                    int ways, float sl2,
                                                                    __nv_bfloat16* __restrict__ o,
                                                                    float* __restrict__ lse) {
  __shared__ SaSeg seg[kSaMaxSegs];
  __shared__ int n_seg;
  __shared__ float4 part[kCbThreads];
  __shared__ float2 part_ml[kCbThreads];
  const int b = blockIdx.x, g = blockIdx.y, tid = threadIdx.x;
  // the plan was complete before the kernel that is waited for let this one start
  if (tid < kSaMaxSegs) {
    const int4 e = __ldcg(reinterpret_cast<const int4*>(plan.segs + static_cast<size_t>(b) * kSaMaxSegs + tid));
    seg[tid] = {e.x, e.y, e.z, e.w};
  }
  if (tid == kSaMaxSegs) n_seg = __ldcg(plan.n_segs + b);
  const int h = blockIdx.z * Gc + tid % Gc, d4 = tid / Gc % 32, way = tid / (32 * Gc);
  __syncthreads();
  const int ns = n_seg;
  int total = 0;
  for (int k = 0; k < ns; ++k) total += seg[k].splits;
  pdl_enter();
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (h < G) {
    int k = 0, s = way;                      // next part: split s of segment k
    for (int p = way; p < total; p += ways * kCbDeep) {
      float2 ml[kCbDeep];
      float4 x[kCbDeep];
#pragma unroll
      for (int i = 0; i < kCbDeep; ++i) {
        ml[i] = make_float2(-INFINITY, 0.f);
        if (p + i * ways >= total) continue;
        while (s >= seg[k].splits) s -= seg[k++].splits;
        const size_t rows = static_cast<size_t>(seg[k].m) * G, at = static_cast<size_t>(seg[k].ro) * G + h;
        const size_t base = seg[k].base + (static_cast<size_t>(s) * Hkv + g) * rows;
        ml[i] = plan.part_ml[base + at];
        x[i] = plan.part_o[base * 32 + d4 * rows + at];
        s += ways;
      }
      float top = M;
#pragma unroll
      for (int i = 0; i < kCbDeep; ++i) top = fmaxf(top, ml[i].x);
      if (top == -INFINITY) continue;
      const float f = M == -INFINITY ? 0.f : sa_ex2((M - top) * sl2);
      acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
      l *= f;
      M = top;
#pragma unroll
      for (int i = 0; i < kCbDeep; ++i) {
        if (ml[i].x == -INFINITY) continue;
        const float e = sa_ex2((ml[i].x - top) * sl2);
        acc.x = fmaf(x[i].x, e, acc.x);
        acc.y = fmaf(x[i].y, e, acc.y);
        acc.z = fmaf(x[i].z, e, acc.z);
        acc.w = fmaf(x[i].w, e, acc.w);
        l = fmaf(ml[i].y, e, l);
      }
    }
  }
  if (ways > 1 && total > 1) {               // uniform
    part[tid] = acc;
    part_ml[tid] = make_float2(M, l);
    __syncthreads();
    if (way == 0) {
      for (int w = 1; w < ways; ++w) {
        const float2 ml = part_ml[tid + w * 32 * Gc];
        const float4 x = part[tid + w * 32 * Gc];
        if (ml.x == -INFINITY) continue;
        const float top = fmaxf(M, ml.x), f = M == -INFINITY ? 0.f : sa_ex2((M - top) * sl2);
        const float e = sa_ex2((ml.x - top) * sl2);
        acc = make_float4(fmaf(x.x, e, acc.x * f), fmaf(x.y, e, acc.y * f), fmaf(x.z, e, acc.z * f),
                          fmaf(x.w, e, acc.w * f));
        l = fmaf(ml.y, e, l * f);
        M = top;
      }
    }
  }
  if (way > 0 || h >= G) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const size_t at = (static_cast<size_t>(b) * Hkv + g) * G + h;
  *reinterpret_cast<uint2*>(o + at * kD + 4 * d4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lse && d4 == 0) lse[at] = M == -INFINITY ? -INFINITY : fmaf(M, sl2, log2f(l)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------- host

namespace {

SaPlan carve_shared_workspace(WsCursor& ws, int B, int Hq, int Hkv) {
  const long long sms = device_sm_count();
  SaPlan p{};
  // With items of the longest length a node has one per tile and KV head: B tiles of leaves
  // and at most 3/4 B (runs of 3 in tiles of 2 rows) at each of the levels; beyond that, room
  // to cut for all SMs.
  p.max_items = static_cast<int>(6LL * B * Hkv + 8 * sms);
  const long long parts = static_cast<long long>(B) * Hq * kSaMaxSegs + 2 * sms * 256;
  p.max_parts = static_cast<int>(parts);
  p.live = ws.take<int>(B);
  p.items = ws.take<SaItem>(p.max_items);
  p.counts = ws.take<int>(2);
  p.segs = ws.take<SaSeg>(static_cast<size_t>(B) * kSaMaxSegs);
  p.n_segs = ws.take<int>(B);
  p.part_ml = ws.take<float2>(p.max_parts);
  p.part_o = ws.take<float4>(static_cast<size_t>(p.max_parts) * 32);
  return p;
}

bool shared_sizes_ok(int B, int Hq, int Hkv) {
  return B >= 1 && B <= kSaMaxRows && Hkv >= 1 && Hkv <= 256 && Hq >= 1 && Hq % Hkv == 0 &&
         Hq / Hkv <= 128 && Hq <= 1024;
}

}  // namespace

}  // namespace msa

using namespace msa;

extern "C" {

size_t msa_decode_shared_workspace_size(int B, int Hq, int Hkv, int max_pages) {
  if (!shared_sizes_ok(B, Hq, Hkv)) return 0;
  if (max_pages >= 1 && short_attn_fits(B, Hq / Hkv, Hkv, max_pages)) return 256;   // nothing is kept there
  WsCursor ws(nullptr);
  carve_shared_workspace(ws, B, Hq, Hkv);
  return ws.used + 256;
}

msa_status_t msa_decode_shared(const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_table, const int32_t* cache_lens, int B,
                               int Hq, int Hkv, int num_pages, int max_pages, float scale, void* o,
                               float* lse, void* workspace, size_t workspace_bytes,
                               msa_stream_t stream) {
  MSA_REQUIRE_PTR(q);
  MSA_REQUIRE_PTR(k_cache);
  MSA_REQUIRE_PTR(v_cache);
  MSA_REQUIRE_PTR(block_table);
  MSA_REQUIRE_PTR(cache_lens);
  MSA_REQUIRE_PTR(o);
  MSA_REQUIRE_PTR(workspace);
  if (lse && !aligned16(lse)) return fail(MSA_ERR_INVALID_ARG, "lse is not 16-byte aligned");
  if (B < 1) return fail(MSA_ERR_INVALID_ARG, "B must be >= 1");
  if (B > kSaMaxRows) return fail(MSA_ERR_UNSUPPORTED, "at most %d rows (got %d)", kSaMaxRows, B);
  MSA_TRY(check_cache_sizes(Hkv, num_pages, max_pages));
  if (Hq < 1 || Hq % Hkv != 0)
    return fail(MSA_ERR_INVALID_ARG, "Hq (%d) must be a positive multiple of Hkv (%d)", Hq, Hkv);
  if (!shared_sizes_ok(B, Hq, Hkv))
    return fail(MSA_ERR_UNSUPPORTED, "at most 128 query heads per KV head and 1024 in all (got %d / %d)", Hq, Hkv);
  if (static_cast<long long>(num_pages) * Hkv > INT32_MAX)
    return fail(MSA_ERR_UNSUPPORTED, "num_pages * Hkv above 2^31");
  if (!(scale >= 0x1p-64f && scale <= 0x1p64f))
    return fail(MSA_ERR_INVALID_ARG, "scale must be from 2^-64 to 2^64");
  // o may be q: a head is read before it is written; other CTAs have yet to read the rest
  const size_t heads = static_cast<size_t>(B) * Hq, ob = heads * kD * sizeof(__nv_bfloat16);
  const size_t rows = static_cast<size_t>(B) * sizeof(int32_t);
  if (o != q && overlap(o, ob, q, ob)) return fail(MSA_ERR_INVALID_ARG, "o overlaps q (it may be q)");
  const struct {
    const void* at;
    size_t bytes;
    const char* name;
  } out[2] = {{o, ob, "o"}, {lse, heads * sizeof(float), "lse"}};
  for (int i = 0; i < (lse ? 2 : 1); ++i)
    if (overlap(out[i].at, out[i].bytes, cache_lens, rows) ||
        overlap(out[i].at, out[i].bytes, block_table, rows * max_pages))
      return fail(MSA_ERR_INVALID_ARG, "%s overlaps the rows", out[i].name);
  if (lse && (overlap(lse, out[1].bytes, q, ob) || overlap(lse, out[1].bytes, o, ob)))
    return fail(MSA_ERR_INVALID_ARG, "lse overlaps q or o");
  if (workspace_bytes < msa_decode_shared_workspace_size(B, Hq, Hkv, max_pages))
    return fail(MSA_ERR_INVALID_ARG, "workspace too small");
  const int G = Hq / Hkv, sms = device_sm_count();
  CUtensorMap tk, tv;
  const uint64_t dims[3] = {static_cast<uint64_t>(kD), static_cast<uint64_t>(kBlock),
                            static_cast<uint64_t>(num_pages) * Hkv};
  const uint32_t box[3] = {64, kBlock, 1};
  if (!make_tmap_bf16(&tk, k_cache, 3, dims, box) || !make_tmap_bf16(&tv, v_cache, 3, dims, box))
    return fail(MSA_ERR_CUDA, "cuTensorMapEncodeTiled failed for the caches");
  if (short_attn_fits(B, G, Hkv, max_pages))
    return launch_short_attn({tk, tv, static_cast<const __nv_bfloat16*>(q), block_table, cache_lens, B, G, Hkv,
                              num_pages, max_pages, scale * kSaLog2e, static_cast<__nv_bfloat16*>(o), lse},
                             static_cast<cudaStream_t>(stream));
  WsCursor ws(workspace);
  const SaPlan plan = carve_shared_workspace(ws, B, Hq, Hkv);
  uint32_t* sw = nullptr;
  MSA_TRY(status_word(&sw));
  MSA_TRY(ensure_smem(shared_attn_kernel, sizeof(SaSmem), "shared_attn_kernel"));
  constexpr size_t kPlanRow = (kPlRowInts + 2 * kPlNodeInts) * sizeof(int);
  const size_t plan_smem = B * kPlanRow;
  MSA_TRY(ensure_smem(shared_plan_kernel, kSaMaxRows * kPlanRow, "shared_plan_kernel"));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope trace_("shared_plan_kernel", st);
    launch_pdl(shared_plan_kernel, 1, B <= 16 ? 256 : kPlThreads, plan_smem, st, block_table, cache_lens, B, G, Hkv,
               max_pages, sms, plan, sw);
  }
  MSA_TRY(check_launch("shared_plan_kernel"));
  {
    TraceScope trace_("shared_attn_kernel", st);
    launch_pdl(shared_attn_kernel, sms, kSaThreads, sizeof(SaSmem), st, tk, tv,
               static_cast<const __nv_bfloat16*>(q), block_table, G, Hkv, num_pages, max_pages,
               scale * kSaLog2e, kSaRescale / (scale * kSaLog2e), plan, sw);
  }
  MSA_TRY(check_launch("shared_attn_kernel"));
  {
    TraceScope trace_("shared_combine_kernel", st);
    // few rows: 4 heads per CTA and 4 ways, so that more parts are in flight; many: the
    // ways only cost (64 rows x 64 heads: 9.5 us with one, 13 with two)
    const bool few = static_cast<long long>(B) * Hq <= 16LL * sms;
    const int most = few ? 4 : 16, Gc = G < most ? G : most, fit = kCbThreads / (32 * Gc);
    const int ways = !few ? 1 : (fit < 4 ? fit : 4);
    launch_pdl(shared_combine_kernel, dim3(B, Hkv, (G + Gc - 1) / Gc), 32 * Gc * ways, 0, st, plan, G, Hkv, Gc,
               ways, scale * kSaLog2e, static_cast<__nv_bfloat16*>(o), lse);
  }
  return check_launch("shared_combine_kernel");
}

}  // extern "C"
