// Upkeep of a paged cache on the device: rows share pages by reference counts
// (fork), lose them (free), grow (extend, with copy on write), and the pool is packed
// to its front (compact).  The tables are small: one CTA decides, with scans
// over rows and pages in place of any host synchronisation, and what it chooses depends
// on the tables alone (free pages go out in ascending order).  The bytes of pages
// are the bulk of the traffic: a persistent grid moves them through shared
// memory with bulk copies (global -> shared -> global), no registers involved.
// Measured: 890 of 4,096 pages of 98 KB moved in 31 us (175 MB read and written, 5.6
// TB/s; chunks of 8 or 32 KB, deeper rings and two CTAs per SM all within 3 %), the
// tables' part of a free and a compaction 8 us.  The one CTA walks all reference counts:
// growing 96 rows by a token takes 4.3 us with 4,096 pages, 22 with 100,000 and 183 with a
// million, a compaction of the tables 5.3, 114 and 1,092 us.
#include "kernels.cuh"

namespace msa {

namespace {

constexpr int kPgThreads = 1024;
constexpr int kPgMaxCaches = 8;
constexpr int kPgChunk = 16384;     // bytes of one bulk copy
constexpr int kPgStages = 8;

__host__ __device__ inline int blocks_of(int len) { return (len + kBlock - 1) / kBlock; }

struct PageCaches {
  uint8_t* base[kPgMaxCaches];
  long long bytes[kPgMaxCaches];    // of a page
  int chunks[kPgMaxCaches + 1];     // prefix sums of the chunks of a page
  int n;
};

// Exclusive scan of v over the CTA (kPgThreads threads); *total = the sum.
__device__ __forceinline__ int block_excl_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warp_sums[wp] = x;
  __syncthreads();
  if (wp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const int before = wp > 0 ? warp_sums[wp - 1] : 0;
  *total = warp_sums[kPgThreads / 32 - 1];
  __syncthreads();                          // warp_sums may be used again
  return before + x - v;
}

__device__ __forceinline__ bool row_ok(int len, int max_pages) {
  return len >= 0 && len <= max_pages * kBlock;
}

}  // namespace

// ---------------------------------------------------------------- fork, free
//
// One CTA settles which pairs hold and the new lengths; a row named twice is
// claimed by the lowest index with atomicMin on its length (claims are negative, lengths
// are not).  Then table entries and reference counts are moved: by the same CTA, a
// warp per pair, when there are few entries (one launch less: 2 us), by a second
// launch with a CTA per pair otherwise.
constexpr long long kPgOneLaunch = 16384;   // entries at most

// Row `to` takes the first entries of row `from`, as many as `len` tokens need.
__device__ __forceinline__ void fork_row(const int32_t* from, int32_t* to, int len, int32_t* ref,
                                         int num_pages, int tid, int nthreads, uint32_t* status) {
  for (int j = tid; j < blocks_of(len); j += nthreads) {
    const int pg = from[j];
    to[j] = pg;
    if (pg < 0 || pg >= num_pages) atomicOr(status, kStatusBounds);
    else atomicAdd(&ref[pg], 1);
  }
}

// Entries of the tokens keep .. keep + drop - 1 leave the row.
__device__ __forceinline__ void free_row(int32_t* row, int keep, int drop, int32_t* ref,
                                         int num_pages, int tid, int nthreads, uint32_t* status) {
  for (int j = blocks_of(keep) + tid; j < blocks_of(keep + drop); j += nthreads) {
    const int pg = row[j];
    row[j] = -1;
    if (pg < 0 || pg >= num_pages) {
      atomicOr(status, kStatusBounds);
    } else if (atomicSub(&ref[pg], 1) <= 0) {      // held more often than counted
      atomicAdd(&ref[pg], 1);
      atomicOr(status, kStatusBounds);
    }
  }
}

__global__ void __launch_bounds__(kPgThreads) pages_fork_claim_kernel(
    const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
    const int32_t* __restrict__ keep, int n, int32_t* lens, int B, int max_pages,
    int32_t* forked, bool all, int32_t* table, int32_t* ref, int num_pages, uint32_t* status) {
  pdl_enter();
  // 1. what every pair would get, from the lengths before the call
  for (int i = threadIdx.x; i < n; i += kPgThreads) {
    const int s = src[i], d = dst[i];
    int len = -1;
    if (s < 0 || s >= B || d < 0 || d >= B) {
      atomicOr(status, kStatusBounds);
    } else {
      const int ls = lens[s];
      if (!row_ok(ls, max_pages)) {
        atomicOr(status, kStatusBounds);
      } else if (s != d && lens[d] == 0) {
        len = ls;
        if (keep) {
          const int k = keep[i];
          if (k < 0 || k > ls) atomicOr(status, kStatusBounds);
          len = max(0, min(k, ls));
        }
      }
    }
    forked[i] = len;
  }
  __syncthreads();
  // 2. claims
  for (int i = threadIdx.x; i < n; i += kPgThreads)
    if (forked[i] >= 0) atomicMin(&lens[dst[i]], i - n);
  __syncthreads();
  // 3. the lowest pair of each row wins; its length is written once all have looked
  for (int i = threadIdx.x; i < n; i += kPgThreads)
    if (forked[i] >= 0 && lens[dst[i]] != i - n) forked[i] = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPgThreads)
    if (forked[i] >= 0) lens[dst[i]] = forked[i];
  if (!all) return;
  for (int i = threadIdx.x >> 5; i < n; i += kPgThreads / 32)
    if (forked[i] > 0)
      fork_row(table + static_cast<size_t>(src[i]) * max_pages,
               table + static_cast<size_t>(dst[i]) * max_pages, forked[i], ref, num_pages,
               threadIdx.x & 31, 32, status);
}

__global__ void __launch_bounds__(128) pages_fork_kernel(const int32_t* __restrict__ src,
                                                         const int32_t* __restrict__ dst,
                                                         const int32_t* __restrict__ forked,
                                                         int32_t* table, int32_t* ref,
                                                         int num_pages, int max_pages,
                                                         uint32_t* status) {
  pdl_enter();
  const int len = forked[blockIdx.x];
  if (len > 0)
    fork_row(table + static_cast<size_t>(src[blockIdx.x]) * max_pages,
             table + static_cast<size_t>(dst[blockIdx.x]) * max_pages, len, ref, num_pages,
             threadIdx.x, blockDim.x, status);
}

// An entry that drops nothing claims nothing (the length stays as it is).
__global__ void __launch_bounds__(kPgThreads) pages_free_claim_kernel(
    const int32_t* __restrict__ rows, const int32_t* __restrict__ keep, int n, int32_t* lens,
    int B, int max_pages, int32_t* dropped, bool all, int32_t* table, int32_t* ref, int num_pages,
    uint32_t* status) {
  pdl_enter();
  for (int i = threadIdx.x; i < n; i += kPgThreads) {
    const int r = rows[i], k = keep ? keep[i] : 0;
    int drop = -1;
    if (r < 0 || r >= B || k < 0 || !row_ok(lens[r], max_pages)) atomicOr(status, kStatusBounds);
    else drop = max(0, lens[r] - k);
    dropped[i] = drop;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPgThreads)
    if (dropped[i] > 0) atomicMin(&lens[rows[i]], i - n);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPgThreads)
    if (dropped[i] > 0 && lens[rows[i]] != i - n) dropped[i] = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPgThreads)
    if (dropped[i] > 0) lens[rows[i]] = keep ? keep[i] : 0;
  if (!all) return;
  for (int i = threadIdx.x >> 5; i < n; i += kPgThreads / 32)
    if (dropped[i] > 0)
      free_row(table + static_cast<size_t>(rows[i]) * max_pages, keep ? keep[i] : 0, dropped[i], ref,
               num_pages, threadIdx.x & 31, 32, status);
}

__global__ void __launch_bounds__(128) pages_free_kernel(const int32_t* __restrict__ rows,
                                                         const int32_t* __restrict__ keep,
                                                         const int32_t* __restrict__ dropped,
                                                         int32_t* table, int32_t* ref,
                                                         int num_pages, int max_pages,
                                                         uint32_t* status) {
  pdl_enter();
  const int drop = dropped[blockIdx.x];
  if (drop > 0)
    free_row(table + static_cast<size_t>(rows[blockIdx.x]) * max_pages, keep ? keep[blockIdx.x] : 0,
             drop, ref, num_pages, threadIdx.x, blockDim.x, status);
}

// ---------------------------------------------------------------- extend

// One CTA.  need(b) = pages that row b lacks, one more when its partly filled
// last page is shared; rows are served while the sum of the needs up to them fits in
// what is free.  Lists the copies to make.
__global__ void __launch_bounds__(kPgThreads) pages_extend_kernel(
    const int32_t* __restrict__ add, int32_t* table, int32_t* lens, int32_t* ref, int B,
    int num_pages, int max_pages, int32_t* __restrict__ done, int2* __restrict__ plan,
    int32_t* __restrict__ free_list, int32_t* __restrict__ copy_src,
    int32_t* __restrict__ copy_dst, int32_t* __restrict__ n_copies, uint32_t* status) {
  pdl_enter();
  __shared__ int warp_sums[kPgThreads / 32];
  __shared__ int copies;
  const int tid = threadIdx.x;
  if (tid == 0) copies = 0;
  // ---- needs: plan[b] = (first place in the free list, need | cow << 30), need -1: refused
  int wanted = 0;
  for (int b0 = 0; b0 < B; b0 += kPgThreads) {
    const int b = b0 + tid;
    int need = 0, cow = 0;
    if (b < B) {
      const int L = lens[b], a = add[b];
      if (a < 0 || !row_ok(L, max_pages)) {
        atomicOr(status, kStatusBounds);
        need = -1;
      } else if (a > max_pages * kBlock - L) {
        need = -1;
      } else if (a > 0) {
        need = blocks_of(L + a) - blocks_of(L);
        if (L % kBlock != 0) {
          const int pg = table[static_cast<size_t>(b) * max_pages + L / kBlock];
          if (pg < 0 || pg >= num_pages || ref[pg] < 1) {
            atomicOr(status, kStatusBounds);
            need = -1;
          } else if (ref[pg] > 1) {
            cow = 1;
            ++need;
          }
        }
      }
    }
    int total;
    const int at = wanted + block_excl_scan(max(need, 0), warp_sums, &total);
    if (b < B) plan[b] = make_int2(at, need < 0 ? -1 : (need | cow << 30));
    wanted += total;
  }
  // ---- free pages in ascending order, as many as are wanted
  const int seg = (num_pages + kPgThreads - 1) / kPgThreads;
  const int p0 = min(num_pages, tid * seg), p1 = min(num_pages, p0 + seg);
  int nfree = 0;
  for (int p = p0; p < p1; ++p) nfree += ref[p] <= 0;
  int avail;
  int at = block_excl_scan(nfree, warp_sums, &avail);
  if (nfree > 0 && at < wanted)
    for (int p = p0; p < p1; ++p)
      if (ref[p] <= 0) {
        if (at < wanted) free_list[at] = p;
        ++at;
      }
  __syncthreads();
  // ---- serve the rows, one warp each
  for (int b = tid >> 5; b < B; b += kPgThreads / 32) {
    const int lane = tid & 31;
    const int2 pl = plan[b];
    const bool refused = pl.y < 0;
    const int need = pl.y & 0x3FFFFFFF, cow = (pl.y >> 30) & 1;
    const bool ok = !refused && (need == 0 || pl.x + need <= avail);
    if (lane == 0) done[b] = ok ? 1 : 0;
    if (!ok) continue;
    const int L = lens[b];
    __syncwarp();                                  // every lane has the old length before it is replaced
    int32_t* row = table + static_cast<size_t>(b) * max_pages;
    for (int j = lane; j < need; j += 32) {
      const int pg = free_list[pl.x + j];
      ref[pg] = 1;
      if (cow && j == 0) {
        const int old = row[L / kBlock];
        const int k = atomicAdd(&copies, 1);
        copy_src[k] = old;
        copy_dst[k] = pg;
        atomicSub(&ref[old], 1);
        row[L / kBlock] = pg;
      } else {
        row[blocks_of(L) + j - cow] = pg;
      }
    }
    if (lane == 0) lens[b] = L + add[b];
  }
  __syncthreads();
  if (tid == 0) *n_copies = copies;
}

// ---------------------------------------------------------------- compact

__global__ void __launch_bounds__(kPgThreads) pages_compact_kernel(
    int32_t* ref, int num_pages, int32_t* __restrict__ page_map, int32_t* __restrict__ n_live,
    int32_t* __restrict__ copy_src, int32_t* __restrict__ copy_dst,
    int32_t* __restrict__ n_copies) {
  pdl_enter();
  __shared__ int warp_sums[kPgThreads / 32];
  const int tid = threadIdx.x;
  const int seg = (num_pages + kPgThreads - 1) / kPgThreads;
  const int p0 = min(num_pages, tid * seg), p1 = min(num_pages, p0 + seg);
  int cnt = 0, live, moves, holes;
  for (int p = p0; p < p1; ++p) cnt += ref[p] > 0;
  block_excl_scan(cnt, warp_sums, &live);
  // pages in use at `live` and behind, free places below: as many of both
  int nm = 0, nh = 0;
  for (int p = p0; p < p1; ++p) {
    const bool used = ref[p] > 0;
    nm += used && p >= live;
    nh += !used && p < live;
  }
  int m = block_excl_scan(nm, warp_sums, &moves);
  int h = block_excl_scan(nh, warp_sums, &holes);
  for (int p = p0; p < p1; ++p) {
    const bool used = ref[p] > 0;
    page_map[p] = used ? p : -1;
    if (used && p >= live) copy_src[m++] = p;
    if (!used && p < live) copy_dst[h++] = p;
  }
  __syncthreads();
  for (int k = tid; k < moves; k += kPgThreads) {
    const int s = copy_src[k], d = copy_dst[k];
    page_map[s] = d;
    ref[d] = ref[s];
    ref[s] = 0;
  }
  if (tid == 0) {
    *n_live = live;
    *n_copies = moves;
  }
}

// ---------------------------------------------------------------- copies
//
// Items are (pair, chunk of a page's caches), cut into equal runs over a
// persistent grid.  Thread 0 of a CTA keeps kPgAhead loads and as many stores of
// 16 KB in flight through a ring in shared memory.  The other threads
// meanwhile rewrite block tables by page_map (compact).
constexpr int kPgAhead = kPgStages / 2;

struct CopySmem {
  alignas(128) uint8_t buf[kPgStages][kPgChunk];
  uint64_t full[kPgStages];
};

__global__ void __launch_bounds__(128) pages_copy_kernel(
    const PageCaches pc, const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n,
    const int32_t* __restrict__ n_dev, int num_pages, int32_t* table,
    const int32_t* __restrict__ lens, const int32_t* __restrict__ page_map, int B, int max_pages,
    uint32_t* status) {
  pdl_enter();
  extern __shared__ __align__(128) uint8_t smem_raw[];
  CopySmem& sm = *reinterpret_cast<CopySmem*>(smem_raw);
  if (threadIdx.x >= 32) {
    if (!page_map) return;
    for (int b = blockIdx.x; b < B; b += gridDim.x) {
      const int L = lens[b];
      if (!row_ok(L, max_pages)) {
        atomicOr(status, kStatusBounds);
        continue;
      }
      int32_t* row = table + static_cast<size_t>(b) * max_pages;
      for (int j = threadIdx.x - 32; j < blocks_of(L); j += blockDim.x - 32) {
        const int pg = row[j];
        const int to = pg >= 0 && pg < num_pages ? page_map[pg] : -1;
        if (to < 0) atomicOr(status, kStatusBounds);
        else if (to != pg) row[j] = to;
      }
    }
    return;
  }
  if (threadIdx.x != 0) return;
  const int per_page = pc.chunks[pc.n];
  if (per_page == 0) return;
  const int pairs = n_dev ? *n_dev : n;
  const long long items = static_cast<long long>(pairs) * per_page;
  // this CTA's run of items; the next pair's pages are read a page ahead
  const long long i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;
  if (i0 >= i1) return;
  for (int i = 0; i < kPgStages; ++i) mbar_init(&sm.full[i], 1);
  fence_mbar_init();
  fence_proxy_async_smem();
  int pair = static_cast<int>(i0 / per_page);
  int ch = static_cast<int>(i0 - static_cast<long long>(pair) * per_page), c = 0;
  long long left = i1 - i0;
  int ps = src[pair], pd = dst[pair], ps_next = -1, pd_next = -1;
  bool skip = false;
  auto enter = [&]() {                             // a pair begins: check it, read the next one
    skip = ps == pd;
    if (ps < 0 || ps >= num_pages || pd < 0 || pd >= num_pages) {
      atomicOr(status, kStatusBounds);
      skip = true;
    }
    if (pair + 1 < pairs) {
      ps_next = src[pair + 1];
      pd_next = dst[pair + 1];
    }
  };
  enter();
  uint8_t* to[kPgStages];
  uint32_t bytes[kPgStages];
  uint32_t nl = 0;                                 // loads issued
  auto load = [&]() {
    bool issued = false;
    while (left > 0 && !issued) {
      if (!skip) {
        while (ch >= pc.chunks[c + 1]) ++c;
        const long long off = static_cast<long long>(ch - pc.chunks[c]) * kPgChunk;
        const long long rest = pc.bytes[c] - off;
        const uint32_t sz = static_cast<uint32_t>(rest < kPgChunk ? rest : kPgChunk);
        const int st = nl % kPgStages;
        to[st] = pc.base[c] + pd * pc.bytes[c] + off;
        bytes[st] = sz;
        mbar_arrive_expect_tx(&sm.full[st], sz);
        bulk_load(sm.buf[st], pc.base[c] + ps * pc.bytes[c] + off, sz, &sm.full[st]);
        ++nl;
        issued = true;
      }
      --left;
      if (++ch == per_page) {
        ch = c = 0;
        ++pair;
        ps = ps_next;
        pd = pd_next;
        if (left > 0) enter();
      }
    }
  };
  for (int i = 0; i < kPgAhead; ++i) load();
  for (uint32_t k = 0; k < nl; ++k) {
    // the stage that the next load takes was stored from kPgAhead stores ago
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kPgAhead - 1) : "memory");
    load();
    const int st = k % kPgStages;
    if (!mbar_wait(&sm.full[st], (k / kPgStages) & 1, status, 90)) {
      // a load never came: wait (again bounded) for those behind it, then leave
      for (uint32_t j = k + 1; j < nl; ++j)
        (void)mbar_wait(&sm.full[j % kPgStages], (j / kPgStages) & 1, status, 91);
      break;
    }
    bulk_store(to[st], sm.buf[st], bytes[st]);
    bulk_commit_group();
  }
  bulk_wait_all();
}

// ---------------------------------------------------------------- host

namespace {

msa_status_t page_caches(void* const* caches, const int64_t* page_bytes, int n, PageCaches* pc) {
  if (n < 0 || n > kPgMaxCaches)
    return fail(MSA_ERR_INVALID_ARG, "n_caches %d outside [0, %d]", n, kPgMaxCaches);
  if (n > 0 && (!caches || !page_bytes))
    return fail(MSA_ERR_INVALID_ARG, "caches or page_bytes is null");
  pc->n = n;
  pc->chunks[0] = 0;
  for (int i = 0; i < n; ++i) {
    if (!caches[i] || !aligned16(caches[i]))
      return fail(MSA_ERR_INVALID_ARG, "cache %d is null or not 16-byte aligned", i);
    if (page_bytes[i] < 16 || page_bytes[i] % 16 != 0 || page_bytes[i] > (1LL << 30))
      return fail(MSA_ERR_INVALID_ARG, "page_bytes[%d] must be a multiple of 16 up to 2^30", i);
    pc->base[i] = static_cast<uint8_t*>(caches[i]);
    pc->bytes[i] = page_bytes[i];
    pc->chunks[i + 1] = pc->chunks[i] + static_cast<int>((page_bytes[i] + kPgChunk - 1) / kPgChunk);
  }
  return MSA_OK;
}

msa_status_t check_tables(const int32_t* table, const int32_t* lens, const int32_t* ref, int B,
                          int num_pages, int max_pages) {
  if (!table || !aligned16(table))
    return fail(MSA_ERR_INVALID_ARG, "block_table is null or not 16-byte aligned");
  if (!lens || !aligned16(lens))
    return fail(MSA_ERR_INVALID_ARG, "cache_lens is null or not 16-byte aligned");
  if (!ref || !aligned16(ref))
    return fail(MSA_ERR_INVALID_ARG, "ref_count is null or not 16-byte aligned");
  if (B < 1 || num_pages < 1 || max_pages < 1)
    return fail(MSA_ERR_INVALID_ARG, "B, num_pages and max_pages must be >= 1");
  if (max_pages > kMaxSeqlen / kBlock)
    return fail(MSA_ERR_UNSUPPORTED, "max_pages %d above the supported %d", max_pages,
                kMaxSeqlen / kBlock);
  if (num_pages > (1 << 28) || B > (1 << 20))
    return fail(MSA_ERR_UNSUPPORTED, "at most 2^28 pages and 2^20 rows");
  return MSA_OK;
}

struct ExtendWorkspace {
  int2* plan;
  int32_t *free_list, *copy_src, *copy_dst, *n_copies;
};

ExtendWorkspace carve_extend_workspace(WsCursor& ws, int B, int num_pages) {
  ExtendWorkspace w;
  w.plan = ws.take<int2>(B);
  w.free_list = ws.take<int32_t>(num_pages);
  w.copy_src = ws.take<int32_t>(B);
  w.copy_dst = ws.take<int32_t>(B);
  w.n_copies = ws.take<int32_t>(1);
  return w;
}

struct CompactWorkspace {
  int32_t *copy_src, *copy_dst, *n_copies;
};

CompactWorkspace carve_compact_workspace(WsCursor& ws, int num_pages) {
  CompactWorkspace w;
  w.copy_src = ws.take<int32_t>(num_pages);
  w.copy_dst = ws.take<int32_t>(num_pages);
  w.n_copies = ws.take<int32_t>(1);
  return w;
}

msa_status_t launch_copy(const PageCaches& pc, const int32_t* src, const int32_t* dst, int n,
                         const int32_t* n_dev, long long most, int num_pages, int32_t* table,
                         const int32_t* lens, const int32_t* page_map, int B, int max_pages,
                         uint32_t* sw, cudaStream_t stream) {
  // `most`: pairs at most; rows of the table to rewrite count as items too
  long long items = most * pc.chunks[pc.n];
  if (page_map && items < B) items = B;
  if (items < 1) return MSA_OK;
  const int sms = device_sm_count();
  const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);
  MSA_TRY(ensure_smem(pages_copy_kernel, sizeof(CopySmem), "pages_copy_kernel"));
  TraceScope trace_("pages_copy_kernel", stream);
  launch_pdl(pages_copy_kernel, grid, 128, sizeof(CopySmem), stream, pc, src, dst, n, n_dev,
             num_pages, table, lens, page_map, B, max_pages, sw);
  return check_launch("pages_copy_kernel");
}

}  // namespace

}  // namespace msa

using namespace msa;

extern "C" {

msa_status_t msa_pages_fork(const int32_t* src, const int32_t* dst, const int32_t* keep, int n,
                            int32_t* block_table, int32_t* cache_lens, int32_t* ref_count, int B,
                            int num_pages, int max_pages, int32_t* forked, msa_stream_t stream) {
  MSA_REQUIRE_PTR(src);
  MSA_REQUIRE_PTR(dst);
  MSA_REQUIRE_PTR(forked);
  if (keep && !aligned16(keep)) return fail(MSA_ERR_INVALID_ARG, "keep is not 16-byte aligned");
  if (n < 1 || n > (1 << 24)) return fail(MSA_ERR_INVALID_ARG, "n %d outside [1, 2^24]", n);
  MSA_TRY(check_tables(block_table, cache_lens, ref_count, B, num_pages, max_pages));
  uint32_t* sw = nullptr;
  MSA_TRY(status_word(&sw));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool all = static_cast<long long>(n) * max_pages <= kPgOneLaunch;
  {
    TraceScope trace_("pages_fork_claim_kernel", st);
    launch_pdl(pages_fork_claim_kernel, 1, kPgThreads, 0, st, src, dst, keep, n, cache_lens, B,
               max_pages, forked, all, block_table, ref_count, num_pages, sw);
  }
  MSA_TRY(check_launch("pages_fork_claim_kernel"));
  if (all) return MSA_OK;
  {
    TraceScope trace_("pages_fork_kernel", st);
    launch_pdl(pages_fork_kernel, n, 128, 0, st, src, dst, forked, block_table, ref_count,
               num_pages, max_pages, sw);
  }
  return check_launch("pages_fork_kernel");
}

msa_status_t msa_pages_free(const int32_t* rows, const int32_t* keep, int n, int32_t* block_table,
                            int32_t* cache_lens, int32_t* ref_count, int B, int num_pages,
                            int max_pages, int32_t* dropped, msa_stream_t stream) {
  MSA_REQUIRE_PTR(rows);
  MSA_REQUIRE_PTR(dropped);
  if (keep && !aligned16(keep)) return fail(MSA_ERR_INVALID_ARG, "keep is not 16-byte aligned");
  if (n < 1 || n > (1 << 24)) return fail(MSA_ERR_INVALID_ARG, "n %d outside [1, 2^24]", n);
  MSA_TRY(check_tables(block_table, cache_lens, ref_count, B, num_pages, max_pages));
  uint32_t* sw = nullptr;
  MSA_TRY(status_word(&sw));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool all = static_cast<long long>(n) * max_pages <= kPgOneLaunch;
  {
    TraceScope trace_("pages_free_claim_kernel", st);
    launch_pdl(pages_free_claim_kernel, 1, kPgThreads, 0, st, rows, keep, n, cache_lens, B,
               max_pages, dropped, all, block_table, ref_count, num_pages, sw);
  }
  MSA_TRY(check_launch("pages_free_claim_kernel"));
  if (all) return MSA_OK;
  {
    TraceScope trace_("pages_free_kernel", st);
    launch_pdl(pages_free_kernel, n, 128, 0, st, rows, keep, dropped, block_table, ref_count,
               num_pages, max_pages, sw);
  }
  return check_launch("pages_free_kernel");
}

size_t msa_pages_extend_workspace_size(int B, int num_pages) {
  if (B < 1 || num_pages < 1) return 0;
  WsCursor ws(nullptr);
  carve_extend_workspace(ws, B, num_pages);
  return ws.used + 256;
}

msa_status_t msa_pages_extend(const int32_t* add, int32_t* block_table, int32_t* cache_lens,
                              int32_t* ref_count, int B, int num_pages, int max_pages,
                              void* const* caches, const int64_t* page_bytes, int n_caches,
                              int32_t* done, void* workspace, size_t workspace_bytes,
                              msa_stream_t stream) {
  MSA_REQUIRE_PTR(add);
  MSA_REQUIRE_PTR(done);
  MSA_REQUIRE_PTR(workspace);
  MSA_TRY(check_tables(block_table, cache_lens, ref_count, B, num_pages, max_pages));
  PageCaches pc{};
  MSA_TRY(page_caches(caches, page_bytes, n_caches, &pc));
  if (workspace_bytes < msa_pages_extend_workspace_size(B, num_pages))
    return fail(MSA_ERR_INVALID_ARG, "workspace too small");
  WsCursor ws(workspace);
  const ExtendWorkspace w = carve_extend_workspace(ws, B, num_pages);
  uint32_t* sw = nullptr;
  MSA_TRY(status_word(&sw));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope trace_("pages_extend_kernel", st);
    launch_pdl(pages_extend_kernel, 1, kPgThreads, 0, st, add, block_table, cache_lens, ref_count,
               B, num_pages, max_pages, done, w.plan, w.free_list, w.copy_src, w.copy_dst,
               w.n_copies, sw);
  }
  MSA_TRY(check_launch("pages_extend_kernel"));
  return launch_copy(pc, w.copy_src, w.copy_dst, 0, w.n_copies, B, num_pages, nullptr, nullptr,
                     nullptr, 0, max_pages, sw, st);
}

size_t msa_pages_compact_workspace_size(int num_pages) {
  if (num_pages < 1) return 0;
  WsCursor ws(nullptr);
  carve_compact_workspace(ws, num_pages);
  return ws.used + 256;
}

msa_status_t msa_pages_compact(int32_t* block_table, const int32_t* cache_lens,
                               int32_t* ref_count, int B, int num_pages, int max_pages,
                               void* const* caches, const int64_t* page_bytes, int n_caches,
                               int32_t* page_map, int32_t* n_live, void* workspace,
                               size_t workspace_bytes, msa_stream_t stream) {
  MSA_REQUIRE_PTR(page_map);
  MSA_REQUIRE_PTR(n_live);
  MSA_REQUIRE_PTR(workspace);
  MSA_TRY(check_tables(block_table, cache_lens, ref_count, B, num_pages, max_pages));
  PageCaches pc{};
  MSA_TRY(page_caches(caches, page_bytes, n_caches, &pc));
  if (workspace_bytes < msa_pages_compact_workspace_size(num_pages))
    return fail(MSA_ERR_INVALID_ARG, "workspace too small");
  WsCursor ws(workspace);
  const CompactWorkspace w = carve_compact_workspace(ws, num_pages);
  uint32_t* sw = nullptr;
  MSA_TRY(status_word(&sw));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  {
    TraceScope trace_("pages_compact_kernel", st);
    launch_pdl(pages_compact_kernel, 1, kPgThreads, 0, st, ref_count, num_pages, page_map, n_live,
               w.copy_src, w.copy_dst, w.n_copies);
  }
  MSA_TRY(check_launch("pages_compact_kernel"));
  return launch_copy(pc, w.copy_src, w.copy_dst, 0, w.n_copies, num_pages, num_pages, block_table,
                     cache_lens, page_map, B, max_pages, sw, st);
}

msa_status_t msa_pages_copy(const int32_t* src, const int32_t* dst, int n, int num_pages,
                            void* const* caches, const int64_t* page_bytes, int n_caches,
                            msa_stream_t stream) {
  MSA_REQUIRE_PTR(src);
  MSA_REQUIRE_PTR(dst);
  if (n < 1 || num_pages < 1)
    return fail(MSA_ERR_INVALID_ARG, "n and num_pages must be >= 1 (got %d, %d)", n, num_pages);
  PageCaches pc{};
  MSA_TRY(page_caches(caches, page_bytes, n_caches, &pc));
  if (n_caches < 1) return fail(MSA_ERR_INVALID_ARG, "no cache given");
  uint32_t* sw = nullptr;
  MSA_TRY(status_word(&sw));
  return launch_copy(pc, src, dst, n, nullptr, n, num_pages, nullptr, nullptr, nullptr, 0, 1, sw,
                     static_cast<cudaStream_t>(stream));
}

}  // extern "C"
