// Page bookkeeping of a paged cache on the device (dsa_cache_*), and the two
// calls that move rows: dsa_cache_copy_pages and dsa_cache_write.
//
// refs[page] is the number of uses of a page; a page is free when it is 0, so
// there is no free list to keep: a call that needs pages takes the lowest free
// ones, found by counting zeros.  Every plan call (fork, extend, compact) is
// one thread-block cluster: each CTA owns a contiguous slice of the pages,
// counts it, and reads the other CTAs' counts from their shared memory after a
// cluster barrier, which gives each slice its place in the ascending order.
// Results do not depend on the order of the integer atomics.  All or nothing:
// the inputs are checked and the free pages counted before anything is taken;
// a call that cannot be carried out writes its inputs through unchanged and
// sets the status word.
//
// Bound: a few cluster barriers and dependent L2 reads.  Fork, extend and compact
// of 16 sequences and 2048 pages take 5.5, 4.3 and 6.6 us, of 256 sequences and
// 98304 pages 15.6, 9.6 and 27 us; the tables and refs are read at L2 rate.
#include <limits.h>

#include "dsa_common.cuh"

namespace dsa {

bool ext_dev_ctx(DevCtx* c);

namespace cache {

// The plan kernels take kThreads (256, 512 or 1024) as a template argument.
constexpr int kMaxThreads = 1024;
constexpr int kMaxCluster = 8;
constexpr int kMaxSeqs = 8192;

struct Dims {
  int n_seqs, n_pages, R, max_pages;
};

struct Shared {                       // what the other CTAs of the cluster read
  int count, more, bad;
  int warp[kMaxThreads / 32];         // block scans
};

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int ld_peer(const int* local, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(local), rank)) : "memory");
  return v;
}
__device__ __forceinline__ int pages_of(int len, int R) { return (int)(((long long)len + R - 1) / R); }

// exclusive prefix of v over the block and its total (all threads call it)
template <int kThreads>
__device__ __forceinline__ int block_scan(int v, Shared& s, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) s.warp[w] = x;
  __syncthreads();
  const int t = lane < kThreads / 32 ? s.warp[lane] : 0;  // every warp: the sums of all warps
  const int below = __reduce_add_sync(0xffffffffu, lane < w ? t : 0);
  *total = __reduce_add_sync(0xffffffffu, t);
  __syncthreads();
  return x - v + below;
}
// the same for a flag
template <int kThreads>
__device__ __forceinline__ int block_rank(bool yes, Shared& s, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const uint32_t bits = __ballot_sync(0xffffffffu, yes);
  if (lane == 0) s.warp[w] = __popc(bits);
  __syncthreads();
  const int t = lane < kThreads / 32 ? s.warp[lane] : 0;
  const int below = __reduce_add_sync(0xffffffffu, lane < w ? t : 0);
  *total = __reduce_add_sync(0xffffffffu, t);
  __syncthreads();
  return below + __popc(bits & ((1u << lane) - 1u));
}
// total of a thread's counts over the block
template <int kThreads>
__device__ __forceinline__ int block_sum(int v, Shared& s) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int x = __reduce_add_sync(0xffffffffu, v);
  if (lane == 0) s.warp[w] = x;
  __syncthreads();
  const int t = __reduce_add_sync(0xffffffffu, lane < kThreads / 32 ? s.warp[lane] : 0);
  __syncthreads();
  return t;
}

// sums of this CTA's `count` over the lower ranks and over all; any CTA's `bad`
struct Totals {
  int before, all, bad;
};
__device__ __forceinline__ Totals gather_totals(const Shared& s, uint32_t rank, uint32_t n) {
  if (n == 1) return {0, s.count, s.bad};
  const uint32_t lane = threadIdx.x & 31;
  const int c = lane < n ? ld_peer(&s.count, lane) : 0, b = lane < n ? ld_peer(&s.bad, lane) : 0;
  Totals t;
  t.before = __reduce_add_sync(0xffffffffu, lane < rank ? c : 0);
  t.all = __reduce_add_sync(0xffffffffu, c);
  t.bad = __reduce_or_sync(0xffffffffu, (uint32_t)b);
  return t;
}
// all CTAs of the cluster, or the one
__device__ __forceinline__ void sync_all(uint32_t n) {
  if (n == 1) __syncthreads();
  else cluster_sync_all();
}

// pages [lo, hi) of this CTA's slice
__device__ __forceinline__ void slice(int n_pages, uint32_t rank, uint32_t n, int* lo, int* hi) {
  const int per = (n_pages + (int)n - 1) / (int)n;
  const long long a = (long long)per * rank, b = a + per;
  *lo = a < n_pages ? (int)a : n_pages;
  *hi = b < n_pages ? (int)b : n_pages;
}

// f(rank, page) for the pages of [lo, hi) that satisfy `pick`, in ascending
// order, ranks from `first`; stops once the rank reaches `limit`
template <int kThreads, typename P, typename F>
__device__ __forceinline__ void in_order(int lo, int hi, int first, int limit, Shared& s, P pick, F f) {
  for (int base = lo; base < hi && first < limit; base += kThreads) {
    const int p = base + threadIdx.x;
    const bool yes = p < hi && pick(p);
    int n;
    const int at = first + block_rank<kThreads>(yes, s, &n);
    if (yes && at < limit) f(at, p);
    first += n;
  }
}
template <int kThreads, typename P>
__device__ __forceinline__ int count_if(int lo, int hi, Shared& s, P pick) {
  int n = 0;
  for (int p = lo + threadIdx.x; p < hi; p += kThreads) n += pick(p) ? 1 : 0;
  return block_sum<kThreads>(n, s);
}

// ---------------------------------- fork ----------------------------------
// table row i <- old row parent[i].  The first child (lowest i) of a parent
// keeps the parent's partial last page, the other children need a page of
// their own for it.
template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1)
    fork_kernel(Dims d, const int32_t* __restrict__ parent, const int32_t* __restrict__ table,
                const int32_t* __restrict__ lens, const int32_t* __restrict__ refs,
                int32_t* __restrict__ table_out, int32_t* __restrict__ lens_out, int32_t* __restrict__ refs_out,
                int32_t* __restrict__ copies, int32_t* __restrict__ n_copies, DevCtx c) {
  __shared__ Shared s;
  extern __shared__ int dyn[];
  int* first = dyn;                   // [n_seqs] lowest child of each parent
  int* needy = dyn + d.n_seqs;        // [n_seqs] sequences that need a page, ascending
  int* par = dyn + 2 * d.n_seqs;      // [n_seqs] parent, lens
  int* len = dyn + 3 * d.n_seqs;
  let_next_launch();
  wait_for_earlier();
  const uint32_t rank = cluster_ctarank(), nc = cluster_nctarank();
  const int n = d.n_seqs, R = d.R, tid = threadIdx.x;
  int lo, hi;
  slice(d.n_pages, rank, nc, &lo, &hi);
  if (tid == 0) s.bad = 0;
  for (int i = tid; i < n; i += kThreads) first[i] = INT_MAX;
  for (int p = lo + tid; p < hi; p += kThreads) refs_out[p] = refs[p];
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const int p = parent[i], l = lens[i];
    par[i] = p;
    len[i] = l;
    if (p < -1 || p >= n || l < 0 || l > (long long)d.max_pages * R) s.bad = 1;
    else if (p >= 0) atomicMin(&first[p], i);
  }
  __syncthreads();
  const bool bad_rows = s.bad != 0;   // the same in every CTA
  sync_all(nc);                 // refs_out initialised
  auto need_page = [&](int i) {
    const int p = par[i];
    return p >= 0 && first[p] != i && len[p] % R != 0;
  };
  if (!bad_rows) {
    // 256 table entries per warp step; uses that do not change are not counted
    const int nch = (d.max_pages + 255) / 256, lane = tid & 31;
    const long long items = (long long)n * nch;
    for (long long it = (long long)rank * (kThreads / 32) + (tid >> 5); it < items;
         it += (long long)nc * (kThreads / 32)) {
      const int i = (int)(it / nch), j0 = (int)(it % nch) * 256;
      const int p = par[i];
      const int po = pages_of(len[i], R), pn = p >= 0 ? pages_of(len[p], R) : 0;
      const int hole = need_page(i) ? pn - 1 : -1;
      int a[8], v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int j = j0 + 32 * u + lane;
        a[u] = j < po ? table[(long long)i * d.max_pages + j] : -1;
        v[u] = j < pn ? table[(long long)p * d.max_pages + j] : -1;
        if ((j < po && (a[u] < 0 || a[u] >= d.n_pages)) || (j < pn && (v[u] < 0 || v[u] >= d.n_pages))) {
          s.bad = 1;
          a[u] = v[u] = -1;
        }
        if (j == hole) v[u] = -1;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int j = j0 + 32 * u + lane;
        if (j >= d.max_pages) continue;
        table_out[(long long)i * d.max_pages + j] = v[u];
        if (a[u] != v[u]) {
          if (a[u] >= 0) atomicAdd(refs_out + a[u], -1);
          if (v[u] >= 0) atomicAdd(refs_out + v[u], 1);
        }
      }
      if (j0 == 0 && lane == 0) lens_out[i] = p >= 0 ? len[p] : 0;
    }
  }
  // the sequences that need a page, in order
  int n_need = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + tid;
    const bool yes = !bad_rows && i < n && need_page(i);
    int t;
    const int at = block_rank<kThreads>(yes, s, &t);
    if (yes) needy[n_need + at] = i;
    n_need += t;
  }
  sync_all(nc);                 // every use counted
  {
    bool neg = false;
    const int free_pages = count_if<kThreads>(lo, hi, s, [&](int p) {
      const int r = __ldcg(refs_out + p);
      neg |= r < 0;
      return r == 0;
    });
    if (neg) s.bad = 1;
    if (tid == 0) s.count = free_pages;
  }
  sync_all(nc);
  const Totals t = gather_totals(s, rank, nc);
  const bool bad = t.bad != 0, fail = bad || n_need > t.all;
  if (!fail) {
    in_order<kThreads>(
        lo, hi, t.before, n_need, s, [&](int p) { return __ldcg(refs_out + p) == 0; },
        [&](int k, int page) {
          const int i = needy[k], p = par[i], last = pages_of(len[p], R) - 1;
          table_out[(long long)i * d.max_pages + last] = page;
          refs_out[page] = 1;
          copies[3 * k] = table[(long long)p * d.max_pages + last];
          copies[3 * k + 1] = page;
          copies[3 * k + 2] = len[p] % R;
        });
    if (rank == 0 && tid == 0) *n_copies = n_need;
  } else {
    for (int p = lo + tid; p < hi; p += kThreads) refs_out[p] = refs[p];
    const long long e = (long long)n * d.max_pages;
    for (long long i = (long long)rank * kThreads + tid; i < e; i += (long long)nc * kThreads) table_out[i] = table[i];
    if (rank == 0) {
      for (int i = tid; i < n; i += kThreads) lens_out[i] = len[i];
      if (tid == 0) {
        *n_copies = 0;
        set_status(c, bad ? DSA_ERR_INDEX : DSA_ERR_PAGES);
      }
    }
  }
  sync_all(nc);                 // the others may still read this CTA's counts
}

// --------------------------------- extend ---------------------------------
template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1)
    extend_kernel(Dims d, const int32_t* __restrict__ n_new, int32_t* table, const int32_t* lens, const int32_t* refs,
                  int32_t* lens_out, int32_t* refs_out, int32_t* __restrict__ slots, int n_slots, DevCtx c) {
  __shared__ Shared s;
  extern __shared__ int dyn[];
  int* len = dyn;                     // [n_seqs] rows before the call
  int* prow = dyn + d.n_seqs;         // [n_seqs + 1] exclusive prefix of the new rows
  int* ppage = prow + d.n_seqs + 1;   // [n_seqs + 1] exclusive prefix of the new pages
  let_next_launch();
  wait_for_earlier();
  const uint32_t rank = cluster_ctarank(), nc = cluster_nctarank();
  const int n = d.n_seqs, R = d.R, tid = threadIdx.x;
  int lo, hi;
  slice(d.n_pages, rank, nc, &lo, &hi);
  if (tid == 0) s.bad = 0;
  __syncthreads();
  int rows = 0, pages = 0;            // running totals
  long long sum = 0;                  // of the new rows, without overflow
  for (int base = 0; base < n; base += kThreads) {
    const int i = base + tid;
    int a = 0, b = 0;
    if (i < n) {
      const int l = lens[i], m = n_new[i];
      len[i] = l;
      if (l < 0 || m < 0 || (long long)l + m > (long long)d.max_pages * R || m > n_slots) {
        s.bad = 1;
      } else {
        a = m;
        b = pages_of(l + m, R) - pages_of(l, R);
        if (m > 0 && l % R != 0) {    // rows go into the last page: it must be this sequence's alone
          const int page = table[(long long)i * d.max_pages + l / R];
          if (page < 0 || page >= d.n_pages || refs[page] != 1) s.bad = 1;
        }
      }
    }
    int ta, tb;
    const int ea = block_scan<kThreads>(a, s, &ta), eb = block_scan<kThreads>(b, s, &tb);
    if (i < n) {
      prow[i] = rows + ea;
      ppage[i] = pages + eb;
    }
    sum += ta;                        // ta <= 1024 * 2^20
    rows += ta;
    pages += tb;
    if (sum > n_slots) {
      if (tid == 0) s.bad = 1;
      rows = 0;
      pages = 0;
      sum = (long long)n_slots + 1;
    }
  }
  if (tid == 0) {
    prow[n] = rows;
    ppage[n] = pages;
  }
  __syncthreads();
  {
    bool neg = false;
    const int free_pages = count_if<kThreads>(lo, hi, s, [&](int p) {
      neg |= refs[p] < 0;
      return refs[p] == 0;
    });
    if (neg) s.bad = 1;
    if (tid == 0) s.count = free_pages;
  }
  sync_all(nc);
  const Totals t = gather_totals(s, rank, nc);
  const bool bad = t.bad != 0, fail = bad || pages > t.all;
  if (refs_out != refs) {
    for (int p = lo + tid; p < hi; p += kThreads) refs_out[p] = refs[p];
    __syncthreads();
  }
  // the sequence whose range of the prefix holds k
  auto find = [&](const int* prefix, int k) {
    int a = 0, b = n;                 // prefix[a] <= k < prefix[b]
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if (prefix[mid] <= k) a = mid;
      else b = mid;
    }
    return a;
  };
  if (!fail) {
    in_order<kThreads>(
        lo, hi, t.before, pages, s, [&](int p) { return refs_out[p] == 0; },
        [&](int k, int page) {
          const int i = find(ppage, k);
          table[(long long)i * d.max_pages + pages_of(len[i], R) + (k - ppage[i])] = page;
          refs_out[page] = 1;
        });
  }
  sync_all(nc);                 // the table is complete; every CTA has its lens
  const int total = fail ? 0 : rows;
  for (int k = (int)rank * kThreads + tid; k < n_slots; k += (int)nc * kThreads) {
    int slot = -1;
    if (k < total) {
      const int i = find(prow, k), pos = len[i] + (k - prow[i]);
      slot = __ldcg(table + (long long)i * d.max_pages + pos / R) * R + pos % R;
    }
    slots[k] = slot;
  }
  if (rank == 0) {
    for (int i = tid; i < n; i += kThreads) lens_out[i] = len[i] + (fail ? 0 : prow[i + 1] - prow[i]);
    if (tid == 0 && fail) set_status(c, bad ? DSA_ERR_INDEX : DSA_ERR_PAGES);
  }
}

// --------------------------------- compact ---------------------------------
// n_live pages are in use: those at n_live and above move, in ascending order,
// into the free ids below n_live, in ascending order.
template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1)
    compact_kernel(Dims d, const int32_t* __restrict__ table, const int32_t* __restrict__ lens,
                   const int32_t* __restrict__ refs, int32_t* __restrict__ table_out, int32_t* __restrict__ refs_out,
                   int32_t* __restrict__ page_map, int32_t* __restrict__ copies, int32_t* __restrict__ n_copies,
                   DevCtx c) {
  __shared__ Shared s;
  let_next_launch();
  wait_for_earlier();
  const uint32_t rank = cluster_ctarank(), nc = cluster_nctarank();
  const int n = d.n_seqs, R = d.R, tid = threadIdx.x, lane = tid & 31;
  int lo, hi;
  slice(d.n_pages, rank, nc, &lo, &hi);
  if (tid == 0) s.bad = 0;
  __syncthreads();
  // f(table offset of entry j0 of a sequence, j0, entries held) for every 256
  // entries of the table, one warp each; lane l takes entries j0 + l + 32 u
  const int nch = (d.max_pages + 255) / 256;
  auto entries = [&](auto f) {
    const int items = n * nch;        // n * max_pages < 2^31
    for (int it = (int)rank * (kThreads / 32) + (tid >> 5); it < items; it += (int)nc * (kThreads / 32)) {
      const int i = it / nch, j0 = (it - i * nch) * 256, len = lens[i];
      const bool ok = len >= 0 && len <= (long long)d.max_pages * R;
      if (!ok) s.bad = 1;
      f((long long)i * d.max_pages + j0, j0, ok ? pages_of(len, R) : 0);
    }
  };
  entries([&](long long e, int j0, int held) {
    int p[8], r[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) p[u] = j0 + 32 * u + lane < held ? table[e + 32 * u + lane] : -2;
    bool wrong = false;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool in = p[u] >= 0 && p[u] < d.n_pages;
      r[u] = in ? refs[p[u]] : (p[u] == -2 && j0 + 32 * u + lane >= held ? 1 : 0);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) wrong |= r[u] <= 0;
    if (wrong) s.bad = 1;
  });
  {
    bool neg = false;
    const int live = count_if<kThreads>(lo, hi, s, [&](int p) {
      neg |= refs[p] < 0;
      return refs[p] > 0;
    });
    if (neg) s.bad = 1;
    if (tid == 0) s.count = live;
  }
  sync_all(nc);
  const Totals t = gather_totals(s, rank, nc);
  const int n_live = t.all, live_here = s.count;
  const bool bad = t.bad != 0;
  sync_all(nc);                       // counts read before they are replaced
  // free ids below n_live and used ones above: here, in the lower slices, in all
  const int mid = n_live < lo ? lo : (n_live > hi ? hi : n_live);  // slice = [lo, mid) low, [mid, hi) high
  const int live_low = count_if<kThreads>(lo, mid, s, [&](int p) { return refs[p] > 0; });
  if (tid == 0) {
    s.count = (mid - lo) - live_low;
    s.more = live_here - live_low;
  }
  sync_all(nc);
  int hole = 0, mover = 0, H = 0;     // ranks of this slice's first hole and mover; holes in all
  if (nc == 1) {
    H = s.count;
  } else {
    const uint32_t l = lane;
    const int a = l < nc ? ld_peer(&s.count, l) : 0, b = l < nc ? ld_peer(&s.more, l) : 0;
    hole = __reduce_add_sync(0xffffffffu, l < rank ? a : 0);
    mover = __reduce_add_sync(0xffffffffu, l < rank ? b : 0);
    H = __reduce_add_sync(0xffffffffu, a);
  }
  if (bad) H = 0;
  for (int base = lo; base < hi && H > 0; base += kThreads) {
    const int p = base + tid;
    const bool used = p < hi && refs[p] > 0;
    const bool is_hole = p < mid && !used, is_mover = p >= mid && used;
    int n;
    const int kh = hole + block_rank<kThreads>(is_hole, s, &n);
    hole += n;
    const int km = mover + block_rank<kThreads>(is_mover, s, &n);
    mover += n;
    if (is_hole) copies[3 * kh + 1] = p;
    if (is_mover) {
      copies[3 * km] = p;
      copies[3 * km + 2] = R;
    }
  }
  sync_all(nc);                 // the list is complete
  for (int p = lo + tid; p < hi; p += kThreads) {
    const int r = refs[p];
    // ids that move are filled in by their copy below
    if (bad || p < n_live ? (bad || r > 0) : r == 0) {
      page_map[p] = r > 0 ? p : -1;
      refs_out[p] = r;
    } else if (p < n_live) {
      page_map[p] = -1;               // a hole: refs_out comes from the page that moves in
    } else {
      refs_out[p] = 0;                // moves away: page_map comes from its copy
    }
  }
  for (int k = (int)rank * kThreads + tid; k < H; k += (int)nc * kThreads) {
    const int src = __ldcg(copies + 3 * k), dst = __ldcg(copies + 3 * k + 1);
    page_map[src] = dst;
    refs_out[dst] = refs[src];
  }
  if (rank == 0 && tid == 0) {
    *n_copies = H;
    if (bad) set_status(c, DSA_ERR_INDEX);
  }
  sync_all(nc);                 // the map is complete
  entries([&](long long e, int j0, int held) {
    int p[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = j0 + 32 * u + lane;
      p[u] = j < (bad ? d.max_pages : held) ? table[e + 32 * u + lane] : -1;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (!bad && p[u] >= 0) p[u] = __ldcg(page_map + p[u]);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (j0 + 32 * u + lane < d.max_pages) table_out[e + 32 * u + lane] = p[u];
  });
}

// ------------------------------- copies / writes -------------------------------
struct Pool {
  uint8_t* base;
  long long layer_stride, page_stride, row_bytes;
  int n_layers;
};

// streamed once: past L1
struct alignas(32) Wide {
  uint32_t w[8];
};
template <typename V>
__device__ __forceinline__ V ld_once(const V* p) {
  return __ldcs(p);
}
template <>
__device__ __forceinline__ Wide ld_once<Wide>(const Wide* p) {
  Wide v;
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                 "=r"(v.w[7])
               : "l"(p)
               : "memory");
  return v;
}
template <typename V>
__device__ __forceinline__ void st_once(V* p, const V& v) {
  __stcs(p, v);
}
template <>
__device__ __forceinline__ void st_once<Wide>(Wide* p, const Wide& v) {
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]),
               "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7])
               : "memory");
}

template <typename V>
__device__ __forceinline__ void copy_span(uint8_t* dst, const uint8_t* src, long long bytes, int t, int nt) {
  const long long nv = bytes / (long long)sizeof(V);
  const V* a = reinterpret_cast<const V*>(src);
  V* b = reinterpret_cast<V*>(dst);
  for (long long i = t; i < nv; i += 4ll * nt) {  // four loads in flight per thread
    V x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + (long long)u * nt < nv) x[u] = ld_once<V>(a + i + (long long)u * nt);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + (long long)u * nt < nv) st_once<V>(b + i + (long long)u * nt, x[u]);
  }
  for (long long j = nv * (long long)sizeof(V) + t; j < bytes; j += nt) dst[j] = src[j];
}

constexpr int kCopyThreads = 256;

// item = (copy, layer, piece of the page).  Bound: HBM.  3,955 pages of 73,728
// bytes: 91 us, 6.4 TB/s read and written (96 % of the copy rate measured on this
// GPU); with 16-byte vectors 96 us.
template <typename V>
__global__ void __launch_bounds__(kCopyThreads)
    copy_pages_kernel(Dims d, Pool pool, const int32_t* __restrict__ copies, const int32_t* __restrict__ n_copies,
                      int max_copies, int pieces, long long piece_bytes, DevCtx c) {
  let_next_launch();
  wait_for_earlier();
  int n = *n_copies;
  if (n > max_copies) n = max_copies;
  const long long per = (long long)pool.n_layers * pieces, items = (long long)n * per;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int k = (int)(it / per), rem = (int)(it % per), layer = rem / pieces, piece = rem % pieces;
    const int src = copies[3 * k], dst = copies[3 * k + 1], rows = copies[3 * k + 2];
    if (src < 0 || src >= d.n_pages || dst < 0 || dst >= d.n_pages || rows < 0 || rows > d.R) {
      if (threadIdx.x == 0) set_status(c, DSA_ERR_INDEX);
      continue;
    }
    const long long begin = piece * piece_bytes, end = rows * pool.row_bytes;
    if (begin >= end) continue;
    const long long bytes = end - begin < piece_bytes ? end - begin : piece_bytes;
    uint8_t* base = pool.base + layer * pool.layer_stride + begin;
    copy_span<V>(base + dst * pool.page_stride, base + src * pool.page_stride, bytes, threadIdx.x, kCopyThreads);
  }
}

// One warp per (layer, row).  Bound: latency for a step's rows (48 rows of 1152
// bytes 1.8 us), HBM for many (65,536 rows 26 us, 5.9 TB/s).
template <typename V>
__global__ void __launch_bounds__(kCopyThreads)
    write_rows_kernel(Dims d, Pool pool, const uint8_t* __restrict__ rows, long long rows_layer_stride, int n_src,
                      const int32_t* __restrict__ slots, const int32_t* __restrict__ row_index, int n_rows, DevCtx c) {
  let_next_launch();
  wait_for_earlier();
  const long long items = (long long)n_rows * pool.n_layers;
  const int lane = threadIdx.x & 31;
  for (long long it = blockIdx.x * (long long)(kCopyThreads / 32) + (threadIdx.x >> 5); it < items;
       it += (long long)gridDim.x * (kCopyThreads / 32)) {
    const int layer = (int)(it / n_rows), i = (int)(it % n_rows);
    const int slot = slots[i];
    if (slot == -1) continue;
    const int src = row_index ? row_index[i] : i;
    if (slot < 0 || slot >= (long long)d.n_pages * d.R || src < 0 || src >= n_src) {
      if (lane == 0) set_status(c, DSA_ERR_INDEX);
      continue;
    }
    copy_span<V>(pool.base + layer * pool.layer_stride + (slot / d.R) * pool.page_stride + (slot % d.R) * pool.row_bytes,
                 rows + layer * rows_layer_stride + src * pool.row_bytes, pool.row_bytes, lane, 32);
  }
}

// --------------------------------- host side ---------------------------------
static int check(const dsa_cache* p, Dims* d) {
  if (!p) return DSA_ERR_INVALID_ARG;
  if (p->n_seqs < 1 || p->n_pages < 1 || p->page_rows < 1 || p->max_pages < 1) return DSA_ERR_INVALID_ARG;
  if (p->n_seqs > kMaxSeqs || p->n_pages > (1ll << 30) || p->page_rows > (1ll << 30) || p->max_pages > (1ll << 30) ||
      p->n_pages * p->page_rows >= (1ll << 31) || p->max_pages * p->page_rows >= (1ll << 31) ||
      p->n_seqs * p->max_pages >= (1ll << 31))
    return DSA_ERR_UNSUPPORTED;
  d->n_seqs = (int)p->n_seqs;
  d->n_pages = (int)p->n_pages;
  d->R = (int)p->page_rows;
  d->max_pages = (int)p->max_pages;
  return DSA_OK;
}
static bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}
// int32 arrays: all there, 4-byte aligned
template <typename... P>
static bool ints(const P*... p) {
  return ((p != nullptr && ((uintptr_t)p & 3u) == 0) && ...);
}

// One CTA while the work is small (a cluster barrier costs more than the other
// CTAs save), else a cluster of eight.  What counts is how often a warp of the one
// CTA goes round: over the steps of 256 table entries (fork, compact) and over the
// pages, in blocks of 1024.  One CTA against eight, us, by steps and pages:
//    16 /  2048: fork  5.9 /  7.8, extend 5.2 / 6.5, compact  6.4 / 10.2
//    32 /  6144:       8.1 /  9.2,        5.7 / 6.8,         11.0 / 11.7
//    64 / 12288:      11.0 / 10.0,        6.4 / 7.5,         17.9 / 13.5
//   256 /  2691:      20.5 /  8.7,        7.0 / 7.6,         21.1 / 10.9
//   128 / 16268:      22.7 / 11.7,       11.9 / 9.1,         29.7 / 14.7
struct Shape {
  int ctas, threads;
};
static int pow2_from(long long x, int lo, int hi) {
  int p = lo;
  while (p < x && p < hi) p *= 2;
  return p;
}
static Shape shape(const Dims& d, int alone_steps, int alone_pages) {
  const long long steps = (long long)d.n_seqs * ((d.max_pages + 255) / 256);
  if (steps > alone_steps || d.n_pages > alone_pages) return {kMaxCluster, kMaxThreads};
  // a warp for each step, but a barrier of few warps is faster: 256, 512, 1024 threads
  // take, us, by steps and pages (extend: by pages; 256 sequences whose free pages are
  // the last of 2691 8.4 with 512, 7.0 with 1024)
  //   4 /   38: fork 4.5, 4.8, 5.0                        extend 3.2, 3.4, 3.7
  //  16 /  512:                     compact 6.1, 4.6, 5.0
  //  16 / 2048: fork 6.5, 5.4, 5.9, compact 8.8, 6.6, 6.4, extend 4.4, 4.6, 5.2
  //  32 / 6144: fork 11.2, 8.6, 8.1                       extend 5.5, 5.4, 5.7
  return {1, 32 * pow2_from(alone_steps == INT_MAX ? d.n_pages / 128 : steps, 8, 32)};
}
template <typename... A, typename... B>
static int launch_plan(void (*k256)(A...), void (*k512)(A...), void (*k1024)(A...), Shape sh, size_t smem,
                       cudaStream_t st, B... args) {
  auto kernel = sh.threads == 256 ? k256 : sh.threads == 512 ? k512 : k1024;
  // (what a kernel may have without asking for more includes its static part)
  constexpr size_t kStatic = 1024;
  static_assert(sizeof(Shared) <= kStatic, "static shared memory of the plan kernels");
  if (smem + kStatic > 48 * 1024 &&
      !cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)))
    return DSA_ERR_CUDA;
  return launch_programmatic(kernel, dim3(sh.ctas), dim3(sh.threads), smem, st, sh.ctas, args...) ? DSA_OK
                                                                                                  : DSA_ERR_CUDA;
}

static int check_pool(const dsa_cache* p, const dsa_pool* pool, Pool* o) {
  if (!pool || !pool->base) return DSA_ERR_INVALID_ARG;
  if (pool->n_layers < 1 || pool->row_bytes < 1) return DSA_ERR_INVALID_ARG;
  if (pool->n_layers > (1 << 20) || pool->row_bytes > (1ll << 30) ||
      p->page_rows * pool->row_bytes > (1ll << 40))
    return DSA_ERR_UNSUPPORTED;
  // pages must not run into each other: layers outside pages, or pages outside layers
  const long long page = p->page_rows * pool->row_bytes, lim = 1ll << 46;
  if (pool->page_stride < 0 || pool->layer_stride < 0) return DSA_ERR_INVALID_ARG;
  if (pool->page_stride > lim / p->n_pages || pool->layer_stride > lim / pool->n_layers) return DSA_ERR_UNSUPPORTED;
  const bool one_layer = pool->n_layers == 1, one_page = p->n_pages == 1;
  const bool layers_outside = (one_page || pool->page_stride >= page) &&
                              (one_layer || pool->layer_stride >= (p->n_pages - 1) * pool->page_stride + page);
  const bool pages_outside = (one_layer || pool->layer_stride >= page) &&
                             (one_page || pool->page_stride >= (pool->n_layers - 1) * pool->layer_stride + page);
  if (!layers_outside && !pages_outside) return DSA_ERR_INVALID_ARG;
  o->base = (uint8_t*)pool->base;
  o->layer_stride = pool->layer_stride;
  o->page_stride = pool->page_stride;
  o->row_bytes = pool->row_bytes;
  o->n_layers = (int)pool->n_layers;
  return DSA_OK;
}
// widest of 16, 4 and 1 bytes that every listed address and stride allows
static int vector_bytes(uintptr_t bits) { return (bits & 15) == 0 ? 16 : (bits & 3) == 0 ? 4 : 1; }
static int sm_count() {
  int dev = 0, sms = 0;
  if (!cuda_ok(cudaGetDevice(&dev)) || !cuda_ok(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)))
    return 0;
  return sms;
}

}  // namespace cache
}  // namespace dsa

using namespace dsa;
using namespace dsa::cache;

extern "C" {

int dsa_cache_fork(const dsa_cache* p, const int32_t* parent, const int32_t* table, const int32_t* lens,
                   const int32_t* refs, int32_t* table_out, int32_t* lens_out, int32_t* refs_out, int32_t* copies,
                   int32_t* n_copies, dsa_stream_t stream) {
  Dims d;
  int rc = check(p, &d);
  if (rc) return rc;
  if (!ints(parent, table, lens, refs, table_out, lens_out, refs_out, copies, n_copies)) return DSA_ERR_INVALID_ARG;
  const size_t nt = (size_t)d.n_seqs * d.max_pages * 4, ns = (size_t)d.n_seqs * 4, np = (size_t)d.n_pages * 4;
  if (overlap(table, nt, table_out, nt) || overlap(lens, ns, lens_out, ns) || overlap(refs, np, refs_out, np) ||
      overlap(parent, ns, lens_out, ns))
    return DSA_ERR_INVALID_ARG;
  DevCtx c;
  if (!ext_dev_ctx(&c)) return DSA_ERR_CUDA;
  return launch_plan(fork_kernel<256>, fork_kernel<512>, fork_kernel<1024>, shape(d, 48, 12288), 4 * ns,
                     (cudaStream_t)stream, d, parent, table, lens, refs, table_out, lens_out, refs_out, copies,
                     n_copies, c);
}

int dsa_cache_extend(const dsa_cache* p, const int32_t* n_new, int32_t* table, const int32_t* lens,
                     const int32_t* refs, int32_t* lens_out, int32_t* refs_out, int32_t* slots, int64_t n_slots,
                     dsa_stream_t stream) {
  Dims d;
  int rc = check(p, &d);
  if (rc) return rc;
  if (!ints(n_new, table, lens, refs, lens_out, refs_out, slots)) return DSA_ERR_INVALID_ARG;
  if (n_slots < 1) return DSA_ERR_INVALID_ARG;
  if (n_slots > (1ll << 20)) return DSA_ERR_UNSUPPORTED;
  const size_t ns = (size_t)d.n_seqs * 4, np = (size_t)d.n_pages * 4;
  // in place or apart, not shifted
  if ((lens != lens_out && overlap(lens, ns, lens_out, ns)) || (refs != refs_out && overlap(refs, np, refs_out, np)))
    return DSA_ERR_INVALID_ARG;
  DevCtx c;
  if (!ext_dev_ctx(&c)) return DSA_ERR_CUDA;
  return launch_plan(extend_kernel<256>, extend_kernel<512>, extend_kernel<1024>, shape(d, INT_MAX, 12288), 3 * ns + 8,
                     (cudaStream_t)stream, d, n_new, table, lens, refs, lens_out, refs_out, slots, (int)n_slots, c);
}

int dsa_cache_compact(const dsa_cache* p, const int32_t* table, const int32_t* lens, const int32_t* refs,
                      int32_t* table_out, int32_t* refs_out, int32_t* page_map, int32_t* copies, int32_t* n_copies,
                      dsa_stream_t stream) {
  Dims d;
  int rc = check(p, &d);
  if (rc) return rc;
  if (!ints(table, lens, refs, table_out, refs_out, page_map, copies, n_copies)) return DSA_ERR_INVALID_ARG;
  const size_t nt = (size_t)d.n_seqs * d.max_pages * 4, np = (size_t)d.n_pages * 4;
  if (overlap(table, nt, table_out, nt) || overlap(refs, np, refs_out, np) || overlap(refs, np, page_map, np))
    return DSA_ERR_INVALID_ARG;
  DevCtx c;
  if (!ext_dev_ctx(&c)) return DSA_ERR_CUDA;
  return launch_plan(compact_kernel<256>, compact_kernel<512>, compact_kernel<1024>, shape(d, 32, 8192), 0,
                     (cudaStream_t)stream, d, table, lens, refs, table_out, refs_out, page_map, copies, n_copies, c);
}

int dsa_cache_copy_pages(const dsa_cache* p, const dsa_pool* pool, const int32_t* copies, const int32_t* n_copies,
                         int64_t max_copies, dsa_stream_t stream) {
  Dims d;
  int rc = check(p, &d);
  if (rc) return rc;
  Pool o;
  rc = check_pool(p, pool, &o);
  if (rc) return rc;
  if (!ints(copies, n_copies) || max_copies < 0 || max_copies > (1ll << 30)) return DSA_ERR_INVALID_ARG;
  if (max_copies == 0) return DSA_OK;
  DevCtx c;
  if (!ext_dev_ctx(&c)) return DSA_ERR_CUDA;
  const int sms = sm_count();
  if (sms <= 0) return DSA_ERR_CUDA;
  const long long page = (long long)d.R * o.row_bytes;
  const uintptr_t bits = (uintptr_t)o.base | (uintptr_t)o.page_stride | (uintptr_t)o.layer_stride;
  const int vb = (bits & 31) == 0 ? 32 : vector_bytes(bits);
  const long long piece = 16384ll;    // a multiple of every vector width
  const long long pieces = (page + piece - 1) / piece;
  if (pieces * o.n_layers > (1ll << 30)) return DSA_ERR_UNSUPPORTED;
  const long long most = max_copies * pieces * o.n_layers;
  const int grid = (int)(most < 8ll * sms ? most : 8ll * sms);
  auto kernel = vb == 32   ? copy_pages_kernel<Wide>
                : vb == 16 ? copy_pages_kernel<uint4>
                : vb == 4  ? copy_pages_kernel<uint32_t>
                           : copy_pages_kernel<uint8_t>;
  return launch_programmatic(kernel, dim3(grid), dim3(kCopyThreads), 0, (cudaStream_t)stream, 1, d, o, copies, n_copies,
                             (int)max_copies, (int)pieces, piece, c)
             ? DSA_OK
             : DSA_ERR_CUDA;
}

int dsa_cache_write(const dsa_cache* p, const dsa_pool* pool, const void* rows, int64_t n_src,
                    int64_t rows_layer_stride, const int32_t* slots, const int32_t* row_index, int64_t n_rows,
                    dsa_stream_t stream) {
  Dims d;
  int rc = check(p, &d);
  if (rc) return rc;
  Pool o;
  rc = check_pool(p, pool, &o);
  if (rc) return rc;
  if (!rows || !ints(slots) || (row_index && !ints(row_index)) || n_src < 1 || n_rows < 0 || rows_layer_stride < 0)
    return DSA_ERR_INVALID_ARG;
  if (n_src > (1ll << 30) || n_rows > (1ll << 30)) return DSA_ERR_UNSUPPORTED;
  if (n_rows == 0) return DSA_OK;
  DevCtx c;
  if (!ext_dev_ctx(&c)) return DSA_ERR_CUDA;
  const int sms = sm_count();
  if (sms <= 0) return DSA_ERR_CUDA;
  const int vb = vector_bytes((uintptr_t)o.base | (uintptr_t)o.page_stride | (uintptr_t)o.layer_stride |
                              (uintptr_t)o.row_bytes | (uintptr_t)rows | (uintptr_t)rows_layer_stride);
  const long long most = (n_rows * o.n_layers + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
  const int grid = (int)(most < 8ll * sms ? most : 8ll * sms);
  auto kernel = vb == 16 ? write_rows_kernel<uint4> : vb == 4 ? write_rows_kernel<uint32_t> : write_rows_kernel<uint8_t>;
  return launch_programmatic(kernel, dim3(grid), dim3(kCopyThreads), 0, (cudaStream_t)stream, 1, d, o,
                             (const uint8_t*)rows, rows_layer_stride, (int)n_src, slots, row_index, (int)n_rows, c)
             ? DSA_OK
             : DSA_ERR_CUDA;
}

}  // extern "C"
