// Bookkeeping of a paged KV cache on the device: rows that grow, shrink or
// end (resize), rows that start as copies of others (fork), and the live
// pages moved to the front of the pool (compact), with the pages' data moved
// along in every layer.
//
// State.  refs[p] counts the page-table entries that hold page p; a page with
// refs[p] <= 0 is free.  There is no free list to keep: a call that needs m
// pages takes the m lowest free ones, in the order of its rows, so the result
// does not depend on timing.
//
// Split.  Each call is two launches.  The tables are a few hundred kilobytes
// at most, and every step of the work depends on the one before (release,
// count, rank, assign), so they go to one cluster of eight CTAs whose steps
// are separated by cluster barriers (hardware barriers, no spinning), with
// counts exchanged through distributed shared memory.  The pages themselves
// are megabytes, so a second kernel on the whole GPU, launched as a
// programmatic dependent, copies them (and, for a fork, the shared entries;
// for a compaction, every entry of the table).
//
// Ranking.  Each warp of the cluster owns a run of pages and turns its
// refs into one bit per page by ballots kept in shared memory; popcounts
// summed over warps and CTAs give every page its rank among the free (or
// live) ones without reading refs a second time.  A release that leaves a
// page unheld clears its bit where it stands, in another CTA if need be.
//
// Measured (one GB300, device time in a graph).  The bookkeeping kernel is a
// chain of dependent reads and three or four cluster barriers, bound by their
// latency: 6.4 us for a decode step of 64 rows over 65,792 pages, launch
// included.  Rows of more than 512 pages are walked by whole CTAs, and by
// several blocks of the finishing kernel: with a warp (a block) a row, one row
// of 65,536 pages took 527 us to grow, 1,155 to free and 64 to fork, now 32,
// 84 and 15; calls on short rows pay 0.4 to 0.8 us for it.  The scan of the
// counts grows with the pool: a decode step of 64 rows takes 7.4 us over
// 65,792 pages, 20 over 2^20 and 35 over 2^21.  The finishing kernel is bound
// by bytes: a compaction of 16,384 pages that moves 3,932 of 64 KB (515 MB
// read and written) takes 84.3 us in all, 91 % of a copy's measured rate, with
// 32 blocks for every SM (8: 90.5 us).
#include "attn_internal.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kPage = 16;
constexpr int kCtas = 8;  // the portable cluster size
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;  // 16-byte vectors in flight per thread
// Table entries of a row past which a whole CTA walks them.  64 rows grown and
// freed in turn: of 200 pages 10.0 us by warps, 11.3 by CTAs; of 600 pages
// 17.8 and 11.9.  The two meet between 200 and 400.
constexpr int kLong = 512;
constexpr int kAtOnce = 4;    // table entries in flight per thread
constexpr int kSegment = kCopyThreads * kAtOnce;  // table entries of a finishing block's step

// ---------------------------------------------------------------- workspace
// Ints: [0] the number of copies; at kHead two lists of num_pages (the free
// pages in order; for a compaction the holes and the movers), the copies as
// pairs (from, to), and a fork's (source row, new row, whole pages) triples.
constexpr int kHead = 4;

__host__ __device__ inline size_t even(int pages) {
  return (static_cast<size_t>(pages) + 1) & ~static_cast<size_t>(1);
}

__device__ __forceinline__ int* ws_list(const PagesArgs& a) { return a.ws + kHead; }
__device__ __forceinline__ int* ws_list2(const PagesArgs& a) {
  return a.ws + kHead + even(a.num_pages);
}
__device__ __forceinline__ int2* ws_copies(const PagesArgs& a) {
  return reinterpret_cast<int2*>(a.ws + kHead + 2 * even(a.num_pages));
}
__device__ __forceinline__ int* ws_forks(const PagesArgs& a) {
  return a.ws + kHead + 3 * even(a.num_pages) + 2 * static_cast<size_t>(a.n);
}

// ---------------------------------------------------------------- cluster
__device__ __forceinline__ int cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}

// Barrier of all threads of the cluster: what any of them wrote before it,
// all of them see after it (global data is read back through L2, __ldcg).
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

// Stores v at the same shared variable of CTA `rank` of the cluster.
__device__ __forceinline__ void st_cluster(unsigned long long* p, int rank, unsigned long long v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"(ptx::smem_addr(p)), "r"(rank));
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

// Sum over the CTA's threads before this one; *total: of all of them.
__device__ __forceinline__ unsigned long long scan_exclusive(unsigned long long v,
                                                             unsigned long long* warp_s,
                                                             unsigned long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) warp_s[warp] = inc;
  __syncthreads();
  unsigned long long w = warp_s[lane];  // kWarps == 32
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long up = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += up;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const unsigned long long before = __shfl_sync(0xffffffffu, w, warp == 0 ? 0 : warp - 1);
  __syncthreads();  // warp_s may be used again
  return (warp == 0 ? 0 : before) + inc - v;
}

// What the CTAs of the cluster tell one another.
struct Shared {
  unsigned long long warp_s[kWarps];
  unsigned long long asked[kCtas];   // pages wanted by the CTA's rows | copies << 44
  unsigned long long counted[kCtas]; // free (or live) pages of the CTA's run
  int warp_off[kWarps];
  unsigned long long holes;           // compaction: pages that move
  int rows, longs;                    // entries of row[] from its front and from its back
  int row[kThreads];                  // the CTA's rows whose page lists a warp or the CTA walks
  int from[kThreads], to[kThreads];   // those rows' first and last table column, by thread
  int start[kThreads];                // rank of the first page the row gets
};

// Puts thread t's row, with table columns [from, to), on the list of rows that
// warps walk, or, from its back, on that of rows the whole CTA walks.
__device__ __forceinline__ void list_row(Shared& sh, int t, int from, int to) {
  sh.from[t] = from;
  sh.to[t] = to;
  if (to - from > kLong)
    sh.row[kThreads - 1 - atomicAdd(&sh.longs, 1)] = t;
  else
    sh.row[atomicAdd(&sh.rows, 1)] = t;
}

// Calls walk(t, column, stride) for every listed row, by its warp or by the
// CTA, with each thread's first column and its step.
template <typename Walk>
__device__ __forceinline__ void walk_rows(const Shared& sh, Walk walk) {
  const int tid = threadIdx.x;
  // one loop over both lists, so that the walk is compiled once, in line
  for (int i = tid >> 5, wide = 0;; i += wide ? 1 : kWarps) {
    if (!wide && i >= sh.rows) {
      wide = 1;
      i = 0;
    }
    if (wide && i >= sh.longs) break;
    const int t = sh.row[wide ? kThreads - 1 - i : i];
    walk(t, sh.from[t] + (wide ? tid : tid & 31), wide ? kThreads : 32);
  }
}

constexpr int kCopyShift = 44;
constexpr unsigned long long kAskMask = (1ull << kCopyShift) - 1;

// The run of pages of warp w of CTA c: words of 32 pages.
struct Run {
  int word0, words;  // first word of the CTA, words of the CTA
  int w0, w1;        // the warp's, of the CTA's
};

__device__ __forceinline__ Run page_run(int num_pages, int cta, int warp) {
  const int total = (num_pages + 31) >> 5;
  const int per = (total + kCtas - 1) / kCtas;
  Run r;
  r.word0 = min(cta * per, total);
  r.words = min(per, total - r.word0);
  const int pw = (r.words + kWarps - 1) / kWarps;
  r.w0 = min(warp * pw, r.words);
  r.w1 = min(r.w0 + pw, r.words);
  return r;
}

// One bit per page, set where the page is live, into bits[word of the CTA];
// returns the warp's number of bits set.  The places of the last word past
// the pool's end read as `past`.
__device__ __forceinline__ int live_bits(const PagesArgs& a, const Run& r, uint32_t* bits,
                                         int past) {
  const int lane = threadIdx.x & 31;
  int live = 0;
  constexpr int kAhead = 8;
  for (int w = r.w0; w < r.w1; w += kAhead) {
    int v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int page = (r.word0 + w + i) * 32 + lane;
      v[i] = w + i < r.w1 && page < a.num_pages ? __ldcg(a.refs + page) : past;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint32_t word = __ballot_sync(0xffffffffu, v[i] > 0);
      if (w + i < r.w1) {
        if (lane == 0) bits[w + i] = word;
        live += __popc(word);
      }
    }
  }
  return live;
}

// Clears a page's bit in the CTA whose run it is in.
__device__ __forceinline__ void clear_bit(int num_pages, uint32_t* bits, int page) {
  const int per = (((num_pages + 31) >> 5) + kCtas - 1) / kCtas;
  const int word = page >> 5, owner = word / per;
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"(ptx::smem_addr(bits + (word - owner * per))), "r"(owner));
  asm volatile("red.relaxed.cluster.shared::cluster.and.b32 [%0], %1;" ::"r"(at),
               "r"(~(1u << (page & 31)))
               : "memory");
}

// Turns per-warp counts into each warp's offset inside the CTA and tells
// every CTA of the cluster the CTA's total.
__device__ __forceinline__ void share_counts(Shared& sh, int cta, int warp_count) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) sh.warp_off[warp] = warp_count;
  __syncthreads();
  if (warp == 0) {
    const int v = sh.warp_off[lane];
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    sh.warp_off[lane] = inc - v;
    const int total = __shfl_sync(0xffffffffu, inc, 31);
    if (lane < kCtas) st_cluster(&sh.counted[cta], lane, static_cast<unsigned long long>(total));
  }
}

__device__ __forceinline__ unsigned long long sum_before(const unsigned long long* v, int cta) {
  unsigned long long s = 0;
  for (int i = 0; i < cta; ++i) s += v[i];
  return s;
}

// Writes the CTA's free pages of rank < wanted to list[rank], lowest first.
__device__ __forceinline__ void list_free(const PagesArgs& a, const Shared& sh, const Run& r,
                                          const uint32_t* bits, int cta, long long wanted) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long rank = static_cast<long long>(sum_before(sh.counted, cta)) + sh.warp_off[warp];
  int* list = ws_list(a);
  for (int w = r.w0; w < r.w1 && rank < wanted; ++w) {
    const uint32_t free = ~bits[w];
    const long long at = rank + __popc(free & ((1u << lane) - 1));
    if ((free >> lane & 1u) && at < wanted) list[at] = (r.word0 + w) * 32 + lane;
    rank += __popc(free);
  }
}

__device__ __forceinline__ int pages_of(int len) { return (len + kPage - 1) / kPage; }

__device__ __forceinline__ bool in_pool(const PagesArgs& a, int page) {
  return page >= 0 && page < a.num_pages;
}

// ---------------------------------------------------------------- resize
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1)
    pages_resize_kernel(const __grid_constant__ PagesArgs a) {
  extern __shared__ uint32_t bits[];
  __shared__ Shared sh;
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = cta_rank();
  const int per = (a.B + kCtas - 1) / kCtas;  // rows of a CTA, one thread each
  const int b = cta * per + tid;
  const bool mine = tid < per && b < a.B;
  int old = 0, n = 0;
  bool ok = mine;
  if (tid == 0) sh.rows = sh.longs = 0;
  __syncthreads();

  // 1. pages past a row's new end are given back, and cleared in the bits of
  // the live pages, which are taken before, where nobody holds them any more
  const Run r = page_run(a.num_pages, cta, warp);
  if (mine) {
    old = __ldcg(a.seqlens + b);
    n = __ldg(a.new_seqlens + b);
    const int most = a.max_pages * kPage;
    ok = old >= 0 && old <= most && n >= 0 && n <= most;
    if (!ok) {
      atomicOr(a.status, kStatusBadInput);
    } else if (pages_of(n) < pages_of(old)) {
      list_row(sh, tid, pages_of(n), pages_of(old));
    }
  }
  live_bits(a, r, bits, 1);
  cluster_sync();
  walk_rows(sh, [&](int t, int first, int step) {
    const int* row = a.page_table + static_cast<size_t>(cta * per + t) * a.max_pages;
    for (int j = first; j < sh.to[t]; j += step) {
      const int page = __ldcg(row + j);
      if (!in_pool(a, page))
        atomicOr(a.status, kStatusBadInput);
      else if (atomicSub(a.refs + page, 1) == 1)
        clear_bit(a.num_pages, bits, page);
    }
  });
  cluster_sync();

  // 2. free pages counted, pages asked for summed.  A row asks for the pages
  // it grows by, and for one more where it grows inside a last page that
  // another row holds too: that page is copied before it is written.
  if (tid == 0) sh.rows = sh.longs = 0;
  int live = 0;
  for (int w = r.w0 + lane; w < r.w1; w += 32) live += __popc(bits[w]);
  live = __reduce_add_sync(0xffffffffu, live);
  int need = 0, last = -1;
  bool split = false;
  if (ok && n > old) {
    need = pages_of(n) - pages_of(old);
    if (a.k_pages != nullptr && old % kPage != 0) {
      last = __ldcg(a.page_table + static_cast<size_t>(b) * a.max_pages + old / kPage);
      if (!in_pool(a, last)) {
        atomicOr(a.status, kStatusBadInput);
        ok = false;
        need = 0;
      } else {
        split = __ldcg(a.refs + last) > 1;
        need += split;
      }
    }
  }
  unsigned long long total;
  unsigned long long before = scan_exclusive(
      static_cast<unsigned long long>(need) | static_cast<unsigned long long>(split) << kCopyShift,
      sh.warp_s, &total);
  share_counts(sh, cta, (r.w1 - r.w0) * 32 - live);
  if (tid < kCtas) st_cluster(&sh.asked[cta], tid, total);
  cluster_sync();

  // 3. the lowest free pages listed in order
  const unsigned long long all = sum_before(sh.asked, kCtas);
  const long long room = static_cast<long long>(sum_before(sh.counted, kCtas));
  const long long asked = static_cast<long long>(all & kAskMask);
  before += sum_before(sh.asked, cta);
  list_free(a, sh, r, bits, cta, asked < room ? asked : room);
  cluster_sync();

  // 4. rows served in order, as long as the pages last
  if (cta == 0 && tid == 0) a.ws[0] = static_cast<int>(all >> kCopyShift);
  const int* list = ws_list(a);
  int2* copies = ws_copies(a) + (before >> kCopyShift);
  const long long start = static_cast<long long>(before & kAskMask);
  if (ok) {
    if (need > 0 && start + need > room) {
      atomicOr(a.status, kStatusNoPages);
      if (split) *copies = make_int2(-1, -1);
    } else {
      int* row = a.page_table + static_cast<size_t>(b) * a.max_pages;
      int at = static_cast<int>(start);
      if (split) {
        const int page = __ldcg(list + at++);
        *copies = make_int2(last, page);
        row[old / kPage] = page;
        a.refs[page] = 1;
        atomicSub(a.refs + last, 1);
      }
      const int c0 = pages_of(old), c1 = pages_of(n);
      if (c1 - c0 == 1) {
        const int page = __ldcg(list + at);
        row[c0] = page;
        a.refs[page] = 1;
      } else if (c1 > c0) {
        sh.start[tid] = at;
        list_row(sh, tid, c0, c1);
      }
      a.seqlens[b] = n;
    }
  }
  __syncthreads();
  walk_rows(sh, [&](int t, int first, int step) {
    int* row = a.page_table + static_cast<size_t>(cta * per + t) * a.max_pages;
    const int* mine = list + sh.start[t] - sh.from[t];
#pragma unroll 4
    for (int j = first; j < sh.to[t]; j += step) {
      const int page = __ldcg(mine + j);
      row[j] = page;
      a.refs[page] = 1;
    }
  });
}

// ---------------------------------------------------------------- fork
// Row dst[i] claims its place with INT_MIN + i in its length, so that of two
// forks into one row the first wins whatever the timing.  Every length is
// read, and one out of range refused, before the first claim is made (a
// cluster barrier lies between, waited for after the counts are read), so no
// stored length is ever taken for a claim.
constexpr int kClaim = static_cast<int>(0x80000000u);

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1)
    pages_fork_kernel(const __grid_constant__ PagesArgs a) {
  extern __shared__ uint32_t bits[];
  __shared__ Shared sh;
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, warp = tid >> 5, cta = cta_rank();
  const int per = (a.n + kCtas - 1) / kCtas;  // forks of a CTA, one thread each
  const int i = cta * per + tid;
  const bool mine = tid < per && i < a.n;

  // 1. what each fork copies; live pages; claims on the new rows
  int src = 0, dst = 0, len = 0, last = -1;
  bool ok = false;
  if (mine) {
    src = __ldg(a.src + i);
    dst = __ldg(a.dst + i);
    ok = src >= 0 && src < a.B && dst >= 0 && dst < a.B && src != dst;
    if (ok) {
      len = __ldcg(a.seqlens + src);
      ok = __ldcg(a.seqlens + dst) == 0 && len >= 0 && len <= a.max_pages * kPage;
    }
  }
  cluster_arrive();
  if (ok && len % kPage != 0) {
    last = __ldcg(a.page_table + static_cast<size_t>(src) * a.max_pages + len / kPage);
    ok = in_pool(a, last);
  }
  const Run r = page_run(a.num_pages, cta, warp);
  const int live = live_bits(a, r, bits, 1);
  cluster_wait();
  if (ok) atomicMin(a.seqlens + dst, kClaim + i);
  share_counts(sh, cta, (r.w1 - r.w0) * 32 - live);
  cluster_sync();

  // 2. pages asked for: one where the source ends inside a page
  const bool won = ok && __ldcg(a.seqlens + dst) == kClaim + i;
  if (mine && !won) atomicOr(a.status, kStatusBadInput);
  const int need = won && last >= 0;
  unsigned long long total;
  unsigned long long before = scan_exclusive(need, sh.warp_s, &total);
  if (tid < kCtas) st_cluster(&sh.asked[cta], tid, total);
  cluster_sync();

  // 3. the lowest free pages listed in order
  const long long asked = static_cast<long long>(sum_before(sh.asked, kCtas));
  const long long room = static_cast<long long>(sum_before(sh.counted, kCtas));
  before += sum_before(sh.asked, cta);
  const long long served = asked < room ? asked : room;
  list_free(a, sh, r, bits, cta, served);
  cluster_sync();

  // 4. new rows; the finishing kernel shares the whole pages
  if (cta == 0 && tid == 0) a.ws[0] = static_cast<int>(served);
  if (mine) {
    const long long start = static_cast<long long>(before);
    const bool granted = won && (!need || start < room);
    int* fork = ws_forks(a) + 3 * static_cast<size_t>(i);
    fork[0] = src;
    fork[1] = dst;
    fork[2] = granted ? len / kPage : 0;
    if (won) a.seqlens[dst] = granted ? len : 0;
    if (won && !granted) atomicOr(a.status, kStatusNoPages);
    if (granted && need) {
      const int page = __ldcg(ws_list(a) + start);
      ws_copies(a)[start] = make_int2(last, page);
      a.page_table[static_cast<size_t>(dst) * a.max_pages + len / kPage] = page;
      a.refs[page] = 1;
    }
  }
}

// ---------------------------------------------------------------- compaction
// With L live pages, the k-th live page at or past L moves to the k-th free
// page before L.  The movers are ranked from the last one down (the live
// pages after a page are the total less those up to it), which needs no
// count at the boundary L; the boundary's own count, the number of movers,
// then turns the ranks round.
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads, 1)
    pages_compact_kernel(const __grid_constant__ PagesArgs a) {
  extern __shared__ uint32_t bits[];
  __shared__ Shared sh;
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = cta_rank();
  if (tid == 0) sh.holes = 0;
  cluster_arrive();
  const Run r = page_run(a.num_pages, cta, warp);
  const int live_count = live_bits(a, r, bits, 0);
  cluster_wait();  // every CTA runs before any writes into another's shared memory
  share_counts(sh, cta, live_count);
  cluster_sync();

  const int total = static_cast<int>(sum_before(sh.counted, kCtas));
  int* holes = ws_list(a);
  int* movers = ws_list2(a);  // last one first
  int seen = static_cast<int>(sum_before(sh.counted, cta)) + sh.warp_off[warp];
  for (int w = r.w0; w < r.w1; ++w) {
    const uint32_t word = bits[w];
    const int page = (r.word0 + w) * 32 + lane;
    const bool live = word >> lane & 1u;
    const int upto = seen + __popc(word & ((1u << lane) - 1));  // live pages before this one
    if (page < a.num_pages) {
      if (!live || page < total) a.new_index[page] = live ? page : -1;
      if (live && page >= total) movers[total - 1 - upto] = page;
      if (!live && page < total) holes[page - upto] = page;
      if (page == total - 1) {
        const unsigned long long h = static_cast<unsigned long long>(total - upto - live);
        for (int c = 0; c < kCtas; ++c) st_cluster(&sh.holes, c, h);
      }
    }
    seen += __popc(word);
  }
  cluster_sync();

  const int moved = static_cast<int>(sh.holes);
  int2* copies = ws_copies(a);
  for (int k = cta * kThreads + tid; k < moved; k += kCtas * kThreads) {
    const int to = __ldcg(holes + k), from = __ldcg(movers + moved - 1 - k);
    copies[k] = make_int2(from, to);
    a.new_index[from] = to;
    a.refs[to] = a.refs[from];
    a.refs[from] = 0;
  }
  if (cta == 0 && tid == 0) {
    a.ws[0] = moved;
    *a.num_live = total;
  }
}

// ---------------------------------------------------------------- finish
enum { kResize, kFork, kCompact };

// The pages' data, in every layer of both pools, and the table entries that
// a fork shares or a compaction renames.  From and to pages never overlap:
// every `to` was free.
template <int kMode>
__global__ void __launch_bounds__(kCopyThreads)
    pages_finish_kernel(const __grid_constant__ PagesArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  // Rows in segments, so that one long row is shared by many blocks.  Their
  // product fits 31 bits: 2^20 rows at most, and a table that fits memory has
  // fewer than 2^27 segments of 1024 entries beyond one a row.
  const int segments = (a.max_pages + kSegment - 1) / kSegment;
  if constexpr (kMode == kFork) {
    for (int it = blockIdx.x; it < a.n * segments; it += gridDim.x) {
      const int i = segments > 1 ? it / segments : it;
      const int j0 = (it - i * segments) * kSegment + tid;
      const int* fork = ws_forks(a) + 3 * static_cast<size_t>(i);
      const int whole = fork[2];
      if (j0 - tid >= whole) continue;
      const int* from = a.page_table + static_cast<size_t>(fork[0]) * a.max_pages;
      int* to = a.page_table + static_cast<size_t>(fork[1]) * a.max_pages;
      int page[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        page[k] = j0 + k * kCopyThreads < whole ? __ldcg(from + j0 + k * kCopyThreads) : 0;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        if (j0 + k * kCopyThreads >= whole) break;
        to[j0 + k * kCopyThreads] = page[k];
        if (in_pool(a, page[k]))
          atomicAdd(a.refs + page[k], 1);
        else
          atomicOr(a.status, kStatusBadInput);
      }
    }
  }
  if constexpr (kMode == kCompact) {
    for (int it = blockIdx.x; it < a.B * segments; it += gridDim.x) {
      const int b = segments > 1 ? it / segments : it;
      const int j0 = (it - b * segments) * kSegment + tid;
      const int len = a.seqlens[b];
      if (len < 0 || len > a.max_pages * kPage) {
        if (tid == 0) atomicOr(a.status, kStatusBadInput);
        continue;
      }
      int* row = a.page_table + static_cast<size_t>(b) * a.max_pages;
      int page[kAtOnce], to[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        page[k] = j0 + k * kCopyThreads < pages_of(len) ? row[j0 + k * kCopyThreads] : -1;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        to[k] = in_pool(a, page[k]) ? __ldcg(a.new_index + page[k]) : -1;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        if (j0 + k * kCopyThreads >= pages_of(len)) break;
        if (to[k] < 0)  // not a page, or one that nothing counts as held
          atomicOr(a.status, kStatusBadInput);
        else if (to[k] != page[k])
          row[j0 + k * kCopyThreads] = to[k];
      }
    }
  }
  constexpr int kPiece = kCopyThreads * kCopyVecs;
  const int pieces = (a.page_vecs + kPiece - 1) / kPiece;
  const int2* copies = ws_copies(a);
  const long long per_copy = 2ll * a.layers * pieces;
  const long long items = a.ws[0] * per_copy;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int c = static_cast<int>(it / per_copy);
    const int rest = static_cast<int>(it - c * per_copy);
    const int piece = rest % pieces, plane = rest / pieces;
    const int2 move = copies[c];
    if (move.x < 0) continue;
    const size_t base = static_cast<size_t>(plane >> 1) * a.num_pages;
    uint4* pool = plane & 1 ? a.v_pages : a.k_pages;
    const uint4* from = pool + (base + move.x) * a.page_vecs;
    uint4* to = pool + (base + move.y) * a.page_vecs;
    const int v0 = piece * kPiece + tid;
    uint4 x[kCopyVecs];
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i)
      if (v0 + i * kCopyThreads < a.page_vecs) x[i] = __ldcs(from + v0 + i * kCopyThreads);
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i)
      if (v0 + i * kCopyThreads < a.page_vecs) to[v0 + i * kCopyThreads] = x[i];
  }
}

// ---------------------------------------------------------------- launches
size_t bits_bytes(int num_pages) {
  const size_t words = (static_cast<size_t>(num_pages) + 31) / 32;
  return (words + kCtas - 1) / kCtas * sizeof(uint32_t);
}

template <typename Kernel>
cudaError_t launch_book(Kernel kernel, const PagesArgs& a, cudaStream_t stream) {
  const size_t smem = bits_bytes(a.num_pages);
  if (smem > 16 * 1024) {
    // beside the static part this passes the default 48 KB.  Always the
    // largest size, so that calls from several threads set the same value.
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(bits_bytes(kPagesMaxPages)));
    if (e != cudaSuccess) return e;
  }
  kernel<<<kCtas, kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

// The finishing kernel may start while the bookkeeping one still runs; its
// first instruction waits for that kernel's end and its writes.
template <int kMode>
cudaError_t launch_finish(const PagesArgs& a, long long most_copies, int rows,
                          cudaStream_t stream) {
  const long long steps =
      static_cast<long long>(rows) * ((a.max_pages + kSegment - 1) / kSegment);
  constexpr int kPiece = kCopyThreads * kCopyVecs;
  const long long items =
      most_copies * 2 * a.layers * ((a.page_vecs + kPiece - 1) / kPiece);
  long long grid = items > steps ? items : steps;
  const long long most = 32ll * a.num_sms;
  if (grid > most) grid = most;
  if (grid < 1) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pages_finish_kernel<kMode>, a);
}

}  // namespace

size_t pages_workspace_bytes(int rows, int num_pages) {
  return sizeof(int) * (kHead + 3 * even(num_pages) + 5 * static_cast<size_t>(rows));
}

cudaError_t launch_pages_resize(const PagesArgs& a, cudaStream_t stream) {
  const cudaError_t e = launch_book(pages_resize_kernel, a, stream);
  if (e != cudaSuccess || a.k_pages == nullptr) return e;
  return launch_finish<kResize>(a, a.B, 0, stream);
}

cudaError_t launch_pages_fork(const PagesArgs& a, cudaStream_t stream) {
  const cudaError_t e = launch_book(pages_fork_kernel, a, stream);
  return e != cudaSuccess ? e : launch_finish<kFork>(a, a.n, a.n, stream);
}

cudaError_t launch_pages_compact(const PagesArgs& a, cudaStream_t stream) {
  const cudaError_t e = launch_book(pages_compact_kernel, a, stream);
  return e != cudaSuccess ? e : launch_finish<kCompact>(a, a.num_pages / 2, a.B, stream);
}

}  // namespace attn
