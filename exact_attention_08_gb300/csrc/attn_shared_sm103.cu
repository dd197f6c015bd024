// One-token decode of rows that share the leading pages of their caches (samples of
// one prompt, chats under one system prompt): the shared keys are read and
// multiplied once for all rows of a group, the rows' own keys by the split decode,
// and the partial results are merged by log-sum-exp.
//
// Prefix kernel.  For one key head the group's queries, (row, head of the head
// group) pairs, are the rows of a product with the prefix's keys: up to 256 of them
// (two 128-row tiles) are an item.  The work is cut into units, a key tile of an item,
// in the order (group, key head, query tile pair, key tile), and each of the
// persistent CTAs (at most one an SM) takes an equal run of units, so one long prompt
// and many short ones alike fill the GPU.  An item that several CTAs share has a
// partial result from each.
//
// Keys.  A page (16 tokens of one head) arrives in one copy, as two halves of [d / 64
// atoms][8 rows][128 bytes]: the eight-row groups of consecutive pages are evenly spaced,
// as the second operand of S needs them, and a page is one step of 16 tokens of the operand of
// O.
//
// Precision.  P is rounded to bf16, the form in which the tensor cores take it beside V, as in the
// split decode; sums, maxima and O are fp32.  O is 2.3e-3 of itself off fp64 by norm, where
// its own rounding to bf16 makes 1.65e-3.
//
// With S = Q K^T and O += P V on the tensor cores and the online softmax between them, a
// key tile keeps an SM busy for less time than HBM needs to bring its keys and values
// while an item has at most 256 rows; more rows find them in L2.
//
// Two streams (d = 64, 128): S buffer, O and four softmax warps each.  An item of more
// than 128 rows has a tile in each stream, and every key tile is a job of both; a
// smaller one has the same tile in both, and they take the key tiles in turn (two
// partial results).  At d = 256 O alone fills half of tensor memory: one stream, two S
// buffers, key tiles of 64.
//
//   tensor memory  S[2], O[streams] (d columns each)
//   shared memory  Q (two tiles; one at d = 256), a ring of K and V tiles
//   warps          0-3, 4-7 softmax of a stream, 8 TMA producer, 9 MMA issuer
#include "attn_internal.h"
#include "sm103_ptx.cuh"

#include <algorithm>
#include <climits>
#include <cmath>

namespace attn {
namespace {

using namespace ptx;

constexpr int kPage = 16;
constexpr int kRows = 128;          // rows of a query tile
constexpr int kItemRows = 2 * kRows;
constexpr int kThr = 320;
constexpr int kWarpProducer = 8;
constexpr int kWarpIssuer = 9;
// O is rescaled only when the running maximum has grown by more than 2^8.
constexpr float kRescaleLog2 = 8.0f;

template <int D>
struct Cfg {
  static constexpr int kStreams = D == 256 ? 1 : 2;
  static constexpr int kTileRows = kStreams * kRows;   // rows of an item at most
  static constexpr int kKeys = D == 256 ? 64 : 128;    // keys of a key tile
  static constexpr int kPages = kKeys / kPage;
  static constexpr int kAtoms = D / 64;
  static constexpr int kQAtom = kRows * 128;
  static constexpr int kQTile = kAtoms * kQAtom;
  static constexpr int kGroup = kAtoms * 1024;         // eight keys
  static constexpr int kPageBytes = 2 * kGroup;
  static constexpr int kSlot = kPages * kPageBytes;    // a K or V tile
  static constexpr int kSlots = D == 64 ? 8 : 5;
  static constexpr int kOffRing = kStreams * kQTile;
  static constexpr int kOffBar = kOffRing + kSlots * kSlot;
  // full, empty of the ring; s_full, p_ready, o_done [2]; rows_full, q_full, q_empty; drain
  static constexpr int kNumBars = 2 * kSlots + 6 + 3 + 1;
  static constexpr int kSmem = kOffBar + (kNumBars + 1) * 8 + 1024;
  static_assert(kSmem + kItemRows * 4 + 16 <= 227 * 1024, "shared memory");
  static constexpr uint32_t kColO = 256;
};

// ---------------------------------------------------------------- plan
// A group shares its prefix where (rows - 1) pages d reaches this.  Rows that read the same
// pages one after the other find them in L2, so sharing a few pages costs more than it saves.
// Its time over that of the rows one by one, 32 heads over 8:
//   64 groups of 8  d = 64   8 pages 1.05, 16 0.95, 32 0.79, 128 0.48
//                   d = 128  1 page 1.30, 8 1.05, 10 1.08, 16 0.93, 128 0.46
//                   d = 256  2 pages 1.07, 4 0.96, 16 0.63
//   200 groups of 2 d = 64   64 pages 1.17, 128 1.10, 192 1.11
//                   d = 128  32 pages 1.20, 64 1.04, 96 1.00
//                   d = 256  16 pages 0.93, 32 0.78
// The border goes by d, as the bytes do; only for pairs the rule is early at d = 64 (by a tenth of
// the time) and late at d = 256.  A single row counts as two: nothing is read less often, but a
// long row is spread over the CTAs, where its few splits would be the last to finish (16 groups
// of 1 to 7 rows, 64 to 256 pages: 70 us, with single rows from 128 pages on 96, by
// themselves 126).
constexpr int kLeastShared = 8192;
// One block: rows to groups, the pages that every group shares, units before each group,
// where each CTA of the prefix kernel begins, first own page of every row, and the rows in
// the order of their own pages, longest first.  Steps that depend on one another, so
// latency is all of it: what later kernels would have to work out again is written down
// as records of 16 bytes.
// Threads of the plan's block: every instruction costs it eight cycles with 32 warps, four with
// 16, and steps over the rows or groups take more of them only when those are many
// (2,000 groups of one row: 69 us with 32 warps, 73 with 16; 64 rows 46.0 and 45.2).
constexpr int kPlanThreads = 512, kPlanMost = 1024, kPlanRows = 1024;
constexpr int kEntries = 4096;  // rows whose list entries fit in shared memory

__device__ __forceinline__ int row_length(const SharedArgs& a, int b) {
  const int L = a.seqlens[b];
  return max(0, min(L, a.max_pages * kPage));
}

__device__ __forceinline__ int ceil_div(int x, int y) { return (x + y - 1) / y; }

__device__ __noinline__ long long divide(long long x, long long y) { return x / y; }

// Sum before this thread and over the block.
template <int kThreads>
__device__ __noinline__ long long block_scan(long long v, long long* part, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) part[warp] = x;
  __syncthreads();
  const long long p = lane < kThreads / 32 ? part[lane] : 0;
  long long sum = p;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  *total = __shfl_sync(0xffffffffu, sum, 31);
  return __shfl_sync(0xffffffffu, sum - p, warp) + x - v;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) attn_shared_plan_kernel(const SharedArgs a) {
  __shared__ int s_cnt[kThreads];
  __shared__ int s_entry[kEntries];
  __shared__ long long s_part[kThreads / 32];
  __shared__ int s_items, s_longest;
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* entry = a.B <= kEntries ? s_entry : a.entry;  // where a row stands in the list
#pragma unroll 1
  for (int b = tid; b < a.B; b += kThreads) {
    entry[b] = INT_MAX;
    a.start[b] = 0;
    a.rowinfo[b] = make_int4(-1, 0, 0, 0);
  }
  s_cnt[tid] = 0;
  if (tid == 0) s_items = s_longest = 0;
  // offsets that decrease or leave the list: no group is used
  bool bad = false;
  if (a.cu_groups != nullptr) {  // (may be null where there are no groups)
#pragma unroll 1
    for (int g = tid; g <= a.n_groups; g += kThreads) {
      const int c = a.cu_groups[g];
      bad |= c < 0 || c > a.n_rows || (g > 0 && c < a.cu_groups[g - 1]);
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) atomicOr(a.status, kStatusBadInput);
  const int n_groups = bad ? 0 : a.n_groups;
  // a row listed more than once belongs where it stands first
  if (n_groups > 0) {
    const int e1 = a.cu_groups[n_groups];
#pragma unroll 1
    for (int e = a.cu_groups[0] + tid; e < e1; e += kThreads) {
      const int b = a.rows ? a.rows[e] : e;
      if (b < 0 || b >= a.B || atomicMin(&entry[b], e) != INT_MAX)
        atomicOr(a.status, kStatusBadInput);
    }
  }
  __syncthreads();
  // Some lanes for each group: its longest row, the pages it shares.  A warp, or as many lanes
  // as a group has rows on average where there are more groups than warps (2,000 groups of one
  // row by a warp each took 45 us).
  int bits = 5;
  if (n_groups > kThreads / 32) {
    const int entries = a.cu_groups[n_groups] - a.cu_groups[0];
#pragma unroll 1
    while (bits > 0 && static_cast<long long>(n_groups) << (bits - 1) >= entries) --bits;
  }
  const int lanes = 1 << bits, part = tid & (lanes - 1);
#pragma unroll 1
  for (int g0 = 0; g0 < n_groups; g0 += kThreads >> bits) {
    const int g = g0 + (tid >> bits);
    int e0 = 0, e1 = 0, prefix = 0;
    if (g < n_groups) e0 = a.cu_groups[g], e1 = a.cu_groups[g + 1], prefix = a.prefix_lens[g];
    long long best = -1;  // length and, downwards, row
    int shortest = INT_MAX;
#pragma unroll 1
    for (int e = e0 + part; e < e1; e += lanes) {
      const int b = a.rows ? a.rows[e] : e;
      if (b < 0 || b >= a.B || entry[b] != e) continue;
      const int L = row_length(a, b);
      best = max(best, static_cast<long long>(L) << 32 | (INT_MAX - b));
      shortest = min(shortest, L);
    }
#pragma unroll 1
    for (int o = lanes / 2; o > 0; o >>= 1) {
      best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
      shortest = min(shortest, __shfl_xor_sync(0xffffffffu, shortest, o));
    }
    const int longest = static_cast<int>(best >> 32);
    const int at = static_cast<int>(INT_MAX - static_cast<uint32_t>(best));  // of any row
    int pages = prefix < 0 ? 0 : min(prefix, max(longest, 0)) / kPage;
    int sharing = e1 - e0;  // rows that share them
    // Only rows that reach the end of the shared pages share them: in the product with the values
    // a weight of zero does not keep out what is not finite, so no row may meet a key behind
    // its end.  Where some rows end before, the pages are those of the longest row or the
    // whole ones of the shortest that holds any, whichever saves more reads.
    if (__any_sync(0xffffffffu, shortest < pages * kPage)) {
      int full = 0, some = 0, least = INT_MAX;
#pragma unroll 1
      for (int e = e0 + part; e < e1; e += lanes) {
        const int b = a.rows ? a.rows[e] : e;
        if (b < 0 || b >= a.B || entry[b] != e) continue;
        const int L = row_length(a, b);
        full += L >= pages * kPage;
        if (L > 0) ++some, least = min(least, L);
      }
#pragma unroll 1
      for (int o = lanes / 2; o > 0; o >>= 1) {
        full += __shfl_xor_sync(0xffffffffu, full, o);
        some += __shfl_xor_sync(0xffffffffu, some, o);
        least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
      }
      if (shortest < pages * kPage) {
        const int all = min(pages, least / kPage);  // (only empty rows may end before)
        const bool fewer = static_cast<long long>(some - 1) * all >
                           static_cast<long long>(full - 1) * pages;
        sharing = fewer ? some : full;
        pages = fewer ? all : pages;
      }
    }
    if (g >= n_groups) continue;  // (the last groups' warps: nothing below is done together)
    if (part == 0 && (prefix < 0 || prefix > a.max_pages * kPage))
      atomicOr(a.status, kStatusBadInput);
    // Too little to share: every row for itself.
    if (static_cast<long long>(max(sharing - 1, 1)) * pages < a.least) pages = 0;
    if (part == 0) a.info[g] = make_int4(pages, e0, (e1 - e0) * a.G, at);
    if (pages == 0) continue;
#pragma unroll 1
    for (int e = e0 + part; e < e1; e += lanes) {
      const int b = a.rows ? a.rows[e] : e;
      if (b < 0 || b >= a.B || entry[b] != e || row_length(a, b) < pages * kPage) continue;
      a.start[b] = pages;
      a.rowinfo[b] = make_int4(g, (e - e0) * a.G, 0, 0);
    }
  }
  __syncthreads();
  // rows by own pages, longest first (a counting sort, of several page counts a bucket where
  // there are more than buckets; rows of one bucket in any order, which only says which
  // CTA runs first)
  const int shift = max(0, 32 - __clz(a.max_pages) - (kThreads == 512 ? 9 : 10));
  auto bucket = [&](int b) {
    return (a.max_pages - ((row_length(a, b) + kPage - 1) / kPage - a.start[b])) >> shift;
  };
  const bool one = a.B <= kThreads;  // a thread a row
  const int mine = one && tid < a.B ? min(bucket(tid), kThreads - 1) : 0;
  if (one) {
    if (tid < a.B) atomicAdd(&s_cnt[mine], 1);
  } else {
#pragma unroll 1
    for (int b = tid; b < a.B; b += kThreads) atomicAdd(&s_cnt[min(bucket(b), kThreads - 1)], 1);
  }
  // units before each group
  long long units = 0;
#pragma unroll 1
  for (int g0 = 0; g0 < n_groups; g0 += kThreads) {
    const int g = g0 + tid;
    long long v = 0, all;
    if (g < n_groups) {
      const int4 info = a.info[g];
      const int tiles = ceil_div(info.x, a.tile_pages);
      v = static_cast<long long>(ceil_div(info.z, a.tile_rows)) * a.Hkv;
      if (tiles > 0) {
        atomicMax(&s_longest, tiles);
        atomicAdd(&s_items, static_cast<int>(min(v, 1024LL)));
      }
      v *= tiles;
    }
    const long long before = block_scan<kThreads>(v, s_part, &all);
    if (g < n_groups) a.base[g] = units + before;
    units += all;
  }
  __syncthreads();
  long long all;
  const int before = static_cast<int>(block_scan<kThreads>(s_cnt[tid], s_part, &all));
  __syncthreads();
  s_cnt[tid] = before;
  __syncthreads();
  if (one) {
    if (tid < a.B) a.order[atomicAdd(&s_cnt[mine], 1)] = tid;
  } else {
#pragma unroll 1
    for (int b = tid; b < a.B; b += kThreads)
      a.order[atomicAdd(&s_cnt[min(bucket(b), kThreads - 1)], 1)] = b;
  }
  // Where each CTA begins.  Every part of an item costs a load of its queries and a partial
  // result that the merge reads, so p parts of t key tiles take about t / p + p: not fewer
  // than sqrt(t) tiles a CTA, and where all items are alike, CTAs that end with an item.  CTAs
  // without units leave their SMs to the rows' own keys.  (64 rows of 32 heads over 8,
  // prefixes of 2,048 and 8,192 tokens: 40 and 46 us; with all CTAs and runs that end
  // anywhere 47 and 57.)
  if (tid <= a.ctas) {
    // (items past 1,024 a group are not counted: then they are more than CTAs)
    const int items = s_items;
    const int least = max(static_cast<int>(ceilf(sqrtf(s_longest))), 1);
    int n = a.ctas;
    if (units < static_cast<long long>(least) * n)
      n = min(n, max(items, static_cast<int>(units) / least));
    if (items > 0 && items <= n && static_cast<long long>(s_longest) * items == units)
      n -= n % items;
    const long long at = tid < n ? divide(units * tid, n) : units;
    a.runs[tid] = at;
    if (at < units) {
      int lo = 0, hi = n_groups - 1;  // the last group with base <= at
#pragma unroll 1
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.base[mid] <= at)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int4 info = a.info[lo];
      const int tiles = ceil_div(info.x, a.tile_pages), mts = ceil_div(info.z, a.tile_rows);
      const long long in = at - a.base[lo];
      const int item = static_cast<int>(divide(in, tiles));
      a.begin[tid] = make_int4(lo, item / mts, item % mts,
                               static_cast<int>(in - static_cast<long long>(item) * tiles));
    }
  }
}

// ---------------------------------------------------------------- items
// One item of the prefix work and this CTA's part of it.
struct Item {
  int h;                  // key head
  int kt, n;              // first key tile of this CTA's part, key tiles in it
  int rows;               // (row, head) pairs of the item
  int row0;               // its first pair among the group's
  int first;              // the group's first list entry
  int source;             // the row whose table names the prefix's pages
  int keys;               // keys of the prefix
  long long part;         // first row of its partial results
};

// A CTA's run: units left, and the item that it continues with.
struct Walk {
  long long left;
  int g, h, mt, kt;
  int4 info;  // of group g
};

__device__ __forceinline__ void walk_begin(const SharedArgs& a, Walk& w) {
  const long long at = a.runs[blockIdx.x];
  const int4 begin = a.begin[blockIdx.x];
  w.left = a.runs[blockIdx.x + 1] - at;
  if (w.left <= 0) return;
  w.g = begin.x;
  w.h = begin.y;
  w.mt = begin.z;
  w.kt = begin.w;
  w.info = a.info[w.g];
}

__device__ __forceinline__ bool walk_next(const SharedArgs& a, Walk& w, Item& it) {
  if (w.left <= 0) return false;
#pragma unroll 1
  while (w.info.x == 0) w.info = a.info[++w.g];  // (a group with pages follows: units are left)
  const int pages = w.info.x, e0 = w.info.y, pairs = w.info.z;
  it.h = w.h;
  it.kt = w.kt;
  it.n = static_cast<int>(min(static_cast<long long>(ceil_div(pages, a.tile_pages) - w.kt), w.left));
  it.row0 = w.mt * a.tile_rows;
  it.rows = min(a.tile_rows, pairs - it.row0);
  it.first = e0;
  it.source = w.info.w;
  it.keys = pages * kPage;
  it.part = 2 * (static_cast<long long>(e0) * a.Hq + static_cast<long long>(w.h) * pairs + it.row0) +
            static_cast<long long>(kItemRows) * blockIdx.x;
  w.left -= it.n;
  w.kt = 0;
  if (it.row0 + a.tile_rows < pairs) {
    ++w.mt;
  } else {
    w.mt = 0;
    if (++w.h == a.Hkv) {
      w.h = 0;
      if (w.left > 0) w.info = a.info[++w.g];
    }
  }
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThr, 1)
    attn_shared_prefix_kernel(const __grid_constant__ CUtensorMap tmK,
                              const __grid_constant__ CUtensorMap tmV, const SharedArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_row[kItemRows];  // rows of q of an item's pairs
  __shared__ int abort_s;
  uint8_t* smem = smem_align1024(smem_raw);
  uint8_t* ring = smem + C::kOffRing;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + C::kSlots;
  uint64_t* s_full = empty + C::kSlots;  // [S buffer]
  uint64_t* p_ready = s_full + 2;        // [S buffer]
  uint64_t* o_done = p_ready + 2;        // [S buffer] O += P V of that buffer's P
  uint64_t* rows_full = o_done + 2;
  uint64_t* q_full = rows_full + 1;
  uint64_t* q_empty = q_full + 1;
  uint64_t* drain = q_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = &abort_s;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 4);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(rows_full, 8);
    mbar_init(q_full, 8);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    abort_s = 0;
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // The plan.  Only then may the decode of the rows' own pages start (it does not wait for
  // the plan itself, but for every CTA here to have seen it).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __threadfence();  // what the plan wrote, to the grid that this lets start
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  Walk w;
  walk_begin(a, w);
  // An item's jobs, in order: S buffer and, with two streams, stream j % 2.  With a tile in
  // both streams job j is key tile j / 2, else key tile j.
  auto split = [&](const Item& it) { return C::kStreams == 2 && it.rows > kRows; };
  Item it;

  if (warp == kWarpProducer) {
    // ============================================================ TMA producer
    int n_load = 0;
    bool ok = true;
    while (ok && walk_next(a, w, it)) {
      const int* row = a.page_table + static_cast<size_t>(it.source) * a.max_pages;
      const int pages = it.keys / kPage;
      auto lookup = [&](int i) -> int {  // page of lane l of the part's key tile i
        if (i >= it.n || lane >= C::kPages) return 0;
        return row[min((it.kt + i) * C::kPages + lane, pages - 1)];
      };
      auto checked = [&](int page) -> int {
        if (page < 0 || page >= a.num_pages) {
          atomicOr(a.status, kStatusBadInput);
          page = a.num_pages;  // out of bounds: zeros, as in the split decode
        }
        return page;
      };
      auto load = [&](const CUtensorMap* map, int page) {
        const int s = n_load % C::kSlots;
        if (n_load >= C::kSlots && !mbar_wait_far(&empty[s], (n_load / C::kSlots - 1) & 1,
                                                   abort_flag, kWaitLimitNs)) {
          ok = false;
          return;
        }
        mbar_arrive_expect_tx_w(&full[s], C::kSlot);
        if (lane < C::kPages)
          tma_load_5d(ring + s * C::kSlot + lane * C::kPageBytes, map, &full[s], 0, 0, 0, it.h,
                      2 * page);
        __syncwarp();
        ++n_load;
      };
      // K(0), K(1), V(0), K(2), V(1), ...
      int now = checked(lookup(0)), next = lookup(1);
      load(&tmK, now);
      for (int i = 0; ok && i < it.n; ++i) {
        const int later = lookup(i + 2);
        if (i + 1 < it.n) {
          next = checked(next);
          load(&tmK, next);
          if (!ok) break;
        }
        load(&tmV, now);
        now = next;
        next = later;
      }
    }
    if (!ok && lane == 0) {
      atomicOr(a.status, kStatusTimeout);
      *abort_flag = 1;
    }
    // every copy issued lands before the CTA leaves
    for (int i = 0; i < C::kSlots; ++i) {
      const int n = n_load > i ? (n_load - 1 - i) / C::kSlots : -1;
      if (n >= 0) mbar_wait(&full[i], n & 1, nullptr, kWaitLimitNs);
    }
  } else if (warp == kWarpIssuer) {
    // ============================================================ MMA issuer
    constexpr uint32_t idesc_s = idesc_bf16_f32(kRows, C::kKeys, false);
    constexpr uint32_t idesc_o = idesc_bf16_f32(kRows, D, true);
    int n_load = 0;        // tiles of the ring before this item
    int jobs[2] = {0, 0};  // jobs of each S buffer so far
    int items = 0;
    bool ok = true;
    // K of the part's key tile i is load 0 (i = 0) or 2 i - 1; V is 2 i + 2, or 2 i + 1 last.
    while (ok && walk_next(a, w, it)) {
      const bool two = split(it);
      const int J = two ? 2 * it.n : it.n;
      auto k_load = [&](int i) { return n_load + (i == 0 ? 0 : 2 * i - 1); };
      auto v_load = [&](int i) { return n_load + (i + 1 < it.n ? 2 * i + 2 : 2 * i + 1); };
      if (!mbar_wait_far(q_full, items & 1, abort_flag, kWaitLimitNs)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      // S of job j = Q K^T
      auto issue_s = [&](int j) -> bool {
        const int i = two ? j / 2 : j, l = k_load(i), s = l % C::kSlots, buf = j & 1;
        if (!(two && (j & 1)) &&
            !mbar_wait_far(&full[s], (l / C::kSlots) & 1, abort_flag, kWaitLimitNs))
          return false;
        tc_fence_after_sync();
        const uint64_t dq =
            sdesc_sw128(smem_addr(smem + (two ? (j & 1) * C::kQTile : 0)), 16, 1024);
        const uint64_t dk = sdesc_sw128(smem_addr(ring + s * C::kSlot), 16, C::kGroup);
#pragma unroll
        for (int at = 0; at < C::kAtoms; ++at)
          mma_ss_atom_w(tmem + buf * C::kKeys, dq + at * (C::kQAtom >> 4), dk + at * (1024 >> 4),
                        idesc_s, at > 0);
        mma_commit_w(&s_full[buf]);
        if (!two || (j & 1)) mma_commit_w(&empty[s]);
        if (j == J - 1) mma_commit_w(q_empty);
        return true;
      };
      ok = issue_s(0);
      for (int j = 0; ok && j < J; ++j) {
        if (j + 1 < J && !issue_s(j + 1)) {
          ok = false;
          break;
        }
        // O += P V: P in the first half of its S buffer's columns, as bf16 pairs
        const int i = two ? j / 2 : j, l = v_load(i), s = l % C::kSlots, buf = j & 1;
        const int stream = C::kStreams == 2 ? buf : 0;
        if (!mbar_wait_far(&p_ready[buf], jobs[buf] & 1, abort_flag, kWaitLimitNs) ||
            !mbar_wait_far(&full[s], (l / C::kSlots) & 1, abort_flag, kWaitLimitNs)) {
          ok = false;
          break;
        }
        ++jobs[buf];
        tc_fence_after_sync();
        const uint64_t dv = sdesc_sw128(smem_addr(ring + s * C::kSlot), 1024, C::kGroup);
        const bool first = j < C::kStreams;  // the stream's first job of the item
#pragma unroll
        for (int kk = 0; kk < C::kKeys / 16; ++kk)
          mma_bf16_ts_w(tmem + C::kColO + stream * D, tmem + buf * C::kKeys + 8 * kk,
                        dv + kk * (C::kPageBytes >> 4), idesc_o, (!first || kk > 0) ? 1u : 0u);
        mma_commit_w(&o_done[buf]);
        if (!two || (j & 1)) mma_commit_w(&empty[s]);
      }
      n_load += 2 * it.n;
      ++items;
    }
    if (!ok && lane == 0) {
      atomicOr(a.status, kStatusTimeout);
      *abort_flag = 1;
    }
    mma_commit_w(drain);
    mbar_wait(drain, 0, nullptr, kWaitLimitNs);
  } else {
    // ============================================================ softmax: warps 0-3, 4-7
    const int stream = warp / 4;
    const int r = tid % kRows;
    const uint32_t lanes = static_cast<uint32_t>((warp % 4) * 32) << 16;
    int done[2] = {0, 0};  // this stream's jobs in each S buffer so far
    int items = 0;
    bool ok = true;
    while (ok && walk_next(a, w, it)) {
      const bool two = split(it);
      const int J = two ? 2 * it.n : it.n;
      // ---- queries: rows 0-127 to Q tile 0, the others to tile 1
      if (items > 0 && !mbar_wait_far(q_empty, (items - 1) & 1, abort_flag, kWaitLimitNs)) {
        ok = false;
        break;
      }
      // This thread's pair and its row of q (both streams' threads work out the same pairs where
      // they share a tile).  The queries then come eight 16-byte chunks at
      // a time: one by one, each behind its row's index, they took 15 us an item.
      const int pr = two ? tid : r;
      {
        int row = -1;
        if (pr < it.rows) {
          const int pair = it.row0 + pr, member = pair / a.G;
          const int b = a.rows ? a.rows[it.first + member] : it.first + member;
          if (b >= 0 && b < a.B) row = b * a.Hq + it.h * a.G + pair - member * a.G;
        }
        s_row[pr] = row;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(rows_full);
      if (!mbar_wait_far(rows_full, items & 1, abort_flag, kWaitLimitNs)) {
        ok = false;
        break;
      }
      {
        constexpr int kChunks = D / 8, kStep = 256 / kChunks;
        const int c = tid % kChunks, rows = two ? kItemRows : kRows;
        const uint32_t dst = (c / 8) * C::kQAtom;
#pragma unroll 1
        for (int r0 = tid / kChunks; r0 < rows; r0 += 8 * kStep) {
          uint4 v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int row = r0 + j * kStep, q = row < rows ? s_row[row] : -1;
            v[j] = make_uint4(0, 0, 0, 0);
            if (q >= 0)
              v[j] = *reinterpret_cast<const uint4*>(a.q + static_cast<size_t>(q) * D + c * 8);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int row = r0 + j * kStep;
            if (row >= rows) break;
            *reinterpret_cast<uint4*>(smem + (row / kRows) * C::kQTile + dst +
                                      (row % kRows) * 128 + (((c & 7) ^ (row & 7)) << 4)) = v[j];
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      ++items;
      if (stream >= C::kStreams) continue;  // d = 256: the other warps only load queries
      float m_run = -INFINITY, m_used = -INFINITY, l = 0.f, corr = 0.f;
      int last = -1;  // S buffer of this stream's last job
      for (int j = C::kStreams == 2 ? stream : 0; j < J; j += C::kStreams) {
        const int buf = j & 1;
        const int i = two ? j / 2 : j;
        if (!mbar_wait_far(&s_full[buf], done[buf] & 1, abort_flag, kWaitLimitNs)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t tS = tmem + lanes + buf * C::kKeys;
        uint32_t x[C::kKeys];
#pragma unroll
        for (int c = 0; c < C::kKeys / 32; ++c) tmem_ld_x32(tS + 32 * c, x + 32 * c);
#pragma unroll
        for (int c = 0; c < C::kKeys / 32; ++c) tmem_ld_wait_x32(x + 32 * c);
        const int ka = (it.kt + i) * C::kKeys;
        if (ka + C::kKeys > it.keys) {
#pragma unroll
          for (int c = 0; c < C::kKeys; ++c)
            if (ka + c >= it.keys) x[c] = __float_as_uint(-INFINITY);
        }
        float mx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) mx[e] = __uint_as_float(x[e]);
#pragma unroll
        for (int c = 8; c < C::kKeys; ++c) mx[c & 7] = fmaxf(mx[c & 7], __uint_as_float(x[c]));
        const float tmax = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                 fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
        m_run = fmaxf(m_run, tmax);
        // The reference maximum moves only when the scores outgrew it by 2^8; O is then
        // scaled once the product before has been added (by the whole warp).
        const bool first = m_used == -INFINITY;
        const bool grow =
            first ? m_run != -INFINITY : (m_run - m_used) * a.scale2 > kRescaleLog2;
        const bool resc = grow && !first;
        if (__any_sync(0xffffffffu, resc)) {
          if (!mbar_wait_far(&o_done[last], (done[last] - 1) & 1, abort_flag, kWaitLimitNs)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const float alpha = resc ? ex2_approx((m_used - m_run) * a.scale2) : 1.f;
          const uint32_t tO = tmem + lanes + C::kColO + stream * D;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld_x32(tO + 32 * c, o);
            tmem_ld_wait_x32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st_x32(tO + 32 * c, o);
          }
          tmem_st_wait();
          l *= alpha;
          corr *= alpha;
        }
        if (grow) m_used = m_run;
        const float nms = m_used == -INFINITY ? 0.f : -m_used * a.scale2;
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int c = 0; c < C::kKeys / 2; c += 16) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p0 = ex2_approx(fmaf(__uint_as_float(x[2 * (c + e)]), a.scale2, nms));
            const float p1 = ex2_approx(fmaf(__uint_as_float(x[2 * (c + e) + 1]), a.scale2, nms));
            if (e & 1)
              sum1 += p0 + p1;
            else
              sum0 += p0 + p1;
            pk[e] = pack_bf16x2(p0, p1);
          }
          tmem_st_x16(tS + c, pk);
        }
        l += sum0 + sum1;
        // O sums P rounded to bf16, l the fp32 values: what the tile's largest lost leaves O's
        // normaliser too
        const float ptop = ex2_approx(fmaf(tmax, a.scale2, nms));
        corr += ptop - __uint_as_float(pack_bf16x2(0.f, ptop) & 0xffff0000u);
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[buf]);
        ++done[buf];
        last = buf;
      }
      if (!ok) break;
      // ---- partial result: O / l and the log-sum-exp, rows of this stream
      if (last >= 0) {
        if (!mbar_wait_far(&o_done[last], (done[last] - 1) & 1, abort_flag, kWaitLimitNs)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
      }
      const bool seen = last >= 0 && l > 0.f;
      const float inv = seen ? 1.f / (l - corr) : 0.f;
      const long long prow = it.part + (two ? pr : stream * it.rows + r);
      if (pr < it.rows) a.part_lse[prow] = seen ? fmaf(m_used, a.scale, logf(l)) : -INFINITY;
      if (last >= 0) {
        float* dst = a.part_o + prow * D;  // (32-byte stores: full sectors, 59.1 -> 57.3 us)
        const uint32_t tO = tmem + lanes + C::kColO + stream * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld_x32(tO + 32 * c, o);
          tmem_ld_wait_x32(o);
          if (pr < it.rows) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = seen ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
#pragma unroll
            for (int e = 0; e < 32; e += 8) st_global_v8(dst + 32 * c + e, o + e);
          }
        }
        // the next item's first product waits for this warp's next p_ready
        tc_fence_before_sync();
      }
    }
    if (!ok && lane == 0) {
      atomicOr(a.status, kStatusTimeout);
      *abort_flag = 1;
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- merge
// A warp for each (row, query head), two at d = 256: the partial results of its group's prefix, CTA by
// CTA, then those of its own pages, split by split, 32 at a time: their log-sum-exps are
// read a lane each, the outputs so far scaled to the new maximum, and kWide outputs are
// under way together.  A chain of reads, so what does not depend on the last one is read beside
// it, and of few (row, head) pairs eight outputs at a time (48 rows that share 65,519 tokens:
// 115 us, with four 118); of more than kMergeFew four, whose registers leave room for more
// warps (1,000 rows of 32 heads 132 us, with eight 141).
constexpr int kMergeThreads = 256, kMergeFew = 4096;
static_assert(kSharedMaxCtas % 32 == 0, "runs a lane holds");

template <int D, int kWide>
__global__ void __launch_bounds__(kMergeThreads)
    attn_shared_merge_kernel(const SharedArgs a, const DecodeLaunch dec) {
  constexpr int kWarps = D == 256 ? 2 : 1;  // warps of a row: 128 columns each at most
  constexpr int kPer = D / 32 / kWarps;      // columns of a lane
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
  const int row = unit / kWarps, column = unit % kWarps * 128 + lane * kPer;
  if (row >= a.B * a.Hq) return;
  const int b = row / a.Hq, hq = row - b * a.Hq, S = dec.num_splits;
  const int4 info = a.rowinfo[b];  // group (-1: none that shares pages), first pair
  long long runs[kSharedMaxCtas / 32];  // (read beside rowinfo, not behind it)
#pragma unroll
  for (int i = 0; i < kSharedMaxCtas / 32; ++i)
    runs[i] = 32 * i + lane < a.ctas ? a.runs[32 * i + lane] : LLONG_MAX;
  // Rows of partial results fit in 32 bits without sign: 2 * 2^30 and the CTAs' 256 each.
  uint32_t part = 0, second = 0;  // the first; distance of the second stream's
  int n_prefix = 0, pairs_of = 0;
  if (info.x >= 0) {
    const int4 group = a.info[info.x];
    const int e0 = group.y, pairs = group.z;
    const int h = hq / a.G, pr = info.y + hq - h * a.G;
    const int mt = pr / a.tile_rows;
    const int rows = min(a.tile_rows, pairs - mt * a.tile_rows);
    const int mts = ceil_div(pairs, a.tile_rows), tiles = ceil_div(group.x, a.tile_pages);
    const long long u = a.base[info.x] + static_cast<long long>(h * mts + mt) * tiles;
    // the CTAs whose runs hold the item's units: runs that start at or before the first and
    // the last of them (those without units start past all)
    int first = 0, last = 0;
#pragma unroll
    for (int i = 0; i < kSharedMaxCtas / 32; ++i) {
      first += runs[i] <= u;
      last += runs[i] < u + tiles;
    }
    const int c0 = __reduce_add_sync(0xffffffffu, first) - 1;
    n_prefix = __reduce_add_sync(0xffffffffu, last) - c0;
    pairs_of = D != 256 && rows <= kRows;  // two partial results a CTA
    second = rows;
    part = 2u * (static_cast<uint32_t>(e0) * a.Hq + static_cast<uint32_t>(h) * pairs +
                 mt * a.tile_rows) +
           (pr - mt * a.tile_rows) + kItemRows * c0;
    n_prefix <<= pairs_of;
  }
  const int n = n_prefix + S;
  const float sg = dec.sink ? dec.sink[hq] : -INFINITY;
  float M = sg, wsum = sg != -INFINITY && lane == 0 ? 1.f : 0.f, acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += 32) {
    // a partial result a lane: its log-sum-exp, and where its output is
    const int i = i0 + lane;
    float l = -INFINITY;
    const float* src = nullptr;
    if (i < n_prefix) {
      const uint32_t p = part + kItemRows * (i >> pairs_of) + (i & pairs_of) * second;
      l = a.part_lse[p];
      src = a.part_o + static_cast<size_t>(p) * D;
    } else if (i < n) {
      const size_t p = static_cast<size_t>(row) * S + (i - n_prefix);
      l = dec.ws_lse[p];
      src = dec.ws_o + p * D;
    }
    float top = l;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top == -INFINITY) continue;
    top = fmaxf(top, M);
    const float keep = M == -INFINITY ? 0.f : expf(M - top), w = expf(l - top);
    M = top;
    wsum = fmaf(wsum, keep, w);
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= keep;
    // (the output of a part without a key is not written)
    uint32_t some = __ballot_sync(0xffffffffu, w > 0.f);
#pragma unroll 1
    while (some != 0) {
      float v[kWide][kPer], wj[kWide];
#pragma unroll
      for (int j = 0; j < kWide; ++j) {
        const int at = some != 0 ? __ffs(some) - 1 : 0;
        wj[j] = some != 0 ? __shfl_sync(0xffffffffu, w, at) : 0.f;
        const float* from = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), at)) + column;
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[j][e] = 0.f;
        if (some != 0) {
          if constexpr (kPer == 2) {
            const float2 x = *reinterpret_cast<const float2*>(from);
            v[j][0] = x.x, v[j][1] = x.y;
          } else {
            const float4 x = *reinterpret_cast<const float4*>(from);
            v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
          }
        }
        some &= some - 1;
      }
#pragma unroll
      for (int j = 0; j < kWide; ++j)
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = fmaf(wj[j], v[j][e], acc[e]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
  const float inv = M != -INFINITY ? 1.f / wsum : 0.f;
  uint32_t out[kPer / 2];
#pragma unroll
  for (int e = 0; e < kPer / 2; ++e) out[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  uint32_t* o =
      reinterpret_cast<uint32_t*>(dec.o) + (static_cast<size_t>(row) * D + column) / 2;
  if constexpr (kPer == 2)
    o[0] = out[0];
  else
    *reinterpret_cast<uint2*>(o) = make_uint2(out[0], out[1]);
  if (dec.lse && lane == 0 && unit % kWarps == 0)
    dec.lse[row] = M != -INFINITY ? M + logf(wsum) : -INFINITY;
}

template <int D>
cudaError_t launch_shared(SharedArgs a, const DecodeLaunch& dec, int num_sms,
                          cudaStream_t stream) {
  using C = Cfg<D>;
  a.tile_rows = C::kTileRows;
  a.tile_pages = C::kPages;
  a.ctas = std::min(num_sms, kSharedMaxCtas);
  a.least = kLeastShared / D;
  static SharedMemoryLimit limit;
  cudaError_t e = limit.raise(attn_shared_prefix_kernel<D>, C::kSmem);
  if (e != cudaSuccess) return e;
  const int rows = std::max(a.B, a.n_groups);
  if (rows <= kPlanRows)
    attn_shared_plan_kernel<kPlanThreads><<<1, kPlanThreads, 0, stream>>>(a);
  else
    attn_shared_plan_kernel<kPlanMost><<<1, kPlanMost, 0, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_dependent(attn_shared_prefix_kernel<D>, dim3(a.ctas), kThr, C::kSmem, stream, a.tmK,
                       a.tmV, a);
  if (e != cudaSuccess) return e;
  if ((e = launch_attn_decode_own(dec, stream)) != cudaSuccess) return e;
  const int per = kMergeThreads / 32 / (D == 256 ? 2 : 1);  // rows of a block
  const int blocks = (a.B * a.Hq + per - 1) / per;
  auto merge = a.B * a.Hq <= kMergeFew ? attn_shared_merge_kernel<D, 8>
                                       : attn_shared_merge_kernel<D, 4>;
  return launch_dependent(merge, dim3(blocks), kMergeThreads, 0, stream, a, dec);
}

}  // namespace

size_t shared_part_rows(int Hq, int Hkv, int d, int n_groups, int n_rows, int max_pages) {
  const size_t tile = d == 256 ? Cfg<256>::kTileRows : Cfg<128>::kTileRows;
  const size_t pages = d == 256 ? Cfg<256>::kPages : Cfg<128>::kPages;
  const size_t pairs = static_cast<size_t>(n_rows) * (Hq / Hkv);
  const size_t units = (pairs / tile + n_groups) * Hkv * ((max_pages + pages - 1) / pages);
  return 2 * static_cast<size_t>(n_rows) * Hq +
         kItemRows * std::min<size_t>(units, kSharedMaxCtas);
}

cudaError_t launch_attn_shared(const SharedArgs& a, const DecodeLaunch& dec, int num_sms,
                               cudaStream_t stream) {
  if (dec.d == 64) return launch_shared<64>(a, dec, num_sms, stream);
  if (dec.d == 128) return launch_shared<128>(a, dec, num_sms, stream);
  if (dec.d == 256) return launch_shared<256>(a, dec, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace attn
