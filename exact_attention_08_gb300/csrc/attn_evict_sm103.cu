// Eviction from a paged cache by accumulated attention weight: of every row,
// layer and key head the keep[b] tokens with the largest mass stay.
//
// Order.  A token ranks by (protected, mass, lowest slot): protected are the
// first positions and the newest ones.  Its 32-bit key is the mass's bits made
// monotone (NaN lowest, both zeros alike), or all ones if protected; ties go to
// the lower slot.  The keep-th largest key T follows from three histogram
// passes over 11, 11 and 10 bits, and with it the tokens that stay: those above
// T, and of those at T the first few by slot.
//
// Moves.  Attention does not depend on the order of the keys, so only tokens
// that stay at or past slot keep[b] move: the k-th of them into the k-th
// evicted slot before keep[b].  Sources and destinations are apart, so no move
// waits for another, and a row 64 tokens over its budget of 1,024 moves about
// 60 tokens where closing the gaps in order would move about a thousand.
//
// Selection.  One CTA per (layer, row, key head).  Its keys go to shared memory once, and
// with them a histogram of their top 11 bits (sign, exponent, two bits of the
// mantissa: some 50 bins in use for masses, so few lanes meet in one); the next bits
// count only the keys of the bin that holds the keep-th largest, and the search ends as
// soon as that bin holds no more than are wanted, after two rounds as a rule.  Another
// look at the keys leaves two bits a token (above T, at T) as words of 32, and ties,
// holes and moves are counted over words.  Rows of up to kSmallRow tokens, of up to kMaxCached
// and longer ones have kernels of their own, which run side by side where the table
// is wide enough for them.  Rows past kMaxCached do not fit in shared memory: they are
// read again from memory for each of six steps (attn_evict_select_long_kernel).
//
// A CTA runs through its code once, so the code's size is its time as much as the work:
// with every loop unrolled (62 KB) rows of 1,088 tokens took 23 us.
//
// Split.  The selecting CTA writes its moves as (from, to) pairs and moves mass and
// position.  The keys and values are then moved by the whole GPU, launched as a
// programmatic dependent, 16 bytes a thread and four in flight.
#include "attn_internal.h"

#include <algorithm>

namespace attn {
namespace {

constexpr int kPage = 16;
constexpr int kThreads = 1024;  // of the kernel for long rows
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;
// Selecting CTAs for every SM, and slots of a row, from and up to which the selecting CTA copies
// too (512 units, 64 tokens over a budget of 1,024: 29.1 us on the device either way, and a
// launch less; 3,000 over it, 100 by two kernels and 113 by one; 128 units, 41 and 76).
constexpr int kFusedPerSm = 2, kFusedSlots = 2048;
constexpr int kMaxCached = 40960;  // tokens whose keys fit in a CTA's shared memory (160 KB)
// Threads of the selecting CTA: rows of up to 4,096 tokens take 256 (a longer block waits
// longer at its barriers), longer ones 384, up to four CTAs an SM.
constexpr int kSmallRow = 4096, kSmallThreads = 256, kLargeThreads = 384;
constexpr uint32_t kProtected = 0xffffffffu;

// Larger mass, larger key; 0 for NaN.
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int2* unit_moves(const EvictArgs& a, int unit) {
  return reinterpret_cast<int2*>(a.ws) + static_cast<size_t>(unit) * a.most_moves;
}
// Row of a pool (page * 16 + token) that holds a slot.
__device__ __forceinline__ int pool_row(const EvictArgs& a, int b, int slot) {
  return a.page_table[static_cast<size_t>(b) * a.max_pages + slot / kPage] * kPage + slot % kPage;
}
__device__ __forceinline__ int* unit_count(const EvictArgs& a, int unit) {
  return a.ws + 2 * static_cast<size_t>(a.units) * a.most_moves + unit;
}

// Sum before this thread and total over the block (warp_part: kWarps ints).
__device__ __forceinline__ int block_scan(int v, int* warp_part, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_part[warp] = x;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int p = warp_part[w];
    if (w < warp) base += p;
    all += p;
  }
  *total = all;
  return base + x - v;
}

// Keys and values of a unit's moves (pool rows), by the threads of one CTA: 2 d / 8 vectors of
// 16 bytes each, all in one index, four in flight a thread.
__device__ __forceinline__ void copy_moves(const EvictArgs& a, int layer, int h, const int2* moves,
                                           int count) {
  const size_t layer0 = static_cast<size_t>(layer) * a.num_pages * kPage;
  const int shift = a.vecs == 8 ? 4 : a.vecs == 16 ? 5 : 6;  // of 2 vecs
  const int total = count << shift, step = blockDim.x;
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < total; i0 += step * kCopyVecs) {
    uint4 v[kCopyVecs];
    uint4* to[kCopyVecs];
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j) {
      const int i = i0 + j * step;
      to[j] = nullptr;
      if (i >= total) continue;
      const int2 m = moves[i >> shift];
      const int r = i & (2 * a.vecs - 1);
      uint4* base = (r < a.vecs ? a.k_pages : a.v_pages) + (r & (a.vecs - 1));
      v[j] = base[((layer0 + m.x) * a.Hkv + h) * a.vecs];
      to[j] = base + ((layer0 + m.y) * a.Hkv + h) * a.vecs;
    }
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j)
      if (to[j] != nullptr) *to[j] = v[j];
  }
}

// Whether a row is to be cut that has more than `from` tokens and `to` at most.
__device__ __forceinline__ bool any_row(const EvictArgs& a, int from, int to) {
  bool any = false;
#pragma unroll 1
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    const int L = a.seqlens[b];
    any |= L > from && L <= to;
  }
  return __syncthreads_or(any);
}

// Selecting kernels for other lengths run side by side (each started by the one before): the
// first block of each leaves only when the kernel before it is done, so that what follows the
// last one follows them all.
__device__ __forceinline__ void leave_last() {
  if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Rows of any length: the keys are formed again for every step.  What bounds it is the loads one
// CTA has in flight: 1,024 threads with four tokens each take a row of 100,000 tokens in
// 163 us, 512 threads with one in 575.
__global__ void __launch_bounds__(kThreads) attn_evict_select_long_kernel(const EvictArgs a) {
  __shared__ int s_hist[kBins];
  __shared__ int s_part[kWarps];
  __shared__ int s_flag, s_newest, s_bin, s_above;
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool any = any_row(a, kMaxCached, INT32_MAX);
#pragma unroll 1
  for (int unit = blockIdx.x; any && unit < a.units; unit += gridDim.x) {
    __syncthreads();
    const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.B, layer = unit / (a.Hkv * a.B);
    const int L = a.seqlens[b], K = a.keep[b];
    const int cap = min(a.slots, a.max_pages * kPage);
    const bool lead = h == 0 && layer == 0;
    if (L <= kMaxCached || L > cap || K <= 0 || K >= L) continue;  // not one of this kernel's
    if (tid == 0) {
      s_flag = 0;
      s_newest = INT32_MIN;
    }
    __syncthreads();
    // Every page of the row must be one of the pool, and the pages written to must
    // be the row's alone.
    {
      const int* row = a.page_table + static_cast<size_t>(b) * a.max_pages;
      const int pages = (L + kPage - 1) / kPage, written = (K + kPage - 1) / kPage;
      bool wrong = false;
#pragma unroll 1
      for (int i = tid; i < pages; i += kThreads) {
        const int p = row[i];
        if (p < 0 || p >= a.num_pages)
          wrong = true;
        else if (a.refs != nullptr && i < written && a.refs[p] > 1)
          wrong = true;
      }
      if (wrong) s_flag = 1;
    }
    float* mass = a.mass + static_cast<size_t>(unit) * a.slots;
    int* pos = a.positions + static_cast<size_t>(unit) * a.slots;
    if (a.recent > 0) {
      int newest = INT32_MIN;
#pragma unroll 4
      for (int t = tid; t < L; t += kThreads) newest = max(newest, pos[t]);
      newest = __reduce_max_sync(0xffffffffu, newest);
      if (lane == 0) atomicMax(&s_newest, newest);
    }
    __syncthreads();
    if (s_flag) {
      if (tid == 0) {
        *unit_count(a, unit) = 0;
        if (lead) a.new_seqlens[b] = L;
        atomicOr(a.status, kStatusBadInput);
      }
      continue;
    }
    const long long recent_from =
        a.recent > 0 ? static_cast<long long>(s_newest) - a.recent : INT64_MAX;
    // The keys of this lane's tokens of the 128 from t on: t + lane, t + 32 + lane, ...  All loads
    // are in flight together; a token past the row's last gets the key of that one.
    auto make_keys = [&](int t, uint32_t (&key)[4]) {
      int p[4];
      float m[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = min(t + 32 * j + lane, L - 1);
        p[j] = pos[at];
        m[j] = mass[at];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        key[j] = (p[j] < a.n_sink || p[j] > recent_from) ? kProtected : mass_key(m[j]);
    };

    // ---- the K-th largest key: its bits from the top, 11, 11 and 10 of them
    uint32_t prefix = 0;
    int want = K;  // how many are still to be found among the keys that share the prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bits = pass == 2 ? 10 : 11;
#pragma unroll 1
      for (int i = tid; i < kBins; i += kThreads) s_hist[i] = 0;
      __syncthreads();
      const uint32_t mask = (1u << bits) - 1u;
#pragma unroll 1
      for (int t = warp * 128; t < L; t += kWarps * 128) {
        uint32_t key[4];
        make_keys(t, key);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t up = pass == 0 ? 0u : key[j] >> (shift + bits);
          if (t + 32 * j + lane < L && up == prefix) atomicAdd(&s_hist[(key[j] >> shift) & mask], 1);
        }
      }
      __syncthreads();
      // from the largest bin down: the bin in which the want-th key falls
      constexpr int kPer = kBins / kThreads;
      int local[kPer], sum = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        local[j] = s_hist[kBins - 1 - (tid * kPer + j)];
        sum += local[j];
      }
      int all;
      int before = block_scan(sum, s_part, &all);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (before < want && want <= before + local[j]) {
          s_bin = kBins - 1 - (tid * kPer + j);
          s_above = before;
        }
        before += local[j];
      }
      __syncthreads();
      prefix = (prefix << bits) | static_cast<uint32_t>(s_bin);
      want -= s_above;
      __syncthreads();
    }
    const uint32_t T = prefix;  // `want` of the tokens with key T stay, the first by slot

    // ---- ranks: every warp owns a run of slots
    const int run = ((L + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int t0 = min(warp * run, L), t1 = min(t0 + run, L);
    const uint32_t below = (1u << lane) - 1u;
    int ties = 0;
#pragma unroll 1
    for (int t = t0; t < t1; t += 128) {
      uint32_t key[4];
      make_keys(t, key);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        ties += __popc(__ballot_sync(0xffffffffu, t + 32 * j + lane < t1 && key[j] == T));
    }
    if (lane == 0) s_part[warp] = ties;
    __syncthreads();
    int tie_base = 0;
#pragma unroll 1
    for (int w = 0; w < warp; ++w) tie_base += s_part[w];
    __syncthreads();
    int2* moves = unit_moves(a, unit);
    int hole_base = 0, mover_base = 0, total = 0;
#pragma unroll 1
    for (int phase = 0; phase < 2; ++phase) {  // count, then write
      int tie_rank = tie_base, holes = hole_base, movers = mover_base;
#pragma unroll 1
      for (int t = t0; t < t1; t += 128) {
        uint32_t key[4];
        make_keys(t, key);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = t + 32 * j + lane;
          const bool valid = at < t1, tie = valid && key[j] == T;
          const uint32_t tie_mask = __ballot_sync(0xffffffffu, tie);
          const bool stays =
              valid && (key[j] > T || (tie && tie_rank + __popc(tie_mask & below) < want));
          tie_rank += __popc(tie_mask);
          const uint32_t hole = __ballot_sync(0xffffffffu, valid && !stays && at < K);
          const uint32_t mover = __ballot_sync(0xffffffffu, stays && at >= K);
          if (phase == 1) {
            if ((hole >> lane) & 1u) moves[holes + __popc(hole & below)].y = at;
            if ((mover >> lane) & 1u) moves[movers + __popc(mover & below)].x = at;
          }
          holes += __popc(hole);
          movers += __popc(mover);
        }
      }
      if (phase == 0) {
        int* s_movers = s_hist;  // free by now
        if (lane == 0) {
          s_part[warp] = holes;
          s_movers[warp] = movers;
        }
        __syncthreads();
#pragma unroll 1
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) {
            hole_base += s_part[w];
            mover_base += s_movers[w];
          }
          total += s_part[w];
        }
      }
    }
    __syncthreads();
#pragma unroll 2
    for (int i = tid; i < total; i += kThreads) {
      const int2 m = moves[i];
      mass[m.y] = mass[m.x];
      pos[m.y] = pos[m.x];
      moves[i] = make_int2(pool_row(a, b, m.x), pool_row(a, b, m.y));
    }
    if (tid == 0) {
      *unit_count(a, unit) = total;
      if (lead) a.new_seqlens[b] = K;
    }
  }
  leave_last();
}

// Sum before this thread and total over a block of up to 16 warps (part: 32 values).
template <typename T>
__device__ __forceinline__ T scan_block(T v, T* part, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  T p = lane < warps ? part[lane] : 0;
  T sum = p;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  *total = __shfl_sync(0xffffffffu, sum, warps - 1);
  return x - v + __shfl_sync(0xffffffffu, sum - p, warp);
}

// Lowest n set bits of x (all of them in every word but one).
__device__ __forceinline__ uint32_t lowest_bits(uint32_t x, int n) {
#pragma unroll 1
  while (__popc(x) > max(n, 0)) x ^= 0x80000000u >> __clz(x);
  return x;
}

// Rows whose keys fit in shared memory: keys [slots rounded up to 32], then two words for
// every 32 of them.
// kFours: rows of mass and positions start on 16 bytes, four tokens a load.  kCopies: the keys
// and values are moved here too.
template <bool kFours, bool kCopies>
__device__ __forceinline__ void select_row(const EvictArgs& a, int words, int unit, int layer, int b,
                                           int h, int L, int K) {
  extern __shared__ __align__(16) uint32_t s_keys[];  // (read four keys at a time)
  __shared__ int s_hist[kBins];
  __shared__ int s_group[kBins / 32];
  __shared__ int s_part[32];
  __shared__ long long s_part2[32];
  __shared__ int s_flag, s_newest, s_bin, s_want;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const int warps = threads >> 5;
  const bool lead = h == 0 && layer == 0;
  float* mass = a.mass + static_cast<size_t>(unit) * a.slots;
  int* pos = a.positions + static_cast<size_t>(unit) * a.slots;
  if (tid == 0) {
    s_flag = 0;
    s_newest = INT32_MIN;
  }
#pragma unroll 1
  for (int i = tid; i < kBins; i += threads) s_hist[i] = 0;
  // Every page of the row must be one of the pool, and the pages written to must
  // be the row's alone.
  bool wrong = false;
  {
    const int* row = a.page_table + static_cast<size_t>(b) * a.max_pages;
    const int pages = (L + kPage - 1) / kPage, written = (K + kPage - 1) / kPage;
#pragma unroll 1
    for (int i = tid; i < pages; i += threads) {
      const int p = row[i];
      if (p < 0 || p >= a.num_pages)
        wrong = true;
      else if (a.refs != nullptr && i < written && a.refs[p] > 1)
        wrong = true;
    }
  }
  // tokens four by four; those of the last, shorter group one by one
  const int fours = kFours ? L / 4 : 0;
  int newest = INT32_MIN;
  if (a.recent > 0) {
#pragma unroll 2
    for (int i = tid; i < fours; i += threads) {
      const int4 p = reinterpret_cast<const int4*>(pos)[i];
      newest = max(max(max(newest, p.x), p.y), max(p.z, p.w));
    }
#pragma unroll 1
    for (int t = 4 * fours + tid; t < L; t += threads) newest = max(newest, pos[t]);
    newest = __reduce_max_sync(0xffffffffu, newest);
  }
  __syncthreads();
  if (lane == 0 && a.recent > 0) atomicMax(&s_newest, newest);
  if (wrong) s_flag = 1;
  __syncthreads();
  if (s_flag) {
    if (tid == 0) {
      *unit_count(a, unit) = 0;
      if (lead) a.new_seqlens[b] = L;
      atomicOr(a.status, kStatusBadInput);
    }
    return;
  }
  const long long recent_from =
      a.recent > 0 ? static_cast<long long>(s_newest) - a.recent : INT64_MAX;
  // (position > recent_from, as a 32-bit comparison: INT32_MAX + 1 stands for none)
  const bool all_recent = recent_from < INT32_MIN;
  const int after = all_recent ? INT32_MIN
                               : static_cast<int>(min(recent_from, static_cast<long long>(INT32_MAX)));
  auto make_key = [&](float m, int p) -> uint32_t {
    const uint32_t k = (p < a.n_sink || p > after || all_recent) ? kProtected : mass_key(m);
    atomicAdd(&s_hist[k >> 21], 1);
    return k;
  };
#pragma unroll 2
  for (int i = tid; i < fours; i += threads) {
    const int4 p = reinterpret_cast<const int4*>(pos)[i];
    const float4 m = reinterpret_cast<const float4*>(mass)[i];
    reinterpret_cast<uint4*>(s_keys)[i] = make_uint4(make_key(m.x, p.x), make_key(m.y, p.y),
                                                     make_key(m.z, p.z), make_key(m.w, p.w));
  }
#pragma unroll 1
  for (int t = 4 * fours + tid; t < L; t += threads) s_keys[t] = make_key(mass[t], pos[t]);
  // whole words of keys from here on: the last one is filled up with the least
  for (int t = L + tid; t < (L + 31) / 32 * 32; t += threads) s_keys[t] = 0u;
  __syncthreads();

  // ---- the threshold's bits from the top, 11, 11 and 10 of them, until the keys that share
  // them are just as many as are still wanted
  uint32_t T = 0;   // the threshold's bits from `shift` up
  int want = K;     // how many of the keys with these bits stay
  int shift = 21;
#pragma unroll 1
  for (;;) {
    // the bin in which the want-th key falls, from the largest down: groups of 32 first
#pragma unroll 1
    for (int j = warp; j < kBins / 32; j += warps) {
      const int n = __reduce_add_sync(0xffffffffu, s_hist[kBins - 1 - (j * 32 + lane)]);
      if (lane == 0) s_group[j] = n;
    }
    __syncthreads();
    if (warp == 0) {
      int lo = s_group[lane], x = lo;
      int hi = s_group[32 + lane], y = hi;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) x += u, y += v;
      }
      y += __shfl_sync(0xffffffffu, x, 31);
      const uint32_t hit0 = __ballot_sync(0xffffffffu, x >= want);
      const uint32_t hit1 = __ballot_sync(0xffffffffu, y >= want);
      const int at = __ffs(hit0 ? hit0 : hit1) - 1;
      const int before = __shfl_sync(0xffffffffu, hit0 ? x - lo : y - hi, at);
      const int group = hit0 ? at : 32 + at;
      const int n = s_hist[kBins - 1 - (group * 32 + lane)];
      x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += u;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, before + x >= want);
      if (lane == __ffs(hit) - 1) {
        s_bin = kBins - 1 - (group * 32 + lane);
        s_want = want - (before + x - n);
      }
    }
    __syncthreads();
    const int bin = s_bin, in_bin = s_hist[bin];
    T = shift == 0 ? (T << 10) | bin : (T << 11) | bin;
    want = s_want;
    if (shift == 0 || in_bin == want) break;
    const int next = shift == 21 ? 10 : 0;
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < kBins; i += threads) s_hist[i] = 0;
    __syncthreads();
    const uint32_t mask = next == 0 ? 0x3ffu : 0x7ffu;
#pragma unroll 1
    for (int i = tid; i < (L + 3) / 4; i += threads) {
      const uint4 k4 = reinterpret_cast<const uint4*>(s_keys)[i];
      const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((k[e] >> shift) == T && 4 * i + e < L) atomicAdd(&s_hist[(k[e] >> next) & mask], 1);
    }
    __syncthreads();
    shift = next;
  }

  // ---- above T and at T, a bit a token
  uint32_t* s_gt = s_keys + words * 32;
  uint32_t* s_eq = s_gt + words;
  const int n_words = (L + 31) / 32;
#pragma unroll 1
  for (int i = warp; i < n_words; i += warps) {
    const int t = i * 32 + lane;
    const uint32_t k = t < L ? s_keys[t] >> shift : 0u;
    const uint32_t gt = __ballot_sync(0xffffffffu, t < L && k > T);
    const uint32_t eq = __ballot_sync(0xffffffffu, t < L && k == T);
    if (lane == 0) {
      s_gt[i] = gt;
      s_eq[i] = eq;
    }
  }
  __syncthreads();
  // ---- ties by slot, then holes and movers: a run of words a thread
  const int per = (n_words + threads - 1) / threads;
  const int w0 = min(tid * per, n_words), w1 = min(w0 + per, n_words);
  int ties = 0;
#pragma unroll 1
  for (int i = w0; i < w1; ++i) ties += __popc(s_eq[i]);
  int all_ties;
  int rank = scan_block(ties, s_part, &all_ties);
  int holes = 0, movers = 0;
#pragma unroll 1
  for (int i = w0; i < w1; ++i) {
    const uint32_t eq = s_eq[i];
    const uint32_t stay = s_gt[i] | lowest_bits(eq, want - rank);
    rank += __popc(eq);
    s_gt[i] = stay;
    // slots of this word before K
    const int below = min(max(K - i * 32, 0), 32);
    const uint32_t low = below == 32 ? 0xffffffffu : (1u << below) - 1u;
    holes += __popc(~stay & low);
    movers += __popc(stay & ~low);
  }
  long long total2;
  const long long first = scan_block((static_cast<long long>(holes) << 32) | movers, s_part2, &total2);
  int at_hole = static_cast<int>(first >> 32), at_mover = static_cast<int>(first & 0xffffffff);
  const int total = static_cast<int>(total2 & 0xffffffff);
  int2* moves = unit_moves(a, unit);
#pragma unroll 1
  for (int i = w0; i < w1; ++i) {
    const uint32_t stay = s_gt[i];
    const int below = min(max(K - i * 32, 0), 32);
    const uint32_t low = below == 32 ? 0xffffffffu : (1u << below) - 1u;
#pragma unroll 1
    for (uint32_t x = ~stay & low; x != 0; x &= x - 1) moves[at_hole++].y = i * 32 + __ffs(x) - 1;
#pragma unroll 1
    for (uint32_t x = stay & ~low; x != 0; x &= x - 1) moves[at_mover++].x = i * 32 + __ffs(x) - 1;
  }
  if (tid == 0) {
    *unit_count(a, unit) = total;
    if (lead) a.new_seqlens[b] = K;
  }
  __syncthreads();
#pragma unroll 2
  for (int i = tid; i < total; i += threads) {
    const int2 m = moves[i];
    mass[m.y] = mass[m.x];
    pos[m.y] = pos[m.x];
    moves[i] = make_int2(pool_row(a, b, m.x), pool_row(a, b, m.y));
  }
  if constexpr (kCopies) {
    __syncthreads();
    copy_moves(a, layer, h, moves, total);
  }
}

// Rows of `to` tokens at most, a CTA each, and those that are not cut.
template <bool kFours, bool kCopies>
__global__ void __launch_bounds__(kLargeThreads, 4) attn_evict_select_kernel(const EvictArgs a,
                                                                             int words, int to) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int unit = blockIdx.x;
  const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.B, layer = unit / (a.Hkv * a.B);
  const int L = a.seqlens[b], K = a.keep[b];
  const bool bad = L < 0 || L > min(a.slots, a.max_pages * kPage) || K < 0;
  if (bad || K >= L || K == 0) {
    if (threadIdx.x == 0) {
      *unit_count(a, unit) = 0;
      if (h == 0 && layer == 0) a.new_seqlens[b] = (bad || K >= L) ? L : 0;
      if (bad) atomicOr(a.status, kStatusBadInput);
    }
    return;
  }
  if (L <= to) select_row<kFours, kCopies>(a, words, unit, layer, b, h, L, K);
}

// Rows of more than kSmallRow tokens, `to` at most.  The table may be far wider than its rows are
// long, so this kernel is launched beside the one above wherever it could be needed, with
// as many CTAs as are resident (64 rows of 1,000 tokens in a table of 8,192 pages: 18 us, with
// one kernel for the longest row possible 62; 8 layers of rows of 8,200 tokens 103 instead
// of 100.5).
template <bool kFours>
__global__ void __launch_bounds__(kLargeThreads, 4) attn_evict_select_wide_kernel(
    const EvictArgs a, int words, int to) {
  asm volatile("griddepcontrol.launch_dependents;");
  const bool any = any_row(a, kSmallRow, to);
#pragma unroll 1
  for (int unit = blockIdx.x; any && unit < a.units; unit += gridDim.x) {
    const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.B, layer = unit / (a.Hkv * a.B);
    const int L = a.seqlens[b], K = a.keep[b];
    if (L <= kSmallRow || L > to || K <= 0 || K >= L) continue;
    __syncthreads();
    select_row<kFours, false>(a, words, unit, layer, b, h, L, K);
  }
  leave_last();
}

// copy_moves by a.copy_blocks blocks a unit.
template <int kVecs>
__global__ void __launch_bounds__(kCopyThreads) attn_evict_copy_kernel(const EvictArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int unit = blockIdx.x / a.copy_blocks, part = blockIdx.x % a.copy_blocks;
  const int h = unit % a.Hkv, layer = unit / (a.Hkv * a.B);
  const int count = *unit_count(a, unit);
  const int2* moves = unit_moves(a, unit);
  const size_t layer0 = static_cast<size_t>(layer) * a.num_pages * kPage;
  const long long total = static_cast<long long>(count) * (2 * kVecs);
  const long long step = static_cast<long long>(a.copy_blocks) * kCopyThreads;
#pragma unroll 1
  for (long long i0 = static_cast<long long>(part) * kCopyThreads + threadIdx.x; i0 < total;
       i0 += step * kCopyVecs) {
    uint4 v[kCopyVecs];
    uint4* to[kCopyVecs];
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j) {
      const long long i = i0 + j * step;
      to[j] = nullptr;
      if (i >= total) continue;
      const int2 m = moves[i / (2 * kVecs)];
      const int r = static_cast<int>(i % (2 * kVecs));
      uint4* base = (r < kVecs ? a.k_pages : a.v_pages) + (r < kVecs ? r : r - kVecs);
      v[j] = base[((layer0 + m.x) * a.Hkv + h) * kVecs];
      to[j] = base + ((layer0 + m.y) * a.Hkv + h) * kVecs;
    }
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j)
      if (to[j] != nullptr) *to[j] = v[j];
  }
}

}  // namespace

cudaError_t launch_attn_evict(EvictArgs a, int num_sms, cudaStream_t stream) {
  const int cap = std::min(a.slots, a.max_pages * kPage);
  // Selecting CTAs that fill the GPU by themselves, of short rows, move their keys and values
  // too; others leave that to a kernel of some sixteen blocks for every SM (and no more than
  // there can be steps).
  const int per_step = kCopyThreads * kCopyVecs;
  const long long most = (static_cast<long long>(a.most_moves) * 2 * a.vecs + per_step - 1) /
                         per_step;
  a.copy_blocks = cap <= kFusedSlots && a.units >= kFusedPerSm * num_sms
                      ? 0
                      : static_cast<int>(std::max(
                            1LL, std::min(most, (16LL * num_sms + a.units - 1) / a.units)));
  cudaError_t e;
  const bool fours = a.slots % 4 == 0 && reinterpret_cast<uintptr_t>(a.mass) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.positions) % 16 == 0;
  const bool copies = a.copy_blocks == 0;
  auto words_of = [](int tokens) { return (tokens + 31) / 32; };
  auto bytes_of = [](int words) { return static_cast<size_t>(words) * 34 * 4; };
  {
    const int to = std::min(cap, kSmallRow), words = words_of(to);
    auto select = fours ? (copies ? attn_evict_select_kernel<true, true>
                                  : attn_evict_select_kernel<true, false>)
                        : (copies ? attn_evict_select_kernel<false, true>
                                  : attn_evict_select_kernel<false, false>);
    select<<<a.units, kSmallThreads, bytes_of(words), stream>>>(a, words, to);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (cap > kSmallRow) {
    const int to = std::min(cap, kMaxCached), words = words_of(to);
    static SharedMemoryLimit limits[2];
    auto select = fours ? attn_evict_select_wide_kernel<true> : attn_evict_select_wide_kernel<false>;
    e = limits[fours].raise(select, bytes_of(words_of(kMaxCached)));
    if (e != cudaSuccess) return e;
    const int resident =
        std::max(1, std::min(4, static_cast<int>((224 << 10) / (bytes_of(words) + (11 << 10)))));
    e = launch_dependent(select, dim3(std::min(a.units, resident * num_sms)), kLargeThreads,
                         bytes_of(words), stream, a, words, to);
    if (e != cudaSuccess) return e;
  }
  if (cap > kMaxCached) {
    e = launch_dependent(attn_evict_select_long_kernel, dim3(std::min(a.units, 2 * num_sms)),
                         kThreads, 0, stream, a);
    if (e != cudaSuccess) return e;
  }
  if (copies) return cudaSuccess;
  auto copy = a.vecs == 8    ? attn_evict_copy_kernel<8>
              : a.vecs == 16 ? attn_evict_copy_kernel<16>
                             : attn_evict_copy_kernel<32>;
  return launch_dependent(copy, dim3(static_cast<unsigned>(a.copy_blocks) * a.units), kCopyThreads,
                          0, stream, a);
}

}  // namespace attn
