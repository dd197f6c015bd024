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
// Split.  One CTA per (layer, row, key head) selects: its keys sit in shared
// memory (16 bytes of histogram and key work a token against 8 read), and it
// writes its moves as (from, to) pairs and moves mass and position.  The keys
// and values are then moved by the whole GPU, launched as a programmatic
// dependent, 16 bytes a thread and four in flight.
#include "attn_internal.h"

#include <algorithm>

namespace attn {
namespace {

constexpr int kPage = 16;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;
constexpr int kMaxCached = 40960;  // tokens whose keys fit in a CTA's shared memory (160 KB)
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

template <bool kCached>
__global__ void __launch_bounds__(kThreads) attn_evict_select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t s_keys[];
  __shared__ int s_hist[kBins];
  __shared__ int s_part[kWarps];
  __shared__ int s_flag, s_newest, s_bin, s_above;
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.x;
  const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.B, layer = unit / (a.Hkv * a.B);
  const int L = a.seqlens[b], K = a.keep[b];
  const int cap = min(a.slots, a.max_pages * kPage);
  const bool lead = h == 0 && layer == 0;
  const bool bad = L < 0 || L > cap || K < 0;
  if (bad || K >= L || K == 0) {
    if (tid == 0) {
      *unit_count(a, unit) = 0;
      if (lead) a.new_seqlens[b] = (bad || K >= L) ? L : 0;
      if (bad) atomicOr(a.status, kStatusBadInput);
    }
    return;
  }
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
    return;
  }
  const long long recent_from =
      a.recent > 0 ? static_cast<long long>(s_newest) - a.recent : INT64_MAX;
  auto make_key = [&](int t) -> uint32_t {
    const int p = pos[t];
    return (p < a.n_sink || p > recent_from) ? kProtected : mass_key(mass[t]);
  };
  if (kCached) {
    for (int t = tid; t < L; t += kThreads) s_keys[t] = make_key(t);
    __syncthreads();
  }
  auto key_of = [&](int t) -> uint32_t { return kCached ? s_keys[t] : make_key(t); };

  // ---- the K-th largest key: its bits from the top, 11, 11 and 10 of them
  uint32_t prefix = 0;
  int want = K;  // how many are still to be found among the keys that share the prefix
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < kBins; i += kThreads) s_hist[i] = 0;
    __syncthreads();
    const uint32_t mask = (1u << bits) - 1u;
    for (int t = tid; t < L; t += kThreads) {
      const uint32_t k = key_of(t);
      const uint32_t up = pass == 0 ? 0u : k >> (shift + bits);
      if (up == prefix) atomicAdd(&s_hist[(k >> shift) & mask], 1);
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
  for (int t = t0; t < t1; t += 32) {
    const bool tie = t + lane < t1 && key_of(t + lane) == T;
    ties += __popc(__ballot_sync(0xffffffffu, tie));
  }
  if (lane == 0) s_part[warp] = ties;
  __syncthreads();
  int tie_base = 0;
  for (int w = 0; w < warp; ++w) tie_base += s_part[w];
  __syncthreads();
  int2* moves = unit_moves(a, unit);
  int hole_base = 0, mover_base = 0, total = 0;
#pragma unroll 1
  for (int phase = 0; phase < 2; ++phase) {  // count, then write
    int tie_rank = tie_base, holes = hole_base, movers = mover_base;
    for (int t = t0; t < t1; t += 32) {
      const int at = t + lane;
      const bool valid = at < t1;
      const uint32_t k = valid ? key_of(at) : 0u;
      const bool tie = valid && k == T;
      const uint32_t tie_mask = __ballot_sync(0xffffffffu, tie);
      const bool stays = valid && (k > T || (tie && tie_rank + __popc(tie_mask & below) < want));
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
    if (phase == 0) {
      int* s_movers = s_hist;  // free by now
      if (lane == 0) {
        s_part[warp] = holes;
        s_movers[warp] = movers;
      }
      __syncthreads();
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
  for (int i = tid; i < total; i += kThreads) {
    const int2 m = moves[i];
    mass[m.y] = mass[m.x];
    pos[m.y] = pos[m.x];
  }
  if (tid == 0) {
    *unit_count(a, unit) = total;
    if (lead) a.new_seqlens[b] = K;
  }
}

// Keys and values of the moves: 2 d / 8 vectors of 16 bytes each, the vectors of
// a unit's moves in one index.
template <int kVecs>
__global__ void __launch_bounds__(kCopyThreads) attn_evict_copy_kernel(const EvictArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int unit = blockIdx.x / a.copy_blocks, part = blockIdx.x % a.copy_blocks;
  const int h = unit % a.Hkv, b = (unit / a.Hkv) % a.B, layer = unit / (a.Hkv * a.B);
  const int count = *unit_count(a, unit);
  const int2* moves = unit_moves(a, unit);
  const int* row = a.page_table + static_cast<size_t>(b) * a.max_pages;
  const size_t pool = static_cast<size_t>(layer) * a.num_pages;
  const long long total = static_cast<long long>(count) * (2 * kVecs);
  const long long step = static_cast<long long>(a.copy_blocks) * kCopyThreads;
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
      uint4* base = r < kVecs ? a.k_pages : a.v_pages;
      const int vec = r < kVecs ? r : r - kVecs;
      auto at = [&](int t) {
        return (((pool + row[t / kPage]) * kPage + t % kPage) * a.Hkv + h) * kVecs + vec;
      };
      v[j] = base[at(m.x)];
      to[j] = base + at(m.y);
    }
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j)
      if (to[j] != nullptr) *to[j] = v[j];
  }
}

}  // namespace

cudaError_t launch_attn_evict(EvictArgs a, int num_sms, cudaStream_t stream) {
  const int cap = std::min(a.slots, a.max_pages * kPage);
  const bool cached = cap <= kMaxCached;
  const size_t smem = cached ? static_cast<size_t>(cap) * 4 : 0;
  auto select = cached ? attn_evict_select_kernel<true> : attn_evict_select_kernel<false>;
  static SharedMemoryLimit limit;
  cudaError_t e = limit.raise(attn_evict_select_kernel<true>, kMaxCached * 4);
  if (e != cudaSuccess) return e;
  select<<<a.units, kThreads, smem, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // about eight blocks for every SM, no more than there can be steps
  const int per_step = kCopyThreads * kCopyVecs;
  const long long most = (static_cast<long long>(a.most_moves) * 2 * a.vecs + per_step - 1) /
                         per_step;
  a.copy_blocks = static_cast<int>(
      std::max(1LL, std::min(most, (8LL * num_sms + a.units - 1) / a.units)));
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(a.copy_blocks * a.units));
  auto copy = a.vecs == 8    ? attn_evict_copy_kernel<8>
              : a.vecs == 16 ? attn_evict_copy_kernel<16>
                             : attn_evict_copy_kernel<32>;
  e = cudaLaunchKernelEx(&cfg, copy, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace attn
