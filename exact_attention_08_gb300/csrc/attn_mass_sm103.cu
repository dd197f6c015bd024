// The attention weight that the keys of a paged cache get from a block of
// queries: mass(b, h, t) += sum over the query heads g of key head h and over
// the block's queries i that see key t of exp(scale q_ig . k_t - LSE_ig), the
// log-sum-exps being those of the block's attention.
//
// Product.  Keys are the rows: S^T = K Q^T, M = 128 keys, N = kQN queries, so a
// thread owns a key and its sum never leaves a register.  A query tile holds
// whole tokens with all their heads of the group (column = token * GP + head),
// loaded as one box of the q tensor.  With the LSE known there is no running
// maximum and no second product: one product and one exponential for each
// (query, key), and the tensor cores' 512 cycles for 128 x 128 x 128 against 512
// of the exponential units.
//
// Precision.  Scores, exponents and sums are fp32 (ex2.approx: 2^-22 of a weight), products
// of bf16 exact: a mass of thousands of weights is some 3.4e-7 of itself off fp64, where fp32
// torch operations on the same inputs are 4.4e-8 off.
//
// Operands.  With both in shared memory, M = N = 128, the tensor cores read 128 bytes
// of it a cycle, all there is, and the tiles' arrival and the LSEs come on top: 1,570
// cycles a unit (two row tiles against one query tile) instead of 1,024.  So a key
// tile with kMinTs query tiles or more is copied to tensor memory once and read from
// there as the A operand; the copy costs about a unit's time.
//
// Rows.  A page (16 tokens of one head) arrives in one copy, as two halves of [d / 64
// atoms][8 rows][128 bytes]: the eight-row groups of consecutive pages are evenly spaced,
// as the product's operand needs.
//
// Tile.  256 keys (two row tiles) against each query tile: one row tile alone
// would read 64 bytes of Q a cycle and SM from L2, more than it delivers.  Eight
// warps for each row tile, and a ring of S buffers, so that the next products run under the
// exponentials of these.
//
//   tensor memory  ring of S (kQN columns each), K of both row tiles (d / 2 columns each)
//   shared memory  K ring (256 keys a slot), Q ring, LSEs, barriers
//   warps          0-3 and 8-11 sums of row tile 0 (half the columns each), 4-7 and
//                  12-15 of row tile 1; 16 TMA producer; 17 MMA issuer (which waits
//                  for the next product's barriers between the halves of this one);
//                  18 LSEs of the query tiles (in column order, loaded a tile ahead)
//
// Split.  The work is cut into units, a query tile against a key tile, in the order
// (sequence, key head, key tile, query tile), and each of the persistent CTAs (one an
// SM) takes an equal run of them: causal triangles, windows and ragged lengths
// balance by themselves, and few keys with many queries still fill the GPU.  A plan
// kernel counts the units of every key tile.  A key tile that several CTAs share has
// one partial sum from each; partial sums go to workspace slot (key tile + CTA), both
// of which only grow along the order, and the last kernel adds them in CTA order
// and updates the mass: the same bits on every call.
//
// A query tile that stays the same from one key tile to the next (few queries that
// judge a long cache) is not loaded again: then the K stream alone is the traffic.
#include "attn_internal.h"
#include "sm103_ptx.cuh"

#include <algorithm>
#include <climits>
#include <cmath>

namespace attn {
namespace {

using namespace ptx;

constexpr int kPage = 16;
constexpr int kRows = 128;            // keys of a row tile
constexpr int kKeys = 2 * kRows;      // keys of a key tile
constexpr int kPagesPerTile = kKeys / kPage;
constexpr int kHalves = 2;  // warps that share 32 rows of a row tile, half the columns each
constexpr int kSumWarps = 8 * kHalves;
constexpr int kWarpProducer = kSumWarps;
constexpr int kWarpIssuer = kSumWarps + 1;
constexpr int kWarpLse = kSumWarps + 2;
constexpr int kThr = 32 * (kSumWarps + 3);
// What starting a key tile costs, in units (8,192 tokens, causal, 32 heads over 8: 245.1 us
// at 0, 235.4 at 2, 234.5 at 3, 234.9 at 4, 236.1 at 6; eight chunks of 8 to 512 queries, d =
// 256, 36.9, 35.6, 36.9, 37.4, 39.0; 64 prompts of 300 tokens 76.6, 80.1, 80.1, 80.0, 82.0; 8 of
// 2,000, 16 heads over 4, 81.2, 78.3, 78.0, 78.4, 79.5).
constexpr int kItemCost = 3;
// Query tiles from which a key tile is copied to tensor memory (8,192 tokens, causal: 257 us, 261
// without; from 8, 16 or 32 tiles on: within 1 % there, up to 3 % either way on short blocks).
constexpr int kMinTs = 4;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
  static constexpr int kAtoms = D / 64;
  static constexpr int kQN = D == 256 ? 64 : 128;  // queries (token, head) of a query tile
  static constexpr int kKSlots = D == 256 ? 1 : 2;
  static constexpr int kQSlots = D == 64 ? 4 : 3;
  static constexpr int kGroup = kAtoms * 1024;     // eight keys
  static constexpr int kPageBytes = 2 * kGroup;
  static constexpr int kKBytes = kPagesPerTile * kPageBytes;  // a K slot
  static constexpr int kQAtom = kQN * 128;
  static constexpr int kQBytes = kAtoms * kQAtom;  // a Q slot
  static constexpr int kOffQ = kKSlots * kKBytes;
  static constexpr int kOffLse = kOffQ + kQSlots * kQBytes;
  static constexpr int kOffBar = kOffLse + 2 * kQN * 4;
  static constexpr int kSBufs = D == 256 ? 4 : 3;
  static constexpr uint32_t kColA = kSBufs * kQN;
  static_assert(kColA + D <= 512, "tensor memory");
  static constexpr int kNumBars = 2 * kKSlots + 2 * kQSlots + 2 * kSBufs + 2 + 2 + 1 + 1;
  static constexpr int kSmem = kOffBar + (kNumBars + 1) * 8 + 1024;
  static_assert(kSmem <= 227 * 1024 - 512, "shared memory (512 bytes of it static)");
};


// One sequence: its queries and keys.  Lengths are at most 2^29 and the window at most the
// longest row, so that sums of three of them stay below 2^31.
struct Seq {
  int Lq, L, off, q_base;
};

__device__ __forceinline__ bool load_seq(const MassArgs& a, int b, Seq& s) {
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], L = a.seqlens_k[b];
  s.q_base = q0;
  s.Lq = q1 - q0;
  s.L = L;
  s.off = s.L - s.Lq;
  return q0 >= 0 && q1 >= q0 && q1 <= a.total_q && q1 - q0 <= a.max_Sq && L >= 0 &&
         L <= min(a.max_pages * kPage, a.slots);
}

__device__ __forceinline__ int key_tiles(const Seq& s) { return (s.L + kKeys - 1) / kKeys; }

// The query tile of a unit: its first token and its head group.
__device__ __forceinline__ int tile_token(const MassArgs& a, int u) {
  return (a.HC == 1 ? u : u / a.HC) * a.TQ;
}
__device__ __forceinline__ int tile_head(const MassArgs& a, int u) {
  return a.HC == 1 ? 0 : (u % a.HC) * a.GP;
}

// Query tiles (of TQ tokens) with a query that sees a key of key tile kt: the first, and how
// many.
__device__ __forceinline__ int query_tiles(const MassArgs& a, const Seq& s, int kt, int* first) {
  const int ka = kt * kKeys, kb = min(ka + kKeys, s.L) - 1;
  int lo = 0, hi = s.Lq - 1;
  if (a.causal) lo = max(lo, ka - s.off);
  if (a.window > 0 && ka >= a.n_sink) hi = min(hi, kb + a.window - 1 - s.off);
  *first = lo / a.TQ;
  return hi < lo ? 0 : hi / a.TQ - *first + 1;
}

__device__ __forceinline__ long long* ws_cum(const MassArgs& a, int b) {
  return a.ws_plan + static_cast<size_t>(b) * (a.max_kt + 1);
}
__device__ __forceinline__ long long* ws_base(const MassArgs& a) {  // [B + 1]
  return a.ws_plan + static_cast<size_t>(a.B) * (a.max_kt + 1);
}
// [B, max_kt] the first query tile of a key tile, and its units.
__device__ __forceinline__ int2* ws_tiles(const MassArgs& a, int b) {
  return reinterpret_cast<int2*>(ws_base(a) + a.B + 1) + static_cast<size_t>(b) * a.max_kt;
}

// ---------------------------------------------------------------- plan
// Work is measured in positions: a key tile with n units has kItemCost + n of them, the units
// last (so that a CTA with many short key tiles gets fewer units).  cum[b][kt]: positions
// of sequence b's key tiles before kt, one key head; cum[b][max_kt]: all.
constexpr int kPlanThreads = 256;
__global__ void __launch_bounds__(kPlanThreads) attn_mass_plan_kernel(const MassArgs a) {
  __shared__ long long s_part[kPlanThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;");
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Seq s;
  const bool ok = load_seq(a, b, s);
  if (!ok && tid == 0) atomicOr(a.status, kStatusBadInput);
  const int n = ok ? key_tiles(s) : 0;
  long long* cum = ws_cum(a, b);
  long long base = 0;
  for (int k0 = 0; k0 < n; k0 += kPlanThreads) {
    const int kt = k0 + tid;
    int first = 0;
    const int units = kt < n ? query_tiles(a, s, kt, &first) * a.HC : 0;
    if (kt < n) ws_tiles(a, b)[kt] = make_int2(first * a.HC, units);
    const long long v = units > 0 ? units + kItemCost : 0;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_part[warp] = x;
    __syncthreads();
    long long before = base, all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) before += s_part[w];
      all += s_part[w];
    }
    if (kt < n) cum[kt] = before + x - v;
    base += all;
  }
  if (tid == 0) cum[a.max_kt] = base;
}

// ---------------------------------------------------------------- the walk
// A CTA's run: the key tiles in order, each with its units.  Every role walks for itself; what
// a key tile has to do was worked out by the plan and is read one key tile ahead.
struct Walk {
  int b, h, kt, n, u;  // key tile; its units, and the next of them (below 0: positions before
                       // its first)
  int tile;            // query tile of unit 0 (times HC, by head groups)
  long long left;      // positions left in the run
  int tiles;           // key tiles of the sequence
  int2 next;           // query tile and units of the key tile behind this one
  const int2* plan;
  Seq s;
};

// Sequence w.b: its key tiles, none if it has no query.
__device__ __forceinline__ void walk_seq(const MassArgs& a, Walk& w) {
  w.tiles = load_seq(a, w.b, w.s) && w.s.Lq > 0 ? key_tiles(w.s) : 0;
}

// Key tile kt, or the first one behind it that a query sees: those between the sink keys and
// every query's window have no units.  (Five rows of 100,000 keys, window 1,024, 256
// queries each: 25 us, and 98 where a CTA walks them one by one.)  Worked out again at each
// step: state kept for it would not fit in the registers (8,192 tokens without a window
// 277 us instead of 242).
__device__ __forceinline__ int walk_tile(const MassArgs& a, const Walk& w, int kt) {
  if (a.window == 0 || kt < (a.n_sink + kKeys - 1u) / kKeys) return kt;
  return max(kt, (w.s.off - a.window + 1) / kKeys);
}

__device__ __forceinline__ void walk_row(const MassArgs& a, Walk& w, int kt) {
  w.plan = ws_tiles(a, w.b);
  w.kt = kt;
  const int2 t = w.plan[kt];
  w.tile = t.x;
  w.n = t.y;
  w.next = w.plan[min(walk_tile(a, w, kt + 1), w.tiles - 1)];
}

// The next key tile with units.
__device__ __forceinline__ bool walk_next(const MassArgs& a, Walk& w) {
  w.u = -kItemCost;
  while (w.left > 0) {
    const int kt = walk_tile(a, w, w.kt + 1);
    if (kt < w.tiles) {
      w.kt = kt;
      w.tile = w.next.x;
      w.n = w.next.y;
      w.next = w.plan[min(walk_tile(a, w, kt + 1), w.tiles - 1)];
    } else {
      if (++w.h >= a.Hkv) {
        w.h = 0;
        do {
          if (++w.b >= a.B) return false;
          walk_seq(a, w);
        } while (w.tiles == 0);
      }
      walk_row(a, w, walk_tile(a, w, 0));
    }
    if (w.n > 0) return true;
  }
  return false;
}

// Takes the positions before the current key tile's first unit; then, how many of its units
// belong to this run (none, if the run ends before them).
__device__ __forceinline__ int walk_units(Walk& w) {
  if (w.u < 0) {
    w.left += w.u;
    w.u = 0;
  }
  return static_cast<int>(max(0LL, min(static_cast<long long>(w.n - w.u), w.left)));
}

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}

// Adds a thread's weights over kCols columns: all of them, those in [lo, hi) where both are
// multiples of four (the group's heads are), or those in any [lo, hi).
enum MaskMode { kAll, kFours, kAny };
template <int kCols, MaskMode kMask>
__device__ __forceinline__ void add_columns(const uint32_t* x, const float* nl, float scale2,
                                            int lo, int hi, float2* acc) {
  const float2 sc = make_float2(scale2, scale2);
#pragma unroll
  for (int c = 0; c < kCols; c += 4) {
    const float4 l = *reinterpret_cast<const float4*>(nl + c);
    float2 u = fma2(make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sc,
                    make_float2(l.x, l.y));
    float2 v = fma2(make_float2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sc,
                    make_float2(l.z, l.w));
    u = make_float2(ex2_approx(u.x), ex2_approx(u.y));
    v = make_float2(ex2_approx(v.x), ex2_approx(v.y));
    if (kMask == kAny) {
      u.x = c >= lo && c < hi ? u.x : 0.f;
      u.y = c + 1 >= lo && c + 1 < hi ? u.y : 0.f;
      v.x = c + 2 >= lo && c + 2 < hi ? v.x : 0.f;
      v.y = c + 3 >= lo && c + 3 < hi ? v.y : 0.f;
    }
    if (kMask == kFours) {
      const bool in = c >= lo && c < hi;
      u.x = in ? u.x : 0.f, u.y = in ? u.y : 0.f, v.x = in ? v.x : 0.f, v.y = in ? v.y : 0.f;
    }
    acc[0] = add2(acc[0], u);
    acc[1] = add2(acc[1], v);
  }
}

template <int D>
__global__ void __launch_bounds__(kThr, 1)
    attn_mass_kernel(const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmQ, const MassArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long s_part[kThr / 32];
  __shared__ long long s_run[2];
  __shared__ int s_start[3];
  __shared__ int abort_s;
  uint8_t* smem = smem_align1024(smem_raw);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* k_empty = k_full + C::kKSlots;
  uint64_t* q_full = k_empty + C::kKSlots;
  uint64_t* q_empty = q_full + C::kQSlots;
  uint64_t* s_full = q_empty + C::kQSlots;
  uint64_t* s_empty = s_full + C::kSBufs;
  uint64_t* l_full = s_empty + C::kSBufs;
  uint64_t* l_empty = l_full + 2;
  uint64_t* a_full = l_empty + 2;  // K of both row tiles is in tensor memory
  uint64_t* drain = a_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = &abort_s;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

  // The mass update starts while this kernel drains; the plan comes first.
  asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0) {
    for (int i = 0; i < C::kKSlots; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::kQSlots; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < C::kSBufs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kSumWarps / 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&l_full[i], 1);
      mbar_init(&l_empty[i], kSumWarps);
    }
    mbar_init(a_full, kSumWarps);
    mbar_init(drain, 1);
    fence_mbar_init();
    abort_s = 0;
    s_start[0] = -1;
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // Rows of a Q slot that no box fills (a group that does not divide the tile) stay zero.
  if (a.GP * a.TQ < C::kQN) {
    for (int i = tid; i < C::kQSlots * C::kQBytes / 16; i += kThr)
      reinterpret_cast<uint4*>(smem + C::kOffQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- this CTA's run: positions [u0, u1) of the T in all
  {
    const int per = (a.B + kThr - 1) / kThr;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += ws_cum(a, b)[a.max_kt] * a.Hkv;
    long long x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_part[warp] = x;
    __syncthreads();
    long long before = x - sum, T = 0;
    for (int w = 0; w < kThr / 32; ++w) {
      if (w < warp) before += s_part[w];
      T += s_part[w];
    }
    // with fewer positions than CTAs the last CTAs have none, the others one each
    const long long n = min(T, static_cast<long long>(gridDim.x)), c = blockIdx.x;
    const long long u0 = c < n ? T * c / n : 0, u1 = c < n ? T * (c + 1) / n : 0;
    for (int b = b0; b < b1; ++b) {
      const long long per_head = ws_cum(a, b)[a.max_kt], here = per_head * a.Hkv;
      if (blockIdx.x == 0) ws_base(a)[b] = before;
      if (u0 < u1 && u0 >= before && u0 < before + here) {
        const long long in = u0 - before;
        const long long v = in % per_head;  // position within the head
        const long long* cum = ws_cum(a, b);
        Seq s;
        load_seq(a, b, s);
        int lo = 0, hi = key_tiles(s) - 1;  // the last key tile with cum <= v
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (cum[mid] <= v)
            lo = mid;
          else
            hi = mid - 1;
        }
        s_start[0] = b;
        s_start[1] = static_cast<int>(in / per_head);
        s_start[2] = lo;
        s_run[0] = v - cum[lo] - kItemCost;
      }
      before += here;
    }
    if (tid == 0) {
      s_run[1] = u1 - u0;
      if (blockIdx.x == 0) ws_base(a)[a.B] = T;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (s_start[0] >= 0) {
    Walk w;
    w.b = s_start[0];
    w.h = s_start[1];
    w.left = s_run[1];
    walk_seq(a, w);
    walk_row(a, w, s_start[2]);
    w.u = static_cast<int>(s_run[0]);  // may stand before the first unit

    if (warp == kWarpProducer) {
      // ============================================================ TMA producer
      int kn = 0, qn = 0;  // K and Q slots filled
      int pb = -1, ph = -1, pu = -1;
      bool ok = true, more = true;
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmQ);
      // Physical page of this lane, read a key tile ahead of its loads.
      auto lookup = [&]() -> int {
        if (lane >= kPagesPerTile) return 0;
        const int page = w.kt * kPagesPerTile + lane;
        if (page * kPage >= w.s.L) return 0;
        return a.page_table[static_cast<size_t>(w.b) * a.max_pages + page];
      };
      int page = lookup();
      while (more) {
        const int units = walk_units(w);
        if (units == 0) break;
        const int pages = min(kPagesPerTile, (w.s.L - w.kt * kKeys + kPage - 1) / kPage);
        const int b = w.b, h = w.h, u0 = w.tile + w.u, q_base = w.s.q_base;
        w.left -= units;
        more = walk_next(a, w);
        if (page < 0 || page >= a.num_pages) {
          atomicOr(a.status, kStatusBadInput);
          page = 0;
        }
        __syncwarp();
        const int ks = kn % C::kKSlots;
        if (kn >= C::kKSlots &&
            !mbar_wait_warp(&k_empty[ks], (kn / C::kKSlots - 1) & 1, abort_flag, kWaitLimitNs)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx_w(&k_full[ks], pages * C::kPageBytes);
        if (lane < pages)
          tma_load_5d(smem + ks * C::kKBytes + lane * C::kPageBytes, &tmK, &k_full[ks], 0, 0, 0, h,
                      2 * page);
        __syncwarp();
        ++kn;
        if (more) page = lookup();
        for (int u = u0; u < u0 + units; ++u) {
          if (b == pb && h == ph && u == pu) continue;
          pb = b, ph = h, pu = u;
          const int qs = qn % C::kQSlots;
          if (qn >= C::kQSlots &&
              !mbar_wait_warp(&q_empty[qs], (qn / C::kQSlots - 1) & 1, abort_flag,
                              kWaitLimitNs)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx_w(&q_full[qs], C::kAtoms * a.GP * a.TQ * 128);
#pragma unroll
          for (int at = 0; at < C::kAtoms; ++at)
            tma_load_4d_w(smem + C::kOffQ + qs * C::kQBytes + at * C::kQAtom, &tmQ, &q_full[qs],
                          at * 64, h * a.G + tile_head(a, u), q_base + tile_token(a, u), 0);
          ++qn;
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) {
        atomicOr(a.status, kStatusTimeout);
        *abort_flag = 1;
      }
      // every copy issued lands before the CTA leaves
      for (int i = 0; i < C::kKSlots; ++i) {
        const int n = kn > i ? (kn - 1 - i) / C::kKSlots : -1;  // last use of the slot
        if (n >= 0) mbar_wait(&k_full[i], n & 1, nullptr, kWaitLimitNs);
      }
      for (int i = 0; i < C::kQSlots; ++i) {
        const int n = qn > i ? (qn - 1 - i) / C::kQSlots : -1;
        if (n >= 0) mbar_wait(&q_full[i], n & 1, nullptr, kWaitLimitNs);
      }
    } else if (warp == kWarpIssuer) {
      // ============================================================ MMA issuer
      // Slots and phases are counted along rather than worked out of running numbers, and the
      // descriptors are sums of constants: one warp issues everything, and each instruction
      // between two products costs it some eight cycles next to the summing warps.
      constexpr uint32_t idesc = idesc_bf16_f32(kRows, C::kQN, false);
      int ks = 0, kphase = 0, aphase = 0;
      int qs = 0, qphase = 0, held = -1;  // next Q slot; the slot of the tile before
      int buf = 0, sphase = 1;            // next S buffer (its first wait passes at once)
      int pb = -1, ph = -1, pu = -1;      // the query tile before
      const uint64_t dq0 = sdesc_sw128(smem_addr(smem + C::kOffQ), 16, 1024);
      const uint64_t dk0 = sdesc_sw128(smem_addr(smem), 16, C::kGroup);
      const uint32_t tA = tmem + C::kColA;
      bool ok = true;
      do {
        int units = walk_units(w);
        if (units == 0) break;
        const bool ts = units >= kMinTs;
        int u = w.tile + w.u;
        bool fresh = !(w.b == pb && w.h == ph && u == pu);  // another query tile
        pb = w.b, ph = w.h, pu = u + units - 1;
        w.left -= units;
        if ((ts ? !mbar_wait_warp(a_full, aphase, abort_flag, kWaitLimitNs)
                : !mbar_wait_warp(&k_full[ks], kphase, abort_flag, kWaitLimitNs)) ||
            (fresh && !mbar_wait_warp(&q_full[qs], qphase, abort_flag, kWaitLimitNs)) ||
            !mbar_wait_warp(&s_empty[buf], sphase, abort_flag, kWaitLimitNs)) {
          ok = false;
          break;
        }
        uint64_t* const k_done = &k_empty[ks];
        const uint64_t dk = dk0 + ks * (C::kKBytes >> 4);
        if (++ks == C::kKSlots) ks = 0, kphase ^= 1;
        if (ts) {
          aphase ^= 1;
          if (lane == 0) mbar_arrive(k_done);
          __syncwarp();
        }
        while (units > 0) {
          if (fresh) {
            // the tile before is done with once its products are
            if (held >= 0) mma_commit_w(&q_empty[held]);
            held = qs;
            if (++qs == C::kQSlots) qs = 0, qphase ^= 1;
          }
          const uint64_t dq = dq0 + held * (C::kQBytes >> 4);
          --units;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            tc_fence_after_sync();
            const uint32_t tS = tmem + buf * C::kQN;
            uint64_t* const s_done = &s_full[buf];
            if (++buf == C::kSBufs) buf = 0, sphase ^= 1;
            // Keys past the last one: whatever the slot holds, in rows that nothing reads.
            auto issue = [&](int at) {
              const uint64_t q = dq + at * (C::kQAtom >> 4);
              if (ts)
                mma_ts_atom_w(tS, tA + t * (D / 2) + 32 * at, q, idesc, at > 0);
              else
                mma_ss_atom_w(tS, dk + ((t * (C::kKBytes / 2) + at * 1024) >> 4), q, idesc, at > 0);
            };
#pragma unroll
            for (int at = 0; at < (C::kAtoms + 1) / 2; ++at) issue(at);
            if (t == 0 || units > 0) {
              if ((t == 1 && !mbar_wait_warp(&q_full[qs], qphase, abort_flag, kWaitLimitNs)) ||
                  !mbar_wait_warp(&s_empty[buf], sphase, abort_flag, kWaitLimitNs)) {
                ok = false;
                break;
              }
            }
#pragma unroll
            for (int at = (C::kAtoms + 1) / 2; at < C::kAtoms; ++at) issue(at);
            mma_commit_w(s_done);
          }
          if (!ok) break;
          fresh = true;  // within a key tile every unit has another query tile
        }
        if (!ok) break;
        if (!ts) mma_commit_w(k_done);
      } while (walk_next(a, w));
      if (!ok && lane == 0) {
        atomicOr(a.status, kStatusTimeout);
        *abort_flag = 1;
      }
      // every product issued has completed before tensor memory is released
      mma_commit_w(drain);
      mbar_wait(drain, 0, nullptr, kWaitLimitNs);
    } else if (warp == kWarpLse) {
      // ============================================================ LSEs
      // -LSE log2 e of every column of a query tile, -inf where there is no query or one that
      // attended to nothing (LSE = -inf); the loads of a tile are in flight while the one
      // before waits for its buffer.
      constexpr int kPer = C::kQN / 32;
      int tok[kPer], head[kPer];  // of this lane's columns
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int c = j * 32 + lane;
        tok[j] = c < a.GP * a.TQ ? c / a.GP : INT_MAX / 2;
        head[j] = c % a.GP;
      }
      int n = 0, units = walk_units(w), i = 0;
      int pb = -1, ph = -1, pu = -1;
      float v[kPer], next[kPer];
      auto fetch = [&] {
        const int u = w.tile + w.u + i;
        if (w.b == pb && w.h == ph && u == pu) return;
        pb = w.b, ph = w.h, pu = u;
        const int t0 = tile_token(a, u);
        const float* lse = a.lse + static_cast<size_t>(w.h * a.G + tile_head(a, u)) * a.total_q +
                           w.s.q_base + t0;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          next[j] = t0 + tok[j] < w.s.Lq
                        ? lse[static_cast<size_t>(head[j]) * a.total_q + tok[j]]
                        : INFINITY;
      };
      bool ok = true, more = units > 0;
      if (more) fetch();
      while (more) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          v[j] = next[j] == -INFINITY ? -INFINITY : next[j] * -kLog2e;
        if (++i == units) {
          w.left -= units;
          more = walk_next(a, w);
          if (more) {
            units = walk_units(w);
            more = units > 0;
            i = 0;
          }
        }
        if (more) fetch();
        if (n >= 2 && !mbar_wait_warp(&l_empty[n & 1], (n / 2 - 1) & 1, abort_flag, kWaitLimitNs)) {
          ok = false;
          break;
        }
        float* nl = reinterpret_cast<float*>(smem + C::kOffLse) + (n & 1) * C::kQN;
#pragma unroll
        for (int j = 0; j < kPer; ++j) nl[j * 32 + lane] = v[j];
        __syncwarp();
        if (lane == 0) mbar_arrive(&l_full[n & 1]);
        ++n;
      }
      if (!ok && lane == 0) {
        atomicOr(a.status, kStatusTimeout);
        *abort_flag = 1;
      }
    } else {
      // ============================================================ sums: warps 0-15
      constexpr int kCols = C::kQN / kHalves;  // columns of this warp
      const int t = (warp / 4) % 2, half = warp / 8, c0 = half * kCols;
      const int r = tid % kRows;  // the row of this thread
      const uint32_t taddr = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16);
      const float* nl = reinterpret_cast<const float*>(smem + C::kOffLse) + c0;
      int kn = 0, lbuf = 0, lphase = 0;  // LSE buffer of the next unit
      int buf = t, phase = 0;            // S buffer of this row tile's next product
      const bool fours = a.GP % 4 == 0;
      bool ok = true;
      do {
        const int ka = w.kt * kKeys + t * kRows, kb = ka + kRows - 1;  // of this row tile
        const int key = ka + r;
        const int units = walk_units(w);
        if (units == 0) break;
        if (units >= kMinTs) {
          // ---- half of this row of K to tensor memory.  The key tile's products before have
          // been read by this warp, so nothing reads the old K any more.
          const int ks = kn % C::kKSlots;
          if (!mbar_wait_warp(&k_full[ks], (kn / C::kKSlots) & 1, abort_flag, kWaitLimitNs)) {
            ok = false;
            break;
          }
          constexpr int kChunks = D / 16;  // 16-byte chunks of half a row
          const uint8_t* src = smem + ks * C::kKBytes + t * (C::kKBytes / 2) +
                               (r / 8) * C::kGroup + (r % 8) * 128;
          const uint32_t dst = taddr + C::kColA + t * (D / 2) + half * (D / 4);
#pragma unroll
          for (int c = 0; c < kChunks; c += 4) {
            uint32_t y[16];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int ch = half * kChunks + c + e;
              const uint4 v = *reinterpret_cast<const uint4*>(
                  src + (ch / 8) * 1024 + (((ch % 8) ^ (r & 7)) << 4));
              y[4 * e] = v.x, y[4 * e + 1] = v.y, y[4 * e + 2] = v.z, y[4 * e + 3] = v.w;
            }
            tmem_st_x16(dst + 4 * c, y);
          }
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(a_full);
        }
        ++kn;
        // Tokens that this row sees, and first tokens of the tiles that all rows see whole.
        int see0 = 0, see1 = w.s.Lq, all0 = 0, all1 = w.s.Lq - a.TQ;
        if (a.causal) {
          see0 = key - w.s.off;
          all0 = kb - w.s.off;
        }
        if (a.window > 0 && key >= a.n_sink)
          see1 = min(see1, key + a.window - w.s.off);
        if (a.window > 0 && kb >= a.n_sink)
          all1 = min(all1, ka + a.window - w.s.off - a.TQ);
        const int u0 = w.tile + w.u;
        int i0 = tile_token(a, u0);
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        for (int i = 0; i < units; ++i) {
          if (!mbar_wait_warp(&s_full[buf], phase, abort_flag, kWaitLimitNs)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          uint32_t x[kCols];
#pragma unroll
          for (int c = 0; c < kCols; c += 32) tmem_ld_x32(taddr + buf * C::kQN + c0 + c, x + c);
          // while they come: the LSEs, and which columns count
          if (!mbar_wait_warp(&l_full[lbuf], lphase, abort_flag, kWaitLimitNs)) {
            ok = false;
            break;
          }
          const float* l = nl + lbuf * C::kQN;
          const bool interior = i0 >= all0 && i0 <= all1;
          const int lo = min(max(see0 - i0, 0), a.TQ) * a.GP - c0;
          const int hi = min(max(see1 - i0, 0), a.TQ) * a.GP - c0;
#pragma unroll
          for (int c = 0; c < kCols; c += 32) tmem_ld_wait_x32(x + c);
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[buf]);
          if (interior)
            add_columns<kCols, kAll>(x, l, a.scale2, 0, 0, acc);
          else if (fours)
            add_columns<kCols, kFours>(x, l, a.scale2, lo, hi, acc);
          else
            add_columns<kCols, kAny>(x, l, a.scale2, lo, hi, acc);
          __syncwarp();
          if (lane == 0) mbar_arrive(&l_empty[lbuf]);
          buf += 2;
          if (buf >= C::kSBufs) buf -= C::kSBufs, phase ^= 1;
          if (++lbuf == 2) lbuf = 0, lphase ^= 1;
          i0 = a.HC == 1 ? i0 + a.TQ : tile_token(a, u0 + i + 1);
        }
        if (!ok) break;
        const size_t slot =
            (static_cast<size_t>(w.b) * a.Hkv + w.h) * a.max_kt + w.kt + blockIdx.x;
        const float2 sum = add2(acc[0], acc[1]);
        a.ws_part[(slot * kHalves + half) * kKeys + t * kRows + r] = sum.x + sum.y;
        w.left -= units;
      } while (walk_next(a, w));
      if (!ok && lane == 0) {
        atomicOr(a.status, kStatusTimeout);
        *abort_flag = 1;
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- the mass
// A block takes four key tiles of one sequence and key head, a thread a token of each.  The
// CTAs whose partial sums a tile has (two divisions of 64 bits) are worked out once, and the
// loads of all four tiles are in flight together (32 queries on 8 rows of 8,000 to 32,000
// tokens: 76 us a call, one tile behind the other 82).
constexpr int kAddThreads = kKeys;
constexpr int kAddTiles = 4;
constexpr int kAddTokens = kAddTiles * kAddThreads;
__global__ void __launch_bounds__(kAddThreads) attn_mass_add_kernel(const MassArgs a, int ctas) {
  __shared__ __align__(16) int2 s_ctas[kAddTiles];  // first and last CTA; none if the last is before the first
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  Seq s;
  if (!load_seq(a, b, s)) return;
  int fresh = a.new_tokens ? a.new_tokens[b] : s.Lq;
  fresh = max(0, min(fresh, s.L));
  const int last = a.last_positions ? a.last_positions[b] : s.L - 1;
  const size_t row = (static_cast<size_t>(b) * a.Hkv + h) * a.slots;
#pragma unroll 1
  for (int t0 = blockIdx.x * kAddTokens; t0 < s.L; t0 += gridDim.x * kAddTokens) {
    __syncthreads();  // (s_ctas of the tiles before has been read)
    if (tid < kAddTiles) {
      const int kt = t0 / kKeys + tid, tiles = key_tiles(s);
      int2 c = make_int2(0, -1);
      if (kt < tiles) {
        const long long* cum = ws_cum(a, b);
        const long long per_head = cum[a.max_kt], T = ws_base(a)[a.B], before = ws_base(a)[b];
        const long long at = cum[kt], n = (kt + 1 < tiles ? cum[kt + 1] : per_head) - at - kItemCost;
        if (n > 0) {
          // of C CTAs with work, position u belongs to CTA ((u + 1) C - 1) / T
          const long long u = before + per_head * h + at + kItemCost;
          const long long C = min(T, static_cast<long long>(ctas));
          c.x = static_cast<int>(((u + 1) * C - 1) / T);
          c.y = static_cast<int>(((u + n) * C - 1) / T);
        }
      }
      s_ctas[tid] = c;
    }
    float old[kAddTiles];
#pragma unroll
    for (int j = 0; j < kAddTiles; ++j) {
      const int t = t0 + j * kAddThreads + tid;
      old[j] = t < s.L - fresh ? a.mass[row + t] : 0.f;
    }
    __syncthreads();
    const float* part = a.ws_part +
                        ((static_cast<size_t>(b) * a.Hkv + h) * a.max_kt + t0 / kKeys) * kHalves * kKeys +
                        tid;
    float w[kAddTiles];
    const int4 c01 = *reinterpret_cast<const int4*>(s_ctas), c23 = *reinterpret_cast<const int4*>(s_ctas + 2);
    const int c0[kAddTiles] = {c01.x, c01.z, c23.x, c23.z}, c1[kAddTiles] = {c01.y, c01.w, c23.y, c23.w};
#pragma unroll
    for (int j = 0; j < kAddTiles; ++j) {
      const float* p = part + static_cast<size_t>(j + c0[j]) * kHalves * kKeys;
      w[j] = 0.f;
      if (c0[j] <= c1[j])
#pragma unroll
        for (int i = 0; i < kHalves; ++i) w[j] += p[i * kKeys];
    }
#pragma unroll
    for (int j = 0; j < kAddTiles; ++j) {
#pragma unroll 1
      for (int c = c0[j] + 1; c <= c1[j]; c += 4) {  // four CTAs' in flight
        float v[4 * kHalves];
#pragma unroll
        for (int i = 0; i < 4 * kHalves; ++i)
          v[i] = c + i / kHalves <= c1[j]
                     ? part[(static_cast<size_t>(j + c) * kHalves + i) * kKeys]
                     : 0.f;
#pragma unroll
        for (int i = 0; i < 4 * kHalves; ++i) w[j] += v[i];
      }
      const int t = t0 + j * kAddThreads + tid;
      if (t >= s.L) break;
      const bool is_new = t >= s.L - fresh;
      a.mass_out[row + t] = is_new ? w[j] : old[j] + w[j];
      if (is_new && a.positions != nullptr) a.positions[row + t] = last - (s.L - 1 - t);
    }
  }
}

template <int D>
cudaError_t launch_mass(const MassArgs& a, int num_sms, cudaStream_t stream) {
  static SharedMemoryLimit limit;
  cudaError_t e = limit.raise(attn_mass_kernel<D>, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  attn_mass_plan_kernel<<<a.B, kPlanThreads, 0, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_dependent(attn_mass_kernel<D>, dim3(num_sms), kThr, Cfg<D>::kSmem, stream, a.tmK,
                       a.tmQ, a);
  if (e != cudaSuccess) return e;
  const long long reach = std::min<long long>(static_cast<long long>(a.max_pages) * kPage, a.slots);
  // (as many blocks as fill the GPU a few times: the table may be far wider than its rows are
  // long)
  const long long units = static_cast<long long>(a.Hkv) * a.B;
  const long long blocks = std::min((reach + kAddTokens - 1) / kAddTokens,
                                    (32LL * num_sms + units - 1) / units);
  const dim3 grid(static_cast<unsigned>(blocks), a.Hkv, a.B);
  return launch_dependent(attn_mass_add_kernel, grid, kAddThreads, 0, stream, a, num_sms);
}

}  // namespace

int mass_query_tile(int d) { return d == 256 ? Cfg<256>::kQN : Cfg<128>::kQN; }
int mass_key_tile() { return kKeys; }
int mass_partial_floats() { return kHalves * kKeys; }

cudaError_t launch_attn_mass(const MassArgs& a, int num_sms, cudaStream_t stream) {
  if (a.d == 64) return launch_mass<64>(a, num_sms, stream);
  if (a.d == 128) return launch_mass<128>(a, num_sms, stream);
  if (a.d == 256) return launch_mass<256>(a, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace attn
