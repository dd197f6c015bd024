// Rotary positions, forward and backward, and the append of new tokens to a
// paged KV cache (rotation of q and k fused with the write of k and v to
// their slots).
//
// Mathematics.  Pair (x, y) of a head row at position p turns by the angle
// p f_i of its pair index i:
//     x' = a (x cos(p f) - y sin(p f)),   y' = a (x sin(p f) + y cos(p f)).
// The backward is the transpose, the same turn by -p f with the same
// amplitude a.  Elements past the rotated part are passed through.
//
// Angles.  p f in fp32 loses the angle of a far position (at p = 10^6 an
// fp32 angle is off by 0.06 rad), so f arrives in fp64 and becomes a 64-bit
// fraction of a turn, f / 2 pi mod 1 in units of 2^-64; an integer product
// with p then drops whole turns exactly.  That costs less than p 2^-63 of a
// turn for f <= 1: 3e-10 at p = 2^31.  The top 32 bits of the fraction, as
// half turns in [-1, 1), go through sincospif in fp32.
// Products and sums are fp32 and are rounded once, to bf16.
//
// Layout.  A block takes a row (token), each of its warps up to 12 heads (at
// d = 128).  The row's cos and sin are formed once by the block's threads,
// passed round through shared memory and held in registers for every head, so
// no table is read from memory and the bytes are those of q and k alone.  A
// lane's unit is eight pairs, two 16-byte loads and two 16-byte stores; all
// its loads are issued before the angles are formed, which hides the
// position's and frequencies' latency.
//
// Bound: bytes.  Measured (one GB300, device time of a call in a graph, inputs
// and outputs rotating over buffers past L2): q, k of 2 x 4096 rows, 32 + 8
// heads, d = 128, 167.8 MB moved: 27.7 us, 6.1 TB/s, 91 % of a copy's
// measured rate (a copy of those bytes takes 26.4 us); 8192 rows, 16 + 16
// heads, 134.2 MB: 22.7 us (copy 21.6; 19.8 into the same outputs each time,
// which L2 holds in part).  On the first, into outputs used again, fp64
// angles took 28.4 us, warps that each formed the angles of their own heads
// 31.1 us, a block for three rows with a division per unit 33.3 us; packed
// fp32 instructions 28.8 us (more registers, fewer blocks on an SM).
#include "attn_internal.h"
#include "sm103_ptx.cuh"

#include <cuda_bf16.h>

namespace attn {
namespace {

constexpr int kThreads = 128;  // of the pair kernel
constexpr int kMaxWarps = 8;   // of a block of the unit kernel
constexpr int kBatch = 3;  // units (passes over heads) of a lane, all in flight at once
constexpr int kWarpsPerSm = 16;

struct RowInfo {
  long long slot;  // append: element offset of the row's cache slot, or -1
  int pos;
  int live;        // 0: the row belongs to no sequence (nothing is written)
};

// f (radians per position) as a fraction of a turn in units of 2^-64, whole
// turns dropped.  With |f| = M 2^(E - 1086), M its 53 significant bits moved
// to the top of 64 and E the biased exponent, f / 2 pi in those units is
// M K 2^(E - 1088) for K = 2^66 / 2 pi: one high product and a shift.  In
// integers because this GPU's fp64 rate is low.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
  const int e = static_cast<int>(bits >> 52 & 0x7ff);
  const uint64_t m = (bits << 11) | (1ull << 63);
  const uint64_t hi = __umul64hi(m, 0xA2F9836E4E441529ull);
  const int up = e - 1024;
  uint64_t r = 0;  // below 2^-64 of a turn (and zero), or all whole turns
  if (up <= 0 && up > -64) r = hi >> -up;
  if (up > 0 && up < 64) r = hi << up;
  return bits >> 63 ? 0 - r : r;
}

// cos and sin of the angle of position pos, times the amplitude; the
// backward's turn is the negated position.
__device__ __forceinline__ void angle(int pos, double f, float amp, float sign, float* c,
                                      float* s) {
  const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turn_fraction(f);
  const int top = static_cast<int>(turns >> 32);
  float sn, cs;
  sincospif(static_cast<float>(top) * 4.656612873077392578125e-10f, &sn, &cs);  // 2^-31
  *c = cs * amp;
  *s = sn * (amp * sign);
}

// Shared-memory place of pair p's cos (and sin): the first four of every
// eight pairs of all units, then the second four, so that the 16-byte reads
// of neighbouring units fall on neighbouring banks.
__device__ __forceinline__ int pair_slot(int p, int npairs) {
  return ((p >> 2) & 1) * (npairs >> 1) + (p >> 3) * 4 + (p & 3);
}

__device__ __forceinline__ uint4 ld16(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void st16(__nv_bfloat16* p, uint4 v) {
  asm volatile("st.global.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Half layout: a holds the first elements of eight pairs, b the second.
__device__ __forceinline__ void rotate_half(uint4& a, uint4& b, const float* c, const float* s) {
  uint32_t* pa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* pb = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = lo_f(pa[i]), x1 = hi_f(pa[i]), y0 = lo_f(pb[i]), y1 = hi_f(pb[i]);
    const float c0 = c[2 * i], c1 = c[2 * i + 1], s0 = s[2 * i], s1 = s[2 * i + 1];
    pa[i] = ptx::pack_bf16x2(x0 * c0 - y0 * s0, x1 * c1 - y1 * s1);
    pb[i] = ptx::pack_bf16x2(x0 * s0 + y0 * c0, x1 * s1 + y1 * c1);
  }
}

// Interleaved layout: every 32-bit word is one pair.
__device__ __forceinline__ void rotate_words(uint4& a, const float* c, const float* s) {
  uint32_t* pa = reinterpret_cast<uint32_t*>(&a);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = lo_f(pa[i]), y = hi_f(pa[i]);
    pa[i] = ptx::pack_bf16x2(x * c[i] - y * s[i], x * s[i] + y * c[i]);
  }
}

// ---------------------------------------------------------------- rows of an append

// The sequence of packed row `row`: the last b in [0, B) with cu[b] <= row,
// by a 32-way search of the whole warp (one round up to 32 sequences, two up
// to 1024).  -1: no such sequence.  Stays inside [0, B) whatever cu holds.
__device__ __forceinline__ int find_sequence(const int* cu, int B, int row) {
  const int lane = static_cast<int>(ptx::lane_id());
  int lo = 0, n = B;
  while (true) {
    const int step = (n + 31) >> 5;
    const int at = lo + lane * step;
    const bool below = lane * step < n && __ldg(cu + at) <= row;
    const int cnt = __popc(__ballot_sync(0xffffffffu, below));
    if (cnt == 0) return -1;
    const int end = lo + n;
    lo += (cnt - 1) * step;
    if (step == 1) return lo;
    n = min(step, end - lo);
  }
}

__device__ __forceinline__ RowInfo append_row(const AppendArgs& p, int row) {
  RowInfo r;
  r.slot = -1;
  r.pos = 0;
  r.live = 0;
  int b = row, end = row + 1;
  if (p.cu_q != nullptr) {
    b = find_sequence(p.cu_q, p.B, row);
    if (b < 0) return r;
    end = __ldg(p.cu_q + b + 1);
    // covers a list that is not in order, too: only rows inside their
    // sequence's own bounds are touched
    if (row >= end || end > p.total_q) return r;
  }
  const int keys = __ldg(p.seqlens_k + b);
  if (keys < 0 || keys > p.max_pages * 16) {
    atomicOr(p.status, kStatusBadInput);
    return r;
  }
  r.live = 1;
  r.pos = keys - (end - row);
  if (r.pos >= 0) {
    const int page =
        __ldg(p.page_table + static_cast<long long>(b) * p.max_pages + (r.pos >> 4));
    if (page < 0 || page >= p.num_pages)
      atomicOr(p.status, kStatusBadInput);
    else
      r.slot = (static_cast<long long>(page) * 16 + (r.pos & 15)) *
               (static_cast<long long>(p.Hkv) * p.d);
  }
  return r;
}

// ---------------------------------------------------------------- rows and heads

// Heads are numbered q, then k, then (append) v.  A row's three pieces, each
// at its first head:
struct RowSource {
  const __nv_bfloat16 *q, *k, *v;
};
struct RowTarget {
  __nv_bfloat16 *q, *k, *v;  // null: not written
};

__device__ __forceinline__ void split_row(const RopeArgs& p, int row, int* b, int* s) {
  *b = p.B > 1 ? row / p.S : 0;
  *s = row - *b * p.S;
}

template <bool kAppend>
__device__ __forceinline__ RowSource row_source(const RopeArgs& p, const AppendArgs& ap, int row) {
  int b, s;
  split_row(p, row, &b, &s);
  RowSource r;
  r.q = p.q + b * p.q_s[0] + s * p.q_s[1];
  r.k = p.k + b * p.k_s[0] + s * p.k_s[1];
  r.v = kAppend ? ap.v + s * ap.v_s[0] : nullptr;
  return r;
}

template <bool kAppend>
__device__ __forceinline__ RowTarget row_target(const RopeArgs& p, const AppendArgs& ap,
                                                const RowInfo& info, int row) {
  int b, s;
  split_row(p, row, &b, &s);
  RowTarget r;
  r.q = kAppend && !info.live ? nullptr : p.qo + b * p.qo_s[0] + s * p.qo_s[1];
  if constexpr (kAppend) {
    r.k = info.slot < 0 ? nullptr : ap.k_pages + info.slot;
    r.v = info.slot < 0 ? nullptr : ap.v_pages + info.slot;
  } else {
    r.k = p.ko + b * p.ko_s[0] + s * p.ko_s[1];
    r.v = nullptr;
  }
  return r;
}

template <bool kAppend>
__device__ __forceinline__ const __nv_bfloat16* source(const RopeArgs& p, const AppendArgs& ap,
                                                       const RowSource& r, int h) {
  if (h < p.Hq) return r.q + h * p.q_s[2];
  h -= p.Hq;
  if (!kAppend || h < p.Hkv) return r.k + h * p.k_s[2];
  return r.v + (h - p.Hkv) * ap.v_s[1];
}

template <bool kAppend>
__device__ __forceinline__ __nv_bfloat16* target(const RopeArgs& p, const RowTarget& r, int h) {
  if (h < p.Hq) return r.q == nullptr ? nullptr : r.q + h * p.qo_s[2];
  h -= p.Hq;
  if (!kAppend) return r.k + h * p.ko_s[2];
  if (r.k == nullptr) return nullptr;
  return h < p.Hkv ? r.k + h * p.d : r.v + (h - p.Hkv) * p.d;
}

// Position (append: and cache slot) of a row; the whole warp calls it.
template <bool kAppend>
__device__ __forceinline__ RowInfo row_info(const RopeArgs& p, const AppendArgs& ap, int row) {
  if constexpr (kAppend) {
    return append_row(ap, row);
  } else {
    RowInfo r;
    r.slot = -1;
    r.live = 1;
    r.pos = p.positions != nullptr ? __ldg(p.positions + row) : row % p.S;
    return r;
  }
}

// Offsets that decrease or leave [0, total_q] are reported; the whole grid
// shares the list.
__device__ __forceinline__ void check_offsets(const AppendArgs& ap) {
  if (ap.cu_q == nullptr) return;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i <= ap.B;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int c = __ldg(ap.cu_q + i);
    const int next = i < ap.B ? __ldg(ap.cu_q + i + 1) : c;
    if (c < 0 || c > ap.total_q || next < c) atomicOr(ap.status, kStatusBadInput);
  }
}

// ---------------------------------------------------------------- the kernels

// rot a multiple of 16: units of eight pairs, 16-byte loads and stores.
template <int D, bool kAppend>
__global__ void __launch_bounds__(kMaxWarps * 32)
    attn_rope_kernel(const __grid_constant__ RopeArgs p, const __grid_constant__ AppendArgs ap) {
  constexpr int kUnits = D / 16;       // per head
  constexpr int kStep = 32 / kUnits;   // heads of one pass of a warp
  __shared__ __align__(16) float sm[D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if constexpr (kAppend) check_offsets(ap);
  // a row's blocks, and the warp's heads of the row
  const int row = p.row_blocks > 1 ? blockIdx.x / p.row_blocks : blockIdx.x;
  const int chunk = (blockIdx.x - row * p.row_blocks) * (blockDim.x >> 5) + warp;
  const int H = p.Hq + p.Hkv + (kAppend ? p.Hkv : 0);
  const int h0 = chunk * p.chunk_heads;
  const int h1 = min(h0 + p.chunk_heads, H);
  const int npairs = p.rot >> 1;
  const int j = lane & (kUnits - 1);
  const bool turn = j < (p.rot >> 4);
  const bool skip = !turn && p.in_place;  // passed through, and already there
  // offsets of the unit's two vectors inside a head
  int va = j * 16, vb = j * 16 + 8;
  if (turn && !p.interleaved) {
    va = j * 8;
    vb = npairs + j * 8;
  }
  const RowSource from = row_source<kAppend>(p, ap, row);
  uint4 xa[kBatch], xb[kBatch];
  const int first = h0 + lane / kUnits;
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int h = first + i * kStep;
    if (h < h1 && !skip) {
      const __nv_bfloat16* src = source<kAppend>(p, ap, from, h);
      xa[i] = ld16(src + va);
      xb[i] = ld16(src + vb);
    }
  }

  const RowInfo info = row_info<kAppend>(p, ap, row);
  for (int pr = threadIdx.x; pr < npairs; pr += blockDim.x) {
    float c, s;
    angle(info.pos, __ldg(p.inv_freq + pr), p.amplitude, p.sign, &c, &s);
    sm[pair_slot(pr, npairs)] = c;
    sm[npairs + pair_slot(pr, npairs)] = s;
  }
  __syncthreads();
  float c[8], s[8];
  if (turn) {
    const float* cs = sm + j * 4;
    *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(cs);
    *reinterpret_cast<float4*>(c + 4) = *reinterpret_cast<const float4*>(cs + (npairs >> 1));
    *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(cs + npairs);
    *reinterpret_cast<float4*>(s + 4) =
        *reinterpret_cast<const float4*>(cs + npairs + (npairs >> 1));
  }
  const RowTarget to = row_target<kAppend>(p, ap, info, row);
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int h = first + i * kStep;
    if (h < h1 && !skip) {
      __nv_bfloat16* dst = target<kAppend>(p, to, h);
      if (turn && (!kAppend || h < p.Hq + p.Hkv)) {
        if (p.interleaved) {
          rotate_words(xa[i], c, s);
          rotate_words(xb[i], c + 4, s + 4);
        } else {
          rotate_half(xa[i], xb[i], c, s);
        }
      }
      if (!kAppend || dst != nullptr) {
        st16(dst + va, xa[i]);
        st16(dst + vb, xb[i]);
      }
    }
  }
}

// Any even rot: one pair per thread, 2-byte loads and stores.  In the half
// layout vectors of eight would straddle the middle of the rotated part; the
// interleaved one, whose vectors are whole pairs, shares the kernel.  A warp
// takes one row.  Far from the floor: 2 x 4096 rows of 32 + 8 heads, d = 128,
// rot = 20 take 101 us in either layout (25 at a copy's rate), 64 rows 23 us.
template <bool kAppend>
__global__ void __launch_bounds__(kThreads)
    attn_rope_pairs_kernel(const __grid_constant__ RopeArgs p,
                           const __grid_constant__ AppendArgs ap) {
  __shared__ float sm[kThreads / 32][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if constexpr (kAppend) check_offsets(ap);
  const int row = blockIdx.x * (kThreads / 32) + warp;
  if (row >= p.rows) return;
  const int npairs = p.rot >> 1;
  const RowInfo info = row_info<kAppend>(p, ap, row);
  for (int pr = lane; pr < npairs; pr += 32)
    angle(info.pos, __ldg(p.inv_freq + pr), p.amplitude, p.sign, &sm[warp][pr],
          &sm[warp][npairs + pr]);
  __syncwarp();
  const RowSource from = row_source<kAppend>(p, ap, row);
  const RowTarget to = row_target<kAppend>(p, ap, info, row);
  const int H = p.Hq + p.Hkv + (kAppend ? p.Hkv : 0);
  const int half = p.d >> 1;  // pairs of a head, the passed-through ones included
  for (int h = 0; h < H; ++h) {
    const __nv_bfloat16* src = source<kAppend>(p, ap, from, h);
    __nv_bfloat16* dst = target<kAppend>(p, to, h);
    if (kAppend && dst == nullptr) continue;
    const bool rotates = !kAppend || h < p.Hq + p.Hkv;
    for (int pr = lane; pr < half; pr += 32) {
      const bool split = pr < npairs && !p.interleaved;
      const int a = split ? pr : 2 * pr, b = split ? pr + npairs : 2 * pr + 1;
      __nv_bfloat16 x = src[a], y = src[b];
      if (pr < npairs && rotates) {
        const float c = sm[warp][pr], s = sm[warp][npairs + pr];
        const float fx = __bfloat162float(x), fy = __bfloat162float(y);
        x = __float2bfloat16_rn(fx * c - fy * s);
        y = __float2bfloat16_rn(fx * s + fy * c);
      }
      dst[a] = x;
      dst[b] = y;
    }
  }
}

template <int D, bool kAppend>
cudaError_t launch_units(RopeArgs p, const AppendArgs& ap, int num_sms, cudaStream_t stream) {
  constexpr int kStep = 32 / (D / 16);
  const int H = p.Hq + p.Hkv + (kAppend ? p.Hkv : 0);
  // A row's heads are dealt to as many warps as give each one batch of loads,
  // and to more, down to one pass each, while that leaves fewer than
  // kWarpsPerSm warps for every SM.  The warps of a block share the row's
  // angles.
  const int passes = (H + kStep - 1) / kStep;
  const long long want = static_cast<long long>(num_sms) * kWarpsPerSm;
  long long chunks = (want + p.rows - 1) / p.rows;
  const int least = (passes + kBatch - 1) / kBatch;
  chunks = chunks < least ? least : chunks > passes ? passes : chunks;
  const int per = static_cast<int>((passes + chunks - 1) / chunks);
  p.chunk_heads = per * kStep;
  const int warps = (passes + per - 1) / per;
  p.row_blocks = (warps + kMaxWarps - 1) / kMaxWarps;
  const int block_warps = (warps + p.row_blocks - 1) / p.row_blocks;
  const long long blocks = static_cast<long long>(p.rows) * p.row_blocks;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  attn_rope_kernel<D, kAppend>
      <<<static_cast<unsigned>(blocks), block_warps * 32, 0, stream>>>(p, ap);
  return cudaGetLastError();
}

template <bool kAppend>
cudaError_t launch(const RopeArgs& p, const AppendArgs& ap, int num_sms, cudaStream_t stream) {
  if (p.rows == 0 || p.Hq + p.Hkv == 0) return cudaSuccess;
  if (p.rot % 16 != 0) {
    constexpr int kWarps = kThreads / 32;
    attn_rope_pairs_kernel<kAppend>
        <<<static_cast<unsigned>((static_cast<long long>(p.rows) + kWarps - 1) / kWarps), kThreads,
           0, stream>>>(p, ap);
    return cudaGetLastError();
  }
  if (p.d == 64) return launch_units<64, kAppend>(p, ap, num_sms, stream);
  if (p.d == 128) return launch_units<128, kAppend>(p, ap, num_sms, stream);
  if (p.d == 256) return launch_units<256, kAppend>(p, ap, num_sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_attn_rope(const RopeArgs& p, int num_sms, cudaStream_t stream) {
  return launch<false>(p, AppendArgs(), num_sms, stream);
}

cudaError_t launch_attn_append(const RopeArgs& p, const AppendArgs& ap, int num_sms,
                               cudaStream_t stream) {
  return launch<true>(p, ap, num_sms, stream);
}

}  // namespace attn
