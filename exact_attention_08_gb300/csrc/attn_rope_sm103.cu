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
// with p then drops whole turns exactly.  The error is p 2^-53 of f / 2 pi:
// below 10^-9 of a turn up to p = 2^23, 1e-7 at p = 2^31.  The top 32 bits
// of the fraction, as half turns in [-1, 1), go through sincospif in fp32.
// Products and sums are fp32 and are rounded once, to bf16.
//
// Layout.  A CTA takes a few consecutive rows (tokens) with all their heads:
// the row's cos and sin are formed once, kept in shared memory and used by
// every head (40 heads in a GQA 32/8 call), so no table is read from memory
// and the bytes are those of q and k alone.  A thread's unit is eight pairs,
// two 16-byte loads and two 16-byte stores; the loads of a thread's first
// units are issued before the angles are formed, which hides the position's
// and frequencies' latency.
#include "attn_internal.h"
#include "sm103_ptx.cuh"

#include <cuda_bf16.h>

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;          // units in flight per thread
constexpr int kMaxRowsPerCta = 32;

struct RowInfo {
  long long slot;  // append: element offset of the row's cache slot, or -1
  int pos;
  int live;        // 0: the row belongs to no sequence (nothing is written)
};

// f (radians per position) as a fraction of a turn in units of 2^-64.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  double t = f * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rz(t * 18446744073709551616.0);
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

// Heads are numbered q, then k, then (append) v.
template <bool kAppend>
__device__ __forceinline__ const __nv_bfloat16* source(const RopeArgs& p, const AppendArgs& ap,
                                                       int row, int h) {
  const int b = p.B > 1 ? row / p.S : 0;
  const long long s = row - b * p.S;
  if (h < p.Hq) return p.q + b * p.q_s[0] + s * p.q_s[1] + h * p.q_s[2];
  if (!kAppend || h < p.Hq + p.Hkv)
    return p.k + b * p.k_s[0] + s * p.k_s[1] + (h - p.Hq) * p.k_s[2];
  return ap.v + s * ap.v_s[0] + (h - p.Hq - p.Hkv) * ap.v_s[1];
}

// Where the head goes; null: it is not written.
template <bool kAppend>
__device__ __forceinline__ __nv_bfloat16* destination(const RopeArgs& p, const AppendArgs& ap,
                                                      const RowInfo* info, int row, int h) {
  if (kAppend && h >= p.Hq) {
    if (info->slot < 0) return nullptr;
    return h < p.Hq + p.Hkv ? ap.k_pages + info->slot + (h - p.Hq) * p.d
                            : ap.v_pages + info->slot + (h - p.Hq - p.Hkv) * p.d;
  }
  if (kAppend && !info->live) return nullptr;
  const int b = p.B > 1 ? row / p.S : 0;
  const long long s = row - b * p.S;
  if (h < p.Hq) return p.qo + b * p.qo_s[0] + s * p.qo_s[1] + h * p.qo_s[2];
  return p.ko + b * p.ko_s[0] + s * p.ko_s[1] + (h - p.Hq) * p.ko_s[2];
}

// Positions (append: and cache slots) of the CTA's rows, then cos and sin of
// their pairs: row r's cos at sm[2 r npairs + place(pair)], its sin npairs
// further on.  The whole CTA calls it; the values may be read on return.
template <bool kAppend, typename Place>
__device__ __forceinline__ void form_angles(const RopeArgs& p, const AppendArgs& ap, int row0,
                                            int nrows, float* sm, RowInfo* rows_s, Place place) {
  const int tid = threadIdx.x;
  const int npairs = p.rot >> 1;
  if constexpr (kAppend) {
    for (int r = tid >> 5; r < nrows; r += kThreads / 32) {
      const RowInfo info = append_row(ap, row0 + r);
      if ((tid & 31) == 0) rows_s[r] = info;
    }
    if (blockIdx.x == 0 && ap.cu_q != nullptr) {
      // offsets that decrease or leave [0, total_q]
      for (int i = tid; i <= ap.B; i += kThreads) {
        const int c = __ldg(ap.cu_q + i);
        const int next = i < ap.B ? __ldg(ap.cu_q + i + 1) : c;
        if (c < 0 || c > ap.total_q || next < c) atomicOr(ap.status, kStatusBadInput);
      }
    }
    __syncthreads();
  }
  for (int e = tid; e < nrows * npairs; e += kThreads) {
    const int r = e / npairs, pr = e - r * npairs;
    const int row = row0 + r;
    int pos;
    if constexpr (kAppend)
      pos = rows_s[r].pos;
    else
      pos = p.positions != nullptr ? __ldg(p.positions + row) : row % p.S;
    float c, s;
    angle(pos, __ldg(p.inv_freq + pr), p.amplitude, p.sign, &c, &s);
    float* at = sm + 2 * r * npairs + place(pr);
    at[0] = c;
    at[npairs] = s;
  }
  __syncthreads();
}

// ---------------------------------------------------------------- the kernels

// rot a multiple of 16: units of eight pairs, 16-byte loads and stores.
template <int D, bool kAppend>
__global__ void __launch_bounds__(kThreads)
    attn_rope_kernel(const __grid_constant__ RopeArgs p, const __grid_constant__ AppendArgs ap) {
  constexpr int kUnits = D / 16;              // per head
  constexpr int kStep = kThreads / kUnits;    // (row, head) pairs of one pass of the CTA
  extern __shared__ __align__(16) float sm[];
  __shared__ RowInfo rows_s[kAppend ? kMaxRowsPerCta : 1];
  const int tid = threadIdx.x;
  const int npairs = p.rot >> 1;
  const int row0 = blockIdx.x * p.rows_per_cta;
  const int nrows = min(p.rows_per_cta, p.rows - row0);
  const int H = p.Hq + p.Hkv + (kAppend ? p.Hkv : 0);
  const int items = nrows * H;
  const int j = tid & (kUnits - 1);
  const bool turn = j < (p.rot >> 4);
  const bool skip = !turn && p.in_place;  // passed through, and already there
  // offsets of the unit's two vectors inside a head
  int va = j * 16, vb = j * 16 + 8;
  if (turn && !p.interleaved) {
    va = j * 8;
    vb = npairs + j * 8;
  }
  uint4 xa[kBatch], xb[kBatch];
  auto load = [&](int first) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int item = first + i * kStep;
      if (item < items && !skip) {
        const int r = item / H;
        const __nv_bfloat16* src = source<kAppend>(p, ap, row0 + r, item - r * H);
        xa[i] = ld16(src + va);
        xb[i] = ld16(src + vb);
      }
    }
  };
  int it = tid / kUnits;
  load(it);
  form_angles<kAppend>(p, ap, row0, nrows, sm, rows_s,
                       [=](int pr) { return pair_slot(pr, npairs); });
  while (true) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int item = it + i * kStep;
      if (item < items && !skip) {
        const int r = item / H, h = item - r * H;
        __nv_bfloat16* dst = destination<kAppend>(p, ap, rows_s + (kAppend ? r : 0), row0 + r, h);
        if (turn && (!kAppend || h < p.Hq + p.Hkv)) {
          float c[8], s[8];
          const float* cs = sm + 2 * r * npairs + j * 4;
          *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(cs);
          *reinterpret_cast<float4*>(c + 4) = *reinterpret_cast<const float4*>(cs + (npairs >> 1));
          *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(cs + npairs);
          *reinterpret_cast<float4*>(s + 4) =
              *reinterpret_cast<const float4*>(cs + npairs + (npairs >> 1));
          if (p.interleaved) {
            rotate_words(xa[i], c, s);
            rotate_words(xb[i], c + 4, s + 4);
          } else {
            rotate_half(xa[i], xb[i], c, s);
          }
        }
        if (dst != nullptr) {
          st16(dst + va, xa[i]);
          st16(dst + vb, xb[i]);
        }
      }
    }
    it += kBatch * kStep;
    if (it >= items) break;
    load(it);
  }
}

// Any even rot: one pair per thread, 2-byte loads and stores.  Vectors of
// eight would straddle the middle of the rotated part.
template <bool kAppend>
__global__ void __launch_bounds__(kThreads)
    attn_rope_pairs_kernel(const __grid_constant__ RopeArgs p,
                           const __grid_constant__ AppendArgs ap) {
  extern __shared__ __align__(16) float sm[];
  __shared__ RowInfo rows_s[kAppend ? kMaxRowsPerCta : 1];
  const int npairs = p.rot >> 1;
  const int row0 = blockIdx.x * p.rows_per_cta;
  const int nrows = min(p.rows_per_cta, p.rows - row0);
  const int H = p.Hq + p.Hkv + (kAppend ? p.Hkv : 0);
  form_angles<kAppend>(p, ap, row0, nrows, sm, rows_s, [](int pr) { return pr; });
  const int half = p.d >> 1;  // pairs of a head, the passed-through ones included
  for (long long u = threadIdx.x; u < static_cast<long long>(nrows) * H * half; u += kThreads) {
    const int item = static_cast<int>(u / half), pr = static_cast<int>(u - (long long)item * half);
    const int r = item / H, h = item - r * H;
    const bool turn = pr < npairs && (!kAppend || h < p.Hq + p.Hkv);
    const bool split = pr < npairs && !p.interleaved;
    const int a = split ? pr : 2 * pr, b = split ? pr + npairs : 2 * pr + 1;
    const __nv_bfloat16* src = source<kAppend>(p, ap, row0 + r, h);
    __nv_bfloat16* dst = destination<kAppend>(p, ap, rows_s + (kAppend ? r : 0), row0 + r, h);
    if (dst == nullptr) continue;
    __nv_bfloat16 x = src[a], y = src[b];
    if (turn) {
      const float c = sm[2 * r * npairs + pr], s = sm[2 * r * npairs + npairs + pr];
      const float fx = __bfloat162float(x), fy = __bfloat162float(y);
      x = __float2bfloat16_rn(fx * c - fy * s);
      y = __float2bfloat16_rn(fx * s + fy * c);
    }
    dst[a] = x;
    dst[b] = y;
  }
}

template <bool kAppend>
cudaError_t launch(RopeArgs p, const AppendArgs& ap, int num_sms, cudaStream_t stream) {
  const int H = p.Hq + p.Hkv + (kAppend ? p.Hkv : 0);
  if (p.rows == 0 || H == 0) return cudaSuccess;
  // Rows of a CTA: one batch of units for every thread where there are rows
  // enough for two CTAs on every SM, fewer where there are not (a decode step
  // has one row per CTA).
  const int units = H * (p.d / 16);
  const int full = (kBatch * kThreads + units - 1) / units;
  const int spread = (p.rows + 2 * num_sms - 1) / (2 * num_sms);
  const int rows = full < spread ? full : spread;
  p.rows_per_cta = rows < 1 ? 1 : rows > kMaxRowsPerCta ? kMaxRowsPerCta : rows;
  const dim3 grid((p.rows + p.rows_per_cta - 1) / p.rows_per_cta);
  const size_t smem = static_cast<size_t>(p.rows_per_cta) * p.rot * sizeof(float);
  if (p.rot % 16 != 0)
    attn_rope_pairs_kernel<kAppend><<<grid, kThreads, smem, stream>>>(p, ap);
  else if (p.d == 64)
    attn_rope_kernel<64, kAppend><<<grid, kThreads, smem, stream>>>(p, ap);
  else if (p.d == 128)
    attn_rope_kernel<128, kAppend><<<grid, kThreads, smem, stream>>>(p, ap);
  else if (p.d == 256)
    attn_rope_kernel<256, kAppend><<<grid, kThreads, smem, stream>>>(p, ap);
  else
    return cudaErrorInvalidValue;
  return cudaGetLastError();
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
