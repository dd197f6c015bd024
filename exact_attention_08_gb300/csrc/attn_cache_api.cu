// C ABI of the operators around the attention kernels: rotary positions, the
// append of new tokens to a paged cache, and the cache's page bookkeeping.
// Argument checks and launches; see include/attn.h for the contract of every
// entry point.
#include "attn.h"
#include "attn_internal.h"

#include <cmath>
#include <cstdint>
#include <cstring>

using namespace attn;

namespace {

// Rows of one call: their numbers stay clear of 2^31 in every index sum.
constexpr int kMaxRows = INT32_MAX - 1024;

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// One tensor's strides: what the caller gave, or the contiguous ones.  A
// dimension of size one has none that matters, and a tensor without heads
// (one left out) none at all.  Outputs must step forward.
int take_strides(long long* out, const long long* given, const long long* contiguous,
                 const long long* sizes, int n, bool output, const char* name) {
  for (int i = 0; i < n; ++i) {
    out[i] = given ? given[i] : contiguous[i];
    if (sizes[i] <= 1 || sizes[n - 1] == 0) {
      out[i] = 0;
      continue;
    }
    if (out[i] % 8 != 0 || out[i] < 0 || (output && out[i] == 0))
      return set_error(ATTN_ERR_INVALID_ARG,
                       "%s: strides must be %s multiples of 8 elements (16 bytes)", name,
                       output ? "positive" : "non-negative");
  }
  return ATTN_OK;
}

int check_rotation(int d, int rotary_dim, int interleaved, float amplitude,
                   const double* inv_freq) {
  if (d != 64 && d != 128 && d != 256)
    return set_error(ATTN_ERR_UNSUPPORTED, "head dim %d (64, 128 or 256)", d);
  if (rotary_dim < 0 || rotary_dim > d || rotary_dim % 2 != 0)
    return set_error(ATTN_ERR_INVALID_ARG, "rotary_dim %d must be even and at most d=%d",
                     rotary_dim, d);
  if (interleaved != 0 && interleaved != 1)
    return set_error(ATTN_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (!std::isfinite(amplitude))
    return set_error(ATTN_ERR_INVALID_ARG, "amplitude must be finite");
  if (rotary_dim > 0 && (inv_freq == nullptr || !aligned(inv_freq, 8)))
    return set_error(ATTN_ERR_INVALID_ARG, "inv_freq must be set and 8-byte aligned");
  return ATTN_OK;
}

int rope_impl(const void* q, const void* k, void* q_out, void* k_out, const int* positions,
              const double* inv_freq, int B, int S, int Hq, int Hkv, int d, int rotary_dim,
              int interleaved, float amplitude, float sign, const long long* q_strides,
              const long long* k_strides, const long long* q_out_strides,
              const long long* k_out_strides, void* stream) {
  clear_error();
  if (B < 0 || S < 0 || Hq < 0 || Hkv < 0)
    return set_error(ATTN_ERR_INVALID_ARG, "negative size (B=%d S=%d Hq=%d Hkv=%d)", B, S, Hq,
                     Hkv);
  int rc = check_rotation(d, rotary_dim, interleaved, amplitude, inv_freq);
  if (rc != ATTN_OK) return rc;
  const long long rows = static_cast<long long>(B) * S;
  if (rows > kMaxRows) return set_error(ATTN_ERR_INVALID_ARG, "%lld rows are too many", rows);
  if (Hq > (1 << 20) || Hkv > (1 << 20))
    return set_error(ATTN_ERR_INVALID_ARG, "more than 2^20 heads");
  if (rows == 0 || Hq + Hkv == 0) return ATTN_OK;
  if ((Hq > 0 && (!q || !q_out)) || (Hkv > 0 && (!k || !k_out)))
    return set_error(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) ||
      !aligned(positions, 4))
    return set_error(ATTN_ERR_INVALID_ARG, "tensors must be 16-byte aligned (positions 4-byte)");
  RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  const long long sq[3] = {B, S, Hq}, sk[3] = {B, S, Hkv};
  const long long cq[3] = {static_cast<long long>(S) * Hq * d, static_cast<long long>(Hq) * d, d};
  const long long ck[3] = {static_cast<long long>(S) * Hkv * d, static_cast<long long>(Hkv) * d,
                           d};
  if ((rc = take_strides(a.q_s, q_strides, cq, sq, 3, false, "q")) != ATTN_OK ||
      (rc = take_strides(a.k_s, k_strides, ck, sk, 3, false, "k")) != ATTN_OK ||
      (rc = take_strides(a.qo_s, q_out_strides, cq, sq, 3, true, "q_out")) != ATTN_OK ||
      (rc = take_strides(a.ko_s, k_out_strides, ck, sk, 3, true, "k_out")) != ATTN_OK)
    return rc;
  const bool q_same = Hq > 0 && q == q_out, k_same = Hkv > 0 && k == k_out;
  if ((q_same && std::memcmp(a.q_s, a.qo_s, sizeof(a.q_s)) != 0) ||
      (k_same && std::memcmp(a.k_s, a.ko_s, sizeof(a.k_s)) != 0))
    return set_error(ATTN_ERR_INVALID_ARG, "in place, the strides must be the input's");
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.qo = static_cast<__nv_bfloat16*>(q_out);
  a.ko = static_cast<__nv_bfloat16*>(k_out);
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.B = B;
  a.S = S;
  a.rows = static_cast<int>(rows);
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.rot = rotary_dim;
  a.interleaved = interleaved;
  a.amplitude = amplitude;
  a.sign = sign;
  a.in_place = (Hq == 0 || q_same) && (Hkv == 0 || k_same);
  int num_sms = 0;
  int* status = nullptr;
  if ((rc = device_info(&num_sms, &status)) != ATTN_OK) return rc;
  const cudaError_t e = launch_attn_rope(a, num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_error(e, "attn_rope launch");
}

// Checks shared by the page bookkeeping calls; fills the common arguments.
int pages_common(PagesArgs* a, int* page_table, int* seqlens, int* refs, int B, int max_pages,
                 int num_pages, void* k_pages, void* v_pages, int layers, int page_size, int Hkv,
                 int d, int rows, void* workspace, size_t workspace_bytes) {
  if (B < 0 || max_pages <= 0 || num_pages <= 0 || layers < 1 || Hkv < 1)
    return set_error(ATTN_ERR_INVALID_ARG, "bad sizes (B=%d max_pages=%d num_pages=%d layers=%d)",
                     B, max_pages, num_pages, layers);
  if (page_size != 16) return set_error(ATTN_ERR_UNSUPPORTED, "page size %d (16)", page_size);
  if (d != 64 && d != 128 && d != 256)
    return set_error(ATTN_ERR_UNSUPPORTED, "head dim %d (64, 128 or 256)", d);
  if (B > kPagesMaxTable)
    return set_error(ATTN_ERR_INVALID_ARG, "%d table rows, at most %d", B, kPagesMaxTable);
  if (rows > kPagesMaxRows)
    return set_error(ATTN_ERR_INVALID_ARG, "%d rows, at most %d in one call", rows,
                     kPagesMaxRows);
  if (num_pages > kPagesMaxPages)
    return set_error(ATTN_ERR_INVALID_ARG, "%d pages, at most %d", num_pages, kPagesMaxPages);
  if (static_cast<long long>(max_pages) * page_size > (1 << 30))
    return set_error(ATTN_ERR_INVALID_ARG, "max_pages_per_seq too large");
  if (Hkv > (1 << 20)) return set_error(ATTN_ERR_INVALID_ARG, "more than 2^20 heads");
  if (layers > (1 << 16)) return set_error(ATTN_ERR_INVALID_ARG, "more than 2^16 layers");
  if (!refs || !workspace || (B > 0 && (!page_table || !seqlens)))
    return set_error(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned(page_table, 4) || !aligned(seqlens, 4) || !aligned(refs, 4) ||
      !aligned16(workspace) || !aligned16(k_pages) || !aligned16(v_pages))
    return set_error(ATTN_ERR_INVALID_ARG, "misaligned pointer");
  const size_t need = pages_workspace_bytes(rows, num_pages);
  if (workspace_bytes < need)
    return set_error(ATTN_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes,
                     need);
  std::memset(a, 0, sizeof(*a));
  a->page_table = page_table;
  a->seqlens = seqlens;
  a->refs = refs;
  a->B = B;
  a->max_pages = max_pages;
  a->num_pages = num_pages;
  a->k_pages = static_cast<uint4*>(k_pages);
  a->v_pages = static_cast<uint4*>(v_pages);
  a->layers = layers;
  a->page_vecs = 16 * Hkv * (d / 8);
  a->ws = static_cast<int*>(workspace);
  return ATTN_OK;
}

}  // namespace

extern "C" {

ATTN_API int attn_rope_inv_freq(int rotary_dim, double base, int scaling, double factor,
                                double original_length, double ramp_low, double ramp_high,
                                double* inv_freq) {
  clear_error();
  if (rotary_dim < 2 || rotary_dim % 2 != 0 || inv_freq == nullptr)
    return set_error(ATTN_ERR_INVALID_ARG, "rotary_dim %d must be even and positive", rotary_dim);
  if (!(base > 0.0) || !std::isfinite(base))
    return set_error(ATTN_ERR_INVALID_ARG, "base must be finite and positive");
  if (scaling < ATTN_ROPE_NONE || scaling > ATTN_ROPE_RAMP)
    return set_error(ATTN_ERR_INVALID_ARG, "scaling %d", scaling);
  if (scaling != ATTN_ROPE_NONE && (!(factor > 0.0) || !std::isfinite(factor)))
    return set_error(ATTN_ERR_INVALID_ARG, "factor must be finite and positive");
  if (scaling == ATTN_ROPE_BASE && rotary_dim == 2)
    return set_error(ATTN_ERR_INVALID_ARG, "a stretched base needs more than one pair");
  if (scaling == ATTN_ROPE_RAMP &&
      (!(original_length > 0.0) || !(ramp_high > ramp_low) || !std::isfinite(original_length) ||
       !std::isfinite(ramp_low) || !std::isfinite(ramp_high)))
    return set_error(ATTN_ERR_INVALID_ARG,
                     "a ramp needs original_length > 0 and ramp_high > ramp_low");
  const double kTwoPi = 6.283185307179586476925;
  if (scaling == ATTN_ROPE_BASE)
    base *= std::pow(factor, static_cast<double>(rotary_dim) / (rotary_dim - 2));
  if (!(base > 0.0) || !std::isfinite(base))
    return set_error(ATTN_ERR_INVALID_ARG, "the stretched base is out of fp64's range");
  const auto frequency = [&](int i) {
    const double f = std::pow(base, -2.0 * i / rotary_dim);
    if (scaling == ATTN_ROPE_LINEAR) return f / factor;
    if (scaling != ATTN_ROPE_RAMP) return f;
    // turns the pair makes over the trained length
    const double turns = original_length * f / kTwoPi;
    double keep = (turns - ramp_low) / (ramp_high - ramp_low);
    keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
    return f * (keep + (1.0 - keep) / factor);
  };
  for (int i = 0; i < rotary_dim / 2; ++i) {
    if (!std::isfinite(frequency(i)))
      return set_error(ATTN_ERR_INVALID_ARG, "frequency %d is out of fp64's range", i);
  }
  for (int i = 0; i < rotary_dim / 2; ++i) inv_freq[i] = frequency(i);
  return ATTN_OK;
}

ATTN_API int attn_rope(const void* q, const void* k, void* q_out, void* k_out,
                       const int* positions, const double* inv_freq, int B, int S, int Hq,
                       int Hkv, int d, int rotary_dim, int interleaved, float amplitude,
                       const long long* q_strides, const long long* k_strides,
                       const long long* q_out_strides, const long long* k_out_strides,
                       void* stream) {
  return rope_impl(q, k, q_out, k_out, positions, inv_freq, B, S, Hq, Hkv, d, rotary_dim,
                   interleaved, amplitude, 1.f, q_strides, k_strides, q_out_strides,
                   k_out_strides, stream);
}

ATTN_API int attn_rope_bwd(const void* dq, const void* dk, void* dq_out, void* dk_out,
                           const int* positions, const double* inv_freq, int B, int S, int Hq,
                           int Hkv, int d, int rotary_dim, int interleaved, float amplitude,
                           const long long* dq_strides, const long long* dk_strides,
                           const long long* dq_out_strides, const long long* dk_out_strides,
                           void* stream) {
  return rope_impl(dq, dk, dq_out, dk_out, positions, inv_freq, B, S, Hq, Hkv, d, rotary_dim,
                   interleaved, amplitude, -1.f, dq_strides, dk_strides, dq_out_strides,
                   dk_out_strides, stream);
}

ATTN_API int attn_append_paged(const void* q, const void* k, const void* v, void* q_out,
                               void* k_pages, void* v_pages, const int* page_table,
                               const int* cu_seqlens_q, const int* seqlens_k,
                               const double* inv_freq, int B, int Hq, int Hkv, int total_q, int d,
                               int rotary_dim, int interleaved, float amplitude, int page_size,
                               int max_pages_per_seq, int num_pages_total,
                               const long long* q_strides, const long long* k_strides,
                               const long long* v_strides, const long long* q_out_strides,
                               void* stream) {
  clear_error();
  if (B < 0 || Hq < 0 || Hkv <= 0 || total_q < 0 || max_pages_per_seq <= 0 ||
      num_pages_total <= 0)
    return set_error(ATTN_ERR_INVALID_ARG, "bad sizes (B=%d Hq=%d Hkv=%d total_q=%d)", B, Hq, Hkv,
                     total_q);
  int rc = check_rotation(d, rotary_dim, interleaved, amplitude, inv_freq);
  if (rc != ATTN_OK) return rc;
  if (page_size != 16) return set_error(ATTN_ERR_UNSUPPORTED, "page size %d (16)", page_size);
  if (static_cast<long long>(max_pages_per_seq) * page_size > (1 << 30))
    return set_error(ATTN_ERR_INVALID_ARG, "max_pages_per_seq too large");
  if (Hq > (1 << 20) || Hkv > (1 << 20))
    return set_error(ATTN_ERR_INVALID_ARG, "more than 2^20 heads");
  if (total_q > kMaxRows || B > kMaxRows)
    return set_error(ATTN_ERR_INVALID_ARG, "%d rows of %d sequences are too many", total_q, B);
  if (cu_seqlens_q == nullptr && total_q != B)
    return set_error(ATTN_ERR_INVALID_ARG,
                     "without cu_seqlens_q every sequence has one new token (total_q=%d, B=%d)",
                     total_q, B);
  if (B == 0 || total_q == 0) return ATTN_OK;
  if (!k || !v || !k_pages || !v_pages || !page_table || !seqlens_k || (Hq > 0 && (!q || !q_out)))
    return set_error(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
      !aligned16(k_pages) || !aligned16(v_pages) || !aligned(page_table, 4) ||
      !aligned(cu_seqlens_q, 4) || !aligned(seqlens_k, 4))
    return set_error(ATTN_ERR_INVALID_ARG, "misaligned pointer");
  RopeArgs a;
  AppendArgs ap;
  std::memset(&a, 0, sizeof(a));
  std::memset(&ap, 0, sizeof(ap));
  const long long sq[2] = {total_q, Hq}, sk[2] = {total_q, Hkv};
  const long long cq[2] = {static_cast<long long>(Hq) * d, d};
  const long long ck[2] = {static_cast<long long>(Hkv) * d, d};
  if ((rc = take_strides(a.q_s + 1, q_strides, cq, sq, 2, false, "q")) != ATTN_OK ||
      (rc = take_strides(a.k_s + 1, k_strides, ck, sk, 2, false, "k")) != ATTN_OK ||
      (rc = take_strides(ap.v_s, v_strides, ck, sk, 2, false, "v")) != ATTN_OK ||
      (rc = take_strides(a.qo_s + 1, q_out_strides, cq, sq, 2, true, "q_out")) != ATTN_OK)
    return rc;
  if (Hq > 0 && q == q_out && std::memcmp(a.q_s, a.qo_s, sizeof(a.q_s)) != 0)
    return set_error(ATTN_ERR_INVALID_ARG, "in place, the strides must be the input's");
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.qo = static_cast<__nv_bfloat16*>(q_out);
  a.inv_freq = inv_freq;
  a.B = 1;
  a.S = a.rows = total_q;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.rot = rotary_dim;
  a.interleaved = interleaved;
  a.amplitude = amplitude;
  a.sign = 1.f;
  ap.v = static_cast<const __nv_bfloat16*>(v);
  ap.k_pages = static_cast<__nv_bfloat16*>(k_pages);
  ap.v_pages = static_cast<__nv_bfloat16*>(v_pages);
  ap.page_table = page_table;
  ap.cu_q = cu_seqlens_q;
  ap.seqlens_k = seqlens_k;
  ap.B = B;
  ap.Hkv = Hkv;
  ap.d = d;
  ap.total_q = total_q;
  ap.max_pages = max_pages_per_seq;
  ap.num_pages = num_pages_total;
  int num_sms = 0;
  if ((rc = device_info(&num_sms, &ap.status)) != ATTN_OK) return rc;
  const cudaError_t e = launch_attn_append(a, ap, num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_error(e, "attn_append_paged launch");
}

ATTN_API size_t attn_pages_workspace_size(int rows, int num_pages_total) {
  if (rows < 0 || rows > kPagesMaxRows || num_pages_total <= 0 || num_pages_total > kPagesMaxPages)
    return 0;
  return pages_workspace_bytes(rows, num_pages_total);
}

ATTN_API int attn_pages_resize(int* page_table, int* seqlens, const int* new_seqlens, int* refs,
                               void* k_pages, void* v_pages, int B, int layers, int Hkv, int d,
                               int page_size, int max_pages_per_seq, int num_pages_total,
                               void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  PagesArgs a;
  int rc = pages_common(&a, page_table, seqlens, refs, B, max_pages_per_seq, num_pages_total,
                        k_pages, v_pages, layers, page_size, Hkv, d, B, workspace,
                        workspace_bytes);
  if (rc != ATTN_OK) return rc;
  if ((k_pages == nullptr) != (v_pages == nullptr))
    return set_error(ATTN_ERR_INVALID_ARG, "k_pages and v_pages must both be given, or neither");
  if (B == 0) return ATTN_OK;
  if (new_seqlens == nullptr || !aligned(new_seqlens, 4))
    return set_error(ATTN_ERR_INVALID_ARG, "new_seqlens must be set and 4-byte aligned");
  a.new_seqlens = new_seqlens;
  if ((rc = device_info(&a.num_sms, &a.status)) != ATTN_OK) return rc;
  const cudaError_t e = launch_pages_resize(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_error(e, "attn_pages_resize launch");
}

ATTN_API int attn_pages_fork(int* page_table, int* seqlens, int* refs, const int* src,
                             const int* dst, int n, void* k_pages, void* v_pages, int B,
                             int layers, int Hkv, int d, int page_size, int max_pages_per_seq,
                             int num_pages_total, void* workspace, size_t workspace_bytes,
                             void* stream) {
  clear_error();
  if (n < 0) return set_error(ATTN_ERR_INVALID_ARG, "n=%d forks", n);
  PagesArgs a;
  int rc = pages_common(&a, page_table, seqlens, refs, B, max_pages_per_seq, num_pages_total,
                        k_pages, v_pages, layers, page_size, Hkv, d, n, workspace,
                        workspace_bytes);
  if (rc != ATTN_OK) return rc;
  if (!k_pages || !v_pages) return set_error(ATTN_ERR_INVALID_ARG, "null pointer");
  if (n == 0) return ATTN_OK;
  if (B == 0) return set_error(ATTN_ERR_INVALID_ARG, "no rows to fork");
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4))
    return set_error(ATTN_ERR_INVALID_ARG, "src and dst must be set and 4-byte aligned");
  a.src = src;
  a.dst = dst;
  a.n = n;
  if ((rc = device_info(&a.num_sms, &a.status)) != ATTN_OK) return rc;
  const cudaError_t e = launch_pages_fork(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_error(e, "attn_pages_fork launch");
}

ATTN_API int attn_pages_compact(int* page_table, const int* seqlens, int* refs, int* new_index,
                                int* num_live, void* k_pages, void* v_pages, int B, int layers,
                                int Hkv, int d, int page_size, int max_pages_per_seq,
                                int num_pages_total, void* workspace, size_t workspace_bytes,
                                void* stream) {
  clear_error();
  PagesArgs a;
  int rc = pages_common(&a, page_table, const_cast<int*>(seqlens), refs, B, max_pages_per_seq,
                        num_pages_total, k_pages, v_pages, layers, page_size, Hkv, d, 0,
                        workspace, workspace_bytes);
  if (rc != ATTN_OK) return rc;
  if (!k_pages || !v_pages || !new_index || !num_live)
    return set_error(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned(new_index, 4) || !aligned(num_live, 4))
    return set_error(ATTN_ERR_INVALID_ARG, "misaligned pointer");
  a.new_index = new_index;
  a.num_live = num_live;
  if ((rc = device_info(&a.num_sms, &a.status)) != ATTN_OK) return rc;
  const cudaError_t e = launch_pages_compact(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_error(e, "attn_pages_compact launch");
}

}  // extern "C"
