// C ABI of the operators on shared and thinned caches: the decode of rows that
// share a prefix, the attention weight that keys accumulate, and the eviction
// by it.  Argument checks and launches; see include/attn.h for the contract of
// every entry point.
#include "attn.h"
#include "attn_internal.h"

#include <cmath>
#include <cstdint>
#include <cstring>

using namespace attn;

namespace {

constexpr int kGridMax = 65535;  // blocks along y or z of a grid
constexpr int kGroupsMax = 1 << 20;
constexpr int kMassMaxTokens = 1 << 29;  // queries, or keys of a row, of attn_mass_paged

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_heads(int B, int Hq, int Hkv, int d, int page_size, int max_pages, int num_pages) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || max_pages <= 0 || num_pages <= 0)
    return set_error(ATTN_ERR_INVALID_ARG, "bad sizes (B=%d Hq=%d Hkv=%d max_pages=%d num_pages=%d)",
                     B, Hq, Hkv, max_pages, num_pages);
  if (Hq % Hkv != 0)
    return set_error(ATTN_ERR_INVALID_ARG, "Hq=%d is not a multiple of Hkv=%d", Hq, Hkv);
  if (d != 64 && d != 128 && d != 256)
    return set_error(ATTN_ERR_UNSUPPORTED, "head dim %d (64, 128 or 256)", d);
  if (page_size != 16) return set_error(ATTN_ERR_UNSUPPORTED, "page size %d (16)", page_size);
  if (static_cast<long long>(max_pages) * page_size > (1 << 30))
    return set_error(ATTN_ERR_INVALID_ARG, "max_pages_per_seq too large");
  if (B > kGridMax || Hq > kGridMax || static_cast<long long>(B) * Hq > (1 << 30))
    return set_error(ATTN_ERR_INVALID_ARG, "B=%d or Hq=%d above %d, or B * Hq above 2^30", B, Hq,
                     kGridMax);
  return ATTN_OK;
}

int check_scale(float scale) {
  if (!(scale > 0.f) || !std::isfinite(scale))
    return set_error(ATTN_ERR_INVALID_ARG, "scale must be finite and positive");
  return ATTN_OK;
}

int check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (workspace == nullptr || !aligned16(workspace))
    return set_error(ATTN_ERR_INVALID_ARG, "workspace must be set and 16-byte aligned");
  if (bytes < need)
    return set_error(ATTN_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", bytes, need);
  return ATTN_OK;
}

// Arguments of the decode calls that attn_decode_paged has too.
int decode_common(DecodeLaunch* a, const void* q, const void* k_pages, const void* v_pages,
                  const int* page_table, const int* seqlens, void* o, float* lse, int B, int Hq,
                  int Hkv, int d, int max_pages, int num_pages, int num_splits, float scale,
                  const float* sink) {
  if (num_splits < 1 || num_splits > 64)
    return set_error(ATTN_ERR_INVALID_ARG, "num_splits %d not in [1, 64]", num_splits);
  int rc = check_scale(scale);
  if (rc != ATTN_OK) return rc;
  if (B == 0) return ATTN_OK;
  if (!q || !k_pages || !v_pages || !page_table || !seqlens || !o)
    return set_error(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o) ||
      !aligned4(page_table) || !aligned4(seqlens) || !aligned4(lse) || !aligned4(sink))
    return set_error(ATTN_ERR_INVALID_ARG, "misaligned pointer");
  std::memset(a, 0, sizeof(*a));
  a->q = q;
  a->o = o;
  a->lse = lse;
  a->sink = sink;
  a->page_table = page_table;
  a->seqlens = seqlens;
  a->B = B;
  a->Hq = Hq;
  a->Hkv = Hkv;
  a->d = d;
  a->page = 16;
  a->max_pages = max_pages;
  a->num_pages = num_pages;
  a->num_splits = num_splits;
  a->scale = scale;
  return ATTN_OK;
}

int decode_maps(DecodeLaunch* a, const void* k_pages, const void* v_pages, int* num_sms) {
  int rc = device_info(num_sms, &a->status);
  if (rc != ATTN_OK) return rc;
  if ((rc = page_pool_map(&a->tmK, k_pages, a->d, a->Hkv, a->num_pages, "k_pages")) != ATTN_OK)
    return rc;
  return page_pool_map(&a->tmV, v_pages, a->d, a->Hkv, a->num_pages, "v_pages");
}

constexpr int kMaxSms = 256;  // SMs that workspaces provide for

// Key tiles of a row's page table.
size_t mass_tiles(int max_pages) {
  return (static_cast<size_t>(max_pages) * 16 + mass_key_tile() - 1) / mass_key_tile();
}

size_t pad16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

// Positions before each key tile and sequence, and the key tiles' units.
size_t mass_plan_bytes(int B, size_t kt) {
  return pad16((static_cast<size_t>(B) * (2 * kt + 2) + 1) * sizeof(long long));
}

// Workspace of attn_decode_paged_shared, in bytes from its start.
struct SharedLayout {
  size_t part_o, part_lse, begin, base, ints, bytes;
};

SharedLayout shared_layout(int B, int Hq, int Hkv, int d, int n_groups, int n_rows, int max_pages,
                           int num_splits) {
  SharedLayout l;
  const size_t rows = shared_part_rows(Hq, Hkv, d, n_groups, n_rows, max_pages);
  // (16 bytes more: from a 16-byte boundary up to one of 32, for the stores of the outputs)
  l.part_o = pad16(attn_decode_workspace_size(B, Hq, d, num_splits)) + 16;
  l.part_lse = l.part_o + rows * d * sizeof(float);
  l.begin = pad16(l.part_lse + rows * sizeof(float));
  l.base = l.begin + (kSharedMaxCtas + 1 + static_cast<size_t>(n_groups) + B) * sizeof(int4);
  l.ints = l.base + (static_cast<size_t>(n_groups) + kSharedMaxCtas + 1) * sizeof(long long);
  l.bytes = l.ints + 3 * static_cast<size_t>(B) * sizeof(int);
  return l;
}

int check_groups(int Hq, int n_groups, int n_rows) {
  if (n_groups < 0 || n_rows < 0 || n_groups > kGroupsMax || n_rows > kGroupsMax ||
      static_cast<long long>(n_rows) * Hq > (1 << 30))
    return set_error(ATTN_ERR_INVALID_ARG, "bad sizes (n_groups=%d n_rows=%d)", n_groups, n_rows);
  return ATTN_OK;
}

}  // namespace

extern "C" {

ATTN_API size_t attn_decode_shared_workspace_size(int B, int Hq, int Hkv, int d, int n_groups,
                                                  int n_rows, int max_pages_per_seq,
                                                  int num_splits) {
  if (check_heads(B, Hq, Hkv, d, 16, max_pages_per_seq, 1) != ATTN_OK ||
      check_groups(Hq, n_groups, n_rows) != ATTN_OK || num_splits < 1 || num_splits > 64) {
    clear_error();
    return 0;
  }
  return shared_layout(B, Hq, Hkv, d, n_groups, n_rows, max_pages_per_seq, num_splits).bytes;
}

ATTN_API int attn_decode_paged_shared(const void* q, const void* k_pages, const void* v_pages,
                                      const int* page_table, const int* seqlens,
                                      const int* cu_groups, const int* prefix_lens,
                                      const int* group_rows, void* o, float* lse, int B, int Hq,
                                      int Hkv, int d, int page_size, int max_pages_per_seq,
                                      int num_pages_total, int n_groups, int n_rows,
                                      int num_splits, float scale, const float* sink_logit,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  int rc = check_heads(B, Hq, Hkv, d, page_size, max_pages_per_seq, num_pages_total);
  if (rc != ATTN_OK) return rc;
  if ((rc = check_groups(Hq, n_groups, n_rows)) != ATTN_OK) return rc;
  if (group_rows == nullptr && n_rows > B)
    return set_error(ATTN_ERR_INVALID_ARG, "n_rows=%d of B=%d rows", n_rows, B);
  DecodeLaunch dec;
  rc = decode_common(&dec, q, k_pages, v_pages, page_table, seqlens, o, lse, B, Hq, Hkv, d,
                     max_pages_per_seq, num_pages_total, num_splits, scale, sink_logit);
  if (rc != ATTN_OK || B == 0) return rc;
  if (n_groups > 0 && (!cu_groups || !prefix_lens))
    return set_error(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned4(cu_groups) || !aligned4(prefix_lens) || !aligned4(group_rows))
    return set_error(ATTN_ERR_INVALID_ARG, "misaligned pointer");
  const SharedLayout l =
      shared_layout(B, Hq, Hkv, d, n_groups, n_rows, max_pages_per_seq, num_splits);
  if ((rc = check_workspace(workspace, workspace_bytes, l.bytes)) != ATTN_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  const size_t rows = static_cast<size_t>(B) * Hq * num_splits;
  SharedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.page_table = page_table;
  a.seqlens = seqlens;
  a.cu_groups = cu_groups;
  a.prefix_lens = prefix_lens;
  a.rows = group_rows;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.n_groups = n_groups;
  a.n_rows = n_rows;
  a.max_pages = max_pages_per_seq;
  a.num_pages = num_pages_total;
  a.scale = scale;
  a.scale2 = scale * 1.4426950408889634f;
  a.part_o = reinterpret_cast<float*>(reinterpret_cast<uintptr_t>(ws + l.part_o) & ~uintptr_t{31});
  a.part_lse = reinterpret_cast<float*>(ws + l.part_lse);
  a.begin = reinterpret_cast<int4*>(ws + l.begin);
  a.info = a.begin + kSharedMaxCtas + 1;
  a.rowinfo = a.info + n_groups;
  a.base = reinterpret_cast<long long*>(ws + l.base);
  a.runs = a.base + n_groups;
  a.entry = reinterpret_cast<int*>(ws + l.ints);
  a.start = a.entry + B;
  a.order = a.start + B;
  dec.ws_o = reinterpret_cast<float*>(ws);
  dec.ws_lse = dec.ws_o + rows * d;
  dec.order = a.order;
  dec.start = a.start;
  int num_sms = 0;
  if ((rc = decode_maps(&dec, k_pages, v_pages, &num_sms)) != ATTN_OK) return rc;
  if ((rc = whole_page_map(&a.tmK, k_pages, d, Hkv, num_pages_total, "k_pages")) != ATTN_OK ||
      (rc = whole_page_map(&a.tmV, v_pages, d, Hkv, num_pages_total, "v_pages")) != ATTN_OK)
    return rc;
  a.status = dec.status;
  const cudaError_t e = launch_attn_shared(a, dec, num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_error(e, "attn_decode_paged_shared launch");
}

ATTN_API size_t attn_decode_mass_workspace_size(int B, int Hq, int d, int max_pages_per_seq,
                                                int num_splits) {
  if (max_pages_per_seq <= 0) return 0;
  const size_t decode = attn_decode_workspace_size(B, Hq, d, num_splits);
  if (decode == 0) return 0;
  return pad16(decode) + static_cast<size_t>(B) * Hq * max_pages_per_seq * 16 * sizeof(float);
}

ATTN_API int attn_decode_paged_mass(const void* q, const void* k_pages, const void* v_pages,
                                    const int* page_table, const int* seqlens, const float* mass,
                                    float* mass_out, int* positions, const int* last_positions,
                                    void* o, float* lse, int B, int Hq, int Hkv, int d,
                                    int page_size, int max_pages_per_seq, int num_pages_total,
                                    int mass_slots, int num_splits, float scale,
                                    const float* sink_logit, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  clear_error();
  int rc = check_heads(B, Hq, Hkv, d, page_size, max_pages_per_seq, num_pages_total);
  if (rc != ATTN_OK) return rc;
  if (mass_slots <= 0) return set_error(ATTN_ERR_INVALID_ARG, "mass_slots=%d", mass_slots);
  DecodeLaunch a;
  rc = decode_common(&a, q, k_pages, v_pages, page_table, seqlens, o, lse, B, Hq, Hkv, d,
                     max_pages_per_seq, num_pages_total, num_splits, scale, sink_logit);
  if (rc != ATTN_OK || B == 0) return rc;
  if (!mass || !mass_out) return set_error(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned4(mass) || !aligned4(mass_out) || !aligned4(positions) || !aligned4(last_positions))
    return set_error(ATTN_ERR_INVALID_ARG, "misaligned pointer");
  const size_t need = attn_decode_mass_workspace_size(B, Hq, d, max_pages_per_seq, num_splits);
  if ((rc = check_workspace(workspace, workspace_bytes, need)) != ATTN_OK) return rc;
  const size_t rows = static_cast<size_t>(B) * Hq * num_splits;
  a.ws_o = static_cast<float*>(workspace);
  a.ws_lse = a.ws_o + rows * d;
  a.order = reinterpret_cast<int*>(a.ws_lse + rows);
  a.ws_scores = reinterpret_cast<float*>(
      static_cast<char*>(workspace) + pad16(attn_decode_workspace_size(B, Hq, d, num_splits)));
  a.mass = mass;
  a.mass_out = mass_out;
  a.positions = positions;
  a.last_positions = last_positions;
  a.mass_slots = mass_slots;
  int num_sms = 0;
  if ((rc = decode_maps(&a, k_pages, v_pages, &num_sms)) != ATTN_OK) return rc;
  const cudaError_t e = launch_attn_decode_mass(a, num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_error(e, "attn_decode_paged_mass launch");
}

ATTN_API size_t attn_mass_workspace_size(int B, int Hkv, int max_pages_per_seq) {
  if (B < 0 || Hkv <= 0 || max_pages_per_seq <= 0) return 0;
  const size_t kt = mass_tiles(max_pages_per_seq);
  return mass_plan_bytes(B, kt) +
         (static_cast<size_t>(B) * Hkv * kt + kMaxSms) * mass_partial_floats() * sizeof(float);
}

ATTN_API int attn_mass_paged(const void* q, const float* lse, const void* k_pages,
                             const int* page_table, const int* cu_seqlens_q, const int* seqlens_k,
                             const float* mass, float* mass_out, int* positions,
                             const int* last_positions, const int* new_tokens, int B, int Hq,
                             int Hkv, int max_Sq, int total_q, int d, int page_size,
                             int max_pages_per_seq, int num_pages_total, int mass_slots,
                             float scale, int causal, int window, int n_sink, void* workspace,
                             size_t workspace_bytes, void* stream) {
  clear_error();
  int rc = check_heads(B, Hq, Hkv, d, page_size, max_pages_per_seq, num_pages_total);
  if (rc != ATTN_OK) return rc;
  if (mass_slots <= 0 || max_Sq < 0 || total_q < 0 || max_Sq > kMassMaxTokens ||
      total_q > kMassMaxTokens || max_pages_per_seq > kMassMaxTokens / 16)
    return set_error(ATTN_ERR_INVALID_ARG,
                     "bad sizes (mass_slots=%d max_Sq=%d total_q=%d max_pages=%d)", mass_slots,
                     max_Sq, total_q, max_pages_per_seq);
  if (causal != 0 && causal != 1) return set_error(ATTN_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (window > 0 && !causal)
    return set_error(ATTN_ERR_INVALID_ARG, "a sliding window requires causal");
  if (n_sink < 0 || (n_sink > 0 && window <= 0))
    return set_error(ATTN_ERR_INVALID_ARG, "n_sink=%d needs a window", n_sink);
  if ((rc = check_scale(scale)) != ATTN_OK) return rc;
  if (B == 0) return ATTN_OK;
  if ((total_q > 0 && (!q || !lse)) || !k_pages || !page_table || !cu_seqlens_q || !seqlens_k ||
      !mass || !mass_out)
    return set_error(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(q) || !aligned16(k_pages) || !aligned4(lse) || !aligned4(page_table) ||
      !aligned4(cu_seqlens_q) || !aligned4(seqlens_k) || !aligned4(mass) || !aligned4(mass_out) ||
      !aligned4(positions) || !aligned4(last_positions) || !aligned4(new_tokens))
    return set_error(ATTN_ERR_INVALID_ARG, "misaligned pointer");
  const size_t need = attn_mass_workspace_size(B, Hkv, max_pages_per_seq);
  if ((rc = check_workspace(workspace, workspace_bytes, need)) != ATTN_OK) return rc;
  MassArgs a;
  std::memset(&a, 0, sizeof(a));
  int num_sms = 0;
  if ((rc = device_info(&num_sms, &a.status)) != ATTN_OK) return rc;
  if (num_sms > kMaxSms) return set_error(ATTN_ERR_UNSUPPORTED, "%d SMs", num_sms);
  a.G = Hq / Hkv;
  // The heads of a query tile: the group, or its largest part that fits.
  const int tile = mass_query_tile(d);
  a.GP = a.G;
  if (a.G > tile) {
    a.GP = tile;
    while (a.G % a.GP != 0) --a.GP;
  }
  a.TQ = tile / a.GP;
  a.HC = a.G / a.GP;
  if ((rc = whole_page_map(&a.tmK, k_pages, d, Hkv, num_pages_total, "k_pages")) != ATTN_OK)
    return rc;
  // with no query at all the map is of nothing that is read
  if ((rc = packed_rows_map(&a.tmQ, total_q > 0 ? q : k_pages, d, total_q > 0 ? Hq : Hkv,
                            total_q > 0 ? total_q : 16, total_q > 0 ? a.GP : 1, a.TQ, "q")) !=
      ATTN_OK)
    return rc;
  a.lse = lse;
  a.page_table = page_table;
  a.cu_q = cu_seqlens_q;
  a.seqlens_k = seqlens_k;
  a.mass = mass;
  a.mass_out = mass_out;
  a.positions = positions;
  a.last_positions = last_positions;
  a.new_tokens = new_tokens;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.max_Sq = max_Sq;
  a.total_q = total_q;
  a.max_pages = max_pages_per_seq;
  a.num_pages = num_pages_total;
  a.slots = mass_slots;
  a.max_kt = static_cast<int>(mass_tiles(max_pages_per_seq));
  a.scale2 = scale * 1.4426950408889634f;
  a.causal = causal;
  const int longest = max_pages_per_seq * 16;
  a.window = window <= 0 ? 0 : window < longest ? window : longest;
  a.n_sink = n_sink;
  a.ws_plan = static_cast<long long*>(workspace);
  a.ws_part = reinterpret_cast<float*>(
      static_cast<char*>(workspace) + mass_plan_bytes(B, a.max_kt));
  const cudaError_t e = launch_attn_mass(a, num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_error(e, "attn_mass_paged launch");
}

ATTN_API size_t attn_evict_workspace_size(int layers, int B, int Hkv, int slots,
                                          int max_pages_per_seq) {
  if (layers <= 0 || B < 0 || Hkv <= 0 || slots <= 0 || max_pages_per_seq <= 0) return 0;
  const long long pool = static_cast<long long>(max_pages_per_seq) * 16;
  const size_t most = static_cast<size_t>(slots < pool ? slots : pool) / 2;
  return static_cast<size_t>(layers) * B * Hkv * (most * 8 + 4);
}

ATTN_API int attn_evict_paged(float* mass, int* positions, const int* page_table,
                              const int* seqlens, const int* keep, const int* refs,
                              int* new_seqlens, void* k_pages, void* v_pages, int B, int layers,
                              int Hkv, int d, int slots, int page_size, int max_pages_per_seq,
                              int num_pages_total, int n_sink, int recent, void* workspace,
                              size_t workspace_bytes, void* stream) {
  clear_error();
  int rc = check_heads(B, Hkv, Hkv, d, page_size, max_pages_per_seq, num_pages_total);
  if (rc != ATTN_OK) return rc;
  if (layers < 1 || layers > (1 << 16) || slots <= 0 || n_sink < 0 || recent < 0)
    return set_error(ATTN_ERR_INVALID_ARG, "bad sizes (layers=%d slots=%d n_sink=%d recent=%d)",
                     layers, slots, n_sink, recent);
  const long long units = static_cast<long long>(layers) * B * Hkv;
  if (units > kEvictMaxUnits)
    return set_error(ATTN_ERR_INVALID_ARG, "%lld rows, layers and heads, at most %d", units,
                     kEvictMaxUnits);
  if (num_pages_total > kPagesMaxPages)
    return set_error(ATTN_ERR_INVALID_ARG, "%d pages, at most %d", num_pages_total, kPagesMaxPages);
  if (B == 0) return ATTN_OK;
  if (!mass || !positions || !page_table || !seqlens || !keep || !new_seqlens || !k_pages ||
      !v_pages)
    return set_error(ATTN_ERR_INVALID_ARG, "null pointer");
  if (!aligned4(mass) || !aligned4(positions) || !aligned4(page_table) || !aligned4(seqlens) ||
      !aligned4(keep) || !aligned4(refs) || !aligned4(new_seqlens) || !aligned16(k_pages) ||
      !aligned16(v_pages))
    return set_error(ATTN_ERR_INVALID_ARG, "misaligned pointer");
  if (new_seqlens == seqlens || new_seqlens == keep)
    return set_error(ATTN_ERR_INVALID_ARG, "new_seqlens must be an array of its own");
  const size_t need = attn_evict_workspace_size(layers, B, Hkv, slots, max_pages_per_seq);
  if ((rc = check_workspace(workspace, workspace_bytes, need)) != ATTN_OK) return rc;
  EvictArgs a;
  std::memset(&a, 0, sizeof(a));
  a.mass = mass;
  a.positions = positions;
  a.page_table = page_table;
  a.seqlens = seqlens;
  a.keep = keep;
  a.refs = refs;
  a.new_seqlens = new_seqlens;
  a.k_pages = static_cast<uint4*>(k_pages);
  a.v_pages = static_cast<uint4*>(v_pages);
  a.units = static_cast<int>(units);
  a.B = B;
  a.Hkv = Hkv;
  a.slots = slots;
  a.max_pages = max_pages_per_seq;
  a.num_pages = num_pages_total;
  a.vecs = d / 8;
  const long long pool = static_cast<long long>(max_pages_per_seq) * 16;
  a.most_moves = static_cast<int>((slots < pool ? slots : pool) / 2);
  a.n_sink = n_sink;
  a.recent = recent;
  a.ws = static_cast<int*>(workspace);
  int num_sms = 0;
  if ((rc = device_info(&num_sms, &a.status)) != ATTN_OK) return rc;
  const cudaError_t e = launch_attn_evict(a, num_sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_error(e, "attn_evict_paged launch");
}

}  // extern "C"
