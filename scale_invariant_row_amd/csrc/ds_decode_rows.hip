// The C ABI of include/ds_decode_rows.h: argument checks and launches.
//
// Every check runs before the first HIP call, so a refused call has touched
// neither the device nor the stream.
#include "ds_decode_rows.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <utility>

#include "decode_launch.hpp"
#include "host_checks.hpp"

namespace {

using namespace dsh;

constexpr int64_t kMostHeadRows = 1 << 23;    // (row, head) pairs of an attention call: a grid's limit
constexpr int64_t kMostSlices = (1 << 24) - 1;   // of a verification: likewise

bool flag_ok(int32_t v) { return v == 0 || v == 1; }

int check_heads(int64_t rows, int32_t nq, int32_t nk, int32_t head_dim) {
  if (rows < 0 || nq < 0 || nk < 0) return DS_ERR_SHAPE;
  if (head_dim < 16 || head_dim > 256 || head_dim % 16 != 0) return DS_ERR_SHAPE;
  return std::max((int64_t)nq, (int64_t)nk) * head_dim > (1 << 24) ? DS_ERR_SHAPE : DS_OK;
}

int check_turn(int32_t rotary_dim, int32_t least, int32_t head_dim, int32_t interleaved,
               float amplitude) {
  if (rotary_dim < least || rotary_dim > head_dim || rotary_dim % 2 != 0) return DS_ERR_SHAPE;
  return flag_ok(interleaved) && std::isfinite(amplitude) ? DS_OK : DS_ERR_ARG;
}

// Both directions of ds_rope_rows.
int rope(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk, const int32_t* positions,
         const float* inv_freq, int32_t rotary_dim, int32_t interleaved, float amplitude, float sign,
         uint16_t* q_out, int64_t ldq_out, uint16_t* k_out, int64_t ldk_out, int64_t rows,
         int32_t nq, int32_t nk, int32_t head_dim, ds_stream_t stream) {
  int st = check_heads(rows, nq, nk, head_dim);
  if (st != DS_OK) return st;
  if ((st = check_turn(rotary_dim, 2, head_dim, interleaved, amplitude)) != DS_OK) return st;
  const int64_t wq = (int64_t)nq * head_dim, wk = (int64_t)nk * head_dim;
  if (rows == 0 || wq + wk == 0) return DS_OK;
  if (positions == nullptr || inv_freq == nullptr) return DS_ERR_NULL;
  if (!aligned(positions, 4) || !aligned(inv_freq, 4)) return DS_ERR_ALIGN;
  const View v[4] = {{q, ldq, wq, false}, {k, ldk, wk, false}, {q_out, ldq_out, wq, true},
                     {k_out, ldk_out, wk, true}};
  const int in_place[2][2] = {{2, 0}, {3, 1}};
  const void* const vecs[2] = {positions, inv_freq};
  const size_t nb[2] = {(size_t)rows * 4, (size_t)rotary_dim * 2};
  if ((st = check_views(v, rows, in_place, 2, vecs, nb, 2)) != DS_OK) return st;
  int cus = 0;
  if ((st = device_cus(&cus)) != DS_OK) return st;
  (void)hipGetLastError();
  return launch_status(launch_in_pieces(rows, dsr::kHeadRows, cus, [&](int64_t r0, int64_t n) {
    dsr::RopeArgs a{};
    a.x[0] = wq > 0 ? q + r0 * ldq : nullptr;
    a.x[1] = wk > 0 ? k + r0 * ldk : nullptr;
    a.y[0] = wq > 0 ? q_out + r0 * ldq_out : nullptr;
    a.y[1] = wk > 0 ? k_out + r0 * ldk_out : nullptr;
    a.pos = positions + r0;
    a.turn = dsr::Turn{inv_freq, rotary_dim, interleaved, amplitude, sign};
    a.ldx[0] = ldq;
    a.ldx[1] = ldk;
    a.ldy[0] = ldq_out;
    a.ldy[1] = ldk_out;
    a.rows = n;
    a.nh[0] = nq;
    a.nh[1] = nk;
    a.hd = head_dim;
    return dsr::launch_rope_rows(a, cus,
                                 (hipStream_t)stream);
  }));
}

int64_t element_bytes(const ds_kv_cache& c) { return c.type == DS_TYPE_E4M3 ? 1 : 2; }

// A cache's sizes (no pointer is looked at).
int check_cache_sizes(const ds_kv_cache& c) {
  if (c.type != DS_TYPE_BF16 && c.type != DS_TYPE_E4M3) return DS_ERR_ARG;
  int st = check_heads(0, 0, c.n_heads, c.head_dim);
  if (st != DS_OK) return st;
  if (c.n_heads < 1 || c.n_pages < 0 || c.n_seqs < 0 || c.pages_per_seq < 0) return DS_ERR_SHAPE;
  if (c.page_size < 1 || c.page_size > DS_MAX_PAGE || (c.page_size & (c.page_size - 1)) != 0)
    return DS_ERR_SHAPE;
  if ((int64_t)c.pages_per_seq * c.page_size > (1 << 30)) return DS_ERR_SHAPE;
  return DS_OK;
}

// Elements from a cache's first to one past its last.
int64_t cache_span(const ds_kv_cache& c) {
  return (c.n_pages - 1) * c.page_stride + (c.page_size - 1) * c.token_stride +
         (c.n_heads - 1) * c.head_stride + c.head_dim;
}

// A whole cache: sizes, strides, pointers, and no element twice in k and v.
int check_cache(const ds_kv_cache& c) {
  int st = check_cache_sizes(c);
  if (st != DS_OK) return st;
  if (c.ld_table < c.pages_per_seq || (c.n_seqs > 0 && c.ld_table > kMostBytes / 4 / c.n_seqs))
    return DS_ERR_SHAPE;
  const int64_t vec = 16 / element_bytes(c);
  std::pair<int64_t, int64_t> dims[4] = {{c.page_stride, c.n_pages}, {c.token_stride, c.page_size},
                                         {c.head_stride, c.n_heads}, {0, 2}};
  for (int i = 0; i < 3; ++i)
    if (dims[i].first < 0 || dims[i].first % vec != 0 ||
        (dims[i].second > 0 && dims[i].first > kMostBytes / 16 / dims[i].second))
      return DS_ERR_SHAPE;
  if (c.n_seqs > 0 && c.pages_per_seq > 0 && c.page_table == nullptr) return DS_ERR_NULL;
  if (!aligned(c.page_table, 4) || !aligned(c.k_scale, 4) || !aligned(c.v_scale, 4))
    return DS_ERR_ALIGN;
  if (c.n_pages == 0) return DS_OK;
  if (c.k == nullptr || c.v == nullptr) return DS_ERR_NULL;
  if (!aligned(c.k, 16) || !aligned(c.v, 16)) return DS_ERR_ALIGN;
  // each dimension's stride clears the extent of those of smaller stride,
  // k and v being a dimension of two
  const uintptr_t k = reinterpret_cast<uintptr_t>(c.k), v = reinterpret_cast<uintptr_t>(c.v);
  dims[3].first = (int64_t)((k < v ? v - k : k - v) / (uintptr_t)element_bytes(c));
  std::sort(dims, dims + 4);
  int64_t extent = c.head_dim;
  for (const auto& d : dims) {
    if (d.second < 2) continue;
    if (d.first < extent) return DS_ERR_ARG;
    extent += d.first * (d.second - 1);
  }
  return DS_OK;
}

// The bytes between k's (v's) first element and its last; where the two lie in
// one buffer, each holds some of the other's.
Buf store_of(const ds_kv_cache& c, const void* p) {
  return c.n_pages == 0 ? Buf{nullptr, 0} : Buf{p, (size_t)(cache_span(c) * element_bytes(c))};
}

size_t table_bytes(const ds_kv_cache& c) {
  return c.n_seqs == 0 ? 0 : ((size_t)(c.n_seqs - 1) * (size_t)c.ld_table + (size_t)c.pages_per_seq) * 4;
}

dsr::CacheView view_of(const ds_kv_cache& c) {
  const int64_t b = element_bytes(c);
  dsr::CacheView v{};
  v.k = static_cast<char*>(c.k);
  v.v = static_cast<char*>(c.v);
  v.k_scale = c.k_scale;
  v.v_scale = c.v_scale;
  v.table = c.page_table;
  v.page_bytes = c.page_stride * b;
  v.token_bytes = c.token_stride * b;
  v.head_bytes = c.head_stride * b;
  v.ld_table = c.ld_table;
  v.e4m3 = c.type == DS_TYPE_E4M3;
  v.n_pages = c.n_pages;
  while ((1 << v.page_shift) < c.page_size) ++v.page_shift;
  v.heads = c.n_heads;
  v.hd = c.head_dim;
  v.seqs = c.n_seqs;
  v.pages_per_seq = c.pages_per_seq;
  return v;
}

}  // namespace

extern "C" {

int ds_rope_rows(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk,
                 const int32_t* positions, const float* inv_freq, int32_t rotary_dim,
                 int32_t interleaved, float amplitude, uint16_t* q_out, int64_t ldq_out,
                 uint16_t* k_out, int64_t ldk_out, int64_t rows, int32_t n_q_heads,
                 int32_t n_kv_heads, int32_t head_dim, ds_stream_t stream) {
  return rope(q, ldq, k, ldk, positions, inv_freq, rotary_dim, interleaved, amplitude, 1.f, q_out,
              ldq_out, k_out, ldk_out, rows, n_q_heads, n_kv_heads, head_dim, stream);
}

int ds_rope_rows_backward(const uint16_t* dq_out, int64_t lddq_out, const uint16_t* dk_out,
                          int64_t lddk_out, const int32_t* positions, const float* inv_freq,
                          int32_t rotary_dim, int32_t interleaved, float amplitude, uint16_t* dq,
                          int64_t lddq, uint16_t* dk, int64_t lddk, int64_t rows,
                          int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                          ds_stream_t stream) {
  return rope(dq_out, lddq_out, dk_out, lddk_out, positions, inv_freq, rotary_dim, interleaved,
              amplitude, -1.f, dq, lddq, dk, lddk, rows, n_q_heads, n_kv_heads, head_dim, stream);
}

int ds_rope_frequencies(float* inv_freq, int32_t rotary_dim, double base, double factor,
                        double original, double low, double high) {
  if (rotary_dim < 2 || rotary_dim > 256 || rotary_dim % 2 != 0) return DS_ERR_SHAPE;
  if (!std::isfinite(base) || base <= 0.0 || !std::isfinite(factor) || factor < 1.0 ||
      !std::isfinite(original) || original <= 0.0 || !std::isfinite(low) || !std::isfinite(high) ||
      low < 0.0 || high < low || (high == low && high > 0.0))
    return DS_ERR_ARG;
  if (inv_freq == nullptr) return DS_ERR_NULL;
  if (!aligned(inv_freq, 4)) return DS_ERR_ALIGN;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rotary_dim);
    const double turns = original * f * 0.15915494309189534;
    const double w = high > low ? std::min(1.0, std::max(0.0, (turns - low) / (high - low))) : 0.0;
    inv_freq[i] = (float)(f * (w + (1.0 - w) / factor));
  }
  return DS_OK;
}

int ds_cache_append_rows(const ds_kv_cache* cache, const uint16_t* q, int64_t ldq,
                         const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                         const int32_t* positions, const int32_t* seqs, const float* inv_freq,
                         int32_t rotary_dim, int32_t interleaved, float amplitude, int32_t rms,
                         const float* q_weight, const float* k_weight, float eps, uint16_t* q_out,
                         int64_t ldq_out, int64_t rows, int32_t n_q_heads, ds_stream_t stream) {
  if (cache == nullptr) return DS_ERR_NULL;
  const ds_kv_cache& c = *cache;
  int st = check_cache(c);
  if (st != DS_OK) return st;
  if ((st = check_heads(rows, n_q_heads, c.n_heads, c.head_dim)) != DS_OK) return st;
  if ((st = check_turn(rotary_dim, 0, c.head_dim, interleaved, amplitude)) != DS_OK) return st;
  if (!flag_ok(rms) || !finite_nonneg(eps) || (rms == 0 && (q_weight != nullptr || k_weight != nullptr)))
    return DS_ERR_ARG;
  if (rows == 0) return DS_OK;
  if (seqs == nullptr && (c.n_seqs == 0 || rows % c.n_seqs != 0)) return DS_ERR_SHAPE;
  if (positions == nullptr || (rotary_dim > 0 && inv_freq == nullptr)) return DS_ERR_NULL;
  if (!aligned(positions, 4) || !aligned(seqs, 4) || !aligned(inv_freq, 4) ||
      !aligned(q_weight, 16) || !aligned(k_weight, 16))
    return DS_ERR_ALIGN;
  const int64_t wq = (int64_t)n_q_heads * c.head_dim, wk = (int64_t)c.n_heads * c.head_dim;
  const View views[4] = {{q, ldq, wq, false}, {k, ldk, wk, false}, {v, ldv, wk, false},
                         {q_out, ldq_out, wq, true}};
  const int in_place[1][2] = {{3, 0}};
  const Buf ks = store_of(c, c.k), vs = store_of(c, c.v);
  const size_t rb = (size_t)rows * 4, wb = (size_t)c.head_dim * 4, sb = (size_t)c.n_heads * 4;
  const void* const vecs[10] = {positions, seqs, inv_freq,  q_weight,  k_weight,
                                ks.p,      vs.p, c.k_scale, c.v_scale, c.page_table};
  const size_t nb[10] = {rb,       rb,       (size_t)rotary_dim * 2, wb, wb,
                         ks.bytes, vs.bytes, sb,                     sb, table_bytes(c)};
  if ((st = check_views(views, rows, in_place, 1, vecs, nb, 10)) != DS_OK) return st;
  const Buf k_out[1] = {ks}, v_out[1] = {vs};
  const Buf ins[11] = {{wq > 0 ? q : nullptr, span_bytes(rows, ldq, wq)},
                       {k, span_bytes(rows, ldk, wk)},
                       {v, span_bytes(rows, ldv, wk)},
                       {positions, rb},
                       {seqs, rb},
                       {inv_freq, (size_t)rotary_dim * 2},
                       {q_weight, wb},
                       {k_weight, wb},
                       {c.k_scale, sb},
                       {c.v_scale, sb},
                       {c.page_table, table_bytes(c)}};
  if (!apart(k_out, ins) || !apart(v_out, ins)) return DS_ERR_ARG;
  int cus = 0;
  if ((st = device_cus(&cus)) != DS_OK) return st;
  (void)hipGetLastError();
  return launch_status(launch_in_pieces(rows, dsr::kHeadRows, cus, [&](int64_t r0, int64_t n) {
    dsr::AppendArgs a{};
    a.x[0] = wq > 0 ? q + r0 * ldq : nullptr;
    a.x[1] = k + r0 * ldk;
    a.x[2] = v + r0 * ldv;
    a.ldx[0] = ldq;
    a.ldx[1] = ldk;
    a.ldx[2] = ldv;
    a.q_out = wq > 0 ? q_out + r0 * ldq_out : nullptr;
    a.ldq_out = ldq_out;
    a.w[0] = q_weight;
    a.w[1] = k_weight;
    a.pos = positions + r0;
    a.seq = seqs != nullptr ? seqs + r0 : nullptr;
    a.turn = dsr::Turn{inv_freq, rotary_dim, interleaved, amplitude, 1.f};
    a.cache = view_of(c);
    a.rows = n;
    a.row0 = r0;
    a.rows_per_seq = c.n_seqs > 0 ? std::max<int64_t>(1, rows / c.n_seqs) : 1;
    a.q_heads = n_q_heads;
    a.rms = rms;
    a.eps = eps;
    return dsr::launch_cache_append(a, cus,
                                    (hipStream_t)stream);
  }));
}

int64_t ds_cache_attention_rows_workspace(const ds_kv_cache* cache, int32_t n_q_heads,
                                          int32_t new_tokens, int32_t window) {
  if (cache == nullptr) return DS_ERR_NULL;
  const ds_kv_cache& c = *cache;
  int st = check_cache_sizes(c);
  if (st != DS_OK) return st;
  if ((st = check_heads(0, n_q_heads, 0, c.head_dim)) != DS_OK) return st;
  if (n_q_heads < 1 || n_q_heads % c.n_heads != 0) return DS_ERR_SHAPE;
  if (new_tokens < 1 || new_tokens > DS_MAX_NEW) return DS_ERR_SHAPE;
  if (window < 0) return DS_ERR_ARG;
  if ((int64_t)c.n_seqs * new_tokens > kMostHeadRows / n_q_heads) return DS_ERR_SHAPE;
  return dsr::attention_workspace(c.n_seqs, (int64_t)c.pages_per_seq * c.page_size, n_q_heads,
                                  c.n_heads, c.head_dim, new_tokens, window);
}

int ds_cache_attention_rows(const ds_kv_cache* cache, const uint16_t* q, int64_t ldq,
                            int32_t n_q_heads, const int32_t* lens, int32_t new_tokens,
                            int32_t window, float scale, uint16_t* out, int64_t ldout, float* lse,
                            void* workspace, int64_t workspace_bytes, ds_stream_t stream) {
  const int64_t need = ds_cache_attention_rows_workspace(cache, n_q_heads, new_tokens, window);
  if (need < 0) return (int)need;
  const ds_kv_cache& c = *cache;
  int st = check_cache(c);
  if (st != DS_OK) return st;
  if (!std::isfinite(scale)) return DS_ERR_ARG;
  if (c.n_seqs == 0) return DS_OK;
  if (lens == nullptr) return DS_ERR_NULL;
  if (!aligned(lens, 4) || !aligned(lse, 4)) return DS_ERR_ALIGN;
  const int64_t rows = (int64_t)c.n_seqs * new_tokens, wq = (int64_t)n_q_heads * c.head_dim;
  const View views[2] = {{q, ldq, wq, false}, {out, ldout, wq, true}};
  const Buf ks = store_of(c, c.k), vs = store_of(c, c.v);
  const size_t lb = (size_t)c.n_seqs * 4, sb = (size_t)c.n_heads * 4;
  const void* const vecs[6] = {lens, ks.p, vs.p, c.k_scale, c.v_scale, c.page_table};
  const size_t nb[6] = {lb, ks.bytes, vs.bytes, sb, sb, table_bytes(c)};
  if ((st = check_views(views, rows, nullptr, 0, vecs, nb, 6)) != DS_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != DS_OK) return st;
  const Buf outs[3] = {{out, span_bytes(rows, ldout, wq)},
                       {lse, (size_t)rows * (size_t)n_q_heads * 4},
                       {workspace, (size_t)need}};
  const Buf ins[6] = {{lens, lb}, ks, vs, {c.k_scale, sb}, {c.v_scale, sb}, {c.page_table, table_bytes(c)}};
  const Buf beside[2] = {outs[1], outs[2]}, qs[1] = {{q, span_bytes(rows, ldq, wq)}};
  if (!apart(outs, ins) || !apart(beside, qs)) return DS_ERR_ARG;
  int cus = 0;
  if ((st = device_cus(&cus)) != DS_OK) return st;
  dsr::AttendArgs a{};
  a.cache = view_of(c);
  a.q = q;
  a.lens = lens;
  a.out = out;
  a.lse = lse;
  a.ldq = ldq;
  a.ldo = ldout;
  a.q_heads = n_q_heads;
  a.n_new = new_tokens;
  a.window = window >= c.pages_per_seq * c.page_size ? 0 : window;   // a window of all is none
  a.scale = scale;
  (void)hipGetLastError();
  return launch_status(dsr::launch_cache_attention(a, cus, workspace, (hipStream_t)stream));
}

int64_t ds_draft_verify_rows_workspace(int64_t n_seqs, int32_t n_drafts, int64_t vocab,
                                       int32_t with_draft) {
  if (n_seqs < 0 || n_drafts < 0 || n_drafts > DS_MAX_DRAFTS || vocab < 1 || vocab > DS_MAX_VOCAB)
    return DS_ERR_SHAPE;
  if (!flag_ok(with_draft)) return DS_ERR_ARG;
  if (n_seqs > kMostSlices / dsr::verify_slices(n_drafts, vocab, with_draft != 0)) return DS_ERR_SHAPE;
  return dsr::verify_workspace(n_seqs, n_drafts, vocab, with_draft != 0);
}

int ds_draft_verify_rows(const void* target, int32_t target_type, int64_t ldt, const float* scale,
                         float inv_temp, const void* draft, int32_t draft_type, int64_t ldd,
                         const float* draft_scale, float draft_inv_temp, const void* drafted,
                         int32_t id_bytes, const float* u_accept, const float* u_sample,
                         int32_t* accepted, int32_t* tokens, float* logp, int64_t n_seqs,
                         int32_t n_drafts, int64_t vocab, void* workspace,
                         int64_t workspace_bytes, ds_stream_t stream) {
  const bool with = draft != nullptr && n_drafts > 0;
  const int64_t need = ds_draft_verify_rows_workspace(n_seqs, n_drafts, vocab, with);
  if (need < 0) return (int)need;
  if (ldt < vocab || (with && ldd < vocab)) return DS_ERR_SHAPE;
  const int64_t t_rows = n_seqs * (n_drafts + 1), d_rows = n_seqs * n_drafts;
  if (t_rows > kMostBytes / 4 / ldt || (with && d_rows > kMostBytes / 4 / ldd)) return DS_ERR_SHAPE;
  if (!type_ok(target_type) || (with && !type_ok(draft_type)) || !id_bytes_ok(id_bytes)) return DS_ERR_ARG;
  if (!std::isfinite(inv_temp) || inv_temp <= 0.f ||
      (with && (!std::isfinite(draft_inv_temp) || draft_inv_temp <= 0.f)))
    return DS_ERR_ARG;
  if (n_seqs == 0) return DS_OK;
  if (target == nullptr || u_sample == nullptr || accepted == nullptr || tokens == nullptr ||
      logp == nullptr || (n_drafts > 0 && (drafted == nullptr || u_accept == nullptr)))
    return DS_ERR_NULL;
  if (!aligned(target, (uintptr_t)type_bytes(target_type)) ||
      (with && !aligned(draft, (uintptr_t)type_bytes(draft_type))) || !aligned(scale, 4) ||
      !aligned(draft_scale, 4) || !aligned(drafted, (uintptr_t)id_bytes) || !aligned(u_accept, 4) ||
      !aligned(u_sample, 4) || !aligned(accepted, 4) || !aligned(tokens, 4) || !aligned(logp, 4))
    return DS_ERR_ALIGN;
  int st = check_workspace(workspace, workspace_bytes, need);
  if (st != DS_OK) return st;
  const size_t sb = (size_t)n_seqs * 4, tb = (size_t)t_rows * 4, vb = (size_t)vocab * 4;
  const Buf outs[4] = {{accepted, sb}, {tokens, tb}, {logp, tb}, {workspace, (size_t)need}};
  const Buf ins[7] = {
      {target, ((size_t)(t_rows - 1) * (size_t)ldt + (size_t)vocab) * (size_t)type_bytes(target_type)},
      {with ? draft : nullptr,
       with ? ((size_t)(d_rows - 1) * (size_t)ldd + (size_t)vocab) * (size_t)type_bytes(draft_type) : 0},
      {scale, vb},
      {with ? draft_scale : nullptr, vb},
      {drafted, (size_t)d_rows * (size_t)id_bytes},
      {u_accept, (size_t)d_rows * 4},
      {u_sample, sb}};
  if (!apart(outs, ins)) return DS_ERR_ARG;
  int cus = 0;
  if ((st = device_cus(&cus)) != DS_OK) return st;
  dsr::VerifyArgs a{};
  a.x[0] = target;
  a.x[1] = with ? draft : nullptr;
  a.ld[0] = ldt;
  a.ld[1] = ldd;
  a.scale[0] = scale;
  a.scale[1] = draft_scale;
  a.inv_temp[0] = inv_temp;
  a.inv_temp[1] = draft_inv_temp;
  a.f32[0] = target_type == DS_TYPE_F32;
  a.f32[1] = draft_type == DS_TYPE_F32;
  a.drafted = drafted;
  a.id_bytes = id_bytes;
  a.u_accept = u_accept;
  a.u_sample = u_sample;
  a.accepted = accepted;
  a.tokens = tokens;
  a.logp = logp;
  a.seqs = (int32_t)n_seqs;
  a.drafts = n_drafts;
  a.vocab = (int32_t)vocab;
  (void)hipGetLastError();
  return launch_status(dsr::launch_draft_verify(a, cus, workspace, (hipStream_t)stream));
}

}  // extern "C"
