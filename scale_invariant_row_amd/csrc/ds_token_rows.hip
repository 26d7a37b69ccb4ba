// The C ABI of include/ds_token_rows.h: argument checks and launches.
//
// Every check runs before the first HIP call, so a refused call has touched
// neither the device nor the stream.
#include "ds_token_rows.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "host_checks.hpp"
#include "token_launch.hpp"

namespace {

using namespace dsh;

constexpr int64_t kMostGradRows = 1 << 30;   // of an embedding's gradient
constexpr int64_t kMostGradBytes = 400ll << 30;   // of its table and of its rows (a grid's limit)

// Shape and types shared by an embedding's two directions.
int check_embed(int32_t type, int64_t vocab, int32_t id_bytes, float scale, int64_t rows,
                int64_t cols) {
  int st = check_matrix(rows, cols, 8, 4);
  if (st != DS_OK) return st;
  if (vocab < 0 || vocab > INT32_MAX || vocab > kMostBytes / (cols * 4)) return DS_ERR_SHAPE;
  if (!type_ok(type) || !id_bytes_ok(id_bytes) || !std::isfinite(scale)) return DS_ERR_ARG;
  return DS_OK;
}

bool grad_sizes_ok(int32_t type, int64_t vocab, int64_t rows, int64_t cols) {
  return rows <= kMostGradRows && rows <= kMostGradBytes / (cols * 2) &&
         vocab <= kMostGradBytes / (cols * type_bytes(type));
}

}  // namespace

extern "C" {

int ds_embed_rows(const void* table, int32_t table_type, int64_t vocab, const void* ids,
                  int32_t id_bytes, float scale, uint16_t* out, int64_t rows, int64_t cols,
                  ds_stream_t stream) {
  int st = check_embed(table_type, vocab, id_bytes, scale, rows, cols);
  if (st != DS_OK || rows == 0) return st;
  if ((vocab > 0 && table == nullptr) || ids == nullptr || out == nullptr) return DS_ERR_NULL;
  if (!aligned(table, 16) || !aligned(out, 16) || !aligned(ids, (uintptr_t)id_bytes))
    return DS_ERR_ALIGN;
  const size_t nb = (size_t)rows * (size_t)cols * 2;
  if (overlaps(out, nb, table, (size_t)vocab * (size_t)cols * (size_t)type_bytes(table_type)) ||
      overlaps(out, nb, ids, (size_t)rows * (size_t)id_bytes))
    return DS_ERR_ARG;
  int cus = 0;
  if ((st = device_cus(&cus)) != DS_OK) return st;
  (void)hipGetLastError();
  return launch_status(launch_in_pieces(rows, 4, cus, [&](int64_t r0, int64_t n) {
    dsr::EmbedArgs a{};
    a.table = table;
    a.ids = static_cast<const char*>(ids) + r0 * id_bytes;
    a.out = out + r0 * cols;
    a.vocab = vocab;
    a.rows = n;
    a.cols = (int32_t)cols;
    a.scale = scale;
    return dsr::launch_embed_rows(table_type == DS_TYPE_F32, id_bytes == 8, a, (int)((n + 3) / 4),
                                  (hipStream_t)stream);
  }));
}

int64_t ds_embed_rows_backward_workspace(int64_t vocab, int64_t rows, int64_t cols) {
  int st = check_embed(DS_TYPE_F32, vocab, 8, 1.f, rows, cols);
  if (st != DS_OK) return st;
  if (!grad_sizes_ok(DS_TYPE_BF16, vocab, rows, cols)) return DS_ERR_SHAPE;
  return vocab == 0 ? 0 : dsr::embed_grad_workspace(vocab, rows, cols);
}

int ds_embed_rows_backward(const uint16_t* dy, const void* ids, int32_t id_bytes, float scale,
                           void* dtable, int32_t grad_type, int32_t accumulate, int64_t vocab,
                           int64_t rows, int64_t cols, void* workspace, int64_t workspace_bytes,
                           ds_stream_t stream) {
  int st = check_embed(grad_type, vocab, id_bytes, scale, rows, cols);
  if (st != DS_OK) return st;
  if (!grad_sizes_ok(grad_type, vocab, rows, cols)) return DS_ERR_SHAPE;
  if (accumulate != 0 && accumulate != 1) return DS_ERR_ARG;
  if (vocab == 0 || (rows == 0 && accumulate)) return DS_OK;
  if (dtable == nullptr || (rows > 0 && (dy == nullptr || ids == nullptr))) return DS_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(dtable, 16) || !aligned(ids, (uintptr_t)id_bytes))
    return DS_ERR_ALIGN;
  const int64_t need = ds_embed_rows_backward_workspace(vocab, rows, cols);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != DS_OK) return st;
  const size_t nd = (size_t)vocab * (size_t)cols * (size_t)type_bytes(grad_type);
  const size_t ny = (size_t)rows * (size_t)cols * 2, ni = (size_t)rows * (size_t)id_bytes;
  if (overlaps(dtable, nd, dy, ny) || overlaps(dtable, nd, ids, ni) ||
      overlaps(workspace, (size_t)need, dtable, nd) || overlaps(workspace, (size_t)need, dy, ny) ||
      overlaps(workspace, (size_t)need, ids, ni))
    return DS_ERR_ARG;
  int cus = 0;
  if ((st = device_cus(&cus)) != DS_OK) return st;
  dsr::EmbedGradArgs a{};
  a.dy = dy;
  a.ids = ids;
  a.dtable = dtable;
  a.vocab = (int32_t)vocab;
  a.rows = (int32_t)rows;
  a.cols = (int32_t)cols;
  a.accumulate = accumulate;
  a.scale = scale;
  (void)hipGetLastError();
  return launch_status(dsr::launch_embed_rows_backward(grad_type == DS_TYPE_F32, id_bytes == 8, a,
                                                       workspace, (hipStream_t)stream));
}

}  // extern "C"

namespace {

int check_qk(int64_t rows, int32_t nq, int32_t nk, int32_t head_dim, float eps, int64_t* wq,
             int64_t* wk) {
  if (rows < 0 || nq < 0 || nk < 0) return DS_ERR_SHAPE;
  if (head_dim < 16 || head_dim > 256 || head_dim % 16 != 0) return DS_ERR_SHAPE;
  if (!finite_nonneg(eps)) return DS_ERR_ARG;
  *wq = (int64_t)nq * head_dim;
  *wk = (int64_t)nk * head_dim;
  return *wq > (1 << 24) || *wk > (1 << 24) ? DS_ERR_SHAPE : DS_OK;
}

}  // namespace

extern "C" {

int ds_qk_rows_rms(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk,
                   const int32_t* positions, const float* inv_freq, const float* q_weight,
                   const float* k_weight, uint16_t* q_out, int64_t ldq_out, uint16_t* k_out,
                   int64_t ldk_out, int64_t rows, int32_t n_q_heads, int32_t n_kv_heads,
                   int32_t head_dim, float eps, ds_stream_t stream) {
  int64_t wq = 0, wk = 0;
  int st = check_qk(rows, n_q_heads, n_kv_heads, head_dim, eps, &wq, &wk);
  if (st != DS_OK || rows == 0 || wq + wk == 0) return st;
  if (positions == nullptr || inv_freq == nullptr) return DS_ERR_NULL;
  const View v[4] = {{q, ldq, wq, false}, {k, ldk, wk, false}, {q_out, ldq_out, wq, true},
                     {k_out, ldk_out, wk, true}};
  const int in_place[2][2] = {{2, 0}, {3, 1}};
  const void* const vecs[4] = {positions, inv_freq, q_weight, k_weight};
  const size_t nb[4] = {(size_t)rows * 4, (size_t)head_dim * 2, (size_t)head_dim * 4,
                        (size_t)head_dim * 4};
  if (!aligned(positions, 4) || !aligned(inv_freq, 16) || !aligned(q_weight, 16) ||
      !aligned(k_weight, 16))
    return DS_ERR_ALIGN;
  if ((st = check_views(v, rows, in_place, 2, vecs, nb, 4)) != DS_OK) return st;
  int cus = 0;
  if ((st = device_cus(&cus)) != DS_OK) return st;
  (void)hipGetLastError();
  const int rpg = dsr::kQkRmsRows;
  return launch_status(launch_in_pieces(rows, rpg, cus, [&](int64_t r0, int64_t n) {
    dsr::QkRmsArgs a{};
    a.x[0] = wq > 0 ? q + r0 * ldq : nullptr;
    a.x[1] = wk > 0 ? k + r0 * ldk : nullptr;
    a.y[0] = wq > 0 ? q_out + r0 * ldq_out : nullptr;
    a.y[1] = wk > 0 ? k_out + r0 * ldk_out : nullptr;
    a.w[0] = q_weight;
    a.w[1] = k_weight;
    a.pos = positions + r0;
    a.inv_freq = inv_freq;
    a.ldx[0] = ldq;
    a.ldx[1] = ldk;
    a.ldy[0] = ldq_out;
    a.ldy[1] = ldk_out;
    a.rows = n;
    a.nh[0] = n_q_heads;
    a.nh[1] = n_kv_heads;
    a.hd = head_dim;
    a.eps = eps;
    return dsr::launch_qk_rows_rms(a, (int)((n + rpg - 1) / rpg), (hipStream_t)stream);
  }));
}

int64_t ds_qk_rows_rms_backward_workspace(int64_t rows, int32_t n_q_heads, int32_t n_kv_heads,
                                          int32_t head_dim) {
  int64_t wq = 0, wk = 0;
  int st = check_qk(rows, n_q_heads, n_kv_heads, head_dim, 0.f, &wq, &wk);
  if (st != DS_OK) return st;
  if (wq + wk == 0) return 0;
  return (int64_t)dsr::qk_rms_backward_groups(rows) * 2 * head_dim * 4;
}

int ds_qk_rows_rms_backward(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk,
                            const int32_t* positions, const float* inv_freq,
                            const float* q_weight, const float* k_weight, const uint16_t* dq_out,
                            int64_t lddq_out, const uint16_t* dk_out, int64_t lddk_out,
                            uint16_t* dq, int64_t lddq, uint16_t* dk, int64_t lddk,
                            float* dq_weight, float* dk_weight, int64_t rows, int32_t n_q_heads,
                            int32_t n_kv_heads, int32_t head_dim, float eps, void* workspace,
                            int64_t workspace_bytes, ds_stream_t stream) {
  int64_t wq = 0, wk = 0;
  int st = check_qk(rows, n_q_heads, n_kv_heads, head_dim, eps, &wq, &wk);
  if (st != DS_OK) return st;
  const bool work = rows > 0 && wq + wk > 0, weights = dq_weight != nullptr || dk_weight != nullptr;
  if (!work && !weights) return DS_OK;
  if (work && (positions == nullptr || inv_freq == nullptr)) return DS_ERR_NULL;
  if (!aligned(positions, 4) || !aligned(inv_freq, 16) || !aligned(q_weight, 16) ||
      !aligned(k_weight, 16) || !aligned(dq_weight, 4) || !aligned(dk_weight, 4))
    return DS_ERR_ALIGN;
  const int64_t need =
      work && weights ? ds_qk_rows_rms_backward_workspace(rows, n_q_heads, n_kv_heads, head_dim) : 0;
  const size_t wb = (size_t)head_dim * 4;
  if (dq_weight != nullptr && dk_weight != nullptr && overlaps(dq_weight, wb, dk_weight, wb))
    return DS_ERR_ARG;
  if (work) {
    const View v[6] = {{q, ldq, wq, false},          {k, ldk, wk, false},
                       {dq_out, lddq_out, wq, false}, {dk_out, lddk_out, wk, false},
                       {dq, lddq, wq, true},          {dk, lddk, wk, true}};
    const int in_place[4][2] = {{4, 0}, {4, 2}, {5, 1}, {5, 3}};
    const void* const vecs[7] = {positions, inv_freq,  q_weight, k_weight,
                                 dq_weight, dk_weight, workspace};
    const size_t nb[7] = {(size_t)rows * 4, (size_t)head_dim * 2, wb, wb, wb, wb, (size_t)need};
    if ((st = check_views(v, rows, in_place, 4, vecs, nb, 7)) != DS_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, need)) != DS_OK) return st;
    // the weight gradients and the workspace against everything that is read
    const void* outs[3] = {dq_weight, dk_weight, workspace};
    const size_t on[3] = {wb, wb, (size_t)need};
    for (int i = 0; i < 3; ++i) {
      if (outs[i] == nullptr) continue;
      for (int j = 0; j < 4; ++j)
        if (vecs[j] != nullptr && overlaps(outs[i], on[i], vecs[j], nb[j])) return DS_ERR_ARG;
      for (int j = 0; j < 4; ++j)
        if (v[j].width > 0 && overlaps(outs[i], on[i], v[j].p, span_bytes(rows, v[j].ld, v[j].width)))
          return DS_ERR_ARG;
      for (int j = 0; j < i; ++j)
        if (outs[j] != nullptr && overlaps(outs[i], on[i], outs[j], on[j])) return DS_ERR_ARG;
    }
  }
  int cus = 0;
  if ((st = device_cus(&cus)) != DS_OK) return st;
  (void)hipGetLastError();
  int groups = 0;
  if (work) {
    dsr::QkRmsArgs a{};
    a.x[0] = q;
    a.x[1] = k;
    a.dy[0] = dq_out;
    a.dy[1] = dk_out;
    a.y[0] = dq;
    a.y[1] = dk;
    a.w[0] = q_weight;
    a.w[1] = k_weight;
    a.pos = positions;
    a.inv_freq = inv_freq;
    a.dw_part = weights ? static_cast<float*>(workspace) : nullptr;
    a.ldx[0] = ldq;
    a.ldx[1] = ldk;
    a.lddy[0] = lddq_out;
    a.lddy[1] = lddk_out;
    a.ldy[0] = lddq;
    a.ldy[1] = lddk;
    a.rows = rows;
    a.nh[0] = n_q_heads;
    a.nh[1] = n_kv_heads;
    a.hd = head_dim;
    a.eps = eps;
    groups = dsr::qk_rms_backward_groups(rows);
    st = launch_status(dsr::launch_qk_rows_rms_backward(a, groups, (hipStream_t)stream));
    if (st != DS_OK) return st;
  }
  if (!weights) return DS_OK;
  return launch_status(dsr::launch_qk_rms_weight_sum(static_cast<const float*>(workspace), groups,
                                                     head_dim, dq_weight, dk_weight,
                                                     (hipStream_t)stream));
}

}  // extern "C"

namespace {

int check_logits(int32_t type, int64_t ld, float inv_temp, int32_t label_bytes, int64_t rows,
                 int64_t vocab) {
  if (rows < 0 || vocab < 1 || vocab > DS_MAX_VOCAB || ld < vocab) return DS_ERR_SHAPE;
  if (rows > kMostBytes / 4 / ld) return DS_ERR_SHAPE;
  if (!type_ok(type) || !id_bytes_ok(label_bytes)) return DS_ERR_ARG;
  if (!std::isfinite(inv_temp) || inv_temp <= 0.f) return DS_ERR_ARG;
  return DS_OK;
}

// Bytes that [rows, vocab] logits of row stride ld span.
size_t logits_span(int32_t type, int64_t rows, int64_t ld, int64_t vocab) {
  return rows == 0 ? 0 : ((size_t)(rows - 1) * (size_t)ld + (size_t)vocab) * (size_t)type_bytes(type);
}

}  // namespace

extern "C" {

int64_t ds_logprob_rows_workspace(int64_t rows, int64_t vocab, int32_t top_k) {
  int st = check_logits(DS_TYPE_F32, vocab, 1.f, 8, rows, vocab);
  if (st != DS_OK) return st;
  if (top_k < 0 || top_k > DS_MAX_TOP || top_k > vocab) return DS_ERR_SHAPE;
  return dsr::logprob_workspace(rows, vocab, top_k);
}

int ds_logprob_rows(const void* logits, int32_t logits_type, int64_t ld, const float* scale,
                    float inv_temp, const void* labels, int32_t label_bytes, float* logp,
                    float* entropy, float* lse, int32_t* top_ids, float* top_logp, int32_t top_k,
                    int64_t rows, int64_t vocab, void* workspace, int64_t workspace_bytes,
                    ds_stream_t stream) {
  int st = check_logits(logits_type, ld, inv_temp, label_bytes, rows, vocab);
  if (st != DS_OK) return st;
  if (top_k < 0 || top_k > DS_MAX_TOP || top_k > vocab) return DS_ERR_SHAPE;
  if (rows == 0) return DS_OK;
  if (logits == nullptr || (logp != nullptr && labels == nullptr) ||
      (top_k > 0 && (top_ids == nullptr || top_logp == nullptr)))
    return DS_ERR_NULL;
  if (!aligned(logits, (uintptr_t)type_bytes(logits_type)) || !aligned(scale, 4) ||
      !aligned(labels, (uintptr_t)label_bytes) || !aligned(logp, 4) || !aligned(entropy, 4) ||
      !aligned(lse, 4) || !aligned(top_ids, 4) || !aligned(top_logp, 4))
    return DS_ERR_ALIGN;
  const int64_t need = ds_logprob_rows_workspace(rows, vocab, top_k);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != DS_OK) return st;
  const size_t rb = (size_t)rows * 4, tb = rb * (size_t)top_k;
  const Buf outs[6] = {{logp, rb}, {entropy, rb}, {lse, rb}, {top_ids, tb}, {top_logp, tb},
                       {workspace, (size_t)need}};
  const Buf ins[3] = {{logits, logits_span(logits_type, rows, ld, vocab)},
                      {scale, (size_t)vocab * 4},
                      {labels, (size_t)rows * (size_t)label_bytes}};
  if (!apart(outs, ins)) return DS_ERR_ARG;
  int cus = 0;
  if ((st = device_cus(&cus)) != DS_OK) return st;
  dsr::LogprobArgs a{};
  a.x = logits;
  a.scale = scale;
  a.labels = labels;
  a.logp = logp;
  a.entropy = entropy;
  a.lse = lse;
  a.top_ids = top_ids;
  a.top_logp = top_logp;
  a.ld = ld;
  a.rows = rows;
  a.vocab = (int32_t)vocab;
  a.top_k = top_k;
  a.label_bytes = label_bytes;
  a.inv_temp = inv_temp;
  (void)hipGetLastError();
  return launch_status(dsr::launch_logprob_rows(logits_type == DS_TYPE_F32, a, workspace,
                                                (hipStream_t)stream));
}

int64_t ds_logprob_rows_backward_workspace(int64_t rows, int64_t vocab) {
  int st = check_logits(DS_TYPE_F32, vocab, 1.f, 8, rows, vocab);
  if (st != DS_OK) return st;
  return dsr::logprob_grad_workspace(rows, vocab);
}

int ds_logprob_rows_backward(const void* logits, int32_t logits_type, int64_t ld,
                             const float* scale, float inv_temp, const void* labels,
                             int32_t label_bytes, const float* lse, const float* entropy,
                             const float* dlogp, const float* dentropy, void* dlogits,
                             int64_t ld_out, float* dscale, int64_t rows, int64_t vocab,
                             void* workspace, int64_t workspace_bytes, ds_stream_t stream) {
  int st = check_logits(logits_type, ld, inv_temp, label_bytes, rows, vocab);
  if (st != DS_OK) return st;
  if (ld_out < vocab || rows > kMostBytes / 4 / ld_out) return DS_ERR_SHAPE;
  if (dscale != nullptr && scale == nullptr) return DS_ERR_ARG;
  if (rows == 0 && dscale == nullptr) return DS_OK;
  if (rows > 0 && (logits == nullptr || dlogits == nullptr || lse == nullptr ||
                   (dlogp != nullptr && labels == nullptr) ||
                   (dentropy != nullptr && entropy == nullptr)))
    return DS_ERR_NULL;
  const uintptr_t ta = (uintptr_t)type_bytes(logits_type);
  if (!aligned(logits, ta) || !aligned(dlogits, ta) || !aligned(scale, 4) ||
      !aligned(labels, (uintptr_t)label_bytes) || !aligned(lse, 4) || !aligned(entropy, 4) ||
      !aligned(dlogp, 4) || !aligned(dentropy, 4) || !aligned(dscale, 4))
    return DS_ERR_ALIGN;
  const int64_t need = dscale != nullptr ? ds_logprob_rows_backward_workspace(rows, vocab) : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != DS_OK) return st;
  const size_t rb = (size_t)rows * 4;
  const bool in_place = dlogits == logits && ld_out == ld;
  const Buf outs[3] = {{dlogits, logits_span(logits_type, rows, ld_out, vocab)},
                       {dscale, (size_t)vocab * 4},
                       {workspace, (size_t)need}};
  const Buf ins[7] = {{in_place ? nullptr : logits, logits_span(logits_type, rows, ld, vocab)},
                      {scale, (size_t)vocab * 4},
                      {labels, (size_t)rows * (size_t)label_bytes},
                      {lse, rb}, {entropy, rb}, {dlogp, rb}, {dentropy, rb}};
  if (!apart(outs, ins)) return DS_ERR_ARG;
  int cus = 0;
  if ((st = device_cus(&cus)) != DS_OK) return st;
  dsr::LogprobGradArgs a{};
  a.x = logits;
  a.scale = scale;
  a.labels = labels;
  a.lse = lse;
  a.entropy = entropy;
  a.dlogp = dlogp;
  a.dentropy = dentropy;
  a.dx = dlogits;
  a.dscale = dscale;
  a.ld = ld;
  a.ldo = ld_out;
  a.rows = rows;
  a.vocab = (int32_t)vocab;
  a.label_bytes = label_bytes;
  a.inv_temp = inv_temp;
  (void)hipGetLastError();
  return launch_status(dsr::launch_logprob_rows_backward(logits_type == DS_TYPE_F32, a, workspace,
                                                         (hipStream_t)stream));
}

}  // extern "C"
