// Host-side launchers of the token row kernels (one translation unit per op).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dsr {

struct EmbedArgs {
  const void* table;
  const void* ids;
  uint16_t* out;
  int64_t vocab;
  int64_t rows;
  int32_t cols;
  float scale;
};
hipError_t launch_embed_rows(bool f32, bool wide_ids, const EmbedArgs& a, int grid,
                             hipStream_t stream);

struct EmbedGradArgs {
  const uint16_t* dy;
  const void* ids;
  void* dtable;
  int32_t vocab;
  int32_t rows;
  int32_t cols;
  int32_t accumulate;
  float scale;
};
int64_t embed_grad_workspace(int64_t vocab, int64_t rows, int64_t cols);
hipError_t launch_embed_rows_backward(bool f32, bool wide_ids, const EmbedGradArgs& a,
                                      void* workspace, hipStream_t stream);

// [0] is q, [1] is k throughout.
struct QkRmsArgs {
  const uint16_t* x[2];
  uint16_t* y[2];               // the output (forward) or dx (backward)
  const uint16_t* dy[2];        // backward only
  const float* w[2];            // may be null: weights of 1
  const int32_t* pos;
  const float* inv_freq;
  float* dw_part;               // backward: [workgroups][2][head_dim], or null
  int64_t ldx[2], ldy[2], lddy[2];
  int64_t rows;
  int32_t nh[2];
  int32_t hd;
  float eps;
};
constexpr int kQkRmsRows = 4;   // rows per workgroup of the forward kernel
int qk_rms_backward_groups(int64_t rows);
hipError_t launch_qk_rows_rms(const QkRmsArgs& a, int grid, hipStream_t stream);
hipError_t launch_qk_rows_rms_backward(const QkRmsArgs& a, int grid, hipStream_t stream);
hipError_t launch_qk_rms_weight_sum(const float* part, int groups, int hd, float* dqw, float* dkw,
                                    hipStream_t stream);

struct LogprobArgs {
  const void* x;
  const float* scale;           // may be null
  const void* labels;           // may be null
  float* logp;
  float* entropy;
  float* lse;
  int32_t* top_ids;
  float* top_logp;
  int64_t ld;
  int64_t rows;
  int32_t vocab;
  int32_t top_k;
  int32_t label_bytes;
  float inv_temp;
};
int64_t logprob_workspace(int64_t rows, int64_t vocab, int top_k);
hipError_t launch_logprob_rows(bool f32, const LogprobArgs& a, void* workspace, hipStream_t stream);

struct LogprobGradArgs {
  const void* x;
  const float* scale;
  const void* labels;
  const float* lse;
  const float* entropy;
  const float* dlogp;
  const float* dentropy;
  void* dx;
  float* dscale;
  int64_t ld, ldo;
  int64_t rows;
  int32_t vocab;
  int32_t label_bytes;
  float inv_temp;
};
int64_t logprob_grad_workspace(int64_t rows, int64_t vocab);
hipError_t launch_logprob_rows_backward(bool f32, const LogprobGradArgs& a, void* workspace,
                                        hipStream_t stream);

}  // namespace dsr
