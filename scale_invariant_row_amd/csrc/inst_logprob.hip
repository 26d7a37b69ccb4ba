// Rows of logits: log probability of a given token, entropy, top alternatives,
// and the gradient.
//
//   z_j = (x_j scale_j) inv_temp;  lse = log sum exp z;  logp = z_label - lse
//   entropy = lse - sum p z = log S - T / S  with  M = max z,
//             S = sum exp(z - M),  T = sum exp(z - M) (z - M)
//
// The row is cut into chunks of kLpChunk columns.  A chunk's (M, S, T) comes
// from its own maximum; the chunks are joined left to right (lp_join), so the
// row's bits depend on the row and its width alone.
//
// exp(-inf) = 0 lets a masked token (z = -inf) drop out of S; in T it would
// be 0 * inf, so the factor z - M is clamped at -200, where exp is 0 already.
#include "row_kernels.hpp"
#include "token_launch.hpp"

namespace dsr {

constexpr int kLpThreads = 256;
constexpr int kLpPer = 32;                            // columns per thread of a chunk
constexpr int kLpChunk = kLpThreads * kLpPer;         // 8,192
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float lp_exp(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

template <bool F32>
__device__ __forceinline__ float lp_load(const void* x, int64_t i) {
  if constexpr (F32) return static_cast<const float*>(x)[i];
  else return __uint_as_float((uint32_t) static_cast<const uint16_t*>(x)[i] << 16);
}

__device__ __forceinline__ float lp_z(float x, const float* scale, int col, float inv_temp) {
  if (scale != nullptr) x = x * scale[col];
  return x * inv_temp;
}

// Label of a row, or -1 for a row to ignore.
__device__ __forceinline__ int lp_label(const void* labels, int label_bytes, int64_t row, int vocab) {
  if (labels == nullptr) return -1;
  const int64_t y = label_bytes == 8 ? static_cast<const int64_t*>(labels)[row]
                                     : (int64_t) static_cast<const int32_t*>(labels)[row];
  return y >= 0 && y < vocab ? (int)y : -1;
}

struct LpSum {
  float M, S, T;
};

// Joins the sums of a stretch with those of the stretch to its right.  With
// every token masked so far, M is -inf and S, T are 0.
__device__ __forceinline__ LpSum lp_join(LpSum a, LpSum b) {
  const float M = fmaxf(a.M, b.M);
  const float base = M == -__builtin_inff() ? 0.f : M;
  const float da = a.M - base, db = b.M - base;
  const float ea = lp_exp(da), eb = lp_exp(db);
  LpSum r;
  r.M = M;
  r.S = a.S * ea + b.S * eb;
  r.T = ea * (a.T + a.S * fmaxf(da, -200.f)) + eb * (b.T + b.S * fmaxf(db, -200.f));
  return r;
}

// A key that orders tokens: larger z first, then the lower column.  0 for a
// token that cannot be listed (masked, or NaN).
__device__ __forceinline__ uint64_t lp_key(float z, int col) {
  if (!(z > -__builtin_inff())) return 0;
  const uint32_t u = __float_as_uint(z + 0.f);        // -0 orders as 0
  const uint32_t k = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return ((uint64_t)k << 32) | (uint32_t)~(uint32_t)col;
}

__device__ __forceinline__ float lp_key_z(uint64_t key) {
  const uint32_t k = (uint32_t)(key >> 32);
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ uint64_t lp_wave_max(uint64_t v) {
  for (int d = 1; d < 64; d *= 2) {
    const uint64_t o = __shfl_xor((unsigned long long)v, d);
    v = o > v ? o : v;
  }
  return v;
}

template <bool F32>
__global__ void __launch_bounds__(kLpThreads) logprob_rows_kernel(const LogprobArgs a) {
  __shared__ float red[4][2];
  __shared__ uint64_t kred[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = blockIdx.x;
  const int64_t at = row * a.ld;
  LpSum sum = {-__builtin_inff(), 0.f, 0.f};
  for (int c0 = 0; c0 < a.vocab; c0 += kLpChunk) {
    float z[kLpPer];
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kLpPer; ++i) {
      const int col = c0 + i * kLpThreads + threadIdx.x;
      z[i] = col < a.vocab ? lp_z(lp_load<F32>(a.x, at + col), a.scale, col, a.inv_temp)
                           : -__builtin_inff();
      m = fmaxf(m, z[i]);
    }
    m = wave_max(m);
    __syncthreads();
    if (lane == 0) red[wave][0] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0]));
    const float base = m == -__builtin_inff() ? 0.f : m;
    float S = 0.f, T = 0.f;
#pragma unroll
    for (int i = 0; i < kLpPer; ++i) {
      const float d = z[i] - base, e = lp_exp(d);
      S += e;
      T = __builtin_fmaf(e, fmaxf(d, -200.f), T);
    }
    S = wave_sum(S);
    T = wave_sum(T);
    __syncthreads();
    if (lane == 0) {
      red[wave][0] = S;
      red[wave][1] = T;
    }
    __syncthreads();
    const LpSum c = {m, ((red[0][0] + red[1][0]) + red[2][0]) + red[3][0],
                     ((red[0][1] + red[1][1]) + red[2][1]) + red[3][1]};
    sum = lp_join(sum, c);
  }
  const bool empty = sum.M == -__builtin_inff() && sum.S == 0.f;
  const float log_s = logf(sum.S);
  const float lse = empty ? -__builtin_inff() : sum.M + log_s;
  if (threadIdx.x == 0) {
    if (a.lse != nullptr) a.lse[row] = lse;
    if (a.entropy != nullptr) a.entropy[row] = empty ? 0.f : log_s - sum.T / sum.S;
    if (a.logp != nullptr) {
      const int y = lp_label(a.labels, a.label_bytes, row, a.vocab);
      float lp = 0.f;
      if (y >= 0) {
        const float z = lp_z(lp_load<F32>(a.x, at + y), a.scale, y, a.inv_temp);
        lp = empty ? -__builtin_inff() : (z - sum.M) - log_s;
      }
      a.logp[row] = lp;
    }
  }
  // the top alternatives, one pass over the row for each: the largest key
  // below the last
  uint64_t last = ~0ull;
  for (int k = 0; k < a.top_k; ++k) {
    uint64_t best = 0;
    for (int col = threadIdx.x; col < a.vocab; col += kLpThreads) {
      const uint64_t key = lp_key(lp_z(lp_load<F32>(a.x, at + col), a.scale, col, a.inv_temp), col);
      if (key < last && key > best) best = key;
    }
    best = lp_wave_max(best);
    __syncthreads();
    if (lane == 0) kred[wave] = best;
    __syncthreads();
    for (int w = 0; w < 4; ++w) best = kred[w] > best ? kred[w] : best;
    last = best;
    if (threadIdx.x == 0) {
      a.top_ids[row * a.top_k + k] = best != 0 ? (int32_t)~(uint32_t)best : -1;
      a.top_logp[row * a.top_k + k] = best != 0 ? (lp_key_z(best) - sum.M) - log_s : -__builtin_inff();
    }
  }
}

hipError_t launch_logprob_rows(bool f32, const LogprobArgs& a, void* workspace,
                               hipStream_t stream) {
  (void)workspace;
  constexpr int64_t kMostRows = 1 << 20;               // rows per launch
  for (int64_t r0 = 0; r0 < a.rows; r0 += kMostRows) {
    LogprobArgs p = a;
    const int64_t n = a.rows - r0 < kMostRows ? a.rows - r0 : kMostRows;
    p.x = static_cast<const char*>(a.x) + r0 * a.ld * (f32 ? 4 : 2);
    if (a.labels != nullptr) p.labels = static_cast<const char*>(a.labels) + r0 * a.label_bytes;
    if (a.logp != nullptr) p.logp = a.logp + r0;
    if (a.entropy != nullptr) p.entropy = a.entropy + r0;
    if (a.lse != nullptr) p.lse = a.lse + r0;
    if (a.top_k > 0) {
      p.top_ids = a.top_ids + r0 * a.top_k;
      p.top_logp = a.top_logp + r0 * a.top_k;
    }
    if (f32) logprob_rows_kernel<true><<<(int)n, kLpThreads, 0, stream>>>(p);
    else logprob_rows_kernel<false><<<(int)n, kLpThreads, 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// What the gradient needs of a row.
struct LpRowGrad {
  float lse, ent, g, gh;       // g: dlogp (0 for an ignored row), gh: dentropy
  int label;
};

__device__ __forceinline__ LpRowGrad lp_row_grad(const LogprobGradArgs& a, int64_t row) {
  LpRowGrad r;
  r.label = lp_label(a.labels, a.label_bytes, row, a.vocab);
  r.lse = a.lse[row];
  r.ent = a.dentropy != nullptr ? a.entropy[row] : 0.f;
  r.g = a.dlogp != nullptr && r.label >= 0 ? a.dlogp[row] : 0.f;
  r.gh = a.dentropy != nullptr ? a.dentropy[row] : 0.f;
  return r;
}

// dz_j inv_temp; 0 for a masked token (and so for a row with all masked).
__device__ __forceinline__ float lp_dz(const LpRowGrad& r, float z, int col, float inv_temp) {
  const float lp = z - r.lse;
  const float p = lp_exp(lp);
  float d = r.gh * (lp + r.ent) + r.g;
  d = (col == r.label ? r.g : 0.f) - p * d;
  return z == -__builtin_inff() ? 0.f : d * inv_temp;
}

template <bool F32>
__global__ void __launch_bounds__(kLpThreads) logprob_grad_kernel(const LogprobGradArgs a) {
  const int64_t row = blockIdx.x;
  const LpRowGrad r = lp_row_grad(a, row);
  for (int col = threadIdx.x; col < a.vocab; col += kLpThreads) {
    const float z = lp_z(lp_load<F32>(a.x, row * a.ld + col), a.scale, col, a.inv_temp);
    float d = lp_dz(r, z, col, a.inv_temp);
    if (a.scale != nullptr) d = d * a.scale[col];
    if constexpr (F32) static_cast<float*>(a.dx)[row * a.ldo + col] = d;
    else static_cast<uint16_t*>(a.dx)[row * a.ldo + col] = (uint16_t)pack_bf16(d, 0.f);
  }
}

// The scale's gradient: one thread per column, down the rows.
template <bool F32>
__global__ void __launch_bounds__(64) logprob_scale_grad_kernel(const LogprobGradArgs a) {
  const int col = blockIdx.x * 64 + threadIdx.x;
  if (col >= a.vocab) return;
  float t = 0.f;
  for (int64_t row = 0; row < a.rows; ++row) {
    const LpRowGrad r = lp_row_grad(a, row);
    const float x = lp_load<F32>(a.x, row * a.ld + col);
    const float d = lp_dz(r, lp_z(x, a.scale, col, a.inv_temp), col, a.inv_temp);
    t += d != 0.f ? d * x : 0.f;
  }
  a.dscale[col] = t;
}

hipError_t launch_logprob_rows_backward(bool f32, const LogprobGradArgs& a, void* workspace,
                                        hipStream_t stream) {
  (void)workspace;
  // dscale first: dlogits may overwrite the logits
  if (a.dscale != nullptr) {
    const int grid = (a.vocab + 63) / 64;
    if (f32) logprob_scale_grad_kernel<true><<<grid, 64, 0, stream>>>(a);
    else logprob_scale_grad_kernel<false><<<grid, 64, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  constexpr int64_t kMostRows = 1 << 20;
  for (int64_t r0 = 0; r0 < a.rows; r0 += kMostRows) {
    LogprobGradArgs p = a;
    const int64_t n = a.rows - r0 < kMostRows ? a.rows - r0 : kMostRows;
    p.x = static_cast<const char*>(a.x) + r0 * a.ld * (f32 ? 4 : 2);
    p.dx = static_cast<char*>(a.dx) + r0 * a.ldo * (f32 ? 4 : 2);
    if (a.labels != nullptr) p.labels = static_cast<const char*>(a.labels) + r0 * a.label_bytes;
    p.lse = a.lse + r0;
    if (a.entropy != nullptr) p.entropy = a.entropy + r0;
    if (a.dlogp != nullptr) p.dlogp = a.dlogp + r0;
    if (a.dentropy != nullptr) p.dentropy = a.dentropy + r0;
    if (f32) logprob_grad_kernel<true><<<(int)n, kLpThreads, 0, stream>>>(p);
    else logprob_grad_kernel<false><<<(int)n, kLpThreads, 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace dsr
