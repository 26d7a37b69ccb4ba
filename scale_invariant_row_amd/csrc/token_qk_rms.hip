// q/k heads: RMS norm with a learned weight, then rotate-half RoPE, and the
// gradient.
//
//   u = x / D, D = sqrt(sum x^2 / HD + eps);  n = u w
//   y = [n1 cos t - n2 sin t, n2 cos t + n1 sin t],  t_i = p inv_freq_i
// and, with d = [dy1 cos t + dy2 sin t, dy2 cos t - dy1 sin t] (dy turned back):
//   dw += d u,   dx = (w d - u <w d, u> / HD) / D
//
// A head spreads over LPH lanes (the power of two at or above HD / 16).  A
// lane holds 8 values of the head's first half and the 8 they rotate with, so
// the rotation needs no exchange between lanes and both loads are 16 bytes;
// 64 / LPH heads go through the wave at a time.  Lanes past the head (a
// head_dim that is no power of two) have their offsets out of the buffer's
// range: loads return 0 and stores are dropped.
//
// Angles: the wave evaluates each of its row's HD/2 angles once and shares
// them through LDS.  The turn p inv_freq / 2 pi is formed and reduced to
// [-1/2, 1/2] in fp64 (exact to 1e-7 turns for any int32 position), its sine
// and cosine in fp32.
#include "token_heads.hpp"
#include "token_launch.hpp"

namespace dsr {

// One wave per row.  CH wave steps of q are loaded before the angles are
// evaluated, then CH at a time.  Bound by memory: 8,192 rows of 16 + 4 heads
// of 256 in 33 us (5.1 TB/s); 39.8 with one step at a time, 35.8 with two or
// three.
template <int LPH>
__global__ void __launch_bounds__(256) qk_rows_rms_kernel(const QkRmsArgs a) {
  constexpr int HPW = 64 / LPH, CH = 4;
  __shared__ __attribute__((aligned(16))) float trig[kQkRmsRows][2][128];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = (int64_t)blockIdx.x * kQkRmsRows + wave;
  if (row >= a.rows) return;
  const int half = a.hd / 2;
  const int at = (lane % LPH) * 8;
  const int hs = lane / LPH;
  const bool active = at < half;
  const float per_hd = 1.f / (float)a.hd;
  const uint32_t head_bytes = (uint32_t)a.hd * 2u;
  const int lane_lo = hs * (int)head_bytes + at * 2;       // of the lane's head in a wave step
  auto offset = [&](int h0) { return active ? h0 * (int)head_bytes + lane_lo : kQkRmsOut; };
  u32x4_t x[CH][2];
  auto load = [&](const RowBuf& ib, int h0) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int lo = offset(h0 + i * HPW);                 // past the last head: loads 0
      x[i][0] = ib.ld16(lo);
      x[i][1] = ib.ld16(active ? lo + a.hd : kQkRmsOut);
    }
  };
  float f[2];
  load_frequencies(f, a.inv_freq, half, lane);             // first: loads return in order
  const RowBuf qb(a.x[0] + row * a.ldx[0], (uint32_t)a.nh[0] * head_bytes);
  load(qb, 0);
  fill_angles(trig[wave], position(a.pos, row), f, half, lane);
  float c[8], s[8];
  read_angles(trig[wave], at, active, c, s);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const int nh = a.nh[which];
    if (nh == 0) continue;
    float w[16];
    load_weights(a.w[which], at, active, w);
    load_weights(a.w[which], half + at, active, w + 8);
    const RowBuf ib(a.x[which] + row * a.ldx[which], (uint32_t)nh * head_bytes);
    const RowBuf ob(a.y[which] + row * a.ldy[which], (uint32_t)nh * head_bytes);
    for (int h0 = 0; h0 < nh; h0 += CH * HPW) {
      if (which > 0 || h0 > 0) load(ib, h0);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (h0 + i * HPW >= nh) break;                     // uniform
        float v[16], y[16];
        unpack8(x[i][0], v);
        unpack8(x[i][1], v + 8);
        int sh;
        const float inv = head_inv_rms<LPH>(v, per_hd, a.eps, sh);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float n1 = v[j] * inv * w[j], n2 = v[8 + j] * inv * w[8 + j];
          y[j] = n1 * c[j] - n2 * s[j];
          y[8 + j] = n2 * c[j] + n1 * s[j];
        }
        const int lo = offset(h0 + i * HPW);
        ob.st16(pack8(y), lo);
        ob.st16(pack8(y + 8), active ? lo + a.hd : kQkRmsOut);
      }
    }
  }
}

// The gradient: the workgroup's four waves walk the rows, each lane summing
// the weight gradients of its 16 head dimensions over the heads it meets; the
// workgroup writes one partial sum per dimension.  The number of workgroups,
// and with it the order of those sums, depends on the row count alone.  The
// next wave step's heads, the next row's first among them, are loaded before
// the present ones are worked on.  16,384 rows of 32 + 8 heads of 128 in 95 us
// (5.3 TB/s), bound by memory and, at some 500 instructions a wave step (a
// third of them the unpacking and the turn back), nearly by the ALUs: 98 us at
// three waves a SIMD, 101 without loading ahead.
template <int LPH>
__global__ void __launch_bounds__(256, 4) qk_rows_rms_backward_kernel(const QkRmsArgs a) {
  constexpr int HPW = 64 / LPH;
  __shared__ __attribute__((aligned(16))) float trig[4][2][128];
  __shared__ float part[4][2][256];
  __shared__ __attribute__((aligned(16))) float weight[2][256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = a.hd / 2;
  const int at = (lane % LPH) * 8;
  const int hs = lane / LPH;
  const bool active = at < half;
  const float per_hd = 1.f / (float)a.hd;
  const uint32_t head_bytes = (uint32_t)a.hd * 2u;
  const int lane_lo = hs * (int)head_bytes + at * 2;       // of the lane's head in a wave step
  for (int i = threadIdx.x; i < 2 * a.hd; i += 256) {
    const int which = i >= a.hd;
    const float* w = a.w[which];
    weight[which][i - which * a.hd] = w != nullptr ? w[i - which * a.hd] : 1.f;
  }
  __syncthreads();
  const int own = active ? at : 0;                         // idle lanes read what they do not use
  float dw[2][16] = {};
  u32x4_t next[4];                                         // x and dy, both halves
  // one place in the code loads (each has its own registers to move from,
  // and moving waits); a row past the end is a buffer of no bytes
  auto load = [&](int64_t row, int which, int h0) {
    const int64_t r = row < a.rows ? row : 0;
    const uint32_t bytes = row < a.rows ? (uint32_t)(which ? a.nh[1] : a.nh[0]) * head_bytes : 0u;
    const RowBuf xb((which ? a.x[1] : a.x[0]) + r * (which ? a.ldx[1] : a.ldx[0]), bytes);
    const RowBuf gb((which ? a.dy[1] : a.dy[0]) + r * (which ? a.lddy[1] : a.lddy[0]), bytes);
    const int lo = active ? h0 * (int)head_bytes + lane_lo : kQkRmsOut;
    const int hi = active ? lo + a.hd : kQkRmsOut;
    next[0] = xb.ld16(lo);
    next[1] = xb.ld16(hi);
    next[2] = gb.ld16(lo);
    next[3] = gb.ld16(hi);
  };
  const int64_t stride = (int64_t)gridDim.x * 4;
  const int start = a.nh[0] > 0 ? 0 : 1;                   // which heads a row begins with
  float f[2];
  load_frequencies(f, a.inv_freq, half, lane);
  int64_t row = (int64_t)blockIdx.x * 4 + wave;
  load(row, start, 0);
  for (; row < a.rows; row += stride) {
    fill_angles(trig[wave], position(a.pos, row), f, half, lane);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const int nh = a.nh[which];
      const RowBuf ob(a.y[which] + row * a.ldy[which], (uint32_t)nh * head_bytes);
      for (int h0 = 0; h0 < nh; h0 += HPW) {
        // angles and weights come from LDS in every step: held, they take
        // the registers that keep a fourth wave on the SIMD
        asm volatile("" ::: "memory");
        float v[16], g[16];
        unpack8(next[0], v);
        unpack8(next[1], v + 8);
        unpack8(next[2], g);
        unpack8(next[3], g + 8);
        const bool more = h0 + HPW < nh, to_k = which == 0 && a.nh[1] > 0;
        load(more || to_k ? row : row + stride, more ? which : to_k ? 1 : start, more ? h0 + HPW : 0);
        int sh;
        float inv = head_inv_rms<LPH>(v, per_hd, a.eps, sh);
        if (h0 + hs >= nh) inv = 0.f;                      // no head here: u = 0
        float a0 = 0.f, a1 = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float cj = trig[wave][0][own + j], sj = trig[wave][1][own + j];
          const float d1 = g[j] * cj + g[8 + j] * sj;
          const float d2 = g[8 + j] * cj - g[j] * sj;
          v[j] *= inv;                                     // u
          v[8 + j] *= inv;
          dw[which][j] = __builtin_fmaf(d1, v[j], dw[which][j]);
          dw[which][8 + j] = __builtin_fmaf(d2, v[8 + j], dw[which][8 + j]);
          g[j] = d1 * weight[which][own + j];
          g[8 + j] = d2 * weight[which][half + own + j];
          a0 = __builtin_fmaf(g[j], v[j], a0);
          a1 = __builtin_fmaf(g[8 + j], v[8 + j], a1);
        }
        const float m = -(lanes_sum<LPH>(a0 + a1) * per_hd);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __builtin_fmaf(v[j], m, g[j]) * inv;
        if (__builtin_amdgcn_ballot_w64(sh != 0) != 0) {   // D was that of the head times 2^sh
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = ldexpf(v[j], sh);
        }
        const int lo = active ? h0 * (int)head_bytes + lane_lo : kQkRmsOut;
        ob.st16(pack8(v), lo);
        ob.st16(pack8(v + 8), active ? lo + a.hd : kQkRmsOut);
      }
    }
  }
  if (a.dw_part == nullptr) return;
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float t = heads_sum<LPH>(dw[which][j]);       // over the heads of the wave step
      if (hs == 0 && active) part[wave][which][(j < 8 ? 0 : half) + at + j % 8] = t;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.hd; i += 256) {
    const int which = i / a.hd, j = i % a.hd;
    a.dw_part[(int64_t)blockIdx.x * 2 * a.hd + i] =
        ((part[0][which][j] + part[1][which][j]) + part[2][which][j]) + part[3][which][j];
  }
}

// Sums the workgroups' partial weight gradients: 16 dimensions a workgroup,
// 64 threads for each, thread k adding parts k, k + 64, ... and the 64 sums
// added in order.  (One thread a dimension, adding 1,024 parts, took 219 us.)
__global__ void __launch_bounds__(1024) qk_rms_weight_sum_kernel(const float* part, int groups,
                                                                 int hd, float* dqw, float* dkw) {
  __shared__ float sums[64][17];
  const int col = threadIdx.x & 15, k = threadIdx.x >> 4;
  const int i = blockIdx.x * 16 + col;                   // 2 hd is a multiple of 16
  float t = 0.f;
#pragma unroll 8
  for (int g = k; g < groups; g += 64) t += part[(int64_t)g * 2 * hd + i];
  sums[k][col] = t;
  __syncthreads();
  if (threadIdx.x >= 16) return;
  t = 0.f;
  for (int j = 0; j < 64; ++j) t += sums[j][col];
  float* out = i < hd ? dqw : dkw;
  if (out != nullptr) out[i < hd ? i : i - hd] = t;
}

int qk_rms_backward_groups(int64_t rows) {
  const int64_t g = (rows + 3) / 4;
  return (int)(g < 1024 ? g : 1024);
}

static int lanes_per_head(int hd) {
  int n = 1;
  while (n * 16 < hd) n *= 2;
  return n;
}

hipError_t launch_qk_rows_rms(const QkRmsArgs& a, int grid, hipStream_t stream) {
  switch (lanes_per_head(a.hd)) {
    case 1: qk_rows_rms_kernel<1><<<grid, 256, 0, stream>>>(a); break;
    case 2: qk_rows_rms_kernel<2><<<grid, 256, 0, stream>>>(a); break;
    case 4: qk_rows_rms_kernel<4><<<grid, 256, 0, stream>>>(a); break;
    case 8: qk_rows_rms_kernel<8><<<grid, 256, 0, stream>>>(a); break;
    case 16: qk_rows_rms_kernel<16><<<grid, 256, 0, stream>>>(a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_qk_rows_rms_backward(const QkRmsArgs& a, int grid, hipStream_t stream) {
  switch (lanes_per_head(a.hd)) {
    case 1: qk_rows_rms_backward_kernel<1><<<grid, 256, 0, stream>>>(a); break;
    case 2: qk_rows_rms_backward_kernel<2><<<grid, 256, 0, stream>>>(a); break;
    case 4: qk_rows_rms_backward_kernel<4><<<grid, 256, 0, stream>>>(a); break;
    case 8: qk_rows_rms_backward_kernel<8><<<grid, 256, 0, stream>>>(a); break;
    case 16: qk_rows_rms_backward_kernel<16><<<grid, 256, 0, stream>>>(a); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_qk_rms_weight_sum(const float* part, int groups, int hd, float* dqw, float* dkw,
                                    hipStream_t stream) {
  qk_rms_weight_sum_kernel<<<2 * hd / 16, 1024, 0, stream>>>(part, groups, hd, dqw, dkw);
  return hipGetLastError();
}

}  // namespace dsr
