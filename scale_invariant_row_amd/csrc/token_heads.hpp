// A head of q or k spread over LPH lanes, 16 values a lane, with 64 / LPH heads
// going through a wave at a time: sums over a head, angles, the RMS factor.
#pragma once

#include "row_kernels.hpp"

namespace dsr {

constexpr int kQkRmsOut = 0x7ffffff0;      // an offset past every buffer

// Sum and maximum over the LPH lanes of a head.
template <int LPH>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (LPH >= 2) v = v + dpp_f<0xB1>(v);
  if constexpr (LPH >= 4) v = v + dpp_f<0x4E>(v);
  if constexpr (LPH >= 8) v = v + dpp_f<0x141>(v);
  if constexpr (LPH >= 16) v = v + dpp_f<0x140>(v);
  return v;
}

template <int LPH>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (LPH >= 2) v = fmaxf(v, dpp_f<0xB1>(v));
  if constexpr (LPH >= 4) v = fmaxf(v, dpp_f<0x4E>(v));
  if constexpr (LPH >= 8) v = fmaxf(v, dpp_f<0x141>(v));
  if constexpr (LPH >= 16) v = fmaxf(v, dpp_f<0x140>(v));
  return v;
}

// Sum over the lanes at the same place of the wave's 64 / LPH heads: rotations
// within 16 lanes, then the swaps across them.
template <int LPH>
__device__ __forceinline__ float heads_sum(float v) {
  if constexpr (LPH <= 1) v = v + dpp_f<0x121>(v);       // row_ror:1
  if constexpr (LPH <= 2) v = v + dpp_f<0x122>(v);
  if constexpr (LPH <= 4) v = v + dpp_f<0x124>(v);
  if constexpr (LPH <= 8) v = v + dpp_f<0x128>(v);
  f32x2_t p = swap16(v);
  p = swap32(p.x + p.y);
  return p.x + p.y;
}

__device__ __forceinline__ void unpack8(u32x4_t t, float* v) {
  v[0] = bf_lo(t.x); v[1] = bf_hi(t.x); v[2] = bf_lo(t.y); v[3] = bf_hi(t.y);
  v[4] = bf_lo(t.z); v[5] = bf_hi(t.z); v[6] = bf_lo(t.w); v[7] = bf_hi(t.w);
}

__device__ __forceinline__ u32x4_t pack8(const float* v) {
  return u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                 pack_bf16(v[6], v[7])};
}

// Eight weights at w + at, or ones.
__device__ __forceinline__ void load_weights(const float* w, int at, bool active, float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = w != nullptr && active ? w[at + j] : 1.f;
}

// A row's position, through the scalar cache: a vector load would have to
// wait for every head asked for before it.  (Positions are only read here.)
__device__ __forceinline__ int32_t position(const int32_t* pos, int64_t row) {
  return *(const __attribute__((address_space(4))) int32_t*)(pos + row);
}

// The frequencies whose angles this lane evaluates: lane and 64 + lane.
__device__ __forceinline__ void load_frequencies(float (&f)[2], const float* inv_freq, int half,
                                                 int lane) {
  f[0] = lane < half ? inv_freq[lane] : 0.f;
  f[1] = 64 + lane < half ? inv_freq[64 + lane] : 0.f;
}

// cos then sin of the row's angles into the wave's own piece of LDS.  LDS
// operations of one wave run in order, so no barrier is needed; the fences
// keep the compiler from moving accesses across.  Nothing here waits for
// memory, so heads that were asked for before stay on their way.
__device__ __forceinline__ void fill_angles(float (&cs)[2][128], int32_t p, const float (&f)[2],
                                            int half, int lane) {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = 64 * k + lane;
    if (64 * k >= half) break;                             // uniform
    double turn = (double)p * (double)f[k] * 0.15915494309189534;
    turn -= rint(turn);
    float s, c;
    sincospif(2.f * (float)turn, &s, &c);
    if (i < half) {
      cs[0][i] = c;
      cs[1][i] = s;
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ void read_angles(const float (&cs)[2][128], int at, bool active,
                                            float* c, float* s) {
  const int i = active ? at : 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c[j] = cs[0][i + j];
    s[j] = cs[1][i + j];
  }
}

// inv = 1 / sqrt(sum / hd + eps) of the head held as v[16] by its LPH lanes.
// Where the sum overflows, or the mean plus eps is below 2^-96, v is scaled by
// 2^sh (exactly) and inv belongs to the scaled head; sh is 0 elsewhere.
template <int LPH>
__device__ __forceinline__ float head_inv_rms(float (&v)[16], float per_hd, float eps, int& sh) {
  float a0 = 0.f, a1 = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    a0 = __builtin_fmaf(v[j], v[j], a0);
    a1 = __builtin_fmaf(v[8 + j], v[8 + j], a1);
  }
  float T = lanes_sum<LPH>(a0 + a1) * per_hd + eps;
  sh = 0;
  const bool need = T == __builtin_inff() || T < kTiny;
  if (__builtin_amdgcn_ballot_w64(need) != 0) {      // any head of the wave
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(v[j]));
    m = lanes_max<LPH>(m);
    if (need && (m > 0.f || eps > 0.f) && m < __builtin_inff()) sh = rescue_shift(m, eps);
    a0 = a1 = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = ldexpf(v[j], sh);
      v[8 + j] = ldexpf(v[8 + j], sh);
      a0 = __builtin_fmaf(v[j], v[j], a0);
      a1 = __builtin_fmaf(v[8 + j], v[8 + j], a1);
    }
    const float T2 = lanes_sum<LPH>(a0 + a1) * per_hd + ldexpf(eps, 2 * sh);
    if (sh != 0) T = T2;
  }
  return inv_sqrt(T);
}

}  // namespace dsr
