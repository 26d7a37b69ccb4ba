// Rotary positions on heads, and a step's keys and values into the paged cache.
//
//   t_i = p inv_freq_i;  (a, b) -> A (a cos t - b sin t, b cos t + a sin t)
// for the pairs (x_i, x_{i + R/2}) or (x_{2i}, x_{2i+1}) of a head's first R
// values.  Appending norms each head first, u = x / sqrt(sum x^2 / HD + eps) w,
// and stores bf16 or e4m3 values where the page table says.
//
// A head spreads over LPH lanes, two 16-byte vectors of 8 values a lane.  Which
// two goes by the pairing, so that as a rule a lane holds whole pairs:
//   halves, R a multiple of 16: vector u of the first R/2 values and the one
//     that turns with it; past R/16 lanes, of the two halves that only pass by
//   neighbours: vector u of the head's first half and of its second
//   halves, any other even R: the same two, and the partners come out of LDS (a
//     wave's heads, 4 KB)
// so loads and stores stay 16 bytes wide for every R, and neighbouring lanes
// touch neighbouring vectors (two vectors in a row a lane, every load and store
// taking half of each line, held 16,384 rows of 32 + 8 heads of 128 at 94 us).  A
// value that does not turn is never multiplied (an infinity beside it would make
// a NaN of it).
//
// Bound by memory: those rows (336 MB) take 57 us, 5.8 TB/s; 8,192 of 16 + 4 heads
// of 256 30.5 us, 5.5; 24 prompts of up to 1,021 tokens, 32 + 2 * 8 heads of 128,
// into a bf16 cache (315 MB) 53 us, 5.9; 16 + 2 * 4 heads of 256, normed, into
// e4m3 (288 MB) 54 us, 5.3.
#include "decode_launch.hpp"
#include "token_heads.hpp"

namespace dsr {

enum { kHalves = 0, kNeighbours = 1, kOddHalves = 2 };

// Where a lane's two vectors lie in its head, and whether they turn.
template <int LPH, int PAIRS>
struct Place {
  int u, a, b;                  // lane within the head; element offsets
  bool active, turns;           // has values; (halves) they turn
  __device__ __forceinline__ Place(int lane, int hd, int rotary) {
    u = lane % LPH;
    active = u * 16 < hd;
    a = 8 * u;
    b = hd / 2 + 8 * u;
    turns = true;
    if constexpr (PAIRS == kHalves) {
      turns = u * 16 < rotary;
      a = turns ? 8 * u : rotary / 2 + 8 * u;
      b = turns ? rotary / 2 + 8 * u : hd / 2 + 8 * u;
    }
  }
};

// cos then sin of the row's R/2 angles, times the amplitude, into the wave's
// own piece of LDS (no barrier: LDS operations of one wave run in order).
__device__ __forceinline__ void fill_turn(float (&cs)[2][128], int32_t p, const Turn& t, int lane) {
  const int half = t.rotary / 2;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = 64 * k + lane;
    if (64 * k >= half) break;                             // uniform
    if (i < half) {
      double turn = (double)p * (double)t.inv_freq[i] * 0.15915494309189534;
      turn -= rint(turn);
      float s, c;
      sincospif(2.f * (float)turn, &s, &c);
      cs[0][i] = c * t.amplitude;
      cs[1][i] = s * t.amplitude * t.sign;
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The angles of a lane's 8 pairs (kOddHalves reads them one by one).
template <int LPH, int PAIRS>
__device__ __forceinline__ void lane_angles(const float (&cs)[2][128], const Place<LPH, PAIRS>& at,
                                            int rotary, float (&c)[8], float (&s)[8]) {
  if constexpr (PAIRS == kOddHalves) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = PAIRS == kHalves ? 8 * at.u + j : (j < 4 ? at.a : at.b) / 2 + j % 4;
    const bool in = 2 * i < rotary;
    c[j] = in ? cs[0][i] : 1.f;
    s[j] = in ? cs[1][i] : 0.f;
  }
}

// Turns a lane's 16 values.  `head`: hd floats of LDS for the head (kOddHalves).
template <int LPH, int PAIRS>
__device__ __forceinline__ void turn16(float (&v)[16], const float (&c)[8], const float (&s)[8],
                                       const Place<LPH, PAIRS>& at, int rotary,
                                       const float (&cs)[2][128], float* head) {
  if constexpr (PAIRS == kHalves) {
    if (at.turns) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = v[j], y = v[8 + j];
        v[j] = x * c[j] - y * s[j];
        v[8 + j] = y * c[j] + x * s[j];
      }
    }
  } else if constexpr (PAIRS == kNeighbours) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = v[2 * j], y = v[2 * j + 1];
      const bool in = (j < 4 ? at.a : at.b) + 2 * (j % 4) < rotary;
      v[2 * j] = in ? x * c[j] - y * s[j] : x;
      v[2 * j + 1] = in ? y * c[j] + x * s[j] : y;
    }
  } else {
    const int half = rotary / 2;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    if (at.active) {
#pragma unroll
      for (int j = 0; j < 16; ++j) head[(j < 8 ? at.a : at.b) + j % 8] = v[j];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (at.active) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int e = (j < 8 ? at.a : at.b) + j % 8;
        if (e < rotary) {
          const bool first = e < half;
          const int i = first ? e : e - half;
          const float y = head[first ? e + half : i], t = y * cs[1][i];
          v[j] = first ? v[j] * cs[0][i] - t : v[j] * cs[0][i] + t;
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // read before the next head's
    __builtin_amdgcn_wave_barrier();
  }
}

template <int PAIRS>
struct Exchange {
  float f[kHeadRows][PAIRS == kOddHalves ? 1024 : 1];
};

// A row's heads in groups of `group`, q's then k's (and v's): 1 << share waves
// take them in turn.  The wave's row and its first head of each kind:
struct Part {
  int64_t row;
  int mine, waves, before;      // before: groups of the kinds gone by
  __device__ __forceinline__ Part(int wave, int share) {
    const int64_t i = (int64_t)blockIdx.x * kHeadRows + wave;
    row = i >> share;
    waves = 1 << share;
    mine = (int)i & (waves - 1);
    before = 0;
  }
  __device__ __forceinline__ int first(int nh, int group) {
    const int g = (mine - before) & (waves - 1);
    before += (nh + group - 1) / group;
    return g * group;
  }
};

// 1 << share waves a row.
template <int LPH, int PAIRS>
__global__ void __launch_bounds__(256) rope_rows_kernel(const RopeArgs a, int share) {
  constexpr int HPW = 64 / LPH, CH = 4;
  __shared__ __attribute__((aligned(16))) float trig[kHeadRows][2][128];
  __shared__ __attribute__((aligned(16))) Exchange<PAIRS> xch;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Part part(wave, share);
  const int64_t row = part.row;
  if (row >= a.rows) return;
  const Place<LPH, PAIRS> at(lane, a.hd, a.turn.rotary);
  const int hs = lane / LPH;
  const uint32_t head_bytes = (uint32_t)a.hd * 2u;
  const int lane_a = hs * (int)head_bytes + at.a * 2, lane_b = hs * (int)head_bytes + at.b * 2;
  auto off = [&](int h0, int lane_off) {
    return at.active ? h0 * (int)head_bytes + lane_off : kQkRmsOut;
  };
  u32x4_t x[CH][2];
  auto load = [&](const RowBuf& ib, int h0) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {                         // past the last head: loads 0
      x[i][0] = ib.ld16(off(h0 + i * HPW, lane_a));
      x[i][1] = ib.ld16(off(h0 + i * HPW, lane_b));
    }
  };
  const RowBuf qb(a.x[0] + row * a.ldx[0], (uint32_t)a.nh[0] * head_bytes);
  load(qb, part.mine * CH * HPW);                          // past q's heads: not used
  fill_turn(trig[wave], position(a.pos, row), a.turn, lane);
  float c[8], s[8];
  lane_angles(trig[wave], at, a.turn.rotary, c, s);
  float* head = xch.f[wave] + (PAIRS == kOddHalves ? hs * a.hd : 0);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const int nh = a.nh[which];
    if (nh == 0) continue;
    const RowBuf ib(a.x[which] + row * a.ldx[which], (uint32_t)nh * head_bytes);
    const RowBuf ob(a.y[which] + row * a.ldy[which], (uint32_t)nh * head_bytes);
    const int start = part.first(nh, CH * HPW);
    for (int h0 = start; h0 < nh; h0 += CH * HPW << share) {
      if (which > 0 || h0 > start) load(ib, h0);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (h0 + i * HPW >= nh) break;                     // uniform
        float v[16];
        unpack8(x[i][0], v);
        unpack8(x[i][1], v + 8);
        turn16(v, c, s, at, a.turn.rotary, trig[wave], head);
        ob.st16(pack8(v), off(h0 + i * HPW, lane_a));
        ob.st16(pack8(v + 8), off(h0 + i * HPW, lane_b));
      }
    }
  }
}

// value / scale, from inv = 1 / scale: one step of Newton's makes the product's
// rounding the quotient's.  Past e4m3's range only the sign matters.
__device__ __forceinline__ float over_scale(float x, float scale, float inv) {
  const float q = x * inv;
  const float r = __builtin_fmaf(__builtin_fmaf(-q, scale, x), inv, q);
  return fabsf(q) < 512.f ? r : q;
}

// Eight values as e4m3: to nearest even, the largest past its range, NaN kept.
__device__ __forceinline__ u32x2_t pack8_e4m3(const float* v, float scale, float inv) {
  float q[8];
  if (inv != 0.f && fabsf(inv) < __builtin_inff()) {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = over_scale(v[j], scale, inv);
  } else {                                   // a scale below 2^-128 or infinite: 1 / scale says nothing of it
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = v[j] / scale;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    q[j] = q[j] > 448.f ? 448.f : q[j] < -448.f ? -448.f : q[j];
  }
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return u32x2_t{(uint32_t)lo, (uint32_t)hi};
}

// Byte offset of sequence `seq`'s token `p`, or -1 where the cache has none.
// (Everything here is the same in the whole wave; the tables are only read.)
__device__ __forceinline__ int64_t token_offset(const CacheView& c, int64_t seq, int32_t p) {
  if (!token_in_table(c, seq, p)) return -1;
  return token_bytes_at(c, position(c.table, table_entry(c, seq, p)), p);
}

// 1 << share waves a row.  Bounds for five waves a SIMD: 24 prompts of up to 1,021
// tokens, 16 + 2 * 4 heads of 256 into e4m3, take 54 us with them, 66 with none and 67
// with bounds for six (registers spilled).
template <int LPH, int PAIRS, bool RMS>
__global__ void __launch_bounds__(256, PAIRS == kOddHalves ? 4 : 5) cache_append_kernel(const AppendArgs a, int share) {
  constexpr int HPW = 64 / LPH, CH = 2;
  __shared__ __attribute__((aligned(16))) float trig[kHeadRows][2][128];
  __shared__ __attribute__((aligned(16))) Exchange<PAIRS> xch;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Part part(wave, share);
  const int64_t row = part.row;
  if (row >= a.rows) return;
  const CacheView& cv = a.cache;
  const int hd = cv.hd, rotary = a.turn.rotary;
  const Place<LPH, PAIRS> at(lane, hd, rotary);
  const int hs = lane / LPH;
  const float per_hd = 1.f / (float)hd;
  const uint32_t head_bytes = (uint32_t)hd * 2u;
  const int lane_a = hs * (int)head_bytes + at.a * 2, lane_b = hs * (int)head_bytes + at.b * 2;
  auto off = [&](int h0, int lane_off) {
    return at.active ? h0 * (int)head_bytes + lane_off : kQkRmsOut;
  };
  const int32_t p = position(a.pos, row);
  const int64_t seq = a.seq != nullptr ? (int64_t)position(a.seq, row) : (a.row0 + row) / a.rows_per_seq;
  const int64_t token = token_offset(cv, seq, p);
  fill_turn(trig[wave], p, a.turn, lane);
  float c[8], s[8];
  lane_angles(trig[wave], at, rotary, c, s);
  float* head = xch.f[wave] + (PAIRS == kOddHalves ? hs * hd : 0);
#pragma unroll
  for (int which = 0; which < 3; ++which) {
    const int nh = which == 0 ? a.q_heads : cv.heads;
    if (nh == 0 || (which > 0 && token < 0)) continue;     // uniform
    const int start = part.first(nh, CH * HPW);
    if (start >= nh) continue;
    float w[16];
    if (RMS && which < 2) {
      load_weights(a.w[which], at.a, at.active, w);
      load_weights(a.w[which], at.b, at.active, w + 8);
    }
    const RowBuf ib(a.x[which] + row * a.ldx[which], (uint32_t)nh * head_bytes);
    const RowBuf ob(which == 0 ? a.q_out + row * a.ldq_out : nullptr,
                    which == 0 ? (uint32_t)nh * head_bytes : 0u);
    char* to = which == 1 ? cv.k : cv.v;
    const float* scales = which == 1 ? cv.k_scale : cv.v_scale;
    for (int h0 = start; h0 < nh; h0 += CH * HPW << share) {
      u32x4_t x[CH][2];
      float scale[CH];
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        x[i][0] = ib.ld16(off(h0 + i * HPW, lane_a));
        x[i][1] = ib.ld16(off(h0 + i * HPW, lane_b));
        scale[i] = which > 0 && scales != nullptr ? scales[min(h0 + i * HPW + hs, nh - 1)] : 1.f;
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int h = h0 + i * HPW;
        if (h >= nh) break;                                // uniform
        float v[16];
        unpack8(x[i][0], v);
        unpack8(x[i][1], v + 8);
        if (which < 2) {
          if constexpr (RMS) {
            int sh;
            const float inv = head_inv_rms<LPH>(v, per_hd, a.eps, sh);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = v[j] * inv * w[j];
          }
          turn16(v, c, s, at, rotary, trig[wave], head);
        }
        if (which == 0) {
          ob.st16(pack8(v), off(h, lane_a));
          ob.st16(pack8(v + 8), off(h, lane_b));
        } else if (at.active && h + hs < nh) {
          char* t = to + token + (int64_t)(h + hs) * cv.head_bytes;
          if (cv.e4m3) {
            const float inv = 1.f / scale[i];
            *(u32x2_t*)(t + at.a) = pack8_e4m3(v, scale[i], inv);
            *(u32x2_t*)(t + at.b) = pack8_e4m3(v + 8, scale[i], inv);
          } else {
            *(u32x4_t*)(t + at.a * 2) = pack8(v);
            *(u32x4_t*)(t + at.b * 2) = pack8(v + 8);
          }
        }
      }
    }
  }
}

static int lanes_per_head(int hd) {
  int n = 1;
  while (n * 16 < hd) n *= 2;
  return n;
}

static int pairing(const Turn& t) {
  return t.interleaved ? kNeighbours : t.rotary % 16 == 0 ? kHalves : kOddHalves;
}

constexpr int kFew = 4;

static int groups(int heads, int group) { return (heads + group - 1) / group; }

// log2 of the waves that share a row of `n` groups: as many as have one each,
// up to a workgroup's four, where that leaves at most kFew waves a SIMD.  64
// rows of 16 + 2 * 4 heads of 256 take 8.6 us by one wave each, 5.6 by four;
// 24,500 rows of 32 + 2 * 8 heads of 128 take 53 by one, 59 by four (each finds
// its row's angles again).
static int waves_of(int64_t rows, int n, int cus) {
  int share = 0;
  while (share < 2 && 1 << share < n && rows << (share + 1) <= (int64_t)cus * 4 * kFew) ++share;
  return share;
}

static int grid_of(int64_t rows, int share) {
  return (int)(((rows << share) + kHeadRows - 1) / kHeadRows);
}

template <int LPH>
static hipError_t rope_lanes(const RopeArgs& a, int cus, hipStream_t stream) {
  const int share = waves_of(a.rows, groups(a.nh[0], 256 / LPH) + groups(a.nh[1], 256 / LPH), cus);
  const int grid = grid_of(a.rows, share);
  switch (pairing(a.turn)) {
    case kHalves: rope_rows_kernel<LPH, kHalves><<<grid, 256, 0, stream>>>(a, share); break;
    case kNeighbours: rope_rows_kernel<LPH, kNeighbours><<<grid, 256, 0, stream>>>(a, share); break;
    default: rope_rows_kernel<LPH, kOddHalves><<<grid, 256, 0, stream>>>(a, share); break;
  }
  return hipGetLastError();
}

hipError_t launch_rope_rows(const RopeArgs& a, int cus, hipStream_t stream) {
  switch (lanes_per_head(a.hd)) {
    case 1: return rope_lanes<1>(a, cus, stream);
    case 2: return rope_lanes<2>(a, cus, stream);
    case 4: return rope_lanes<4>(a, cus, stream);
    case 8: return rope_lanes<8>(a, cus, stream);
    case 16: return rope_lanes<16>(a, cus, stream);
    default: return hipErrorInvalidValue;
  }
}

template <int LPH, bool RMS>
static hipError_t append_lanes(const AppendArgs& a, int cus, hipStream_t stream) {
  const int share = waves_of(
      a.rows, groups(a.q_heads, 128 / LPH) + 2 * groups(a.cache.heads, 128 / LPH), cus);
  const int grid = grid_of(a.rows, share);
  switch (pairing(a.turn)) {
    case kHalves: cache_append_kernel<LPH, kHalves, RMS><<<grid, 256, 0, stream>>>(a, share); break;
    case kNeighbours: cache_append_kernel<LPH, kNeighbours, RMS><<<grid, 256, 0, stream>>>(a, share); break;
    default: cache_append_kernel<LPH, kOddHalves, RMS><<<grid, 256, 0, stream>>>(a, share); break;
  }
  return hipGetLastError();
}

template <int LPH>
static hipError_t append_norm(const AppendArgs& a, int cus, hipStream_t stream) {
  return a.rms ? append_lanes<LPH, true>(a, cus, stream) : append_lanes<LPH, false>(a, cus, stream);
}

hipError_t launch_cache_append(const AppendArgs& a, int cus, hipStream_t stream) {
  switch (lanes_per_head(a.cache.hd)) {
    case 1: return append_norm<1>(a, cus, stream);
    case 2: return append_norm<2>(a, cus, stream);
    case 4: return append_norm<4>(a, cus, stream);
    case 8: return append_norm<8>(a, cus, stream);
    case 16: return append_norm<16>(a, cus, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dsr
