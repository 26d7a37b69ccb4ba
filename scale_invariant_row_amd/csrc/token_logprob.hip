// Rows of logits: log probability of a given token, entropy, top alternatives,
// and the gradient.
//
//   z_j = (x_j scale_j) inv_temp;  lse = log sum exp z;  logp = z_label - lse
//   entropy = lse - sum p z = log S - T / S  with  M = max z,
//             S = sum exp(z - M),  T = sum exp(z - M) (z - M)
//
// The row is cut into chunks of kLpChunk columns.  One wave holds a chunk in
// registers (32 values a lane, read once), takes its maximum, and then its S
// and T about that maximum, so no exponential is ever rescaled inside a
// chunk.  The chunks' (M, S, T) are joined by a tree that the number of chunks
// fixes, whoever computed them: the row's bits depend on the row and its width
// alone, and a row may be spread over any number of waves.
//
// Cost per value beside its load: unpack, scale, half a maximum, one fused
// multiply-add to log2 units, exp2 (four issue slots), a sum and a fused
// multiply-add: 10 slots, 270 us for 8,192 x 131,072 bf16 values, under the
// time their 2.1 GB take from memory.  Measured: 409 us (5.3 TB/s) with the 5
// best of each row, 363 without.
//
// Masked tokens (z = -inf) have exp 0 but 0 * -inf in T.  The fast sums go
// without a test for them: a chunk whose T comes out NaN (a masked token in it,
// or nothing above -inf) or that lies millions from 0 is summed again in the
// careful form (lp_careful), where the factor is clamped at -200 (exp is 0
// there already); a NaN of the row's own stays NaN.  With a token masked in
// every chunk that is every chunk twice: 8,192 x 131,072 with 30 % of the
// columns at -inf takes 565 us, with -1e30 there 409.
#include <algorithm>
#include <type_traits>

#include "row_kernels.hpp"
#include "token_launch.hpp"

namespace dsr {

constexpr int kLpPer = 32;                            // columns per lane of a chunk
constexpr int kLpChunk = 64 * kLpPer;                 // 2,048
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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

// Joins the sums of two stretches.  With every token of a stretch masked, M
// is -inf and S, T are 0.
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

// The joined sums of n chunks, in every lane: lane l takes chunks l, l + 64,
// ... in order, then the lanes pair up.  get(c) gives chunk c's sums.
template <class F>
__device__ __forceinline__ LpSum lp_join_all(int n, int lane, F&& get) {
  LpSum s = {-__builtin_inff(), 0.f, 0.f};
  for (int c = lane; c < n; c += 64) s = lp_join(s, get(c));
  for (int d = 1; d < 64; d *= 2) {
    const LpSum o = {__shfl_xor(s.M, d), __shfl_xor(s.S, d), __shfl_xor(s.T, d)};
    s = lp_join(s, o);
  }
  return s;
}

// -------------------------------------------------------- top alternatives
//
// A key orders tokens: larger z first, then the lower column.  0 stands for a
// token that cannot be listed (masked, or NaN).  A wave keeps its best tokens
// as a sorted list over its lanes (lane i the i-th best); a chunk's values
// are looked at one by one only where a lane's maximum beats the list's k-th.

__device__ __forceinline__ uint32_t lp_order(float z) {
  const uint32_t u = __float_as_uint(z + 0.f);        // -0 orders as 0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float lp_unorder(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ uint64_t lp_key(float z, int col) {
  return z > -__builtin_inff() ? ((uint64_t)lp_order(z) << 32) | (uint32_t)~(uint32_t)col : 0;
}

__device__ __forceinline__ uint64_t lp_read_lane(uint64_t v, int lane) {
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), lane);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane);
  return ((uint64_t)hi << 32) | lo;
}

// v of the lane below (lane 0 keeps its own).
__device__ __forceinline__ uint64_t lp_lane_below(uint64_t v) {
  const int hi = (int)(v >> 32), lo = (int)(uint32_t)v;
  const uint32_t h = (uint32_t)__builtin_amdgcn_update_dpp(hi, hi, 0x138, 0xF, 0xF, false);
  const uint32_t l = (uint32_t)__builtin_amdgcn_update_dpp(lo, lo, 0x138, 0xF, 0xF, false);
  return ((uint64_t)h << 32) | l;
}

struct LpTop {
  uint64_t key = 0;        // lane i: the i-th best so far, 0 past the end
  uint64_t kth = 0;        // the k-th best (uniform)

  // One key (uniform) into its place.
  __device__ __forceinline__ void insert(uint64_t k, int top_k, int lane) {
    const int pos = __builtin_popcountll(__builtin_amdgcn_ballot_w64(key > k));
    const uint64_t below = lp_lane_below(key);
    key = lane < pos ? key : lane == pos ? k : below;
    kth = lp_read_lane(key, top_k - 1);
  }

  // Every lane's key that belongs in the list, lowest lane first.
  __device__ __forceinline__ void add(uint64_t k, int top_k, int lane) {
    uint64_t hits = __builtin_amdgcn_ballot_w64(k > kth);
    while (hits != 0) {
      const int l = __builtin_ctzll(hits);
      insert(lp_read_lane(k, l), top_k, lane);
      hits &= __builtin_amdgcn_ballot_w64(k > kth);
      hits &= ~(1ull << l);
    }
  }
};

// A lower bound of the k-th largest of the lanes' values (in lp_order's
// order): its upper 16 bits, found bit by bit.  At least k lanes reach it.
__device__ __forceinline__ uint32_t lp_kth_lane(uint32_t u, int k) {
  uint32_t t = 0;
#pragma unroll
  for (int b = 31; b >= 16; --b) {
    const uint32_t c = t | (1u << b);
    if (__builtin_popcountll(__builtin_amdgcn_ballot_w64(u >= c)) >= k) t = c;
  }
  return t;
}

// ------------------------------------------------------------ chunk of a row
//
// Lane l holds, of each stretch of 64 vectors, the l-th: 8 bf16 or 4 fp32
// columns, 16 bytes, at whatever alignment the row has (global loads need
// none beyond the element's).

typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));
typedef f32x4_t f32x4_a4 __attribute__((aligned(4)));

template <bool F32>
struct LpRaw {
  static constexpr int VE = F32 ? 4 : 8;              // columns per vector
  static constexpr int NV = kLpPer / VE;
  u32x4_t r[NV];

  static __device__ __forceinline__ int col(int c0, int v, int lane) {
    return c0 + (v * 64 + lane) * VE;
  }

  // The chunk at column c0; columns past the row read as -inf.
  __device__ __forceinline__ void load(const void* x, int64_t at, int c0, int vocab, int lane) {
    using V = typename std::conditional<F32, u32x4_a4, u32x4_a2>::type;
    using E = typename std::conditional<F32, uint32_t, uint16_t>::type;
    const E* row = static_cast<const E*>(x) + at;
    if (c0 + kLpChunk <= vocab) {                     // uniform
#pragma unroll
      for (int v = 0; v < NV; ++v)
        r[v] = __builtin_nontemporal_load(reinterpret_cast<const V*>(row + col(c0, v, lane)));
      return;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = col(c0, v, lane);
      if (c + VE <= vocab) {
        r[v] = *reinterpret_cast<const V*>(row + c);
      } else {
        uint32_t e[VE];
#pragma unroll
        for (int k = 0; k < VE; ++k)
          e[k] = c + k < vocab ? (uint32_t)row[c + k] : F32 ? 0xff800000u : 0xff80u;
        if constexpr (F32) r[v] = u32x4_t{e[0], e[1], e[2], e[3]};
        else r[v] = u32x4_t{e[0] | e[1] << 16, e[2] | e[3] << 16, e[VE - 4] | e[VE - 3] << 16,
                            e[VE - 2] | e[VE - 1] << 16};
      }
    }
  }

  __device__ __forceinline__ float at(int i) const {  // i-th of the lane's 32 values
    const u32x4_t t = r[i / VE];
    const int w = i % VE;
    if constexpr (F32) return __uint_as_float(t[w]);
    else return w % 2 == 0 ? bf_lo(t[w / 2]) : bf_hi(t[w / 2]);
  }
};

// The scale of a lane's 32 columns (1 past the row).
template <bool F32>
__device__ __forceinline__ void lp_load_scale(float (&sc)[kLpPer], const float* scale, int c0,
                                              int vocab, int lane) {
  using R = LpRaw<F32>;
  const bool whole = c0 + kLpChunk <= vocab;
#pragma unroll
  for (int v = 0; v < R::NV; ++v) {
    const int c = R::col(c0, v, lane);
    if (whole || c + R::VE <= vocab) {
#pragma unroll
      for (int h = 0; h < R::VE; h += 4) {
        const f32x4_t t = *reinterpret_cast<const f32x4_a4*>(scale + c + h);
        sc[v * R::VE + h] = t.x; sc[v * R::VE + h + 1] = t.y;
        sc[v * R::VE + h + 2] = t.z; sc[v * R::VE + h + 3] = t.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < R::VE; ++k) sc[v * R::VE + k] = c + k < vocab ? scale[c + k] : 1.f;
    }
  }
}

// The wave's maximum of a value that is no NaN, in every lane.  Ordered as whole
// numbers, so that each step is one instruction (fmaxf would quiet NaNs of both
// sides first): within 16 lanes, then row after row into the last lane.
template <int CTRL>
__device__ __forceinline__ int lp_max_step(int v) {
  const int o = __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true);
  return v > o ? v : o;
}

__device__ __forceinline__ float lp_wave_max(float m) {
  const int u = __builtin_bit_cast(int, m);
  int v = u ^ ((u >> 31) & 0x7fffffff);
  v = lp_max_step<0xB1>(v);    // quad_perm [1,0,3,2]
  v = lp_max_step<0x4E>(v);    // quad_perm [2,3,0,1]
  v = lp_max_step<0x141>(v);   // row_half_mirror
  v = lp_max_step<0x140>(v);   // row_mirror
  v = lp_max_step<0x142>(v);   // row_bcast:15 (the first row gets 0: not lane 63's)
  v = lp_max_step<0x143>(v);   // row_bcast:31
  v = __builtin_amdgcn_readlane(v, 63);
  return __builtin_bit_cast(float, v ^ ((v >> 31) & 0x7fffffff));
}

// S and T about the chunk's maximum M with every step guarded: see the head of
// this file.
__device__ __forceinline__ LpSum lp_careful(const float (&z)[kLpPer], float M) {
  const float base = M == -__builtin_inff() ? 0.f : M;
  float S = 0.f, T = 0.f;
#pragma unroll
  for (int i = 0; i < kLpPer; ++i) {
    const float d = z[i] - base, e = lp_exp(d);
    S += e;
    T = __builtin_fmaf(e, fmaxf(d, -200.f), T);
  }
  return LpSum{M, wave_sum(S), wave_sum(T)};
}

// A chunk's sums, the same in every lane; m: the lane's maximum.  They are
// about the chunk's own maximum M: the top's term is 1, S >= 1, and neither
// log S nor T / S is larger than it has to be.  A base that needs no exchange
// between lanes (lane 0's maximum: 405 us where this takes 409) lets both grow
// to some 13 in rows whose top stands out, and they lose that many digits to
// each other: 1.5e-5 of an entropy, 3e-6 of a log probability, 2e-6 and 8e-7
// here (3,000 rows with a top 2 to 14 above the rest).  With c = fp32(M log2 e)
// the sums are about c in log2 units, z log2 e - c one fused multiply-add; r,
// the rounding error of c (a fused multiply-add gives it exactly), turns them
// into those about M:  z log2 e - c = (z - M) log2 e + r.  Beside a c past 2^24
// r is no longer a fraction (a chunk masked with -1e30 has one of 1e21, and S
// would be 0 or infinite): the careful form then.
__device__ __forceinline__ LpSum lp_chunk_sum(const float (&z)[kLpPer], float m) {
  const float M = lp_wave_max(m);
  const float c = M * kLog2e;
  float S = 0.f, T = 0.f;
#pragma unroll
  for (int i = 0; i < kLpPer; ++i) {
    const float d = __builtin_fmaf(z[i], kLog2e, -c), e = __builtin_amdgcn_exp2f(d);
    S += e;
    T = __builtin_fmaf(e, d, T);
  }
  S = wave_sum(S);
  T = wave_sum(T);
  const float r = __builtin_fmaf(M, kLog2e, -c);
  if (!(T == T && fabsf(r) <= 0.5f)) return lp_careful(z, M);   // uniform
  const float f = __builtin_amdgcn_exp2f(-r);
  return LpSum{M, S * f, (T - r * S) * f * kLn2};
}

// A wave's share of a row: the sums of one chunk at a time, and the list.
template <bool F32, bool SCALED>
struct LpRow {
  LpTop top;

  __device__ __forceinline__ LpSum chunk(const LpRaw<F32>& raw, const float (&sc)[kLpPer],
                                         float inv_temp, int c0, int top_k, int lane) {
    using R = LpRaw<F32>;
    constexpr int G = 8;                              // values of a group
    float z[kLpPer], gm[kLpPer / G];                  // and the groups' maxima
#pragma unroll
    for (int i = 0; i < kLpPer; ++i) {
      z[i] = raw.at(i);
      if constexpr (SCALED) z[i] = z[i] * sc[i];
    }
    if (inv_temp != 1.f) {                            // uniform; * 1 changes nothing
#pragma unroll
      for (int i = 0; i < kLpPer; ++i) z[i] = z[i] * inv_temp;
    }
    float m = -__builtin_inff();
#pragma unroll
    for (int g = 0; g < kLpPer / G; ++g) {
      gm[g] = z[g * G];
#pragma unroll
      for (int i = 1; i < G; ++i) gm[g] = fmaxf(gm[g], z[g * G + i]);
      m = fmaxf(m, gm[g]);
    }
    const LpSum s = lp_chunk_sum(z, m);
    if (top_k > 0) {
      // the least z that can enter the list: above the k-th best so far
      // (columns only rise, so an equal value comes too late)
      uint32_t least = top.kth != 0 ? (uint32_t)(top.kth >> 32) + 1 : lp_order(-__builtin_inff()) + 1;
      const uint64_t hits = __builtin_amdgcn_ballot_w64(m >= lp_unorder(least));
      if (hits != 0) {
        // many lanes: only values that reach the k-th largest lane maximum
        // can be among the chunk's k best
        if (__builtin_popcountll(hits) > top_k) {
          const uint32_t t = lp_kth_lane(m > -__builtin_inff() ? lp_order(m) : 0u, top_k);
          least = t > least ? t : least;
        }
        const float lz = lp_unorder(least);
#pragma unroll
        for (int g = 0; g < kLpPer / G; ++g) {
          if (__builtin_amdgcn_ballot_w64(gm[g] >= lz) == 0) continue;
#pragma unroll
          for (int i = g * G; i < (g + 1) * G; ++i) {
            const bool may = z[i] >= lz;
            if (__builtin_amdgcn_ballot_w64(may) != 0)
              top.add(may ? lp_key(z[i], R::col(c0, i / R::VE, lane) + i % R::VE) : 0, top_k, lane);
          }
        }
      }
    }
    return s;
  }
};

// Writes a row's three numbers and its list from the joined sums; zy is the
// label's z (read ahead), y its column or -1.
__device__ __forceinline__ void lp_write_row(const LogprobArgs& a, int64_t row, LpSum sum,
                                             uint64_t key, int y, float zy, int lane) {
  const bool empty = sum.M == -__builtin_inff() && sum.S == 0.f;
  const float log_s = logf(sum.S);
  if (lane == 0) {
    if (a.lse != nullptr) a.lse[row] = empty ? -__builtin_inff() : sum.M + log_s;
    if (a.entropy != nullptr) a.entropy[row] = empty ? 0.f : log_s - sum.T / sum.S;
    if (a.logp != nullptr)
      a.logp[row] = y < 0 ? 0.f : empty ? -__builtin_inff() : (zy - sum.M) - log_s;
  }
  if (lane < a.top_k) {
    a.top_ids[row * a.top_k + lane] = key != 0 ? (int32_t)~(uint32_t)key : -1;
    a.top_logp[row * a.top_k + lane] =
        key != 0 ? (lp_unorder((uint32_t)(key >> 32)) - sum.M) - log_s : -__builtin_inff();
  }
}

// One workgroup of four waves per ROWS rows.  Each wave takes every fourth
// chunk of all of them, so a chunk's scale is loaded once for ROWS rows (with
// two rows 8,192 x 131,072 scaled bf16 took 457 us where four took 434); the
// next row's values are on their way while one is summed (ROWS is 1 or even:
// two buffers take turns).  Dynamic LDS: the chunks' sums, [ROWS][chunks].
template <bool F32, bool SCALED, int ROWS>
__global__ void __launch_bounds__(256) logprob_rows_kernel(const LogprobArgs a, int chunks) {
  extern __shared__ float sums[];
  __shared__ uint64_t lists[ROWS][4][32];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row0 = (int64_t)blockIdx.x * ROWS;
  const int rows = (int)(a.rows - row0 < ROWS ? a.rows - row0 : ROWS);
  // wave r writes row r: its label's z on the way
  int y = -1;
  float zy = 0.f;
  if (wave < rows) {
    y = lp_label(a.labels, a.label_bytes, row0 + wave, a.vocab);
    if (y >= 0) zy = lp_z(lp_load<F32>(a.x, (row0 + wave) * a.ld + y), a.scale, y, a.inv_temp);
  }
  // a last workgroup of fewer rows works on its last one again
  LpRow<F32, SCALED> st[ROWS];
  LpRaw<F32> raw[2];
  auto load = [&](LpRaw<F32>& to, int r, int c) {
    if (c < chunks) to.load(a.x, (row0 + (r < rows ? r : rows - 1)) * a.ld, c * kLpChunk, a.vocab, lane);
  };
  load(raw[0], 0, wave);
  for (int c = wave; c < chunks; c += 4) {
    float sc[kLpPer];
    if constexpr (SCALED) lp_load_scale<F32>(sc, a.scale, c * kLpChunk, a.vocab, lane);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      LpRaw<F32>&now = raw[r % 2], &next = raw[(r + 1) % 2];
      load(next, r + 1 < ROWS ? r + 1 : 0, r + 1 < ROWS ? c : c + 4);
      const LpSum s = st[r].chunk(now, sc, a.inv_temp, c * kLpChunk, a.top_k, lane);
      if (lane == 0) {
        float* p = sums + ((int64_t)r * chunks + c) * 3;
        p[0] = s.M; p[1] = s.S; p[2] = s.T;
      }
      if constexpr (ROWS == 1) raw[0] = raw[1];
    }
  }
  if (a.top_k > 0 && lane < a.top_k) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) lists[r][wave][lane] = st[r].top.key;
  }
  __syncthreads();
  if (wave >= rows) return;
  const LpSum sum = lp_join_all(chunks, lane, [&](int c) {
    const float* p = sums + ((int64_t)wave * chunks + c) * 3;
    return LpSum{p[0], p[1], p[2]};
  });
  LpTop top;
  if (a.top_k > 0) {
    const bool in = lane < a.top_k;
    top.key = in ? lists[wave][0][lane] : 0;
    top.kth = lp_read_lane(top.key, a.top_k - 1);
    for (int w = 1; w < 4; ++w) top.add(in ? lists[wave][w][lane] : 0, a.top_k, lane);
  }
  lp_write_row(a, row0 + wave, sum, top.key, y, zy, lane);
}

// Few rows: a row is spread over `splits` workgroups; wave w of the row's
// 4 splits takes chunks w, w + 4 splits, ...  The chunks' sums and the waves'
// lists go to the workspace, sums [rows][chunks][3], then keys
// [rows][top_k][waves].
template <bool F32, bool SCALED>
__global__ void __launch_bounds__(256)
logprob_split_kernel(const LogprobArgs a, int chunks, int splits, float* sums, uint64_t* keys) {
  const int lane = threadIdx.x & 63;
  const int64_t row = blockIdx.x / splits;
  const int waves = splits * 4;
  const int w = (int)(blockIdx.x % splits) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  LpRow<F32, SCALED> st;
  for (int c = w; c < chunks; c += waves) {
    LpRaw<F32> raw;
    float sc[kLpPer];
    raw.load(a.x, row * a.ld, c * kLpChunk, a.vocab, lane);
    if constexpr (SCALED) lp_load_scale<F32>(sc, a.scale, c * kLpChunk, a.vocab, lane);
    const LpSum s = st.chunk(raw, sc, a.inv_temp, c * kLpChunk, a.top_k, lane);
    if (lane == 0) {
      float* p = sums + (row * chunks + c) * 3;
      p[0] = s.M; p[1] = s.S; p[2] = s.T;
    }
  }
  if (lane < a.top_k) keys[(row * a.top_k + lane) * waves + w] = st.top.key;
}

// Joins a split row: one wave per row.  The lists are sorted, so once no wave
// of 64 has a place-j key for the list, their deeper ones have none either.
template <bool F32>
__global__ void __launch_bounds__(64)
logprob_join_kernel(const LogprobArgs a, int chunks, int waves, const float* sums,
                    const uint64_t* keys) {
  constexpr int AT_ONCE = 8;                          // places of the lists loaded together
  const int lane = threadIdx.x;
  const int64_t row = blockIdx.x;
  uint64_t k[AT_ONCE];
  auto load = [&](int j0, int w0) {
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j)
      k[j] = j0 + j < a.top_k && w0 + lane < waves
                 ? keys[(row * a.top_k + j0 + j) * waves + w0 + lane] : 0;
  };
  load(0, 0);                                         // on its way during the sums
  const int y = lp_label(a.labels, a.label_bytes, row, a.vocab);
  const LpSum sum = lp_join_all(chunks, lane, [&](int c) {
    const float* p = sums + (row * chunks + c) * 3;
    return LpSum{p[0], p[1], p[2]};
  });
  const float zy = y >= 0 ? lp_z(lp_load<F32>(a.x, row * a.ld + y), a.scale, y, a.inv_temp) : 0.f;
  LpTop top;
  for (int j0 = 0; j0 < a.top_k; j0 += AT_ONCE) {
    uint64_t any = 0;
    for (int w0 = 0; w0 < waves; w0 += 64) {
      if (j0 > 0 || w0 > 0) load(j0, w0);
      // as in a chunk: only keys that reach the k-th largest first place
      uint32_t least = 0;
      if (j0 == 0 && w0 == 0) least = lp_kth_lane((uint32_t)(k[0] >> 32), a.top_k);
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j) {
        const uint64_t in = (uint32_t)(k[j] >> 32) >= least ? k[j] : 0;
        any = __builtin_amdgcn_ballot_w64(in > top.kth);
        if (any == 0) break;                          // uniform: deeper places hold less
        top.add(in, a.top_k, lane);
      }
    }
    if (waves <= 64 && any == 0) break;
  }
  lp_write_row(a, row, sum, top.key, y, zy, lane);
}

static int lp_chunks(int64_t vocab) { return (int)((vocab + kLpChunk - 1) / kLpChunk); }

// Workgroups a row is spread over: enough for about 2,048 waves in all (two
// for each SIMD), as far as it has chunks.  Results do not depend on it.
static int lp_splits(int64_t rows, int chunks) {
  const int64_t want = (512 + rows - 1) / (rows > 0 ? rows : 1);
  const int most = (chunks + 3) / 4;
  return (int)(want < most ? want : most);
}

int64_t logprob_workspace(int64_t rows, int64_t vocab, int top_k) {
  const int chunks = lp_chunks(vocab), splits = lp_splits(rows, chunks);
  if (rows == 0 || splits <= 1) return 0;
  const int64_t sums = (rows * chunks * 12 + 15) / 16 * 16;
  return sums + rows * top_k * splits * 4 * 8;
}

template <bool F32, bool SCALED>
static hipError_t run_logprob(const LogprobArgs& a, void* workspace, hipStream_t stream) {
  const int chunks = lp_chunks(a.vocab), splits = lp_splits(a.rows, chunks);
  if (splits > 1) {                                   // at most 511 rows
    float* sums = static_cast<float*>(workspace);
    auto* keys = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) +
                                             (a.rows * chunks * 12 + 15) / 16 * 16);
    logprob_split_kernel<F32, SCALED>
        <<<(int)a.rows * splits, 256, 0, stream>>>(a, chunks, splits, sums, keys);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    logprob_join_kernel<F32><<<(int)a.rows, 64, 0, stream>>>(a, chunks, splits * 4, sums, keys);
    return hipGetLastError();
  }
  constexpr int64_t kMostRows = 1 << 20;              // rows per launch
  for (int64_t r0 = 0; r0 < a.rows; r0 += kMostRows) {
    LogprobArgs p = a;
    p.rows = a.rows - r0 < kMostRows ? a.rows - r0 : kMostRows;
    p.x = static_cast<const char*>(a.x) + r0 * a.ld * (F32 ? 4 : 2);
    if (a.labels != nullptr) p.labels = static_cast<const char*>(a.labels) + r0 * a.label_bytes;
    if (a.logp != nullptr) p.logp = a.logp + r0;
    if (a.entropy != nullptr) p.entropy = a.entropy + r0;
    if (a.lse != nullptr) p.lse = a.lse + r0;
    if (a.top_k > 0) {
      p.top_ids = a.top_ids + r0 * a.top_k;
      p.top_logp = a.top_logp + r0 * a.top_k;
    }
    // four rows a workgroup share each load of the scale, once there are
    // workgroups enough
    const bool many = SCALED && a.rows >= 4096;
    if constexpr (SCALED) {
      if (many)
        logprob_rows_kernel<F32, true, 4>
            <<<(int)((p.rows + 3) / 4), 256, (size_t)4 * chunks * 12, stream>>>(p, chunks);
    }
    if (!many)
      logprob_rows_kernel<F32, SCALED, 1><<<(int)p.rows, 256, (size_t)chunks * 12, stream>>>(p, chunks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_logprob_rows(bool f32, const LogprobArgs& a, void* workspace,
                               hipStream_t stream) {
  if (f32)
    return a.scale != nullptr ? run_logprob<true, true>(a, workspace, stream)
                              : run_logprob<true, false>(a, workspace, stream);
  return a.scale != nullptr ? run_logprob<false, true>(a, workspace, stream)
                            : run_logprob<false, false>(a, workspace, stream);
}

// ------------------------------------------------------------- the gradient
//
//   dz = tau (dlogp [j = label] - p (dlogp + dentropy (log p + entropy)))
//
// Given lse, every element stands by itself.  A workgroup takes a strip of
// columns (16 bytes a thread) down a tile of rows, so a column's scale is
// loaded, and its gradient summed, once per tile; the tiles' sums go to the
// workspace and are added in order by a second kernel.  What a row needs is
// folded into five numbers in LDS:  d = p (gh lp + c), lp = z - lse.  Bound by
// memory: 8,192 x 131,072 bf16 with dscale in 801 us (5.4 TB/s; 777 on another
// GPU); eight rows loaded together where the logits stream (844 us with four),
// four where they come from the cache (15.5 against 16.8 us for 509 x 32,003).
//
// lp is clamped at -200, where p is 0, and x and the scale at the largest
// finite value where d multiplies them, so that a masked token's 0 * inf does
// not arise; c is NaN where lse is, so that row's NaN is kept.

// An infinity as the largest finite value of its sign.
__device__ __forceinline__ float lp_finite(float v) {
  return __builtin_amdgcn_fmed3f(v, -0x1.fffffep127f, 0x1.fffffep127f);
}

struct LpRowGrad {
  float lse, gh, c, hot;       // hot: tau dlogp, added at the label
  int label;
};

__device__ __forceinline__ LpRowGrad lp_row_grad(const LogprobGradArgs& a, int64_t row) {
  LpRowGrad r;
  r.label = lp_label(a.labels, a.label_bytes, row, a.vocab);
  r.lse = a.lse[row];
  const float g = a.dlogp != nullptr && r.label >= 0 ? a.dlogp[row] * a.inv_temp : 0.f;
  const float h = a.dentropy != nullptr ? a.dentropy[row] * a.inv_temp : 0.f;
  r.gh = -h;
  r.c = a.dentropy != nullptr ? -__builtin_fmaf(h, a.entropy[row], g) : -g;
  r.hot = g;
  if (r.lse != r.lse) r.c = r.lse;
  // Past 2^24 fp32 holds the row's maximum, but no log of the sum beside it: p
  // comes out 1 for every token at the maximum.  That is right where one token
  // holds it alone.  An entropy below log 2 = 0.693 says so: n tokens that share
  // the maximum have log n at least.  Any other row (a finite mask over every
  // token; and every token masked, lse -inf) has no gradient.
  if (fabsf(r.lse) >= 0x1p24f &&
      !(a.entropy != nullptr && a.entropy[row] < 0.6875f && fabsf(r.lse) < __builtin_inff())) {
    r.lse = __builtin_inff();
    r.hot = 0.f;
  }
  return r;
}

constexpr int kLpTileRows = 32;                       // most rows of a tile

// A thread's 16 bytes.  STREAM: the logits do not fit the last-level cache, so
// their loads are non-temporal (869 against 885 us for 4.3 GB in and out);
// smaller ones are read through it, where their producer left them (15.0
// against 18.0 us for 65 MB).  Stores are non-temporal either way (a cached
// store: 19.5 us).
template <bool F32, bool STREAM>
struct LpVec {
  static constexpr int VE = F32 ? 4 : 8;
  using V = typename std::conditional<F32, u32x4_a4, u32x4_a2>::type;
  using E = typename std::conditional<F32, uint32_t, uint16_t>::type;

  static __device__ __forceinline__ u32x4_t load(const void* x, int64_t at, int c, int vocab) {
    const E* p = static_cast<const E*>(x) + at + c;
    if (c + VE <= vocab) {
      if constexpr (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
      else return *reinterpret_cast<const V*>(p);
    }
    uint32_t e[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k) e[k] = c + k < vocab ? (uint32_t)p[k] : 0u;
    if constexpr (F32) return u32x4_t{e[0], e[1], e[2], e[3]};
    else return u32x4_t{e[0] | e[1] << 16, e[2] | e[3] << 16, e[VE - 4] | e[VE - 3] << 16,
                        e[VE - 2] | e[VE - 1] << 16};
  }

  static __device__ __forceinline__ void store(void* x, int64_t at, int c, int vocab, u32x4_t t) {
    E* p = static_cast<E*>(x) + at + c;
    if (c + VE <= vocab) {
      __builtin_nontemporal_store(t, reinterpret_cast<V*>(p));
      return;
    }
#pragma unroll
    for (int k = 0; k < VE; ++k)
      if (c + k < vocab) p[k] = (E)(F32 ? t[k] : t[k / 2] >> (16 * (k % 2)));
  }

  static __device__ __forceinline__ float get(u32x4_t t, int k) {
    if constexpr (F32) return __uint_as_float(t[k]);
    else return k % 2 == 0 ? bf_lo(t[k / 2]) : bf_hi(t[k / 2]);
  }

  static __device__ __forceinline__ u32x4_t put(const float (&d)[VE]) {
    if constexpr (F32)
      return u32x4_t{__float_as_uint(d[0]), __float_as_uint(d[1]), __float_as_uint(d[2]),
                     __float_as_uint(d[3])};
    else
      return u32x4_t{pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]), pack_bf16(d[VE - 4], d[VE - 3]),
                     pack_bf16(d[VE - 2], d[VE - 1])};
  }
};

template <bool F32, bool SCALED, bool STREAM>
__global__ void __launch_bounds__(256)
logprob_grad_kernel(const LogprobGradArgs a, int strips, int tile_rows, float* parts) {
  using L = LpVec<F32, STREAM>;
  constexpr int VE = L::VE, AHEAD = STREAM ? 8 : 4;   // rows loaded together
  __shared__ LpRowGrad rg[kLpTileRows];
  const int64_t tile = blockIdx.x / strips;
  const int c0 = (int)(blockIdx.x % strips) * 256 * VE;
  const int c = c0 + threadIdx.x * VE;
  const int64_t row0 = tile * tile_rows;
  const int rows = (int)(a.rows - row0 < tile_rows ? a.rows - row0 : tile_rows);
  if ((int)threadIdx.x < rows) rg[threadIdx.x] = lp_row_grad(a, row0 + threadIdx.x);
  float sc[VE], sum[VE] = {};
#pragma unroll
  for (int k = 0; k < VE; ++k) sc[k] = SCALED && c + k < a.vocab ? a.scale[c + k] : 1.f;
  __syncthreads();
  if (c >= a.vocab) return;
  // whole tiles begin in turn at each of their groups of rows: workgroups that
  // run side by side are then not all at the same address modulo a power of
  // two (801 against 822 us for 8,192 x 131,072)
  const int turn = rows == tile_rows ? (int)(tile % (rows / AHEAD)) * AHEAD : 0;
  for (int q0 = 0; q0 < rows; q0 += AHEAD) {
    const int r0 = q0 + turn < rows ? q0 + turn : q0 + turn - rows;
    u32x4_t t[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (r0 + i < rows) t[i] = L::load(a.x, (row0 + r0 + i) * a.ld, c, a.vocab);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (r0 + i >= rows) break;
      const LpRowGrad r = rg[r0 + i];
      float d[VE];
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        float z = L::get(t[i], k);
        if constexpr (SCALED) z = z * sc[k];
        if (a.inv_temp != 1.f) z = z * a.inv_temp;
        const float lp = fmaxf(z - r.lse, -200.f);
        d[k] = lp_exp(lp) * __builtin_fmaf(r.gh, lp, r.c);
      }
      if (r.label >= c0 && r.label < c0 + 256 * VE) {               // uniform
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          float z = L::get(t[i], k);
          if constexpr (SCALED) z = z * sc[k];
          if (c + k == r.label && z * a.inv_temp > -__builtin_inff()) d[k] += r.hot;
        }
      }
      if constexpr (SCALED) {
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          if (parts != nullptr)
            sum[k] = __builtin_fmaf(d[k], lp_finite(L::get(t[i], k)), sum[k]);
          d[k] = d[k] * lp_finite(sc[k]);
        }
      }
      L::store(a.dx, (row0 + r0 + i) * a.ldo, c, a.vocab, L::put(d));
    }
  }
  if constexpr (SCALED) {
    if (parts != nullptr) {
#pragma unroll
      for (int k = 0; k < VE; ++k)
        if (c + k < a.vocab) parts[tile * a.vocab + c + k] = sum[k];
    }
  }
}

// Adds the tiles' column sums, in order and in fp64: millions of rows are tens
// of thousands of tiles, and an fp32 sum would lose what is below 2^-24 of it at
// every step (2^25 rows of one sign: 3e-5 of dscale).  It costs 1.4 us of the
// gradient's 72 for 8,192 x 4,096 (one addition after another; by pairs the
// same), nothing measurable for 8,192 x 131,072.
__global__ void __launch_bounds__(64)
logprob_scale_sum_kernel(const float* parts, int64_t tiles, int vocab, float* dscale) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= vocab) return;
  double t = 0.;
#pragma unroll 8
  for (int64_t i = 0; i < tiles; ++i) t += parts[i * vocab + c];
  dscale[c] = (float)t;
}

static int lp_strips(bool f32, int64_t vocab) {
  const int64_t w = f32 ? 1024 : 2048;
  return (int)((vocab + w - 1) / w);
}

// Rows of a tile: 8 to 32, about 2,048 workgroups in all.  (8,192 x 131,072
// bf16 on one GPU: 777 us with tiles of 32, 820 with 16 or 64; 864 with 128.)  A rule of the
// sizes alone (the type's strip width aside: bf16's, the wider, counts for
// both), so the order of dscale's sums is too.
static int lp_tile_rows(int64_t rows, int64_t vocab) {
  const int64_t want = rows * lp_strips(false, vocab) / 2048;
  int t = 8;
  while (t < kLpTileRows && t < want) t *= 2;
  return t;
}

int64_t logprob_grad_workspace(int64_t rows, int64_t vocab) {
  const int t = lp_tile_rows(rows, vocab);
  return (rows + t - 1) / t * vocab * 4;
}

template <bool F32, bool SCALED>
static hipError_t run_logprob_grad(const LogprobGradArgs& a, float* parts, hipStream_t stream) {
  const int strips = lp_strips(F32, a.vocab), t = lp_tile_rows(a.rows, a.vocab);
  const int64_t tiles = (a.rows + t - 1) / t;
  const bool large = a.rows * a.vocab > (256 << 20) / (F32 ? 8 : 4);   // in and out: 256 MiB
  // launches of at most 2^20 tiles' strips (a grid's limit is 2^31 threads)
  const int64_t most = std::max<int64_t>(1, (1 << 20) / strips);
  for (int64_t t0 = 0; t0 < tiles; t0 += most) {
    const int64_t n = std::min(most, tiles - t0), r0 = t0 * t;
    LogprobGradArgs p = a;
    p.rows = std::min(n * t, a.rows - r0);
    p.x = static_cast<const char*>(a.x) + r0 * a.ld * (F32 ? 4 : 2);
    p.dx = static_cast<char*>(a.dx) + r0 * a.ldo * (F32 ? 4 : 2);
    if (a.labels != nullptr) p.labels = static_cast<const char*>(a.labels) + r0 * a.label_bytes;
    p.lse = a.lse + r0;
    if (a.entropy != nullptr) p.entropy = a.entropy + r0;
    if (a.dlogp != nullptr) p.dlogp = a.dlogp + r0;
    if (a.dentropy != nullptr) p.dentropy = a.dentropy + r0;
    float* to = parts != nullptr ? parts + t0 * a.vocab : nullptr;
    if (large)
      logprob_grad_kernel<F32, SCALED, true><<<(int)(n * strips), 256, 0, stream>>>(p, strips, t, to);
    else
      logprob_grad_kernel<F32, SCALED, false><<<(int)(n * strips), 256, 0, stream>>>(p, strips, t, to);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dscale == nullptr) return hipSuccess;        // (no rows: no parts, and zeros)
  logprob_scale_sum_kernel<<<(a.vocab + 63) / 64, 64, 0, stream>>>(parts, tiles, a.vocab, a.dscale);
  return hipGetLastError();
}

hipError_t launch_logprob_rows_backward(bool f32, const LogprobGradArgs& a, void* workspace,
                                        hipStream_t stream) {
  float* parts = a.dscale != nullptr ? static_cast<float*>(workspace) : nullptr;
  if (f32)
    return a.scale != nullptr ? run_logprob_grad<true, true>(a, parts, stream)
                              : run_logprob_grad<true, false>(a, parts, stream);
  return a.scale != nullptr ? run_logprob_grad<false, true>(a, parts, stream)
                            : run_logprob_grad<false, false>(a, parts, stream);
}

}  // namespace dsr
