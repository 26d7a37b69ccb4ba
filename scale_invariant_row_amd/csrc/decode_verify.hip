// Drafted tokens against a model's probabilities, from given random numbers.
//
//   p = softmax(target row), q = softmax(draft row)      in fp64
//   accept d_i while u_i q_i(d_i) < p_i(d_i); then the first j with
//   sum_{k <= j} w_k > u sum w,  w = max(p - q, 0)
// The first launch sums exp over slices of every row.  In the last a workgroup
// takes a part of the one row that its sequence's token is sampled from and sums
// w over it; the last workgroup of a sequence to finish finds the part that the
// random number falls into, and the token in it.  (Which row that is, a few
// numbers decide, in the last launch or one before it.)
//
// fp64, because a token's choice hangs on every border of the cumulated
// distribution at once: with weights known to 1e-7 and a vocabulary of 1e5,
// about one choice in a thousand would fall on the other side of a border.
// That makes it bound by the ALUs: 25 instructions an element, 13 of them fp64
// (at fp32's rate), are 47 us of the first launch's 61 over 576 rows of 131,072
// bf16 logits (151 MB), and 10 of the last's 32.  Rows that end within a slice take
// longer (load_as).
#include "decode_launch.hpp"
#include "powers_of_two.hpp"
#include "row_kernels.hpp"

namespace dsr {

constexpr int kSlice = 8192;          // columns a workgroup of the first launch takes
constexpr int kPart = 4096;           // and of the last
constexpr int kSumThreads = 256, kPickThreads = 512;   // 256 at least: they fill ExpTable
constexpr int kMaxRowsPerSeq = 72;    // >= 2 DS_MAX_DRAFTS + 1
constexpr int kMaxSlices = 128;       // DS_MAX_VOCAB / kSlice
constexpr int kMaxParts = 256;        // DS_MAX_VOCAB / kPart

// What a slice of a row sums to: exp(z - m) over it, m its largest.  A NaN or
// +infinity makes sum NaN; a slice masked whole has m -infinity and sum 0.
struct Slice {
  float m, pad;
  double sum;
};

typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));
typedef f32x4_t f32x4_a4 __attribute__((aligned(4)));

__device__ __forceinline__ float scaled(const VerifyArgs& a, int which, float x, int col) {
  return (a.scale[which] != nullptr ? x * a.scale[which][col] : x) * a.inv_temp[which];
}

__device__ __forceinline__ float logit(const VerifyArgs& a, int which, int64_t row, int col) {
  const float x = a.f32[which] ? ((const float*)a.x[which])[row * a.ld[which] + col]
                               : bf_lo(((const uint16_t*)a.x[which])[row * a.ld[which] + col]);
  return scaled(a, which, x, col);
}

// N vectors of 8 scaled logits, the i-th from column col + i * step on, -infinity
// past the vocabulary.  `whole`: none is past it (the same for the workgroup).
// There all loads are asked for before any value is used; rows may have any alignment
// (global loads do not need theirs).  Where the row ends within, each column is loaded
// under a condition and waited for by itself, and the launch lasts as long as those
// workgroups: 576 rows of 128,256 take 164 us, of 131,072 (16 whole slices) 55.
template <int N, bool F32, bool SCALED>
__device__ __forceinline__ void load_as(const VerifyArgs& a, int which, int64_t row, int col, int step, bool whole,
                                        float (&z)[N][8]) {
  const float* scale = a.scale[which];
  const float inv_temp = a.inv_temp[which];
  if (whole) {
    u32x4_t raw[N][F32 ? 2 : 1];
    f32x4_t f[N][SCALED ? 2 : 1];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t at = row * a.ld[which] + col + i * step;
      if constexpr (F32) {
        const float* p = (const float*)a.x[which] + at;
        raw[i][0] = __builtin_bit_cast(u32x4_t, (f32x4_t) * (const f32x4_a4*)p);
        raw[i][1] = __builtin_bit_cast(u32x4_t, (f32x4_t) * (const f32x4_a4*)(p + 4));
      } else {
        raw[i][0] = *(const u32x4_a2*)((const uint16_t*)a.x[which] + at);
      }
      if constexpr (SCALED) {
        f[i][0] = *(const f32x4_a4*)(scale + col + i * step);
        f[i][1] = *(const f32x4_a4*)(scale + col + i * step + 4);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (F32)
          z[i][j] = __uint_as_float(raw[i][j / 4][j % 4]);
        else
          z[i][j] = j % 2 ? bf_hi(raw[i][0][j / 2]) : bf_lo(raw[i][0][j / 2]);
        z[i][j] = (SCALED ? z[i][j] * f[i][j / 4][j % 4] : z[i][j]) * inv_temp;
      }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = col + i * step + j;
        z[i][j] = c < a.vocab ? logit(a, which, row, c) : -__builtin_inff();
      }
  }
}

template <int N>
__device__ __forceinline__ void load_logits(const VerifyArgs& a, int which, int64_t row, int col, int step, bool whole,
                                            float (&z)[N][8]) {
  if (a.f32[which]) {
    if (a.scale[which] != nullptr)
      load_as<N, true, true>(a, which, row, col, step, whole, z);
    else
      load_as<N, true, false>(a, which, row, col, step, whole, z);
  } else {
    if (a.scale[which] != nullptr)
      load_as<N, false, true>(a, which, row, col, step, whole, z);
    else
      load_as<N, false, false>(a, which, row, col, step, whole, z);
  }
}

// exp to fp64's precision: with k ln 2 / 256 next to d and r what is left of d,
// 2^(k / 256) from a table in LDS times exp(r) to its fourth power.  Off by at most
// (2 + |d| / 3) 2^-53 of itself: half a unit each for the table and the last
// rounding, 0.4 for the fifth power at half a step, (ln 2 / 512)^5 / 120, and 0.3 |d|
// for ln 2 / 256 in one part.  13 fp64 instructions an element, a sum among them; a
// table of 128 and a cubic, 12, are 2.2e-12 off and take as long.
struct ExpTable {
  double t[256];
  static_assert(kSumThreads >= 256 && kPickThreads >= 256);
  __device__ __forceinline__ void fill() {               // by 256 threads at least; a barrier follows
    if (threadIdx.x < 256) t[threadIdx.x] = kPowersOfTwo[threadIdx.x];
  }
  // exp(z - m) for z <= m, m finite
  __device__ __forceinline__ double operator()(float z, float m) const {
    constexpr double kPer = 369.3299304675746;           // 256 / ln 2
    constexpr double kStep = 0.0027076061740622863;      // ln 2 / 256
    constexpr double kMagic = 6755399441055744.0;        // 1.5 * 2^52: the sum's low bits are the whole number
    const double d = fmax((double)z - (double)m, -800.0);   // exp(-800) is 0, and so is a masked token's
    const double y = __builtin_fma(d, kPer, kMagic);
    const double r = __builtin_fma(kMagic - y, kStep, d);
    const int k = (int)__builtin_bit_cast(int64_t, y);
    double v = __builtin_fma(r, 1.0 / 24.0, 1.0 / 6.0);
    v = __builtin_fma(v, r, 0.5);
    v = __builtin_fma(v, r, 1.0);
    const double from = t[k & 255];
    v = __builtin_fma(from, v * r, from);
    return __builtin_amdgcn_ldexp(v, k >> 8);
  }
};

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Sums of the lanes up to this one.
__device__ __forceinline__ double wave_scan_f64(double v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double t = __shfl_up(v, d);
    if (lane >= d) v += t;
  }
  return v;
}

// Row r of a sequence: its target rows, then its draft rows.
__global__ void __launch_bounds__(kSumThreads) verify_sums_kernel(const VerifyArgs a, Slice* slices, uint32_t* done,
                                                          int rows_per_seq, int n_slices) {
  __shared__ ExpTable table;
  __shared__ float tops[4];
  __shared__ double sums[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t id = blockIdx.x;
  const int slice = (int)(id % n_slices);
  const int64_t row = id / n_slices, seq = row / rows_per_seq;
  const int r = (int)(row % rows_per_seq), which = r > a.drafts;
  const int64_t at = which ? seq * a.drafts + r - a.drafts - 1 : seq * (a.drafts + 1) + r;
  if (slice == 0 && r == 0 && threadIdx.x == 0) done[seq] = 0;   // for the second launch
  constexpr int kVecs = kSlice / kSumThreads / 8;
  float z[kVecs][8], top = -__builtin_inff();
  load_logits(a, which, at, slice * kSlice + (int)threadIdx.x * 8, kSumThreads * 8, (slice + 1) * kSlice <= a.vocab, z);
  table.fill();
#pragma unroll
  for (int i = 0; i < kVecs * 8; ++i) top = __builtin_elementwise_maximum(top, z[i / 8][i % 8]);   // keeps a NaN
  bool odd = !(top < __builtin_inff());
  top = wave_max(top);
  if (lane == 0) tops[wave] = top;
  odd = __syncthreads_or(odd);
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  double sum = 0.0;
  if (top > -__builtin_inff() && !odd) {
#pragma unroll
    for (int i = 0; i < kVecs * 8; ++i) sum += table(z[i / 8][i % 8], top);
  }
  sum = wave_sum_f64(sum);
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    Slice s;
    s.m = odd ? 0.f : top;
    s.pad = 0.f;
    s.sum = odd ? __builtin_nan("") : ((sums[0] + sums[1]) + sums[2]) + sums[3];
    slices[id] = s;
  }
}

// A row's largest logit and sum of exp: p = exp(z - m) / sum.  sum 0: the row
// says nothing (masked whole, or not a number somewhere).
struct Norm {
  float m;
  double sum;
};

// Norms of a sequence's rows, by the whole workgroup: as many rows a wave at a
// time as their slices fit its lanes (the sums of the lanes in one order).
__device__ __forceinline__ void join_slices(const Slice* s, int rows, int n, const ExpTable& table, Norm* norms) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  int width = 1;                                           // lanes a row
  while (width < n && width < 64) width *= 2;
  const int each = 64 / width, i0 = lane & (width - 1);
  for (int r0 = wave * each; r0 < rows; r0 += waves * each) {
    const int r = r0 + lane / width;
    Slice t[kMaxSlices / 64];
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kMaxSlices / 64; ++i) {
      t[i] = Slice{-__builtin_inff(), 0.f, 0.0};
      if (r < rows && i0 + i * 64 < n) t[i] = s[(int64_t)r * n + i0 + i * 64];
      m = fmaxf(m, t[i].m);
    }
    for (int d = width / 2; d > 0; d /= 2) m = fmaxf(m, __shfl_xor(m, d));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kMaxSlices / 64; ++i)
      if (t[i].m > -__builtin_inff()) sum += t[i].sum * table(t[i].m, m);
    for (int d = width / 2; d > 0; d /= 2) sum += __shfl_xor(sum, d);
    if (i0 == 0 && r < rows) norms[r] = Norm{m, sum == sum ? sum : 0.0};
  }
}

// Where a sequence stands after its drafts: how many were accepted (the next
// token comes from that row), whether the one after was refused by a draft row
// that counts, and which token that was.
struct Choice {
  int accepted, refused, token;
  Norm p, q;
};

struct Decision {                     // LDS of the workgroup that decides
  Norm norms[kMaxRowsPerSeq];
  int accepted, refused, token;
};

__device__ __forceinline__ int64_t drafted_id(const VerifyArgs& a, int64_t i) {
  return a.id_bytes == 8 ? ((const int64_t*)a.drafted)[i] : ((const int32_t*)a.drafted)[i];
}

// By the whole workgroup: wave 0's lanes ask for the drafted tokens' logits
// while the waves join the rows' slices, then decide one draft each.
__device__ __forceinline__ Choice decide(const VerifyArgs& a, const Slice* slices, int64_t seq,
                                         int rows_per_seq, int n_slices, const ExpTable& table,
                                         Decision& d) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t id = -1;
  float zp = 0.f, zq = 0.f, u = 0.f;
  if (wave == 0 && lane < a.drafts) {
    id = drafted_id(a, seq * a.drafts + lane);
    u = a.u_accept[seq * a.drafts + lane];
    if (id >= 0 && id < a.vocab) {
      zp = logit(a, 0, seq * (a.drafts + 1) + lane, (int)id);
      if (a.x[1] != nullptr) zq = logit(a, 1, seq * a.drafts + lane, (int)id);
    }
  }
  __syncthreads();                                         // the table is there
  join_slices(slices + seq * rows_per_seq * n_slices, rows_per_seq, n_slices, table, d.norms);
  __syncthreads();
  if (wave == 0) {
    bool ends = true, says = false, ok = false;            // no draft here; its draft row counts; accepted
    if (id >= 0 && id < a.vocab && lane < a.drafts) {
      ends = false;
      const Norm p = d.norms[lane];
      const double pd = p.sum > 0.0 ? table(zp, p.m) / p.sum : 0.0;
      double qd = 1.0;
      says = true;
      if (a.x[1] != nullptr) {
        const Norm q = d.norms[a.drafts + 1 + lane];
        says = q.sum > 0.0;
        if (says) qd = table(zq, q.m) / q.sum;
      }
      ok = says && p.sum > 0.0 && (double)u * qd < pd;     // (a u below 0 is below p = 0 too)
    }
    const uint64_t stops = __builtin_amdgcn_ballot_w64(!ok);   // (lanes past the drafts stop)
    const int first = __builtin_ctzll(stops);
    if (lane == first) {
      d.accepted = lane;
      d.refused = !ends && says;
      d.token = (int)id;
    }
  }
  __syncthreads();
  Choice c;
  c.accepted = d.accepted;
  c.refused = d.refused;
  c.token = d.token;
  c.p = d.norms[c.accepted];
  c.q = Norm{0.f, 1.0};
  if (a.x[1] != nullptr && c.refused) c.q = d.norms[a.drafts + 1 + c.accepted];
  return c;
}

// Calls f(i, j, w, p) for N vectors of 8 columns: each column's weight in the
// distribution that the next token comes from, and the target's own (both 0
// past the vocabulary).
template <int N, class F>
__device__ __forceinline__ void for_weights(const VerifyArgs& a, const Choice& c, const ExpTable& table, int64_t seq,
                                            int col, int step, bool whole, F&& f) {
  if (!(c.p.sum > 0.0)) {
#pragma unroll
    for (int i = 0; i < N * 8; ++i) f(i / 8, i % 8, 0.0, 0.0);
    return;
  }
  float z[N][8], zq[N][8];
  const bool draft = c.refused && a.x[1] != nullptr;
  load_logits(a, 0, seq * (a.drafts + 1) + c.accepted, col, step, whole, z);
  const double inv = 1.0 / c.p.sum, inv_q = 1.0 / c.q.sum;
  if (draft) {
    load_logits(a, 1, seq * a.drafts + c.accepted, col, step, whole, zq);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double p = table(z[i][j], c.p.m) * inv;
        f(i, j, fmax(p - table(zq[i][j], c.q.m) * inv_q, 0.0), p);
      }
  } else {
    const int off = c.refused ? c.token : -1;              // its p - 1 is not above 0
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double p = table(z[i][j], c.p.m) * inv;
        f(i, j, col + i * step + j == off ? 0.0 : p, p);
      }
  }
}

// The part of the row that u times the total falls into (one wave; -1: no weight
// anywhere), what is left of u times the total there, and whether it goes by p.
struct Place {
  int part, whole;
  double left;
};

__device__ __forceinline__ Place find_part(const double* of, int n, double u, int lane) {
  double w[2][kMaxParts / 64], total[2] = {0.0, 0.0};
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < kMaxParts / 64; ++i) {
      w[k][i] = 0.0;
      // written by other workgroups of this launch: past this one's caches
      if (i * 64 + lane < n) w[k][i] = __hip_atomic_load(of + (i * 64 + lane) * 2 + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (i * 64 < n) total[k] += wave_sum_f64(w[k][i]);
    }
  Place at{-1, !(total[0] > 0.0), 0.0};                    // p = q: nothing is left over
  // at or above 1, or NaN: past every sum, whose order may bring one to the total early
  const double edge = u < 1.0 ? u * total[at.whole] : __builtin_inf();
  double before = 0.0;
#pragma unroll
  for (int i = 0; i < kMaxParts / 64; ++i) {
    if (i * 64 >= n) break;
    const double mine = at.whole ? w[1][i] : w[0][i];
    const double upto = before + wave_scan_f64(mine, lane);
    const uint64_t past = __builtin_amdgcn_ballot_w64(mine > 0.0 && upto > edge);
    const uint64_t some = __builtin_amdgcn_ballot_w64(mine > 0.0);
    const int l = past != 0 ? __builtin_ctzll(past) : 63 - __builtin_clzll(some | 1);
    if (past != 0 || some != 0) {                          // the last of any weight, at least
      at.part = i * 64 + l;
      at.left = edge - (__shfl(upto, l) - __shfl(mine, l));
    }
    if (past != 0) break;
    before = __shfl(upto, 63);
  }
  return at;
}

// What is known of a sequence's outputs once its drafts are decided: the count,
// the accepted tokens, -1 past the next one (by the whole workgroup).
__device__ __forceinline__ void write_accepted(const VerifyArgs& a, const Choice& c, int64_t seq, const Norm* norms) {
  const int i = threadIdx.x;
  if (i == 0) a.accepted[seq] = c.accepted;
  if (i > a.drafts || i == c.accepted) return;
  const int64_t at = seq * (a.drafts + 1) + i;
  const int t = i < c.accepted ? (int)drafted_id(a, seq * a.drafts + i) : -1;
  a.tokens[at] = t;
  a.logp[at] = t < 0 ? 0.f : (float)((double)logit(a, 0, at, t) - (double)norms[i].m - log(norms[i].sum));
}

// One workgroup a sequence, where the second launch has many a sequence.
__global__ void __launch_bounds__(kSumThreads) verify_decide_kernel(const VerifyArgs a, const Slice* slices,
                                                                    Choice* choices, int rows_per_seq, int n_slices) {
  __shared__ ExpTable table;
  __shared__ Decision d;
  const int64_t seq = blockIdx.x;
  table.fill();
  const Choice c = decide(a, slices, seq, rows_per_seq, n_slices, table, d);
  write_accepted(a, c, seq, d.norms);
  if (threadIdx.x == 0) choices[seq] = c;
}

// Sums of w (and of p itself) over a part of the row; the last workgroup of a sequence
// picks the token.  DECIDED: the choices are there already.
template <bool DECIDED>
__global__ void __launch_bounds__(kPickThreads) verify_pick_kernel(const VerifyArgs a, const Slice* slices,
                                                                   const Choice* choices, uint32_t* done,
                                                                   double* sums, int rows_per_seq, int n_slices,
                                                                   int n_parts) {
  constexpr int kVecs = kPart / kPickThreads / 8, kWaves = kPickThreads / 64;
  __shared__ ExpTable table;
  __shared__ Decision d;
  __shared__ double part[2][kWaves];
  __shared__ int is_last, found[kWaves], last[kWaves];
  __shared__ Place place;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t seq = blockIdx.x / n_parts;
  const int here = (int)(blockIdx.x % n_parts);
  table.fill();
  Choice c;
  if constexpr (DECIDED) {
    c = choices[seq];
    __syncthreads();                                       // the table is there
  } else {
    c = decide(a, slices, seq, rows_per_seq, n_slices, table, d);
    if (here == 0) write_accepted(a, c, seq, d.norms);
  }
  double ws = 0.0, ps = 0.0;
  for_weights<kVecs>(a, c, table, seq, here * kPart + (int)threadIdx.x * 8, kPickThreads * 8,
                     (here + 1) * kPart <= a.vocab, [&](int, int, double w, double p) {
                       ws += w;
                       ps += p;
                     });
  ws = wave_sum_f64(ws);
  ps = wave_sum_f64(ps);
  if (lane == 0) {
    part[0][wave] = ws;
    part[1][wave] = ps;
  }
  __syncthreads();
  double* of = sums + seq * n_parts * 2;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      double sum = part[k][0];
      for (int i = 1; i < kWaves; ++i) sum += part[k][i];
      __hip_atomic_store(of + here * 2 + k, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    // The sums are stored past this die's caches, and waited for, before the count
    // is added to: who counts last reads them all, past its own caches.  That order
    // is this chip's, not the memory model's, to which relaxed accesses of two places
    // have none: a store of agent scope is counted until it lies where every die reads
    // it.  The wait is an instruction that no access may be moved across, so the source
    // alone keeps it.  (An atomic that releases and acquires whole caches, which the
    // model would ask for, takes 62 us where this takes 34.)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    is_last = __hip_atomic_fetch_add(done + seq, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)n_parts - 1;
  }
  __syncthreads();
  if (!is_last) return;
  if (wave == 0) {
    const double u = (double)a.u_sample[seq];
    const Place at = find_part(of, n_parts, u < 0.0 ? 0.0 : u, lane);
    if (lane == 0) place = at;
  }
  __syncthreads();
  int token = -1;
  if (place.part >= 0) {                                  // a thread's columns in a row, in ascending order
    const int col = place.part * kPart + (int)threadIdx.x * (kVecs * 8);
    double e[kVecs * 8], run = 0.0;
    for_weights<kVecs>(a, c, table, seq, col, 8, (place.part + 1) * kPart <= a.vocab,
                       [&](int i, int j, double w, double p) { run += e[i * 8 + j] = place.whole ? p : w; });
    const double upto = wave_scan_f64(run, lane);
    if (lane == 63) part[0][wave] = upto;
    __syncthreads();
    run = upto - run;
    for (int i = 0; i < wave; ++i) run += part[0][i];
    int hit = 0x7fffffff, any = -1;
#pragma unroll
    for (int i = 0; i < kVecs * 8; ++i) {
      run += e[i];
      if (e[i] > 0.0) {
        any = col + i;
        if (run > place.left && hit == 0x7fffffff) hit = col + i;
      }
    }
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) {
      hit = min(hit, __shfl_xor(hit, k));
      any = max(any, __shfl_xor(any, k));
    }
    if (lane == 0) {
      found[wave] = hit;
      last[wave] = any;
    }
    __syncthreads();
    for (int i = 0; i < kWaves; ++i) {
      hit = min(hit, found[i]);
      any = max(any, last[i]);
    }
    token = hit != 0x7fffffff ? hit : any;
  }
  if (threadIdx.x == 0) {
    const int64_t at = seq * (a.drafts + 1) + c.accepted;
    a.tokens[at] = token;
    a.logp[at] = token < 0 ? 0.f : (float)((double)logit(a, 0, at, token) - (double)c.p.m - log(c.p.sum));
  }
}

static int slices_of(int64_t vocab) { return (int)((vocab + kSlice - 1) / kSlice); }
static int parts_of(int64_t vocab) { return (int)((vocab + kPart - 1) / kPart); }

int64_t verify_slices(int drafts, int64_t vocab, bool with_draft) {
  const int64_t rows = drafts + 1 + (with_draft ? drafts : 0), n = slices_of(vocab);
  return n * (rows > 4 ? rows : 4);   // the last launch's threads too are under a grid's limit
}

// Slices of every row, a choice, two sums for each part of one row, a count.
int64_t verify_workspace(int64_t seqs, int drafts, int64_t vocab, bool with_draft) {
  return seqs * ((drafts + 1 + (with_draft ? drafts : 0)) * (int64_t)slices_of(vocab) * (int64_t)sizeof(Slice) + (int64_t)sizeof(Choice) +
                 parts_of(vocab) * 16 + 4);
}

// With few workgroups in the last launch each decides by itself (one user's 3
// drafts of 32,003 tokens: 10.6 us, against 9.5 + 3.1 and a launch more); with
// more than twice the compute units a launch of its own decides once a sequence
// (64 sequences of 4 drafts of 131,072 tokens: 5.4 + 33.5 us, against 48.5).
hipError_t launch_draft_verify(const VerifyArgs& a, int cus, void* workspace, hipStream_t stream) {
  const int n = slices_of(a.vocab), rows = a.drafts + 1 + (a.x[1] != nullptr ? a.drafts : 0);
  const int parts = parts_of(a.vocab);
  Slice* slices = static_cast<Slice*>(workspace);
  Choice* choices = reinterpret_cast<Choice*>(slices + (int64_t)a.seqs * rows * n);
  double* sums = reinterpret_cast<double*>(choices + a.seqs);
  uint32_t* done = reinterpret_cast<uint32_t*>(sums + (int64_t)a.seqs * parts * 2);
  verify_sums_kernel<<<(uint32_t)((int64_t)a.seqs * rows * n), kSumThreads, 0, stream>>>(a, slices, done, rows, n);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const uint32_t grid = (uint32_t)((int64_t)a.seqs * parts);
  if (grid <= 2u * (uint32_t)cus) {
    verify_pick_kernel<false><<<grid, kPickThreads, 0, stream>>>(a, slices, choices, done, sums, rows, n, parts);
    return hipGetLastError();
  }
  verify_decide_kernel<<<a.seqs, kSumThreads, 0, stream>>>(a, slices, choices, rows, n);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  verify_pick_kernel<true><<<grid, kPickThreads, 0, stream>>>(a, slices, choices, done, sums, rows, n, parts);
  return hipGetLastError();
}

}  // namespace dsr
