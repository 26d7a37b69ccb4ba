// Attention of each sequence's newest tokens over the paged cache.
//
//   z_u = scale <q, K_u>,  lse = log sum exp z_u,  out = sum exp(z_u - lse) V_u
// over the tokens u that a row sees, in one pass: with m the largest z so far,
// l = sum exp(z - m) and O = sum exp(z - m) V are rescaled when m rises.
//
// The n new tokens of a sequence and the G = q heads / kv heads that share a
// kv head make n G rows over the same keys and values, 16 of them a tile of
// the matrix instruction (16 x 16 x 32): S^T = K Q^T has a lane hold 4 keys of
// one row, which is how P^T has to lie for O^T = V^T P^T, so P never leaves its
// lane.  V^T's 8 keys of one dimension a lane come out of LDS transposed
// (ds_read_tr16).  A wave takes 32 keys at a time; a workgroup's four waves
// share out a chunk of the sequence and join at its end; chunks of one sequence
// are joined by a second kernel.  How a sequence is cut goes by its own length
// alone, so a row's bits do not depend on the batch.
#include <algorithm>
#include <type_traits>

#include "decode_launch.hpp"
#include "row_kernels.hpp"

namespace dsr {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kNegInf = -__builtin_inff();

struct Split {
  float* sums;                       // [row][head][max_chunks][hd]
  float* stats;                      // [row][head][max_chunks][2]: m (of z log2 e), l
  int32_t max_chunks;
  int32_t workers;                   // workgroups a sequence, kv head and row group
  int32_t row_groups;
};

__device__ __forceinline__ int32_t scalar_load(const int32_t* p) {
  return *(const __attribute__((address_space(4))) int32_t*)p;
}

__device__ __forceinline__ Span span_here(const AttendArgs& a, int seq) {
  const int cap = a.cache.pages_per_seq << a.cache.page_shift;
  int len = scalar_load(a.lens + seq);
  len = len < 0 ? 0 : len > cap ? cap : len;
  return span_of(len, a.n_new, a.window);
}

// Maximum and sum over the four lanes that hold a row's keys.
__device__ __forceinline__ float row_max(float v) {
  f32x2_t p = swap16(v);
  p = swap32(fmaxf(p.x, p.y));
  return fmaxf(p.x, p.y);
}
__device__ __forceinline__ float row_sum(float v) {
  f32x2_t p = swap16(v);
  p = swap32(p.x + p.y);
  return p.x + p.y;
}

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// Four e4m3 values as bf16 (exact).
__device__ __forceinline__ u32x2_t widen4(uint32_t w) {
  const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false);
  const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true);
  return u32x2_t{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}

// HB: head_dim in blocks of 32, rounded up.  RT: tiles of 16 rows a workgroup.
//
// A wave walks its tiles of 32 keys, across the chunks of its workgroup, one
// ahead with its loads: the next tile's K is asked for as soon as this one's has
// gone into S, its V as soon as this one's is in LDS, the page of the one after
// before either.  Nothing but the join of a chunk waits for another wave.
template <int HB, bool E4M3, int RT>
__global__ void __launch_bounds__(256, HB * RT <= 4 ? 2 : 1) cache_attention_kernel(const AttendArgs a, const Split sp) {
  constexpr int HP = HB * 32, DB = HB * 2;                 // padded head_dim; its blocks of 16
  constexpr int VS = HP + 16;                              // bf16 a row of V in LDS: rows start 8 banks apart
  constexpr int OS = HP + 4;                               // floats a row of O
  constexpr int VP = E4M3 ? HB : 2 * HB, PPR = E4M3 ? 2 * HB : 4 * HB;   // V's 16-byte pieces a lane, a row
  constexpr int kVBytes = 4 * kTile * VS * 2, kOBytes = 4 * 16 * OS * 4;
  __shared__ __attribute__((aligned(16))) char pool[kVBytes > kOBytes ? kVBytes : kOBytes];
  __shared__ int64_t places[4][kTile];                     // byte offset of a key's token, or -1
  __shared__ float stat[4][RT][16][2];
  const int lane = threadIdx.x & 63, col = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const CacheView& cv = a.cache;
  const int hd = cv.hd;
  int id = blockIdx.x;
  const int worker = id % sp.workers;
  id /= sp.workers;
  const int group0 = id % sp.row_groups * RT;              // first row tile
  id /= sp.row_groups;
  const int head = id % cv.heads, seq = id / cv.heads;
  const Span span = span_here(a, seq);
  // this workgroup's chunks
  const int c_begin = (int)((int64_t)span.n * worker / sp.workers);
  const int c_end = (int)((int64_t)span.n * (worker + 1) / sp.workers);
  if (c_begin == c_end) return;
  const int G = a.q_heads / cv.heads, rows = G * a.n_new;
  if (span.len == 0) {                                     // nothing is seen (and there may be no table)
    const int first = group0 * 16, n = min(rows - first, RT * 16);
    for (int i = threadIdx.x; i < n * hd; i += 256) {
      const int row = first + i / hd, qh = head * G + row % G;
      const int64_t qr = (int64_t)seq * a.n_new + row / G;
      a.out[qr * a.ldo + (int64_t)qh * hd + i % hd] = 0;
      if (i % hd == 0 && a.lse != nullptr) a.lse[qr * a.q_heads + qh] = kNegInf;
    }
    return;
  }

  // this lane's row of each tile: its token, and q as the matrix operand
  int t_row[RT];
  bf16x8_t q[RT][HB];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = (group0 + r) * 16 + col;
    const int j = row / G;
    t_row[r] = span.len - a.n_new + j;
    // a row past the last takes the first's values, set to 0
    const uint16_t* p = a.q + ((int64_t)seq * a.n_new + (row < rows ? j : 0)) * a.ldq +
                        (int64_t)(head * G + (row < rows ? row % G : 0)) * hd;
#pragma unroll
    for (int k = 0; k < HB; ++k) {
      const int d = k * 32 + grp * 8;
      u32x4_t v = *(const u32x4_t*)(p + min(d, hd - 8));
      if (row >= rows || d >= hd) v = u32x4_t{0, 0, 0, 0};
      q[r][k] = __builtin_bit_cast(bf16x8_t, v);
    }
  }
  const int last_row = min(rows, (group0 + RT) * 16) - 1;
  const int t_first = span.len - a.n_new + group0 * 16 / G, t_last = span.len - a.n_new + last_row / G;
  const float z_scale = a.scale * (cv.k_scale != nullptr ? cv.k_scale[head] : 1.f) * kLog2e;
  const float v_scale = cv.v_scale != nullptr ? cv.v_scale[head] : 1.f;
  const char* kbase = cv.k + head * cv.head_bytes;
  const char* vbase = cv.v + head * cv.head_bytes;
  uint16_t* vt = (uint16_t*)pool + wave * kTile * VS;      // this wave's V tile
  int64_t* place = places[wave];

  // The wave's tiles in order: key `first key`, in chunk `c`; c_end past the last.
  struct Tile {
    int c, k0;
  };
  auto chunk_lo = [&](int c) { return span.start + c * span.chunk; };
  auto settle = [&](Tile t) {                              // on to the next chunk that has one
    while (t.c < c_end && t.k0 >= min(span.len, chunk_lo(t.c) + span.chunk)) {
      ++t.c;
      t.k0 = chunk_lo(t.c) + wave * kTile;
    }
    return t;
  };
  auto first_from = [&](int c) { return settle(Tile{c, chunk_lo(c) + wave * kTile}); };
  auto after = [&](Tile t) { return settle(Tile{t.c, t.k0 + 4 * kTile}); };
  // the page of this lane's key (lanes 0..31; of the last key past it)
  auto ask_page = [&](Tile t) {
    return cv.table[table_entry(cv, seq, min(t.k0 + (lane & 31), span.len - 1))];
  };
  typedef std::conditional_t<E4M3, u32x2_t, u32x4_t> kword_t;   // eight values
  kword_t kw[2][HB];                                       // a tile on its way
  u32x4_t vw[VP];
  uint32_t valid = 0;                                      // which of its keys are in the cache and seen
  auto put_places = [&](Tile t, int32_t page) {
    const int key = t.k0 + (lane & 31);
    const int64_t at = t.c < c_end && key >= span.first && key < span.len ? token_bytes_at(cv, page, key) : -1;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    if (lane < 32) place[lane] = at < 0 ? 0 : at;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    return (uint32_t)__builtin_amdgcn_ballot_w64(at >= 0);
  };
  // Every lane loads, one without a key of its own the cache's first token (and
  // the first dimensions in place of those past the head): a load under a
  // condition is waited for at once.  What no row sees is masked where it is used.
  const int past_k = (hd - 1) / 8 * 8;
  auto ask_k = [&]() {                                     // lane (col, grp): key col, dims 8 grp.. of each 32
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const char* at = kbase + place[half * 16 + col];
#pragma unroll
      for (int k = 0; k < HB; ++k) {
        const int d = min(k * 32 + grp * 8, past_k);
        if constexpr (E4M3)
          kw[half][k] = *(const kword_t*)(at + d);
        else
          kw[half][k] = *(const kword_t*)(at + d * 2);
      }
    }
  };
  auto ask_v = [&]() {                                     // 16 bytes at a time, rows side by side
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const int piece = i * 64 + lane, d = piece % PPR * (E4M3 ? 16 : 8);
      vw[i] = *(const u32x4_t*)(vbase + place[piece / PPR] + min(d, hd - (E4M3 ? 16 : 8)) * (E4M3 ? 1 : 2));
    }
  };
  Tile cur = first_from(c_begin), ahead = after(cur);
  int32_t page_ahead;
  auto prime = [&]() {                                     // the loads of `cur`, the page of `ahead`
    const int32_t page = ask_page(cur);
    page_ahead = ask_page(ahead);
    valid = put_places(cur, page);
    // K's loads before V's, as in the loop, and on every way into it: how many
    // younger loads a tile may leave on their way there is the least of them all
    __builtin_amdgcn_sched_barrier(0);
    ask_k();
    __builtin_amdgcn_sched_barrier(0);
    ask_v();
    __builtin_amdgcn_sched_barrier(0);
  };
  prime();

  // A second pass over a chunk is for sums that came out infinite or NaN: where V
  // holds an infinity, its products with the two parts of a P may cancel to NaN,
  // so the lanes with such sums take P rounded to one part there (the others do
  // again what they did).
  bool one_part[RT] = {}, again = false;
  for (int c = c_begin; c < c_end;) {
    float m[RT], l[RT];
    f32x4_t o[RT][DB];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      m[r] = kNegInf;
      l[r] = 0.f;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[r][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    while (cur.c == c) {
      const int k0 = cur.k0;
      const uint32_t seen_keys = valid;
      const bool whole = seen_keys == 0xffffffffu && k0 + kTile - 1 <= t_first &&
                         (a.window == 0 || k0 > t_last - a.window);
      f32x4_t z[RT][2];
#pragma unroll
      for (int r = 0; r < RT; ++r) z[r][0] = z[r][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < HB; ++k)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          u32x4_t w;
          if constexpr (E4M3) {
            const u32x2_t a0 = widen4(kw[half][k].x), a1 = widen4(kw[half][k].y);
            w = u32x4_t{a0.x, a0.y, a1.x, a1.y};
          } else {
            w = kw[half][k];
          }
          if (k == HB - 1 || k == HB - 2)                  // dimensions past the head: 0, as q is
            if (k * 32 + grp * 8 >= hd) w = u32x4_t{0, 0, 0, 0};
#pragma unroll
          for (int r = 0; r < RT; ++r)
            z[r][half] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w), q[r][k],
                                                                 z[r][half], 0, 0, 0);
        }
      // ask for the next tile's K, and the page of the one after it
      cur = ahead;
      ahead = after(cur);
      valid = put_places(cur, page_ahead);
      page_ahead = ask_page(ahead);
      __builtin_amdgcn_sched_barrier(0);
      ask_k();
      __builtin_amdgcn_sched_barrier(0);
      bf16x8_t p_hi[RT], p_lo[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float zs[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) zs[i] = z[r][i / 4][i % 4] * z_scale;
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int b = i / 4 * 16 + grp * 4 + i % 4, key = k0 + b;
            const bool seen = ((seen_keys >> b) & 1u) != 0 && key <= t_row[r] &&
                              (a.window == 0 || key > t_row[r] - a.window);
            zs[i] = seen ? zs[i] : kNegInf;
          }
        }
        float top = zs[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, zs[i]);
        const float m_new = fmaxf(m[r], row_max(top));
        const float base = m_new == kNegInf ? 0.f : m_new;
        const float shrink = exp2_fast(m[r] - base);
        m[r] = m_new;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = exp2_fast(zs[i] - base);
          sum += p;
          p_hi[r][i] = (__bf16)p;
          p_lo[r][i] = (__bf16)(p - (float)p_hi[r][i]);
        }
        l[r] = l[r] * shrink + sum;
#pragma unroll
        for (int d = 0; d < DB; ++d) o[r][d] *= shrink;
      }
      // V into LDS, and transposed out of it
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < VP; ++i) {
        const int piece = i * 64 + lane;
        uint16_t* to = vt + piece / PPR * VS + piece % PPR * (E4M3 ? 16 : 8);
        if constexpr (E4M3) {
          const u32x2_t a0 = widen4(vw[i].x), a1 = widen4(vw[i].y), a2 = widen4(vw[i].z), a3 = widen4(vw[i].w);
          ((u32x4_t*)to)[0] = u32x4_t{a0.x, a0.y, a1.x, a1.y};
          ((u32x4_t*)to)[1] = u32x4_t{a2.x, a2.y, a3.x, a3.y};
        } else {
          *(u32x4_t*)to = vw[i];
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      ask_v();                                             // the next tile's
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        // 16 lanes read 4 keys of 16 dimensions and get them by dimension
        typedef short s16x8_t __attribute__((ext_vector_type(8)));
        typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
        const uint16_t* from = vt + (grp * 4 + col / 4) * VS + d * 16 + col % 4 * 4;
        const s16x4_t x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)from);
        const s16x4_t x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(from + 16 * VS));
        const s16x8_t x = __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
        if (whole) {
          const bf16x8_t v = __builtin_bit_cast(bf16x8_t, x);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            o[r][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p_hi[r], o[r][d], 0, 0, 0);
            const f32x4_t s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p_lo[r], o[r][d], 0, 0, 0);
            o[r][d] = again && one_part[r] ? o[r][d] : s;
          }
        } else {
          // a key that a row does not see must not reach it even as 0 times an
          // infinity: each new token's rows get V with its own keys
          f32x4_t was[RT];
#pragma unroll
          for (int r = 0; r < RT; ++r) was[r] = o[r][d];
          for (int t = t_first; t <= t_last; ++t) {
            s16x8_t y;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int b = i / 4 * 16 + grp * 4 + i % 4, key = k0 + b;
              const bool seen = ((seen_keys >> b) & 1u) != 0 && key <= t && (a.window == 0 || key > t - a.window);
              y[i] = seen ? x[i] : (short)0;
            }
            const bf16x8_t v = __builtin_bit_cast(bf16x8_t, y);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
              const f32x4_t h = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p_hi[r], was[r], 0, 0, 0);
              const f32x4_t s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p_lo[r], h, 0, 0, 0);
              if (t_row[r] == t) o[r][d] = again && one_part[r] ? h : s;
            }
          }
        }
      }
    }

    // join the four waves: their sums into LDS as they are, weighed as they are added
    bool odd = false;
    if (!again) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        one_part[r] = false;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) one_part[r] = one_part[r] || !(fabsf(o[r][d][i]) < __builtin_inff());
        odd = odd || one_part[r];
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      l[r] = row_sum(l[r]);
      if (grp == 0) {
        stat[wave][r][col][0] = m[r];
        stat[wave][r][col][1] = l[r];
      }
    }
    if (__syncthreads_or(odd)) {
      again = true;
      cur = first_from(c);
      ahead = after(cur);
      prime();
      continue;
    }
    again = false;
    float* ob = (float*)pool;                              // [wave][row][OS]
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      if ((group0 + r) * 16 >= rows) break;                // uniform
      if ((group0 + r) * 16 + col < rows) {
#pragma unroll
        for (int d = 0; d < DB; ++d) *(f32x4_t*)(ob + (wave * 16 + col) * OS + d * 16 + grp * 4) = o[r][d];
      }
      __syncthreads();
      const int n_rows = min(16, rows - (group0 + r) * 16);
      for (int i = threadIdx.x; i < n_rows * (HP / 4); i += 256) {
        const int row16 = i / (HP / 4), d = i % (HP / 4) * 4, row = (group0 + r) * 16 + row16;
        if (d >= hd) continue;
        float t = kNegInf, sum = 0.f;
        for (int w = 0; w < 4; ++w) t = fmaxf(t, stat[w][r][row16][0]);
        const float base = t == kNegInf ? 0.f : t;
        f32x4_t s = {0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < 4; ++w) {
          const float f = exp2_fast(stat[w][r][row16][0] - base);
          sum += f * stat[w][r][row16][1];
          s += *(const f32x4_t*)(ob + (w * 16 + row16) * OS + d) * f;
        }
        const int64_t qr = (int64_t)seq * a.n_new + row / G;
        const int qh = head * G + row % G;
        const int64_t at = qr * a.q_heads + qh;
        if (span.n == 1) {
          const float inv = sum == 0.f ? 0.f : v_scale / sum;
          uint16_t* to = a.out + qr * a.ldo + (int64_t)qh * hd + d;
          *(u32x2_t*)to = u32x2_t{pack_bf16(s.x * inv, s.y * inv), pack_bf16(s.z * inv, s.w * inv)};
          if (d == 0 && a.lse != nullptr) a.lse[at] = sum == 0.f ? kNegInf : t * kLn2 + logf(sum);
        } else {
          *(f32x4_t*)(sp.sums + (at * sp.max_chunks + c) * hd + d) = s;
          if (d == 0) {
            sp.stats[(at * sp.max_chunks + c) * 2] = t;
            sp.stats[(at * sp.max_chunks + c) * 2 + 1] = sum;
          }
        }
      }
      __syncthreads();
    }
    ++c;
  }
}

// Joins the chunks of a row's head: out = sum f_c O_c / sum f_c l_c with
// f_c = exp(m_c - max m).  One workgroup a head; wave w adds chunks w, w + 4, ...
__global__ void __launch_bounds__(256) cache_attention_join_kernel(const AttendArgs a, const Split sp) {
  __shared__ float factor[kMaxChunks];
  __shared__ __attribute__((aligned(16))) float part[4][256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t at = blockIdx.x;
  const int qh = (int)(at % a.q_heads);
  const int64_t row = at / a.q_heads;
  const Span span = span_here(a, (int)(row / a.n_new));
  if (span.n == 1) return;                                 // written already
  const float* stats = sp.stats + at * sp.max_chunks * 2;
  float m[kMaxChunks / 64], l[kMaxChunks / 64], top = kNegInf;
#pragma unroll
  for (int i = 0; i < kMaxChunks / 64; ++i) {
    const int c = i * 64 + lane;
    m[i] = c < span.n ? stats[c * 2] : kNegInf;
    l[i] = c < span.n ? stats[c * 2 + 1] : 0.f;
    top = fmaxf(top, m[i]);
  }
  top = wave_max(top);
  const float base = top == kNegInf ? 0.f : top;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxChunks / 64; ++i) {
    const float f = exp2_fast(m[i] - base);
    if (wave == 0) factor[i * 64 + lane] = f;
    sum += f * l[i];
  }
  sum = wave_sum(sum);
  __syncthreads();
  const int hd = a.cache.hd, d = lane * 4;
  f32x4_t s = {0.f, 0.f, 0.f, 0.f};
  if (d < hd) {
    const float* sums = sp.sums + at * sp.max_chunks * hd + d;
#pragma unroll 4
    for (int c = wave; c < span.n; c += 4) s += *(const f32x4_t*)(sums + (int64_t)c * hd) * factor[c];
    *(f32x4_t*)(part[wave] + d) = s;
  }
  __syncthreads();
  if (wave != 0 || d >= hd) return;
  for (int w = 1; w < 4; ++w) s += *(const f32x4_t*)(part[w] + d);
  const float v_scale = a.cache.v_scale != nullptr ? a.cache.v_scale[qh / (a.q_heads / a.cache.heads)] : 1.f;
  const float inv = sum == 0.f ? 0.f : v_scale / sum;
  *(u32x2_t*)(a.out + row * a.ldo + (int64_t)qh * hd + d) =
      u32x2_t{pack_bf16(s.x * inv, s.y * inv), pack_bf16(s.z * inv, s.w * inv)};
  if (lane == 0 && a.lse != nullptr) a.lse[at] = sum == 0.f ? kNegInf : top * kLn2 + logf(sum);
}

int64_t attention_workspace(int64_t seqs, int64_t capacity, int q_heads, int hd, int n_new, int window) {
  const int n = most_chunks(capacity, n_new, window);
  return n == 1 ? 0 : seqs * n_new * q_heads * n * (hd + 2) * 4;
}

template <int HB, bool E4M3>
static void attend(const AttendArgs& a, const Split& sp, int tiles, int grid, hipStream_t stream) {
  if (tiles == 1)
    cache_attention_kernel<HB, E4M3, 1><<<grid, 256, 0, stream>>>(a, sp);
  else
    cache_attention_kernel<HB, E4M3, 2><<<grid, 256, 0, stream>>>(a, sp);
}

template <int HB>
static void attend_type(const AttendArgs& a, const Split& sp, int tiles, int grid, hipStream_t stream) {
  if (a.cache.e4m3)
    attend<HB, true>(a, sp, tiles, grid, stream);
  else
    attend<HB, false>(a, sp, tiles, grid, stream);
}

hipError_t launch_cache_attention(const AttendArgs& args, int cus, void* workspace, hipStream_t stream) {
  AttendArgs a = args;
  CacheView& cv = a.cache;
  if (cv.n_pages == 0) {                                   // no token is seen: loads go where some memory is
    cv.k = cv.v = (char*)const_cast<uint16_t*>(a.q);
    cv.head_bytes = 0;
  }
  const int64_t capacity = (int64_t)cv.pages_per_seq << cv.page_shift;
  const int tiles = (a.q_heads / cv.heads * a.n_new + 15) / 16;
  Split sp;
  sp.max_chunks = most_chunks(capacity, a.n_new, a.window);
  const int64_t heads = (int64_t)cv.seqs * a.n_new * a.q_heads;
  sp.sums = static_cast<float*>(workspace);
  sp.stats = sp.sums + heads * sp.max_chunks * cv.hd;
  sp.row_groups = (tiles + 1) / 2;
  const int64_t pairs = (int64_t)cv.seqs * cv.heads * sp.row_groups;
  sp.workers = (int)std::min<int64_t>(sp.max_chunks, std::max<int64_t>(1, (cus * 16 + pairs - 1) / pairs));
  const int grid = (int)(pairs * sp.workers);
  switch ((cv.hd + 31) / 32) {
    case 1: attend_type<1>(a, sp, tiles, grid, stream); break;
    case 2: attend_type<2>(a, sp, tiles, grid, stream); break;
    case 3: attend_type<3>(a, sp, tiles, grid, stream); break;
    case 4: attend_type<4>(a, sp, tiles, grid, stream); break;
    case 5:
    case 6: attend_type<6>(a, sp, tiles, grid, stream); break;
    case 7:
    case 8: attend_type<8>(a, sp, tiles, grid, stream); break;
    default: return hipErrorInvalidValue;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || sp.max_chunks == 1) return e;
  cache_attention_join_kernel<<<(int)heads, 256, 0, stream>>>(a, sp);
  return hipGetLastError();
}

}  // namespace dsr
