// Attention of each sequence's newest tokens over the paged cache.
//
//   z_u = scale <q, K_u>,  lse = log sum exp z_u,  out = sum exp(z_u - lse) V_u
// over the tokens u that a row sees, in one pass: with m about the largest
// z so far, l = sum exp(z - m) and O = sum exp(z - m) V are rescaled when m rises.
//
// The n new tokens of a sequence and the G = q heads / kv heads that share a
// kv head make n G rows over the same keys and values, 16 of them a tile of
// the matrix instruction (16 x 16 x 32): S^T = K Q^T has a lane hold 4 keys of
// one row, which is how P^T has to lie for O^T = V^T P^T, so P (three bf16 parts
// of it, all 24 bits) never leaves its lane.  V^T's 8 keys of one dimension a lane
// come out of LDS transposed (ds_read_tr16).  A wave takes a chunk of a sequence, 32
// keys at a time; the chunks of a sequence are joined by a second kernel.  How a
// sequence is cut goes by its own length alone, so a row's bits do not depend on the
// batch.
//
// Bound by the cache's bytes, each read once for up to 32 rows a kv head (every 32
// more read them again: 35 rows take 134 us where 30 take 89): 64 sequences of up to
// 8,192 tokens over 4 heads of 256 (1.09 GB) take 236 us, 4.6 TB/s, and 10 to join; 4
// of up to 131,072 over 8 heads of 128 in e4m3 (0.67 GB) 132 us, 5.1 TB/s, and 8.5; a
// kernel that only reads reaches 6.0.  A wave issues for a quarter of its time and
// waits for loads for the rest; without the stores of the chunks' sums (35 MB), whose
// acknowledgement the next loads' count waits for, the first takes 214.
#include <algorithm>
#include <type_traits>

#include "decode_launch.hpp"
#include "row_kernels.hpp"

namespace dsr {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kNegInf = -__builtin_inff();
constexpr float kRise = 8.f;         // of z log2 e
constexpr float kReduce = 0x1p-32f;

struct Split {
  float* sums;                       // [row][head][max_chunks][hd]
  float* stats;                      // [row][head][max_chunks][2]: m (of z log2 e), l
  int32_t max_chunks;
  int32_t row_groups;
};

template <class T>
__device__ __forceinline__ T scalar_load(const T* p) {
  return *(const __attribute__((address_space(4))) T*)p;
}

__device__ __forceinline__ Span span_here(const AttendArgs& a, int seq) {
  const int cap = a.cache.pages_per_seq << a.cache.page_shift;
  int len = scalar_load(a.lens + seq);
  len = len < 0 ? 0 : len > cap ? cap : len;
  return span_of(len, a.n_new, a.window, a.cache.heads);
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

__device__ __forceinline__ float scale_of_z(float scale, float k_scale) { return scale * k_scale * kLog2e; }

// log sum exp from m, a maximum of z log2 e, and l.  m carries the roundings of
// z_scale, which the factor back to z takes out again.
__device__ __forceinline__ float lse_of(float m, float l, double scale, float z_scale) {
  if (l == 0.f) return kNegInf;
  const double back = z_scale != 0.f ? scale / (double)z_scale : 0.6931471805599453;
  return (float)((double)m * back + (double)logf(l));
}

// Four e4m3 values as bf16 (exact).
__device__ __forceinline__ u32x2_t widen4(uint32_t w) {
  const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false);
  const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true);
  return u32x2_t{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}

// The work is a list of chunks: of sequence 0 its heads' (and row groups'), one
// after the other, then of sequence 1.  Wave i of W takes the i-th of W equal
// stretches of the list, counted in chunks.  Those hold 128 keys, 256 or, of a
// sequence that would make more than 128 of them, more, so waves that take long
// sequences' chunks are done last: of 4 sequences of 32,768 to 131,072 tokens a wave
// takes 512 to 2,048 keys, and one of 131,072 beside 63 of 100 takes 189 us, alone
// 164.  Each wave finds its place by reading all lengths, 512 at a time, which is most
// of the time of many sequences with hardly a token (16,384 of 8: 550 us).
struct Item {
  int seq, part, c;                  // part: row group * heads + head; c: chunk
  Span span;                         // of the sequence
};

// The number of chunks (of one part) of sequence s0 + lane, 0 past the last.
__device__ __forceinline__ int chunks_of(const AttendArgs& a, int s0, int lane) {
  const int last = a.cache.seqs - 1, cap = a.cache.pages_per_seq << a.cache.page_shift;
  const int len = a.lens[min(s0 + lane, last)];
  const int n = span_of(len < 0 ? 0 : len > cap ? cap : len, a.n_new, a.window, a.cache.heads).n;
  return s0 + lane > last ? 0 : n;
}

// And of the N * 64 sequences from s0 on together, their lengths asked for at once.
template <int N>
__device__ __forceinline__ int chunks_from(const AttendArgs& a, int s0, int lane) {
  int sum = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) sum += chunks_of(a, s0 + i * 64, lane);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  return __builtin_amdgcn_readfirstlane(sum);
}

__device__ __forceinline__ int64_t list_length(const AttendArgs& a, int parts, int lane) {
  if (a.cache.seqs <= 64) return (int64_t)chunks_from<1>(a, 0, lane) * parts;
  int sum = 0;
  for (int s0 = 0; s0 < a.cache.seqs; s0 += 512) sum += chunks_from<8>(a, s0, lane);
  return (int64_t)sum * parts;
}

// The item at place `at` of the list.
__device__ __forceinline__ Item item_at(const AttendArgs& a, int parts, int64_t at, int lane) {
  Item it{0, 0, 0, {}};
  int before = 0, s0 = 0;                                  // chunks of the sequences before s0
  for (; s0 + 64 < a.cache.seqs; s0 += 512) {
    const int sum = chunks_from<8>(a, s0, lane);
    if (at < (int64_t)(before + sum) * parts) break;
    before += sum;
  }
  for (; s0 < a.cache.seqs; s0 += 64) {
    const int n = chunks_of(a, s0, lane);
    int upto = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int t = __shfl_up(upto, d);
      if (lane >= d) upto += t;
    }
    upto += before;
    const uint64_t past = __builtin_amdgcn_ballot_w64(at < (int64_t)upto * parts);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      it.seq = s0 + l;
      before = __builtin_amdgcn_readlane(upto - n, l);
      break;
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  it.span = span_here(a, it.seq);
  const int rest = (int)(at - (int64_t)before * parts);
  it.part = rest / it.span.n;
  it.c = rest % it.span.n;
  return it;
}

// O of one row's head over one chunk, key by key in fp32 (the wave's lanes share
// its dimensions), from its m and l: what the matrix instructions cannot keep
// apart is handed here.  Its sums are kReduce times O (weights reach 2^kRise, a
// chunk 2^23 keys): what is written of them for a join has l < 0.
template <bool E4M3>
__device__ __forceinline__ void plain_row(const AttendArgs& a, const Split& sp, const Item& item, int head, int row,
                                          float m, float l, float z_scale, float v_scale, int lane) {
  const CacheView& cv = a.cache;
  const int hd = cv.hd, G = a.q_heads / cv.heads;
  const int64_t qr = (int64_t)item.seq * a.n_new + row / G;
  const int qh = head * G + row % G;
  const int t = item.span.len - a.n_new + row / G;
  int lo = item.span.start + item.c * item.span.chunk;
  const int hi = min(min(item.span.len, lo + item.span.chunk), t + 1);
  lo = max(lo, item.span.first);
  if (a.window != 0) lo = max(lo, t - a.window + 1);
  auto value = [&](const char* p, int d) {
    if constexpr (E4M3)
      return __builtin_amdgcn_cvt_f32_fp8(*(const uint8_t*)(p + d), 0);
    else
      return bf_lo(*(const uint16_t*)(p + d * 2));
  };
  const float base = m == kNegInf ? 0.f : m;
  float q[4], o[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = i * 64 + lane;
    q[i] = d < hd ? bf_lo(a.q[qr * a.ldq + (int64_t)qh * hd + d]) : 0.f;
  }
  for (int key = lo; key < hi; ++key) {
    const int64_t at = token_bytes_at(cv, cv.table[table_entry(cv, item.seq, key)], key);
    if (at < 0) continue;
    const char* k = cv.k + head * cv.head_bytes + at;
    const char* v = cv.v + head * cv.head_bytes + at;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i * 64 + lane < hd) z = __builtin_fmaf(q[i], value(k, i * 64 + lane), z);
    z = wave_sum(z) * z_scale;
    if (z == kNegInf) continue;                            // masked
    const float p = exp2_fast(z - base) * kReduce;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i * 64 + lane < hd) o[i] += p * value(v, i * 64 + lane);
  }
  const int64_t part_at = (qr * a.q_heads + qh) * sp.max_chunks + item.c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = i * 64 + lane;
    if (d >= hd) continue;
    if (item.span.n == 1)
      a.out[qr * a.ldo + (int64_t)qh * hd + d] = (uint16_t)pack_bf16(l == 0.f ? 0.f : o[i] / (l * kReduce) * v_scale, 0.f);
    else
      sp.sums[part_at * hd + d] = o[i];
  }
  if (item.span.n > 1 && lane == 0) *(f32x2_t*)(sp.stats + part_at * 2) = f32x2_t{m, -l};
}

// HB: head_dim in blocks of 32, rounded up.  RT: tiles of 16 rows a wave.
//
// A wave walks its chunks by blocks of 128 keys, whose places it looks up
// together, a block ahead, and those by tiles of 32, a tile ahead with their
// loads: the next tile's K is asked for as soon as this one's has gone into S,
// its V as soon as this one's is in LDS.  No wave waits for another.
template <int HB, bool E4M3, int RT>
__global__ void __launch_bounds__(256, HB * RT <= 2 ? 3 : HB <= (RT == 1 ? 4 : 2) ? 2 : 1) cache_attention_kernel(const AttendArgs a,
                                                                                    const Split sp) {
  constexpr int HP = HB * 32, DB = HB * 2;                 // padded head_dim; its blocks of 16
  constexpr int VS = HP + 16;                              // bf16 a row of V in LDS: rows start 8 banks apart
  constexpr int VP = E4M3 ? HB : 2 * HB, PPR = E4M3 ? 2 * HB : 4 * HB;   // V's 16-byte pieces a lane, a row
  constexpr int EB = E4M3 ? 1 : 2;                         // bytes an element
  __shared__ __attribute__((aligned(16))) uint16_t v_tiles[4][kTile * VS];
  __shared__ int64_t places[4][2][kBlock];            // byte offset of a key's token
  const int lane = threadIdx.x & 63, col = lane & 15, grp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const CacheView& cv = a.cache;
  const int hd = cv.hd;
  const int G = a.q_heads / cv.heads, rows = G * a.n_new;
  const int parts = cv.heads * sp.row_groups;
  const int64_t total = list_length(a, parts, lane);
  const int64_t id = (int64_t)blockIdx.x * 4 + wave, ids = (int64_t)gridDim.x * 4;
  const int64_t list_lo = total * id / ids, list_hi = total * (id + 1) / ids;
  if (list_lo == list_hi) return;
  Item item = item_at(a, parts, list_lo, lane);
  int left = (int)(list_hi - list_lo);                     // items still to do, this one too

  auto chunk_lo = [](const Item& t) { return t.span.start + t.c * t.span.chunk; };
  auto chunk_hi = [&](const Item& t) { return min(t.span.len, chunk_lo(t) + t.span.chunk); };
  auto next_item = [&](Item& t) {
    if (++t.c < t.span.n) return;
    t.c = 0;
    if (++t.part < parts) return;
    t.part = 0;
    ++t.seq;
    if (t.seq < cv.seqs) t.span = span_here(a, t.seq);
  };
  // A block ahead of the one at work (two, from the last tile of it on): its item,
  // how many items come after that (-1: there is no such block), its first key.
  Item soon;
  int soon_after, soon_k0;
  auto soon_from = [&]() {                                 // on to an item that has keys
    while (soon_after >= 0 && soon_k0 >= chunk_hi(soon)) {
      if (--soon_after < 0) break;
      next_item(soon);
      soon_k0 = chunk_lo(soon);
    }
  };
  // the pages of its keys: this lane's and the 64th after it (of the last key past it)
  int32_t pages[2];
  auto ask_pages = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = min(soon_k0 + i * 64 + lane, soon.span.len - 1);
      pages[i] = cv.table[soon_after >= 0 ? table_entry(cv, soon.seq, key) : 0];
    }
  };
  uint64_t valid[2], soon_valid[2];                        // which keys are in the cache and seen
  int64_t soon_head = 0;                                   // the byte offset of its head
  auto put_places = [&](int64_t* to) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    asm volatile("" : "+v"(pages[0]), "+v"(pages[1]));     // not looked at before this place
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = soon_k0 + i * 64 + lane;
      const int64_t at = soon_after >= 0 && key >= soon.span.first && key < soon.span.len
                             ? token_bytes_at(cv, pages[i], key) : -1;
      to[i * 64 + lane] = at < 0 ? 0 : at;
      soon_valid[i] = __builtin_amdgcn_ballot_w64(at >= 0);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    soon_head = soon_after >= 0 ? (soon.part % cv.heads) * cv.head_bytes : 0;
    // the block after that: its pages are asked for before the tile's K, so they
    // are there when a K is
    soon_k0 += kBlock;
    soon_from();
    ask_pages();
    __builtin_amdgcn_sched_barrier(0);
  };
  typedef std::conditional_t<E4M3, u32x2_t, u32x4_t> kword_t;   // eight values
  kword_t kw[2][HB];                                       // a tile on its way
  u32x4_t vw[VP];
  uint16_t* vt = v_tiles[wave];
  // Every lane loads, one without a key of its own the cache's first token (and
  // dimensions of the head in place of those past it): a load under a condition
  // is waited for at once.  What no row sees is masked where it is used.
  int k_off[2];                                            // the last two blocks of 32 dimensions
#pragma unroll
  for (int i = 0; i < 2; ++i) k_off[i] = min((HB - 2 + i) * 32 + grp * 8, hd - 8) * EB;
  auto ask_k = [&](int64_t head, const int64_t* at) {      // lane (col, grp): key col, dims 8 grp.. of each 32
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const char* p = cv.k + (head + at[half * 16 + col]);
#pragma unroll
      for (int k = 0; k < HB; ++k) {
        if (k >= HB - 2)
          kw[half][k] = *(const kword_t*)(p + k_off[k - HB + 2]);
        else
          kw[half][k] = *(const kword_t*)(p + grp * 8 * EB + k * 32 * EB);
      }
    }
  };
  auto ask_v = [&](int64_t head, const int64_t* at) {      // 16 bytes at a time, rows side by side
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const int piece = i * 64 + lane, d = min(piece % PPR * (16 / EB), hd - 16 / EB);
      vw[i] = *(const u32x4_t*)(cv.v + (head + at[piece / PPR]) + d * EB);
    }
  };
  int buf = 0;                                             // which places are the block's at work
  auto prime = [&]() {                                     // from `item` on
    soon = item;
    soon_after = left - 1;
    soon_k0 = chunk_lo(item);
    soon_from();
    ask_pages();
    put_places(places[wave][buf]);
    // K's loads before V's, as in the loop, and on every way into it: how many
    // younger loads a tile may leave on their way there is the least of them all
    __builtin_amdgcn_sched_barrier(0);
    ask_k(soon_head, places[wave][buf]);
    __builtin_amdgcn_sched_barrier(0);
    ask_v(soon_head, places[wave][buf]);
    __builtin_amdgcn_sched_barrier(0);
  };
  prime();

  int t_row[RT], at_row[RT];                               // this lane's row of each row tile: its token, its
  bf16x8_t q[RT][HB];                                      // place among (row, head) pairs (-1: no row), its q
  int q_seq = -1, q_part = -1;
  while (left > 0) {
    const Span span = item.span;
    const int head = item.part % cv.heads, group0 = item.part / cv.heads * RT;   // first row tile
    if (item.seq != q_seq || item.part != q_part) {
      q_seq = item.seq;
      q_part = item.part;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int row = (group0 + r) * 16 + col;
        const int j = row / G;
        t_row[r] = span.len - a.n_new + j;
        at_row[r] = row < rows ? (item.seq * a.n_new + j) * a.q_heads + head * G + row % G : -1;
        // a row past the last takes the first's values, set to 0
        const uint16_t* p = a.q + ((int64_t)item.seq * a.n_new + (row < rows ? j : 0)) * a.ldq +
                            (int64_t)(head * G + (row < rows ? row % G : 0)) * hd;
#pragma unroll
        for (int k = 0; k < HB; ++k) {
          const int d = k * 32 + grp * 8;
          u32x4_t v = *(const u32x4_t*)(p + min(d, hd - 8));
          if (row >= rows || d >= hd) v = u32x4_t{0, 0, 0, 0};
          q[r][k] = __builtin_bit_cast(bf16x8_t, v);
        }
      }
      __builtin_amdgcn_s_waitcnt(0x0f70);                  // vmcnt(0): nothing younger than V's loads in the loop
    }
    const int last_row = min(rows, (group0 + RT) * 16) - 1;
    const int t_first = span.len - a.n_new + group0 * 16 / G, t_last = span.len - a.n_new + last_row / G;
    const float k_scale = cv.k_scale != nullptr ? scalar_load(cv.k_scale + head) : 1.f;
    const float z_scale = scale_of_z(a.scale, k_scale);
    float m[RT], l[RT];
    f32x4_t o[RT][DB];
    bool odd[RT];                                          // this row is to be summed by itself, below
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      m[r] = kNegInf;
      l[r] = 0.f;
      odd[r] = false;
#pragma unroll
      for (int d = 0; d < DB; ++d) o[r][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    const int hi = chunk_hi(item);
    for (int kb = chunk_lo(item); kb < hi; kb += kBlock) {
      valid[0] = soon_valid[0];
      valid[1] = soon_valid[1];
      const int64_t block_head = soon_head;
      const int tiles = (min(hi - kb, kBlock) + kTile - 1) / kTile;
      for (int tile = 0; tile < tiles; ++tile) {
        const int k0 = kb + tile * kTile;
        const uint32_t keys = (uint32_t)((tile < 2 ? valid[0] : valid[1]) >> (tile % 2 * 32));
        // every row sees every key; there may be keys that some row does not see
        const bool whole = keys == 0xffffffffu && k0 + kTile - 1 <= t_first &&
                           (a.window == 0 || k0 > t_last - a.window);
        const bool mixed = a.n_new > 1 && (k0 + kTile - 1 > t_first || (a.window != 0 && k0 <= t_last - a.window));
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
            if (k >= HB - 2)                               // dimensions past the head: 0, as q is
              if (k * 32 + grp * 8 >= hd) w = u32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int r = 0; r < RT; ++r)
              z[r][half] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w), q[r][k],
                                                                   z[r][half], 0, 0, 0);
          }
        // the next tile, of this block or of the one after it
        if (tile == tiles - 1) put_places(places[wave][buf ^ 1]);
        const int64_t* next = tile == tiles - 1 ? places[wave][buf ^ 1] : places[wave][buf] + (tile + 1) * kTile;
        const int64_t next_head = tile == tiles - 1 ? soon_head : block_head;
        __builtin_amdgcn_sched_barrier(0);
        ask_k(next_head, next);
        __builtin_amdgcn_sched_barrier(0);
        bf16x8_t p[RT][3];                                 // weights: their first, next and last 8 bits
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          float zs[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) zs[i] = z[r][i / 4][i % 4] * z_scale;
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int b = i / 4 * 16 + grp * 4 + i % 4, key = k0 + b;
              const bool seen = ((keys >> b) & 1u) != 0 && key <= t_row[r] &&
                                (a.window == 0 || key > t_row[r] - a.window);
              zs[i] = seen ? zs[i] : kNegInf;
            }
          }
          float top = zs[0];
#pragma unroll
          for (int i = 1; i < 8; ++i) top = fmaxf(top, zs[i]);
          // m follows the largest z only where that is kRise above it: sums stay
          // within 2^kRise of the largest weight, and are rescaled seldom
          top = row_max(top);
          const float m_new = top > m[r] + kRise ? top : m[r];
          const float base = m_new == kNegInf ? 0.f : m_new;
          const float shrink = exp2_fast(m[r] - base);
          m[r] = m_new;
          float sum = 0.f;
          // Three parts hold a weight's 24 bits.  Two, 16 bits, move about one output
          // of 1,000 to a neighbouring bf16 value, and take 235 us instead of 237 over
          // 64 sequences of up to 8,192 tokens, 84 instead of 85.5 with two row tiles.
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float w = exp2_fast(zs[i] - base);
            sum += w;
#pragma unroll
            for (int b = 0; b < 3; ++b) {                  // (the differences are exact)
              p[r][b][i] = (__bf16)w;
              w -= (float)p[r][b][i];
            }
          }
          l[r] = l[r] * shrink + sum;
          if (__builtin_amdgcn_ballot_w64(shrink != 1.f) != 0) {
#pragma unroll
            for (int d = 0; d < DB; ++d) o[r][d] *= shrink;
          }
        }
        // A key that a row does not see must not reach it even as 0 times an
        // infinity.  What is not among the sequence's keys is made zeros; so is one
        // that holds infinities or NaN and that some row does not see, and the rows
        // that see it are summed by themselves.
        if (mixed) {
          const int from = a.window != 0 ? t_last - a.window : -1;
          uint32_t bad_keys = 0;
#pragma unroll
          for (int i = 0; i < VP; ++i) {
            const int b = (i * 64 + lane) / PPR, key = k0 + b;
            bool bad = false;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if constexpr (E4M3) {
#pragma unroll
                for (int k = 0; k < 32; k += 8) bad = bad || ((vw[i][j] >> k) & 0x7fu) == 0x7fu;
              } else {
                bad = bad || (vw[i][j] & 0x7f80u) == 0x7f80u || (vw[i][j] & 0x7f800000u) == 0x7f800000u;
              }
            if (bad && ((keys >> b) & 1u) != 0 && (key > t_first || key <= from)) {
              vw[i] = u32x4_t{0, 0, 0, 0};
              bad_keys |= 1u << b;
            }
          }
          if (__builtin_amdgcn_ballot_w64(bad_keys != 0) != 0) {
#pragma unroll
            for (int i = 32; i > 0; i >>= 1) bad_keys |= __shfl_xor(bad_keys, i);
#pragma unroll
            for (int r = 0; r < RT; ++r)
              for (int b = 0; b < kTile; ++b)
                odd[r] = odd[r] || (((bad_keys >> b) & 1u) != 0 && k0 + b <= t_row[r] &&
                                    (a.window == 0 || k0 + b > t_row[r] - a.window));
          }
        }
        // V into LDS
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < VP; ++i) {
          const int piece = i * 64 + lane;
          uint16_t* to = vt + piece / PPR * VS + piece % PPR * (16 / EB);
          u32x4_t w = vw[i];
          if (keys != 0xffffffffu)
            if (((keys >> (piece / PPR)) & 1u) == 0) w = u32x4_t{0, 0, 0, 0};
          if constexpr (E4M3) {
            const u32x2_t a0 = widen4(w.x), a1 = widen4(w.y), a2 = widen4(w.z), a3 = widen4(w.w);
            ((u32x4_t*)to)[0] = u32x4_t{a0.x, a0.y, a1.x, a1.y};
            ((u32x4_t*)to)[1] = u32x4_t{a2.x, a2.y, a3.x, a3.y};
          } else {
            *(u32x4_t*)to = w;
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_sched_barrier(0);
        ask_v(next_head, next);
        __builtin_amdgcn_sched_barrier(0);
        // and transposed out of it: 16 lanes read 4 keys of 16 dimensions and get
        // them by dimension
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          typedef short s16x8_t __attribute__((ext_vector_type(8)));
          typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
          const uint16_t* from = vt + (grp * 4 + col / 4) * VS + d * 16 + col % 4 * 4;
          const s16x4_t x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)from);
          const s16x4_t x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(from + 16 * VS));
          const s16x8_t x = __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
          const bf16x8_t v = __builtin_bit_cast(bf16x8_t, x);
#pragma unroll
          for (int b = 0; b < 3; ++b)
#pragma unroll
            for (int r = 0; r < RT; ++r)
              o[r][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[r][b], o[r][d], 0, 0, 0);
        }
      }
      buf ^= 1;
    }

    // Rows to be summed by themselves: those whose scores are numbers and whose sums
    // are not finite, for an infinity's products with the parts of a P may cancel
    // to NaN, and a sum of large V may overflow where its quotient by l does not.
    const float v_scale = cv.v_scale != nullptr ? scalar_load(cv.v_scale + head) : 1.f;
    uint32_t alone[RT];                                    // their columns
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      l[r] = row_sum(l[r]);
      float none = 0.f;                                    // NaN if any is not finite
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) none = __builtin_fmaf(o[r][d][i], 0.f, none);
      const uint64_t lanes = __builtin_amdgcn_ballot_w64((odd[r] || none != none) && l[r] == l[r] && at_row[r] >= 0);
      alone[r] = (uint32_t)(lanes | (lanes >> 16) | (lanes >> 32) | (lanes >> 48)) & 0xffffu;
      if (at_row[r] < 0) continue;
      const bool mine = ((alone[r] >> col) & 1u) == 0;
      if (span.n == 1) {
        float inv = l[r] == 0.f ? 0.f : v_scale / l[r];
        if (fabsf(v_scale) < 0x1p-64f) {                   // (uniform) few bits may be left of the quotient
          const float share = l[r] == 0.f ? 0.f : 1.f / l[r];
#pragma unroll
          for (int d = 0; d < DB; ++d) o[r][d] *= share;
          inv = v_scale;
        }
        uint16_t* to = a.out + at_row[r] / a.q_heads * a.ldo + at_row[r] % a.q_heads * hd + grp * 4;
#pragma unroll
        for (int d = 0; d < DB; ++d)
          if (mine && d * 16 < hd)
            *(u32x2_t*)(to + d * 16) = u32x2_t{pack_bf16(o[r][d].x * inv, o[r][d].y * inv),
                                               pack_bf16(o[r][d].z * inv, o[r][d].w * inv)};
        if (grp == 0 && a.lse != nullptr) a.lse[at_row[r]] = lse_of(m[r], l[r], (double)a.scale * k_scale, z_scale);
      } else {
        const int64_t part_at = (int64_t)at_row[r] * sp.max_chunks + item.c;
        float* to = sp.sums + part_at * hd + grp * 4;
#pragma unroll
        for (int d = 0; d < DB; ++d)
          if (mine && d * 16 < hd) *(f32x4_t*)(to + d * 16) = o[r][d];
        if (grp == 0 && mine) *(f32x2_t*)(sp.stats + part_at * 2) = f32x2_t{m[r], l[r]};
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
      for (uint32_t cols = alone[r]; cols != 0; cols &= cols - 1) {
        const int c = __builtin_ctz(cols);
        plain_row<E4M3>(a, sp, item, head, (group0 + r) * 16 + c, __shfl(m[r], c), __shfl(l[r], c), z_scale, v_scale,
                        lane);
      }
    --left;
    next_item(item);
  }
}

// Joins the chunks of a row's head: out = sum w_c O_c with w_c = f_c / sum f_c l_c,
// f_c = exp(m_c - max m).  One workgroup a head; wave w adds chunks w, w + 4, ...
// (bound by latency: 4 us for a row of 8 chunks, 10 for 64 rows of 16 heads).
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
  float m[kMaxChunks / 64], l[kMaxChunks / 64], f[kMaxChunks / 64], top = kNegInf;
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
    f[i] = exp2_fast(m[i] - base);
    sum += f[i] * fabsf(l[i]);
  }
  sum = wave_sum(sum);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < kMaxChunks / 64; ++i)
    if (wave == 0) factor[i * 64 + lane] = f[i] * inv * (l[i] < 0.f ? 1.f / kReduce : 1.f);
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
  const float v_scale = sum == 0.f ? 0.f                   // (0 times an infinite scale)
                        : a.cache.v_scale != nullptr ? a.cache.v_scale[qh / (a.q_heads / a.cache.heads)] : 1.f;
  *(u32x2_t*)(a.out + row * a.ldo + (int64_t)qh * hd + d) =
      u32x2_t{pack_bf16(s.x * v_scale, s.y * v_scale), pack_bf16(s.z * v_scale, s.w * v_scale)};
  if (lane == 0 && a.lse != nullptr) {
    const float k_scale = a.cache.k_scale != nullptr ? a.cache.k_scale[qh / (a.q_heads / a.cache.heads)] : 1.f;
    a.lse[at] = lse_of(top, sum, (double)a.scale * k_scale, scale_of_z(a.scale, k_scale));
  }
}

int64_t attention_workspace(int64_t seqs, int64_t capacity, int q_heads, int heads, int hd, int n_new,
                            int window) {
  const int n = most_chunks(capacity, n_new, window, heads);
  return n == 1 ? 0 : seqs * n_new * q_heads * n * (hd + 2) * 4;
}

// As many workgroups as the chip holds at once (by their registers), or one for
// each chunk, whose waves then lie on as many compute units as they can (96
// chunks: 10.4 us, in a quarter of the workgroups 11.5).  A workgroup that starts
// later would start its loads from nothing.
template <int HB, bool E4M3, int RT>
static void attend(const AttendArgs& a, const Split& sp, int64_t most, int cus, hipStream_t stream) {
  constexpr int kHeld = HB * RT <= 2 ? 3 : HB <= (RT == 1 ? 4 : 2) ? 2 : 1;
  const int grid = (int)std::min<int64_t>(most, (int64_t)cus * kHeld);
  cache_attention_kernel<HB, E4M3, RT><<<grid, 256, 0, stream>>>(a, sp);
}

template <int HB>
static void attend_type(const AttendArgs& a, const Split& sp, int tiles, int64_t most, int cus, hipStream_t stream) {
  if (a.cache.e4m3) {
    if (tiles == 1)
      attend<HB, true, 1>(a, sp, most, cus, stream);
    else
      attend<HB, true, 2>(a, sp, most, cus, stream);
  } else {
    if (tiles == 1)
      attend<HB, false, 1>(a, sp, most, cus, stream);
    else
      attend<HB, false, 2>(a, sp, most, cus, stream);
  }
}

hipError_t launch_cache_attention(const AttendArgs& args, int cus, void* workspace, hipStream_t stream) {
  AttendArgs a = args;
  CacheView& cv = a.cache;
  if (cv.n_pages == 0) {                                   // no token is seen: loads go where some memory is
    cv.k = cv.v = (char*)const_cast<uint16_t*>(a.q);
    cv.head_bytes = 0;
  }
  if (cv.pages_per_seq == 0) cv.table = a.lens;
  const int64_t capacity = (int64_t)cv.pages_per_seq << cv.page_shift;
  const int tiles = (a.q_heads / cv.heads * a.n_new + 15) / 16;
  Split sp;
  sp.max_chunks = most_chunks(capacity, a.n_new, a.window, cv.heads);
  const int64_t heads = (int64_t)cv.seqs * a.n_new * a.q_heads;
  sp.sums = static_cast<float*>(workspace);
  sp.stats = sp.sums + heads * sp.max_chunks * cv.hd;
  sp.row_groups = (tiles + 1) / 2;
  const int64_t most = (int64_t)cv.seqs * cv.heads * sp.row_groups * sp.max_chunks;
  switch ((cv.hd + 31) / 32) {
    case 1: attend_type<1>(a, sp, tiles, most, cus, stream); break;
    case 2: attend_type<2>(a, sp, tiles, most, cus, stream); break;
    case 3: attend_type<3>(a, sp, tiles, most, cus, stream); break;
    case 4: attend_type<4>(a, sp, tiles, most, cus, stream); break;
    case 5:
    case 6: attend_type<6>(a, sp, tiles, most, cus, stream); break;
    case 7:
    case 8: attend_type<8>(a, sp, tiles, most, cus, stream); break;
    default: return hipErrorInvalidValue;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || sp.max_chunks == 1) return e;
  cache_attention_join_kernel<<<(int)heads, 256, 0, stream>>>(a, sp);
  return hipGetLastError();
}

}  // namespace dsr
