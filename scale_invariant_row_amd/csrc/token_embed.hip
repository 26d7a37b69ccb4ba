// Embedding rows by token id, and the table's gradient.
//
//   out_i     = bf16(scale * table[ids_i])          (zeros for an id outside the table)
//   dtable[t] = scale * sum_{i : ids_i = t} dy_i    fp32 sums in ascending i
#include <type_traits>

#include "row_kernels.hpp"
#include "token_launch.hpp"

namespace dsr {

// Token id i, or -1 for one outside [0, vocab).
template <class Id>
__device__ __forceinline__ int32_t token_at(const void* ids, int64_t i, int64_t vocab) {
  const int64_t t = static_cast<const Id*>(ids)[i];
  return t >= 0 && t < vocab ? (int32_t)t : -1;
}

// One wave per row and 16 bytes a lane and load: 4 fp32 or 8 bf16 columns,
// four loads ahead.  The table is read through the caches (frequent tokens come
// again), the rows written past them.  Bound by memory: 32,768 rows of 4,096
// from an fp32 table in 91 us (0.63 GB read and written, 6.9 TB/s).
template <bool F32, class Id>
__global__ void __launch_bounds__(256) embed_rows_kernel(const EmbedArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (row >= a.rows) return;
  const int32_t t = __builtin_amdgcn_readfirstlane(token_at<Id>(a.ids, row, a.vocab));
  const int64_t at = (int64_t)(t < 0 ? 0 : t) * a.cols;
  // an unknown token's buffer holds no bytes: every load returns 0
  const uint32_t bytes = t < 0 ? 0u : (uint32_t)a.cols * (F32 ? 4u : 2u);
  const RowBuf ib(F32 ? (const void*)(static_cast<const float*>(a.table) + at)
                      : (const void*)(static_cast<const uint16_t*>(a.table) + at), bytes);
  const RowBuf ob(a.out + row * a.cols, (uint32_t)a.cols * 2u);
  const float scale = t < 0 ? 0.f : a.scale;               // +0 under a negative scale too
  constexpr int STEP = F32 ? 256 : 512, N = 4;             // columns a load of the wave, loads ahead
  for (int c0 = 0; c0 < a.cols; c0 += STEP * N) {
    f32x4_t x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = ib.ld16f_cached((c0 + i * STEP) * (F32 ? 4 : 2) + lane * 16);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (F32) {
        ob.st8(u32x2_t{pack_bf16(x[i].x * scale, x[i].y * scale),
                       pack_bf16(x[i].z * scale, x[i].w * scale)},
               (c0 + i * STEP) * 2 + lane * 8);
      } else {
        const u32x4_t b = __builtin_bit_cast(u32x4_t, x[i]);
        ob.st16(u32x4_t{pack_bf16(bf_lo(b.x) * scale, bf_hi(b.x) * scale),
                        pack_bf16(bf_lo(b.y) * scale, bf_hi(b.y) * scale),
                        pack_bf16(bf_lo(b.z) * scale, bf_hi(b.z) * scale),
                        pack_bf16(bf_lo(b.w) * scale, bf_hi(b.w) * scale)},
                (c0 + i * STEP) * 2 + lane * 16);
      }
    }
  }
}

hipError_t launch_embed_rows(bool f32, bool wide_ids, const EmbedArgs& a, int grid,
                             hipStream_t stream) {
  if (f32 && wide_ids) embed_rows_kernel<true, int64_t><<<grid, 256, 0, stream>>>(a);
  else if (f32) embed_rows_kernel<true, int32_t><<<grid, 256, 0, stream>>>(a);
  else if (wide_ids) embed_rows_kernel<false, int64_t><<<grid, 256, 0, stream>>>(a);
  else embed_rows_kernel<false, int32_t><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

// ---------------------------------------------------------------- gradient
//
// Three steps: sort the rows by token, clearing the table meanwhile
// (embed_sort_kernel), sum them by blocks of 32 sorted rows
// (embed_sum_kernel), and join the sums of tokens that span blocks
// (embed_join_kernel).  A token's rows are added in ascending order within a
// block and its blocks in order, so the ids fix the order of every sum, and no
// wave takes all rows of a token that occurs often, only its blocks' sums.
//
// Tokens are dealt over `parts` groups, a power of two: token t is number
// t / parts of group t mod parts, so that the frequent low ids of a frequency-
// sorted vocabulary fall into different groups.  Sorted order is by group,
// then token, then row.

constexpr int kSortThreads = 1024;
constexpr int kSortRows = 4;                              // ids a lane holds of a block
constexpr int kSortBlock = kSortThreads * kSortRows;      // 4,096 ids
constexpr int kSortCap = kSortBlock;                      // rows kept in LDS
constexpr int kClearVectors = 8 * kSortThreads;           // cleared by a workgroup: 128 KiB
constexpr int kSortBins = 2048;                           // most tokens of a group
constexpr int kRun = 32;

// The workspace: start[parts * bins + 1] (first sorted row of each token),
// order[rows] and token[rows] (row and token in sorted order), parts of sums
// [blocks of 32 rows][2][cols].
struct EmbedSort {
  int32_t log_parts, bins, bin_bits;
  int32_t* start;
  int32_t* order;
  int32_t* token;
  float* part;
};

// One workgroup per group.  It reads every id, 4,096 at a time, and keeps its
// own rows in LDS in their order (a wave's ids are 256 in a row, so ballots and
// the counts of the waves before give each its place), counting them by token
// and counting the rows of the groups before.  The counts give each token its
// first place; the rows then go to their places in order: ballots over the
// bits of the token's number find a lane's equals among 64 rows, the first of
// them moves the token's cursor for all, and the waves take turns.  Only a
// group of more than 4,096 rows reads the ids a second time.  Reading all ids
// in every workgroup costs parts * rows * 8 bytes from L2 (67 MB for 32,768
// ids); one launch takes the place of the dozen of a device-wide radix sort.
//
// The workgroups past the groups clear the table meanwhile (`vectors` of 16
// bytes; none when the gradient is added to what is there).  The rows of
// tokens that occur are written again (160 MB of 2.1 GB for 32,768 Zipf-like
// ids of 131,072), which costs less than looking up, row by row, which do
// not: together with the sort and the sums 478 us, where a launch that wrote
// zeros or sums token by token took 468 to 517 in its variants, but 32 instead
// of 27 us for 1,021 ids of 50,304 x 768.  In a launch of its own the clearing
// took 351 us and the sort 24 behind it.
template <class Id>
__global__ void __launch_bounds__(kSortThreads, 8)     // 64 VGPRs: two workgroups a compute unit
embed_sort_kernel(const void* ids, int rows, int vocab, const EmbedSort w, u32x4_t* table,
                  int64_t vectors) {
  __shared__ uint32_t cursor[kSortBins];
  __shared__ uint32_t pos[kSortCap];
  __shared__ uint16_t bin[kSortCap];
  __shared__ uint32_t wsum[2][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = blockIdx.x, mask = (1 << w.log_parts) - 1;
  if (group > mask) {
    const int64_t v0 = (int64_t)(group - mask - 1) * kClearVectors + tid;
#pragma unroll
    for (int i = 0; i < kClearVectors / kSortThreads; ++i)
      if (v0 + i * kSortThreads < vectors) table[v0 + i * kSortThreads] = u32x4_t{0u, 0u, 0u, 0u};
    return;
  }
  const uint64_t below = (1ull << lane) - 1;
  int flip = 0;
  // exclusive prefix over the waves of v (uniform in a wave), and the total;
  // one barrier, the two buffers alternate
  auto wave_prefix = [&](uint32_t v, uint32_t& total) {
    if (lane == 0) wsum[flip][wave] = v;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
    for (int i = 0; i < 16; ++i) {
      const uint32_t t = wsum[flip][i];
      before += i < wave ? t : 0;
      total += t;
    }
    flip ^= 1;
    return before;
  };

  for (int i = tid; i < w.bins; i += kSortThreads) cursor[i] = 0;
  __syncthreads();

  // Writes the n rows kept in pos, bin to their places.
  auto flush = [&](uint32_t n) {
    __syncthreads();
    uint32_t p[kSortRows], q[kSortRows];
    uint64_t same[kSortRows];
#pragma unroll
    for (int j = 0; j < kSortRows; ++j) {
      const uint32_t e = wave * 64 * kSortRows + j * 64 + lane;
      p[j] = e < n ? pos[e] : 0;
      q[j] = e < n ? bin[e] : 0;
      same[j] = __builtin_amdgcn_ballot_w64(e < n);
      if (same[j] == 0) continue;
      for (int b = 0; b < w.bin_bits; ++b) {
        const uint64_t ones = __builtin_amdgcn_ballot_w64((q[j] >> b & 1) != 0);
        same[j] &= (q[j] >> b & 1) != 0 ? ones : ~ones;
      }
    }
    const int turns = (int)((n + 64 * kSortRows - 1) / (64 * kSortRows));
    for (int v = 0; v < turns; ++v) {
      if (v == wave) {
        uint32_t at[kSortRows];
#pragma unroll
        for (int j = 0; j < kSortRows; ++j) {
          const bool first = (same[j] & below) == 0 && (same[j] >> lane & 1) != 0;
          at[j] = first ? atomicAdd(&cursor[q[j]], (uint32_t)__builtin_popcountll(same[j])) : 0;
        }
#pragma unroll
        for (int j = 0; j < kSortRows; ++j) {
          const uint32_t base = __shfl(at[j], same[j] != 0 ? __builtin_ctzll(same[j]) : 0);
          if ((same[j] >> lane & 1) != 0) {
            const uint32_t to = base + __builtin_popcountll(same[j] & below);
            w.order[to] = (int32_t)p[j];
            w.token[to] = (int32_t)((q[j] << w.log_parts) | (uint32_t)group);
          }
        }
      }
      __syncthreads();
    }
  };

  // first reading: count, and keep the first 4,096
  uint32_t kept = 0, less = 0;
  int32_t t[kSortRows], next[kSortRows];
  auto read = [&](int base, int32_t (&to)[kSortRows]) {
#pragma unroll
    for (int j = 0; j < kSortRows; ++j) {
      const int64_t i = (int64_t)base + wave * 64 * kSortRows + j * 64 + lane;
      to[j] = i < rows ? token_at<Id>(ids, i, vocab) : -1;
    }
  };
  // the block's rows of this group into pos, bin from `at` on
  uint64_t hits[kSortRows];
  auto place = [&](int base, uint32_t at) {
#pragma unroll
    for (int j = 0; j < kSortRows; ++j) {
      if (hits[j] == 0) continue;
      const uint32_t to = at + __builtin_popcountll(hits[j] & below);
      if ((hits[j] >> lane & 1) != 0 && to < kSortCap) {
        pos[to] = (uint32_t)(base + wave * 64 * kSortRows + j * 64 + lane);
        bin[to] = (uint16_t)(t[j] >> w.log_parts);
      }
      at += __builtin_popcountll(hits[j]);
    }
  };
  auto count = [&]() {
    uint32_t n = 0;
#pragma unroll
    for (int j = 0; j < kSortRows; ++j) {
      hits[j] = __builtin_amdgcn_ballot_w64(t[j] >= 0 && (t[j] & mask) == group);
      n += __builtin_popcountll(hits[j]);
    }
    return n;
  };
  read(0, next);
  for (int64_t base = 0; base < rows; base += kSortBlock) {
#pragma unroll
    for (int j = 0; j < kSortRows; ++j) t[j] = next[j];
    if (base + kSortBlock < rows) read((int)(base + kSortBlock), next);
#pragma unroll
    for (int j = 0; j < kSortRows; ++j) {
      if (t[j] >= 0 && (t[j] & mask) < group) ++less;
      if (t[j] >= 0 && (t[j] & mask) == group) atomicAdd(&cursor[t[j] >> w.log_parts], 1u);
    }
    uint32_t total;
    const uint32_t before = wave_prefix(count(), total);
    if (total == 0) continue;
    place((int)base, kept + before);
    kept += total;
  }
  // rows of the groups before: over the lanes, then the waves
  for (int d = 1; d < 64; d *= 2) less += __shfl_xor(less, d);
  uint32_t base_row;
  (void)wave_prefix(less, base_row);
  // counts -> first sorted row of each token: two tokens a thread
  const uint32_t c0 = 2 * tid < w.bins ? cursor[2 * tid] : 0;
  const uint32_t c1 = 2 * tid + 1 < w.bins ? cursor[2 * tid + 1] : 0;
  uint32_t run = c0 + c1;
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_up(run, d);
    if (lane >= d) run += o;
  }
  uint32_t all;
  const uint32_t ahead = wave_prefix(__builtin_amdgcn_readlane(run, 63), all);
  const uint32_t s0 = base_row + ahead + run - c0 - c1;
  if (2 * tid < w.bins) {
    cursor[2 * tid] = s0;
    w.start[(int64_t)group * w.bins + 2 * tid] = (int32_t)s0;
  }
  if (2 * tid + 1 < w.bins) {
    cursor[2 * tid + 1] = s0 + c0;
    w.start[(int64_t)group * w.bins + 2 * tid + 1] = (int32_t)(s0 + c0);
  }
  if (group == mask && tid == 0) w.start[((int64_t)mask + 1) * w.bins] = (int32_t)(base_row + all);
  if (kept <= kSortCap) {
    flush(kept);
    return;
  }
  kept = 0;
  for (int64_t base = 0; base < rows; base += kSortBlock) {
    read((int)base, t);
    uint32_t total;
    const uint32_t before = wave_prefix(count(), total);
    if (kept + total > kSortCap) {                        // uniform
      flush(kept);
      kept = 0;
    }
    place((int)base, kept + before);
    kept += total;
  }
  flush(kept);
}

// A wave's columns: VE a lane, 4 where the table is fp32 and 8 where it is
// bf16, so that its stores cover 1 KiB without gaps (with 8 columns a lane,
// non-temporal fp32 stores of alternate 16 bytes reached 2.3 TB/s).
template <bool F32, bool ACC>
struct EmbedCols {
  static constexpr int VE = F32 ? 4 : 8;
  using Raw = typename std::conditional<F32, u32x2_t, u32x4_t>::type;   // of a row of dy
  using Old = u32x4_t;                                                  // of a row of the table
  float v[VE];

  static __device__ __forceinline__ Raw load(const EmbedGradArgs& a, int row, int c) {
    const RowBuf b(a.dy + (int64_t)row * a.cols, (uint32_t)a.cols * 2u);
    if constexpr (F32) return b.ld8(c * 2);
    else return b.ld16(c * 2);
  }

  __device__ __forceinline__ void add(Raw x) {
#pragma unroll
    for (int j = 0; j < VE / 2; ++j) {
      v[2 * j] += bf_lo(x[j]);
      v[2 * j + 1] += bf_hi(x[j]);
    }
  }

  // sums of a part of a token's rows, in the workspace
  static __device__ __forceinline__ RowBuf part(const EmbedGradArgs& a, const EmbedSort& w, int k,
                                                int which) {
    return RowBuf(w.part + ((int64_t)k * 2 + which) * a.cols, (uint32_t)a.cols * 4u);
  }
  __device__ __forceinline__ void store_part(const RowBuf& b, int c) const {
#pragma unroll
    for (int h = 0; h < VE; h += 4)
      b.st16(__builtin_bit_cast(u32x4_t, f32x4_t{v[h], v[h + 1], v[h + 2], v[h + 3]}), (c + h) * 4);
  }
  __device__ __forceinline__ void add_part(const RowBuf& b, int c) {
#pragma unroll
    for (int h = 0; h < VE; h += 4) {
      const f32x4_t x = b.ld16f((c + h) * 4);
      v[h] += x.x; v[h + 1] += x.y; v[h + 2] += x.z; v[h + 3] += x.w;
    }
  }

  static __device__ __forceinline__ RowBuf table(const EmbedGradArgs& a, int t) {
    return RowBuf(F32 ? (const void*)(static_cast<float*>(a.dtable) + (int64_t)t * a.cols)
                      : (const void*)(static_cast<uint16_t*>(a.dtable) + (int64_t)t * a.cols),
                  (uint32_t)a.cols * (F32 ? 4u : 2u));
  }
  static __device__ __forceinline__ Old load_old(const EmbedGradArgs& a, int t, int c) {
    return table(a, t).ld16(c * (F32 ? 4 : 2));
  }
  // scale times the sum, plus what was there (if accumulating), to token t
  __device__ __forceinline__ void store(const EmbedGradArgs& a, int t, int c, Old old) const {
    float d[VE];
#pragma unroll
    for (int j = 0; j < VE; ++j) d[j] = v[j] * a.scale;
    if constexpr (F32) {
      if constexpr (ACC) {
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] += __uint_as_float(old[j]);
      }
      table(a, t).st16(__builtin_bit_cast(u32x4_t, f32x4_t{d[0], d[1], d[2], d[3]}), c * 4);
    } else {
      if constexpr (ACC) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          d[2 * j] += bf_lo(old[j]);
          d[VE - 7 + 2 * j] += bf_hi(old[j]);
        }
      }
      table(a, t).st16(u32x4_t{pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]),
                               pack_bf16(d[VE - 4], d[VE - 3]), pack_bf16(d[VE - 2], d[VE - 1])},
                       c * 2);
    }
  }
};

// Sums by blocks of 32 sorted rows: one wave per block and 64 VE columns, all
// its loads in flight together (half of them, where the table's old rows take
// registers too).  The rows of a token that lies in the block give its row of
// the table; of one that came from the block before, part 0 of the block; of
// one that only goes on into the next, part 1.
//
// Bound by memory: for 32,768 x 4,096 (0.43 GB read and written) 96 us.  For
// 1,021 x 768 rows the whole gradient takes 24.0 us with 32 loads together,
// 24.6 with 16 and 25.5 with eight.  Waves that gathered all rows of
// one token, four at a time, needed their whole runs of 32 summed by a launch
// before (28 us) and took 83 us more, held up by the frequent tokens.
template <bool F32, bool ACC>
__global__ void __launch_bounds__(256) embed_sum_kernel(const EmbedGradArgs a, const EmbedSort w, int tiles) {
  constexpr int kAhead = ACC ? kRun / 2 : kRun;          // rows loaded at a time
  using C = EmbedCols<F32, ACC>;
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t block = wave / tiles;
  if (block * kRun >= a.rows) return;
  const int k = (int)block, p0 = k * kRun;
  const int c = (int)(wave % tiles) * (64 * C::VE) + lane * C::VE;   // past the row: loads 0, stores nothing
  // all loads at once: what lies past the known rows is not used
  const int known = __builtin_amdgcn_readfirstlane(w.start[(int64_t)w.bins << w.log_parts]);
  const bool in = p0 + lane < a.rows && lane <= kRun;    // the block and one more
  const int tok = in ? w.token[p0 + lane] : -1;
  const int row = in ? w.order[p0 + lane] : 0;
  const int left = k > 0 ? __builtin_amdgcn_readfirstlane(w.token[p0 - 1]) : -1;
  const int n = min(kRun, known - p0);
  if (n <= 0) return;
  const int next = __shfl_down(tok, 1);
  uint32_t ends = (uint32_t)__builtin_amdgcn_ballot_w64(lane < n && (lane == n - 1 || next != tok));
  const bool from_left = left == __builtin_amdgcn_readlane(tok, 0);
  const bool to_right = n == kRun && p0 + kRun < known &&
                        __builtin_amdgcn_readlane(tok, kRun) == __builtin_amdgcn_readlane(tok, kRun - 1);
  C acc{};
  bool first = true;
#pragma unroll 1
  for (int j0 = 0; j0 < n; j0 += kAhead) {
    typename C::Raw x[kAhead];
    typename C::Old old[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (j0 + j < n) x[j] = C::load(a, __builtin_amdgcn_readlane(row, j0 + j), c);
    if constexpr (ACC) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (ends >> (j0 + j) & 1) old[j] = C::load_old(a, __builtin_amdgcn_readlane(tok, j0 + j), c);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (j0 + j >= n) break;
      acc.add(x[j]);
      if (!(ends >> (j0 + j) & 1)) continue;
      const bool l = first && from_left, r = j0 + j == n - 1 && to_right;
      if (l || r) acc.store_part(C::part(a, w, k, l ? 0 : 1), c);
      else acc.store(a, __builtin_amdgcn_readlane(tok, j0 + j), c, old[j]);
      acc = C{};
      first = false;
    }
  }
}

// Tokens that span blocks: the wave of the block that a token starts in adds
// part 1 of it and part 0 of the blocks that follow, in order.  11 us where the
// most frequent of 32,768 tokens fills some 60 blocks.  A token that fills the
// whole batch is bound by this one wave for each 64 VE columns: 1,023 parts of
// 4,096 columns take 91 us into an fp32 row, 251 into a bf16 one (half the
// waves), beside 119 of sorting (one workgroup places every row) and 45 to 49
// of sums.
template <bool F32, bool ACC>
__global__ void __launch_bounds__(256)
embed_join_kernel(const EmbedGradArgs a, const EmbedSort w, int tiles) {
  using C = EmbedCols<F32, ACC>;
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t block = wave / tiles;
  if ((block + 1) * kRun >= a.rows) return;
  const int k = (int)block, p0 = k * kRun;
  const int known = __builtin_amdgcn_readfirstlane(w.start[(int64_t)w.bins << w.log_parts]);
  // lane 0: the token left of the block; 1 and 2: its first and last; 3: the next
  const int p = lane == 0 ? p0 - 1 : lane == 1 ? p0 : lane == 2 ? p0 + kRun - 1 : p0 + kRun;
  const int tok = p >= 0 ? w.token[p] : -1;
  const int t = __builtin_amdgcn_readlane(tok, 2);
  if (p0 + kRun >= known || __builtin_amdgcn_readlane(tok, 3) != t) return;     // it ends here
  if (__builtin_amdgcn_readlane(tok, 0) == t && __builtin_amdgcn_readlane(tok, 1) == t) return;   // began before
  const int64_t slot = (int64_t)(t & ((1 << w.log_parts) - 1)) * w.bins + (t >> w.log_parts);
  const int last = (__builtin_amdgcn_readfirstlane(w.start[slot + 1]) - 1) / kRun;
  const int c = (int)(wave % tiles) * (64 * C::VE) + lane * C::VE;
  C acc{};
  acc.add_part(C::part(a, w, k, 1), c);
  typename C::Old old{};
  if constexpr (ACC) old = C::load_old(a, t, c);
#pragma unroll 8
  for (int b = k + 1; b <= last; ++b) acc.add_part(C::part(a, w, b, 0), c);
  acc.store(a, t, c, old);
}

static EmbedSort embed_sort_plan(int64_t vocab, int64_t rows, int64_t cols, void* workspace,
                                 int64_t* bytes) {
  EmbedSort w{};
  // up to 256 groups (one workgroup for each compute unit), more only where a
  // group would hold over 2,048 tokens
  while ((1 << w.log_parts) < 256 && (2ll << w.log_parts) <= vocab) ++w.log_parts;
  while ((((int64_t)kSortBins) << w.log_parts) < vocab) ++w.log_parts;
  w.bins = (int32_t)((vocab + (1ll << w.log_parts) - 1) >> w.log_parts);
  while ((1 << w.bin_bits) < w.bins) ++w.bin_bits;
  auto round = [](int64_t n) { return (n + 15) / 16 * 16; };
  const int64_t ns = round((((int64_t)w.bins << w.log_parts) + 1) * 4), nr = round(rows * 4);
  char* p = static_cast<char*>(workspace);
  w.start = reinterpret_cast<int32_t*>(p);
  w.order = reinterpret_cast<int32_t*>(p + ns);
  w.token = reinterpret_cast<int32_t*>(p + ns + nr);
  w.part = reinterpret_cast<float*>(p + ns + 2 * nr);
  *bytes = ns + 2 * nr + (rows + kRun - 1) / kRun * 2 * cols * 4;
  return w;
}

int64_t embed_grad_workspace(int64_t vocab, int64_t rows, int64_t cols) {
  int64_t bytes = 0;
  (void)embed_sort_plan(vocab, rows, cols, nullptr, &bytes);
  return bytes;
}

template <bool F32, bool ACC>
static hipError_t run_embed_grad(const EmbedGradArgs& a, const EmbedSort& w, hipStream_t stream) {
  constexpr int W = 64 * EmbedCols<F32, ACC>::VE;
  const int tiles = (a.cols + W - 1) / W;
  const int64_t waves = ((int64_t)a.rows + kRun - 1) / kRun * tiles;
  embed_sum_kernel<F32, ACC><<<(int)((waves + 3) / 4), 256, 0, stream>>>(a, w, tiles);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.rows <= kRun) return e;
  embed_join_kernel<F32, ACC><<<(int)((waves + 3) / 4), 256, 0, stream>>>(a, w, tiles);
  return hipGetLastError();
}

hipError_t launch_embed_rows_backward(bool f32, bool wide_ids, const EmbedGradArgs& a,
                                      void* workspace, hipStream_t stream) {
  int64_t bytes = 0;
  const EmbedSort w = embed_sort_plan(a.vocab, a.rows, a.cols, workspace, &bytes);
  const int64_t vectors = a.accumulate ? 0 : (int64_t)a.vocab * a.cols / (f32 ? 4 : 8);
  const int grid = (1 << w.log_parts) + (int)((vectors + kClearVectors - 1) / kClearVectors);
  auto* table = static_cast<u32x4_t*>(a.dtable);
  if (wide_ids)
    embed_sort_kernel<int64_t><<<grid, kSortThreads, 0, stream>>>(a.ids, a.rows, a.vocab, w, table, vectors);
  else
    embed_sort_kernel<int32_t><<<grid, kSortThreads, 0, stream>>>(a.ids, a.rows, a.vocab, w, table, vectors);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.rows == 0) return e;
  if (a.accumulate)
    return f32 ? run_embed_grad<true, true>(a, w, stream) : run_embed_grad<false, true>(a, w, stream);
  return f32 ? run_embed_grad<true, false>(a, w, stream) : run_embed_grad<false, false>(a, w, stream);
}

}  // namespace dsr
