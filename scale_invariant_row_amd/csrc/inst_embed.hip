// Embedding rows by token id, and the table's gradient.
//
//   out_i     = bf16(scale * table[ids_i])          (zeros for an id outside the table)
//   dtable[t] = scale * sum_{i : ids_i = t} dy_i    fp32 sums in ascending i
#include "row_kernels.hpp"
#include "token_launch.hpp"

namespace dsr {

// Token id i, or -1 for one outside [0, vocab).
template <class Id>
__device__ __forceinline__ int32_t token_at(const void* ids, int64_t i, int64_t vocab) {
  const int64_t t = static_cast<const Id*>(ids)[i];
  return t >= 0 && t < vocab ? (int32_t)t : -1;
}

// One wave per row; lane l holds 8 columns of each stretch of 512.
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
  for (int c = lane * 8; c < a.cols; c += 512) {
    float v[8];
    if constexpr (F32) {
      const f32x4_t x = ib.ld16f_cached(c * 4), y = ib.ld16f_cached(c * 4 + 16);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    } else {
      const u32x4_t x = __builtin_bit_cast(u32x4_t, ib.ld16f_cached(c * 2));
      v[0] = bf_lo(x.x); v[1] = bf_hi(x.x); v[2] = bf_lo(x.y); v[3] = bf_hi(x.y);
      v[4] = bf_lo(x.z); v[5] = bf_hi(x.z); v[6] = bf_lo(x.w); v[7] = bf_hi(x.w);
    }
    const u32x4_t o = {pack_bf16(v[0] * a.scale, v[1] * a.scale),
                       pack_bf16(v[2] * a.scale, v[3] * a.scale),
                       pack_bf16(v[4] * a.scale, v[5] * a.scale),
                       pack_bf16(v[6] * a.scale, v[7] * a.scale)};
    ob.st16(o, c * 2);
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
// Three steps: sort the rows by token (embed_sort_kernel), sum every whole
// run of 32 sorted rows that share one token (embed_run_kernel), and write the
// table (embed_table_kernel).  A token's rows are added in ascending order,
// its whole runs by their sums, so the order is fixed by the ids and no token,
// however often it occurs, makes one wave read more than 62 rows and a 32nd
// of the rest.
//
// Tokens are dealt over `parts` groups, a power of two: token t is number
// t / parts of group t mod parts, so that the frequent low ids of a frequency-
// sorted vocabulary fall into different groups.  Sorted order is by group,
// then token, then row.

constexpr int kSortThreads = 1024;
constexpr int kSortRows = 4;                              // ids a lane holds of a block
constexpr int kSortBlock = kSortThreads * kSortRows;      // 4,096 ids
constexpr int kSortCap = kSortBlock;                      // rows sorted at once
constexpr int kSortBins = 2048;                           // most tokens of a group
constexpr int kRun = 32;

// The workspace: start[parts * bins + 1] (first sorted row of each token),
// order[rows] and token[rows] (row and token in sorted order), run sums
// [rows / 32][cols].
struct EmbedSort {
  int32_t log_parts, bins, bin_bits;
  int32_t* start;
  int32_t* order;
  int32_t* token;
  float* run;
};

// One workgroup per group.  It reads every id, 4,096 at a time, and keeps its
// own in LDS in their order (a wave's ids are 256 in a row, so ballots and the
// counts of the waves before give each its place), counting them by token and
// counting the rows of the groups before.  Then a stable sort by token: a
// split by each bit of the token's number.  Only a group of more than 4,096
// rows reads the ids a second time, and sorts 4,096 at a time, each going
// behind what its token already has.  Reading all ids in every workgroup
// costs parts * rows * 8 bytes from L2 (67 MB for 32,768 ids), and one launch
// takes the place of the dozen that a device-wide radix sort would need.
template <class Id>
__global__ void __launch_bounds__(kSortThreads)
embed_sort_kernel(const void* ids, int rows, int vocab, const EmbedSort w) {
  __shared__ uint32_t cursor[kSortBins];
  __shared__ uint32_t pos[2][kSortCap];
  __shared__ uint16_t bin[2][kSortCap];
  __shared__ uint32_t wsum[2][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = blockIdx.x, mask = (1 << w.log_parts) - 1;
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

  // Sorts the n rows in pos[0], bin[0] by token and writes them out behind
  // their tokens' cursors.
  auto flush = [&](uint32_t n) {
    int f = 0;
    __syncthreads();
    for (int b = 0; b < w.bin_bits; ++b) {
      uint32_t p[kSortRows], q[kSortRows];
      uint64_t zeros[kSortRows];
      uint32_t nz = 0;
#pragma unroll
      for (int j = 0; j < kSortRows; ++j) {
        const uint32_t e = wave * 64 * kSortRows + j * 64 + lane;
        p[j] = e < n ? pos[f][e] : 0;
        q[j] = e < n ? bin[f][e] : 0;
        zeros[j] = __builtin_amdgcn_ballot_w64(e < n && ((q[j] >> b) & 1) == 0);
        nz += __builtin_popcountll(zeros[j]);
      }
      uint32_t total;
      uint32_t z = wave_prefix(nz, total);
#pragma unroll
      for (int j = 0; j < kSortRows; ++j) {
        const uint32_t e = wave * 64 * kSortRows + j * 64 + lane;
        const uint32_t mine = z + __builtin_popcountll(zeros[j] & below);   // zeros before e
        const uint32_t to = ((q[j] >> b) & 1) == 0 ? mine : total + e - mine;
        if (e < n) {
          pos[f ^ 1][to] = p[j];
          bin[f ^ 1][to] = (uint16_t)q[j];
        }
        z += __builtin_popcountll(zeros[j]);
      }
      f ^= 1;
      __syncthreads();
    }
    uint32_t first[kSortRows];
#pragma unroll
    for (int j = 0; j < kSortRows; ++j) {
      const uint32_t e = tid + j * kSortThreads;
      if (e >= n) continue;
      const uint32_t q = bin[f][e];
      uint32_t lo = 0, hi = e;                            // first entry of e's token
      while (lo < hi) {
        const uint32_t mid = (lo + hi) / 2;
        if (bin[f][mid] < q) lo = mid + 1;
        else hi = mid;
      }
      first[j] = lo;
      const uint32_t to = cursor[q] + (e - lo);
      w.order[to] = (int32_t)pos[f][e];
      w.token[to] = (int32_t)((q << w.log_parts) | (uint32_t)group);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortRows; ++j) {
      const uint32_t e = tid + j * kSortThreads;
      if (e < n && (e + 1 == n || bin[f][e + 1] != bin[f][e])) cursor[bin[f][e]] += e + 1 - first[j];
    }
    __syncthreads();
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
  // the block's rows of this group into pos[0], bin[0] from `at` on
  auto place = [&](int base, uint32_t at) {
#pragma unroll
    for (int j = 0; j < kSortRows; ++j) {
      const bool mine = t[j] >= 0 && (t[j] & mask) == group;
      const uint64_t hits = __builtin_amdgcn_ballot_w64(mine);
      const uint32_t to = at + __builtin_popcountll(hits & below);
      if (mine && to < kSortCap) {
        pos[0][to] = (uint32_t)(base + wave * 64 * kSortRows + j * 64 + lane);
        bin[0][to] = (uint16_t)(t[j] >> w.log_parts);
      }
      at += __builtin_popcountll(hits);
    }
  };
  auto count = [&]() {
    uint32_t n = 0;
#pragma unroll
    for (int j = 0; j < kSortRows; ++j)
      n += __builtin_popcountll(__builtin_amdgcn_ballot_w64(t[j] >= 0 && (t[j] & mask) == group));
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

// v[VN][8] += the bf16 row at `row`, columns c + 512 k of the lane.
template <int VN>
__device__ __forceinline__ void load_row(u32x4_t (&x)[VN], const uint16_t* dy, int64_t row,
                                         int cols, int c) {
  const RowBuf b(dy + row * cols, (uint32_t)cols * 2u);
#pragma unroll
  for (int k = 0; k < VN; ++k) x[k] = b.ld16((c + 512 * k) * 2);
}

template <int VN>
__device__ __forceinline__ void add_row(float (&acc)[VN][8], const u32x4_t (&x)[VN]) {
#pragma unroll
  for (int k = 0; k < VN; ++k) {
    acc[k][0] += bf_lo(x[k].x); acc[k][1] += bf_hi(x[k].x);
    acc[k][2] += bf_lo(x[k].y); acc[k][3] += bf_hi(x[k].y);
    acc[k][4] += bf_lo(x[k].z); acc[k][5] += bf_hi(x[k].z);
    acc[k][6] += bf_lo(x[k].w); acc[k][7] += bf_hi(x[k].w);
  }
}

// acc += the rows order[from .. to), in order, four loads ahead.
template <int VN>
__device__ __forceinline__ void add_rows(float (&acc)[VN][8], const uint16_t* dy,
                                         const int32_t* order, int from, int to, int cols, int c,
                                         int lane) {
  for (int p0 = from; p0 < to; p0 += 64) {
    const int n = min(64, to - p0);
    const int mine = lane < n ? order[p0 + lane] : 0;
    for (int i = 0; i < n; i += 4) {
      u32x4_t x[4][VN];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u < n) load_row<VN>(x[u], dy, __builtin_amdgcn_readlane(mine, i + u), cols, c);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u < n) add_row<VN>(acc, x[u]);
    }
  }
}

// Sums of the whole runs of 32 sorted rows that share a token, one wave per
// run and 512 VN columns.
template <int VN>
__global__ void __launch_bounds__(256) embed_run_kernel(const EmbedGradArgs a, const EmbedSort w) {
  const int lane = threadIdx.x & 63;
  const int k = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int known = w.start[(int64_t)w.bins << w.log_parts];
  if ((int64_t)(k + 1) * kRun > known || w.token[k * kRun] != w.token[k * kRun + kRun - 1]) return;
  const int c = blockIdx.y * 512 * VN + lane * 8;
  float acc[VN][8] = {};
  add_rows<VN>(acc, a.dy, w.order, k * kRun, (k + 1) * kRun, a.cols, c, lane);
  const RowBuf b(w.run + (int64_t)k * a.cols, (uint32_t)a.cols * 4u);
#pragma unroll
  for (int v = 0; v < VN; ++v) {
    b.st16(__builtin_bit_cast(u32x4_t, f32x4_t{acc[v][0], acc[v][1], acc[v][2], acc[v][3]}),
           (c + 512 * v) * 4);
    b.st16(__builtin_bit_cast(u32x4_t, f32x4_t{acc[v][4], acc[v][5], acc[v][6], acc[v][7]}),
           (c + 512 * v) * 4 + 16);
  }
}

// The table, one wave per token: zeros, or its rows' sum.
template <bool F32, int VN>
__global__ void __launch_bounds__(256) embed_table_kernel(const EmbedGradArgs a, const EmbedSort w) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= a.vocab) return;
  const int64_t slot = (t & ((1 << w.log_parts) - 1)) * w.bins + (t >> w.log_parts);
  const int s = __builtin_amdgcn_readfirstlane(w.start[slot]);
  const int e = __builtin_amdgcn_readfirstlane(w.start[slot + 1]);
  if (s == e && a.accumulate) return;
  const RowBuf ob(F32 ? (const void*)(static_cast<float*>(a.dtable) + t * a.cols)
                      : (const void*)(static_cast<uint16_t*>(a.dtable) + t * a.cols),
                  (uint32_t)a.cols * (F32 ? 4u : 2u));
  // every lane takes every turn (add_rows passes row numbers between lanes);
  // columns past the row load 0 and store nothing
  for (int c = lane * 8; c - lane * 8 < a.cols; c += 512 * VN) {
    float acc[VN][8] = {};
    const int k0 = (s + kRun - 1) / kRun, k1 = e / kRun;
    if (k0 < k1) {
      add_rows<VN>(acc, a.dy, w.order, s, k0 * kRun, a.cols, c, lane);
      for (int k = k0; k < k1; ++k) {
        const RowBuf b(w.run + (int64_t)k * a.cols, (uint32_t)a.cols * 4u);
#pragma unroll
        for (int v = 0; v < VN; ++v) {
          const f32x4_t x = b.ld16f((c + 512 * v) * 4), y = b.ld16f((c + 512 * v) * 4 + 16);
          acc[v][0] += x.x; acc[v][1] += x.y; acc[v][2] += x.z; acc[v][3] += x.w;
          acc[v][4] += y.x; acc[v][5] += y.y; acc[v][6] += y.z; acc[v][7] += y.w;
        }
      }
      add_rows<VN>(acc, a.dy, w.order, k1 * kRun, e, a.cols, c, lane);
    } else if (s < e) {
      add_rows<VN>(acc, a.dy, w.order, s, e, a.cols, c, lane);
    }
#pragma unroll
    for (int v = 0; v < VN; ++v) {
      const int at = c + 512 * v;
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = acc[v][j] * a.scale;
      if constexpr (F32) {
        if (a.accumulate) {
          const f32x4_t x = ob.ld16f(at * 4), y = ob.ld16f(at * 4 + 16);
          d[0] += x.x; d[1] += x.y; d[2] += x.z; d[3] += x.w;
          d[4] += y.x; d[5] += y.y; d[6] += y.z; d[7] += y.w;
        }
        ob.st16(__builtin_bit_cast(u32x4_t, f32x4_t{d[0], d[1], d[2], d[3]}), at * 4);
        ob.st16(__builtin_bit_cast(u32x4_t, f32x4_t{d[4], d[5], d[6], d[7]}), at * 4 + 16);
      } else {
        if (a.accumulate) {
          const u32x4_t x = ob.ld16(at * 2);
          d[0] += bf_lo(x.x); d[1] += bf_hi(x.x); d[2] += bf_lo(x.y); d[3] += bf_hi(x.y);
          d[4] += bf_lo(x.z); d[5] += bf_hi(x.z); d[6] += bf_lo(x.w); d[7] += bf_hi(x.w);
        }
        ob.st16(u32x4_t{pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]), pack_bf16(d[4], d[5]),
                        pack_bf16(d[6], d[7])}, at * 2);
      }
    }
  }
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
  w.run = reinterpret_cast<float*>(p + ns + 2 * nr);
  *bytes = ns + 2 * nr + rows / kRun * cols * 4;
  return w;
}

int64_t embed_grad_workspace(int64_t vocab, int64_t rows, int64_t cols) {
  int64_t bytes = 0;
  (void)embed_sort_plan(vocab, rows, cols, nullptr, &bytes);
  return bytes;
}

template <bool F32, int VN>
static hipError_t run_embed_grad(const EmbedGradArgs& a, const EmbedSort& w, hipStream_t stream) {
  if (a.rows >= kRun) {
    const dim3 grid((unsigned)((a.rows / kRun + 3) / 4), (unsigned)((a.cols + 512 * VN - 1) / (512 * VN)));
    embed_run_kernel<VN><<<grid, 256, 0, stream>>>(a, w);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  embed_table_kernel<F32, VN><<<(int)(((int64_t)a.vocab + 3) / 4), 256, 0, stream>>>(a, w);
  return hipGetLastError();
}

hipError_t launch_embed_rows_backward(bool f32, bool wide_ids, const EmbedGradArgs& a,
                                      void* workspace, hipStream_t stream) {
  int64_t bytes = 0;
  const EmbedSort w = embed_sort_plan(a.vocab, a.rows, a.cols, workspace, &bytes);
  const int groups = 1 << w.log_parts;
  if (wide_ids)
    embed_sort_kernel<int64_t><<<groups, kSortThreads, 0, stream>>>(a.ids, a.rows, a.vocab, w);
  else
    embed_sort_kernel<int32_t><<<groups, kSortThreads, 0, stream>>>(a.ids, a.rows, a.vocab, w);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // a wave's columns: 512, 1,024 or 2,048 at a time
  if (a.cols <= 512) return f32 ? run_embed_grad<true, 1>(a, w, stream) : run_embed_grad<false, 1>(a, w, stream);
  if (a.cols <= 1024) return f32 ? run_embed_grad<true, 2>(a, w, stream) : run_embed_grad<false, 2>(a, w, stream);
  return f32 ? run_embed_grad<true, 4>(a, w, stream) : run_embed_grad<false, 4>(a, w, stream);
}

}  // namespace dsr
