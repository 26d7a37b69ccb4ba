// Drafted tokens against a model's probabilities, from given random numbers.
//
//   p = softmax(target row), q = softmax(draft row)      in fp64
//   accept d_i while u_i q_i(d_i) < p_i(d_i); then the first j with
//   sum_{k <= j} w_k > u sum w,  w = max(p - q, 0)
// Three launches: sums of exp by chunks of every row; the decisions and the
// chunks' sums of w (of the one row that a token is sampled from); the chunk
// that the random number falls into, and the token in it.
//
// fp64, because a token's choice hangs on every border of the cumulated
// distribution at once: with weights known to 1e-7 and a vocabulary of 1e5,
// about one choice in a thousand would fall on the other side of a border.
#include <algorithm>

#include "decode_launch.hpp"
#include "row_kernels.hpp"

namespace dsr {

constexpr int kSlice = 2048;          // columns a workgroup takes: 8 a thread
constexpr int kMaxRowsPerSeq = 72;    // >= 2 DS_MAX_DRAFTS + 1

// What a slice of a row sums to: exp(z - m) over it, m its largest.  A NaN or
// +infinity makes sum NaN; a slice masked whole has m -infinity and sum 0.
struct Slice {
  float m, pad;
  double sum;
};

__device__ __forceinline__ float logit(const VerifyArgs& a, int which, int64_t row, int col) {
  const float x = a.f32[which] ? ((const float*)a.x[which])[row * a.ld[which] + col]
                               : bf_lo(((const uint16_t*)a.x[which])[row * a.ld[which] + col]);
  return (a.scale[which] != nullptr ? x * a.scale[which][col] : x) * a.inv_temp[which];
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// exp of the distance from m, 0 for a masked token.
__device__ __forceinline__ double weight_of(float z, float m) { return exp((double)z - (double)m); }

// Row r of a sequence: its target rows, then its draft rows.
__global__ void __launch_bounds__(256) verify_sums_kernel(const VerifyArgs a, Slice* slices, int rows_per_seq,
                                                          int n_slices) {
  __shared__ float tops[4];
  __shared__ double sums[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t id = blockIdx.x;
  const int slice = (int)(id % n_slices);
  const int64_t row = id / n_slices, seq = row / rows_per_seq;
  const int r = (int)(row % rows_per_seq), which = r > a.drafts;
  const int64_t at = which ? seq * a.drafts + r - a.drafts - 1 : seq * (a.drafts + 1) + r;
  float z[8], top = -__builtin_inff();
  bool odd = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = slice * kSlice + j * 256 + (int)threadIdx.x;
    z[j] = c < a.vocab ? logit(a, which, at, c) : -__builtin_inff();
    odd = odd || !(z[j] < __builtin_inff());
    top = fmaxf(top, z[j]);
  }
  top = wave_max(top);
  if (lane == 0) tops[wave] = top;
  odd = __syncthreads_or(odd);
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  double sum = 0.0;
  if (top > -__builtin_inff() && !odd) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += weight_of(z[j], top);
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

// A row's largest logit and its log-sum's factor: p = exp(z - m) / sum.  sum 0:
// the row says nothing (masked whole, or not a number somewhere).
struct Norm {
  float m;
  double sum;
};

__device__ __forceinline__ Norm join_slices(const Slice* s, int n, int lane) {
  float m = -__builtin_inff();
  for (int i = lane; i < n; i += 64) m = fmaxf(m, s[i].m);
  m = wave_max(m);
  double sum = 0.0;
  for (int i = lane; i < n; i += 64) {
    const Slice t = s[i];
    sum += t.m == -__builtin_inff() ? t.sum : t.sum * exp((double)t.m - (double)m);
  }
  sum = wave_sum_f64(sum);
  return Norm{m, sum == sum ? sum : 0.0};
}

// Where a sequence stands after its drafts: the row that the next token comes
// from, whether its draft row is taken off, and the one token that is (certain
// drafts), with the rows' norms.
struct Choice {
  int accepted, refused, token;       // token: the refused one
  Norm p, q;
};

__device__ __forceinline__ int64_t drafted_id(const VerifyArgs& a, int64_t i) {
  return a.id_bytes == 8 ? ((const int64_t*)a.drafted)[i] : ((const int32_t*)a.drafted)[i];
}

// The whole workgroup finds its sequence's choice; `norms` is LDS.
__device__ __forceinline__ Choice decide(const VerifyArgs& a, const Slice* slices, int64_t seq,
                                         int rows_per_seq, int n_slices, Norm* norms) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  for (int r = wave; r < rows_per_seq; r += waves) {
    const Norm n = join_slices(slices + (seq * rows_per_seq + r) * n_slices, n_slices, lane);
    if (lane == 0) norms[r] = n;
  }
  __syncthreads();
  Choice c{0, 0, -1, norms[0], Norm{0.f, 0.0}};
  for (; c.accepted < a.drafts; ++c.accepted) {
    const int i = c.accepted;
    const int64_t d = drafted_id(a, seq * a.drafts + i);
    if (d < 0 || d >= a.vocab) break;                      // no draft here: nothing to refuse
    const Norm p = norms[i];
    const double pd =
        p.sum > 0.0 ? weight_of(logit(a, 0, seq * (a.drafts + 1) + i, (int)d), p.m) / p.sum : 0.0;
    double qd = 1.0;
    bool says = true;                                      // the draft row does
    if (a.x[1] != nullptr) {
      c.q = norms[a.drafts + 1 + i];
      says = c.q.sum > 0.0;
      if (says) qd = weight_of(logit(a, 1, seq * a.drafts + i, (int)d), c.q.m) / c.q.sum;
    }
    if (!(says && (double)a.u_accept[seq * a.drafts + i] * qd < pd)) {
      c.refused = says;
      c.token = (int)d;
      break;
    }
  }
  c.p = norms[c.accepted];
  return c;
}

// Weight of column `col` in the distribution that the next token comes from.
__device__ __forceinline__ double residual(const VerifyArgs& a, const Choice& c, int64_t seq, int col,
                                           bool whole) {
  if (!(c.p.sum > 0.0)) return 0.0;
  const double p = weight_of(logit(a, 0, seq * (a.drafts + 1) + c.accepted, col), c.p.m) / c.p.sum;
  if (whole || !c.refused) return p;
  double q = col == c.token ? 1.0 : 0.0;
  if (a.x[1] != nullptr) q = weight_of(logit(a, 1, seq * a.drafts + c.accepted, col), c.q.m) / c.q.sum;
  return fmax(p - q, 0.0);
}

// Sums of w over a slice's columns: thread t has the 8 columns 8 t.. (ascending
// order is what the cumulated sum goes by).  Two sums a slice: w, and p itself.
__global__ void __launch_bounds__(256) verify_weights_kernel(const VerifyArgs a, const Slice* slices, double* sums,
                                                             int rows_per_seq, int n_slices) {
  __shared__ Norm norms[kMaxRowsPerSeq];
  __shared__ double part[4][2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t seq = blockIdx.x / n_slices;
  const int slice = (int)(blockIdx.x % n_slices);
  const Choice c = decide(a, slices, seq, rows_per_seq, n_slices, norms);
  double w = 0.0, p = 0.0;
  for (int j = 0; j < 8; ++j) {
    const int col = slice * kSlice + (int)threadIdx.x * 8 + j;
    if (col >= a.vocab) break;
    w += residual(a, c, seq, col, false);
    p += residual(a, c, seq, col, true);
  }
  w = wave_sum_f64(w);
  p = wave_sum_f64(p);
  if (lane == 0) {
    part[wave][0] = w;
    part[wave][1] = p;
  }
  __syncthreads();
  if (threadIdx.x < 2)
    sums[(int64_t)blockIdx.x * 2 + threadIdx.x] =
        ((part[0][threadIdx.x] + part[1][threadIdx.x]) + part[2][threadIdx.x]) + part[3][threadIdx.x];
}

// One workgroup a sequence: the slice that u * total falls into, the token in
// it, and the outputs.
__global__ void __launch_bounds__(256) verify_pick_kernel(const VerifyArgs a, const Slice* slices, const double* sums,
                                                          int rows_per_seq, int n_slices) {
  __shared__ Norm norms[kMaxRowsPerSeq];
  __shared__ double ends[256];
  __shared__ int32_t found, last;
  __shared__ int slice_of;
  __shared__ double before;
  const int64_t seq = blockIdx.x;
  const Choice c = decide(a, slices, seq, rows_per_seq, n_slices, norms);
  const double* of = sums + seq * n_slices * 2;
  double u = (double)a.u_sample[seq];
  u = u < 0.0 ? 0.0 : u;                                   // (a NaN stays one)
  if (threadIdx.x == 0) {
    double total = 0.0;
    int whole = 0;
    for (int i = 0; i < n_slices; ++i) total += of[i * 2];
    if (!(total > 0.0)) {                                  // p = q: nothing is left over
      whole = 1;
      total = 0.0;
      for (int i = 0; i < n_slices; ++i) total += of[i * 2 + 1];
    }
    const double edge = u * total;
    double sum = 0.0, start = 0.0;
    int at = -1;
    for (int i = 0; i < n_slices; ++i) {
      const double w = of[i * 2 + whole];
      if (w > 0.0) {                                       // the last one of any weight, at least
        at = i;
        start = sum;
        if (sum + w > edge) break;
      }
      sum += w;
    }
    slice_of = at < 0 ? -1 : at * 2 + whole;
    before = edge - start;
    found = 0x7fffffff;
    last = -1;
  }
  __syncthreads();
  int token = -1;
  if (slice_of >= 0) {
    const bool whole = slice_of & 1;
    const int col0 = slice_of / 2 * kSlice + (int)threadIdx.x * 8;
    double w[8], sum = 0.0;
    for (int j = 0; j < 8; ++j) {
      w[j] = col0 + j < a.vocab ? residual(a, c, seq, col0 + j, whole) : 0.0;
      sum += w[j];
    }
    ends[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      double run = 0.0;
      for (int i = 0; i < 256; ++i) {
        const double t = ends[i];
        ends[i] = run;
        run += t;
      }
    }
    __syncthreads();
    double run = ends[threadIdx.x];
    for (int j = 0; j < 8; ++j) {
      run += w[j];
      if (w[j] > 0.0) {
        atomicMax(&last, col0 + j);
        if (run > before) {
          atomicMin(&found, col0 + j);
          break;
        }
      }
    }
    __syncthreads();
    token = found != 0x7fffffff ? found : last;
  }
  for (int i = threadIdx.x; i <= a.drafts; i += 256) {
    const int64_t at = seq * (a.drafts + 1) + i;
    const int t = i < c.accepted ? (int)drafted_id(a, seq * a.drafts + i) : i == c.accepted ? token : -1;
    a.tokens[at] = t;
    const Norm n = norms[i];
    a.logp[at] = t < 0 ? 0.f : (float)((double)logit(a, 0, at, t) - (double)n.m - log(n.sum));
  }
  if (threadIdx.x == 0) a.accepted[seq] = c.accepted;
}

static int slices_of(int64_t vocab) { return (int)((vocab + kSlice - 1) / kSlice); }

int64_t verify_slices(int drafts, int64_t vocab, bool with_draft) {
  return (int64_t)slices_of(vocab) * (drafts + 1 + (with_draft ? drafts : 0));
}

int64_t verify_workspace(int64_t seqs, int drafts, int64_t vocab, bool with_draft) {
  return seqs * (verify_slices(drafts, vocab, with_draft) * (int64_t)sizeof(Slice) + slices_of(vocab) * 16);
}

hipError_t launch_draft_verify(const VerifyArgs& a, void* workspace, hipStream_t stream) {
  const int n = slices_of(a.vocab), rows = a.drafts + 1 + (a.x[1] != nullptr ? a.drafts : 0);
  Slice* slices = static_cast<Slice*>(workspace);
  double* sums = reinterpret_cast<double*>(slices + (int64_t)a.seqs * rows * n);
  verify_sums_kernel<<<(uint32_t)((int64_t)a.seqs * rows * n), 256, 0, stream>>>(a, slices, rows, n);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  verify_weights_kernel<<<(uint32_t)((int64_t)a.seqs * n), 256, 0, stream>>>(a, slices, sums, rows, n);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  verify_pick_kernel<<<a.seqs, 256, 0, stream>>>(a, slices, sums, rows, n);
  return hipGetLastError();
}

}  // namespace dsr
