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

constexpr int kEmbedRun = 32;     // rows of a token summed together before they join the total

// One wave per (token, 512 columns): it looks at every id, 64 at a time, and
// adds the rows of its token as they come.
template <bool F32, class Id>
__global__ void __launch_bounds__(256) embed_grad_scan_kernel(const EmbedGradArgs a) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = (blockIdx.y * 64 + lane) * 8;
  const uint32_t in_bytes = (uint32_t)a.cols * 2u;
  for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < a.vocab; t += (int64_t)gridDim.x * 4) {
    float total[8] = {}, run[8] = {};
    int n = 0;
    for (int64_t i0 = 0; i0 < a.rows; i0 += 64) {
      const bool mine = i0 + lane < a.rows && token_at<Id>(a.ids, i0 + lane, a.vocab) == t;
      uint64_t hits = __builtin_amdgcn_ballot_w64(mine);
      while (hits != 0) {
        const int64_t i = i0 + __builtin_ctzll(hits);
        hits &= hits - 1;
        const u32x4_t x = RowBuf(a.dy + i * a.cols, in_bytes).ld16(c * 2);
        const float v[8] = {bf_lo(x.x), bf_hi(x.x), bf_lo(x.y), bf_hi(x.y),
                            bf_lo(x.z), bf_hi(x.z), bf_lo(x.w), bf_hi(x.w)};
        if (n > 0 && n % kEmbedRun == 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            total[k] += run[k];
            run[k] = 0.f;
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) run[k] += v[k];
        ++n;
      }
    }
    if (n == 0 && a.accumulate) continue;
    const uint32_t out_bytes = (uint32_t)a.cols * (F32 ? 4u : 2u);
    const int64_t at = t * a.cols;
    const RowBuf ob(F32 ? (const void*)(static_cast<float*>(a.dtable) + at)
                        : (const void*)(static_cast<uint16_t*>(a.dtable) + at), out_bytes);
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = (total[k] + run[k]) * a.scale;
    if constexpr (F32) {
      if (a.accumulate) {
        const f32x4_t x = ob.ld16f(c * 4), y = ob.ld16f(c * 4 + 16);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
      }
      ob.st16(__builtin_bit_cast(u32x4_t, f32x4_t{v[0], v[1], v[2], v[3]}), c * 4);
      ob.st16(__builtin_bit_cast(u32x4_t, f32x4_t{v[4], v[5], v[6], v[7]}), c * 4 + 16);
    } else {
      if (a.accumulate) {
        const u32x4_t x = ob.ld16(c * 2);
        v[0] += bf_lo(x.x); v[1] += bf_hi(x.x); v[2] += bf_lo(x.y); v[3] += bf_hi(x.y);
        v[4] += bf_lo(x.z); v[5] += bf_hi(x.z); v[6] += bf_lo(x.w); v[7] += bf_hi(x.w);
      }
      ob.st16(u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                      pack_bf16(v[6], v[7])}, c * 2);
    }
  }
}

hipError_t launch_embed_rows_backward(bool f32, bool wide_ids, const EmbedGradArgs& a,
                                      void* workspace, hipStream_t stream) {
  (void)workspace;
  const int64_t groups = ((int64_t)a.vocab + 3) / 4;
  const dim3 grid((unsigned)(groups < 65536 ? groups : 65536), (unsigned)((a.cols + 511) / 512));
  if (f32 && wide_ids) embed_grad_scan_kernel<true, int64_t><<<grid, 256, 0, stream>>>(a);
  else if (f32) embed_grad_scan_kernel<true, int32_t><<<grid, 256, 0, stream>>>(a);
  else if (wide_ids) embed_grad_scan_kernel<false, int64_t><<<grid, 256, 0, stream>>>(a);
  else embed_grad_scan_kernel<false, int32_t><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace dsr
