// Host-side launchers of the decoding step's kernels (one translation unit per
// kind), and what they share of the paged cache.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dsr {

// The turn of a head's first `rotary` values.
struct Turn {
  const float* inv_freq;
  int32_t rotary;               // 0: nothing turns
  int32_t interleaved;
  float amplitude;
  float sign;                   // -1 turns back
};

// [0] is q, [1] is k throughout.
struct RopeArgs {
  const uint16_t* x[2];
  uint16_t* y[2];
  const int32_t* pos;
  Turn turn;
  int64_t ldx[2], ldy[2];
  int64_t rows;
  int32_t nh[2];
  int32_t hd;
};

// Byte strides; a token's byte offset is page * page + token * token + head * head.
struct CacheView {
  char* k;
  char* v;
  const float* k_scale;         // may be null
  const float* v_scale;
  const int32_t* table;
  int64_t page_bytes, token_bytes, head_bytes;
  int64_t ld_table;
  int32_t e4m3;
  int32_t n_pages;
  int32_t page_shift;
  int32_t heads;
  int32_t hd;
  int32_t seqs;
  int32_t pages_per_seq;
};

// The bounds of everything that the kernels read from a page table: whether
// sequence `seq`'s row of it has an entry for token `t`, which entry that is, and
// the byte offset of the token in page `page` (-1: no page of the cache).
__host__ __device__ inline bool token_in_table(const CacheView& c, int64_t seq, int32_t t) {
  return seq >= 0 && seq < c.seqs && t >= 0 && (t >> c.page_shift) < c.pages_per_seq;
}
__host__ __device__ inline int64_t table_entry(const CacheView& c, int64_t seq, int32_t t) {
  return seq * c.ld_table + (t >> c.page_shift);
}
__host__ __device__ inline int64_t token_bytes_at(const CacheView& c, int32_t page, int32_t t) {
  if (page < 0 || page >= c.n_pages) return -1;
  return page * c.page_bytes + (int64_t)(t & ((1 << c.page_shift) - 1)) * c.token_bytes;
}

// The keys that a sequence's new rows see, and how they are cut into chunks: by
// the sequence's own length, the window and the number of kv heads, so that a
// row's bits do not depend on the batch.
constexpr int kTile = 32;            // keys a wave takes at a time
constexpr int kBlock = 128;          // keys whose places it looks up together
constexpr int kMaxChunks = 128;      // of one sequence

struct Span {
  int len, first, start, chunk, n;   // first key seen; start: first rounded down to a tile
};

// The least chunk is one block, or two where one block makes more than 512 chunks
// of the sequence's heads.  One sequence over 4 heads of 256 takes 21 us (and 5
// to join) for 8,000 tokens with one block, 27 with two, and 1,021 tokens over 12
// heads of 64 take 10.4 and 14; 32 sequences of up to 4,096 tokens over 8 heads of
// 128, 5 new ones each, 86 and 12.6 with one, 86 and 10.4 with two (half as many sums
// are written and read again).  Half a block would take 8.4 us for those 1,021 tokens,
// but 252 and 16.5 for 64 sequences of up to 8,192 over 4 heads of 256 instead of 238
// and 10.
constexpr int64_t kFine = 512 * kBlock;      // keys times heads

__host__ __device__ inline int least_chunk(int64_t keys, int heads) {
  return keys * heads <= kFine ? kBlock : 2 * kBlock;
}

__host__ __device__ inline Span span_of(int len, int n_new, int window, int heads) {
  Span s;
  s.len = len;
  const int64_t lo = window > 0 ? (int64_t)len - n_new - window + 1 : 0;
  s.first = lo > 0 ? (int)lo : 0;
  s.start = s.first & ~(kTile - 1);
  const int keys = len > s.start ? len - s.start : 0;
  const int least = least_chunk(keys, heads);
  s.chunk = least * (((keys + least - 1) / least + kMaxChunks - 1) / kMaxChunks);
  if (s.chunk == 0) s.chunk = least;
  s.n = (keys + s.chunk - 1) / s.chunk;
  if (s.n == 0) s.n = 1;             // no keys: one empty chunk writes the zeros
  return s;
}

// Most chunks of a sequence of at most `capacity` tokens: of the longest that is
// cut into single blocks, or of the longest.
inline int most_chunks(int64_t capacity, int n_new, int window, int heads) {
  int64_t keys = capacity;
  if (window > 0) {
    const int64_t seen = (int64_t)window + n_new - 1 + kTile - 1;
    keys = keys < seen ? keys : seen;
  }
  const int64_t most = kFine / heads, small = keys < most ? keys : most;
  const int64_t least = least_chunk(keys, heads);
  int64_t n = (keys + least - 1) / least;
  if ((small + kBlock - 1) / kBlock > n) n = (small + kBlock - 1) / kBlock;
  return n < 1 ? 1 : n > kMaxChunks ? kMaxChunks : (int)n;
}

struct AppendArgs {
  const uint16_t* x[3];         // q, k, v
  int64_t ldx[3];
  uint16_t* q_out;
  int64_t ldq_out;
  const float* w[2];            // may be null: weights of 1
  const int32_t* pos;
  const int32_t* seq;           // may be null: row0 + row over rows_per_seq
  Turn turn;
  CacheView cache;
  int64_t rows, row0, rows_per_seq;
  int32_t q_heads;
  int32_t rms;
  float eps;
};

constexpr int kHeadRows = 4;    // rows a workgroup of both kernels
hipError_t launch_rope_rows(const RopeArgs& a, int cus, hipStream_t stream);
hipError_t launch_cache_append(const AppendArgs& a, int cus, hipStream_t stream);

struct AttendArgs {
  CacheView cache;
  const uint16_t* q;
  const int32_t* lens;
  uint16_t* out;
  float* lse;                   // may be null
  int64_t ldq, ldo;
  int32_t q_heads;
  int32_t n_new;
  int32_t window;
  float scale;
};
int64_t attention_workspace(int64_t seqs, int64_t capacity, int q_heads, int heads, int hd, int n_new,
                            int window);
hipError_t launch_cache_attention(const AttendArgs& a, int cus, void* workspace,
                                  hipStream_t stream);

struct VerifyArgs {
  const void* x[2];             // target, draft (may be null)
  int64_t ld[2];
  const float* scale[2];        // may be null
  float inv_temp[2];
  int32_t f32[2];
  const void* drafted;
  int32_t id_bytes;
  const float* u_accept;
  const float* u_sample;
  int32_t* accepted;
  int32_t* tokens;
  float* logp;
  int32_t seqs;
  int32_t drafts;
  int32_t vocab;
};
int64_t verify_slices(int drafts, int64_t vocab, bool with_draft);   // of one sequence
int64_t verify_workspace(int64_t seqs, int drafts, int64_t vocab, bool with_draft);
hipError_t launch_draft_verify(const VerifyArgs& a, int cus, void* workspace, hipStream_t stream);

}  // namespace dsr
