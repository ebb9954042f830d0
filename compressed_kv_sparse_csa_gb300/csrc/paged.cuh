// The paged 4-bit cache: row addressing and launchers shared by the paged
// translation units.  Row and page layout as include/ds4x.h describes them.
#pragma once

#include "ds4x_internal.cuh"

namespace ds4x {

constexpr int kPgCodeBytes = DS4X_KV_NOPE / 2;       // 224
constexpr int kPgTailBytes = 2 * DS4X_KV_ROPE;       // 128
constexpr int kPgScaleBytes = 16;
constexpr int kPgBlocks = DS4X_KV_NOPE / 32;         // 14 blocks of 32 codes
constexpr int kPgTailScale = kPgBlocks;              // the RoPE part's scale byte
static_assert(kPgCodeBytes + kPgTailBytes + kPgScaleBytes == DS4X_PAGED_ROW_BYTES, "row bytes");
constexpr int kPgExpMin = -96, kPgExpMax = 96;       // scale exponents

struct PagedCache {
  uint8_t *pages;
  int64_t n_pages;
  const int32_t *table;
  int64_t table_stride;
  const int32_t *cu;     // [n_seqs + 1]
  int32_t n_seqs, seq_pages;
  int32_t page_log2;     // page_rows = 1 << page_log2
};

// Where a row lies: its page's first byte and its number in the page.
struct PagedRow {
  const uint8_t *page;   // null: the table places the row nowhere
  int32_t at;
};

// The page of row r of sequence s (s checked by the caller).
__device__ __forceinline__ PagedRow paged_row(const PagedCache &c, int32_t s, int64_t r) {
  PagedRow p{nullptr, 0};
  const int64_t j = r >> c.page_log2;
  if (r < 0 || j >= c.seq_pages) return p;
  const int32_t page = __ldcg(c.table + int64_t(s) * c.table_stride + j);
  if (page < 0 || page >= c.n_pages) return p;
  p.page = c.pages + (int64_t(page) << c.page_log2) * DS4X_PAGED_ROW_BYTES;
  p.at = int32_t(r & ((1 << c.page_log2) - 1));
  return p;
}
__device__ __forceinline__ int64_t paged_code_off(const PagedRow &p) { return int64_t(p.at) * kPgCodeBytes; }
__device__ __forceinline__ int64_t paged_tail_off(const PagedCache &c, const PagedRow &p) {
  return (int64_t(kPgCodeBytes) << c.page_log2) + int64_t(p.at) * kPgTailBytes;
}
__device__ __forceinline__ int64_t paged_scale_off(const PagedCache &c, const PagedRow &p) {
  return (int64_t(kPgCodeBytes + kPgTailBytes) << c.page_log2) + int64_t(p.at) * kPgScaleBytes;
}

// The sequence of token t: the s with cu[s] <= t < cu[s + 1], or -1 (padding,
// or a cu that is not what it should be); its first token and the one behind its
// last.  One warp searches, 32 ways a step.
struct PagedSeq {
  int32_t s, from, to;
};
__device__ __forceinline__ PagedSeq paged_seq_of(const PagedCache &c, int64_t t, int lane) {
  int32_t lo = 0, n = c.n_seqs;  // the answer, if any, is in [lo, lo + n)
  while (n > 1) {
    const int32_t step = (n + 31) / 32;
    const int32_t at = lo + lane * step;
    const bool below = lane * step < n && int64_t(__ldcg(c.cu + at)) <= t;
    const uint32_t b = __ballot_sync(0xffffffffu, below);
    const int32_t k = b ? 31 - __clz(b) : 0;  // the last pivot at or below t
    const int32_t left = n - k * step;
    lo += k * step;
    n = step < left ? step : left;
  }
  const int32_t from = __ldcg(c.cu + lo), to = __ldcg(c.cu + lo + 1);
  return PagedSeq{from <= t && t < to ? lo : -1, from, to};
}

cudaError_t launch_paged_append(const PagedCache &c, const int64_t *row0, const void *in, bool in_bf16,
                                int64_t in_stride, int64_t n, const int64_t *pos, const float *inv_freq, bool halves,
                                void *ws, cudaStream_t stream);
cudaError_t launch_paged_gather(const PagedCache &c, const int64_t *row0, void *out, bool out_bf16,
                                int64_t out_stride, int64_t n, void *ws, cudaStream_t stream);

// Moves row row0 + path[i] of each sequence to row0 + i, i < n_path.
cudaError_t launch_paged_keep(const PagedCache &c, const int64_t *row0, const int32_t *path, const int32_t *n_path,
                              int64_t n, void *ws, cudaStream_t stream);

// The walk over drafted tokens (csrc/verify.cu).
struct Verify {
  const int32_t *cu;
  int32_t n_seqs;
  int64_t n_tokens;
  const int32_t *parent, *tokens;
  const void *target, *draft;  // draft may be null
  int64_t target_stride, draft_stride;
  int32_t vocab;
  const float *u;
  int32_t *path, *out, *n_path;
};
cudaError_t launch_verify(const Verify &v, bool bf16, void *ws, cudaStream_t stream);

// Attention over row ranges (idx null: [row_begin, row_end) per token), lists
// (idx [n][k] with n_rows per sequence) or trees (parent [n] with tree_row0 per
// sequence; row_begin a position).
struct PagedAttn {
  PagedCache c;
  const int64_t *row_begin, *row_end;
  const int64_t *n_rows;
  const int32_t *idx;
  int32_t k;
  int32_t n_tokens, n_heads;
  const uint16_t *q;
  int64_t q_stride;
  float scale;
  uint16_t *out;
  int64_t out_stride;
  float *lse;
  const int64_t *tree_row0;
  const int32_t *parent;
};
size_t paged_attn_ws_bytes();
cudaError_t launch_paged_attn(const PagedAttn &a, void *ws, cudaStream_t stream);

}  // namespace ds4x
