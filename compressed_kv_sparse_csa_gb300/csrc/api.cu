// Host side of the C ABI declared in include/ds4x.h: argument checks (all
// before any CUDA call, so a bad call launches nothing), the device
// architecture check, workspace sizing and dispatch to the kernels.
#include <atomic>
#include <cstdlib>
#include <cstring>

#include "ds4x_internal.cuh"
#include "paged.cuh"

using namespace ds4x;

namespace {

bool aligned_to(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool aligned16(const void *p) { return aligned_to(p, 16); }

// Per-device cache of the architecture check: 0 unknown, 1 GB300, 2 other.
std::atomic<int> g_arch_ok[64];

int check_arch() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DS4X_ECUDA;
  if (dev >= 0 && dev < 64) {
    const int c = g_arch_ok[dev].load(std::memory_order_relaxed);
    if (c != 0) return c == 1 ? DS4X_OK : DS4X_EARCH;
  }
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
    return DS4X_ECUDA;
  }
  const bool ok = (major == 10 && minor == 3);
  if (dev >= 0 && dev < 64) g_arch_ok[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
  return ok ? DS4X_OK : DS4X_EARCH;
}

int from_cuda(cudaError_t e) { return e == cudaSuccess ? DS4X_OK : DS4X_ECUDA; }

// DS4X_SCORER=two_stage selects the score-then-select path (A/B and debug);
// the default is the fused tensor-core scorer.
bool use_two_stage() {
  static const bool v = [] {
    const char *e = std::getenv("DS4X_SCORER");
    return e != nullptr && std::strcmp(e, "two_stage") == 0;
  }();
  return v;
}

}  // namespace

extern "C" {

const char *ds4x_status_str(int status) {
  switch (status) {
    case DS4X_OK: return "ok";
    case DS4X_EINVAL: return "invalid argument (null or misaligned pointer, bad size or k)";
    case DS4X_ERANGE: return "rows outside the cache capacity";
    case DS4X_EWORKSPACE: return "workspace too small";
    case DS4X_EARCH: return "device is not compute capability 10.3 (GB300)";
    case DS4X_ECUDA: return "CUDA runtime error";
    case DS4X_ETIMEOUT: return "bounded device wait gave up";
    case DS4X_EDEVICE: return "kernel-detected invalid input (index out of range)";
    case DS4X_EFORMAT: return "not a checkpoint of this layout, or corrupt or truncated";
    case DS4X_EVERSION: return "a checkpoint of another payload version";
    default: return "unknown status";
  }
}

int ds4x_abi_version(void) { return DS4X_ABI_VERSION; }

int64_t ds4x_cache_bytes(int64_t L) {
  if (L < 0) return -1;
  const int64_t ring = int64_t(43) * 256 * DS4X_KV_ROW_BYTES;
  const int64_t csa = int64_t(21) * (L / 4 + 2) * (DS4X_KV_ROW_BYTES + DS4X_IDX_ROW_BYTES);
  const int64_t hca = int64_t(20) * (L / 128 + 2) * DS4X_KV_ROW_BYTES;
  return ring + csa + hca;
}

int ds4x_workspace_init(void *ws, size_t ws_bytes, ds4x_stream_t stream) {
  if (ws == nullptr || !aligned16(ws) || ws_bytes < kWsHeaderBytes) return DS4X_EINVAL;
  const int a = check_arch();
  if (a != DS4X_OK) return a;
  return from_cuda(cudaMemsetAsync(ws, 0, ws_bytes, stream));
}

int ds4x_copy_async(void *dst, const void *src, size_t bytes, ds4x_stream_t stream) {
  if (dst == nullptr || src == nullptr || !aligned16(dst) || !aligned16(src)) return DS4X_EINVAL;
  const uintptr_t d = reinterpret_cast<uintptr_t>(dst), s = reinterpret_cast<uintptr_t>(src);
  if (bytes > 0 && d < s + bytes && s < d + bytes) return DS4X_EINVAL;  // overlapping
  if (bytes == 0) return DS4X_OK;
  const int a = check_arch();
  if (a != DS4X_OK) return a;
  return from_cuda(launch_copy(dst, src, bytes, stream));
}

int ds4x_workspace_status(void *ws, ds4x_stream_t stream, int32_t *status_host) {
  if (ws == nullptr || status_host == nullptr || !aligned16(ws)) return DS4X_EINVAL;
  const int a = check_arch();
  if (a != DS4X_OK) return a;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return DS4X_ECUDA;
  int32_t v = 0;
  if (cudaMemcpy(&v, ws, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess) return DS4X_ECUDA;
  const int32_t zero = 0;
  if (cudaMemcpy(ws, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess) return DS4X_ECUDA;
  *status_host = v;
  return DS4X_OK;
}

int ds4x_cache_append(uint8_t *kv_rows, uint8_t *idx_rows, int64_t capacity, int64_t pos,
                      const float *kv_in, const float *idx_in, int64_t n, ds4x_stream_t stream) {
  if (kv_rows == nullptr && idx_rows == nullptr) return DS4X_EINVAL;
  if (kv_rows != nullptr && (kv_in == nullptr || !aligned16(kv_in) || !aligned16(kv_rows))) return DS4X_EINVAL;
  if (idx_rows != nullptr && (idx_in == nullptr || !aligned16(idx_in) || !aligned16(idx_rows))) return DS4X_EINVAL;
  if (n < 1 || capacity < 1) return DS4X_EINVAL;
  if (pos < 0 || pos > capacity || n > capacity - pos) return DS4X_ERANGE;
  const int a = check_arch();
  if (a != DS4X_OK) return a;
  return from_cuda(launch_cache_append(kv_rows, idx_rows, pos, kv_in, idx_in, n, stream));
}

size_t ds4x_index_score_topk_workspace(int64_t n_rows, int32_t k) {
  (void)k;
  if (n_rows < 1) n_rows = 1;
  const size_t a = score_two_stage_ws_bytes(n_rows), b = score_fused_ws_bytes();
  return a > b ? a : b;
}

int ds4x_index_score_topk(const uint8_t *idx_rows, int64_t n_rows, const uint16_t *q_bf16,
                          const float *w, int32_t k, int32_t *out_idx, float *out_score, void *ws,
                          size_t ws_bytes, ds4x_stream_t stream) {
  if (idx_rows == nullptr || q_bf16 == nullptr || w == nullptr || out_idx == nullptr || ws == nullptr)
    return DS4X_EINVAL;
  if (!aligned16(idx_rows) || !aligned16(q_bf16) || !aligned16(w) || !aligned16(out_idx) ||
      !aligned16(ws) || (out_score != nullptr && !aligned16(out_score)))
    return DS4X_EINVAL;
  if (n_rows < 1 || n_rows > int64_t(INT32_MAX) || k < 1 || k > DS4X_TOPK_MAX) return DS4X_EINVAL;
  if (ws_bytes < ds4x_index_score_topk_workspace(n_rows, k)) return DS4X_EWORKSPACE;
  const int a = check_arch();
  if (a != DS4X_OK) return a;
  if (use_two_stage())
    return from_cuda(launch_score_two_stage(idx_rows, n_rows, q_bf16, w, k, out_idx, out_score, ws, stream));
  return from_cuda(launch_score_fused(idx_rows, n_rows, q_bf16, w, k, out_idx, out_score, ws, stream));
}

size_t ds4x_sparse_attn_decode_workspace(int32_t k) {
  if (k < 1) k = 1;
  if (k > DS4X_TOPK_MAX) k = DS4X_TOPK_MAX;
  return attn_decode_ws_bytes(k);
}

int ds4x_sparse_attn_decode(const uint8_t *kv_rows, int64_t n_rows, const int32_t *idx, int32_t k,
                            const uint16_t *q_bf16, float softmax_scale, uint16_t *out_bf16,
                            float *lse, void *ws, size_t ws_bytes, ds4x_stream_t stream) {
  if (kv_rows == nullptr || idx == nullptr || q_bf16 == nullptr || out_bf16 == nullptr || ws == nullptr)
    return DS4X_EINVAL;
  if (!aligned16(kv_rows) || !aligned16(idx) || !aligned16(q_bf16) || !aligned16(out_bf16) ||
      !aligned16(ws) || (lse != nullptr && !aligned16(lse)))
    return DS4X_EINVAL;
  if (n_rows < 1 || k < 1 || k > DS4X_TOPK_MAX) return DS4X_EINVAL;
  if (ws_bytes < ds4x_sparse_attn_decode_workspace(k)) return DS4X_EWORKSPACE;
  const int a = check_arch();
  if (a != DS4X_OK) return a;
  return from_cuda(launch_attn_decode(kv_rows, n_rows, idx, k, q_bf16, softmax_scale, out_bf16, lse,
                                      ws, stream));
}

size_t ds4x_csa_decode_step_workspace(int64_t n_rows, int32_t k) {
  const size_t a = ds4x_index_score_topk_workspace(n_rows, k), b = ds4x_sparse_attn_decode_workspace(k);
  return a > b ? a : b;
}

int ds4x_csa_decode_step(const uint8_t *idx_rows, const uint8_t *kv_rows, int64_t n_rows, const uint16_t *q_idx_bf16,
                         const float *w, int32_t k, const uint16_t *q_attn_bf16, float softmax_scale,
                         int32_t *out_idx, float *out_score, uint16_t *out_bf16, float *lse, void *ws,
                         size_t ws_bytes, ds4x_stream_t stream) {
  if (idx_rows == nullptr || kv_rows == nullptr || q_idx_bf16 == nullptr || w == nullptr || q_attn_bf16 == nullptr ||
      out_idx == nullptr || out_bf16 == nullptr || ws == nullptr)
    return DS4X_EINVAL;
  if (!aligned16(idx_rows) || !aligned16(kv_rows) || !aligned16(q_idx_bf16) || !aligned16(w) ||
      !aligned16(q_attn_bf16) || !aligned16(out_idx) || !aligned16(out_bf16) || !aligned16(ws) ||
      (out_score != nullptr && !aligned16(out_score)) || (lse != nullptr && !aligned16(lse)))
    return DS4X_EINVAL;
  if (n_rows < 1 || n_rows > int64_t(INT32_MAX) || k < 1 || k > DS4X_TOPK_MAX) return DS4X_EINVAL;
  if (ws_bytes < ds4x_csa_decode_step_workspace(n_rows, k)) return DS4X_EWORKSPACE;
  const int a = check_arch();
  if (a != DS4X_OK) return a;
  // the attention shares the scorer's workspace header (it only ever sets its status word)
  cudaError_t e = use_two_stage()
                      ? launch_score_two_stage(idx_rows, n_rows, q_idx_bf16, w, k, out_idx, out_score, ws, stream)
                      : launch_score_fused(idx_rows, n_rows, q_idx_bf16, w, k, out_idx, out_score, ws, stream);
  if (e != cudaSuccess) return DS4X_ECUDA;
  return from_cuda(launch_attn_decode(kv_rows, n_rows, out_idx, k, q_attn_bf16, softmax_scale, out_bf16, lse, ws,
                                      stream));
}

size_t ds4x_index_score_topk_batched_workspace(int32_t n_sess, int32_t k) {
  (void)n_sess;
  (void)k;
  return score_fused_ws_bytes();
}

int ds4x_index_score_topk_batched(const uint8_t *const *idx_rows, const int64_t *n_rows, int32_t n_sess,
                                  const uint16_t *q_bf16, const float *w, int32_t k, int32_t *out_idx,
                                  float *out_score, void *ws, size_t ws_bytes, ds4x_stream_t stream) {
  if (idx_rows == nullptr || n_rows == nullptr || q_bf16 == nullptr || w == nullptr || out_idx == nullptr ||
      ws == nullptr)
    return DS4X_EINVAL;
  if (!aligned16(idx_rows) || !aligned16(n_rows) || !aligned16(q_bf16) || !aligned16(w) || !aligned16(out_idx) ||
      !aligned16(ws) || (out_score != nullptr && !aligned16(out_score)))
    return DS4X_EINVAL;
  if (n_sess < 1 || n_sess > DS4X_MAX_SESSIONS || k < 1 || k > DS4X_TOPK_MAX) return DS4X_EINVAL;
  if (ws_bytes < ds4x_index_score_topk_batched_workspace(n_sess, k)) return DS4X_EWORKSPACE;
  const int a = check_arch();
  if (a != DS4X_OK) return a;
  ScoreBatch sb{};
  sb.rows_arr = idx_rows;
  sb.n_arr = n_rows;
  sb.n_sess = n_sess;
  sb.q = q_bf16;
  sb.w = w;
  sb.k = k;
  sb.out_idx = out_idx;
  sb.out_score = out_score;
  return from_cuda(launch_score_batch(sb, 0, ws, stream));
}

int ds4x_sparse_attn_decode_batched(const uint8_t *const *kv_rows, const int64_t *n_rows, int32_t n_sess,
                                    const int32_t *idx, int32_t k, const uint16_t *q_bf16, float softmax_scale,
                                    uint16_t *out_bf16, float *lse, void *ws, size_t ws_bytes,
                                    ds4x_stream_t stream) {
  if (kv_rows == nullptr || n_rows == nullptr || idx == nullptr || q_bf16 == nullptr || out_bf16 == nullptr ||
      ws == nullptr)
    return DS4X_EINVAL;
  if (!aligned16(kv_rows) || !aligned16(n_rows) || !aligned16(idx) || !aligned16(q_bf16) || !aligned16(out_bf16) ||
      !aligned16(ws) || (lse != nullptr && !aligned16(lse)))
    return DS4X_EINVAL;
  if (n_sess < 1 || n_sess > DS4X_MAX_SESSIONS || k < 1 || k > DS4X_TOPK_MAX) return DS4X_EINVAL;
  if (ws_bytes < ds4x_sparse_attn_decode_workspace(k)) return DS4X_EWORKSPACE;
  const int a = check_arch();
  if (a != DS4X_OK) return a;
  AttnBatch ab{};
  ab.kv_arr = kv_rows;
  ab.n_arr = n_rows;
  ab.idx = idx;
  ab.k = k;
  ab.scale = softmax_scale;
  ab.q = q_bf16;
  ab.out = out_bf16;
  ab.lse = lse;
  return from_cuda(launch_attn_batch(ab, n_sess, ws, stream));
}

int ds4x_sparse_attn_prefill(const uint8_t *kv_rows, int64_t n_rows, const int32_t *idx, int32_t n_queries,
                             int32_t k, const uint16_t *q_bf16, float softmax_scale, uint16_t *out_bf16,
                             float *lse, void *ws, size_t ws_bytes, ds4x_stream_t stream) {
  if (kv_rows == nullptr || idx == nullptr || q_bf16 == nullptr || out_bf16 == nullptr || ws == nullptr)
    return DS4X_EINVAL;
  if (!aligned16(kv_rows) || !aligned16(idx) || !aligned16(q_bf16) || !aligned16(out_bf16) || !aligned16(ws) ||
      (lse != nullptr && !aligned16(lse)))
    return DS4X_EINVAL;
  if (n_rows < 1 || n_queries < 1 || n_queries > DS4X_PREFILL_MAX_QUERIES || k < 1 || k > DS4X_TOPK_MAX)
    return DS4X_EINVAL;
  if (ws_bytes < ds4x_sparse_attn_decode_workspace(k) || ws_bytes < attn_prefill_ws_bytes()) return DS4X_EWORKSPACE;
  const int a = check_arch();
  if (a != DS4X_OK) return a;
  return from_cuda(launch_attn_prefill(kv_rows, n_rows, idx, n_queries, k, q_bf16, softmax_scale, out_bf16, lse, ws,
                                       stream));
}

size_t ds4x_dense_attn_decode_workspace(int64_t n_rows) {
  if (n_rows < 1) n_rows = 1;
  if (n_rows > DS4X_DENSE_MAX_ROWS) n_rows = DS4X_DENSE_MAX_ROWS;
  return dense_attn_ws_bytes(n_rows);
}

int ds4x_dense_attn_decode(const uint8_t *kv_rows, int64_t n_rows, const uint16_t *q_bf16, float softmax_scale,
                           uint16_t *out_bf16, float *lse, void *ws, size_t ws_bytes, ds4x_stream_t stream) {
  if (kv_rows == nullptr || q_bf16 == nullptr || out_bf16 == nullptr || ws == nullptr) return DS4X_EINVAL;
  if (!aligned16(kv_rows) || !aligned16(q_bf16) || !aligned16(out_bf16) || !aligned16(ws) ||
      (lse != nullptr && !aligned16(lse)))
    return DS4X_EINVAL;
  if (n_rows < 1 || n_rows > DS4X_DENSE_MAX_ROWS) return DS4X_EINVAL;
  if (ws_bytes < ds4x_dense_attn_decode_workspace(n_rows)) return DS4X_EWORKSPACE;
  const int a = check_arch();
  if (a != DS4X_OK) return a;
  return from_cuda(launch_dense_attn(kv_rows, n_rows, q_bf16, softmax_scale, out_bf16, lse, ws, stream));
}

size_t ds4x_window_sparse_attn_decode_workspace(void) { return window_attn_ws_bytes(); }

int ds4x_window_sparse_attn_decode(const uint8_t *kv_rows, int64_t n_rows, const int32_t *idx, int32_t k,
                                   const uint8_t *ring_rows, int32_t ring_pos, int32_t w, const uint16_t *q_bf16,
                                   float softmax_scale, uint16_t *out_bf16, float *lse, void *ws, size_t ws_bytes,
                                   ds4x_stream_t stream) {
  if (kv_rows == nullptr || idx == nullptr || ring_rows == nullptr || q_bf16 == nullptr || out_bf16 == nullptr ||
      ws == nullptr)
    return DS4X_EINVAL;
  if (!aligned16(kv_rows) || !aligned16(idx) || !aligned16(ring_rows) || !aligned16(q_bf16) ||
      !aligned16(out_bf16) || !aligned16(ws) || (lse != nullptr && !aligned16(lse)))
    return DS4X_EINVAL;
  if (n_rows < 1 || k < 1 || k > DS4X_TOPK_MAX || ring_pos < 0 || ring_pos >= DS4X_RING_ROWS || w < 0 ||
      w > DS4X_RING_ROWS)
    return DS4X_EINVAL;
  if (ws_bytes < ds4x_window_sparse_attn_decode_workspace()) return DS4X_EWORKSPACE;
  const int a = check_arch();
  if (a != DS4X_OK) return a;
  return from_cuda(launch_window_attn(kv_rows, n_rows, idx, k, ring_rows, ring_pos, w, q_bf16, softmax_scale,
                                      out_bf16, lse, ws, stream));
}

int ds4x_quantize_query_e4m3(const float *q, int64_t n_vec128, uint8_t *codes, uint8_t *scales,
                              ds4x_stream_t stream) {
  if (q == nullptr || codes == nullptr || scales == nullptr) return DS4X_EINVAL;
  if (!aligned16(q) || !aligned16(codes) || !aligned16(scales)) return DS4X_EINVAL;
  if (n_vec128 < 1 || n_vec128 > (int64_t(1) << 34)) return DS4X_EINVAL;
  const int a = check_arch();
  if (a != DS4X_OK) return a;
  return from_cuda(launch_quantize_query(q, n_vec128, codes, scales, stream));
}

size_t ds4x_index_score_topk_prefill_workspace(int64_t n_rows, int32_t n_queries, int32_t k) {
  (void)k;
  return prefill_ws_bytes(n_rows, n_queries);
}

int ds4x_index_score_topk_prefill(const uint8_t *idx_rows, int64_t n_rows, const uint8_t *q_codes,
                                  const uint8_t *q_scales, const float *w, int32_t n_queries, int64_t causal_base,
                                  int32_t k, int32_t *out_idx, float *out_score, void *ws, size_t ws_bytes,
                                  ds4x_stream_t stream) {
  if (idx_rows == nullptr || q_codes == nullptr || q_scales == nullptr || w == nullptr || out_idx == nullptr ||
      ws == nullptr)
    return DS4X_EINVAL;
  if (!aligned16(idx_rows) || !aligned16(q_codes) || !aligned16(q_scales) || !aligned16(w) || !aligned16(out_idx) ||
      !aligned16(ws) || (out_score != nullptr && !aligned16(out_score)))
    return DS4X_EINVAL;
  if (n_rows < 1 || n_rows > int64_t(INT32_MAX) || n_queries < 1 || n_queries > DS4X_PREFILL_MAX_QUERIES ||
      k < 1 || k > DS4X_TOPK_MAX)
    return DS4X_EINVAL;
  if (ws_bytes < ds4x_index_score_topk_prefill_workspace(n_rows, n_queries, k)) return DS4X_EWORKSPACE;
  const int a = check_arch();
  if (a != DS4X_OK) return a;
  return from_cuda(launch_score_prefill(idx_rows, n_rows, q_codes, q_scales, w, n_queries, causal_base, k, out_idx,
                                        out_score, ws, stream));
}

namespace {

// The cache's arguments, common to the paged calls.
int paged_cache(const uint8_t *pages, int64_t n_pages, int32_t page_rows, const int32_t *table, int32_t n_seqs,
                int32_t seq_pages, int64_t table_stride, const int32_t *cu_tokens, const void *ws, PagedCache *c) {
  if (pages == nullptr || table == nullptr || cu_tokens == nullptr || ws == nullptr) return DS4X_EINVAL;
  if (!aligned16(pages) || !aligned16(ws)) return DS4X_EINVAL;
  if (!aligned_to(table, 4) || !aligned_to(cu_tokens, 4)) return DS4X_EINVAL;
  if (n_pages < 1 || n_pages > int64_t(INT32_MAX) || n_seqs < 1 || n_seqs == INT32_MAX || seq_pages < 1)
    return DS4X_EINVAL;
  int lg = 4;
  while (lg < 8 && (1 << lg) != page_rows) ++lg;
  if ((1 << lg) != page_rows) return DS4X_EINVAL;
  if ((int64_t(seq_pages) << lg) > int64_t(INT32_MAX) || table_stride < seq_pages) return DS4X_EINVAL;
  *c = PagedCache{const_cast<uint8_t *>(pages), n_pages, table, table_stride, cu_tokens, n_seqs, seq_pages, lg};
  return DS4X_OK;
}

// A row array of n vectors of `dim` elements, `stride` elements apart, in whole 16 bytes.
bool paged_vectors(const void *p, int32_t type, int64_t stride, int64_t dim) {
  if (p == nullptr || !aligned16(p) || (type != DS4X_F32 && type != DS4X_BF16)) return false;
  return stride >= dim && stride <= (int64_t(1) << 40) && stride % (type == DS4X_BF16 ? 8 : 4) == 0;
}

// Whether two arrays of n vectors of `vec` bytes, as far apart as given, share a byte.
// Vectors that interleave at one stride do not; of other strides only arrays apart.
bool paged_overlap(const void *a, int64_t a_stride, const void *b, int64_t b_stride, int64_t vec, int64_t n) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  if (a0 >= b0 + uintptr_t(b_stride * (n - 1) + vec) || b0 >= a0 + uintptr_t(a_stride * (n - 1) + vec)) return false;
  if (n == 1 || a_stride != b_stride) return true;
  const uintptr_t s = uintptr_t(a_stride), d = b0 >= a0 ? (b0 - a0) % s : (s - (a0 - b0) % s) % s;
  return d < uintptr_t(vec) || s - d < uintptr_t(vec);
}

// Whether two arrays share no byte.
bool apart(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 >= b0 + uintptr_t(b_bytes) || b0 >= a0 + uintptr_t(a_bytes);
}

int paged_attn(PagedAttn &a, const uint8_t *pages, int64_t n_pages, int32_t page_rows, const int32_t *table,
               int32_t n_seqs, int32_t seq_pages, int64_t table_stride, const int32_t *cu_tokens, void *ws,
               size_t ws_bytes, ds4x_stream_t stream) {
  const int e = paged_cache(pages, n_pages, page_rows, table, n_seqs, seq_pages, table_stride, cu_tokens, ws, &a.c);
  if (e != DS4X_OK) return e;
  if (a.n_tokens < 1 || a.n_tokens > DS4X_PAGED_MAX_TOKENS || a.n_heads < 1 || a.n_heads > DS4X_PAGED_MAX_HEADS)
    return DS4X_EINVAL;
  const int64_t vec = int64_t(a.n_heads) * DS4X_KV_DIM;
  if (!paged_vectors(a.q, DS4X_BF16, a.q_stride, vec) || !paged_vectors(a.out, DS4X_BF16, a.out_stride, vec))
    return DS4X_EINVAL;
  if (a.lse != nullptr && !aligned_to(a.lse, 4)) return DS4X_EINVAL;
  // a token's heads may be computed apart, so its output must not lie where its query does
  if (paged_overlap(a.q, 2 * a.q_stride, a.out, 2 * a.out_stride, 2 * vec, a.n_tokens)) return DS4X_EINVAL;
  if (ws_bytes < paged_attn_ws_bytes()) return DS4X_EWORKSPACE;
  const int arch = check_arch();
  if (arch != DS4X_OK) return arch;
  return from_cuda(launch_paged_attn(a, ws, stream));
}

}  // namespace

int ds4x_paged_append(uint8_t *pages, int64_t n_pages, int32_t page_rows, const int32_t *table, int32_t n_seqs,
                      int32_t seq_pages, int64_t table_stride, const int32_t *cu_tokens, const int64_t *row0,
                      const void *kv_in, int32_t in_type, int64_t in_stride, int64_t n_tokens, const int64_t *pos,
                      const float *inv_freq, int32_t rope_style, void *ws, size_t ws_bytes, ds4x_stream_t stream) {
  PagedCache c;
  const int e = paged_cache(pages, n_pages, page_rows, table, n_seqs, seq_pages, table_stride, cu_tokens, ws, &c);
  if (e != DS4X_OK) return e;
  if (row0 == nullptr || !aligned_to(row0, 8) || !aligned_to(pos, 8) || !aligned_to(inv_freq, 4)) return DS4X_EINVAL;
  if (!paged_vectors(kv_in, in_type, in_stride, DS4X_KV_DIM)) return DS4X_EINVAL;
  if (n_tokens < 1 || n_tokens > int64_t(INT32_MAX)) return DS4X_EINVAL;
  if (rope_style != DS4X_ROPE_INTERLEAVED && rope_style != DS4X_ROPE_HALVES) return DS4X_EINVAL;
  if (ws_bytes < kWsHeaderBytes) return DS4X_EWORKSPACE;
  const int arch = check_arch();
  if (arch != DS4X_OK) return arch;
  return from_cuda(launch_paged_append(c, row0, kv_in, in_type == DS4X_BF16, in_stride, n_tokens, pos, inv_freq,
                                       rope_style == DS4X_ROPE_HALVES, ws, stream));
}

int ds4x_paged_gather(const uint8_t *pages, int64_t n_pages, int32_t page_rows, const int32_t *table, int32_t n_seqs,
                      int32_t seq_pages, int64_t table_stride, const int32_t *cu_tokens, const int64_t *row0,
                      void *out, int32_t out_type, int64_t out_stride, int64_t n_tokens, void *ws, size_t ws_bytes,
                      ds4x_stream_t stream) {
  PagedCache c;
  const int e = paged_cache(pages, n_pages, page_rows, table, n_seqs, seq_pages, table_stride, cu_tokens, ws, &c);
  if (e != DS4X_OK) return e;
  if (row0 == nullptr || !aligned_to(row0, 8)) return DS4X_EINVAL;
  if (!paged_vectors(out, out_type, out_stride, DS4X_KV_DIM)) return DS4X_EINVAL;
  if (n_tokens < 1 || n_tokens > int64_t(INT32_MAX)) return DS4X_EINVAL;
  if (ws_bytes < kWsHeaderBytes) return DS4X_EWORKSPACE;
  const int arch = check_arch();
  if (arch != DS4X_OK) return arch;
  return from_cuda(launch_paged_gather(c, row0, out, out_type == DS4X_BF16, out_stride, n_tokens, ws, stream));
}

int ds4x_paged_keep(uint8_t *pages, int64_t n_pages, int32_t page_rows, const int32_t *table, int32_t n_seqs,
                    int32_t seq_pages, int64_t table_stride, const int32_t *cu_tokens, const int64_t *row0,
                    const int32_t *path, const int32_t *n_path, int64_t n_tokens, void *ws, size_t ws_bytes,
                    ds4x_stream_t stream) {
  PagedCache c;
  const int e = paged_cache(pages, n_pages, page_rows, table, n_seqs, seq_pages, table_stride, cu_tokens, ws, &c);
  if (e != DS4X_OK) return e;
  if (row0 == nullptr || path == nullptr || n_path == nullptr) return DS4X_EINVAL;
  if (!aligned_to(row0, 8) || !aligned_to(path, 4) || !aligned_to(n_path, 4)) return DS4X_EINVAL;
  if (n_tokens < 1 || n_tokens > int64_t(INT32_MAX)) return DS4X_EINVAL;
  if (ws_bytes < kWsHeaderBytes) return DS4X_EWORKSPACE;
  const int arch = check_arch();
  if (arch != DS4X_OK) return arch;
  return from_cuda(launch_paged_keep(c, row0, path, n_path, n_tokens, ws, stream));
}

int ds4x_verify_drafts(const int32_t *cu_tokens, int32_t n_seqs, int64_t n_tokens, const int32_t *parent,
                       const int32_t *tokens, const void *target, int64_t target_stride, const void *draft,
                       int64_t draft_stride, int32_t type, int32_t vocab, const float *u, int32_t *path,
                       int32_t *out_tokens, int32_t *n_path, void *ws, size_t ws_bytes, ds4x_stream_t stream) {
  if (cu_tokens == nullptr || parent == nullptr || tokens == nullptr || u == nullptr || path == nullptr ||
      out_tokens == nullptr || n_path == nullptr || ws == nullptr)
    return DS4X_EINVAL;
  if (!aligned_to(cu_tokens, 4) || !aligned_to(parent, 4) || !aligned_to(tokens, 4) || !aligned_to(u, 4) ||
      !aligned_to(path, 4) || !aligned_to(out_tokens, 4) || !aligned_to(n_path, 4) || !aligned16(ws))
    return DS4X_EINVAL;
  if (n_seqs < 1 || n_seqs == INT32_MAX || n_tokens < 1 || n_tokens > int64_t(INT32_MAX) || vocab < 1 ||
      vocab > DS4X_VERIFY_MAX_VOCAB)
    return DS4X_EINVAL;
  if (!paged_vectors(target, type, target_stride, vocab) ||
      (draft != nullptr && !paged_vectors(draft, type, draft_stride, vocab)))
    return DS4X_EINVAL;
  // no output shares memory with another array
  const int64_t tb = 4 * n_tokens, sb = 4 * int64_t(n_seqs), row = vocab * int64_t(type == DS4X_BF16 ? 2 : 4);
  const struct {
    const void *p;
    int64_t bytes;
  } with[] = {{path, tb}, {out_tokens, tb}, {n_path, sb}, {cu_tokens, sb + 4}, {parent, tb}, {tokens, tb}, {u, tb},
              {ws, int64_t(kWsHeaderBytes)},
              {target, row + (n_tokens - 1) * target_stride * (type == DS4X_BF16 ? 2 : 4)},
              {draft, draft != nullptr ? row + (n_tokens - 1) * draft_stride * (type == DS4X_BF16 ? 2 : 4) : 0}};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 10; ++j)
      if (with[j].bytes > 0 && !apart(with[i].p, with[i].bytes, with[j].p, with[j].bytes)) return DS4X_EINVAL;
  if (ws_bytes < kWsHeaderBytes) return DS4X_EWORKSPACE;
  const int arch = check_arch();
  if (arch != DS4X_OK) return arch;
  return from_cuda(launch_verify(Verify{cu_tokens, n_seqs, n_tokens, parent, tokens, target, draft, target_stride,
                                        draft_stride, vocab, u, path, out_tokens, n_path},
                                 type == DS4X_BF16, ws, stream));
}

size_t ds4x_paged_attn_workspace(void) { return paged_attn_ws_bytes(); }

int ds4x_paged_attn(const uint8_t *pages, int64_t n_pages, int32_t page_rows, const int32_t *table, int32_t n_seqs,
                    int32_t seq_pages, int64_t table_stride, const int32_t *cu_tokens, const int64_t *row_begin,
                    const int64_t *row_end, int32_t n_tokens, int32_t n_heads, const uint16_t *q_bf16,
                    int64_t q_stride, float softmax_scale, uint16_t *out_bf16, int64_t out_stride, float *lse,
                    void *ws, size_t ws_bytes, ds4x_stream_t stream) {
  if (row_end == nullptr || !aligned_to(row_end, 8) || !aligned_to(row_begin, 8)) return DS4X_EINVAL;
  PagedAttn a{PagedCache{}, row_begin, row_end, nullptr, nullptr, 0, n_tokens, n_heads, q_bf16, q_stride,
              softmax_scale, out_bf16, out_stride, lse};
  return paged_attn(a, pages, n_pages, page_rows, table, n_seqs, seq_pages, table_stride, cu_tokens, ws, ws_bytes,
                    stream);
}

int ds4x_paged_sparse_attn(const uint8_t *pages, int64_t n_pages, int32_t page_rows, const int32_t *table,
                           int32_t n_seqs, int32_t seq_pages, int64_t table_stride, const int32_t *cu_tokens,
                           const int64_t *n_rows, const int32_t *idx, int32_t k, int32_t n_tokens, int32_t n_heads,
                           const uint16_t *q_bf16, int64_t q_stride, float softmax_scale, uint16_t *out_bf16,
                           int64_t out_stride, float *lse, void *ws, size_t ws_bytes, ds4x_stream_t stream) {
  if (n_rows == nullptr || idx == nullptr || !aligned_to(n_rows, 8) || !aligned_to(idx, 4)) return DS4X_EINVAL;
  if (k < 1 || k > DS4X_PAGED_MAX_LIST) return DS4X_EINVAL;
  PagedAttn a{PagedCache{}, nullptr, nullptr, n_rows, idx, k, n_tokens, n_heads, q_bf16, q_stride,
              softmax_scale, out_bf16, out_stride, lse};
  return paged_attn(a, pages, n_pages, page_rows, table, n_seqs, seq_pages, table_stride, cu_tokens, ws, ws_bytes,
                    stream);
}

int ds4x_paged_tree_attn(const uint8_t *pages, int64_t n_pages, int32_t page_rows, const int32_t *table,
                         int32_t n_seqs, int32_t seq_pages, int64_t table_stride, const int32_t *cu_tokens,
                         const int64_t *row0, const int32_t *parent, const int64_t *row_begin, int32_t n_tokens,
                         int32_t n_heads, const uint16_t *q_bf16, int64_t q_stride, float softmax_scale,
                         uint16_t *out_bf16, int64_t out_stride, float *lse, void *ws, size_t ws_bytes,
                         ds4x_stream_t stream) {
  if (row0 == nullptr || parent == nullptr || !aligned_to(row0, 8) || !aligned_to(parent, 4) ||
      !aligned_to(row_begin, 8))
    return DS4X_EINVAL;
  PagedAttn a{PagedCache{}, row_begin, nullptr, nullptr, nullptr, 0, n_tokens, n_heads, q_bf16, q_stride,
              softmax_scale, out_bf16, out_stride, lse, row0, parent};
  return paged_attn(a, pages, n_pages, page_rows, table, n_seqs, seq_pages, table_stride, cu_tokens, ws, ws_bytes,
                    stream);
}

}  // extern "C"
