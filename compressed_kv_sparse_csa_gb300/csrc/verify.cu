// Which drafted tokens stand: the walk over each sequence's draft by the target's
// and the draft's probabilities (include/ds4x.h, ds4x_verify_drafts).
//
// A block a sequence.
#include <cuda_bf16.h>

#include "paged.cuh"

namespace ds4x {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ float prob(const void *p, int64_t at) {
  const float v = BF16 ? __bfloat162float(__ushort_as_bfloat16(__ldcg(static_cast<const uint16_t *>(p) + at)))
                       : __ldcg(static_cast<const float *>(p) + at);
  return fmaxf(v, 0.0f);
}

__device__ __forceinline__ double block_sum(double v, double *red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = 0.0;
  for (int k = 0; k < kThreads / 32; ++k) v += red[k];
  return v;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) verify_kernel(Verify v, WsHeader *__restrict__ hdr) {
  __shared__ double red[kThreads / 32];
  __shared__ int16_t parent[DS4X_TREE_MAX_NODES];
  __shared__ int found;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t from = max(0, __ldcg(v.cu + s)), to = min(v.n_tokens, int64_t(__ldcg(v.cu + s + 1)));
  const int64_t all = max(int64_t(0), to - from);
  const bool many = all > DS4X_TREE_MAX_NODES;
  const int nodes = many ? 0 : int(all);
  bool odd = many;
  for (int64_t i = tid; i < all; i += kThreads) {
    v.path[from + i] = v.out[from + i] = -1;
    if (many) continue;
    const int32_t p = __ldcg(v.parent + from + i);
    const bool bad = p < -1 || p >= i;
    odd = odd || bad;
    parent[i] = int16_t(bad ? -1 : p);
  }
  if (odd) atomicExch(&hdr->status, int32_t(DS4X_EDEVICE));
  __syncthreads();
  if (nodes == 0) {
    if (tid == 0) v.n_path[s] = 0;
    return;
  }
  // the walk, the same in every thread
  int cur = 0, count = 1, last = 0;  // last: the latest child of cur that was tried (0: none)
  double t = 0.0, C = 1.0;
  if (tid == 0) v.path[from] = 0;
  const auto p_at = [&](int64_t y) { return prob<BF16>(v.target, (from + cur) * v.target_stride + y); };
  const auto q_at = [&](int64_t y) { return prob<BF16>(v.draft, (from + cur) * v.draft_stride + y); };
  const auto tried = [&](int32_t y) {  // without the draft's probabilities
    for (int j = cur + 1; j <= last; ++j)
      if (parent[j] == cur && __ldcg(v.tokens + from + j) == y) return true;
    return false;
  };
  const auto weight = [&](int32_t y) {
    if (v.draft != nullptr) return fmax(double(p_at(y)) - t * double(q_at(y)), 0.0);
    return tried(y) ? 0.0 : double(p_at(y));
  };
  for (int j = 1; j < nodes; ++j) {
    if (parent[j] != cur) continue;
    const int32_t x = __ldcg(v.tokens + from + j);
    const bool in = x >= 0 && x < v.vocab;
    if (!in && tid == 0) atomicExch(&hdr->status, int32_t(DS4X_EDEVICE));
    const double w = in ? weight(x) : 0.0, q = v.draft == nullptr ? 1.0 : in ? double(q_at(x)) : 0.0;
    if (double(__ldcg(v.u + from + j)) * q * C < w) {
      if (tid == 0) {
        v.path[from + count] = j;
        v.out[from + count - 1] = x;
      }
      cur = j;
      ++count;
      last = 0;
      t = 0.0;
      C = 1.0;
      continue;
    }
    last = j;
    if (v.draft != nullptr) {
      t += C;
      double sum = 0.0;
      for (int y = tid; y < v.vocab; y += kThreads) sum += weight(y);
      C = block_sum(sum, red);
    } else {
      C -= w;
    }
  }
  // the last token
  double sum = 0.0;
  for (int y = tid; y < v.vocab; y += kThreads) sum += weight(y);
  const double total = block_sum(sum, red), want = double(__ldcg(v.u + from)) * total;
  double before = 0.0;
  if (tid == 0) found = -1;
  int latest = -1;  // the last token with a weight
  for (int y0 = 0; y0 < v.vocab; y0 += kThreads) {
    const int y = y0 + tid;
    const double w = y < v.vocab ? weight(y) : 0.0;
    double incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) red[warp] = incl;
    __syncthreads();
    double base = before, whole = before;
    for (int k = 0; k < kThreads / 32; ++k) {
      if (k < warp) base += red[k];
      whole += red[k];
    }
    if (w > 0.0) {
      latest = y;
      if (base + incl > want) atomicCAS(&found, -1, y), atomicMin(&found, y);
    }
    __syncthreads();
    if (found >= 0) break;
    before = whole;
  }
  if (found < 0) {  // (rounding, or no weight at all)
    __syncthreads();
    atomicMax(&found, latest);
    __syncthreads();
  }
  if (tid == 0) {
    v.out[from + count - 1] = found;
    v.n_path[s] = count;
    if (found < 0) atomicExch(&hdr->status, int32_t(DS4X_EDEVICE));
  }
}

}  // namespace

cudaError_t launch_verify(const Verify &v, bool bf16, void *ws, cudaStream_t stream) {
  return launch_pdl(bf16 ? verify_kernel<true> : verify_kernel<false>, unsigned(v.n_seqs), unsigned(kThreads), 0, stream,
                    v, static_cast<WsHeader *>(ws));
}

}  // namespace ds4x
