// Attention over the paged 4-bit cache.
//
//   l_hj = scale * (q_h . v_j),  o_h = sum_j softmax_j(l_h)_j v_j,
//   lse_h = log sum_j e^(l_hj)
//
// over a token's rows: the range [row_begin, row_end) of its sequence, or its
// own list of rows.  A CTA takes one token and eight heads, a head a warp (16
// of the 512 values a lane): tiles of 32 rows are widened to fp32 in shared
// memory, read by all eight warps, and each warp runs the softmax online with
// a running maximum and sum in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.cuh"

namespace ds4x {
namespace {

constexpr int kHeadsCta = 8;
constexpr int kThreads = kHeadsCta * 32;
constexpr int kTile = 32;

struct Smem {
  float v[kTile][DS4X_KV_DIM];
  int ok[kTile];
};

__device__ __forceinline__ float pow2_byte(uint32_t b) {
  return b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

__global__ void __launch_bounds__(kThreads) paged_attn_kernel(PagedAttn a, WsHeader *hdr) {
  extern __shared__ uint8_t smem_raw[];
  Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.x, h = blockIdx.y * kHeadsCta + warp;
  const int32_t s = paged_seq_of(a.c, t, lane);
  if (s < 0) return;
  int64_t r0 = 0, n;
  if (a.idx != nullptr) {
    n = a.k;
  } else {
    r0 = a.row_begin != nullptr ? max(int64_t(0), int64_t(__ldcg(a.row_begin + t))) : 0;
    // no further than the table goes (a range past it is the caller's error)
    const int64_t room = int64_t(a.c.seq_pages) << a.c.page_log2, end = __ldcg(a.row_end + t);
    if (end > room && tid == 0) atomicExch(&hdr->status, int32_t(DS4X_EDEVICE));
    n = max(int64_t(0), min(end, room) - r0);
  }
  const int64_t n_rows = a.idx != nullptr ? __ldcg(a.n_rows + s) : 0;
  float q[16], o[16], m = -INFINITY, sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    q[i] = h < a.n_heads ? __uint_as_float(uint32_t(a.q[t * a.q_stride + h * DS4X_KV_DIM + 32 * i + lane]) << 16) : 0.0f;
    o[i] = 0.0f;
  }
  for (int64_t j0 = 0; j0 < n; j0 += kTile) {
    __syncthreads();
    for (int j = warp; j < kTile; j += kHeadsCta) {
      PagedRow p{nullptr, 0};
      if (j0 + j < n) {
        int64_t r = r0 + j0 + j;
        bool bad = false;
        if (a.idx != nullptr) {
          r = __ldcg(a.idx + int64_t(t) * a.k + j0 + j);
          bad = r < -1 || r >= n_rows;
        }
        if (!bad && r >= 0) p = paged_row(a.c, s, r);
        if (p.page == nullptr && (bad || r >= 0) && lane == 0) atomicExch(&hdr->status, int32_t(DS4X_EDEVICE));
      }
      if (lane == 0) sm.ok[j] = p.page != nullptr;
      if (p.page == nullptr) continue;
      const uint8_t *sc = p.page + paged_scale_off(a.c, p), *co = p.page + paged_code_off(p);
#pragma unroll
      for (int i = 0; i < 7; ++i) {  // byte 32 i + lane: elements 64 i + 2 lane, + 1
        const uint32_t b = __ldcg(co + 32 * i + lane);
        const float f = pow2_byte(__ldcg(sc + 2 * i + (lane >> 4)));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t c4 = (b >> (4 * u)) & 15u;
          const float x = __half2float(__ushort_as_half(uint16_t((c4 & 7u) << 9))) * 16384.0f;
          sm.v[j][64 * i + 2 * lane + u] = (c4 & 8u ? -x : x) * f;
        }
      }
      const uint32_t w = __ldcg(reinterpret_cast<const uint32_t *>(p.page + paged_tail_off(a.c, p)) + lane);
      const float f = pow2_byte(__ldcg(sc + kPgTailScale));
      sm.v[j][DS4X_KV_NOPE + 2 * lane] = __half2float(__ushort_as_half(uint16_t(w))) * f;
      sm.v[j][DS4X_KV_NOPE + 2 * lane + 1] = __half2float(__ushort_as_half(uint16_t(w >> 16))) * f;
    }
    __syncthreads();
    for (int j = 0; j < kTile && j0 + j < n; ++j) {
      if (!sm.ok[j]) continue;
      float v[16], d = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[i] = sm.v[j][32 * i + lane];
        d = fmaf(q[i], v[i], d);
      }
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) d += __shfl_xor_sync(0xffffffffu, d, k);
      const float l = d * a.scale, mn = fmaxf(m, l);
      const float al = expf(m - mn), p = expf(l - mn);
      m = mn;
      sum = fmaf(sum, al, p);
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = fmaf(o[i], al, p * v[i]);
    }
  }
  if (h >= a.n_heads) return;
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    a.out[t * a.out_stride + h * DS4X_KV_DIM + 32 * i + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i] * inv));
  if (lane == 0 && a.lse != nullptr) a.lse[int64_t(t) * a.n_heads + h] = sum > 0.0f ? m + logf(sum) : -INFINITY;
}

}  // namespace

size_t paged_attn_ws_bytes() { return kWsHeaderBytes; }

cudaError_t launch_paged_attn(const PagedAttn &a, void *ws, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_set{0};
  const int smem = int(sizeof(Smem));
  cudaError_t e = set_max_smem_once(paged_attn_kernel, smem, smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(a.n_tokens), unsigned((a.n_heads + kHeadsCta - 1) / kHeadsCta));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_attn_kernel, a, reinterpret_cast<WsHeader *>(ws));
}

}  // namespace ds4x
