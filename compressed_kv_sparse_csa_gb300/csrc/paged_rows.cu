// The paged 4-bit cache's writer and reader.
//
// Append: one warp a row.  Lane L holds the row's 8-value chunks L and 32 + L:
// chunks 0-55 are non-RoPE values (four lanes to a 32-value block), chunks
// 56-63 (lanes 24-31) the RoPE part.  The rotation's 32 pairs take a lane
// each for their angle.  pos * inv_freq is formed as a fraction of a turn in
// 64-bit fixed point: f = inv_freq / 2 pi (its whole turns dropped) has 64
// fraction bits, and pos * f wraps modulo 2^64 = modulo a turn by itself.  So
// the angle is off by the last of those bits, pos * 2^-63 turns at most for
// frequencies below 2^9 turns (a float product would be off by 2^-5 radians at
// position 2^20); its upper 32 bits go to sincospi.  Scales by exact comparisons (block_exponent), codes by the
// hardware's round-to-nearest-even conversion.
//
// Global loads here and in the attention go by L2 (ld.global.cg): the kernels
// are programmatic dependents, so a line that an earlier kernel left in L1 may
// be older than what the previous kernel wrote.
//
// What bounds them: bytes in the end (append: 1024 or 2048 in and 368 out a row,
// gather: 367 in and 1024 or 2048 out), so loads and stores are 16 bytes a lane but
// for the codes (4 bytes a lane, 128 consecutive bytes a warp); at the sizes that a
// step has, the chain cu -> row0 -> table -> page, a round trip to memory each.
// 16384 tokens in bf16 appended and read back: 23.4 us, 2.0 TB/s (in a graph, rows in L2,
// 13.1 and 8.6 us); one token: 17 us, of which the calls' host side is 15.  Several tokens
// a warp let one search, one page and one forming of the turns serve them, and the next
// one's words are on their way while one is worked on.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "paged.cuh"

namespace ds4x {
namespace {

constexpr int kWarps = 8;
constexpr int kTailLane = 24;  // lanes 24-31: the RoPE part (chunks 56-63)
constexpr double kInv2PiHi = 0.15915494309189535, kInv2PiLo = -9.839338337591243e-18;  // 1 / 2 pi

// Two floats -> one byte of two E2M1 codes: `lo` in bits 0-3, `hi` in bits 4-7.
__device__ __forceinline__ uint32_t cvt_e2m1x2(float hi, float lo) {
  uint16_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u16.u8 %0, t;\n\t}"
      : "=h"(r) : "f"(hi), "f"(lo));
  return r & 0xffu;
}
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float s) {
  return cvt_e2m1x2(v[1] * s, v[0] * s) | cvt_e2m1x2(v[3] * s, v[2] * s) << 8 | cvt_e2m1x2(v[5] * s, v[4] * s) << 16 |
         cvt_e2m1x2(v[7] * s, v[6] * s) << 24;
}
// block_exponent (ds4x_internal.cuh) with this format's exponent range; an
// all-zero block takes the least exponent.
__device__ __forceinline__ int paged_exponent(float amax, float g, int G) {
  if (amax == 0.0f) return kPgExpMin;
  return max(kPgExpMin, min(kPgExpMax, block_exponent(amax, g, G)));
}
// The largest |v|; NaN where one is.
__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[i])));
  return m;
}
// NaN to zero, infinities to the largest floats.
__device__ __forceinline__ float finite(float v) {
  return v == v ? fminf(fmaxf(v, -FLT_MAX), FLT_MAX) : 0.0f;
}

// Eight values as they lie in memory.
template <bool BF16>
struct Words {
  uint4 w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void *in, int64_t at) {
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(in) + at * (BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) w[i] = __ldcg(p + i);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (BF16) {
          v[2 * k] = __uint_as_float(u[k] << 16);
          v[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
        } else {
          v[4 * i + k] = __uint_as_float(u[k]);
        }
      }
    }
  }
};

// The tokens of a warp: `per` in a row, so that a sequence found serves the next.
struct Tokens {
  int64_t t, end;
  __device__ __forceinline__ Tokens(int64_t n, int64_t per) {
    t = (int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * per;
    end = min(n, t + per);
  }
};

// Where token after token lies: the sequence and the page found for one serve the
// next while they hold.
struct Places {
  PagedSeq sq{-1, 0, 0};
  int64_t first_row = 0, r = 0;
  PagedRow p{nullptr, 0};
  // false: padding
  __device__ __forceinline__ bool find(const PagedCache &c, const int64_t *row0, int64_t t, int lane) {
    const int64_t before = r;
    const bool known = sq.s >= 0 && t < sq.to;
    if (!known) {
      sq = paged_seq_of(c, t, lane);
      if (sq.s < 0) return false;
      first_row = __ldcg(row0 + sq.s);
    }
    r = first_row + (t - sq.from);
    if (known && p.page != nullptr && r >> c.page_log2 == before >> c.page_log2)
      p.at = int32_t(r & ((1 << c.page_log2) - 1));
    else
      p = paged_row(c, sq.s, r);
    return true;
  }
};

template <bool BF16>
__global__ void __launch_bounds__(kWarps * 32)
paged_append_kernel(PagedCache c, const int64_t *__restrict__ row0, const void *__restrict__ in, int64_t in_stride,
                    int64_t n, int64_t per, const int64_t *__restrict__ pos, const float *__restrict__ inv_freq,
                    int halves, WsHeader *__restrict__ hdr) {
  __shared__ unsigned long long turn[32];  // pair i's turn a position, 2^-64 turns
  // launched as a programmatic dependent: past this wait the previous kernel
  // (say the one that formed kv_in) is complete and visible
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  Tokens tk(n, per);
  // (the block's one warp that does it: 64-bit floating point is slow here, and a
  // warp a token spent more time on it than on everything else)
  if (inv_freq != nullptr && threadIdx.x < 32) {
    // inv_freq / 2 pi as t + e, 1 / 2 pi in two doubles; the whole turns of t
    // dropped exactly, then 64 fraction bits of both
    const double w = double(__ldcg(inv_freq + lane));
    const double t0 = w * kInv2PiHi, e0 = fma(w, kInv2PiHi, -t0) + w * kInv2PiLo;
    const double fr = t0 - floor(t0);
    turn[lane] = (fr < 1.0 ? (unsigned long long)(fr * 18446744073709551616.0) : 0ull) +
                 (unsigned long long)((long long)(e0 * 18446744073709551616.0));
  }
  Places at_row;
  bool ready = inv_freq == nullptr;
  // (a named barrier: a warp without a token waits at another place than the rest)
  auto turns_made = [] { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); };
  if (tk.t >= tk.end && !ready) turns_made();
  Words<BF16> wa, wb;  // the next token's, on their way while one is worked on
  int64_t next_pos = 0;
  auto load = [&](int64_t t) {
    wa.load(in, t * in_stride + 8 * lane);
    wb.load(in, t * in_stride + 256 + 8 * lane);
    next_pos = pos != nullptr ? __ldcg(pos + t) : 0;
  };
  if (tk.t < tk.end) load(tk.t);
  for (; tk.t < tk.end; ++tk.t) {
    const int64_t t = tk.t;
    const bool token = at_row.find(c, row0, t, lane);
    const PagedRow p = token ? at_row.p : PagedRow{nullptr, 0};
    const int64_t r = at_row.r, place = next_pos;
    float a[8], b[8];
    wa.values(a);
    wb.values(b);
    if (t + 1 < tk.end) load(t + 1);
    if (!ready) {
      turns_made();
      ready = true;
    }
    if (p.page == nullptr) {
      if (token && lane == 0) atomicExch(&hdr->status, int32_t(DS4X_EDEVICE));
      continue;
    }
    if (inv_freq != nullptr) {
      // lane i: pair i's angle
      const uint64_t at = turn[lane] * uint64_t(pos != nullptr ? place : r);
      float sn, cs;
      sincospif(float(int32_t(uint32_t(at >> 32))) * 4.656612873077393e-10f, &sn, &cs);  // half turns: * 2^-31
      const bool tail = lane >= kTailLane;
      if (halves) {  // elements i and 32 + i: lanes 24-27 hold the first of each pair, 28-31 the second
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int pair = 8 * (lane & 3) + i;
          const float ci = __shfl_sync(0xffffffffu, cs, pair), si = __shfl_sync(0xffffffffu, sn, pair);
          const float o = __shfl_xor_sync(0xffffffffu, b[i], 4);
          if (tail) b[i] = (lane & 4) ? b[i] * ci + o * si : b[i] * ci - o * si;
        }
      } else {  // elements 2 i and 2 i + 1
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int pair = (4 * (lane - kTailLane) + i) & 31;
          const float ci = __shfl_sync(0xffffffffu, cs, pair), si = __shfl_sync(0xffffffffu, sn, pair);
          const float x = b[2 * i], y = b[2 * i + 1];
          if (tail) {
            b[2 * i] = x * ci - y * si;
            b[2 * i + 1] = x * si + y * ci;
          }
        }
      }
    }
    // block maxima over four lanes, the RoPE part's over lanes 24-31
    float ma = amax8(a), mb = amax8(b);
    if (__any_sync(0xffffffffu, !(ma <= FLT_MAX && mb <= FLT_MAX))) {  // rows hold finite values only
      if (lane == 0) atomicExch(&hdr->status, int32_t(DS4X_EDEVICE));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = finite(a[i]);
        b[i] = finite(b[i]);
      }
      ma = amax8(a);
      mb = amax8(b);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, o));
      mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
    }
    const float m4 = __shfl_xor_sync(0xffffffffu, mb, 4);
    const int ea = paged_exponent(ma, 0.75f, 3);  // 6 = 0.75 * 2^3
    const int eb = lane < kTailLane ? paged_exponent(mb, 0.75f, 3)
                                    : paged_exponent(fmaxf(mb, m4), 0.5f, 4);  // 8 = 0.5 * 2^4
    const int E = __reduce_max_sync(0xffffffffu, max(ea, eb));  // the RoPE part's: the row's largest

    uint8_t *page = const_cast<uint8_t *>(p.page);
    uint8_t *codes = page + paged_code_off(p);
    *reinterpret_cast<uint32_t *>(codes + 4 * lane) = codes8(a, pow2_neg(ea));
    if (lane < kTailLane) {
      *reinterpret_cast<uint32_t *>(codes + 128 + 4 * lane) = codes8(b, pow2_neg(eb));
    } else {
      const float f = pow2_neg(E);
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = fminf(fmaxf(b[2 * i] * f, -65504.0f), 65504.0f);
        const float hi = fminf(fmaxf(b[2 * i + 1] * f, -65504.0f), 65504.0f);
        const __half2 v = __floats2half2_rn(lo, hi);
        h[i] = *reinterpret_cast<const uint32_t *>(&v);
      }
      *reinterpret_cast<uint4 *>(page + paged_tail_off(c, p) + 16 * (lane - kTailLane)) =
          make_uint4(h[0], h[1], h[2], h[3]);
    }
    // the scale record: byte i < 8 from lane 4 i's first chunk, 8 .. 13 from lane
    // 4 (i - 8)'s second, 14 the RoPE part's
    const uint32_t ba = uint32_t(ea + 127), bb = uint32_t(eb + 127);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2] |= __shfl_sync(0xffffffffu, ba, 4 * i) << (8 * (i & 3));
#pragma unroll
    for (int i = 8; i < kPgBlocks; ++i) w[i >> 2] |= __shfl_sync(0xffffffffu, bb, 4 * (i - 8)) << (8 * (i & 3));
    w[3] |= uint32_t(E + 127) << 16;
    if (lane == 0) *reinterpret_cast<uint4 *>(page + paged_scale_off(c, p)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Eight values as bf16 or f32.
template <bool BF16>
__device__ __forceinline__ void store8(void *out, int64_t at, const float (&v)[8]) {
  if (BF16) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ float pow2_byte(uint32_t b) {  // 2^(b - 127), any byte (255: infinity)
  return b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}
__device__ __forceinline__ void decode8(uint32_t w, float s, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t n = (w >> (4 * i)) & 15u;
    // E2M1 as a half: exponent and mantissa bits moved up read 2^-14 times the value
    const float m = __half2float(__ushort_as_half(uint16_t((n & 7u) << 9))) * 16384.0f;
    v[i] = (n & 8u ? -m : m) * s;
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kWarps * 32)
paged_gather_kernel(PagedCache c, const int64_t *__restrict__ row0, void *__restrict__ out, int64_t out_stride,
                    int64_t n, int64_t per, WsHeader *__restrict__ hdr) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  // a row's words, the next one's on their way while one is worked on
  struct Row {
    bool token, placed;
    uint32_t a, b, sa, sb;
    uint4 h;
  };
  Places at_row;
  auto load = [&](int64_t t) {
    Row w;
    w.token = at_row.find(c, row0, t, lane);
    const PagedRow p = at_row.p;
    w.placed = w.token && p.page != nullptr;
    if (w.placed) {
      const uint8_t *codes = p.page + paged_code_off(p), *sc = p.page + paged_scale_off(c, p);
      w.a = __ldcg(reinterpret_cast<const uint32_t *>(codes + 4 * lane));
      w.sa = __ldcg(sc + (lane >> 2));
      if (lane < kTailLane) {
        w.b = __ldcg(reinterpret_cast<const uint32_t *>(codes + 128 + 4 * lane));
        w.sb = __ldcg(sc + 8 + (lane >> 2));
      } else {
        w.h = __ldcg(reinterpret_cast<const uint4 *>(p.page + paged_tail_off(c, p) + 16 * (lane - kTailLane)));
        w.sb = __ldcg(sc + kPgTailScale);
      }
    }
    return w;
  };
  Tokens tk(n, per);
  Row next{};
  if (tk.t < tk.end) next = load(tk.t);
  for (; tk.t < tk.end; ++tk.t) {
    const int64_t t = tk.t;
    const Row w = next;
    if (t + 1 < tk.end) next = load(t + 1);
    if (!w.token) continue;
    float a[8], b[8];
    if (!w.placed) {
      if (lane == 0) atomicExch(&hdr->status, int32_t(DS4X_EDEVICE));
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = b[i] = 0.0f;
    } else {
      const float f = pow2_byte(w.sb);
      if (lane < kTailLane) {
        decode8(w.b, f, b);
      } else {
        const uint32_t u[4] = {w.h.x, w.h.y, w.h.z, w.h.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
          b[2 * i] = v.x * f;
          b[2 * i + 1] = v.y * f;
        }
      }
      decode8(w.a, pow2_byte(w.sa), a);
    }
    store8<BF16>(out, t * out_stride + 8 * lane, a);
    store8<BF16>(out, t * out_stride + 256 + 8 * lane, b);
  }
}

}  // namespace

namespace {
// Tokens a warp, so that the grid is at most what the GPU holds at once (4 blocks an
// SM, by the registers).  16384 tokens appended and read back take 23.2 us so, 24.3
// with 8 blocks an SM, 25.4 with 2, 33 with a token a warp.
cudaError_t tokens_per_warp(int64_t n, int64_t *per, unsigned *blocks) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t warps = int64_t(sms) * 4 * kWarps;
  *per = (n + warps - 1) / warps;
  *blocks = unsigned((n + *per * kWarps - 1) / (*per * kWarps));
  return cudaSuccess;
}
}  // namespace

cudaError_t launch_paged_append(const PagedCache &c, const int64_t *row0, const void *in, bool in_bf16,
                                int64_t in_stride, int64_t n, const int64_t *pos, const float *inv_freq, bool halves,
                                void *ws, cudaStream_t stream) {
  int64_t per;
  unsigned blocks;
  const cudaError_t e = tokens_per_warp(n, &per, &blocks);
  if (e != cudaSuccess) return e;
  WsHeader *hdr = static_cast<WsHeader *>(ws);
  return launch_pdl(in_bf16 ? paged_append_kernel<true> : paged_append_kernel<false>, blocks, kWarps * 32, 0, stream,
                    c, row0, in, in_stride, n, per, pos, inv_freq, int(halves), hdr);
}

cudaError_t launch_paged_gather(const PagedCache &c, const int64_t *row0, void *out, bool out_bf16,
                                int64_t out_stride, int64_t n, void *ws, cudaStream_t stream) {
  int64_t per;
  unsigned blocks;
  const cudaError_t e = tokens_per_warp(n, &per, &blocks);
  if (e != cudaSuccess) return e;
  WsHeader *hdr = static_cast<WsHeader *>(ws);
  return launch_pdl(out_bf16 ? paged_gather_kernel<true> : paged_gather_kernel<false>, blocks, kWarps * 32, 0, stream,
                    c, row0, out, out_stride, n, per, hdr);
}

}  // namespace ds4x
