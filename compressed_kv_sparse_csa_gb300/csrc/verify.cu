// Which drafted tokens stand: the walk over each sequence's draft by the target's
// and the draft's probabilities (include/ds4x.h, ds4x_verify_drafts).
//
// With p and q of the node where the walk stands and t draws of q taken off, the
// rest of p is max(p - t q, 0) / C.  One rejection more makes it max(that - q, 0),
// renormalised: max(p - (t + C) q, 0) / C'.  So a node's whole history is the two
// numbers t and C, and each rejection is one pass over the rows for the next C.
// Without q the rest is p without the tokens tried, and C = 1 less theirs.
// Exact rows leave nothing only where a rejection has probability 0.  Rounded ones do in
// earnest (a bf16 probability from 0.998 up is 1, so p and q can be the same there and q larger
// elsewhere): then the last token is drawn from p as it is, which takes a pass over q's row
// (is it a distribution beside p?) and one over p's.
//
// What is read.  A child's decision needs p and q at one token: those of all
// children are fetched at once, beforehand, so the walk runs in shared memory.
// Only the node where it ends, and nodes with a second child, need rows: one pass
// of V probabilities each, which also leaves a sum for each 1024 of them, so that
// the last token is found by prefix sums and one look at 1024 again.
//
// Sums.  A token is chosen among up to 2^20 by where u falls between partial sums,
// so those must be far better than fp32: pairs of floats, hi + lo, by error-free
// additions (Knuth's two-sum) and products (by fma), good to 2^-44 or so of what is
// added, before t q is taken off.  Not fp64:
// a warp's instruction takes some 50 cycles of an SM's one pipe.  256 sequences of
// 131,072 tokens took 2.77 ms in fp64 throughout, and 206 us with fp64 from a warp's
// 1024 on alone.
//
// Work split.  A cluster of 1 to 16 blocks a sequence, a contiguous slice of the
// vocabulary each; every block walks by itself (the same numbers, the same order, so
// the same decisions), and after a pass each gives its sum to all blocks by an
// asynchronous store that counts on their barriers (a cluster barrier took 0.7 us
// longer a pass).  That wait is bounded (0.5 s).  Whether it ran out is agreed on by the
// whole block, so that its warps never part: after a time-out (DS4X_ETIMEOUT) a block makes
// no further pass, writes nothing and leaves with its cluster.  Another block may then
// miss its sum, and runs out in its turn, once.
//
// What bounds it.  Many sequences: DRAM, 256 chains of 8 over 131,072 tokens take 49.2 us
// (5.4 TB/s), 8 us of them before and after the rows; in bf16 36.2 us, the additions as
// many for half the bytes; without a draft 32.5 us, in bf16 27.4.  Few: latency, one chain of
// 6 takes 7.3 us, 16 trees of 32 nodes 10.4 us.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace ds4x {
namespace {

using namespace ptx;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunk = 1024;          // probabilities a warp sums at a time
constexpr int kMaxChunks = DS4X_VERIFY_MAX_VOCAB / kChunk;
constexpr int kMaxCluster = 16;
constexpr int kMaxNodes = DS4X_TREE_MAX_NODES;
constexpr unsigned long long kTimeoutNs = 500ull * 1000 * 1000;
constexpr unsigned long long kDrainNs = 10ull * 1000 * 1000;

// A number in two floats, hi + lo (|lo| at most half a step of hi).
struct __align__(8) Pair {
  float h, l;
};
__device__ __forceinline__ Pair pair(float h, float l) {  // |l| below |h|
  const float s = __fadd_rn(h, l);
  return Pair{s, __fadd_rn(l, -__fadd_rn(s, -h))};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const float s = __fadd_rn(a.h, b.h), bb = __fadd_rn(s, -a.h);
  const float e = __fadd_rn(__fadd_rn(a.h, -__fadd_rn(s, -bb)), __fadd_rn(b.h, -bb));
  return pair(s, __fadd_rn(e, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Pair operator*(float a, Pair b) {
  const float h = __fmul_rn(a, b.h);
  return pair(h, __fmaf_rn(a, b.l, __fmaf_rn(a, b.h, -h)));
}
__device__ __forceinline__ Pair operator-(Pair a) { return Pair{-a.h, -a.l}; }
__device__ __forceinline__ bool operator>(Pair a, Pair b) {
  return __fadd_rn(__fadd_rn(a.h, -b.h), __fadd_rn(a.l, -b.l)) > 0.0f;
}
__device__ __forceinline__ bool some(Pair a) { return a.h > 0.0f; }
__device__ __forceinline__ Pair shfl_up(Pair a, int o) {
  return Pair{__shfl_up_sync(0xffffffffu, a.h, o), __shfl_up_sync(0xffffffffu, a.l, o)};
}
__device__ __forceinline__ Pair shfl(Pair a, int lane) {
  return Pair{__shfl_sync(0xffffffffu, a.h, lane), __shfl_sync(0xffffffffu, a.l, lane)};
}
// A lane's sum over the lanes up to it.
__device__ __forceinline__ Pair warp_scan(Pair v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair x = shfl_up(v, o);
    if (lane >= o) v = x + v;
  }
  return v;
}

// A sum over each N lanes, the same in all of them.
template <int N = 32>
__device__ __forceinline__ Pair warp_sum(Pair v) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    const float h = __shfl_xor_sync(0xffffffffu, v.h, o), l = __shfl_xor_sync(0xffffffffu, v.l, o);
    const float s = __fadd_rn(v.h, h), bb = __fadd_rn(s, -v.h);
    const float e = __fadd_rn(__fadd_rn(v.h, -__fadd_rn(s, -bb)), __fadd_rn(h, -bb));
    v = Pair{s, __fadd_rn(e, __fadd_rn(v.l, l))};  // (made a pair once, at the end)
  }
  return pair(v.h, v.l);
}
// The first of n numbers where base and the sum up to it pass `want`, and has a part in it;
// without one (by rounding) the last that is not 0, or -1.  base: what comes before it then.
__device__ __forceinline__ int first_past(const Pair *v, int n, Pair want, Pair &base, int lane) {
  int found = -1;
  Pair found_base = base;
  for (int b = 0; b < n; b += 32) {
    const Pair mine = b + lane < n ? v[b + lane] : Pair{0.0f, 0.0f};
    const Pair upto = base + warp_scan(mine, lane);
    const uint32_t any = __ballot_sync(0xffffffffu, some(mine));
    const uint32_t over = __ballot_sync(0xffffffffu, some(mine) && upto > want);
    const int k = over != 0 ? __ffs(int(over)) - 1 : any != 0 ? 31 - __clz(any) : 0;
    const Pair prev = shfl(upto, max(k - 1, 0));
    if (any != 0) {
      found = b + k;
      found_base = k > 0 ? prev : base;
    }
    if (over != 0) break;
    base = shfl(upto, 31);
  }
  base = found_base;
  return found;
}

struct Shared {
  Pair sums[kMaxChunks];              // the block's chunks' sums of the latest pass
  Pair total[2][kMaxCluster];         // the blocks' (written by all of them), of this pass and the one before
  Pair red[kWarps];
  float p[kMaxNodes], q[kMaxNodes], u[kMaxNodes];  // of each node's token, after its parent
  int32_t token[kMaxNodes];           // outside the vocabulary: -1
  int16_t parent[kMaxNodes], path[kMaxNodes];
  Pair base, drafted;                 // (drafted: the sum of a draft's whole row)
  int chunk, found, abort_flag;
  unsigned long long given[2];        // barriers of the totals
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// *p of the cluster's block r, and eight bytes on its barrier
__device__ __forceinline__ void give(Pair *p, unsigned long long *bar, uint32_t r, Pair v) {
  const unsigned long long bits =
      (unsigned long long)(__float_as_uint(v.l)) << 32 | (unsigned long long)(__float_as_uint(v.h));
  asm volatile(
      "{\n\t.reg .b32 x, y;\n\tmapa.shared::cluster.u32 x, %0, %2;\n\tmapa.shared::cluster.u32 y, %1, %2;\n\t"
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [x], %3, [y];\n\t}" ::"r"(smem_u32(p)),
      "r"(smem_u32(bar)), "r"(r), "l"(bits)
      : "memory");
}

__device__ __forceinline__ unsigned long long globaltimer() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Whether the phase came in time (a thread's own finding: others may find otherwise).
__device__ __forceinline__ bool wait_slowly(Shared &sm, uint32_t bar, uint32_t parity, WsHeader *hdr) {
  const unsigned long long t0 = globaltimer();
  for (;;) {
    for (int k = 0; k < 64; ++k)
      if (mbar_try_wait_sleep(bar, parity, 2000)) return true;
    if (*reinterpret_cast<volatile int *>(&sm.abort_flag)) return false;
    if (globaltimer() - t0 > kTimeoutNs) {
      atomicExch(&hdr->status, int32_t(DS4X_ETIMEOUT));
      *reinterpret_cast<volatile int *>(&sm.abort_flag) = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_bar(Shared &sm, unsigned long long *bar, uint32_t parity, WsHeader *hdr) {
  const uint32_t b = smem_u32(bar);
  return mbar_try_wait(b, parity) || wait_slowly(sm, b, parity, hdr);
}

// NaN and negative ones count as zero.
__device__ __forceinline__ float clean(float v) { return fmaxf(v, 0.0f); }

// N probabilities in a row, from element y on (a multiple of N; from `end` on: 0).
template <bool BF16, int N>
struct Probs {
  static_assert(N * (BF16 ? 2 : 4) <= 16, "one load");
  uint32_t w[N * (BF16 ? 2 : 4) / 4];
  __device__ __forceinline__ void load(const void *row, int y, int end) {
    if (y + N <= end) {
      const uint8_t *at = static_cast<const uint8_t *>(row) + int64_t(y) * (BF16 ? 2 : 4);
      if constexpr (sizeof(w) == 16) {
        const uint4 v = __ldcg(reinterpret_cast<const uint4 *>(at));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      } else {
        const uint2 v = __ldcg(reinterpret_cast<const uint2 *>(at));
        w[0] = v.x, w[1] = v.y;
      }
    } else {
#pragma unroll
      for (uint32_t &v : w) v = 0;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (y + i < end) {
          if constexpr (BF16)
            w[i / 2] |= uint32_t(__ldcg(static_cast<const uint16_t *>(row) + y + i)) << (16 * (i & 1));
          else
            w[i] = __ldcg(static_cast<const uint32_t *>(row) + y + i);
        }
    }
  }
  __device__ __forceinline__ float2 two(int k) const {  // elements 2 k, 2 k + 1
    const float a = __uint_as_float(BF16 ? w[k] << 16 : w[2 * k]);
    const float b = __uint_as_float(BF16 ? w[k] & 0xffff0000u : w[2 * k + 1]);
    return make_float2(clean(a), clean(b));
  }
};

// Two pairs, by instructions of two fp32 operations.
struct Pair2 {
  float2 hi, lo;
  __device__ __forceinline__ Pair first() const { return pair(hi.x, lo.x); }
  __device__ __forceinline__ Pair second() const { return pair(hi.y, lo.y); }
};
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.0f, -1.0f), a); }
// hi + lo = a + b, exactly
__device__ __forceinline__ Pair2 two_sum(float2 a, float2 b) {
  const float2 s = add2(a, b), bb = sub2(s, a);
  return Pair2{s, add2(sub2(a, sub2(s, bb)), sub2(b, bb))};
}
// Where a node's sums are: to be made or made of what is left, or of the whole rows.
enum class Sums { kNone, kLeft, kDraft, kTarget };
// What is left of the target's probabilities: all of them, max(p - q, 0) or max(p - t q, 0).
enum class Rest { kAll, kOne, kAny };
template <Rest R>
__device__ __forceinline__ Pair2 rest(float2 p, float2 q, Pair t) {
  if (R == Rest::kAll) return Pair2{p, make_float2(0.0f, 0.0f)};
  if (R == Rest::kOne) {
    // p - min(p, q): the rounding error of a difference from what is not larger takes two
    // operations, and nothing has to be compared
    const float2 m = make_float2(fminf(q.x, p.x), fminf(q.y, p.y)), s = sub2(p, m);
    return Pair2{s, sub2(sub2(p, s), m)};
  }
  const float2 minus = make_float2(-t.h, -t.h), h = mul2(minus, q);  // -th q = h + e
  const float2 e = fma2(make_float2(-t.l, -t.l), q, fma2(minus, q, make_float2(-h.x, -h.y)));
  Pair2 d = two_sum(p, h);
  d.lo = add2(d.lo, e);
  const float2 s = add2(d.hi, d.lo);
  if (!(s.x > 0.0f)) d.hi.x = d.lo.x = 0.0f;
  if (!(s.y > 0.0f)) d.hi.y = d.lo.y = 0.0f;
  return d;
}

// Where the walk stands.
struct Stand {
  int cur;        // the node
  int last;       // its latest child tried, or itself
  Pair t, C;
};

// The rows of the node where it stands, and what is taken off them.
struct Rows {
  const void *p, *q;
  Pair t;
  Rest kind;
};

// Whether some child of `cur` up to node `end` - 1 has token y.  All lanes ask alike.
__device__ __forceinline__ bool among_children(const Shared &sm, int cur, int end, int32_t y, int lane) {
  for (int b = cur + 1; b < end; b += 32) {
    const int i = b + lane;
    if (__any_sync(0xffffffffu, i < end && sm.parent[i] == cur && sm.token[i] == y)) return true;
  }
  return false;
}

// A chunk's sum, by a warp.  `nodes`: the draft's, where tokens tried are left out, else 0.
// AtOnce: 16-byte words of a row that a lane has on their way.
template <bool BF16, int AtOnce, Rest R>
__device__ __forceinline__ Pair chunk_sum(const Shared &sm, const Rows &r, int chunk, int vocab, int cur, int nodes,
                                            int lane) {
  constexpr int N = BF16 ? 8 : 4, kSteps = kChunk / (32 * N), kAtOnce = AtOnce < kSteps ? AtOnce : kSteps;
  Pair2 acc{make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
  for (int s0 = 0; s0 < kSteps; s0 += kAtOnce) {
    Probs<BF16, N> p[kAtOnce], q[kAtOnce];
    const int y0 = chunk * kChunk + 32 * N * s0 + N * lane;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      p[k].load(r.p, y0 + 32 * N * k, vocab);
      if (R != Rest::kAll) q[k].load(r.q, y0 + 32 * N * k, vocab);
    }
    for (int b = cur + 1; R == Rest::kAll && b < nodes; b += 32) {
      const int i = b + lane;
      const int32_t at = i < nodes && sm.parent[i] == cur && sm.token[i] >= 0
                             ? sm.token[i] - (chunk * kChunk + 32 * N * s0) : -1;
      for (uint32_t m = __ballot_sync(0xffffffffu, at >= 0 && at < 32 * N * kAtOnce); m != 0; m &= m - 1) {
        const int x = __shfl_sync(0xffffffffu, at, __ffs(int(m)) - 1);  // of step x / (32 N), lane (x / N) % 32
        // (in every word without a branch: one word by its number would put them all in local memory)
        const int word = (x / N) % 32 == lane ? 4 * (x / (32 * N)) + (BF16 ? x % N / 2 : x % N) : -1;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
          for (int w = 0; w < 4; ++w)
            p[k].w[w] &= word == 4 * k + w ? (BF16 ? (x & 1 ? 0x0000ffffu : 0xffff0000u) : 0u) : 0xffffffffu;
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const Pair2 w = rest<R>(p[k].two(i), R != Rest::kAll ? q[k].two(i) : make_float2(0.0f, 0.0f), r.t);
        const Pair2 s = two_sum(acc.hi, w.hi);
        acc.hi = s.hi;
        acc.lo = add2(acc.lo, R != Rest::kAll ? add2(s.lo, w.lo) : s.lo);
      }
  }
  return warp_sum(acc.first() + acc.second());
}

template <bool BF16, int AtOnce>
__global__ void __launch_bounds__(kThreads, AtOnce > 4 ? 2 : 4) verify_kernel(Verify v, WsHeader *__restrict__ hdr) {
  __shared__ Shared sm;
  // (waited for below: no block writes to one that has not made its barriers)
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&sm.given[0]), 1);
    mbar_init(smem_u32(&sm.given[1]), 1);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank(), blocks = cluster_size();
  const int s = int(blockIdx.x / blocks);
  const int64_t from = max(0, __ldcg(v.cu + s)), to = min(v.n_tokens, int64_t(__ldcg(v.cu + s + 1)));
  const int64_t all = max(int64_t(0), to - from);
  const bool many = all > kMaxNodes;
  const int nodes = many ? 0 : int(all);
  const int size = BF16 ? 2 : 4;
  const auto row_of = [&](const void *m, int64_t stride, int node) {
    return static_cast<const void *>(static_cast<const uint8_t *>(m) + (from + node) * stride * size);
  };
  const auto one = [&](const void *row, int y) {
    Probs<BF16, 2> p;
    if constexpr (BF16)
      p.w[0] = __ldcg(static_cast<const uint16_t *>(row) + y);
    else
      p.w[0] = __ldcg(static_cast<const uint32_t *>(row) + y);
    return clean(__uint_as_float(BF16 ? p.w[0] << 16 : p.w[0]));
  };
  // (bytes that no block gives: the time-out's test)
  const uint32_t extra = tid == 0 && __ldcg(&hdr->wait_extra) != 0 ? 8u : 0u;
  bool odd = many;
  for (int i = tid; i < nodes; i += kThreads) {
    const int32_t up = __ldcg(v.parent + from + i);
    int32_t x = __ldcg(v.tokens + from + i);
    sm.u[i] = __ldcg(v.u + from + i);
    const bool bad = up < -1 || up >= i;
    const int at = bad ? -1 : up;
    if (x < 0 || x >= v.vocab) x = -1;
    odd = odd || bad || (x < 0 && i > 0);
    sm.parent[i] = int16_t(at);
    sm.token[i] = x;
    if (at >= 0 && x >= 0) {
      sm.p[i] = one(row_of(v.target, v.target_stride, at), x);
      if (v.draft != nullptr) sm.q[i] = one(row_of(v.draft, v.draft_stride, at), x);
    } else {
      sm.p[i] = sm.q[i] = 0.0f;
    }
  }
  if (odd && rank == 0) atomicExch(&hdr->status, int32_t(DS4X_EDEVICE));
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (nodes == 0) {  // (all blocks of the cluster leave here)
    for (int64_t i = rank * kThreads + tid; i < all; i += blocks * kThreads) v.path[from + i] = v.out[from + i] = -1;
    if (rank == 0 && tid == 0) v.n_path[s] = 0;
    return;
  }

  // the block's chunks
  const int chunks = (v.vocab + kChunk - 1) / kChunk, per = (chunks + int(blocks) - 1) / int(blocks);
  const int c0 = min(chunks, int(rank) * per), c1 = min(chunks, c0 + per);
  int passes = 0;
  bool aborted = false;
  // sums of what is left at the node, by chunk, by block and in all
  Rows rows{nullptr, nullptr, Pair{0.0f, 0.0f}, Rest::kAll};
  const auto pass = [&](const Stand &at, Sums of) {
    rows.p = of == Sums::kDraft ? row_of(v.draft, v.draft_stride, at.cur) : row_of(v.target, v.target_stride, at.cur);
    rows.kind = v.draft == nullptr || !some(at.t) ? Rest::kAll : at.t.h == 1.0f && at.t.l == 0.0f ? Rest::kOne : Rest::kAny;
    if (rows.kind != Rest::kAll) rows.q = row_of(v.draft, v.draft_stride, at.cur);
    rows.t = at.t;
    // (a barrier is used again two passes on, when every warp here is past its first use: the one between)
    unsigned long long *given = &sm.given[passes & 1];
    Pair *total = sm.total[passes & 1];
    if (tid == 0) mbar_arrive_expect_tx(smem_u32(given), 8 * blocks + extra);
    Pair mine{0.0f, 0.0f};
    for (int c = c0 + warp; c < c1; c += kWarps) {
      const int tried = v.draft == nullptr ? at.last + 1 : 0;
      const Pair sum = rows.kind == Rest::kAll   ? chunk_sum<BF16, AtOnce, Rest::kAll>(sm, rows, c, v.vocab, at.cur, tried, lane)
                       : rows.kind == Rest::kOne ? chunk_sum<BF16, AtOnce, Rest::kOne>(sm, rows, c, v.vocab, at.cur, 0, lane)
                                                 : chunk_sum<BF16, AtOnce, Rest::kAny>(sm, rows, c, v.vocab, at.cur, 0, lane);
      if (lane == 0) sm.sums[c - c0] = sum;
      mine = mine + sum;
    }
    if (lane == 0) sm.red[warp] = mine;
    __syncthreads();
    if (warp == 0) {
      const Pair sum = warp_sum<kWarps>(sm.red[lane % kWarps]);
      if (lane < int(blocks)) give(&total[rank], given, uint32_t(lane), sum);
    }
    const bool came = wait_bar(sm, given, (passes >> 1) & 1, hdr);
    __syncwarp();
    aborted = __syncthreads_or(!came) != 0;
    ++passes;
    return warp_sum<kMaxCluster>(lane % kMaxCluster < int(blocks) ? total[lane % kMaxCluster] : Pair{0.0f, 0.0f});
  };

  // ---- the walk, the same in every warp -------------------------------------------------
  Stand at{0, 0, Pair{0.0f, 0.0f}, Pair{1.0f, 0.0f}};
  int count = 1;
  Sums sums = Sums::kNone;
  Pair left{0.0f, 0.0f};
  if (tid == 0) sm.path[0] = 0;
  for (;;) {
    bool ends = sums > Sums::kLeft;
    while (!ends) {
      int j = -1;  // the next child
      for (int b = at.last + 1; b < nodes && j < 0; b += 32) {
        const int i = b + lane;
        const uint32_t m = __ballot_sync(0xffffffffu, i < nodes && sm.parent[i] == at.cur);
        if (m != 0) j = b + __ffs(int(m)) - 1;
      }
      ends = j < 0;
      if (ends) break;
      const int32_t x = sm.token[j];
      Pair w{sm.p[j], 0.0f}, bar = sm.u[j] * at.C;
      if (v.draft != nullptr) {
        const float q = sm.q[j];
        // (not max(.., 0): what it is compared with is not below 0)
        if (some(at.t)) w = w + -(q * at.t);
        bar = q * bar;
      } else if (at.last > at.cur && among_children(sm, at.cur, j, x, lane)) {
        w.h = 0.0f;
      }
      if (w > bar) {
        if (tid == 0) sm.path[count] = int16_t(j);
        ++count;
        at = Stand{j, j, Pair{0.0f, 0.0f}, Pair{1.0f, 0.0f}};
        sums = Sums::kNone;
        continue;
      }
      at.last = j;
      if (v.draft != nullptr) {
        at.t = at.t + at.C;
        break;
      }
      at.C = at.C + -w;
    }
    if (!ends || sums != Sums::kLeft) left = pass(at, sums);
    if (aborted) break;
    if (!ends) {
      at.C = left;
      sums = Sums::kLeft;
      continue;
    }
    // nothing left after a rejection: the draft's row, then the target's
    if (sums == Sums::kTarget || (sums != Sums::kDraft && (some(left) || at.last == at.cur))) break;
    const bool draft = sums != Sums::kDraft && v.draft != nullptr;
    if (tid == 0) sm.drafted = sums == Sums::kDraft ? left : Pair{0.0f, 0.0f};  // (read behind the next pass's barriers)
    sums = draft ? Sums::kDraft : Sums::kTarget;
    at = Stand{at.cur, at.cur, Pair{0.0f, 0.0f}, Pair{1.0f, 0.0f}};
  }

  // (no block ends while another may still store into it)
  __syncwarp();
  if (blocks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const auto leave = [&]() {
    __syncwarp();
    if (blocks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  };
  if (aborted) {
    leave();
    // Not all stores have come; none is begun any more.  One takes about a microsecond.
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < kDrainNs) __nanosleep(1000);
    return;
  }

  // ---- the last token ---------------------------------------------------------------------
  const Pair want = sm.u[0] * left;
  // the block in whose slice it lies, then its chunk
  Pair base{0.0f, 0.0f};
  // (the draft's sum twice the target's or more: no distribution beside it)
  const bool none = sums == Sums::kTarget && !(left + left > sm.drafted);
  const int holder = none ? -1 : first_past(sm.total[(passes - 1) & 1], int(blocks), want, base, lane);
  if (rank == 0) {
    __syncthreads();  // `path`
    for (int i = tid; i < nodes; i += kThreads) {
      v.path[from + i] = i < count ? sm.path[i] : -1;
      if (i != count - 1) v.out[from + i] = i < count ? sm.token[sm.path[i + 1]] : -1;
    }
    if (tid == 0) {
      v.n_path[s] = count;
      if (holder < 0) {
        v.out[from + count - 1] = -1;
        atomicExch(&hdr->status, int32_t(DS4X_EDEVICE));
      }
    }
  }
  if (holder != int(rank)) {
    leave();
    return;
  }
  if (warp == 0) {
    const int pick = first_past(sm.sums, c1 - c0, want, base, lane);
    if (lane == 0) {
      sm.chunk = c0 + max(pick, 0);  // (there is one, save where probabilities were infinite)
      sm.base = base;
      sm.found = INT32_MAX;
    }
  }
  __syncthreads();
  // its tokens, four a lane
  const int y0 = sm.chunk * kChunk + 4 * tid;
  Probs<BF16, 4> p, q;
  p.load(rows.p, y0, v.vocab);
  if (rows.kind != Rest::kAll) q.load(rows.q, y0, v.vocab);
  Pair w[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    Pair2 d{p.two(i), make_float2(0.0f, 0.0f)};
    if (rows.kind == Rest::kOne) d = rest<Rest::kOne>(d.hi, q.two(i), rows.t);
    if (rows.kind == Rest::kAny) d = rest<Rest::kAny>(d.hi, q.two(i), rows.t);
    w[2 * i] = d.first();
    w[2 * i + 1] = d.second();
  }
  if (v.draft == nullptr)
    for (int i = at.cur + 1; i <= at.last; ++i) {
      const int k = sm.parent[i] == at.cur ? sm.token[i] - y0 : -1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j].h = k == j ? 0.0f : w[j].h;
        w[j].l = k == j ? 0.0f : w[j].l;
      }
    }
  const Pair upto = warp_scan((w[0] + w[1]) + (w[2] + w[3]), lane);
  if (lane == 31) sm.red[warp] = upto;
  const Pair prev = shfl_up(upto, 1);
  __syncthreads();
  Pair sum = sm.base;
  for (int k = 0; k < warp; ++k) sum = sum + sm.red[k];
  if (lane > 0) sum = sum + prev;
  int first = INT32_MAX, latest = -1;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    sum = sum + w[k];
    if (some(w[k])) {
      latest = y0 + k;
      if (sum > want) first = min(first, y0 + k);
    }
  }
  first = __reduce_min_sync(0xffffffffu, first);
  if (lane == 0 && first != INT32_MAX) atomicMin(&sm.found, first);
  __syncthreads();
  if (sm.found == INT32_MAX) {  // (by rounding)
    __syncthreads();
    if (tid == 0) sm.chunk = -1;
    __syncthreads();
    atomicMax(&sm.chunk, latest);
    __syncthreads();
    if (tid == 0) sm.found = sm.chunk;
  }
  if (tid == 0) v.out[from + count - 1] = sm.found;
  leave();
}

}  // namespace

cudaError_t launch_verify(const Verify &v, bool bf16, void *ws, cudaStream_t stream) {
  static std::atomic<uint64_t> set[3];
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // As many blocks a sequence as are resident at once and find a chunk for each warp (61
  // sequences of 50,257 tokens: 20.1 us with 8 blocks each, some 8 % more with 4).
  const int chunks = (v.vocab + kChunk - 1) / kChunk;
  int blocks = 1;
  while (blocks < kMaxCluster && 2 * int64_t(blocks) * v.n_seqs <= 4 * int64_t(sms) && blocks * kWarps < chunks) blocks *= 2;
  // Where each block may have half an SM a lane has all of its chunk on its way (one sequence
  // of 131,072 tokens: 7.3 us, some 0.6 more with half of it), else half, and twice the blocks an
  // SM (256 sequences: 49.2 us, some 13 % more with all of it).
  const bool wide = !bf16 && int64_t(blocks) * v.n_seqs <= 2 * int64_t(sms);
  auto *kernel = bf16 ? verify_kernel<true, 4> : wide ? verify_kernel<false, 8> : verify_kernel<false, 4>;
  std::atomic<uint64_t> &known = set[bf16 ? 0 : wide ? 1 : 2];
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(known.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    known.fetch_or(bit, std::memory_order_acq_rel);
  }
  return launch_pdl_clusters(kernel, unsigned(blocks), unsigned(v.n_seqs) * unsigned(blocks), unsigned(kThreads), size_t(0),
                             stream, v, static_cast<WsHeader *>(ws));
}

}  // namespace ds4x
