// Attention over the paged 4-bit cache on the tensor cores.
//
//   l_hj = scale * (q_h . v_j),  o_h = sum_j softmax_j(l_h)_j v_j,
//   lse_h = log sum_j e^(l_hj)
//
// over a token's rows: the range [row_begin, row_end) of its sequence, or its
// own list of rows.  A unit is a token and up to 64 of its heads, or, where heads
// are few, several neighbouring tokens of one sequence with all their heads
// (paged_plan_kernel): up to 64 query vectors, its columns.  Its rows come in tiles
// of 64.  Two tcgen05.mma (kind::f16, fp16 operands, fp32 sums in tensor memory) a
// tile:
//
//   S^T[64 rows][columns] = V'[64 rows][512] . Q'[columns][512]^T
//   O^T[512 dims][columns] += V'^T[512][64 rows] . P^T[64 rows][columns]
//
// V' is the tile's rows widened once to fp16, in shared memory, as eight
// 128-byte-swizzled panels of 64 dims (16-byte chunk c of row r at c ^ (r % 8); which
// dims, see v_chunk): the first product reads them K-major, the second the same
// bytes MN-major.
//
// Exact operands.  Row j's exponent E_j is its RoPE part's, the row's largest:
// V'_j = v_j 2^-E_j, at most 8, is exact in fp16 while a block's scale lies
// within 2^14 of 2^E_j (smaller blocks round at 2^-25 of 2^E_j); the RoPE part's
// fp16 values are V' as they are.  Q' = q 2^c in fp16, c taking the vector's
// largest |q| into [2^14, 2^15): a bf16 value is exact down to 2^-32 of it.  (One c
// a unit was 1.5 % faster and let a large head round away a small one beside it.)
//
// Softmax in the log2 domain, online, with the row's exponent kept apart:
// x_j = l_j log2 e + E_j, w_j = 2^(x_j - m) is what multiplies V'_j, and the
// denominator is sum_j w_j 2^-(E_j + 7).  m is 7 below a column's running maximum of x,
// lazily: it moves (and O^T and the sums are rescaled) only when a tile's x exceeds it
// by more than 15, so the largest w lies between 2^7 and 2^15.  w enters the second
// product as fp16: half a step is 2^-12 to 2^-11 of it, an eighth of the bf16 output's
// own step (hi + lo parts would double that product), while it is above 2^-21 of the
// largest, and at most 2^-32 of the largest below that.  (With the largest at 1 a sink
// row took a flat history's part of the output with it.)
//
// Sums are fp32, over runs of at most 512 tiles of a unit: both the denominator's and
// the tensor core's drop a term that is 2^-24 of the sum so far.  Over 2^20 rows at once
// that was 2.5 % of the output and 2^-9 of the denominator; over 2^15 it is below 2^-10
// and 2^-14.  A longer share of a unit is joined run by run in the CTA's own part of the
// workspace, by its log-sum-exp (152 units of 2^20 rows: 25.2 ms, 24.7 by 1024 tiles at
// twice the error, 24.2 in one sum).  E_j is within +-96, so a run's denominator stays
// inside fp32 (the 2^7 is left out of it).
//
// Work split.  All units' tiles, in order, are cut into one run a CTA (one CTA
// an SM), so any mix of lengths fills the GPU; a cut that falls near a unit's
// end moves there.  A unit that one CTA covers goes straight to the output; the
// parts of the others go to the workspace in fp32, normalised, with their
// log-sum-exp, and a second kernel joins them in a fixed order.  The cuts
// depend on the lengths alone, so results do not depend on timing.
//
// Roles (20 warps).  L (warp 0): finds the rows of the tiles to come (list entry,
// page table), four tiles ahead, and asks for them into L2.  W (4-11): widens the
// tiles into two V' buffers in turn, two rows a lane, with the 16-byte words of the
// next two tiles on their way into registers meanwhile.
// X (12-19): the softmax, four 16-row quarters of S^T by two halves of the columns;
// when a unit ends, the next one's Q' first, then the output.  M (1-3): issue the
// products, a thread each for S of the even tiles, S of the odd ones and O: a
// thread that has committed MMAs is held at its next barrier until they are done,
// so one thread for all of them left the tensor core idle between tiles.
// Registers go from L, M and W to X (setmaxnreg): the softmax must not spill,
// because local loads queue behind W's.
//
// What bounds it.  Long histories and chunks: the chain of a tile, widen -> S ->
// softmax -> O, about 3400 cycles a tile with the two V' buffers that shared memory
// holds (64 KB each beside 64 KB of Q'), of which the products fill 56 % (M = 64
// rows make S run at half the tensor rate): 64 heads over 1,048,576 rows 191 us
// (2.0 TB/s of packed rows, 0.72 PFLOP/s), a chunk of 2048 tokens over 8192 rows
// 2.51 ms (0.77 PFLOP/s).  Two tiles' loads in flight and a third product queue
// took it there from 307 us.  Short histories: latency, 10 us for the kernel (its
// launch, the cuts, one round trip to the rows, three tiles' chain) and 1.4 to 3.5
// us for the join: 777 rows 13.4 us, 8192 rows 18.9 us.
//
// Every wait is bounded (0.5 s): a time-out sets DS4X_ETIMEOUT, after which no
// wait blocks, so every role runs to its end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace ds4x {
namespace {

using namespace ptx;

constexpr int kDim = DS4X_KV_DIM;  // 512
constexpr int kTile = 64;          // rows a tile
constexpr int kHeads = 64;         // heads a unit, at most
constexpr int kMWarp0 = 1;                           // S of even tiles, S of odd tiles, O
constexpr int kWWarp0 = 4, kWWarps = 8, kXWarp0 = 12, kXWarps = 8;
constexpr int kXThreads = 32 * kXWarps;
constexpr int kThreads = 32 * (kXWarp0 + kXWarps);  // 640
// registers a thread: at launch, then by role
constexpr int kRegs = 96, kRegsLM = 64, kRegsW = 96, kRegsX = 104;
static_assert(4 * kRegsLM + kWWarps * kRegsW + kXWarps * kRegsX <= kThreads / 32 * kRegs, "register split");
constexpr int kAhead = 4;                            // L's ring of found tiles
constexpr int kMaxCtas = 160;
constexpr int kPackTokens = 8;     // tokens a unit, at most
constexpr int kFewUnits = 16;      // up to so many units are joined by a block a head's half each
constexpr uint32_t kOCol = 0;      // O^T: dims 128 i .. as columns 64 i .. 64 i + 63
constexpr uint32_t kSCol = 256;    // S^T: two buffers of 64 columns
constexpr unsigned long long kTimeoutNs = 500ull * 1000 * 1000;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTop = 7;                       // log2 of the largest weight, when a maximum has moved
constexpr float kLazy = 8.0f + kTop;          // ... and at most
constexpr int kTame = 20;
constexpr int kRunTiles = 512;     // tiles that one sum goes over, at most
enum { kBarX = 1, kBarEnd = 2 };  // named barriers

// Where a row lies: its codes (null: no row), and from there to its RoPE part and
// its scale record.
struct __align__(16) Found {
  const uint8_t *codes;
  int32_t tail, scales;
};

struct __align__(1024) Smem {
  uint8_t q[kHeads * kDim * 2];     // Q': 8 panels of 64 dims, 8 KB each
  uint8_t v[2][kTile * kDim * 2];   // V': 8 panels of 8 KB, two tiles
  uint8_t p[2][kTile * kHeads * 2]; // P^T: one panel, two tiles
  float4 rowe[2][kTile];            // 2^E_j, E_j, 2^-(E_j + 7), E_j + 7; a row that is not there: 0, -inf, 0, 0
  Found found[kAhead][kTile];
  float red[4][kHeads];
  float alpha[kHeads];
  float mh[kHeads], hinv[kHeads];
  float qscale[kHeads];             // the unit's columns' scale log2 e 2^-c
  float qodd[kHeads];               // NaN for a column with NaN or infinity, else 0
  float run2[kHeads], keep[kHeads]; // a share of several runs: log2 of the denominator so far; its part of the joined output
  unsigned long long vfull[2], sfull[2], pfull[2], pvdone[2][2], lfull[kAhead], lfree[kAhead], qfull, qtaken, drain;
  long long scan[kThreads / 32];
  long long cut0, cut1, all;        // the CTA's run of tiles, and all tiles
  int unit0, off0;                  // where it begins: tile off0 of unit unit0
  int row0, rows;                   // that unit's rows
  int total;                        // its tiles
  uint32_t tmem_base;
  int abort_flag;
  unsigned long long wide[2];       // bit r: the tile's row r has an exponent beyond +-kTame
  int2 seen[kPackTokens];           // packed: the rows that each token sees, from the unit's first
  long long out_at[kHeads];         // packed: a column's output (-1: no column)
  int end_unit, end_part;           // the CTA's last unit (-1: W has no part in its output), and its part (-1: the whole unit)
};
static_assert(sizeof(Smem) <= 232448, "shared-memory budget");

// The workspace behind its header.  Part 2 c: CTA c's share of a unit that an
// earlier CTA began; part 2 c + 1: of one that it begins and a later one ends.
struct Parts {
  int32_t unit[2 * kMaxCtas];            // the part's unit, or -1
  int2 span[kFewUnits];                  // with few units: a unit's first CTA, and how many have a part of it
  float lse2[2 * kMaxCtas][kHeads];      // log2 of the denominator
  float o[2 * kMaxCtas][kHeads][kDim];   // normalised, dims as V' has them (v_chunk)
};

// With several tokens a unit: its tokens t0 .. t0 + count - 1, of one sequence, and
// the rows that any of them sees.
struct __align__(16) Pack {
  int32_t t0, count, r0, n;
};
struct Plan {
  int32_t n_units, pad[3];
  Pack unit[DS4X_PAGED_MAX_TOKENS];
};

struct Args {
  PagedAttn a;
  const Plan *plan;   // several tokens a unit (n_heads columns each), or null
  int32_t groups;     // head groups a token
  int32_t group;      // a unit's columns at most: heads a group (the last may have fewer), or tokens x heads
  int32_t per_head;   // 2^16 / n_heads, rounded up
  int32_t n_cols;     // `group` rounded up to 16: the products' N
  uint64_t per_grid;  // 2^64 / CTAs, rounded up
  int32_t few;        // at most kFewUnits units
  __device__ __forceinline__ bool packed() const { return plan != nullptr; }
};
// The same where the kernel is compiled for either: unpacked units cost nothing for the others.
template <bool P>
struct ArgsFor : Args {
  ArgsFor(const Args &g) : Args(g) {}
  static __device__ __forceinline__ constexpr bool packed() { return P; }
};

__device__ __forceinline__ unsigned long long globaltimer() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __noinline__ void wait_failed(Smem &sm, WsHeader *hdr) {
  atomicExch(&hdr->status, int32_t(DS4X_ETIMEOUT));
  *reinterpret_cast<volatile int *>(&sm.abort_flag) = 1;
}
__device__ __forceinline__ void wait_bar(Smem &sm, unsigned long long *bar, uint32_t parity, WsHeader *hdr) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try_wait(b, parity)) return;
  const unsigned long long t0 = globaltimer();
  for (;;) {
#pragma unroll 1
    for (int k = 0; k < 64; ++k)  // (a try may itself wait a while; the clock is looked at now and then)
      if (mbar_try_wait_sleep(b, parity, 2000)) return;
    if (*reinterpret_cast<volatile int *>(&sm.abort_flag)) return;
    if (globaltimer() - t0 > kTimeoutNs) {
      wait_failed(sm, hdr);
      return;
    }
  }
}

// Shared-memory descriptor, 128-byte swizzle.  K-major: sbo = distance of
// 8-row groups.  MN-major: lbo = distance of 64-wide panels along M (N), sbo =
// distance of 8-row groups along K.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t((lbo >> 4) & 0x3FFFu) << 16) |
         (uint64_t((sbo >> 4) & 0x3FFFu) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// Registers a thread of this warpgroup from here on (all four warps).
template <int N>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// One lane of a converged warp, chosen so that the compiler knows the branch to
// be one thread's: its MMA descriptors then stay in uniform registers (an issuer
// picked by lane number took 78 cycles an MMA beside busy warps, this one 32).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// 16 lanes x 32 columns: register 4 j + 2 r + c of lane T holds lane T / 4 + 8 r,
// column 8 j + 2 (T % 4) + c.
__device__ __forceinline__ void tc_ld_16x256_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // e in [-126, 127]
// 2^d twice, as fp16, for d <= 0 (0 below the smallest subnormal 2^-24: the
// conversion's rounding does it).
__device__ __forceinline__ uint32_t pow2_half2(int d) {
  const float f = pow2f(max(d, -32));
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(r) : "f"(f));
  return r;
}
__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d));
}

// A unit's query vectors ("columns"): heads h0 .. of token t0, or, packed, all heads
// of count tokens from t0, head by head.
struct Columns {
  int32_t t0, h0, n;
  template <class A>
  __device__ __forceinline__ Columns(const A &g, int unit) {
    if (g.packed()) {
      const int2 p = __ldcg(reinterpret_cast<const int2 *>(&g.plan->unit[unit]));
      t0 = p.x;
      h0 = 0;
      n = p.y * g.a.n_heads;
    } else {
      t0 = unit / g.groups;
      h0 = (unit % g.groups) * g.group;
      n = min(g.group, g.a.n_heads - h0);
    }
  }
  // column c's token and head (c < 64 and n_heads <= 64: the product is the quotient)
  template <class A>
  __device__ __forceinline__ int64_t at(const A &g, int c, int64_t token_stride, int head_stride) const {
    const int j = g.packed() ? (c * g.per_head) >> 16 : 0;
    return int64_t(t0 + j) * token_stride + (h0 + c - j * g.a.n_heads) * head_stride;
  }
};

// A token's rows: n of them, from row r0 of its sequence (or of its list).
struct Rows {
  int64_t r0;
  int32_t n;
};
__device__ __forceinline__ Rows token_rows(const PagedAttn &a, int t) {
  if (a.idx != nullptr) return Rows{0, a.k};
  // no further than the table goes (a range past it is flagged by find_cuts)
  const int64_t room = int64_t(a.c.seq_pages) << a.c.page_log2;
  const int64_t b = a.row_begin != nullptr ? max(int64_t(0), int64_t(__ldcg(a.row_begin + t))) : 0;
  const int64_t e = min(room, int64_t(__ldcg(a.row_end + t)));
  return b < e ? Rows{b, int32_t(e - b)} : Rows{0, 0};
}
// Whether token t sees a row past what the table can place.
__device__ __forceinline__ bool past_table(const PagedAttn &a, int t) {
  const int64_t e = __ldcg(a.row_end + t);
  return e > (int64_t(a.c.seq_pages) << a.c.page_log2) && (a.row_begin == nullptr || __ldcg(a.row_begin + t) < e);
}
template <class A>
__device__ __forceinline__ Rows unit_rows(const A &g, int unit) {
  if (!g.packed()) return token_rows(g.a, unit / g.groups);
  const int2 p = __ldcg(reinterpret_cast<const int2 *>(&g.plan->unit[unit]) + 1);
  return Rows{p.x, p.y};
}
// A token without a row still has a tile (of rows that are not there): it writes the zeros.
__device__ __forceinline__ int rows_tiles(int n) { return n > 0 ? (n - 1) / kTile + 1 : 1; }

// Walks the CTA's tiles (numbered from 0 locally), a run of a unit's share at a time.
struct Walk {
  int unit, from;  // the share's unit, and its first tile within it
  int off;         // the run's first tile within the unit
  int i0, i1;      // the run's tiles, locally
  int tiles;       // the unit's tiles
  int r0, n;       // the token's rows
  __device__ __forceinline__ void end_run(int total) {
    i1 = int(min(int64_t(total), int64_t(i0) + min(tiles - off, kRunTiles)));
  }
  __device__ __forceinline__ void set(int row0, int rows, int total) {
    r0 = row0;
    n = rows;
    tiles = rows_tiles(n);
    end_run(total);
  }
  __device__ __forceinline__ void begin(const Smem &sm, int total) {
    unit = sm.unit0;
    from = off = sm.off0;
    i0 = 0;
    set(sm.row0, sm.rows, total);
  }
  // another run of this unit follows
  __device__ __forceinline__ bool more(int total) const { return i1 < total && off + (i1 - i0) < tiles; }
  template <class A>
  __device__ __forceinline__ void next(const A &g, int total) {
    if (more(total)) {
      off += i1 - i0;
      i0 = i1;
      end_run(total);
      return;
    }
    ++unit;
    from = off = 0;
    i0 = i1;
    const Rows r = unit_rows(g, unit);
    set(int(r.r0), r.n, total);
  }
};

// ---- the cuts ------------------------------------------------------------------

// Fewer than 16 tiles a CTA: cuts at whole multiples of this many, else (0) fractional.
// The longest run is as long and there are fewer parts to join (24000 rows: 23.6 us a
// call, was 25.3).  Above kOnes tiles, two in one CTA are quicker than one each in two,
// because every part is 128 KB written and read (6200 rows, 97 tiles: 16.2 us by ones,
// 16.4 by twos; 8192 rows, 128 tiles: 20.5, 18.0; 16384 rows 23.1, 21.8).
constexpr int kOnes = 100;
template <class A>
__device__ __forceinline__ int cut_step(const A &g, long long total) {
  const int n = int(gridDim.x);
  if (total >= 16 * n) return 0;
  const int even = int(__umul64hi((unsigned long long)total + (n - 1), g.per_grid));  // (one CTA: 0)
  return max(total > kOnes ? 2 : 1, even);
}
// Cut c of `total` tiles: at c total / CTAs, or, with few, at c steps.  (total < 2^43
// and c <= 160: the high word of the product with the rounded-up reciprocal is the
// quotient.)
template <class A>
__device__ __forceinline__ long long cut_at(const A &g, unsigned c, long long total) {
  if (c >= gridDim.x) return total;
  if (const int step = cut_step(g, total)) return min((long long)(c * step), total);
  return (long long)(__umul64hi(c * (unsigned long long)total, g.per_grid));
}
// A cut at most so far from a unit's end moves there: a sixteenth of a run, or up to
// kSnap tiles where that is at most a quarter of it (a part costs its CTA a start and
// an end and is written and read again: 88 lists of 456 rows for 100 heads 45.7 us, 53.2
// without; 762 of 195 rows 78.4, 84.0; 770 tokens over up to 771 rows 123.9, 129.4).
constexpr int kSnap = 4;
template <class A>
__device__ __forceinline__ long long cut_tolerance(const A &g, long long total) {
  const long long run = (long long)(__umul64hi((unsigned long long)total, g.per_grid));
  return max(run >> 4, min((long long)kSnap, run >> 2));
}
// How many CTAs from this one on have a part of a unit that ends with tile end - 1,
// that this one begins and does not end: the cuts inside it that do not move to its
// end, and one.  (c total / CTAs < e for the c below e CTAs / total.)
template <class A>
__device__ __forceinline__ int unit_parts(const A &g, long long end, long long total) {
  const long long e = end - cut_tolerance(g, total), n = gridDim.x;
  if (const int step = cut_step(g, total)) return 1 + (int(e) - 1) / step - int(blockIdx.x);
  const long long last = (long long)(((unsigned long long)(e) * n + total - 1) / (unsigned long long)total) - 1;
  return 1 + int(min(last, n - 1) - (long long)(blockIdx.x));
}

// The run of CTA c of g: unit0, off0, total; the first unit's rows.  All threads.
template <class A>
__device__ void find_cuts(const A &g, Smem &sm, Parts *parts, WsHeader *hdr) {
  const PagedAttn &a = g.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kThreads / 32;
  // a thread takes `per` tokens in a row (or packed units; of all that there may be:
  // the count of valid ones is on its way with their rows)
  const int per = (a.n_tokens + kThreads - 1) / kThreads;
  const int t0 = min(a.n_tokens, tid * per), t1 = min(a.n_tokens, t0 + per);
  auto rows_of = [&](int t) { return g.packed() ? unit_rows(g, t) : token_rows(a, t); };
  const Rows first_rows = t0 < t1 ? rows_of(t0) : Rows{0, 0};
  // tokens behind are padding
  const int valid = g.packed() ? __ldcg(&g.plan->n_units) : __ldcg(a.c.cu + a.c.n_seqs);
  auto tiles_of = [&](int t) { return t < valid ? rows_tiles(rows_of(t).n) : 0; };
  const int first = t0 < min(t1, valid) ? rows_tiles(first_rows.n) : 0;
  long long mine = first;
  for (int t = t0 + 1; t < t1; ++t) mine += tiles_of(t);
  mine *= g.groups;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sm.scan[warp] = incl;
  if (tid == 0) sm.unit0 = sm.off0 = sm.row0 = sm.rows = 0;
  __syncthreads();
  long long ws = lane < kWarps ? sm.scan[lane] : 0;
  long long wi = ws;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, wi, o);
    if (lane >= o) wi += v;
  }
  const long long total = __shfl_sync(0xffffffffu, wi, 31);
  const long long before = __shfl_sync(0xffffffffu, wi - ws, warp) + incl - mine;
  if (tid == 0) sm.all = total;
  const long long tol = cut_tolerance(g, total);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const long long x = cut_at(g, blockIdx.x + e, total);
    if (x >= total) {
      if (tid == 0) (e ? sm.cut1 : sm.cut0) = total;
      continue;
    }
    if (x < before || x >= before + mine) continue;
    long long p = before;  // tile x lies in this thread's tokens
    for (int t = t0; t < t1; ++t) {
      const int tiles = t == t0 ? first : tiles_of(t);
      const long long w = (long long)(tiles)*g.groups;
      if (x < p + w) {
        int k = 0;  // the head group
        long long off = x - p;
        while (off >= tiles) off -= tiles, ++k;
        long long at = x;
        if (off <= tol) {
          at -= off;
          off = 0;
        } else if (tiles - off <= tol) {
          at += tiles - off;
          off = 0;
          ++k;
        }
        if (k == g.groups) k = 0, ++t;
        if (e == 0) {
          sm.cut0 = at;
          sm.unit0 = t * g.groups + k;
          sm.off0 = int(off);
          if (at < total) {
            const Rows r = t == t0 ? first_rows : rows_of(t);
            sm.row0 = int(r.r0);
            sm.rows = r.n;
          }
        } else {
          sm.cut1 = at;
        }
        break;
      }
      p += w;
    }
  }
  __syncthreads();
  if (tid == 0) {
    const long long run = sm.cut1 - sm.cut0;
    if (run > INT32_MAX - 8) atomicExch(&hdr->status, int32_t(DS4X_EDEVICE));  // (months of work)
    sm.total = int(min(run, (long long)(INT32_MAX - 8)));
  }
  // (padding has no parts)
  if (blockIdx.x == 0 && g.few && tid < kFewUnits && tid / g.groups >= valid) parts->span[tid] = make_int2(0, 0);
  // a range past what the table can place
  if (blockIdx.x == gridDim.x - 1 && a.idx == nullptr && !g.packed())
    for (int t = t0; t < min(t1, valid); ++t)
      if (past_table(a, t)) atomicExch(&hdr->status, int32_t(DS4X_EDEVICE));
  __syncthreads();
}

// ---- L: finding rows ------------------------------------------------------------

// A unit's queries toward L2: X converts them when the
// unit before it is done, some tiles from now (a chunk of 2048 lists: 255 us, was 264).
template <class A>
__device__ __forceinline__ void prefetch_queries(const A &g, int unit) {
  const Columns col(g, unit);
  const auto fetch = [](const void *p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
  };
  const int heads = A::packed() ? g.a.n_heads : col.n;
  for (int c = 0; c < col.n; c += heads)
    fetch(g.a.q + col.at(g, c, g.a.q_stride, kDim), uint32_t(heads) * kDim * 2);
}
template <class A>
__device__ __forceinline__ void load_entries(const A &g, int t, int pos, int n, int (&entry)[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (pos + 32 * k < n) entry[k] = __ldcg(g.a.idx + int64_t(t) * g.a.k + pos + 32 * k);
}

template <class A>
__device__ __forceinline__ void role_l(const A &g, Smem &sm, WsHeader *hdr) {
  const PagedAttn &a = g.a;
  const int total = sm.total;
  const int lane = threadIdx.x & 31;  // finds the tile's rows lane and 32 + lane
  PagedSeq sq{-1, 0, 0};
  int n_rows = 0;
  Walk w;
  w.begin(sm, total);
  for (;;) {
    const int t = g.packed() ? __ldcg(&g.plan->unit[w.unit].t0) : w.unit / g.groups;
    if (lane == 0 && w.i0 > 0 && w.off == w.from) prefetch_queries(g, w.unit);
    bool fresh = true;
    // a list's entries are on their way a tile ahead
    int entry[2] = {0, 0};
    if (a.idx != nullptr) load_entries(g, t, w.off * kTile + lane, w.n, entry);
    for (int i = w.i0; i < w.i1; ++i) {
      const int pos = (w.off + (i - w.i0)) * kTile + lane;
      int row[2];  // -1: none (a table reaches at most row 2^31 - 2)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        row[k] = -1;
        if (pos < w.n - 32 * k) row[k] = a.idx != nullptr ? entry[k] : w.r0 + pos + 32 * k;
      }
      if (a.idx != nullptr && i + 1 < w.i1) load_entries(g, t, pos + kTile, w.n, entry);
      if (fresh) {  // (looked up while the first entries are on their way)
        if (sq.s < 0 || t >= sq.to) {
          sq = paged_seq_of(a.c, t, lane);
          n_rows = INT32_MAX;
          if (a.idx != nullptr && sq.s >= 0)  // (below 0: no row)
            n_rows = int(max(int64_t(0), min(int64_t(INT32_MAX), int64_t(__ldcg(a.n_rows + sq.s)))));
        }
        fresh = false;
      }
      const int seq = sq.s;
      int2 at[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (seq < 0) row[k] = -1;
        const int j = row[k] >> a.c.page_log2;
        const bool in = row[k] >= 0 && j < a.c.seq_pages;
        const int32_t page = in ? __ldcg(a.c.table + int64_t(seq) * a.c.table_stride + j) : -1;
        at[k] = make_int2(page < a.c.n_pages ? max(page, -1) : -1, row[k] & ((1 << a.c.page_log2) - 1));
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (row[k] >= n_rows) at[k].x = -1;
        if (row[k] != -1 && at[k].x < 0) atomicExch(&hdr->status, int32_t(DS4X_EDEVICE));
      }
      Found f[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        f[k] = Found{nullptr, 0, 0};
        if (at[k].x >= 0) {
          const PagedRow p{a.c.pages + (int64_t(at[k].x) << a.c.page_log2) * DS4X_PAGED_ROW_BYTES, at[k].y};
          const int32_t co = int32_t(paged_code_off(p));
          f[k] = Found{p.page + co, int32_t(paged_tail_off(a.c, p)) - co, int32_t(paged_scale_off(a.c, p)) - co};
          // toward L2: the code lines (224 bytes lie in two or three) and the RoPE part's
          asm volatile("prefetch.global.L2 [%0];" ::"l"(f[k].codes));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(f[k].codes + 112));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(f[k].codes + 223));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(f[k].codes + f[k].tail));
        }
      }
      const int slot = i % kAhead;
      if (i >= kAhead) wait_bar(sm, &sm.lfree[slot], (i / kAhead - 1) & 1, hdr);
      sm.found[slot][lane] = f[0];
      sm.found[slot][32 + lane] = f[1];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.lfull[slot]));
    }
    if (w.i1 >= total) break;
    w.next(g, total);
  }
}

// ---- W: widening ----------------------------------------------------------------

// Eight lanes (a quarter-warp) take a row at a time, so that each of its loads is
// a row's 128 consecutive bytes: lane l of them the codes of block l, those of
// block 8 + l (l < 6) and chunk l of the RoPE part.  (Eight lanes on eight rows
// took 21 passes of the load pipe an instruction instead of 4 to 8.)  To store a
// block's words without bank conflicts the chunks of 8 values are dealt to V''s
// panels by word, not by block: word u of block b < 8 is chunk b of panel u; word u
// of block 8 + l is number l + 6 u of the 24 chunks of panels 4 to 6; the RoPE part
// is panel 7.  Q' is laid out alike, and the output's dims are put back.
__device__ __forceinline__ int v_chunk(int C) {  // where chunk C (values 8 C ..) lies: 8 panel + chunk
  if (C < 32) return 8 * (C & 3) + (C >> 2);
  if (C < 56) return 32 + ((C - 32) >> 2) + 6 * (C & 3);
  return C;
}
__device__ __forceinline__ int v_chunk_back(int P) {  // the C of place P
  if (P < 32) return 4 * (P & 7) + (P >> 3);
  if (P < 56) return 32 + 4 * ((P - 32) % 6) + (P - 32) / 6;
  return P;
}

struct Raw {
  uint4 a, b, t, sc;  // (the scale record's zero byte: 255 marks a row that is not there)
};
__device__ __forceinline__ void load_raw(const Found &at, int l, Raw &w) {
  const uint4 z = make_uint4(0, 0, 0, 0);
  if (at.codes != nullptr) {
    const uint8_t *lane = at.codes + 16 * l;
    w.sc = __ldcg(reinterpret_cast<const uint4 *>(at.codes + at.scales));
    w.a = __ldcg(reinterpret_cast<const uint4 *>(lane));
    w.b = l < 6 ? __ldcg(reinterpret_cast<const uint4 *>(lane + 128)) : z;
    w.t = __ldcg(reinterpret_cast<const uint4 *>(lane + at.tail));
  } else {
    w.a = w.b = w.t = z;
    w.sc = make_uint4(0, 0, 0, 0xff000000u);
  }
}

// NaN and infinities to the largest fp16 values.
__device__ __forceinline__ uint32_t finite_half2(uint32_t v) {
  asm("{\n\t.reg .b32 t;\n\tmax.f16x2 t, %0, %1;\n\tmin.f16x2 %0, t, %2;\n\t}" : "+r"(v) : "r"(0xfbfffbffu), "r"(0x7bff7bffu));
  return v;
}
// Eight codes times the factor pair f, as fp16, to shared memory.
__device__ __forceinline__ void widen8(uint32_t addr, uint32_t w, uint32_t f) {
  uint32_t h0, h1, h2, h3;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h0), "=r"(h1), "=r"(h2), "=r"(h3)
      : "r"(w));
  sts16(addr, hmul2_bits(h0, f), hmul2_bits(h1, f), hmul2_bits(h2, f), hmul2_bits(h3, f));
}
// A row (at `row`) of V', x = 16 (row % 8): panels 0 to 3, then 4 to 7.
__device__ __forceinline__ void widen_low(uint32_t row, uint32_t x, int l, const Raw &w) {
  const int E = int((w.sc.w >> 16) & 0xffu);
  const uint32_t f = pow2_half2(min(0, int(((l & 4 ? w.sc.y : w.sc.x) >> (8 * (l & 3))) & 0xffu) - E));
  const uint32_t pa = row + (uint32_t(l << 4) ^ x);
  widen8(pa, w.a.x, f);
  widen8(pa + 8192, w.a.y, f);
  widen8(pa + 2 * 8192, w.a.z, f);
  widen8(pa + 3 * 8192, w.a.w, f);
}
template <class A>
__device__ __forceinline__ void widen_high(uint32_t row, uint32_t x, int l, const uint32_t (&off_b)[4], const Raw &w) {
  const int E = int((w.sc.w >> 16) & 0xffu);
  // (packed: a row that only one token sees must not reach the others by 0 * NaN)
  auto t = [](uint32_t v) { return A::packed() ? finite_half2(v) : v; };
  sts16(row + 7 * 8192 + (uint32_t(l << 4) ^ x), t(w.t.x), t(w.t.y), t(w.t.z), t(w.t.w));
  if (l < 6) {
    const uint32_t f = pow2_half2(min(0, int(((l & 4 ? w.sc.w : w.sc.z) >> (8 * (l & 3))) & 0xffu) - E));
    widen8(row + (off_b[0] ^ x), w.b.x, f);
    widen8(row + (off_b[1] ^ x), w.b.y, f);
    widen8(row + (off_b[2] ^ x), w.b.z, f);
    widen8(row + (off_b[3] ^ x), w.b.w, f);
  }
}

// A unit's output (part -1), or its part: O^T over the denominator, M tiles k0 .. k1
// - 1, 128 dims each, by 32 heads (`half`); the warp's dims are 32 qd .. of each M
// tile.  (A step's loads are waited for before the loop goes round: a register that a
// load is still to write must not be moved.)
template <class A>
__device__ __forceinline__ void store_output(const A &g, Smem &sm, uint32_t tmem, Parts *parts, int unit, int part,
                                             int qd, int half, int k0, int k1) {
  const int lane = threadIdx.x & 31;
  const Columns col(g, unit);
#pragma unroll 1
  for (int k = k0; k < k1; ++k) {
    uint32_t o[2][16];
    const uint32_t ta = tmem + (uint32_t(32 * qd) << 16) + kOCol + 64u * k + 32u * half;
    tc_ld_x16(ta, o[0]);
    tc_ld_x16(ta + 16u, o[1]);
    tc_wait_ld();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int hc = 32 * half + 16 * j;  // heads hc .. hc + 15
      if (part >= 0) {
        float *po = &parts->o[part][hc][128 * k + 32 * qd + lane];
#pragma unroll
        for (int u = 0; u < 16; ++u)
          if (hc + u < col.n) po[u * kDim] = __uint_as_float(o[j][u]) * sm.hinv[hc + u];
      } else {
        // neighbouring lanes swap one of two heads, so each stores two dims of one head
        const int odd = lane & 1, d = 8 * v_chunk_back(16 * k + 4 * qd + (lane >> 3)) + (lane & 6);
        uint16_t *out = g.a.out + d + (A::packed() ? 0 : col.at(g, hc + odd, g.a.out_stride, kDim));
#pragma unroll
        for (int u = 0; u < 16; u += 2) {
          const float v0 = __uint_as_float(o[j][u]) * sm.hinv[hc + u];
          const float v1 = __uint_as_float(o[j][u + 1]) * sm.hinv[hc + u + 1];
          const float got = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
          const __nv_bfloat162 pr = odd ? __floats2bfloat162_rn(got, v1) : __floats2bfloat162_rn(v0, got);
          const int c = hc + u + odd;
          if (A::packed()) {
            const long long at = sm.out_at[c];
            if (at >= 0) *reinterpret_cast<__nv_bfloat162 *>(out + at) = pr;
          } else if (c < col.n) {
            *reinterpret_cast<__nv_bfloat162 *>(out + u * kDim) = pr;
          }
        }
      }
    }
  }
}

// A run's output joined to what the part holds of the runs before it (`again`); after
// a whole unit's last one (`done`) the output from there.  X's warps.
template <class A>
__device__ __noinline__ void store_run(const A &g, Smem &sm, uint32_t tmem, Parts *parts, int unit, int part, int xw,
                                       bool again, bool done) {
  const int lane = threadIdx.x & 31, qd = xw & 3, half = xw >> 2;
  const Columns col(g, unit);
  if (32 * half < g.n_cols) {
#pragma unroll 1
    for (int k = 0; k < 2 * kDim / 128; ++k) {
      const int hc = 32 * half + 16 * (k & 1);
      uint32_t o[16];
      tc_ld_x16(tmem + (uint32_t(32 * qd) << 16) + kOCol + 64u * (k >> 1) + uint32_t(hc), o);
      tc_wait_ld();
      float *po = &parts->o[part][hc][128 * (k >> 1) + 32 * qd + lane];
#pragma unroll
      for (int u = 0; u < 16; ++u)
        if (hc + u < col.n) {
          float v = __uint_as_float(o[u]) * sm.hinv[hc + u];
          if (again) v = fmaf(po[u * kDim], sm.keep[hc + u], v);
          po[u * kDim] = v;
        }
    }
  }
  if (!done) return;
  named_bar_sync(kBarX, kXThreads);
  for (int c = xw; c < col.n; c += kXWarps)
    for (int d0 = 4 * lane; d0 < kDim; d0 += 128) {
      const float4 o = __ldcg(reinterpret_cast<const float4 *>(&parts->o[part][c][d0]));
      const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
      const int d = 8 * v_chunk_back(d0 >> 3) + (d0 & 4);
      *reinterpret_cast<uint2 *>(g.a.out + col.at(g, c, g.a.out_stride, kDim) + d) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    }
}

template <class A>
__device__ __forceinline__ void role_w(const A &g, Smem &sm, Parts *parts, WsHeader *hdr) {
  const int total = sm.total;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - kWWarp0;
  const int l = lane & 7, q = lane >> 3;
  const int r = 8 * warp + q;            // the tile's rows that this lane helps to widen: r and r + 4
  uint32_t off_b[4];                     // block 8 + l's words, within a row
#pragma unroll
  for (int u = 0; u < 4; ++u) off_b[u] = uint32_t(4 + ((l + 6 * u) >> 3)) * 8192u + (uint32_t((l + 6 * u) & 7) << 4);
  const uint32_t row0 = smem_u32(sm.v[0]) + r * 128, x = uint32_t(q) << 4;
  auto load = [&](int i, Raw (&raw)[2]) {
    if (i >= total) return;
    const int slot = i % kAhead;
    wait_bar(sm, &sm.lfull[slot], (i / kAhead) & 1, hdr);
    const Found at0 = sm.found[slot][r], at1 = sm.found[slot][r + 4];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.lfree[slot]));
    load_raw(at0, l, raw[0]);
    load_raw(at1, l, raw[1]);
  };
  auto tile = [&](int i, int buf, Raw (&raw)[2]) {
    const uint32_t row = row0 + 65536u * buf;
    // the buffer's lower and upper panels come free one after the other
    if (i >= 2) wait_bar(sm, &sm.pvdone[buf][0], ((i >> 1) - 1) & 1, hdr);
    widen_low(row, x, l, raw[0]);
    widen_low(row + 4 * 128, x ^ 64u, l, raw[1]);
    if (i >= 2) wait_bar(sm, &sm.pvdone[buf][1], ((i >> 1) - 1) & 1, hdr);
    widen_high<A>(row, x, l, off_b, raw[0]);
    widen_high<A>(row + 4 * 128, x ^ 64u, l, off_b, raw[1]);
    bool wide = false;
    if (l < 2) {
      const uint32_t scw = l ? raw[1].sc.w : raw[0].sc.w;
      const int E = int((scw >> 16) & 0xffu) - 127;
      const bool none = scw >> 24;
      // (2^-(E + 7) finite for any byte: another token's bytes that are no row meet it as 0 times it)
      sm.rowe[buf][r + 4 * l] =
          none ? make_float4(0.0f, -INFINITY, 0.0f, 0.0f)
               : make_float4(pow2f(E), float(E), pow2f(-min(E, kPgExpMax) - kTop), float(E + kTop));
      wide = !none && (E > kTame || E < -kTame);
    }
    // lane 8 q + l: the warp's row q + 4 l
    const uint32_t wides = __ballot_sync(0xffffffffu, wide);
    if (lane == 0) {
      uint32_t rows = 0;
      if (wides != 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) rows |= (wides >> (8 * (k & 3) + (k >> 2)) & 1u) << k;
      }
      reinterpret_cast<uint8_t *>(&sm.wide[buf])[warp] = uint8_t(rows);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm.vfull[buf]));
    load(i + 2, raw);
  };
  Raw even[2], odd[2];
  load(0, even);
  load(1, odd);
  for (int i = 0; i < total; i += 2) {
    tile(i, 0, even);
    if (i + 1 < total) tile(i + 1, 1, odd);
  }
  // half of the last unit's output (a lone small call waits for little else)
  named_bar_sync(kBarEnd, kXThreads + 32 * kWWarps);
  const int half = warp >> 2, end = total - 1;
  wait_bar(sm, &sm.pvdone[end & 1][1], (end >> 1) & 1, hdr);
  tc_fence_after();
  if (sm.end_unit >= 0 && 32 * half < g.n_cols)
    store_output(g, sm, sm.tmem_base, parts, sm.end_unit, sm.end_part, warp & 3, half, kDim / 256, kDim / 128);
  tc_fence_before();
}

// ---- M: the products --------------------------------------------------------------
// The proxy fence between what W and X stored and what the tensor core reads is
// here, behind the barrier that orders their stores: in W it would wait for W's
// loads in flight.

// S of the tiles of one parity.
template <class A>
__device__ __forceinline__ void role_s(const A &g, Smem &sm, int b, WsHeader *hdr) {
  const int total = sm.total;
  const uint32_t tmem = sm.tmem_base;
  const uint32_t idS = idesc_f16(kTile, uint32_t(g.n_cols), 0, 0);  // V' K-major, Q' K-major
  const uint64_t dS_a = desc_sw128(smem_u32(sm.v[b]), 16, 1024), dS_b = desc_sw128(smem_u32(sm.q), 16, 1024);
  Walk w;
  w.begin(sm, total);
  for (int seg = 0;; ++seg) {
    wait_bar(sm, &sm.qfull, seg & 1, hdr);
    mbar_arrive(smem_u32(&sm.qtaken));
    for (int i = w.i0 + ((w.i0 ^ b) & 1); i < w.i1; i += 2) {
      wait_bar(sm, &sm.vfull[b], (i >> 1) & 1, hdr);
      fence_proxy_async_smem();
      tc_fence_after();
      // K step 4 p + ks: 16 dims, 32 ks bytes into panel p (descriptor addresses count 16 bytes)
#pragma unroll 2
      for (uint32_t p = 0; p < kDim / 64; ++p)
#pragma unroll
        for (uint32_t ks = 0; ks < 4; ++ks)
          mma_f16_ss(tmem + kSCol + 64u * b, dS_a + uint64_t(512 * p + 2 * ks), dS_b + uint64_t(512 * p + 2 * ks), idS,
                     p + ks);
      tc_commit(smem_u32(&sm.sfull[b]));
    }
    if (w.i1 >= total) break;
    w.next(g, total);
  }
  tc_commit(smem_u32(&sm.drain));  // nothing may still write this CTA's memory when it exits
  wait_bar(sm, &sm.drain, 0, hdr);
}

// O of every tile, in order.
template <class A>
__device__ __forceinline__ void role_o(const A &g, Smem &sm, WsHeader *hdr) {
  const int total = sm.total;
  const uint32_t tmem = sm.tmem_base;
  const uint32_t idO = idesc_f16(128, uint32_t(g.n_cols), 1, 1);  // V'^T MN-major, P^T MN-major
  const uint64_t dO_a0 = desc_sw128(smem_u32(sm.v[0]), 8192, 1024), dO_b0 = desc_sw128(smem_u32(sm.p[0]), 8192, 1024);
  Walk w;
  w.begin(sm, total);
  for (;;) {
    for (int i = w.i0; i < w.i1; ++i) {
      const int b = i & 1;
      wait_bar(sm, &sm.pfull[b], (i >> 1) & 1, hdr);
      fence_proxy_async_smem();
      tc_fence_after();
      const uint64_t dO_a = dO_a0 + uint64_t(4096 * b), dO_b = dO_b0 + uint64_t(512 * b);
      const uint32_t acc = i > w.i0 ? 1u : 0u;
      // M tile mi: panels 2 mi, 2 mi + 1; K step ks: 16 rows (2 KB)
#pragma unroll
      for (int mi = 0; mi < kDim / 128; ++mi) {
#pragma unroll
        for (int ks = 0; ks < kTile / 16; ++ks)
          mma_f16_ss(tmem + kOCol + 64u * mi, dO_a + uint64_t(1024 * mi + 128 * ks), dO_b + uint64_t(128 * ks), idO,
                     ks > 0 ? 1u : acc);
        if (mi & 1) tc_commit(smem_u32(&sm.pvdone[b][mi >> 1]));  // the lower panels are read, all are
      }
    }
    if (w.i1 >= total) break;
    w.next(g, total);
  }
  tc_commit(smem_u32(&sm.drain));
  wait_bar(sm, &sm.drain, 0, hdr);
}

// ---- X: softmax and output ------------------------------------------------------------

// Q' of a unit: warp w of X converts columns 8 w .. 8 w + 7, lane L the 16-byte
// chunks L and 32 + L of each; columns that the unit does not have are zeros.  All of
// a warp's loads are in flight at once (64 registers: the unit's maxima and sums
// must be in shared memory by then).
template <class A>
__device__ __forceinline__ void make_query(const A &g, Smem &sm, int unit, int xw, int lane) {
  const Columns col(g, unit);
  if (g.packed() && xw == 0 && lane < kPackTokens) {  // (warp 0)
    const Rows u = unit_rows(g, unit);
    const Rows r = lane * g.a.n_heads < col.n ? token_rows(g.a, col.t0 + lane) : Rows{0, 0};
    const int lo = r.n > 0 ? int(r.r0 - u.r0) : 0;
    sm.seen[lane] = make_int2(lo, lo + r.n);
  }
  const long long mine = col.at(g, 8 * xw + (A::packed() ? lane & 7 : 0), g.a.q_stride, kDim);
  const uint4 *q = reinterpret_cast<const uint4 *>(g.a.q + (A::packed() ? 0 : mine)) + lane;
  uint4 qv[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = 8 * xw + (i >> 1);
    const long long at = A::packed() ? __shfl_sync(0xffffffffu, mine, i >> 1) / 8 + 32 * (i & 1) : 32 * i;
    qv[i] = c < col.n ? __ldcg(q + at) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    // the column's largest exponent field e, and the scale that brings it to 14
    uint32_t m = 0;
#pragma unroll
    for (int i = 2 * k; i < 2 * k + 2; ++i) {
      const uint32_t w4[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) m = __vmaxu2(m, w4[u] & 0x7fff7fffu);
    }
    const int e = int(__reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16)) >> 7);
    const int c = max(-113, min(126, 14 + 127 - max(e, 1)));
    const float f = pow2f(c);
    const int h = 8 * xw + k;
    // A column with NaN or infinity (all its logits are, so all its results) is computed
    // as zeros, so that rows that are not there stay out, and marked: out and lse are NaN.
    const bool odd = e == 255;
    if (lane == 0) {
      sm.qscale[h] = g.a.scale * kLog2e * pow2f(-c);
      sm.qodd[h] = odd ? __int_as_float(0x7fffffff) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int P = v_chunk(32 * i + lane);
      const uint4 v = qv[2 * k + i];
      const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        o[u] = odd ? 0u : half2_bits(__uint_as_float(w4[u] << 16) * f, __uint_as_float(w4[u] & 0xffff0000u) * f);
      sts16(smem_u32(sm.q) + (P >> 3) * 8192 + h * 128 + (((P & 7) ^ (h & 7)) << 4), o[0], o[1], o[2], o[3]);
    }
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&sm.qfull));
}

template <class A>
__device__ __forceinline__ void role_x(const A &g, Smem &sm, Parts *parts, WsHeader *hdr) {
  const int total = sm.total;
  const uint32_t tmem = sm.tmem_base;
  const PagedAttn &a = g.a;
  const int lane = threadIdx.x & 31, xw = (threadIdx.x >> 5) - kXWarp0, xt = threadIdx.x - 32 * kXWarp0;
  const int qd = xw & 3, half = xw >> 2;        // tile rows 16 qd .., heads 32 half ..
  const bool busy = 32 * half < g.n_cols;
  const int r0 = 16 * qd + (lane >> 2);         // this lane's rows r0 and r0 + 8
  const int hb = 32 * half + 2 * (lane & 3);    // this lane's heads hb + 8 j + c
  const uint32_t lane_base = uint32_t(32 * qd) << 16;
  // P^T: row r0, heads hb, hb + 1; heads 8 j on at the 16-byte chunk's number ^ j
  const uint32_t p0 = smem_u32(sm.p[0]) + r0 * 128 + (((4 * half) ^ (r0 & 7)) << 4) + 4 * (lane & 3);
  make_query(g, sm, sm.unit0, xw, lane);
  if (A::packed()) named_bar_sync(kBarX, kXThreads);  // `seen`
  Walk w;
  w.begin(sm, total);
  for (int seg = 0;; ++seg) {
    float m[8], sum[8];  // head hb + 8 j + c: 2 j + c (m: kTop below the maximum)
#pragma unroll
    for (int k = 0; k < 8; ++k) m[k] = 0.0f, sum[k] = 0.0f;
    // bit k: no row so far for that head (for all heads or none, unless packed); m is 0
    // and not a maximum yet
    uint32_t fresh = busy ? 0xffu : 0u;
    // bit k: that head has had a row with an exponent beyond +-kTame (for all heads or none, unless
    // packed).  In the tiles' order and the run's own, so that nothing else shows in the sums' rounding.
    uint32_t wide = 0;
    int lo = 0, hi = INT32_MAX;          // packed: the rows that all of the unit's tokens see
    if (A::packed()) {
      const int count = __ldcg(&g.plan->unit[w.unit].count);
      for (int j = 0; j < count; ++j) {
        lo = max(lo, sm.seen[j].x);
        hi = min(hi, sm.seen[j].y);
      }
    }
    for (int i = w.i0; i < w.i1; ++i) {
      const int b = i & 1;
      wait_bar(sm, &sm.sfull[b], (i >> 1) & 1, hdr);
      tc_fence_after();
      float d[16];  // x - m of row r0 + 8 r: d[4 j + 2 r + c]
      float inv[2] = {0.0f, 0.0f}, er[2] = {0.0f, 0.0f};  // the rows' 2^-(E_j + 7), E_j + 7
      float over = -INFINITY;
      if (busy) {
        uint32_t s[16];
        tc_ld_16x256_x4(tmem + lane_base + kSCol + 64u * b + 32u * half, s);
        const float4 e0 = sm.rowe[b][r0], e1 = sm.rowe[b][r0 + 8];
        const float ef[2] = {e0.y, e1.y};
        if (const unsigned long long rows = sm.wide[b]) {
          if (!A::packed()) {
            wide = 0xffu;
          } else {
            const int first = (w.off + (i - w.i0)) * kTile;
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
              const int j = ((hb + 8 * (k >> 1) + (k & 1)) * g.per_head) >> 16;
              if (j >= kPackTokens) break;
              const int from = max(0, sm.seen[j].x - first), to = min(kTile, sm.seen[j].y - first);
              if (to > from && (rows >> from & ~0ull >> (kTile - (to - from)))) wide |= 1u << k;
            }
          }
        }
        inv[0] = e0.z, inv[1] = e1.z;
        er[0] = e0.w, er[1] = e1.w;
        float2 qs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) qs[k] = *reinterpret_cast<const float2 *>(&sm.qscale[hb + 8 * k]);
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const int row = (k >> 1) & 1, h = 2 * (k >> 2);
          const float er2 = row ? e1.x : e0.x;
          float2 x = fma2(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])),
                          mul2(qs[k >> 2], make_float2(er2, er2)), make_float2(ef[row], ef[row]));
          x = add2(x, make_float2(-m[h], -m[h + 1]));
          d[k] = x.x;
          d[k + 1] = x.y;
          over = fmaxf(fmaxf(over, d[k]), d[k + 1]);
        }
      }
      bool moves = over > kLazy || fresh != 0;
      if (A::packed()) {
        const int first = (w.off + (i - w.i0)) * kTile;
        if (busy && (first < lo || first > hi - kTile)) {  // rows that some token does not see
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int row = first + r0 + 8 * ((k >> 1) & 1), j = ((hb + 8 * (k >> 2) + (k & 1)) * g.per_head) >> 16;
            if (j < kPackTokens && (row < sm.seen[j].x || row >= sm.seen[j].y)) d[k] = -INFINITY;
          }
        }
        moves = false;  // a maximum is passed, or a first row sets one, however small
#pragma unroll
        for (int k = 0; k < 16; ++k)
          moves = moves || d[k] > ((fresh >> (2 * (k >> 2) + (k & 1)) & 1) ? -INFINITY : kLazy);
        moves = moves && busy;
      }
      if (named_bar_or(kBarX, kXThreads, moves)) {
        // some head's maximum moves: each head's maximum over the tile
        if (busy) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float mx = fmaxf(d[4 * (k >> 1) + (k & 1)], d[4 * (k >> 1) + 2 + (k & 1)]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (lane < 4) sm.red[qd][hb + 8 * (k >> 1) + (k & 1)] = mx;
          }
        }
        named_bar_sync(kBarX, kXThreads);
        if (busy) {
          const uint32_t was_fresh = fresh;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int h = hb + 8 * (k >> 1) + (k & 1);
            float up = fmaxf(fmaxf(sm.red[0][h], sm.red[1][h]), fmaxf(sm.red[2][h], sm.red[3][h]));
            // (columns past the unit's hold what an earlier kernel left in tensor memory: where
            // that is NaN in every row, it must not end the others' wait for a first row)
            const bool none = !(up > -INFINITY);
            up = none || !((was_fresh >> k & 1) || up > kLazy) ? 0.0f : up - kTop;
            if (!none) fresh &= A::packed() ? ~(1u << k) : 0u;
            m[k] += up;
            d[4 * (k >> 1) + (k & 1)] -= up;
            d[4 * (k >> 1) + 2 + (k & 1)] -= up;
            // what there is so far times 2^-up (zeros, before a first row, whose `up` may be far
            // below zero); in halves for the sum (rows far apart in size: 2^-up itself may underflow)
            up = fmaxf(up, 0.0f);
            const float half_al = ex2(-0.5f * up);
            sum[k] = sum[k] * half_al * half_al;
            if (qd == 0 && lane < 4) sm.alpha[h] = ex2(-up);
          }
        }
        named_bar_sync(kBarX, kXThreads);
        if (i > w.i0 && busy) {
          // O^T of the unit so far, once the previous tile's product is done
          wait_bar(sm, &sm.pvdone[b ^ 1][1], ((i - 1) >> 1) & 1, hdr);
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < 2 * kDim / 128; ++k) {
            const uint32_t ta = tmem + lane_base + kOCol + 64u * (k >> 1) + 32u * half + 16u * (k & 1);
            uint32_t o[16];
            tc_ld_x16(ta, o);
            tc_wait_ld();
#pragma unroll
            for (int u = 0; u < 16; ++u)
              o[u] = __float_as_uint(__uint_as_float(o[u]) * sm.alpha[32 * half + 16 * (k & 1) + u]);
            tc_st_x16(ta, o);
          }
          tc_wait_st();
        }
      }
      if (busy) {
        // Rows of very different size: a weight 2^(l_j + E_j - m) may underflow although
        // its part of the denominator, 2^-(E_j + 7) as large, does not; then that is formed
        // by itself.  (While all |E_j| <= kTame a lost part is below 2^-86 of the whole.)
        if (wide) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int h = 2 * (k >> 2) + (k & 1);
            if (!A::packed() || (wide >> h & 1)) sum[h] += ex2(d[k] - er[(k >> 1) & 1]);
          }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) d[k] = ex2(d[k]);
        if (wide != 0xffu) {
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const int row = (k >> 1) & 1, h = 2 * (k >> 2);
            const float2 t = fma2(make_float2(d[k], d[k + 1]), make_float2(inv[row], inv[row]),
                                  make_float2(sum[h], sum[h + 1]));
            if (!A::packed() || !(wide >> h & 1)) sum[h] = t.x;
            if (!A::packed() || !(wide >> (h + 1) & 1)) sum[h + 1] = t.y;
          }
        }
#pragma unroll
        for (int k = 0; k < 16; k += 2)  // (rows r0 and r0 + 8 have the same place in their 8 rows)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"((p0 ^ uint32_t((k >> 2) << 4)) + 8192u * b +
                                                       1024u * ((k >> 1) & 1)),
                       "r"(half2_bits(d[k], d[k + 1])));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.pfull[b]));
    }
    // ---- the unit's share is done: sums over the rows ------------------------------------
#pragma unroll
    for (int k = 0; k < 8; ++k) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
    }
    // (the mark is read before this barrier: behind it other warps write the next unit's)
    if (busy && qd == 0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) m[k] += kTop + sm.qodd[hb + 8 * (k >> 1) + (k & 1)];
    }
    named_bar_sync(kBarX, kXThreads);  // the last readers of red, mh and hinv are done
    if (busy && lane < 4) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int h = hb + 8 * (k >> 1) + (k & 1);
        sm.red[qd][h] = sum[k];
        if (qd == 0) sm.mh[h] = m[k];
      }
    }
    // the next unit's Q' (this one's last first product is done: its softmax is)
    const bool last = w.i1 >= total, more = w.more(total);
    if (!last) {
      wait_bar(sm, &sm.qtaken, seg & 1, hdr);  // (an S thread without a tile in this unit may not have seen its Q' yet)
      if (!more) {
        make_query(g, sm, w.unit + 1, xw, lane);
      } else if (lane == 0) {
        mbar_arrive(smem_u32(&sm.qfull));  // the same
      }
    }
    named_bar_sync(kBarX, kXThreads);
    const bool whole = w.from == 0 && w.off + (w.i1 - w.i0) == w.tiles;
    const bool again = w.off != w.from, runs = more || again;  // not the share's first run; not its only one
    const int part = 2 * int(blockIdx.x) + (w.from == 0 ? 1 : 0);
    if (A::packed() && xt < kHeads) {  // (all 64: store_output looks at 32 at a time)
      const Columns col(g, w.unit);
      sm.out_at[xt] = xt < col.n ? col.at(g, xt, a.out_stride, kDim) : -1;
    }
    if (xt < g.n_cols) {
      const float tot = (sm.red[0][xt] + sm.red[1][xt]) + (sm.red[2][xt] + sm.red[3][xt]);
      // (m is finite or NaN)
      float inv = tot > 0.0f ? __frcp_rn(tot) * pow2f(-kTop) + 0.0f * sm.mh[xt] : 0.0f;
      float l2 = tot > 0.0f ? sm.mh[xt] + log2f(tot) : -INFINITY;
      if (runs) {
        const float l0 = again ? sm.run2[xt] : -INFINITY, mx = fmaxf(l0, l2);
        const float a = l0 == -INFINITY ? 0.0f : exp2f(l0 - mx), b = l2 == -INFINITY ? 0.0f : exp2f(l2 - mx), z = a + b;
        if (z != 0.0f) {  // (NaN stays)
          inv *= b / z;
          l2 = mx + log2f(z);
        }
        sm.keep[xt] = z != 0.0f ? a / z : 0.0f;
        sm.run2[xt] = l2;
      }
      sm.hinv[xt] = inv;
      const Columns col(g, w.unit);
      if (xt < col.n && !more) {
        if (!whole)
          parts->lse2[part][xt] = l2;
        else if (a.lse != nullptr)
          a.lse[col.at(g, xt, a.n_heads, 1)] = l2 * 0.6931471805599453f;
      }
    }
    if (xt == 0 && !whole && !more) parts->unit[part] = w.unit;
    if (xt == 0 && g.few && w.from == 0 && !more) {
      parts->span[w.unit] = make_int2(int(blockIdx.x), whole ? 1 : unit_parts(g, sm.cut0 + w.i0 - w.off + w.tiles, sm.all));
    }
    named_bar_sync(kBarX, kXThreads);
    wait_bar(sm, &sm.pvdone[(w.i1 - 1) & 1][1], ((w.i1 - 1) >> 1) & 1, hdr);
    tc_fence_after();
    if (last) {
      if (xt == 0) {
        sm.end_unit = runs ? -1 : w.unit;
        sm.end_part = whole ? -1 : part;
      }
      named_bar_sync(kBarEnd, kXThreads + 32 * kWWarps);  // W, done with its tiles, takes half of the output
    }
    if (runs)
      store_run(g, sm, tmem, parts, w.unit, part, xw, again, whole);
    else if (busy)
      store_output(g, sm, tmem, parts, w.unit, whole ? -1 : part, qd, half, 0, last ? kDim / 256 : kDim / 128);
    tc_fence_before();
    if (w.i1 >= total) break;
    w.next(g, total);
  }
}

// Packs tokens into units: the tokens of a sequence in order, as many as n_heads
// goes into 64 columns, so that a row is widened once for all of them and the
// products' 64 columns are full.  One block; bound by latency (about 3 us).
constexpr int kPlanThreads = 1024, kPlanSeqs = 4096;
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(PagedAttn a, int pack, Plan *__restrict__ plan,
                                                                  WsHeader *__restrict__ hdr) {
  __shared__ int32_t cus[kPlanSeqs + 1], warps[kPlanThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_seqs = a.c.n_seqs;
  const bool held = n_seqs <= kPlanSeqs;
  if (held)
    for (int i = tid; i <= n_seqs; i += kPlanThreads) cus[i] = __ldcg(a.c.cu + i);
  const int valid = max(0, min(a.n_tokens, __ldcg(a.c.cu + n_seqs)));
  __syncthreads();
  auto cu = [&](int s) { return held ? cus[s] : __ldcg(a.c.cu + s); };
  int base = 0;
  for (int c0 = 0; c0 < valid; c0 += kPlanThreads) {
    const int t = c0 + tid;
    int count = 0, units = 0;  // the tokens from t on, and the units they make
    Pack u{t, 1, 0, 0};
    if (t < valid) {
      int s = 0, n = n_seqs;  // the last sequence that begins at or before t
      while (n > 1) {
        const int half = n / 2;
        if (cu(s + half) <= t) s += half, n -= half;
        else n = half;
      }
      const int from = cu(s), to = min(valid, cu(s + 1));
      if (!(from <= t && t < to)) {  // (cu is not what it should be: a unit without a row)
        units = 1;
      } else if ((t - from) % pack == 0) {
        count = min(pack, to - t);
        int rest = 0;  // tokens whose rows do not meet those from lo to hi
        int64_t lo = 0, hi = 0;
        for (int j = 0; j < count; ++j) {
          if (past_table(a, t + j)) atomicExch(&hdr->status, int32_t(DS4X_EDEVICE));
          const Rows r = token_rows(a, t + j);
          if (r.n == 0) continue;
          if (hi == 0) lo = r.r0, hi = r.r0 + r.n;
          else if (r.r0 > hi || r.r0 + r.n < lo) ++rest;
          else lo = min(lo, r.r0), hi = max(hi, r.r0 + r.n);
        }
        // Rows between the tokens' ranges, which no token sees, must not be read (and
        // would be work for nothing): then each token is its own unit.
        units = rest > 0 ? count : 1;
        u = Pack{t, count, int32_t(lo), int32_t(hi - lo)};
      }
    }
    int incl = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
    int at = base + incl - units;
    for (int k = 0; k < kPlanThreads / 32; ++k) {
      if (k < warp) at += warps[k];
      base += warps[k];
    }
    if (units == 1) plan->unit[at] = u;
    if (units > 1)
      for (int j = 0; j < count; ++j) {
        const Rows r = token_rows(a, t + j);
        plan->unit[at + j] = Pack{t + j, 1, int32_t(r.r0), r.n};
      }
    __syncthreads();
  }
  if (tid == 0) plan->n_units = base;
}

template <bool P>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(ArgsFor<P> g, Parts *__restrict__ parts,
                                                                 WsHeader *__restrict__ hdr) {
  // (no static shared memory: the dynamic begins at the window's start, as aligned as Smem asks)
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sm.vfull[b]), kWWarps);
      mbar_init(smem_u32(&sm.sfull[b]), 1);
      mbar_init(smem_u32(&sm.pfull[b]), kXWarps);
      mbar_init(smem_u32(&sm.pvdone[b][0]), 1);
      mbar_init(smem_u32(&sm.pvdone[b][1]), 1);
    }
    for (int k = 0; k < kAhead; ++k) {
      mbar_init(smem_u32(&sm.lfull[k]), 1);
      mbar_init(smem_u32(&sm.lfree[k]), kWWarps);
    }
    mbar_init(smem_u32(&sm.qfull), kXWarps);
    mbar_init(smem_u32(&sm.qtaken), 2);
    mbar_init(smem_u32(&sm.drain), 3);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMWarp0) {
    tmem_alloc(smem_u32(&sm.tmem_base), 512);
    tmem_relinquish();
  }
  // Launched as a programmatic dependent: nothing above touches global memory.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid < 2) parts->unit[2 * blockIdx.x + tid] = -1;
  tc_fence_before();
  find_cuts(g, sm, parts, hdr);  // (its barriers also publish the barriers and the tensor memory's address)
  tc_fence_after();
  if (sm.total > 0) {
    if (warp >= kXWarp0) {
      set_regs_up<kRegsX>();
      role_x(g, sm, parts, hdr);
    } else if (warp >= kWWarp0) {
      set_regs_down<kRegsW>();
      role_w(g, sm, parts, hdr);
    } else {
      set_regs_down<kRegsLM>();
      if (warp < kMWarp0) {
        role_l(g, sm, hdr);
      } else {
        if (elect_one()) {
          if (warp < kMWarp0 + 2)
            role_s(g, sm, warp - kMWarp0, hdr);
          else
            role_o(g, sm, hdr);
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMWarp0) {
    tc_fence_after();
    tmem_dealloc(sm.tmem_base, 512);
  }
}

// Joins the parts of the units that several CTAs share.  A warp takes 128 dims (a
// float4 a lane) of a head, eight parts on their way at once.  Where the unit has at
// most 16 parts, a block's 16 warps take four heads; else 128 dims of one head, its
// parts dealt over them (a unit split over every CTA has 64 heads to go round: 256
// blocks then read 9 or 10 parts a warp).  Sums go in a fixed order.
constexpr int kJoinWarps = 16, kJoinThreads = 32 * kJoinWarps, kJoinFew = 16;

__global__ void __launch_bounds__(kJoinThreads, 2) paged_combine_kernel(Args g, const Parts *__restrict__ parts,
                                                                         int ctas) {
  __shared__ int unit[2 * kMaxCtas];
  // the shared units: the CTA that begins each, its parts, the items before it
  __shared__ int first[kMaxCtas], count[kMaxCtas], item0[kMaxCtas + 1], n_units;
  __shared__ float wts[kJoinWarps][kMaxCtas];
  __shared__ float4 part_sum[kJoinWarps][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = tid; i < 2 * kMaxCtas; i += kJoinThreads) unit[i] = i < 2 * ctas ? __ldcg(parts->unit + i) : -1;
  __syncthreads();
  if (warp == 0) {
    constexpr int kWords = kMaxCtas / 32;
    uint32_t more[kWords];  // bit c: CTA c goes on with the unit that the CTA before it went on with
    int n = 0;
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const int c = 32 * k + lane, u = unit[2 * c];
      more[k] = __ballot_sync(0xffffffffu, c > 0 && u >= 0 && u == unit[2 * c - 2]);
    }
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const int c = 32 * k + lane;
      const bool is = unit[2 * c + 1] >= 0;
      const uint32_t b = __ballot_sync(0xffffffffu, is);
      if (is) first[n + __popc(b & ((1u << lane) - 1))] = c;
      n += __popc(b);
    }
    __syncwarp();
    int items = 0;
    for (int e0 = 0; e0 < n; e0 += 32) {
      const int e = e0 + lane;
      int mine = 0;
      if (e < n) {
        int c = first[e] + 1;  // the unit's next part is CTA c's, then those of a run of set bits
        if (c < kMaxCtas && unit[2 * c] == unit[2 * c - 1]) ++c;
#pragma unroll
        for (int k = 0; k < kWords; ++k)
          if (c >= 32 * k && c < 32 * k + 32) {
            const uint32_t clear = ~more[k] >> (c & 31);  // (shifted-in zeros: the word's end)
            c = clear != 0 ? c + __ffs(int(clear)) - 1 : 32 * k + 32;
          }
        count[e] = c - first[e];
        const int heads = Columns(g, unit[2 * first[e] + 1]).n;
        mine = count[e] <= kJoinFew ? (heads + 3) / 4 : 4 * heads;
      }
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (e < n) item0[e] = items + incl - mine;
      items += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      n_units = n;
      item0[n] = items;
    }
  }
  __syncthreads();
  const int items = item0[n_units];
  for (int item = blockIdx.x, e = 0; item < items; item += gridDim.x) {
    while (item >= item0[e + 1]) ++e;
    const int c0 = first[e], n = count[e], u = unit[2 * c0 + 1];
    const Columns col(g, u);
    const int heads = col.n;
    const bool few = n <= kJoinFew;
    const int it = item - item0[e], quarter = few ? warp & 3 : it & 3;
    const int h = few ? 4 * it + (warp >> 2) : it >> 2;
    const int k0 = few ? 0 : warp, step = few ? 1 : kJoinWarps;
    const bool writes = few || warp == 0;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (h < heads) {  // (a block's warps differ in it only where few)
      auto slot = [&](int k) { return k == 0 ? 2 * c0 + 1 : 2 * (c0 + k); };
      float m = -INFINITY, s = 0.0f;
      for (int k = lane; k < n; k += 32) m = fmaxf(m, wts[warp][k] = __ldcg(&parts->lse2[slot(k)][h]));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      for (int k = lane; k < n; k += 32) {
        const float x = wts[warp][k], w = x == -INFINITY ? 0.0f : exp2f(x - m);
        wts[warp][k] = w;
        s += w;
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      __syncwarp();
      const float inv = s > 0.0f ? 1.0f / s : 0.0f;
      const int d0 = 128 * quarter + 4 * lane;
      for (int k = k0; k < n; k += 8 * step) {
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i * step < n) v[i] = __ldcg(reinterpret_cast<const float4 *>(&parts->o[slot(k + i * step)][h][d0]));
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i * step < n) {
            const float w = wts[warp][k + i * step] * inv;
            o.x = fmaf(w, v[i].x, o.x);
            o.y = fmaf(w, v[i].y, o.y);
            o.z = fmaf(w, v[i].z, o.z);
            o.w = fmaf(w, v[i].w, o.w);
          }
      }
      if (!few) part_sum[warp][lane] = o;
      if (lane == 0 && quarter == 0 && writes && g.a.lse != nullptr)
        g.a.lse[col.at(g, h, g.a.n_heads, 1)] = s == 0.0f ? -INFINITY : (m + log2f(s)) * 0.6931471805599453f;
    }
    if (!few) {
      __syncthreads();
      if (warp == 0)
#pragma unroll
        for (int k = 1; k < kJoinWarps; ++k) {
          const float4 v = part_sum[k][lane];
          o = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
        }
      __syncthreads();
    }
    if (h < heads && writes) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
      const int d = 8 * v_chunk_back(16 * quarter + (lane >> 1)) + 4 * (lane & 1);
      *reinterpret_cast<uint2 *>(g.a.out + col.at(g, h, g.a.out_stride, kDim) + d) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    }
    __syncwarp();  // wts is read
  }
}

// The same for at most kFewUnits units, where a call's latency counts: a block takes
// 256 dims of a head, its parts dealt over four pairs of warps; no list to make first
// (the units' spans are written by the CTAs that begin them).  A call over 777 rows
// takes 13.4 us so, 15.6 by the list.  Up to 16 units (kFewUnits), with cold caches: 9 of
// 4096 to 8192 rows 38.9 us, 51.2 by the list, 16 of 600 to 1200 rows 34.8, 36.8; above,
// 32 of those 43.0, 41.0, while 32 lists of 512 rows would take 28.7, 32.8.
constexpr int kFewThreads = 256;
__global__ void __launch_bounds__(kFewThreads) paged_combine_few_kernel(Args g, const Parts *__restrict__ parts) {
  __shared__ float wts[kMaxCtas], lsum, lmax;
  __shared__ float4 part_sum[kFewThreads / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = blockIdx.x >> 7, h = (blockIdx.x >> 1) & 63;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (h >= g.n_cols) return;
  const int2 span = __ldcg(&parts->span[u]);
  const int c0 = span.x, n = span.y;
  if (n <= 1) return;  // one CTA wrote it all
  const Columns col(g, u);
  if (h >= col.n) return;
  auto slot = [&](int k) { return k == 0 ? 2 * c0 + 1 : 2 * (c0 + k); };
  const int d0 = 256 * (blockIdx.x & 1) + 128 * (warp & 1) + 4 * lane, deal = warp >> 1;
  // the first parts on their way, then the weights
  float4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (deal + 4 * i < n) v[i] = __ldcg(reinterpret_cast<const float4 *>(&parts->o[slot(deal + 4 * i)][h][d0]));
  if (warp == 0) {
    float x[kMaxCtas / 32], m = -INFINITY, s = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxCtas / 32; ++i) {
      x[i] = lane + 32 * i < n ? __ldcg(&parts->lse2[slot(lane + 32 * i)][h]) : -INFINITY;
      m = fmaxf(m, x[i]);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
#pragma unroll
    for (int i = 0; i < kMaxCtas / 32; ++i) {
      const float w = x[i] == -INFINITY ? 0.0f : exp2f(x[i] - m);
      wts[lane + 32 * i] = w;
      s += w;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) {
      lsum = s;
      lmax = m;
    }
  }
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = deal;;) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + 4 * i < n) {
        const float w = wts[k + 4 * i];
        o.x = fmaf(w, v[i].x, o.x);
        o.y = fmaf(w, v[i].y, o.y);
        o.z = fmaf(w, v[i].z, o.z);
        o.w = fmaf(w, v[i].w, o.w);
      }
    k += 32;
    if (k >= n) break;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + 4 * i < n) v[i] = __ldcg(reinterpret_cast<const float4 *>(&parts->o[slot(k + 4 * i)][h][d0]));
  }
  part_sum[warp][lane] = o;
  __syncthreads();
  if (deal != 0) return;
  const float s = lsum, inv = s > 0.0f ? 1.0f / s : 0.0f;
#pragma unroll
  for (int k = 1; k < 4; ++k) {
    const float4 p = part_sum[warp + 2 * k][lane];
    o = make_float4(o.x + p.x, o.y + p.y, o.z + p.z, o.w + p.w);
  }
  const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  const int d = 8 * v_chunk_back(d0 >> 3) + (d0 & 4);
  *reinterpret_cast<uint2 *>(g.a.out + col.at(g, h, g.a.out_stride, kDim) + d) =
      make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
  if (threadIdx.x == 0 && (blockIdx.x & 1) == 0 && g.a.lse != nullptr)
    g.a.lse[col.at(g, h, g.a.n_heads, 1)] = s == 0.0f ? -INFINITY : (lmax + log2f(s)) * 0.6931471805599453f;
}

// The same where a unit has at most kShortParts tiles (short lists): a warp takes 128
// dims of a head with all its parts on their way at once, and nothing is shared (16
// sessions' lists of 512 rows: 17.5 us a call, 20.8 by the kernel above).
constexpr int kShortParts = 16, kShortThreads = 256;
__global__ void __launch_bounds__(kShortThreads) paged_combine_short_kernel(Args g, const Parts *__restrict__ parts) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = blockIdx.x >> 5, h = 2 * (blockIdx.x & 31) + (warp >> 2);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (h >= g.n_cols) return;
  const int2 span = __ldcg(&parts->span[u]);
  const int c0 = span.x, n = span.y;
  if (n <= 1) return;  // one CTA wrote it all
  const Columns col(g, u);
  if (h >= col.n) return;
  auto slot = [&](int k) { return k == 0 ? 2 * c0 + 1 : 2 * (c0 + k); };
  const int d0 = 128 * (warp & 3) + 4 * lane;
  const float x = lane < n ? __ldcg(&parts->lse2[slot(lane)][h]) : -INFINITY;
  float4 v[kShortParts];
#pragma unroll
  for (int k = 0; k < kShortParts; ++k)
    if (k < n) v[k] = __ldcg(reinterpret_cast<const float4 *>(&parts->o[slot(k)][h][d0]));
  float m = x;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float w = x == -INFINITY ? 0.0f : exp2f(x - m);
  float s = w;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  const float inv = s > 0.0f ? 1.0f / s : 0.0f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kShortParts; ++k) {
    const float wk = __shfl_sync(0xffffffffu, w, k) * inv;
    if (k < n) {
      o.x = fmaf(wk, v[k].x, o.x);
      o.y = fmaf(wk, v[k].y, o.y);
      o.z = fmaf(wk, v[k].z, o.z);
      o.w = fmaf(wk, v[k].w, o.w);
    }
  }
  const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
  const int d = 8 * v_chunk_back(d0 >> 3) + (d0 & 4);
  *reinterpret_cast<uint2 *>(g.a.out + col.at(g, h, g.a.out_stride, kDim) + d) =
      make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
  if (lane == 0 && (warp & 3) == 0 && g.a.lse != nullptr)
    g.a.lse[col.at(g, h, g.a.n_heads, 1)] = s == 0.0f ? -INFINITY : (m + log2f(s)) * 0.6931471805599453f;
}

}  // namespace

size_t paged_attn_ws_bytes() { return kWsHeaderBytes + sizeof(Parts) + sizeof(Plan); }

cudaError_t launch_paged_attn(const PagedAttn &a, void *ws, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_set[2];
  const int smem = int(sizeof(Smem));
  cudaError_t e = set_max_smem_once(paged_attn_kernel<false>, smem, smem_set[0]);
  if (e == cudaSuccess) e = set_max_smem_once(paged_attn_kernel<true>, smem, smem_set[1]);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  WsHeader *hdr = static_cast<WsHeader *>(ws);
  Parts *parts = reinterpret_cast<Parts *>(hdr + 1);
  Plan *plan = reinterpret_cast<Plan *>(parts + 1);
  // no more CTAs than there can be tiles
  const int64_t rows = a.idx != nullptr ? a.k : int64_t(a.c.seq_pages) << a.c.page_log2;
  const int groups = (a.n_heads + kHeads - 1) / kHeads;
  const int64_t most = int64_t(a.n_tokens) * groups * ((rows + kTile - 1) / kTile);
  const int ctas = int(most < sms ? most : sms) < kMaxCtas ? int(most < sms ? most : sms) : kMaxCtas;
  // Several tokens a unit where two or more fit its columns, some sequence must have
  // two, and single tokens could fill more than two tiles a CTA: below that the plan's
  // launch costs more than the passes that it saves.  Packed / single, us a call:
  // 1 sequence x 2 tokens x 20 heads x 700 rows 17.1 / 12.2, 8 x 2 x 16 x 2000
  // 22.4 / 23.0, 24 x 5 x 20 x 4500 66 / 130, 1 x 512 x 16 x 4096 124 / 420.
  const int pack = kHeads / a.n_heads < kPackTokens ? kHeads / a.n_heads : kPackTokens;
  const bool packed = a.idx == nullptr && pack > 1 && a.n_tokens > a.c.n_seqs && most > 2 * ctas;
  Args g{a, packed ? plan : nullptr, groups, 0, 0, 0, 0, 0};
  g.few = int64_t(a.n_tokens) * g.groups <= kFewUnits;
  g.group = packed ? pack * a.n_heads : (a.n_heads + g.groups - 1) / g.groups;
  g.per_head = 65536 / a.n_heads + 1;
  g.n_cols = (g.group + 15) / 16 * 16;
  g.per_grid = ~uint64_t(0) / uint64_t(ctas) + 1;  // (one CTA: 0, and its one inner cut is 0)
  if (packed) {
    e = launch_pdl(paged_plan_kernel, 1u, unsigned(kPlanThreads), size_t(0), stream, a, pack, plan, hdr);
    if (e != cudaSuccess) return e;
  }
  e = packed ? launch_pdl(paged_attn_kernel<true>, unsigned(ctas), unsigned(kThreads), size_t(smem), stream,
                          ArgsFor<true>(g), parts, hdr)
             : launch_pdl(paged_attn_kernel<false>, unsigned(ctas), unsigned(kThreads), size_t(smem), stream,
                          ArgsFor<false>(g), parts, hdr);
  if (e != cudaSuccess) return e;
  if (ctas == 1) return cudaSuccess;  // nothing is split
  if (g.few && (rows + kTile - 1) / kTile <= kShortParts)
    return launch_pdl(paged_combine_short_kernel, unsigned(a.n_tokens * g.groups * kHeads / 2),
                      unsigned(kShortThreads), size_t(0), stream, g, static_cast<const Parts *>(parts));
  if (g.few)
    return launch_pdl(paged_combine_few_kernel, unsigned(a.n_tokens * g.groups * 2 * kHeads), unsigned(kFewThreads),
                      size_t(0), stream, g, static_cast<const Parts *>(parts));
  return launch_pdl(paged_combine_kernel, unsigned(2 * sms), unsigned(kJoinThreads), size_t(0), stream, g,
                    static_cast<const Parts *>(parts), ctas);
}

}  // namespace ds4x
