// nvfp4_attention.cu -- attention of one new token per sequence over a paged
// key-value cache.
//
//   s_t = scale ks (q . k_t), m = max s_t, l = sum exp(s_t - m),
//   out = vs / l sum exp(s_t - m) v_t, lse = m + ln l, over the visible tokens.
//
// Bound: HBM.  Every visible key and value is read once; the products are
// 4 flop per element and query head of the group, far below the tensor cores'
// rate, so the work is to keep enough copies in flight.  Measured: 16 x 32768
// tokens (64 heads on 8 of 128, bf16) 308 us, 7.0 TB/s; 3 x 65536 (E4M3) 70 us, 5.8
// TB/s; 61 ragged sequences of up to 2048 (32 heads on 8, bf16) 48 us, 5.4 TB/s.
// Short items are bound by their instructions and their latency instead: 256
// sequences, window 128, 16 E4M3 heads of 64 take 30 us, where an item of 4 tiles is
// 3000 warp instructions over all roles; one sequence of 517 tokens takes 8.4 us.
// So are the large head blocks that leave one CTA per SM, with one consuming warp
// per scheduler: 16 x 8192 tokens with 32 heads on one of 128 take 36 us in bf16 and
// 30 in E4M3 (2.2 TB/s), with 16 on one of 256 38 and 33.  Heads of 256 in groups of
// up to 8 (16 x 8192, 16 heads on 4) take 88 us, 6.1 TB/s, and 51 in E4M3, 5.3 TB/s.
//
// Work split: an item is one sequence and one block of up to 8 NT query heads
// that share a cache head.  Its visible tokens are cut into tiles of KT, and the
// tiles of all items form one sequence; CTA c takes the contiguous range
// [c T / G, (c + 1) T / G) of it (an item counts kAttItemCost tiles more than
// it has), so ragged lengths balance without the host
// knowing them.  The part of an item inside a CTA's range is a segment.  The
// kAttWarps consuming warps share a segment's tiles, each with a running maximum,
// sum and output of its own (no barrier inside a segment), and meet in shared
// memory at the segment's end, which costs about 4000 clocks; so an item of few
// tiles is one warp's alone: of as many as its ring holds, because the loads of
// more would hold up the other warps' where two share a loading warp, and leave
// them idle at a range's end (with up to 12 tiles in rings of 2, 256 x 300 tokens of
// bf16 heads of 128 took 45 us instead of 40).  An item inside one CTA is finished
// there; the parts of a longer one go to the workspace, where a second launch
// (k_attend_join) adds them in CTA order, so that results do not depend on
// timing.  (When the CTA that came last added them, behind a fence and a counter,
// it cost up to 14 us under load: 61 ragged sequences of up to 2048 tokens took
// 62 us.)
//
// Loads: two or four more warps fill a ring of S tiles per consuming warp by TMA, across
// segments (keys and values of a page as boxes of 128-byte rows, 128-byte
// swizzle; pages outside the cache read as zeros), and the queries of each
// segment.  When the consumers asked for their own tiles, that took 700 clocks
// of each tile's 1700.
//
// Products: mma.sync with the tokens as the M side, S^T = K Q^T and
// O^T = V^T P^T: 16 tokens x 8 heads fill an m16n8 tile, so a group of 8 heads
// wastes nothing, and S^T and O^T keep a head in the same lanes, so the running
// maximum never moves between lanes.  (tcgen05 would want 64 or 128 rows of
// tokens per instruction and the softmax through tensor memory; at 4 flop per
// byte per head the legacy path is not the limit.)  bf16 keys and values enter
// as they are, and P as the sum of two bf16 numbers, 16 bits together: rounded to
// one, it was the largest error before the output's own rounding (61 ragged
// sequences: 1.86e-3 of the output's norm off against 1.66e-3), and the second
// product costs 0 to 1 % where HBM is the bound (16 x 32768: 308 us with and
// without), 5 to 7 % where instructions are (256 x 300, window 128, heads of 64,
// 43.1 -> 45.1 us).  E4M3 ones are converted exactly to f16; q is scaled by a power
// of two per head to fit f16 (its entries keep their 8 bits down to 2^-27 of the
// head's largest), and P, scaled by 2^14, keeps 11 bits, which the output's error
// does not show (1.658e-3 against 1.656e-3 in fp32).
#include <algorithm>
#include <cstring>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {

constexpr int kAttWarps = 4;
constexpr int kAttConsumers = kAttWarps * 32;
constexpr int kAttMinTiles = 4;      // tiles per CTA below which fewer CTAs take part
constexpr int kAttMaxCtas = 1024;
constexpr int kAttItemCost = 6;      // an item's cost apart from its tiles, in tiles
constexpr int kAttTries = 2000;      // x 1 ms: bound of a wait for a copy

template <int D, bool E4M3, int NT>
struct AttCfg {
  static constexpr int kElem = E4M3 ? 1 : 2;
  static constexpr int kRow = D * kElem;                       // bytes of a token's key
  static constexpr int kBoxRow = kRow < 128 ? kRow : 128;      // bytes of a box's row = swizzle span
  static constexpr int kBoxes = kRow / kBoxRow;
  static constexpr int KT = kRow <= 128 ? 32 : 16;             // tokens per tile
  static constexpr int kHalf = KT * kRow;                      // bytes of a tile's keys
  static constexpr int kTile = 2 * kHalf;
  static constexpr int kHeads = 8 * NT;
  // Loading warps, each for the rings of kAttWarps / kLoaders consumers.  A
  // consumer each takes 256 x 300 tokens (window 128, E4M3, heads of 64) from
  // 34.6 to 31.9 us; where registers are short, the threads of four would cost
  // more than they give (16 x 8192 tokens, E4M3, heads of 256: 34.5 -> 42.4 us,
  // 12 heads per cache head of 64: 26.4 -> 28.2 us).
  static constexpr int kLoaders = NT == 1 && D < 256 ? 4 : 2;
  static constexpr int kThreads = kAttConsumers + 32 * kLoaders;
  static constexpr int kRedStride = D + 4;                     // floats; keeps the lanes of a store in distinct banks
  static constexpr int kRed = kAttWarps * kHeads * kRedStride * 4;
  static constexpr int kQRow = D * 2;                          // bytes of a staged query head
  static constexpr int kQ = kHeads * kQRow;
  static constexpr int NQ = NT == 1 && D < 256 ? 8 : 2;        // segments whose queries are staged ahead
  static constexpr int kBudget = 113 * 1024 - 2048;  // dynamic shared memory of one of the CTAs per SM
  static constexpr int S0 = (kBudget - 1024 - kRed - NQ * kQ) / (kAttWarps * kTile);
  static constexpr int S = S0 >= 6 ? 6 : S0 >= 2 ? S0 : 2;
  static constexpr int kRing = kAttWarps * S * kTile;
  static constexpr size_t kSmem = 1024 + kRing + kRed + NQ * kQ;
  static_assert(kSmem <= 226 * 1024, "shared memory");
};

__device__ __forceinline__ uint32_t att_smem(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ float att_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// c += a b, 16 x 8 x 16, fp32 accumulators; f16 or bf16 operands.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two E4M3 bytes -> two f16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;\n\t}" : "=r"(r) : "r"(b));
  return r;
}

// {lo, hi} fp32 -> packed 16-bit pair.
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

// Orders this thread's reads of shared memory before copies into it that other
// threads start once they have been told: without it the last loads of a tile
// could still be on their way when the next tile landed (one tile in a million
// took dimensions 112 .. 127 of its values from the next one).
__device__ __forceinline__ void att_reads_done() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One thread of a converged warp, known as such to the compiler.
__device__ __forceinline__ bool att_elect() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

__device__ __forceinline__ bool att_wait(uint32_t mb, uint32_t parity, int tries) {
  for (int i = 0; i < tries; ++i) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(done) : "r"(mb), "r"(parity), "r"(1000000u) : "memory");
    if (done) return true;
  }
  return false;
}

// An item that several CTAs share, from CTA c on: what k_attend_join needs.
struct AttShared {
  int64_t row;       // sequence * q_heads + first head
  int heads, parts;  // parts 0: no such item begins in this CTA
};

// What the kernel needs beside the caller's arguments.
struct AttLaunch {
  AttendArgs a;
  AttShared *shared;  // [G]
  float *part;        // [2 G][heads][D] sums, then [2 G][heads][2] maxima and sums
  int blocks;         // head blocks per cache head
  int piece_shift;    // log2 of the rows of a box: min(page, KT)
};

// Quotient of non-negative integers; the 64-bit one only where it is needed.
__device__ __forceinline__ int64_t att_div(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The even split of T tiles over G CTAs (at most T): the first T mod G take one more.
struct AttSplit {
  int64_t q;  // T / G
  int r;      // T mod G
  __device__ __forceinline__ AttSplit(int64_t T, int G) {
    q = att_div(T, G);
    r = (int)(T - q * G);
  }
  __device__ __forceinline__ int64_t first(int c) const { return c * q + min(c, r); }
  __device__ __forceinline__ int cta_of(int64_t g) const {
    const int64_t longer = r * (q + 1);
    return (int)(g < longer ? att_div(g, q + 1) : r + att_div(g - longer, q));
  }
};

// A position in a CTA's range: a segment (tiles [first, first + count) of
// sequence b, head block hg) and what is left behind it.  The split counts
// units: an item's tiles and, before them, kAttItemCost more, which stand for
// what an item costs apart from its tiles.
struct AttSeg {
  int b, hg;
  int kh, blk;       // hg = kh * blocks + blk
  int first, count;  // tiles, numbered from token 0
  int off, total;    // the segment's place among the item's tiles, and their number
  int unit;          // the segment's place among the item's units
  int units;         // the segment's units
  int64_t left;      // units of the range behind this segment
  int n, lo;         // visible tokens [lo, n)
};

__device__ __forceinline__ void att_visible(const AttendArgs &a, int b, int &n, int &lo) {
  const int64_t cap = a.kv.table_width << a.kv.page_shift;  // at most 2^30
  n = (int)max((int64_t)0, min((int64_t)__ldg(a.lengths + b), cap));
  lo = a.window > 0 && n > a.window ? n - (int)a.window : 0;
}
template <int KT>
__device__ __forceinline__ int att_tiles(int n, int lo) { return n > 0 ? (n - 1) / KT - lo / KT + 1 : 0; }

__device__ __forceinline__ int att_units(int tiles) { return tiles > 0 ? tiles + kAttItemCost : 0; }

// The segment from unit `unit` of item (b, hg) on, at most `left` units long.
template <int KT>
__device__ __forceinline__ void att_segment(AttSeg &s, int unit, int64_t left) {
  s.unit = unit;
  s.units = (int)min((int64_t)(att_units(s.total) - unit), left);
  s.left = left - s.units;
  s.off = max(unit - kAttItemCost, 0);
  s.count = max(unit + s.units - kAttItemCost, 0) - s.off;
  s.first = s.lo / KT + s.off;
}
// Who takes a segment's tiles: one warp all of them, or tile j warp
// (first + j) % 4; the next segment begins with the warp after the last one.
// Loaders and consumers each count along.  (Handing out by the tiles that each
// warp has been given balances no better, and every warp pays for it at every
// segment.)
struct AttTeam {
  int next = 0;
  bool solo;
  int first;
  __device__ __forceinline__ void take(const AttSeg &s, int most) {
    solo = s.count == s.total && s.count <= most;
    first = next;
    next = (next + (solo ? 1 : s.count)) & (kAttWarps - 1);
  }
};

// Moves to the next segment that has tiles; false: there is none.
template <int KT>
__device__ __forceinline__ bool att_next(const AttendArgs &a, AttSeg &s, int groups, int blocks) {
  do {
    if (s.left == 0) return false;
    if (++s.blk == blocks) {
      s.blk = 0;
      ++s.kh;
    }
    if (++s.hg == groups) {
      s.hg = s.kh = 0;
      do {  // (a later sequence holds the units that are left)
        att_visible(a, ++s.b, s.n, s.lo);
      } while (s.n == 0);
      s.total = att_tiles<KT>(s.n, s.lo);
    }
    att_segment<KT>(s, 0, s.left);
  } while (s.count == 0);
  return true;
}

// 14: the scale 2^14 of E4M3's weights, which the sums have too.
template <bool E4M3>
__device__ __forceinline__ float att_lse(float ref, float sum) {
  return (ref - (E4M3 ? 14.0f : 0.0f) + log2f(sum)) * 0.69314718055994531f;
}

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(AttCfg<D, E4M3, NT>::kThreads) k_attend(const __grid_constant__ CUtensorMap kmap,
                                                        const __grid_constant__ CUtensorMap vmap,
                                                        const __grid_constant__ AttLaunch p) {
  using C = AttCfg<D, E4M3, NT>;
  constexpr int KT = C::KT, S = C::S, SUB = KT / 16, KS = D / 16;
  extern __shared__ uint8_t dsm[];
  // full: a tile has landed; empty: it has been read; q_*: the queries of a segment
  __shared__ __align__(8) uint64_t full[kAttWarps * S], empty[kAttWarps * S], q_full[C::NQ], q_empty[C::NQ];
  __shared__ int64_t s_sum[C::kThreads / 32];
  __shared__ int s_start[6], s_fail;
  __shared__ float s_ml[kAttWarps][C::kHeads][2];
  const AttendArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.q_heads / a.kv.kv_heads, groups = a.kv.kv_heads * p.blocks;
  const uint32_t raw = att_smem(dsm), base = (raw + 1023u) & ~1023u;
  float *red = reinterpret_cast<float *>(dsm + (base - raw) + C::kRing);  // [warps][heads][kRedStride]
  const uint32_t qs_smem = base + C::kRing + C::kRed;
  pdl_launch_dependents();  // k_attend_join waits for the whole grid all the same

  for (int i = tid; i < kAttWarps * S; i += C::kThreads) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(att_smem(&full[i])) : "memory");
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(att_smem(&empty[i])) : "memory");
  }
  if (tid < C::NQ) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(att_smem(&q_full[tid])) : "memory");
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(att_smem(&q_empty[tid])), "r"(kAttWarps) : "memory");
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (tid == 0) s_fail = 0;

  // ---- all tiles, this CTA's range of them, and the item where it begins: a
  // run of sequences per thread
  const int c = blockIdx.x;
  const int per = (a.sequences + C::kThreads - 1) / C::kThreads;
  const int sb0 = min(tid * per, a.sequences), sb1 = min(sb0 + per, a.sequences);
  int64_t mine = 0;
  for (int b = sb0; b < sb1; ++b) {
    int n, lo;
    att_visible(a, b, n, lo);
    mine += att_units(att_tiles<KT>(n, lo));
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int64_t T = 0;
#pragma unroll
  for (int w = 0; w < C::kThreads / 32; ++w) {
    if (w < warp) incl += s_sum[w];
    T += s_sum[w];
  }
  T *= groups;
  const int G = (int)min((int64_t)gridDim.x, max((int64_t)1, (T + kAttMinTiles - 1) / kAttMinTiles));
  const AttSplit split(T, G);
  const int64_t g0 = c < G ? split.first(c) : T, g1 = c < G ? split.first(c + 1) : T;
  AttSeg seg = {};
  if (g0 < g1 && (incl - mine) * groups <= g0 && g0 < incl * groups) {  // one thread
    int64_t rem = g0 - (incl - mine) * groups;
    for (seg.b = sb0;; ++seg.b) {
      att_visible(a, seg.b, seg.n, seg.lo);
      seg.total = att_tiles<KT>(seg.n, seg.lo);
      const int64_t all = (int64_t)att_units(seg.total) * groups;
      if (rem < all) break;
      rem -= all;
    }
    s_start[0] = seg.b;
    s_start[1] = (int)att_div(rem, att_units(seg.total));
    s_start[2] = (int)(rem - (int64_t)s_start[1] * att_units(seg.total));
    s_start[3] = seg.n;
    s_start[4] = seg.lo;
    s_start[5] = seg.total;
  }
  __syncthreads();
  if (g0 < g1) {
    seg.b = s_start[0];
    seg.hg = s_start[1];
    seg.kh = seg.hg / p.blocks;
    seg.blk = seg.hg - seg.kh * p.blocks;
    seg.n = s_start[3];
    seg.lo = s_start[4];
    seg.total = s_start[5];
    att_segment<KT>(seg, s_start[2], g1 - g0);
  }
  const bool any = g0 < g1 && (seg.count > 0 || att_next<KT>(a, seg, groups, p.blocks));  // tiles in the range

  AttTeam team;
  if (warp >= kAttWarps) {
    // ---- loads: a consumer's u-th tile goes to stage u % S of its ring
    constexpr int kMine = kAttWarps / C::kLoaders;  // consumers of this loader: kMine * loader ..
    const int loader = warp - kAttWarps;
    int given = 0;  // lane w: tiles given to consumer w
    if (any) {
      const int piece = 1 << p.piece_shift, pp = KT >> p.piece_shift;  // pieces (pages) per tile: 1, 2 or 4
      const int page_mask = (1 << a.kv.page_shift) - 1;
      int ids_b = -1, ids_base = 0, ids = -1;  // this lane's page number, for tiles of ids_b from ids_base on
      bool ok = true;
      for (int k = 0; ok; ++k) {  // segments
        const int kh = seg.kh, h0 = kh * group + seg.blk * C::kHeads;
        const int heads = min(C::kHeads, (kh + 1) * group - h0), qb = k % C::NQ;
        if (loader == 0) {
          // (a warp gives up as a whole: its lanes meet in the shuffles and elections below)
          if (!__all_sync(0xFFFFFFFFu, att_wait(att_smem(&q_empty[qb]), ((uint32_t)(k / C::NQ) & 1u) ^ 1u, kAttTries))) break;
          if (att_elect()) {
            const uint32_t q_bar = att_smem(&q_full[qb]);
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + seg.b * a.q_stride + (int64_t)h0 * D;
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(q_bar), "r"(heads * D * 2) : "memory");
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                         ::"r"(qs_smem + qb * C::kQ), "l"(q), "r"(heads * D * 2), "r"(q_bar) : "memory");
          }
          __syncwarp();
        }
        team.take(seg, S);
        for (int j = 0; j < seg.count; ++j) {
          const int t = seg.first + j, w = team.solo ? team.first : (team.first + j) & (kAttWarps - 1);
          if (w / kMine != loader) continue;
          if (ids_b != seg.b || t < ids_base || t >= ids_base + 32 / pp) {  // page numbers of 32 / pp tiles, a lane each
            ids_b = seg.b;
            ids_base = t;
            const int tok = (t + lane / pp) * KT + (lane % pp) * piece;
            ids = tok < seg.n ? __ldg(a.kv.table + seg.b * a.kv.table_stride + (tok >> a.kv.page_shift)) : -1;
          }
          const int t0 = t * KT, pieces = min(pp, (seg.n - t0 + piece - 1) >> p.piece_shift);
          int page[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (x == 0 || pp > 1) page[x] = __shfl_sync(0xFFFFFFFFu, ids, ((t - ids_base) * pp + x) & 31);
          const int u = __shfl_sync(0xFFFFFFFFu, given, w), at = w * S + u % S;
          if (!__all_sync(0xFFFFFFFFu, att_wait(att_smem(&empty[at]), ((uint32_t)(u / S) & 1u) ^ 1u, kAttTries))) {
            ok = false;
            break;
          }
          if (att_elect()) {
            const uint32_t mb = att_smem(&full[at]), dst = base + at * C::kTile;
            // (the pieces of a tile are whole pages, except where a page holds the whole tile)
            const int y = (kh << a.kv.page_shift) + (pp == 1 ? t0 & page_mask : 0);
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                         ::"r"(mb), "r"(2 * pieces * piece * C::kRow) : "memory");
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (x < pieces) {
#pragma unroll
                for (int i = 0; i < 2 * C::kBoxes; ++i) {
                  const int kind = i / C::kBoxes, box = i % C::kBoxes;
                  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                               " [%0], [%1, {%2, %3, %4}], [%5];"
                               ::"r"(dst + kind * C::kHalf + box * (KT * C::kBoxRow) + x * piece * C::kBoxRow),
                                 "l"(kind ? &vmap : &kmap), "r"(box * (C::kBoxRow / C::kElem)), "r"(y), "r"(page[x]), "r"(mb)
                               : "memory");
                }
              }
          }
          __syncwarp();
          if (lane == w) ++given;
        }
        if (!att_next<KT>(a, seg, groups, p.blocks)) break;
      }
    }
    __syncthreads();  // the consumers are done
    if (s_fail)       // copies that nothing waited for: let them land
      for (int w = kMine * loader; w < kMine * (loader + 1); ++w) {
        const int n = __shfl_sync(0xFFFFFFFFu, given, w);
        for (int u = max(0, n - S); u < n; ++u) att_wait(att_smem(&full[w * S + u % S]), (uint32_t)(u / S) & 1u, kAttTries);
      }
    return;
  }

  // ---- rows of empty sequences
  for (int b = blockIdx.x; b < a.sequences; b += gridDim.x) {
    int n, lo;
    att_visible(a, b, n, lo);
    if (n > 0) continue;
    uint4 *o = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + (int64_t)b * a.q_heads * D);
    for (int i = tid; i < a.q_heads * D / 8; i += kAttConsumers) o[i] = make_uint4(0u, 0u, 0u, 0u);
    if (a.lse)
      for (int i = tid; i < a.q_heads; i += kAttConsumers) a.lse[(int64_t)b * a.q_heads + i] = -INFINITY;
  }
  AttShared shared = {0, 0, 0};
  if (!any) {
    if (tid == 0) p.shared[c] = shared;
    __syncthreads();
    return;
  }

  int stage = 0;            // of this warp's next tile
  uint32_t full_ph = 0u;
  bool bad = false;         // a copy did not arrive in time: this warp's sums become NaN
  bool dead = false;        // nor later: nothing is waited for or handed back any more
  int tries = p.a.first_tries >= 0 && warp == 0 ? p.a.first_tries : kAttTries;
  // ldmatrix rows and chunks of this lane
  const int krow = (lane & 7) + ((lane >> 3) & 1) * 8, kchk = lane >> 4;
  const int vrow = E4M3 ? krow : (lane & 7) + ((lane >> 4) & 1) * 8, vchk = E4M3 ? kchk : (lane >> 3) & 1;
  auto chunk_at = [&](int row, int ch) {  // byte offset of 16-byte chunk ch of a row of a tile's half
    constexpr int kPer = C::kBoxRow / 16;
    const int sw = C::kBoxRow == 128 ? row & 7 : (row >> 1) & 3;
    return (uint32_t)((ch / kPer) * (KT * C::kBoxRow) + row * C::kBoxRow + (((ch % kPer) ^ sw) << 4));
  };

  for (int k = 0;; ++k) {
    team.take(seg, S);
    const int turn = (warp - team.first) & (kAttWarps - 1);  // this warp's first tile of the segment
    // (Every warp waits for and hands back the queries of every segment, with
    // tiles in it or not: a warp that skipped some could be two phases off the
    // mbarrier, which a parity cannot tell from none.)
    const int qb = k % C::NQ;
    if (!dead && !__all_sync(0xFFFFFFFFu, att_wait(att_smem(&q_full[qb]), (uint32_t)(k / C::NQ) & 1u, kAttTries)))
      bad = dead = true;
    if (team.solo && turn != 0) {  // another warp's
      if (lane == 0 && !dead)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(att_smem(&q_empty[qb])) : "memory");
      if (!att_next<KT>(a, seg, groups, p.blocks)) break;
      continue;
    }
    const int kh = seg.kh, h0 = kh * group + seg.blk * C::kHeads;
    const int heads = min(C::kHeads, (kh + 1) * group - h0);
    const float sc = a.scale * (E4M3 && a.kv.k_scale ? __ldg(a.kv.k_scale + kh) : 1.0f) * 1.4426950408889634f;

    // ---- q as the B side: this lane's head is 8 nt + lane / 4
    uint32_t qf[NT][KS][2];
    float qs[NT][2];  // factor of the scores of heads 8 nt + 2 (lane % 4) + j
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // (rows past the last head hold anything: their columns of S^T and O^T are not used)
      const uint32_t qrow = qs_smem + qb * C::kQ + (8 * nt + (lane & 7)) * C::kQRow;
      if (E4M3) {  // dimensions 4c .. 4c + 3 of the step: the order in which ldmatrix hands out bytes
        const uint32_t at = qs_smem + qb * C::kQ + (8 * nt + (lane >> 2)) * C::kQRow + 8 * (lane & 3);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(qf[nt][ks][0]), "=r"(qf[nt][ks][1]) : "r"(at + 32 * ks) : "memory");
      } else {
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2) {
          uint32_t r[4];
          ldsm4<false>(qrow + 32 * ks + 16 * (lane >> 3), r);
          qf[nt][ks][0] = r[0], qf[nt][ks][1] = r[1], qf[nt][ks + 1][0] = r[2], qf[nt][ks + 1][1] = r[3];
        }
      }
      qs[nt][0] = qs[nt][1] = sc;
      if (E4M3) {
        uint32_t top = 0u;  // bf16 bits of the head's largest |q|
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w = qf[nt][ks][j] & 0x7FFF7FFFu;
            top = max(top, max(w & 0xFFFFu, w >> 16));
          }
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // 2^-up takes the largest into [2^13, 2^14); inf and NaN heads stay as they are
        const int e = (int)(top >> 7), up = e == 255 ? 0 : max(e, 1) - 127 - 13;
        const float f1 = __uint_as_float((uint32_t)(127 - up / 2) << 23), f2 = __uint_as_float((uint32_t)(127 - (up - up / 2)) << 23);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w = qf[nt][ks][j];
            qf[nt][ks][j] = pack16<true>(__uint_as_float(w << 16) * f1 * f2, __uint_as_float(w & 0xFFFF0000u) * f1 * f2);
          }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int u = __shfl_sync(0xFFFFFFFFu, up, 4 * (2 * (lane & 3) + j));
          qs[nt][j] = sc * __uint_as_float((uint32_t)(127 + u / 2) << 23) * __uint_as_float((uint32_t)(127 + u - u / 2) << 23);
        }
      }
    }

    float o[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int d = 0; d < KS; ++d)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][d][j] = 0.0f;
    }

    for (int t = seg.first + turn; t < seg.first + seg.count; t += team.solo ? 1 : kAttWarps) {
      const int at = warp * S + stage;
      if (!dead && !__all_sync(0xFFFFFFFFu, att_wait(att_smem(&full[at]), full_ph, tries))) {
        bad = true;  // (a stage goes back only once its copy has landed)
        dead = !__all_sync(0xFFFFFFFFu, att_wait(att_smem(&full[at]), full_ph, kAttTries));
      }
      tries = kAttTries;
      const uint32_t kb = base + at * C::kTile, vb = kb + C::kHalf;
      const int t0 = t * KT;
      const bool edge = t0 < seg.lo || t0 + KT > seg.n;
      if (edge) {
        // values outside [lo, n) become zeros: their weights are zero, but what is stored there need not be finite
        for (int i = lane; i < KT * (C::kRow / 16); i += 32) {
          const int row = i / (C::kRow / 16);
          if (t0 + row < seg.lo || t0 + row >= seg.n)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vb + chunk_at(row, i % (C::kRow / 16))), "r"(0)
                         : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next copy into this stage
        __syncwarp();
      }

      // ---- S^T: 16 SUB tokens x 8 NT heads
      float s[SUB][NT][4];
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[u][nt][j] = 0.0f;
      if (E4M3) {
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2)
#pragma unroll
          for (int u = 0; u < SUB; ++u) {
            uint32_t r[4];
            ldsm4<false>(kb + chunk_at(16 * u + krow, ks + kchk), r);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t f[4] = {e4m3x2_f16x2(r[2 * x]), e4m3x2_f16x2(r[2 * x + 1]), e4m3x2_f16x2_hi(r[2 * x]),
                                     e4m3x2_f16x2_hi(r[2 * x + 1])};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<true>(s[u][nt], f, qf[nt][ks + x][0], qf[nt][ks + x][1]);
            }
          }
      } else {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int u = 0; u < SUB; ++u) {
            uint32_t r[4];
            ldsm4<false>(kb + chunk_at(16 * u + krow, 2 * ks + kchk), r);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<false>(s[u][nt], r, qf[nt][ks][0], qf[nt][ks][1]);
          }
      }

      // ---- running maximum and sum: this lane's tokens lane / 4 (+ 8), heads 2 (lane % 4) + {0, 1}
      bool grew = false;
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = -INFINITY;
#pragma unroll
          for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float &v = s[u][nt][2 * r + j];
              v *= qs[nt][j];
              if (edge) {
                const int tok = t0 + 16 * u + 8 * r + (lane >> 2);
                if (tok < seg.lo || tok >= seg.n) v = -INFINITY;
              }
              x = fmaxf(x, v);
            }
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, w));
          top[nt][j] = fmaxf(m[nt][j], x);
          grew |= top[nt][j] > m[nt][j];
        }
      if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float f = top[nt][j] == m[nt][j] ? 1.0f : att_exp2(m[nt][j] - top[nt][j]);
            m[nt][j] = top[nt][j];
            l[nt][j] *= f;
#pragma unroll
            for (int d = 0; d < KS; ++d) {
              o[nt][d][j] *= f;
              o[nt][d][2 + j] *= f;
            }
          }
      }
      uint32_t pf[SUB][NT][2], pl[SUB][NT][2];  // (pl: bf16 only)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float ref[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) ref[j] = m[nt][j] == -INFINITY ? 0.0f : E4M3 ? m[nt][j] - 14.0f : m[nt][j];
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float x = att_exp2(s[u][nt][2 * r] - ref[0]), y = att_exp2(s[u][nt][2 * r + 1] - ref[1]);
            l[nt][0] += x;
            l[nt][1] += y;
            const uint32_t w = pack16<E4M3>(x, y);
            pf[u][nt][r] = transpose8x8(w);
            if (!E4M3)
              pl[u][nt][r] = transpose8x8(pack16<false>(x - __uint_as_float(w << 16), y - __uint_as_float(w & 0xFFFF0000u)));
          }
      }

      // ---- O^T += V^T P^T
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        if (E4M3) {
#pragma unroll
          for (int d = 0; d < KS; d += 2) {
            uint32_t r[4];
            ldsm4<true>(vb + chunk_at(16 * u + vrow, d + vchk), r);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t w0 = __byte_perm(r[2 * x], 0u, 0x3120), w1 = __byte_perm(r[2 * x + 1], 0u, 0x3120);
              const uint32_t f[4] = {e4m3x2_f16x2(w0), e4m3x2_f16x2_hi(w0), e4m3x2_f16x2(w1), e4m3x2_f16x2_hi(w1)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<true>(o[nt][d + x], f, pf[u][nt][0], pf[u][nt][1]);
            }
          }
        } else {
#pragma unroll
          for (int d = 0; d < KS; ++d) {
            uint32_t r[4];
            ldsm4<true>(vb + chunk_at(16 * u + vrow, 2 * d + vchk), r);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816<false>(o[nt][d], r, pf[u][nt][0], pf[u][nt][1]);
              mma16816<false>(o[nt][d], r, pl[u][nt][0], pl[u][nt][1]);
            }
          }
        }
      }
      att_reads_done();
      __syncwarp();  // every lane has read the stage
      if (lane == 0 && !dead)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(att_smem(&empty[at])) : "memory");
      if (++stage == S) {
        stage = 0;
        full_ph ^= 1u;
      }
    }

    // The queries go back only once products have used them: handed back right
    // behind the loads, 16 heads of 256 of a one-tile item were still being read
    // when the next copy landed.
    att_reads_done();
    __syncwarp();
    if (lane == 0 && !dead)
      asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(att_smem(&q_empty[qb])) : "memory");

    // ---- the warps' parts meet: those of the segment's first tiles
    const int parts = team.solo ? 1 : min(kAttWarps, seg.count);
    if (turn < parts) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = l[nt][j];
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, w);
          const int h = 8 * nt + 2 * (lane & 3) + j;
          if (lane < 4) {
            s_ml[warp][h][0] = m[nt][j];
            s_ml[warp][h][1] = bad ? __int_as_float(0x7FC00000) : x;
          }
          float *to = red + (warp * C::kHeads + h) * C::kRedStride;
#pragma unroll
          for (int d = 0; d < KS; ++d) {
            // rows g and g + 8 of a 16-row tile: dimensions g, g + 8, or 2 g, 2 g + 1 (E4M3)
            const int d0 = 16 * d + (E4M3 ? 2 : 1) * (lane >> 2);
            to[d0] = o[nt][d][j];
            to[d0 + (E4M3 ? 1 : 8)] = o[nt][d][2 + j];
          }
        }
    }
    if (dead) s_fail = 1;
    if (team.solo) __syncwarp();
    else asm volatile("bar.sync 1, %0;" ::"n"(kAttConsumers) : "memory");
    const bool whole = seg.count == seg.total;
    // parts of an item: the first in its CTA's slot 2c + 1, the others in their CTAs' slots 2c
    const int64_t slot = 2 * c + (seg.off == 0 ? 1 : 0);
    const float vs = E4M3 && a.kv.v_scale ? __ldg(a.kv.v_scale + kh) : 1.0f;
    float2 *ml_all = reinterpret_cast<float2 *>(p.part + (int64_t)2 * gridDim.x * C::kHeads * D);
    for (int i = team.solo ? lane : tid; i < heads * (D / 8); i += team.solo ? 32 : kAttConsumers) {
      const int h = i / (D / 8), d = i % (D / 8) * 8;
      float mx = -INFINITY, sum = 0.0f, v[8] = {};
      for (int j = 0; j < parts; ++j) mx = fmaxf(mx, s_ml[(team.first + j) & (kAttWarps - 1)][h][0]);
      const float ref = mx == -INFINITY ? 0.0f : mx;
      for (int j = 0; j < parts; ++j) {
        const int w = (team.first + j) & (kAttWarps - 1);
        const float f = att_exp2(s_ml[w][h][0] - ref);
        sum += s_ml[w][h][1] * f;
        const float4 *x = reinterpret_cast<const float4 *>(red + (w * C::kHeads + h) * C::kRedStride + d);
        const float4 x0 = x[0], x1 = x[1];
        v[0] = fmaf(x0.x, f, v[0]), v[1] = fmaf(x0.y, f, v[1]), v[2] = fmaf(x0.z, f, v[2]), v[3] = fmaf(x0.w, f, v[3]);
        v[4] = fmaf(x1.x, f, v[4]), v[5] = fmaf(x1.y, f, v[5]), v[6] = fmaf(x1.z, f, v[6]), v[7] = fmaf(x1.w, f, v[7]);
      }
      if (whole) {
        const float r = sum == 0.0f ? 0.0f : vs / sum;
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack16<false>(v[2 * j] * r, v[2 * j + 1] * r);
        const int64_t row = (int64_t)seg.b * a.q_heads + h0 + h;
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + row * D + d) = make_uint4(w[0], w[1], w[2], w[3]);
        if (d == 0 && a.lse) a.lse[row] = att_lse<E4M3>(ref, sum);
      } else {
        float4 *to = reinterpret_cast<float4 *>(p.part + (slot * C::kHeads + h) * D + d);
        to[0] = make_float4(v[0], v[1], v[2], v[3]);
        to[1] = make_float4(v[4], v[5], v[6], v[7]);
        if (d == 0) ml_all[slot * C::kHeads + h] = make_float2(mx, sum);
      }
    }
    if (!whole && seg.off == 0) {  // this CTA holds the item's first part: the range's last segment
      shared.row = (int64_t)seg.b * a.q_heads + h0;
      shared.heads = heads;
      // (the unit of the item's last tile)
      shared.parts = split.cta_of(g1 - seg.left - seg.units - seg.unit + kAttItemCost + seg.total - 1) - c + 1;
    }
    if (!att_next<KT>(a, seg, groups, p.blocks)) break;
    // red and s_ml are free again
    if (team.solo) __syncwarp();
    else asm volatile("bar.sync 1, %0;" ::"n"(kAttConsumers) : "memory");
  }
  if (tid == 0) p.shared[c] = shared;
  __syncthreads();
}

// Adds the parts of the items that several CTAs share, in a fixed order; block
// c has the one that begins in CTA c, if any.  Rows of D / 4 threads: row r
// takes parts r / heads, + PG, ... of head r % heads, four in flight, and the
// PG rows of a head meet in shared memory.
template <bool E4M3, int THREADS>
__global__ void __launch_bounds__(THREADS) k_attend_join(const __grid_constant__ AttLaunch p, int D, int heads, int grid) {
  __shared__ float4 s_v[THREADS];
  __shared__ float2 s_ml[THREADS];
  pdl_wait();
  const int c = blockIdx.x;
  const AttShared it = p.shared[c];
  if (it.parts == 0) return;
  const AttendArgs &a = p.a;
  const float2 *ml = reinterpret_cast<const float2 *>(p.part + (int64_t)2 * grid * heads * D);
  const int d4 = D / 4, rows = THREADS / d4, row = threadIdx.x / d4, d = threadIdx.x % d4 * 4;
  const int step = min(rows, it.heads), pg = min(rows / step, it.parts);  // heads at a time, rows per head
  const int kh = (int)(it.row % a.q_heads) / (a.q_heads / a.kv.kv_heads);
  const float vs = E4M3 && a.kv.v_scale ? __ldg(a.kv.v_scale + kh) : 1.0f;
  for (int h0 = 0; h0 < it.heads; h0 += step) {
    const int h = h0 + row % step, first = row / step;
    const bool on = h < it.heads && first < pg;
    float mx = -INFINITY, sum = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int j0 = first; on && j0 < it.parts; j0 += 4 * pg) {
      float2 e[4];
      float4 x[4];
      float top = mx;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int part = j0 + j * pg < it.parts ? j0 + j * pg : first;
        const int64_t s = (int64_t)(2 * (c + part) + (part == 0 ? 1 : 0)) * heads + h;
        e[j] = ml[s];
        x[j] = *reinterpret_cast<const float4 *>(p.part + s * D + d);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j0 + j * pg >= it.parts) e[j] = make_float2(-INFINITY, 0.0f);
        top = fmaxf(top, e[j].x);
      }
      const float ref = top == -INFINITY ? 0.0f : top, f0 = att_exp2(mx - ref);
      sum *= f0, v.x *= f0, v.y *= f0, v.z *= f0, v.w *= f0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j0 + j * pg < it.parts) {
          const float f = att_exp2(e[j].x - ref);
          sum = fmaf(e[j].y, f, sum);
          v.x = fmaf(x[j].x, f, v.x), v.y = fmaf(x[j].y, f, v.y), v.z = fmaf(x[j].z, f, v.z), v.w = fmaf(x[j].w, f, v.w);
        }
      mx = top;
    }
    s_v[threadIdx.x] = v;
    s_ml[threadIdx.x] = make_float2(mx, sum);
    __syncthreads();
    if (on && first == 0) {
      for (int g = 1; g < pg; ++g) mx = fmaxf(mx, s_ml[threadIdx.x + g * step * d4].x);
      const float ref = mx == -INFINITY ? 0.0f : mx;
      sum = 0.0f;
      v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int g = 0; g < pg; ++g) {
        const float2 e = s_ml[threadIdx.x + g * step * d4];
        const float4 x = s_v[threadIdx.x + g * step * d4];
        const float f = att_exp2(e.x - ref);
        sum = fmaf(e.y, f, sum);
        v.x = fmaf(x.x, f, v.x), v.y = fmaf(x.y, f, v.y), v.z = fmaf(x.z, f, v.z), v.w = fmaf(x.w, f, v.w);
      }
      const float r = sum == 0.0f ? 0.0f : vs / sum;
      const int64_t at = it.row + h;
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at * D + d) =
          make_uint2(pack16<false>(v.x * r, v.y * r), pack16<false>(v.z * r, v.w * r));
      if (d == 0 && a.lse) a.lse[at] = att_lse<E4M3>(ref, sum);
    }
    __syncthreads();
  }
}

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_att_encode = nullptr;

// NT of a launch: the smallest block of 8 NT heads that holds the group; larger
// groups take the largest block that the registers hold and read the cache
// once per block.
int att_nt(int head_dim, int group) {
  const int most = head_dim == 256 ? 2 : 4;
  return group <= 8 ? 1 : group <= 16 || most == 2 ? 2 : 4;
}

template <int D, bool E4M3, int NT>
int att_ctas_per_sm() {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_attend<D, E4M3, NT>, AttCfg<D, E4M3, NT>::kThreads,
                                                    AttCfg<D, E4M3, NT>::kSmem) != cudaSuccess || n < 1)
    n = 1;
  return n;
}

// Calls f<D, E4M3, NT>() for the runtime values.
template <typename F>
auto att_dispatch(int head_dim, bool e4m3, int nt, F &&f) {
#define NVFP4_ATT(D, N) (e4m3 ? f.template operator()<D, true, N>() : f.template operator()<D, false, N>())
  if (head_dim == 64) return nt == 1 ? NVFP4_ATT(64, 1) : nt == 2 ? NVFP4_ATT(64, 2) : NVFP4_ATT(64, 4);
  if (head_dim == 128) return nt == 1 ? NVFP4_ATT(128, 1) : nt == 2 ? NVFP4_ATT(128, 2) : NVFP4_ATT(128, 4);
  return nt == 1 ? NVFP4_ATT(256, 1) : NVFP4_ATT(256, 2);
#undef NVFP4_ATT
}

struct AttGrid {
  int sms;
  template <int D, bool E4M3, int NT>
  int operator()() const {
    static const int per_sm = att_ctas_per_sm<D, E4M3, NT>();
    return std::min(kAttMaxCtas, sms * per_sm);
  }
};

struct AttPrepare {
  template <int D, bool E4M3, int NT>
  cudaError_t operator()() const {
    return cudaFuncSetAttribute(k_attend<D, E4M3, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)AttCfg<D, E4M3, NT>::kSmem);
  }
};

struct AttRun {
  const AttendArgs &a;
  int grid_max, nt;
  void *ws;
  cudaStream_t st;
  template <int D, bool E4M3, int NT>
  cudaError_t operator()() const {
    using C = AttCfg<D, E4M3, NT>;
    AttLaunch p;
    p.a = a;
    const int group = a.q_heads / a.kv.kv_heads, page = 1 << a.kv.page_shift, piece = std::min(page, C::KT);
    p.blocks = (group + C::kHeads - 1) / C::kHeads;
    p.piece_shift = 0;
    while ((1 << p.piece_shift) < piece) ++p.piece_shift;
    // The units of the longest possible lengths bound the grid; so it never limits
    // the kernel's G, and the order of the additions does not depend on the table's width.
    const int64_t cap = a.kv.table_width << a.kv.page_shift;
    const int64_t seen = a.window > 0 ? std::min<int64_t>(cap, std::min<int64_t>(a.window, cap) + C::KT) : cap;
    const int64_t items = (int64_t)a.sequences * a.kv.kv_heads * p.blocks, units = (seen / C::KT + 1 + kAttItemCost) * items;
    const int grid = (int)std::min<int64_t>(grid_max, (units + kAttMinTiles - 1) / kAttMinTiles);
    p.shared = static_cast<AttShared *>(ws);
    p.part = reinterpret_cast<float *>(static_cast<char *>(ws) + kAttMaxCtas * sizeof(AttShared));
    CUtensorMap m[2];
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.kv.kv_heads << a.kv.page_shift, (cuuint64_t)a.kv.pages};
    const cuuint32_t box[3] = {(cuuint32_t)(C::kBoxRow / C::kElem), (cuuint32_t)piece, 1u}, es[3] = {1u, 1u, 1u};
    for (int i = 0; i < 2; ++i) {
      const cuuint64_t strides[2] = {(cuuint64_t)C::kRow,
                                     (cuuint64_t)(i ? a.kv.v_page_stride : a.kv.k_page_stride) * C::kElem};
      if (g_att_encode(&m[i], E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                       i ? a.kv.v : a.kv.k, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       C::kBoxRow == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    }
    k_attend<D, E4M3, NT><<<grid, C::kThreads, C::kSmem, st>>>(m[0], m[1], p);
    const cudaError_t e = cudaGetLastError();
    // the parts of split items; one CTA splits none
    if (e != cudaSuccess || grid == 1) return e;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    // Small blocks fit beside the attention's CTAs and start at once; where
    // items are cut into many parts, large ones share the parts of a head
    // (1 x 8192 tokens, 38 parts: 6 us with 256 threads, 4.5 with 1024).  They
    // add in different orders: the choice goes by the device and the number of items.
    const bool many = grid_max > 8 * items;
    cfg.blockDim = dim3(many ? 1024 : 256);
    return cudaLaunchKernelEx(&cfg, many ? k_attend_join<E4M3, 1024> : k_attend_join<E4M3, 256>, p, D, C::kHeads, grid);
  }
};

}  // namespace

size_t attend_workspace_bytes(const KvArgs &kv, int q_heads, int sms) {
  const int nt = att_nt(kv.head_dim, q_heads / kv.kv_heads);
  const size_t grid = (size_t)att_dispatch(kv.head_dim, kv.e4m3, nt, AttGrid{sms});
  return kAttMaxCtas * sizeof(AttShared) + 2 * grid * 8 * nt * (kv.head_dim + 2) * sizeof(float);
}

cudaError_t launch_attend(const AttendArgs &a, int sms, void *ws, cudaStream_t st) {
  if (!g_att_encode) return cudaErrorInitializationError;
  const int nt = att_nt(a.kv.head_dim, a.q_heads / a.kv.kv_heads);
  const int grid = att_dispatch(a.kv.head_dim, a.kv.e4m3, nt, AttGrid{sms});
  return att_dispatch(a.kv.head_dim, a.kv.e4m3, nt, AttRun{a, grid, nt, ws, st});
}

cudaError_t prepare_attention_kernels() {
  void *fn = nullptr;
  cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
  cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
  if (e != cudaSuccess) return e;
  if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorSymbolNotFound;
  g_att_encode = reinterpret_cast<EncodeTiledFn>(fn);
  for (const int dim : {64, 128, 256})
    for (const bool e4m3 : {false, true})
      for (const int nt : {1, 2, 4})
        if (e == cudaSuccess && !(dim == 256 && nt == 4)) e = att_dispatch(dim, e4m3, nt, AttPrepare{});
  return e;
}

}  // namespace nvfp4
