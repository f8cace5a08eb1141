// nvfp4_moe.cu -- the experts' products of a mixture-of-experts layer for a few
// tokens, on NVFP4 weights:
//   h[t,s] = act(alpha_g sum_c q Delta x[t][c]) * (alpha_u sum_c q Delta x[t][c]),  expert ids[t][s]
//   y[t]   = bf16( residual[t] + sum_s weights[t][s] alpha_d sum_j q Delta h[t,s][j] ).
//
// Floor: reading once the weights of every expert that some token names
// (0.5625 B each); a token's share of x, h and y is small beside them.  Measured
// with cold weights, and those weights' bytes over the time (a copy reads and writes
// 6.77 TB/s):
//   33 tokens 7168 x 2048, 8 of 256  612 to 646 us   5.7 to 6.0 TB/s (by the box)
//    5 tokens 4096 x 14336, 2 of 8        105      4.7
//   61 tokens 2048 x 768, 8 of 128         79      3.8
//   256 tokens 2064 x 1424, 6 of 60       164      1.2  (no gate; 26 pairs an expert, 110 TFLOP/s)
//    1 token 2048 x 768, 8 of 128          17      1.2
// What the largest leaves is the plan, the first fetches (4 to 6 us a launch) and
// CTAs that end apart (5 to 10); with less work those weigh more, with many pairs an
// expert the MMAs of their n-tiles and their vectors' way into shared memory.
//
// An expert's weights are gone over once for each of its jobs, and a job's pairs are
// limited by its vectors, which lie whole in shared memory: 32 up to about 1500 columns,
// 24 to 29 at 2048, 13 to 16 at 4096, 7 to 9 at 7168, 3 to 5 at 14336.  So many pairs on wide
// experts fetch, form and multiply the same weights again (in brackets how many times):
//   4096 x 14336, 2 of 8:  5 tokens 107 us (1.07 times)    16 tokens 214 (1.2)
//                          33       292    (1.9)           64        478 (2.9)    256  1645 (10.3)
//   256 tokens 7168 x 2048, 8 of 256: 2046 us (1.4); 4096 x 2048, 6 of 64: 477 (2.0)
//
// Three launches, each waiting for the one before through a programmatic
// dependency: gate and up with the activation (h, f16 with a power of two for each
// 8 entries, to the workspace), down (each slot's product, fp32, to the workspace),
// and the sum over a token's slots in slot order.  No atomics take part in a sum and
// no CTA waits for another, so a workspace may hold anything and results repeat bit
// for bit.
//
// Jobs: every CTA sorts the call's (token, slot) pairs by expert in shared
// memory; an expert with n pairs makes ceil(n / N) jobs of up to N pairs.  The
// row tiles of all jobs, job after job, are cut by measured costs into one
// contiguous range per CTA (two of 8 warps on an SM, or one of 16 where the vectors
// leave no room for two), and the units (16 rows by 256 columns) of a range's part of
// one job into contiguous runs, one per warp.  A warp that does a whole tile finishes it
// from its registers; sums of a tile cut between warps meet in shared memory, in
// warp order.  Codes come by asynchronous copies, kMoeDepth units ahead, across
// tiles and jobs.
//
// Products: mma.sync m16n8k16 (f16 x f16 -> fp32), 16 rows of W by 8 pairs.
// q * Delta is formed in registers, exactly: six significant bits between 2^-10
// and 2688.  The vectors go to f16 in shared memory, each scaled by a power of
// two that puts its largest entry into [2^14, 2^15): x keeps its 8 bits down to
// 2^-31 of its largest entry.  h is rounded to f16's 11 bits, which loses an
// eighth of what bf16 would, under a scale for each 8 entries (a whole vector's is
// not known before all of them are), and then brought to one scale, exactly down
// to 2^-29 of its largest entry.  With a gate the 16 rows are 8 of the gate's
// and the 8 of up's that they multiply, so that h is formed in registers.
#include <algorithm>
#include <climits>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"
#include "nvfp4_epilogue.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {

constexpr int kMoeDepth = 2;            // units of 256 columns in flight per warp (3: 650 -> 764 us on the
                                        // largest case, the rows' lines come less often from an open DRAM page)
constexpr int kMoeMaxWarps = 16;        // of a CTA
constexpr int kMoeSmem = 226 * 1024;    // dynamic shared memory of a CTA that has an SM to itself
constexpr int kMoeHalfSmem = 112 * 1024;  // of one of two
constexpr int kMoeFewPairs = 32;        // a warp sorts so many by itself

struct MoeLaunch {
  MoeArgs a;
  __half *h;          // [pairs][inner], each 8 entries times a power of two
  int8_t *h_up;       // [pairs][up_pitch]: its exponent
  float *part;        // [pairs][hidden]
  int up_pitch;       // inner / 8, rounded up to 16
  int pairs;          // tokens * top_k
  int group;          // pairs of a job at most
  int steps;          // of 256 columns
  int tiles;          // of a job
  int job_cost;       // of a job besides its tiles and vectors
  int more_cost;      // of a tile for each further n-tile, in eighths of a tile's
  uint32_t share;     // of the cost, of a CTA: 2^32 / CTAs
  int64_t cols;       // of this launch's matrices
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The power of two (its exponent) that brings a largest magnitude of these bits
// into [2^14, 2^15), or up to 2^126; for an infinity or a NaN one that leaves it what it is.
// (2^126 is enough: it brings bf16's smallest, 2^-133, to 2^-7, which f16 holds with all of
// bf16's bits, and half of f16's last step, 2^-25, back to 2^-151, below fp32's own 2^-150.)
__device__ __forceinline__ int f16_up(unsigned top) { return min(14 + 127 - (int)(top >> 23), 126); }

// How a unit's codes and scales reach shared memory, by what their rows' addresses allow:
//   kWide   rows of codes are whole multiples of 16 bytes and of scales of 4, and so
//           aligned: 16 bytes and a word at a time;
//   kOdd    a tile's codes begin on 16 bytes, but its odd rows perhaps 8 behind: each
//           row's 16-byte pieces from the last such boundary before it, nine instead
//           of eight; scales on any byte, in the two words that hold a lane's four;
//   kAny    codes on any 8 bytes: 8 at a time, which takes 1.7 times as long as kOdd.
enum MoeLoads { kWide = 0, kOdd = 1, kAny = 2 };
__host__ __device__ constexpr int moe_code_slot(int loads) { return loads == kOdd ? 16 * 144 : 16 * 128; }
__host__ __device__ constexpr int moe_slot(int loads) { return moe_code_slot(loads) + (loads == kWide ? 256 : 512); }
__host__ __device__ constexpr int moe_up_pitch(int64_t cols) { return (int)((cols / 8 + 15) / 16 * 16); }
// Shared memory: the vectors (with h's exponents), the warps' units in flight
// and partial sums, the vectors' scales, the plan.
__host__ __device__ constexpr int64_t moe_smem(int group, int64_t cols, bool down, int warps, int loads, int experts, int pairs) {
  return (cols + 255) / 256 * 512 * (group | 1) + (down ? (int64_t)group * moe_up_pitch(cols) : 0) +
         (int64_t)warps * (kMoeDepth * moe_slot(loads) + (group + 7) / 8 * 512) + 512 +
         (pairs > kMoeFewPairs ? (int64_t)experts * 8 : 0) + ((int64_t)pairs + 1) * 14 + 64;
}

// A job: an expert's pairs order[at .. at + n).
__device__ __forceinline__ uint32_t moe_job(int expert, int at, int n) { return (uint32_t)expert << 17 | (uint32_t)at << 6 | (uint32_t)n; }
static_assert(kMaxExperts <= 1024 && kMoeSlicePairs <= 2048, "a job's fields");
// A tile's cost: its weights' way, and a part of that for each further n-tile of pairs.
// Measured: 61 tokens 2048 x 768, 8 of 128 (kWide): a tile of 9 .. 16 pairs took
// 1.44 times one of up to 8; 256 tokens 2064 x 1424, 6 of 60 (rows on 8 bytes): 1.2, and
// 1.4 with a third n-tile.  (Weighing the pairs within an n-tile too made 33 tokens
// 7168 x 2048, 8 of 256 slower, 645 -> 652 us.)
__device__ __forceinline__ int moe_tile_cost(const MoeLaunch &p, int pairs) { return 8 + p.more_cost * ((pairs - 1) / 8); }
// A job's besides its tiles: a vector's way into shared memory takes about a third of a
// tile's time (256 tokens 2064 x 1424, 6 of 60: a weight of 0 181 us, 3 176, 5 178).
__device__ __forceinline__ int moe_begin_cost(const MoeLaunch &p, int pairs) { return p.job_cost + 3 * pairs; }
__device__ __forceinline__ int moe_job_cost(const MoeLaunch &p, int pairs) { return moe_begin_cost(p, pairs) + p.tiles * moe_tile_cost(p, pairs); }

// The plan: the pairs that have an expert by expert, ascending, so that every
// CTA cuts an expert's into the same jobs; the jobs, and the cost of those
// before each.
struct MoePlan {
  uint32_t *jobs;   // [pairs]
  int *start;       // [pairs + 1]
  uint16_t *order;  // [pairs]
  int *count, *end; // [experts]: pairs of an expert, and where they end (unused with few pairs)
  uint16_t *named;  // [pairs]: their experts
  uint16_t *found;  // [pairs]: by expert, as they came (where that is not yet the order)
  int *total;       // jobs
};

// By one warp, one pair per lane.
__device__ void moe_plan_few(const MoeLaunch &p, const MoePlan &o, int lane) {
  const int N = p.group;
  const int id = lane < p.pairs ? p.a.ids[lane] : -1;
  const bool there = id >= 0 && id < p.a.experts;
  const int e = there ? id : INT_MAX;
  const uint32_t same = __match_any_sync(~0u, e), before = same & ((1u << lane) - 1u);
  const int pos = __popc(before), n = min(N, __popc(same) - pos);  // pairs from here to the job's end, at a job's first
  const bool first = there && pos % N == 0;
  const int cost = first ? moe_job_cost(p, n) : 0;
  int rank = 0, job = 0, start = 0;
#pragma unroll 4
  for (int l = 0; l < p.pairs; ++l) {
    const int el = __shfl_sync(~0u, e, l), cl = __shfl_sync(~0u, cost, l);
    if (el < e || (el == e && l < lane)) ++rank, job += cl > 0, start += cl;
  }
  if (there) o.order[rank] = (uint16_t)lane;
  if (first) {
    o.jobs[job] = moe_job(e, rank, n);
    o.start[job] = start;
  }
  const int total = __popc(__ballot_sync(~0u, first)), all = __reduce_add_sync(~0u, cost);
  if (lane == 0) o.start[total] = all, *o.total = total;
}

// By the whole CTA.
__device__ void moe_plan(const MoeLaunch &p, const MoePlan &o, int tid, int threads, int (*scan)[kMoeMaxWarps]) {
  const int N = p.group, E = p.a.experts, warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e < E; e += threads) o.count[e] = 0;
  __syncthreads();
  for (int i = tid; i < p.pairs; i += threads) {
    const int e = p.a.ids[i];
    const bool there = e >= 0 && e < E;
    o.named[i] = there ? (uint16_t)e : (uint16_t)0xFFFFu;
    if (there) atomicAdd(&o.count[e], 1);
  }
  __syncthreads();
  int total = 0, named = 0, cost = 0;  // jobs; pairs that have an expert; the jobs' cost
  bool many = false;                   // an expert of this thread has several jobs
  for (int e0 = 0; e0 < E; e0 += threads) {
    const int e = e0 + tid, n = e < E ? o.count[e] : 0, j = (n + N - 1) / N;
    many |= j > 1;
    const int full = moe_job_cost(p, N), c = j > 0 ? (j - 1) * full + moe_job_cost(p, n - (j - 1) * N) : 0;
    int sn = n, sj = j, sc = c;  // inclusive sums over the warp, then over the warps
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int un = __shfl_up_sync(~0u, sn, d), uj = __shfl_up_sync(~0u, sj, d), uc = __shfl_up_sync(~0u, sc, d);
      if (lane >= d) sn += un, sj += uj, sc += uc;
    }
    if (lane == 31) scan[0][warp] = sn, scan[1][warp] = sj, scan[2][warp] = sc;
    __syncthreads();
    int bn = named + sn - n, bj = total + sj - j, bc = cost + sc - c;
    for (int w = 0; w < threads / 32; ++w) {
      const int wn = scan[0][w], wj = scan[1][w], wc = scan[2][w];
      if (w < warp) bn += wn, bj += wj, bc += wc;
      named += wn, total += wj, cost += wc;
    }
    if (e < E) {
      o.end[e] = bn;  // (its first pair, until they are found)
      for (int i = 0; i < j; ++i) {
        o.jobs[bj + i] = moe_job(e, bn + i * N, min(N, n - i * N));
        o.start[bj + i] = bc + i * full;
      }
    }
    __syncthreads();
  }
  if (tid == 0) o.start[total] = cost, *o.total = total;
  // (in an expert's only job a pair's place just decides which column of an MMA it takes)
  const bool several = __syncthreads_or(many);
  uint16_t *to = several ? o.found : o.order;
  for (int i = tid; i < p.pairs; i += threads) {
    const int e = o.named[i];
    if (e != 0xFFFF) to[atomicAdd(&o.end[e], 1)] = (uint16_t)i;
  }
  if (!several) return;
  __syncthreads();
  for (int q = tid; q < named; q += threads) {
    const int i = o.found[q], e = o.named[i], n = o.count[e], b = o.end[e] - n;
    int at = q;
    if (n > N) {
      at = b;
      for (int f = b; f < b + n; ++f) at += o.found[f] < i;
    }
    o.order[at] = (uint16_t)i;
  }
}

// DOWN: the second product (h -> part), else the first (x -> h).  GATED: the
// first product's tiles hold 8 rows of gate and 8 of up.  LOADS: MoeLoads.  NT:
// n-tiles that the group's pairs fill at most.
template <int NT, bool DOWN, bool GATED, int LOADS>
__global__ void __launch_bounds__(kMoeMaxWarps * 32, 1) k_moe(const __grid_constant__ MoeLaunch p) {
  // Rows of codes lie in whole 128-byte lines of shared memory: where they lay across
  // two, each copy took four times the requests to L2 and 2.5 times the sectors.
  extern __shared__ __align__(128) uint4 dsm[];
  __shared__ int scan[3][kMoeMaxWarps], jobs_there, bound[2][2];
  const MoeArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cq = lane & 3;
  const int threads = blockDim.x, warps = threads >> 5, warps_bits = 31 - __clz(warps);  // (8 or 16)
  const int nk = p.steps, N = p.group, NB = (N + 7) / 8, P = N | 1;  // P: vectors' places (odd, see `chunks`)
  constexpr bool WIDE = LOADS == kWide;
  constexpr int kSlot = moe_slot(LOADS), kScales = moe_code_slot(LOADS);  // of a slot: its bytes, where its scales begin
  uint4 *xs = dsm;                                                        // [nk][8][P][4] 16-byte units of f16
  uint4 *slots = dsm + (size_t)nk * 32 * P;                               // [warps][depth][kSlot / 16]: units in flight
  float4 *own = reinterpret_cast<float4 *>(slots + warps * kMoeDepth * (kSlot / 16));  // [warps][NB][32]
  slots += warp * kMoeDepth * (kSlot / 16);
  int8_t *ups = reinterpret_cast<int8_t *>(own + warps * NB * 32);        // [N][up_pitch]
  float *xdown = reinterpret_cast<float *>(ups + (DOWN ? N * p.up_pitch : 0));  // [2][32]: the vectors' scales, undone
  int *xtop = reinterpret_cast<int *>(xdown + 64);                        // [2][32]: their largest entries' bits, or their scales' exponents
  MoePlan o;
  o.start = xtop + 64;
  o.jobs = reinterpret_cast<uint32_t *>(o.start + p.pairs + 1);
  o.count = reinterpret_cast<int *>(o.jobs + p.pairs);
  o.end = o.count + (p.pairs > kMoeFewPairs ? a.experts : 0);
  o.order = reinterpret_cast<uint16_t *>(o.end + (p.pairs > kMoeFewPairs ? a.experts : 0));
  o.named = o.order + p.pairs;
  o.found = o.named + p.pairs;
  o.total = &jobs_there;

  // The second product waits for the first only where it needs h: ids and
  // weights were there before the first began, since that lets the second start
  // after its own wait only.
  if constexpr (!DOWN) {
    pdl_wait();
    pdl_launch_dependents();
  }
  if (tid < 64) xtop[tid] = DOWN ? INT_MAX : INT_MIN;
  if (p.pairs <= kMoeFewPairs) {
    if (warp == 0) moe_plan_few(p, o, lane);
  } else {
    moe_plan(p, o, tid, threads, scan);
  }
  __syncthreads();

  // ---- this CTA's tiles: the job and the tile at two places of the total cost
  const int total = jobs_there, cost = o.start[total];
  {
    // (p.share: 2^32 / CTAs)
    const uint32_t at0 = __umulhi(blockIdx.x * p.share, (uint32_t)cost),
                   at1 = blockIdx.x + 1 == gridDim.x ? (uint32_t)cost : __umulhi((blockIdx.x + 1) * p.share, (uint32_t)cost);
    for (int j = tid; j <= total; j += threads) {  // one j holds each place
      const uint32_t from = (uint32_t)o.start[j], to = j < total ? (uint32_t)o.start[j + 1] : ~0u;
      const int np = (int)(o.jobs[max(min(j, total - 1), 0)] & 63u), begin = moe_begin_cost(p, np), c = moe_tile_cost(p, np);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t at = i ? at1 : at0;
        if (from <= at && at < to) bound[i][0] = j, bound[i][1] = j < total ? max((int)(at - from) - begin, 0) / c : 0;
      }
    }
    __syncthreads();
  }
  int j0 = bound[0][0], t0 = bound[0][1], j1 = bound[1][0], t1 = bound[1][1];
  if (j0 == j1 && t0 == t1) {
    if constexpr (DOWN) {
      pdl_wait();
      pdl_launch_dependents();
    }
    return;
  }
  if (t1 == 0) --j1, t1 = p.tiles;

  // ---- this warp's units: its run of the range's part of each job
  struct Run {
    int t0, u0, u1;  // the part's first tile; the warp's units, counted from there
  };
  auto run_of = [&](int j, int w) {
    const int from = j == j0 ? t0 : 0, units = ((j == j1 ? t1 : p.tiles) - from) * nk;
    return Run{from, w * units >> warps_bits, (w + 1) * units >> warps_bits};
  };
  // Units go to the ring kMoeDepth ahead.  Codes: 16 rows of 128 bytes, the 16-byte
  // chunk c of row r at place c ^ (r % 8), so that both the copies (full rows) and
  // the reads (two chunks of each of eight rows at once) spread over the banks.
  // A lane takes 64 columns (four blocks) of rows g and g + 8; it copies their
  // scales itself, a word each, or (where a row need not begin on a word) the two
  // words that hold them.
  const int64_t nblk = p.cols / 16, pitch = 8 * nblk;     // blocks and code bytes of a row
  constexpr int kTileRows = GATED && !DOWN ? 8 : 16;      // rows between tiles
  constexpr int kPiece = LOADS == kAny ? 8 : 16, kRows = 4 * kPiece / 16, kCopies = 16 / kRows;  // of a copy by the warp
  const int row0 = lane / (32 / kRows), byte0 = lane % (32 / kRows) * kPiece;
  // bytes of the last step's piece and scales (past the end come zeros, from no address)
  const int code_tail = max(0, min(kPiece, (int)(pitch - (int64_t)(nk - 1) * 128) - byte0));
  const int scale_tail = max(0, min(4, (int)(nblk - (int64_t)(nk - 1) * 16) - 4 * cq));
  const uint32_t slot_at = static_cast<uint32_t>(__cvta_generic_to_shared(slots)), scale_to = slot_at + kScales + lane * 4;
  // the lane's place in rows 0 .. 7: copies 0 and 1 of the wide form's two
  const uint32_t code_to0 = slot_at + row0 * 128 + (((byte0 >> 4) ^ row0) << 4) + (byte0 & 15),
                 code_to1 = slot_at + (row0 + 4) * 128 + (((byte0 >> 4) ^ (row0 + 4)) << 4);
  // kOdd: piece i of the lane is 16 bytes of row odd_row(i) from `odd_from`, of which
  // 8 may belong to the row before; `back`: how far behind a boundary odd rows begin
  const int back = LOADS == kOdd && (pitch & 8) ? 8 : 0;
  auto odd_row = [&](int i) { return (i * 32 + lane) / 9; };
  auto odd_chunk = [&](int i) { return (i * 32 + lane) % 9; };
  struct {
    int j, k, left;     // the next unit's job and step; units left of the run
    uint32_t at;        // its scales' offset in the matrix (and an eighth of its codes')
    const uint8_t *code[2], *scale[2];  // this lane's rows 0 and 8 of the matrix
  } next = {j0 - 1, 0, 0, 0u, {nullptr, nullptr}, {nullptr, nullptr}};
  const uint32_t rows4 = (uint32_t)(kRows * pitch), wrap = (uint32_t)(kTileRows * nblk - (int64_t)(nk - 1) * 16);
  auto open_run = [&]() {  // the next unit's rows, in the next job with units for this warp
    while (next.left == 0 && next.j < j1) {
      const Run r = run_of(++next.j, warp);
      next.left = r.u1 - r.u0;
      const int e = (int)(o.jobs[next.j] >> 17), t = r.u0 / nk;
      next.k = r.u0 - t * nk;
      next.at = (uint32_t)((r.t0 + t) * kTileRows * nblk) + 16 * next.k;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const MoeMatrix &m = DOWN ? a.down : GATED && h == 0 ? a.gate : a.up;
        const int64_t row = GATED && !DOWN ? 0 : 8 * h;
        next.code[h] = m.codes + e * m.code_stride + (LOADS == kOdd ? row * pitch : (row + row0) * pitch + byte0);
        next.scale[h] = m.scales + e * m.scale_stride + (row + g) * nblk + 4 * cq;
      }
    }
  };
  uint32_t fill = 0;  // the ring's place for the next unit
  auto fetch = [&]() {
    if (next.left == 0) open_run();
    if (next.left > 0) {
      const bool last = next.k == nk - 1;
      const int sb = last ? scale_tail : 4;
      if constexpr (LOADS == kOdd) {
        const int row_left = last ? (int)(pitch - (int64_t)(nk - 1) * 128) : 128;  // bytes of a row from here
#pragma unroll
        for (int i = 0; i < 5; ++i) {
          const int r = odd_row(i), from = odd_chunk(i) * 16 - (r & 1 ? back : 0);  // counted from the row's place here
          if (i < 4 || r < 16) {
            // (pieces that begin past the row's end are zeros; one that reaches past it takes in the next row's
            // bytes, which there are: such a row is an even one)
            const int bytes = from < row_left ? 16 : 0;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                         ::"r"(slot_at + r * 144 + odd_chunk(i) * 16 + fill),
                           "l"((r >= 8 ? next.code[1] : next.code[0]) + (int64_t)next.at * 8 + (r & 7) * (int)pitch + from), "r"(bytes) : "memory");
          }
        }
      } else {
        const int cb = last ? code_tail : kPiece;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          const uint8_t *from = next.code[i / (kCopies / 2)] + (uint64_t)next.at * 8 + (i % (kCopies / 2)) * rows4;
          if (WIDE) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                         ::"r"((i & 1 ? code_to1 : code_to0) + (i >> 1) * 1024 + fill), "l"(from), "r"(cb) : "memory");
          } else {
            const int r = i * kRows + row0;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;"
                         ::"r"(slot_at + r * 128 + (((byte0 >> 4) ^ (r & 7)) << 4) + (byte0 & 15) + fill), "l"(from), "r"(cb) : "memory");
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t *from = next.scale[h] + next.at;
        if (WIDE) {
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(scale_to + h * 128 + fill), "l"(from), "r"(sb) : "memory");
        } else {
          const int off = (int)(reinterpret_cast<uintptr_t>(from) & 3u), end = sb ? off + sb : 0;  // bytes of the two words
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(scale_to + h * 256 + fill), "l"(from - off), "r"(min(end, 4)) : "memory");
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                       ::"r"(scale_to + h * 256 + 128 + fill), "l"(from - off + 4), "r"(max(end - 4, 0)) : "memory");
        }
      }
      --next.left;
      next.k = last ? 0 : next.k + 1;
      next.at += last ? wrap : 16;
    }
    fill = fill == (kMoeDepth - 1) * kSlot ? 0 : fill + kSlot;
    asm volatile("cp.async.commit_group;" ::: "memory");  // (one per unit, empty after the last, for the waits to count)
  };
  // A job's vectors into shared memory, 8 columns (a unit) at a time: copies of
  // what lies in memory, bf16 or f16 of eighths, to their places.
  const int wide = (int)(p.cols / 8);  // units of a vector (nk * 32 with those past the end)
  // unit u: step u / 32, lane quarter (u / 8) % 4, pair of k-steps u % 8
  auto unit_at = [&](int n, int u) { return xs + (((u >> 5) * 8 + (u & 7)) * P + n) * 4 + ((u >> 3) & 3); };
  // This warp's chunks of 32 units of `count` vectors: (vector, the lane's unit).  Eight
  // lanes in a row have two pairs of k-steps of four lane quarters: with P odd their places are
  // in different banks (in the order of u, eight met in one: 5 tokens 4096 x 14336, 2 of 8,
  // took 122 us instead of 105).
  auto chunks = [&](int count, auto f) {
    int n = warp / nk, c = warp - n * nk;
    while (n < count) {
      f(n, c * 32 + ((lane & 3) << 3 | lane >> 2));
      c += warps;
      while (c >= nk) c -= nk, ++n;
    }
  };
  auto take_in = [&](uint32_t job) {
    const int np = (int)(job & 63u);
    const uint16_t *pair = o.order + (job >> 6 & 2047u);
    if constexpr (DOWN) {
      const int pieces = p.up_pitch / 16;
      for (int i = tid; i < np * pieces; i += threads) {
        const int n = i / pieces, q = i - n * pieces;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                     ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(ups + n * p.up_pitch + 16 * q))),
                     "l"(p.h_up + (int64_t)pair[n] * p.up_pitch + 16 * q) : "memory");
      }
    }
    chunks(np, [&](int n, int u) {
      const int from = pair[n];
      const void *v = DOWN ? (const void *)(p.h + (int64_t)from * p.cols)
                           : (const void *)(static_cast<const __nv_bfloat16 *>(a.x) + (int64_t)(from / a.top_k) * a.x_stride);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                   ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(unit_at(n, u)))),
                   "l"(static_cast<const uint4 *>(v) + (u < wide ? u : 0)), "r"(u < wide ? 16 : 0) : "memory");
    });
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // (x before the weights, which take longer; h is not there yet)
  if constexpr (!DOWN) take_in(o.jobs[j0]);
#pragma unroll 1
  for (int i = 0; i < kMoeDepth; ++i) fetch();
  if constexpr (DOWN) {
    pdl_wait();
    pdl_launch_dependents();
  }

  // ---- the jobs.  xtop and xdown alternate between two places: a warp may
  // still finish a job's sums while others take in the next one's vectors.
  int par = 0, take = 0;  // take: the ring's place of the next unit
  for (int j = j0; j <= j1; ++j, par ^= 1) {
    const int e = (int)(o.jobs[j] >> 17), np = (int)(o.jobs[j] & 63u);
    const uint16_t *pair = o.order + (o.jobs[j] >> 6 & 2047u);

    // the vectors; the scale of each; and, in place, f16 of that scale
    if (DOWN || j > j0) {
      take_in(o.jobs[j]);
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group %0;" ::"n"(kMoeDepth) : "memory");
    }
    if constexpr (DOWN) {  // (a thread reads what it copied itself, here and below)
      const int pieces = p.up_pitch / 16;
      for (int i = tid; i < np * pieces; i += threads) {
        const int n = i / pieces, q = i - n * pieces;
        const uint4 r = *reinterpret_cast<const uint4 *>(ups + n * p.up_pitch + 16 * q);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        uint32_t low = 0x7F7F7F7Fu;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int valid = wide - 16 * q - 4 * b;  // bytes of this word
          const uint32_t mask = valid >= 4 ? 0u : valid <= 0 ? ~0u : ~0u << 8 * valid;
          low = __vmins4(low, (w[b] & ~mask) | (0x7F7F7F7Fu & mask));
        }
        low = __vmins4(low, low >> 16 | 0x7F7F0000u);
        low = __vmins4(low, low >> 8 | 0x7F7F7F00u);
        atomicMin(&xtop[par * 32 + n], (int)(int8_t)(low & 0xFFu));
      }
    } else {
      chunks(np, [&](int n, int u) {
        const uint4 r = *unit_at(n, u);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        uint32_t m = 0u;  // (magnitudes of bf16 are in the order of their bits, NaN above infinity)
#pragma unroll
        for (int b = 0; b < 4; ++b) m = __vmaxu2(m, w[b] & 0x7FFF7FFFu);
        const unsigned top = __reduce_max_sync(~0u, max(m & 0xFFFFu, m >> 16));
        if (lane == 0) atomicMax(&xtop[par * 32 + n], (int)(top << 16));
      });
    }
    __syncthreads();
    chunks(np, [&](int n, int u) {
      const int up = DOWN ? xtop[par * 32 + n] : f16_up((unsigned)xtop[par * 32 + n]);
      if (u == 0) xdown[par * 32 + n] = pow2(-up);
      // h: 2^(up of the vector - up of the unit), at least 2^-126, where nothing is left of 16 bits
      const float f = pow2(DOWN ? max(up - (u < wide ? (int)ups[n * p.up_pitch + u] : up), -126) : up);
      uint4 *to = unit_at(n, u);
      const uint4 r = *to;
      uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        float2 x;
        if constexpr (DOWN) x = __half22float2(*reinterpret_cast<const __half2 *>(&w[b]));
        else x = make_float2(__uint_as_float(w[b] << 16), __uint_as_float(w[b] & 0xFFFF0000u));
        const __half2 y = __floats2half2_rn(x.x * f, x.y * f);
        w[b] = *reinterpret_cast<const uint32_t *>(&y);
      }
      *to = make_uint4(w[0], w[1], w[2], w[3]);
    });
    if (tid < 32) xtop[(par ^ 1) * 32 + tid] = DOWN ? INT_MAX : INT_MIN;
    __syncthreads();

    // ---- the run, with as many n-tiles as the job's pairs fill (three and four by one
    // form of four: 256 tokens 2064 x 1424, 6 of 60 took 177 us instead of 164)
    auto products = [&](auto tiles_of_pairs) {
      constexpr int A = decltype(tiles_of_pairs)::value;
      const Run r = run_of(j, warp);
      float acc[A][4];
      auto clear = [&] {
#pragma unroll
        for (int nt = 0; nt < A; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
      };
      clear();
      const MoeMatrix &mv = DOWN ? a.down : a.up;
      const float av = mv.alpha[e * mv.alpha_stride];
      [[maybe_unused]] const float ag = GATED && !DOWN ? a.gate.alpha[e * a.gate.alpha_stride] : 0.0f;
      // a tile's finished sums
      auto finish_tile = [&](int t) {
#pragma unroll
        for (int nt = 0; nt < A; ++nt) {
          const int n0 = 8 * nt + 2 * cq, m0 = min(n0, np - 1), m1 = min(n0 + 1, np - 1);
          const bool one = n0 < np, two = n0 + 1 < np;
          const int64_t p0 = pair[m0], p1 = pair[m1];
          const float d0 = xdown[par * 32 + m0], d1 = xdown[par * 32 + m1];
          if constexpr (DOWN) {
            float *q = p.part + (int64_t)t * 16 + g;
            if (one) {
              q[p0 * a.hidden] = acc[nt][0] * av * d0;
              q[p0 * a.hidden + 8] = acc[nt][2] * av * d0;
            }
            if (two) {
              q[p1 * a.hidden] = acc[nt][1] * av * d1;
              q[p1 * a.hidden + 8] = acc[nt][3] * av * d1;
            }
          } else {
            // h of eight rows (this lane's and those of the other g): a common power of two
            auto put = [&](float v, int64_t pr, int64_t row8, bool there) {
              unsigned top = __float_as_uint(v) & 0x7FFFFFFFu;
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
              const int up = f16_up(top);
              if (!there) return;
              p.h[pr * a.inner + row8 * 8 + g] = __float2half_rn(v * pow2(up));
              if (g == 0) p.h_up[pr * p.up_pitch + row8] = (int8_t)up;
            };
            if constexpr (GATED) {
              float v[2] = {acc[nt][0] * ag * d0, acc[nt][1] * ag * d1};
              activate(v, a.act);
              put(v[0] * (acc[nt][2] * av * d0), p0, t, one);
              put(v[1] * (acc[nt][3] * av * d1), p1, t, two);
            } else {
              float v[4] = {acc[nt][0] * av * d0, acc[nt][1] * av * d1, acc[nt][2] * av * d0, acc[nt][3] * av * d1};
              activate(v, a.act);
              put(v[0], p0, 2 * (int64_t)t, one);
              put(v[1], p1, 2 * (int64_t)t, two);
              put(v[2], p0, 2 * (int64_t)t + 1, one);
              put(v[3], p1, 2 * (int64_t)t + 1, two);
            }
          }
        }
      };
      int ct = r.u0 / nk, ck = r.u0 - ct * nk;  // counted from the part's first tile
      bool mine = ck == 0;  // this warp takes the current tile's first step
      auto put_own = [&] {
#pragma unroll
        for (int nt = 0; nt < A; ++nt)
          if (8 * nt < np) own[(warp * NB + nt) * 32 + lane] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
      };
      const uint4 *xl[A], *xk[A];  // this lane's column of the vectors, and its place in the current step
#pragma unroll
      for (int nt = 0; nt < A; ++nt) {
        xl[nt] = xs + min(8 * nt + g, np - 1) * 4 + cq;
        xk[nt] = xl[nt] + ck * 32 * P;
      }
      [[maybe_unused]] const int chunk0 = g * 8 + ((2 * cq) ^ g), chunk1 = g * 8 + ((2 * cq + 1) ^ g);
      [[maybe_unused]] const int odd_at = g * 144 + (g & 1 ? back : 0) + 32 * cq;
      for (int left = r.u1 - r.u0; left > 0; --left) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kMoeDepth - 1) : "memory");
        __syncwarp();
        const uint4 *here = slots + take;
        take = take == (kMoeDepth - 1) * (kSlot / 16) ? 0 : take + kSlot / 16;
        uint32_t sc[2][2][2];  // [half][row][block]: f16 pairs {Delta, Delta}
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t *words = reinterpret_cast<const uint32_t *>(here + kScales / 16) + lane;
          uint32_t word;
          if constexpr (WIDE) {
            word = words[h * 32];
          } else {
            const MoeMatrix &m = DOWN ? a.down : GATED && h == 0 ? a.gate : a.up;
            const int64_t row = (int64_t)(r.t0 + ct) * kTileRows + (GATED && !DOWN ? 0 : 8 * h) + g;
            const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(m.scales) + e * m.scale_stride + row * nblk) & 3u;
            word = __funnelshift_r(words[h * 64], words[h * 64 + 32], 8 * off);
          }
          uint32_t f[2];
          asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
              : "=r"(f[0]), "=r"(f[1]) : "r"(word));
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            sc[half][h][0] = __byte_perm(f[half], 0u, 0x1010);
            sc[half][h][1] = __byte_perm(f[half], 0u, 0x3232);
          }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint4 c0, c1;
          if constexpr (LOADS == kOdd) {
            const uint2 *from = reinterpret_cast<const uint2 *>(reinterpret_cast<const uint8_t *>(here) + odd_at) + 2 * half;
            const uint2 l0 = from[0], h0 = from[1], l1 = from[8 * 18], h1 = from[8 * 18 + 1];
            c0 = make_uint4(l0.x, l0.y, h0.x, h0.y), c1 = make_uint4(l1.x, l1.y, h1.x, h1.y);
          } else {
            c0 = here[half ? chunk1 : chunk0], c1 = here[64 + (half ? chunk1 : chunk0)];
          }
          const uint32_t cw[2][4] = {{c0.x, c0.y, c0.z, c0.w}, {c1.x, c1.y, c1.z, c1.w}};
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) {  // a word of codes: 8 columns, two k-steps
            uint32_t w[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              e2m1x8_f16(cw[h][jj], w[h]);
#pragma unroll
              for (int b = 0; b < 4; ++b) w[h][b] = mul_f16x2(w[h][b], sc[half][h][jj >> 1]);
            }
#pragma unroll
            for (int nt = 0; nt < A; ++nt) {
              const uint4 xb = xk[nt][(half * 4 + jj) * (4 * P)];
              mma_f16(acc[nt], w[0][0], w[1][0], w[0][1], w[1][1], xb.x, xb.y);
              mma_f16(acc[nt], w[0][2], w[1][2], w[0][3], w[1][3], xb.z, xb.w);
            }
          }
        }
        __syncwarp();
        fetch();  // into the place just read
#pragma unroll
        for (int nt = 0; nt < A; ++nt) xk[nt] += 32 * P;
        if (++ck == nk) {  // the tile's last step
          if (mine) finish_tile(r.t0 + ct);
          else put_own();
          clear();
#pragma unroll
          for (int nt = 0; nt < A; ++nt) xk[nt] = xl[nt];
          ck = 0;
          ++ct;
          mine = true;
        }
      }
      const bool open = ck > 0 && r.u1 > r.u0;  // the run ends inside a tile
      if (open && !mine) put_own();
      __syncthreads();
      if (open && mine) {  // that it began: the next warps have the rest
        for (int w = warp + 1; w < warps; ++w) {
          const Run o = run_of(j, w);
          if (o.u0 >= (ct + 1) * nk) break;
          if (o.u0 == o.u1) continue;
#pragma unroll
          for (int nt = 0; nt < A; ++nt) {
            if (8 * nt >= np) break;
            const float4 v = own[(w * NB + nt) * 32 + lane];
            acc[nt][0] += v.x, acc[nt][1] += v.y, acc[nt][2] += v.z, acc[nt][3] += v.w;
          }
        }
        finish_tile(r.t0 + ct);
      }
    };
    if (np <= 8) products(std::integral_constant<int, 1>());
    else if constexpr (NT > 1) {
      if (np <= 16) products(std::integral_constant<int, 2>());
      else if (np <= 24) products(std::integral_constant<int, 3>());
      else products(std::integral_constant<int, 4>());
    }
  }
}

// y = residual + the sum of a token's slots, in slot order; four columns a thread.
// What was there before the products is read before they end.
__global__ void __launch_bounds__(256) k_moe_join(const __grid_constant__ MoeLaunch p) {
  const MoeArgs &a = p.a;
  const int64_t quads = a.hidden / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool mine = i < quads * a.tokens;
  const int64_t t = i / quads, c = (i - t * quads) * 4;
  constexpr int kSlots = 8;  // slots read at a time
  float w[kSlots];
  bool there[kSlots];
  auto slots = [&](int s0) {
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const int64_t at = t * a.top_k + min(s0 + s, a.top_k - 1);
      const int e = mine ? a.ids[at] : -1;
      there[s] = s0 + s < a.top_k && e >= 0 && e < a.experts;
      w[s] = mine ? a.weights[at] : 0.0f;
    }
  };
  slots(0);
  float r[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const __nv_bfloat16 *res = static_cast<const __nv_bfloat16 *>(a.residual);
  if (res && mine) {
#pragma unroll
    for (int b = 0; b < 4; ++b) r[b] = __bfloat162float(res[t * a.residual_stride + c + b]);
  }
  pdl_wait();
  pdl_launch_dependents();
  if (!mine) return;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s0 = 0; s0 < a.top_k; s0 += kSlots) {
    if (s0 > 0) slots(s0);
    float4 o[kSlots];
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      o[s] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (there[s]) o[s] = *reinterpret_cast<const float4 *>(p.part + (t * a.top_k + s0 + s) * a.hidden + c);
    }
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
      if (there[s]) v[0] = fmaf(w[s], o[s].x, v[0]), v[1] = fmaf(w[s], o[s].y, v[1]), v[2] = fmaf(w[s], o[s].z, v[2]), v[3] = fmaf(w[s], o[s].w, v[3]);
  }
  __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y) + t * a.y_stride + c;
#pragma unroll
  for (int b = 0; b < 4; ++b) y[b] = __float2bfloat16(v[b] + r[b]);
}

namespace {

// Pairs of a job at most, of those wanted, for the vectors' room in shared memory.
int moe_group(int wanted, int64_t cols, bool down, int warps, int loads, int experts, int pairs, int64_t room) {
  for (int n = wanted; n > 0; --n)
    if (moe_smem(n, cols, down, warps, loads, experts, pairs) <= room) return n;
  return 0;
}

template <typename F>
auto with_kernel(int nt, bool down, bool gated, int loads, F f) {
  auto pick = [&](auto l, auto n) {
    constexpr int L = decltype(l)::value, N = decltype(n)::value;
    return down ? f(k_moe<N, true, false, L>) : gated ? f(k_moe<N, false, true, L>) : f(k_moe<N, false, false, L>);
  };
  auto pick_nt = [&](auto l) {
    return nt == 1 ? pick(l, std::integral_constant<int, 1>()) : pick(l, std::integral_constant<int, 4>());
  };
  return loads == kWide ? pick_nt(std::integral_constant<int, kWide>())
         : loads == kOdd ? pick_nt(std::integral_constant<int, kOdd>()) : pick_nt(std::integral_constant<int, kAny>());
}

template <typename K>
cudaError_t launch_dependent(K *k, int grid, int threads, size_t smem, const MoeLaunch &p, cudaStream_t st) {
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p);
}

cudaError_t launch_product(MoeLaunch p, bool down, int sms, cudaStream_t st) {
  const MoeArgs &a = p.a;
  p.cols = down ? a.inner : a.hidden;
  p.steps = (int)((p.cols + 255) / 256);
  p.tiles = (int)(down ? a.hidden / 16 : a.gated ? a.inner / 8 : a.inner / 16);
  auto loads_of = [&](const MoeMatrix &m) -> int {
    if ((reinterpret_cast<uintptr_t>(m.codes) | m.code_stride) % 16) return kAny;
    return p.cols % 64 || (reinterpret_cast<uintptr_t>(m.scales) | m.scale_stride) % 4 ? kOdd : kWide;
  };
  const int loads = down ? loads_of(a.down) : std::max(loads_of(a.up), a.gated ? loads_of(a.gate) : (int)kWide);
  // Pairs that a job should take: few experts have more than three times the mean and four.
  const int wanted = std::min({p.pairs, 32, 4 + 3 * p.pairs / a.experts});
  p.job_cost = std::min(368 / p.steps, p.tiles);
  p.more_cost = loads == kWide ? 3 : 2;
  // Little work: one small CTA per SM, so that the next launch's CTAs find room beside
  // it (1 token 2048 x 768, 8 of 128: 7 % less time than with two).
  const bool little = (int64_t)std::min(p.pairs, a.experts) * p.tiles * p.steps <= (int64_t)64 * sms;
  int warps = 8, ctas = little ? sms : 2 * sms;
  auto fit = [&](int64_t room) { p.group = moe_group(wanted, p.cols, down, warps, loads, a.experts, p.pairs, room); };
  fit(kMoeHalfSmem);
  if (p.group < wanted) {
    warps = kMoeMaxWarps, ctas = sms;
    fit(kMoeSmem);
  }
  if (p.group == 0) {  // vectors too long for that many units in flight
    warps = 8;
    fit(kMoeSmem);
  }
  p.share = (uint32_t)((uint64_t{1} << 32) / (uint32_t)ctas);
  const size_t smem = (size_t)moe_smem(p.group, p.cols, down, warps, loads, a.experts, p.pairs);
  return with_kernel(p.group <= 8 ? 1 : 4, down, a.gated, loads,
                     [&](auto *k) { return launch_dependent(k, ctas, warps * 32, smem, p, st); });
}

size_t moe_h_bytes(int64_t inner, int pairs) { return ((size_t)pairs * inner * 2 + 255) / 256 * 256; }
size_t moe_up_bytes(int64_t inner, int pairs) { return ((size_t)pairs * moe_up_pitch(inner) + 255) / 256 * 256; }

}  // namespace

bool moe_fits(int64_t hidden, int64_t inner, int experts, int pairs) {
  return moe_group(1, hidden, false, 8, kOdd, experts, pairs, kMoeSmem) > 0 &&
         moe_group(1, inner, true, 8, kOdd, experts, pairs, kMoeSmem) > 0;
}

size_t moe_workspace_bytes(int64_t hidden, int64_t inner, int pairs) {
  return moe_h_bytes(inner, pairs) + moe_up_bytes(inner, pairs) + (size_t)pairs * hidden * 4;
}

cudaError_t launch_moe(const MoeArgs &a, int sms, void *ws, cudaStream_t st) {
  MoeLaunch p = {};
  p.a = a;
  p.pairs = a.tokens * a.top_k;
  p.up_pitch = moe_up_pitch(a.inner);
  char *at = static_cast<char *>(ws);
  p.h = reinterpret_cast<__half *>(at);
  p.h_up = reinterpret_cast<int8_t *>(at += moe_h_bytes(a.inner, p.pairs));
  p.part = reinterpret_cast<float *>(at += moe_up_bytes(a.inner, p.pairs));
  cudaError_t e = launch_product(p, false, sms, st);
  if (e == cudaSuccess) e = launch_product(p, true, sms, st);
  if (e != cudaSuccess) return e;
  return launch_dependent(k_moe_join, (int)((a.hidden / 4 * a.tokens + 255) / 256), 256, 0, p, st);
}

cudaError_t prepare_moe_kernels() {
  cudaError_t e = cudaSuccess;
  for (int nt : {1, 4})
    for (int form : {0, 1, 2})
      for (int loads : {kWide, kOdd, kAny})
        if (e == cudaSuccess)
          e = with_kernel(nt, form == 2, form == 1, loads,
                          [](auto *k) { return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoeSmem); });
  return e;
}

}  // namespace nvfp4
