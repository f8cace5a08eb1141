// nvfp4_linear_tc.cu -- nvfp4_linear on tcgen05, for more vectors than
// nvfp4_linear.cu takes.
//
// The dequantized weights never touch shared memory: the producers write them
// to tensor memory, where tcgen05.mma takes its A operand, lane = row.  Shared
// memory carries the codes (64 B per row and step) and X only; with A there as
// well a 128 x 128 step would move 64 KiB more through its 128 B per clock.
//
// Types: q * Delta has six significant bits between 2^-10 and 2688, so both
// f16 and bf16 hold it exactly; the two operands of an MMA must be of one type.
//   - f16 weights take two instructions per pair to form, but x has to be
//     turned into f16 first (k_linear_x, each vector scaled by a power of two
//     that takes its largest entry into [2^13, 2^14): 8 bits stay exact down
//     to 2^-27 of that entry, an entry below is off by at most 2^-38 of it).
//     The product starts early (programmatic dependent launch) and has its
//     weights in flight meanwhile.
//   - bf16 weights take five, and x is read as it is, in one launch.
//
// Bound: up to 64 vectors nominally HBM, in fact the set-up and a step's fixed
// cost; at 256 vectors the tensor pipe.  Measured: 13 vectors 14336 x 4096 17.7 us
// (1.9 TB/s; of a CTA's 28000 clocks 2200 pass until it has its tensor memory,
// 6000 until the first codes are there, 16000 over 24 steps, 2000 from the last
// MMA to its end); 16 vectors 8192 x 28672 37 us (3.6 TB/s, 540 clocks a step), 52 us
// with 28640 columns (no TMA for the codes); 128 vectors 50 us; 256 vectors 80 us (1.50 PFLOP/s, the tensor pipe 78 % busy).
//
// Work: row tiles of 128 by column steps of 128.  With `tiles` tiles on G CTAs
// (one per SM), each CTA takes floor(tiles / G) whole tiles; the steps of the
// tiles left over are cut into equal contiguous ranges of at least one step, one
// per CTA, which does it first.  The part of a tile inside a CTA is a segment with an accumulator of
// its own.  A whole tile is finished by its CTA; the parts of a shared one meet
// in the workspace, where a second launch (k_linear_join) adds them in CTA
// order with all SMs: when the last CTA of a tile did it, four parts of a tile
// took 2 us at 16 vectors and 10 us at 256.
//
// Roles inside a CTA (736 threads), every hand-off through an mbarrier:
//   - warps 0-15, four groups of four that take the steps in turn: a thread
//     forms the 128 weights of one row and stores them with tcgen05.st;
//   - warps 16-19 read finished accumulators back (the last one with the
//     producers' help);
//   - warp 20 (one lane) issues the eight tcgen05.mma of a step (M = 128,
//     K = 16, N = the vectors rounded up to 16);
//   - warp 21 (one lane) loads X by TMA;
//   - warp 22 (one lane) loads codes and scales by TMA where their rows are
//     whole multiples of 16 bytes; otherwise the producers copy their own with
//     cp.async.
// Every wait is bounded; a CTA that gives up lets its copies and MMAs in
// flight finish (bounded), and its outputs are NaN.
#include <algorithm>
#include <cmath>
#include <cstring>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"
#include "nvfp4_epilogue.cuh"
#include "nvfp4_internal.h"
#include "nvfp4_tc.cuh"

namespace nvfp4 {

constexpr int kLtM = 128, kLtK = 128;
constexpr int kLtProducers = 512;
constexpr int kLtEpiWarp0 = 16, kLtMmaWarp = 20, kLtXWarp = 21, kLtCodeWarp = 22;
constexpr int kLtThreads = 736;
constexpr int kLtGroups = 4;       // of producers
// ring slot: by TMA [128][64 B] codes (64-byte swizzle), then [128][16 B] scales;
// by the producers 80 B per row: 64 of codes, 12 of scales
constexpr uint32_t kLtSlot = 10240;
constexpr int kLtDyn = 227 * 1024 - 2048;
// Steps per CTA up to which the operands are bf16.  24 vectors take (us, f16 and
// bf16) 4096 x 4096 (7 steps) 12.3 and 12.3, 14336 x 4096 (24) 17.6 and 18.5, 8192 x
// 8192 (27) 18.2 and 19.3, 8192 x 28672 (94) 38.3 and 43.3; f16 is a launch more, which
// costs a program that does not capture its calls 2 us.  (Above 128 vectors
// the MMAs hide the producers, and it is always bf16.)
constexpr int kLtBfSteps = 24;

// CAP: vectors that a launch's shared and tensor memory are laid out for.
template <int CAP>
struct LtCfg {
  // A stage of A holds P steps; up to 128 vectors it has the steps' X too, and
  // one pair of mbarriers for both.  The issuing thread competes with sixteen
  // busy warps for issue slots, and a wait or a commit costs it about 150
  // clocks: with two of each per step it took 690 clocks a step (8192 x 28672,
  // 16 vectors), with one 540, while the MMAs of a step take 75.  At 256
  // vectors they take 1024, and an atom of X per stage keeps four loads going.
  static constexpr int P = CAP <= 64 ? 2 : 1;
  static constexpr bool kOne = CAP <= 128;
  static constexpr int H = kOne ? 2 * P : 1;         // 64-column atoms of X per stage
  static constexpr uint32_t kAtom = CAP * 128u;
  static constexpr uint32_t kXStage = H * kAtom;
  static constexpr int SA = CAP <= 64 ? 3 : 4;       // A stages
  static constexpr int SX = kOne ? SA : 4;
  static constexpr int D0 = (int)((kLtDyn - 1024 - SX * kXStage) / kLtSlot) / kLtGroups * kLtGroups;
  static constexpr int D = D0 > 16 ? 16 : D0;
  static constexpr int NB = CAP <= 128 ? 2 : 1;      // accumulators
  static constexpr uint32_t kA = NB * CAP;           // tensor-memory column of the first A stage
  static constexpr size_t kSmem = 1024 + (size_t)SX * kXStage + (size_t)D * kLtSlot;
  static_assert(kA + SA * P * 64 <= 512, "tensor memory");
  static_assert(D >= 2 * kLtGroups, "ring");
};

struct LtArgs {
  LinearArgs a;
  int K;            // steps per tile
  int64_t R;        // shared tiles: tiles 0 .. R - 1
  int W;            // whole tiles per CTA: R + CTA, + G, ...
  const int *up;    // [batch]: x was divided by 2^up (f16)
  float *part;      // [2 CTAs][batch][128]
  int tma;          // codes and scales by TMA
  int wide;         // else: rows of codes are whole multiples of 16 bytes, aligned
  int first_tries;  // < 0: normal (test hook)
};

// x -> f16, one CTA per vector: one pass over memory for up to 8 * kLxKeep *
// kLxThreads entries (they stay in registers between the maximum and the
// conversion), a second one for the entries behind those.
constexpr int kLxThreads = 1024, kLxKeep = 4;
__global__ void __launch_bounds__(kLxThreads) k_linear_x(const uint4 *__restrict__ x, int64_t x_stride8, int64_t units,
                                                         uint4 *__restrict__ xf, int *__restrict__ up_out) {
  __shared__ uint32_t s_top[kLxThreads / 32];
  pdl_launch_dependents();
  const int64_t b = blockIdx.x;
  const uint4 *from = x + b * x_stride8;
  uint32_t m = 0u;
  auto take = [&](const uint4 &v) {
    asm("{\n\t.reg .b32 s, t;\n\tmax.xorsign.abs.bf16x2 s, %1, %2;\n\tmax.xorsign.abs.bf16x2 t, %3, %4;\n\t"
        "max.xorsign.abs.bf16x2 s, s, t;\n\tmax.xorsign.abs.bf16x2 %0, %0, s;\n\t}"
        : "+r"(m) : "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
  };
  uint4 keep[kLxKeep];
#pragma unroll
  for (int i = 0; i < kLxKeep; ++i) {
    const int64_t u = threadIdx.x + i * kLxThreads;
    keep[i] = u < units ? __ldg(from + u) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kLxKeep; ++i) take(keep[i]);
  for (int64_t u = threadIdx.x + kLxKeep * kLxThreads; u < units; u += kLxThreads) take(__ldg(from + u));
  m &= 0x7FFF7FFFu;
  m = __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = m;
  __syncthreads();
  m = __reduce_max_sync(0xFFFFFFFFu, s_top[threadIdx.x & 31]);
  const int e = (int)(m >> 7), up = e == 255 ? 0 : max(e, 1) - 127 - 13;  // (inf and NaN stay as they are)
  const float f1 = pow2(-up / 2), f2 = pow2(-up - (-up / 2));            // (2^-up alone may be out of range)
  auto give = [&](int64_t u, const uint4 &v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("cvt.rn.f16x2.f32 %0, %1, %2;"
          : "=r"(o[i]) : "f"(__uint_as_float(w[i] & 0xFFFF0000u) * f1 * f2), "f"(__uint_as_float(w[i] << 16) * f1 * f2));
    xf[b * units + u] = make_uint4(o[0], o[1], o[2], o[3]);
  };
#pragma unroll
  for (int i = 0; i < kLxKeep; ++i) {
    const int64_t u = threadIdx.x + i * kLxThreads;
    if (u < units) give(u, keep[i]);
  }
  for (int64_t u = threadIdx.x + kLxKeep * kLxThreads; u < units; u += kLxThreads) give(u, __ldg(from + u));
  if (threadIdx.x == 0) up_out[b] = up;
}
static_assert(kLxThreads == 1024, "one maximum per lane");

// Bounded wait, polling: a waiting thread that suspends with a time hint (as
// tc_wait's does) wakes late.  Gives up once another role has raised `fail`,
// and raises it itself after about 2 s.
__device__ __forceinline__ bool lt_wait(uint32_t mb, uint32_t parity, volatile int *fail) {
  if (mbar_test(mb, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
      uint32_t done;
      asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                   "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(done) : "r"(mb), "r"(parity) : "memory");
      if (done) return true;
    }
    if (*fail) return false;
    if (clock64() - t0 > 4000000000LL) {
      *fail = 1;
      return false;
    }
  }
}

// One thread of a converged warp.  With this predicate the compiler knows that
// a single thread issues, and feeds tcgen05 and TMA instructions from uniform
// registers: 90 clocks per tcgen05.mma issued in a plain loop, against 157 for
// "lane == 0" (N = 16, M = 128).
__device__ __forceinline__ bool lt_elect() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// Instruction descriptor of kind::f16: fp32 accumulator (bits 4-5 = 1), types
// of A and B (bits 7-9 and 10-12: 0 f16, 1 bf16), both K-major, N >> 3 at bits
// 17-22, M >> 4 at bits 24-28.
template <bool BF>
__device__ __forceinline__ uint32_t lt_idesc(int n) {
  return (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kLtM >> 4) << 24);
}

// 16 words of a lane to 16 consecutive columns of tensor memory.
__device__ __forceinline__ void lt_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
               "%14, %15, %16};"
               ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                 "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}

// Two blocks (16 code bytes, scales in the low two bytes of s) -> 16 pairs of
// q * Delta in f16 or bf16.
template <bool BF>
__device__ __forceinline__ void lt_weights(const uint4 &c, uint32_t s, uint32_t (&w)[16]) {
  uint32_t f;
  asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(f) : "r"(s));
  const uint32_t sc[2] = {__byte_perm(f, 0u, 0x1010), __byte_perm(f, 0u, 0x3232)};
  const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t q[4];
    e2m1x8_f16(cw[j], q);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t v = mul_f16x2(q[b], sc[j >> 1]);
      if (BF) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&v));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[4 * j + b]) : "f"(x.y), "f"(x.x));
      } else {
        w[4 * j + b] = v;
      }
    }
  }
}

// CTAs 0 .. lt_sharers - 1 have steps of the shared tiles, each at least one
// (so that every part that the join adds has been written).
__host__ __device__ __forceinline__ int64_t lt_sharers(const LtArgs &p, int64_t G) { return p.R * p.K < G ? p.R * p.K : G; }

// The CTAs c0 .. c0 + n - 1 that share tile t.
struct LtParts {
  int64_t c0;
  int n;
};
__device__ __forceinline__ LtParts lt_parts(const LtArgs &p, int64_t t, int64_t T, int64_t GS) {
  LtParts q;
  q.c0 = tc_cta_of(t * p.K, T, GS);
  q.n = (int)(tc_cta_of((t + 1) * p.K - 1, T, GS) - q.c0) + 1;
  return q;
}
// Adds the parts of rows r8 .. r8 + 7 of tile t and vector b in CTA order
// (eight loads in flight) and finishes them.
__device__ __forceinline__ void lt_join(const LtArgs &p, float alpha, bool vec, const LtParts &q, int64_t t, int b, int r8, int up) {
  const LinearArgs &a = p.a;
  float w[8] = {};
  for (int j0 = 0; j0 < q.n; j0 += 4) {
    float4 o[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t s = 2 * (q.c0 + j0 + j) + (j0 + j == 0 ? 1 : 0);
      const float4 *from = reinterpret_cast<const float4 *>(p.part + (s * a.batch + b) * kLtM + r8);
      o[j][0] = j0 + j < q.n ? __ldcg(from) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      o[j][1] = j0 + j < q.n ? __ldcg(from + 1) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[0] += o[j][0].x, w[1] += o[j][0].y, w[2] += o[j][0].z, w[3] += o[j][0].w;
      w[4] += o[j][1].x, w[5] += o[j][1].y, w[6] += o[j][1].z, w[7] += o[j][1].w;
    }
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) w[u] = w[u] * pow2(up / 2) * pow2(up - up / 2);
  const int64_t r0 = t * kLtM + r8;
  if (vec && r0 + 8 <= a.rows) finish_rows8(a, alpha, w, b, r0);
  else finish<8>(a, alpha, w, [&](int u) { return r0 + u < a.rows; }, [&](int) { return (int64_t)b; },
                 [&](int u) { return r0 + u; });
}

template <int CAP, bool BF>
__global__ void __launch_bounds__(kLtThreads, 1) k_linear_tc(const __grid_constant__ CUtensorMap xmap,
                                                             const __grid_constant__ CUtensorMap cmap,
                                                             const __grid_constant__ CUtensorMap smap,
                                                             const __grid_constant__ LtArgs p) {
  using C = LtCfg<CAP>;
  constexpr int SX = C::SX, SA = C::SA, D = C::D, NB = C::NB, H = C::H, P = C::P;
  extern __shared__ uint8_t dsm[];
  __shared__ __align__(8) uint64_t full_a[SA], empty_a[SA], full_x[SX], empty_x[SX], acc_full[NB], acc_empty[NB],
      ring_full[D], ring_empty[D];
  __shared__ uint32_t tmem_slot;
  __shared__ int fail;
  __shared__ int16_t s_up[CAP];
  const LinearArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t raw = tc_smem(dsm), base = (raw + 1023u) & ~1023u;  // swizzle atoms need 1024-byte alignment
  uint8_t *ring = dsm + (base - raw) + SX * C::kXStage;
  const int64_t G = gridDim.x, c = blockIdx.x, T = p.R * p.K, GS = lt_sharers(p, G);
  const int64_t g0 = c < GS ? tc_first_step(c, T, GS) : T, g1 = c < GS ? tc_first_step(c + 1, T, GS) : T;  // of the shared tiles' steps
  const int nr = (int)(g1 - g0), n = nr + p.W * p.K;                           // steps: shared ones first
  const int64_t t_first = g0 / p.K;
  const int nsh = nr > 0 ? (int)((g1 - 1) / p.K - t_first + 1) : 0, nseg = nsh + p.W;
  const int nv = (a.batch + 15) & ~15;  // MMA columns
  volatile int *vfail = &fail;

  if (tid == 0) fail = 0;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem(&tmem_slot)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == kLtMmaWarp * 32) {
    for (int s = 0; s < SA; ++s) {
      mbar_init(tc_smem(&full_a[s]), 4 * P + (C::kOne ? 1 : 0));  // the producing warps (and X's loader)
      mbar_init(tc_smem(&empty_a[s]), 1);
    }
    for (int s = 0; s < SX; ++s) {
      mbar_init(tc_smem(&full_x[s]), 1);
      mbar_init(tc_smem(&empty_x[s]), 1);
    }
    for (int d = 0; d < D; ++d) {
      mbar_init(tc_smem(&ring_full[d]), 1);
      mbar_init(tc_smem(&ring_empty[d]), 4);
    }
    for (int b = 0; b < NB; ++b) {
      mbar_init(tc_smem(&acc_full[b]), 1);
      mbar_init(tc_smem(&acc_empty[b]), 4);  // one per epilogue warp
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }

  // A place in the CTA's steps: step i is column step ks of tile t.
  struct Place {
    int64_t t;
    int ks, i;
  };
  auto advance = [&](Place &q, int by) {
    const bool was_shared = q.i < nr;
    q.i += by;
    q.ks += by;
    if (was_shared && q.i >= nr) {  // on to the whole tiles
      q.t = p.R + c;
      q.ks = q.i - nr;
    }
    const int64_t next = q.i < nr ? 1 : G;
    for (; q.ks >= p.K; q.ks -= p.K) q.t += next;
  };
  Place start;
  start.i = 0;
  start.t = nr > 0 ? t_first : p.R + c;
  start.ks = nr > 0 ? (int)(g0 - t_first * p.K) : 0;

  // ---- producers: warp 4 group + row / 32 takes the steps i with i % 4 == group
  const int grp = warp >> 2, row = 32 * (warp & 3) + lane;
  const int64_t cb = a.cols / 16;
  Place me = start, f;
  if (warp < kLtProducers / 32) advance(me, grp);
  f = me;
  // this warp's 32 rows of step i, at `f`: eight (or four) lanes a row,
  // so that an instruction touches few lines
  auto fetch = [&](int i) {
    const uint32_t to = tc_smem(ring) + (uint32_t)(i % D) * kLtSlot + (uint32_t)(32 * (warp & 3)) * 80u;
    const int64_t r0 = f.t * kLtM + 32 * (warp & 3), blk = (int64_t)f.ks * 8;
    advance(f, kLtGroups);
    const int have = (int)min((int64_t)8, cb - blk), rows = (int)max((int64_t)0, min((int64_t)32, a.rows - r0));
    if (p.wide) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 8 * j + (lane >> 2), b = 2 * (lane & 3);
        const bool in = r < rows && b < have;  // (an even number of blocks per row)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     ::"r"(to + r * 80 + 8 * b), "l"(in ? a.codes + ((r0 + r) * cb + blk + b) * 8 : a.codes), "r"(in ? 16 : 0) : "memory");
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = 4 * j + (lane >> 3), b = lane & 7;
        const bool in = r < rows && b < have;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;"
                     ::"r"(to + r * 80 + 8 * b), "l"(in ? a.codes + ((r0 + r) * cb + blk + b) * 8 : a.codes), "r"(in ? 8 : 0) : "memory");
      }
    }
    // the aligned words that hold a row's scale bytes (rows may start at any byte)
    const uint8_t *end = a.scales + a.rows * cb;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const int w = lane + 32 * j, r = w / 3;
      const uint8_t *ps = a.scales + (r0 + r) * cb + blk;
      const uint8_t *wp = ps - (reinterpret_cast<uintptr_t>(ps) & 3) + 4 * (w - 3 * r);
      const uint32_t at = to + r * 80 + 64 + 4 * (w - 3 * r);
      const bool need = r < rows && wp < ps + have;
      if (need && wp < a.scales) {  // the array's first word, not aligned: a byte at a time
        uint32_t v = 0u;
        for (int b = 0; b < 4; ++b)
          if (wp + b >= a.scales && wp + b < end) v |= (uint32_t)__ldg(wp + b) << (8 * b);
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
      } else {
        const int bytes = need ? (int)min((int64_t)4, (int64_t)(end - wp)) : 0;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(at), "l"(need ? wp : a.codes), "r"(bytes) : "memory");
      }
    }
  };
  if (warp < kLtProducers / 32 && !p.tma) {
#pragma unroll 1
    for (int i = grp; i < D; i += kLtGroups) {  // one commit group per step of this warp's group
      if (i < n) fetch(i);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;");
  const uint32_t tmem = tmem_slot;

  int hi = 0;  // loaders: stages or steps asked for, [0, hi)
  if (warp < kLtProducers / 32) {
    // ---- dequantize: step i to half i % P of A stage (i / P) % SA
    const uint32_t ta = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + C::kA + 64u * (grp % P);
    const uint32_t sw = p.tma ? (uint32_t)(row >> 1) & 3u : 0u;  // the code tile's 64-byte swizzle
    int slot = grp, st = grp / P;
    uint32_t rph = 0u, aph = 1u;  // parities of ring_full[slot] and empty_a[st] (an untouched stage is empty)
#pragma unroll 1
    for (int i = grp; i < (n + P - 1) / P * P; i += kLtGroups) {
      if (P > 1 && i >= n) {  // a stage's second step that does not exist: its warps arrive all the same
        if (!__all_sync(0xFFFFFFFFu, lt_wait(tc_smem(&empty_a[st]), aph, vfail))) break;
      } else {
        const uint8_t *sl = ring + (uint32_t)slot * kLtSlot, *src = sl + row * (p.tma ? 64 : 80);
        uint2 sc;
        if (p.tma) {
          if (!__all_sync(0xFFFFFFFFu, lt_wait(tc_smem(&ring_full[slot]), rph, vfail))) break;
          sc = *reinterpret_cast<const uint2 *>(sl + 8192 + row * 16 + (me.ks & 1) * 8);
        } else {
          asm volatile("cp.async.wait_group %0;" ::"n"(D / kLtGroups - 1) : "memory");  // this step's bytes have landed
          __syncwarp();
          const uint4 w = *reinterpret_cast<const uint4 *>(src + 64);
          const int64_t blk = (int64_t)me.ks * 8;
          const uint32_t by = 8u * (uint32_t)((reinterpret_cast<uintptr_t>(a.scales) + (me.t * kLtM + row) * cb + blk) & 3);
          sc = make_uint2(__funnelshift_r(w.x, w.y, by), __funnelshift_r(w.y, w.z, by));
          if (blk + 8 > cb) {  // bytes of the next row
            const int have = (int)(cb - blk);
            sc.x &= have >= 4 ? 0xFFFFFFFFu : (1u << (8 * have)) - 1u;
            sc.y &= have <= 4 ? 0u : (1u << (8 * (have - 4))) - 1u;
          }
        }
        if (!__all_sync(0xFFFFFFFFu, lt_wait(tc_smem(&empty_a[st]), aph, vfail))) break;
        asm volatile("tcgen05.fence::after_thread_sync;");
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t w[16];
          lt_weights<BF>(*reinterpret_cast<const uint4 *>(src + ((j ^ sw) << 4)), (j < 2 ? sc.x : sc.y) >> (16 * (j & 1)), w);
          lt_st16(ta + 64u * P * st + 16u * j, w);
        }
        // the slot just read takes step i + D (its reads are ordered before the copy, which is another proxy's)
        if (p.tma) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (p.tma) {
          if (lane == 0) mbar_arrive(tc_smem(&ring_empty[slot]));
        } else {
          if (i + D < n) fetch(i + D);
          asm volatile("cp.async.commit_group;" ::: "memory");
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;");
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(tc_smem(&full_a[st]));
      advance(me, kLtGroups);
      if ((slot += kLtGroups) >= D) {
        slot -= D;
        rph ^= 1u;
      }
      if ((st += kLtGroups / P) >= SA) {
        st -= SA;
        aph ^= 1u;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // no copy outlives the CTA
  } else if (warp == kLtMmaWarp) {
    // ---- MMAs
    if (lt_elect()) {
      const uint32_t idesc = lt_idesc<BF>(nv);
      const uint64_t xd0 = tc_desc(base);
      int st = 0, sub = 0, sx = 0, last = 0, left = nr, in_tile = p.K - start.ks;
      uint32_t aph = 0u, xph = 0u, bph = 0u, last_ph = 0u;
      bool issued = false, ok = true;
#pragma unroll 1
      for (int seg = 0; seg < nseg && ok; ++seg) {
        const int b = NB == 2 ? seg & 1 : 0;
        // the accumulator must have been read back
        if (seg >= NB && !lt_wait(tc_smem(&acc_empty[b]), bph, vfail)) break;
        if (seg >= NB && b == NB - 1) bph ^= 1u;
        const uint32_t acc_t = tmem + (uint32_t)b * CAP;
        uint32_t acc = 0u;
        int steps = p.K;
        if (seg < nsh) {
          steps = min(left, in_tile);
          left -= steps;
          in_tile = p.K;
        }
#pragma unroll 1
        for (; steps > 0; --steps) {
          if (sub == 0) {
            const bool ready = !issued && p.first_tries >= 0 ? tc_wait_tries(tc_smem(&full_a[st]), 0u, vfail, p.first_tries)
                                                             : lt_wait(tc_smem(&full_a[st]), aph, vfail);
            if (!ready) {
              ok = false;
              break;
            }
          }
          const uint32_t a_t = tmem + C::kA + 64u * (P * st + sub);
#pragma unroll
          for (int h = 0; h < (C::kOne ? 1 : 2); ++h) {
            if (!C::kOne && !lt_wait(tc_smem(&full_x[sx]), xph, vfail)) {
              ok = false;
              break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;");
            const uint64_t xd = xd0 + (uint64_t)((C::kOne ? st * C::kXStage + sub * 2 * C::kAtom : sx * C::kXStage) >> 4);
#pragma unroll
            for (int kk = 0; kk < (C::kOne ? 8 : 4); ++kk) {
              asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                           "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                           ::"r"(acc_t), "r"(a_t + 8u * (4 * h + kk)),
                             "l"(xd + (uint64_t)(((kk >> 2) * C::kAtom + 32u * (kk & 3)) >> 4)), "r"(idesc), "r"(acc));
              acc = 1u;
            }
            if (!C::kOne) {
              asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                           ::"r"(tc_smem(&empty_x[sx])) : "memory");
              if (++sx == SX) {
                sx = 0;
                xph ^= 1u;
              }
            }
          }
          if (!ok) break;
          issued = true;
          if (++sub == P) {  // (a half-filled last stage has no next use)
            asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                         ::"r"(tc_smem(&empty_a[st])) : "memory");
            sub = 0;
            last = st;
            last_ph = aph;
            if (++st == SA) {
              st = 0;
              aph ^= 1u;
            }
          }
        }
        if (ok)
          asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                       ::"r"(tc_smem(&acc_full[b])) : "memory");
      }
      // after a failure: let the MMAs already issued finish before the CTA leaves
      if (*vfail && issued) {
        if (sub != 0) {  // the stage under way has no commit yet
          asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                       ::"r"(tc_smem(&empty_a[st])) : "memory");
          last = st;
          last_ph = aph;
        }
        tc_drain(tc_smem(&empty_a[last]), last_ph);
      }
    }
    __syncwarp();
  } else if (warp == kLtXWarp) {
    // ---- X by TMA
    if (lt_elect()) {
      if (!BF) pdl_wait();  // x in f16 is there
      const uint64_t tmap = reinterpret_cast<uint64_t>(&xmap);
      Place q = start;
      const int stages = C::kOne ? (n + P - 1) / P : 2 * n;
#pragma unroll 1
      for (int x = 0; x < stages; ++x) {
        const int sx = x % SX;
        if (x >= SX && !lt_wait(tc_smem(C::kOne ? &empty_a[sx] : &empty_x[sx]), (uint32_t)(((x - SX) / SX) & 1), vfail)) break;
        const uint32_t mb = tc_smem(C::kOne ? &full_a[sx] : &full_x[sx]);
        mbar_expect_tx(mb, (uint32_t)(H * nv) * 128u);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const int col = q.ks * kLtK + 64 * (C::kOne ? h & 1 : x & 1);
          asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                       " [%0], [%1, {%2, %3}], [%4];"
                       ::"r"(base + sx * C::kXStage + h * C::kAtom), "l"(tmap), "r"(col), "r"(0), "r"(mb) : "memory");
          if (C::kOne ? h & 1 : x & 1) advance(q, 1);
        }
        hi = x + 1;
      }
    }
    __syncwarp();
  } else if (warp == kLtCodeWarp) {
    // ---- codes and scales by TMA: step i into slot i % D
    if (p.tma && lt_elect()) {
      const uint64_t cm = reinterpret_cast<uint64_t>(&cmap), sm = reinterpret_cast<uint64_t>(&smap);
      Place q = start;
#pragma unroll 1
      for (int i = 0; i < n; ++i, advance(q, 1)) {
        const int slot = i % D;
        if (i >= D && !lt_wait(tc_smem(&ring_empty[slot]), (uint32_t)(((i - D) / D) & 1), vfail)) break;
        const uint32_t mb = tc_smem(&ring_full[slot]), dst = tc_smem(ring) + (uint32_t)slot * kLtSlot;
        mbar_expect_tx(mb, 8192u + 2048u);
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%2, %3}], [%4];"
                     ::"r"(dst), "l"(cm), "r"(q.ks * 64), "r"((int)(q.t * kLtM)), "r"(mb) : "memory");
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%2, %3}], [%4];"
                     ::"r"(dst + 8192u), "l"(sm), "r"((q.ks * 8) & ~15), "r"((int)(q.t * kLtM)), "r"(mb) : "memory");
        hi = i + 1;
      }
    }
    __syncwarp();
  }

  // Segment k of this CTA: its tile, whether it is the whole tile, its slot
  // (the first part of a tile in 2c + 1, the others in their CTAs' 2c).
  auto tile_of = [&](int k) { return k < nsh ? t_first + k : p.R + c + (k - nsh) * G; };
  auto whole = [&](int k) { return k >= nsh || ((t_first + k) * p.K >= g0 && (t_first + k + 1) * p.K <= g1); };
  auto slot_of = [&](int k) { return 2 * c + ((t_first + k) * p.K >= g0 ? 1 : 0); };
  auto unscale = [&](float v, int b) {
    if (BF) return v;
    const int up = s_up[b];
    return v * pow2(up / 2) * pow2(up - up / 2);
  };
  // Reads segment k's accumulator back, lanes 32 (warp % 4) .., the 16-column
  // pieces `first`, first + by, ...: to the outputs if the segment is its whole
  // tile, else to the workspace.  The next piece is on its way while one is
  // stored.
  auto read_back = [&](int k, int first, int by, float alpha) {
    const int q = warp & 3;
    const bool all = whole(k);
    const int64_t r = tile_of(k) * kLtM + 32 * q + lane;
    float *dst = p.part + (all ? 0 : slot_of(k) * a.batch * kLtM) + 32 * q + lane;
    const uint32_t tb = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(k % NB) * CAP;
    uint32_t v[16];
    if (16 * first < a.batch) tc_ld16(tb + 16u * first, v);
#pragma unroll 1
    for (int n0 = 16 * first; n0 < a.batch; n0 += 16 * by) {
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
      float w[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) w[u] = __uint_as_float(v[u]);
      if (n0 + 16 * by < a.batch) tc_ld16(tb + (uint32_t)(n0 + 16 * by), v);
      if (!all) {
#pragma unroll
        for (int u = 0; u < 16; ++u)
          if (n0 + u < a.batch) __stcg(dst + (int64_t)(n0 + u) * kLtM, w[u]);
      } else {
#pragma unroll
        for (int h = 0; h < 16; h += 8)
          if (n0 + h < a.batch && r < a.rows) {
            float x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = unscale(w[h + u], min(n0 + h + u, a.batch - 1));
            finish_row<8>(a, alpha, x, n0 + h, r);
          }
      }
    }
  };
  if (warp >= kLtEpiWarp0 && warp < kLtEpiWarp0 + 4) {
    // ---- every segment but the last
    if (!BF) {
      pdl_wait();
      for (int i = tid - kLtEpiWarp0 * 32; i < a.batch; i += 128) s_up[i] = (int16_t)__ldcg(p.up + i);
      asm volatile("bar.sync 1, 128;" ::: "memory");
    }
    const float alpha = *a.alpha;
#pragma unroll 1
    for (int k = 0; k + 1 < nseg; ++k) {
      const int b = k % NB;
      if (!__all_sync(0xFFFFFFFFu, tc_wait<500>(tc_smem(&acc_full[b]), (uint32_t)((k / NB) & 1), vfail))) break;
      asm volatile("tcgen05.fence::after_thread_sync;");
      read_back(k, 0, 1, alpha);
      asm volatile("tcgen05.fence::before_thread_sync;");
      __syncwarp();
      if (lane == 0) mbar_arrive(tc_smem(&acc_empty[b]));
    }
  }
  __syncthreads();
  // ---- the last segment: the producers have nothing left to do and help
  if (warp < kLtEpiWarp0 + 4) {
    const int k = nseg - 1, b = k % NB;
    if (__all_sync(0xFFFFFFFFu, lt_wait(tc_smem(&acc_full[b]), (uint32_t)((k / NB) & 1), vfail))) {
      asm volatile("tcgen05.fence::after_thread_sync;");
      read_back(k, warp >> 2, kLtEpiWarp0 / 4 + 1, *a.alpha);
    }
  }

  asm volatile("tcgen05.fence::before_thread_sync;");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;");
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  if (!BF) pdl_wait();
  if (*vfail) {
    // Copies that nothing has waited for land first, whichever role gave up
    // and when (a shared phase may never complete: then the bounded wait outlasts
    // the copy).
    if (warp == kLtXWarp)
      for (int x = max(0, hi - SX); x < hi; ++x) tc_drain(tc_smem(C::kOne ? &full_a[x % SX] : &full_x[x % SX]), (uint32_t)((x / SX) & 1));
    if (warp == kLtCodeWarp)
      for (int i = max(0, hi - D); i < hi; ++i) tc_drain(tc_smem(&ring_full[i % D]), (uint32_t)((i / D) & 1));
    // report the failure through every output of this CTA
    const float nan = __int_as_float(0x7FC00000);
    for (int k = 0; k < nseg; ++k)
      for (int i = tid; i < a.batch * kLtM; i += kLtThreads) {
        const int64_t r = tile_of(k) * kLtM + i % kLtM;
        if (!whole(k)) __stcg(p.part + slot_of(k) * a.batch * kLtM + i, nan);
        else if (r < a.rows)
          static_cast<__nv_bfloat16 *>(a.y)[(int64_t)(i / kLtM) * a.y_stride + r] = __float2bfloat16(nan);
      }
  }
}

// The parts of the shared tiles, added in CTA order and finished.
__global__ void __launch_bounds__(256) k_linear_join(const __grid_constant__ LtArgs p, int64_t GS) {
  pdl_wait();
  const int64_t T = p.R * p.K, per = (int64_t)p.a.batch * (kLtM / 8);
  const float alpha = *p.a.alpha;
  const bool vec = rows8_aligned(p.a);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.R * per; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / per;
    const int j = (int)(i - t * per), b = j / (kLtM / 8);
    const LtParts q = lt_parts(p, t, T, GS);
    if (q.n > 1) lt_join(p, alpha, vec, q, t, b, j % (kLtM / 8) * 8, p.up ? __ldg(p.up + b) : 0);
  }
}

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_lt_encode = nullptr;

struct LtPlan {
  int64_t tiles, K, G;
  bool bf;                     // bf16 operands
  size_t up, xf, part, bytes;  // offsets in the workspace, and its size
};

LtPlan lt_plan(int64_t rows, int64_t cols, int batch, int sms) {
  LtPlan p;
  p.tiles = (rows + kLtM - 1) / kLtM;
  p.K = (cols + kLtK - 1) / kLtK;
  // CTAs per tile: a step takes about max(0.2, 0.0021 N) us, adding one more
  // part of a tile about 0.0034 N us (its 512 N bytes go through one SM), so
  // K / parts steps and the parts cost least at sqrt(K step / part).
  const double step = std::max(0.2, 0.0021 * batch), part = 0.0034 * batch;
  const int64_t parts = std::max<int64_t>(1, (int64_t)(std::sqrt((double)p.K * step / part) + 0.5));
  p.G = std::min<int64_t>({p.tiles * p.K, sms, p.tiles * parts});
  p.bf = batch > 128 || p.tiles * p.K <= kLtBfSteps * p.G;
  p.up = 0;
  p.xf = p.up + kLinearSlice * sizeof(int);
  p.part = (p.xf + (p.bf ? 0 : (size_t)batch * cols * 2) + 255) / 256 * 256;
  p.bytes = p.part + 2 * (size_t)p.G * batch * kLtM * sizeof(float);
  return p;
}

bool lt_map(CUtensorMap *m, CUtensorMapDataType type, const void *ptr, uint64_t width, uint64_t height, uint64_t pitch,
            uint32_t box_w, uint32_t box_h, CUtensorMapSwizzle sw, CUtensorMapL2promotion promo) {
  const cuuint64_t dims[2] = {width, height}, strides[1] = {pitch};
  const cuuint32_t box[2] = {box_w, box_h}, es[2] = {1u, 1u};
  return g_lt_encode(m, type, 2, const_cast<void *>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, promo,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CAP, bool BF>
cudaError_t lt_launch(const CUtensorMap &xm, const CUtensorMap &cm, const CUtensorMap &sm, const LtArgs &p, int grid,
                      cudaStream_t st) {
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kLtThreads);
  cfg.dynamicSmemBytes = LtCfg<CAP>::kSmem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = BF ? 0 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_linear_tc<CAP, BF>, xm, cm, sm, p);
  if (e != cudaSuccess || p.R == 0) return e;
  cfg.gridDim = dim3((unsigned)std::min<int64_t>((p.R * p.a.batch * (kLtM / 8) + 255) / 256, 1 << 20));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_linear_join, p, lt_sharers(p, grid));
}

template <int CAP, bool BF>
cudaError_t lt_prepare() {
  return cudaFuncSetAttribute(k_linear_tc<CAP, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)LtCfg<CAP>::kSmem);
}

}  // namespace

size_t linear_tc_workspace_bytes(int64_t rows, int64_t cols, int batch, int sms) {
  return lt_plan(rows, cols, batch, sms).bytes;
}

cudaError_t launch_linear_tc(const LinearArgs &a, int sms, void *ws, int first_tries, LinearKernel *took, cudaStream_t st) {
  if (!g_lt_encode) return cudaErrorInitializationError;
  if (a.cols >= (int64_t(1) << 31)) return cudaErrorInvalidValue;  // a TMA coordinate
  const LtPlan q = lt_plan(a.rows, a.cols, a.batch, sms);
  *took = q.bf ? kLinearTcBf16 : kLinearTcF16;
  char *w = static_cast<char *>(ws);
  const int64_t whole = q.tiles / q.G;
  if (whole * q.K >= (int64_t(1) << 30)) return cudaErrorInvalidValue;  // steps of a CTA
  LtArgs p = {a, (int)q.K, q.tiles - whole * q.G, (int)whole, q.bf ? nullptr : reinterpret_cast<int *>(w + q.up),
              reinterpret_cast<float *>(w + q.part), 0,
              a.cols % 32 == 0 && reinterpret_cast<uintptr_t>(a.codes) % 16 == 0, first_tries};
  const int nv = (a.batch + 15) & ~15;
  CUtensorMap xm, cm, sm;
  if (!(q.bf ? lt_map(&xm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.cols, a.batch, a.x_stride * 2, 64u, nv,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B)
             : lt_map(&xm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, w + q.xf, a.cols, a.batch, a.cols * 2, 64u, nv,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B)))
    return cudaErrorInvalidValue;
  memset(&cm, 0, sizeof(cm));
  memset(&sm, 0, sizeof(sm));
  p.tma = a.cols % 256 == 0 && a.rows < (int64_t(1) << 31) && reinterpret_cast<uintptr_t>(a.codes) % 16 == 0 &&
          reinterpret_cast<uintptr_t>(a.scales) % 16 == 0 &&
          lt_map(&cm, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.codes, a.cols / 2, a.rows, a.cols / 2, 64u, kLtM,
                 CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B) &&
          lt_map(&sm, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.scales, a.cols / 16, a.rows, a.cols / 16, 16u, kLtM,
                 CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
  const int grid = (int)q.G;
  if (q.bf)
    return a.batch <= 64 ? lt_launch<64, true>(xm, cm, sm, p, grid, st)
                         : a.batch <= 128 ? lt_launch<128, true>(xm, cm, sm, p, grid, st) : lt_launch<256, true>(xm, cm, sm, p, grid, st);
  k_linear_x<<<a.batch, kLxThreads, 0, st>>>(static_cast<const uint4 *>(a.x), a.x_stride / 8, a.cols / 8,
                                             reinterpret_cast<uint4 *>(w + q.xf), reinterpret_cast<int *>(w + q.up));
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return a.batch <= 64 ? lt_launch<64, false>(xm, cm, sm, p, grid, st) : lt_launch<128, false>(xm, cm, sm, p, grid, st);
}

cudaError_t prepare_linear_tc_kernels() {
  if (!g_lt_encode) {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorSymbolNotFound;
    g_lt_encode = reinterpret_cast<EncodeTiledFn>(fn);
  }
  cudaError_t e = lt_prepare<64, false>();
  if (e == cudaSuccess) e = lt_prepare<64, true>();
  if (e == cudaSuccess) e = lt_prepare<128, false>();
  if (e == cudaSuccess) e = lt_prepare<128, true>();
  if (e == cudaSuccess) e = lt_prepare<256, true>();
  return e;
}

}  // namespace nvfp4
