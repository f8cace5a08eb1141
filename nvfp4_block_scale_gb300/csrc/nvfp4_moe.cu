// nvfp4_moe.cu -- the experts' products of a mixture-of-experts layer for a few
// tokens, on NVFP4 weights:
//   h[t,s] = act(alpha_g sum_c q Delta x[t][c]) * (alpha_u sum_c q Delta x[t][c]),  expert ids[t][s]
//   y[t]   = bf16( residual[t] + sum_s weights[t][s] alpha_d sum_j q Delta h[t,s][j] ).
//
// Bound: reading once the weights of every expert that some token names
// (0.5625 B each); a token's share of x, h and y is small beside them.
//
// Three launches, each waiting for the one before through a programmatic
// dependency: gate and up with the activation (h, fp32, to the workspace), down
// (each slot's product, fp32, to the workspace), and the sum over a token's
// slots in slot order.  No atomics take part in a sum and no CTA waits for
// another, so a workspace may hold anything and results repeat bit for bit.
//
// Jobs: every CTA sorts the call's (token, slot) pairs by expert in shared
// memory; an expert with n pairs makes ceil(n / N) jobs of up to N pairs.  The
// row tiles of all jobs, job after job, are cut into one contiguous range per
// SM, and the (tile, column step) units of a range's part of one job into 16
// contiguous runs, one per warp.  A warp that does a whole tile finishes it
// from its registers; sums of a tile cut between warps meet in shared memory, in
// warp order.  Loads run kMoeDepth units ahead, across jobs.
//
// Products: mma.sync m16n8k16 (f16 x f16 -> fp32), 16 rows of W by 8 pairs.
// q * Delta is formed in registers, exactly: six significant bits between 2^-10
// and 2688.  The vectors go to f16 in shared memory, each scaled by a power of
// two that puts its largest entry into [2^14, 2^15): x keeps its 8 bits down to
// 2^-31 of its largest entry; h, fp32 until then, is rounded to 11 bits, an
// eighth of what bf16 would lose.  With a gate the 16 rows are 8 of the gate's
// and the 8 of up's that they multiply, so that h is formed in registers.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"
#include "nvfp4_epilogue.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {

constexpr int kMoeWarps = 16;
constexpr int kMoeThreads = kMoeWarps * 32;
constexpr int kMoeDepth = 4;            // steps in flight per warp
constexpr int kMoeSmem = 226 * 1024;    // dynamic shared memory of the one CTA per SM

struct MoeLaunch {
  MoeArgs a;
  float *h, *part;    // [pairs][inner], [pairs][hidden]
  int pairs;          // tokens * top_k
  int group;          // pairs of a job at most
  int steps;          // of 128 columns
  int tiles;          // of a job
  int64_t cols;       // of this launch's matrices
};

// One step of a lane: 32 columns (two blocks) of its two rows.
struct MoeLoad {
  uint4 c[2];
  uint32_t s[2];
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight consecutive entries of a vector, as fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
  const uint4 r = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 r = reinterpret_cast<const float4 *>(p)[i];
    v[4 * i] = r.x, v[4 * i + 1] = r.y, v[4 * i + 2] = r.z, v[4 * i + 3] = r.w;
  }
}

// Shared memory besides the vectors: the plan, and a partial sum per warp.
__host__ __device__ constexpr int64_t moe_fixed_smem(int experts, int pairs, int nt) {
  return (int64_t)experts * 8 + (int64_t)pairs * 8 + 512 + (int64_t)kMoeWarps * nt * 512 + 128;
}

// DOWN: the second product (h -> part), else the first (x -> h).  GATED: the
// first product's tiles hold 8 rows of gate and 8 of up.  WIDE: rows of codes
// are whole multiples of 16 bytes and of scales of 2, and so aligned; otherwise
// a block at a time.
template <int NT, bool DOWN, bool GATED, bool WIDE>
__global__ void __launch_bounds__(kMoeThreads, 1) k_moe(const __grid_constant__ MoeLaunch p) {
  extern __shared__ uint4 dsm[];
  __shared__ int scan[2][kMoeWarps];
  const MoeArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cq = lane & 3;
  const int nk = p.steps, N = p.group;
  uint4 *xs = dsm;                                                        // [nk][4][N][4] 16-byte units of f16
  float4 *own = reinterpret_cast<float4 *>(dsm + (size_t)nk * 16 * N);    // [warps][NT][32]
  float *xdown = reinterpret_cast<float *>(own + kMoeWarps * NT * 32);    // [2][32]: the vectors' scales, undone
  unsigned *xmax = reinterpret_cast<unsigned *>(xdown + 64);              // [2][32]: their largest entries
  int *count = reinterpret_cast<int *>(xmax + 64);                        // [experts]
  int *end = count + a.experts;                                           // [experts]: where its pairs end in `order`
  uint32_t *jobs = reinterpret_cast<uint32_t *>(end + a.experts);       // [jobs]: expert << 16 | group
  uint16_t *order = reinterpret_cast<uint16_t *>(jobs + p.pairs);         // [pairs], by expert
  uint16_t *found = order + p.pairs;                                      // [pairs], by expert, as they came

  for (int e = tid; e < a.experts; e += kMoeThreads) count[e] = 0;
  if (tid < 64) xmax[tid] = 0u;
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();

  // ---- the plan: pairs by expert, jobs
  for (int i = tid; i < p.pairs; i += kMoeThreads) {
    const int e = a.ids[i];
    if (e >= 0 && e < a.experts) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  int total = 0, named = 0;  // jobs; pairs that have an expert
  {
    for (int e0 = 0; e0 < a.experts; e0 += kMoeThreads) {
      const int e = e0 + tid, n = e < a.experts ? count[e] : 0, j = (n + N - 1) / N;
      int sn = n, sj = j;  // inclusive sums over the warp, then over the warps
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int un = __shfl_up_sync(~0u, sn, o), uj = __shfl_up_sync(~0u, sj, o);
        if (lane >= o) sn += un, sj += uj;
      }
      if (lane == 31) scan[0][warp] = sn, scan[1][warp] = sj;
      __syncthreads();
      int bn = named, bj = total;
#pragma unroll
      for (int w = 0; w < kMoeWarps; ++w) {
        const int wn = scan[0][w], wj = scan[1][w];
        if (w < warp) bn += wn, bj += wj;
        named += wn, total += wj;
      }
      if (e < a.experts) {
        end[e] = bn + sn - n;  // (its first pair, until they are put in order)
        for (int i = 0; i < j; ++i) jobs[bj + sj - j + i] = (uint32_t)e << 16 | (uint32_t)i;
      }
      __syncthreads();
    }
  }
  const int64_t tiles = (int64_t)total * p.tiles;
  const int64_t T0 = blockIdx.x * tiles / gridDim.x, T1 = (blockIdx.x + 1) * tiles / gridDim.x;
  if (T0 == T1) return;
  const int j0 = (int)(T0 / p.tiles), j1 = (int)((T1 - 1) / p.tiles);
  // Pairs by expert, ascending inside an expert that has several jobs: every CTA
  // has to cut it alike.  (In one job a pair's place only decides which column of
  // an MMA it takes.)
  for (int i = tid; i < p.pairs; i += kMoeThreads) {
    const int e = a.ids[i];
    if (e >= 0 && e < a.experts) found[atomicAdd(&end[e], 1)] = (uint16_t)i;
  }
  __syncthreads();
  for (int q = tid; q < named; q += kMoeThreads) {
    const int i = found[q], e = a.ids[i], n = count[e], b = end[e] - n;
    int to = q;
    if (n > N) {
      to = b;
      for (int o = b; o < b + n; ++o) to += found[o] < i;
    }
    order[to] = (uint16_t)i;
  }
  __syncthreads();

  // ---- this warp's units: its run of the range's part of each job
  struct Run {
    int t0, u0, u1;  // the part's first tile; the warp's units, counted from there
  };
  auto run_of = [&](int j, int w) {
    const int t0 = j == j0 ? (int)(T0 - (int64_t)j0 * p.tiles) : 0;
    const int units = ((j == j1 ? (int)(T1 - (int64_t)j1 * p.tiles) : p.tiles) - t0) * nk;
    return Run{t0, w * units / kMoeWarps, (w + 1) * units / kMoeWarps};
  };
  const int64_t nblk = p.cols / 16, tile_blk = (GATED && !DOWN ? 8 : 16) * nblk;  // blocks of a row, between tiles
  int fj = j0 - 1, fk = 0, fleft = 0;  // next unit to load: its job, its step; units left of the run
  const uint8_t *fc[2], *fs[2];        // its rows' codes and scales
  fc[0] = fc[1] = fs[0] = fs[1] = nullptr;
  auto fetch = [&](MoeLoad &d) {  // (nothing once the range's units are loaded)
    while (fleft == 0) {
      if (fj == j1) return;
      const Run r = run_of(++fj, warp);
      fleft = r.u1 - r.u0;
      if (fleft == 0) continue;
      const int e = (int)(jobs[fj] >> 16), t = r.t0 + r.u0 / nk;
      fk = r.u0 % nk;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const MoeMatrix &m = DOWN ? a.down : GATED && h == 0 ? a.gate : a.up;
        const int64_t row = GATED && !DOWN ? (int64_t)t * 8 + g : (int64_t)t * 16 + 8 * h + g;
        fc[h] = m.codes + e * m.code_stride + row * nblk * 8;
        fs[h] = m.scales + e * m.scale_stride + row * nblk;
      }
    }
    // columns past the end read the last blocks: the vectors are zero there
    const int blk = fk * 8 + 2 * cq;
    if (WIDE) {
      const int64_t at = min((int64_t)blk, nblk - 2);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        d.c[h] = __ldcs(reinterpret_cast<const uint4 *>(fc[h] + 8 * at));
        d.s[h] = __ldg(reinterpret_cast<const uint16_t *>(fs[h] + at));
      }
    } else {
      const int64_t at = min((int64_t)blk, nblk - 1), at1 = min((int64_t)blk + 1, nblk - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 lo = __ldcs(reinterpret_cast<const uint2 *>(fc[h]) + at), hi = __ldcs(reinterpret_cast<const uint2 *>(fc[h]) + at1);
        d.c[h] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        d.s[h] = (uint32_t)__ldg(fs[h] + at) | (uint32_t)__ldg(fs[h] + at1) << 8;
      }
    }
    --fleft;
    if (++fk == nk) {
      fk = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) fc[h] += 8 * tile_blk, fs[h] += tile_blk;
    }
  };
  MoeLoad buf[kMoeDepth];
#pragma unroll
  for (int i = 0; i < kMoeDepth; ++i) fetch(buf[i]);

  // ---- the jobs.  xmax and xdown alternate between two places: a warp may
  // still finish a job's sums while others take in the next one's vectors.
  int par = 0, turn = 0;  // turn: the buffer that holds the next unit
  for (int j = j0; j <= j1; ++j, par ^= 1) {
    const int e = (int)(jobs[j] >> 16), at0 = end[e] - count[e] + (int)(jobs[j] & 0xFFFFu) * N;
    const int np = min(N, end[e] - at0);  // pairs of this job
    const uint16_t *pair = order + at0;

    // vectors into shared memory, 8 columns at a time: first the largest entry
    // of each, then (from L1 or L2) the scaled f16.  A vector's columns are
    // shared by several warps where there are fewer vectors than warps.
    const int nu = nk * 16, wide = (int)(p.cols / 8);
    const int share = kMoeWarps / np > 0 ? kMoeWarps / np : 1;
    auto vector = [&](int n) {
      const int i = pair[n];
      if constexpr (DOWN) return (const float *)p.h + (int64_t)i * p.cols;
      else return static_cast<const __nv_bfloat16 *>(a.x) + (int64_t)(i / a.top_k) * a.x_stride;
    };
    for (int i = warp; i < np * share; i += kMoeWarps) {
      const int n = i / share, s = i - n * share;
      const auto *v = vector(n);
      float top = 0.0f;
      bool nan = false;
      for (int u = s * 32 + lane; u < wide; u += share * 32) {
        float x[8];
        load8(v + 8 * u, x);
#pragma unroll
        for (int b = 0; b < 8; ++b) top = fmaxf(top, fabsf(x[b])), nan |= x[b] != x[b];
      }
      const unsigned m = __reduce_max_sync(~0u, nan ? 0x7F800000u : __float_as_uint(top));
      if (lane == 0) atomicMax(&xmax[par * 32 + n], m);
    }
    __syncthreads();
    for (int i = warp; i < np * share; i += kMoeWarps) {
      const int n = i / share, s = i - n * share;
      const auto *v = vector(n);
      const int up = min(14 + 127 - (int)(xmax[par * 32 + n] >> 23), 126);
      if (s == 0 && lane == 0) xdown[par * 32 + n] = pow2(-up);
      for (int u = s * 32 + lane; u < nu; u += share * 32) {
        uint4 o = make_uint4(0u, 0u, 0u, 0u);
        if (u < wide) {
          float x[8];
          load8(v + 8 * u, x);
          uint32_t w[4];
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const __half2 f = __floats2half2_rn(x[2 * b] * pow2(up), x[2 * b + 1] * pow2(up));
            w[b] = *reinterpret_cast<const uint32_t *>(&f);
          }
          o = make_uint4(w[0], w[1], w[2], w[3]);
        }
        // unit u: step u / 16, lane quarter (u / 4) % 4, pair of k-steps u % 4
        xs[(((u >> 4) * 4 + (u & 3)) * N + n) * 4 + ((u >> 2) & 3)] = o;
      }
    }
    if (tid < 32) xmax[(par ^ 1) * 32 + tid] = 0u;
    __syncthreads();

    // ---- the run
    const Run r = run_of(j, warp);
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
    // a tile's finished sums
    auto finish_tile = [&](int t) {
      float av = 0.0f, ag = 0.0f;  // (read here: once per tile, from L1)
      if constexpr (DOWN) av = a.down.alpha[e * a.down.alpha_stride];
      else av = a.up.alpha[e * a.up.alpha_stride];
      if constexpr (GATED && !DOWN) ag = a.gate.alpha[e * a.gate.alpha_stride];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int n0 = 8 * nt + 2 * cq;
        if (n0 >= np) continue;
        const bool two = n0 + 1 < np;
        const int p0 = pair[n0], p1 = pair[two ? n0 + 1 : n0];
        const float d0 = xdown[par * 32 + n0], d1 = xdown[par * 32 + (two ? n0 + 1 : n0)];
        if constexpr (DOWN) {
          float *q = p.part + (int64_t)t * 16 + g;
          q[p0 * a.hidden] = acc[nt][0] * av * d0;
          q[p0 * a.hidden + 8] = acc[nt][2] * av * d0;
          if (two) {
            q[p1 * a.hidden] = acc[nt][1] * av * d1;
            q[p1 * a.hidden + 8] = acc[nt][3] * av * d1;
          }
        } else if constexpr (GATED) {
          float v[2] = {acc[nt][0] * ag * d0, acc[nt][1] * ag * d1};
          activate(v, a.act);
          float *q = p.h + (int64_t)t * 8 + g;
          q[p0 * a.inner] = v[0] * (acc[nt][2] * av * d0);
          if (two) q[p1 * a.inner] = v[1] * (acc[nt][3] * av * d1);
        } else {
          float v[4] = {acc[nt][0] * av * d0, acc[nt][1] * av * d1, acc[nt][2] * av * d0, acc[nt][3] * av * d1};
          activate(v, a.act);
          float *q = p.h + (int64_t)t * 16 + g;
          q[p0 * a.inner] = v[0];
          q[p0 * a.inner + 8] = v[2];
          if (two) {
            q[p1 * a.inner] = v[1];
            q[p1 * a.inner + 8] = v[3];
          }
        }
      }
    };
    int ct = r.u0 / nk, ck = r.u0 - ct * nk;  // counted from the part's first tile
    bool mine = ck == 0;  // this warp takes the current tile's first step
    const uint4 *xl[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xl[nt] = xs + min(8 * nt + g, np - 1) * 4 + cq;
    auto unit = [&](MoeLoad &d) {
      uint32_t sc[2][2];  // f16 pairs {Delta, Delta} of the lane's two blocks, of both rows
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t f;
        asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(f) : "r"(d.s[h]));
        sc[h][0] = __byte_perm(f, 0u, 0x1010);
        sc[h][1] = __byte_perm(f, 0u, 0x3232);
      }
      const uint32_t cw[2][4] = {{d.c[0].x, d.c[0].y, d.c[0].z, d.c[0].w}, {d.c[1].x, d.c[1].y, d.c[1].z, d.c[1].w}};
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {  // a word of codes: 8 columns, two k-steps
        uint32_t w[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          e2m1x8_f16(cw[h][jj], w[h]);
#pragma unroll
          for (int b = 0; b < 4; ++b) w[h][b] = mul_f16x2(w[h][b], sc[h][jj >> 1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (nt > 0 && 8 * nt >= np) break;
          const uint4 xb = xl[nt][(ck * 4 + jj) * (4 * N)];
          mma_f16(acc[nt], w[0][0], w[1][0], w[0][1], w[1][1], xb.x, xb.y);
          mma_f16(acc[nt], w[0][2], w[1][2], w[0][3], w[1][3], xb.z, xb.w);
        }
      }
      fetch(d);
      if (++ck == nk) {  // the tile's last step
        if (mine) {
          finish_tile(r.t0 + ct);
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) own[(warp * NT + nt) * 32 + lane] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
        ck = 0;
        ++ct;
        mine = true;
      }
    };
    // the buffers take turns: this run begins with the one that follows the last run's last
    int left = r.u1 - r.u0;
    while (left > 0) {
#pragma unroll
      for (int i = 0; i < kMoeDepth; ++i)
        if (left > 0 && turn == i) {
          unit(buf[i]);
          --left;
          turn = (i + 1) % kMoeDepth;
        }
    }
    if (ck > 0 && r.u1 > r.u0 && !mine) {  // the run lies inside a tile
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) own[(warp * NT + nt) * 32 + lane] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
    }
    __syncthreads();
    if (ck > 0 && r.u1 > r.u0 && mine) {  // the run ends inside a tile that it began: the next warps have the rest
      for (int w = warp + 1; w < kMoeWarps; ++w) {
        const Run o = run_of(j, w);
        if (o.u0 >= (ct + 1) * nk) break;
        if (o.u0 == o.u1) continue;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float4 v = own[(w * NT + nt) * 32 + lane];
          acc[nt][0] += v.x, acc[nt][1] += v.y, acc[nt][2] += v.z, acc[nt][3] += v.w;
        }
      }
      finish_tile(r.t0 + ct);
    }
  }
}

// y = residual + the sum of a token's slots, in slot order; four columns a thread.
__global__ void __launch_bounds__(256) k_moe_join(const __grid_constant__ MoeLaunch p) {
  const MoeArgs &a = p.a;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t quads = a.hidden / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads * a.tokens) return;
  const int64_t t = i / quads, c = (i - t * quads) * 4;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < a.top_k; ++s) {
    const int64_t at = t * a.top_k + s;
    const int e = a.ids[at];
    if (e < 0 || e >= a.experts) continue;
    const float w = a.weights[at];
    const float4 o = *reinterpret_cast<const float4 *>(p.part + at * a.hidden + c);
    v[0] = fmaf(w, o.x, v[0]), v[1] = fmaf(w, o.y, v[1]), v[2] = fmaf(w, o.z, v[2]), v[3] = fmaf(w, o.w, v[3]);
  }
  const __nv_bfloat16 *res = static_cast<const __nv_bfloat16 *>(a.residual);
  if (res) {
    __nv_bfloat16 rv[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) rv[b] = res[t * a.residual_stride + c + b];
#pragma unroll
    for (int b = 0; b < 4; ++b) v[b] += __bfloat162float(rv[b]);
  }
  __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y) + t * a.y_stride + c;
#pragma unroll
  for (int b = 0; b < 4; ++b) y[b] = __float2bfloat16(v[b]);
}

namespace {

// Pairs of a job: as many as the vectors' room in shared memory allows, up to
// 32 (four n-tiles of accumulators), no more than the call has.
int moe_group(int64_t cols, int experts, int pairs) {
  for (int n = std::min(pairs, 32); n > 0; --n) {
    const int nt = n <= 8 ? 1 : n <= 16 ? 2 : 4;
    if ((cols + 127) / 128 * 256 * n + moe_fixed_smem(experts, pairs, nt) <= kMoeSmem) return n;
  }
  return 0;
}

template <typename F>
auto with_kernel(int nt, bool down, bool gated, bool wide, F f) {
  auto pick_wide = [&](auto w, auto n) {
    constexpr bool W = decltype(w)::value;
    constexpr int N = decltype(n)::value;
    return down ? f(k_moe<N, true, false, W>) : gated ? f(k_moe<N, false, true, W>) : f(k_moe<N, false, false, W>);
  };
  auto pick_nt = [&](auto w) {
    return nt == 1 ? pick_wide(w, std::integral_constant<int, 1>()) : nt == 2 ? pick_wide(w, std::integral_constant<int, 2>())
                                                                             : pick_wide(w, std::integral_constant<int, 4>());
  };
  return wide ? pick_nt(std::true_type()) : pick_nt(std::false_type());
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
  p.steps = (int)((p.cols + 127) / 128);
  p.tiles = (int)(down ? a.hidden / 16 : a.gated ? a.inner / 8 : a.inner / 16);
  p.group = moe_group(p.cols, a.experts, p.pairs);
  const int nt = p.group <= 8 ? 1 : p.group <= 16 ? 2 : 4;
  const size_t smem = (size_t)p.steps * 256 * p.group + moe_fixed_smem(a.experts, p.pairs, nt);
  auto wide_matrix = [&](const MoeMatrix &m) {
    return ((reinterpret_cast<uintptr_t>(m.codes) | m.code_stride) % 16 | (reinterpret_cast<uintptr_t>(m.scales) | m.scale_stride) % 2) == 0;
  };
  const bool wide = p.cols % 32 == 0 && (down ? wide_matrix(a.down) : wide_matrix(a.up) && (!a.gated || wide_matrix(a.gate)));
  return with_kernel(nt, down, a.gated, wide, [&](auto *k) { return launch_dependent(k, sms, kMoeThreads, smem, p, st); });
}

size_t moe_h_bytes(int64_t inner, int pairs) { return ((size_t)pairs * inner * 4 + 255) / 256 * 256; }

}  // namespace

bool moe_fits(int64_t hidden, int64_t inner, int experts, int pairs) {
  return moe_group(hidden, experts, pairs) > 0 && moe_group(inner, experts, pairs) > 0;
}

size_t moe_workspace_bytes(int64_t hidden, int64_t inner, int pairs) {
  return moe_h_bytes(inner, pairs) + (size_t)pairs * hidden * 4;
}

cudaError_t launch_moe(const MoeArgs &a, int sms, void *ws, cudaStream_t st) {
  MoeLaunch p = {};
  p.a = a;
  p.pairs = a.tokens * a.top_k;
  p.h = static_cast<float *>(ws);
  p.part = reinterpret_cast<float *>(static_cast<char *>(ws) + moe_h_bytes(a.inner, p.pairs));
  cudaError_t e = launch_product(p, false, sms, st);
  if (e == cudaSuccess) e = launch_product(p, true, sms, st);
  if (e != cudaSuccess) return e;
  return launch_dependent(k_moe_join, (int)((a.hidden / 4 * a.tokens + 255) / 256), 256, 0, p, st);
}

cudaError_t prepare_moe_kernels() {
  cudaError_t e = cudaSuccess;
  for (int nt : {1, 2, 4})
    for (int form : {0, 1, 2})
      for (bool wide : {false, true})
        if (e == cudaSuccess)
          e = with_kernel(nt, form == 2, form == 1, wide,
                          [](auto *k) { return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoeSmem); });
  return e;
}

}  // namespace nvfp4
