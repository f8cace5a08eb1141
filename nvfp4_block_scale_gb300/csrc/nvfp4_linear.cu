// nvfp4_linear.cu -- the W4A16 product with its epilogue:
//   y[b][r] = bf16( residual + gate * act( alpha * sum_c q Delta x[b][c] + bias ) ).
//
// Many vectors and large tensors go to the tcgen05 product
// (nvfp4_linear_tc.cu).  The others are bound by latency, then by reading the
// weights once (0.5625 B each), and run here, without tensor memory (1 vector
// 4096 x 4096: 8.3 us, 1.1 TB/s, 10.0 with cold weights; 2048 x 8192: 7.9 and 9.1; 8
// vectors 4096 x 6144: 10.3 and 12.7; a second launch in a stream costs 1 to 2 us of
// these, the first bytes' way from HBM and a CTA's set-up another 3):
//
// Products: mma.sync m16n8k16 (bf16 x bf16 -> fp32), 16 rows of W by 8 vectors.
// q * Delta is formed in registers, exactly: six significant bits between
// 2^-10 and 2688, in f16 first (two instructions per pair), then bf16 (three
// more), so that x is used as it is.
//
// Work split: a CTA owns a rectangle of W, `tiles` row tiles of 16 by `steps`
// column steps of 128, and keeps x for its columns in shared memory in the
// order in which the MMAs read it.  The rectangle's (tile, step) units, tile
// by tile, are cut into eight contiguous runs of equal length, one per warp,
// so no warp waits for another until the end.  A warp's sums of a tile go to
// shared memory: to the tile's place if the warp took the tile's first step,
// else (its run began inside the tile) to a place of the warp's own; after one
// barrier they are added in warp order.  The sums of rectangles that share rows
// meet in the workspace, where a second launch adds them in column order.
//
// Loads: a lane takes 16 consecutive code bytes (32 columns) of two rows per
// step, kLinDepth steps ahead, straight into registers.  The order of the
// columns inside a step is permuted alike on both sides, so that those bytes
// feed the MMAs without a shuffle.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"
#include "nvfp4_epilogue.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {

// This kernel takes up to 16 vectors, and W up to so many blocks of 16 x 128
// per CTA of a full wave.  Measured against the tcgen05 product (us): 1 vector
// 4096 x 4096 (27 blocks) 9.0 against 12.1, 8192 x 4096 (54) 13.0 against 13.9,
// 14336 x 4096 (94) 17.9 against 17.6; 8 vectors 4096 x 11008 (72) 16.3 against
// 16.2; 16 vectors 2048 x 4096 (13) 9.0 against 11.0, 4096 x 6144 (40) 13.3 either
// way, 8192 x 4096 14.8 against 14.2.
constexpr int kLinVecs = 16, kLinBlocks8 = 72, kLinBlocks16 = 40;
constexpr int kLinWarps = 8;
constexpr int kLinThreads = kLinWarps * 32;
constexpr int kLinDepth = 4;       // steps in flight per warp
constexpr int kLinSmem = 88 * 1024;  // dynamic shared memory of one of two CTAs per SM

// Shared memory of a rectangle: x, the tiles' sums, the warps' own.
__host__ __device__ constexpr int64_t lin_smem(int nt, int64_t steps, int64_t tiles) {
  return steps * nt * 2048 + (tiles + kLinWarps) * nt * 512;
}

struct LinPlan {
  int steps, tiles;         // of W
  int ranges, groups;       // column ranges, row groups
  int max_steps, max_tiles; // of a rectangle
};

struct LinLaunch {
  LinearArgs a;
  LinPlan p;
  float4 *part;     // [ranges][tiles][NT][32]: sums in the MMA's lane order
  int min_steps, long_ranges, min_tiles, long_groups;  // steps = min_steps * ranges + long_ranges, tiles likewise
};

// One step of a lane: 32 columns (two blocks) of rows g and g + 8.
struct LinLoad {
  uint4 c[2];
  uint32_t s[2];
};

// f16 pair -> bf16 pair (exact for six significant bits).
__device__ __forceinline__ uint32_t f16x2_bf16x2(uint32_t v) {
  const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&v));
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x.y), "f"(x.x));
  return r;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The finished sums of one lane's fragment: rows g, g + 8 of a tile, vectors 8 nt + 2 cq + {0, 1}.
__device__ __forceinline__ void finish4(const LinearArgs &a, float alpha, int64_t tile, int nt, int lane, const float4 &v) {
  const float w[4] = {v.x, v.y, v.z, v.w};
  auto b = [&](int j) { return (int64_t)(8 * nt + 2 * (lane & 3) + (j & 1)); };
  auto r = [&](int j) { return tile * 16 + 8 * (j >> 1) + (lane >> 2); };
  finish<4>(a, alpha, w, [&](int j) { return b(j) < a.batch && r(j) < a.rows; }, b, r);
}

// WIDE: rows of codes are whole multiples of 16 bytes and of scales of 2, and
// so aligned; otherwise a block at a time.
template <int NT, bool WIDE>
__global__ void __launch_bounds__(kLinThreads, 2) k_linear(const __grid_constant__ LinLaunch p) {
  constexpr int N = 8 * NT;
  extern __shared__ uint4 dsm[];
  const LinearArgs &a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cq = lane & 3;
  pdl_launch_dependents();  // k_linear_sum waits for the whole grid all the same
  // the first (steps mod ranges) ranges and (tiles mod groups) groups are one longer
  const int group = blockIdx.x / (uint32_t)p.p.ranges, range = blockIdx.x - group * p.p.ranges;
  const int nk = p.min_steps + (range < p.long_ranges), k0 = range * p.min_steps + min(range, p.long_ranges);
  const int ntile = p.min_tiles + (group < p.long_groups), t0 = group * p.min_tiles + min(group, p.long_groups);
  uint4 *xs = dsm;                                                              // [nk][4][N][4] 16-byte units
  float4 *sums = reinterpret_cast<float4 *>(dsm + (size_t)p.p.max_steps * NT * 128);  // [tiles][NT][32], then [warps][NT][32]
  float4 *own = sums + p.p.max_tiles * NT * 32;

  // ---- this warp's run of units and its first loads.  Rows and columns past
  // the end read the last ones: those rows are not written, and x is zero there.
  const int units = ntile * nk;  // (a CTA's rectangle fits its shared memory: 8 units is far below 2^31)
  const int u0 = warp * units / kLinWarps, u1 = (warp + 1) * units / kLinWarps;
  const int64_t nblk = a.cols / 16;
  int ft = u0 / nk, fk = u0 - ft * nk;  // next unit to load
  const uint8_t *fc[2], *fs[2];         // its rows' codes and scales, from the lane's first column
  const int last = (int)min(nblk - 1, (int64_t)INT32_MAX);
  auto rows_of = [&](int t) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t row = min((int64_t)(t0 + t) * 16 + 8 * h + g, a.rows - 1);
      fc[h] = a.codes + row * nblk * 8;
      fs[h] = a.scales + row * nblk;
    }
  };
  rows_of(ft);
  auto fetch = [&](LinLoad &d) {
    const int blk = (k0 + fk) * 8 + 2 * cq;
    if (WIDE) {
      const int64_t at = min(blk, last - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        d.c[h] = __ldcs(reinterpret_cast<const uint4 *>(fc[h] + 8 * at));
        d.s[h] = __ldg(reinterpret_cast<const uint16_t *>(fs[h] + at));
      }
    } else {
      const int64_t at = min(blk, last), at1 = min(blk + 1, last);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 lo = __ldcs(reinterpret_cast<const uint2 *>(fc[h]) + at), hi = __ldcs(reinterpret_cast<const uint2 *>(fc[h]) + at1);
        d.c[h] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        d.s[h] = (uint32_t)__ldg(fs[h] + at) | (uint32_t)__ldg(fs[h] + at1) << 8;
      }
    }
    if (++fk == nk) {
      fk = 0;
      rows_of(++ft);
    }
  };
  LinLoad buf[kLinDepth];
  int ahead = u0;  // units loaded
#pragma unroll
  for (int i = 0; i < kLinDepth; ++i)
    if (ahead < u1) {
      fetch(buf[i]);
      ++ahead;
    }

  // ---- x into shared memory, 16 bytes (8 columns) at a time; zeros past the
  // last vector and column
  const int xu = nk * 16;  // 8-column units of a vector
  for (int i = tid; i < N * xu; i += kLinThreads) {
    const int n = i / xu, u = i - n * xu;
    const int64_t col = (int64_t)k0 * 128 + 8 * u;
    const bool in = n < a.batch && col < a.cols;
    // unit u of the range: step u / 16, lane quarter (u / 4) % 4, pair of k-steps u % 4
    const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(xs + (((u >> 4) * 4 + (u & 3)) * N + n) * 4 + ((u >> 2) & 3)));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"(to), "l"(static_cast<const __nv_bfloat16 *>(a.x) + (in ? n * a.x_stride + col : 0)), "r"(in ? 16 : 0) : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  // ---- the run
  {
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[nt][j] = 0.0f;
    int ct = u0 / nk, ck = u0 - ct * nk;
    bool mine = ck == 0;  // this warp takes the current tile's first step
    const uint4 *xl = xs + g * 4 + cq;
    auto unit = [&](LinLoad &d) {
      uint32_t sc[2][2];  // rows g, g + 8: f16 pairs {Delta, Delta} of the lane's two blocks
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t f;
        asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(f) : "r"(d.s[h]));
        sc[h][0] = __byte_perm(f, 0u, 0x1010);
        sc[h][1] = __byte_perm(f, 0u, 0x3232);
      }
      const uint32_t cw[2][4] = {{d.c[0].x, d.c[0].y, d.c[0].z, d.c[0].w}, {d.c[1].x, d.c[1].y, d.c[1].z, d.c[1].w}};
      const uint4 *xk = xl + ck * (16 * N);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {  // a word of codes: 8 columns, two k-steps
        uint4 xb[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) xb[nt] = xk[jj * (4 * N) + nt * 32];
        uint32_t w[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          e2m1x8_f16(cw[h][jj], w[h]);
#pragma unroll
          for (int b = 0; b < 4; ++b) w[h][b] = f16x2_bf16x2(mul_f16x2(w[h][b], sc[h][jj >> 1]));
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_bf16(acc[nt], w[0][0], w[1][0], w[0][1], w[1][1], xb[nt].x, xb[nt].y);
          mma_bf16(acc[nt], w[0][2], w[1][2], w[0][3], w[1][3], xb[nt].z, xb[nt].w);
        }
      }
      if (ahead < u1) {
        fetch(d);
        ++ahead;
      }
      if (++ck == nk) {  // the tile's last step
        float4 *to = mine ? sums + ct * NT * 32 : own + warp * NT * 32;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          to[nt * 32 + lane] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
          acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.0f;
        }
        ck = 0;
        ++ct;
        mine = true;
      }
    };
    int left = u1 - u0;
    while (left > 0) {
#pragma unroll
      for (int i = 0; i < kLinDepth; ++i)
        if (left > 0) {
          unit(buf[i]);
          --left;
        }
    }
    if (ck > 0 && u1 > u0) {  // the run ends inside a tile
      float4 *to = mine ? sums + ct * NT * 32 : own + warp * NT * 32;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) to[nt * 32 + lane] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
    }
  }
  __syncthreads();

  // ---- each tile's sum, and its way out
  const float alpha = *a.alpha;
  for (int i = tid; i < ntile * NT * 32; i += kLinThreads) {
    const int t = i / (NT * 32), f = i - t * (NT * 32), nt = f >> 5, l = f & 31;
    float4 v = sums[i];
    // warps whose run began inside the tile: those holding its units after the first
    const int wa = ((t * nk + 1) * kLinWarps - 1) / units, wb = ((t + 1) * nk * kLinWarps - 1) / units;
    for (int w = wa + 1; w <= wb; ++w) {
      if (w * units / kLinWarps == (w + 1) * units / kLinWarps) continue;  // an empty run
      const float4 o = own[w * NT * 32 + f];
      v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
    }
    if (p.p.ranges == 1) finish4(a, alpha, t0 + t, nt, l, v);
    else p.part[((int64_t)range * p.p.tiles + t0) * NT * 32 + i] = v;
  }
}

// Adds the column ranges' sums in column order and finishes them.
template <int NT>
__global__ void __launch_bounds__(256) k_linear_sum(const __grid_constant__ LinLaunch p) {
  pdl_wait();
  const int64_t all = (int64_t)p.p.tiles * NT * 32, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= all) return;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int k = 0; k < p.p.ranges; ++k) {
    const float4 o = p.part[k * all + i];
    v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
  }
  finish4(p.a, *p.a.alpha, i / (NT * 32), (int)(i % (NT * 32)) >> 5, (int)i & 31, v);
}

// cols == 0: the epilogue of a zero sum.
__global__ void __launch_bounds__(256) k_linear_empty(const __grid_constant__ LinearArgs a) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.rows * a.batch; i += (int64_t)gridDim.x * 256) {
    const float zero[1] = {0.0f};
    finish<1>(a, *a.alpha, zero, [](int) { return true; }, [&](int) { return i / a.rows; }, [&](int) { return i % a.rows; });
  }
}

namespace {

int lin_nt(int batch) { return batch <= 8 ? 1 : 2; }

// The cut into rectangles, for one wave of 2 CTAs per SM where it fits: whole
// rows, or eight column ranges (more where those would leave three quarters of
// the CTAs without work, or x of a range does not fit).  Both have an estimated
// cost in bytes of weights that a CTA reads meanwhile: the rectangle itself, x
// (which all CTAs read through one L2), and the second launch that adds the
// ranges' sums, counted as the 2 us that it takes a program which does not
// capture its calls (on the GPU it takes 1).  Measured (us on the GPU, whole rows
// and eight ranges): 8 vectors 4096 x 1024 8.4 and 6.2; 1 vector 2048 x 8192 12.2
// and 9.0, 11008 x 1024 7.7 and 8.7; 8 vectors 1000 x 1008 4.2 and 5.0.  Where the
// count decides (cold weights on the GPU, then called back to back): 1 vector
// 4096 x 4096 10.0 and 10.0, 12.4 and 12.3; 8192 x 4096 14.5 and 14.1, 16.3 and 16.5;
// 1024 x 4096 6.9 and 6.0, 8.8 and 10.8; 4 vectors 4096 x 1024 7.3 and 6.5, 9.4 and
// 10.7: what a captured step would gain the others would lose.  Other numbers of ranges lie within 3 % of the better of the two or
// behind it (4 vectors 4096 x 4096: 1, 2, 4, 6, 8, 12 and 16 ranges take 11.7,
// 10.4, 9.5, 10.4, 9.2, 11.3 and 10.9).  false: the tcgen05 product runs.
bool lin_plan(int64_t rows, int64_t cols, int batch, int sms, LinPlan *best) {
  const int nt = lin_nt(batch), ctas = 2 * sms;
  const int64_t steps = (cols + 127) / 128, tiles = (rows + 15) / 16;
  if (batch > kLinVecs || tiles > (int64_t)ctas * kLinBlocks8 ||
      steps * tiles > (int64_t)ctas * (batch <= 8 ? kLinBlocks8 : kLinBlocks16))
    return false;
  int64_t many = 8;
  while (lin_smem(nt, (steps + many - 1) / many, 1) > kLinSmem || (4 * tiles * many <= ctas && 4 * many <= steps)) many *= 2;
  int64_t least = -1;
  for (const int64_t ranges : {int64_t(1), std::min(many, steps)}) {
    const int64_t ms = (steps + ranges - 1) / ranges;
    const int64_t most = (kLinSmem - lin_smem(nt, ms, 0)) / (nt * 512);  // tiles that fit
    if (most < 1) continue;
    int64_t groups = std::min<int64_t>(tiles, std::max<int64_t>(1, ctas / ranges));
    if ((tiles + groups - 1) / groups > most) groups = (tiles + most - 1) / most;
    const int64_t mt = (tiles + groups - 1) / groups, waves = (groups * ranges + ctas - 1) / ctas;
    const int64_t cost = waves * (mt * ms * 1152 + ms * batch * 1000 * std::min<int64_t>(groups * ranges, ctas) / ctas) +
                         (ranges > 1 ? 44000 : 0);
    if (least < 0 || cost < least) {
      least = cost;
      *best = LinPlan{(int)steps, (int)tiles, (int)ranges, (int)groups, (int)ms, (int)mt};
    }
  }
  return least >= 0;
}

template <int NT>
cudaError_t lin_launch(const LinLaunch &p, bool wide, cudaStream_t st) {
  const size_t smem = (size_t)lin_smem(NT, p.p.max_steps, p.p.max_tiles);
  const int grid = p.p.ranges * p.p.groups;
  if (wide) k_linear<NT, true><<<grid, kLinThreads, smem, st>>>(p);
  else k_linear<NT, false><<<grid, kLinThreads, smem, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.p.ranges == 1) return e;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.p.tiles * NT * 32 + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_linear_sum<NT>, p);
}

}  // namespace

size_t linear_workspace_bytes(int64_t rows, int64_t cols, int batch, int sms) {
  LinPlan p;
  if (!lin_plan(rows, cols, batch, sms, &p))
    return linear_tc_workspace_bytes(rows, cols, batch, sms);
  return p.ranges == 1 ? 0 : (size_t)p.ranges * p.tiles * lin_nt(batch) * 512;
}

cudaError_t launch_linear(const LinearArgs &a, int sms, void *ws, int first_tries, LinearKernel *took, cudaStream_t st) {
  *took = kLinearRegisters;
  if (a.cols == 0) {
    k_linear_empty<<<(int)std::min<int64_t>((a.rows * a.batch + 255) / 256, 8 * sms), 256, 0, st>>>(a);
    return cudaGetLastError();
  }
  LinPlan plan;
  if (!lin_plan(a.rows, a.cols, a.batch, sms, &plan))
    return launch_linear_tc(a, sms, ws, first_tries, took, st);
  const LinLaunch p = {a, plan, static_cast<float4 *>(ws), plan.steps / plan.ranges,
                       plan.steps % plan.ranges, plan.tiles / plan.groups, plan.tiles % plan.groups};
  const bool wide = a.cols % 32 == 0 && reinterpret_cast<uintptr_t>(a.codes) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(a.scales) % 2 == 0;
  return a.batch <= 8 ? lin_launch<1>(p, wide, st) : lin_launch<2>(p, wide, st);
}

cudaError_t prepare_linear_kernels() {
  auto set = [](auto *k) { return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kLinSmem); };
  cudaError_t e = cudaSuccess;
  for (auto *k : {k_linear<1, true>, k_linear<1, false>, k_linear<2, true>, k_linear<2, false>})
    if (e == cudaSuccess) e = set(k);
  return e;
}

}  // namespace nvfp4
