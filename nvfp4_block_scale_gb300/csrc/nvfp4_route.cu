// nvfp4_route.cu -- the router of a mixture-of-experts layer: a token's scores
// against every expert, its top_k experts and their weights.
//   l[e] = sum_c x[c] router[e][c];  chosen by l, or by sigmoid(l) + bias
//   weights: softmax of l over all experts, or sigmoid(l); renormalized; scaled.
//
// The choice is the result, and a whole number: two experts whose scores fp32
// cannot tell apart have to come out in the right order.  So a lane keeps its
// sum of products (exact in fp32 for a bf16 router) as two fp32 numbers, the
// sum and the sum of its rounding errors (each found exactly by Knuth's
// two-sum: 7 operations a product), lanes meet in fp64, and scores are fp64.
//
// Bound: latency for a few tokens (1 token 2048, 8 of 128: 6.4 us, of which a launch
// and the router's first bytes are 3); from about 64 tokens on the 7 fp32 operations a
// product, so many tokens take the tensor cores, and those operations only where the
// tensor cores leave the order of two experts open (61 tokens 4096, 2 of 8: 8.3 us;
// 256 x 7168, 8 of 256: 47 us, 20 TFLOP/s, where the operations for all took 266; 17 to
// 25 of them are loads and products, 5 the choice, up to 8 the doubtful experts).
//
// Work split: a cluster of 8 or 16 CTAs takes G tokens; each CTA has its
// share of the experts, its warps an expert each, or a range of an expert's
// columns where there are fewer experts than warps.  The logits of a token meet
// in the shared memory of one CTA of the cluster, where a warp chooses: in each of
// top_k rounds every lane offers the first of its own that is left.  No global
// memory, no second launch.
#include <algorithm>
#include <climits>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {

namespace cg = cooperative_groups;

constexpr int kRouteThreads = 512, kRouteWarps = kRouteThreads / 32;
constexpr int kRouteMaxCtas = 16;  // of a cluster (8 where a device cannot place more)
constexpr int kTcCtas = 8, kTcThreads = 256, kTcWarps = kTcThreads / 32;  // of the kernel for many tokens

// Adds a * b to the sum hi + lo.
__device__ __forceinline__ void add_product(float a, float b, float &hi, float &lo, bool exact) {
  const float s = fmaf(a, b, hi);
  if (exact) {  // a * b is one fp32 number
    const float t = s - hi;
    lo += (hi - (s - t)) + fmaf(a, b, -t);
  } else {  // s = fl(hi + ab): p + e = ab, then the same with p, and e
    const float p = a * b, e = fmaf(a, b, -p), q = hi + p, t = q - hi;
    lo += ((hi - (q - t)) + (p - t)) + e;
    hi = q;
    return;
  }
  hi = s;
}

template <typename R>
struct RouterLoad;
template <>
struct RouterLoad<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void get(const __nv_bfloat16 *p) { w = __ldg(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t v = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
    return __uint_as_float(i & 1 ? v & 0xFFFF0000u : v << 16);
  }
};
template <>
struct RouterLoad<float> {
  float4 w[2];
  __device__ __forceinline__ void get(const float *p) {
    w[0] = __ldg(reinterpret_cast<const float4 *>(p));
    w[1] = __ldg(reinterpret_cast<const float4 *>(p) + 1);
  }
  __device__ __forceinline__ float at(int i) const {
    const float4 v = w[i >> 2];
    return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
  }
};

// A number's place in the order of scores, above 0: NaN below everything.
__device__ __forceinline__ uint64_t score_key(double v) {
  if (v != v) return 1;
  if (v == 0.0) v = 0.0;  // (-0 and 0 are equal)
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  return b >> 63 ? ~b : b | 1ull << 63;
}

// A warp's sum of the products of two rows, in units [u0, u1) of eight columns.
template <typename R>
__device__ __forceinline__ double exact_dot(const __nv_bfloat16 *x, const R *w, int u0, int u1, int lane) {
  float hi = 0.0f, lo = 0.0f;
  constexpr int kAhead = 4;
  for (int u = u0 + lane; u < u1; u += 32 * kAhead) {  // (u1 > u0 wherever this loads)
    RouterLoad<R> r[kAhead];
    RouterLoad<__nv_bfloat16> v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = min(u + 32 * i, u1 - 1);
      r[i].get(w + 8 * at);
      v[i].get(x + 8 * at);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (u + 32 * i >= u1) break;
#pragma unroll
      for (int c = 0; c < 8; ++c) add_product(r[i].at(c), v[i].at(c), hi, lo, sizeof(R) == 2);
    }
  }
  double d = (double)hi + (double)lo;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(~0u, d, o);
  return d;
}

__device__ __forceinline__ float sigmoid(float v) { return __fdiv_rn(1.0f, 1.0f + expf(-v)); }
__device__ __forceinline__ double route_score(const RouteArgs &a, double logit, int e) {
  return a.sigmoid ? 1.0 / (1.0 + exp(-logit)) + (a.bias ? (double)a.bias[e] : 0.0) : logit;
}
// The same in fp32, off by at most 2^-21 of itself and (a sigmoid's) of 1: fp64's
// exponentials take longer than everything else about a choice.
__device__ __forceinline__ float route_score_fp32(const RouteArgs &a, double logit, int e) {
  return a.sigmoid ? sigmoid((float)logit) + (a.bias ? a.bias[e] : 0.0f) : (float)logit;
}

// A token's top_k experts in order, by one warp: in each of top_k rounds every lane
// offers the first of its own (e = lane, lane + 32, ..) that is left.  Lane i has
// the i-th in the end.
__device__ __forceinline__ int choose(const RouteArgs &a, uint64_t *keys, int lane) {
  uint64_t best = 0;
  int at = INT_MAX, chosen = 0;
  auto look = [&] {
    best = 0, at = INT_MAX;
#pragma unroll 4
    for (int e = lane; e < a.experts; e += 32) {
      const uint64_t k = keys[e];
      if (k > best) best = k, at = e;
    }
  };
  look();
  for (int i = 0; i < a.top_k; ++i) {
    const uint32_t hi = __reduce_max_sync(~0u, (uint32_t)(best >> 32));
    const uint32_t lo = __reduce_max_sync(~0u, (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
    const bool first = (uint32_t)(best >> 32) == hi && (uint32_t)best == lo;
    const int e = (int)__reduce_min_sync(~0u, first ? (unsigned)at : ~0u);
    if (lane == i) chosen = e;
    if (e == at) {
      keys[e] = 0;
      look();
    }
  }
  return chosen;
}

// Its weights, by the same warp; lane i's expert is the i-th.
__device__ __forceinline__ void weigh(const RouteArgs &a, int64_t t, const double *l, int e, int lane) {
  const double m = l[__shfl_sync(~0u, e, 0)];  // softmax: the first choice has the largest logit
  float w = 0.0f, z = 1.0f;
  if (a.sigmoid) {
    // exp(min(l, 0)) / (1 + exp(-|l|)).  Of a sum the exponentials' largest cancels, so that the
    // weights of logits below -87, whose sigmoids fp32 does not hold, still have one.
    const float v = (float)l[e];
    float most = 0.0f;
    if (a.renormalize) most = -__uint_as_float(__reduce_min_sync(~0u, lane >= a.top_k ? ~0u : v < 0.0f ? __float_as_uint(-v) : 0u));
    if (lane < a.top_k) w = __fdiv_rn(expf((float)(fmin(l[e], 0.0) - (double)most)), 1.0f + expf(-fabsf(v)));
  } else if (lane < a.top_k) {
    w = expf((float)(l[e] - m));
  }
  if (a.renormalize) {
    z = w;
  } else if (!a.sigmoid) {
    z = 0.0f;
    for (int o = lane; o < a.experts; o += 32) z += expf((float)(l[o] - m));
  }
  if (a.renormalize || !a.sigmoid) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(~0u, z, o);
  }
  if (lane < a.top_k) {
    a.ids[t * a.top_k + lane] = e;
    a.weights[t * a.top_k + lane] = __fdiv_rn(w, z) * a.scale;
  }
}

struct RouteLaunch {
  RouteArgs a;
  int per;     // experts of a CTA at most
  int splits;  // warps of an expert
};

template <typename R, int G>
__global__ void __launch_bounds__(kRouteThreads) k_moe_route(const __grid_constant__ RouteLaunch p) {
  // [splits][per][G] sums, later [experts] keys; then the logits of this CTA's token [experts]
  extern __shared__ double sums[];
  const RouteArgs &a = p.a;
  const auto cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = (int)cluster.block_rank();
  static_assert(G <= 8, "a token per CTA of the cluster at most");
  const int64_t t0 = (int64_t)(blockIdx.x / cluster.num_blocks()) * G;
  const int tokens = (int)min((int64_t)G, a.tokens - t0);
  const int e0 = rank * p.per, mine = max(0, min(p.per, a.experts - e0));
  double *const logits = sums + max(p.splits * p.per * G, a.experts);
  cluster_begun();
  pdl_wait();
  pdl_launch_dependents();

  // ---- products: task (expert, range of columns) per warp
  const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.x) + t0 * a.x_stride;
  const int eighths = (int)(a.hidden / 8);
  for (int task = warp; task < mine * p.splits; task += kRouteWarps) {
    const int e = task / p.splits, s = task - e * p.splits;
    const int u0 = (int)((int64_t)s * eighths / p.splits), u1 = (int)((int64_t)(s + 1) * eighths / p.splits);
    const R *w = static_cast<const R *>(a.router) + (int64_t)(e0 + e) * a.router_stride;
    float hi[G], lo[G];
#pragma unroll
    for (int g = 0; g < G; ++g) hi[g] = lo[g] = 0.0f;
    constexpr int kAhead = G == 1 ? 8 : G == 2 ? 4 : 2;
    for (int u = u0 + lane; u < u1; u += 32 * kAhead) {
      RouterLoad<R> r[kAhead];
      RouterLoad<__nv_bfloat16> v[kAhead][G];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int at = min(u + 32 * i, u1 - 1);
        r[i].get(w + 8 * at);
#pragma unroll
        for (int g = 0; g < G; ++g) v[i][g].get(x + (int64_t)min(g, tokens - 1) * a.x_stride + 8 * at);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (u + 32 * i >= u1) break;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int c = 0; c < 8; ++c) add_product(r[i].at(c), v[i][g].at(c), hi[g], lo[g], sizeof(R) == 2);
      }
    }
    // lanes meet: halves of the tokens at a time, then all lanes of a token
    double d[G];
#pragma unroll
    for (int g = 0; g < G; ++g) d[g] = (double)hi[g] + (double)lo[g];
    int off = 16;
#pragma unroll
    for (int n = G; n > 1; n >>= 1, off >>= 1) {
      const bool up = lane & off;
#pragma unroll
      for (int g = 0; g < n / 2; ++g) {
        const double keep = up ? d[g + n / 2] : d[g], send = up ? d[g] : d[g + n / 2];
        d[g] = keep + __shfl_xor_sync(~0u, send, off);
      }
    }
#pragma unroll
    for (; off > 0; off >>= 1) d[0] += __shfl_xor_sync(~0u, d[0], off);
    constexpr int kLanes = 32 / G;  // of a token: the lanes with its bits on top, in the order of the halvings
    if (lane % kLanes == 0) sums[((size_t)s * p.per + e) * G + lane / kLanes] = d[0];
  }
  __syncthreads();
  cluster_wait_begun();
  // ---- every logit to the CTA of its token
  for (int i = tid; i < mine * tokens; i += kRouteThreads) {
    const int e = i / tokens, g = i - e * tokens;
    double v = 0.0;
    for (int s = 0; s < p.splits; ++s) v += sums[((size_t)s * p.per + e) * G + g];
    cluster.map_shared_rank(logits, g)[e0 + e] = v;
  }
  cluster.sync();

  // ---- the choice
  if (rank >= tokens) return;
  uint64_t *keys = reinterpret_cast<uint64_t *>(sums);  // (the sums are spent)
  for (int e = tid; e < a.experts; e += kRouteThreads) keys[e] = score_key(route_score(a, logits[e], e));
  __syncthreads();
  if (warp > 0) return;
  const int e = choose(a, keys, lane);
  weigh(a, t0 + rank, logits, e, lane);
}

// Many tokens: the products on the tensor cores (mma.sync m16n8k16, 16 experts by 8
// tokens), two steps (32 columns) summed there from zero and then added to a sum in
// two fp32 numbers.  Such a logit is off by less than kBand ||x|| ||r||: products of
// two bf16 numbers are exact, and 32 additions, truncated at worst, lose 2^-23 of
// sum |x r| <= ||x|| ||r|| each: 2^-18.  An fp32 router's entry enters as three bf16
// numbers (all of its 24 bits), with three times the additions: 2^-16.4.  Where that
// leaves open which of two experts comes first, and one of them may be chosen, their
// logits are formed once more, exactly (a token in twenty, two experts each, at
// 256 experts x 7168).
// (The factor of two between the bounds and kBand covers the norms' roundings.)
template <typename R>
constexpr float kBand = sizeof(R) == 2 ? 0x1p-17f : 0x1p-15f;
constexpr int kTcTokens = 16;  // of a cluster

__device__ __forceinline__ void route_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The sum of squares of eight bf16 numbers (of an fp32 router their leading parts), within 2^-6 of it.
__device__ __forceinline__ float squares(const uint4 &v) {
  uint32_t s = 0u;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("fma.rn.bf16x2 %0, %1, %1, %0;" : "+r"(s) : "r"(w[i]));
  return __uint_as_float(s << 16) + __uint_as_float(s & 0xFFFF0000u);
}

template <typename R>
__global__ void __launch_bounds__(kTcThreads, 2) k_moe_route_tc(const __grid_constant__ RouteLaunch p) {
  // [splits][tiles * 16][kTcTokens] sums, later [2][experts] keys; the logits of this CTA's two tokens [2][experts];
  // norms of the router's rows [experts], of this CTA's by split, of the tokens by split, whether a token has an
  // entry other than 0, and the scores of the two tokens [2][experts]
  extern __shared__ double sums[];
  __shared__ int doubtful, list[2 * kMaxExperts];
  __shared__ uint16_t candidates[2][kMaxExperts];
  __shared__ double parts[kTcWarps][kTcWarps];
  const RouteArgs &a = p.a;
  const auto cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cq = lane & 3, rank = (int)cluster.block_rank();
  const int64_t t0 = (int64_t)(blockIdx.x / kTcCtas) * kTcTokens;
  const int tokens = (int)min((int64_t)kTcTokens, a.tokens - t0);
  const int e0 = rank * p.per, mine = max(0, min(p.per, a.experts - e0));
  const int tiles = (p.per + 15) / 16, rows = tiles * 16;
  double *const logits = sums + max(p.splits * rows * kTcTokens, 2 * a.experts);
  float *const row_norm = reinterpret_cast<float *>(logits + 2 * a.experts);  // [experts]
  float *const row_part = row_norm + a.experts;                               // [splits][rows]
  float *const token_part = row_part + p.splits * rows;                       // [splits][kTcTokens]
  uint32_t *const token_any = reinterpret_cast<uint32_t *>(token_part + p.splits * kTcTokens);  // [splits][kTcTokens]
  float *const scores = reinterpret_cast<float *>(token_any + p.splits * kTcTokens);            // [2][experts]
  if (tid == 0) doubtful = 0;
  cluster_begun();
  pdl_wait();
  pdl_launch_dependents();

  const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.x) + t0 * a.x_stride;
  const int eighths = (int)(a.hidden / 8), steps = (eighths + 3) / 4;
  for (int task = warp; task < tiles * p.splits; task += kTcWarps) {
    const int tile = task / p.splits, s = task - tile * p.splits;
    const int k0 = (int)((int64_t)s * steps / p.splits), k1 = (int)((int64_t)(s + 1) * steps / p.splits);
    const R *w[2];
    const __nv_bfloat16 *v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] = static_cast<const R *>(a.router) + (int64_t)min(e0 + tile * 16 + 8 * h + g, a.experts - 1) * a.router_stride;
      v[h] = x + (int64_t)min(8 * h + g, tokens - 1) * a.x_stride;
    }
    float hi[2][4], lo[2][4], nr[2] = {0.0f, 0.0f}, nx[2] = {0.0f, 0.0f};
    uint32_t any[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) hi[i][c] = lo[i][c] = 0.0f;
    constexpr int kAhead = sizeof(R) == 2 ? 4 : 2;
    struct Step {
      RouterLoad<R> r[2];
      RouterLoad<__nv_bfloat16> t[2];
    };
    auto load = [&](Step &d, int k) {
      const int u = min(4 * min(k, k1 - 1) + cq, eighths - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        d.r[h].get(w[h] + 8 * u);
        d.t[h].get(v[h] + 8 * u);
      }
    };
    Step d[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(d[i], k0 + i);
    for (int k = k0; k < k1; k += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (k + i >= k1) break;
        if (4 * (k + i) + cq >= eighths)  // columns past the end
#pragma unroll
          for (int h = 0; h < 2; ++h) d[i].t[h].w = make_uint4(0u, 0u, 0u, 0u);
        uint4 big[2], small[2], rest[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (sizeof(R) == 2) {
            big[h] = d[i].r[h].w;
          } else {
            uint32_t b[4], m[4], l[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float f0 = d[i].r[h].at(2 * c), f1 = d[i].r[h].at(2 * c + 1);
              b[c] = pack_bf16(f0, f1);
              const float g0 = f0 - __uint_as_float(b[c] << 16), g1 = f1 - __uint_as_float(b[c] & 0xFFFF0000u);
              m[c] = pack_bf16(g0, g1);
              l[c] = pack_bf16(g0 - __uint_as_float(m[c] << 16), g1 - __uint_as_float(m[c] & 0xFFFF0000u));
            }
            big[h] = make_uint4(b[0], b[1], b[2], b[3]);
            small[h] = make_uint4(m[0], m[1], m[2], m[3]);
            rest[h] = make_uint4(l[0], l[1], l[2], l[3]);
          }
          if (tile == 0) {
            const uint4 &tw = d[i].t[h].w;
            nx[h] += squares(tw);
            any[h] |= (tw.x | tw.y | tw.z | tw.w) & 0x7FFF7FFFu;
          }
          nr[h] += squares(big[h]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // eight tokens
          const uint4 b = d[i].t[h].w;
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          route_mma(c, big[0].x, big[1].x, big[0].y, big[1].y, b.x, b.y);
          route_mma(c, big[0].z, big[1].z, big[0].w, big[1].w, b.z, b.w);
          if constexpr (sizeof(R) == 4) {
            route_mma(c, small[0].x, small[1].x, small[0].y, small[1].y, b.x, b.y);
            route_mma(c, small[0].z, small[1].z, small[0].w, small[1].w, b.z, b.w);
            route_mma(c, rest[0].x, rest[1].x, rest[0].y, rest[1].y, b.x, b.y);
            route_mma(c, rest[0].z, rest[1].z, rest[0].w, rest[1].w, b.z, b.w);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // hi + lo += c, the rounding of hi kept
            const float q = hi[h][j] + c[j], t = q - hi[h][j];
            lo[h][j] += (hi[h][j] - (q - t)) + (c[j] - t);
            hi[h][j] = q;
          }
        }
        load(d[i], k + i + kAhead);
      }
    }
    double *to = sums + ((size_t)s * rows + tile * 16) * kTcTokens;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        to[(g + 8 * (j >> 1)) * kTcTokens + 8 * h + 2 * cq + (j & 1)] = (double)hi[h][j] + (double)lo[h][j];
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        nr[h] += __shfl_xor_sync(~0u, nr[h], o), nx[h] += __shfl_xor_sync(~0u, nx[h], o);
        any[h] |= __shfl_xor_sync(~0u, any[h], o);
      }
      if (cq == 0) row_part[s * rows + tile * 16 + 8 * h + g] = nr[h];
      if (cq == 0 && tile == 0) token_part[s * kTcTokens + 8 * h + g] = nx[h], token_any[s * kTcTokens + 8 * h + g] = any[h];
    }
  }
  __syncthreads();
  cluster_wait_begun();
  // ---- every logit to the CTA of its token, every row's norm to all
  for (int i = tid; i < mine * kTcTokens; i += kTcThreads) {
    const int e = i / kTcTokens, t = i - e * kTcTokens;
    double v = 0.0;
    for (int s = 0; s < p.splits; ++s) v += sums[((size_t)s * rows + e) * kTcTokens + t];
    cluster.map_shared_rank(logits, t % kTcCtas)[(t / kTcCtas) * a.experts + e0 + e] = v;
  }
  for (int i = tid; i < mine * kTcCtas; i += kTcThreads) {
    const int e = i / kTcCtas, r = i - e * kTcCtas;
    float n = 0.0f;
    for (int s = 0; s < p.splits; ++s) n += row_part[s * rows + e];
    cluster.map_shared_rank(row_norm, r)[e0 + e] = sqrtf(n + 0x1p-100f);  // (an upper bound where squares underflow)
  }
  cluster.sync();

  // ---- the choice of each of this CTA's tokens, by a warp
  uint64_t *const keys = reinterpret_cast<uint64_t *>(sums);  // (the sums are spent)
  auto make_keys = [&](bool fp64) {
    for (int i = tid; i < 2 * a.experts; i += kTcThreads) {
      const int r = i >= a.experts, e = i - r * a.experts;
      if (rank + r * kTcCtas >= tokens) continue;
      const float s = route_score_fp32(a, logits[i], e);
      keys[i] = score_key(fp64 ? route_score(a, logits[i], e) : (double)s);
      scores[i] = s;
    }
    __syncthreads();
  };
  make_keys(false);
  const int t = rank + warp * kTcCtas;  // this warp's token
  const bool has = warp < 2 && t < tokens;
  int e = 0;
  if (has) {
    const float *score = scores + (size_t)warp * a.experts;
    uint64_t *const key = keys + (size_t)warp * a.experts;
    float norm = 0.0f;
    uint32_t any = 0u;
    for (int s = 0; s < p.splits; ++s) norm += token_part[s * kTcTokens + t], any |= token_any[s * kTcTokens + t];
    if (!any && a.bias) {  // a token of zeros: its logits are exact, and so are its scores in fp64
      for (int o = lane; o < a.experts; o += 32) key[o] = score_key(0.5 + (double)a.bias[o]);
      __syncwarp();
    }
    e = choose(a, key, lane);
    // (squares that may have underflowed bound nothing)
    norm = norm > 0x1p-100f ? sqrtf(norm) * kBand<R> : INFINITY;
    // how far arithmetic may have moved an expert's score (a sigmoid's slope is at most 1/4)
    auto off = [&](int o, float s) {  // (a bias of -inf or inf leaves nothing open)
      if (fabsf(s) == INFINITY) return 0.0f;
      return norm * row_norm[o] * (a.sigmoid ? 0.25f : 1.0f) + 0x1p-21f * (fabsf(s) + (a.sigmoid ? 1.0f : 0.0f));
    };
    // those that may be among the chosen reach up to where the last of these may have come from
    const float s0 = lane < a.top_k ? score[e] : INFINITY, low = lane < a.top_k ? s0 - off(e, s0) : INFINITY;
    float least = low;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) least = fminf(least, __shfl_xor_sync(~0u, least, o));
    // Candidates: an expert that is none lies below all of the chosen whatever
    // arithmetic did, and so does a candidate that is near no other.
    int n = 0;
    for (int o0 = 0; any && o0 < a.experts; o0 += 32) {
      const int o = o0 + lane;
      const float so = o < a.experts ? score[o] : 0.0f;
      const bool is = o < a.experts && !(so + off(o, so) < least);
      const uint32_t all = __ballot_sync(~0u, is);
      if (is) candidates[warp][n + __popc(all & ((1u << lane) - 1u))] = (uint16_t)o;
      n += __popc(all);
    }
    __syncwarp();
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int c = candidates[warp][min(i0 + lane, n - 1)];
      const float sc = score[c], bc = off(c, sc);
      bool near = n > 128;  // (too many to compare: all of them)
      for (int q = 0; q < n && n <= 128; ++q) {
        const int o = candidates[warp][q];
        const float so = score[o];
        near |= o != c && !(fabsf(so - sc) > bc + off(o, so));
      }
      if (near && i0 + lane < n) list[atomicAdd(&doubtful, 1)] = warp * a.experts + c;
    }
  }
  __syncthreads();
  const int count = doubtful;
  if (count > 0) {  // those once more, exactly
    auto dot = [&](int i, int u0, int u1) {
      const int r = list[i] >= a.experts, c = list[i] - r * a.experts;
      return exact_dot(x + (int64_t)(rank + r * kTcCtas) * a.x_stride,
                       static_cast<const R *>(a.router) + (int64_t)c * a.router_stride, u0, u1, lane);
    };
    if (count <= kTcWarps) {  // all warps on each
      for (int i = 0; i < count; ++i) {
        const double v = dot(i, warp * eighths / kTcWarps, (warp + 1) * eighths / kTcWarps);
        if (lane == 0) parts[i][warp] = v;
      }
      __syncthreads();
      if (tid < count) {
        double v = 0.0;
        for (int w = 0; w < kTcWarps; ++w) v += parts[tid][w];
        logits[list[tid]] = v;
      }
    } else {
      for (int i = warp; i < count; i += kTcWarps) {
        const double v = dot(i, 0, eighths);
        if (lane == 0) logits[list[i]] = v;
      }
    }
    __syncthreads();
    make_keys(true);
    if (has) e = choose(a, keys + (size_t)warp * a.experts, lane);
  }
  if (has) weigh(a, t0 + t, logits + (size_t)warp * a.experts, e, lane);
}

namespace {

template <typename F>
auto with_route(bool fp32, int g, F f) {
  auto pick = [&](auto r) {
    using R = decltype(r);
    return g == 1 ? f(k_moe_route<R, 1>) : g == 2 ? f(k_moe_route<R, 2>) : g == 4 ? f(k_moe_route<R, 4>) : f(k_moe_route<R, 8>);
  };
  return fp32 ? pick(0.0f) : pick(__nv_bfloat16());
}

size_t route_smem(const RouteLaunch &p, int g) {
  return ((size_t)std::max(p.splits * p.per * g, p.a.experts) + (size_t)p.a.experts) * sizeof(double);
}

size_t route_tc_smem(const RouteLaunch &p) {
  const int rows = (p.per + 15) / 16 * 16, e = p.a.experts;
  return ((size_t)std::max(p.splits * rows * kTcTokens, 2 * e) + 2 * (size_t)e) * sizeof(double) +
         (3 * (size_t)e + (size_t)p.splits * (rows + 2 * kTcTokens)) * sizeof(float);
}

}  // namespace

cudaError_t prepare_route_kernels(int *ctas) {
  // splits * rows <= 128 rows of 16 tokens, and 1024 experts
  const int most = (128 * kTcTokens + 4 * kMaxExperts) * 8 + (3 * kMaxExperts + 128 + kTcWarps * 2 * kTcTokens) * 4;
  cudaError_t e = cudaFuncSetAttribute(k_moe_route_tc<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_moe_route_tc<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  for (const bool fp32 : {false, true})
    if (e == cudaSuccess)
      e = with_route(fp32, 1, [](auto *k) { return cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); });
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = kRouteMaxCtas;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kRouteMaxCtas);
  cfg.blockDim = dim3(kRouteThreads);
  cfg.dynamicSmemBytes = 48 * 1024;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, k_moe_route<float, 1>, &cfg) != cudaSuccess) cudaGetLastError();  // (8 then)
  *ctas = clusters > 0 ? kRouteMaxCtas : 8;
  return cudaSuccess;
}

cudaError_t launch_route(const RouteArgs &a, int sms, int most_ctas, cudaStream_t st) {
  RouteLaunch p = {a, 0, 1};
  // The tensor cores where there are many scores.  Measured with a bf16 router, softmax (us, then the
  // other kernel's), where the rule takes them: 64 tokens 7168, 256 experts 31 and 53; 32 tokens 31 and 34;
  // 128 tokens 2048, 128 experts 16 and 20; 128 tokens 4096, 60 experts 17 and 20; 256 tokens 4096, 8 experts
  // 14 and 28; 64 tokens 4096, 128 experts 18 and 19; and where it does not: 31 tokens 2048, 128 experts 13
  // and 11; 64 tokens 4096, 60 experts 16 and 14; 64 tokens 4096, 8 experts 11 and 9.  It looks at tokens and
  // scores alone, since the accuracy of the weights goes by it, and so takes the slower kernel near its edges:
  // 64 tokens 2048, 128 experts 16 and 15 (1024: 15 and 11), 128 tokens 4096, 8 experts 12 and 10 (256, 32
  // experts: 9 and 6), and the other way 16 tokens 7168, 256 experts 28 and 33, 127 tokens 4096, 64 experts 17
  // and 20.  With an fp32 router both take longer: 64 tokens 7168, 256 experts 45 and 62; 64 tokens 4096, 128
  // experts 24 and 22; 128 tokens 4096, 8 experts 17 and 11.
  const bool tc = a.tokens >= 128 || (a.tokens >= 16 && a.tokens * a.experts >= 8192);
  int g = kTcTokens, ctas = kTcCtas, threads = kTcThreads;
  p.per = (a.experts + ctas - 1) / ctas;
  if (tc) {
    p.splits = std::max(1, std::min(kTcWarps / ((p.per + 15) / 16), (int)((a.hidden + 31) / 32)));
  } else {
    // as few tokens per cluster as one wave of CTAs allows: a router row's way
    // through L2 is shared by a cluster's tokens, but a lane's work is theirs together
    g = 1, threads = kRouteThreads;
    // (1 token 7168, 256 experts: 23 us with clusters of 8, 14 with 16; 2048, 128 experts: 7.9 and 6.6)
    if (a.experts >= 32 && a.tokens * kRouteMaxCtas <= sms) ctas = most_ctas;
    p.per = (a.experts + ctas - 1) / ctas;
    p.splits = std::max(1, std::min<int>(kRouteWarps / p.per, (int)(a.hidden / 256)));
    while (g < 8 && (a.tokens + g - 1) / g * ctas > 2 * sms) g *= 2;
  }
  const int64_t groups = (a.tokens + g - 1) / g;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * ctas));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = tc ? route_tc_smem(p) : route_smem(p, g);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  if (tc) return a.fp32 ? cudaLaunchKernelEx(&cfg, k_moe_route_tc<float>, p) : cudaLaunchKernelEx(&cfg, k_moe_route_tc<__nv_bfloat16>, p);
  return with_route(a.fp32, g, [&](auto *k) { return cudaLaunchKernelEx(&cfg, k, p); });
}

}  // namespace nvfp4
