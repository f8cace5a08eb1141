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
// Bound: latency for a few tokens; from about 64 tokens on the 7 fp32
// operations a product.
//
// Work split: a cluster of kRouteCtas CTAs takes G tokens; each CTA has its
// share of the experts, its warps an expert each, or a range of an expert's
// columns where there are fewer experts than warps.  The logits of a token meet
// in the shared memory of one CTA of the cluster, which ranks them: an
// expert's rank is the number of those before it.  No global memory, no second
// launch.
#include <algorithm>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {

namespace cg = cooperative_groups;

constexpr int kRouteCtas = 8;
constexpr int kRouteThreads = 512, kRouteWarps = kRouteThreads / 32;

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

// A number's place in the order of scores: NaN below everything.
__device__ __forceinline__ uint64_t score_key(double v) {
  if (v != v) return 0;
  if (v == 0.0) v = 0.0;  // (-0 and 0 are equal)
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  return b >> 63 ? ~b : b | 1ull << 63;
}

// A warp's sum of the products of two rows, in units [u0, u1) of eight columns.
template <typename R>
__device__ __forceinline__ double exact_dot(const __nv_bfloat16 *x, const R *w, int u0, int u1, int lane) {
  float hi = 0.0f, lo = 0.0f;
  for (int u = u0 + lane; u < u1; u += 32) {
    RouterLoad<R> r;
    RouterLoad<__nv_bfloat16> v;
    r.get(w + 8 * u);
    v.get(x + 8 * u);
#pragma unroll
    for (int c = 0; c < 8; ++c) add_product(r.at(c), v.at(c), hi, lo, sizeof(R) == 2);
  }
  double d = (double)hi + (double)lo;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(~0u, d, o);
  return d;
}

__device__ __forceinline__ double route_score(const RouteArgs &a, double logit, int e) {
  return a.sigmoid ? 1.0 / (1.0 + exp(-logit)) + (a.bias ? (double)a.bias[e] : 0.0) : logit;
}

// A token's experts and weights from its logits, by the whole CTA.
__device__ void choose(const RouteArgs &a, int64_t t, const double *l, uint64_t *keys, int *best, float *partial) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e < a.experts; e += kRouteThreads) keys[e] = score_key(route_score(a, l[e], e));
  if (tid < kMaxTopK) best[tid] = 0;
  __syncthreads();
  for (int e = tid; e < a.experts; e += kRouteThreads) {
    const uint64_t k = keys[e];
    int before = 0;
    for (int o = 0; o < a.experts; ++o) before += keys[o] > k || (keys[o] == k && o < e);
    if (before < a.top_k) best[before] = e;
  }
  __syncthreads();
  // softmax: its maximum is the first choice's logit; its sum in a fixed order
  const double m = l[best[0]];
  if (!a.sigmoid && !a.renormalize) {
    float z = 0.0f;
    for (int e = tid; e < a.experts; e += kRouteThreads) z += expf((float)(l[e] - m));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(~0u, z, o);
    if (lane == 0) partial[warp] = z;
  }
  __syncthreads();
  if (warp == 0) {
    const int e = best[min(lane, a.top_k - 1)];
    float w = lane < a.top_k ? a.sigmoid ? (float)(1.0 / (1.0 + exp(-l[e]))) : expf((float)(l[e] - m)) : 0.0f;
    float z = 1.0f;
    if (a.renormalize) {
      z = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(~0u, z, o);
    } else if (!a.sigmoid) {
      z = 0.0f;
      for (int i = 0; i < kRouteWarps; ++i) z += partial[i];
    }
    if (lane < a.top_k) {
      a.ids[t * a.top_k + lane] = e;
      a.weights[t * a.top_k + lane] = __fdiv_rn(w, z) * a.scale;
    }
  }
  __syncthreads();
}

struct RouteLaunch {
  RouteArgs a;
  int per;     // experts of a CTA at most
  int splits;  // warps of an expert
};

template <typename R, int G>
__global__ void __launch_bounds__(kRouteThreads) k_moe_route(const __grid_constant__ RouteLaunch p) {
  // [splits][per][G] sums, later [experts] keys; then the logits of this CTA's tokens [ceil(G / kRouteCtas)][experts]
  extern __shared__ double sums[];
  __shared__ int best[kMaxTopK];
  __shared__ float partial[kRouteWarps];
  const RouteArgs &a = p.a;
  const auto cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = (int)cluster.block_rank();
  const int64_t t0 = (int64_t)(blockIdx.x / kRouteCtas) * G;
  const int tokens = (int)min((int64_t)G, a.tokens - t0);
  const int e0 = rank * p.per, mine = max(0, min(p.per, a.experts - e0));
  double *const logits = sums + max(p.splits * p.per * G, a.experts);
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
    constexpr int kAhead = G <= 2 ? 4 : 2;
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
  // ---- every logit to the CTA of its token
  for (int i = tid; i < mine * tokens; i += kRouteThreads) {
    const int e = i / tokens, g = i - e * tokens;
    double v = 0.0;
    for (int s = 0; s < p.splits; ++s) v += sums[((size_t)s * p.per + e) * G + g];
    cluster.map_shared_rank(logits, g % kRouteCtas)[(g / kRouteCtas) * a.experts + e0 + e] = v;
  }
  cluster.sync();

  // ---- the choice
  for (int g = rank, r = 0; g < tokens; g += kRouteCtas, ++r)
    choose(a, t0 + g, logits + (size_t)r * a.experts, reinterpret_cast<uint64_t *>(sums), best, partial);  // (the sums are spent)
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
__global__ void __launch_bounds__(kRouteThreads) k_moe_route_tc(const __grid_constant__ RouteLaunch p) {
  // [splits][tiles * 16][kTcTokens] sums, later [experts] keys and [experts] fp32 scores; the logits of this CTA's
  // tokens [2][experts]; norms of the router's rows [experts], of this CTA's by split, of the tokens by split, and
  // whether a token has an entry other than 0
  extern __shared__ double sums[];
  __shared__ int best[kMaxTopK], doubtful, list[kMaxExperts];
  __shared__ float partial[kRouteWarps];
  const RouteArgs &a = p.a;
  const auto cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cq = lane & 3, rank = (int)cluster.block_rank();
  const int64_t t0 = (int64_t)(blockIdx.x / kRouteCtas) * kTcTokens;
  const int tokens = (int)min((int64_t)kTcTokens, a.tokens - t0);
  const int e0 = rank * p.per, mine = max(0, min(p.per, a.experts - e0));
  const int tiles = (p.per + 15) / 16, rows = tiles * 16;
  double *const logits = sums + max(p.splits * rows * kTcTokens, 2 * a.experts);
  float *const row_norm = reinterpret_cast<float *>(logits + 2 * a.experts);  // [experts]
  float *const row_part = row_norm + a.experts;                               // [splits][rows]
  float *const token_part = row_part + p.splits * rows;                       // [splits][kTcTokens]
  uint32_t *const token_any = reinterpret_cast<uint32_t *>(token_part + p.splits * kTcTokens);  // [splits][kTcTokens]
  pdl_wait();
  pdl_launch_dependents();

  const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(a.x) + t0 * a.x_stride;
  const int eighths = (int)(a.hidden / 8), steps = (eighths + 3) / 4;
  if (warp < tiles * p.splits) {
    const int tile = warp / p.splits, s = warp - tile * p.splits;
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
    constexpr int kAhead = 2;
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
  // ---- every logit to the CTA of its token, every row's norm to all
  for (int i = tid; i < mine * kTcTokens; i += kRouteThreads) {
    const int e = i / kTcTokens, t = i - e * kTcTokens;
    double v = 0.0;
    for (int s = 0; s < p.splits; ++s) v += sums[((size_t)s * rows + e) * kTcTokens + t];
    cluster.map_shared_rank(logits, t % kRouteCtas)[(t / kRouteCtas) * a.experts + e0 + e] = v;
  }
  for (int i = tid; i < mine * kRouteCtas; i += kRouteThreads) {
    const int e = i / kRouteCtas, r = i - e * kRouteCtas;
    float n = 0.0f;
    for (int s = 0; s < p.splits; ++s) n += row_part[s * rows + e];
    cluster.map_shared_rank(row_norm, r)[e0 + e] = sqrtf(n);
  }
  cluster.sync();

  // ---- experts in doubt, exactly; the choice
  float *const scores = reinterpret_cast<float *>(sums + a.experts);  // (the sums are spent)
  for (int t = rank, r = 0; t < tokens; t += kRouteCtas, ++r) {
    double *l = logits + (size_t)r * a.experts;
    float norm = 0.0f;
    uint32_t any = 0u;
    for (int s = 0; s < p.splits; ++s) norm += token_part[s * kTcTokens + t], any |= token_any[s * kTcTokens + t];
    // (squares that may have underflowed bound nothing; a token of zeros has exact logits)
    norm = norm > 0x1p-100f ? sqrtf(norm) * kBand<R> : INFINITY;
    if (tid == 0) doubtful = 0;
    for (int e = tid; e < a.experts; e += kRouteThreads) scores[e] = (float)route_score(a, l[e], e);
    __syncthreads();
    for (int e = any ? tid : a.experts; e < a.experts; e += kRouteThreads) {
      const float s = scores[e], own = norm * row_norm[e];
      int before = 0;
      bool near = false;
      for (int o = 0; o < a.experts; ++o) {
        // scores' distance that arithmetic explains (a sigmoid's slope is at most 1/4; 2^-22 for the scores' own roundings)
        const float band = (own + norm * row_norm[o]) * (a.sigmoid ? 0.25f : 1.0f) + 0x1p-22f * (fabsf(s) + fabsf(scores[o]));
        const float d = scores[o] - s;
        before += d > band;
        near |= o != e && !(fabsf(d) > band);
      }
      if (near && before < a.top_k) list[atomicAdd(&doubtful, 1)] = e;
    }
    __syncthreads();
    const int count = doubtful;
    for (int i = warp; i < count; i += kRouteWarps) {
      const int e = list[i];
      const double v = exact_dot(x + (int64_t)t * a.x_stride, static_cast<const R *>(a.router) + (int64_t)e * a.router_stride, 0, eighths, lane);
      if (lane == 0) l[e] = v;
    }
    __syncthreads();
    choose(a, t0 + t, l, reinterpret_cast<uint64_t *>(sums), best, partial);
  }
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
  return ((size_t)std::max(p.splits * p.per * g, p.a.experts) + (size_t)((g + kRouteCtas - 1) / kRouteCtas) * p.a.experts) * sizeof(double);
}

size_t route_tc_smem(const RouteLaunch &p) {
  const int rows = (p.per + 15) / 16 * 16, e = p.a.experts;
  return ((size_t)std::max(p.splits * rows * kTcTokens, 2 * e) + 2 * (size_t)e) * sizeof(double) +
         ((size_t)e + (size_t)p.splits * (rows + 2 * kTcTokens)) * sizeof(float);
}

}  // namespace

cudaError_t prepare_route_kernels() {
  // splits * rows <= 256 rows of 16 tokens, and 1024 experts
  const int most = (256 * kTcTokens + 2 * kMaxExperts) * 8 + (kMaxExperts + 256 + kRouteWarps * 2 * kTcTokens) * 4;
  const cudaError_t e = cudaFuncSetAttribute(k_moe_route_tc<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(k_moe_route_tc<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

cudaError_t launch_route(const RouteArgs &a, int sms, cudaStream_t st) {
  RouteLaunch p = {a, (a.experts + kRouteCtas - 1) / kRouteCtas, 1};
  p.splits = std::max(1, std::min<int>(kRouteWarps / p.per, (int)(a.hidden / 256)));
  // The tensor cores where they fill their tiles.  Measured (us): XXX
  const bool tc = a.tokens >= 32 && a.experts >= 64;
  if (tc) {
    const int tiles = (p.per + 15) / 16;
    p.splits = std::min(kRouteWarps / tiles, (int)((a.hidden + 31) / 32));
  }
  // as few tokens per cluster as one wave of CTAs allows: a router row's way
  // through L2 is shared by a cluster's tokens, but a lane's work is theirs together
  int g = tc ? kTcTokens : 1;
  while (!tc && g < 8 && (a.tokens + g - 1) / g * kRouteCtas > 2 * sms) g *= 2;
  const int64_t groups = (a.tokens + g - 1) / g;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kRouteCtas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * kRouteCtas));
  cfg.blockDim = dim3(kRouteThreads);
  cfg.dynamicSmemBytes = tc ? route_tc_smem(p) : route_smem(p, g);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  if (tc) return a.fp32 ? cudaLaunchKernelEx(&cfg, k_moe_route_tc<float>, p) : cudaLaunchKernelEx(&cfg, k_moe_route_tc<__nv_bfloat16>, p);
  return with_route(a.fp32, g, [&](auto *k) { return cudaLaunchKernelEx(&cfg, k, p); });
}

}  // namespace nvfp4
