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
  for (int g = rank, row = 0; g < tokens; g += kRouteCtas, ++row) {
    double *l = logits + (size_t)row * a.experts;
    uint64_t *keys = reinterpret_cast<uint64_t *>(sums);  // (the sums are spent)
    for (int e = tid; e < a.experts; e += kRouteThreads) {
      double score = l[e];
      if (a.sigmoid) score = 1.0 / (1.0 + exp(-score)) + (a.bias ? (double)a.bias[e] : 0.0);
      keys[e] = score_key(score);
    }
    if (tid < kMaxTopK) best[tid] = 0;
    __syncthreads();
    for (int e = tid; e < a.experts; e += kRouteThreads) {
      const uint64_t k = keys[e];
      int before = 0;
      for (int o = 0; o < a.experts; ++o) before += keys[o] > k || (keys[o] == k && o < e);
      if (before < a.top_k) best[before] = e;
    }
    // softmax: its maximum is the first choice's logit; its sum in a fixed order
    __syncthreads();
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
        const int64_t at = (t0 + g) * a.top_k + lane;
        a.ids[at] = e;
        a.weights[at] = __fdiv_rn(w, z) * a.scale;
      }
    }
    __syncthreads();
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

}  // namespace

cudaError_t launch_route(const RouteArgs &a, int sms, cudaStream_t st) {
  RouteLaunch p = {a, (a.experts + kRouteCtas - 1) / kRouteCtas, 1};
  p.splits = std::max(1, std::min<int>(kRouteWarps / p.per, (int)(a.hidden / 256)));
  // as few tokens per cluster as one wave of CTAs allows: a router row's way
  // through L2 is shared by a cluster's tokens, but a lane's work is theirs together
  int g = 1;
  while (g < 8 && (a.tokens + g - 1) / g * kRouteCtas > 2 * sms) g *= 2;
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
  cfg.dynamicSmemBytes = route_smem(p, g);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return with_route(a.fp32, g, [&](auto *k) { return cudaLaunchKernelEx(&cfg, k, p); });
}

}  // namespace nvfp4
