// nvfp4_attention.cu -- attention of one new token per sequence over a paged
// key-value cache.
//
// One CTA per query head and sequence; each warp takes every fourth token, a
// lane head_dim / 32 dimensions, with a running maximum and sum; the warps'
// parts meet in shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {

constexpr int kAttWarps = 4;

__device__ __forceinline__ float kv_value(const void *p, int64_t i, bool e4m3) {
  if (e4m3) return e4m3_value(static_cast<const uint8_t *>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

template <int D>
__global__ void __launch_bounds__(kAttWarps * 32) k_attend(const __grid_constant__ AttendArgs a) {
  constexpr int N = D / 32;
  __shared__ float sm[kAttWarps], sl[kAttWarps], so[kAttWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x, s = blockIdx.y, kh = h / (a.q_heads / a.kv.kv_heads);
  const int64_t cap = a.kv.table_width << a.kv.page_shift;
  const int64_t n = max((int64_t)0, min((int64_t)a.lengths[s], cap));
  const int64_t lo = a.window > 0 && n > a.window ? n - a.window : 0;
  const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + s * a.q_stride + (int64_t)h * D;
  float qv[N], o[N], m = -INFINITY, l = 0.0f;
  const float sc = a.scale * (a.kv.k_scale ? a.kv.k_scale[kh] : 1.0f);
  for (int i = 0; i < N; ++i) {
    qv[i] = __bfloat162float(q[lane + 32 * i]);
    o[i] = 0.0f;
  }
  for (int64_t t = lo + warp; t < n; t += kAttWarps) {
    const int64_t page = a.kv.table[s * a.kv.table_stride + (t >> a.kv.page_shift)];
    const bool in = page >= 0 && page < a.kv.pages;
    const int64_t row = (((int64_t)kh << a.kv.page_shift) + (t & ((1 << a.kv.page_shift) - 1))) * D + lane;
    float dot = 0.0f;
    for (int i = 0; i < N; ++i)
      dot = fmaf(qv[i], in ? kv_value(a.kv.k, page * a.kv.k_page_stride + row + 32 * i, a.kv.e4m3) : 0.0f, dot);
    for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, x);
    dot *= sc;
    const float m1 = fmaxf(m, dot), base = m1 == -INFINITY ? 0.0f : m1;
    const float f = expf(m - base), p = expf(dot - base);
    l = l * f + p;
    for (int i = 0; i < N; ++i)
      o[i] = o[i] * f + p * (in ? kv_value(a.kv.v, page * a.kv.v_page_stride + row + 32 * i, a.kv.e4m3) : 0.0f);
    m = m1;
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  for (int i = 0; i < N; ++i) so[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float top = -INFINITY, sum = 0.0f;
  for (int w = 0; w < kAttWarps; ++w) top = fmaxf(top, sm[w]);
  const float base = top == -INFINITY ? 0.0f : top;
  for (int w = 0; w < kAttWarps; ++w) sum += sl[w] * expf(sm[w] - base);
  const int64_t at = (int64_t)s * a.q_heads + h;
  for (int d = threadIdx.x; d < D; d += kAttWarps * 32) {
    float v = 0.0f;
    for (int w = 0; w < kAttWarps; ++w) v += so[w][d] * expf(sm[w] - base);
    v = sum == 0.0f ? 0.0f : v * (a.kv.v_scale ? a.kv.v_scale[kh] : 1.0f) / sum;
    static_cast<__nv_bfloat16 *>(a.out)[at * D + d] = __float2bfloat16(v);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[at] = base + logf(sum);
}

size_t attend_workspace_bytes(const KvArgs &, int, int) { return kCounterBytes; }

cudaError_t launch_attend(const AttendArgs &a, int, void *, cudaStream_t st) {
  const dim3 grid((unsigned)a.q_heads, (unsigned)a.sequences);
  switch (a.kv.head_dim) {
    case 64: k_attend<64><<<grid, kAttWarps * 32, 0, st>>>(a); break;
    case 128: k_attend<128><<<grid, kAttWarps * 32, 0, st>>>(a); break;
    default: k_attend<256><<<grid, kAttWarps * 32, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace nvfp4
