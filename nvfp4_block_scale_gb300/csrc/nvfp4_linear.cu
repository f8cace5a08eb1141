// nvfp4_linear.cu -- the W4A16 product with its epilogue:
//   y[b][r] = bf16( residual + gate * act( alpha * sum_c q Delta x[b][c] + bias ) ).
//
// One warp per row and group of kLinVecs vectors, a lane every 32nd block of
// 16 columns, fp32 sums joined by a butterfly.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"
#include "nvfp4_epilogue.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {

constexpr int kLinWarps = 8;
constexpr int kLinVecs = 4;

__device__ __forceinline__ float e2m1_value(uint32_t n) {
  const float m = (n & 6u) ? (float)(2u + (n & 1u)) * 0.5f * (float)(1u << ((n & 7u) >> 1)) * 0.5f : 0.5f * (float)(n & 1u);
  return n & 8u ? -m : m;
}

__global__ void __launch_bounds__(kLinWarps * 32) k_linear(const __grid_constant__ LinearArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kLinWarps + (threadIdx.x >> 5);
  const int b0 = blockIdx.y * kLinVecs;
  if (row >= a.rows) return;
  const int64_t nblk = a.cols / 16;
  float acc[kLinVecs] = {};
  for (int64_t j = lane; j < nblk; j += 32) {
    const uint2 c = reinterpret_cast<const uint2 *>(a.codes)[row * nblk + j];
    const float s = e4m3_value(a.scales[row * nblk + j]);
    for (int i = 0; i < 16; ++i) {
      const float w = e2m1_value(((i < 8 ? c.x : c.y) >> (4 * (i & 7))) & 15u) * s;
#pragma unroll
      for (int v = 0; v < kLinVecs; ++v)
        if (b0 + v < a.batch)
          acc[v] = fmaf(w, __bfloat162float(static_cast<const __nv_bfloat16 *>(a.x)[(b0 + v) * a.x_stride + 16 * j + i]),
                        acc[v]);
    }
  }
#pragma unroll
  for (int v = 0; v < kLinVecs; ++v) {
    for (int o = 16; o > 0; o >>= 1) acc[v] += __shfl_xor_sync(0xFFFFFFFFu, acc[v], o);
    if (lane == 0 && b0 + v < a.batch) finish(a, *a.alpha, b0 + v, row, acc[v]);
  }
}

size_t linear_workspace_bytes(int64_t rows, int64_t cols, int batch, int sms) {
  return kCounterBytes + (batch > 16 ? gemm_tc_workspace_bytes(rows, cols, batch, sms) : 0);
}

cudaError_t launch_linear(const LinearArgs &a, int sms, void *ws, cudaStream_t st) {
  if (a.cols > 0 && a.batch > 16) {
    float *part = reinterpret_cast<float *>(static_cast<char *>(ws) + kCounterBytes);
    const cudaError_t e = launch_gemm_tc(a.codes, a.scales, nullptr, a.rows, a.cols, a.x, a.x_stride, a.batch, sms, part,
                                         -1, st);
    return e != cudaSuccess ? e : launch_linear_reduce(part, a, sms, st);
  }
  const int64_t gx = (a.rows + kLinWarps - 1) / kLinWarps;
  if (gx > INT32_MAX) return cudaErrorInvalidValue;
  k_linear<<<dim3((unsigned)gx, (unsigned)((a.batch + kLinVecs - 1) / kLinVecs)), kLinWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace nvfp4
