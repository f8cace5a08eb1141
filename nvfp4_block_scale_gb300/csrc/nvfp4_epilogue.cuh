// nvfp4_epilogue.cuh -- the epilogue of the W4A16 product: alpha, bias,
// activation, gate and residual on one fp32 sum, rounded once to bf16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/nvfp4.h"
#include "nvfp4_internal.h"

namespace nvfp4 {

// The activations by their formulas, with CUDA's own exp, tanh and erf.
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case NVFP4_ACT_RELU: return v < 0.0f ? 0.0f : v;
    case NVFP4_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    case NVFP4_ACT_GELU_TANH:
      return 0.5f * v * (1.0f + tanhf(0.79788456080286536f * fmaf(0.044715f * v * v, v, v)));
    case NVFP4_ACT_SILU: return __fdiv_rn(v, 1.0f + expf(-v));
    default: return v;
  }
}

// Finishes output (b, r) from its sum over the columns.
__device__ __forceinline__ void finish(const LinearArgs &a, float alpha, int b, int64_t r, float sum) {
  float v = alpha * sum;
  if (a.bias) v += __bfloat162float(static_cast<const __nv_bfloat16 *>(a.bias)[r]);
  v = activate(v, a.act);
  if (a.gate) v *= __bfloat162float(static_cast<const __nv_bfloat16 *>(a.gate)[b * a.gate_stride + r]);
  if (a.residual) v += __bfloat162float(static_cast<const __nv_bfloat16 *>(a.residual)[b * a.residual_stride + r]);
  static_cast<__nv_bfloat16 *>(a.y)[b * a.y_stride + r] = __float2bfloat16(v);
}

}  // namespace nvfp4
