// nvfp4_epilogue.cuh -- what the kernels of nvfp4_linear share: f16 weights
// from codes and scales, and the epilogue (alpha, bias, activation, gate and
// residual on one fp32 sum, rounded once to bf16).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/nvfp4.h"
#include "nvfp4_internal.h"

namespace nvfp4 {

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Eight E2M1 codes -> four f16 pairs (exact).
__device__ __forceinline__ void e2m1x8_f16(uint32_t c, uint32_t (&w)[4]) {
  asm("{\n\t.reg .b8 t, u, v, x;\n\tmov.b32 {t, u, v, x}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, u;\n\tcvt.rn.f16x2.e2m1x2 %2, v;\n\tcvt.rn.f16x2.e2m1x2 %3, x;\n\t}"
      : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(c));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }  // |e| <= 126

// The activations by their formulas, with CUDA's own exp, tanh and erf.  One
// branch for all values: a branch per value would put every function's code
// between two values, and waiting for instructions then costs more than the
// arithmetic.
template <int COUNT>
__device__ __forceinline__ void activate(float (&v)[COUNT], int act) {
  switch (act) {
    case NVFP4_ACT_RELU:
#pragma unroll
      for (int i = 0; i < COUNT; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];
      break;
    case NVFP4_ACT_GELU:
#pragma unroll
      for (int i = 0; i < COUNT; ++i) v[i] = 0.5f * v[i] * (1.0f + erff(v[i] * 0.70710678118654752f));
      break;
    case NVFP4_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < COUNT; ++i)
        v[i] = 0.5f * v[i] * (1.0f + tanhf(0.79788456080286536f * fmaf(0.044715f * v[i] * v[i], v[i], v[i])));
      break;
    case NVFP4_ACT_SILU:
#pragma unroll
      for (int i = 0; i < COUNT; ++i) v[i] = __fdiv_rn(v[i], 1.0f + expf(-v[i]));
      break;
    default: break;
  }
}

// Finishes COUNT outputs from their sums over the columns (times 2^-up; see
// the callers): output i is (b(i), r(i)), skipped where ok(i) is false.  All
// gates and residuals are read before the first output is written: y may be
// the residual, so the compiler could not move them itself, and each would
// wait for memory in turn.
template <int COUNT, typename Ok, typename B, typename R>
__device__ __forceinline__ void finish(const LinearArgs &a, float alpha, const float (&sum)[COUNT], Ok ok, B b, R r) {
  const __nv_bfloat16 *bias = static_cast<const __nv_bfloat16 *>(a.bias), *gate = static_cast<const __nv_bfloat16 *>(a.gate),
                      *res = static_cast<const __nv_bfloat16 *>(a.residual);
  const __nv_bfloat16 zero = __float2bfloat16(0.0f);
  __nv_bfloat16 bi[COUNT], ga[COUNT], re[COUNT];
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    bi[i] = bias && ok(i) ? bias[r(i)] : zero;
    ga[i] = gate && ok(i) ? gate[b(i) * a.gate_stride + r(i)] : zero;
    re[i] = res && ok(i) ? res[b(i) * a.residual_stride + r(i)] : zero;
  }
  float v[COUNT];
#pragma unroll
  for (int i = 0; i < COUNT; ++i) v[i] = bias ? alpha * sum[i] + __bfloat162float(bi[i]) : alpha * sum[i];
  activate(v, a.act);
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    if (gate) v[i] *= __bfloat162float(ga[i]);
    if (res) v[i] += __bfloat162float(re[i]);
    if (ok(i)) static_cast<__nv_bfloat16 *>(a.y)[b(i) * a.y_stride + r(i)] = __float2bfloat16(v[i]);
  }
}

// The same for COUNT consecutive vectors b .. of one row.
template <int COUNT>
__device__ __forceinline__ void finish_row(const LinearArgs &a, float alpha, float (&v)[COUNT], int64_t b, int64_t r) {
  const __nv_bfloat16 *gate = static_cast<const __nv_bfloat16 *>(a.gate) + b * a.gate_stride + r,
                      *res = static_cast<const __nv_bfloat16 *>(a.residual) + b * a.residual_stride + r;
  const int n = a.batch - (int)b;  // vectors that exist
  __nv_bfloat16 ga[COUNT], re[COUNT];
  if (a.gate) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) ga[i] = gate[(i < n ? i : 0) * a.gate_stride];
  }
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) re[i] = res[(i < n ? i : 0) * a.residual_stride];
  }
  const float bias = a.bias ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.bias)[r]) : 0.0f;
#pragma unroll
  for (int i = 0; i < COUNT; ++i) v[i] = a.bias ? alpha * v[i] + bias : alpha * v[i];
  activate(v, a.act);
  __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y) + b * a.y_stride + r;
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    if (a.gate) v[i] *= __bfloat162float(ga[i]);
    if (a.residual) v[i] += __bfloat162float(re[i]);
    if (i < n) y[i * a.y_stride] = __float2bfloat16(v[i]);
  }
}

// Whether rows r .. r + 7 (r a multiple of 8) of every operand lie in one
// aligned 16-byte word.
__device__ __forceinline__ bool rows8_aligned(const LinearArgs &a) {
  uintptr_t bits = reinterpret_cast<uintptr_t>(a.y) | (uintptr_t)(2 * a.y_stride);
  if (a.gate) bits |= reinterpret_cast<uintptr_t>(a.gate) | (uintptr_t)(2 * a.gate_stride);
  if (a.residual) bits |= reinterpret_cast<uintptr_t>(a.residual) | (uintptr_t)(2 * a.residual_stride);
  if (a.bias) bits |= reinterpret_cast<uintptr_t>(a.bias);
  return (bits & 15) == 0;
}

// The same for rows r .. r + 7 of vector b, 16 bytes at a time.
__device__ __forceinline__ void finish_rows8(const LinearArgs &a, float alpha, float (&v)[8], int64_t b, int64_t r) {
  auto load = [&](const void *p, int64_t at) { return *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + at); };
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint4 bi = a.bias ? load(a.bias, r) : zero, ga = a.gate ? load(a.gate, b * a.gate_stride + r) : zero,
              re = a.residual ? load(a.residual, b * a.residual_stride + r) : zero;
  auto get = [](const uint4 &u, int i) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = a.bias ? alpha * v[i] + get(bi, i) : alpha * v[i];
  activate(v, a.act);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (a.gate) v[i] *= get(ga, i);
    if (a.residual) v[i] += get(re, i);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
  *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.y) + b * a.y_stride + r) = make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace nvfp4
