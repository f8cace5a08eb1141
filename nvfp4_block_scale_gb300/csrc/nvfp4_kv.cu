// nvfp4_kv.cu -- rotated append to a paged key-value cache.
//
// Per token: q and k heads are rotated by position, (a, b) -> (a cos - b sin,
// b cos + a sin), q goes to q_out, k and v to the token's slot of the cache
// (bf16, or E4M3 of value * fl(1 / scale)).  Every product and sum is rounded
// to fp32 separately (no fused multiply-add), so the stored codes are those
// of the elementary operations.
//
// Bound: HBM.  Each input is read once and each output written once with 16-
// or 8-byte accesses; the cosines and sines of a token are loaded once per
// thread and serve all of the heads that it handles.  8192 tokens (bf16 rows of
// 64 + 2 x 8 heads of 128 into an E4M3 cache) take 54.6 us, 5.9 TB/s; 3001 (bf16,
// heads of 256) 14.9 us, 5.0 TB/s; one 1.9 us, which is a launch.
//
// Work split: a thread handles one 16-dimension unit of several heads of one
// token: two runs of 8 consecutive dimensions that rotate into each other
// (dimensions 8u.. and rotary/2 + 8u..; 16 consecutive ones when interleaved
// or not rotated), always the same unit of each head so that the angles stay
// in registers.  A token's slot takes three dependent lookups (its position, its
// page, then the store), so the first head's loads go out before them and
// each further head's before the previous one is stored (3001 tokens: 15.8 us
// with all of a head's loads behind the lookups).
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "nvfp4_device.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {

constexpr int kAppendThreads = 128;

// Eight elements as they lie in memory, and their values.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  uint4 w[2];
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 w[1];
};
template <typename T>
__device__ __forceinline__ void load8(const T *p, Raw8<T> &v) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v.w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
}
__device__ __forceinline__ void values(const Raw8<float> &r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.w[i].x), v[4 * i + 1] = __uint_as_float(r.w[i].y);
    v[4 * i + 2] = __uint_as_float(r.w[i].z), v[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}
__device__ __forceinline__ void values(const Raw8<__nv_bfloat16> &r, float (&v)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void store8_bf16(__nv_bfloat16 *p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8_e4m3(uint8_t *p, const float (&v)[8], float r) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(w[i])
        : "f"(__fmul_rn(v[4 * i], r)), "f"(__fmul_rn(v[4 * i + 1], r)), "f"(__fmul_rn(v[4 * i + 2], r)),
          "f"(__fmul_rn(v[4 * i + 3], r)));
  *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

// grid: (tokens, head groups); blockDim.x = kAppendThreads, a multiple of the
// head_dim / 16 units of a head.
template <typename T, bool E4M3>
__global__ void __launch_bounds__(kAppendThreads) k_kv_append(const __grid_constant__ AppendArgs a) {
  const int D = a.kv.head_dim, units = D >> 4;
  const int u = threadIdx.x & (units - 1), lane_head = threadIdx.x / units, step = kAppendThreads / units;
  const int64_t tok = blockIdx.x;
  const int hk = a.kv.kv_heads, heads = a.q_heads + 2 * hk;
  const T *row = static_cast<const T *>(a.qkv) + tok * a.qkv_stride;

  // this thread's unit of a rotated head: dimensions d0.. and d1..
  const int half = a.rotary >> 1;
  const bool turns = u < (a.rotary >> 4);
  const int d0 = turns && !a.interleaved ? 8 * u : 16 * u;
  const int d1 = turns && !a.interleaved ? half + 8 * u : 16 * u + 8;
  auto place = [&](int h, int &e0, int &e1) {
    const bool value = h >= a.q_heads + hk;
    e0 = value ? 16 * u : d0;
    e1 = value ? 16 * u + 8 : d1;
  };
  Raw8<T> rx, ry;
  auto fetch = [&](int h) {
    int e0, e1;
    place(h, e0, e1);
    load8<T>(row + (int64_t)h * D + e0, rx);
    load8<T>(row + (int64_t)h * D + e1, ry);
  };
  const int h0 = blockIdx.y * step + lane_head, h_step = gridDim.y * step;
  if (h0 < heads) fetch(h0);

  const int seq = __ldg(a.seq + tok), pos = __ldg(a.pos + tok);
  const int entry = pos >> a.kv.page_shift;  // (arithmetic shift: a negative pos stays negative)
  bool ok = seq >= 0 && seq < a.sequences && pos >= 0 && entry < a.kv.table_width &&
            (a.rotary == 0 || pos < a.positions);
  int64_t page = ok ? __ldg(a.kv.table + seq * a.kv.table_stride + entry) : -1;
  ok = ok && page >= 0 && page < a.kv.pages;

  float c[8], s[8];
  if (turns && ok) {
    const float *cs = a.cos_sin + (int64_t)pos * a.rotary + 8 * u;
    Raw8<float> r;
    load8<float>(cs, r);
    values(r, c);
    load8<float>(cs + half, r);
    values(r, s);
  }
  const int in_page = pos & ((1 << a.kv.page_shift) - 1);
  __nv_bfloat16 *q_out = static_cast<__nv_bfloat16 *>(a.q_out) + tok * a.q_heads * D;

  for (int h = h0; h < heads; h += h_step) {
    const bool value = h >= a.q_heads + hk;
    int e0, e1;
    place(h, e0, e1);
    float x[8], y[8];
    values(rx, x);
    values(ry, y);
    if (h + h_step < heads) fetch(h + h_step);
    if (!ok) {
      if (h < a.q_heads) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.0f;
        store8_bf16(q_out + h * D + e0, x);
        store8_bf16(q_out + h * D + e1, x);
      }
      continue;
    }
    if (turns && !value) {
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // pair i: dimensions 2i, 2i + 1 of the 16
          float &p = i < 4 ? x[2 * i] : y[2 * i - 8], &q = i < 4 ? x[2 * i + 1] : y[2 * i - 7];
          const float t = __fsub_rn(__fmul_rn(p, c[i]), __fmul_rn(q, s[i]));
          q = __fadd_rn(__fmul_rn(q, c[i]), __fmul_rn(p, s[i]));
          p = t;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float t = __fsub_rn(__fmul_rn(x[i], c[i]), __fmul_rn(y[i], s[i]));
          y[i] = __fadd_rn(__fmul_rn(y[i], c[i]), __fmul_rn(x[i], s[i]));
          x[i] = t;
        }
      }
    }
    if (h < a.q_heads) {
      store8_bf16(q_out + h * D + e0, x);
      store8_bf16(q_out + h * D + e1, y);
      continue;
    }
    const int kh = value ? h - a.q_heads - hk : h - a.q_heads;
    const int64_t off = page * (value ? a.kv.v_page_stride : a.kv.k_page_stride) +
                        (((int64_t)kh << a.kv.page_shift) + in_page) * D;
    void *base = value ? a.kv.v : a.kv.k;
    if (E4M3) {
      const float *sc = value ? a.kv.v_scale : a.kv.k_scale;
      const float r = sc ? __fdiv_rn(1.0f, __ldg(sc + kh)) : 1.0f;
      store8_e4m3(static_cast<uint8_t *>(base) + off + e0, x, r);
      store8_e4m3(static_cast<uint8_t *>(base) + off + e1, y, r);
    } else {
      store8_bf16(static_cast<__nv_bfloat16 *>(base) + off + e0, x);
      store8_bf16(static_cast<__nv_bfloat16 *>(base) + off + e1, y);
    }
  }
}

cudaError_t launch_kv_append(const AppendArgs &a, int sms, cudaStream_t st) {
  const int units = a.kv.head_dim / 16, heads = a.q_heads + 2 * a.kv.kv_heads;
  const int groups = (heads * units + kAppendThreads - 1) / kAppendThreads;
  // few tokens: one pass over the heads per CTA, the heads spread over the
  // CTAs; many: one CTA per token, so that the angles are loaded once
  const dim3 grid((unsigned)a.tokens, a.tokens * groups <= 8 * sms ? (unsigned)groups : 1u);
  if (a.fp32) {
    if (a.kv.e4m3) k_kv_append<float, true><<<grid, kAppendThreads, 0, st>>>(a);
    else k_kv_append<float, false><<<grid, kAppendThreads, 0, st>>>(a);
  } else {
    if (a.kv.e4m3) k_kv_append<__nv_bfloat16, true><<<grid, kAppendThreads, 0, st>>>(a);
    else k_kv_append<__nv_bfloat16, false><<<grid, kAppendThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace nvfp4
