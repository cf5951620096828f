// The epilogue of a dense layer: bias, activation and residual on fp32 sums.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/flce.h"
#include "flce_device.cuh"

namespace flce {

// Where a dense layer's output goes: y[M, N] (row length ld = N) = act(z) + residual, and z itself
// in bf16 for the backward (preact), each pointer but y or NULL.
struct LinearOut {
  const __nv_bfloat16* bias;
  const void* residual;
  void* y;
  __nv_bfloat16* preact;
  int64_t ld;
  int32_t act;
  int32_t out_f32;
  int32_t wide;  // rows and arrays are 32-byte aligned, 16 columns at a time
};

__device__ __forceinline__ float sigmoid_fast(float x) {
  return fast_rcp(1.0f + fast_ex2(-kLog2e * x));
}

// tanh(u) = 2 sigmoid(2 u) - 1, so z / 2 (1 + tanh(u)) = z sigmoid(2 u): no cancellation
// where the tanh is near -1.
constexpr float kGeluK = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// The lower tail Phi(-|z|) and e = exp(-z^2 / 2):  with x = |z| / sqrt(2),
// erfc(x) = exp(-x^2) g(1 / (1 + x / 3)) for a polynomial g, least squares reweighted towards the
// largest relative error of exp(x^2) erfc(x) on [0, 9]: 1.3e-7, 4e-7 with fp32's roundings.  One exponential and one
// reciprocal, no branch, and no cancellation where the tail is small.
__device__ __forceinline__ float normal_tail(float z, float& e) {
  const float t = fast_rcp(fmaf(fabsf(z), 0.7071067811865476f / 3.0f, 1.0f));
  e = fast_ex2(-0.5f * kLog2e * z * z);
  float g = -0.12484309822320938f;
  g = fmaf(g, t, 0.401925265789032f);
  g = fmaf(g, t, -0.26398417353630066f);
  g = fmaf(g, t, 0.33701184391975403f);
  g = fmaf(g, t, 0.08211106061935425f);
  g = fmaf(g, t, 0.19337718188762665f);
  g = fmaf(g, t, 0.1862521916627884f);
  g = fmaf(g, t, 0.1881496012210846f);
  return 0.5f * g * t * e;
}

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case FLCE_ACT_RELU: return z < 0.0f ? 0.0f : z;  // NaN stays
    case FLCE_ACT_GELU: {
      float e;
      const float tail = normal_tail(z, e);
      return z * (z > 0.0f ? 1.0f - tail : tail);
    }
    case FLCE_ACT_GELU_TANH: return z * sigmoid_fast(2.0f * kGeluK * fmaf(kGeluA * z, z * z, z));
    case FLCE_ACT_SILU: return z * sigmoid_fast(z);
    default: return z;
  }
}

__device__ __forceinline__ float activate_slope(float z, int act) {
  switch (act) {
    case FLCE_ACT_RELU: return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    case FLCE_ACT_GELU: {
      float e;
      const float tail = normal_tail(z, e);
      return fmaf(z, 0.3989422804014327f * e, z > 0.0f ? 1.0f - tail : tail);
    }
    case FLCE_ACT_GELU_TANH: {
      const float s = sigmoid_fast(2.0f * kGeluK * fmaf(kGeluA * z, z * z, z));
      const float du = 2.0f * kGeluK * fmaf(3.0f * kGeluA * z, z, 1.0f);
      return fmaf(z * s * (1.0f - s), du, s);
    }
    case FLCE_ACT_SILU: {
      const float s = sigmoid_fast(z);
      return s * fmaf(z, 1.0f - s, 1.0f);
    }
    default: return 1.0f;
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void unpack_bf16x8(const uint4& q, float (&x)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

template <int N>
__device__ __forceinline__ void activate_all(float (&v)[N], int act) {
  switch (act) {  // outside the loops: one copy of each activation's code
    case FLCE_ACT_NONE: break;
    case FLCE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate(v[i], FLCE_ACT_RELU);
      break;
    case FLCE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate(v[i], FLCE_ACT_GELU);
      break;
    case FLCE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate(v[i], FLCE_ACT_GELU_TANH);
      break;
    default:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = activate(v[i], FLCE_ACT_SILU);
  }
}

// Sixteen bf16 values to 32 aligned bytes: one full sector of L2.  (16 bytes at a time are two half
// sectors, and L2's traffic is what the tensor cores' operands need.)
__device__ __forceinline__ void store_sector(__nv_bfloat16* p, const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  st_global_v8(p, w);
}

// Sixteen neighbouring sums of a row that starts at element `base`, of which the first `cols` are
// the row's (16 or 8), all arrays 16-byte aligned there.
__device__ __forceinline__ void linear_store16(const LinearOut& o, int64_t base, int col, int cols,
                                               float (&v)[16]) {
  const bool all = cols >= 16;
  if (o.bias) {
    const __nv_bfloat16* p = o.bias + col;
    float b[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && !all) break;
      if (reinterpret_cast<uintptr_t>(p) & 15) {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = __bfloat162float(p[8 * h + i]);
      } else {
        unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(p) + h), b);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * h + i] += b[i];
    }
  }
  auto put = [&](__nv_bfloat16* p) {
    if (all && o.wide) {
      store_sector(p, v);
    } else {
      reinterpret_cast<uint4*>(p)[0] =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                     pack_bf16x2(v[6], v[7]));
      if (all)
        reinterpret_cast<uint4*>(p)[1] =
            make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]),
                       pack_bf16x2(v[12], v[13]), pack_bf16x2(v[14], v[15]));
    }
  };
  if (o.preact) put(o.preact + base + col);
  activate_all(v, o.act);
  if (o.out_f32) {
    float* y = static_cast<float*>(o.y) + base + col;
    const float* r = static_cast<const float*>(o.residual) + base + col;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      if (h >= 2 && !all) break;
      float4 u = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
      if (o.residual) {
        const float4 t = reinterpret_cast<const float4*>(r)[h];
        u.x += t.x; u.y += t.y; u.z += t.z; u.w += t.w;
      }
      v[4 * h] = u.x; v[4 * h + 1] = u.y; v[4 * h + 2] = u.z; v[4 * h + 3] = u.w;
      if (!(all && o.wide)) reinterpret_cast<float4*>(y)[h] = u;
    }
    if (all && o.wide) {
      st_global_v8f(y, v);
      st_global_v8f(y + 8, v + 8);
    }
  } else {
    if (o.residual) {
      const uint4* r = reinterpret_cast<const uint4*>(
          static_cast<const __nv_bfloat16*>(o.residual) + base + col);
      float t[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 1 && !all) break;
        unpack_bf16x8(r[h], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * h + i] += t[i];
      }
    }
    put(static_cast<__nv_bfloat16*>(o.y) + base + col);
  }
}

// One sum, element `at` of the output.
__device__ __forceinline__ void linear_store1(const LinearOut& o, int64_t at, float bias, float v) {
  v += bias;
  if (o.preact) o.preact[at] = __float2bfloat16_rn(v);
  v = activate(v, o.act);
  if (o.out_f32) {
    if (o.residual) v += static_cast<const float*>(o.residual)[at];
    static_cast<float*>(o.y)[at] = v;
  } else {
    if (o.residual) v += __bfloat162float(static_cast<const __nv_bfloat16*>(o.residual)[at]);
    static_cast<__nv_bfloat16*>(o.y)[at] = __float2bfloat16_rn(v);
  }
}

}  // namespace flce
