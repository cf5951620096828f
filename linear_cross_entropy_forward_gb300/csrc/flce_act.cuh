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
};

__device__ __forceinline__ float sigmoid_fast(float x) {
  return fast_rcp(1.0f + fast_ex2(-kLog2e * x));
}

// tanh(u) = 2 sigmoid(2 u) - 1, so z / 2 (1 + tanh(u)) = z sigmoid(2 u): no cancellation
// where the tanh is near -1.
constexpr float kGeluK = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case FLCE_ACT_RELU: return z < 0.0f ? 0.0f : z;  // NaN stays
    case FLCE_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.7071067811865476f));
    case FLCE_ACT_GELU_TANH: return z * sigmoid_fast(2.0f * kGeluK * fmaf(kGeluA * z, z * z, z));
    case FLCE_ACT_SILU: return z * sigmoid_fast(z);
    default: return z;
  }
}

__device__ __forceinline__ float activate_slope(float z, int act) {
  switch (act) {
    case FLCE_ACT_RELU: return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    case FLCE_ACT_GELU: {
      const float cdf = 0.5f * (1.0f + erff(z * 0.7071067811865476f));
      return fmaf(z, 0.3989422804014327f * fast_ex2(-0.5f * kLog2e * z * z), cdf);
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

// Eight neighbouring sums of a row that starts at element `base`, all arrays 16-byte aligned there.
__device__ __forceinline__ void linear_store8(const LinearOut& o, int64_t base, int col,
                                              float (&v)[8]) {
  if (o.bias) {
    float b[8];
    if (reinterpret_cast<uintptr_t>(o.bias) & 15) {
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = __bfloat162float(o.bias[col + i]);
    } else {
      unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(o.bias + col)), b);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  if (o.preact) *reinterpret_cast<uint4*>(o.preact + base + col) = pack_bf16x8(v);
  switch (o.act) {  // outside the loops: one copy of each activation's code
    case FLCE_ACT_NONE: break;
    case FLCE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = activate(v[i], FLCE_ACT_RELU);
      break;
    case FLCE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = activate(v[i], FLCE_ACT_GELU);
      break;
    case FLCE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = activate(v[i], FLCE_ACT_GELU_TANH);
      break;
    default:
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = activate(v[i], FLCE_ACT_SILU);
  }
  if (o.out_f32) {
    float* y = static_cast<float*>(o.y) + base + col;
    if (o.residual) {
      const float4* r = reinterpret_cast<const float4*>(static_cast<const float*>(o.residual) + base + col);
      const float4 r0 = r[0], r1 = r[1];
      v[0] += r0.x; v[1] += r0.y; v[2] += r0.z; v[3] += r0.w;
      v[4] += r1.x; v[5] += r1.y; v[6] += r1.z; v[7] += r1.w;
    }
    reinterpret_cast<float4*>(y)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(y)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    if (o.residual) {
      float r[8];
      unpack_bf16x8(*reinterpret_cast<const uint4*>(
                        static_cast<const __nv_bfloat16*>(o.residual) + base + col), r);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(o.y) + base + col) = pack_bf16x8(v);
  }
}

// One sum, of row `base` and column col.
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
