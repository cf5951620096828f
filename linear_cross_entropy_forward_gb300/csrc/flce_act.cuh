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

// Arrays that a call writes (NULL: none), of which nothing may be taken for a result if a wait runs out.
// Whole 2-byte elements from a 16-byte boundary on.
struct Results {
  void* p[2];
  int64_t bytes[2];
};

// Whether `left` rows (as many as `most` of them) of a column from element `at` on lie in the output.
__device__ __forceinline__ bool column_ok(const LinearOut& o, const Results& r, int64_t at, int left, int most) {
  const int rows = left < most ? left : most;
  return rows <= 0 || (at >= 0 && (at + (rows - 1) * o.ld) * (o.out_f32 ? 4 : 2) < r.bytes[0]);
}

// Every bit set is NaN in bf16 and in fp32.  By all threads of a block whose wait ran out, at its end: what
// it has left out is NaN then, and so is what other blocks finished before, seconds ago.
__device__ __forceinline__ void leave_nan(const Results& r) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint8_t* p = static_cast<uint8_t*>(r.p[k]);
    if (!p) continue;
    const int64_t whole = r.bytes[k] / 16 * 16;
    for (int64_t i = int64_t(threadIdx.x) * 16; i < whole; i += int64_t(blockDim.x) * 16)
      *reinterpret_cast<uint4*>(p + i) = make_uint4(~0u, ~0u, ~0u, ~0u);
    for (int64_t i = whole + threadIdx.x * 2; i < r.bytes[k]; i += blockDim.x * 2)
      *reinterpret_cast<uint16_t*>(p + i) = 0xffff;
  }
}

__device__ __forceinline__ float sigmoid_fast(float x) {
  return fast_rcp(1.0f + fast_ex2(-kLog2e * x));
}

// tanh(u) = 2 sigmoid(2 u) - 1, so z / 2 (1 + tanh(u)) = z sigmoid(2 u): no cancellation
// where the tanh is near -1.
constexpr float kGeluK = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// The lower tail Phi(-|z|) and e = exp(-z^2 / 2):  with x = |z| / sqrt(2),
// erfc(x) = exp(-x^2) g(1 / (1 + x / 3)) for a polynomial g, least squares reweighted towards the
// largest relative error of exp(x^2) erfc(x) on [0, 9]: 1.3e-7.  One exponential and one reciprocal, no branch, and
// no cancellation where the tail is small: GELU is 6e-7 off, relative to itself, from -2 on; below, the rounding of
// the exponent grows with it (1.3e-6 at -5, 7e-6 at -12, where the value is 1e-32).
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

// One column of TOKENS rows, `left` of which are there, element `at` of the output on.  The residual's
// bits are asked for ahead of the sums that they are added to, and all before any is looked at (a
// conversion beside its load waits for it, and so does a load behind a store).
template <int TOKENS>
__device__ __forceinline__ void linear_residual(const LinearOut& o, int64_t at, int left,
                                                uint32_t (&r)[TOKENS]) {
  if (!o.residual) return;
  if (o.out_f32) {
    const uint32_t* p = static_cast<const uint32_t*>(o.residual) + at;
    if (left >= TOKENS) {
#pragma unroll
      for (int i = 0; i < TOKENS; ++i) r[i] = p[i * o.ld];
    } else {
#pragma unroll
      for (int i = 0; i < TOKENS; ++i)
        if (i < left) r[i] = p[i * o.ld];
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(o.residual) + at;
    if (left >= TOKENS) {
#pragma unroll
      for (int i = 0; i < TOKENS; ++i) r[i] = p[i * o.ld];
    } else {
#pragma unroll
      for (int i = 0; i < TOKENS; ++i)
        if (i < left) r[i] = p[i * o.ld];
    }
  }
}
template <int TOKENS>
__device__ __forceinline__ void linear_store_column(const LinearOut& o, int64_t at, int left,
                                                    float bias, const uint32_t (&r)[TOKENS],
                                                    float (&v)[TOKENS]) {
  if (left <= 0) return;
#pragma unroll
  for (int i = 0; i < TOKENS; ++i) v[i] += bias;
  if (o.preact) {
    __nv_bfloat16* p = o.preact + at;
#pragma unroll
    for (int i = 0; i < TOKENS; ++i)
      if (i < left) p[i * o.ld] = __float2bfloat16_rn(v[i]);
  }
  activate_all(v, o.act);
  if (o.residual) {
    const int bits = o.out_f32 ? 0 : 16;
#pragma unroll
    for (int i = 0; i < TOKENS; ++i) v[i] += __uint_as_float(r[i] << bits);
  }
  if (o.out_f32) {
    float* p = static_cast<float*>(o.y) + at;
#pragma unroll
    for (int i = 0; i < TOKENS; ++i)
      if (i < left) p[i * o.ld] = v[i];
  } else {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(o.y) + at;
#pragma unroll
    for (int i = 0; i < TOKENS; ++i)
      if (i < left) p[i * o.ld] = __float2bfloat16_rn(v[i]);
  }
}

}  // namespace flce
