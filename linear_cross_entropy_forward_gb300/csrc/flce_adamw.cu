// AdamW over many tensors in one launch, and the norm of their gradients.
//
//   g' = c g,  c = grad_scale min(1, max_norm / (norm + 1e-6))
//   m = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// Elementwise over tensors of all sizes: bound by the bytes of the weights, the gradients
// and the states, each read and written once.  A unit is 2048 elements of one tensor, 8 per
// thread; the blocks of one wave share all tensors' units in contiguous runs (a run's tensor
// is searched once, then followed).  The table of tensors travels in the launch's arguments,
// so a step copies nothing from the host and can be captured.
//
// States: fp32, or 8 bits: m and s = sqrt(v) (half the range of exponents that v needs) as
// e4m3 codes in units of 1 / 448 of the largest of each 128 elements, which 16 lanes hold.
// A magnitude goes to one of its two neighbouring codes, the upper one with the probability
// that keeps the mean: rounded to nearest, a decay of 0.1 % a step would never leave a code
// whose neighbours are 6 to 12 % away.  The random bits are a mixing of (seed, step, element),
// so a step repeats bit for bit.  s > 0 is never rounded to 0 (m / eps would follow).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "flce_device.cuh"
#include "flce_host.h"

namespace flce {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                    // elements per thread
constexpr int kUnit = kThreads * kPer;     // elements per unit
constexpr int kBlockElems = 128;           // elements per scale of the 8-bit states
constexpr int kSmall = 40, kLarge = 680;   // tensors in one launch's arguments
constexpr float kTiny = 7.703719777548943e-34f;  // 2^-110: blocks below are held as zeros
constexpr int kNormBlocks = 4;             // blocks per SM of the norm
constexpr int64_t kMaxUnits = int64_t(1) << 31;

struct Slot {
  void* param;
  const void* grad;
  int64_t n, offset;
  float decay;
  int32_t kind;  // dtype * 2 + (gradient in fp32 beside a 16-bit parameter)
};

template <int CAP>
struct Table {
  int32_t count;
  uint32_t units;
  uint32_t first[CAP];  // first unit of each tensor
  Slot slot[CAP];
};

struct StepArgs {
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* s_scale;
  const float* lr_ptr;
  const float* norm;
  int64_t* step;
  uint32_t* ticket;
  float lr, beta1, omb1, beta2, rb2, romb2, eps, grad_scale, max_norm;  // r: root of
  double ln1, ln2;  // logarithms of the betas
  uint32_t seed;
  int32_t skip, last;
};

struct NormArgs {
  double* partial;   // of all launches of the call
  uint32_t* ticket;
  float* norm;
  float scale;
  int32_t base, last;
};

// ------------------------------------------------------------------ elements
template <typename T>
__device__ __forceinline__ float widen(T x) {
  if constexpr (std::is_same_v<T, float>) return x;
  else if constexpr (std::is_same_v<T, __nv_bfloat16>) return __bfloat162float(x);
  else return __half2float(x);
}
template <typename T>
__device__ __forceinline__ T narrow(float x) {
  if constexpr (std::is_same_v<T, float>) return x;
  else if constexpr (std::is_same_v<T, __nv_bfloat16>) return __float2bfloat16_rn(x);
  else return __float2half_rn(x);
}

__device__ __forceinline__ void ld_cs_v8(const float* p, float (&x)[kPer]) {
  asm volatile("ld.global.cs.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]),
                 "=f"(x[6]), "=f"(x[7])
               : "l"(p));
}

// 8 elements from p, `n` of them there (the others 0)
template <typename T>
__device__ __forceinline__ void load8(const T* p, int64_t n, float (&x)[kPer]) {
  if (n >= kPer && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    if constexpr (sizeof(T) == 4) {
      if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        ld_cs_v8(reinterpret_cast<const float*>(p), x);
        return;
      }
    }
    alignas(16) T t[kPer];
    uint4* q = reinterpret_cast<uint4*>(t);
#pragma unroll
    for (int i = 0; i < int(sizeof(T) * kPer / 16); ++i)
      q[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = widen(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = i < n ? widen(p[i]) : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int64_t n, const float (&x)[kPer]) {
  if (n >= kPer && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    if constexpr (sizeof(T) == 4) {
      if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        st_global_cs_v8f(reinterpret_cast<float*>(p), x);
        return;
      }
    }
    alignas(16) T t[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) t[i] = narrow<T>(x[i]);
    const uint4* q = reinterpret_cast<const uint4*>(t);
#pragma unroll
    for (int i = 0; i < int(sizeof(T) * kPer / 16); ++i)
      __stcs(reinterpret_cast<uint4*>(p) + i, q[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < n) p[i] = narrow<T>(x[i]);
  }
}

// ------------------------------------------------------------------ 8-bit states
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

__device__ __forceinline__ uint16_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void from_e4m3_pair(uint16_t c, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  const __half2 v = *reinterpret_cast<const __half2*>(&h);
  lo = __low2float(v);
  hi = __high2float(v);
}

__device__ __forceinline__ void unpack8(uint2 c, float (&x)[kPer]) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    from_e4m3_pair(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))), x[2 * i], x[2 * i + 1]);
}

// |x| unit to an e4m3 value, the upper neighbour where the 20 random bits carry into the
// code's last place.  e4m3 keeps 3 of fp32's 23 mantissa bits; below 2^-6 its step is that of
// [2^-6, 2^-5), so adding 2^-6 first makes the same 20 bits the ones cut off.
__device__ __forceinline__ float round_up_or_down(float a, uint32_t r20) {
  const float low = a < 0.015625f ? 0.015625f : 0.0f;
  return __uint_as_float((__float_as_uint(a + low) + r20) & 0xFFF00000u) - low;
}

// The largest of 16 lanes' x (lanes 0-15 and 16-31 of a warp hold a block each).
__device__ __forceinline__ float block_max(float x) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}

// Codes of 8 elements and their block's scale.  ROOT: non-negative values, 0 for 0 alone.
template <bool ROOT>
__device__ __forceinline__ uint2 pack8(const float (&x)[kPer], const uint32_t (&r)[kPer],
                                       float& scale) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) top = fmaxf(top, fabsf(x[i]));
  top = block_max(top);
  const bool none = top < kTiny;
  const float unit = none ? 0.0f : __fdiv_rn(448.0f, top);
  scale = none ? 0.0f : __fdiv_rn(top, 448.0f);
  float y[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    // a quotient just above 448, carried up to 480, is 448 again as a code
    const float a = fabsf(x[i]) * unit;
    float q = round_up_or_down(a, r[i]);
    if (ROOT) {
      if (a > 0.0f && q == 0.0f) q = 0.001953125f;  // 2^-9, the smallest code
      y[i] = q;
    } else {
      y[i] = copysignf(q, x[i]);
    }
  }
  uint2 c;
  c.x = e4m3_pair(y[0], y[1]) | (static_cast<uint32_t>(e4m3_pair(y[2], y[3])) << 16);
  c.y = e4m3_pair(y[4], y[5]) | (static_cast<uint32_t>(e4m3_pair(y[6], y[7])) << 16);
  return c;
}

// ------------------------------------------------------------------ the step
// m = b1 m + cm grad;  v = (rb2 s)^2 + (cs grad)^2 (8 bits) or b2 v + (cs grad)^2, with the root
// s = sqrt(v);  p = p (1 - lr wd) - step_size m / (root_c2 s + eps)
struct Coef {
  float beta1, beta2, rb2, cm, cs, eps, lr, step_size, root_c2;
  uint32_t key;
};

__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));  // subnormals are kept
  return y;
}

// One thread's 8 elements: element e0 of the tensor on, the state's offset `at`.
template <typename P, typename G, bool STATE8, bool MASTER>
__device__ __forceinline__ void update8(const Slot& s, const StepArgs& a, const Coef& k,
                                        int64_t e0) {
  const int64_t left = s.n - e0, at = s.offset + e0;
  // past the tensor's last block of 128 there is no state; 16 lanes leave or stay together
  const bool in = (e0 & ~int64_t(kBlockElems - 1)) < s.n;
  float g[kPer], w[kPer], m[kPer], v[kPer];
  float scale_m = 0.0f, scale_s = 0.0f;
  uint2 cm = make_uint2(0, 0), cs = make_uint2(0, 0);
  if (in) {
    load8(static_cast<const G*>(s.grad) + e0, left, g);
    if constexpr (MASTER) load8(a.master + at, kPer, w);
    else load8(static_cast<const P*>(s.param) + e0, left, w);
    if constexpr (STATE8) {
      cm = __ldcs(reinterpret_cast<const uint2*>(static_cast<uint8_t*>(a.m) + at));
      cs = __ldcs(reinterpret_cast<const uint2*>(static_cast<uint8_t*>(a.v) + at));
      scale_m = a.m_scale[at / kBlockElems];
      scale_s = a.s_scale[at / kBlockElems];
    } else {
      load8(static_cast<const float*>(a.m) + at, kPer, m);
      load8(static_cast<const float*>(a.v) + at, kPer, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) g[i] = w[i] = m[i] = v[i] = 0.0f;
  }
  if constexpr (STATE8) {
    unpack8(cm, m);
    unpack8(cs, v);
  }
  const float shrink = 1.0f - k.lr * s.decay;
  const uint64_t shrink2 = f2_pack(shrink, shrink), minus = f2_pack(-k.step_size, -k.step_size),
                 eps2 = f2_pack(k.eps, k.eps), cm2 = f2_pack(k.cm, k.cm), cs2 = f2_pack(k.cs, k.cs),
                 root2 = f2_pack(k.root_c2, k.root_c2);
  const float keep_m = STATE8 ? k.beta1 * scale_m : k.beta1;
  const float keep_v = STATE8 ? k.rb2 * scale_s : k.beta2;
  const uint64_t keep_m2 = f2_pack(keep_m, keep_m), keep_v2 = f2_pack(keep_v, keep_v);
#pragma unroll
  for (int i = 0; i < kPer; i += 2) {
    const uint64_t x = f2_pack(g[i], g[i + 1]);
    const uint64_t m2 = f2_fma(x, cm2, f2_mul(f2_pack(m[i], m[i + 1]), keep_m2));
    const uint64_t y = f2_mul(x, cs2);
    uint64_t old = f2_mul(f2_pack(v[i], v[i + 1]), keep_v2);
    if constexpr (STATE8) old = f2_mul(old, old);
    const uint64_t v2 = f2_fma(y, y, old);
    float v0, v1, d0, d1;
    f2_unpack(v2, v0, v1);
    const float s0 = sqrt_approx(v0), s1 = sqrt_approx(v1);
    f2_unpack(f2_fma(f2_pack(s0, s1), root2, eps2), d0, d1);
    const uint64_t u = f2_mul(m2, f2_pack(fast_rcp(d0), fast_rcp(d1)));
    f2_unpack(f2_fma(u, minus, f2_mul(f2_pack(w[i], w[i + 1]), shrink2)), w[i], w[i + 1]);
    f2_unpack(m2, m[i], m[i + 1]);
    v[i] = STATE8 ? s0 : v0;
    v[i + 1] = STATE8 ? s1 : v1;
  }
  if constexpr (STATE8) {
    uint32_t r1[kPer], r2[kPer];
    const uint32_t key = mix(k.key + static_cast<uint32_t>(static_cast<uint64_t>(at) >> 32));
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t h = mix((static_cast<uint32_t>(at) + i) ^ key);
      r1[i] = h >> 12;
      r2[i] = (h * 0x9E3779B1u) >> 12;
    }
    cm = pack8<false>(m, r1, scale_m);
    cs = pack8<true>(v, r2, scale_s);
  }
  if (!in) return;
  if constexpr (MASTER) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i >= left) w[i] = 0.0f;  // the padding of the states stays zero
    store8(a.master + at, kPer, w);
  }
  store8(static_cast<P*>(s.param) + e0, left, w);
  if constexpr (STATE8) {
    __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + at), cm);
    __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + at), cs);
    if ((at & (kBlockElems - 1)) == 0) {
      a.m_scale[at / kBlockElems] = scale_m;
      a.s_scale[at / kBlockElems] = scale_s;
    }
  } else {
    store8(static_cast<float*>(a.m) + at, kPer, m);
    store8(static_cast<float*>(a.v) + at, kPer, v);
  }
}

// First and last unit of this block's run, and the tensor that holds the first.
template <int CAP>
__device__ __forceinline__ int find_run(const Table<CAP>& t, uint32_t& u, uint32_t& end) {
  const uint64_t U = t.units;
  u = static_cast<uint32_t>(U * blockIdx.x / gridDim.x);
  end = static_cast<uint32_t>(U * (blockIdx.x + 1) / gridDim.x);
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <bool STATE8, bool MASTER, int CAP>
__global__ void __launch_bounds__(kThreads)
    adamw_kernel(const __grid_constant__ Table<CAP> t, const __grid_constant__ StepArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t step = *a.step + 1;
  float c = a.grad_scale;
  bool skip = false;
  if (a.norm) {
    const float norm = *a.norm;
    skip = a.skip && !isfinite(norm);
    const float clip = a.max_norm / (norm + 1e-6f);
    if (a.max_norm > 0.0f && !(clip >= 1.0f)) c *= clip;  // a NaN norm leaves NaN
  }
  if (!skip) {
    Coef k;
    k.beta1 = a.beta1;
    k.beta2 = a.beta2;
    k.rb2 = a.rb2;
    k.cm = c * a.omb1;
    k.cs = c * a.romb2;
    k.eps = a.eps;
    k.lr = a.lr_ptr ? *a.lr_ptr : a.lr;
    // 1 - b^t = -(e^{t ln b} - 1): exact to fp32 for small t ln b too
    const double ts = static_cast<double>(step);
    k.step_size = k.lr / -expm1f(static_cast<float>(ts * a.ln1));
    k.root_c2 = sqrtf(1.0f / -expm1f(static_cast<float>(ts * a.ln2)));
    k.key = mix(a.seed + 0x9E3779B9u * static_cast<uint32_t>(step));
    uint32_t u, end;
    int i = find_run(t, u, end);
    for (; u < end; ++u) {
      while (i + 1 < t.count && t.first[i + 1] <= u) ++i;
      const Slot& s = t.slot[i];
      const int64_t e0 = static_cast<int64_t>(u - t.first[i]) * kUnit + threadIdx.x * kPer;
      switch (s.kind) {
        case 2 * FLCE_BF16:
          update8<__nv_bfloat16, __nv_bfloat16, STATE8, MASTER>(s, a, k, e0);
          break;
        case 2 * FLCE_BF16 + 1:
          update8<__nv_bfloat16, float, STATE8, MASTER>(s, a, k, e0);
          break;
        case 2 * FLCE_F16:
          update8<__half, __half, STATE8, MASTER>(s, a, k, e0);
          break;
        case 2 * FLCE_F16 + 1:
          update8<__half, float, STATE8, MASTER>(s, a, k, e0);
          break;
        default:
          update8<float, float, STATE8, MASTER>(s, a, k, e0);
      }
    }
  }
  // the last block to have read the step counts it, and leaves the ticket at 0
  if (a.last && threadIdx.x == 0 && !skip) {
    __threadfence();
    if (atomicAdd(a.ticket, 1u) == gridDim.x - 1) {
      *a.ticket = 0;
      *a.step = step;
    }
  }
}

// ------------------------------------------------------------------ the norm
// Sum of (scale g)^2: up to 512 squares in fp32, from there on in 64 bits (whose units are few:
// one addition per 8 squares took longer than the bytes), in a fixed order.
constexpr int kNormDepth = 4;  // units in flight
constexpr int kNormFold = 64;  // units whose squares a thread sums in fp32

__device__ __forceinline__ float squares(const float (&x)[kPer], float scale) {
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float y = scale * x[i];
    sum = fmaf(y, y, sum);
  }
  return sum;
}

// `units` units of one tensor from element e0 on (this thread's first)
template <typename G>
__device__ __forceinline__ double sum_units(const void* grad, int64_t n, int64_t e0, int64_t units,
                                            float scale) {
  const G* p = static_cast<const G*>(grad);
  double total = 0.0;
  for (int64_t u = 0; u < units; u += kNormFold) {
    const int64_t end = u + kNormFold < units ? u + kNormFold : units;
    float part[kNormDepth] = {};
    for (int64_t v = u; v < end; v += kNormDepth) {
      float x[kNormDepth][kPer];
#pragma unroll
      for (int d = 0; d < kNormDepth; ++d) {
        const int64_t e = e0 + (v + d) * kUnit;
        load8(p + e, v + d < end ? n - e : 0, x[d]);
      }
#pragma unroll
      for (int d = 0; d < kNormDepth; ++d) part[d] += squares(x[d], scale);
    }
    total += (part[0] + part[1]) + (part[2] + part[3]);
  }
  return total;
}

__device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.0;
  for (int i = 0; i < kThreads / 32; ++i) x += part[i];
  return x;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads)
    norm_kernel(const __grid_constant__ Table<CAP> t, const __grid_constant__ NormArgs a) {
  uint32_t u, end;
  int i = find_run(t, u, end);
  double total = 0.0;
  while (u < end) {
    while (i + 1 < t.count && t.first[i + 1] <= u) ++i;
    const Slot& s = t.slot[i];
    const uint32_t stop = i + 1 < t.count && t.first[i + 1] < end ? t.first[i + 1] : end;
    const int64_t e0 = static_cast<int64_t>(u - t.first[i]) * kUnit + threadIdx.x * kPer;
    const bool f32 = (s.kind & 1) || s.kind == 2 * FLCE_F32;
    total += f32 ? sum_units<float>(s.grad, s.n, e0, stop - u, a.scale)
             : s.kind == 2 * FLCE_BF16
                 ? sum_units<__nv_bfloat16>(s.grad, s.n, e0, stop - u, a.scale)
                 : sum_units<__half>(s.grad, s.n, e0, stop - u, a.scale);
    u = stop;
  }
  total = block_sum(total);
  __shared__ bool is_last;
  if (threadIdx.x == 0) {
    a.partial[a.base + blockIdx.x] = total;
    __threadfence();
    is_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!is_last) return;
  if (threadIdx.x == 0) *a.ticket = 0;
  if (!a.last) return;
  __threadfence();
  double sum = 0.0;
  const int count = a.base + static_cast<int>(gridDim.x);
  for (int j = threadIdx.x; j < count; j += kThreads) sum += __ldcg(a.partial + j);
  sum = block_sum(sum);
  if (threadIdx.x == 0) *a.norm = static_cast<float>(sqrt(sum));
}

// ------------------------------------------------------------------ host
inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int rc_of(cudaError_t e) {
  if (e == cudaSuccess) return FLCE_OK;
  cudaGetLastError();  // reported here, not by a later call
  return FLCE_ERR_CUDA;
}

bool fraction(double x) { return x >= 0.0 && x < 1.0; }

int check(const flce_adamw_params* p) {
  if (!p) return FLCE_ERR_BAD_ARG;
  if (p->state_bits != 32 && p->state_bits != 8) return FLCE_ERR_BAD_ARG;
  if (!fraction(p->beta1) || !fraction(p->beta2)) return FLCE_ERR_BAD_ARG;
  if (!(p->lr >= 0.0) || isinf(p->lr) || !(p->eps >= 0.0) || isinf(p->eps) ||
      !(p->max_norm >= 0.0) || !isfinite(p->grad_scale))
    return FLCE_ERR_BAD_ARG;
  if (p->n_tensors < 0 || p->n_tensors > (int64_t(1) << 24) || p->numel < 0 ||
      p->numel % kBlockElems != 0)
    return FLCE_ERR_BAD_SHAPE;
  return FLCE_OK;
}

// The tensors' types, sizes and addresses; with `step` what the step writes too.
int check_tensors(const flce_adamw_params* p, const flce_adamw_tensor* t, bool step) {
  if (p->n_tensors > 0 && !t) return FLCE_ERR_BAD_ARG;
  for (int64_t i = 0; i < p->n_tensors; ++i) {
    const flce_adamw_tensor& x = t[i];
    if (x.dtype < FLCE_F32 || x.dtype > FLCE_F16 ||
        (x.grad_dtype != x.dtype && x.grad_dtype != FLCE_F32) || !(x.weight_decay >= 0.0f) ||
        isinf(x.weight_decay))
      return FLCE_ERR_BAD_ARG;
    if (x.n < 0 || x.n > int64_t(1) << 42) return FLCE_ERR_BAD_SHAPE;
    if (x.n == 0) continue;
    if (!x.grad || (step && !x.param)) return FLCE_ERR_BAD_ARG;
    if (addr(x.grad) & (x.grad_dtype == FLCE_F32 ? 3 : 1) ||
        (step && addr(x.param) & (x.dtype == FLCE_F32 ? 3 : 1)))
      return FLCE_ERR_ALIGN;
    if (step && (x.offset < 0 || x.offset % kBlockElems != 0 || x.offset > p->numel ||
                 cdiv(x.n, kBlockElems) * kBlockElems > p->numel - x.offset))
      return FLCE_ERR_BAD_SHAPE;
  }
  return FLCE_OK;
}

// Tensors of a launch: as many as fit its arguments, with elements, from *i on.
template <int CAP>
int fill(Table<CAP>* out, const flce_adamw_params* p, const flce_adamw_tensor* t, int64_t* i) {
  out->count = 0;
  int64_t units = 0;
  for (; *i < p->n_tensors && out->count < CAP; ++*i) {
    const flce_adamw_tensor& x = t[*i];
    if (x.n == 0) continue;
    const int64_t more = cdiv(x.n, kUnit);
    if (units + more >= kMaxUnits) return FLCE_ERR_BAD_SHAPE;
    out->first[out->count] = static_cast<uint32_t>(units);
    out->slot[out->count] = Slot{x.param, x.grad, x.n, x.offset, x.weight_decay,
                                 2 * x.dtype + (x.grad_dtype != x.dtype)};
    units += more;
    ++out->count;
  }
  out->units = static_cast<uint32_t>(units);
  return FLCE_OK;
}

int64_t with_elements(const flce_adamw_params* p, const flce_adamw_tensor* t) {
  int64_t n = 0;
  for (int64_t i = 0; i < p->n_tensors; ++i) n += t[i].n > 0;
  return n;
}

// Whether tensors with elements come from i on.
bool more_from(const flce_adamw_params* p, const flce_adamw_tensor* t, int64_t i) {
  for (; i < p->n_tensors; ++i)
    if (t[i].n > 0) return true;
  return false;
}

template <typename K, typename A, typename B>
int launch(K kernel, unsigned blocks, bool wait, cudaStream_t st, A& a, B& b) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = wait ? 1 : 0;
  void* params[] = {&a, &b};
  return rc_of(cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), params));
}

template <int CAP>
int run_norm(const flce_adamw_params* p, const flce_adamw_tensor* t, float* norm, uint8_t* ws,
             int sms, cudaStream_t st) {
  NormArgs a{};
  a.partial = reinterpret_cast<double*>(ws + 256);
  a.ticket = reinterpret_cast<uint32_t*>(ws);
  a.norm = norm;
  a.scale = static_cast<float>(p->grad_scale);
  int64_t i = 0;
  do {
    Table<CAP> table;
    int rc = fill(&table, p, t, &i);
    if (rc) return rc;
    const int64_t cap = static_cast<int64_t>(sms) * kNormBlocks;
    const unsigned blocks = static_cast<unsigned>(table.units < cap ? table.units : cap);
    a.last = !more_from(p, t, i);
    if ((rc = launch(norm_kernel<CAP>, blocks, false, st, table, a))) return rc;
    a.base += static_cast<int32_t>(blocks);
  } while (!a.last);
  return FLCE_OK;
}

template <bool STATE8, bool MASTER, int CAP>
int run_step(const flce_adamw_params* p, const flce_adamw_tensor* t, StepArgs a, int sms,
             cudaStream_t st) {
  static std::atomic<int> per_sm{0};
  int per = per_sm.load();
  if (per == 0) {
    if (rc_of(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, adamw_kernel<STATE8, MASTER, CAP>,
                                                            kThreads, 0)) || per < 1)
      return FLCE_ERR_CUDA;
    per_sm.store(per);
  }
  int64_t i = 0;
  do {
    Table<CAP> table;
    int rc = fill(&table, p, t, &i);
    if (rc) return rc;
    const int64_t cap = static_cast<int64_t>(sms) * per;
    const unsigned blocks = static_cast<unsigned>(table.units < cap ? table.units : cap);
    a.last = !more_from(p, t, i);
    if ((rc = launch(adamw_kernel<STATE8, MASTER, CAP>, blocks, true, st, table, a))) return rc;
  } while (!a.last);
  return FLCE_OK;
}

template <bool STATE8, bool MASTER>
int run_step_cap(const flce_adamw_params* p, const flce_adamw_tensor* t, const StepArgs& a,
                 int64_t tensors, int sms, cudaStream_t st) {
  return tensors <= kSmall ? run_step<STATE8, MASTER, kSmall>(p, t, a, sms, st)
                           : run_step<STATE8, MASTER, kLarge>(p, t, a, sms, st);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_adamw_check_params(const flce_adamw_params* p) { return check(p); }

size_t flce_adamw_workspace_size(const flce_adamw_params* p) {
  if (check(p) != FLCE_OK) return 0;
  // partial sums of the norm: at most kNormBlocks per SM (up to 256 SMs) and launch
  const int64_t launches = 1 + p->n_tensors / kLarge;
  return 256 + static_cast<size_t>(launches) * kNormBlocks * 256 * sizeof(double);
}

int flce_grad_norm(const flce_adamw_params* p, const flce_adamw_tensor* tensors, float* norm,
                   void* workspace, size_t ws_bytes, void* stream) {
  int rc = check(p);
  if (rc || (rc = check_tensors(p, tensors, false))) return rc;
  if (!norm || !workspace) return FLCE_ERR_BAD_ARG;
  if (addr(norm) & 3 || addr(workspace) & 255) return FLCE_ERR_ALIGN;
  if (ws_bytes < flce_adamw_workspace_size(p)) return FLCE_ERR_WS_TOO_SMALL;
  int sms;
  if ((rc = require_device(&sms))) return rc;
  if (sms > 256) return FLCE_ERR_DEVICE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t count = with_elements(p, tensors);
  if (count == 0) return rc_of(cudaMemsetAsync(norm, 0, sizeof(float), st));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return count <= kSmall ? run_norm<kSmall>(p, tensors, norm, ws, sms, st)
                         : run_norm<kLarge>(p, tensors, norm, ws, sms, st);
}

int flce_adamw_step(const flce_adamw_params* p, const flce_adamw_tensor* tensors, float* master,
                    void* exp_avg, void* exp_avg_sq, float* exp_avg_scale, float* exp_rms_scale,
                    const float* lr, const float* norm, int64_t* step, void* workspace,
                    size_t ws_bytes, void* stream) {
  int rc = check(p);
  if (rc || (rc = check_tensors(p, tensors, true))) return rc;
  if (!exp_avg || !exp_avg_sq || !step || !workspace) return FLCE_ERR_BAD_ARG;
  const bool state8 = p->state_bits == 8;
  if (state8 && (!exp_avg_scale || !exp_rms_scale)) return FLCE_ERR_BAD_ARG;
  if ((p->max_norm > 0.0 || p->skip_nonfinite) && !norm) return FLCE_ERR_BAD_ARG;
  if ((addr(master) | addr(exp_avg) | addr(exp_avg_sq)) & 15 ||
      (addr(exp_avg_scale) | addr(exp_rms_scale) | addr(lr) | addr(norm)) & 3 || addr(step) & 7 ||
      addr(workspace) & 255)
    return FLCE_ERR_ALIGN;
  if (ws_bytes < 256) return FLCE_ERR_WS_TOO_SMALL;
  const int64_t count = with_elements(p, tensors);
  int sms;
  if ((rc = require_device(&sms))) return rc;
  if (count == 0) return FLCE_OK;
  StepArgs a{};
  a.master = master;
  a.m = exp_avg;
  a.v = exp_avg_sq;
  a.m_scale = exp_avg_scale;
  a.s_scale = exp_rms_scale;
  a.lr_ptr = lr;
  a.norm = norm;
  a.step = step;
  a.ticket = static_cast<uint32_t*>(workspace) + 1;
  a.lr = static_cast<float>(p->lr);
  a.beta1 = static_cast<float>(p->beta1);
  a.omb1 = static_cast<float>(1.0 - p->beta1);
  a.beta2 = static_cast<float>(p->beta2);
  a.rb2 = static_cast<float>(sqrt(p->beta2));
  a.romb2 = static_cast<float>(sqrt(1.0 - p->beta2));
  a.eps = static_cast<float>(p->eps);
  a.grad_scale = static_cast<float>(p->grad_scale);
  a.max_norm = static_cast<float>(p->max_norm);
  a.ln1 = log(p->beta1);
  a.ln2 = log(p->beta2);
  a.seed = p->seed;
  a.skip = p->skip_nonfinite != 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (state8)
    return master ? run_step_cap<true, true>(p, tensors, a, count, sms, st)
                  : run_step_cap<true, false>(p, tensors, a, count, sms, st);
  return master ? run_step_cap<false, true>(p, tensors, a, count, sms, st)
                : run_step_cap<false, false>(p, tensors, a, count, sms, st);
}

}  // extern "C"
