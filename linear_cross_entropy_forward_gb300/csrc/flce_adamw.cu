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
// so a step repeats bit for bit.  s > 0 is never rounded to 0 (m / eps would follow).  What a code is
// made of is rounded after every operation, in the order of the formulas, so that the codes are the
// definition's and not this kernel's; the weights, which no code depends on, take fused and
// approximate operations.
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
constexpr int kNormBlocks = 8;             // blocks per SM of the norm, of kNormUnits at least
constexpr int kNormUnits = 4;               // (2.1M: 9.9 us; of one unit 14.0)
constexpr int64_t kMaxUnits = int64_t(1) << 31;

struct Slot {
  void* param;
  const void* grad;
  int64_t n, offset;
  float decay;
  int16_t dtype, grad_dtype;
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
  float lr, beta1, omb1, beta2, omb2, eps, grad_scale, max_norm;
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
__device__ __forceinline__ void ld_v8(const float* p, float (&x)[kPer]) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]),
                 "=f"(x[6]), "=f"(x[7])
               : "l"(p));
}

__device__ __forceinline__ void st_v8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
               "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// Eight elements of any type as they are in memory (16-bit ones in q[0]).  The type is looked at
// when they are converted, by branches that a warp takes together, so that there is one copy of
// the rest of the code for all types.
struct Raw {
  uint4 q[2];
};

// `left` elements are there; what is not aligned, and a tensor's last, goes element by element
// through memory of the thread's own, in rolled loops that take no registers from the rest.
__device__ __forceinline__ void load_raw(const void* base, int64_t e, int64_t left, int dtype, Raw& r) {
  const bool wide = dtype == FLCE_F32;
  const uint8_t* p = static_cast<const uint8_t*>(base) + e * (wide ? 4 : 2);
  if (left >= kPer && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    r.q[0] = __ldcs(reinterpret_cast<const uint4*>(p));
    if (wide) r.q[1] = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
  } else {
    Raw own;
    own.q[0] = own.q[1] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
    for (int i = 0; i < kPer && i < left; ++i) {
      if (wide) reinterpret_cast<uint32_t*>(&own)[i] = reinterpret_cast<const uint32_t*>(p)[i];
      else reinterpret_cast<uint16_t*>(&own)[i] = reinterpret_cast<const uint16_t*>(p)[i];
    }
    r = own;
  }
}
__device__ __forceinline__ void widen(const Raw& r, int dtype, float (&x)[kPer]) {
  const uint32_t w[8] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w,
                         r.q[1].x, r.q[1].y, r.q[1].z, r.q[1].w};
  if (dtype == FLCE_F32) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = __uint_as_float(w[i]);
  } else if (dtype == FLCE_BF16) {
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      x[i] = __uint_as_float(w[i / 2] << 16);
      x[i + 1] = __uint_as_float(w[i / 2] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i / 2]));
      x[i] = f.x;
      x[i + 1] = f.y;
    }
  }
}
__device__ __forceinline__ void store_raw(void* base, int64_t e, int64_t left, int dtype,
                                          const float (&x)[kPer]) {
  const bool wide = dtype == FLCE_F32;
  uint8_t* p = static_cast<uint8_t*>(base) + e * (wide ? 4 : 2);
  uint32_t w[8] = {};
  if (wide) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) w[i] = __float_as_uint(x[i]);
  } else if (dtype == FLCE_BF16) {
#pragma unroll
    for (int i = 0; i < kPer; i += 2) w[i / 2] = pack_bf16x2(x[i], x[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      const __half2 h = __floats2half2_rn(x[i], x[i + 1]);
      w[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  Raw r;
  r.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
  r.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  if (left >= kPer && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    __stcs(reinterpret_cast<uint4*>(p), r.q[0]);
    if (wide) __stcs(reinterpret_cast<uint4*>(p) + 1, r.q[1]);
  } else {
#pragma unroll 1
    for (int i = 0; i < kPer && i < left; ++i) {
      if (wide) reinterpret_cast<uint32_t*>(p)[i] = reinterpret_cast<const uint32_t*>(&r)[i];
      else reinterpret_cast<uint16_t*>(p)[i] = reinterpret_cast<const uint16_t*>(&r)[i];
    }
  }
}

// ------------------------------------------------------------------ 8-bit states
// Chris Wellons' lowbias32 (xor-shifts and odd multipliers found by a search for the least bias).
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
  // (a NaN of larger bits would become 0 by the addition)
  const uint32_t bits = min(__float_as_uint(a + low), 0x7FC00000u);
  return __uint_as_float((bits + r20) & 0xFFF00000u) - low;
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
  const float unit = none ? 0.0f : 448.0f * __frcp_rn(top);
  scale = none ? 0.0f : top * (1.0f / 448.0f);
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
// g = c grad;  m = beta1 m + omb1 g;  v = beta2 v + omb2 g^2;
// p = p (1 - lr wd) - step_size m / (root_c2 sqrt(v) + eps)
struct Coef {
  float c, beta1, omb1, beta2, omb2, eps, lr, step_size, root_c2;
  uint32_t key;
};

// fp32 states: to a unit in the last place or two, subnormals kept; 8-bit states: rounded.
template <bool STATE8>
__device__ __forceinline__ float root(float x) {
  if constexpr (STATE8) return __fsqrt_rn(x);
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// a b + c d, rounded after each product and the sum: not by the packed operations, of which a
// multiplication is fused with the addition behind it even where both say .rn.
__device__ __forceinline__ float sum_of_products(float a, float b, float c, float d) {
  return __fadd_rn(__fmul_rn(a, b), __fmul_rn(c, d));
}

// One thread's 8 elements as they are in memory.
template <bool STATE8, bool MASTER>
struct Fetched {
  Raw g, w;
  float master[MASTER ? kPer : 1], m[STATE8 ? 1 : kPer], v[STATE8 ? 1 : kPer];
  uint2 cm, cs;
  float scale_m, scale_s;
};

// Elements e0 on of the tensor, the states' (32-byte aligned) from s.offset + e0 on.  Past the
// tensor's last block of 128 there is no state; the 16 lanes of a block leave or stay together.
__device__ __forceinline__ bool has_state(const Slot& s, int64_t e0) {
  return (e0 & ~int64_t(kBlockElems - 1)) < s.n;
}

template <bool STATE8, bool MASTER>
__device__ __forceinline__ void fetch(const Slot& s, const StepArgs& a, int64_t e0,
                                      Fetched<STATE8, MASTER>& f) {
  if (!has_state(s, e0)) return;
  const int64_t left = s.n - e0, at = s.offset + e0;
  load_raw(s.grad, e0, left, s.grad_dtype, f.g);
  if constexpr (MASTER) ld_v8(a.master + at, f.master);
  else load_raw(s.param, e0, left, s.dtype, f.w);
  if constexpr (STATE8) {
    f.cm = __ldcs(reinterpret_cast<const uint2*>(static_cast<uint8_t*>(a.m) + at));
    f.cs = __ldcs(reinterpret_cast<const uint2*>(static_cast<uint8_t*>(a.v) + at));
    f.scale_m = a.m_scale[at / kBlockElems];
    f.scale_s = a.s_scale[at / kBlockElems];
  } else {
    ld_v8(static_cast<const float*>(a.m) + at, f.m);
    ld_v8(static_cast<const float*>(a.v) + at, f.v);
  }
}

template <bool STATE8, bool MASTER>
__device__ __forceinline__ void update8(const Slot& s, const StepArgs& a, const Coef& k,
                                        int64_t e0, const Fetched<STATE8, MASTER>& f) {
  const int64_t left = s.n - e0, at = s.offset + e0;
  const bool in = has_state(s, e0);
  if (!STATE8 && !in) return;
  float g[kPer], w[kPer], m[kPer], v[kPer];
  float scale_m = f.scale_m, scale_s = f.scale_s;
  widen(f.g, s.grad_dtype, g);
  if constexpr (MASTER) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) w[i] = f.master[i];
  } else {
    widen(f.w, s.dtype, w);
  }
  if constexpr (STATE8) {
    unpack8(f.cm, m);
    unpack8(f.cs, v);
    if (!in) {  // no part in another block's largest: zeros throughout
      scale_m = scale_s = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) g[i] = m[i] = v[i] = 0.0f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      m[i] = f.m[i];
      v[i] = f.v[i];
    }
  }
  const float shrink = 1.0f - k.lr * s.decay;
  const uint64_t shrink2 = f2_pack(shrink, shrink), minus = f2_pack(-k.step_size, -k.step_size),
                 eps2 = f2_pack(k.eps, k.eps), c2 = f2_pack(k.c, k.c),
                 beta1 = f2_pack(k.beta1, k.beta1), omb1 = f2_pack(k.omb1, k.omb1),
                 beta2 = f2_pack(k.beta2, k.beta2), omb2 = f2_pack(k.omb2, k.omb2),
                 root2 = f2_pack(k.root_c2, k.root_c2);
  const uint64_t unit_m = f2_pack(scale_m, scale_m), unit_s = f2_pack(scale_s, scale_s);
#pragma unroll
  for (int i = 0; i < kPer; i += 2) {
    const uint64_t x = f2_mul(f2_pack(g[i], g[i + 1]), c2);
    uint64_t m2 = f2_pack(m[i], m[i + 1]), v2 = f2_pack(v[i], v[i + 1]);
    if constexpr (STATE8) {
      m2 = f2_mul(m2, unit_m);
      v2 = f2_mul(v2, unit_s);
      v2 = f2_mul(v2, v2);
      float x0, x1, y0, y1, p0, p1, q0, q1;
      f2_unpack(x, x0, x1);
      f2_unpack(f2_mul(x, x), y0, y1);
      f2_unpack(m2, p0, p1);
      f2_unpack(v2, q0, q1);
      m2 = f2_pack(sum_of_products(p0, k.beta1, x0, k.omb1), sum_of_products(p1, k.beta1, x1, k.omb1));
      v2 = f2_pack(sum_of_products(q0, k.beta2, y0, k.omb2), sum_of_products(q1, k.beta2, y1, k.omb2));
    } else {
      m2 = f2_fma(m2, beta1, f2_mul(x, omb1));
      v2 = f2_fma(v2, beta2, f2_mul(f2_mul(x, x), omb2));
    }
    float v0, v1, d0, d1;
    f2_unpack(v2, v0, v1);
    const float s0 = root<STATE8>(v0), s1 = root<STATE8>(v1);
    f2_unpack(f2_fma(f2_pack(s0, s1), root2, eps2), d0, d1);
    const uint64_t u = f2_mul(m2, f2_pack(fast_rcp(d0), fast_rcp(d1)));
    f2_unpack(f2_fma(u, minus, f2_mul(f2_pack(w[i], w[i + 1]), shrink2)), w[i], w[i + 1]);
    f2_unpack(m2, m[i], m[i + 1]);
    v[i] = STATE8 ? s0 : v0;
    v[i + 1] = STATE8 ? s1 : v1;
  }
  // Behind the tensor's last element the states are zero, as they have been so far: 0 / eps is NaN for an eps
  // of 0, and so is 0 times a factor that is not finite.
  if (left < kPer) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i >= left) w[i] = m[i] = v[i] = 0.0f;
  }
  uint2 cm, cs;
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
  if constexpr (MASTER) st_v8(a.master + at, w);
  store_raw(s.param, e0, left, s.dtype, w);
  if constexpr (STATE8) {
    __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + at), cm);
    __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + at), cs);
    if ((at & (kBlockElems - 1)) == 0) {
      a.m_scale[at / kBlockElems] = scale_m;
      a.s_scale[at / kBlockElems] = scale_s;
    }
  } else {
    st_v8(static_cast<float*>(a.m) + at, m);
    st_v8(static_cast<float*>(a.v) + at, v);
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

// Two blocks per SM's worth of registers for fp32 states, whose loads are all of a unit's bytes (600M
// with masters 2.66 ms, 6.3 TB/s; for four blocks 2 % more), four for 8 bits, bound by their arithmetic, some 85
// instructions per element (300M with masters: 0.97 ms, 5.0 TB/s; for two 7 % more).
template <bool STATE8, bool MASTER, int CAP>
__global__ void __launch_bounds__(kThreads, STATE8 ? 4 : 2)
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
    k.c = c;
    k.beta1 = a.beta1;
    k.omb1 = a.omb1;
    k.beta2 = a.beta2;
    k.omb2 = a.omb2;
    k.eps = a.eps;
    k.lr = a.lr_ptr ? *a.lr_ptr : a.lr;
    // 1 - b^t = -(e^{t ln b} - 1): exact to fp32 for small t ln b too
    const double ts = static_cast<double>(step);
    k.step_size = k.lr / -expm1f(static_cast<float>(ts * a.ln1));
    k.root_c2 = sqrtf(1.0f / -expm1f(static_cast<float>(ts * a.ln2)));
    k.key = mix(a.seed + 0x9E3779B9u * static_cast<uint32_t>(step));
    uint32_t u, end;
    int i = find_run(t, u, end);
    while (u < end) {
      while (i + 1 < t.count && t.first[i + 1] <= u) ++i;
      const Slot& s = t.slot[i];
      const uint32_t stop = i + 1 < t.count && t.first[i + 1] < end ? t.first[i + 1] : end;
      int64_t e0 = static_cast<int64_t>(u - t.first[i]) * kUnit + threadIdx.x * kPer;
      Fetched<STATE8, MASTER> f;
      if (STATE8) fetch(s, a, e0, f);
#pragma unroll 1
      for (; u < stop; ++u, e0 += kUnit) {
        if constexpr (STATE8) {
          // the next unit is asked for ahead of the arithmetic, which is as long as the bytes take
          const Fetched<STATE8, MASTER> now = f;
          if (u + 1 < stop) fetch(s, a, e0 + kUnit, f);
          update8(s, a, k, e0, now);
        } else {
          fetch(s, a, e0, f);
          update8(s, a, k, e0, f);
        }
      }
    }
  }
  // A block's ticket says that all of its threads have read the step; the last one counts it, and leaves
  // the ticket at 0.  (a.last and skip are the same for all threads.)
  if (a.last && !skip) {
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      if (atomicAdd(a.ticket, 1u) == gridDim.x - 1) {
        *a.ticket = 0;
        *a.step = step;
      }
    }
  }
}

// ------------------------------------------------------------------ the norm
// Sum of (scale g)^2: those of eight elements in fp32, four additions deep, and these sums in a pair of
// floats per lane of a packed addition, whose rounding errors are added up beside it.  The roundings of
// many eights cancel: 2^-24 / sqrt(n / 8) or so is left of them.  (Two 64-bit additions per 16 squares
// took longer than their bytes do, and so did every pair of squares in the pair of floats: 600M in bf16
// 370 us; so 238, 5.0 TB/s, and in fp32 337, 7.1 TB/s.)
constexpr int kNormDepth = 2;  // units in flight (four, for half the blocks per SM: 600M in bf16 329 us)

struct PairSum {
  uint64_t hi = 0, lo = 0;  // two lanes each

  // (a + b and what it lost: the two-sum of Knuth)
  __device__ __forceinline__ void add(uint64_t x) {
    const uint64_t sign = 0x8000000080000000ull;
    const uint64_t sum = f2_add(hi, x), part = f2_add(sum, hi ^ sign);
    const uint64_t lost = f2_add(f2_add(hi, f2_add(sum, part ^ sign) ^ sign), f2_add(x, part ^ sign));
    hi = sum;
    lo = f2_add(lo, lost);
  }
  __device__ __forceinline__ double value() const {
    float h0, h1, l0, l1;
    f2_unpack(hi, h0, h1);
    f2_unpack(lo, l0, l1);
    // an infinity's lost part is NaN
    if (!isfinite(h0) || !isfinite(h1)) return static_cast<double>(h0) + h1;
    return (static_cast<double>(h0) + l0) + (static_cast<double>(h1) + l1);
  }
};

// `units` units of one tensor from element e0 on (this thread's first)
__device__ __forceinline__ void sum_units(const Slot& s, int64_t e0, int64_t units, float scale,
                                          PairSum& sum) {
  const uint64_t scale2 = f2_pack(scale, scale);
#pragma unroll 1
  for (int64_t v = 0; v < units; v += kNormDepth) {
    Raw r[kNormDepth];
#pragma unroll
    for (int d = 0; d < kNormDepth; ++d) {
      const int64_t e = e0 + (v + d) * kUnit;
      r[d].q[0] = r[d].q[1] = make_uint4(0, 0, 0, 0);
      if (v + d < units && e < s.n) load_raw(s.grad, e, s.n - e, s.grad_dtype, r[d]);
    }
#pragma unroll
    for (int d = 0; d < kNormDepth; ++d) {
      float x[kPer];
      widen(r[d], s.grad_dtype, x);
      uint64_t squares = 0;
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        const uint64_t y = f2_mul(f2_pack(x[i], x[i + 1]), scale2);
        squares = f2_fma(y, y, squares);
      }
      sum.add(squares);
    }
  }
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
__global__ void __launch_bounds__(kThreads, kNormBlocks)
    norm_kernel(const __grid_constant__ Table<CAP> t, const __grid_constant__ NormArgs a) {
  uint32_t u, end;
  int i = find_run(t, u, end);
  PairSum sum_of;
  while (u < end) {
    while (i + 1 < t.count && t.first[i + 1] <= u) ++i;
    const Slot& s = t.slot[i];
    const uint32_t stop = i + 1 < t.count && t.first[i + 1] < end ? t.first[i + 1] : end;
    const int64_t e0 = static_cast<int64_t>(u - t.first[i]) * kUnit + threadIdx.x * kPer;
    sum_units(s, e0, stop - u, a.scale, sum_of);
    u = stop;
  }
  const double total = block_sum(sum_of.value());
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
                                 static_cast<int16_t>(x.dtype), static_cast<int16_t>(x.grad_dtype)};
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
    const int64_t enough = cdiv(table.units, kNormUnits);
    const unsigned blocks = static_cast<unsigned>(enough < cap ? enough : cap);
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
    const int64_t enough = cdiv(table.units, kNormUnits);
    const unsigned blocks = static_cast<unsigned>(enough < cap ? enough : cap);
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
  const bool state8 = p->state_bits == 8;
  if (!step || !workspace) return FLCE_ERR_BAD_ARG;
  if (p->numel > 0 && (!exp_avg || !exp_avg_sq || (state8 && (!exp_avg_scale || !exp_rms_scale))))
    return FLCE_ERR_BAD_ARG;
  if ((p->max_norm > 0.0 || p->skip_nonfinite) && !norm) return FLCE_ERR_BAD_ARG;
  if ((addr(master) | addr(exp_avg) | addr(exp_avg_sq)) & 31 ||
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
  a.omb2 = static_cast<float>(1.0 - p->beta2);
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
