// Dense layer  y = act(x W + b) + r  and its gradients.
//
// Two GEMM kernels, both tcgen05 with operands brought by TMA:
//
//   pair     flce_gemm.cuh's CTA pairs on 256 x 256 tiles, for shapes with enough tiles to fill
//            the GPU in whole rounds: bound by the tensor cores.
//   split    (here) for all others, above all few tokens, which are bound by the bytes of the
//            weight.  The product is taken transposed, y^T = W^T x^T: 128 columns of y are the
//            128 TMEM lanes and up to 256 tokens its columns, so that a tile has no rows for
//            tokens that are not there, and a warp's stores run along y's rows whatever N is.
//            Where there are fewer tiles than SMs, the blocks of a cluster share a tile's depth and
//            add up their sums over distributed shared memory: one launch, no workspace.
//            (Cutting the line of all tiles' 64-deep blocks into equal pieces per SM, with partial
//            sums in the workspace and a second launch to join them: one token through 4096 x 4096
//            11.8 us, against 8.8; 200 tokens 34.7 against 16.5.)
//
// Results repeat bit for bit: either adds in a fixed order.
//
// The backward forms dz = dout act'(z) in bf16 (the tensor cores' type) and db, the sum of the
// unrounded dz over tokens, in one pass, then dx and dW as GEMMs side by side.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "flce_act.cuh"
#include "flce_gemm.cuh"
#include "flce_host.h"

namespace flce {
namespace {

constexpr size_t kHeader = 256;       // error word, the pair kernels' counters
constexpr size_t kSched = 128;
constexpr int kRows = 128;            // columns of y per tile of the split kernel
constexpr int kMaxTokens = 256;       // tokens per tile

// ------------------------------------------------------------------ tcgen05, one CTA
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void umma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, uint64_t* bar,
                                         int32_t x, int32_t y, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "l"(policy)
      : "memory");
}
// 16 fp32 columns of this warp's 32 TMEM lanes; tmem_wait before they are looked at
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// (the registers go through the wait, so that nothing reads them before it)
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

template <bool MN, int ROWS>
__device__ __forceinline__ void load_rows(uint8_t* dst, const CUtensorMap* map, uint64_t* bar,
                                          int mn0, int k0, uint64_t policy) {
  if constexpr (!MN) {
    tma_load(dst, map, bar, k0, mn0, policy);
  } else {
    static_assert(ROWS % 64 == 0, "operand rows");
#pragma unroll
    for (int j = 0; j < ROWS / 64; ++j)
      tma_load(dst + j * PIECE_BYTES, map, bar, mn0 + 64 * j, k0, policy);
  }
}

// ------------------------------------------------------------------ split kernel
// A block per tile of 128 columns of y and tt tokens (a multiple of 16) and share of the depth; the
// blocks of a cluster share a tile's depth, leave their sums in shared memory, and each adds up and
// finishes a part of the tile's tokens, in the blocks' order.
//
// The tensor cores cut off what an addition to an accumulator loses, so that its error grows with the
// additions: 4.4e-6 of fp32 logits after a depth of 4096.  A block's depth goes to as many accumulators
// one after the other as TMEM holds beside another block (eight at most: 4.8e-7), whose sums are then
// added with rounding.  A bf16 output, whose rounding is 2^-8, takes one.
struct SplitArgs {
  int32_t M, N;
  int32_t tt, m_tiles, k_blocks, stages;
  int32_t parts;  // accumulators that the depth is spread over
  LinearOut out;
  uint32_t* err;
  int32_t clear;
  int64_t a_inner, a_outer, b_inner, b_outer;
};
constexpr int kSplitThreads = 320;  // producer, issuer, eight epilogue warps

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kSplitThreads, 2)
    split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ SplitArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  constexpr int kABytes = kRows * BK * 2;
  const int b_bytes = a.tt * BK * 2, stages = a.stages;
  uint8_t* sA = smem;
  uint8_t* sB = smem + stages * kABytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sB + stages * b_bytes);
  uint64_t* empty = full + stages;
  uint64_t* done = empty + stages;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  uint32_t size;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  const int tile = blockIdx.x / size;
  const int n0 = tile / a.m_tiles * kRows, m0 = tile % a.m_tiles * a.tt;
  const int kb0 = static_cast<int>(int64_t(a.k_blocks) * rank / size);
  const int kb1 = static_cast<int>(int64_t(a.k_blocks) * (rank + 1) / size);
  const int width = a.tt * a.parts;
  const uint32_t cols = width <= 32 ? 32 : width <= 64 ? 64 : width <= 128 ? 128 : 256;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) tmem_alloc(tmem_holder, cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.clear) *a.err = 0;

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol_a = l2_policy(a.m_tiles == 1 ? L2_EVICT_FIRST : L2_NORMAL),
                     pol_b = l2_policy(L2_EVICT_LAST);
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, a.err)) break;
        const int k0 = kb * BK;
#if FLCE_DEBUG
        const bool in_a = A_MN ? tma_box_ok(n0, k0, a.a_inner, a.a_outer)
                               : tma_box_ok(k0, n0, a.a_inner, a.a_outer);
        const bool in_b = B_MN ? tma_box_ok(m0, k0, a.b_inner, a.b_outer)
                               : tma_box_ok(k0, m0, a.b_inner, a.b_outer);
        if (!in_a || !in_b) {
          atomicOr(a.err, FLCE_DEVERR_BOUNDS);
          *abort_flag = 1;
          break;
        }
#endif
        mbar_arrive_expect_tx(&full[stage], kABytes + b_bytes);
        load_rows<A_MN, kRows>(sA + stage * kABytes, &tmA, &full[stage], n0, k0, pol_a);
        if constexpr (B_MN) {
          for (int j = 0; j < a.tt / 64; ++j)
            tma_load(sB + stage * b_bytes + j * PIECE_BYTES, &tmB, &full[stage], m0 + 64 * j, k0, pol_b);
        } else {
          tma_load(sB + stage * b_bytes, &tmB, &full[stage], k0, m0, pol_b);
        }
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(kRows, 0, A_MN, B_MN) | (static_cast<uint32_t>(a.tt >> 3) << 17);
      GemmShape strides{};
      strides.mn_lbo = MN_ATOM_BYTES;
      strides.mn_sbo = 1024;
      const uint64_t a0 = operand_desc<A_MN>(smem_u32(sA), 0, strides);
      const uint64_t b0 = operand_desc<B_MN>(smem_u32(sB), 0, strides);
      constexpr uint64_t kKA = (A_MN ? UK * 128 : UK * 2) >> 4;
      constexpr uint64_t kKB = (B_MN ? UK * 128 : UK * 2) >> 4;
      int stage = 0, part = 0, until = kb0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full[stage], phase, abort_flag, a.err)) break;
        tc_fence_after();
        const bool begin = kb == until;  // of an accumulator
        if (begin) until = kb0 + (kb1 - kb0) * ++part / a.parts;
        const uint32_t d = tmem + (part - 1) * a.tt;
        const uint64_t as = a0 + stage * (kABytes >> 4), bs = b0 + stage * (b_bytes >> 4);
#pragma unroll
        for (int kk = 0; kk < BK / UK; ++kk)
          umma_bf16(d, as + kk * kKA, bs + kk * kKB, idesc, begin && kk == 0 ? 0u : 1u);
        umma_commit(&empty[stage]);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      umma_commit(done);
    }
    __syncwarp();
  }
  // all warps: the sums are complete, and the ring is free
  const bool ok = mbar_wait(done, 0, abort_flag, a.err);
  __syncwarp();
  tc_fence_after();
  const int rows = a.M - m0 < a.tt ? a.M - m0 : a.tt;
  const int q = warp & 3, half = (warp - 2) >> 2, nl = q * 32 + lane, n = n0 + nl;
  const bool n_ok = n < a.N;
  float* part = reinterpret_cast<float*>(smem);
  const float bias = warp >= 2 && a.out.bias && n_ok ? __bfloat162float(a.out.bias[n]) : 0.0f;
  if (warp >= 2 && ok) {
    const uint32_t tbase = tmem + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
    for (int c = half * 16; c < rows; c += 32) {
      float x[16] = {};
      __syncwarp();
      // the accumulators' columns, two on their way
      uint32_t u[16], v[16];
      for (int p = 0; p < a.parts; p += 2) {
        tmem_ld16(tbase + p * a.tt + c, u);
        if (p + 1 < a.parts) tmem_ld16(tbase + (p + 1) * a.tt + c, v);
        tmem_wait(u);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] += __uint_as_float(u[i]);
        if (p + 1 < a.parts) {
          tmem_wait(v);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] += __uint_as_float(v[i]);
        }
      }
      if (size > 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * kRows + nl] = x[i];
      } else if (n_ok) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (c + i < rows) linear_store1(a.out, int64_t(m0 + c + i) * a.out.ld + n, bias, x[i]);
      }
    }
  }
  tc_fence_before();
  if (size > 1) {
    __syncwarp();
    cluster_sync();
    if (warp >= 2 && ok && n_ok) {
      const int r0 = rows * rank / static_cast<int>(size), r1 = rows * (rank + 1) / static_cast<int>(size);
      const uint32_t own = smem_u32(part) + nl * 4;
      constexpr int kDeep = 4;  // tokens whose sums are on their way
      for (int m = r0 + half * kDeep; m < r1; m += 2 * kDeep) {
        float sum[kDeep] = {};
        for (uint32_t j = 0; j < size; ++j) {
          const uint32_t from = mapa_shared(own, j);
#pragma unroll
          for (int i = 0; i < kDeep; ++i)
            if (m + i < r1) sum[i] += ld_cluster(from + (m + i) * kRows * 4);
        }
#pragma unroll
        for (int i = 0; i < kDeep; ++i)
          if (m + i < r1) linear_store1(a.out, int64_t(m0 + m + i) * a.out.ld + n, bias, sum[i]);
      }
    }
    __syncwarp();
    cluster_sync();  // no block leaves while another reads its sums
  } else {
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, cols);
}

// ------------------------------------------------------------------ dz and db
constexpr int kDzThreads = 256;

struct DzArgs {
  const void* dout;
  const __nv_bfloat16* preact;
  __nv_bfloat16* dz;  // NULL: dout serves
  float* part;        // [strips, N], or NULL
  int64_t M, N, ld_dz, strip;
  int32_t act, dout_f32;
};

// A thread takes VEC columns and a strip of rows, a block neighbouring columns: whole kilobytes of a
// row at a time, four rows on their way, and the columns' sums stay in the thread.
template <int VEC>
__global__ void __launch_bounds__(kDzThreads) dz_kernel(const __grid_constant__ DzArgs a) {
  const int64_t n = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) * VEC;
  const int64_t m0 = blockIdx.y * a.strip;
  const int64_t m1 = m0 + a.strip < a.M ? m0 + a.strip : a.M;
  if (n >= a.N) return;
  constexpr int kDeep = VEC == 8 ? 4 : 8;
  float sum[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
  const bool act = a.act != FLCE_ACT_NONE;
  for (int64_t m = m0; m < m1; m += kDeep) {
    uint4 graw[kDeep], zraw[kDeep];
    float4 gwide[kDeep];
    float g1[kDeep], z1[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (m + d >= m1) continue;
      const int64_t at = (m + d) * a.N + n;
      if constexpr (VEC == 8) {
        if (a.dout_f32) {
          const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.dout) + at);
          gwide[d] = __ldcs(p);
          const float4 v = __ldcs(p + 1);
          graw[d] = make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z),
                               __float_as_uint(v.w));
        } else {
          graw[d] = __ldcs(reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(a.dout) + at));
        }
        if (act) zraw[d] = __ldcs(reinterpret_cast<const uint4*>(a.preact + at));
      } else {
        g1[d] = a.dout_f32 ? static_cast<const float*>(a.dout)[at]
                           : __bfloat162float(static_cast<const __nv_bfloat16*>(a.dout)[at]);
        if (act) z1[d] = __bfloat162float(a.preact[at]);
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (m + d >= m1) continue;
      float g[VEC], z[VEC];
      if constexpr (VEC == 8) {
        if (a.dout_f32) {
          g[0] = gwide[d].x; g[1] = gwide[d].y; g[2] = gwide[d].z; g[3] = gwide[d].w;
          g[4] = __uint_as_float(graw[d].x); g[5] = __uint_as_float(graw[d].y);
          g[6] = __uint_as_float(graw[d].z); g[7] = __uint_as_float(graw[d].w);
        } else {
          unpack_bf16x8(graw[d], g);
        }
        if (act) unpack_bf16x8(zraw[d], z);
      } else {
        g[0] = g1[d];
        if (act) z[0] = z1[d];
      }
      switch (a.act) {
        case FLCE_ACT_NONE: break;
        case FLCE_ACT_RELU:
#pragma unroll
          for (int i = 0; i < VEC; ++i) g[i] *= activate_slope(z[i], FLCE_ACT_RELU);
          break;
        case FLCE_ACT_GELU:
#pragma unroll
          for (int i = 0; i < VEC; ++i) g[i] *= activate_slope(z[i], FLCE_ACT_GELU);
          break;
        case FLCE_ACT_GELU_TANH:
#pragma unroll
          for (int i = 0; i < VEC; ++i) g[i] *= activate_slope(z[i], FLCE_ACT_GELU_TANH);
          break;
        default:
#pragma unroll
          for (int i = 0; i < VEC; ++i) g[i] *= activate_slope(z[i], FLCE_ACT_SILU);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum[i] += g[i];
      if (a.dz) {
        __nv_bfloat16* o = a.dz + (m + d) * a.ld_dz + n;
        if constexpr (VEC == 8) *reinterpret_cast<uint4*>(o) = pack_bf16x8(g);
        else *o = __float2bfloat16_rn(g[0]);
      }
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < VEC; ++i) a.part[blockIdx.y * a.N + n + i] = sum[i];
}

// db: the strips' sums, eight groups of strips side by side, then those
__global__ void __launch_bounds__(256) db_kernel(const float* part, int64_t strips, int64_t N,
                                                 __nv_bfloat16* db) {
  __shared__ float sums[8][32];
  const int group = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n = int64_t(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (n < N) {
#pragma unroll 8
    for (int64_t i = group; i < strips; i += 8) s += __ldcg(part + i * N + n);
  }
  sums[group][lane] = s;
  __syncthreads();
  if (group == 0 && n < N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sums[i][lane];
    db[n] = __float2bfloat16_rn(s);
  }
}

// ------------------------------------------------------------------ host
inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline int rc_of(cudaError_t e) {
  if (e == cudaSuccess) return FLCE_OK;
  cudaGetLastError();  // reported here, not by a later call
  return FLCE_ERR_CUDA;
}

int check(const flce_linear_params* p) {
  if (!p) return FLCE_ERR_BAD_ARG;
  if (p->weight_layout != FLCE_WEIGHT_HV && p->weight_layout != FLCE_WEIGHT_VH)
    return FLCE_ERR_BAD_ARG;
  if (p->activation < FLCE_ACT_NONE || p->activation > FLCE_ACT_SILU) return FLCE_ERR_BAD_ARG;
  if (p->out_dtype != FLCE_BF16 && p->out_dtype != FLCE_F32) return FLCE_ERR_BAD_ARG;
  constexpr int64_t most = (int64_t(1) << 31) - 1 - 256;
  if (p->M < 0 || p->N < 1 || p->K < 8 || p->M > most || p->N > most || p->K > most)
    return FLCE_ERR_BAD_SHAPE;
  if (p->K % 8 != 0) return FLCE_ERR_ALIGN;
  if (p->weight_layout == FLCE_WEIGHT_HV && p->N % 8 != 0) return FLCE_ERR_ALIGN;
  return FLCE_OK;
}

// One product out[rows, cols] = A B^T of the kernels' operands: "rows" are those of `out`.
// left: [rows, depth] K-major, or its transpose stored [depth, rows] (left_mn); right the same
// for [cols, depth].
struct Product {
  const void* left;
  const void* right;
  int64_t rows, cols, depth;
  int64_t ld_left, ld_right;
  bool left_mn, right_mn;
};

// How a product is done: by CTA pairs on tiles of 256 x `width`, or split, with tiles of tt rows and
// `size` blocks along the depth; whichever should take the fewest microseconds.  What the estimates
// are made of was measured: a 64-deep block of a pair's 256 x 256 tile takes 0.33 us (the tensor
// cores' rate), of 256 x 128 0.27 (an SM takes about 100 KB from L2 in a microsecond, which bounds it
// and the split tiles); 3 to 5 us pass from the launch to the first product, and the last tile's epilogue
// and the join of a cluster are in nobody's shadow.  512 x 4096 x 4096: 256 x 256 pairs 28.7 us, 128 x
// 128 split 28.2; 200 x 4096 x 4096: 28.8 and (64 rows, depth in two) 16.5; 24 x 4096 x 128256: split
// 162, depth in two 174.
struct Plan {
  int width;  // of a pair's tiles; 0: split
  int tt, size, stages;
};

Plan choose(const Product& g, int sms, bool f32 = false) {
  const double kb = static_cast<double>(cdiv(g.depth, BK));
  Plan best{};
  double least = 1e30;
  if (g.cols % 8 == 0) {
    for (int width = 256; width >= (f32 ? 256 : 128); width /= 2) {
      const int64_t rounds = cdiv(cdiv(g.rows, 256) * cdiv(g.cols, width), sms / 2);
      const double us = rounds * kb * (width == 256 ? 0.33 : 0.27) + (width == 256 ? 8.0 : 7.0) +
                        (rounds > 1 ? 2.0 : 0.0);
      const double dram = (static_cast<double>(g.rows) + g.cols) * g.depth * 2 / 5.8e6 + 6.0;
      const double t = us > dram ? us : dram;
      if (t < least) {
        least = t;
        best = Plan{width, 0, 0, 0};
      }
    }
  }
  const int unit = g.left_mn ? 64 : 16;
  const int64_t fewest = cdiv(g.rows, kMaxTokens);
  for (int64_t mt = fewest; mt <= fewest + 4; ++mt) {
    const int tt = static_cast<int>(cdiv(cdiv(g.rows, mt), unit) * unit);
    if (tt > kMaxTokens) continue;
    const int64_t tiles = cdiv(g.cols, kRows) * cdiv(g.rows, tt);
    for (int size = 1; size <= 8 && size <= kb; size *= 2) {
      const int64_t blocks = tiles * size;
      const int stage = (kRows + tt) * BK * 2;
      // two blocks per SM where there are blocks for it and half the memory holds a deep enough ring
      const bool two = blocks > sms && tt <= 64;
      int stages = ((two ? SMEM_LIMIT / 2 - 1024 : SMEM_LIMIT) - 1024 - 512) / stage;
      if (stages > 12) stages = 12;
      if (size > 1 && stages * stage < tt * kRows * 4) continue;  // a tile's sums do not fit
      const double mma = 0.34 * tt / 256, bytes = stage / 100e3;
      const double rounds = !two ? static_cast<double>(cdiv(blocks, sms)) : static_cast<double>(blocks) / sms;
      const double us = rounds * (kb / size * (mma > bytes ? mma : bytes) + 1.0 + tt * 0.012) + 3.0 +
                        (size > 1 ? 1.5 + tt * 0.01 : 0.0);
      const double dram = (static_cast<double>(g.rows) + g.cols) * g.depth * 2 / 6.2e6 + 4.0;
      const double t = us > dram ? us : dram;
      if (t < least) {
        least = t;
        best = Plan{0, tt, size, stages};
      }
    }
  }
  return best;
}

template <bool A_MN, bool B_MN>
int launch_split(const Product& g, const Plan& s, const LinearOut& out, uint32_t* err, bool clear,
                 cudaStream_t st) {
  auto kernel = split_kernel<A_MN, B_MN>;
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  int rc = rc_of(cudaGetDevice(&dev));
  if (rc) return rc;
  if (!(ready.load() >> (dev & 63) & 1)) {
    if ((rc = rc_of(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT))))
      return rc;
    ready.fetch_or(uint64_t(1) << (dev & 63));
  }
  CUtensorMap A, B;
  if (!(A_MN ? tensor_map(&A, g.right, g.cols, g.depth, g.ld_right, 64, BK)
             : tensor_map(&A, g.right, g.depth, g.cols, g.ld_right, BK, kRows)) ||
      !(B_MN ? tensor_map(&B, g.left, g.rows, g.depth, g.ld_left, 64, BK)
             : tensor_map(&B, g.left, g.depth, g.rows, g.ld_left, BK, s.tt)))
    return FLCE_ERR_CUDA;
  SplitArgs a{};
  a.M = static_cast<int32_t>(g.rows);
  a.N = static_cast<int32_t>(g.cols);
  a.tt = s.tt;
  a.m_tiles = static_cast<int32_t>(cdiv(g.rows, s.tt));
  a.k_blocks = static_cast<int32_t>(cdiv(g.depth, BK));
  a.stages = s.stages;
  // parts of a block's share of the depth, of one 64-deep block at least
  const int share = a.k_blocks / s.size;
  a.parts = !out.out_f32 ? 1 : 256 / s.tt < 8 ? 256 / s.tt : 8;
  if (a.parts > share) a.parts = share;
  a.out = out;
  a.err = err;
  a.clear = clear;
  a.a_inner = A_MN ? g.cols : g.depth;
  a.a_outer = A_MN ? g.depth : g.cols;
  a.b_inner = B_MN ? g.rows : g.depth;
  a.b_outer = B_MN ? g.depth : g.rows;
  const int64_t blocks = int64_t(a.m_tiles) * cdiv(g.cols, kRows) * s.size;
  if (blocks > (int64_t(1) << 31) - 1) return FLCE_ERR_BAD_SHAPE;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = 1024 + static_cast<size_t>(s.stages) * (kRows * BK * 2 + s.tt * BK * 2) + 512;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(s.size);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return rc_of(cudaLaunchKernelEx(&cfg, kernel, A, B, a));
}

int run_split(const Product& g, const Plan& s, const LinearOut& out, uint32_t* err, bool clear,
              cudaStream_t st) {
  if (g.left_mn) return launch_split<true, true>(g, s, out, err, clear, st);  // dweight: both are
  return g.right_mn ? launch_split<true, false>(g, s, out, err, clear, st)
                    : launch_split<false, false>(g, s, out, err, clear, st);
}

// Whether every pair has one tile at most, so that the schedule's counters are not needed.
bool one_round(const Product& g, int width) {
  return cdiv(g.rows, PAIR_BM) * cdiv(g.cols, width) <= pair_capacity();
}

// The product by CTA pairs; kind 0: a layer's output, 1: dx, 2: dweight.
int run_pair(const Product& g, int width, int kind, const LinearOut& out, uint32_t* err, int slot,
             bool clear, cudaStream_t st) {
  CUtensorMap A, B;
  if (!(g.left_mn ? tensor_map(&A, g.left, g.rows, g.depth, g.ld_left, 64, BK)
                  : tensor_map(&A, g.left, g.depth, g.rows, g.ld_left, BK, 64)) ||
      !(g.right_mn ? tensor_map(&B, g.right, g.cols, g.depth, g.ld_right, 64, BK)
                   : tensor_map(&B, g.right, g.depth, g.cols, g.ld_right, BK, 64)))
    return FLCE_ERR_CUDA;
  GemmShape sh = pair_shape(L2_EVICT_LAST, L2_NORMAL);
  sh.m_tiles = static_cast<int>(cdiv(g.rows, PAIR_BM));
  sh.n_tiles = static_cast<int>(cdiv(g.cols, width));
  sh.k_blocks = static_cast<int>(cdiv(g.depth, BK));
  sh.raster = 0;
  sh.sched = reinterpret_cast<unsigned int*>(reinterpret_cast<uint8_t*>(err) + kSched + 8 * slot);
  sh.one_round = one_round(g, width);
  sh.a_inner = g.left_mn ? g.rows : g.depth;
  sh.a_outer = g.left_mn ? g.depth : g.rows;
  sh.b_inner = g.right_mn ? g.cols : g.depth;
  sh.b_outer = g.right_mn ? g.depth : g.cols;
  plan_pair(&sh, int64_t(PAIR_BM) * g.depth * 2);
  EpiArgs ea{};
  ea.rows = static_cast<int>(g.rows);
  ea.cols = static_cast<int>(g.cols);
  ea.err = err;
  ea.clear = clear;
  const bool wide = width == 256;
  if (kind == 0) {
    ea.lin = out;
    if (out.out_f32)
      return rc_of((g.right_mn ? launch_linear_f32 : launch_linear_vh_f32)(A, B, sh, ea, st));
    return rc_of((g.right_mn ? (wide ? launch_linear : launch_linear_128)
                             : (wide ? launch_linear_vh : launch_linear_vh_128))(A, B, sh, ea, st));
  }
  if (kind == 1) {
    ea.acc_out = static_cast<__nv_bfloat16*>(out.y);
    ea.acc_mode = ACC_ONLY;
    ea.ld_acc = out.ld;
    return rc_of((g.right_mn ? (wide ? launch_bwd_dhidden_vh : launch_linear_dx_vh_128)
                             : (wide ? launch_bwd_dhidden : launch_linear_dx_128))(A, B, sh, ea, st));
  }
  ea.out = static_cast<__nv_bfloat16*>(out.y);
  ea.ld_out = out.ld;
  return rc_of((wide ? launch_bwd_dweight : launch_linear_dweight_128)(A, B, sh, ea, st));
}

Product forward_product(const flce_linear_params* p, const void* x, const void* w) {
  const bool hv = p->weight_layout == FLCE_WEIGHT_HV;
  return Product{x, w, p->M, p->N, p->K, p->K, hv ? p->N : p->K, false, hv};
}
// dx = dz W^T: W [K,N] is K-major over n, [N,K] MN-major
Product dx_product(const flce_linear_params* p, const void* dz, int64_t ld_dz, const void* w) {
  const bool hv = p->weight_layout == FLCE_WEIGHT_HV;
  return Product{dz, w, p->M, p->K, p->N, ld_dz, hv ? p->N : p->K, false, !hv};
}
// dweight [K,N] = x^T dz, or [N,K] = dz^T x
Product dw_product(const flce_linear_params* p, const void* dz, int64_t ld_dz, const void* x) {
  if (p->weight_layout == FLCE_WEIGHT_HV)
    return Product{x, dz, p->K, p->N, p->M, p->K, ld_dz, true, true};
  return Product{dz, x, p->N, p->K, p->M, ld_dz, p->K, true, true};
}

// Rows per strip of the dz kernel: at most 256 strips, and as short as 16 rows where the columns
// alone give few threads.
int64_t dz_strip(const flce_linear_params* p) {
  const int64_t threads = cdiv(p->N, p->N % 8 == 0 ? 8 : 1);
  int64_t strip = cdiv(p->M * threads, int64_t(1) << 18);  // about 2^18 threads
  if (strip < 16) strip = 16;
  const int64_t least = cdiv(p->M, 256);
  return strip < least ? least : strip;
}

struct BwdLayout {
  size_t dz, db, total;
  int64_t ld_dz, strips;
};

BwdLayout bwd_layout(const flce_linear_params* p) {
  BwdLayout L{};
  L.ld_dz = cdiv(p->N, 8) * 8;
  L.strips = cdiv(p->M, dz_strip(p));
  size_t off = kHeader;
  L.dz = off; off += align256(static_cast<size_t>(p->M) * L.ld_dz * 2);
  L.db = off; off += align256(static_cast<size_t>(L.strips) * p->N * 4);
  L.total = off;
  return L;
}

template <int VEC>
int launch_dz(const DzArgs& a, int64_t strips, cudaStream_t st) {
  const int64_t lanes = cdiv(a.N, VEC);
  const int threads = lanes >= kDzThreads ? kDzThreads : static_cast<int>(cdiv(lanes, 32) * 32);
  const int64_t cols = cdiv(lanes, threads);
  if (cols > (int64_t(1) << 31) - 1) return FLCE_ERR_BAD_SHAPE;
  dz_kernel<VEC><<<dim3(static_cast<unsigned>(cols), static_cast<unsigned>(strips)), threads, 0, st>>>(a);
  return rc_of(cudaGetLastError());
}

// One gradient's product, by whichever kernel suits it.
int run_gradient(const Product& g, int kind, void* out, uint32_t* err, int slot, int sms,
                 cudaStream_t st) {
  LinearOut o{};
  o.y = out;
  o.ld = g.cols;
  const Plan plan = choose(g, sms);
  return plan.width ? run_pair(g, plan.width, kind, o, err, slot, false, st)
                    : run_split(g, plan, o, err, false, st);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_linear_check_params(const flce_linear_params* p) { return check(p); }

size_t flce_linear_workspace_size(const flce_linear_params* p, int backward) {
  if (check(p) != FLCE_OK) return 0;
  if (backward) return bwd_layout(p).total;
  return kHeader;
}

int flce_linear(const flce_linear_params* p, const void* x, const void* weight, const void* bias,
                const void* residual, void* y, void* preact, void* workspace, size_t ws_bytes,
                void* stream) {
  int rc = check(p);
  if (rc) return rc;
  if (!weight || !workspace || (p->M > 0 && (!x || !y))) return FLCE_ERR_BAD_ARG;
  if ((addr(x) | addr(weight) | addr(residual) | addr(y) | addr(preact)) & 15 || addr(bias) & 1 ||
      addr(workspace) & 255)
    return FLCE_ERR_ALIGN;
  if (ws_bytes < flce_linear_workspace_size(p, 0)) return FLCE_ERR_WS_TOO_SMALL;
  int sms;
  if ((rc = require_device(&sms))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* err = static_cast<uint32_t*>(workspace);
  if (p->M == 0) {
    if ((rc = rc_of(cudaMemsetAsync(ws, 0, kHeader, st)))) return rc;
    return p->validate ? read_status(ws, st) : FLCE_OK;
  }
  LinearOut o{};
  o.bias = static_cast<const __nv_bfloat16*>(bias);
  o.residual = residual;
  o.y = y;
  o.preact = static_cast<__nv_bfloat16*>(preact);
  o.ld = p->N;
  o.act = p->activation;
  o.out_f32 = p->out_dtype == FLCE_F32;
  o.wide = p->N % 16 == 0 && ((addr(y) | addr(preact)) & 31) == 0;
  const Product g = forward_product(p, x, weight);
  const Plan plan = choose(g, sms, o.out_f32);
  // The header is cleared ahead where the schedule's counters are needed (and in the bounds-checking
  // build, whose first findings a kernel could wipe out), else by the kernel: a memset is a
  // microsecond or two of a small layer's ten.
  const bool ahead = FLCE_DEBUG || (plan.width && !one_round(g, plan.width));
  if (ahead && (rc = rc_of(cudaMemsetAsync(ws, 0, kHeader, st)))) return rc;
  rc = plan.width ? run_pair(g, plan.width, 0, o, err, 0, !ahead, st)
                  : run_split(g, plan, o, err, !ahead, st);
  if (rc) return rc;
  return p->validate ? read_status(ws, st) : FLCE_OK;
}

int flce_linear_backward(const flce_linear_params* p, const void* dout, const void* x,
                         const void* weight, const void* preact, void* dx, void* dweight,
                         void* dbias, void* workspace, size_t ws_bytes, void* stream) {
  int rc = check(p);
  if (rc) return rc;
  if (!workspace || (p->M > 0 && (!dout || (dx && !weight) || (dweight && !x) ||
                                  (p->activation != FLCE_ACT_NONE && !preact))))
    return FLCE_ERR_BAD_ARG;
  if ((addr(dout) | addr(x) | addr(weight) | addr(preact) | addr(dx) | addr(dweight)) & 15 ||
      addr(dbias) & 1 || addr(workspace) & 255)
    return FLCE_ERR_ALIGN;
  const BwdLayout L = bwd_layout(p);
  if (ws_bytes < L.total) return FLCE_ERR_WS_TOO_SMALL;
  int sms;
  if ((rc = require_device(&sms))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* err = static_cast<uint32_t*>(workspace);
  if ((rc = rc_of(cudaMemsetAsync(ws, 0, kHeader, st)))) return rc;
  if (p->M == 0) {  // sums over no tokens
    if (dweight && (rc = rc_of(cudaMemsetAsync(dweight, 0, size_t(p->N) * p->K * 2, st)))) return rc;
    if (dbias && (rc = rc_of(cudaMemsetAsync(dbias, 0, size_t(p->N) * 2, st)))) return rc;
    return p->validate ? read_status(ws, st) : FLCE_OK;
  }
  // dz: dout itself where nothing changes it and TMA can read it
  const bool f32 = p->out_dtype == FLCE_F32;
  const bool own_dz = p->activation != FLCE_ACT_NONE || f32 || p->N % 8 != 0;
  const void* dz = own_dz ? static_cast<const void*>(ws + L.dz) : dout;
  const int64_t ld_dz = own_dz ? L.ld_dz : p->N;
  if ((own_dz && (dx || dweight)) || dbias) {
    DzArgs a{};
    a.dout = dout;
    a.preact = static_cast<const __nv_bfloat16*>(preact);
    a.dz = own_dz && (dx || dweight) ? reinterpret_cast<__nv_bfloat16*>(ws + L.dz) : nullptr;
    a.part = dbias ? reinterpret_cast<float*>(ws + L.db) : nullptr;
    a.M = p->M;
    a.N = p->N;
    a.ld_dz = L.ld_dz;
    a.strip = dz_strip(p);
    a.act = p->activation;
    a.dout_f32 = f32;
    rc = p->N % 8 == 0 ? launch_dz<8>(a, L.strips, st) : launch_dz<1>(a, L.strips, st);
    if (rc) return rc;
  }
  if (dbias) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(cdiv(p->N, 32)));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    if ((rc = rc_of(cudaLaunchKernelEx(&cfg, db_kernel, reinterpret_cast<const float*>(ws + L.db),
                                       L.strips, p->N, static_cast<__nv_bfloat16*>(dbias)))))
      return rc;
  }
  // dx on the caller's stream, dweight beside it, as the head's backward does
  cudaStream_t side = st;
  const bool both = dx && dweight;
  if (both && (rc = side_fork(st, &side))) return rc;
  if (dx && (rc = run_gradient(dx_product(p, dz, ld_dz, weight), 1, dx, err, 0, sms, st)))
    return rc;
  if (dweight &&
      (rc = run_gradient(dw_product(p, dz, ld_dz, x), 2, dweight, err, 1, sms, side)))
    return rc;
  if (both && (rc = side_join(st))) return rc;
  return p->validate ? read_status(ws, st) : FLCE_OK;
}

}  // extern "C"
