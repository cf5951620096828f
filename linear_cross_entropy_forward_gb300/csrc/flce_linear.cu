// Dense layer  y = act(x W + b) + r  and its gradients.
//
// Two GEMM kernels, both tcgen05 with operands brought by TMA:
//
//   pair     flce_gemm.cuh's CTA pairs on 256 x 256 tiles, for shapes with enough tiles to fill
//            the GPU in whole rounds: bound by the tensor cores (8192 x 4096 x 16384: 565 us, 1.95
//            PFLOP/s with its operands in L2).
//   split    (here) for few tokens, which are bound by the bytes of the weight (24 x 4096 x 128256:
//            161 us, 6.6 TB/s), and for shallow products, bound by their outputs.  Tiles are 128
//            columns of y by up to 256 tokens, so that a tile has no rows for tokens that are not
//            there, and two blocks of an SM take turns at the tensor cores and the stores.
//
// Both take the product transposed, y^T = W^T x^T: y's columns are the TMEM lanes, and a warp's stores
// run along y's rows whatever N is.  (With a row of y per lane, pairs take multiples of 8 alone, and
// 8192 x 4096 x 4097 by the split kernel is 361 us; so 173.)
//
// Where there are fewer split tiles than SMs, the blocks of a cluster share a tile's depth and add up
// their sums over distributed shared memory: one launch, no workspace.  (Cutting the line of all tiles'
// 64-deep blocks into equal pieces per SM, with partial sums in the workspace and a second launch to
// join them: one token through 4096 x 4096 11.8 us, against 9.0; 200 tokens 34.7 against 15.2.)
//
// Results repeat bit for bit: either adds in a fixed order.
//
// The backward forms dz = dout act'(z) in bf16 and db, the sum of the unrounded dz over tokens, in one pass,
// then dx and dW as GEMMs side by side.  dz is rounded because x and W are bf16 and the tensor cores take
// one type (split into a high and a low half the products would take twice as long); z comes in bf16 from
// the forward, half the bytes to write and to read again.  dx and dW are 2.4e-3 off by 2-norm, where the
// rounding of dz leaves 2.35e-3 and that of the outputs alone 1.7e-3.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

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
// additions: 4.4e-6 of fp32 logits after a depth of 4096.  A block's depth goes to several accumulators
// one after the other (eight, where TMEM holds them beside another block: 4.8e-7), whose sums are then
// added with rounding.  A bf16 output, whose rounding is 2^-8, takes one.
struct SplitArgs {
  int32_t M, N;
  int32_t tt, m_tiles, k_blocks, stages;
  int32_t parts;  // accumulators that the depth is spread over
  int32_t lost;   // the self-test of the bounded waits: the first block's copies end halfway down its depth
  LinearOut out;
  uint32_t* err;
  int32_t clear;
  int64_t a_inner, a_outer, b_inner, b_outer;
  Results results;
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
      const int last = a.lost && blockIdx.x == 0 ? (kb0 + kb1) / 2 : kb1;
      for (int kb = kb0; kb < last; ++kb) {
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
      uint32_t res[16];
      const int64_t at = int64_t(m0 + c) * a.out.ld + n;
      if (size == 1) linear_residual(a.out, at, n_ok ? rows - c : 0, res);
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
      } else if (n_ok && FLCE_CHECK(column_ok(a.out, a.results, at, rows - c, 16), a.err)) {
        linear_store_column(a.out, at, rows - c, bias, res, x);
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
        uint32_t res[kDeep];
        const int64_t at = int64_t(m0 + m) * a.out.ld + n;
        linear_residual(a.out, at, r1 - m, res);
        for (uint32_t j = 0; j < size; ++j) {
          const uint32_t from = mapa_shared(own, j);
#pragma unroll
          for (int i = 0; i < kDeep; ++i)
            if (m + i < r1) sum[i] += ld_cluster(from + (m + i) * kRows * 4);
        }
        if (FLCE_CHECK(column_ok(a.out, a.results, at, r1 - m, kDeep), a.err))
          linear_store_column(a.out, at, r1 - m, bias, res, sum);
      }
    }
    __syncwarp();
    cluster_sync();  // no block leaves while another reads its sums
  } else {
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, cols);
  if (*abort_flag) leave_nan(a.results);  // (behind what the cluster's other blocks made of its sums)
}

// ------------------------------------------------------------------ dz and db
constexpr int kDzThreads = 256;

struct DzArgs {
  const void* dout;
  const __nv_bfloat16* preact;
  __nv_bfloat16* dz;  // NULL: dout serves
  float* part;        // [strips, N], or NULL
  uint32_t* header;   // the workspace's, cleared for the launches behind
  int64_t M, N, ld_dz, strip;
  int32_t act, dout_f32;
};

// Eight neighbouring elements, from element `at` on, of an array of 16-byte aligned beginning and
// `total` elements.  ALIGNED: at is a multiple of 8.  Else the aligned 16-byte pieces that they lie in
// are read (neighbouring threads' pieces are the same lines of L1) and shifted; elements behind the
// array's end are not touched.
template <bool ALIGNED>
struct Eight16 {
  uint4 q[ALIGNED ? 1 : 2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int64_t at, int64_t total) {
    if constexpr (ALIGNED) {
      q[0] = __ldcs(reinterpret_cast<const uint4*>(p + at));
    } else {
      const int64_t piece = at >> 3;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        q[i] = make_uint4(0, 0, 0, 0);
        const int64_t first = (piece + i) * 8;
        if (first + 8 <= total) {
          q[i] = __ldg(reinterpret_cast<const uint4*>(p) + piece + i);
        } else if (first < total) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t x = first + j < total
                                   ? reinterpret_cast<const uint16_t*>(p)[first + j] : 0u;
            w[j / 2] = j & 1 ? w[j / 2] | x << 16 : x;
          }
          q[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
  __device__ __forceinline__ void get(int64_t at, float (&x)[8]) const {
    if constexpr (ALIGNED) {
      unpack_bf16x8(q[0], x);
    } else {
      const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
      uint32_t u[6], v[5], o[4];
#pragma unroll
      for (int i = 0; i < 6; ++i) u[i] = at & 4 ? w[i + 2] : w[i];
#pragma unroll
      for (int i = 0; i < 5; ++i) v[i] = at & 2 ? u[i + 1] : u[i];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(v[i], v[i + 1], (at & 1) * 16);
      unpack_bf16x8(make_uint4(o[0], o[1], o[2], o[3]), x);
    }
  }
};
template <bool ALIGNED>
struct Eight32 {
  uint4 q[ALIGNED ? 2 : 3];
  __device__ __forceinline__ void load(const float* p, int64_t at, int64_t total) {
    const int64_t piece = at >> 2;
#pragma unroll
    for (int i = 0; i < (ALIGNED ? 2 : 3); ++i) {
      const int64_t first = (piece + i) * 4;
      if (ALIGNED) {
        q[i] = __ldcs(reinterpret_cast<const uint4*>(p) + piece + i);
      } else if (first + 4 <= total) {
        q[i] = __ldg(reinterpret_cast<const uint4*>(p) + piece + i);
      } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
        q[i].x = first < total ? w[first] : 0u;
        q[i].y = first + 1 < total ? w[first + 1] : 0u;
        q[i].z = first + 2 < total ? w[first + 2] : 0u;
        q[i].w = 0;
      }
    }
  }
  __device__ __forceinline__ void get(int64_t at, float (&x)[8]) const {
    if constexpr (ALIGNED) {
      const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    } else {
      const uint32_t w[12] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w,
                              q[2].x, q[2].y, q[2].z, q[2].w};
      uint32_t u[9];
#pragma unroll
      for (int i = 0; i < 9; ++i) u[i] = at & 2 ? w[i + 2] : w[i];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(at & 1 ? u[i + 1] : u[i]);
    }
  }
};

// A thread takes eight columns and a strip of rows, a block neighbouring columns: whole kilobytes of a
// row at a time, four rows on their way (two where they are not aligned), and the columns' sums stay
// in the thread.
template <bool ALIGNED, bool F32>
__global__ void __launch_bounds__(kDzThreads) dz_kernel(const __grid_constant__ DzArgs a) {
  const int64_t n = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) * 8;
  const int64_t m0 = blockIdx.y * a.strip;
  const int64_t m1 = m0 + a.strip < a.M ? m0 + a.strip : a.M;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < int(kHeader / 4); i += blockDim.x) a.header[i] = 0;
  if (n >= a.N) return;
  constexpr int kDeep = ALIGNED ? 4 : 2;
  const int64_t total = a.M * a.N;
  const int left = a.N - n < 8 ? static_cast<int>(a.N - n) : 8;
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
  const bool act = a.act != FLCE_ACT_NONE;
  for (int64_t m = m0; m < m1; m += kDeep) {
    std::conditional_t<F32, Eight32<ALIGNED>, Eight16<ALIGNED>> graw[kDeep];
    Eight16<ALIGNED> zraw[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (m + d >= m1) continue;
      const int64_t at = (m + d) * a.N + n;
      if constexpr (F32) graw[d].load(static_cast<const float*>(a.dout), at, total);
      else graw[d].load(static_cast<const __nv_bfloat16*>(a.dout), at, total);
      if (act) zraw[d].load(a.preact, at, total);
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (m + d >= m1) continue;
      const int64_t at = (m + d) * a.N + n;
      float g[8], z[8];
      graw[d].get(at, g);
      if (act) zraw[d].get(at, z);
      switch (a.act) {
        case FLCE_ACT_NONE: break;
        case FLCE_ACT_RELU:
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] *= activate_slope(z[i], FLCE_ACT_RELU);
          break;
        case FLCE_ACT_GELU:
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] *= activate_slope(z[i], FLCE_ACT_GELU);
          break;
        case FLCE_ACT_GELU_TANH:
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] *= activate_slope(z[i], FLCE_ACT_GELU_TANH);
          break;
        default:
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] *= activate_slope(z[i], FLCE_ACT_SILU);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += g[i];
      // (rows of dz are padded to eight columns; nothing reads the padding)
      if (a.dz) *reinterpret_cast<uint4*>(a.dz + (m + d) * a.ld_dz + n) = pack_bf16x8(g);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < left) a.part[blockIdx.y * a.N + n + i] = sum[i];
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

// Tiles of CTA pairs; a layer's output is made transposed.
int64_t pair_tiles(const Product& g, bool layer, int width) {
  return layer ? cdiv(g.cols, PAIR_BM) * cdiv(g.rows, width)
               : cdiv(g.rows, PAIR_BM) * cdiv(g.cols, width);
}

// fp32 outputs of a depth that one accumulator should not add up.
bool drained(const Product& g, const LinearOut& o) {
  return o.out_f32 && cdiv(g.depth, BK) > kWholeBlocks;
}

// Accumulators of a split block with fp32 output for a share of the depth: eight, or as many more as
// it takes, and TMEM holds beside another block, but none without a 64-deep block.
int parts_of(int tt, int share) {
  int parts = static_cast<int>(cdiv(share, kWholeBlocks));
  if (parts < 8) parts = 8;
  if (parts > 256 / tt) parts = 256 / tt;
  return parts < share ? parts : share;
}

// How a product is done: by CTA pairs on tiles of 256 x `width`, or split, with tiles of tt rows,
// `size` blocks along the depth and one or two blocks per SM; whichever should take the fewest
// microseconds.  What the estimates are made of was measured: a 64-deep block of a pair's 256 x 256
// tile takes 0.33 us (the tensor cores' rate), of 256 x 128 0.27 (an SM takes about 100 KB from L2 in a
// microsecond, which bounds it and the split tiles); 3 to 5 us pass from the launch to the first
// product.  An SM's share of the output, 128 columns of 256 tokens, takes 4.5 us for its stores, and
// more with an activation, preact and a residual; pairs do it beside the next tile's products, and so do
// two split blocks of one SM, if less well.  The blocks of a cluster share it.
struct Plan {
  int width;  // of a pair's tiles; 0: split
  int tt, size, stages;
  double us;  // what it should take
};

Plan choose(const Product& g, int sms, bool layer, const LinearOut& o) {
  const double kb = static_cast<double>(cdiv(g.depth, BK));
  const double output = 4.5 + (o.act != FLCE_ACT_NONE ? 1.7 : 0.0) + (o.preact ? 2.5 : 0.0) +
                        (o.residual ? 3.5 : 0.0) + (o.out_f32 ? 1.0 : 0.0);
  const double traffic = (static_cast<double>(g.rows) + g.cols) * g.depth * 2 / 6.2e6 + 4.0;
  Plan best{0, 0, 0, 0, 1e30};
  auto consider = [&](double us, const Plan& p) {
    if (us < best.us) {
      best = p;
      best.us = us;
    }
  };
  const bool drain = drained(g, o);
  for (int width = 256; width >= (drain ? 256 : 128); width /= 2) {
    const int64_t rounds = cdiv(pair_tiles(g, layer, width), sms / 2);
    const double feed = kb * (width == 256 ? 0.33 : 0.27), finish = output * width / 256;
    const double us = rounds * (feed > finish ? feed : finish) + (feed > finish ? finish : feed) +
                      (drain ? rounds * finish / 2 : 0.0) + 5.0 + (rounds > 1 ? 2.0 : 0.0);
    consider(us > traffic + 3.0 ? us : traffic + 3.0, Plan{width, 0, 0, 0, us});
  }
  const int unit = g.left_mn ? 64 : 16;
  const int64_t fewest = cdiv(g.rows, kMaxTokens);
  for (int64_t mt = fewest; mt <= fewest + 4; ++mt) {
    const int tt = static_cast<int>(cdiv(cdiv(g.rows, mt), unit) * unit);
    if (tt > kMaxTokens) continue;
    const int64_t tiles = cdiv(g.cols, kRows) * cdiv(g.rows, tt);
    for (int size = 1; size <= 8 && size <= kb; size *= 2) {
      for (int per_sm = 1; per_sm <= 2; ++per_sm) {
        const int64_t blocks = tiles * size;
        if (per_sm == 2 && blocks <= sms) continue;
        const int stage = (kRows + tt) * BK * 2;
        int stages = ((per_sm == 2 ? SMEM_LIMIT / 2 - 1024 : SMEM_LIMIT) - 1024 - 512) / stage;
        if (stages > 12) stages = 12;
        if (size > 1 && stages * stage < tt * kRows * 4) continue;  // a tile's sums do not fit
        const int share = static_cast<int>(kb) / size;
        if (o.out_f32 && share > kWholeBlocks * parts_of(tt, share)) continue;
        const double mma = 0.34 * tt / 256, bytes = stage / 100e3;
        const double feed = kb / size * (mma > bytes ? mma : bytes);
        const double finish = 1.0 + output * tt / 256 / size + (size > 1 ? 1.5 + tt * 0.01 : 0.0);
        const double rounds = static_cast<double>(cdiv(blocks, per_sm * sms));
        const double us = rounds * (per_sm == 2 ? 2 * feed + 1.3 * finish : feed + finish) + 3.0;
        // the memory rests while an SM's only block finishes
        const double memory = traffic + (per_sm == 1 ? rounds * finish : 0.0);
        consider(us > memory ? us : memory, Plan{0, tt, size, stages, us});
      }
    }
  }
  return best;
}

Results results_of(const Product& g, const LinearOut& o) {
  const int64_t n = g.rows * g.cols;
  return Results{{o.y, o.preact}, {n * (o.out_f32 ? 4 : 2), n * 2}};
}

template <bool A_MN, bool B_MN>
int launch_split(const Product& g, const Plan& s, const LinearOut& out, uint32_t* err, bool clear,
                 bool lost, cudaStream_t st) {
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
  a.parts = out.out_f32 ? parts_of(s.tt, a.k_blocks / s.size) : 1;
  a.out = out;
  a.results = results_of(g, out);
  a.err = err;
  a.clear = clear;
  a.lost = lost;
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
              bool lost, cudaStream_t st) {
  if (g.left_mn) return launch_split<true, true>(g, s, out, err, clear, lost, st);  // dweight: both are
  return g.right_mn ? launch_split<true, false>(g, s, out, err, clear, lost, st)
                    : launch_split<false, false>(g, s, out, err, clear, lost, st);
}

// Whether every pair has one tile at most, so that the schedule's counters are not needed.
bool one_round(const Product& g, bool layer, int width) {
  return pair_tiles(g, layer, width) <= pair_capacity();
}

// The product by CTA pairs; kind 0: a layer's output, 1: dx, 2: dweight.
int run_pair(const Product& p, int width, int kind, const LinearOut& out, uint32_t* err, int slot,
             bool clear, bool lost, cudaStream_t st) {
  const Product g = kind ? p
                         : Product{p.right, p.left, p.cols, p.rows, p.depth, p.ld_right, p.ld_left,
                                   p.right_mn, p.left_mn};
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
  sh.one_round = one_round(p, kind == 0, width);
  sh.lost = lost;
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
  ea.results = results_of(p, out);
  const bool wide = width == 256;
  if (kind == 0) {
    ea.lin = out;
    if (drained(g, out))
      return rc_of((g.left_mn ? launch_linear_f32 : launch_linear_vh_f32)(A, B, sh, ea, st));
    return rc_of((g.left_mn ? (wide ? launch_linear : launch_linear_128)
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
  const int64_t threads = cdiv(p->N, 8);
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

int launch_dz(const DzArgs& a, int64_t strips, cudaStream_t st) {
  const int64_t lanes = cdiv(a.N, 8);
  const int threads = lanes >= kDzThreads ? kDzThreads : static_cast<int>(cdiv(lanes, 32) * 32);
  const int64_t cols = cdiv(lanes, threads);
  if (cols > (int64_t(1) << 31) - 1) return FLCE_ERR_BAD_SHAPE;
  auto kernel = a.N % 8 == 0 ? (a.dout_f32 ? dz_kernel<true, true> : dz_kernel<true, false>)
                             : (a.dout_f32 ? dz_kernel<false, true> : dz_kernel<false, false>);
  kernel<<<dim3(static_cast<unsigned>(cols), static_cast<unsigned>(strips)), threads, 0, st>>>(a);
  return rc_of(cudaGetLastError());
}

// One gradient's product.
int run_gradient(const Product& g, const Plan& plan, int kind, void* out, uint32_t* err, int slot,
                 bool lost, cudaStream_t st) {
  LinearOut o{};
  o.y = out;
  o.ld = g.cols;
  return plan.width ? run_pair(g, plan.width, kind, o, err, slot, false, lost, st)
                    : run_split(g, plan, o, err, false, lost, st);
}

// Below this many microseconds of the smaller of two products, running them side by side costs the host
// more than it saves the GPU.
constexpr double kSideBySide = 10.0;

// The calls; lost: the self-test of the bounded waits.
int forward(const flce_linear_params* p, const void* x, const void* weight, const void* bias,
            const void* residual, void* y, void* preact, void* workspace, size_t ws_bytes,
            void* stream, bool lost) {
  int rc = check(p);
  if (rc) return rc;
  if (!weight || !workspace || (p->M > 0 && (!x || !y))) return FLCE_ERR_BAD_ARG;
  if ((addr(x) | addr(weight) | addr(residual) | addr(y) | addr(preact)) & 15 || addr(bias) & 1 ||
      addr(workspace) & 255)
    return FLCE_ERR_ALIGN;
  if (ws_bytes < kHeader) return FLCE_ERR_WS_TOO_SMALL;
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
  const Product g = forward_product(p, x, weight);
  const Plan plan = choose(g, sms, true, o);
  // The header is cleared ahead where the schedule's counters are needed (and in the bounds-checking
  // build, whose first findings a kernel could wipe out), else by the kernel: a memset is a
  // microsecond or two of a small layer's ten.
  const bool ahead = FLCE_DEBUG || (plan.width && !one_round(g, true, plan.width));
  if (ahead && (rc = rc_of(cudaMemsetAsync(ws, 0, kHeader, st)))) return rc;
  rc = plan.width ? run_pair(g, plan.width, 0, o, err, 0, !ahead, lost, st)
                  : run_split(g, plan, o, err, !ahead, lost, st);
  if (rc) return rc;
  return p->validate ? read_status(ws, st) : FLCE_OK;
}

int backward(const flce_linear_params* p, const void* dout, const void* x,
             const void* weight, const void* preact, void* dx, void* dweight, void* dbias,
             void* workspace, size_t ws_bytes, void* stream, bool lost) {
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
  if (p->M == 0) {  // sums over no tokens
    if ((rc = rc_of(cudaMemsetAsync(ws, 0, kHeader, st)))) return rc;
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
    a.header = err;
    a.part = dbias ? reinterpret_cast<float*>(ws + L.db) : nullptr;
    a.M = p->M;
    a.N = p->N;
    a.ld_dz = L.ld_dz;
    a.strip = dz_strip(p);
    a.act = p->activation;
    a.dout_f32 = f32;
    rc = launch_dz(a, L.strips, st);
    if (rc) return rc;
  } else if ((rc = rc_of(cudaMemsetAsync(ws, 0, kHeader, st)))) {
    return rc;
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
  const Product x_product = dx_product(p, dz, ld_dz, weight), w_product = dw_product(p, dz, ld_dz, x);
  Plan x_plan{}, w_plan{};
  if (dx) x_plan = choose(x_product, sms, false, LinearOut{});
  if (dweight) w_plan = choose(w_product, sms, false, LinearOut{});
  cudaStream_t side = st;
  const bool both = dx && dweight && x_plan.us >= kSideBySide && w_plan.us >= kSideBySide;
  if (both && (rc = side_fork(st, &side))) return rc;
  if (dx && (rc = run_gradient(x_product, x_plan, 1, dx, err, 0, lost, st))) return rc;
  if (dweight && (rc = run_gradient(w_product, w_plan, 2, dweight, err, 1, lost, side))) return rc;
  if (both && (rc = side_join(st))) return rc;
  return p->validate ? read_status(ws, st) : FLCE_OK;
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
  return forward(p, x, weight, bias, residual, y, preact, workspace, ws_bytes, stream, false);
}

int flce_linear_backward(const flce_linear_params* p, const void* dout, const void* x,
                         const void* weight, const void* preact, void* dx, void* dweight,
                         void* dbias, void* workspace, size_t ws_bytes, void* stream) {
  return backward(p, dout, x, weight, preact, dx, dweight, dbias, workspace, ws_bytes, stream, false);
}

int flce_selftest_linear_timeout(const flce_linear_params* p, const void* x, const void* weight,
                                 const void* residual, void* y, void* preact, void* workspace,
                                 size_t ws_bytes, void* stream) {
  return forward(p, x, weight, nullptr, residual, y, preact, workspace, ws_bytes, stream, true);
}

int flce_selftest_linear_backward_timeout(const flce_linear_params* p, const void* dout, const void* x,
                                          const void* weight, const void* preact, void* dx, void* dweight,
                                          void* workspace, size_t ws_bytes, void* stream) {
  return backward(p, dout, x, weight, preact, dx, dweight, nullptr, workspace, ws_bytes, stream, true);
}

}  // extern "C"
