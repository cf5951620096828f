// Dense layer  y = act(x W + b) + r  and its gradients.
//
// Two GEMM kernels, both tcgen05 with operands brought by TMA:
//
//   pair     flce_gemm.cuh's CTA pairs on 256 x 256 tiles, for shapes with enough tiles to fill
//            the GPU in whole rounds: bound by the tensor cores.
//   stream   (here) for all others, above all few tokens, which are bound by the bytes of the
//            weight.  The product is taken transposed, y^T = W^T x^T: 128 columns of y are the
//            128 TMEM lanes and up to 256 tokens its columns, so that a tile has no rows for
//            tokens that are not there, and a warp's stores run along y's rows whatever N is.
//            The k-blocks of all tiles, in order, are one line that is cut into equal pieces, one
//            per SM: every SM streams the same number of bytes, whatever the tile count.  A tile
//            cut between SMs leaves fp32 partial sums in the workspace, which join_kernel adds in
//            the line's order, and finishes.
//
// Either gives the same sums for any number of SMs at a time, in a fixed order: results repeat
// bit for bit.
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
constexpr int kRows = 128;            // columns of y per tile of the stream kernel
constexpr int kStreamThreads = 192;   // producer, issuer, four epilogue warps
constexpr int kMaxTokens = 256;       // tokens per tile
constexpr int kStreamCtas = 160;      // partial slots: two per block, at most this many blocks

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
// 16 fp32 columns of this warp's 32 TMEM lanes
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// ------------------------------------------------------------------ stream kernel
struct StreamArgs {
  int32_t M, N;                 // tokens and columns of y
  int32_t m_tiles, tiles;       // token tiles vary fastest
  int32_t k_blocks;
  int64_t blocks;               // k-blocks of all tiles
  LinearOut out;
  float* part;                  // [2 * grid][TT][128]
  uint32_t* err;
  int32_t clear;                // err is not cleared yet
  int64_t a_inner, a_outer, b_inner, b_outer;  // FLCE_DEBUG: extents behind the maps
};

// Piece c of g: k-blocks [cut(c), cut(c + 1)) of the line.
__host__ __device__ __forceinline__ int64_t cut(int64_t blocks, int64_t c, int64_t g) {
  return blocks * c / g;
}

template <int TT>
struct StreamCfg {
  static constexpr int A_BYTES = kRows * BK * 2;
  static constexpr int B_BYTES = TT * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int FIT = (SMEM_LIMIT - 1024 - 512) / STAGE_BYTES;
  static constexpr int STAGES = FIT > 12 ? 12 : FIT;
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + 512;
  static constexpr int NACC = 2;
  static_assert((2 * STAGES + 2 * NACC) * 8 + 8 <= 512, "barrier area");
};

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

template <bool A_MN, bool B_MN, int TT>
__global__ void __launch_bounds__(kStreamThreads, 1)
    stream_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ StreamArgs a) {
  using C = StreamCfg<TT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + C::STAGES * C::A_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sB + C::STAGES * C::B_BYTES);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + C::NACC;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(tempty + C::NACC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint32_t kTmem = 2 * TT < 32 ? 32 : 2 * TT;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < C::NACC; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) tmem_alloc(tmem_holder, kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  // the error word of a launch whose waits all end in time: a timeout is seconds away
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.clear) *a.err = 0;
  // what follows may start: it waits for this launch's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int64_t r0 = cut(a.blocks, blockIdx.x, gridDim.x);
  const int64_t r1 = cut(a.blocks, blockIdx.x + 1, gridDim.x);
  const int first = static_cast<int>(r0 / a.k_blocks);
  const int k_first = static_cast<int>(r0 - int64_t(first) * a.k_blocks);

  if (warp == 0) {
    if (lane == 0) {
      // the weight is read once, by one SM: it goes first; x is read by every tile
      const uint64_t pol_a = l2_policy(L2_NORMAL), pol_b = l2_policy(L2_EVICT_LAST);
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      int tile = first, kb = k_first;
      for (int64_t r = r0; r < r1 && ok; ++r) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, a.err)) {
          ok = false;
          break;
        }
        const int n0 = tile / a.m_tiles * kRows, m0 = tile % a.m_tiles * TT, k0 = kb * BK;
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
        mbar_arrive_expect_tx(&full[stage], C::STAGE_BYTES);
        load_rows<A_MN, kRows>(sA + stage * C::A_BYTES, &tmA, &full[stage], n0, k0, pol_a);
        load_rows<B_MN, TT>(sB + stage * C::B_BYTES, &tmB, &full[stage], m0, k0, pol_b);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        if (++kb == a.k_blocks) {
          kb = 0;
          ++tile;
        }
      }
      // every filled stage has been released before the block ends
      for (int i = 0; i < C::STAGES && ok; ++i) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, a.err)) break;
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t IDESC = idesc_bf16_f32(kRows, TT, A_MN, B_MN);
      GemmShape strides{};
      strides.mn_lbo = MN_ATOM_BYTES;
      strides.mn_sbo = 1024;
      const uint64_t a0 = operand_desc<A_MN>(smem_u32(sA), 0, strides);
      const uint64_t b0 = operand_desc<B_MN>(smem_u32(sB), 0, strides);
      constexpr uint64_t kKA = (A_MN ? UK * 128 : UK * 2) >> 4;
      constexpr uint64_t kKB = (B_MN ? UK * 128 : UK * 2) >> 4;
      uint32_t stage = 0, phase = 0;
      int kb = k_first, it = 0;
      bool begin = true;  // of an accumulator
      for (int64_t r = r0; r < r1; ++r) {
        const int acc = it & 1;
        const uint32_t d = tmem_base + acc * TT;
        if (begin) {
          if (!mbar_wait(&tempty[acc], ((it >> 1) & 1) ^ 1u, abort_flag, a.err)) break;
          tc_fence_after();
        }
        if (!mbar_wait(&full[stage], phase, abort_flag, a.err)) break;
        tc_fence_after();
        const uint64_t as = a0 + stage * (C::A_BYTES >> 4), bs = b0 + stage * (C::B_BYTES >> 4);
#pragma unroll
        for (int kk = 0; kk < BK / UK; ++kk)
          umma_bf16(d, as + kk * kKA, bs + kk * kKB, IDESC, begin && kk == 0 ? 0u : 1u);
        umma_commit(&empty[stage]);
        begin = false;
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        if (++kb == a.k_blocks || r + 1 == r1) {
          kb = 0;
          umma_commit(&tfull[acc]);
          ++it;
          begin = true;
        }
      }
    }
    __syncwarp();
  } else {
    const int q = warp & 3;
    int it = 0;
    int64_t r = r0;
    for (int tile = first; r < r1; ++tile, ++it) {
      const int64_t t0 = int64_t(tile) * a.k_blocks, t1 = t0 + a.k_blocks;
      const int64_t end = t1 < r1 ? t1 : r1;
      const bool whole = r == t0 && end == t1;
      const int acc = it & 1;
      if (!mbar_wait(&tfull[acc], (it >> 1) & 1, abort_flag, a.err)) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * TT;
      const int n = tile / a.m_tiles * kRows + q * 32 + lane, m0 = tile % a.m_tiles * TT;
      const int rows = a.M - m0 < TT ? a.M - m0 : TT;  // tokens of the tile
      const bool n_ok = n < a.N;
      // a block's first piece of a tile may be one, and its last
      float* part = a.part + (int64_t(blockIdx.x) * 2 + (r == r0 ? 0 : 1)) * TT * kRows +
                    q * 32 + lane;
      const float bias =
          whole && a.out.bias && n_ok ? __bfloat162float(a.out.bias[n]) : 0.0f;
#pragma unroll 1
      for (int c = 0; c < rows; c += 16) {
        float x[16];
        __syncwarp();
        tmem_ld16(tbase + c, x);
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c + i < rows) part[(c + i) * kRows] = x[i];
        } else if (n_ok) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c + i < rows)
              linear_store1(a.out, int64_t(m0 + c + i) * a.out.ld + n, bias, x[i]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_local(&tempty[acc]);
      r = end;
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, kTmem);
}

// Tiles cut between blocks of the stream kernel: their partial sums in the line's order, then
// the epilogue.  A block of 128 threads per (tile, 16 tokens).
template <int TT>
__global__ void __launch_bounds__(kRows) join_kernel(const __grid_constant__ StreamArgs a, int grid) {
  const int tile = blockIdx.x, m0 = tile % a.m_tiles * TT + blockIdx.y * 16;
  const int n = tile / a.m_tiles * kRows + threadIdx.x;
  // every block waits: what follows this launch follows the one before it too
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (m0 >= a.M) return;
  const int64_t t0 = int64_t(tile) * a.k_blocks, t1 = t0 + a.k_blocks;
  // the blocks that hold the tile's first and last k-block
  int64_t c0 = t0 * grid / a.blocks, c1 = (t1 - 1) * grid / a.blocks;
  while (cut(a.blocks, c0 + 1, grid) <= t0) ++c0;
  while (cut(a.blocks, c1 + 1, grid) <= t1 - 1) ++c1;
  if (c0 == c1) return;  // whole
  const float bias = a.out.bias && n < a.N ? __bfloat162float(a.out.bias[n]) : 0.0f;
  const int rows = a.M - m0 < 16 ? a.M - m0 : 16;
  float sum[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) sum[i] = 0.0f;
  for (int64_t c = c0; c <= c1; ++c) {
    // the piece is the block's first unless the block began with an earlier tile
    const bool later = cut(a.blocks, c, grid) < t0;
    const float* p = a.part + (c * 2 + later) * TT * kRows + int64_t(blockIdx.y) * 16 * kRows +
                     threadIdx.x;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < rows) sum[i] += __ldcg(p + i * kRows);
  }
  if (n >= a.N) return;
#pragma unroll 1
  for (int i = 0; i < rows; ++i) {
    float v = sum[0];
#pragma unroll
    for (int j = 1; j < 16; ++j)
      if (j == i) v = sum[j];
    linear_store1(a.out, int64_t(m0 + i) * a.out.ld + n, bias, v);
  }
}

// ------------------------------------------------------------------ dz and db
constexpr int kDzThreads = 256;
constexpr int kDzWarps = kDzThreads / 32;

struct DzArgs {
  const void* dout;
  const __nv_bfloat16* preact;
  __nv_bfloat16* dz;  // NULL: dout serves
  float* part;        // [strips, N], or NULL
  int64_t M, N, ld_dz, strip;
  int32_t act, dout_f32;
};

// A block takes a strip of rows and 32 * VEC columns; a warp's rows are kDzWarps apart, and a
// thread sums its columns over them.
template <int VEC>
__global__ void __launch_bounds__(kDzThreads) dz_kernel(const __grid_constant__ DzArgs a) {
  __shared__ float sums[kDzWarps][32 * VEC];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t n = (int64_t(blockIdx.x) * 32 + lane) * VEC;
  const int64_t m0 = blockIdx.y * a.strip;
  const int64_t m1 = m0 + a.strip < a.M ? m0 + a.strip : a.M;
  float sum[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
  if (n < a.N) {
#pragma unroll 2
    for (int64_t m = m0 + warp; m < m1; m += kDzWarps) {
      const int64_t at = m * a.N + n;
      float g[VEC], z[VEC];
      if constexpr (VEC == 8) {
        if (a.dout_f32) {
          const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.dout) + at);
          const float4 u = __ldg(p), v = __ldg(p + 1);
          g[0] = u.x; g[1] = u.y; g[2] = u.z; g[3] = u.w;
          g[4] = v.x; g[5] = v.y; g[6] = v.z; g[7] = v.w;
        } else {
          unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(
                            static_cast<const __nv_bfloat16*>(a.dout) + at)), g);
        }
        if (a.act != FLCE_ACT_NONE)
          unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(a.preact + at)), z);
      } else {
        g[0] = a.dout_f32 ? static_cast<const float*>(a.dout)[at]
                          : __bfloat162float(static_cast<const __nv_bfloat16*>(a.dout)[at]);
        if (a.act != FLCE_ACT_NONE) z[0] = __bfloat162float(a.preact[at]);
      }
      if (a.act != FLCE_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) g[i] *= activate_slope(z[i], a.act);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum[i] += g[i];
      if (a.dz) {
        __nv_bfloat16* o = a.dz + m * a.ld_dz + n;
        if constexpr (VEC == 8) *reinterpret_cast<uint4*>(o) = pack_bf16x8(g);
        else *o = __float2bfloat16_rn(g[0]);
      }
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < VEC; ++i) sums[warp][lane * VEC + i] = sum[i];
  __syncthreads();
  for (int j = threadIdx.x; j < 32 * VEC; j += kDzThreads) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kDzWarps; ++w) s += sums[w][j];
    const int64_t c = int64_t(blockIdx.x) * 32 * VEC + j;
    if (c < a.N) a.part[blockIdx.y * a.N + c] = s;
  }
}

__global__ void __launch_bounds__(128) db_kernel(const float* part, int64_t strips, int64_t N,
                                                 __nv_bfloat16* db) {
  const int64_t n = int64_t(blockIdx.x) * 128 + threadIdx.x;
  if (n >= N) return;
  float s = 0.0f;
#pragma unroll 8
  for (int64_t i = 0; i < strips; ++i) s += __ldcg(part + i * N + n);
  db[n] = __float2bfloat16_rn(s);
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

// Token tile of the stream kernel: 16 to 256, the tokens' own number rounded up.
int token_tile(int64_t rows, bool left_mn) {
  int tt = left_mn ? 64 : 16;  // an MN-major operand comes in pieces of 64
  while (tt < kMaxTokens && tt < rows) tt *= 2;
  return tt;
}

struct StreamPlan {
  int tt;
  int64_t m_tiles, tiles, k_blocks, blocks;
  int grid;
  size_t part_bytes;
};

StreamPlan stream_plan(const Product& g, int sms) {
  StreamPlan s{};
  s.tt = token_tile(g.rows, g.left_mn);
  s.m_tiles = cdiv(g.rows, s.tt);
  s.tiles = s.m_tiles * cdiv(g.cols, kRows);
  s.k_blocks = cdiv(g.depth, BK);
  s.blocks = s.tiles * s.k_blocks;
  const int most = sms < kStreamCtas ? sms : kStreamCtas;
  s.grid = static_cast<int>(s.blocks < most ? s.blocks : most);
  s.part_bytes = align256(size_t(2) * most * s.tt * kRows * 4);
  return s;
}

// Whether the pair kernel takes a product.  Its rounds of 256 x 256 tiles over the CTA pairs
// against the stream kernel's even share of all tiles' k-blocks: kEven is what the latter's rate is
// of the former's.
bool use_pair(const Product& g, int pairs) {
  const int64_t tiles = cdiv(g.rows, 256) * cdiv(g.cols, 256);
  if (g.cols % 8 != 0 || tiles < pairs / 2) return false;
  const int64_t rounds = cdiv(tiles, pairs);
  const StreamPlan s = stream_plan(g, 2 * pairs);
  const double stream = static_cast<double>(s.tiles) * s.tt * kRows / (256.0 * 256.0) / pairs;
  constexpr double kEven = 0.80;
  return static_cast<double>(rounds) * kEven <= stream;
}

template <bool A_MN, bool B_MN, int TT>
int launch_stream(const Product& g, const StreamPlan& s, StreamArgs a, cudaStream_t st) {
  using C = StreamCfg<TT>;
  auto kernel = stream_kernel<A_MN, B_MN, TT>;
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  int rc = rc_of(cudaGetDevice(&dev));
  if (rc) return rc;
  if (!(ready.load() >> (dev & 63) & 1)) {
    if ((rc = rc_of(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::SMEM_BYTES))))
      return rc;
    ready.fetch_or(uint64_t(1) << (dev & 63));
  }
  CUtensorMap A, B;
  if (!(A_MN ? tensor_map(&A, g.right, g.cols, g.depth, g.ld_right, 64, BK)
             : tensor_map(&A, g.right, g.depth, g.cols, g.ld_right, BK, kRows)) ||
      !(B_MN ? tensor_map(&B, g.left, g.rows, g.depth, g.ld_left, 64, BK)
             : tensor_map(&B, g.left, g.depth, g.rows, g.ld_left, BK, TT)))
    return FLCE_ERR_CUDA;
  a.a_inner = A_MN ? g.cols : g.depth;
  a.a_outer = A_MN ? g.depth : g.cols;
  a.b_inner = B_MN ? g.rows : g.depth;
  a.b_outer = B_MN ? g.depth : g.rows;
  kernel<<<static_cast<unsigned>(s.grid), kStreamThreads, C::SMEM_BYTES, st>>>(A, B, a);
  if ((rc = rc_of(cudaGetLastError()))) return rc;
  if (s.blocks % s.grid == 0 && (s.blocks / s.grid) % s.k_blocks == 0) return FLCE_OK;  // no tile is cut
  const int64_t groups = cdiv(g.rows < TT ? g.rows : TT, 16);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(s.tiles), static_cast<unsigned>(groups));
  cfg.blockDim = dim3(kRows);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return rc_of(cudaLaunchKernelEx(&cfg, join_kernel<TT>, a, s.grid));
}

template <bool A_MN, bool B_MN>
int launch_stream_tt(const Product& g, const StreamPlan& s, const StreamArgs& a, cudaStream_t st) {
  if constexpr (!B_MN) {
    if (s.tt == 16) return launch_stream<A_MN, B_MN, 16>(g, s, a, st);
    if (s.tt == 32) return launch_stream<A_MN, B_MN, 32>(g, s, a, st);
  }
  if (s.tt == 64) return launch_stream<A_MN, B_MN, 64>(g, s, a, st);
  if (s.tt == 128) return launch_stream<A_MN, B_MN, 128>(g, s, a, st);
  return launch_stream<A_MN, B_MN, 256>(g, s, a, st);
}

int run_stream(const Product& g, const LinearOut& out, uint8_t* part, uint32_t* err, bool clear,
               int sms, cudaStream_t st) {
  const StreamPlan s = stream_plan(g, sms);
  if (s.tiles > (int64_t(1) << 31) - 1) return FLCE_ERR_BAD_SHAPE;
  StreamArgs a{};
  a.M = static_cast<int32_t>(g.rows);
  a.N = static_cast<int32_t>(g.cols);
  a.m_tiles = static_cast<int32_t>(s.m_tiles);
  a.tiles = static_cast<int32_t>(s.tiles);
  a.k_blocks = static_cast<int32_t>(s.k_blocks);
  a.blocks = s.blocks;
  a.out = out;
  a.part = reinterpret_cast<float*>(part);
  a.err = err;
  a.clear = clear;
  if (g.left_mn) return launch_stream_tt<true, true>(g, s, a, st);  // dweight: both are
  return g.right_mn ? launch_stream_tt<true, false>(g, s, a, st)
                    : launch_stream_tt<false, false>(g, s, a, st);
}

// The product by CTA pairs; kind 0: a layer's output, 1: dx, 2: dweight.
int run_pair(const Product& g, int kind, const LinearOut& out, uint32_t* err, int slot,
             cudaStream_t st) {
  CUtensorMap A, B;
  if (!(g.left_mn ? tensor_map(&A, g.left, g.rows, g.depth, g.ld_left, 64, BK)
                  : tensor_map(&A, g.left, g.depth, g.rows, g.ld_left, BK, 64)) ||
      !(g.right_mn ? tensor_map(&B, g.right, g.cols, g.depth, g.ld_right, 64, BK)
                   : tensor_map(&B, g.right, g.depth, g.cols, g.ld_right, BK, 64)))
    return FLCE_ERR_CUDA;
  GemmShape sh = pair_shape(L2_EVICT_LAST, L2_NORMAL);
  sh.m_tiles = static_cast<int>(cdiv(g.rows, PAIR_BM));
  sh.n_tiles = static_cast<int>(cdiv(g.cols, 256));
  sh.k_blocks = static_cast<int>(cdiv(g.depth, BK));
  sh.raster = 0;
  sh.sched = reinterpret_cast<unsigned int*>(reinterpret_cast<uint8_t*>(err) + kSched + 8 * slot);
  sh.a_inner = g.left_mn ? g.rows : g.depth;
  sh.a_outer = g.left_mn ? g.depth : g.rows;
  sh.b_inner = g.right_mn ? g.cols : g.depth;
  sh.b_outer = g.right_mn ? g.depth : g.cols;
  plan_pair(&sh, int64_t(PAIR_BM) * g.depth * 2);
  EpiArgs ea{};
  ea.rows = static_cast<int>(g.rows);
  ea.cols = static_cast<int>(g.cols);
  ea.err = err;
  if (kind == 0) {
    ea.lin = out;
    return rc_of((g.right_mn ? launch_linear : launch_linear_vh)(A, B, sh, ea, st));
  }
  if (kind == 1) {
    ea.acc_out = static_cast<__nv_bfloat16*>(out.y);
    ea.acc_mode = ACC_ONLY;
    ea.ld_acc = out.ld;
    return rc_of((g.right_mn ? launch_bwd_dhidden_vh : launch_bwd_dhidden)(A, B, sh, ea, st));
  }
  ea.out = static_cast<__nv_bfloat16*>(out.y);
  ea.ld_out = out.ld;
  return rc_of(launch_bwd_dweight(A, B, sh, ea, st));
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

// Workspace sizes hold for any number of SMs up to kStreamCtas, so that they need no device.
size_t part_size(const Product& g) { return stream_plan(g, kStreamCtas).part_bytes; }

int64_t dz_strip(int64_t M) {
  // strips of 64 rows, at most 256 of them
  const int64_t s = cdiv(M, 256);
  return s < 64 ? 64 : cdiv(s, kDzWarps) * kDzWarps;
}

struct BwdLayout {
  size_t dz, db, part[2], total;
  int64_t ld_dz, strips;
};

BwdLayout bwd_layout(const flce_linear_params* p) {
  BwdLayout L{};
  L.ld_dz = cdiv(p->N, 8) * 8;
  L.strips = cdiv(p->M, dz_strip(p->M));
  size_t off = kHeader;
  L.dz = off; off += align256(static_cast<size_t>(p->M) * L.ld_dz * 2);
  L.db = off; off += align256(static_cast<size_t>(L.strips) * p->N * 4);
  L.part[0] = off; off += part_size(dx_product(p, nullptr, L.ld_dz, nullptr));
  L.part[1] = off; off += part_size(dw_product(p, nullptr, L.ld_dz, nullptr));
  L.total = off;
  return L;
}

template <int VEC>
int launch_dz(const DzArgs& a, int64_t strips, cudaStream_t st) {
  const int64_t cols = cdiv(a.N, 32 * VEC);
  if (cols > (int64_t(1) << 31) - 1) return FLCE_ERR_BAD_SHAPE;
  dz_kernel<VEC><<<dim3(static_cast<unsigned>(cols), static_cast<unsigned>(strips)), kDzThreads, 0,
                   st>>>(a);
  return rc_of(cudaGetLastError());
}

// One gradient's product, by whichever kernel suits it.
int run_gradient(const Product& g, int kind, void* out, uint8_t* ws, size_t part, int slot, int sms,
                 cudaStream_t st) {
  LinearOut o{};
  o.y = out;
  o.ld = g.cols;
  uint32_t* err = reinterpret_cast<uint32_t*>(ws);
  if (use_pair(g, pair_capacity())) return run_pair(g, kind, o, err, slot, st);
  return run_stream(g, o, ws + part, err, false, sms, st);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_linear_check_params(const flce_linear_params* p) { return check(p); }

size_t flce_linear_workspace_size(const flce_linear_params* p, int backward) {
  if (check(p) != FLCE_OK) return 0;
  if (backward) return bwd_layout(p).total;
  return kHeader + part_size(forward_product(p, nullptr, nullptr));
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
  const Product g = forward_product(p, x, weight);
  if (use_pair(g, pair_capacity())) {
    if ((rc = rc_of(cudaMemsetAsync(ws, 0, kHeader, st)))) return rc;
    rc = run_pair(g, 0, o, err, 0, st);
  } else {
    rc = run_stream(g, o, ws + kHeader, err, true, sms, st);
  }
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
    a.strip = dz_strip(p->M);
    a.act = p->activation;
    a.dout_f32 = f32;
    rc = p->N % 8 == 0 ? launch_dz<8>(a, L.strips, st) : launch_dz<1>(a, L.strips, st);
    if (rc) return rc;
  }
  if (dbias) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(cdiv(p->N, 128)));
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    if ((rc = rc_of(cudaLaunchKernelEx(&cfg, db_kernel, reinterpret_cast<const float*>(ws + L.db),
                                       L.strips, p->N, static_cast<__nv_bfloat16*>(dbias)))))
      return rc;
  }
  // dx on the caller's stream, dweight beside it, as the head's backward does
  cudaStream_t side = st;
  const bool both = dx && dweight;
  if (both && (rc = side_fork(st, &side))) return rc;
  if (dx && (rc = run_gradient(dx_product(p, dz, ld_dz, weight), 1, dx, ws, L.part[0], 0, sms, st)))
    return rc;
  if (dweight &&
      (rc = run_gradient(dw_product(p, dz, ld_dz, x), 2, dweight, ws, L.part[1], 1, sms, side)))
    return rc;
  if (both && (rc = side_join(st))) return rc;
  return p->validate ? read_status(ws, st) : FLCE_OK;
}

}  // extern "C"
