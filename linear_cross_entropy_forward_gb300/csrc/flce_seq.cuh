// Tokens in sequences: the layouts of the losses over sequences of tokens (the policy
// and preference losses) and the parts their kernels share.
//
// A batch is padded, [B, S] with a row stride per array, or packed, S tokens of which
// sequence i owns [cu[i], cu[i + 1]).  Both are one axis of positions: sequence i of a
// padded batch starts at position i * S, and an array's element for position p of
// sequence i is base[p + i * skip] with skip = row stride - S (0 when packed).
//
// The axis is cut at every multiple of kTile positions and at every sequence's start.
// The pieces need no list: the piece of sequence i in tile j has number i + j (each new
// piece moves on to the next tile or to the next sequence), so the first piece of
// sequence i is f(i) = start(i) / kTile + i, which rises strictly, and piece u belongs
// to the last i with f(i) <= u.  There are at most S / kTile + B + 1 numbers; the unused
// ones are empty pieces.  One long sequence is spread over the GPU as well as many short
// ones, whatever their lengths, and nothing about them is read on the host.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/flce.h"

namespace flce {

constexpr int kSeqThreads = 256;
constexpr int kSeqWarps = kSeqThreads / 32;
constexpr int kSeqPerThread = 4;
constexpr int64_t kTile = int64_t(kSeqThreads) * kSeqPerThread;
// Blocks an SM holds at once (the launch bounds of the kernels): the grid of a
// cooperative launch is at most this times the SM count.
constexpr int kSeqBlocksPerSm = 4;

struct Seqs {
  int64_t B, S, total;  // total: positions (B * S padded, S packed)
  const void* cu;       // NULL: padded
  int cu64;
  const void* mask;     // NULL: every token counts
  int mask_labels;      // 0: bytes, non-zero counts; 1: int64 labels != ignore_index
  int64_t ignore_index;
  int64_t mask_skip;
};

inline int64_t seq_pieces(int64_t B, int64_t total) { return total / kTile + B + 1; }

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) {
  return x < lo ? lo : (x > hi ? hi : x);
}

// Start of sequence i (i = B: the end of the last), inside [0, total] whatever the
// array holds, so that no offset built from it leaves the arrays.
__device__ __forceinline__ int64_t seq_start(const Seqs& q, int64_t i) {
  if (!q.cu) return i * q.S;
  const int64_t v = q.cu64 ? __ldg(static_cast<const long long*>(q.cu) + i)
                           : __ldg(static_cast<const int*>(q.cu) + i);
  return clamp64(v, 0, q.total);
}

__device__ __forceinline__ int64_t seq_first_piece(const Seqs& q, int64_t i) {
  return seq_start(q, i) / kTile + i;
}

struct Piece {
  int64_t seq, begin, end;  // empty: begin >= end
};

// The piece with number u; called by the whole block (a search over cu takes one
// coalesced load per 256-fold narrowing instead of a chain of dependent ones).
__device__ __forceinline__ Piece find_piece(const Seqs& q, int64_t u) {
  int64_t i;
  if (!q.cu) {
    // f(i) = i * S / kTile + i: off by at most one from the real quotient
    i = clamp64(static_cast<int64_t>(static_cast<double>(u) * kTile / (q.S + kTile)), 0, q.B - 1);
    while (i > 0 && i * q.S / kTile + i > u) --i;
    while (i + 1 < q.B && (i + 1) * q.S / kTile + i + 1 <= u) ++i;
  } else {
    int64_t lo = 0, n = q.B;  // the answer is in [lo - 1, lo + n)
    while (n > 0) {
      const int64_t step = (n + kSeqThreads - 1) / kSeqThreads;
      const int64_t k = threadIdx.x * step;
      const int below =
          __syncthreads_count(k < n && seq_first_piece(q, lo + k) <= u);
      if (below == 0) break;
      const int64_t from = (below - 1) * step;
      const int64_t left = n - from;
      lo += from + 1;
      n = (left < step ? left : step) - 1;
    }
    i = lo - 1;
  }
  Piece p{i, 0, 0};
  if (i < 0) return p;
  const int64_t a = seq_start(q, i), b = seq_start(q, i + 1);
  const int64_t tile = (u - i) * kTile;
  p.begin = a > tile ? a : tile;
  p.end = b < tile + kTile ? b : tile + kTile;
  return p;
}

__device__ __forceinline__ bool token_counts(const Seqs& q, int64_t i, int64_t p) {
  if (!q.mask) return true;
  const int64_t o = p + i * q.mask_skip;
  if (q.mask_labels) return __ldg(static_cast<const long long*>(q.mask) + o) != q.ignore_index;
  return __ldg(static_cast<const unsigned char*>(q.mask) + o) != 0;
}

__device__ __forceinline__ float load_f(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p)))
                         << 16);
}
__device__ __forceinline__ float load_f(const __half* p) { return __half2float(__ldg(p)); }
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_f(__half* p, float v) { *p = __float2half_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Sums of NF floats and NI counts over the block, in a fixed order; valid in thread 0.
template <int NF, int NI>
__device__ __forceinline__ void block_sums(float (&f)[NF], int (&c)[NI]) {
  __shared__ float sf[NF][kSeqWarps];
  __shared__ int sc[NI][kSeqWarps];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < NF; ++k) f[k] = warp_sum(f[k]);
#pragma unroll
  for (int k = 0; k < NI; ++k) c[k] = __reduce_add_sync(~0u, c[k]);
  __syncthreads();  // the previous sums have been read
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < NF; ++k) sf[k][w] = f[k];
#pragma unroll
    for (int k = 0; k < NI; ++k) sc[k][w] = c[k];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int k = 0; k < NF; ++k) {
      f[k] = 0.0f;
      for (int j = 0; j < kSeqWarps; ++j) f[k] += sf[k][j];
    }
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      c[k] = 0;
      for (int j = 0; j < kSeqWarps; ++j) c[k] += sc[k][j];
    }
  }
}

template <typename T>
__device__ __forceinline__ T block_total(T v) {
  __shared__ T s[kSeqWarps];
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  T t = 0;
  for (int j = 0; j < kSeqWarps; ++j) t += s[j];
  return t;
}

// Everything written by any block before is visible to every block after.  A grid of
// one block is launched plainly, larger ones cooperatively.
__device__ __forceinline__ void grid_barrier() {
  if (gridDim.x == 1)
    __syncthreads();
  else
    cooperative_groups::this_grid().sync();
}

// Whether cu is in order and inside the axis (block-wide).
__device__ __forceinline__ bool seqs_ok(const Seqs& q) {
  int bad = 0;
  if (q.cu)
    for (int64_t i = threadIdx.x; i < q.B; i += kSeqThreads) {
      const int64_t a = q.cu64 ? __ldg(static_cast<const long long*>(q.cu) + i)
                               : __ldg(static_cast<const int*>(q.cu) + i);
      const int64_t b = q.cu64 ? __ldg(static_cast<const long long*>(q.cu) + i + 1)
                               : __ldg(static_cast<const int*>(q.cu) + i + 1);
      bad |= a < 0 || b < a || b > q.total;
    }
  return __syncthreads_or(bad) == 0;
}

// exp(x) - 1 - x for |x| <= 20: near 0 the series x^2 (1/2! + x/3! + x^2/4! + ...), whose
// terms do not cancel (the difference itself would leave nothing of a small x^2 / 2).
__device__ __forceinline__ float exp_m1_mx(float x) {
  if (fabsf(x) < 0.5f) {
    float s = 1.0f / 3628800.0f;
    s = fmaf(s, x, 1.0f / 362880.0f);
    s = fmaf(s, x, 1.0f / 40320.0f);
    s = fmaf(s, x, 1.0f / 5040.0f);
    s = fmaf(s, x, 1.0f / 720.0f);
    s = fmaf(s, x, 1.0f / 120.0f);
    s = fmaf(s, x, 1.0f / 24.0f);
    s = fmaf(s, x, 1.0f / 6.0f);
    s = fmaf(s, x, 0.5f);
    return x * x * s;
  }
  return expf(x) - 1.0f - x;
}

// Host: the layout of an entry point's arguments; FLCE_OK or the refusal.
inline int make_seqs(const flce_seqs* a, Seqs* q) {
  if (a->B < 0 || a->S < 0) return FLCE_ERR_BAD_SHAPE;
  const int64_t lim = (int64_t(1) << 31) - 1;
  if (a->B > lim || a->S > (int64_t(1) << 40)) return FLCE_ERR_BAD_SHAPE;
  if (a->dtype < FLCE_F32 || a->dtype > FLCE_F16) return FLCE_ERR_BAD_ARG;
  if (a->cu_kind < 0 || a->cu_kind > 2 || a->mask_kind < 0 || a->mask_kind > 2)
    return FLCE_ERR_BAD_ARG;
  if (a->cu_kind == 0 && a->B > 0 && a->S > (int64_t(1) << 40) / a->B) return FLCE_ERR_BAD_SHAPE;
  if ((a->cu_kind != 0) != (a->cu_seqlens != nullptr)) return FLCE_ERR_BAD_ARG;
  if ((a->mask_kind != 0) != (a->mask != nullptr)) return FLCE_ERR_BAD_ARG;
  const uintptr_t cu = reinterpret_cast<uintptr_t>(a->cu_seqlens);
  if (cu & (a->cu_kind == 2 ? 7 : 3)) return FLCE_ERR_ALIGN;
  if (a->mask_kind == 2 && (reinterpret_cast<uintptr_t>(a->mask) & 7)) return FLCE_ERR_ALIGN;
  q->B = a->B;
  q->S = a->S;
  q->total = a->cu_kind ? a->S : a->B * a->S;
  q->cu = a->cu_seqlens;
  q->cu64 = a->cu_kind == 2;
  q->mask = a->mask;
  q->mask_labels = a->mask_kind == 2;
  q->ignore_index = a->ignore_index;
  q->mask_skip = a->cu_kind ? 0 : a->ld_mask - a->S;
  return FLCE_OK;
}

inline int seq_elem_bytes(int dtype) { return dtype == FLCE_F32 ? 4 : 2; }

// Plain for one block, cooperative (all blocks resident, as the barrier needs) otherwise.
template <typename Args>
inline cudaError_t launch_seq(void (*kernel)(Args), const Args& args, int64_t blocks,
                              cudaStream_t st) {
  Args a = args;
  void* params[] = {&a};
  const dim3 grid(static_cast<unsigned>(blocks)), block(kSeqThreads);
  return blocks == 1 ? cudaLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, params, 0, st)
                     : cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kernel), grid,
                                                   block, params, 0, st);
}

}  // namespace flce
