// Tokens in sequences: the layouts of the losses over sequences of tokens (the policy
// and preference losses) and the parts their kernels share.
//
// A batch is padded, [B, S] with a row stride per array, or packed, S tokens of which
// sequence i owns [cu[i], cu[i + 1]).  Both are one axis of positions: sequence i of a
// padded batch starts at position i * S, and an array's element for position p of
// sequence i is base[p + i * skip] with skip = row stride - S (0 when packed).
//
// The axis is cut into pieces of at most kTile positions, none of which holds tokens of
// two sequences; a warp takes a piece.  A padded row has ceil(S / kTile) of them.  A packed
// axis is cut at every multiple of kTile and at every sequence's start, which needs no
// list: the piece of sequence i in tile j has number i + j (each new piece moves on to the
// next tile or to the next sequence), so the first piece of sequence i is
// f(i) = start(i) / kTile + i, which rises strictly, and piece u belongs to the last i with
// f(i) <= u.  The numbers that no piece has (a sequence that ends at a cut) are empty
// pieces.  The tokens of one long sequence are spread over the GPU as well as those of many,
// and nothing about their lengths is read on the host.  What a piece costs beside its tokens (a
// search of cu, the sums) is not: 100000 sequences of 10 tokens take the policy loss 585 us, as
// many tokens in 256 sequences 23.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/flce.h"
#include "flce_device.cuh"

namespace flce {

constexpr int kSeqThreads = 1024;  // one block per SM, 64 registers: few blocks to meet
constexpr int kSeqWarps = kSeqThreads / 32;
constexpr int kVec = 4;             // a lane's consecutive tokens
constexpr int kGroup4 = 32 * kVec;  // a warp's
constexpr int kGroups = 2;
constexpr int kTile = kGroups * kGroup4;
constexpr int kClusterBlocks = 8;   // the portable cluster size
// Piece numbers are 32-bit, and a loop over them looks one step past the last: a step is a
// grid's warps at most (or a block's threads, which are fewer).
constexpr int kMaxBlocks = 1024;
constexpr int64_t kMaxPieces = (int64_t(1) << 31) - 1 - int64_t(kMaxBlocks) * kSeqWarps;
static_assert(kMaxBlocks * kSeqWarps >= kSeqThreads, "the longest step");

// How the blocks of a grid meet between the phases of a kernel.
enum : int { MEET_BLOCK = 0, MEET_CLUSTER = 1, MEET_GRID = 2 };

struct Seqs {
  int64_t B, S, total;  // total: positions (B * S padded, S packed)
  const void* cu;       // NULL: padded
  int cu64;
  const void* mask;     // NULL: every token counts
  int mask_labels;      // 0: bytes, non-zero counts; 1: int64 labels != ignore_index
  int64_t ignore_index;
  int64_t mask_skip;
  int per_row;          // pieces of a padded row
  int pieces;
  int meet;
  int kept;             // pieces per warp that shared memory holds values of
  unsigned int awaited; // sequences (pairs) that the second meeting waits for
};

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) {
  return x < lo ? lo : (x > hi ? hi : x);
}

// What a packed batch says of the start of sequence i.
__device__ __forceinline__ int64_t raw_start(const Seqs& q, int64_t i) {
  return q.cu64 ? __ldg(static_cast<const long long*>(q.cu) + i)
                : __ldg(static_cast<const int*>(q.cu) + i);
}

// Start of sequence i (i = B: the end of the last), inside [0, total] whatever the
// array holds, so that no offset built from it leaves the arrays.
__device__ __forceinline__ int64_t seq_start(const Seqs& q, int64_t i) {
  return q.cu ? clamp64(raw_start(q, i), 0, q.total) : i * q.S;
}

// The pieces of sequence i: [first, last), the empty ones left out of a packed axis.  False
// where its offsets are out of order or outside the axis: pieces may then cover a token twice
// or not at all, and no result is to be had.
__device__ __forceinline__ bool seq_pieces(const Seqs& q, int64_t i, int& first, int& last) {
  if (!q.cu) {
    first = static_cast<int>(i) * q.per_row;
    last = first + q.per_row;
    return true;
  }
  const int64_t a = seq_start(q, i), b = seq_start(q, i + 1);
  first = static_cast<int>(a / kTile + i);
  last = b > a ? static_cast<int>((b - 1) / kTile + i + 1) : first;
  return a <= b && a == raw_start(q, i) && b == raw_start(q, i + 1);
}

struct Piece {
  int seq;
  int len;        // 0: empty
  int64_t begin;  // position
};

// The piece with number u; called by a whole warp (a search over cu takes one load by all
// lanes per 32-fold narrowing).
__device__ __forceinline__ Piece find_piece(const Seqs& q, int u) {
  Piece p{-1, 0, 0};
  if (!q.cu) {
    p.seq = static_cast<int>(static_cast<unsigned>(u) / static_cast<unsigned>(q.per_row));
    const int64_t off = int64_t(u - p.seq * q.per_row) * kTile;
    p.begin = p.seq * q.S + off;
    const int64_t left = q.S - off;
    p.len = static_cast<int>(left < kTile ? left : kTile);
    return p;
  }
  int lo = 0, n = static_cast<int>(q.B);  // the answer is in [lo - 1, lo + n)
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int64_t k = int64_t(threadIdx.x & 31) * step;
    const int below =
        __popc(__ballot_sync(~0u, k < n && seq_start(q, lo + k) / kTile + lo + k <= u));
    if (below == 0) break;
    const int from = (below - 1) * step;
    const int left = n - from;
    lo += from + 1;
    n = (left < step ? left : step) - 1;
  }
  p.seq = lo - 1;
  if (p.seq < 0) return p;
  const int64_t a = seq_start(q, p.seq), b = seq_start(q, p.seq + 1);
  const int64_t tile = int64_t(u - p.seq) * kTile;
  p.begin = a > tile ? a : tile;
  const int64_t end = b < tile + kTile ? b : tile + kTile;
  p.len = end > p.begin ? static_cast<int>(end - p.begin) : 0;
  return p;
}

__device__ __forceinline__ float load_f(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p)))
                         << 16);
}
__device__ __forceinline__ float load_f(const __half* p) { return __half2float(__ldg(p)); }
// Four consecutive values: as one access where `vec` (the pointer is aligned and all four are
// inside), else those of `in`.
__device__ __forceinline__ void load4(const float* p, bool vec, unsigned int in, float (&v)[kVec]) {
  if (vec) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = in >> j & 1 ? __ldg(p + j) : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void load4(const T* p, bool vec, unsigned int in, float (&v)[kVec]) {
  static_assert(sizeof(T) == 2, "16-bit types");
  if (vec) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    const T* h = reinterpret_cast<const T*>(&x);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = static_cast<float>(h[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = in >> j & 1 ? load_f(p + j) : 0.0f;
  }
}
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_f(__half* p, float v) { *p = __float2half_rn(v); }
template <typename T>
__device__ __forceinline__ void store4(T* p, bool vec, unsigned int in, const float (&v)[kVec]) {
  if (vec) {
    struct alignas(kVec * sizeof(T)) { T x[kVec]; } o;
#pragma unroll
    for (int j = 0; j < kVec; ++j) store_f(&o.x[j], v[j]);
    *reinterpret_cast<decltype(o)*>(p) = o;
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (in >> j & 1) store_f(p + j, v[j]);
  }
}

// Whether every given array (NULL: not there) takes four values in one access.
template <typename T>
__device__ __forceinline__ uintptr_t misfit(const T* p, bool there) {
  return there ? reinterpret_cast<uintptr_t>(p) & (kVec * sizeof(T) - 1) : 0;
}

// Which of a piece's tokens count.
struct Counted {
  const void* mask;
  int labels;
  int64_t ignore_index;
  bool vec;
  __device__ __forceinline__ Counted(const Seqs& q, const Piece& p)
      : mask(nullptr), labels(q.mask_labels), ignore_index(q.ignore_index), vec(false) {
    const int64_t o = p.begin + p.seq * q.mask_skip;
    if (q.mask)
      mask = labels ? static_cast<const void*>(static_cast<const long long*>(q.mask) + o)
                    : static_cast<const void*>(static_cast<const unsigned char*>(q.mask) + o);
    // four bytes, or two pairs of labels
    vec = (reinterpret_cast<uintptr_t>(mask) & (labels ? 15 : 3)) == 0;
  }
  // Of the four tokens from t on, those of `in` that count.
  __device__ __forceinline__ unsigned int operator()(int t, unsigned int in) const {
    if (!mask) return in;
    unsigned int on = 0;
    if (labels) {
      const long long* m = static_cast<const long long*>(mask) + t;
      if (vec && in == 15u) {
        const longlong2 a = __ldg(reinterpret_cast<const longlong2*>(m));
        const longlong2 b = __ldg(reinterpret_cast<const longlong2*>(m) + 1);
        on = (a.x != ignore_index) | (a.y != ignore_index) << 1 | (b.x != ignore_index) << 2 |
             (b.y != ignore_index) << 3;
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (in >> j & 1) on |= static_cast<unsigned int>(__ldg(m + j) != ignore_index) << j;
      }
    } else {
      const unsigned char* m = static_cast<const unsigned char*>(mask) + t;
      if (vec && in == 15u) {
        const unsigned int x = __ldg(reinterpret_cast<const unsigned int*>(m));
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          on |= static_cast<unsigned int>((x >> (8 * j) & 255u) != 0) << j;
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (in >> j & 1) on |= static_cast<unsigned int>(__ldg(m + j) != 0) << j;
      }
    }
    return on;
  }
};

// Of the four tokens from t on, those inside [t0, t1).
__device__ __forceinline__ unsigned int tokens_in(int t, int t0, int t1) {
  unsigned int in = 15u;
  if (t < t0) in = t0 - t >= kVec ? 0u : in << (t0 - t) & 15u;
  if (t + kVec > t1) in &= t >= t1 ? 0u : (1u << (t1 - t)) - 1;
  return in;
}

// A sum as an unevaluated pair of floats (h + l, about 48 bits): the sums over pieces and
// sequences, whose terms have both signs.  fp64 adds run at a small fraction of the
// fp32 rate here: when the sums became pairs, the policy kernel went from 58 us at a million
// tokens to 44.
struct Pair {
  float h, l;
  __device__ __forceinline__ float value() const {
    return fabsf(h) <= 3.4028235e38f ? h + l : h;  // infinities and NaN: l means nothing
  }
};

__device__ __forceinline__ Pair operator+(Pair a, float b) {
  const float s = __fadd_rn(a.h, b);
  const float z = __fadd_rn(s, -a.h);
  const float e = __fadd_rn(__fadd_rn(a.h, -__fadd_rn(s, -z)), __fadd_rn(b, -z));
  return {s, __fadd_rn(a.l, e)};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  Pair s = a + b.h;
  s.l = __fadd_rn(s.l, b.l);
  return s;
}
__device__ __forceinline__ Pair operator-(Pair a) { return {-a.h, -a.l}; }
__device__ __forceinline__ Pair operator*(Pair a, float s) {
  const float x = __fmul_rn(a.h, s);
  return {x, fmaf(a.h, s, -x) + a.l * s};
}
// The quotient, and the quotient of what it leaves.
__device__ __forceinline__ Pair operator/(Pair a, float s) {
  const float x = a.value() / s;
  return {x, fabsf(x) <= 3.4028235e38f ? (fmaf(-x, s, a.h) + a.l) / s : 0.0f};
}

// Sums over a warp or a block.  Their loops stay rolled: a launch finds the instruction
// caches cold, and with every SM fetching the same lines at once straight-line code cost
// some 60 cycles an instruction (when these loops were rolled, the sums' unrolled forms took 40000
// of the policy kernel's 88000 cycles at a million tokens).
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(~0u, v[k], o);
  }
}

// Pairs and floats in one loop.
template <int N, int M>
__device__ __forceinline__ void warp_sums(Pair (&p)[N], float (&v)[M]) {
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      p[k] = p[k] + Pair{__shfl_xor_sync(~0u, p[k].h, o), __shfl_xor_sync(~0u, p[k].l, o)};
#pragma unroll
    for (int k = 0; k < M; ++k) v[k] += __shfl_xor_sync(~0u, v[k], o);
  }
}

template <int N>
__device__ __forceinline__ void warp_sums(Pair (&v)[N]) {
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      v[k] = v[k] + Pair{__shfl_xor_sync(~0u, v[k].h, o), __shfl_xor_sync(~0u, v[k].l, o)};
  }
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(~0u, v); }

// 0 <= v < 2^38, as its low 20 and its other bits.
__device__ __forceinline__ long long warp_sum(long long v) {
  const int lo = __reduce_add_sync(~0u, static_cast<int>(v & 0xfffff));
  const int hi = __reduce_add_sync(~0u, static_cast<int>(v >> 20));
  return (static_cast<long long>(hi) << 20) + lo;
}

// In a fixed order, valid in warp 0; only the threads below `used` hold values.
template <int N>
__device__ __forceinline__ void block_sums(Pair (&v)[N], int64_t used) {
  __shared__ Pair s[kSeqWarps][N];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int busy = used < kSeqThreads ? static_cast<int>(used + 31) / 32 : kSeqWarps;
#pragma unroll 1
  for (int stage = 0; stage < 2; ++stage) {
    if (w < busy) warp_sums(v);
    if (stage == 1) break;
    if (lane == 0 && w < busy) {
#pragma unroll
      for (int k = 0; k < N; ++k) s[w][k] = v[k];
    }
    __syncthreads();
    if (w > 0) break;
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = lane < busy ? s[lane][k] : Pair{0.0f, 0.0f};
  }
}

// Sums of non-negative whole numbers below 2^38, the same in any order, in every thread.
// Two calls have a barrier between them.  (32-bit halves: a 64-bit atomic in shared memory is a loop.)
template <int N>
__device__ __forceinline__ void block_counts(long long (&c)[N]) {
  __shared__ unsigned int s[2][N];
  if (threadIdx.x < 2 * N) s[threadIdx.x / N][threadIdx.x % N] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const unsigned int lo = __reduce_add_sync(~0u, static_cast<unsigned int>(c[k] & 0xfffff));
    const unsigned int hi = __reduce_add_sync(~0u, static_cast<unsigned int>(c[k] >> 20));
    if ((threadIdx.x & 31) == 0 && (lo | hi)) {
      atomicAdd(&s[0][k], lo);
      atomicAdd(&s[1][k], hi);
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) c[k] = (static_cast<long long>(s[1][k]) << 20) + s[0][k];
}

// Everything written by any block before is visible to every block after.
__device__ __forceinline__ void meet(int how) {
  if (how == MEET_GRID)
    cooperative_groups::this_grid().sync();
  else if (how == MEET_CLUSTER)
    cooperative_groups::this_cluster().sync();
  else
    __syncthreads();
}

// How the sums of `items` sequences (or pairs) are shared out: a warp each, or, where there
// are few and long ones, a block each.  The policy loss of one sequence of a million tokens
// takes 27 us with a block and 64 with a warp, of four such 64 and 102; the preference loss of a
// pair of 16384 tokens each, whose 128 pieces a warp goes through four times, 11.9 with a block
// and 11.2 with a warp.  The rule looks at the average length: a sequence of a million tokens
// beside 60 of 100 is a warp's, 66 us where a block would take 27.
struct SeqShare {
  bool wide;
  int64_t first, stride;
  int offset, step;  // of this thread in an item's pieces
  __device__ __forceinline__ SeqShare(const Seqs& q, int64_t items)
      : wide(items <= gridDim.x && q.pieces / 256 > items),
        first(wide ? blockIdx.x : blockIdx.x * kSeqWarps + (threadIdx.x >> 5)),
        stride(wide ? gridDim.x : int64_t(gridDim.x) * kSeqWarps),
        offset(wide ? threadIdx.x : threadIdx.x & 31),
        step(wide ? kSeqThreads : 32) {}
  // Whether this thread writes the item's results, and whether its warp counts it.
  __device__ __forceinline__ bool writes() const { return offset == 0; }
  __device__ __forceinline__ bool counts() const { return !wide || threadIdx.x < 32; }
  // The item's sums; valid in the warp that counts it.
  template <int N, int M>
  __device__ __forceinline__ void sum(Pair (&f)[N], long long (&c)[M]) const {
    if (wide) {
      block_sums(f, kSeqThreads);
      block_counts(c);
    } else {
      warp_sums(f);
#pragma unroll
      for (int k = 0; k < M; ++k) c[k] = warp_sum(c[k]);
    }
  }
};

// What the sequences add up to: whole numbers, the same in any order.  Cleared before the
// first meeting.
struct SeqTotals {
  unsigned long long tokens;  // counted tokens
  unsigned int live;          // sequences (pairs) that count, and kBadSeqs
  unsigned int done;          // sequences (pairs) summed up
};
// Whether the offsets of a sequence are out of order or out of range: in a word that is read
// anyway (a load of its own after the second meeting takes the losses 0.5 us).
constexpr unsigned int kBadSeqs = 1u << 31;

// The second meeting, by a warp that has summed up `mine` sequences.  Most blocks of a grid
// have nothing left to do there: polled at full speed by all of them, the barrier's word kept
// its part of L2 from the few that still read (their sums took 15000 cycles instead of
// 1700).  So a grid's blocks wait for the count of finished sequences, and sleep between
// looks.  A wait ends after 2 s at the latest, with the time-out bit set; true (in the whole
// block) says so: the totals are not to be trusted then.
__device__ __forceinline__ bool meet_sequences(const Seqs& q, SeqTotals* t,
                                               unsigned long long tokens, unsigned int live,
                                               unsigned int mine, uint32_t* err) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0 && mine > 0) {
    if (tokens) atomicAdd(&t->tokens, tokens);
    if (live) atomicAdd(&t->live, live);
    if (q.meet == MEET_GRID) {
      __threadfence();
      atomicAdd(&t->done, mine);
    }
  }
  if (q.meet != MEET_GRID) {
    meet(q.meet);
    return false;
  }
  int late = 0;
  if (threadIdx.x == 0) {
    const uint64_t t0 = global_timer_ns();
    unsigned int n;
    while (true) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(&t->done) : "memory");
      if (n >= q.awaited) break;
      if (global_timer_ns() - t0 > FLCE_WAIT_LIMIT_NS) {
        atomicOr(err, FLCE_DEVERR_TIMEOUT);
        late = 1;
        break;
      }
      __nanosleep(100);
    }
  }
  return __syncthreads_or(late) != 0;
}

// exp(x) - 1 - x given e = exp(x), |x| <= 20: near 0 the series x^2 (1/2! + x/3! + x^2/4! +
// ...), whose terms do not cancel (the difference would leave nothing of a small x^2 / 2).
__device__ __forceinline__ float exp_m1_mx(float x, float e) {
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
  return e - 1.0f - x;
}

// Host: the layout of an entry point's arguments; FLCE_OK or the refusal.
inline int make_seqs(const flce_seqs* a, Seqs* q) {
  if (a->B < 0 || a->S < 0) return FLCE_ERR_BAD_SHAPE;
  const int64_t lim = (int64_t(1) << 31) - 1;
  if (a->B > lim || a->S > (int64_t(1) << 38)) return FLCE_ERR_BAD_SHAPE;
  if (a->dtype < FLCE_F32 || a->dtype > FLCE_F16) return FLCE_ERR_BAD_ARG;
  if (a->ld_mask < 0 || a->cu_kind < 0 || a->cu_kind > 2 || a->mask_kind < 0 || a->mask_kind > 2)
    return FLCE_ERR_BAD_ARG;
  if (a->cu_kind == 0 && a->B > 0 && a->S > (int64_t(1) << 38) / a->B) return FLCE_ERR_BAD_SHAPE;
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
  const int64_t per_row = a->S > 0 ? (a->S + kTile - 1) / kTile : 1;
  const int64_t pieces = a->cu_kind ? q->total / kTile + q->B + 1 : q->B * per_row;
  if (pieces > kMaxPieces) return FLCE_ERR_BAD_SHAPE;
  q->per_row = a->cu_kind ? 0 : static_cast<int>(per_row);
  q->pieces = static_cast<int>(pieces);
  q->awaited = static_cast<unsigned int>(a->B);
  return FLCE_OK;
}

inline int seq_elem_bytes(int dtype) { return dtype == FLCE_F32 ? 4 : 2; }

// A grid whose blocks meet: plain for one block, one cluster (of 2, 4 or 8 blocks), or
// cooperative.
inline cudaError_t launch_meeting(const void* kernel, void* args, int64_t blocks, int threads,
                                  int meet, cudaStream_t st, int smem = 0) {
  void* params[] = {args};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  if (meet == MEET_CLUSTER) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cfg.gridDim.x;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  } else {
    attr.id = cudaLaunchAttributeCooperative;
    attr.val.cooperative = 1;
  }
  cfg.attrs = &attr;
  cfg.numAttrs = meet == MEET_BLOCK ? 0 : 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, params);
  if (e != cudaSuccess) cudaGetLastError();  // reported here, not by a later call
  return e;
}

// A warp per piece: one block where its warps suffice, else a cluster of at most eight
// (whose hardware barrier is faster: the policy loss of 16 x 1024 tokens takes 20.0 us with
// a cluster and 20.9 with a grid, of 64 x 1024 21.2 and 22.2), else a cooperative grid of at
// most one block per SM, whose warps take several pieces each.
// `kept` bytes of dynamic shared memory per warp's piece, for at most kKept of them (the
// policy loss of 4 x 1M tokens takes 64 us with four pieces kept and 82 with one).
constexpr int kKept = 4;

template <typename Args>
inline cudaError_t launch_seq(void (*kernel)(Args), const Args& args, int kept, int sms,
                              cudaStream_t st) {
  Args a = args;
  int64_t blocks = (int64_t(a.q.pieces) + kSeqWarps - 1) / kSeqWarps;
  if (blocks < 1) blocks = 1;
  a.q.meet = blocks == 1 ? MEET_BLOCK : blocks <= kClusterBlocks ? MEET_CLUSTER : MEET_GRID;
  if (a.q.meet == MEET_CLUSTER) blocks = blocks <= 2 ? 2 : blocks <= 4 ? 4 : 8;
  if (blocks > sms) blocks = sms;
  if (blocks > kMaxBlocks) blocks = kMaxBlocks;
  const int64_t rounds = (a.q.pieces + blocks * kSeqWarps - 1) / (blocks * kSeqWarps);
  a.q.kept = static_cast<int>(rounds < kKept ? rounds : kKept);
  const int smem = kept * kSeqWarps * a.q.kept;
  const void* k = reinterpret_cast<const void*>(kernel);
  if (smem > 40 * 1024) {  // more than the default, beside the kernel's static arrays
    // the most that any launch takes, not this one's: the limit is the kernel's own, and
    // another thread may set it between here and the launch
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kept * kSeqWarps * kKept);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return e;
    }
  }
  return launch_meeting(k, &a, blocks, kSeqThreads, a.q.meet, st, smem);
}

}  // namespace flce
