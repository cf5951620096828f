// Rows of logits as a sampler sees them, their logsumexp, the log-probability of a label and
// the entropy under them, and the gradient by the logits.
//
//   z = (seen ? (l > 0 ? l / rp : l rp) : l) - fp n - pp [n > 0] + (sum of the biases on it)
//   z = -inf where not allowed;  z = z / T
//
// (the divisions are multiplications by the rounded reciprocals, a rounding of fp32 more)
// n counts a token among the row's generated tokens, seen says whether it is among prompt or
// generated ones.  One pass over the logits, so bound by their bytes, in and out.
//
// A row is shared by a cluster of blocks, each with a run of columns and a counter per column in its
// shared memory.  Each block reads all of the row's tokens, which come from L2, and counts those of
// its own columns.  384 x 256000 in bf16 after up to 8192 tokens each: 148 us, 2.7 TB/s; without a
// history and statistics 62 us, 6.3 TB/s.  A block lives for some 10 us, of which its 20 to 40 KB of logits
// need 2 to 5 at the memory's rate; what goes on the rest is the row's parameters and lengths, its
// tokens, and the statistics' join.  (Reading each token once and adding into the other blocks' counters over
// distributed shared memory took 5 to 8 cycles of an SM per token; laying the tokens out by owner
// and fetching them, three meetings of the cluster: 384 x 256000 in bf16 after 1 and after 8192
// tokens 114 and 250 us, against 79 and 174 at the time.  A list of the changed columns, worked off by a
// thread per entry beside the pass over all logits: 87 and 240.  Sorting a row's tokens by blocks in a
// launch ahead: 192 against 195 after 8192 tokens, 205 against 190 for 700 x 152064 after 4000, and ahead
// only after tens of thousands.)  Biases only mark their columns' counters; a
// marked column adds its biases from the row's list, one by one in the list's order.
//
// The running maximum m, d = sum 2^u and s = sum 2^u u with u = log2(e) (z - m) stay in registers, are
// joined in the block and then in the cluster, in a fixed order:  lse = m + ln d,
// H = ln d - ln 2 s / d.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "flce_device.cuh"
#include "flce_host.h"

namespace flce {
namespace logits {

// 256 threads and 64 KB (three blocks per SM): 512 threads took 204 us where 256 took 173 (384 x 256000
// in bf16 after up to 8192 tokens each), 128 threads and half the memory 189; four blocks of 48 KB 150
// where three take 148 (700 x 152064 with masks, both directions, 360 against 330).
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocks = 3;           // per SM
constexpr int kFill = 6;             // blocks per SM that a row's are multiplied up to (12: 200 us, 4: 206)
constexpr int kMaxCluster = 16;
constexpr int kStage = 16384;        // bytes of logits per copy into shared memory, two on their way
constexpr int kRoom = 32768;         // bytes of counters
constexpr int kDeep = 2;             // 16-byte words of tokens on their way per thread
constexpr int kMaxBias = 2048;       // entries of a row's list: 16 KB of shared memory

// Counters: occurrences among the generated tokens, and flags of the prompt's tokens and of
// columns with a bias.  16 bits hold the count of histories below 2^14 tokens.
struct NoCounter {
  using Word = uint16_t;
  static constexpr uint32_t kSeen = 0, kBiased = 0, kCount = 0;
};
template <typename W>
struct Counter {
  using Word = W;
  static constexpr int kBits = sizeof(W) * 8;
  static constexpr uint32_t kSeen = 1u << (kBits - 1), kBiased = 1u << (kBits - 2),
                            kCount = kBiased - 1;
};

struct Args {
  const void* logits;
  void* out;  // MODE_FORWARD: processed logits (NULL: none); MODE_BACKWARD: dlogits
  int64_t R, V, ld, ld_out;
  const void* tokens;
  int64_t T, ld_tokens;
  const void* prompt_lens;
  const void* lengths;
  const float* rep;
  const float* freq;
  const float* pres;
  const float* temp;
  float rep1, freq1, pres1, temp1;  // without an array
  const void* bias_ids;
  const float* bias_values;
  int64_t n_bias, ld_bias_ids, ld_bias_values;
  const void* allowed;
  int64_t ld_allowed;
  const int64_t* labels;
  int64_t ignore_index;
  float* lse;  // [R], or with `split` [2, R]: what its rounding left off behind it
  float* logp;
  float* entropy;
  const float* g_logp;
  const float* g_entropy;
  uint32_t* err;
  int64_t columns, room;  // per block, and of them at a time (whole vectors)
  int32_t passes, stage_bytes;
  int32_t ids64, lens64, bias64, mask_kind, out_f32, stats, split;
};

// PROCESS: z, with or without lse.  FORWARD: whatever is asked for.
enum { MODE_FORWARD = 0, MODE_BACKWARD = 1, MODE_PROCESS = 2 };

// (one per source: what a source has set up for its kernels is not shared with another build of them in
// the same process)
namespace {

// The 4 or 8 values of 16 bytes.
template <typename T>
__device__ __forceinline__ void widen(const uint4& q, float (&x)[16 / sizeof(T)]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same_v<T, float>) {
      x[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 narrow(const float (&x)[16 / sizeof(T)]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same_v<T, float>) {
      w[i] = __float_as_uint(x[i]);
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ float widen1(T x) {
  if constexpr (std::is_same_v<T, float>) return x;
  else if constexpr (std::is_same_v<T, __nv_bfloat16>) return __bfloat162float(x);
  else return __half2float(x);
}
template <typename T>
__device__ __forceinline__ T narrow1(float x) {
  if constexpr (std::is_same_v<T, float>) return x;
  else if constexpr (std::is_same_v<T, __nv_bfloat16>) return __float2bfloat16_rn(x);
  else return __float2half_rn(x);
}

__device__ __forceinline__ int64_t whole(const void* p, int64_t i, int is64) {
  return is64 ? __ldg(static_cast<const long long*>(p) + i)
              : static_cast<int64_t>(__ldg(static_cast<const int*>(p) + i));
}

// Statistics of a part of a row: m the largest z, d and s as above (m = -inf: nothing).
struct Stats {
  float m, d, s;
};

// The join of lanes 0 to n - 1 (a power of two; the others' are not looked at by them), in every one
// of them: first the largest m, then sums in its units.
__device__ __forceinline__ Stats join_warp(Stats x, int n) {
  float m = x.m;
  for (int j = n / 2; j > 0; j >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, j));
  if (m != -INFINITY) {
    const float t = x.m == -INFINITY ? 0.0f : (x.m - m) * kLog2e;
    const float e = fast_ex2(t);
    x.s = e != 0.0f ? e * fmaf(t, x.d, x.s) : 0.0f;
    x.d *= e;
  }
  for (int j = n / 2; j > 0; j >>= 1) {
    x.d += __shfl_xor_sync(0xffffffffu, x.d, j);
    x.s += __shfl_xor_sync(0xffffffffu, x.s, j);
  }
  return Stats{m, x.d, x.s};
}
__device__ __forceinline__ void st_remote(uint32_t a, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// The cluster's barrier in two halves (every thread of every block, in warps).
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One more (FLAG: seen) at the counter of column `at` where there is one and the id's upper half,
// `high`, is 0; without a branch, as some
// lane of a warp nearly always has a column here.
template <typename COUNTER, bool FLAG>
__device__ __forceinline__ void bump(uint32_t at, uint32_t high, uint32_t columns, uint32_t counters) {
  constexpr bool WIDE = sizeof(typename COUNTER::Word) == 4;
  const uint32_t to = counters + (WIDE ? at * 4 : (at * 2 & ~3u));
  const uint32_t one = FLAG ? COUNTER::kSeen : 1u;
  // (the funnel shift takes its distance modulo 32: 16 for odd columns)
  const uint32_t value = WIDE ? one : __funnelshift_l(0u, one, at << 4);
  if (FLAG)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.lt.u32 p, %0, %1;\n\tsetp.eq.and.u32 p, %4, 0, p;\n\t"
        "@p red.shared::cta.or.b32 [%2], %3;\n\t}" ::"r"(at), "r"(columns), "r"(to), "r"(value), "r"(high)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.lt.u32 p, %0, %1;\n\tsetp.eq.and.u32 p, %4, 0, p;\n\t"
        "@p red.shared::cta.add.u32 [%2], %3;\n\t}" ::"r"(at), "r"(columns), "r"(to), "r"(value), "r"(high)
        : "memory");
}

// Counts tokens [t0, t1) of a row that fall on the `columns` columns from id `first` on (FLAG: marks
// them as seen), 16 bytes of tokens at a time, the next ones asked for ahead.  The counter of an id
// outside the row is never looked at.
template <typename COUNTER, bool FLAG, typename ID>
__device__ __forceinline__ void count(const ID* tokens, int t0, int t1, int first, uint32_t columns,
                                      uint32_t counters) {
  constexpr int kIds = 16 / sizeof(ID);
  const uint32_t none = 0xffffffffu;  // no column
  auto add = [&](const uint4& q) {
    if constexpr (sizeof(ID) == 8) {
      bump<COUNTER, FLAG>(q.x - first, q.y, columns, counters);
      bump<COUNTER, FLAG>(q.z - first, q.w, columns, counters);
    } else {
      bump<COUNTER, FLAG>(q.x - first, 0u, columns, counters);
      bump<COUNTER, FLAG>(q.y - first, 0u, columns, counters);
      bump<COUNTER, FLAG>(q.z - first, 0u, columns, counters);
      bump<COUNTER, FLAG>(q.w - first, 0u, columns, counters);
    }
  };
  if (t1 <= t0) return;
  // whole 16-byte words from a to b, a few tokens before and behind them
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(tokens + t0) & 15) / sizeof(ID));
  const int a = min(skew ? t0 + kIds - skew : t0, t1), words = (t1 - a) / kIds, b = a + words * kIds;
  const int tid = threadIdx.x;
  if (tid < 2 * kIds) {
    const int t = tid < kIds ? t0 + tid : b + tid - kIds;
    if (tid < kIds ? t < a : t < t1) {
      const int64_t id = tokens[t];
      bump<COUNTER, FLAG>(static_cast<uint32_t>(id) - first, static_cast<uint32_t>(id >> 32), columns,
                          counters);
    }
  }
  const uint4* from = reinterpret_cast<const uint4*>(tokens + a);
  const uint4 nothing = make_uint4(none, none, none, none);
  uint4 next[kDeep];
#pragma unroll
  for (int j = 0; j < kDeep; ++j)
    next[j] = tid + j * kThreads < words ? __ldg(from + tid + j * kThreads) : nothing;
#pragma unroll 1
  for (int i = 0; i < words; i += kDeep * kThreads) {
    uint4 q[kDeep];
#pragma unroll
    for (int j = 0; j < kDeep; ++j) q[j] = next[j];
    const int n = i + kDeep * kThreads + tid;
#pragma unroll
    for (int j = 0; j < kDeep; ++j)
      next[j] = n + j * kThreads < words ? __ldg(from + n + j * kThreads) : nothing;
#pragma unroll
    for (int j = 0; j < kDeep; ++j) add(q[j]);
  }
}

// Four mask bytes as bits: bit i set where byte i is not 0.
__device__ __forceinline__ uint32_t byte_bits(uint32_t w) {
  // bit 0 of each byte that is not 0, then the four of them side by side
  const uint32_t t = ((((w & 0x7f7f7f7fu) + 0x7f7f7f7fu) | w) >> 7) & 0x01010101u;
  return (t * 0x01020408u) >> 24 & 15u;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Counters i and i + 1 of those in words n32: what marks a column as seen, and the count.
template <typename COUNTER>
__device__ __forceinline__ void split_counter(const uint32_t* n32, int i, uint32_t& seen0, uint32_t& seen1,
                                              float& count0, float& count1) {
  constexpr uint32_t kMark = COUNTER::kSeen | COUNTER::kCount;
  if constexpr (sizeof(typename COUNTER::Word) == 2) {
    const uint32_t w = n32[i / 2], n = w & (COUNTER::kCount | COUNTER::kCount << 16);
    seen0 = w & kMark;
    seen1 = w & kMark << 16;
    // below 2^23 a whole number is the end of a float of that exponent: no conversion
    f2_unpack(f2_add(f2_pack(__uint_as_float(__byte_perm(n, 0x4B00, 0x5410)),
                             __uint_as_float(__byte_perm(n, 0x4B00, 0x5432))),
                     f2_pack(-8388608.0f, -8388608.0f)),
              count0, count1);
  } else {
    seen0 = n32[i] & kMark;
    seen1 = n32[i + 1] & kMark;
    count0 = static_cast<float>(n32[i] & COUNTER::kCount);
    count1 = static_cast<float>(n32[i + 1] & COUNTER::kCount);
  }
}

// Zeros for logits [l0, l1) of an output row.
template <typename T>
__device__ __forceinline__ void zero_columns(const Args& a, uint8_t* out, int l0, int l1) {
  const int bytes = a.out_f32 ? 4 : sizeof(T);
  uint8_t* p = out + static_cast<int64_t>(max(l0, 0)) * bytes;
  uint8_t* end = out + static_cast<int64_t>(l1) * bytes;
  uint8_t* first = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 15) & ~uintptr_t(15));
  if (first > end) first = end;
  uint8_t* last = first + (end - first) / 16 * 16;
  const int tid = threadIdx.x;
  for (uint8_t* q = first + tid * 16; q < last; q += kThreads * 16)
    __stcs(reinterpret_cast<uint4*>(q), make_uint4(0, 0, 0, 0));
  if (tid < 8 && p + tid * 2 < first) *reinterpret_cast<uint16_t*>(p + tid * 2) = 0;
  if (tid < 8 && last + tid * 2 < end) *reinterpret_cast<uint16_t*>(last + tid * 2) = 0;
}

// What all of a block needs to know of its row, found out by one thread.
struct RowArgs {
  float rep, inv_rep, freq, pres, inv_temp;
  float lse, low, g, h, ent;  // the gradient: -p (g + h (ln p + H)) + g [label], ln p = (z - lse) - low
  int label, length, prompt;
  int ignored, bad, zero;    // zero: a gradient of zeros
};

template <bool COUNT, bool BACKWARD>
__device__ __forceinline__ void read_row(const Args& a, int64_t row, RowArgs& r) {
  const int64_t y = a.labels ? a.labels[row] : -1;
  const float temp = a.temp ? a.temp[row] : a.temp1;
  if (COUNT) {
    r.rep = a.rep ? a.rep[row] : a.rep1;
    r.freq = a.freq ? a.freq[row] : a.freq1;
    r.pres = a.pres ? a.pres[row] : a.pres1;
    const int64_t n = !a.tokens ? 0 : a.lengths ? whole(a.lengths, row, a.lens64) : a.T;
    const int64_t q = a.prompt_lens ? whole(a.prompt_lens, row, a.lens64) : 0;
    r.inv_rep = __fdiv_rn(1.0f, r.rep);
    r.length = static_cast<int>(n < 0 ? 0 : n < a.T ? n : a.T);
    if (r.rep == 1.0f && r.freq == 0.0f && r.pres == 0.0f) r.length = 0;
    r.prompt = static_cast<int>(q < 0 ? 0 : q < r.length ? q : r.length);
  }
  r.ignored = a.labels && y == a.ignore_index;
  r.label = y >= 0 && y < a.V ? static_cast<int>(y) : -1;
  r.bad = a.labels && !r.ignored && r.label < 0;
  r.inv_temp = temp > 0.0f ? __fdiv_rn(1.0f, temp) : 1.0f;
  r.zero = 0;
  if (BACKWARD) {
    r.lse = a.lse[row];
    r.low = a.split ? a.lse[a.R + row] : 0.0f;
    r.g = a.g_logp ? a.g_logp[row] : 0.0f;
    r.h = a.g_entropy ? a.g_entropy[row] : 0.0f;
    r.ent = a.entropy ? a.entropy[row] : 0.0f;
    r.zero = r.ignored || r.lse == -INFINITY;
  }
}

// A running maximum and the sums below it, of one thread.
struct Running {
  float top = -INFINITY, d = 0.0f, s = 0.0f;

  template <int N>
  __device__ __forceinline__ void add(const float (&z)[N], bool entropy) {
    float m = z[0];
    if constexpr (N > 1) {
      m = fmaxf(z[0], z[1]);
#pragma unroll
      for (int i = 2; i + 1 < N; i += 2) m = fmax3(m, z[i], z[i + 1]);
    }
    if (m > top) {
      const float t = (top - m) * kLog2e;  // -inf before the first
      const float e = fast_ex2(t);
      s = e != 0.0f ? e * fmaf(t, d, s) : 0.0f;
      d *= e;
      top = m;
    }
    // nothing yet: -inf alone, or NaN, which makes d NaN
    const float base = top == -INFINITY ? 0.0f : top;
    if constexpr (N == 1) {
      const float u = (z[0] - base) * kLog2e, e = fast_ex2(u);
      d += e;
      s = fmaf(e, fmaxf(u, -200.0f), s);
    } else {
      const uint64_t base2 = f2_pack(-base, -base), log2 = f2_pack(kLog2e, kLog2e);
      uint64_t sum = 0, dot = 0;
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        float u0, u1;
        f2_unpack(f2_mul(f2_add(f2_pack(z[i], z[i + 1]), base2), log2), u0, u1);
        const uint64_t e = f2_pack(fast_ex2(u0), fast_ex2(u1));
        sum = f2_add(sum, e);
        if (entropy)  // 2^u is 0 below, and u may be -inf
          dot = f2_fma(e, f2_pack(fmaxf(u0, -200.0f), fmaxf(u1, -200.0f)), dot);
      }
      float a0, a1;
      f2_unpack(sum, a0, a1);
      d += a0 + a1;
      if (entropy) {
        f2_unpack(dot, a0, a1);
        s += a0 + a1;
      }
    }
  }
};

// Columns are numbered from the row's last 16-byte boundary at or before its first logit, so
// that vectors of VEC columns are aligned in every row; `pre` columns before the row are not
// there.  Column c of that numbering is logit c - pre.  A block's columns go by passes of as many
// as it has counters for, a pass by copies of kStage bytes, two on their way at a time; the vectors
// at a row's ends that are not whole are done element by element.
//
// A loop of fewer instructions is worth a kernel of its own, as the warps of three blocks, each at
// another place of it, wait for instructions a fifth of their time: with masks (MASK) and biases (BIAS)
// left in, 384 x 256000 in bf16 after up to 8192 tokens takes 195 us, without 169, and without entropies
// and labels (MODE_PROCESS) 160.
template <typename T, typename COUNTER, int MODE, bool MASK, bool BIAS>
__global__ void __launch_bounds__(kThreads, kBlocks)
    logits_kernel(const __grid_constant__ Args a) {
  constexpr int VEC = 16 / sizeof(T);
  constexpr uint32_t kAll = (1u << VEC) - 1;
  constexpr int kColumns = kStage / sizeof(T);  // per copy
  constexpr bool COUNT = !std::is_same_v<COUNTER, NoCounter>, BACKWARD = MODE == MODE_BACKWARD,
                 PROCESS = MODE == MODE_PROCESS;
  using Word = typename COUNTER::Word;
  // two copies of logits, counters, the biases' columns and values
  extern __shared__ __align__(16) uint8_t shared[];
  __shared__ uint64_t landed[2];
  __shared__ int gave_up;
  __shared__ RowArgs r;
  __shared__ Stats part[kWarps];
  __shared__ float4 from[kMaxCluster];  // each block's statistics and, if it has it, the label's z
  __shared__ float label_z;
  __shared__ uint32_t mask_bits[2][kColumns / 32];  // of two copies, a bit per column
  const uint32_t rank = cluster_ctarank(), size = cluster_size();
  const int64_t row = blockIdx.x / size;
  const int V = static_cast<int>(a.V), tid = threadIdx.x, lane = tid & 31;
  const T* x = static_cast<const T*>(a.logits) + row * a.ld;
  const int pre = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const int span = V + pre, columns = static_cast<int>(a.columns), room = static_cast<int>(a.room);
  const int n_bias = BIAS ? static_cast<int>(a.n_bias) : 0, mask_kind = MASK ? a.mask_kind : 0;
  uint8_t* counters = shared + a.stage_bytes;
  int* bias_col = reinterpret_cast<int*>(counters + (COUNT ? room * sizeof(Word) : 0));
  float* bias_val = reinterpret_cast<float*>(bias_col + n_bias);
  const uint8_t* mask = static_cast<const uint8_t*>(a.allowed) +
                        row * a.ld_allowed * (mask_kind == 2 ? 4 : 1);
  uint8_t* out = static_cast<uint8_t*>(a.out);
  if (PROCESS || out) out += row * a.ld_out * (a.out_f32 ? 4 : sizeof(T));
  const int begin = static_cast<int>(rank) * columns, end = min(begin + columns, span);
  // whole vectors of the row among the block's columns
  const int in0 = max(begin, pre ? VEC : 0), in1 = max(in0, min(end, span / VEC * VEC));
  const int copies = (in1 - in0 + kColumns - 1) / kColumns;

  auto copy = [&](int k) {  // by one thread
    const int c = in0 + k * kColumns;
    const uint32_t bytes = static_cast<uint32_t>(min(kColumns, in1 - c)) * sizeof(T);
    mbar_arrive_expect_tx(&landed[k & 1], bytes);
    bulk_load(smem_u32(shared) + (k & 1) * kStage, x + (c - pre), bytes, &landed[k & 1]);
  };
  if (tid == 0) {
    mbar_init(&landed[0], 1);
    mbar_init(&landed[1], 1);
    gave_up = 0;
    label_z = -INFINITY;
    fence_mbar_init();
    if (copies > 0) copy(0);
    if (copies > 1) copy(1);
  }
  // The mask of a copy's columns: a thread's 32 of them are asked for a copy ahead, and made bits of
  // when the copy before is done.
  static_assert(kColumns / 32 <= kThreads, "a word of mask bits per thread");
  uint32_t raw[9];
  int raw_off = 0;  // bytes: where they begin in raw; -1: raw[0] is the bits already
  auto load_mask = [&](int k) {
    const int c = in0 + k * kColumns + 32 * tid, l = c - pre;
    if (k >= copies || c >= min(in0 + (k + 1) * kColumns, in1)) return;
    if (mask_kind == 2) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(mask) + (l >> 5);
      raw[0] = __ldg(w);
      raw[1] = (l & 31) && ((l >> 5) + 1) * 32 < V ? __ldg(w + 1) : 0u;
    } else {
      const uint8_t* p = mask + l;
      raw_off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 3);
      if (l + 32 <= V && (raw_off == 0 || (l >= 4 && l + 36 <= V))) {  // whole words inside the row
        const uint32_t* w = reinterpret_cast<const uint32_t*>(p - raw_off);
        if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
          const uint4 u = __ldcs(reinterpret_cast<const uint4*>(w)),
                      v = __ldcs(reinterpret_cast<const uint4*>(w) + 1);
          raw[0] = u.x; raw[1] = u.y; raw[2] = u.z; raw[3] = u.w;
          raw[4] = v.x; raw[5] = v.y; raw[6] = v.z; raw[7] = v.w;
          raw[8] = 0;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) raw[j] = __ldcs(w + j);
          raw[8] = raw_off ? __ldcs(w + 8) : 0u;
        }
      } else {
        uint32_t bits = 0;
#pragma unroll 1
        for (int i = 0; i < 32 && l + i < V; ++i) bits |= (p[i] != 0 ? 1u : 0u) << i;
        raw[0] = bits;
        raw_off = -1;
      }
    }
  };
  auto store_mask = [&](int k) {
    const int c = in0 + k * kColumns + 32 * tid;
    if (k >= copies || c >= min(in0 + (k + 1) * kColumns, in1)) return;
    uint32_t bits;
    if (mask_kind == 2) {
      bits = __funnelshift_r(raw[0], raw[1], static_cast<uint32_t>(c - pre));
    } else if (raw_off < 0) {
      bits = raw[0];
    } else {
      bits = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        bits |= byte_bits(__funnelshift_r(raw[j], raw[j + 1], 8 * raw_off)) << (4 * j);
    }
    mask_bits[k & 1][tid] = bits;
  };
  if (mask_kind) load_mask(0);
  if (tid == kThreads - 1) read_row<COUNT, BACKWARD>(a, row, r);
  auto clear = [&] {
    for (int i = tid; i < room * int(sizeof(Word)) / 16; i += kThreads)
      reinterpret_cast<uint4*>(counters)[i] = make_uint4(0, 0, 0, 0);
  };
  if (COUNT) clear();
  if (COUNT) {
    for (int j = tid; j < n_bias; j += kThreads) {
      const int64_t id = whole(a.bias_ids, row * a.ld_bias_ids + j, a.bias64);
      bias_col[j] = id >= 0 && id < V ? static_cast<int>(id) + pre : -1;
      bias_val[j] = a.bias_values[row * a.ld_bias_values + j];
    }
  }
  if (!BACKWARD && a.stats) cluster_arrive();  // waited for before another block's memory is written
  if (mask_kind) store_mask(0);
  __syncthreads();
  const bool zero = BACKWARD && r.zero;

  if (zero) {  // the same columns, without a look at the logits
    zero_columns<T>(a, out, begin - pre, end - pre);
    if (copies > 0) mbar_wait(&landed[0], 0, &gave_up, a.err);  // nothing is on its way when it ends
    if (copies > 1) mbar_wait(&landed[1], 0, &gave_up, a.err);
    return;
  }
  // z of the sum so far, by its counter; the slope by its logit goes into k
  auto change = [&](float y, uint32_t n, int c, float& k) {
    if (n & (COUNTER::kSeen | COUNTER::kCount)) {
      k = y > 0.0f ? r.inv_rep : r.rep;
      y *= k;
      if (n & COUNTER::kCount) y = fmaf(-r.freq, static_cast<float>(n & COUNTER::kCount), y) - r.pres;
    }
    if (n & COUNTER::kBiased) {
#pragma unroll 1
      for (int j = 0; j < n_bias; ++j)
        if (bias_col[j] == c) y += bias_val[j];
    }
    return y;
  };
  auto gradient = [&](float z, float slope, bool label) {
    const float q = fmaxf(z - r.lse, -200.0f), e = fast_ex2(fmaf(q, kLog2e, -r.low * kLog2e));
    const float dz = -e * (fmaf(r.h, q + (r.ent - r.low), r.g) + (r.lse - r.lse)) + (label ? r.g : 0.0f);
    return slope * dz;
  };
  Running run;
  float inv_temp = r.inv_temp;
  const float rep = COUNT ? r.rep : 1.0f, inv_rep = COUNT ? r.inv_rep : 1.0f;
  const float freq = COUNT ? r.freq : 0.0f, pres = COUNT ? r.pres : 0.0f;
  const bool counted = freq != 0.0f || pres != 0.0f;
  // The gradient of a column that is not the label's: p (down_h (z - lse) + down_g), where down_g has the rest
  // of ln p; a row whose lse is NaN has NaN.  z - lse is exact where p is not small, so that p keeps its digits
  // whatever the size of the logits: without `low`, up to half a step of the lse is the relative error of p, and
  // 1 - p of a label at 0.9998 is off by up to 2 % at a size of 100, by up to 60 % at 3000.
  const float down_h = BACKWARD ? -r.h * inv_temp : 0.0f;
  float down_g = BACKWARD ? -fmaf(r.h, r.ent - r.low, r.g) * inv_temp + (r.lse - r.lse) : 0.0f;
  const bool stats = !BACKWARD && a.stats, entropy = !PROCESS && a.entropy;
  const int label = PROCESS ? -1 : r.label;
  int copied = 0;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int c0 = begin + pass * room, c1 = min(c0 + room, end);
    if (c0 >= c1) break;
    if constexpr (COUNT) {
      if (pass > 0) {
        __syncthreads();  // the last pass's counters are done with
        clear();
        __syncthreads();
      }
      if (r.length > 0) {
        const uint32_t at = smem_u32(counters);
        if (a.ids64) {
          const auto* t = static_cast<const int64_t*>(a.tokens) + row * a.ld_tokens;
          count<COUNTER, true>(t, 0, r.prompt, c0 - pre, c1 - c0, at);
          count<COUNTER, false>(t, r.prompt, r.length, c0 - pre, c1 - c0, at);
        } else {
          const auto* t = static_cast<const int32_t*>(a.tokens) + row * a.ld_tokens;
          count<COUNTER, true>(t, 0, r.prompt, c0 - pre, c1 - c0, at);
          count<COUNTER, false>(t, r.prompt, r.length, c0 - pre, c1 - c0, at);
        }
      }
      for (int j = tid; j < n_bias; j += kThreads) {
        const int c = bias_col[j];
        if (c < c0 || c >= c1) continue;
        const uint32_t byte = (c - c0) * sizeof(Word);
        atomicOr(reinterpret_cast<uint32_t*>(counters + (byte & ~3u)),
                 COUNTER::kBiased << (8 * (byte & 3u)));
      }
      __syncthreads();
    }
    // a row's first and last columns where they are no whole vector
    for (int edge = 0; edge < 2; ++edge) {
      const int c = edge == 0 ? (pre ? 0 : -1) : (span % VEC ? span / VEC * VEC : -1);
      if (c < c0 || c >= c1 || (edge == 1 && pre && c == 0) || tid != edge * 32) continue;
#pragma unroll 1
      for (int i = 0; i < VEC; ++i) {
        const int l = c + i - pre;
        if (l < 0 || l >= V) continue;
        bool ok = true;
        if (mask_kind == 2)
          ok = reinterpret_cast<const uint32_t*>(mask)[l >> 5] >> (l & 31) & 1;
        else if (mask_kind == 1)
          ok = mask[l] != 0;
        float z = widen1(x[l]), k = 1.0f;
        if constexpr (COUNT) {
          const uint32_t n = reinterpret_cast<const Word*>(counters)[c + i - c0];
          if (n) z = change(z, n, c + i, k);
        }
        z = ok ? z * inv_temp : -INFINITY;
        if (stats) {
          const float one[1] = {z};
          run.add(one, entropy);
          if (l == label) label_z = z;
        }
        if (BACKWARD) z = gradient(z, ok ? k * inv_temp : 0.0f, l == label);
        if (out) {
          if (a.out_f32) reinterpret_cast<float*>(out)[l] = z;
          else reinterpret_cast<T*>(out)[l] = narrow1<T>(z);
        }
      }
    }
    // the pass's whole vectors, copy by copy
    const int p1 = min(c1, in1);
    for (int c = max(c0, in0); c < p1;) {
      const int k = (c - in0) / kColumns, base = in0 + k * kColumns;
      const int stop = min(base + kColumns, p1);  // of this pass and copy
      if (k >= copied) {
        // a wait that runs out leaves NaN in the outputs; every thread goes the same way on
        if (!mbar_wait(&landed[k & 1], (k >> 1) & 1, &gave_up, a.err)) inv_temp = down_g = NAN;
        copied = k + 1;
      }
      const uint8_t* staged = shared + (k & 1) * kStage;
      const bool ends = stop == min(base + kColumns, in1);  // the copy, not just the pass
      if (mask_kind && ends) load_mask(k + 1);
#pragma unroll 1
      for (int cv = c + tid * VEC; cv < stop; cv += kThreads * VEC) {
        const int l = cv - pre;
        float z[VEC];
        uint32_t any = 0, biased = 0;    // columns that are changed, and by a bias
        float times[COUNT ? VEC : 1];    // where any: the slope by the repetition penalty
        widen<T>(*reinterpret_cast<const uint4*>(staged + (cv - base) * sizeof(T)), z);
        if constexpr (COUNT) {
          constexpr int WORDS = VEC * sizeof(Word) / 4;
          uint32_t n32[WORDS];
          const uint8_t* src = counters + (cv - c0) * sizeof(Word);
          if constexpr (WORDS == 2) {
            *reinterpret_cast<uint2*>(n32) = *reinterpret_cast<const uint2*>(src);
          } else {
#pragma unroll
            for (int j = 0; j < WORDS; j += 4)
              *reinterpret_cast<uint4*>(n32 + j) = *reinterpret_cast<const uint4*>(src + 4 * j);
          }
#pragma unroll
          for (int j = 0; j < WORDS; ++j) any |= n32[j];
          if (any) {
            // without branches, as lanes differ, and two columns at a time
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
              uint32_t seen0, seen1;  // not 0: among the row's tokens
              float count0, count1;
              split_counter<COUNTER>(n32, i, seen0, seen1, count0, count1);
              const float k0 = z[i] > 0.0f ? inv_rep : rep, k1 = z[i + 1] > 0.0f ? inv_rep : rep;
              times[i] = seen0 ? k0 : 1.0f;
              times[i + 1] = seen1 ? k1 : 1.0f;
              uint64_t y = f2_mul(f2_pack(z[i], z[i + 1]), f2_pack(times[i], times[i + 1]));
              if (counted) {
                y = f2_fma(f2_pack(count0, count1), f2_pack(-freq, -freq), y);
                y = f2_add(y, f2_pack(count0 > 0.0f ? -pres : 0.0f, count1 > 0.0f ? -pres : 0.0f));
              }
              f2_unpack(y, z[i], z[i + 1]);
            }
            biased = any & (COUNTER::kBiased | (sizeof(Word) == 2 ? COUNTER::kBiased << 16 : 0u));
          }
          if (n_bias > 0) {
            // the lanes of a warp look through 32 entries at a time, for all of its columns
            const int cw = cv - lane * VEC;
            const uint32_t lanes = stop - cw >= 32 * VEC ? 0xffffffffu
                                                         : (1u << ((stop - cw + VEC - 1) / VEC)) - 1u;
            if (__any_sync(lanes, biased)) {
              const int width = __popc(lanes);
#pragma unroll 1
              for (int j0 = 0; j0 < n_bias; j0 += width) {
                const int at = j0 + lane < n_bias ? bias_col[j0 + lane] - cw : -1;
                const float value = j0 + lane < n_bias ? bias_val[j0 + lane] : 0.0f;
                for (uint32_t hits = __ballot_sync(lanes, at >= 0 && at < width * VEC); hits;
                     hits &= hits - 1) {
                  const int from_lane = __ffs(hits) - 1;
                  const int i = __shfl_sync(lanes, at, from_lane) - lane * VEC;
                  const float v = __shfl_sync(lanes, value, from_lane);
#pragma unroll
                  for (int q = 0; q < VEC; ++q) z[q] += q == i ? v : 0.0f;
                }
              }
            }
          }
        }
        const uint64_t inv2 = f2_pack(inv_temp, inv_temp);
#pragma unroll
        for (int i = 0; i < VEC; i += 2)
          f2_unpack(f2_mul(f2_pack(z[i], z[i + 1]), inv2), z[i], z[i + 1]);
        uint32_t there = kAll;
        if (mask_kind) {
          const int at = cv - base;
          there = mask_bits[k & 1][at >> 5] >> (at & 31) & kAll;
          if (there != kAll) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
              if (!(there >> i & 1)) z[i] = -INFINITY;
          }
        }
        if constexpr (!BACKWARD) {
          if (stats) {
            run.add(z, entropy);
            if (!PROCESS && static_cast<uint32_t>(label - l) < VEC) {
              float zy = z[0];
#pragma unroll
              for (int i = 1; i < VEC; ++i)
                if (i == label - l) zy = z[i];
              label_z = zy;
            }
          }
          if (!PROCESS && !out) continue;
        } else {
          // p and its logarithm from q = max(z - lse, -200): p is 0 there, and -inf stays out of the sums
          const float rest = -r.low * kLog2e;
          const uint64_t minus = f2_pack(-r.lse, -r.lse), log2 = f2_pack(kLog2e, kLog2e), rest2 = f2_pack(rest, rest);
          const uint64_t h2 = f2_pack(down_h, down_h), g2 = f2_pack(down_g, down_g);
#pragma unroll
          for (int i = 0; i < VEC; i += 2) {
            float q0, q1, t0, t1;
            f2_unpack(f2_add(f2_pack(z[i], z[i + 1]), minus), q0, q1);
            const uint64_t q = f2_pack(fmaxf(q0, -200.0f), fmaxf(q1, -200.0f));
            f2_unpack(f2_fma(q, log2, rest2), t0, t1);
            const uint64_t p = f2_pack(fast_ex2(t0), fast_ex2(t1));
            f2_unpack(f2_mul(p, f2_fma(h2, q, g2)), z[i], z[i + 1]);
          }
          if (static_cast<uint32_t>(label - l) < VEC) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
              if (i == label - l && (there >> i & 1)) z[i] += r.g * inv_temp;
          }
          if constexpr (COUNT) {
            if (any) {
#pragma unroll
              for (int i = 0; i < VEC; ++i) z[i] *= times[i];
            }
          }
        }
        if (a.out_f32) {
          float* o = reinterpret_cast<float*>(out) + l;
          if ((reinterpret_cast<uintptr_t>(o) & 15) == 0) {
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i)
              __stcs(reinterpret_cast<float4*>(o) + i,
                     make_float4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]));
          } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = z[i];
          }
        } else {
          T* o = reinterpret_cast<T*>(out) + l;
          if ((reinterpret_cast<uintptr_t>(o) & 15) == 0) {
            __stcs(reinterpret_cast<uint4*>(o), narrow<T>(z));
          } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = narrow1<T>(z[i]);
          }
        }
      }
      c = stop;
      if (ends && k + 1 < copies && (mask_kind || k + 2 < copies)) {
        if (mask_kind) store_mask(k + 1);
        __syncthreads();  // the copy is done with, the next one's mask is there
        if (tid == 0 && k + 2 < copies) {
          asm volatile("fence.proxy.async;" ::: "memory");
          copy(k + 2);
        }
      }
    }
  }
  if (stats) {
    __syncwarp();
    Stats mine = join_warp(Stats{run.top, run.d, run.s}, 32);
    if ((tid & 31) == 0) part[tid >> 5] = mine;
    __syncthreads();
    cluster_wait();
    if (tid < 32) {
      mine = join_warp(tid < kWarps ? part[tid] : Stats{-INFINITY, 0.0f, 0.0f}, kWarps);
      if (tid == 0) {
        const uint32_t at = mapa_shared(smem_u32(&from[rank]), 0);
        st_remote(at, mine.m);
        st_remote(at + 4, mine.d);
        st_remote(at + 8, mine.s);
        st_remote(at + 12, label_z);
      }
    }
    cluster_arrive();  // the other blocks are done; their memory is not written by any
    if (rank != 0) return;
    cluster_wait();
    if (tid < 32) {
      const float4 one = tid < size ? from[tid] : make_float4(-INFINITY, 0.0f, 0.0f, -INFINITY);
      const Stats all = join_warp(Stats{one.x, one.y, one.z}, kMaxCluster);
      float zy = one.w;  // a NaN there is in all.d too
#pragma unroll
      for (int j = kMaxCluster / 2; j > 0; j >>= 1)
        zy = fmaxf(zy, __shfl_xor_sync(0xffffffffu, zy, j));
      if (tid != 0) return;
      const float log_d = logf(all.d);
      const bool none = all.m == -INFINITY && all.d == 0.0f;  // nothing is left
      if (a.lse) {
        const float lse = none ? -INFINITY : all.m + log_d, part_d = lse - all.m;
        a.lse[row] = lse;
        // (what the sum lost, by Knuth's two-sum)
        if (a.split)
          a.lse[a.R + row] = isfinite(lse) ? (all.m - (lse - part_d)) + (log_d - part_d) : 0.0f;
      }
      if (a.logp)
        a.logp[row] = r.ignored ? 0.0f
                      : r.bad   ? NAN
                      : none    ? -INFINITY
                                : (zy - all.m) - log_d;
      if (a.entropy) {
        const float H = none ? 0.0f : log_d - kLn2 * __fdiv_rn(all.s, all.d);
        a.entropy[row] = r.ignored ? 0.0f : r.bad ? NAN : H;
      }
      if (r.bad && a.err) atomicOr(a.err, FLCE_DEVERR_LABEL);
    }
  }
}

// ------------------------------------------------------------------ host
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int rc_of(cudaError_t e) {
  if (e == cudaSuccess) return FLCE_OK;
  cudaGetLastError();  // reported here, not by a later call
  return FLCE_ERR_CUDA;
}

template <typename T, typename COUNTER, int MODE, bool MASK, bool BIAS>
int run(Args a, int sms, cudaStream_t st) {
  auto kernel = logits_kernel<T, COUNTER, MODE, MASK, BIAS>;
  constexpr bool COUNT = !std::is_same_v<COUNTER, NoCounter>;
  constexpr int VEC = 16 / sizeof(T);
  constexpr int64_t wide = int64_t(kThreads) * VEC;
  // whole 16-byte words of counters, whole vectors
  using Word = typename COUNTER::Word;
  constexpr int64_t unit = 16 / sizeof(Word) > VEC ? 16 / sizeof(Word) : VEC;
  constexpr int64_t most = kRoom / sizeof(Word);
  const int64_t span = a.V + VEC - 1;  // with what may stand before a row
  // Blocks per row: few rows take as many as are resident at once, as a second round of blocks costs more
  // than shorter ones save (64 x 128256 in fp32 with a mask: 23.6 us by 4, 30.6 by 16; 200 x 32000: 13.3 by
  // 2, 19.0 by 8); more rows as few as fill the GPU several times over, so that the last round is a small
  // part (384 x 256000: 156 us by 4, 161 by 1).  None has less than a vector for half of its threads.
  const int64_t resident = int64_t(kBlocks) * sms;
  const bool few = 2 * a.R <= resident;
  int size = 1;
  while (size < kMaxCluster && (few ? 2 * a.R * size <= resident : a.R * size < kFill * sms) &&
         span > size * wide / 2)
    size *= 2;
  a.columns = cdiv(cdiv(span, size), unit) * unit;
  a.passes = static_cast<int32_t>(COUNT ? cdiv(a.columns, most) : 1);
  a.room = cdiv(cdiv(a.columns, a.passes), unit) * unit;
  const int64_t bytes = a.columns * static_cast<int64_t>(sizeof(T));
  a.stage_bytes = bytes < 2 * kStage ? static_cast<int32_t>(cdiv(bytes, 16) * 16) : 2 * kStage;
  const size_t smem = a.stage_bytes + (COUNT ? a.room * sizeof(Word) : 0) + a.n_bias * 8;
  constexpr int kMostShared = 2 * kStage + (COUNT ? kRoom : 0) + kMaxBias * 8;
  // the same values from every thread that gets here, once per device
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  int rc = rc_of(cudaGetDevice(&dev));
  if (rc) return rc;
  if (!(ready.load() >> (dev & 63) & 1)) {
    if ((rc = rc_of(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kMostShared))) ||
        (rc = rc_of(cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                         1))))
      return rc;
    ready.fetch_or(uint64_t(1) << (dev & 63));
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.R * size));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(size);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return rc_of(cudaLaunchKernelEx(&cfg, kernel, a));
}

template <typename T, typename COUNTER, bool MASK, bool BIAS>
int run_mode(const Args& a, int mode, int sms, cudaStream_t st) {
  return mode == MODE_PROCESS   ? run<T, COUNTER, MODE_PROCESS, MASK, BIAS>(a, sms, st)
         : mode == MODE_FORWARD ? run<T, COUNTER, MODE_FORWARD, MASK, BIAS>(a, sms, st)
                                : run<T, COUNTER, MODE_BACKWARD, MASK, BIAS>(a, sms, st);
}

// count 0: no counters, else their bits.  Histories of 2^14 tokens and more take the kernels that can do
// everything.
template <typename T>
int run_type(const Args& a, int count, int mode, int sms, cudaStream_t st) {
  const bool mask = a.mask_kind != 0, bias = a.n_bias != 0;
  if (count == 32) return run_mode<T, Counter<uint32_t>, true, true>(a, mode, sms, st);
  if (count == 16)
    return bias ? (mask ? run_mode<T, Counter<uint16_t>, true, true>(a, mode, sms, st)
                        : run_mode<T, Counter<uint16_t>, false, true>(a, mode, sms, st))
                : (mask ? run_mode<T, Counter<uint16_t>, true, false>(a, mode, sms, st)
                        : run_mode<T, Counter<uint16_t>, false, false>(a, mode, sms, st));
  return mask ? run_mode<T, NoCounter, true, false>(a, mode, sms, st)
              : run_mode<T, NoCounter, false, false>(a, mode, sms, st);
}

}  // namespace

// by the logits' type, each in a source of its own
int run_f32(const Args& a, int count, int mode, int sms, cudaStream_t st);
int run_bf16(const Args& a, int count, int mode, int sms, cudaStream_t st);
int run_f16(const Args& a, int count, int mode, int sms, cudaStream_t st);

}  // namespace logits
}  // namespace flce
