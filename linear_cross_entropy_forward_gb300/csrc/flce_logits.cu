// Rows of logits as a sampler sees them, their logsumexp, the log-probability of a label and
// the entropy under them, and the gradient by the logits.
//
//   z = (seen ? (l > 0 ? l / rp : l rp) : l) - fp n - pp [n > 0] + (sum of the biases on it)
//   z = -inf where not allowed;  z = z / T
//
// n counts a token among the row's generated tokens, seen says whether it is among prompt or
// generated ones.  One pass over the logits, so bound by their bytes, in and out.
//
// A row is shared by a cluster of blocks, each with a run of columns and a 32-bit counter per
// column in its shared memory.  The row's tokens are read once: each block takes a share of
// them and adds into the counter of the block that has the column, over distributed shared
// memory.  Biases only mark their columns' counters; a marked column sums its biases from the
// row's list, in the list's order.  The running maximum m, d = sum 2^u and s = sum 2^u u with
// u = log2(e) (z - m) stay in registers, are joined in the block and then in the cluster, in a
// fixed order:  lse = m + ln d,  H = ln d - ln 2 s / d.
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

#ifndef FLCE_LOGITS_THREADS
#define FLCE_LOGITS_THREADS 256
#endif
#ifndef FLCE_LOGITS_FILL
#define FLCE_LOGITS_FILL 4
#endif
#ifndef FLCE_LOGITS_ROOM
#define FLCE_LOGITS_ROOM 65536
#endif
constexpr int kThreads = FLCE_LOGITS_THREADS;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;            // vectors in flight per thread
constexpr int kMaxCluster = 16;
constexpr int kRoom = FLCE_LOGITS_ROOM;  // bytes of counters per block
constexpr int kMaxBias = 2048;       // entries of a row's list: 16 KB of shared memory

// Counters: occurrences among the generated tokens, and flags of the prompt's tokens and of
// columns with a bias.  16 bits hold the count of histories below 2^14 tokens.
struct NoCounter {
  using Word = uint16_t;
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
  float* lse;
  float* logp;
  float* entropy;
  const float* g_logp;
  const float* g_entropy;
  uint32_t* err;
  int64_t columns, passes;  // per block and pass; runs of whole vectors
  int32_t ids64, lens64, bias64, mask_kind, out_f32, stats;
};

enum { MODE_FORWARD = 0, MODE_BACKWARD = 1 };

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

__device__ __forceinline__ int64_t whole(const void* p, int64_t i, int is64) {
  return is64 ? __ldg(static_cast<const long long*>(p) + i)
              : static_cast<int64_t>(__ldg(static_cast<const int*>(p) + i));
}

// Statistics of a part of a row: m the largest z, d and s as above (m = -inf: nothing).
struct Stats {
  float m, d, s;
};

__device__ __forceinline__ Stats join(const Stats& a, const Stats& b) {
  const float m = fmaxf(a.m, b.m);
  Stats r{m, a.d + b.d, a.s + b.s};
  if (m == -INFINITY) return r;
  // a part without anything has d = s = 0: its exponent may be anything finite
  const float ta = a.m == -INFINITY ? 0.0f : (a.m - m) * kLog2e;
  const float tb = b.m == -INFINITY ? 0.0f : (b.m - m) * kLog2e;
  const float ea = fast_ex2(ta), eb = fast_ex2(tb);
  r.d = fmaf(ea, a.d, eb * b.d);
  r.s = (ea != 0.0f ? ea * fmaf(ta, a.d, a.s) : 0.0f) +
        (eb != 0.0f ? eb * fmaf(tb, b.d, b.s) : 0.0f);
  return r;
}

// What a row's columns are changed by.
struct Row {
  float rep, inv_rep, freq, pres, inv_temp;
  const uint8_t* mask;
};

// Address of a shared variable of this block's in block `rank` of the cluster.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  return mapa_shared(smem_u32(p), rank);
}
__device__ __forceinline__ void red_add(uint32_t a, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void red_or(uint32_t a, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void st_remote(uint32_t a, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
// All blocks of the cluster, whatever paths the threads of a warp came by.
__device__ __forceinline__ void meet() {
  __syncwarp();
  cluster_sync();
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// VEC mask bytes at p (that of logit l of a row of V) as bits: bit i set where byte i is not 0.
template <int VEC>
__device__ __forceinline__ uint32_t byte_mask(const uint8_t* p, int64_t l, int64_t V) {
  uint32_t w[VEC / 4];
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 3);
  if (off == 0 || (l >= 4 && l + VEC + 4 <= V)) {  // whole words inside the row
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p - off);
    uint32_t lo = __ldg(q);
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j) {
      const uint32_t hi = j + 1 < VEC / 4 || off ? __ldg(q + j + 1) : 0u;
      w[j] = __funnelshift_r(lo, hi, 8 * off);
      lo = hi;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j)
      w[j] = p[4 * j] | p[4 * j + 1] << 8 | p[4 * j + 2] << 16 | uint32_t(p[4 * j + 3]) << 24;
  }
  uint32_t bits = 0;
#pragma unroll
  for (int j = 0; j < VEC / 4; ++j) {
    // bit 7 of each byte that is not 0, then the four of them side by side
    const uint32_t t = ((((w[j] & 0x7f7f7f7fu) + 0x7f7f7f7fu) | w[j]) >> 7) & 0x01010101u;
    bits |= ((t * 0x01020408u) >> 24 & 15u) << (4 * j);
  }
  return bits;
}

// Columns are numbered from the row's last 16-byte boundary at or before its first logit, so
// that vectors of VEC columns are aligned in every row; `pre` columns before the row are not
// there.  Column c of that numbering is logit c - pre.
template <typename T, typename COUNTER, int MODE>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    logits_kernel(const __grid_constant__ Args a) {
  constexpr int VEC = 16 / sizeof(T);
  constexpr bool COUNT = !std::is_same_v<COUNTER, NoCounter>;
  using Word = typename COUNTER::Word;
  extern __shared__ __align__(16) uint8_t shared[];  // counters, then the biases' columns and values
  __shared__ Stats part[kWarps];
  __shared__ Stats from[kMaxCluster];
  __shared__ float label_z;
  Word* counters = reinterpret_cast<Word*>(shared);
  const uint32_t rank = cluster_ctarank(), size = cluster_size();
  const int64_t row = blockIdx.x / size;
  const T* x = static_cast<const T*>(a.logits) + row * a.ld;
  const int pre = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const int64_t span = a.V + pre;
  const int64_t per_pass = a.columns * size;
  int* bias_col = reinterpret_cast<int*>(shared + a.columns * sizeof(Word));
  float* bias_val = reinterpret_cast<float*>(bias_col + a.n_bias);

  // the first vectors are asked for before anything is waited for
  alignas(16) T in[kBatch][VEC];
  auto load = [&](int64_t v0, int64_t c1) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int64_t c = v0 + int64_t(b) * kThreads * VEC, l = c - pre;
      if (c >= c1) continue;
      if (l >= 0 && l + VEC <= a.V) {
        *reinterpret_cast<uint4*>(in[b]) = __ldcs(reinterpret_cast<const uint4*>(x + l));
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          in[b][i] = l + i >= 0 && l + i < a.V ? x[l + i] : narrow<T>(0.0f);
      }
    }
  };
  {
    const int64_t c0 = rank * a.columns;
    load(c0 + threadIdx.x * VEC, c0 + a.columns < span ? c0 + a.columns : span);
  }

  int64_t label = -1;
  bool ignored = false, bad = false;
  if (a.labels) {
    const int64_t y = a.labels[row];
    ignored = y == a.ignore_index;
    if (y >= 0 && y < a.V) label = y;
    else bad = !ignored;
  }
  // the gradient's constants: -p (g + h (ln p + H)) + g [label]
  float lse = 0.0f, g = 0.0f, h = 0.0f, ent = 0.0f;
  bool zero = false;
  if (MODE == MODE_BACKWARD) {
    lse = a.lse[row];
    if (!ignored) {
      g = a.g_logp ? a.g_logp[row] : 0.0f;
      h = a.g_entropy ? a.g_entropy[row] : 0.0f;
    }
    ent = a.entropy ? a.entropy[row] : 0.0f;
    zero = ignored || lse == -INFINITY;
  }
  Row p;
  p.rep = a.rep ? a.rep[row] : a.rep1;
  p.inv_rep = __fdiv_rn(1.0f, p.rep);
  p.freq = a.freq ? a.freq[row] : a.freq1;
  p.pres = a.pres ? a.pres[row] : a.pres1;
  const float temp = a.temp ? a.temp[row] : a.temp1;
  p.inv_temp = temp > 0.0f ? __fdiv_rn(1.0f, temp) : 1.0f;
  p.mask = static_cast<const uint8_t*>(a.allowed) +
           row * a.ld_allowed * (a.mask_kind == 2 ? 4 : 1);
  int64_t length = 0, prompt = 0;
  if (COUNT && a.tokens) {
    length = a.lengths ? whole(a.lengths, row, a.lens64) : a.T;
    length = length < a.T ? length : a.T;
    prompt = a.prompt_lens ? whole(a.prompt_lens, row, a.lens64) : 0;
    if (p.rep == 1.0f && p.freq == 0.0f && p.pres == 0.0f) length = 0;
  }
  if (COUNT && !zero) {
    for (int64_t j = threadIdx.x; j < a.n_bias; j += kThreads) {
      const int64_t id = whole(a.bias_ids, row * a.ld_bias_ids + j, a.bias64);
      // columns are below 2^31; -1 is no column
      bias_col[j] = id >= 0 && id < a.V ? static_cast<int>(id + pre) : -1;
      bias_val[j] = a.bias_values[row * a.ld_bias_values + j];
    }
  }
  if (a.stats && threadIdx.x == 0 && rank == 0) label_z = -INFINITY;

  Stats mine{-INFINITY, 0.0f, 0.0f};
  for (int64_t pass = 0; pass < a.passes; ++pass) {
    const int64_t base = pass * per_pass;  // of the pass's columns
    const int64_t c0 = base + rank * a.columns;
    const int64_t c1 = c0 + a.columns < span ? c0 + a.columns : span;
    if (COUNT && !zero) {
      // every block of the cluster clears its counters before any adds to them
      if (pass > 0) __syncthreads();
      uint4* clear = reinterpret_cast<uint4*>(shared);
      for (int i = threadIdx.x; i < a.columns * int(sizeof(Word)) / 16; i += kThreads)
        clear[i] = make_uint4(0, 0, 0, 0);
      meet();
      if constexpr (COUNT) {
        const int64_t share = (length + size - 1) / size;
        const int64_t t0 = rank * share;
        const int64_t t1 = t0 + share < length ? t0 + share : length;
        const uint32_t columns = static_cast<uint32_t>(a.columns);
        for (int64_t t = t0 + threadIdx.x; t < t1; t += kThreads) {
          const int64_t id = whole(a.tokens, row * a.ld_tokens + t, a.ids64);
          const int64_t c = id + pre - base;
          if (id < 0 || id >= a.V || c < 0 || c >= per_pass) continue;
          const uint32_t owner = static_cast<uint32_t>(c) / columns;
          const uint32_t byte = (static_cast<uint32_t>(c) - owner * columns) * sizeof(Word);
          const uint32_t at = remote(shared + (byte & ~3u), owner), shift = 8 * (byte & 3u);
          if (t < prompt) red_or(at, COUNTER::kSeen << shift);
          else red_add(at, 1u << shift);
        }
        for (int j = threadIdx.x; j < a.n_bias; j += kThreads) {
          const int64_t c = bias_col[j];  // every block marks its own columns
          if (c < c0 || c >= c1) continue;
          const uint32_t byte = static_cast<uint32_t>(c - c0) * sizeof(Word);
          atomicOr(reinterpret_cast<uint32_t*>(shared + (byte & ~3u)),
                   COUNTER::kBiased << (8 * (byte & 3u)));
        }
      }
      meet();
    } else if (MODE == MODE_FORWARD && a.stats && pass == 0) {
      meet();  // label_z of the first block is there, and cleared
    }
    for (int64_t v0 = c0 + threadIdx.x * VEC; v0 < c1; v0 += int64_t(kThreads) * VEC * kBatch) {
      if ((pass > 0 || v0 >= c0 + int64_t(kThreads) * VEC) && !zero) load(v0, c1);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int64_t c = v0 + int64_t(b) * kThreads * VEC;
        if (c >= c1) continue;
        const int64_t l = c - pre;
        const bool inside = l >= 0 && l + VEC <= a.V;
        constexpr uint32_t kAll = (1u << VEC) - 1;
        uint32_t real = kAll;  // bit i: column c + i is a logit
        if (!inside) {
          real = 0;
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            if (l + i >= 0 && l + i < a.V) real |= 1u << i;
        }
        uint32_t there = real;  // and allowed
        if (a.mask_kind == 2) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(p.mask);
          if (l >= 0) {
            const uint32_t lo = __ldg(w + (l >> 5));
            const uint32_t hi = (l & 31) + VEC > 32 && ((l >> 5) + 1) * 32 < a.V
                                    ? __ldg(w + (l >> 5) + 1) : 0u;
            there &= __funnelshift_r(lo, hi, static_cast<uint32_t>(l & 31));
          } else {
            there &= __ldg(w) << static_cast<uint32_t>(-l);
          }
        } else if (a.mask_kind == 1) {
          if (inside) {
            there = byte_mask<VEC>(p.mask + l, l, a.V);
          } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
              if ((real >> i & 1) && p.mask[l + i] == 0) there &= ~(1u << i);
          }
        }
        float z[VEC], slope[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          z[i] = widen(in[b][i]);
          slope[i] = p.inv_temp;
        }
        if constexpr (COUNT) {
          constexpr int WORDS = VEC * sizeof(Word) / 4;
          uint32_t n32[WORDS];
          uint32_t any = 0;
          if (!zero) {
            const uint32_t* src = reinterpret_cast<const uint32_t*>(counters + (c - c0));
            if constexpr (WORDS == 2) {
              *reinterpret_cast<uint2*>(n32) = *reinterpret_cast<const uint2*>(src);
            } else {
#pragma unroll
              for (int j = 0; j < WORDS; j += 4)
                *reinterpret_cast<uint4*>(n32 + j) = *reinterpret_cast<const uint4*>(src + j);
            }
#pragma unroll
            for (int j = 0; j < WORDS; ++j) any |= n32[j];
          }
          if (any) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              const uint32_t n = sizeof(Word) == 4
                                     ? n32[i % WORDS] : n32[i / 2 % WORDS] >> (16 * (i & 1)) & 0xffffu;
              if (n == 0) continue;
              float y = z[i];
              if (n & (COUNTER::kSeen | COUNTER::kCount)) {
                const float k = y > 0.0f ? p.inv_rep : p.rep;
                y *= k;
                slope[i] *= k;
              }
              if (n & COUNTER::kCount)
                y = fmaf(-p.freq, static_cast<float>(n & COUNTER::kCount), y) - p.pres;
              if (n & COUNTER::kBiased) {
                float sum = 0.0f;
#pragma unroll 1
                for (int j = 0; j < a.n_bias; ++j)
                  if (bias_col[j] == static_cast<int>(c) + i) sum += bias_val[j];
                y += sum;
              }
              z[i] = y;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) z[i] *= p.inv_temp;
        if (there != kAll) {
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            if (!(there >> i & 1)) {
              z[i] = -INFINITY;
              slope[i] = 0.0f;
            }
        }
        const int64_t yl = label - l;  // the label's place in this vector
        if (MODE == MODE_FORWARD) {
          if (a.stats) {
            float top = z[0];
#pragma unroll
            for (int i = 1; i < VEC; ++i) top = fmaxf(top, z[i]);
            if (top > mine.m) {
              const float t = (mine.m - top) * kLog2e;  // -inf before the first
              const float e = fast_ex2(t);
              mine.s = e != 0.0f ? e * fmaf(t, mine.d, mine.s) : 0.0f;
              mine.d *= e;
              mine.m = top;
            }
            if (mine.m != -INFINITY) {
#pragma unroll
              for (int i = 0; i < VEC; ++i) {
                const float t = (z[i] - mine.m) * kLog2e;
                const float e = fast_ex2(t);
                mine.d += e;
                mine.s += e != 0.0f ? e * t : 0.0f;
              }
            } else {
#pragma unroll
              for (int i = 0; i < VEC; ++i) mine.d += z[i] != z[i] ? z[i] : 0.0f;  // NaN alone
            }
            if (yl >= 0 && yl < VEC) {
              float zy = z[0];
#pragma unroll
              for (int i = 1; i < VEC; ++i)
                if (i == yl) zy = z[i];
              st_remote(remote(&label_z, 0), zy);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float q = z[i] - lse;
            const float e = fast_ex2(q * kLog2e);
            float d = e != 0.0f ? -e * fmaf(h, q + ent, g) : 0.0f;
            if (i == yl) d += g;
            z[i] = zero ? 0.0f : slope[i] * d;
          }
        }
        if (a.out) {
          if (a.out_f32) {
            float* o = static_cast<float*>(a.out) + row * a.ld_out + l;
            if (inside && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
#pragma unroll
              for (int i = 0; i < VEC / 4; ++i)
                __stcs(reinterpret_cast<float4*>(o) + i,
                       make_float4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]));
            } else {
#pragma unroll
              for (int i = 0; i < VEC; ++i)
                if (real >> i & 1) o[i] = z[i];
            }
          } else {
            T* o = static_cast<T*>(a.out) + row * a.ld_out + l;
            if (inside && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
              alignas(16) T t[VEC];
#pragma unroll
              for (int i = 0; i < VEC; ++i) t[i] = narrow<T>(z[i]);
              __stcs(reinterpret_cast<uint4*>(o), *reinterpret_cast<uint4*>(t));
            } else {
#pragma unroll
              for (int i = 0; i < VEC; ++i)
                if (real >> i & 1) o[i] = narrow<T>(z[i]);
            }
          }
        }
      }
    }
  }
  if (MODE == MODE_FORWARD && a.stats) {
    __syncwarp();
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const Stats o{__shfl_down_sync(0xffffffffu, mine.m, d),
                    __shfl_down_sync(0xffffffffu, mine.d, d),
                    __shfl_down_sync(0xffffffffu, mine.s, d)};
      mine = join(mine, o);
    }
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w) mine = join(mine, part[w]);
      const uint32_t at = remote(&from[rank], 0);
      st_remote(at, mine.m);
      st_remote(at + 4, mine.d);
      st_remote(at + 8, mine.s);
    }
    meet();
    if (rank == 0 && threadIdx.x == 0) {
      Stats r = from[0];
      for (uint32_t i = 1; i < size; ++i) r = join(r, from[i]);
      const float log_d = logf(r.d);
      const float all = r.m == -INFINITY && r.d == 0.0f ? -INFINITY : r.m + log_d;
      if (a.lse) a.lse[row] = all;
      if (a.logp)
        a.logp[row] = ignored ? 0.0f
                      : bad   ? NAN
                              : label_z == -INFINITY ? -INFINITY : label_z - all;
      if (a.entropy) {
        const float H = all == -INFINITY ? 0.0f : log_d - kLn2 * __fdiv_rn(r.s, r.d);
        a.entropy[row] = ignored ? 0.0f : bad ? NAN : H;
      }
      if (bad && a.err) atomicOr(a.err, FLCE_DEVERR_LABEL);
    }
  }
}

// ------------------------------------------------------------------ host
inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int rc_of(cudaError_t e) {
  if (e == cudaSuccess) return FLCE_OK;
  cudaGetLastError();  // reported here, not by a later call
  return FLCE_ERR_CUDA;
}

int check(const flce_logits_params* p) {
  if (!p) return FLCE_ERR_BAD_ARG;
  if (p->dtype < FLCE_F32 || p->dtype > FLCE_F16) return FLCE_ERR_BAD_ARG;
  if (p->out_dtype != p->dtype && p->out_dtype != FLCE_F32) return FLCE_ERR_BAD_ARG;
  if (p->mask_kind < 0 || p->mask_kind > 2) return FLCE_ERR_BAD_ARG;
  // NaN is refused with the others
  if (!(p->repetition_penalty > 0.0) || isinf(p->repetition_penalty) ||
      !isfinite(p->frequency_penalty) || !isfinite(p->presence_penalty) ||
      !(p->temperature >= 0.0) || isinf(p->temperature))
    return FLCE_ERR_BAD_ARG;
  constexpr int64_t most = (int64_t(1) << 30);
  if (p->R < 0 || p->V < 1 || p->V > most || p->T < 0 || p->T >= most || p->n_bias < 0 ||
      p->n_bias > kMaxBias || p->R > (int64_t(1) << 31) / kMaxCluster - 1)
    return FLCE_ERR_BAD_SHAPE;
  if (p->ld_logits < 0 || p->ld_out < 0 || p->ld_tokens < 0 || p->ld_bias_ids < 0 ||
      p->ld_bias_values < 0 || p->ld_allowed < 0)
    return FLCE_ERR_BAD_SHAPE;
  if (p->R > 1 && p->ld_out < p->V) return FLCE_ERR_BAD_SHAPE;  // rows written would overlap
  return FLCE_OK;
}

template <typename T, typename COUNTER, int MODE>
int run(Args a, int sms, cudaStream_t st) {
  auto kernel = logits_kernel<T, COUNTER, MODE>;
  constexpr bool COUNT = !std::is_same_v<COUNTER, NoCounter>;
  constexpr int VEC = 16 / sizeof(T);
  constexpr int64_t wide = int64_t(kThreads) * VEC;
  // whole 16-byte words of counters, whole vectors
  constexpr int64_t unit = 16 / sizeof(typename COUNTER::Word) > VEC
                               ? 16 / sizeof(typename COUNTER::Word) : VEC;
  constexpr int64_t most = kRoom / sizeof(typename COUNTER::Word);
  const int64_t span = a.V + VEC - 1;  // with what may stand before a row
  // As few blocks per row as fill the GPU's block slots, but no more than have a vector for half
  // of their threads; the counters' room asks for more.
  int size = 1;
  while (size < kMaxCluster && ((a.R * size < FLCE_LOGITS_FILL * sms && span > size * wide / 2) ||
                                (COUNT && span > size * most)))
    size *= 2;
  a.columns = cdiv(cdiv(span, size), unit) * unit;
  a.passes = 1;
  if (COUNT && a.columns > most) {
    a.columns = most;
    a.passes = cdiv(span, size * most);
  }
  const size_t smem = COUNT ? a.columns * sizeof(typename COUNTER::Word) + a.n_bias * 8 : 0;
  // the same values from every thread that gets here, once per device
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  int rc = rc_of(cudaGetDevice(&dev));
  if (rc) return rc;
  if (!(ready.load() >> (dev & 63) & 1)) {
    if ((rc = rc_of(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kRoom + kMaxBias * 8))) ||
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

// count 0: no counters, else their bits
template <typename T>
int run_type(const Args& a, int count, bool backward, int sms, cudaStream_t st) {
  if (count == 16)
    return backward ? run<T, Counter<uint16_t>, MODE_BACKWARD>(a, sms, st)
                    : run<T, Counter<uint16_t>, MODE_FORWARD>(a, sms, st);
  if (count == 32)
    return backward ? run<T, Counter<uint32_t>, MODE_BACKWARD>(a, sms, st)
                    : run<T, Counter<uint32_t>, MODE_FORWARD>(a, sms, st);
  return backward ? run<T, NoCounter, MODE_BACKWARD>(a, sms, st)
                  : run<T, NoCounter, MODE_FORWARD>(a, sms, st);
}

// What both calls have in common: the checks and the kernel's arguments.
int common(const flce_logits_params* p, const flce_logits_rows* r, const void* logits,
           const int64_t* labels, void* out, void* workspace, size_t ws_bytes, Args* a) {
  const int rc = check(p);
  if (rc) return rc;
  if (!r || (p->R > 0 && !logits)) return FLCE_ERR_BAD_ARG;
  if (p->T > 0 && p->R > 0 && !r->tokens) return FLCE_ERR_BAD_ARG;
  if (p->n_bias > 0 && p->R > 0 && (!r->bias_ids || !r->bias_values)) return FLCE_ERR_BAD_ARG;
  if (p->mask_kind && p->R > 0 && !r->allowed) return FLCE_ERR_BAD_ARG;
  if (p->validate && !workspace) return FLCE_ERR_BAD_ARG;
  const int b = p->dtype == FLCE_F32 ? 4 : 2, ob = p->out_dtype == FLCE_F32 ? 4 : 2;
  if (addr(logits) & (b - 1) || addr(out) & (ob - 1) || addr(labels) & 7 ||
      (addr(r->repetition_penalty) | addr(r->frequency_penalty) | addr(r->presence_penalty) |
       addr(r->temperature) | addr(r->bias_values)) & 3 ||
      addr(r->tokens) & (p->tokens_int64 ? 7 : 3) ||
      (addr(r->prompt_lens) | addr(r->lengths)) & (p->lens_int64 ? 7 : 3) ||
      addr(r->bias_ids) & (p->bias_int64 ? 7 : 3) || (p->mask_kind == 2 && addr(r->allowed) & 3) ||
      addr(workspace) & 255)
    return FLCE_ERR_ALIGN;
  if (p->validate && ws_bytes < 256) return FLCE_ERR_WS_TOO_SMALL;
  Args& x = *a;
  x = Args{};
  x.logits = logits;
  x.out = out;
  x.R = p->R;
  x.V = p->V;
  x.ld = p->ld_logits;
  x.ld_out = p->ld_out;
  x.tokens = p->T > 0 ? r->tokens : nullptr;
  x.T = p->T;
  x.ld_tokens = p->ld_tokens;
  x.prompt_lens = r->prompt_lens;
  x.lengths = r->lengths;
  x.rep = r->repetition_penalty;
  x.freq = r->frequency_penalty;
  x.pres = r->presence_penalty;
  x.temp = r->temperature;
  x.rep1 = static_cast<float>(p->repetition_penalty);
  x.freq1 = static_cast<float>(p->frequency_penalty);
  x.pres1 = static_cast<float>(p->presence_penalty);
  x.temp1 = static_cast<float>(p->temperature);
  x.bias_ids = r->bias_ids;
  x.bias_values = r->bias_values;
  x.n_bias = p->n_bias;
  x.ld_bias_ids = p->ld_bias_ids;
  x.ld_bias_values = p->ld_bias_values;
  x.allowed = r->allowed;
  x.ld_allowed = p->ld_allowed;
  x.mask_kind = p->mask_kind;
  x.labels = labels;
  x.ignore_index = p->ignore_index;
  x.ids64 = p->tokens_int64;
  x.lens64 = p->lens_int64;
  x.bias64 = p->bias_int64;
  x.out_f32 = p->out_dtype == FLCE_F32;
  return FLCE_OK;
}

int launch(const flce_logits_params* p, Args a, bool backward, void* workspace, cudaStream_t st) {
  int rc, sms;
  if ((rc = require_device(&sms))) return rc;
  if (p->validate) {
    a.err = static_cast<uint32_t*>(workspace);
    if ((rc = rc_of(cudaMemsetAsync(workspace, 0, 256, st)))) return rc;
  }
  if (p->R > 0) {
    const bool penalties = a.rep || a.freq || a.pres || a.rep1 != 1.0f || a.freq1 != 0.0f ||
                           a.pres1 != 0.0f;
    if (!penalties) a.tokens = nullptr;
    const int count = a.tokens && a.T >= 1 << 14 ? 32 : a.tokens || a.n_bias > 0 ? 16 : 0;
    rc = p->dtype == FLCE_F32    ? run_type<float>(a, count, backward, sms, st)
         : p->dtype == FLCE_BF16 ? run_type<__nv_bfloat16>(a, count, backward, sms, st)
                                 : run_type<__half>(a, count, backward, sms, st);
    if (rc) return rc;
  }
  return p->validate ? read_status(workspace, st) : FLCE_OK;
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_logits_check_params(const flce_logits_params* p) { return check(p); }

int flce_logits(const flce_logits_params* p, const flce_logits_rows* rows, const void* logits,
                const int64_t* labels, void* out, float* lse, float* logp, float* entropy,
                void* workspace, size_t ws_bytes, void* stream) {
  Args a;
  int rc = common(p, rows, logits, labels, out, workspace, ws_bytes, &a);
  if (rc) return rc;
  if (!out && !lse && !logp && !entropy && p->R > 0) return FLCE_ERR_BAD_ARG;
  if (logp && !labels && p->R > 0) return FLCE_ERR_BAD_ARG;
  if ((addr(lse) | addr(logp) | addr(entropy)) & 3) return FLCE_ERR_ALIGN;
  a.lse = lse;
  a.logp = logp;
  a.entropy = entropy;
  a.stats = lse || logp || entropy;
  return launch(p, a, false, workspace, static_cast<cudaStream_t>(stream));
}

int flce_logits_backward(const flce_logits_params* p, const flce_logits_rows* rows,
                         const void* logits, const int64_t* labels, const float* lse,
                         const float* entropy, const float* g_logp, const float* g_entropy,
                         void* dlogits, void* workspace, size_t ws_bytes, void* stream) {
  Args a;
  int rc = common(p, rows, logits, labels, dlogits, workspace, ws_bytes, &a);
  if (rc) return rc;
  if (p->R > 0 && (!dlogits || !lse || !labels || (g_entropy && !entropy))) return FLCE_ERR_BAD_ARG;
  if ((addr(lse) | addr(entropy) | addr(g_logp) | addr(g_entropy)) & 3) return FLCE_ERR_ALIGN;
  a.lse = const_cast<float*>(lse);
  a.entropy = const_cast<float*>(entropy);
  a.g_logp = g_logp;
  a.g_entropy = g_entropy;
  return launch(p, a, true, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
