// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[n] = scale * weight[ids[n]]
//   dweight[v] (+)= scale * sum over { n : ids[n] = v }, in the order of n, of dout[n]
//
// The gradient sorts the tokens by id first: a stable radix sort with digits of at most
// 9 bits (18-bit ids: two passes), all passes in one cooperative launch of at most 64
// blocks.  The sorted order is then cut into units of 32 positions.  A warp takes 256
// (16-bit types) columns of a unit, adds the rows of each run of equal ids in fp32 and
// stores a run that lies inside the unit at once, rounded once.  A run that crosses a
// unit's border leaves its part in fp32, and a last launch joins each such run's parts in
// order.  Frequent ids (padding, the commonest words) are thus spread over many warps;
// no atomics add anything, so results do not change from run to run.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "../../include/flce.h"
#include "flce_device.cuh"
#include "flce_host.h"

namespace flce {

namespace {

constexpr int kUnit = 32;        // sorted positions per unit
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigit = 9;
constexpr int kBins = 1 << kMaxDigit;
constexpr int kSortBlocks = 64;  // every block reads every block's histogram: 64 x 2 KB
constexpr int64_t kSortChunk = 1024;

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// VEC values of T moved as one access.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC < 16 ? sizeof(T) * VEC : 16) Pack {
  T v[VEC];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float x, float& o) { o = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16& o) { o = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(float x, __half& o) { o = __float2half_rn(x); }

struct Ids {
  const void* ids;
  int ids64;
  int64_t N, V, v_offset, v_total;
  int64_t padding;  // -1: none
};

__device__ __forceinline__ int64_t load_id(const Ids& d, int64_t n) {
  return d.ids64 ? __ldg(static_cast<const long long*>(d.ids) + n)
                 : __ldg(static_cast<const int*>(d.ids) + n);
}

// ------------------------------------------------------------------ lookup
// A warp moves kFwdVecs vectors per lane of one row: with 16-byte vectors, 2 KB, loaded
// before the first is stored.
constexpr int kFwdVecs = 4;
constexpr int kFwdThreads = 256;

struct EmbedArgs {
  Ids d;
  const void* weight;
  void* out;
  int64_t H;
  float scale;
  int64_t parts;  // warps per row
  uint32_t* err;
};

template <typename T, int VEC>
__global__ void __launch_bounds__(kFwdThreads) embedding_kernel(EmbedArgs a) {
  using P = Pack<T, VEC>;
  const int64_t w = blockIdx.x * int64_t(kFwdThreads / 32) + (threadIdx.x >> 5);
  const int64_t n = w / a.parts;
  if (n >= a.d.N) return;
  const int64_t c0 = ((w - n * a.parts) * kFwdVecs * 32 + (threadIdx.x & 31)) * VEC;
  const int64_t id = load_id(a.d, n);
  const bool in = id >= 0 && id < a.d.v_total;
  const int64_t v = id - a.d.v_offset;
  const bool here = in && v >= 0 && v < a.d.V;
  P x[kFwdVecs];
  if (here) {
    const T* row = static_cast<const T*>(a.weight) + v * a.H;
#pragma unroll
    for (int k = 0; k < kFwdVecs; ++k) {
      const int64_t c = c0 + k * 32 * VEC;
      if (c < a.H) x[k] = *reinterpret_cast<const P*>(row + c);
    }
    if (a.scale != 1.0f) {
#pragma unroll
      for (int k = 0; k < kFwdVecs; ++k)
#pragma unroll
        for (int j = 0; j < VEC; ++j) from_f(to_f(x[k].v[j]) * a.scale, x[k].v[j]);
    }
  } else {
    // another shard's row is zero (the shards' sum is the lookup); an id of no row NaN
    const float fill = in ? 0.0f : __int_as_float(0x7fc00000);
#pragma unroll
    for (int k = 0; k < kFwdVecs; ++k)
#pragma unroll
      for (int j = 0; j < VEC; ++j) from_f(fill, x[k].v[j]);
    if (!in && a.err && c0 == 0) atomicOr(a.err, FLCE_DEVERR_LABEL);
  }
  T* out = static_cast<T*>(a.out) + n * a.H;
#pragma unroll
  for (int k = 0; k < kFwdVecs; ++k) {
    const int64_t c = c0 + k * 32 * VEC;
    if (c < a.H) *reinterpret_cast<P*>(out + c) = x[k];
  }
}

// ------------------------------------------------------------------ sort
struct SortArgs {
  Ids d;
  int64_t chunk;  // tokens per block, a multiple of kSortThreads
  int passes, digit;
  uint32_t *key[2], *pos[2];  // the sorted result is in [passes & 1]
  uint32_t* hist;             // [blocks][kBins]
  uint32_t* err;
};

// The sort key of token n: its row here, or V (behind every row) where it has none.
__device__ __forceinline__ uint32_t token_key(const Ids& d, int64_t n, bool* bad) {
  const int64_t id = load_id(d, n);
  *bad = id < 0 || id >= d.v_total;
  const int64_t v = id - d.v_offset;
  if (*bad || id == d.padding || v < 0 || v >= d.V) return static_cast<uint32_t>(d.V);
  return static_cast<uint32_t>(v);
}

// Ranks are stable: a warp owns consecutive tokens and goes through them 32 at a time in
// order; warps, blocks and digits follow in order by the prefix sums.
__global__ void __launch_bounds__(kSortThreads) sort_kernel(SortArgs a) {
  __shared__ uint32_t cnt[kSortWarps][kBins];
  __shared__ uint32_t base[kBins];
  __shared__ uint32_t wsum[kSortWarps];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t per_warp = a.chunk / kSortWarps;
  const int64_t n0 = blockIdx.x * a.chunk + w * per_warp;
  const int64_t n1 = n0 + per_warp < a.d.N ? n0 + per_warp : a.d.N;
  const uint32_t mask = (1u << a.digit) - 1;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.err = 0u;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.digit;
    const uint32_t* ikey = a.key[pass & 1];
    const uint32_t* ipos = a.pos[pass & 1];
    uint32_t* okey = a.key[(pass + 1) & 1];
    uint32_t* opos = a.pos[(pass + 1) & 1];
    for (int i = threadIdx.x; i < kSortWarps * kBins; i += kSortThreads) (&cnt[0][0])[i] = 0;
    __syncthreads();
    for (int64_t b = n0; b < n1; b += 32) {
      const bool have = b + lane < n1;
      bool bad = false;
      uint32_t key = 0;
      if (have) key = pass ? ikey[b + lane] : token_key(a.d, b + lane, &bad);
      const uint32_t dig = have ? (key >> shift) & mask : kBins;
      const uint32_t same = __match_any_sync(~0u, dig);
      if (have && (same & ((1u << lane) - 1)) == 0) cnt[w][dig] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    // threads are digits: the warps' counts become offsets inside the block
    uint32_t run = 0;
    for (int k = 0; k < kSortWarps; ++k) {
      const uint32_t c = cnt[k][threadIdx.x];
      cnt[k][threadIdx.x] = run;
      run += c;
    }
    uint32_t total = run, before = 0;
    if (gridDim.x > 1) {
      a.hist[blockIdx.x * kBins + threadIdx.x] = run;
      cooperative_groups::this_grid().sync();
      total = 0;
#pragma unroll 8
      for (int b = 0; b < gridDim.x; ++b) {
        const uint32_t c = a.hist[b * kBins + threadIdx.x];
        if (b < blockIdx.x) before += c;
        total += c;
      }
    }
    uint32_t incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) wsum[w] = incl;
    __syncthreads();
    uint32_t lower = 0;
    for (int k = 0; k < w; ++k) lower += wsum[k];
    base[threadIdx.x] = lower + incl - total + before;
    __syncthreads();
    for (int64_t b = n0; b < n1; b += 32) {
      const bool have = b + lane < n1;
      bool bad = false;
      uint32_t key = 0, pos = static_cast<uint32_t>(b + lane);
      if (have) {
        if (pass) {
          key = ikey[b + lane];
          pos = ipos[b + lane];
        } else {
          key = token_key(a.d, b + lane, &bad);
        }
      }
      const uint32_t dig = have ? (key >> shift) & mask : kBins;
      const uint32_t same = __match_any_sync(~0u, dig);
      const uint32_t ahead = __popc(same & ((1u << lane) - 1));
      uint32_t to = 0;
      if (have) to = base[dig] + cnt[w][dig] + ahead;
      __syncwarp();
      if (have && ahead == 0) cnt[w][dig] += __popc(same);
      __syncwarp();
      if (have) {
        okey[to] = key;
        opos[to] = pos;
      }
      // block 0 cleared the word before the histograms met
      if (bad) atomicOr(a.err, FLCE_DEVERR_LABEL);
    }
    if (pass + 1 < a.passes) {
      if (gridDim.x > 1)
        cooperative_groups::this_grid().sync();
      else
        __syncthreads();
    }
  }
}

// ------------------------------------------------------------------ sums
constexpr int kSumThreads = 128;
constexpr int kSumWarps = kSumThreads / 32;
constexpr int kFillRows = 64;  // table rows per filling block

struct SumArgs {
  const uint32_t *key, *pos;  // sorted
  int64_t N, H, V;
  const void* dout;
  void* dweight;
  float* part;  // [units][2][H]: a unit's run from the left, a run that goes on to the right
  float scale;
  int accumulate;
  int64_t units, slabs, sum_blocks;
};

template <typename TO, int VEC>
__device__ __forceinline__ void store_row(TO* p, const float (&acc)[VEC], float scale,
                                          bool accumulate) {
  using P = Pack<TO, VEC>;
  P o;
  if (accumulate) {
    const P old = *reinterpret_cast<const P*>(p);
#pragma unroll
    for (int j = 0; j < VEC; ++j) from_f(fmaf(scale, acc[j], to_f(old.v[j])), o.v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) from_f(scale * acc[j], o.v[j]);
  }
  *reinterpret_cast<P*>(p) = o;
}

// The first sorted position whose key is not below k.
__device__ __forceinline__ int64_t lower_bound(const uint32_t* key, int64_t N, uint32_t k) {
  int64_t lo = 0, n = N;
  while (n > 0) {
    const int64_t h = n / 2;
    if (key[lo + h] < k) {
      lo += h + 1;
      n -= h + 1;
    } else {
      n = h;
    }
  }
  return lo;
}

template <typename T, typename TO, int VEC>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(SumArgs a) {
  if (blockIdx.x >= a.sum_blocks) {
    // zeros for the rows of this block that no token names
    __shared__ int used[kFillRows];
    __shared__ int64_t range[2];
    const int64_t v0 = (blockIdx.x - a.sum_blocks) * int64_t(kFillRows);
    const int64_t v1 = v0 + kFillRows < a.V ? v0 + kFillRows : a.V;
    if (threadIdx.x < kFillRows) used[threadIdx.x] = 0;
    if (threadIdx.x < 2)
      range[threadIdx.x] =
          lower_bound(a.key, a.N, static_cast<uint32_t>(threadIdx.x ? v1 : v0));
    __syncthreads();
    for (int64_t i = range[0] + threadIdx.x; i < range[1]; i += kSumThreads)
      used[a.key[i] - v0] = 1;
    __syncthreads();
    Pack<TO, VEC> z;
#pragma unroll
    for (int j = 0; j < VEC; ++j) from_f(0.0f, z.v[j]);
    const int64_t vecs = a.H / VEC;
    for (int64_t r = threadIdx.x >> 5; r < v1 - v0; r += kSumWarps) {
      if (used[r]) continue;
      TO* row = static_cast<TO*>(a.dweight) + (v0 + r) * a.H;
      for (int64_t c = threadIdx.x & 31; c < vecs; c += 32)
        *reinterpret_cast<Pack<TO, VEC>*>(row + c * VEC) = z;
    }
    return;
  }
  const int64_t w = blockIdx.x * int64_t(kSumWarps) + (threadIdx.x >> 5);
  const int64_t u = w / a.slabs;
  if (u >= a.units) return;
  const int lane = threadIdx.x & 31;
  const int64_t c = ((w - u * a.slabs) * 32 + lane) * VEC;
  const int64_t s0 = u * kUnit;
  const int rows = static_cast<int>(a.N - s0 < kUnit ? a.N - s0 : kUnit);
  const uint32_t none = static_cast<uint32_t>(a.V);
  const uint32_t key = lane < rows ? a.key[s0 + lane] : none;
  const uint32_t pos = lane < rows ? a.pos[s0 + lane] : 0;
  const uint32_t left = u > 0 ? a.key[s0 - 1] : none;
  const uint32_t right = s0 + kUnit < a.N ? a.key[s0 + kUnit] : none;
  // keys rise: those of no row are at the end
  const int live = __popc(__ballot_sync(~0u, key != none));
  const bool col = c < a.H;
  const T* dout = static_cast<const T*>(a.dout) + c;
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = 0.0f;
  bool first = true;  // the unit's first run
  for (int b = 0; b < live; b += 8) {
    Pack<T, VEC> x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t n = __shfl_sync(~0u, pos, (b + k) & 31);
      if (b + k < live && col)
        x[k] = *reinterpret_cast<const Pack<T, VEC>*>(dout + int64_t(n) * a.H);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t id = __shfl_sync(~0u, key, (b + k) & 31);
      const uint32_t next = __shfl_sync(~0u, key, (b + k + 1) & 31);
      if (b + k >= live) continue;
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] += to_f(x[k].v[j]);
      const bool end = b + k + 1 == live;
      if (!end && next == id) continue;
      // the run ends here, or the unit does
      const bool from_left = first && left == id;
      const bool to_right = b + k + 1 == kUnit && right == id;
      if (col) {
        if (from_left || to_right) {
          Pack<float, VEC> o;
#pragma unroll
          for (int j = 0; j < VEC; ++j) o.v[j] = acc[j];
          *reinterpret_cast<Pack<float, VEC>*>(a.part + (2 * u + (from_left ? 0 : 1)) * a.H + c) =
              o;
        } else {
          store_row<TO, VEC>(static_cast<TO*>(a.dweight) + int64_t(id) * a.H + c, acc, a.scale,
                             a.accumulate);
        }
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] = 0.0f;
      first = false;
    }
  }
}

// ------------------------------------------------------------------ joins
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

// A block per unit; those whose last run starts there and goes on to the right add the
// run's parts: each warp a consecutive share of the units, the shares in order.
template <typename TO>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(SumArgs a) {
  __shared__ float share[kJoinWarps][32];
  __shared__ int64_t s_end;
  const int64_t u = blockIdx.x;
  const int64_t s1 = (u + 1) * kUnit;
  if (s1 >= a.N) return;
  const uint32_t id = a.key[s1 - 1];
  if (id == static_cast<uint32_t>(a.V) || a.key[s1] != id) return;
  // a run that came from the left is joined where it started
  if (a.key[s1 - kUnit] == id && u > 0 && a.key[s1 - kUnit - 1] == id) return;
  if (threadIdx.x == 0) s_end = lower_bound(a.key + s1, a.N - s1, id + 1) + s1;
  __syncthreads();
  const int64_t n = (s_end - 1) / kUnit - u;  // units after this one
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t per = (n + kJoinWarps - 1) / kJoinWarps;
  const int64_t k0 = w * per, k1 = k0 + per < n ? k0 + per : n;
  for (int64_t c = lane + blockIdx.y * 32; c - lane < a.H; c += 32 * gridDim.y) {
    float acc = 0.0f;
    if (c < a.H) {
      if (w == 0) acc = a.part[(2 * u + 1) * a.H + c];
#pragma unroll 8
      for (int64_t k = k0; k < k1; ++k) acc += a.part[2 * (u + 1 + k) * a.H + c];
    }
    share[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < a.H) {
      for (int k = 1; k < kJoinWarps; ++k) acc += share[k][lane];
      const float one[1] = {acc};
      store_row<TO, 1>(static_cast<TO*>(a.dweight) + int64_t(id) * a.H + c, one, a.scale,
                       a.accumulate);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host
int check(const flce_embedding_params* p) {
  if (!p) return FLCE_ERR_BAD_ARG;
  const int64_t lim = (int64_t(1) << 31) - 2;
  if (p->N < 0 || p->H < 1 || p->V < 1 || p->N > lim || p->H > lim || p->V > lim)
    return FLCE_ERR_BAD_SHAPE;
  if (p->N > 0 && p->H > (int64_t(1) << 46) / p->N) return FLCE_ERR_BAD_SHAPE;
  if (p->dtype < FLCE_F32 || p->dtype > FLCE_F16) return FLCE_ERR_BAD_ARG;
  if (p->grad_dtype != p->dtype && p->grad_dtype != FLCE_F32) return FLCE_ERR_BAD_ARG;
  if ((p->ids_int64 | 1) != 1 || (p->accumulate | 1) != 1) return FLCE_ERR_BAD_ARG;
  if (!std::isfinite(p->scale)) return FLCE_ERR_BAD_ARG;
  if (p->v_total < 0 || p->v_offset < 0 || (p->v_total == 0 && p->v_offset != 0))
    return FLCE_ERR_BAD_ARG;
  if (p->v_total > 0 && (p->v_total > lim || p->v_offset + p->V > p->v_total))
    return FLCE_ERR_BAD_SHAPE;
  if (p->padding_idx < -1 || p->padding_idx >= (p->v_total ? p->v_total : p->V))
    return FLCE_ERR_BAD_ARG;
  return FLCE_OK;
}

struct Layout {
  size_t key[2], pos[2], hist, part, total;
  int64_t chunk, blocks, units;
  int passes, digit;
};

Layout layout(const flce_embedding_params* p) {
  Layout L{};
  const int64_t per = cdiv(p->N, kSortBlocks);
  L.chunk = cdiv(per > kSortChunk ? per : kSortChunk, kSortThreads) * kSortThreads;
  L.blocks = p->N > 0 ? cdiv(p->N, L.chunk) : 1;
  L.units = cdiv(p->N, kUnit);
  int bits = 1;
  while ((p->V >> bits) != 0) ++bits;  // keys are 0 .. V
  L.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  L.digit = (bits + L.passes - 1) / L.passes;
  size_t off = 256;
  for (int k = 0; k < 2; ++k) {
    L.key[k] = off; off += align256(p->N * 4);
    L.pos[k] = off; off += align256(p->N * 4);
  }
  L.hist = off; off += align256(L.blocks * kBins * 4);
  L.part = off; off += align256(static_cast<size_t>(L.units) * 2 * p->H * 4);
  L.total = off;
  return L;
}

Ids make_ids(const flce_embedding_params* p, const void* ids) {
  return Ids{ids, p->ids_int64, p->N, p->V, p->v_offset, p->v_total ? p->v_total : p->V,
             p->padding_idx};
}

inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// The widest vector, in elements of the 16-bit or 32-bit type `bytes`, that rows of H
// elements and the given pointers allow.
int vec_for(int bytes, int64_t H, uintptr_t ptrs) {
  int v = 16 / bytes;
  while (v > 1 && (H % v != 0 || ptrs % (v * bytes) != 0)) v /= 2;
  return v;
}

inline int rc_of(cudaError_t e) { return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA; }

template <typename T, int VEC>
int launch_lookup(EmbedArgs a, cudaStream_t st) {
  a.parts = cdiv(a.H, int64_t(32) * VEC * kFwdVecs);
  const int64_t blocks = cdiv(a.d.N * a.parts, kFwdThreads / 32);
  if (blocks > (int64_t(1) << 31) - 1) return FLCE_ERR_BAD_SHAPE;
  embedding_kernel<T, VEC><<<static_cast<unsigned>(blocks), kFwdThreads, 0, st>>>(a);
  return rc_of(cudaGetLastError());
}

template <typename T>
int launch_lookup_vec(const EmbedArgs& a, int vec, cudaStream_t st) {
  if constexpr (sizeof(T) == 2)
    if (vec == 8) return launch_lookup<T, 8>(a, st);
  if (vec == 4) return launch_lookup<T, 4>(a, st);
  if (vec == 2) return launch_lookup<T, 2>(a, st);
  return launch_lookup<T, 1>(a, st);
}

template <typename T, typename TO, int VEC>
int launch_sum(SumArgs a, cudaStream_t st) {
  a.slabs = cdiv(a.H, 32 * VEC);
  a.sum_blocks = cdiv(a.units * a.slabs, kSumWarps);
  const int64_t blocks = a.sum_blocks + (a.accumulate ? 0 : cdiv(a.V, kFillRows));
  if (blocks > (int64_t(1) << 31) - 1) return FLCE_ERR_BAD_SHAPE;
  if (blocks == 0) return FLCE_OK;  // no token, nothing to add
  sum_kernel<T, TO, VEC><<<static_cast<unsigned>(blocks), kSumThreads, 0, st>>>(a);
  int rc = rc_of(cudaGetLastError());
  if (rc || a.units < 2) return rc;
  const int64_t y = cdiv(a.H, 32);
  join_kernel<TO><<<dim3(static_cast<unsigned>(a.units), static_cast<unsigned>(y < 16 ? y : 16)),
                    kJoinThreads, 0, st>>>(a);
  return rc_of(cudaGetLastError());
}

template <typename T, typename TO>
int launch_sum_vec(const SumArgs& a, int vec, cudaStream_t st) {
  if constexpr (sizeof(T) == 2)
    if (vec == 8) return launch_sum<T, TO, 8>(a, st);
  if (vec == 4) return launch_sum<T, TO, 4>(a, st);
  if (vec == 2) return launch_sum<T, TO, 2>(a, st);
  return launch_sum<T, TO, 1>(a, st);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_embedding_check_params(const flce_embedding_params* p) { return check(p); }

size_t flce_embedding_workspace_size(const flce_embedding_params* p) {
  return check(p) == FLCE_OK ? layout(p).total : 0;
}

int flce_embedding(const flce_embedding_params* p, const void* ids, const void* weight, void* out,
                   void* workspace, size_t ws_bytes, void* stream) {
  int rc = check(p);
  if (rc) return rc;
  if (p->N > 0 && (!ids || !weight || !out)) return FLCE_ERR_BAD_ARG;
  if (p->validate && !workspace) return FLCE_ERR_BAD_ARG;
  const int b = p->dtype == FLCE_F32 ? 4 : 2;
  if ((addr(weight) | addr(out)) & (b - 1) || addr(ids) & (p->ids_int64 ? 7 : 3) ||
      addr(workspace) & 255)
    return FLCE_ERR_ALIGN;
  if (p->validate && ws_bytes < 256) return FLCE_ERR_WS_TOO_SMALL;
  int sms;
  if ((rc = require_device(&sms))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  EmbedArgs a{};
  a.d = make_ids(p, ids);
  a.weight = weight;
  a.out = out;
  a.H = p->H;
  a.scale = static_cast<float>(p->scale);
  if (p->validate) {
    a.err = static_cast<uint32_t*>(workspace);
    if ((rc = rc_of(cudaMemsetAsync(workspace, 0, 256, st)))) return rc;
  }
  if (p->N > 0) {
    const int vec = vec_for(b, p->H, addr(weight) | addr(out));
    rc = p->dtype == FLCE_F32    ? launch_lookup_vec<float>(a, vec, st)
         : p->dtype == FLCE_BF16 ? launch_lookup_vec<__nv_bfloat16>(a, vec, st)
                                 : launch_lookup_vec<__half>(a, vec, st);
    if (rc) return rc;
  }
  return p->validate ? read_status(workspace, st) : FLCE_OK;
}

int flce_embedding_backward(const flce_embedding_params* p, const void* dout, const void* ids,
                            void* dweight, void* workspace, size_t ws_bytes, void* stream) {
  int rc = check(p);
  if (rc) return rc;
  if (!dweight || !workspace || (p->N > 0 && (!ids || !dout))) return FLCE_ERR_BAD_ARG;
  const int b = p->dtype == FLCE_F32 ? 4 : 2, gb = p->grad_dtype == FLCE_F32 ? 4 : 2;
  if (addr(dout) & (b - 1) || addr(dweight) & (gb - 1) || addr(ids) & (p->ids_int64 ? 7 : 3) ||
      addr(workspace) & 255)
    return FLCE_ERR_ALIGN;
  const Layout L = layout(p);
  if (ws_bytes < L.total) return FLCE_ERR_WS_TOO_SMALL;
  int sms;
  if ((rc = require_device(&sms))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SortArgs s{};
  s.d = make_ids(p, ids);
  s.chunk = L.chunk;
  s.passes = L.passes;
  s.digit = L.digit;
  for (int k = 0; k < 2; ++k) {
    s.key[k] = reinterpret_cast<uint32_t*>(ws + L.key[k]);
    s.pos[k] = reinterpret_cast<uint32_t*>(ws + L.pos[k]);
  }
  s.hist = reinterpret_cast<uint32_t*>(ws + L.hist);
  s.err = reinterpret_cast<uint32_t*>(ws);
  void* params[] = {&s};
  const void* sort = reinterpret_cast<const void*>(sort_kernel);
  const dim3 grid(static_cast<unsigned>(L.blocks)), block(kSortThreads);
  rc = rc_of(L.blocks == 1 ? cudaLaunchKernel(sort, grid, block, params, 0, st)
                           : cudaLaunchCooperativeKernel(sort, grid, block, params, 0, st));
  if (rc) return rc;
  SumArgs a{};
  a.key = s.key[L.passes & 1];
  a.pos = s.pos[L.passes & 1];
  a.N = p->N;
  a.H = p->H;
  a.V = p->V;
  a.dout = dout;
  a.dweight = dweight;
  a.part = reinterpret_cast<float*>(ws + L.part);
  a.scale = static_cast<float>(p->scale);
  a.accumulate = p->accumulate;
  a.units = L.units;
  // a fp32 gradient of 16-bit rows is stored in 16-byte halves of a vector
  const int align_to = gb > b ? 16 : 16 / b * gb;
  int vec = vec_for(b, p->H, addr(dout));
  while (vec > 1 && addr(dweight) % (vec * gb < align_to ? vec * gb : align_to) != 0) vec /= 2;
  if (p->dtype == FLCE_F32)
    rc = launch_sum_vec<float, float>(a, vec, st);
  else if (p->dtype == FLCE_BF16)
    rc = gb == 4 ? launch_sum_vec<__nv_bfloat16, float>(a, vec, st)
                 : launch_sum_vec<__nv_bfloat16, __nv_bfloat16>(a, vec, st);
  else
    rc = gb == 4 ? launch_sum_vec<__half, float>(a, vec, st)
                 : launch_sum_vec<__half, __half>(a, vec, st);
  if (rc) return rc;
  return p->validate ? read_status(workspace, st) : FLCE_OK;
}

}  // extern "C"
