// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[n] = scale * weight[ids[n]]
//   dweight[v] (+)= scale * sum over { n : ids[n] = v } of dout[n]
//
// The gradient sorts the tokens by id first: a stable radix sort with digits of at most
// 9 bits (18-bit ids: two passes), all passes in one launch: one block up to 512 tokens, a
// cluster of at most eight up to 16384, a cooperative grid of at most 64 beyond.  The
// sorted order is then cut into units of 32 positions.  A warp takes 256 (16-bit types)
// columns of a unit, adds the rows of each run of equal ids in fp32 and stores a run that
// lies inside the unit at once, rounded once.  A run that crosses a unit's border leaves
// its part in fp32, and a last launch joins each such run's parts in order.  Frequent ids
// (padding, the commonest words) are thus spread over many warps; no atomics add anything,
// so results do not change from run to run: rows are added in the order of n inside a unit, and
// the units' sums in order (those of a run over more than nine units in 32 groups first).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "../../include/flce.h"
#include "flce_device.cuh"
#include "flce_host.h"
#include "flce_seq.cuh"

namespace flce {

namespace {

constexpr int kUnit = 32;        // sorted positions per unit
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigit = 9;
constexpr int kBins = 1 << kMaxDigit;
constexpr int kSortBlocks = 64;  // every block reads every block's histogram: 64 x 2 KB
// A cluster's eight blocks meet in a fraction of a grid's time, a grid has more SMs: the
// gradient of 8192 tokens took 33.0 us with the one and 34.3 with the other, that of 32768
// tokens 48.5 and 44.1.
constexpr int64_t kSortSmall = 16384;
constexpr int kSortBatch = 4;    // a lane's tokens that are loaded together
constexpr int64_t kSortChunk = kSortThreads;  // a block has as many tokens at least

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// VEC values of T moved as one access.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC < 16 ? sizeof(T) * VEC : 16) Pack {
  T v[VEC];
};

// First to leave L2: rows that are written once push out no others.  The lookup of 16384
// rows of 7 KB takes 27.6 us with such stores and 32.7 without.
template <typename P>
__device__ __forceinline__ void store_stream(P* to, const P& x) {
  if constexpr (sizeof(P) >= 16) {
#pragma unroll
    for (int k = 0; k < static_cast<int>(sizeof(P) / 16); ++k)
      __stcs(reinterpret_cast<uint4*>(to) + k, reinterpret_cast<const uint4*>(&x)[k]);
  } else {
    *to = x;
  }
}

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
constexpr int kFwdThreads = 128;

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
    if (c < a.H) store_stream(reinterpret_cast<P*>(out + c), x[k]);
  }
}

// The gradient's three launches follow each other by programmatic dependence: the blocks
// of the next are placed as soon as all of this one's run, and wait for its end there.
__device__ __forceinline__ void next_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_launch() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------ sort
struct SortArgs {
  Ids d;
  int64_t chunk;  // tokens per block, a multiple of kSortThreads
  int passes, digit;
  uint2 *kp0, *kp1;  // (key, token), the sorted result in [passes & 1]
  int meet;
  uint32_t* hist;   // [blocks][kBins]
  uint32_t* lists;  // the join's two counts, cleared here
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
  __shared__ uint32_t mine[kBins];  // this block's histogram
  __shared__ uint32_t base[kBins];
  __shared__ uint32_t wsum[kSortWarps];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t lower_lanes = (1u << lane) - 1;
  const int64_t per_warp = a.chunk / kSortWarps;
  const int64_t n0 = blockIdx.x * a.chunk + w * per_warp;
  const int64_t n1 = n0 + per_warp < a.d.N ? n0 + per_warp : a.d.N;
  const bool one_batch = per_warp <= 32 * kSortBatch;
  const uint32_t mask = (1u << a.digit) - 1;
  next_launch();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *a.err = 0u;
    a.lists[0] = a.lists[1] = 0u;
  }
  bool bad = false;
#pragma unroll 1
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.digit;
    const uint2* in = pass & 1 ? a.kp1 : a.kp0;
    // key and token as one store: the scattered stores are what the placing waits for
    uint2* out = pass & 1 ? a.kp0 : a.kp1;
    for (int i = threadIdx.x; i < kSortWarps * kBins / 4; i += kSortThreads)
      reinterpret_cast<uint4*>(&cnt[0][0])[i] = make_uint4(0, 0, 0, 0);
    uint32_t key[kSortBatch], pos[kSortBatch];
    __syncthreads();
    // twice over the warp's tokens: their digits' counts, then, with every count known,
    // their places
#pragma unroll 1
    for (int place = 0; place < 2; ++place) {
#pragma unroll 1
      for (int64_t b = n0; b < n1; b += 32 * kSortBatch) {
        if (!(place && one_batch)) {
#pragma unroll
          for (int k = 0; k < kSortBatch; ++k) {
            const int64_t n = b + 32 * k + lane;
            key[k] = 0;
            pos[k] = static_cast<uint32_t>(n);
            if (n < n1) {
              if (pass == 0) {
                bool none;
                key[k] = token_key(a.d, n, &none);
                bad |= none;
              } else {
                const uint2 x = in[n];
                key[k] = x.x;
                pos[k] = x.y;
              }
            }
          }
        }
#pragma unroll
        for (int k = 0; k < kSortBatch; ++k) {
          if (b + 32 * k >= n1) break;
          const bool have = b + 32 * k + lane < n1;
          const uint32_t dig = (key[k] >> shift) & mask;
          if (!place) {
            if (have) atomicAdd(&cnt[w][dig], 1u);
            continue;
          }
          // the lanes with this digit, bit by bit (a little faster than __match_any_sync:
          // the sort of 16384 tokens took 15 us instead of 17)
          uint32_t same = __ballot_sync(~0u, have);
#pragma unroll
          for (int i = 0; i < kMaxDigit; ++i) {
            const uint32_t ones = __ballot_sync(~0u, dig >> i & 1);
            same &= dig >> i & 1 ? ones : ~ones;
          }
          const uint32_t ahead = __popc(same & lower_lanes);
          if (have) {
            const uint32_t to = base[dig] + cnt[w][dig] + ahead;
            out[to] = make_uint2(key[k], pos[k]);
          }
          __syncwarp();
          if (have && ahead == 0) cnt[w][dig] += __popc(same);
          __syncwarp();
        }
      }
      if (place) break;
      __syncthreads();
      // threads are digits: the warps' counts become offsets inside the block
      uint32_t run = 0;
#pragma unroll
      for (int k = 0; k < kSortWarps; ++k) {
        const uint32_t c = cnt[k][threadIdx.x];
        cnt[k][threadIdx.x] = run;
        run += c;
      }
      uint32_t total = run, before = 0;
      if (a.meet != MEET_BLOCK) {
        if (a.meet == MEET_CLUSTER)
          mine[threadIdx.x] = run;
        else
          a.hist[blockIdx.x * kBins + threadIdx.x] = run;
        meet(a.meet);
        total = 0;
#pragma unroll 8
        for (int b = 0; b < gridDim.x; ++b) {
          const uint32_t c =
              a.meet == MEET_CLUSTER
                  ? cooperative_groups::this_cluster().map_shared_rank(mine, b)[threadIdx.x]
                  : a.hist[b * kBins + threadIdx.x];
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
      const uint32_t lower = __reduce_add_sync(~0u, lane < w ? wsum[lane] : 0u);  // 16 warps
      base[threadIdx.x] = lower + incl - total + before;
      __syncthreads();
    }
    // also before the end: a block's shared memory may still be read by its cluster
    if (pass + 1 < a.passes || a.meet == MEET_CLUSTER) meet(a.meet);
  }
  // block 0 cleared the word before the histograms met
  if (bad) atomicOr(a.err, FLCE_DEVERR_LABEL);
}

// ------------------------------------------------------------------ sums
constexpr int kSumThreads = 128;
constexpr int kSumWarps = kSumThreads / 32;
constexpr int kFillRows = 64;  // table rows per filling block
constexpr int kRing = 16;      // rows of a warp's slab in flight or in use
constexpr int kGroup = 4;      // rows per asynchronous copy group
// Units beyond its head from which a block joins a run, not a warp: with 2, 8 and 30 the
// gradient of 65536 tokens of 4096 columns took 198, 187 and 189 us, of 16384 45.8, 43.6, 45.3.
constexpr int kLong = 8;

struct SumArgs {
  const uint2* kp;  // sorted (key, token)
  int64_t N, H, V;
  const void* dout;
  void* dweight;
  float* part;  // [units][2][H]: a unit's run from the left, a run that goes on to the right
  uint4* jobs[2];  // runs to join, (head's unit, slab, row, units after it): short, long
  uint32_t* lists;    // their numbers
  float scale;
  int accumulate;
  int64_t units, slabs, sum_blocks;
};

template <typename TO, int VEC>
__device__ __forceinline__ void store_row(TO* p, const float (&acc)[VEC],
                                          const Pack<TO, VEC>& old, float scale,
                                          bool accumulate) {
  using P = Pack<TO, VEC>;
  P o;
  if (accumulate) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) from_f(fmaf(scale, acc[j], to_f(old.v[j])), o.v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) from_f(scale * acc[j], o.v[j]);
  }
  *reinterpret_cast<P*>(p) = o;
}

// Copies one lane's vector to shared memory: asynchronously where the hardware does (4, 8
// and 16 bytes), else at once.
template <typename P>
__device__ __forceinline__ void copy_vec(P* to, const P* from) {
  if constexpr (sizeof(P) < 4) {
    *to = *from;
  } else {
    constexpr int step = sizeof(P) < 16 ? sizeof(P) : 16;
#pragma unroll
    for (int o = 0; o < static_cast<int>(sizeof(P)); o += step) {
      const uint32_t dst = smem_u32(to) + o;
      const char* src = reinterpret_cast<const char*>(from) + o;
      if constexpr (step == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(step)
                     : "memory");
    }
  }
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The first sorted position whose key is not below k.
__device__ __forceinline__ int64_t lower_bound(const uint2* kp, int64_t N, uint32_t k) {
  int64_t lo = 0, n = N;
  while (n > 0) {
    const int64_t h = n / 2;
    if (kp[lo + h].x < k) {
      lo += h + 1;
      n -= h + 1;
    } else {
      n = h;
    }
  }
  return lo;
}

// What a unit's warps need to know of its 32 positions.
struct Unit {
  uint32_t key, pos;  // this lane's
  int live;           // positions with a row (they come first: keys rise)
  uint32_t ends;      // positions that end a run, or the unit
  uint32_t whole;     // those of runs that lie inside the unit
  bool from_left, to_right;
};

// How many units after unit u begin with `id` (whole warp); a run's are consecutive.  First
// powers of two, then 32 places of what is left at a time.
__device__ __forceinline__ uint32_t units_after(const SumArgs& a, int64_t u, uint32_t id) {
  const int lane = threadIdx.x & 31;
  auto begins = [&](int64_t k) {
    const int64_t s = (u + k) * kUnit;
    return s < a.N && a.kp[s].x == id;
  };
  uint32_t hits = __ballot_sync(~0u, begins(int64_t(1) << lane));
  hits = __popc(hits & ~(hits + 1));  // from the first on
  if (hits == 0) return 0;
  int64_t lo = int64_t(1) << (hits - 1), n = lo - 1;  // lo begins so; n more may
  while (n > 0) {
    const int64_t step = (n + 31) / 32;
    const int64_t k = (lane + 1) * step;
    const int more = __popc(__ballot_sync(~0u, k <= n && begins(lo + k)));
    const int64_t left = n - more * step;
    lo += more * step;
    n = left < step - 1 ? left : step - 1;
  }
  return static_cast<uint32_t>(lo);
}

__device__ __forceinline__ Unit load_unit(const SumArgs& a, int64_t u) {
  const int lane = threadIdx.x & 31;
  const int64_t s0 = u * kUnit;
  const uint32_t none = static_cast<uint32_t>(a.V);
  Unit t;
  const uint2 kp = s0 + lane < a.N ? a.kp[s0 + lane] : make_uint2(none, 0);
  const uint32_t left = u > 0 ? a.kp[s0 - 1].x : none;
  const uint32_t right = s0 + kUnit < a.N ? a.kp[s0 + kUnit].x : none;
  t.key = kp.x;
  t.pos = kp.y;
  t.live = __popc(__ballot_sync(~0u, t.key != none));
  const uint32_t next = __shfl_down_sync(~0u, t.key, 1);
  t.ends = __ballot_sync(~0u, lane < t.live && (lane + 1 == t.live || next != t.key));
  t.from_left = t.live > 0 && left == __shfl_sync(~0u, t.key, 0);
  t.to_right = t.live == kUnit && right == __shfl_sync(~0u, t.key, kUnit - 1);
  t.whole = t.ends;
  if (t.from_left) t.whole &= t.whole - 1;  // the first run's end
  if (t.to_right) t.whole &= ~(1u << (kUnit - 1));
  return t;
}

// The rows pass through a ring of shared memory that each warp fills for itself, twelve to
// sixteen rows ahead: the copies in flight need no registers, and the loop over the rows
// stays short (unrolled over rows in registers it took 44 us where this one takes 30, a
// launch's instructions being fetched cold by every SM at once).
template <typename T, typename TO, int VEC>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(SumArgs a) {
  extern __shared__ __align__(16) unsigned char ring_bytes[];
  next_launch();
  wait_launch();
  if (blockIdx.x >= a.sum_blocks) {
    // zeros for the rows of this block that no token names
    __shared__ int used[kFillRows];
    __shared__ int64_t range[2];
    const int64_t v0 = (blockIdx.x - a.sum_blocks) * int64_t(kFillRows);
    const int64_t v1 = v0 + kFillRows < a.V ? v0 + kFillRows : a.V;
    if (threadIdx.x < kFillRows) used[threadIdx.x] = 0;
    if (threadIdx.x < 2)
      range[threadIdx.x] =
          lower_bound(a.kp, a.N, static_cast<uint32_t>(threadIdx.x ? v1 : v0));
    __syncthreads();
    for (int64_t i = range[0] + threadIdx.x; i < range[1]; i += kSumThreads)
      used[a.kp[i].x - v0] = 1;
    __syncthreads();
    Pack<TO, VEC> z;
#pragma unroll
    for (int j = 0; j < VEC; ++j) from_f(0.0f, z.v[j]);
    const int64_t vecs = a.H / VEC;
    for (int64_t r = threadIdx.x >> 5; r < v1 - v0; r += kSumWarps) {
      if (used[r]) continue;
      TO* row = static_cast<TO*>(a.dweight) + (v0 + r) * a.H;
      for (int64_t c = threadIdx.x & 31; c < vecs; c += 32)
        store_stream(reinterpret_cast<Pack<TO, VEC>*>(row + c * VEC), z);
    }
    return;
  }
  using PT = Pack<T, VEC>;
  using PO = Pack<TO, VEC>;
  const int64_t w = blockIdx.x * int64_t(kSumWarps) + (threadIdx.x >> 5);
  const int64_t u = w / a.slabs;
  if (u >= a.units) return;
  const int lane = threadIdx.x & 31;
  const int64_t c = ((w - u * a.slabs) * 32 + lane) * VEC;
  const bool col = c < a.H;
  const Unit t = load_unit(a, u);
  const char* dout = reinterpret_cast<const char*>(static_cast<const T*>(a.dout) + c);
  char* dweight = reinterpret_cast<char*>(static_cast<TO*>(a.dweight) + c);
  const uint32_t row_bytes = static_cast<uint32_t>(a.H * sizeof(T));
  const uint32_t out_bytes = static_cast<uint32_t>(a.H * sizeof(TO));
  PT* rows = reinterpret_cast<PT*>(ring_bytes) + (threadIdx.x >> 5) * kRing * 32 + lane;
  PO* olds = reinterpret_cast<PO*>(ring_bytes + sizeof(PT) * kSumThreads * kRing) +
             (threadIdx.x >> 5) * kRing * 32 + lane;
  // positions whose rows this lane copies; and whose old rows
  const uint32_t want = !col ? 0u : t.live == kUnit ? ~0u : (1u << t.live) - 1;
  const uint32_t want_old = a.accumulate ? want & t.whole : 0u;
  auto fetch = [&](int g) {
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      const int j = g * kGroup + k;  // past the unit's end: nothing wanted
      if (j >= kUnit) break;
      const uint32_t n = __shfl_sync(~0u, t.pos, j);
      const uint32_t id = __shfl_sync(~0u, t.key, j);
      const int slot = (j & (kRing - 1)) * 32;
      if (want >> j & 1)
        copy_vec(rows + slot, reinterpret_cast<const PT*>(dout + uint64_t(n) * row_bytes));
      if (want_old >> j & 1)
        copy_vec(olds + slot, reinterpret_cast<const PO*>(dweight + uint64_t(id) * out_bytes));
    }
    copy_commit();
  };
#pragma unroll 1
  for (int g = 0; g < kRing / kGroup; ++g) fetch(g);
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = 0.0f;
  int side = t.from_left ? 0 : 1;  // of a part, until the first run has ended
  uint32_t ends = t.ends;
#pragma unroll 1
  for (int g = 0; g * kGroup < t.live; ++g, ends >>= kGroup) {
    copy_wait<kRing / kGroup - 1>();  // lanes read back what they copied themselves
    const PT* in = rows + (g * kGroup & (kRing - 1)) * 32;
    const int count = t.live - g * kGroup < kGroup ? t.live - g * kGroup : kGroup;
#pragma unroll 1
    for (int k = 0; k < count; ++k) {
      const PT x = in[k * 32];
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += to_f(x.v[i]);
      if (!(ends >> k & 1)) continue;
      const int j = g * kGroup + k;
      const uint32_t id = __shfl_sync(~0u, t.key, j);
      if (col) {
        if (t.whole >> j & 1) {
          store_row<TO, VEC>(reinterpret_cast<TO*>(dweight + uint64_t(id) * out_bytes), acc,
                             olds[(j & (kRing - 1)) * 32], a.scale, a.accumulate);
        } else {
          Pack<float, VEC> o;
#pragma unroll
          for (int i = 0; i < VEC; ++i) o.v[i] = acc[i];
          *reinterpret_cast<Pack<float, VEC>*>(a.part + (2 * u + side) * a.H + c) = o;
        }
      }
      side = 1;
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
    }
    fetch(g + kRing / kGroup);
  }
  // the head of a run that goes on: a job for the join
  if (t.to_right && !(t.from_left && t.ends == 1u << (kUnit - 1))) {
    const uint32_t id = __shfl_sync(~0u, t.key, kUnit - 1);
    const uint32_t n = units_after(a, u, id);
    if (lane == 0) {
      const bool is_long = n > kLong;
      uint4* jobs = is_long ? a.jobs[1] : a.jobs[0];
      jobs[atomicAdd(a.lists + is_long, 1u)] =
          make_uint4(static_cast<uint32_t>(u), static_cast<uint32_t>(w - u * a.slabs), id, n);
    }
  }
}

// ------------------------------------------------------------------ joins
constexpr int kJoinThreads = 1024;
constexpr int kJoinWarps = kJoinThreads / 32;

// Adds up the parts of the runs that cross units.  Their number is known on the GPU alone:
// the grid is fixed and strides over the two lists, a block per long run's slab (each warp
// takes consecutive units, and their sums follow in order), a warp per short one's.  The
// lists' order changes from run to run; nothing depends on it.
template <typename TO, int VEC>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(SumArgs a) {
  using PF = Pack<float, VEC>;
  using PO = Pack<TO, VEC>;
  __shared__ PF share[kJoinWarps][32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_launch();
  // a block's jobs: a long run's slab, or a short one's for each warp
  const uint32_t n_short = a.lists[0], n_long = a.lists[1];
  const uint32_t items = n_long + (n_short + kJoinWarps - 1) / kJoinWarps;
#pragma unroll 1
  for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
    const bool list = item < n_long;
    const uint32_t k = list ? item : (item - n_long) * kJoinWarps + w;
    if (list || k < n_short) {
      const uint4 job = list ? a.jobs[1][k] : a.jobs[0][k];
      const int64_t u = job.x, n = job.w;
      const int64_t c = (int64_t(job.y) * 32 + lane) * VEC;
      const uint32_t id = job.z;
      const int64_t per = list ? (n + kJoinWarps - 1) / kJoinWarps : n;
      const int64_t k0 = list ? w * per : 0, k1 = k0 + per < n ? k0 + per : n;
      const bool head = !list || w == 0;
      float acc[VEC];
      PO old{};
      TO* row = static_cast<TO*>(a.dweight) + int64_t(id) * a.H + c;
      const float* part = a.part + 2 * u * a.H + c;
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] = 0.0f;
      if (c < a.H) {
        if (head && a.accumulate) old = *reinterpret_cast<const PO*>(row);
        if (head) {
          const PF x = *reinterpret_cast<const PF*>(part + a.H);
#pragma unroll
          for (int j = 0; j < VEC; ++j) acc[j] = x.v[j];
        }
#pragma unroll 4
        for (int64_t i = k0; i < k1; ++i) {
          const PF x = *reinterpret_cast<const PF*>(part + 2 * (i + 1) * a.H);
#pragma unroll
          for (int j = 0; j < VEC; ++j) acc[j] += x.v[j];
        }
      }
      if (list) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) share[w][lane].v[j] = acc[j];
        __syncthreads();
        if (w == 0) {
#pragma unroll 1
          for (int i = 1; i < kJoinWarps; ++i) {
            const PF x = share[i][lane];
#pragma unroll
            for (int j = 0; j < VEC; ++j) acc[j] += x.v[j];
          }
        }
        __syncthreads();
      }
      if (head && c < a.H) store_row<TO, VEC>(row, acc, old, a.scale, a.accumulate);
    }
  }
}

// ------------------------------------------------------------------ host
int check(const flce_embedding_params* p) {
  if (!p) return FLCE_ERR_BAD_ARG;
  const int64_t lim = (int64_t(1) << 31) - 2;
  if (p->N < 0 || p->H < 1 || p->V < 1 || p->N > lim || p->H > lim || p->V > lim)
    return FLCE_ERR_BAD_SHAPE;
  if (p->H > (int64_t(1) << 28)) return FLCE_ERR_BAD_SHAPE;  // a row's bytes are 32-bit
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
  size_t kp[2], hist, jobs[2], part, total;
  int64_t chunk, blocks, units;
  int passes, digit, meet;
};

Layout layout(const flce_embedding_params* p) {
  Layout L{};
  const int64_t per = cdiv(p->N, p->N <= kSortSmall ? kClusterBlocks : kSortBlocks);
  L.chunk = cdiv(per > kSortChunk ? per : kSortChunk, kSortThreads) * kSortThreads;
  L.blocks = p->N > 0 ? cdiv(p->N, L.chunk) : 1;
  L.meet = L.blocks == 1 ? MEET_BLOCK : p->N <= kSortSmall ? MEET_CLUSTER : MEET_GRID;
  if (L.meet == MEET_CLUSTER) L.blocks = L.blocks <= 2 ? 2 : L.blocks <= 4 ? 4 : 8;
  L.units = cdiv(p->N, kUnit);
  int bits = 1;
  while ((p->V >> bits) != 0) ++bits;  // keys are 0 .. V
  L.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  L.digit = (bits + L.passes - 1) / L.passes;
  size_t off = 256;
  for (int k = 0; k < 2; ++k) {
    L.kp[k] = off; off += align256(p->N * 8);
  }
  L.hist = off; off += align256(L.blocks * kBins * 4);
  // a unit has one run at most that goes on; the most slabs are those of 32 columns
  for (int k = 0; k < 2; ++k) {
    L.jobs[k] = off; off += align256(static_cast<size_t>(L.units) * cdiv(p->H, 32) * 16);
  }
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

inline int rc_of(cudaError_t e) {
  if (e == cudaSuccess) return FLCE_OK;
  cudaGetLastError();  // reported here, not by a later call
  return FLCE_ERR_CUDA;
}

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

// A launch that waits for the one before it on the GPU (wait_launch).
int launch_next(void (*kernel)(SumArgs), const SumArgs& a, int64_t blocks, int threads, int smem,
                cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  SumArgs copy = a;
  void* params[] = {&copy};
  return rc_of(cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), params));
}

template <typename T, typename TO, int VEC>
int launch_sum(SumArgs a, int sms, cudaStream_t st) {
  a.slabs = cdiv(a.H, 32 * VEC);
  a.sum_blocks = cdiv(a.units * a.slabs, kSumWarps);
  const int64_t blocks = a.sum_blocks + (a.accumulate ? 0 : cdiv(a.V, kFillRows));
  if (blocks > (int64_t(1) << 31) - 1) return FLCE_ERR_BAD_SHAPE;
  if (blocks == 0) return FLCE_OK;  // no token, nothing to add
  // the rows' ring, and the old rows' where there are any
  const int ring = kSumThreads * kRing *
                   static_cast<int>(sizeof(Pack<T, VEC>) +
                                    (a.accumulate ? sizeof(Pack<TO, VEC>) : 0));
  if (ring > 47 * 1024) {  // beside the static 272 bytes
    const int rc = rc_of(cudaFuncSetAttribute(
        sum_kernel<T, TO, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, ring));
    if (rc) return rc;
  }
  int rc = launch_next(sum_kernel<T, TO, VEC>, a, blocks, kSumThreads, ring, st);
  if (rc || a.units < 2) return rc;
  const int64_t join = cdiv(a.units * a.slabs, kJoinWarps), cap = sms;
  return launch_next(join_kernel<TO, VEC>, a, join < cap ? join : cap, kJoinThreads, 0, st);
}

template <typename T, typename TO>
int launch_sum_vec(const SumArgs& a, int vec, int sms, cudaStream_t st) {
  if constexpr (sizeof(T) == 2)
    if (vec == 8) return launch_sum<T, TO, 8>(a, sms, st);
  if (vec == 4) return launch_sum<T, TO, 4>(a, sms, st);
  if (vec == 2) return launch_sum<T, TO, 2>(a, sms, st);
  return launch_sum<T, TO, 1>(a, sms, st);
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
  s.meet = L.meet;
  s.kp0 = reinterpret_cast<uint2*>(ws + L.kp[0]);
  s.kp1 = reinterpret_cast<uint2*>(ws + L.kp[1]);
  s.lists = reinterpret_cast<uint32_t*>(ws + 64);
  s.hist = reinterpret_cast<uint32_t*>(ws + L.hist);
  s.err = reinterpret_cast<uint32_t*>(ws);
  if ((rc = rc_of(launch_meeting(reinterpret_cast<const void*>(sort_kernel), &s, L.blocks,
                                 kSortThreads, L.meet, st))))
    return rc;
  SumArgs a{};
  a.kp = L.passes & 1 ? s.kp1 : s.kp0;
  a.lists = s.lists;
  for (int k = 0; k < 2; ++k) a.jobs[k] = reinterpret_cast<uint4*>(ws + L.jobs[k]);
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
    rc = launch_sum_vec<float, float>(a, vec, sms, st);
  else if (p->dtype == FLCE_BF16)
    rc = gb == 4 ? launch_sum_vec<__nv_bfloat16, float>(a, vec, sms, st)
                 : launch_sum_vec<__nv_bfloat16, __nv_bfloat16>(a, vec, sms, st);
  else
    rc = gb == 4 ? launch_sum_vec<__half, float>(a, vec, sms, st)
                 : launch_sum_vec<__half, __half>(a, vec, sms, st);
  if (rc) return rc;
  return p->validate ? read_status(workspace, st) : FLCE_OK;
}

}  // extern "C"
