// Preference loss over pairs of sequences, and its gradient.
//
// Sequence i scores s_i = sum_t (lp_t - ref_t) over its counted tokens (divided by their
// number where lengths are normalised); a pair of a chosen c and a rejected sequence r has
//   h = beta (s_c - s_r) - margin
//   sigmoid  -(1 - e) ln sig(h) - e ln sig(-h)          (e: label smoothing)
//   robust   (-(1 - e) ln sig(h) + e ln sig(-h)) / (1 - 2e)
//   hinge    max(0, 1 - h)
//   ipo      (h / beta - 1 / (2 beta))^2
// plus nll_coef times the chosen side's mean negative log-likelihood.  A pair with a side
// of which nothing counts is left out.  The gradient of a counted token is its sequence's
// coefficient.
//
// One launch: sums of the pieces; a warp per pair (a block, where they are few and long), which
// adds its two sequences' pieces in a fixed order in pairs of floats; the number of pairs by
// atomics; the loss and the gradients.  The gradient pass reads only the mask.  256 packed pairs
// of 1M tokens take 16.4 us, of which the bytes need 2: two meetings and three memory latencies.
#include <cmath>

#include "flce_device.cuh"
#include "flce_host.h"
#include "flce_seq.cuh"

namespace flce {

namespace {

struct PrefPiece {
  Pair score, like;  // a score meets reference scores of its size: every digit counts
  int n;
  int pad;
};

struct PrefArgs {
  Seqs q;
  const void *lp, *ref;
  int64_t lp_skip, ref_skip;
  const float* ref_scores;
  float beta, margin, smooth, nll;
  int kind, norm, interleaved, reduction, want_loss;
  const float* g_loss;
  float *loss, *rewards;
  void* dlp;
  uint32_t* err;
  SeqTotals* totals;
  PrefPiece* piece;
  float* coef;       // [B] gradient of the pair's own loss by a token of sequence i
  float* pair_loss;  // [B / 2]
};

__device__ __forceinline__ float softplus(float x) {  // ln(1 + e^x)
  return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x)));
}
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// The pair's loss and its derivative by h.
__device__ void pair_value(const PrefArgs& a, float h, float& l, float& dh) {
  const float e = a.smooth;
  switch (a.kind) {
    case FLCE_PREF_SIGMOID:
      l = (1.0f - e) * softplus(-h) + e * softplus(h);
      dh = -(1.0f - e) * sigmoid(-h) + e * sigmoid(h);
      break;
    case FLCE_PREF_ROBUST:
      l = ((1.0f - e) * softplus(-h) - e * softplus(h)) / (1.0f - 2.0f * e);
      dh = (-(1.0f - e) * sigmoid(-h) - e * sigmoid(h)) / (1.0f - 2.0f * e);
      break;
    case FLCE_PREF_HINGE:
      l = h < 1.0f ? 1.0f - h : (h != h ? h : 0.0f);
      dh = h < 1.0f ? -1.0f : 0.0f;
      break;
    default: {
      const float u = (h - 0.5f) / a.beta;
      l = u * u;
      dh = 2.0f * u / a.beta;
    }
  }
}

// In the place of the losses and the gradient where the sums mean nothing: NaN, and the reason.
template <typename T>
__device__ __noinline__ void poison(const PrefArgs& a, uint32_t why) {
  const float nan = __int_as_float(0x7fc00000);
  const int64_t thread = blockIdx.x * int64_t(kSeqThreads) + threadIdx.x;
  const int64_t threads = gridDim.x * int64_t(kSeqThreads);
  if (thread == 0) atomicOr(a.err, why);
  if (a.want_loss) {
    // the losses by the threads that wrote them; the rewards are there since the meeting
    const int64_t losses = a.reduction == FLCE_RED_NONE ? a.q.B / 2 : 1;
    if (blockIdx.x == 0) {
      for (int64_t i = threadIdx.x; i < losses; i += kSeqThreads) a.loss[i] = nan;
      for (int64_t i = threadIdx.x; i < a.q.B; i += kSeqThreads) a.rewards[i] = nan;
    }
  }
  if (a.dlp)
    for (int64_t p = thread; p < a.q.total; p += threads) store_f(static_cast<T*>(a.dlp) + p, nan);
}

template <typename T>
__global__ void __launch_bounds__(kSeqThreads, 1) preference_kernel(PrefArgs a) {
  const Seqs& q = a.q;
  const int lane = threadIdx.x & 31;
  const int warp = blockIdx.x * kSeqWarps + (threadIdx.x >> 5);
  const int warps = gridDim.x * kSeqWarps;
  if (warp == 0 && lane == 0) {
    *a.totals = SeqTotals{};
    *a.err = 0;
  }
  for (int u = warp; u < q.pieces; u += warps) {
    const Piece pc = find_piece(q, u);
    const Counted counted(q, pc);
    const T* lp_ = static_cast<const T*>(a.lp) + pc.begin + pc.seq * a.lp_skip;
    const T* ref_ = static_cast<const T*>(a.ref) + pc.begin + pc.seq * a.ref_skip;
    Pair f[2] = {};
    int n = 0;
    const bool vec_in = !(misfit(lp_, true) | misfit(ref_, a.ref));
    // the loads of all the lane's tokens first, masked ones' too
    float lp[kGroups][kVec] = {}, ref[kGroups][kVec] = {};
    unsigned int on[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int t = g * kGroup4 + lane * kVec;
      const unsigned int in = tokens_in(t, 0, pc.len);
      const bool vec = vec_in && in == 15u;
      on[g] = counted(t, in);
      load4(lp_ + t, vec, in, lp[g]);
      if (a.ref) load4(ref_ + t, vec, in, ref[g]);
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      n += __popc(on[g]);
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (on[g] >> j & 1) {
          f[0] = f[0] + lp[g][j] + -ref[g][j];
          f[1] = f[1] + lp[g][j];
        }
    }
    warp_sums(f);
    n = warp_sum(n);
    if (lane == 0) a.piece[u] = {f[0], f[1], n, 0};
  }
  meet(q.meet);

  const int64_t pairs = q.B / 2;
  unsigned int my_live = 0, my_pairs = 0;
  const SeqShare share(q, pairs);
  for (int64_t i = share.first; i < pairs; i += share.stride) {
    int64_t id[2];
    Pair score[2] = {}, like{};
    long long n[2] = {0, 0};
    id[0] = a.interleaved ? 2 * i : i;
    id[1] = a.interleaved ? 2 * i + 1 : pairs + i;
#pragma unroll 1
    for (int side = 1; side >= 0; --side) {
      int first, last;
      if (!seq_pieces(q, id[side], first, last)) atomicOr(&a.totals->live, kBadSeqs);
      Pair f[2] = {};
      long long c[1] = {0};
      for (int u = first + share.offset; u < last; u += share.step) {
        const PrefPiece r = a.piece[u];
        f[0] = f[0] + r.score;
        f[1] = f[1] + r.like;
        c[0] += r.n;
      }
      share.sum(f, c);
      score[1] = side == 1 ? f[0] : score[1];
      score[0] = f[0];
      like = f[1];
      n[1] = side == 1 ? c[0] : n[1];
      n[0] = c[0];
    }
    if (share.writes()) {
      const float per[2] = {n[0] > 0 ? 1.0f / static_cast<float>(n[0]) : 0.0f,
                            n[1] > 0 ? 1.0f / static_cast<float>(n[1]) : 0.0f};
      for (int side = 0; side < 2; ++side) {
        if (a.norm && n[side] > 0) score[side] = score[side] / static_cast<float>(n[side]);
        if (a.ref_scores) score[side] = score[side] + -__ldg(a.ref_scores + id[side]);
        if (n[side] == 0) score[side] = {};
      }
      const bool ok = n[0] > 0 && n[1] > 0;
      float l = 0.0f, dh = 0.0f;
      if (ok) {
        pair_value(a, fmaf(a.beta, (score[0] + -score[1]).value(), -a.margin), l, dh);
        l -= a.nll * like.value() * per[0];
      }
      a.pair_loss[i] = l;
      const float d = a.beta * dh;
      a.coef[id[0]] = ok ? d * (a.norm ? per[0] : 1.0f) - a.nll * per[0] : 0.0f;
      a.coef[id[1]] = ok ? -d * (a.norm ? per[1] : 1.0f) : 0.0f;
      if (a.want_loss) {
        a.rewards[id[0]] = a.beta * score[0].value();
        a.rewards[id[1]] = a.beta * score[1].value();
      }
    }
    if (share.counts()) {
      my_live += n[0] > 0 && n[1] > 0;
      ++my_pairs;
    }
  }
  const bool late = meet_sequences(q, a.totals, 0, my_live, my_pairs, a.err);
  const float nan = __int_as_float(0x7fc00000);

  const unsigned int live = __ldcg(&a.totals->live);
  Pair l[1] = {};
  if (blockIdx.x == 0 && a.want_loss) {
    for (int64_t i = threadIdx.x; i < pairs; i += kSeqThreads) {
      const float v = late ? nan : a.pair_loss[i];
      if (a.reduction == FLCE_RED_NONE) a.loss[i] = v;
      l[0] = l[0] + v;
    }
    block_sums(l, pairs);
  }
  float scale = a.reduction == FLCE_RED_MEAN
                    ? (live > 0 ? 1.0f / static_cast<float>(live) : 0.0f)
                    : 1.0f;
  if (late) scale = nan;  // totals of a wait that ran out: no loss, no gradients of this block's pieces
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.want_loss && a.reduction != FLCE_RED_NONE)
    a.loss[0] = l[0].value() * scale;
  if (live & kBadSeqs) {
    poison<T>(a, FLCE_DEVERR_SEQS);
    return;
  }
  T* dlp_ = static_cast<T*>(a.dlp);
  if (!dlp_) return;
  if (q.cu) {
    const int64_t begin = seq_start(q, 0), end = seq_start(q, q.B);
    for (int64_t p = warp * int64_t(32) + lane; p < q.total; p += warps * int64_t(32))
      if (p < begin || p >= end) store_f(dlp_ + p, 0.0f);
  }
  for (int u = warp; u < q.pieces; u += warps) {
    const Piece pc = find_piece(q, u);
    if (pc.len == 0) continue;
    const Counted counted(q, pc);
    float g = a.coef[pc.seq] * scale;
    if (a.g_loss) {
      const int64_t pair = a.interleaved ? pc.seq / 2 : pc.seq % pairs;
      g *= __ldg(a.g_loss + (a.reduction == FLCE_RED_NONE ? pair : 0));
    }
    T* out = dlp_ + pc.begin;
    const bool vec_out = !misfit(out, true);
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const int t = k * kGroup4 + lane * kVec;
      const unsigned int in = tokens_in(t, 0, pc.len), on = counted(t, in);
      float o[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) o[j] = on >> j & 1 ? g : 0.0f;
      store4(out + t, vec_out && in == 15u, in, o);
    }
  }
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct PrefLayout {
  size_t piece, coef, pair_loss, total;
};

PrefLayout pref_layout(const Seqs& q) {
  PrefLayout L{};
  const int64_t B = q.B > 0 ? q.B : 1;
  size_t off = 256;
  L.piece = off; off += align256(static_cast<size_t>(q.pieces) * sizeof(PrefPiece));
  L.coef = off; off += align256(B * 4);
  L.pair_loss = off; off += align256(B * 4);
  L.total = off;
  return L;
}

int pref_check(const flce_preference_params* p, Seqs* q) {
  if (!p) return FLCE_ERR_BAD_ARG;
  const int rc = make_seqs(&p->seqs, q);
  if (rc) return rc;
  if (q->B % 2) return FLCE_ERR_BAD_SHAPE;
  if ((p->ld_logp | p->ld_ref) < 0) return FLCE_ERR_BAD_ARG;
  if (p->kind < FLCE_PREF_SIGMOID || p->kind > FLCE_PREF_IPO) return FLCE_ERR_BAD_ARG;
  if (p->reduction < FLCE_RED_NONE || p->reduction > FLCE_RED_SUM) return FLCE_ERR_BAD_ARG;
  if (!(p->beta > 0.0) || !std::isfinite(p->beta) || !std::isfinite(p->margin) ||
      !std::isfinite(p->nll_coef))
    return FLCE_ERR_BAD_ARG;
  if (!(p->label_smoothing >= 0.0 && p->label_smoothing < 0.5)) return FLCE_ERR_BAD_ARG;
  // smoothing flips labels: only the logistic losses have that reading
  if (p->label_smoothing != 0.0 && p->kind != FLCE_PREF_SIGMOID && p->kind != FLCE_PREF_ROBUST)
    return FLCE_ERR_BAD_ARG;
  if ((p->length_normalised | p->interleaved | 1) != 1) return FLCE_ERR_BAD_ARG;
  return FLCE_OK;
}

inline bool misaligned(const void* p, int bytes) {
  return reinterpret_cast<uintptr_t>(p) & (bytes - 1);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

int flce_preference_check_params(const flce_preference_params* p) {
  Seqs q;
  return pref_check(p, &q);
}

size_t flce_preference_workspace_size(const flce_preference_params* p) {
  Seqs q;
  return pref_check(p, &q) == FLCE_OK ? pref_layout(q).total : 0;
}

}  // extern "C"

namespace {

// `missing`: pairs that the second meeting waits for in vain (the self-test's).
int preference_loss(const flce_preference_params* p, const void* logp, const void* ref_logp,
                    const float* ref_scores, const float* g_loss, float* loss, float* rewards,
                    void* dlogp, void* workspace, size_t ws_bytes, void* stream,
                    unsigned int missing) {
  PrefArgs a{};
  int rc = pref_check(p, &a.q);
  if (rc) return rc;
  if (!workspace || (!loss && !dlogp) || (loss && !rewards && a.q.B > 0)) return FLCE_ERR_BAD_ARG;
  if (a.q.total > 0 && !logp) return FLCE_ERR_BAD_ARG;
  const int dt = p->seqs.dtype, eb = seq_elem_bytes(dt);
  if (misaligned(logp, eb) || misaligned(ref_logp, eb) || misaligned(dlogp, eb) ||
      misaligned(ref_scores, 4) || misaligned(g_loss, 4) || misaligned(loss, 4) ||
      misaligned(rewards, 4) || misaligned(workspace, 256))
    return FLCE_ERR_ALIGN;
  const PrefLayout L = pref_layout(a.q);
  if (ws_bytes < L.total) return FLCE_ERR_WS_TOO_SMALL;
  int sms;
  if ((rc = require_device(&sms))) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool packed = p->seqs.cu_kind != 0;
  a.q.awaited = static_cast<unsigned int>(a.q.B / 2) + missing;
  a.lp = logp;
  a.ref = ref_logp;
  a.lp_skip = packed ? 0 : p->ld_logp - p->seqs.S;
  a.ref_skip = packed ? 0 : p->ld_ref - p->seqs.S;
  a.ref_scores = ref_scores;
  a.beta = static_cast<float>(p->beta);
  a.margin = static_cast<float>(p->margin);
  a.smooth = static_cast<float>(p->label_smoothing);
  a.nll = static_cast<float>(p->nll_coef);
  a.kind = p->kind;
  a.norm = p->length_normalised;
  a.interleaved = p->interleaved;
  a.reduction = p->reduction;
  a.want_loss = loss != nullptr;
  a.g_loss = g_loss;
  a.loss = loss;
  a.rewards = rewards;
  a.dlp = dlogp;
  a.err = reinterpret_cast<uint32_t*>(ws);
  a.totals = reinterpret_cast<SeqTotals*>(ws + 64);
  a.piece = reinterpret_cast<PrefPiece*>(ws + L.piece);
  a.coef = reinterpret_cast<float*>(ws + L.coef);
  a.pair_loss = reinterpret_cast<float*>(ws + L.pair_loss);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dt == FLCE_F32)
    e = launch_seq(preference_kernel<float>, a, 0, sms, st);
  else if (dt == FLCE_BF16)
    e = launch_seq(preference_kernel<__nv_bfloat16>, a, 0, sms, st);
  else
    e = launch_seq(preference_kernel<__half>, a, 0, sms, st);
  if (e != cudaSuccess) return FLCE_ERR_CUDA;
  return p->validate ? read_status(workspace, st) : FLCE_OK;
}

}  // namespace

extern "C" {

int flce_preference_loss(const flce_preference_params* p, const void* logp, const void* ref_logp,
                         const float* ref_scores, const float* g_loss, float* loss,
                         float* rewards, void* dlogp, void* workspace, size_t ws_bytes,
                         void* stream) {
  return preference_loss(p, logp, ref_logp, ref_scores, g_loss, loss, rewards, dlogp, workspace,
                         ws_bytes, stream, 0);
}

int flce_selftest_preference_timeout(const flce_preference_params* p, const void* logp,
                                     float* loss, float* rewards, void* dlogp, void* workspace,
                                     size_t ws_bytes, void* stream) {
  return preference_loss(p, logp, nullptr, nullptr, nullptr, loss, rewards, dlogp, workspace,
                         ws_bytes, stream, 1);
}

}  // extern "C"
