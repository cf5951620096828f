// Clipped policy loss with a KL term and an entropy bonus, and its gradients.
//
// Per token with log-probability lp, the rollout's old and a reference's ref:
//   d = lp - old,  r = exp(d) (d clamped to +-20),  A the advantage,
//   l = -min(r A, clip(r, 1 - lo, 1 + hi) A)      (A < 0 with a dual clip c: at most -c A)
//       + kl_coef K(lp, ref) - ent_coef H,
//   loss = sum_i w_i sum_{t in i, counted} l_t,
// with w from the aggregate: 1 / tokens, 1 / (sequences n_i), 1 / sequences, or a scale.
//
// One launch does all of it, loss and gradients:
//   A  a block per piece of at most 1024 tokens: its sums;
//   S  a warp per sequence: its pieces' sums, added in order in fp64;
//   B  the totals (each block for itself, over the sequences' records), the loss (block
//      0), and a second pass over the tokens for the gradients, which by then sit in L2.
// between which the blocks of the (cooperative) grid meet.  The sums have a fixed order:
// results do not change from run to run.
//
// Clipping tests compare d, not r, with log(1 + hi), log(1 - lo), log c: d is formed as
// an exact sum of two floats and the borders are given the same way, so a token at a
// border falls on the side that the exact difference falls on.
#include <cmath>

#include "flce_device.cuh"
#include "flce_policy.cuh"

namespace flce {

namespace {

constexpr float kLogRatioLimit = 20.0f;

__device__ __forceinline__ bool pair_above(float h, float l, float bh, float bl) {
  return __fadd_rn(__fadd_rn(h, -bh), __fadd_rn(l, -bl)) > 0.0f;
}

// a - b as an unevaluated sum h + l (exact).
__device__ __forceinline__ void exact_diff(float a, float b, float& h, float& l) {
  h = __fadd_rn(a, -b);
  const float z = __fadd_rn(h, -a);
  l = __fadd_rn(__fadd_rn(a, -__fadd_rn(h, -z)), __fadd_rn(-b, -z));
}

struct Ratio {
  float value;  // the objective is value * A
  bool live;    // whether it moves with d
  bool clipped, dual;
};

__device__ __forceinline__ Ratio clip_ratio(const PolicyArgs& a, float h, float l, float adv) {
  Ratio o{0.0f, true, false, false};
  if (adv > 0.0f && pair_above(h, l, a.hi_h, a.hi_l)) {
    o = {a.r_hi, false, true, false};
  } else if (adv < 0.0f && pair_above(-h, -l, -a.lo_h, -a.lo_l)) {
    o = {a.r_lo, false, true, false};
  } else if (adv < 0.0f && a.r_dual != 0.0f && pair_above(h, l, a.dual_h, a.dual_l)) {
    o = {a.r_dual, false, false, true};
  } else {
    o.value = expf(fminf(fmaxf(h, -kLogRatioLimit), kLogRatioLimit));
    // a NaN log-ratio stays one (fmaxf would drop it)
    if (h != h) o.value = h;
    o.live = !(fabsf(h) > kLogRatioLimit);
  }
  return o;
}

// K(lp, ref) and its derivative by lp.
__device__ __forceinline__ void kl_term(int kind, float lp, float ref, float& k, float& dk) {
  const float e = ref - lp;
  if (kind == FLCE_KL_K1) {
    k = -e;
    dk = 1.0f;
  } else if (kind == FLCE_KL_K2) {
    k = 0.5f * e * e;
    dk = -e;
  } else {
    const float c = e != e ? e : fminf(fmaxf(e, -kLogRatioLimit), kLogRatioLimit);
    k = exp_m1_mx(c);
    dk = fabsf(e) > kLogRatioLimit ? 0.0f : -(c + k);  // 1 - exp(c)
  }
}

template <typename T>
__global__ void __launch_bounds__(kSeqThreads, kSeqBlocksPerSm) policy_kernel(PolicyArgs a) {
  const Seqs& q = a.q;
  const T* lp_ = static_cast<const T*>(a.lp);
  const T* old_ = static_cast<const T*>(a.old_lp);
  const T* ref_ = static_cast<const T*>(a.ref);
  const T* ent_ = static_cast<const T*>(a.ent);
  const bool want_loss = a.what & POLICY_LOSS;
  const bool by_seq = a.ratio == FLCE_RATIO_SEQUENCE;

  // ---- A: sums of the pieces
  for (int64_t u = blockIdx.x; u < a.pieces; u += gridDim.x) {
    const Piece pc = find_piece(q, u);
    float f[5] = {0, 0, 0, 0, 0};
    int c[3] = {0, 0, 0};
#pragma unroll
    for (int k = 0; k < kSeqPerThread; ++k) {
      const int64_t p = pc.begin + threadIdx.x + k * kSeqThreads;
      if (p >= pc.end || !token_counts(q, pc.seq, p)) continue;
      ++c[0];
      if (!want_loss && !by_seq) continue;
      const float lp = a.lp_sign * load_f(lp_ + p + pc.seq * a.lp_skip);
      float h = 0.0f, l = 0.0f;
      if (old_) exact_diff(lp, load_f(old_ + p + pc.seq * a.old_skip), h, l);
      if (by_seq) {
        f[4] += h;
      } else {
        const float adv = __ldg(a.adv + (a.adv_per_token ? p + pc.seq * a.adv_skip : pc.seq));
        const Ratio r = clip_ratio(a, h, l, adv);
        f[0] -= r.value * adv;
        c[1] += r.clipped;
        c[2] += r.dual;
      }
      if (!want_loss) continue;
      const float hc = h != h ? h : fminf(fmaxf(h, -kLogRatioLimit), kLogRatioLimit);
      f[3] += exp_m1_mx(hc);
      if (ref_) {
        float kl, dkl;
        kl_term(a.kl, lp, load_f(ref_ + p + pc.seq * a.ref_skip), kl, dkl);
        f[1] += kl;
      }
      if (ent_) f[2] += load_f(ent_ + p + pc.seq * a.ent_skip);
    }
    block_sums(f, c);
    if (threadIdx.x == 0) a.piece[u] = {f[0], f[1], f[2], f[3], f[4], c[0], c[1], c[2]};
  }
  grid_barrier();

  // ---- S: sums of the sequences
  for (int64_t i = blockIdx.x * int64_t(kSeqWarps) + (threadIdx.x >> 5); i < q.B;
       i += gridDim.x * int64_t(kSeqWarps)) {
    const int64_t s0 = seq_start(q, i), s1 = seq_start(q, i + 1);
    double f[5] = {0, 0, 0, 0, 0};
    long long c[3] = {0, 0, 0};
    const int64_t last = s1 > s0 ? (s1 - 1) / kTile + i : -1;
    for (int64_t u = s0 / kTile + i + (threadIdx.x & 31); u <= last; u += 32) {
      const PolicyPiece r = a.piece[u];
      f[0] += r.pg;
      f[1] += r.kl;
      f[2] += r.ent;
      f[3] += r.old_kl;
      f[4] += r.d;
      c[0] += r.n;
      c[1] += r.clipped;
      c[2] += r.dual;
    }
#pragma unroll
    for (int k = 0; k < 5; ++k) f[k] = warp_sum(f[k]);
#pragma unroll
    for (int k = 0; k < 3; ++k) c[k] = warp_sum(c[k]);
    if ((threadIdx.x & 31) == 0) {
      PolicySeq o{f[0], f[1], f[2], f[3], c[0], static_cast<int>(c[1]), static_cast<int>(c[2]),
                  0.0f, 0};
      if (by_seq) {
        o.clipped = o.dual = 0;
        o.pg = 0.0;
        if (c[0] > 0) {
          const double s = f[4] / static_cast<double>(c[0]);
          const float h = static_cast<float>(s), l = static_cast<float>(s - h);
          const float adv = __ldg(a.adv + i);
          const Ratio r = clip_ratio(a, h, l, adv);
          o.pg = -static_cast<double>(c[0]) * (static_cast<double>(r.value) * adv);
          o.coef = r.live ? -r.value * adv : 0.0f;
          o.clipped = r.clipped;
          o.dual = r.dual;
        }
      }
      a.seq[i] = o;
    }
  }
  grid_barrier();

  // ---- B: totals and the loss
  long long tokens = 0, live = 0;
  for (int64_t i = threadIdx.x; i < q.B; i += kSeqThreads) {
    const long long n = a.seq[i].n;
    tokens += n;
    live += n > 0;
  }
  tokens = block_total(tokens);
  live = block_total(live);
  const bool mean_seq = a.aggregate == FLCE_AGG_SEQ_MEAN_TOKEN_MEAN;
  // fp64 runs at a fraction of the fp32 rate: one thread for the block
  __shared__ double s_one_token, s_w_all;
  __shared__ float s_wg;
  if (threadIdx.x == 0) {
    s_one_token = tokens > 0 ? 1.0 / static_cast<double>(tokens) : 0.0;
    const double one_seq = live > 0 ? 1.0 / static_cast<double>(live) : 0.0;
    s_w_all = a.aggregate == FLCE_AGG_TOKEN_MEAN ? s_one_token
              : a.aggregate == FLCE_AGG_SUM      ? a.scale
                                                 : one_seq;
    s_wg = static_cast<float>((a.g_loss ? __ldg(a.g_loss) : 1.0f) * s_w_all);
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    const bool ok = seqs_ok(q);
    if (threadIdx.x == 0) {
      if (a.err_store)
        *a.err = ok ? 0u : FLCE_DEVERR_SEQS;
      else if (!ok)
        atomicOr(a.err, FLCE_DEVERR_SEQS);
    }
  }
  if (want_loss && blockIdx.x == 0) {
    double f[6] = {0, 0, 0, 0, 0, 0};
    long long c[2] = {0, 0};
    for (int64_t i = threadIdx.x; i < q.B; i += kSeqThreads) {
      const PolicySeq r = a.seq[i];
      const double w = mean_seq && r.n > 0 ? 1.0 / static_cast<double>(r.n) : 1.0;
      f[0] += w * r.pg;
      f[1] += w * (a.kl_coef * r.kl - a.ent_coef * r.ent);
      f[2] += r.kl;
      f[3] += r.ent;
      f[4] += r.old_kl;
      c[0] += r.clipped;
      c[1] += r.dual;
    }
#pragma unroll
    for (int k = 0; k < 5; ++k) f[k] = block_total(f[k]);
    c[0] = block_total(c[0]);
    c[1] = block_total(c[1]);
    const bool ok = seqs_ok(q);
    if (threadIdx.x == 0) {
      const float nan = __int_as_float(0x7fc00000);
      const double w_all = s_w_all, one_token = s_one_token;
      a.loss[0] = ok ? static_cast<float>(w_all * (f[0] + f[1])) : nan;
      a.stats[0] = ok ? static_cast<float>(w_all * f[0]) : nan;
      a.stats[1] = static_cast<float>(one_token * f[2]);
      a.stats[2] = static_cast<float>(one_token * f[3]);
      a.stats[3] = static_cast<float>(one_token * f[4]);
      a.counts[0] = tokens;
      a.counts[1] = live;
      a.counts[2] = c[0];
      a.counts[3] = c[1];
    }
  }
  if (a.lp_out) {
    // positions of a packed axis (the head's tokens)
    for (int64_t p = blockIdx.x * int64_t(kSeqThreads) + threadIdx.x; p < q.total;
         p += gridDim.x * int64_t(kSeqThreads))
      a.lp_out[p] = 0.0f + a.lp_sign * load_f(lp_ + p);
  }
  if (!(a.what & POLICY_GRAD)) return;

  // ---- B: gradients
  T* dlp_ = static_cast<T*>(a.dlp);
  T* dent_ = static_cast<T*>(a.dent);
  if (q.cu) {
    // positions outside every sequence
    const int64_t first = seq_start(q, 0), end = seq_start(q, q.B);
    for (int64_t p = a.g_begin + blockIdx.x * int64_t(kSeqThreads) + threadIdx.x; p < a.g_end;
         p += gridDim.x * int64_t(kSeqThreads))
      if (p < first || p >= end) {
        if (dlp_) store_f(dlp_ + p, 0.0f);
        if (dent_) store_f(dent_ + p, 0.0f);
      }
  }
  for (int64_t u = blockIdx.x; u < a.pieces; u += gridDim.x) {
    const Piece pc = find_piece(q, u);
    const int64_t b = pc.begin > a.g_begin ? pc.begin : a.g_begin;
    const int64_t e = pc.end < a.g_end ? pc.end : a.g_end;
    if (b >= e) continue;
    float wg = s_wg, coef = 0.0f;
    if (mean_seq || by_seq) {
      const PolicySeq& r = a.seq[pc.seq];
      if (mean_seq) wg = r.n > 0 ? wg / static_cast<float>(r.n) : 0.0f;
      coef = r.coef;
    }
#pragma unroll
    for (int k = 0; k < kSeqPerThread; ++k) {
      const int64_t p = b + threadIdx.x + k * kSeqThreads;
      if (p >= e) continue;
      float dl = 0.0f, dh = 0.0f;
      if (token_counts(q, pc.seq, p)) {
        if (dlp_) {
          const float lp = a.lp_sign * load_f(lp_ + p + pc.seq * a.lp_skip);
          if (by_seq) {
            dl = coef;
          } else {
            float h = 0.0f, l = 0.0f;
            if (old_) exact_diff(lp, load_f(old_ + p + pc.seq * a.old_skip), h, l);
            const float adv = __ldg(a.adv + (a.adv_per_token ? p + pc.seq * a.adv_skip : pc.seq));
            const Ratio r = clip_ratio(a, h, l, adv);
            dl = r.live ? -r.value * adv : 0.0f;
          }
          if (ref_ && a.kl_coef != 0.0f) {
            float kl, dkl;
            kl_term(a.kl, lp, load_f(ref_ + p + pc.seq * a.ref_skip), kl, dkl);
            dl = fmaf(a.kl_coef, dkl, dl);
          }
          dl *= wg * a.lp_sign;
        }
        dh = -a.ent_coef * wg;
      }
      // outputs are dense: a padded batch's position is its index
      if (dlp_) store_f(dlp_ + p, dl);
      if (dent_) store_f(dent_ + p, dh);
    }
  }
}

// A border b as a sum of two floats (an infinite one as its high part alone).
void split(double b, float* h, float* l) {
  *h = static_cast<float>(b);
  *l = std::isfinite(*h) ? static_cast<float>(b - *h) : 0.0f;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline bool misaligned(const void* p, int dtype) {
  return reinterpret_cast<uintptr_t>(p) & (seq_elem_bytes(dtype) - 1);
}

}  // namespace

int policy_check(const flce_policy_params* p) {
  if (!p) return FLCE_ERR_BAD_ARG;
  Seqs q;
  const int rc = make_seqs(&p->seqs, &q);
  if (rc) return rc;
  if (p->kl < FLCE_KL_K1 || p->kl > FLCE_KL_K3) return FLCE_ERR_BAD_ARG;
  if (p->ratio != FLCE_RATIO_TOKEN && p->ratio != FLCE_RATIO_SEQUENCE) return FLCE_ERR_BAD_ARG;
  if (p->aggregate < FLCE_AGG_TOKEN_MEAN || p->aggregate > FLCE_AGG_SUM) return FLCE_ERR_BAD_ARG;
  if (!(p->clip_low >= 0.0 && p->clip_low < 1.0) || !(p->clip_high >= 0.0))
    return FLCE_ERR_BAD_ARG;
  if (!(p->dual_clip == 0.0 || p->dual_clip > 1.0)) return FLCE_ERR_BAD_ARG;
  if (!std::isfinite(p->kl_coef) || !std::isfinite(p->entropy_coef) || !std::isfinite(p->scale))
    return FLCE_ERR_BAD_ARG;
  if (p->adv_per_token != 0 && p->adv_per_token != 1) return FLCE_ERR_BAD_ARG;
  // a sequence's ratio has one advantage
  if (p->ratio == FLCE_RATIO_SEQUENCE && p->adv_per_token) return FLCE_ERR_BAD_ARG;
  return FLCE_OK;
}

size_t policy_workspace(const flce_policy_params* p) {
  Seqs q;
  if (make_seqs(&p->seqs, &q)) return 0;
  return 256 + align256(seq_pieces(q.B, q.total) * sizeof(PolicyPiece)) +
         align256((q.B > 0 ? q.B : 1) * sizeof(PolicySeq));
}

int policy_args(const flce_policy_params* p, void* workspace, PolicyArgs* a) {
  *a = PolicyArgs{};
  const int rc = make_seqs(&p->seqs, &a->q);
  if (rc) return rc;
  const bool packed = p->seqs.cu_kind != 0;
  const int64_t S = p->seqs.S;
  a->lp_skip = packed ? 0 : p->ld_logp - S;
  a->old_skip = packed ? 0 : p->ld_old - S;
  a->ref_skip = packed ? 0 : p->ld_ref - S;
  a->ent_skip = packed ? 0 : p->ld_entropy - S;
  a->adv_skip = packed ? 0 : p->ld_adv - S;
  a->adv_per_token = p->adv_per_token;
  a->lp_sign = 1.0f;
  split(std::log1p(p->clip_high), &a->hi_h, &a->hi_l);
  split(std::log1p(-p->clip_low), &a->lo_h, &a->lo_l);
  if (p->dual_clip != 0.0) split(std::log(p->dual_clip), &a->dual_h, &a->dual_l);
  a->r_hi = static_cast<float>(1.0 + p->clip_high);
  a->r_lo = static_cast<float>(1.0 - p->clip_low);
  a->r_dual = static_cast<float>(p->dual_clip);
  a->kl_coef = static_cast<float>(p->kl_coef);
  a->ent_coef = static_cast<float>(p->entropy_coef);
  a->scale = p->scale;
  a->kl = p->kl;
  a->ratio = p->ratio;
  a->aggregate = p->aggregate;
  a->pieces = seq_pieces(a->q.B, a->q.total);
  a->g_end = a->q.total;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a->err = reinterpret_cast<uint32_t*>(ws);
  a->err_store = 1;
  a->piece = reinterpret_cast<PolicyPiece*>(ws + 256);
  a->seq = reinterpret_cast<PolicySeq*>(ws + 256 + align256(a->pieces * sizeof(PolicyPiece)));
  return FLCE_OK;
}

int launch_policy(const PolicyArgs& a, int dtype, int sms, cudaStream_t st) {
  const int64_t cap = int64_t(sms) * kSeqBlocksPerSm;
  const int64_t blocks = a.pieces < cap ? a.pieces : cap;
  cudaError_t e;
  if (dtype == FLCE_F32)
    e = launch_seq(policy_kernel<float>, a, blocks, st);
  else if (dtype == FLCE_BF16)
    e = launch_seq(policy_kernel<__nv_bfloat16>, a, blocks, st);
  else
    e = launch_seq(policy_kernel<__half>, a, blocks, st);
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

}  // namespace flce

using namespace flce;

extern "C" {

int flce_policy_check_params(const flce_policy_params* p) { return policy_check(p); }

size_t flce_policy_workspace_size(const flce_policy_params* p) {
  return policy_check(p) == FLCE_OK ? policy_workspace(p) : 0;
}

int flce_policy_loss(const flce_policy_params* p, const void* logp, const void* old_logp,
                     const void* ref_logp, const void* entropy, const float* advantages,
                     const float* g_loss, float* loss, float* stats, int64_t* counts,
                     void* dlogp, void* dentropy, void* workspace, size_t ws_bytes,
                     void* stream) {
  int rc = policy_check(p);
  if (rc) return rc;
  if (!workspace || (loss == nullptr) != (stats == nullptr) ||
      (loss == nullptr) != (counts == nullptr))
    return FLCE_ERR_BAD_ARG;
  if (!loss && !dlogp && !dentropy) return FLCE_ERR_BAD_ARG;
  PolicyArgs a;
  if ((rc = policy_args(p, workspace, &a))) return rc;
  if (a.q.total > 0 && (!logp || !advantages)) return FLCE_ERR_BAD_ARG;
  if (a.q.total > 0 && ((p->kl_coef != 0.0 && !ref_logp) ||
                        ((p->entropy_coef != 0.0 || dentropy) && !entropy)))
    return FLCE_ERR_BAD_ARG;
  const int dt = p->seqs.dtype;
  if (misaligned(logp, dt) || misaligned(old_logp, dt) || misaligned(ref_logp, dt) ||
      misaligned(entropy, dt) || misaligned(dlogp, dt) || misaligned(dentropy, dt) ||
      misaligned(advantages, FLCE_F32) || misaligned(g_loss, FLCE_F32) ||
      misaligned(loss, FLCE_F32) || misaligned(stats, FLCE_F32) ||
      (reinterpret_cast<uintptr_t>(counts) & 7) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255))
    return FLCE_ERR_ALIGN;
  if (ws_bytes < policy_workspace(p)) return FLCE_ERR_WS_TOO_SMALL;
  int sms;
  if ((rc = require_device(&sms))) return rc;
  a.lp = logp;
  a.old_lp = old_logp;
  a.ref = ref_logp;
  a.ent = entropy;
  a.adv = advantages;
  a.g_loss = g_loss;
  a.loss = loss;
  a.stats = stats;
  a.counts = reinterpret_cast<long long*>(counts);
  a.dlp = dlogp;
  a.dent = dentropy;
  a.what = (loss ? POLICY_LOSS : 0) | (dlogp || dentropy ? POLICY_GRAD : 0);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((rc = launch_policy(a, dt, sms, st))) return rc;
  return p->validate ? read_status(workspace, st) : FLCE_OK;
}

}  // extern "C"
