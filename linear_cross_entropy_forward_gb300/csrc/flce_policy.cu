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
//   1  a warp per piece of at most 256 tokens: its sums;
//   2  a warp per sequence (a block, where they are few and long): its pieces' sums, added in
//      a fixed order in pairs of floats, and the counts of tokens and sequences by atomics;
//   3  the loss (block 0, over the sequences' records) and the gradients: of a warp's first
//      four pieces from what pass 1 left in shared memory, of further ones (beyond 5M tokens) by
//      a second pass over the tokens,
// between which the blocks meet.  The sums have a fixed order: results do not change from
// run to run.  The two passes over the tokens share one body of code: a launch finds the
// instruction cache cold, and a second copy would be fetched while nothing else runs.
//
// What bounds it: up to a piece per warp, latency (4 x 64 tokens 9.6 us in one block, 16 x 1024 20
// in a cluster, 256 x 4096 22.8 in a grid, whose bytes need 4.5); beyond, that a warp loads a
// piece, waits, computes and sums it before the next one's loads: 13 us for each further million
// tokens (1024 x 4096 62 us, 29 % of the copy rate).
//
// Clipping tests compare d, not r, with log(1 + hi), log(1 - lo), log c: d is formed as
// an exact sum of two floats and the borders are given the same way, so a token at a
// border falls on the side that the exact difference falls on.  (A border beyond +-20, which
// the clamped d does not reach, clips nothing.)
#include <cmath>

#include "flce_policy.cuh"

namespace flce {

namespace {

constexpr float kLogRatioLimit = 20.0f;

__device__ __forceinline__ bool pair_above(float h, float l, float bh, float bl) {
  return __fadd_rn(__fadd_rn(h, -bh), __fadd_rn(l, -bl)) > 0.0f;
}

// a - b as an unevaluated sum h + l (exact; an infinite one is h alone).
__device__ __forceinline__ void exact_diff(float a, float b, float& h, float& l) {
  h = __fadd_rn(a, -b);
  const float z = __fadd_rn(h, -a);
  l = __fadd_rn(__fadd_rn(a, -__fadd_rn(h, -z)), __fadd_rn(-b, -z));
  if (!(fabsf(h) <= 3.4028235e38f)) l = 0.0f;
}

// A NaN stays one (fmaxf alone would drop it).
__device__ __forceinline__ float clamp_ratio(float h) {
  return h != h ? h : fminf(fmaxf(h, -kLogRatioLimit), kLogRatioLimit);
}

struct Ratio {
  float value, low;  // the objective is (value + low) * A
  bool live;    // whether it moves with d
  bool clipped, dual;
};

// The clipped ratio of the log-ratio h + l; e = exp(hc), k = e - 1 - hc of the clamped hc.
// Near 1 the ratio is 1 + (hc + k), more exact than e: where the objective's terms cancel,
// its last bits are what the loss is made of.
__device__ __forceinline__ Ratio clip_ratio(const PolicyArgs& a, float h, float l, float hc,
                                            float e, float k, float adv) {
  // above the upper border where A > 0, below the lower where A < 0
  const bool up = adv > 0.0f, down = adv < 0.0f;
  Ratio o;
  o.clipped = (up || down) && pair_above(up ? h : -h, up ? l : -l, up ? a.hi_h : -a.lo_h,
                                         up ? a.hi_l : -a.lo_l);
  o.dual = false;
  if (a.r_dual != 0.0f) o.dual = down && pair_above(h, l, a.dual_h, a.dual_l);
  o.value = e;
  o.low = 0.0f;
  if (fabsf(hc) < 0.5f) {
    const float y = hc + k;
    o.value = 1.0f + y;
    o.low = y - (o.value - 1.0f) + l;
  }
  if (o.clipped) {
    o.value = up ? a.r_hi : a.r_lo;
    o.low = up ? a.r_hi_l : a.r_lo_l;
  } else if (o.dual) {
    o.value = a.r_dual;
    o.low = a.r_dual_l;
  }
  o.live = !(o.clipped || o.dual || fabsf(h) > kLogRatioLimit);
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
    const float c = clamp_ratio(e);
    k = exp_m1_mx(c, expf(c));
    dk = fabsf(e) > kLogRatioLimit ? 0.0f : -(c + k);  // 1 - exp(c)
  }
}

template <typename T>
__global__ void __launch_bounds__(kSeqThreads, 1) policy_kernel(PolicyArgs a) {
  const Seqs& q = a.q;
  const bool want_loss = a.what & POLICY_LOSS;
  const bool by_seq = a.ratio == FLCE_RATIO_SEQUENCE;
  const bool mean_seq = a.aggregate == FLCE_AGG_SEQ_MEAN_TOKEN_MEAN;
  const int lane = threadIdx.x & 31;
  const int warp = blockIdx.x * kSeqWarps + (threadIdx.x >> 5);
  const int warps = gridDim.x * kSeqWarps;
  // gradients before their weight, and which tokens count, of this warp's first pieces
  extern __shared__ float4 kept[];  // [piece][kGroups][kSeqThreads]
  unsigned int kept_on = 0;
  const bool keep_all = a.what == (POLICY_LOSS | POLICY_GRAD);
  if (warp == 0 && lane == 0) {
    *a.totals = SeqTotals{};
    if (a.err_store) *a.err = 0;
  }
  float wg_all = 0.0f;  // the gradients' weight before a sequence's own
  float g_up = 1.0f;    // the upstream gradient, a factor with a rounding of its own

#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const bool grad = pass == 1;
    if (grad && !(a.what & POLICY_GRAD)) break;
    // the first pass of a launch without the loss counts tokens, no more
    // (and a second pass of a sequence's ratio without a reference knows the gradient)
    const bool values = grad ? !by_seq || a.ref : want_loss || by_seq;
    // (a weight of NaN, from bad offsets: no pieces to go by, the gradients are written already)
#pragma unroll 1
    for (int u = wg_all == wg_all ? warp : q.pieces, round = 0; u < q.pieces;
         u += warps, ++round) {
      const Piece pc = find_piece(q, u);
      int t0 = 0, t1 = pc.len;
      float wg = wg_all, coef = 0.0f;
      if (grad) {
        if (pc.len == 0 || pc.begin >= a.g_end || pc.begin + pc.len <= a.g_begin) continue;
        if (pc.begin < a.g_begin) t0 = static_cast<int>(a.g_begin - pc.begin);
        if (pc.begin + pc.len > a.g_end) t1 = static_cast<int>(a.g_end - pc.begin);
        if (mean_seq || by_seq) {
          const PolicySeq& r = a.seq[pc.seq];
          if (mean_seq) wg = r.n > 0 ? wg / static_cast<float>(r.n) : 0.0f;
          coef = r.coef;
        }
      }
      const bool keep = keep_all && round < q.kept;
      const float w_lp = wg * a.lp_sign, w_ent = -a.ent_coef * wg;
      const Counted counted(q, pc);
      const T* lp_ = static_cast<const T*>(a.lp) + pc.begin + pc.seq * a.lp_skip;
      const T* old_ = static_cast<const T*>(a.old_lp) + pc.begin + pc.seq * a.old_skip;
      const T* ref_ = static_cast<const T*>(a.ref) + pc.begin + pc.seq * a.ref_skip;
      const T* ent_ = static_cast<const T*>(a.ent) + pc.begin + pc.seq * a.ent_skip;
      const float* adv_ = a.adv + (a.adv_per_token ? pc.begin + pc.seq * a.adv_skip : pc.seq);
      T* dlp_ = static_cast<T*>(a.dlp) + pc.begin;  // outputs are dense
      T* dent_ = static_cast<T*>(a.dent) + pc.begin;
      const bool vec_in = !(misfit(lp_, a.lp) | misfit(old_, a.old_lp) | misfit(ref_, a.ref) |
                            misfit(ent_, a.ent) | misfit(adv_, a.adv_per_token));
      const bool vec_out = !(misfit(dlp_, a.dlp) | misfit(dent_, a.dent));
      float adv_seq = 0.0f;
      if (!a.adv_per_token && !by_seq && pc.len > 0) adv_seq = __ldg(adv_);
      Pair f[3] = {};  // policy term, KL, log-ratio: terms of both signs
      float pos[2] = {0, 0};  // entropy, KL to the old policy
      int c[3] = {0, 0, 0};
#pragma unroll 1
      for (int g = 0; g < kGroups && g * kGroup4 < t1; ++g) {
        const int t = g * kGroup4 + lane * kVec;
        const unsigned int in = tokens_in(t, t0, t1);
        unsigned int on;
        float dl[kVec];
        if (grad && keep) {
          on = kept_on >> ((round * kGroups + g) * kVec);
          const float4 x = kept[(round * kGroups + g) * kSeqThreads + threadIdx.x];
          dl[0] = x.x; dl[1] = x.y; dl[2] = x.z; dl[3] = x.w;
        } else {
          // every load first, masked tokens' too: one wait
          float lp[kVec] = {}, old[kVec] = {}, ref[kVec] = {}, ent[kVec] = {}, adv[kVec] = {};
          const bool vec = vec_in && in == 15u;
          on = counted(t, in);
          if (values) {
            load4(lp_ + t, vec, in, lp);
            if (a.old_lp) load4(old_ + t, vec, in, old);
            if (a.ref) load4(ref_ + t, vec, in, ref);
            if (a.ent && !grad) load4(ent_ + t, vec, in, ent);
            if (a.adv_per_token && !by_seq) load4(adv_ + t, vec, in, adv);
          }
#pragma unroll
          for (int j = 0; j < kVec; ++j) {
            const bool counts = on >> j & 1;
            const float x = a.lp_sign * lp[j];
            float h = 0.0f, l = 0.0f;
            if (a.old_lp) exact_diff(x, old[j], h, l);
            const float hc = clamp_ratio(h), e = expf(hc), k = exp_m1_mx(hc, e);
            dl[j] = 0.0f;
            if (by_seq) {
              if (counts) {
                f[2] = f[2] + h;
                f[2].l += l;
              }
            } else {
              const float A = a.adv_per_token ? adv[j] : adv_seq;
              const Ratio r = clip_ratio(a, h, l, hc, e, k, A);
              const float ra = r.value * A;
              dl[j] = r.live ? -ra : 0.0f;
              if (counts) {
                f[0] = f[0] + -ra;
                f[0].l -= fmaf(r.value, A, -ra) + r.low * A;
                c[1] += r.clipped;
                c[2] += r.dual;
              }
            }
            if (a.ref) {
              float kl, dkl;
              kl_term(a.kl, x, ref[j], kl, dkl);
              if (counts) f[1] = f[1] + kl;
              dl[j] = fmaf(a.kl_coef, dkl, dl[j]);
            }
            if (!grad && counts) {
              pos[1] += k;
              pos[0] += ent[j];
            }
          }
          c[0] += __popc(on);
          if (!grad && keep) {
            kept[(round * kGroups + g) * kSeqThreads + threadIdx.x] =
                make_float4(dl[0], dl[1], dl[2], dl[3]);
            kept_on |= on << ((round * kGroups + g) * kVec);
          }
        }
        if (grad) {
          float o[kVec];
#pragma unroll
          for (int j = 0; j < kVec; ++j)
            o[j] = on >> j & 1 ? __fadd_rn(dl[j], coef) * w_lp * g_up : 0.0f;
          const bool vec = vec_out && in == 15u;
          if (a.dlp) store4(dlp_ + t, vec, in, o);
#pragma unroll
          for (int j = 0; j < kVec; ++j) o[j] = on >> j & 1 ? w_ent * g_up : 0.0f;
          if (a.dent) store4(dent_ + t, vec, in, o);
        }
      }
      if (!grad) {
        warp_sums(f, pos);
#pragma unroll
        for (int k = 0; k < 3; ++k) c[k] = warp_sum(c[k]);
        if (lane == 0) a.piece[u] = {f[0], f[1], f[2], pos[0], pos[1], c[0], c[1], c[2], 0};
      }
    }
    if (grad) break;
    meet(q.meet);

    // ---- sums of the sequences
    unsigned long long my_tokens = 0;
    unsigned int my_live = 0, my_seqs = 0;
    const SeqShare share(q, q.B);
    for (int64_t i = share.first; i < q.B; i += share.stride) {
      int first, last;
      if (!seq_pieces(q, i, first, last)) atomicOr(&a.totals->live, kBadSeqs);
      Pair f[5] = {};
      long long c[3] = {0, 0, 0};
      for (int u = first + share.offset; u < last; u += share.step) {
        const PolicyPiece r = a.piece[u];
        f[0] = f[0] + r.pg;
        f[1] = f[1] + r.kl;
        f[2] = f[2] + r.ent;
        f[3] = f[3] + r.old_kl;
        f[4] = f[4] + r.d;
        c[0] += r.n;
        c[1] += r.clipped;
        c[2] += r.dual;
      }
      share.sum(f, c);
      const long long n = c[0];
      if (share.writes()) {
        PolicySeq o{f[0], f[1], f[2], f[3], n, c[1], c[2], 0.0f};
        if (by_seq && n > 0) {
          const float fn = static_cast<float>(n);
          const Pair d = f[4] / fn;
          const float adv = __ldg(a.adv + i);
          const float hc = clamp_ratio(d.h), e = expf(hc);
          const Ratio r = clip_ratio(a, d.h, d.l, hc, e, exp_m1_mx(hc, e), adv);
          const float ra = r.value * adv;
          o.pg = Pair{-ra, -(fmaf(r.value, adv, -ra) + r.low * adv)} * fn;
          o.coef = r.live ? -ra : 0.0f;
          o.clipped = r.clipped;
          o.dual = r.dual;
        }
        a.seq[i] = o;
      }
      if (share.counts()) {
        my_tokens += n;
        my_live += n > 0;
        ++my_seqs;
      }
    }
    const bool late = meet_sequences(q, a.totals, my_tokens, my_live, my_seqs, a.err);

    // ---- totals and the loss
    const bool first_block = blockIdx.x == 0;
    const unsigned long long tokens = __ldcg(&a.totals->tokens);
    const unsigned int live = __ldcg(&a.totals->live);
    Pair f[5] = {};
    long long c[2] = {0, 0};
    if (first_block && want_loss) {
      for (int64_t i = threadIdx.x; i < q.B; i += kSeqThreads) {
        const PolicySeq& r = a.seq[i];
        const float n = mean_seq && r.n > 0 ? static_cast<float>(r.n) : 1.0f;
        f[0] = f[0] + r.pg / n;
        f[1] = f[1] + (r.kl * a.kl_coef + r.ent * -a.ent_coef) / n;
        f[2] = f[2] + r.kl;
        f[3] = f[3] + r.ent;
        f[4] = f[4] + r.old_kl;
        c[0] += r.clipped;
        c[1] += r.dual;
      }
      block_counts(c);
      block_sums(f, q.B);
    }
    float one_token = tokens > 0 ? 1.0f / static_cast<float>(tokens) : 0.0f;
    const float one_seq = live > 0 ? 1.0f / static_cast<float>(live) : 0.0f;
    float w_all = a.aggregate == FLCE_AGG_TOKEN_MEAN ? one_token
                  : a.aggregate == FLCE_AGG_SUM      ? a.scale
                                                     : one_seq;
    if (a.g_loss) g_up = __ldg(a.g_loss);
    wg_all = w_all;
    // no result where the offsets are bad, or the totals of a wait that ran out: NaN in the place
    // of loss, means and gradients (with the latter, those of this block's pieces)
    const bool bad = live & kBadSeqs;
    if (bad || late) w_all = one_token = __int_as_float(0x7fc00000);
    if (bad) wg_all = w_all;
    if (late) g_up = w_all;
    if (first_block && threadIdx.x == 0 && bad) atomicOr(a.err, FLCE_DEVERR_SEQS);
    if (first_block && want_loss && threadIdx.x == 0) {
      a.loss[0] = ((f[0] + f[1]) * w_all).value();
      a.stats[0] = w_all * f[0].value();
      a.stats[1] = one_token * f[2].value();
      a.stats[2] = one_token * f[3].value();
      a.stats[3] = one_token * f[4].value();
      a.counts[0] = static_cast<long long>(tokens);
      a.counts[1] = live & ~kBadSeqs;
      a.counts[2] = c[0];
      a.counts[3] = c[1];
    }
    const int64_t thread = warp * int64_t(32) + lane, threads = warps * int64_t(32);
    if (a.lp_out)  // the head's tokens: a packed axis
      for (int64_t p = thread; p < q.total; p += threads)
        a.lp_out[p] = 0.0f + a.lp_sign * load_f(static_cast<const T*>(a.lp) + p);
    if (q.cu && (a.what & POLICY_GRAD)) {
      // positions outside every sequence: all of them where the offsets are bad
      const int64_t begin = bad ? a.g_end : seq_start(q, 0), end = seq_start(q, q.B);
      const float fill = bad ? w_all : 0.0f;
      for (int64_t p = a.g_begin + thread; p < a.g_end; p += threads)
        if (p < begin || p >= end) {
          if (a.dlp) store_f(static_cast<T*>(a.dlp) + p, fill);
          if (a.dent) store_f(static_cast<T*>(a.dent) + p, fill);
        }
    }
  }
}

// A number as a sum of two floats (an infinite one as its high part alone).
void split(double b, float* h, float* l) {
  *h = static_cast<float>(b);
  *l = std::isfinite(*h) ? static_cast<float>(b - *h) : 0.0f;
}

// A border of the log-ratio likewise.  The clamped log-ratio reaches no border at or beyond the
// limit, whatever the log-ratio itself: such a border is put where nothing reaches it.
void split_border(double b, float* h, float* l) {
  split(std::fabs(b) < kLogRatioLimit ? b : std::copysign(HUGE_VAL, b), h, l);
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
  if ((p->ld_logp | p->ld_old | p->ld_ref | p->ld_entropy | p->ld_adv) < 0) return FLCE_ERR_BAD_ARG;
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
  return 256 + align256(static_cast<size_t>(q.pieces) * sizeof(PolicyPiece)) +
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
  split_border(std::log1p(p->clip_high), &a->hi_h, &a->hi_l);
  split_border(std::log1p(-p->clip_low), &a->lo_h, &a->lo_l);
  if (p->dual_clip != 0.0) split_border(std::log(p->dual_clip), &a->dual_h, &a->dual_l);
  split(1.0 + p->clip_high, &a->r_hi, &a->r_hi_l);
  split(1.0 - p->clip_low, &a->r_lo, &a->r_lo_l);
  split(p->dual_clip, &a->r_dual, &a->r_dual_l);
  a->kl_coef = static_cast<float>(p->kl_coef);
  a->ent_coef = static_cast<float>(p->entropy_coef);
  a->scale = static_cast<float>(p->scale);
  a->kl = p->kl;
  a->ratio = p->ratio;
  a->aggregate = p->aggregate;
  a->g_end = a->q.total;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a->err = reinterpret_cast<uint32_t*>(ws);
  a->err_store = 1;
  a->totals = reinterpret_cast<SeqTotals*>(ws + 64);
  a->piece = reinterpret_cast<PolicyPiece*>(ws + 256);
  a->seq = reinterpret_cast<PolicySeq*>(ws + 256 + align256(static_cast<size_t>(a->q.pieces) * sizeof(PolicyPiece)));
  return FLCE_OK;
}

int launch_policy(const PolicyArgs& a, int dtype, int sms, cudaStream_t st) {
  // loss and gradients in one launch: gradients wait in shared memory
  const int kept = a.what == (POLICY_LOSS | POLICY_GRAD) ? kTile * 4 : 0;
  cudaError_t e;
  if (dtype == FLCE_F32)
    e = launch_seq(policy_kernel<float>, a, kept, sms, st);
  else if (dtype == FLCE_BF16)
    e = launch_seq(policy_kernel<__nv_bfloat16>, a, kept, sms, st);
  else
    e = launch_seq(policy_kernel<__half>, a, kept, sms, st);
  return e == cudaSuccess ? FLCE_OK : FLCE_ERR_CUDA;
}

}  // namespace flce

using namespace flce;

extern "C" {

int flce_policy_check_params(const flce_policy_params* p) { return policy_check(p); }

size_t flce_policy_workspace_size(const flce_policy_params* p) {
  return policy_check(p) == FLCE_OK ? policy_workspace(p) : 0;
}

}  // extern "C"

namespace {

// `missing`: sequences that the second meeting waits for in vain (the self-test's).
int policy_loss(const flce_policy_params* p, const void* logp, const void* old_logp,
                const void* ref_logp, const void* entropy, const float* advantages,
                const float* g_loss, float* loss, float* stats, int64_t* counts, void* dlogp,
                void* dentropy, void* workspace, size_t ws_bytes, void* stream,
                unsigned int missing) {
  int rc = policy_check(p);
  if (rc) return rc;
  if (!workspace || (loss == nullptr) != (stats == nullptr) ||
      (loss == nullptr) != (counts == nullptr))
    return FLCE_ERR_BAD_ARG;
  if (!loss && !dlogp && !dentropy) return FLCE_ERR_BAD_ARG;
  PolicyArgs a;
  if ((rc = policy_args(p, workspace, &a))) return rc;
  // (no sequences, no advantages: an empty array has no address)
  if (a.q.total > 0 && (!logp || (!advantages && (a.q.B > 0 || a.adv_per_token))))
    return FLCE_ERR_BAD_ARG;
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
  a.q.awaited += missing;
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

}  // namespace

extern "C" {

int flce_policy_loss(const flce_policy_params* p, const void* logp, const void* old_logp,
                     const void* ref_logp, const void* entropy, const float* advantages,
                     const float* g_loss, float* loss, float* stats, int64_t* counts,
                     void* dlogp, void* dentropy, void* workspace, size_t ws_bytes,
                     void* stream) {
  return policy_loss(p, logp, old_logp, ref_logp, entropy, advantages, g_loss, loss, stats, counts,
                     dlogp, dentropy, workspace, ws_bytes, stream, 0);
}

int flce_selftest_policy_timeout(const flce_policy_params* p, const void* logp,
                                 const float* advantages, float* loss, float* stats,
                                 int64_t* counts, void* dlogp, void* workspace, size_t ws_bytes,
                                 void* stream) {
  return policy_loss(p, logp, nullptr, nullptr, nullptr, advantages, nullptr, loss, stats, counts,
                     dlogp, nullptr, workspace, ws_bytes, stream, 1);
}

}  // extern "C"
