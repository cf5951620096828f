// The clipped policy loss: host arguments of its one kernel (flce_policy.cu), which the
// head's gradient-in-forward call also launches on ranges of its tokens.
#pragma once

#include "flce_host.h"
#include "flce_seq.cuh"

namespace flce {

// One sequence's sums over its tokens.
struct PolicySeq {
  Pair pg, kl, ent, old_kl;
  long long n;
  long long clipped, dual;
  float coef;  // d(loss)/d(mean log-ratio) before the weight (sequence ratios only)
};

// A piece's sums.
struct PolicyPiece {
  Pair pg, kl, d;  // of both signs
  float ent, old_kl;
  int n, clipped, dual, pad;
};

// What a launch is for.
enum : int {
  POLICY_LOSS = 1,   // the loss, the means and the counts
  POLICY_GRAD = 2    // the gradients of the positions [g_begin, g_end)
};

struct PolicyArgs {
  Seqs q;
  const void *lp, *old_lp, *ref, *ent;
  int64_t lp_skip, old_skip, ref_skip, ent_skip, adv_skip;
  const float* adv;
  int adv_per_token;
  float lp_sign;  // -1: lp holds negative log-probabilities, as does the gradient
  // clipping borders of the log-ratio, as unevaluated sums of two floats
  float hi_h, hi_l, lo_h, lo_l, dual_h, dual_l;
  // the ratio beyond the borders, as sums of two floats; r_dual 0: no dual clip
  float r_hi, r_hi_l, r_lo, r_lo_l, r_dual, r_dual_l;
  float kl_coef, ent_coef;
  float scale;
  int kl, ratio, aggregate, what;
  int64_t g_begin, g_end;
  const float* g_loss;
  float *loss, *stats;
  long long* counts;
  void *dlp, *dent;
  float* lp_out;
  uint32_t* err;
  int err_store;  // the word is this launch's own and cleared by it
  SeqTotals* totals;
  PolicyPiece* piece;
  PolicySeq* seq;
};

size_t policy_workspace(const flce_policy_params* p);
// Checks of the parameters alone.
int policy_check(const flce_policy_params* p);
// The arguments every launch of these parameters shares; the workspace has
// policy_workspace() bytes.
int policy_args(const flce_policy_params* p, void* workspace, PolicyArgs* a);
int launch_policy(const PolicyArgs& a, int dtype, int sms, cudaStream_t st);

}  // namespace flce
