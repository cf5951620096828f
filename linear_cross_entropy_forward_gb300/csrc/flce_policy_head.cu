// The policy loss on top of the head: the gradient-in-forward call (flce_api.cu) with its
// upstream gradients formed on the way.  Once a chunk's rows have their log-probabilities
// and entropies, a launch of the policy kernel writes the two gradients per row that the
// chunk's dlogits need; their weights depend on the labels alone, so no later chunk is
// waited for.  With one chunk (the usual case) that launch also forms the loss; with
// several, a last one does.
//
// The dlogits are bf16, as in flce_backward and flce_forward_backward: both gradient products
// take them as tensor-core operands, and a second operand for their low bits would double the
// products.  At 4096 x 4096 x 32000 the gradients are off by 2.3e-3 (2-norm, relative), by
// 1.7e-3 where only the outputs are rounded.  The loss of the head's log-probabilities is within
// 3e-7; these are themselves some 4e-6 too large there, from the tensor cores' accumulation.
#include "flce_policy.cuh"

namespace flce {

namespace {

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct HeadLayout {
  size_t policy, ce, lse, ez, g_loss, g_ent, total;
};

HeadLayout head_layout(const flce_params* p, const flce_policy_params* q) {
  HeadLayout L{};
  const size_t row = align256(static_cast<size_t>(p->N) * 4);
  size_t off = align256(flce_workspace_size(p, 3));
  L.policy = off; off += align256(policy_workspace(q));
  L.ce = off; off += row;
  L.lse = off; off += row;
  L.ez = off; off += row;
  L.g_loss = off; off += row;
  L.g_ent = off; off += row;
  L.total = off;
  return L;
}

int head_check(const flce_params* p, const flce_policy_params* q) {
  int rc = flce_check_params(p);
  if (rc || (rc = policy_check(q))) return rc;
  if (p->reduction != FLCE_RED_NONE || p->zloss_coef != 0.0f || p->label_smoothing != 0.0f ||
      p->class_weight || (p->v_total > 0 && p->v_total != p->V))
    return FLCE_ERR_BAD_ARG;
  if (q->seqs.dtype != FLCE_F32 || q->seqs.mask_kind != 0) return FLCE_ERR_BAD_ARG;
  if (q->seqs.S != p->N || (q->seqs.cu_kind == 0 && q->seqs.B != 1)) return FLCE_ERR_BAD_SHAPE;
  // a sequence's ratio is known once all its tokens are
  if (q->ratio == FLCE_RATIO_SEQUENCE && fused_chunks(p) > 1) return FLCE_ERR_BAD_ARG;
  return FLCE_OK;
}

struct HeadCtx {
  PolicyArgs a;
  int sms;
};

void head_begin(void* ctx, uint32_t* err) {
  PolicyArgs& a = static_cast<HeadCtx*>(ctx)->a;
  a.err = err;  // the call's own word: bits are added
  a.err_store = 0;
}

int head_mid(void* ctx, int64_t n0, int64_t rows, int64_t chunks, cudaStream_t st) {
  const HeadCtx* h = static_cast<HeadCtx*>(ctx);
  PolicyArgs a = h->a;
  a.what = POLICY_GRAD | (chunks == 1 ? POLICY_LOSS : 0);
  a.g_begin = n0;
  a.g_end = n0 + rows;
  if (chunks > 1) a.lp_out = nullptr;
  return launch_policy(a, FLCE_F32, h->sms, st);
}

int head_end(void* ctx, int64_t chunks, cudaStream_t st) {
  if (chunks == 1) return FLCE_OK;
  const HeadCtx* h = static_cast<HeadCtx*>(ctx);
  PolicyArgs a = h->a;
  a.what = POLICY_LOSS;
  return launch_policy(a, FLCE_F32, h->sms, st);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

size_t flce_policy_head_workspace_size(const flce_params* p, const flce_policy_params* q) {
  return head_check(p, q) == FLCE_OK ? head_layout(p, q).total : 0;
}

int flce_policy_forward_backward(const flce_params* p, const flce_policy_params* q,
                                 const void* hidden, const void* weight, const int64_t* labels,
                                 const float* old_logp, const float* ref_logp,
                                 const float* advantages, const float* g_loss, float* loss,
                                 float* stats, int64_t* counts, float* logp, float* entropy,
                                 void* dhidden, void* dweight, void* workspace,
                                 size_t ws_bytes, void* stream) {
  int rc = head_check(p, q);
  if (rc) return rc;
  if (!workspace || !loss || !stats || !counts) return FLCE_ERR_BAD_ARG;
  const bool no_adv = !advantages && (q->seqs.B > 0 || q->adv_per_token);
  if (p->N > 0 && (no_adv || !entropy || !logp || !labels || (q->kl_coef != 0.0 && !ref_logp)))
    return FLCE_ERR_BAD_ARG;
  const uintptr_t f4 = reinterpret_cast<uintptr_t>(old_logp) |
                       reinterpret_cast<uintptr_t>(ref_logp) |
                       reinterpret_cast<uintptr_t>(advantages) |
                       reinterpret_cast<uintptr_t>(g_loss) | reinterpret_cast<uintptr_t>(loss) |
                       reinterpret_cast<uintptr_t>(stats) | reinterpret_cast<uintptr_t>(logp);
  if ((f4 & 3) || (reinterpret_cast<uintptr_t>(counts) & 7) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255))
    return FLCE_ERR_ALIGN;
  const HeadLayout L = head_layout(p, q);
  if (ws_bytes < L.total) return FLCE_ERR_WS_TOO_SMALL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  HeadCtx h{};
  if ((rc = policy_args(q, ws + L.policy, &h.a))) return rc;
  if ((rc = require_device(&h.sms))) return rc;
  PolicyArgs& a = h.a;
  float* ce = reinterpret_cast<float*>(ws + L.ce);
  if (!entropy) entropy = ce;  // no rows
  a.q.mask = labels;
  a.q.mask_labels = 1;
  a.q.ignore_index = p->ignore_index;
  a.q.mask_skip = 0;
  a.lp = ce;
  a.lp_sign = -1.0f;
  a.old_lp = old_logp;
  a.ref = ref_logp;
  a.ent = entropy;
  a.lp_skip = a.old_skip = a.ref_skip = a.ent_skip = a.adv_skip = 0;
  a.adv = advantages;
  a.g_loss = g_loss;
  a.loss = loss;
  a.stats = stats;
  a.counts = reinterpret_cast<long long*>(counts);
  a.dlp = ws + L.g_loss;
  a.dent = ws + L.g_ent;
  a.lp_out = logp;
  flce_params p2 = *p;
  p2.validate |= q->validate;
  const GradHook hook{&h, head_mid, head_end, head_begin};
  return forward_backward(&p2, hidden, weight, labels, reinterpret_cast<float*>(ws + L.g_loss),
                          reinterpret_cast<float*>(ws + L.g_ent), ce, entropy,
                          reinterpret_cast<float*>(ws + L.lse),
                          reinterpret_cast<float*>(ws + L.ez), dhidden, dweight, workspace,
                          flce_workspace_size(p, 3), stream, &hook);
}

}  // extern "C"
