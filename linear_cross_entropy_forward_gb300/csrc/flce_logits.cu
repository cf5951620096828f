// C entries of the processed logits: checks, and the kernels' arguments.
#include "flce_logits.cuh"

namespace flce {
namespace {

using namespace logits;

inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }
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
  x.split = p->split_lse != 0;
  return FLCE_OK;
}

int launch(const flce_logits_params* p, Args a, int mode, void* workspace, cudaStream_t st) {
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
    if (!a.tokens) a.T = 0;
    const int count = !a.tokens && a.n_bias == 0 ? 0 : a.T >= 1 << 14 ? 32 : 16;
    rc = (p->dtype == FLCE_F32 ? run_f32 : p->dtype == FLCE_BF16 ? run_bf16 : run_f16)(a, count, mode,
                                                                                      sms, st);
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
  return launch(p, a, out && !labels && !logp && !entropy ? MODE_PROCESS : MODE_FORWARD, workspace, static_cast<cudaStream_t>(stream));
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
  return launch(p, a, MODE_BACKWARD, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
