/*
 * flce.h -- C ABI of the fused linear cross-entropy + entropy library (libflce.so)
 * for NVIDIA GB300 (sm_103a).
 *
 * The operation (verl PR #462, "Equivalent compute logic" and "API"):
 *     logits  = hidden[N,H] @ weight[H,V]                (never stored)
 *     z       = softcap * tanh(logits / softcap)          (softcap > 0 only;
 *                                                          Liger-Kernel issue #127)
 *     p       = softmax(z) over the vocabulary
 *     lse_n   = logsumexp_v z_nv,   Ez_n = sum_v p_nv z_nv
 *     ce_n    = lse_n - z_{n,y_n}                         (the page returns -ce as logprobs)
 *     ent_n   = lse_n - Ez_n                              (entropy of p_n)
 *     loss_n  = ce_n + zloss_coef * lse_n^2               (z-loss: Liger-Kernel PR #435,
 *                                                          "Changes Made"; formula is a reading)
 *   With label smoothing eps and per-class weights w (options named in the
 *   Liger-Kernel PR #551 review; defined as torch's cross_entropy(weight,
 *   label_smoothing)): ce_n = (1-eps) w_{y_n} (lse_n - z_{n,y_n})
 *                             + eps/V sum_v w_v (lse_n - z_nv);
 *   the mean then divides the sum of ce_n by the sum of w_{y_n} over non-ignored
 *   rows, while z-loss and entropy stay unweighted (divided by the row count).
 *   Rows whose label equals ignore_index contribute exactly 0 to loss and entropy
 *   (Liger-Kernel PR #551, review: mean divides by the non-ignored count).
 *   Reduction (Liger-Kernel PR #435, "Summary"): NONE returns loss[N], entropy[N];
 *   SUM returns the sums over non-ignored rows; MEAN divides both sums by the
 *   number of non-ignored rows (0 when every row is ignored).
 *
 *   Backward, for upstream gradients g_loss, g_entropy (per token for NONE,
 *   scalars otherwise; scaled by 1/n_valid for MEAN; zero on ignored rows):
 *     dz_nv   = gl_n (p_nv - [v == y_n] + 2 coef lse_n p_nv) - ge_n p_nv (z_nv - Ez_n)
 *     dz'_nv  = dz_nv (1 - (z_nv/softcap)^2)              (soft-cap chain rule)
 *     dhidden = dz' @ weight^T,   dweight = hidden^T @ dz'
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers to dense row-major arrays, owned by
 *     the caller; the library allocates no device memory and keeps no state
 *     between calls apart from per-device caches (device attributes, the no-alloc
 *     scratch address) and the per-thread side streams described below.
 *   - hidden, weight, dhidden, dweight: bf16 (IEEE bfloat16 bit patterns; dhidden fp32
 *     when params->dhidden_fp32 is set); weight and dweight are [H,V] or [V,H] as
 *     params->weight_layout says.
 *     labels: int64.  Everything else: fp32.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  All work is
 *     enqueued asynchronously on it; nothing synchronises unless params->validate
 *     is set.  The backward passes run their dweight GEMM beside dhidden on an
 *     internal stream (one per host thread and device, created on first use and
 *     destroyed when the thread exits) that
 *     is forked from `stream` by an event and joined back before the call returns,
 *     so every call's work still follows the work enqueued on `stream` before it and
 *     precedes the work enqueued after it.
 *   - Return value: FLCE_OK or one of the FLCE_ERR_* codes below.  Argument errors
 *     are detected on the host before anything is enqueued.  Device-side
 *     conditions (a label outside [0,V) that is not ignore_index, a pipeline wait
 *     that timed out) are recorded in an error word inside the workspace; they
 *     are returned by flce_status(), or directly when params->validate != 0.
 *   - Requirements: N >= 0, H >= 8, V >= 1, H % 8 == 0, and V % 8 == 0 for a [H,V]
 *     weight (16-byte row strides for the TMA engine; a [V,H] weight takes any V).
 *     Row lengths that are multiples of 64 elements (whole 128-byte lines) run
 *     faster: ~11 % in the forward GEMM otherwise.  Every tensor pointer 16-byte aligned (g_loss,
 *     g_entropy and class_weight: 4-byte; an fp32 dhidden: 32-byte), every workspace
 *     256-byte aligned.
 */
#ifndef FLCE_H_
#define FLCE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Storage of weight (and of dweight, which always matches it).  WEIGHT_HV is the
 * [H,V] matrix of the pages' logits = hidden @ weight (verl PR #462, "API");
 * WEIGHT_VH is the transposed [V,H] layout of a torch nn.Linear LM head (the
 * layout Liger-Kernel issue #127 works with), logits = hidden @ weight^T. */
typedef enum {
  FLCE_WEIGHT_HV = 0,
  FLCE_WEIGHT_VH = 1
} flce_weight_layout;

typedef enum {
  FLCE_RED_NONE = 0,
  FLCE_RED_MEAN = 1,
  FLCE_RED_SUM = 2
} flce_reduction;

enum {
  FLCE_OK = 0,
  FLCE_ERR_BAD_ARG = 1,       /* NULL pointer, bad reduction, negative coefficient */
  FLCE_ERR_BAD_SHAPE = 2,     /* N, H or V out of the supported range; cu_seqlens out of order */
  FLCE_ERR_ALIGN = 3,         /* H (or a [H,V] weight's V) not a multiple of 8, or a pointer
                               * not 16-byte aligned */
  FLCE_ERR_WS_TOO_SMALL = 4,  /* ws_bytes < flce_workspace_size(...) */
  FLCE_ERR_LABEL = 5,         /* a label outside [0, V) that is not ignore_index */
  FLCE_ERR_TIMEOUT = 6,       /* a device pipeline wait exceeded its time limit */
  FLCE_ERR_CUDA = 7,          /* a CUDA runtime/driver call failed */
  FLCE_ERR_DEVICE = 8,        /* current device is not an sm_103 GPU */
  FLCE_ERR_SCRATCH_LIMIT = 9, /* problem needs more than FLCE_NOALLOC_SCRATCH_BYTES */
  FLCE_ERR_BOUNDS = 10        /* libflce_debug.so only: an in-kernel bounds check failed
                               * (the access was skipped; results are not valid) */
};

typedef struct {
  int64_t N;             /* tokens (rows of hidden) */
  int64_t H;             /* hidden size */
  int64_t V;             /* vocabulary size */
  int64_t ignore_index;  /* label value that marks an ignored row (usually -100) */
  int32_t reduction;     /* flce_reduction */
  float zloss_coef;      /* z-loss coefficient, 0 = off */
  float softcap;         /* tanh logit soft-cap c, 0 = off */
  int32_t validate;      /* != 0: synchronise at the end and report device errors */
  int64_t chunk_v;       /* backward vocabulary chunk width (multiple of 256), 0 = auto:
                          * the widest whose bf16 dlogits [N, chunk_v] fit 2 GiB */
  int32_t weight_layout; /* flce_weight_layout: how weight and dweight are stored */
  float label_smoothing; /* eps in [0, 1], 0 = off */
  const float* class_weight; /* [V] fp32 device pointer, per-class target weights; NULL = all 1 */
  /* Vocabulary sharding (see flce_shard_stats).  v_total = 0: weight holds the whole
   * vocabulary.  v_total > 0: weight holds columns [v_offset, v_offset + V) of a
   * vocabulary of v_total entries, and labels are indices into the whole vocabulary.
   * Sharding excludes label_smoothing and class_weight. */
  int64_t v_offset;
  int64_t v_total;
  /* flce_forward_backward's token chunk (a multiple of 512), 0 = auto: the largest
   * chunk whose fp32 logits and bf16 dlogits fit in 8 GiB. */
  int64_t chunk_n;
  /* 0: dhidden is bf16 [N,H].  1: dhidden is fp32 [N,H] (32-byte aligned), the
   * unrounded fp32 accumulation -- for a vocabulary shard's dhidden term, so that the
   * sum over the shards is rounded once, after the exchange, not once per shard. */
  int32_t dhidden_fp32;
} flce_params;

/* FLCE_OK, or the status every entry point returns for these parameters (checked
 * on the host before any pointer is looked at): FLCE_ERR_BAD_ARG, FLCE_ERR_BAD_SHAPE
 * or FLCE_ERR_ALIGN. */
int flce_check_params(const flce_params* params);

/* Bytes of device workspace that flce_forward / flce_shard_stats (phase 0),
 * flce_backward (phase 1), flce_combine_shards (phase 2) or flce_forward_backward
 * (phase 3) needs for these parameters; 0 when the parameters are invalid.  The workspace is scratch: its
 * contents need not be preserved between calls. */
size_t flce_workspace_size(const flce_params* params, int phase);

/* Forward pass.
 *   hidden  [N,H] bf16, weight [H,V] (or [V,H]) bf16, labels [N] int64.
 *   loss, entropy: [N] fp32 for FLCE_RED_NONE, [1] fp32 otherwise (overwritten).
 *   lse, ez: [N] fp32, per-row logsumexp and softmax mean E_p[z] of the capped
 *     logits, written for every row (ignored ones too); flce_backward needs them.
 *   workspace: >= flce_workspace_size(params, 0) bytes, 256-byte aligned. */
int flce_forward(const flce_params* params, const void* hidden, const void* weight,
                 const int64_t* labels, float* loss, float* entropy, float* lse, float* ez,
                 void* workspace, size_t ws_bytes, void* stream);

/* Backward pass (logits are recomputed tile by tile; no [N,V] array exists).
 *   hidden, weight, labels: as given to flce_forward.
 *   lse, ez: the [N] outputs of flce_forward for the same inputs and params.
 *   g_loss, g_entropy: upstream gradients of loss and entropy, [N] for
 *     FLCE_RED_NONE, [1] otherwise; NULL means zero.
 *   dhidden [N,H] bf16 (fp32 with params->dhidden_fp32), dweight [H,V] (or [V,H], as
 *   weight) bf16: overwritten.
 *   workspace: >= flce_workspace_size(params, 1) bytes, 256-byte aligned. */
int flce_backward(const flce_params* params, const void* hidden, const void* weight,
                  const int64_t* labels, const float* lse, const float* ez,
                  const float* g_loss, const float* g_entropy, void* dhidden, void* dweight,
                  void* workspace, size_t ws_bytes, void* stream);

/* Forward and backward in one call, for callers that know the upstream gradients
 * when they run the forward (Liger-Kernel PR #551, "gradient in forward"; in a
 * training step the loss's gradient is 1, scaled by the reduction).  Per chunk of
 * params->chunk_n tokens the logits are computed once, kept in the workspace in
 * fp32 next to their online-softmax statistics, turned into dlogits once the
 * rows' logsumexp is known, and contracted into dhidden and dweight: 6*N*H*V
 * flops instead of flce_forward + flce_backward's 8*N*H*V (no recompute), at the
 * cost of an [chunk_n, V] fp32 + bf16 workspace.
 *   Arguments: as flce_forward's and flce_backward's (g_loss, g_entropy: [N] for
 *   FLCE_RED_NONE, [1] otherwise, NULL = zero).  loss, entropy, lse, ez,
 *   dhidden and dweight are all written, with the values the two-call path
 *   gives (the dlogits are bitwise the same).  Vocabulary sharding
 *   (v_total > 0 with a partial shard) is rejected with FLCE_ERR_BAD_ARG.
 *   workspace: >= flce_workspace_size(params, 3) bytes, 256-byte aligned. */
int flce_forward_backward(const flce_params* params, const void* hidden, const void* weight,
                          const int64_t* labels, const float* g_loss, const float* g_entropy,
                          float* loss, float* entropy, float* lse, float* ez, void* dhidden,
                          void* dweight, void* workspace, size_t ws_bytes, void* stream);

/* x[i] = bf16(g[0] * x[i]) for the n bf16 values at x (16-byte aligned), on
 * `stream`, with a zero product stored as +0 (so rows of zeros stay bitwise zero
 * under a negative g[0]); the kernel returns at once when g[0] == 1.  It scales
 * flce_forward_backward's dhidden and dweight when the upstream gradient of the
 * loss becomes known only after the forward (autograd's backward).  Not part of
 * the pages' method: a helper of the gradient-in-forward mode. */
int flce_scale_bf16(void* x, int64_t n, const float* g, void* stream);

/* Vocabulary-parallel forward, step 1 (the softmax statistics are split over
 * shards of the vocabulary and merged with the online-softmax max-rescale).
 *   params: V, v_offset, v_total describe this shard; weight is its slice, stored
 *   as params->weight_layout says ([H,V] or [V,H] with V the shard width).
 *   stats: [4, N] fp32, overwritten: per row, over the shard's columns, the maximum
 *   m of log2e * z, d = sum 2^(log2e z - m), s = sum 2^(log2e z - m) (log2e z - m),
 *   and the label's logit z_y if the label falls in the shard (else 0).
 *   workspace: >= flce_workspace_size(params, 0) bytes. */
int flce_shard_stats(const flce_params* params, const void* hidden, const void* weight,
                     const int64_t* labels, float* stats, void* workspace, size_t ws_bytes,
                     void* stream);

/* Vocabulary-parallel forward, step 2: merge the stats of all shards.
 *   stats: [n_shards, 4, N] fp32, each shard's flce_shard_stats output (as an
 *   all-gather across ranks produces it).  Outputs as flce_forward's, for the whole
 *   vocabulary (params->v_total entries).  workspace: >= flce_workspace_size(params, 2).
 *   Of params only N, ignore_index, reduction, zloss_coef, validate and v_total are
 *   used; the shard fields (V, v_offset, weight_layout) need only be a valid shard of
 *   v_total, e.g. the whole vocabulary as one [V,H] shard, which takes any v_total. 
 * The backward of a shard is flce_backward with the same sharded params and weight
 * slice: it writes that shard's dweight and this shard's term of dhidden, which the
 * caller sums over the shards. */
int flce_combine_shards(const flce_params* params, const float* stats, int32_t n_shards,
                        const int64_t* labels, float* loss, float* entropy, float* lse,
                        float* ez, void* workspace, size_t ws_bytes, void* stream);

/* Synchronises `stream` and returns the device-side status recorded in the
 * workspace header by the last call that used this workspace (FLCE_OK,
 * FLCE_ERR_LABEL, FLCE_ERR_BAD_SHAPE for cu_seqlens out of order, FLCE_ERR_TIMEOUT or, with
 * libflce_debug.so, FLCE_ERR_BOUNDS), or FLCE_ERR_CUDA. */
int flce_status(const void* workspace, void* stream);

/* Number of kernels one call with these parameters enqueues (memsets not counted):
 * phase 0 flce_forward, 1 flce_backward, 2 flce_combine_shards, 3 flce_shard_stats,
 * 4 flce_forward_backward; -1 when invalid. */
int flce_kernel_launches(const flce_params* params, int phase);

/* Self-test of the device-side failure detection (no counterpart on the pages): one
 * kernel thread waits, with the bounded wait every pipeline kernel uses, on an
 * mbarrier that nothing arrives on, gives up after limit_ns of global time
 * (0 < limit_ns <= 2 s) and records the timeout in the workspace header, then returns.
 * Afterwards flce_status(workspace, stream) reports FLCE_ERR_TIMEOUT and the CUDA
 * context stays usable.  workspace: >= 256 bytes, 256-byte aligned.  Returns
 * FLCE_OK once the kernel is enqueued (the timeout is the expected outcome). */
int flce_selftest_wait_timeout(void* workspace, size_t ws_bytes, uint64_t limit_ns, void* stream);

/* Diagnostic (no counterpart on the pages): the schedule the library plans for one of
 * its GEMMs, from the GEMM's shape in tiles and the GPU's capacity; host arithmetic
 * only, usable without a GPU.
 *   m_tiles, n_tiles: output tiles (256 rows x 256 columns); raster: 0 = the M tiles
 *   vary fastest in the persistent schedule, 1 = the N tiles; panel_bytes: bytes of the
 *   operand every tile of a raster group revisits, per tile of the fast dimension;
 *   a_hint, b_hint: the L2 policy wanted for the A / B loads (0 normal, 1 evict-first,
 *   2 evict-last); pairs: CTA pairs the GPU holds at once (76 on a 152-SM GB300).
 *   out[3] receives: tiles of the fast dimension per raster group, and the L2
 *   policies of the A and B loads.
 * Returns FLCE_OK, or FLCE_ERR_BAD_ARG for a NULL out or an out-of-range argument. */
int flce_plan_tiles(int32_t m_tiles, int32_t n_tiles, int32_t raster, int64_t panel_bytes,
                    int32_t a_hint, int32_t b_hint, int32_t pairs, int32_t* out);

/* Static, NUL-terminated description of a status code. */
const char* flce_strerror(int code);

/* Forward pass for callers that cannot allocate device memory.  (The pages have
 * no counterpart: this entry point serves callers that can't call cudaMalloc, e.g.
 * code whose device memory a framework or serving runtime hands out up front and
 * keeps, or code under an allocator it does not own, which therefore cannot
 * provide the workspace flce_forward needs.)
 *   Same arguments and results as flce_forward, minus the workspace, and the same
 *   kernels in the same order, so the results are bitwise flce_forward's.  The
 *   scratch it uses is a static device array of FLCE_NOALLOC_SCRATCH_BYTES (64 MiB)
 *   held by every GPU that loads the library until the process exits; problems
 *   whose flce_workspace_size(params, 0) exceeds it return FLCE_ERR_SCRATCH_LIMIT
 *   without enqueueing anything.  Nothing is allocated (no cudaMalloc/cudaFree).
 *   The first call on a device looks up the array's device address (once, with
 *   that device current, through the runtime's symbol lookup).  All calls
 *   share the array (its header is cleared on every call; the rest is fully
 *   rewritten), so calls that may overlap on the GPU -- other streams, other
 *   threads -- race and must be serialised by the caller.  flce_status() is not
 *   available for it; set params->validate to get device-side errors returned
 *   (the call then waits for `stream` and copies the error word to the host
 *   before it returns). */
#define FLCE_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
int flce_forward_noalloc(const flce_params* params, const void* hidden, const void* weight,
                         const int64_t* labels, float* loss, float* entropy, float* lse,
                         float* ez, void* stream);

/* ------------------------------------------------------------------------------------
 * Losses over sequences of tokens, and the embedding lookup: what stands before and
 * behind the head in a fine-tuning step.  Conventions as above; these calls use one
 * launch each for the losses (loss and gradients together), and three for the
 * embedding's gradient.  Their sums have a fixed order: results repeat bit for bit.
 * Grids of up to eight blocks are clusters, the losses' and the sort's larger ones cooperative
 * launches.
 * ---------------------------------------------------------------------------------- */

enum { FLCE_F32 = 0, FLCE_BF16 = 1, FLCE_F16 = 2 };

/* A batch of B sequences of tokens, B * S at most 2^38 (S, where packed), and about 2^31
 * pieces of 256 tokens, no two sequences in one.
 *   padded (cu_kind 0): arrays [B, S], each with its own row stride ld_* in elements
 *     (>= 0; the last dimension dense);
 *   packed: arrays [S] (S tokens in all), sequence i owning [cu_seqlens[i],
 *     cu_seqlens[i + 1]), cu_seqlens [B + 1] int32 (cu_kind 1) or int64 (cu_kind 2), rising,
 *     inside [0, S].  Tokens before the first or behind the last sequence do not count
 *     and have zero gradients.  Offsets out of order or out of range are reported as
 *     FLCE_ERR_BAD_SHAPE by flce_status (or with validate); the loss, its means or
 *     rewards, and all gradients are then NaN, and no access leaves the arrays.
 *   mask_kind 0: every token counts; 1: bytes, non-zero counts; 2: int64 labels, those
 *     other than ignore_index count.  What does not count is not looked at: it may hold
 *     anything, infinities and NaN included.
 *   dtype: of the log-probabilities, entropies and their gradients. */
typedef struct {
  int64_t B, S;
  const void* cu_seqlens;
  const void* mask;
  int64_t ld_mask;
  int64_t ignore_index;
  int32_t cu_kind;
  int32_t mask_kind;
  int32_t dtype;
} flce_seqs;

enum { FLCE_KL_K1 = 1, FLCE_KL_K2 = 2, FLCE_KL_K3 = 3 };
enum { FLCE_RATIO_TOKEN = 0, FLCE_RATIO_SEQUENCE = 1 };
enum {
  FLCE_AGG_TOKEN_MEAN = 0,          /* sum over tokens / counted tokens */
  FLCE_AGG_SEQ_MEAN_TOKEN_MEAN = 1, /* mean over sequences of the token means */
  FLCE_AGG_SEQ_MEAN_TOKEN_SUM = 2,  /* mean over sequences of the token sums */
  FLCE_AGG_SUM = 3                  /* scale * sum over tokens */
};

/* Clipped policy loss.  Per counted token, with d = logp - old_logp (0 without old_logp),
 * r = exp(d), A the advantage:
 *   l = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)   (A < 0, dual_clip c > 1: not
 *                                                            above -c A)
 *       + kl_coef K(logp, ref_logp) - entropy_coef H
 *   K: k1 = logp - ref, k2 = (logp - ref)^2 / 2, k3 = exp(ref - logp) - 1 - (ref - logp)
 * d, and ref - logp in k3, are clamped to +-20, with zero gradient beyond.  With
 * FLCE_RATIO_SEQUENCE d is its mean over the sequence's counted tokens and A is per
 * sequence.  Sequences without a counted token do not count.  clip_high may be infinite. */
typedef struct {
  flce_seqs seqs;
  int64_t ld_logp, ld_old, ld_ref, ld_entropy, ld_adv;
  double clip_low, clip_high, dual_clip, kl_coef, entropy_coef, scale;
  int32_t kl, ratio, aggregate;
  int32_t adv_per_token; /* advantages [B, S] / [S] (ld_adv), else [B] */
  int32_t validate;
} flce_policy_params;

int flce_policy_check_params(const flce_policy_params* params);
size_t flce_policy_workspace_size(const flce_policy_params* params);

/* Loss and gradients in one launch.
 *   logp, old_logp, ref_logp, entropy: seqs.dtype (old_logp NULL: the policy itself;
 *     ref_logp NULL with kl_coef 0; entropy NULL with entropy_coef 0); advantages fp32.
 *   loss [1], stats [4] fp32 = aggregated policy term, mean KL to the reference, mean
 *     entropy, mean KL to the old policy (k3), means over counted tokens; counts [4] int64 =
 *     counted tokens, sequences with one, clipped tokens (sequences), dual-clipped ones.
 *     All three or none.
 *   dlogp, dentropy: dense [B, S] or [S], seqs.dtype: the gradients times g_loss[0] (NULL: 1).
 *     Either may be NULL. */
int flce_policy_loss(const flce_policy_params* params, const void* logp, const void* old_logp,
                     const void* ref_logp, const void* entropy, const float* advantages,
                     const float* g_loss, float* loss, float* stats, int64_t* counts, void* dlogp,
                     void* dentropy, void* workspace, size_t ws_bytes, void* stream);

/* flce_forward_backward of the policy loss on top of the head: log-probabilities and
 * entropies of the labels from hidden and weight, the loss, dhidden and dweight, at
 * 6*N*H*V flops (the logits are not recomputed).
 *   params: as flce_forward_backward's with reduction FLCE_RED_NONE, without z-loss, label
 *     smoothing, class weights or shards; N tokens.
 *   policy: packed (cu_seqlens) or one sequence (padded, B = 1), S = N, dtype FLCE_F32,
 *     mask_kind 0: the labels other than ignore_index count.  A sequence ratio needs all
 *     tokens in one chunk (chunk_n >= N).
 *   logp, entropy: [N] fp32 outputs.  The others as in the two calls.
 *   workspace: >= flce_policy_head_workspace_size(params, policy). */
size_t flce_policy_head_workspace_size(const flce_params* params,
                                       const flce_policy_params* policy);
int flce_policy_forward_backward(const flce_params* params, const flce_policy_params* policy,
                                 const void* hidden, const void* weight, const int64_t* labels,
                                 const float* old_logp, const float* ref_logp,
                                 const float* advantages, const float* g_loss, float* loss,
                                 float* stats, int64_t* counts, float* logp, float* entropy,
                                 void* dhidden, void* dweight, void* workspace,
                                 size_t ws_bytes, void* stream);

enum {
  FLCE_PREF_SIGMOID = 0, /* -(1 - e) ln sig(h) - e ln sig(-h) */
  FLCE_PREF_ROBUST = 1,  /* (-(1 - e) ln sig(h) + e ln sig(-h)) / (1 - 2 e) */
  FLCE_PREF_HINGE = 2,   /* max(0, 1 - h) */
  FLCE_PREF_IPO = 3      /* (h / beta - 1 / (2 beta))^2 */
};

/* Preference loss over B / 2 pairs of sequences (B even): chosen c, rejected r,
 *   s_i = sum over counted tokens of (logp - ref_logp)  [/ their number: length_normalised]
 *         - ref_scores[i],
 *   h = beta (s_c - s_r) - margin; the loss of the pair by kind, plus
 *   nll_coef * (-(mean over c's counted tokens of logp)).
 * interleaved 0: sequence i < B / 2 is chosen and B / 2 + i its rejected one; 1: 2i and
 * 2i + 1.  Pairs with a side without a counted token do not count. */
typedef struct {
  flce_seqs seqs;
  int64_t ld_logp, ld_ref;
  double beta, margin, label_smoothing, nll_coef;
  int32_t kind, length_normalised, interleaved;
  int32_t reduction; /* flce_reduction, over the counted pairs */
  int32_t validate;
} flce_preference_params;

int flce_preference_check_params(const flce_preference_params* params);
size_t flce_preference_workspace_size(const flce_preference_params* params);

/* Loss and gradient in one launch.
 *   ref_logp: as logp, or NULL; ref_scores: [B] fp32 reference scores, or NULL.
 *   loss: [1], or [B / 2] for FLCE_RED_NONE; rewards [B] = beta s_i (0 where nothing
 *     counts).  Both or none.
 *   dlogp: dense, seqs.dtype, times g_loss ([1], or [B / 2] for FLCE_RED_NONE; NULL: 1). */
int flce_preference_loss(const flce_preference_params* params, const void* logp,
                         const void* ref_logp, const float* ref_scores, const float* g_loss,
                         float* loss, float* rewards, void* dlogp, void* workspace,
                         size_t ws_bytes, void* stream);

/* Self-tests of the bounded wait between the blocks of these two losses: the call with one
 * sequence (pair) awaited that never comes.  A batch of more than 256 pieces takes a grid whose
 * blocks give up after 2 s: loss, means and the gradients of counted tokens are then NaN, and
 * flce_status (or validate) reports FLCE_ERR_TIMEOUT.  Smaller batches do not wait that way. */
int flce_selftest_policy_timeout(const flce_policy_params* params, const void* logp,
                                 const float* advantages, float* loss, float* stats,
                                 int64_t* counts, void* dlogp, void* workspace, size_t ws_bytes,
                                 void* stream);
int flce_selftest_preference_timeout(const flce_preference_params* params, const void* logp,
                                     float* loss, float* rewards, void* dlogp, void* workspace,
                                     size_t ws_bytes, void* stream);

/* Embedding lookup out[n] = scale * weight[ids[n]] and its gradient. */
typedef struct {
  int64_t N, H, V;     /* ids, row length, rows of weight (1 <= H <= 2^28) */
  int64_t v_offset;    /* weight holds rows [v_offset, v_offset + V) of a table of v_total */
  int64_t v_total;     /* 0: the whole table */
  int64_t padding_idx; /* an id without a gradient, -1: none */
  double scale;
  int32_t dtype;       /* of weight, out and dout */
  int32_t grad_dtype;  /* of dweight: dtype or FLCE_F32 */
  int32_t ids_int64;   /* 1: int64, 0: int32 */
  int32_t accumulate;  /* backward: add to dweight, whose other rows stay untouched */
  int32_t validate;
} flce_embedding_params;

int flce_embedding_check_params(const flce_embedding_params* params);
size_t flce_embedding_workspace_size(const flce_embedding_params* params);

/* Lookup.  A row of another shard is zero; an id outside the table gives a row of NaN and
 * FLCE_ERR_LABEL with validate, which needs a workspace of 256 bytes (else NULL, 0). */
int flce_embedding(const flce_embedding_params* params, const void* ids, const void* weight,
                   void* out, void* workspace, size_t ws_bytes, void* stream);

/* dweight[v] = scale * sum of dout[n] over the n with ids[n] = v (added to dweight[v] with
 * accumulate), summed in fp32 in a fixed order (32 rows of n at a time, then those) and
 * rounded once.  Ids outside the table
 * are left out and reported as FLCE_ERR_LABEL by flce_status. */
int flce_embedding_backward(const flce_embedding_params* params, const void* dout,
                            const void* ids, void* dweight, void* workspace, size_t ws_bytes,
                            void* stream);

/* ------------------------------------------------------------------------------------
 * What stands around the head in a rollout and behind it in a training step: a dense layer,
 * the distribution that a sampler sees, and the optimizer.  Conventions as above.
 * ---------------------------------------------------------------------------------- */

enum {
  FLCE_ACT_NONE = 0,
  FLCE_ACT_RELU = 1,
  FLCE_ACT_GELU = 2,      /* z Phi(z) */
  FLCE_ACT_GELU_TANH = 3, /* z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) */
  FLCE_ACT_SILU = 4       /* z / (1 + e^-z) */
};

/* Dense layer  y[M,N] = act(z) + residual,  z = x[M,K] @ W + bias.
 *   x, weight, bias: bf16; weight [K,N] (FLCE_WEIGHT_HV: N % 8 == 0) or [N,K] (FLCE_WEIGHT_VH);
 *   K % 8 == 0.  residual and y: out_dtype, bf16 or fp32, sums in fp32, rounded once. */
typedef struct {
  int64_t M, N, K;
  int32_t weight_layout;
  int32_t activation;
  int32_t out_dtype; /* FLCE_BF16 or FLCE_F32 */
  int32_t validate;
} flce_linear_params;

int flce_linear_check_params(const flce_linear_params* params);
/* backward 0: flce_linear, 1: flce_linear_backward */
size_t flce_linear_workspace_size(const flce_linear_params* params, int backward);

/* bias, residual: or NULL.  preact: [M,N] bf16, z for the backward, or NULL.  x, weight, y,
 * residual and preact 16-byte aligned, bias 2-byte.  y may be the residual itself; outputs otherwise
 * share no memory with one another or with what is read, here and in the backward. */
int flce_linear(const flce_linear_params* params, const void* x, const void* weight,
                const void* bias, const void* residual, void* y, void* preact, void* workspace,
                size_t ws_bytes, void* stream);

/* Gradients by x [M,K], weight and bias, bf16, each or NULL (that by the residual is dout):
 *   dz = dout act'(preact), in bf16;  dx = dz W^T,  dweight = x^T dz,  dbias = sum_m of the
 *   unrounded dz, in fp32.  dout: out_dtype.  preact: or NULL without an activation.  x (weight) may
 *   be NULL where dweight (dx) is. */
int flce_linear_backward(const flce_linear_params* params, const void* dout, const void* x,
                         const void* weight, const void* preact, void* dx, void* dweight,
                         void* dbias, void* workspace, size_t ws_bytes, void* stream);

/* A wait of these two calls' products that runs out (2 s) is reported by flce_status and validate, as
 * FLCE_ERR_TIMEOUT, and what the product writes is then NaN throughout.  Self-tests: the calls with
 * copies that never come, at the first block (pair of blocks) of each product. */
int flce_selftest_linear_timeout(const flce_linear_params* params, const void* x, const void* weight,
                                 const void* residual, void* y, void* preact, void* workspace,
                                 size_t ws_bytes, void* stream);
int flce_selftest_linear_backward_timeout(const flce_linear_params* params, const void* dout,
                                          const void* x, const void* weight, const void* preact,
                                          void* dx, void* dweight, void* workspace, size_t ws_bytes,
                                          void* stream);

/* Rows of logits as a sampler sees them, per row in fp32:
 *   l = seen ? (l > 0 ? l / repetition : l * repetition) : l
 *   l = l - frequency * n - presence * [n > 0] + the sum of its biases
 *   l = -inf where not allowed;  z = l / temperature  (temperature 0: z = l)
 * with n its occurrences among the row's generated tokens, seen whether it is among its prompt
 * or generated tokens.  An array of flce_logits_rows takes the place of the value here. */
typedef struct {
  int64_t R, V, T;          /* rows, columns (<= 2^30), tokens per row (< 2^30) */
  int64_t ld_logits, ld_out, ld_tokens;      /* row strides in elements */
  int64_t n_bias, ld_bias_ids, ld_bias_values; /* entries of a row's list (<= 2048) */
  int64_t ld_allowed;       /* in bytes (mask_kind 1) or words (2); 0: one mask for all rows */
  int64_t ignore_index;
  double repetition_penalty, frequency_penalty, presence_penalty, temperature;
  int32_t dtype, out_dtype; /* of the logits, and of z: dtype or FLCE_F32 */
  int32_t tokens_int64, lens_int64, bias_int64; /* 1: int64, 0: int32 */
  int32_t mask_kind;        /* 0: none, 1: bytes, non-zero allows, 2: bits, v % 32 of word v / 32 */
  int32_t validate;
  int32_t split_lse;        /* lse is [2, R]: behind it what its rounding to fp32 left off */
} flce_logits_params;

/* Of each row, or NULL.  tokens [R, T]: the first lengths[r] count (NULL: all), of them the first
 * prompt_lens[r] are the prompt's (NULL: none).  Tokens and bias ids outside [0, V) are left out;
 * an id that comes twice in a list has both biases. */
typedef struct {
  const void* tokens;
  const void* prompt_lens;
  const void* lengths;
  const float* repetition_penalty;
  const float* frequency_penalty;
  const float* presence_penalty;
  const float* temperature;
  const void* bias_ids;
  const float* bias_values;
  const void* allowed;
} flce_logits_rows;

int flce_logits_check_params(const flce_logits_params* params);

/* out [R, V]: z (may be logits itself where the types are the same); lse [R]; logp [R], of
 * labels[r] under softmax(z); entropy [R].  Each or NULL, one at least.  A row whose label is
 * ignore_index has logp = entropy = 0, one whose label is outside [0, V) NaN, reported as
 * FLCE_ERR_LABEL with validate, which needs a workspace of 256 bytes (else NULL, 0); labels NULL:
 * every row counts.  A row with nothing left has lse = logp = -inf and entropy 0; one with a NaN or
 * +inf left, NaN. */
int flce_logits(const flce_logits_params* params, const flce_logits_rows* rows,
                const void* logits, const int64_t* labels, void* out, float* lse, float* logp,
                float* entropy, void* workspace, size_t ws_bytes, void* stream);

/* dlogits [R, V] (out_dtype, ld_out) = g_logp * d logp / d logits + g_entropy * d entropy / d logits
 * (NULL: 0), with lse and entropy (or NULL without g_entropy) of flce_logits.  Without split_lse a
 * probability is off by the rounding of lse, 2^-24 |lse| of itself; with it, by that of z - lse.  Rows
 * that are ignored or have nothing left get zeros. */
int flce_logits_backward(const flce_logits_params* params, const flce_logits_rows* rows,
                         const void* logits, const int64_t* labels, const float* lse,
                         const float* entropy, const float* g_logp, const float* g_entropy,
                         void* dlogits, void* workspace, size_t ws_bytes, void* stream);

/* AdamW over many tensors.  With c = grad_scale * min(1, max_norm / (norm + 1e-6)) (max_norm 0:
 * no clipping), t the steps so far plus one:
 *   g = c * grad;  m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * States, of numel elements for all tensors together, each tensor's at a multiple of 128:
 *   state_bits 32: m and v in fp32;
 *   state_bits 8: m and sqrt(v) as e4m3 codes with an fp32 scale per 128 elements, the largest of
 *     them / 448 (zero where that is below 2^-110).  A magnitude in units of the scale goes to a
 *     neighbouring code, up where the upper 20 of 32 random bits, a mixing of (seed, t, element),
 *     carry; a root that isn't 0 is not rounded to 0.  What a code is made of is rounded to fp32
 *     after every operation, in the order of the formulas; a magnitude in units is that times
 *     448 * (1 / largest).
 * master: fp32 weights in the same layout, or NULL: the parameters themselves are updated, and
 * rounded, in their own type.  Elements of the states behind a tensor's last stay 0. */
typedef struct {
  void* param;
  const void* grad;   /* dense, as param */
  int64_t n, offset;  /* elements; where its states begin (a multiple of 128) */
  float weight_decay;
  int32_t dtype;      /* of param */
  int32_t grad_dtype; /* dtype or FLCE_F32 */
} flce_adamw_tensor;

typedef struct {
  int64_t n_tensors, numel;
  double lr, beta1, beta2, eps, grad_scale, max_norm;
  int32_t state_bits;
  uint32_t seed;
  int32_t skip_nonfinite; /* a norm that is not finite: nothing changes, t neither */
} flce_adamw_params;

int flce_adamw_check_params(const flce_adamw_params* params);
/* Of both calls below.  The first 256 bytes are zero before the first call that uses the
 * workspace and after each. */
size_t flce_adamw_workspace_size(const flce_adamw_params* params);

/* norm [1] = 2-norm of grad_scale * (all gradients); `tensors` is read on the host. */
int flce_grad_norm(const flce_adamw_params* params, const flce_adamw_tensor* tensors, float* norm,
                   void* workspace, size_t ws_bytes, void* stream);

/* exp_avg_sq: v, or the codes of sqrt(v).  lr: a device value in the place of params->lr, or
 * NULL.  norm: of flce_grad_norm, where max_norm or skip_nonfinite asks for it.  step [1]: t,
 * counted up by the call. */
int flce_adamw_step(const flce_adamw_params* params, const flce_adamw_tensor* tensors,
                    float* master, void* exp_avg, void* exp_avg_sq, float* exp_avg_scale,
                    float* exp_rms_scale, const float* lr, const float* norm, int64_t* step,
                    void* workspace, size_t ws_bytes, void* stream);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int flce_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FLCE_H_ */
