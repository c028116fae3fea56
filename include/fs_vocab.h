/*
 * fs_vocab.h -- C ABI of the operators beside the sampler at the vocabulary
 * ends of a model, for NVIDIA GB300 (sm_103a):
 *
 *   fs_logprobs       log-probabilities of given tokens, the entropy of the
 *                     row's distribution and its most probable tokens, from
 *                     hidden states H and LM-head weight W
 *   fs_logprobs_grad  gradient of the log-probabilities and entropies to H, W
 *   fs_embed          embedding lookup with scaling
 *   fs_embed_grad     its gradient to the table, by sorted tokens
 *
 * Conventions are the sampler's (fs_sample.h): device pointers owned by the
 * caller, no allocation per call, asynchronous on the given stream, argument
 * errors returned before anything is launched, status codes fs_status, device
 * timeouts reported by fs_last_device_error.  Results do not depend on the
 * stream, on graph capture, or on other work: every sum has a fixed order.
 */
#ifndef FS_VOCAB_H_
#define FS_VOCAB_H_

#include "fs_sample.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of alternatives fs_logprobs returns. */
#define FS_LOGPROBS_TOPK_MAX 20

/*
 * With l[b,v] = sum_k H[b,k] W[v,k] (fp32 accumulation), x[b,v] = l[b,v] / T_b
 * and sums over the row's allowed ids v:
 *   lse[b]     = log sum_v exp(x[b,v])
 *   logp[b]    = x[b, token_b] - lse[b]
 *   entropy[b] = -sum_v p log p,  p = exp(x[b,v] - lse[b])
 *   top K      = the K allowed ids of the largest l[b,v], best first, ties to
 *                the lower id, with their log-probabilities
 * The [B,V] logits never reach device memory.
 *
 * The logits of the token and of K + 4 candidates (the best by their tensor-core
 * sums in fp32, ties to the lower id) are summed again in compensated fp32, about
 * 45 bits, and ranked on that.  So alternatives come in the order of their exact
 * logits, also where those differ by less than fp32 resolves, and do not depend on
 * B or on how the work was split.  One of the K largest is missed only where K + 4
 * other ids' fp32 sums are no smaller than its own: where more than 4 ids lie within
 * those sums' error (about 1e-6 of the sum of |H W|) of the K-th.
 *
 * The tensor core cuts its fp32 sums off towards zero, on average by 1.55e-8 of the
 * logit for every 16 products, which is corrected.  The ids that decide a row do not
 * depend on that: the token, the K + 4 candidates and, with K = 0, one id of a logit near
 * the largest enter the row's sums with the logits summed again.  The other ids'
 * probabilities are off by a quarter of the mean, each in its own way (1e-6 |x| at
 * d = 4096, relative), or by all of it where a row's sums are exact on the way, as with
 * few non-zeros in H (4e-6 |x|).
 *
 * Conventions: T_b <= 0, NaN or +inf (greedy rows of the sampler) means T = 1, a T_b
 * below 2^-126 counts as 2^-126.
 * A token below 0 means "no token": logp 0.  A token that the mask clears, or
 * that lies outside [vocab_offset, vocab_offset + V), has logp -inf.  A fully
 * masked row has lse -inf and entropy 0; alternatives past the allowed count
 * are id -1, log-probability -inf.  Whatever W holds for a masked id -- NaN or
 * infinity too -- changes nothing; a NaN or +inf logit of an allowed id makes
 * the row's lse, entropy and log-probabilities NaN, also those of missing
 * alternatives (ids with a NaN logit are not listed).
 */
typedef struct fs_logprobs_args {
  /* As in fs_sample_args: bf16 [B, d] and [V, d], 16-byte aligned, row strides
   * multiples of 8; fp32 [B] or NULL; uint32 [B, mask_ld] allow-bits or NULL. */
  const void *H;
  const void *W;
  const float *temperature;
  const uint32_t *vocab_mask;
  int64_t mask_ld;
  const int64_t *tokens; /* int64 [B] global ids, or NULL: no log-probabilities */
  int64_t B, d, V, ldh, ldw;
  int64_t vocab_offset;  /* global id of W's first row (>= 0) */
  int64_t K;             /* alternatives per row, 0..FS_LOGPROBS_TOPK_MAX */
  float *out_logp;       /* fp32 [B]; given exactly when tokens is */
  float *out_entropy;    /* fp32 [B] or NULL */
  float *out_lse;        /* fp32 [B] or NULL */
  int64_t *out_topk_idx; /* int64 [B, K]; given exactly when K > 0 */
  float *out_topk_logp;  /* fp32 [B, K]; given exactly when K > 0 */
  /* 256-byte aligned, fs_logprobs_workspace_size(B, V, K) bytes, no
   * initialisation needed.  Calls that may overlap need different ones. */
  void *workspace;
  size_t workspace_bytes;
  uint32_t flags; /* FS_FLAG_OVERLAP_PREVIOUS or 0 */
} fs_logprobs_args;

/* 0 for sizes fs_logprobs rejects. */
size_t fs_logprobs_workspace_size(int64_t B, int64_t V, int64_t K);

/* Limits: 1 <= B <= 65535, 1 <= d, 1 <= V, vocab_offset + V < 2^31. */
fs_status fs_logprobs(const fs_logprobs_args *args, void *stream);

/*
 * Gradient of  sum_b grad_logp[b] logp[b] + grad_entropy[b] entropy[b]:
 *   G[b,v]  = (1/T_b) (grad_logp[b] (1[v = token_b] - p)
 *                      - grad_entropy[b] p (log p + entropy[b])),  0 if masked
 *   dH[b,:] = sum_v G[b,v] W[v,:]        dW[v,:] = sum_b G[b,v] H[b,:]
 * The logits are computed again; G goes through the workspace in bf16 (each
 * term rounded once, relative error at most 2^-8, sums in fp32), but for G at the
 * row's token, most of a row's gradient: that comes from the token's logit in
 * compensated fp32, and what rounding takes of it is kept in fp32 and added to the
 * sums; dH, dW are rounded to bf16 once.  An id other than the token that holds
 * most of a row repeats its rounding in the row of dH and in its own of dW: their
 * error is then up to twice that of rounding them to bf16.  The probabilities of the
 * other ids are those of the tensor core's logits, as far off as said above (and never
 * above 1), and all are off by the rounding of lse, 2^-24 |lse|.  lse and entropy are fs_logprobs' outputs; on
 * a shard of the vocabulary they are those of the whole vocabulary, and the shards' dH
 * add up to the whole one.  A token below 0 or cleared by the mask (logp 0 or -inf)
 * gets no gradient from logp; for a token outside [vocab_offset, vocab_offset +
 * V) the one-hot term lies in another shard and only the p term is added here.
 * A fully masked row (lse -inf) gets no gradient.
 * H and W must be finite, masked ids' rows of W and fully masked rows of H too:
 * where G is 0 they are multiplied by 0, and 0 times NaN is NaN.  dH and dW must
 * not overlap H, W, the workspace or one another.
 */
typedef struct fs_logprobs_grad_args {
  const void *H;
  const void *W;
  const float *temperature;
  const uint32_t *vocab_mask;
  int64_t mask_ld;
  const int64_t *tokens;     /* int64 [B] global ids */
  const float *lse;          /* fp32 [B] */
  const float *entropy;      /* fp32 [B]; needed exactly when grad_entropy is given */
  const float *grad_logp;    /* fp32 [B] */
  const float *grad_entropy; /* fp32 [B] or NULL */
  int64_t B, d, V, ldh, ldw;
  int64_t vocab_offset;
  void *out_dH; /* bf16 [B, d], row stride lddh; or NULL */
  void *out_dW; /* bf16 [V, d], row stride lddw; or NULL (not both) */
  int64_t lddh, lddw; /* multiples of 8, >= d; bases 16-byte aligned */
  void *workspace;
  size_t workspace_bytes;
} fs_logprobs_grad_args;

/* 0 for sizes fs_logprobs_grad rejects. */
size_t fs_logprobs_grad_workspace_size(int64_t B, int64_t d, int64_t V);

fs_status fs_logprobs_grad(const fs_logprobs_grad_args *args, void *stream);

/* Element types of the embedding operators. */
#define FS_BF16 0
#define FS_F32 1

/*
 * Embedding lookup: out[n,:] = scale * E[ids[n] - vocab_offset, :] for n < N,
 * computed in fp32 and rounded once to the table's type (scale 1 copies); rows
 * whose id lies outside [vocab_offset, vocab_offset + V) -- padding ids below
 * 0, another shard's ids -- are 0, so the shards' outputs add up to the whole.
 * ids: int64 [N]; E: [V, d] and out: [N, d] of `dtype`, unit column stride, row
 * strides lde, ldo >= d elements, bases aligned to the element (rows on 16-byte
 * boundaries are copied 16 bytes at a time, others element by element).  out
 * must not overlap E.  N = 0 does nothing.
 * Limits: 0 <= N < 2^31 - 2^16, 1 <= d < 2^31 - 2^11, V >= 1, vocab_offset >= 0,
 * vocab_offset + V < 2^31.
 */
fs_status fs_embed(const int64_t *ids, int64_t N, const void *E, int64_t V, int64_t d,
                   int64_t lde, int dtype, float scale, int64_t vocab_offset, void *out,
                   int64_t ldo, void *stream);

/*
 * Gradient of fs_embed to the table: dE[v,:] = scale * sum of dY[n,:] over the
 * n with ids[n] = vocab_offset + v (added to what dE holds if accumulate is
 * not 0; otherwise every row of dE is written, 0 where no id names it).
 * The ids are sorted on the device, stably, and each row's terms are summed in
 * fp32 in the order of n in runs of fixed length, so the result is the same on
 * every call; it is rounded once to dE's type (with accumulate, after adding).
 * dY: [N, d] of y_dtype; dE: [V, d] of e_dtype (FS_BF16 or FS_F32; FS_F32 when
 * y_dtype is FS_F32); row strides and alignment as fs_embed; dY and dE must not
 * overlap.  workspace: 256-byte aligned, fs_embed_grad_workspace_size(N, d)
 * bytes, no initialisation needed (may be NULL for N = 0).
 */
size_t fs_embed_grad_workspace_size(int64_t N, int64_t d);

fs_status fs_embed_grad(const int64_t *ids, int64_t N, const void *dY, int64_t V, int64_t d,
                        int64_t ldy, int y_dtype, float scale, int64_t vocab_offset, void *dE,
                        int64_t lde, int e_dtype, int accumulate, void *workspace,
                        size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FS_VOCAB_H_ */
