/*
 * fs_speculate.h -- C ABI of the operators of speculative decoding at the LM
 * head, for NVIDIA GB300 (sm_103a):
 *
 *   fs_quantize    bf16 / fp32 matrix to 8-bit floating point (e4m3) with a
 *                  scale for each block of 128: hidden states, or a head's weight
 *   fs_matmul_fp8  product of two such matrices: logits from an 8-bit head
 *   fs_probs       probabilities from logits, with the sampler's temperatures and
 *                  masks: the drafter's and the target's
 *   fs_verify      verification of drafted tokens against the target's
 *                  probabilities, from given random numbers
 *
 * Conventions are the sampler's (fs_sample.h): device pointers owned by the
 * caller, no allocation and no workspace, asynchronous on the given stream,
 * argument errors returned before anything is launched, status codes fs_status,
 * device timeouts reported by fs_last_device_error.  Results do not depend on
 * the stream, on graph capture, or on other work: every sum has a fixed order.
 * Element types are FS_BF16 and FS_F32 (fs_vocab.h).  Row strides are in elements
 * and at least the row's length; of a single row they are not used.  Outputs must
 * not overlap inputs unless it is said.
 */
#ifndef FS_SPECULATE_H_
#define FS_SPECULATE_H_

#include "fs_sample.h"
#include "fs_vocab.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Columns (and, of a weight, rows) that share a scale. */
#define FS_FP8_BLOCK 128

/*
 * 8-bit floating point with a scale for each block: x[n,k] stands as
 * values[n,k] * scale[n / block_rows, k / 128], values in e4m3 (largest 448).
 *   a     = max(max |x| over the block, 2^-100)
 *   scale = a / 448,   values = e4m3(x * (448 / a))
 * in fp32, each division and product rounded to nearest, e4m3 to nearest even
 * (a product just above 448 becomes 448).  block_rows is 1 (activations: a scale
 * for 128 columns of a row) or 128 (weights: for 128 x 128).  A block with a NaN has
 * scale NaN; one with an infinity has scale +inf, values 0 and, for the infinity,
 * NaN: either way no product with it is finite.  Blocks at the right and lower edge
 * are of what is there.
 * x: [N, d] of x_dtype, row stride ldx, base aligned to the element (16 bytes, with
 * ldx a multiple of 16 bytes, is faster); values: bytes [N, d], row stride ldv;
 * scale: fp32 [ceil(N / block_rows), ceil(d / 128)], row stride lds.  N = 0 does
 * nothing.  Limits: 0 <= N < 2^31 - 128, 1 <= d < 2^31 - 128.
 */
fs_status fs_quantize(const void *x, int64_t N, int64_t d, int64_t ldx, int x_dtype,
                      int block_rows, void *values, int64_t ldv, float *scale, int64_t lds,
                      void *stream);

/*
 * out[m,v] = sum over blocks k of a_scale[m,k] w_scale[v/128,k] *
 *            (sum over the block's columns j of A[m,j] W[v,j])
 * with A [M, d] and W [V, d] in e4m3, as fs_quantize leaves them (block_rows 1 and
 * 128).  Products are exact, a block's sum is the tensor core's fp32, blocks are added
 * in fp32 in their order, with the product of the two scales rounded to fp32, and
 * the result is rounded once to out's type.
 */
typedef struct fs_matmul_fp8_args {
  const void *A;        /* e4m3 [M, d]: 16-byte aligned base, lda % 16 == 0 */
  const float *a_scale; /* fp32 [M, ceil(d/128)], row stride lda_scale */
  const void *W;        /* e4m3 [V, d]: 16-byte aligned base, ldw % 16 == 0 */
  const float *w_scale; /* fp32 [ceil(V/128), ceil(d/128)], row stride ldw_scale */
  int64_t M, d, V, lda, lda_scale, ldw, ldw_scale;
  void *out; /* [M, V] of out_dtype, row stride ldo, base aligned to the element
              * (rows on 16-byte boundaries are faster) */
  int64_t ldo;
  int out_dtype;
  /* FS_FLAG_OVERLAP_PREVIOUS or 0: with it W streams while the kernel before on the
   * stream ends, which may write A and a_scale but neither W nor w_scale.  If that kernel was
   * itself launched so and lets its dependents start at once (an overlapping sampling call),
   * neither may the one before it.  The product lets its dependents start once the
   * kernel before it has ended, with the flag and without. */
  uint32_t flags;
} fs_matmul_fp8_args;

/* Limits: 0 <= M (0 does nothing), 1 <= d, 1 <= V, each below 2^31 - 512, and
 * ceil(M / 128) * ceil(V / 64) < 2^31. */
fs_status fs_matmul_fp8(const fs_matmul_fp8_args *args, void *stream);

/*
 * out[n,v] = exp(logits[n,v] / T_n - lse_n), lse_n = log of the sum of
 * exp(logits[n,v] / T_n) over the row's allowed ids; 0 for the other ids.
 * As in the sampler, T_n <= 0, NaN or +inf selects greedy decoding: 1 at the
 * allowed id of the largest logit (the lowest of equal ones; a NaN logit is never the
 * largest), 0 elsewhere.  A T_n below 2^-126 counts as 2^-126.  A row with no allowed id, or
 * whose allowed logits are all -inf, is 0.  A NaN or +inf logit of an allowed id makes the allowed
 * ids of a row that is not greedy NaN; logits of masked ids change nothing.
 * Computed in fp32 and rounded once to out's type.  out may be logits itself (same
 * address, type and stride), or must not overlap it.  Rows on 16-byte boundaries are faster,
 * rows of more than 262144 ids much slower (one thread block reads a row three times).
 */
typedef struct fs_probs_args {
  const void *logits; /* [N, V] of dtype, row stride ldl, base aligned to the element */
  int64_t N, V, ldl;
  const float *temperature;   /* fp32 [N] or NULL: T = 1 */
  const uint32_t *vocab_mask; /* uint32 [N, mask_ld] allow-bits or NULL, as fs_sample's */
  int64_t mask_ld;
  void *out; /* [N, V] of out_dtype, row stride ldo, base aligned to the element */
  int64_t ldo;
  int dtype, out_dtype;
} fs_probs_args;

/* Limits: 0 <= N < 2^28 (0 does nothing), 1 <= V < 2^31 - 2^16. */
fs_status fs_probs(const fs_probs_args *args, void *stream);

/* Largest K of fs_verify. */
#define FS_VERIFY_DRAFTS_MAX 1024

/*
 * Verification of drafted tokens, so that what comes out is distributed as
 * samples of the target alone.  Sequence b has drafted tokens x_0 .. x_(K-1), drawn
 * from the drafter's probabilities q[b,i,:], the target's p[b,i,:] at the K + 1
 * positions, and uniform random numbers u[b,0..K]:
 *   1. for i = 0, 1, ..: x_i is accepted if u_i q[i, x_i] < p[i, x_i] (compared
 *      exactly); the first one that is not ends the loop;
 *   2. n accepted: one more token is drawn with weights
 *        w[v] = max(p[n,v] - q[n,v], 0) (fp32)   if x_n was rejected
 *        w[v] = p[n,v]                           if there was no x_n
 *      as the lowest id v with  sum_{j<=v} w[j] > u_K sum_j w[j].
 * out_ids[b] = x_0 .. x_(n-1), the drawn token, -1 ..;  out_accepted[b] = n.
 * q NULL: a drafter that names its token (an n-gram table, a greedy drafter):
 * q is 1 at x_i, so x_i is accepted with probability p[i, x_i], and after a rejection
 * w is p without x_n.
 * K = 0 draws from p[b,0,:].  An id below 0 ends a sequence's drafts there (drafts
 * of different lengths); an id of V or more has probability 0 and is rejected.
 *
 * The sums are held to about 2^-45 of the row's total, in an order that depends on V
 * alone, so the drawn id is that of exact sums but where u_K falls within that of a
 * border.  p and q need not be normalised (sums below 2^100); a weight that is negative or
 * not finite counts as 0.  If every weight max(p - q, 0) is 0 after a rejection, the
 * draw is from p; if every weight is 0 then, the drawn id is -1.  A u below 0, or NaN, counts as 0,
 * one of 1 or more as 1 - 2^-24.
 *
 * Reads one row of p, and of q after a rejection, and the drafted tokens' elements:
 * whatever the other rows hold changes nothing.
 */
typedef struct fs_verify_args {
  const void *p; /* [B, K + 1, V] of dtype: strides p_seq, p_pos, 1 */
  const void *q; /* [B, K, V] of dtype: strides q_seq, q_pos, 1; or NULL */
  const int64_t *draft_ids; /* int64 [B, K], row stride ld_ids; may be NULL for K = 0 */
  const float *u;           /* fp32 [B, K + 1], row stride ldu */
  int64_t B, K, V;
  int64_t p_seq, p_pos, q_seq, q_pos, ld_ids, ldu;
  int64_t *out_ids; /* int64 [B, K + 1], row stride ld_out */
  int64_t ld_out;
  int64_t *out_accepted; /* int64 [B] or NULL */
  int dtype;
} fs_verify_args;

/* Limits: 0 <= B < 2^24 (0 does nothing), 0 <= K <= FS_VERIFY_DRAFTS_MAX,
 * 1 <= V < 2^31 - 2^16; strides of p and q at least 0 (one row for several
 * sequences or positions is allowed). */
fs_status fs_verify(const fs_verify_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FS_SPECULATE_H_ */
