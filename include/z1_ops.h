/*
 * z1_ops.h -- C ABI of the operators next to the ZeRO-1 shard step (z1.h):
 * what makes the gradients the step accumulates, and a second update rule.
 *
 *   z1_muon_*            momentum, Newton-Schulz orthogonalisation and the
 *                        fp32 master / bf16 weight update of whole matrices
 *   z1_embed_*           embedding lookup with scaling, and its gradient
 *                        summed in fp32 by sorted tokens (bit-reproducible)
 *   z1_token_logprob, z1_logprob_grad
 *                        log-probability of one target per logits row, and
 *                        its gradient in the logits
 *   z1_policy_loss       clipped policy loss with a KL term and its gradient
 *                        in the logits, in one pass over the logits
 *   z1_preference_loss   paired log-ratio preference loss and its gradient in
 *                        the token log-probabilities
 *
 * The conventions of z1.h hold: caller-owned device buffers, work enqueued on
 * the given stream of the GPU that is current, no host synchronisation,
 * arguments validated on the host before anything is enqueued, status codes,
 * no C++ exception across the interface.  No call here allocates except
 * z1_muon_create.  Two calls that run at the same time on different streams
 * must not share a workspace or a z1_muon.  Results are bit-reproducible: no
 * call adds floating-point values in an order that timing decides.  Every
 * call can be captured into a HIP graph; its scalar arguments are baked in.
 *
 * Target and token ids live on the device, so the host cannot check their
 * values: an id below zero marks an empty position (nothing of its row counts,
 * its outputs are zero), and an id of vocab or more gives NaN in its outputs
 * (and is skipped by z1_embed_grad); neither makes the kernels read or write
 * outside the buffers.
 */
#ifndef Z1_OPS_H
#define Z1_OPS_H

#include "z1.h"

#ifdef __cplusplus
extern "C" {
#endif

#define Z1_OPS_ABI_VERSION 1

typedef enum z1_dtype { Z1_F32 = 0, Z1_BF16 = 1, Z1_F16 = 2 } z1_dtype;
typedef enum z1_itype { Z1_I64 = 0, Z1_I32 = 1 } z1_itype;

int32_t z1_ops_abi_version(void);

/* ------------------------------------------------------------------------
 * Muon.  For a matrix with gradient G (rows x cols):
 *
 *   g   = c G,  c = min(1, clip / (sqrt(S) + 1e-6))   (c = 1 for clip <= 0)
 *   mom = mu mom + g
 *   U   = g + mu mom  (nesterov)  or  mom
 *   O   = q(U / (|U|_F + eps)),  q = p applied ns_steps times,
 *         p(X) = a X + (b A + c A A) X,  A = X X^T   (X transposed if tall)
 *   master = master (1 - lr wd_scale wd) - lr lr_scale O
 *   weights = bf16(master), to nearest even
 *
 * The products take fp16 operands (a fixed power of two above their range's
 * top, see z1_muon.hip) with fp32 accumulators; X itself is carried in 22 bits.
 * What that leaves of O against the definition, of its norm: 1.2e-3 to 1.9e-3
 * for gaussian U of sides from 100 on, 2e-3 to 3.3e-3 for sides of 8 to 100,
 * up to 1e-2 for a few elements; 1e-4 to 1e-3 for low-rank and decaying
 * spectra.  A handle of z1_muon_create_wide takes all operands in 22 bits.
 * A zero U gives a zero O.  A NaN or infinity anywhere in U spreads over O.
 * ------------------------------------------------------------------------ */
typedef struct z1_muon z1_muon;

typedef struct z1_muon_bind {
    int32_t n;               /* matrices, >= 0                              */
    int32_t grad_dtype;      /* Z1_F32 (the step's acc arena) or Z1_BF16    */
    const int64_t *rows;     /* host [n], each in [1, 2^20]                 */
    const int64_t *cols;     /* host [n], each in [1, 2^20]                 */
    /* host arrays [n] of device pointers to row-major contiguous matrices.
     * momentum, master, weights: all three, or none (z1_muon_orthogonalize
     * only).  ortho: bf16 outputs of z1_muon_orthogonalize, or NULL.  Base
     * pointers are aligned to their element type only.                     */
    const void *const *grad;
    float *const *momentum;
    float *const *master;
    void *const *weights;
    void *const *ortho;
    const double *lr_scale;  /* host [n] or NULL (all 1)                    */
    const double *wd_scale;  /* host [n] or NULL (all 1)                    */
    double a, b, c;          /* coefficients of p                           */
    double eps;              /* >= 0                                        */
    int32_t ns_steps;        /* in [1, 32]                                  */
    int32_t reserved;        /* 0                                           */
} z1_muon_bind;

typedef struct z1_muon_hp {
    double lr, momentum, weight_decay, clip;
    int32_t nesterov;        /* 0 or 1                                      */
    int32_t reserved;        /* 0                                           */
} z1_muon_hp;

/* Creates the handle on the current GPU: tile tables and the workspace (8
 * bytes per element and 4 per element of the smaller side squared, padded to
 * tiles of up to 256; none for matrices that fit one workgroup, up to about 64
 * x 512 or 128 x 160).  Waits for its upload.  Errors: Z1_EINVAL for null
 * pointers, sizes (or more than about 1.7e10 elements in all), an unknown
 * dtype, or coefficients for which p leaves the range the fp16 operands hold (|p| > 3.9
 * or |b s + c s^2| > 3.9 somewhere on the values the iteration can reach;
 * ns_steps included); Z1_EALIGN; Z1_ENOMEM; Z1_EHIP. */
z1_status z1_muon_create(z1_muon **out, const z1_muon_bind *bind, z1_stream stream);

/* The same, with every operand as two fp16 numbers (22 bits), every product as
 * three, and X carried in fp32: O is then 1e-6 (gaussian U) to 3e-5 (low-rank
 * U) of its norm off, about a third of what fp32 products leave of large
 * matrices, at two to three times the time.  16 bytes of workspace an element and 8 per element of the smaller
 * side squared, and no one-workgroup path. */
z1_status z1_muon_create_wide(z1_muon **out, const z1_muon_bind *bind, z1_stream stream);
z1_status z1_muon_destroy(z1_muon *m);

/* One update of every matrix.  d_S: device double, the squared global
 * gradient norm (z1_grad_norm_sq); read only when clip > 0, may be NULL
 * otherwise.  Needs momentum, master and weights bound (else Z1_ESTATE). */
z1_status z1_muon_step(z1_muon *m, const z1_muon_hp *hp, const double *d_S, z1_stream stream);

/* ortho[i] = q(grad[i] / (|grad[i]|_F + eps)) as bf16; momentum and weights
 * untouched.  Needs ortho bound (else Z1_ESTATE). */
z1_status z1_muon_orthogonalize(z1_muon *m, z1_stream stream);

/* ------------------------------------------------------------------------
 * Embedding.
 *   out[t, :] = scale * weight[ids[t], :]            rounded once
 *   dweight[v, :] (+)= scale * sum over t with ids[t] == v of dout[t, :]
 * Rows are contiguous; ld* is the distance of two rows in elements.
 * ------------------------------------------------------------------------ */
typedef struct z1_embed_args {
    int64_t n_ids;           /* T, in [0, 2^30]                             */
    int64_t vocab;           /* V, in [1, 2^24]                             */
    int64_t dim;             /* d, in [1, 2^20]                             */
    const void *ids;         /* device [T]                                  */
    int32_t id_type;         /* z1_itype                                    */
    int32_t dtype;           /* of weight / out, or of dout                 */
    double scale;
} z1_embed_args;

z1_status z1_embed_lookup(const z1_embed_args *args, const void *weight, int64_t ld_weight,
                          void *out, int64_t ld_out, z1_stream stream);

/* Bytes of device workspace z1_embed_grad needs for these sizes. */
z1_status z1_embed_grad_workspace(int64_t n_ids, int64_t vocab, int64_t dim, int64_t *bytes);

/* dweight: fp32 [vocab, dim], contiguous.  accumulate 0 writes all of it
 * (zero rows for absent ids), 1 adds to the rows of the ids that occur.
 * The sums run in fp32 in token order, in pieces of fixed size that are
 * joined in order.  workspace: 16-byte aligned (Z1_EALIGN), at least
 * z1_embed_grad_workspace bytes (Z1_EINVAL). */
z1_status z1_embed_grad(const z1_embed_args *args, const void *dout, int64_t ld_dout,
                        float *dweight, int32_t accumulate, void *workspace,
                        int64_t workspace_bytes, z1_stream stream);

/* ------------------------------------------------------------------------
 * Losses over logits.  logits: [n_rows, vocab] of dtype, rows contiguous,
 * ld >= vocab elements apart; targets [n_rows].  With
 *   lse_r = log sum_v exp x_rv,   logp_r = x_{r, y_r} - lse_r
 * a row whose target is negative has logp 0 and lse 0, and a zero gradient
 * row, whatever its logits hold.
 * ------------------------------------------------------------------------ */
typedef struct z1_logits {
    int64_t n_rows;          /* in [0, 2^31 - 1]                            */
    int64_t vocab;           /* in [1, 2^30]                                */
    const void *logits;
    int64_t ld;
    const void *targets;
    int32_t target_type;     /* z1_itype                                    */
    int32_t dtype;           /* z1_dtype                                    */
} z1_logits;

/* logp, lse: fp32 [n_rows]; lse may be NULL. */
z1_status z1_token_logprob(const z1_logits *x, float *logp, float *lse, z1_stream stream);

/* dlogits_rv = dlogp_r (1[v == y_r] - exp(x_rv - lse_r)), rounded once to
 * dtype, ld_d elements between rows; dlogits may be the logits themselves
 * (with the same row distance, else Z1_EINVAL), but not overlap them otherwise.
 * Where |lse| is 64 or more, and is the row's own as z1_token_logprob gave it,
 * the exponent is taken from the row's maximum and log-sum anew (one more
 * read of that row), so that lse's rounding does not reach the gradient. */
z1_status z1_logprob_grad(const z1_logits *x, const float *lse, const float *dlogp,
                          void *dlogits, int64_t ld_d, z1_stream stream);

/* Clipped policy loss.  Per counted row (target >= 0 and weight != 0):
 *   rho = exp(logp - old_logp)
 *   l   = -min(rho A, clamp(rho, 1 - clip_low, 1 + clip_high) A)
 *         + kl_coef (exp(ref - logp) - (ref - logp) - 1)
 *   loss = scale * sum_r w_r l_r      dlogits = d loss / d logits
 * token_loss gets l_r (0 where not counted).  ref_logp may be NULL and kl_coef 0
 * (either: no KL term, and ref_logp is not read), weights NULL (all 1), dlogits NULL (no gradient), logp NULL;
 * dlogits may be the logits themselves, as above.  Where the minimum's two sides are
 * equal with rho outside the clamp (A = 0), the gradient is the clamp's. */
typedef struct z1_policy_args {
    const float *old_logp, *ref_logp, *advantages, *weights; /* fp32 [n_rows] */
    double clip_low, clip_high, kl_coef, scale;
    float *loss;             /* [1]                                         */
    float *token_loss;       /* [n_rows]                                    */
    float *logp;             /* [n_rows] or NULL                            */
    void *dlogits;           /* [n_rows, vocab] of dtype or NULL            */
    int64_t ld_dlogits;
} z1_policy_args;

z1_status z1_policy_loss(const z1_logits *x, const z1_policy_args *args, z1_stream stream);

/* Preference loss.  cu_seqlens: device [2 n_pairs + 1], ascending row
 * offsets; sequence 2p is pair p's chosen answer, 2p + 1 its rejected one
 * (either may be empty).  With r_s = sum over the counted rows of sequence s
 * of (logp - ref_logp):
 *   z_p = beta (r_2p - r_2p+1)
 *   l_p = -(1 - e) log sigmoid(z_p) - e log sigmoid(-z_p)   e = label_smoothing
 *   loss = scale * sum_p l_p,   dlogp = d loss / d logp  (0 outside every
 *   sequence and where the target is negative)
 * Offsets are clamped to [0, n_rows]. */
typedef struct z1_preference_args {
    int64_t n_rows;
    int64_t n_pairs;         /* in [0, 2^23]                                */
    const float *logp, *ref_logp;
    const void *targets;     /* [n_rows]                                    */
    const void *cu_seqlens;
    int32_t target_type, cu_type;   /* z1_itype                             */
    double beta, label_smoothing, scale;
    float *loss;             /* [1]                                         */
    float *pair_loss;        /* [n_pairs]                                   */
    float *margins;          /* [n_pairs] z_p, or NULL                      */
    float *dlogp;            /* [n_rows] or NULL                            */
} z1_preference_args;

z1_status z1_preference_loss(const z1_preference_args *args, z1_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* Z1_OPS_H */
