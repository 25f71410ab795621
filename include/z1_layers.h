/*
 * z1_layers.h -- C ABI of the layers whose gradients the ZeRO-1 shard step
 * (z1.h) accumulates, between the embedding and the losses of z1_ops.h.
 *
 *   z1_linear            matrix product with bias, activation, elementwise
 *                        product, dropout and residual in its epilogue
 *   z1_linear_dz         the gradient through that epilogue, and of the bias
 *   z1_linear_grad       the gradients of the product's two operands, the
 *                        weight's straight onto the step's accumulator
 *   z1_dropout           dropout whose mask is drawn from a counter each time
 *                        and never stored, with a residual
 *   z1_qk_norm_rope      norm of queries and keys for each head with the
 *                        rotation by position, and z1_qk_norm_rope_grad
 *
 * The conventions of z1_ops.h hold: caller-owned device buffers, work enqueued
 * on the given stream of the GPU that is current, no host synchronisation, no
 * allocation, arguments validated on the host before anything is enqueued,
 * status codes, results that do not depend on timing.  Every call can be
 * captured into a HIP graph; its scalar arguments are baked in.  Two calls that
 * run at the same time must not share a workspace.
 *
 * Matrices are row-major: a pointer and the distance of two rows in elements,
 * at least the row's length.  Base pointers are aligned to their element type
 * only.  A buffer that is written overlaps no other one of the call, but for
 * the pairs named below, which may be the same buffer with the same row
 * distance.
 *
 * Errors of every call: Z1_EINVAL for null pointers, sizes, types, values that
 * are not finite, a workspace that is too small, a stream of another GPU, an
 * output that is another buffer of the call at the same address and may not be;
 * Z1_EALIGN for a misaligned pointer; Z1_EHIP for a failed launch.
 */
#ifndef Z1_LAYERS_H
#define Z1_LAYERS_H

#include "z1_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

#define Z1_LAYERS_ABI_VERSION 1

int32_t z1_layers_abi_version(void);

/* ------------------------------------------------------------------------
 * Dropout.  Element (r, c) of a matrix is kept where
 *   u(r, c) >= round(65536 p),
 * and scaled by 65536 / (65536 - round(65536 p)): the probability is a
 * multiple of 2^-16 and the scale is exact for it (p = 1: nothing is kept).
 * u(r, c) is 16 of the 128 bits of Philox4x32-10 (Salmon et al., "Parallel
 * random numbers: as easy as 1, 2, 3", 2011) under the key
 *   (seed low, seed high)      words of 32 bits
 * at the counter
 *   (c / 8, r, offset low, offset high):
 * half c mod 2 (0: the low one) of word (c mod 8) / 2.  A dropped element is
 * zero whatever it was.
 *
 * rng: device [2], seed and offset; the offset used is rng[1] + offset modulo
 * 2^64.  A step advances rng[1] (on the device, so that a replayed graph draws
 * new masks) and tells its layers apart by `offset`; the gradient takes the
 * same rng and offset as the forward pass.  rng NULL or p 0: no dropout.
 * ------------------------------------------------------------------------ */
typedef struct z1_drop {
    const uint64_t *rng;     /* device [2], or NULL                         */
    uint64_t offset;
    double p;                /* in [0, 1]                                   */
} z1_drop;

/* y = residual + drop(x) of rows x cols elements of dtype, rounded once; the
 * gradient is the same call on dy without a residual.  residual may be NULL; y
 * may be x or residual.  rows in [0, 2^31 - 1], cols in [1, 2^24]. */
typedef struct z1_dropout_args {
    int64_t rows, cols;
    const void *x, *residual;
    void *y;
    int64_t ld_x, ld_residual, ld_y;
    z1_drop drop;
    int32_t dtype;           /* z1_dtype                                    */
    int32_t reserved;        /* 0                                           */
} z1_dropout_args;

z1_status z1_dropout(const z1_dropout_args *args, z1_stream stream);

/* ------------------------------------------------------------------------
 * Linear.  x [rows, in], weight [out, in], bias [out], mul, residual, pre, y
 * [rows, out], all of dtype:
 *   z   = x weight^T + bias                   sums in fp32
 *   pre = z                                   rounded, where pre is given
 *   y   = residual + drop(act(z) mul)         from the unrounded z, rounded once
 * bias, mul, residual and pre may be NULL (none).  y may be residual or mul.
 * dtype Z1_F32 takes fp32 products.
 *   act      NONE z, RELU max(z, 0), GELU z Phi(z), SILU z / (1 + e^-z),
 *            GELU_TANH z / (1 + exp(-2 sqrt(2 / pi) (z + 0.044715 z^3))),
 *            RELU2 max(z, 0)^2
 * rows in [0, 2^30], in and out in [1, 2^20], row distances of x and weight
 * below 2^21; an output of any of the products has fewer than 2^24 tiles of 256 x
 * 256 elements (fp32: 128 x 128), which one that fits the GPU has by far.
 * ------------------------------------------------------------------------ */
typedef enum z1_act {
    Z1_ACT_NONE = 0, Z1_ACT_RELU = 1, Z1_ACT_GELU = 2, Z1_ACT_GELU_TANH = 3, Z1_ACT_SILU = 4,
    Z1_ACT_RELU2 = 5
} z1_act;

typedef struct z1_linear_args {
    int64_t rows, in, out;
    const void *x, *weight, *bias, *mul, *residual;
    void *pre, *y;
    int64_t ld_x, ld_weight, ld_mul, ld_residual, ld_pre, ld_y;
    z1_drop drop;
    int32_t dtype;           /* z1_dtype                                    */
    int32_t act;             /* z1_act                                      */
} z1_linear_args;

/* Bytes of device workspace the call needs for these sizes, row distances and
 * alignments of x and weight (0 for many, and for up to 4 rows): copies of
 * operands whose rows are not 16-byte aligned throughout, and partial sums where
 * a deep product of few tiles is split.  Only sizes, dtype, x, weight and their
 * distances are read. */
z1_status z1_linear_workspace(const z1_linear_args *args, int64_t *bytes);

/* workspace: 16-byte aligned, may be NULL where no byte is needed. */
z1_status z1_linear(const z1_linear_args *args, void *workspace, int64_t workspace_bytes,
                    z1_stream stream);

/* ------------------------------------------------------------------------
 * The gradient through the epilogue: with g = drop(dy) (the forward's mask),
 *   dz   = g mul act'(pre)                    rounded once
 *   dmul = g act(pre)                         rounded once
 *   dbias (+)= sum over rows of dz            fp32, from the unrounded dz
 * pre is needed for any act but NONE, and for dmul.  mul, dz, dmul and dbias
 * may be NULL (none; not all of the last three); the gradient of the residual
 * is dy itself.  Where g is dropped dz and dmul are 0 whatever mul and pre are.  dz may be dy or pre or mul, dmul may be mul or pre.
 * accumulate 0 writes dbias, 1 adds to it.  act' is 0 at z = 0 for RELU; where pre
 * is infinite (an fp16 one whose z was not) act and act' are their limits.
 * ------------------------------------------------------------------------ */
typedef struct z1_linear_dz_args {
    int64_t rows, out;
    const void *dy, *pre, *mul;
    void *dz, *dmul;
    float *dbias;            /* [out]                                       */
    int64_t ld_dy, ld_pre, ld_mul, ld_dz, ld_dmul;
    z1_drop drop;
    int32_t dtype, act;
    int32_t accumulate;      /* 0 or 1                                      */
    int32_t reserved;        /* 0                                           */
} z1_linear_dz_args;

/* Bytes of device workspace for dbias: partial sums.  None without dbias. */
z1_status z1_linear_dz_workspace(int64_t rows, int64_t out, int64_t *bytes);
z1_status z1_linear_dz(const z1_linear_dz_args *args, void *workspace, int64_t workspace_bytes,
                       z1_stream stream);

/* ------------------------------------------------------------------------
 * The gradients of the product, from dz [rows, out]:
 *   dx      = dz weight (+ add)      [rows, in], rounded once
 *   dweight (+)= dz^T x              [out, in], of dweight_dtype, rounded once
 * Either of dx and dweight may be NULL (then weight and add, or x, are not
 * read).  add [rows, in] may be NULL, and dx may be add.  dweight_dtype is
 * dtype or Z1_F32: with Z1_F32, accumulate 0 writes and 1 adds, so that
 * micro-batches are summed on the step's accumulator; with another type it is
 * written (a micro-batch slot).
 * ------------------------------------------------------------------------ */
typedef struct z1_linear_grad_args {
    int64_t rows, in, out;
    const void *dz, *x, *weight, *add;
    void *dx, *dweight;
    int64_t ld_dz, ld_x, ld_weight, ld_add, ld_dx, ld_dweight;
    int32_t dtype;           /* of all but dweight                          */
    int32_t dweight_dtype;
    int32_t accumulate;      /* 0 or 1; 1 only for a Z1_F32 dweight         */
    int32_t reserved;        /* 0                                           */
} z1_linear_grad_args;

/* As z1_linear_workspace; read are sizes, dtype, dz, x, weight, their
 * distances, and whether dx and dweight are NULL. */
z1_status z1_linear_grad_workspace(const z1_linear_grad_args *args, int64_t *bytes);
z1_status z1_linear_grad(const z1_linear_grad_args *args, void *workspace, int64_t workspace_bytes,
                         z1_stream stream);

/* ------------------------------------------------------------------------
 * Norm and rotation of queries and keys.  For each token t and head h, with v
 * the head's dim elements and w the weight of its kind (q or k):
 *   n   = v / sqrt(mean(v^2) + eps) * w       (w NULL: n = v, no norm)
 *   out = n with its first 2 n_freq elements turned, pair i by the angle
 *         positions[t] * inv_freq[i]:
 *         (a, b) -> (a cos - b sin, b cos + a sin)
 * Pair i is elements (i, n_freq + i), or (2 i, 2 i + 1) with interleaved.  The
 * angle is taken in binary64, everything else in fp32, rounded once.
 *
 * q and k are [tokens, heads, dim]: element (t, h, i) at t * token_stride + h *
 * head_stride + i.  The heads of one token do not overlap, nor do tokens;
 * either kind may have no heads.  out may be the input with the same strides.
 * inv_freq: device binary64 [n_freq], so that any scaling of the frequencies is
 * the caller's.  positions: any integers.
 * ------------------------------------------------------------------------ */
typedef struct z1_heads {
    int64_t heads;           /* in [0, 2^16]                                */
    const void *x;           /* input; may be NULL in the gradient w/o norm */
    void *out;               /* forward: out; gradient: d input             */
    const void *dout;        /* gradient only: d out                        */
    const void *weight;      /* [dim] of dtype, or NULL: no norm            */
    float *dweight;          /* gradient only: [dim], or NULL               */
    int64_t x_token, x_head, out_token, out_head, dout_token, dout_head; /* strides */
} z1_heads;

typedef struct z1_qk_args {
    int64_t tokens;          /* in [0, 2^31 - 1]                            */
    int32_t dim;             /* in [1, 512]                                 */
    int32_t n_freq;          /* in [0, dim / 2]                             */
    z1_heads q, k;
    const void *positions;   /* device [tokens]                             */
    const double *inv_freq;  /* device [n_freq]                             */
    double eps;              /* >= 0                                        */
    int32_t position_type;   /* z1_itype                                    */
    int32_t dtype;           /* z1_dtype                                    */
    int32_t interleaved;     /* 0 or 1                                      */
    int32_t accumulate;      /* gradient: 0 writes the dweights, 1 adds     */
} z1_qk_args;

z1_status z1_qk_norm_rope(const z1_qk_args *args, z1_stream stream);

/* d input = the gradient through rotation and norm (out may be dout with the
 * same strides); dweight (+)= its sum over tokens and heads in fp32.  Queries and
 * keys have dweights of their own, also where they share a weight. */
z1_status z1_qk_norm_rope_grad_workspace(int64_t tokens, int64_t q_heads, int64_t k_heads,
                                         int32_t dim, int64_t *bytes);
z1_status z1_qk_norm_rope_grad(const z1_qk_args *args, void *workspace, int64_t workspace_bytes,
                               z1_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* Z1_LAYERS_H */
