/*
 * linear.h - C ABI of the linear layers around the triangle update and the atom
 * attention on B200 (sm_100a), their gradients, and activations kept in 8 bits
 * between the forward and the backward.
 *
 *   forward    p = x W^T + b;  y = act(p) + residual
 *   backward   D = dy * act'(p) (p recomputed from x)
 *              dx = D W,  dW = D^T x,  db = sum of D over the rows
 *              (the residual's gradient is dy itself)
 *
 *   act: identity, relu max(p, 0), sigmoid 1 / (1 + e^-p), silu p / (1 + e^-p).
 *   relu' is 1 where p > 0 and 0 elsewhere.
 *
 * Layouts (row-major, contiguous, bf16): x, dx [rows][in_features]; y, dy,
 * residual [rows][out_features]; weight, dW [out_features][in_features] (PyTorch
 * Linear layout); bias, db [out_features]. in_features and out_features are
 * multiples of 8, at most 16384; 1 <= rows <= 2^30. Every pointer but bias and db
 * must be 16-byte aligned (those 2-byte). y and the gradients must not overlap an
 * input, each other or the workspace, with one exception: y may be the residual
 * itself (the residual stream updated in place).
 *
 * Precision: bf16 operands on tcgen05 tensor cores, fp32 accumulation, bias,
 * activation and residual in fp32, one rounding to bf16 at the end. The backward
 * rounds D to bf16 before it enters the products dx and dW (with identity or relu
 * D is dy or 0, exactly); db sums D before that rounding. Where p is so near 0
 * that its sums' rounding could turn its sign (under a bound from the norms of its
 * rows of x and W), relu' takes p again in 64 bits: the sign is right down to
 * 2^-53 of the products' sizes. Gradients have the parameters' type. Sums over the
 * rows are taken in parts of at most 65536 rows each, and the parts added in fp32.
 * Every sum is taken in a fixed order, so equal calls give equal bits.
 *
 * Ownership, threading and errors follow trimul.h: the caller owns every buffer,
 * a call enqueues on `stream` and returns TRIMUL_OK or a negative trimul_status,
 * argument errors are found on the host before any work is enqueued, and a bounded
 * in-kernel wait that runs out is recorded in the status word, the workspace's or
 * the caller's own (trimul_linear_device_status). Calls that may overlap in time need workspaces of
 * their own, captured graphs included. All pointers must be memory of the current
 * device.
 */
#ifndef TRIMUL_LINEAR_H
#define TRIMUL_LINEAR_H

#include "trimul.h"

#ifdef __cplusplus
extern "C" {
#endif

enum trimul_act {
    TRIMUL_ACT_NONE = 0,
    TRIMUL_ACT_RELU = 1,
    TRIMUL_ACT_SIGMOID = 2,
    TRIMUL_ACT_SILU = 3
};

typedef struct trimul_linear_params {
    long long rows;
    int in_features, out_features;
    int act;                /* enum trimul_act */
    const void *weight;     /* [out_features][in_features] */
    const void *bias;       /* [out_features] or NULL */
    void *workspace;        /* device memory, 256-byte aligned */
    size_t workspace_bytes;
    uint32_t timeout_ms;    /* bound on each in-kernel wait; 0 = 2000 ms */
    void *status;           /* NULL: the status word is the workspace's, cleared by each call;
                               else one that calls do not clear (trimul_status_word) */
} trimul_linear_params;

/* Bytes of workspace of the forward (the device status word). With p->status, a
 * call whose workspace would hold nothing else needs none (workspace NULL). */
size_t trimul_linear_workspace_size(void);

/* y = act(x W^T + b) + residual (residual may be NULL). Asynchronous. */
int trimul_linear_forward(const void *x, const void *residual, const trimul_linear_params *p, void *y,
                          trimul_stream_t stream);

/* ---- activations in 8 bits ---------------------------------------------------
 * A bf16 array kept as MXFP8 between the forward and the backward, in the reading
 * of OCP Microscaling v1.0 that the MXFP8 contraction takes (trimul.h): each block
 * of 32 consecutive channels has one E8M0 scale byte s (2^(s - 127), with
 * s - 127 = floor(log2 max|v|) - 8, at least -127; an all-zero block has s = 0) and
 * 32 E4M3 codes of v / 2^(s - 127), rounded to nearest even and saturated at
 * +-448. 33/32 bytes per value instead of 2. A value is kept to within 2^-4 of its
 * own size while it lies within 2^-14 of its block's largest, except that a value
 * above 1.75 times its block's power of two becomes 1.75 times it (at most 1/8
 * lower). An infinity or NaN is kept as NaN and does not change its block's scale.
 * (A scale byte of 255, which packing never writes, stands for NaN.)
 *
 * codes [rows][channels], scales [rows][channels / 32], one byte each, both 16-byte
 * aligned; channels a multiple of 32, at most 16384; 1 <= rows <= 2^30. */
typedef struct trimul_act8 {
    const void *codes, *scales;
} trimul_act8;

int trimul_act8_pack(const void *x, long long rows, int channels, void *codes, void *scales,
                     trimul_stream_t stream);

/* x = the values that the codes stand for, in bf16 (exact, but for values under
 * 2^-126, which round to nearest even). */
int trimul_act8_unpack(const void *codes, const void *scales, long long rows, int channels, void *x,
                       trimul_stream_t stream);

/* ---- backward ------------------------------------------------------------------
 * dx, dW and db for one forward call with the same x and params. Exactly one of x
 * and x8 is given: with x8 (in_features a multiple of 32) the gradients are those
 * at the values that the codes stand for. A NULL dx, dw or db skips that gradient.
 * p->workspace must hold trimul_linear_backward_workspace_size bytes.
 * Asynchronous. */
size_t trimul_linear_backward_workspace_size(long long rows, int in_features, int out_features, int act, int from8);

int trimul_linear_backward(const void *x, const trimul_act8 *x8, const void *dy, const trimul_linear_params *p,
                           void *dx, void *dw, void *db, trimul_stream_t stream);

/* Synchronises `stream`, then reads the params' status word: TRIMUL_OK,
 * TRIMUL_ERR_TIMEOUT or TRIMUL_ERR_DEVICE; detail[4] (optional) receives code,
 * site, block, aux. */
int trimul_linear_device_status(const trimul_linear_params *p, trimul_stream_t stream, int *detail);

#ifdef __cplusplus
}
#endif

#endif /* TRIMUL_LINEAR_H */
