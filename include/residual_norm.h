/*
 * residual_norm.h -- C ABI of the residual norm, forward and backward (part of
 * libspectre_mix), on NVIDIA B200 (sm_100a): the four forms that the spectral mix
 * fuses (enum spectre_norm), as an operator of its own.
 *
 * For every row of C values, with N the norm over the row:
 *
 *   SPECTRE_NORM_POST_LN, _POST_RMS:  y = N(out + x)
 *   SPECTRE_NORM_PRE_LN,  _PRE_RMS:   y = N(out) + x
 *   LayerNorm: N(z) = (z - mean) / sqrt(var + eps) * gamma + beta   (biased variance)
 *   RMSNorm:   N(z) = z / sqrt(mean(z^2) + eps) * gamma + beta
 *
 * Backward, with n = (z - mean) r, r = 1 / sqrt(var + eps) and dn = dy * gamma:
 *
 *   LayerNorm: dz = r (dn - mean(dn) - n mean(dn * n));  RMSNorm: without mean(dn)
 *   dgamma = sum over rows of dy * n,  dbeta = sum over rows of dy
 *
 * dz is the gradient of out, and of x too in the POST forms; in the PRE forms the
 * gradient of x is dy itself, and x is not read.
 *
 * Shapes: 1 <= C <= 8192; any T >= 0.  Numbers: rows are of the plan's dtype
 * (SPECTRE_F32 or SPECTRE_BF16); gamma, beta, dgamma and dbeta are fp32 [C].  All
 * sums are fp32 in a fixed order (equal inputs give equal bits); bf16 outputs are
 * rounded once, to nearest even.
 *
 * Rows: T rows with a row stride in elements, their C values contiguous.  Input
 * rows may overlap, output rows may not, and an output may not overlap an input.
 * Pointers need their element's alignment (SPECTRE_ERR_ALIGN); where every pointer
 * and row is 16-byte aligned the rows are moved 16 bytes at a time, otherwise
 * element by element.
 *
 * Ownership and errors as in gated_scan.h: the caller owns tensors and workspace,
 * the handle holds no device memory and serves several streams and threads at once.
 */
#ifndef RESIDUAL_NORM_H
#define RESIDUAL_NORM_H

#include "spectre_mix.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct residual_norm_s *residual_norm_t;

enum residual_norm_option {
    /* 0 (default).  1, for tests of the failure path only: a wait for copies of rows gives up at once (they
     * are waited for again before the block goes on without them).  Only the backward pass has such waits,
     * over rows of more than 128 values that are aligned for copies. */
    RESIDUAL_NORM_OPT_TEST_WAIT_TIMEOUT = 1,
};

/* Create a plan for rows of C values on the current CUDA device; norm: enum
 * spectre_norm; eps finite and > 0.  Returns SPECTRE_OK, SPECTRE_ERR_ARG,
 * SPECTRE_ERR_DEVICE (no sm_100 device) or SPECTRE_ERR_NOMEM. */
int residual_norm_create(residual_norm_t *out, int C, int dtype, int norm, float eps);

/* Set an option (enum residual_norm_option) of later calls; not while another thread uses the
 * handle.  Returns SPECTRE_OK or SPECTRE_ERR_ARG. */
int residual_norm_set_option(residual_norm_t h, int option, int value);

/* Enqueue y for T rows on `stream`.  T = 0 does nothing.  Returns SPECTRE_ERR_ARG (a
 * NULL pointer, T < 0, a bad stride), SPECTRE_ERR_ALIGN, SPECTRE_ERR_DEVICE when the
 * handle's device is not current, SPECTRE_ERR_CUDA. */
int residual_norm_run(residual_norm_t h, long long T, const void *out, long long out_stride,
                      const void *x, long long x_stride, const float *gamma, const float *beta,
                      void *y, long long y_stride, void *stream);

/* Workspace of one residual_norm_backward over T rows; 0 for a NULL handle. */
size_t residual_norm_workspace_bytes(residual_norm_t h, long long T);

/* Enqueue the backward pass: dz for T rows, and dgamma, dbeta (set to 0 when T = 0).
 * x may be NULL in the PRE forms.  work: device, 256-byte aligned. */
int residual_norm_backward(residual_norm_t h, long long T, const void *dy, long long dy_stride,
                           const void *out, long long out_stride, const void *x,
                           long long x_stride, const float *gamma, void *dz, long long dz_stride,
                           float *dgamma, float *dbeta, void *work, size_t work_bytes,
                           void *stream);

/* Synchronise `stream`; SPECTRE_ERR_TIMEOUT if a bounded wait for a copy gave up in any
 * residual norm on the handle's device since the last call (its row, and others that the
 * block takes behind it, are NaN, and dgamma and dbeta with them), else SPECTRE_OK.  Clears the record. */
int residual_norm_device_status(residual_norm_t h, void *stream);

/* Release the handle.  NULL-safe; returns SPECTRE_OK. */
int residual_norm_destroy(residual_norm_t h);

#ifdef __cplusplus
}
#endif

#endif /* RESIDUAL_NORM_H */
