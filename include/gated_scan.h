/*
 * gated_scan.h -- C ABI of the gated linear recurrence (part of libspectre_mix),
 * a causal token mixer in the layout of the spectral mix, on NVIDIA B200 (sm_100a).
 *
 * The operation, for every sequence and every channel c = h * D + d of C = H * D:
 *
 *   h_t = a_t h_{t-1} + b_t,   y_t = h_t,   h_{-1} = the initial state (or 0)
 *
 *   GATED_SCAN_SIGMOID: a_t = s(g_t), b_t = (1 - s(g_t)) v_t, s the logistic function.
 *                       g = +infinity holds the state whatever v is; g = -infinity
 *                       replaces it by v.
 *   GATED_SCAN_EXP:     a_t = exp(g_t), b_t = v_t; g is a log decay, g_t <= 0.
 *                       g = 0 with v = 0 holds the state; g = -infinity starts it again.
 *
 * A factor that is exactly zero (a_t, a product of consecutive a_t that is zero in
 * fp32, or 1 - s) takes its operand out, NaN and infinities included: nothing
 * before a gate of zero reaches the rows behind it.  Decays above one (g > 0 with
 * GATED_SCAN_EXP) are taken as they are; then the products of consecutive a_t must
 * stay finite in fp32.
 *
 * The gate is one value per channel ([.., C]) or one per head ([.., H], shared by
 * the head's D channels; its gradient is the sum over them).
 *
 * Numbers: v, y, dy and dv are of the plan's dtype, g and dg of its gate dtype
 * (SPECTRE_F32 or SPECTRE_BF16; an fp32 plan has an fp32 gate).  States (h0, hT,
 * dhT, dh0, states, the step's pool) are fp32, and so is all arithmetic; each
 * bf16 output is rounded once, to nearest even.  The smaller of s(g) and 1 - s(g) is within
 * 16 * 2^-24 of itself; in the scans of a bf16 plan, which take the hardware's exp2, within
 * (1.25 |g| + 16) * 2^-24, and zero below 2^-126, so a step's state may differ from a scan's
 * in its last bits.  A run's results do not depend on
 * how its blocks were scheduled: equal inputs give equal bits.
 *
 * Rows: a tensor of rows is a pointer with a batch stride and a row stride in
 * elements; the C (or H) values of a row are contiguous.  Input rows may overlap
 * (a stride of 0 included), output rows may not, and an output may not overlap an
 * input.  Pointers need their element's own alignment (SPECTRE_ERR_ALIGN); rows
 * aligned to four elements with D (per head) or C (per channel) a multiple of four
 * are read and written four elements at a time, others one by one.
 *
 * Packed sequences: with cu_seqlens (device, nseq + 1 non-decreasing int32), B is 1
 * and sequence n has the rows [cu_seqlens[n], cu_seqlens[n+1]) of the L rows; it may
 * be empty.  h0, hT, dhT and dh0 then have nseq rows.  Rows in no sequence are
 * neither read nor written, or set to zero with zero_outside.  Offsets outside
 * [0, L] or out of order give wrong results but no access outside the tensors.
 *
 * Ownership: the caller owns every tensor and the workspace; the handle holds no
 * device memory and is not changed by a run, so one handle may be used on several
 * streams and threads at once, each call with a workspace of its own.  Long sequences
 * of few channels are one cooperative launch: its blocks start together, when the
 * device has room for all of them.
 *
 * Errors: the spectre_status codes of spectre_mix.h; no function throws or exits.
 */
#ifndef GATED_SCAN_H
#define GATED_SCAN_H

#include "spectre_mix.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gated_scan_s *gated_scan_t;

enum gated_scan_gate { GATED_SCAN_SIGMOID = 0, GATED_SCAN_EXP = 1 };
enum gated_scan_per { GATED_SCAN_PER_CHANNEL = 0, GATED_SCAN_PER_HEAD = 1 };

enum gated_scan_option {
    /* 0 (default).  For tests of the failure path only: 1, a block's first wait for copies of rows gives
     * up at once (it waits for them again before it goes on without them); 2, every wait for the state
     * ahead of a block of rows does.  Rows that are not aligned for copies have no waits of the first kind,
     * and sequences that one block takes alone none of the second. */
    GATED_SCAN_OPT_TEST_WAIT_TIMEOUT = 1,
};

/* Rows between two saved states (see gated_scan_args.states). */
#define GATED_SCAN_CHUNK 128

/*
 * Create a plan on the current CUDA device.  H, D >= 1 with H * D <= 2^20 channels.
 * Returns SPECTRE_OK, SPECTRE_ERR_ARG, SPECTRE_ERR_DEVICE (no sm_100 device) or
 * SPECTRE_ERR_NOMEM.
 */
int gated_scan_create(gated_scan_t *out, int H, int D, int gate, int per, int dtype,
                      int gate_dtype);

/* Set an option (enum gated_scan_option) of later calls; not while another thread uses the
 * handle.  Returns SPECTRE_OK or SPECTRE_ERR_ARG. */
int gated_scan_set_option(gated_scan_t h, int option, int value);

/* A tensor of rows: element (b, t, i) is data[b * batch_stride + t * row_stride + i]. */
typedef struct gated_scan_rows {
    void *data;
    long long batch_stride, row_stride;
} gated_scan_rows;

typedef struct gated_scan_args {
    long long B, L;            /* B sequences of L rows; packed: B = 1, L rows in all */
    const int *cu_seqlens;     /* NULL for dense sequences */
    long long nseq;            /* packed: sequences; ignored when dense */
    gated_scan_rows g, v;      /* inputs of both directions */
    gated_scan_rows y;         /* run: output */
    gated_scan_rows dy;        /* backward: input */
    gated_scan_rows dg, dv;    /* backward: outputs */
    const float *h0;           /* initial states [B or nseq][C], or NULL for 0 */
    float *hT;                 /* run: final states [B or nseq][C], or NULL */
    const float *dhT;          /* backward: gradient of hT, or NULL for 0 */
    float *dh0;                /* backward: gradient of h0, or NULL */
    float *states;             /* [B][ceil(L / GATED_SCAN_CHUNK)][C]: the state before each
                                  chunk's first row.  run writes it (NULL: it does not),
                                  backward reads it */
    void *work;                /* device, 256-byte aligned, gated_scan_workspace_bytes */
    size_t work_bytes;
    int zero_outside;          /* packed: 1 sets output rows outside every sequence to 0 */
} gated_scan_args;

/* Workspace of one gated_scan_run (backward = 0) or gated_scan_backward
 * (backward = 1) over B sequences of L rows; 0 for a NULL handle. */
size_t gated_scan_workspace_bytes(gated_scan_t h, long long B, long long L, int backward);

/*
 * Enqueue the forward recurrence on `stream` (a cudaStream_t, NULL for the legacy
 * default stream).  Reads g, v and h0; writes y, and hT and states where given.
 * B = 0 does nothing; L = 0 sets hT to h0 (or 0).  Returns SPECTRE_ERR_ARG (a NULL
 * pointer, a bad size or stride, a short workspace), SPECTRE_ERR_ALIGN,
 * SPECTRE_ERR_DEVICE when the handle's device is not current, SPECTRE_ERR_CUDA.
 */
int gated_scan_run(gated_scan_t h, const gated_scan_args *a, void *stream);

/*
 * Enqueue the backward pass: reads dy, g, v, h0, dhT and the states that
 * gated_scan_run wrote for the same inputs; writes dg, dv and, where given, dh0.
 * L = 0 sets dh0 to dhT (or 0).
 *   dh_t = dy_t + a_{t+1} dh_{t+1};  dh0 = a_0 dh_0
 *   sigmoid: dv = dh (1 - a), dg = dh (h_{t-1} - v) a (1 - a);
 *   exp:     dv = dh,         dg = dh h_{t-1} a
 * dg is zero where a (or 1 - a) is, whatever dh and the states are.
 * The states between are recomputed in fp32 from `states`; y is not read.
 */
int gated_scan_backward(gated_scan_t h, const gated_scan_args *a, void *stream);

/*
 * One token of each of B sequences: y[i] = new_state[slots[i]] = a state[slots[i]] + b.
 *   g, v, y   : B rows with a row stride in elements.
 *   state     : [S][C] fp32 pool; new_state: [S][C], may be `state` itself (updated in
 *               place) and may not overlap it otherwise.  Pool rows that no slot names
 *               are left as they are.
 *   slots     : [B] int32 (device), or NULL: row i has slot i, and S >= B.
 *               A row whose slot is outside [0, S) is skipped: its y is left as it is, or
 *               set to zero with zero_skipped.
 *               Rows that name the same slot are taken in order, one after another.  Every block
 *               looks through all slots for them, B^2 words in all: no matter to some ten thousand
 *               rows, but seconds for millions.
 */
int gated_scan_step(gated_scan_t h, long long B, const void *g, long long g_stride,
                    const void *v, long long v_stride, const float *state, long long S,
                    const int *slots, void *y, long long y_stride, float *new_state,
                    int zero_skipped, void *stream);

/*
 * Synchronise `stream` and report device-side failures of earlier gated scans on the
 * handle's device: SPECTRE_ERR_TIMEOUT if a bounded wait (for a copy, or for the state
 * ahead of a block of rows) gave up in any run since the last call, else SPECTRE_OK.
 * Clears the record.  A wait that gives up, after some seconds, leaves NaN in the rows
 * behind it, so the failure shows in the output as well.
 */
int gated_scan_device_status(gated_scan_t h, void *stream);

/* Release the handle.  NULL-safe; returns SPECTRE_OK. */
int gated_scan_destroy(gated_scan_t h);

#ifdef __cplusplus
}
#endif

#endif /* GATED_SCAN_H */
