/*
 * atlas_ops.h -- C ABI of the operators around the memory update in a recurrent
 * layer, in the same library (libatlasmem.so):
 *
 *   norm  residual addition and root-mean-square norm, output in 32, 16 or 8 bits
 *   conv  short causal convolution per channel, optionally through SiLU
 *   scan  selective state space scan: a diagonal recurrence whose decay depends on
 *         token, channel and state
 *
 * each forward and backward; conv and scan run whole sequences, packed sequences of
 * unequal lengths and single tokens (L = 1) through the same entry point.
 *
 * The conventions of atlas_mem.h hold: device pointers owned by the caller, work
 * enqueued on `stream` without synchronising, argument errors reported before
 * anything is launched, no device memory allocated, scratch from the caller's
 * workspace, status codes ATLAS_OK / ATLAS_ERR_*.  A call may be captured into a
 * graph; two calls that can run at the same time need workspaces of their own.
 * Results do not depend on the order in which thread blocks run (no floating-point
 * atomics): the same call on the same inputs gives the same bits.
 *
 * Sources: "[Paper Review] Titans 논문 이해하기" (the layer around the memory:
 * short convolutions of q, k, v and SiLU) and "It's All Connected: ... (Miras)"
 * (projections, convolution and norm of q and k, output gate).  The scan is the
 * recurrence with a diagonal decay that both pages list among the models whose
 * state has a fixed size.
 *
 * Tensors: the channel index is always innermost and contiguous.  Batch and token
 * strides are in elements and may be any value >= 0 as long as no two written
 * elements share an address; 0 for both asks for the contiguous layout.  Any
 * alignment to the element's size is accepted; 16-byte aligned pointers and strides
 * of a multiple of 16 bytes take the wide loads.  No output may overlap an input or
 * another output, except where an entry point says so.
 */
#ifndef ATLAS_OPS_H
#define ATLAS_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "atlas_mem.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types beyond ATLAS_F32 (0) and ATLAS_BF16 (1) */
#define ATLAS_F16 2
#define ATLAS_E4M3 3 /* 8 bits: 4 exponent, 3 mantissa bits, largest value 448 */

/* activation of the convolution */
#define ATLAS_ACT_NONE 0
#define ATLAS_ACT_SILU 1 /* p / (1 + exp(-p)) */

/* ------------------------------------------------------------------ norm
 * Per row of d channels:
 *   h = x + residual            (h = x without a residual), in 32 bits
 *   y = h / sqrt(mean(h^2) + eps) * weight
 * residual_out receives h rounded to r_dtype; y is taken from the unrounded h.
 * An 8-bit output is stored with one scale per group of `group` channels (the last
 * group of a row may be shorter; group = 0: the whole row):
 *   scale = max(max |y| over the group, 1e-30) / 448,   q = e4m3(y / scale)
 * rounded to nearest even (the quotient in 32 bits, as y times 1 / scale), so that
 * y = q * scale.  A row of zeros gives zeros, with eps = 0 too (its dx is then dh, and it
 * adds nothing to dw).  h^2 and its mean are taken in 32 bits: with eps = 0 a row that is
 * not zero but whose mean of squares is below 2^-149 is not normalised.
 * With a row of keys or queries (d = the head's width) and weight = 1 / sqrt(d)
 * this is the l2 normalisation that the memory update expects of K and Q. */
typedef struct atlas_norm_cfg {
  long rows;       /* >= 0 */
  int d;           /* channels of a row, 1 .. ATLAS_NORM_MAX_D */
  int dtype;       /* x and y's gradient: ATLAS_F32, ATLAS_BF16, ATLAS_F16 */
  int r_dtype;     /* residual, residual_out and their gradients (same three) */
  int w_dtype;     /* weight (same three) */
  int out_dtype;   /* y: the same three or ATLAS_E4M3 */
  int group;       /* channels per scale of an ATLAS_E4M3 output, 0 = the whole row */
  float eps;       /* >= 0 */
  long x_stride, r_stride, y_stride; /* elements from row to row, 0 = d */
  void* workspace; /* backward only */
  size_t workspace_bytes;
} atlas_norm_cfg;
#define ATLAS_NORM_MAX_D 32768

/*   x            [rows, d] dtype
 *   residual     [rows, d] r_dtype or NULL
 *   weight       [d] w_dtype or NULL (ones)
 *   y            [rows, d] out_dtype out
 *   residual_out [rows, d] r_dtype out, or NULL; may be `residual` itself
 *   scale        [rows, groups] fp32 out, contiguous; NULL unless out_dtype is ATLAS_E4M3 */
int atlas_norm_forward(const void* x, const void* residual, const void* weight,
                       const atlas_norm_cfg* cfg, void* y, void* residual_out, float* scale,
                       void* stream);

size_t atlas_norm_backward_workspace_bytes(const atlas_norm_cfg* cfg);

/* Gradients of L with dy = dL/dy (of the output before its rounding to 8 bits) and,
 * where h goes on as the residual stream, dh = dL/d residual_out:
 *   dx = dL/dh = dL/dx = dL/d residual,   dw = dL/d weight
 *   h   [rows, d] r_dtype: what the norm was taken of (the forward's residual_out, or
 *       x itself when there was no residual, with r_dtype = dtype), r_stride
 *   dy  [rows, d] dtype, y_stride;   dh [rows, d] r_dtype or NULL, r_stride
 *   dx  [rows, d] r_dtype out, r_stride; may be dh itself
 *   dw  [d] fp32 out, or NULL (required to be NULL when weight is NULL) */
int atlas_norm_backward(const void* h, const void* weight, const void* dy, const void* dh,
                        const atlas_norm_cfg* cfg, void* dx, float* dw, void* stream);

/* ------------------------------------------------- sequences and their states
 * conv and scan take B sequences in one of two forms:
 *   seq_start == NULL  every sequence has L tokens: row t of sequence b lies at
 *                      b * batch_stride + t * token_stride
 *   seq_start != NULL  the sequences are packed: L rows in all, sequence b has rows
 *                      seq_start[b] .. seq_start[b + 1] - 1 (device int [B + 1]; empty
 *                      sequences allowed; row r lies at r * token_stride).  Rows before
 *                      the first and behind the last sequence are neither read nor
 *                      written.
 * A sequence's state is read from state_in and written to state_out (either may be
 * NULL: start from zeros, do not return it; both may be the same buffer).  The state
 * of an empty sequence is passed on unchanged.
 *   slot   NULL: sequence b has state b.  Else device int [B]: sequence b has state
 *          slot[b] of n_slots; a negative entry marks b as padding: nothing of it is
 *          written and its state is not read (its rows may be).
 *   carry  NULL: every sequence starts from its state.  Else device bytes [B]: a
 *          sequence with carry[b] == 0 starts from zeros.
 * The arrays on the device cannot be checked before the launch.  The kernels check
 * them: a sequence whose rows are not 0 <= seq_start[b] <= seq_start[b + 1] <= L, whose
 * slot is >= n_slots, or whose slot an earlier sequence has too, is left out like padding, and
 * so is every sequence from the first fall of seq_start on (seq_start[b + 1] < seq_start[b]),
 * behind which rows could belong to two; *status_dev (when given) is set to
 * ATLAS_ERR_INVALID.  (Slots have to differ because two sequences with one state would
 * race.  A backward call with a bad seq_start reports it and stays inside its tensors; its
 * outputs are then not defined.) */

/* ------------------------------------------------------------------ conv
 *   p_t[c] = bias[c] + sum_{k < W} weight[c][k] x_{t - W + 1 + k}[c],   y = SiLU(p) or p
 * Inputs before a sequence's first token come from its state, its last W - 1 inputs:
 * state [.., W - 1, C], oldest first, in dtype. */
typedef struct atlas_conv_cfg {
  int B, L, C;     /* sequences, tokens (packed: rows), channels */
  int W;           /* taps, 1 .. ATLAS_CONV_MAX_W */
  int act;         /* ATLAS_ACT_* */
  int dtype;       /* x, y, state, dy, dx: ATLAS_F32, ATLAS_BF16, ATLAS_F16 */
  int w_dtype;     /* weight and bias (same three) */
  int head_dim;    /* 0: y is token-major like x.  > 0 (divides C): y is head-major,
                      channel c of token t at (c / head_dim) * y_head_stride +
                      t * y_token_stride + c % head_dim: with the strides 0
                      [B, C / head_dim, L, head_dim], what atlas_mem_forward reads
                      (packed: [C / head_dim, L, head_dim]) */
  long x_batch_stride, x_token_stride;
  long y_batch_stride, y_token_stride, y_head_stride;
  const int* seq_start;
  const int* slot;
  int n_slots;
  const uint8_t* carry;
  int* status_dev;
  void* workspace; /* backward only */
  size_t workspace_bytes;
} atlas_conv_cfg;
#define ATLAS_CONV_MAX_W 8

/*   x [.., L, C] dtype;  weight [C, W], bias [C] or NULL, w_dtype, contiguous
 *   y [.., L, C] dtype out;  state_in, state_out [n, W - 1, C] dtype, contiguous, or NULL */
int atlas_conv_forward(const void* x, const void* weight, const void* bias,
                       const atlas_conv_cfg* cfg, void* y, const void* state_in, void* state_out,
                       void* stream);

size_t atlas_conv_backward_workspace_bytes(const atlas_conv_cfg* cfg);

/* Gradients for L with dL/dy = dy and dL/d state_out = dstate.  slot must be NULL.
 *   dy     [.., L, C] dtype, y's strides;  state_in [B, W - 1, C] as in the forward
 *   dstate [B, W - 1, C] fp32 in/out or NULL: dL/d state_out on entry, dL/d state_in on
 *          return (zero for a sequence with carry[b] == 0)
 *   dx     [.., L, C] dtype out, x's strides
 *   dw [C, W], dbias [C] fp32 out (dbias may be NULL) */
int atlas_conv_backward(const void* x, const void* weight, const void* bias,
                        const atlas_conv_cfg* cfg, const void* state_in, const void* dy,
                        float* dstate, void* dx, float* dw, float* dbias, void* stream);

/* ------------------------------------------------------------------ scan
 * Per channel c of D (in group g = c / (D / G)) with N states:
 *   dt_t[c] = softplus(dt_raw_t[c] + dt_bias[c])      (without softplus: the sum)
 *   h_t[c][n] = exp(dt_t[c] A[c][n]) h_{t-1}[c][n] + dt_t[c] B_t[g][n] x_t[c]
 *   y_t[c] = (sum_n C_t[g][n] h_t[c][n] + D[c] x_t[c]) * SiLU(z_t[c])
 * The state h [.., D, N], every sum and every exponential are held in 32 bits. */
typedef struct atlas_scan_cfg {
  int B, L, D;     /* sequences (at most 65535), tokens (packed: rows), channels */
  int N;           /* states per channel, 1 .. ATLAS_SCAN_MAX_N */
  int G;           /* groups that share B and C, divides D */
  int dtype;       /* x, dt, B, C, z, y and their gradients: ATLAS_F32, ATLAS_BF16, ATLAS_F16 */
  int softplus;    /* 0: dt is used as it is (plus dt_bias) */
  long x_batch_stride, x_token_stride;
  long dt_batch_stride, dt_token_stride;
  long z_batch_stride, z_token_stride;
  long y_batch_stride, y_token_stride;
  long b_batch_stride, b_token_stride; /* B: [.., L, G, N], the last two contiguous */
  long c_batch_stride, c_token_stride; /* C: likewise */
  const int* seq_start;
  const int* slot;
  int n_slots;
  const uint8_t* carry;
  int* status_dev;
  void* workspace;
  size_t workspace_bytes;
} atlas_scan_cfg;
#define ATLAS_SCAN_MAX_N 128

/* Bytes of workspace atlas_scan_forward needs (may be 0); (size_t)-1 for an invalid
 * description. */
size_t atlas_scan_workspace_bytes(const atlas_scan_cfg* cfg);

/*   x, dt, z [.., L, D] dtype (z may be NULL: no gate);  B, C [.., L, G, N] dtype
 *   A [D, N], Dskip [D] or NULL, dt_bias [D] or NULL: fp32, contiguous
 *   y [.., L, D] dtype out;  h_in, h_out [n, D, N] fp32, contiguous, or NULL */
int atlas_scan_forward(const void* x, const void* dt, const float* A, const void* B, const void* C,
                       const float* Dskip, const void* z, const float* dt_bias,
                       const atlas_scan_cfg* cfg, void* y, const float* h_in, float* h_out,
                       void* stream);

size_t atlas_scan_backward_workspace_bytes(const atlas_scan_cfg* cfg);

/* Gradients for L with dL/dy = dy and dL/d h_out = dh, the forward's states computed
 * again.  slot must be NULL.
 *   dy [.., L, D] dtype, y's strides;  h_in [B, D, N] as in the forward, or NULL
 *   dh [B, D, N] fp32 in/out or NULL: dL/d h_out on entry, dL/d h_in on return (zero for a
 *      sequence with carry[b] == 0)
 *   dx, ddt (of dt_raw), dB, dC, dz: dtype out, with the strides of x, dt, B, C, z; dz is
 *      NULL exactly when z is
 *   dA [D, N], dD [D] (NULL exactly when Dskip is), ddt_bias [D] (NULL exactly when dt_bias
 *      is): fp32 out */
int atlas_scan_backward(const void* x, const void* dt, const float* A, const void* B,
                        const void* C, const float* Dskip, const void* z, const float* dt_bias,
                        const atlas_scan_cfg* cfg, const float* h_in, const void* dy, float* dh,
                        void* dx, void* ddt, float* dA, void* dB, void* dC, float* dD, void* dz,
                        float* ddt_bias, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ATLAS_OPS_H */
