/*
 * zo_block.h - C ABI of the selective state-space block on B200 (sm_100a): the
 * operators beside its dense projections, which are plain library products.
 *
 *   zo_conv        the short causal convolution over time, with its SiLU
 *   zo_scan        the selective scan (a recurrent layer beside the LSTM cell)
 *   zo_block_norm  the norm after a block with its gate and residual scale, the
 *                  residual addition and the norm before the next block
 *
 * conv and scan have a form for prompts (and for the forwards of probe
 * losses), a backward pass, and a form for single tokens; the norm has a
 * forward and a backward pass (its rows are tokens).
 *
 * Parameter sets.  A probe chunk of CD-RGE evaluates one model at many
 * perturbed parameter copies, and this block's parameters besides the
 * projections are small (A, skip, biases, taps, norm weights: the kind of
 * segment that is copied per probe sign).  So every call takes `sets` copies of
 * them and `rows` rows, rows a multiple of sets, and row r uses set
 * r / (rows / sets): all copies of a chunk run in one call.  sets = 1 is the
 * ordinary use.  A parameter shared by all sets has stride 0.  Gradients of
 * parameters are per set.
 *
 * Conventions shared by every call (the same as include/zo.h):
 *   - Every call returns a ZO_* status.  No C++ exception crosses this
 *     interface.  Argument errors are found on the host before anything is
 *     launched, and then nothing is written.
 *   - Calls only enqueue work on `stream` (a cudaStream_t as void*, NULL = the
 *     legacy default stream) of the current device, which must be the one that
 *     holds the tensors.  They never synchronise or allocate and keep nothing
 *     between calls: calls on different streams do not disturb one another as
 *     long as each has its own workspace and outputs, and a call can be captured
 *     into a CUDA graph.
 *   - There is at least one row and one step; steps and channels are at most
 *     2^30.
 *   - All pointers are device pointers owned by the caller, aligned to their
 *     element type.  Strides count elements and may be any value that keeps
 *     the elements of an output apart; the innermost dimension (channels, or
 *     states of a group) is contiguous.  Full speed needs rows and steps that
 *     start on 16 bytes.
 *   - Parameters, their gradients and recurrent states are fp32.  Activations
 *     are fp32, bf16 or fp16 (`dtype`), converted exactly to fp32, computed with
 *     in fp32 and rounded once to nearest even.
 *   - Infinite and NaN inputs give what the formulas give in fp32 (what a length or an absent
 *     tensor leaves out does not count); only dB and dC of zo_scan may be NaN in place of infinite
 *     where B or C itself is infinite.
 *   - Outputs must not overlap inputs, except where a call says so.
 *   - Results do not depend on timing: no floating-point atomics.
 */
#ifndef ZO_BLOCK_H_
#define ZO_BLOCK_H_

#include "zo.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ZO_DTYPE_FP16 2  /* beside ZO_DTYPE_FP32 and ZO_DTYPE_BF16: activations here */

#define ZO_MAX_TAPS 8      /* most taps of zo_conv            */
#define ZO_MAX_STATES 128  /* most states per channel of zo_scan */
#define ZO_MAX_NORM_WIDTH 16384 /* widest row of zo_block_norm */

/* A [rows][steps][contiguous] tensor of activations: element strides of a row
 * and of a step.  ptr NULL = absent, where a call allows that. */
typedef struct zo_tensor {
  void* ptr;
  int64_t row, step;
} zo_tensor;

/* An fp32 array whose leading dimension (parameter sets, or rows for recurrent
 * states) has a stride in elements; the rest is contiguous. */
typedef struct zo_f32 {
  float* ptr;
  int64_t stride;
} zo_f32;

/* ---- short causal convolution ------------------------------------------- */

#define ZO_CONV_SILU 1 /* flags: out = pre * sigmoid(pre), else out = pre */

/* pre_t = bias + sum_k weight[k] x_{t - taps + 1 + k} per channel. */
typedef struct zo_conv_args {
  int32_t rows, seq, channels;
  int32_t taps;               /* 1..ZO_MAX_TAPS                                   */
  int32_t sets, dtype, flags;
  zo_tensor x, out;           /* [rows][seq][channels]                            */
  zo_f32 weight;              /* [sets][taps][channels]; tap taps-1 meets x_t     */
  zo_f32 bias;                /* [sets][channels]; optional                       */
  const int32_t* lengths;     /* [rows], optional: steps of each row, 0..seq      */
  zo_tensor state_in;         /* [rows][taps-1][channels], optional (zeros): the  */
                              /* inputs before x_0, oldest first                  */
  zo_tensor state_out;        /* the same after the last step; optional; may be   */
                              /* state_in itself                                  */
  int32_t* status;            /* optional: ZO_ERR_BOUNDS is stored here if a      */
                              /* length is outside 0..seq (it is then clamped)    */
} zo_conv_args;

/* The whole of every row.  Steps at or behind a row's length read nothing and
 * give 0.  state_out holds the last taps-1 inputs before the row's length (those
 * of state_in included where the row is shorter). */
ZO_API int zo_conv(const zo_conv_args* args, void* stream);

/* One step: seq = 1, state_in required, lengths unused.  state_out is the
 * window moved by one (it may be state_in itself); without it the window is
 * left as it is. */
ZO_API int zo_conv_step(const zo_conv_args* args, void* stream);

/* Gradients from dout.  dx, dweight and dbias are written whole (0 at steps
 * behind a row's length); `out` and state_out of args are not used. */
typedef struct zo_conv_grads {
  zo_tensor dout, dx;         /* [rows][seq][channels]                            */
  zo_f32 dweight;             /* [sets][taps][channels]                           */
  zo_f32 dbias;               /* [sets][channels]; optional                       */
  zo_tensor dstate_out;       /* gradient of state_out; optional (zeros)          */
  zo_tensor dstate_in;        /* gradient of state_in; optional                   */
} zo_conv_grads;

/* Bytes of workspace that zo_conv_backward needs for these sizes (only the
 * integer fields of args are read); -1 for sizes that it refuses. */
ZO_API int64_t zo_conv_backward_workspace(const zo_conv_args* args);
ZO_API int zo_conv_backward(const zo_conv_args* args, const zo_conv_grads* grads, void* workspace,
                            int64_t workspace_bytes, void* stream);

/* ---- selective scan ------------------------------------------------------- */

#define ZO_SCAN_SOFTPLUS 1 /* flags: d = log(1 + exp(delta + bias)), else d = delta + bias */
#define ZO_SCAN_CHUNK 16   /* steps between two kept states (checkpoints) */

/* Per row, channel c (of group c / (channels / groups)) and state n:
 *   d_t = softplus(delta_t + delta_bias)
 *   h_t[n] = exp(d_t A[n]) h_{t-1}[n] + d_t u_t B_t[n]
 *   out_t = (sum_n C_t[n] h_t[n] + skip u_t) silu(z_t)                        */
typedef struct zo_scan_args {
  int32_t rows, seq, channels;
  int32_t groups;             /* divides channels; B and C are shared in a group  */
  int32_t states;             /* N: 1..ZO_MAX_STATES                              */
  int32_t sets, dtype, flags;
  zo_tensor u, delta, out;    /* [rows][seq][channels]                            */
  zo_tensor z;                /* the gate; optional                               */
  zo_tensor B, C;             /* [rows][seq][groups * N]                          */
  zo_f32 A;                   /* [sets][channels][N]; beyond 2.3e38 (the largest  */
                              /* fp32 over log2(e)) it counts as that             */
  zo_f32 skip, delta_bias;    /* [sets][channels]; optional                       */
  const int32_t* lengths;     /* [rows], optional: steps of each row, 0..seq      */
  zo_f32 state_in;            /* [rows][channels][N]; optional (zeros)            */
  zo_f32 state_out;           /* after each row's last step; optional; may be     */
                              /* state_in itself                                  */
  float* checkpoints;         /* [rows][ceil(seq / ZO_SCAN_CHUNK)][channels][N],  */
                              /* 16-byte aligned: the states before steps 0,      */
                              /* ZO_SCAN_CHUNK, ...; written by zo_scan where     */
                              /* given, read by zo_scan_backward                  */
  int32_t* status;            /* as in zo_conv_args                               */
} zo_scan_args;

/* Bytes of workspace of the two calls for these sizes (only the integer fields
 * are read; 0 is possible); -1 for sizes that they refuse. */
ZO_API int64_t zo_scan_workspace(const zo_scan_args* args);
ZO_API int64_t zo_scan_backward_workspace(const zo_scan_args* args);

/* The whole of every row.  Steps at or behind a row's length read nothing,
 * leave the state as it is and give 0. */
ZO_API int zo_scan(const zo_scan_args* args, void* workspace, int64_t workspace_bytes,
                   void* stream);

/* One step: seq = 1, state_in required, lengths unused.  state_out may be
 * state_in itself; without it the state is left as it is. */
ZO_API int zo_scan_step(const zo_scan_args* args, void* stream);

/* Gradients from dout, with the checkpoints that zo_scan wrote for the same
 * inputs.  Everything is written whole (0 at steps behind a row's length); `out`,
 * state_in and state_out of args are not used. */
typedef struct zo_scan_grads {
  zo_tensor dout;             /* [rows][seq][channels]                            */
  zo_tensor du, ddelta;       /* [rows][seq][channels]                            */
  zo_tensor dz;               /* required where z is given                        */
  zo_tensor dB, dC;           /* [rows][seq][groups * N]                          */
  zo_f32 dA;                  /* [sets][channels][N]                              */
  zo_f32 dskip, ddelta_bias;  /* [sets][channels]; optional                       */
  zo_f32 dstate_out;          /* [rows][channels][N]: gradient of state_out;      */
                              /* optional (zeros)                                 */
  zo_f32 dstate_in;           /* gradient of state_in; optional                   */
} zo_scan_grads;
ZO_API int zo_scan_backward(const zo_scan_args* args, const zo_scan_grads* grads, void* workspace,
                            int64_t workspace_bytes, void* stream);

/* ---- norms around a block --------------------------------------------------- */

#define ZO_NORM_GATE_FIRST 1 /* flags: the gate multiplies o before its norm, else after */

/* With rms(v) = v / sqrt(mean(v^2) + eps) over a row:
 *   p = rms(o) w_post silu(gate)          or, with ZO_NORM_GATE_FIRST,
 *   p = rms(o silu(gate)) w_post
 *   x_out = x + scale p
 *   n_out = rms(x_out) w_pre              (from the unrounded x_out)
 * Without o, x_out = x (the norm before a first block); without gate, its
 * factor is 1; without w_post there is no norm after the block; without scale it
 * is 1. */
typedef struct zo_norm_args {
  int32_t rows, channels;     /* channels: 1..ZO_MAX_NORM_WIDTH                   */
  int32_t sets;
  int32_t dtype;              /* o, gate, n_out                                   */
  int32_t x_dtype;            /* x, x_out: dtype or ZO_DTYPE_FP32                 */
  int32_t flags;
  float eps;                  /* > 0                                              */
  zo_tensor x, x_out;         /* [rows][channels] (step strides unused); x_out    */
                              /* is optional where n_out is given, and may be x   */
  zo_tensor o, gate;          /* [rows][channels]; optional (gate only with o)    */
  zo_tensor n_out;            /* [rows][channels]; with w_pre only; optional      */
  zo_f32 w_post, scale;       /* [sets][channels]; optional, only with o          */
  zo_f32 w_pre;               /* [sets][channels]; given exactly where n_out (or  */
                              /* its gradient) is                                 */
} zo_norm_args;
ZO_API int zo_block_norm(const zo_norm_args* args, void* stream);

/* Gradients from dn (of n_out) and dx_out (of x_out), either optional but not
 * both.  args.x_out is an input here, as zo_block_norm stored it; args.x and
 * args.n_out are not used.  All gradients of what was given are written. */
typedef struct zo_norm_grads {
  zo_tensor dn;               /* [rows][channels] dtype; with w_pre               */
  zo_tensor dx_out;           /* [rows][channels] x_dtype                         */
  zo_tensor dx;               /* [rows][channels] x_dtype; may be dx_out itself   */
  zo_tensor d_o, dgate;       /* [rows][channels] dtype, required with o, gate    */
  zo_f32 dw_post, dscale, dw_pre; /* [sets][channels]; each required with its     */
                              /* parameter                                        */
} zo_norm_grads;
ZO_API int64_t zo_block_norm_backward_workspace(const zo_norm_args* args);
ZO_API int zo_block_norm_backward(const zo_norm_args* args, const zo_norm_grads* grads,
                                  void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZO_BLOCK_H_ */
