/*
 * ttt_ops.h -- C ABI of the operators that stand beside the TTT layer in a
 * sequence-mixing block, each with its gradient:
 *
 *   ttt_rope_*  rotary positions with several axes (time, height, width), for the
 *               keys and queries of image, video and text layers
 *   ttt_scan_*  the gated linear recurrence h_t = a_t h_{t-1} + u_t, a per-channel
 *               state that is carried from call to call as the layer's W is
 *   ttt_norm_*  group norm with an activation, channels last, which also reads the
 *               layer's heads-first output with one group a head
 *
 * The web pages that define the layer name none of these operators; the
 * formulas below define them.
 *
 * Conventions (those of ttt.h, and)
 *   - Tensors are described by ttt_strides, in elements; the channels of a row are
 *     contiguous.  Any strides are read (a stride of 0 broadcasts); the elements of
 *     a written tensor must not overlap one another (TTT_ERR_INVALID_ARG).  Device
 *     pointers are aligned to their element type; 16-byte alignment of pointers
 *     and strides is faster.  A written tensor may not share elements with one
 *     that is read, except where a call says so.
 *   - A handle holds host-side configuration only and is never changed by a call:
 *     calls on one handle may run at once, on any streams, threads and devices.
 *   - Calls enqueue on `stream` and return; they allocate nothing and may be
 *     captured into a CUDA graph.  The workspace is the caller's, its contents
 *     before a call do not matter, and calls whose GPU work overlaps need a
 *     workspace each (two captured graphs that replay at once among them).
 *   - `status` (optional, 4 bytes of device memory) collects the device status bits:
 *     a call that goes wrong on the device sets bits, and its outputs are then not to
 *     be used; no call clears them.  Bit 1 (value 2): a bounded device wait ran out
 *     (2 s, as in ttt.h).  Only the recurrence waits on other blocks: rotary positions
 *     take no status, and the norm takes one, as all calls with a workspace do, and
 *     never sets it.
 *   - Results do not depend on timing: the same call gives the same bits.  Rows that
 *     start on other alignments or strides may take another kernel, of the same
 *     definition and arithmetic, whose last bits may differ.
 */
#ifndef TTT_OPS_H_
#define TTT_OPS_H_

#include "ttt.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ttt_strides {
  int64_t batch; /* elements between batch entries */
  int64_t head;  /* elements between heads (rope) or groups (norm); not used by scan */
  int64_t token; /* elements between tokens */
} ttt_strides;

/* ------------------------------------------------------------------ rotary positions
 * A token has `axes` coordinates.  Axis a owns pairs[a] pairs of channels; pair j of
 * the axis turns by phi = p_a * base[a]^(-j / pairs[a]).  With i the running number of
 * the pair over all axes and M = sum of pairs:
 *   y[p] = x[p] cos phi - x[q] sin phi,   y[q] = x[q] cos phi + x[p] sin phi,
 *   (p, q) = (i, i + M) with TTT_ROPE_HALVES, (2i, 2i + 1) with TTT_ROPE_INTERLEAVED.
 * Channels from 2M on are copied.  Angles are formed and reduced in 64 bits.  Before
 * its rounding to `dtype` an output is off by 2^-22 (|x[p]| + |x[q]|) at most in fp32, by
 * 2^-20 of them in bf16.
 * TTT_ERR_UNSUPPORTED: d above 4096, more than TTT_ROPE_MAX_PAIRS pairs, N above 2^40. */
typedef enum { TTT_ROPE_HALVES = 0, TTT_ROPE_INTERLEAVED = 1 } ttt_rope_pairing;
typedef enum { TTT_POS_I32 = 0, TTT_POS_F32 = 1 } ttt_pos_dtype;
#define TTT_ROPE_MAX_AXES 4
#define TTT_ROPE_MAX_PAIRS 256

typedef struct ttt_rope_config {
  int32_t d;                        /* channels of a head, >= 2 * sum(pairs), at most 4096 */
  int32_t axes;                     /* 1..TTT_ROPE_MAX_AXES */
  int32_t pairs[TTT_ROPE_MAX_AXES]; /* pairs of each axis, each >= 1, at most TTT_ROPE_MAX_PAIRS in all */
  double base[TTT_ROPE_MAX_AXES];   /* each finite and > 0 */
  int32_t pairing;                  /* ttt_rope_pairing */
  int32_t dtype;                    /* ttt_dtype of x and y */
} ttt_rope_config;

typedef struct ttt_rope ttt_rope;
int ttt_rope_create(const ttt_rope_config* cfg, ttt_rope** out);
void ttt_rope_destroy(ttt_rope* handle);

/* y = rotated x, [B, H, N, d].  pos: [N, axes], or with pos_batch != 0 one such block
 * for each batch entry, pos_batch elements apart.  inverse = 1 turns by -phi: the
 * inverse rotation, which is also the gradient (x is then dL/dy and y is dL/dx).
 * y may be x (same pointer and strides).  B, H >= 1; N >= 0 (0: nothing to do). */
int ttt_rope_apply(const ttt_rope* handle, int32_t B, int32_t H, int64_t N, const void* x, const ttt_strides* xs,
                   const void* pos, int32_t pos_dtype, int64_t pos_batch, void* y, const ttt_strides* ys,
                   int32_t inverse, void* stream);

/* ------------------------------------------------------------ gated linear recurrence
 * Per batch entry and channel, over tokens t = 1..len:
 *   h_t = a_t h_{t-1} + u_t,  h_0 = h0 (or 0)
 *   a = g | sigma(g) | exp(g);   u = x | (1 - a) x
 * Backward, for the gradients dh of every h_t and dh_last of h_len:
 *   lam_t = dh_t + a_{t+1} lam_{t+1}  (lam_len = dh_len + dh_last)
 *   dx = lam | (1 - a) lam;  da = lam h_{t-1} | lam (h_{t-1} - x);  dg = da a'(g);  dh0 = a_1 lam_1
 * States and products are fp32; g, x, h, dh, dg, dx are in `dtype`.  Products of the
 * gates of up to 256 tokens in a row are formed: gates that grow a state (|a| > 1) have to
 * keep them, and the states, within fp32's range; beyond it, and from an infinite state
 * on, results are infinite or NaN, in their channel and batch entry alone.
 * TTT_ERR_UNSUPPORTED: L above 2^30; with c channels a column (bf16: 64, fp32: 32),
 * B ceil(D / c) ceil(L / 256) above 2^30 forward, B ceil(D / c) ceil(L / 128) backward
 * (sequences of up to 16 tokens are not cut so: for them, B ceil(D / 2) in bf16 or B D in
 * fp32 above 2^38). */
typedef enum { TTT_GATE_VALUE = 0, TTT_GATE_SIGMOID = 1, TTT_GATE_EXP = 2 } ttt_gate_kind;
typedef enum { TTT_SCAN_PLAIN = 0, TTT_SCAN_COMPLEMENT = 1 } ttt_scan_input;

typedef struct ttt_scan_config {
  int32_t D;     /* channels, >= 1 */
  int32_t gate;  /* ttt_gate_kind */
  int32_t input; /* ttt_scan_input */
  int32_t dtype; /* ttt_dtype */
} ttt_scan_config;

typedef struct ttt_scan ttt_scan;
int ttt_scan_create(const ttt_scan_config* cfg, ttt_scan** out);
void ttt_scan_destroy(ttt_scan* handle);

/* Workspace bytes of a call (16-byte aligned buffer) and bytes of the state that a
 * forward call leaves for its backward call (opaque, 16-byte aligned).  0: none
 * needed, the pointer may be NULL. */
size_t ttt_scan_workspace_size(const ttt_scan* handle, int32_t B, int64_t L);
size_t ttt_scan_saved_size(const ttt_scan* handle, int32_t B, int64_t L);

/* g, x, h: [B, L, D].  B >= 1, 0 <= L <= 2^30.  lengths: [B] int32 or NULL (then L
 * everywhere; values are clamped to 0..L): rows of h from a sequence's length on are
 * left as they were, whatever g and x hold there.  h0: [B, D] fp32 or NULL.
 * h_last: [B, D] fp32 or NULL, the state after the last token (h0 where there is
 * none); it may be h0.  saved: for ttt_scan_backward, or NULL. */
int ttt_scan_forward(const ttt_scan* handle, int32_t B, int64_t L, const void* g, const ttt_strides* gs,
                     const void* x, const ttt_strides* xs, const float* h0, const int32_t* lengths, void* h,
                     const ttt_strides* hs, float* h_last, void* saved, void* workspace, size_t workspace_bytes,
                     unsigned* status, void* stream);

/* The gradients of a forward call with the same g, x, lengths and L, which left `saved`.
 * dh_last: [B, D] fp32 or NULL (zero).  dg, dx: [B, L, D], rows from a sequence's
 * length on left as they were.  dh0: [B, D] fp32 or NULL. */
int ttt_scan_backward(const ttt_scan* handle, int32_t B, int64_t L, const void* dh, const ttt_strides* dhs,
                      const float* dh_last, const void* g, const ttt_strides* gs, const void* x,
                      const ttt_strides* xs, const int32_t* lengths, const void* saved, void* dg,
                      const ttt_strides* dgs, void* dx, const ttt_strides* dxs, float* dh0, void* workspace,
                      size_t workspace_bytes, unsigned* status, void* stream);

/* Zeroes the rows of y [B, L, D] from each sequence's length on (lengths as above, not
 * NULL): what forward and backward leave as it was, for a tensor that is new. */
int ttt_scan_clear(const ttt_scan* handle, int32_t B, int64_t L, const int32_t* lengths, void* y,
                   const ttt_strides* ys, void* stream);

/* -------------------------------------------------- group norm with an activation
 * Channel c = k (C / groups) + i of group k; mean and variance (divided by n) over the
 * group's channels of all N tokens of a batch entry:
 *   xhat = (x - mean) / sqrt(var + eps);  z = xhat weight[c] + bias[c]
 *   y = z | z sigma(z) | z Phi(z)     (SiLU; GELU with the normal distribution function)
 * Backward, dz = dy y'(z):
 *   dweight = sum dz xhat, dbias = sum dz (over tokens and batch entries); with q = dz weight
 *   dx = (q - mean(q) - xhat mean(q xhat)) / sqrt(var + eps)
 * Statistics, weight, bias and their gradients are fp32; x, y, dx, dy are in `dtype`.
 * The statistics are those of all N tokens of the call: each output depends on later tokens
 * as on earlier ones, and tokens that are handed over in parts, or one at a time, have
 * other statistics than the whole.  It fits layers that see a whole image, view or clip, not
 * causal or streamed ones (the layer's causal form, a state carried by the recurrence).
 * The strides' `head` is the distance between groups: C / groups for channels last
 * [B, N, C]; the layer's O [B, H, N, d] is read with groups = H. */
typedef enum { TTT_ACT_NONE = 0, TTT_ACT_SILU = 1, TTT_ACT_GELU = 2 } ttt_act_kind;

typedef struct ttt_norm_config {
  int32_t C;      /* channels, a multiple of groups, at most 65536 */
  int32_t groups; /* >= 1 */
  int32_t act;    /* ttt_act_kind */
  float eps;      /* finite, >= 0 */
  int32_t dtype;  /* ttt_dtype */
} ttt_norm_config;

typedef struct ttt_norm ttt_norm;
int ttt_norm_create(const ttt_norm_config* cfg, ttt_norm** out);
void ttt_norm_destroy(ttt_norm* handle);
size_t ttt_norm_workspace_size(const ttt_norm* handle, int32_t B, int64_t N, int32_t backward);

/* x, y: 1 <= B <= 65535, 1 <= N <= 2^30 tokens of C channels.  weight, bias: [C] fp32 or NULL (one, zero).
 * stats: [B, groups, 2] fp32 (mean, 1 / sqrt(var + eps)) for the backward call, or
 * NULL.  y may be x (same pointer and strides), which leaves no x for a backward call. */
int ttt_norm_forward(const ttt_norm* handle, int32_t B, int64_t N, const void* x, const ttt_strides* xs,
                     const float* weight, const float* bias, void* y, const ttt_strides* ys, float* stats,
                     void* workspace, size_t workspace_bytes, unsigned* status, void* stream);

/* dweight, dbias: [C] fp32, overwritten, or NULL.  dx may be dy (same pointer and strides). */
int ttt_norm_backward(const ttt_norm* handle, int32_t B, int64_t N, const void* dy, const ttt_strides* dys,
                      const void* x, const ttt_strides* xs, const float* weight, const float* bias,
                      const float* stats, void* dx, const ttt_strides* dxs, float* dweight, float* dbias,
                      void* workspace, size_t workspace_bytes, unsigned* status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* TTT_OPS_H_ */
