/*
 * gl_delta.h -- C ABI of the gated delta rule and of the query / key norms with
 * the position rotation (libglscan.so, beside gl_scan.h, whose status codes,
 * dtypes, ownership and error rules hold here too).
 *
 * The gated delta rule is the fast weight whose costate is its own: with the
 * token loss |S k_t - v_t|^2 / 2 the costate is S k_t - v_t, so the serial
 * learner of gl_scan.h needs no costates from outside.  Per sequence and value
 * head, S [dv][dk], S_0 given or zero:
 *
 *     e_t = v_t - a_t S_{t-1} k_t            a_t = exp(log_alpha_t)
 *     S_t = a_t S_{t-1} + beta_t e_t k_t^T
 *     y_t = scale S_t q_t                    read from the updated weight
 *
 * Layouts, last index contiguous; the first three may have any strides
 * (elements; an all-zero gl_strides_t means the dense order shown):
 *   q, k, dq, dk                    [B][Hk][T][dk]   io dtype
 *   v, y, dy, dv                    [B][H][T][dv]    io dtype
 *   log_alpha, beta and gradients   [B][H][T]        gate dtype
 *   states                          [n][H][dv][dk]   dense, fp64 if io is F64, else fp32
 * Pointers are 16-byte aligned; those of gates, and of q, k, v, y and their
 * gradients off the matrix-core paths, only to their elements (a forward that
 * saves nothing takes the other path by itself where they are not).
 * Value head h reads query and key head h / (H / Hk); dq and dk sum over the
 * value heads that share them.
 * state_out may be state_in itself, and dstate_in dstate_out (every path has read
 * what it writes over); no other output may overlap an input.
 *
 * Packed sequences: with n_seq > 0, B is 1, the T tokens hold n_seq sequences
 * one after another and cu_seqlens (device, int32, n_seq + 1 values, first 0,
 * last T, not decreasing) says where each begins.  States then number n_seq;
 * otherwise B.  A sequence may be empty: its state passes through.  Values out
 * of range are clamped to it, so that no call reads or writes outside its
 * tensors; where the sequences do not cover 0..T-1 once, what the outputs hold
 * at the other tokens is undefined.
 *
 * Numerical preconditions (not checked on the device): finite q, k, v, beta,
 * dy and states; log_alpha <= 0, minus infinity included (the state is
 * forgotten before that token is written).  With |k_t| <= 1 and 0 <= beta <= 1
 * every factor of the recurrence is a contraction; other keys are taken as
 * they are.  A value that is not finite reaches every token of its chunk of 64
 * and all later ones on the matrix-core paths (only later ones token by token).
 *
 * Arithmetic: F32 and F64 io compute in their own type.  BF16 io keeps the
 * states and every accumulator in fp32.  Its matrix-core path carries the
 * recurrences (states in both directions, e_t) through operands split into two
 * bf16 terms (16 significand bits): final states and the gradient of the first
 * hold 3.5e-6 (relative 2-norm).  dlog_alpha, before it is rounded to the gate
 * dtype, is a running sum where tokens keep more than 0.022 of the state: 1e-5 where
 * they keep nearly all, growing as 1 / alpha (uniform log_alpha -3, 4096 tokens:
 * 2e-3); a token that keeps less has the sum of what crosses it (1e-3, up to 6e-3 for
 * single heads).  y and dv are rounded once, at the end (1.7e-3).  dq and
 * dk come from products of two bf16 operands of which one (states, e_t, dv / beta)
 * was rounded once: 3.1e-3; dbeta takes e_t rounded once: 2.5e-3.
 *
 * Kernels: BF16 io with dk and dv multiples of 8, and F32 io with multiples of
 * 4, run in chunks of 64 tokens on the matrix cores.  Everything else goes token
 * by token on the vector ALU, and so do sequences of fewer than 4 tokens on
 * average (fewer than 24 in a forward that saves nothing): a long sequence packed
 * with very many short ones is faster in a call of its own.
 */
#ifndef GL_DELTA_H
#define GL_DELTA_H

#include "gl_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t b, h, t;  /* elements between batches, heads, tokens */
} gl_strides_t;

typedef struct {
  int64_t B, T;        /* batch and tokens; either may be 0 (no token)          */
  int64_t H, Hk;       /* value heads, query / key heads; H a multiple of Hk    */
  int64_t dk, dv;      /* 1..128 each                                           */
  int64_t n_seq;       /* packed sequences (B must be 1), 0 = B of T tokens     */
  int32_t io_dtype;    /* gl_dtype_t                                            */
  int32_t gate_dtype;  /* the io dtype, or F32 with BF16 io                     */
  uint32_t flags;      /* GL_FLAG_GENERIC: the token-serial vector kernels      */
  uint32_t segments;   /* BF16 matrix-core kernels: parts of a sequence that run
                          at once; 0 = chosen by the number of heads and chunks,
                          n = n (at most one per chunk), the same in a forward
                          and the backward of what it saved; elsewhere not used */
  double scale;        /* of y                                                  */
  gl_strides_t sq, sk, sv, sy, sg;      /* q, k, v, y, log_alpha and beta       */
  gl_strides_t sdq, sdk, sdv, sdy, sdg; /* their gradients (gl_delta_bwd)       */
} gl_delta_desc_t;

/* Bytes of `saved` (what gl_delta_fwd leaves for gl_delta_bwd; opaque) and of
 * the workspaces.  have_saved as in gl_scan_workspace_size: without it the
 * backward runs the forward again inside its own, larger workspace. */
gl_status_t gl_delta_saved_size(const gl_delta_desc_t* desc, size_t* saved_bytes);
gl_status_t gl_delta_workspace_size(const gl_delta_desc_t* desc, int have_saved,
                                    size_t* fwd_ws_bytes, size_t* bwd_ws_bytes);

/* Training forward and prefill.  state_in NULL = zero; state_out and saved may
 * be NULL; cu_seqlens is NULL unless n_seq > 0. */
gl_status_t gl_delta_fwd(const gl_delta_desc_t* desc, const void* q, const void* k, const void* v,
                         const void* log_alpha, const void* beta, const void* state_in,
                         const int32_t* cu_seqlens, void* y, void* state_out, void* saved,
                         void* ws, size_t ws_bytes, void* stream);

/* Gradients of L = sum <dy_t, y_t> + <dstate_out, S_T>.  `saved` is NULL or
 * what gl_delta_fwd left for the same inputs; dstate_out NULL = zero; dstate_in
 * may be NULL. */
gl_status_t gl_delta_bwd(const gl_delta_desc_t* desc, const void* q, const void* k, const void* v,
                         const void* log_alpha, const void* beta, const void* state_in,
                         const int32_t* cu_seqlens, const void* dy, const void* dstate_out,
                         const void* saved, void* dq, void* dk, void* dv, void* dlog_alpha,
                         void* dbeta, void* dstate_in, void* ws, size_t ws_bytes, void* stream);

/* Serving: one token of B sequences against a pool of n_slots states
 * [n_slots][H][dv][dk], updated in place.  Row b uses state slots[b] (device
 * int32; NULL = b, n_slots >= B); a slot outside 0..n_slots-1 marks a row with
 * nothing to do: its y is zero and no state changes.  No two rows may name one
 * slot.  desc->T is checked and not used (q, k are [B][Hk][dk], v, y [B][H][dv], gates
 * [B][H]; the t strides are not used), n_seq must be 0. */
gl_status_t gl_delta_step(const gl_delta_desc_t* desc, const void* q, const void* k, const void* v,
                          const void* log_alpha, const void* beta, const int32_t* slots,
                          int64_t n_slots, void* state, void* y, void* stream);

/* Name of the kernels chosen for desc ("delta-mfma-bf16-128x128",
 * "delta-serial-f32", ...), or NULL if desc is unsupported. */
const char* gl_delta_path_name(const gl_delta_desc_t* desc);

/* ---- Norms of queries and keys per head, and the position rotation, in one
 * pass over each:
 *
 *   n = x / sqrt(mean(x^2) + eps),  z = w * n,  out = scale Rot_p(z)
 *
 * for each row of d elements of q [B][Hq][T][d] and k [B][Hk][T][d] (strided as
 * above; all pointers here aligned to their elements, the workspace to 16
 * bytes), w = wq or wk [d] io dtype (NULL = ones), scale = q_scale or k_scale
 * (1 / sqrt(d) gives rows of unit length).  Rot_p turns the pairs (i, i + rot/2)
 * of the first rot columns ((2i, 2i + 1) with GL_FLAG_INTERLEAVED) by the angle
 * whose cosine and sine are cos[p][i], sin[p][i] (tables [n_pos][rot/2], fp32,
 * fp64 if io is F64); rot = 0: no rotation, the tables may be NULL.  p is
 * pos[b][t] (device int32 [B][T]), or pos0 + t if pos is NULL; p outside the
 * table is clamped into it.
 *
 * The backward reads x again (no saved tensor) and returns dq, dk and the sums
 * dwq, dwk [d] (fp32, fp64 if io is F64; NULL = not wanted), in a fixed order
 * of addition. */
#define GL_FLAG_INTERLEAVED 8u

typedef struct {
  int64_t B, T, Hq, Hk, d; /* Hq or Hk may be 0; d in 1..256                    */
  int64_t rot;             /* even, 0..d                                        */
  int64_t n_pos, pos0;
  int32_t io_dtype;
  uint32_t flags;          /* GL_FLAG_INTERLEAVED                               */
  double eps, q_scale, k_scale;
  gl_strides_t sq, sk, soq, sok;      /* q, k and what is made of them          */
  gl_strides_t sdoq, sdok, sdq, sdk;  /* gradients: given, returned             */
} gl_qknorm_desc_t;

gl_status_t gl_qknorm_rope_fwd(const gl_qknorm_desc_t* desc, const void* q, const void* k,
                               const void* wq, const void* wk, const void* cos, const void* sin,
                               const int32_t* pos, void* out_q, void* out_k, void* stream);
gl_status_t gl_qknorm_rope_workspace_size(const gl_qknorm_desc_t* desc, size_t* bwd_ws_bytes);
gl_status_t gl_qknorm_rope_bwd(const gl_qknorm_desc_t* desc, const void* q, const void* k,
                               const void* wq, const void* wk, const void* cos, const void* sin,
                               const int32_t* pos, const void* dout_q, const void* dout_k,
                               void* dq, void* dk, void* dwq, void* dwk, void* ws,
                               size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GL_DELTA_H */
