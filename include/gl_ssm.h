/*
 * gl_ssm.h -- C ABI of the selective state space scan, of the short causal
 * convolution before it, and of the norms before and after a block with its gate
 * and residual scale (libglscan.so, beside gl_scan.h, whose status codes, dtypes,
 * ownership and error rules hold here too).
 *
 * Rows are D (or d) channels, contiguous; tensors [B][T][D] (and [B][T][G][n])
 * may have any strides of their first dimensions (elements; an all-zero
 * gl_rows_t means the dense order shown).  io is the io dtype; par is fp64 if io
 * is F64, else fp32.  Pointers are aligned to their elements, workspaces and
 * saved states to 16 bytes; tensors whose rows begin on 16 bytes take the
 * faster kernels where there are two.  Unless said otherwise no output may
 * overlap an input or another output.  Sizes of which a launch would have 2^32
 * threads or more are not supported; a call says so before it writes anything.
 *
 * Packed sequences: with n_seq > 0, B is 1, the T tokens hold n_seq sequences
 * one after another and cu_seqlens (device, int32, n_seq + 1 values, first 0,
 * last T or less, not decreasing) says where each begins.  States then number
 * n_seq; otherwise B.  A sequence may be empty: its state passes through.  Tokens
 * behind the last sequence belong to none: whatever they hold adds nothing to any
 * sum, and all outputs and gradients are zero there.  Values out of range are
 * clamped to it, so that no call reads or writes outside its tensors; where a
 * table is not as said, what the outputs hold is undefined.
 */
#ifndef GL_SSM_H
#define GL_SSM_H

#include "gl_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t b, t, g;  /* elements between batches, tokens, groups */
} gl_rows_t;

/* ---- Short causal convolution, per channel d:
 *
 *   p_t = bias[d] + sum_j w[d][j] x_(t - K + 1 + j)[d],   y_t = p_t
 *
 * or y_t = p_t / (1 + e^-p_t) with GL_FLAG_SILU.  Before a sequence's first token
 * x is its state, the last K - 1 inputs before it (oldest first), or zero.
 *   x, y, dy, dx        [B][T][D]       io
 *   w, bias             [D][K], [D]     io, dense (bias NULL = zero)
 *   states              [n][K-1][D]     io, dense
 *   dw, dbias           [D][K], [D]     par (sums over the tokens in a fixed order)
 */
#define GL_FLAG_SILU 16u

typedef struct {
  int64_t B, T, D, K;  /* K in 1..8 */
  int64_t n_seq;
  int32_t io_dtype;
  uint32_t flags;      /* GL_FLAG_SILU */
  gl_rows_t sx, sy, sdy, sdx;
} gl_conv_desc_t;

/* state_in NULL = zero; state_out (the last K - 1 inputs) may be NULL. */
gl_status_t gl_conv_fwd(const gl_conv_desc_t* desc, const void* x, const void* w, const void* bias,
                        const void* state_in, const int32_t* cu_seqlens, void* y, void* state_out, void* stream);

/* Gradients of L = sum <dy_t, y_t> + <dstate_out, state_out>; dstate_out NULL =
 * zero; dw, dbias, dstate_in NULL = not wanted. */
gl_status_t gl_conv_workspace_size(const gl_conv_desc_t* desc, size_t* bwd_ws_bytes);
gl_status_t gl_conv_bwd(const gl_conv_desc_t* desc, const void* x, const void* w, const void* bias,
                        const void* state_in, const int32_t* cu_seqlens, const void* dy, const void* dstate_out,
                        void* dx, void* dw, void* dbias, void* dstate_in, void* ws, size_t ws_bytes, void* stream);

/* One token of B sequences, x, y [B][D] (row strides sx.b, sy.b), against a pool
 * of n_slots states, moved on by one input in place.  Row b uses state slots[b]
 * (device int32; NULL = b, n_slots >= B); a slot outside 0..n_slots-1 marks a
 * row with nothing to do: its y is zero and no state changes.  No two rows may
 * name one slot.  desc->T is not used (any T >= 0), n_seq must be 0. */
gl_status_t gl_conv_step(const gl_conv_desc_t* desc, const void* x, const void* w, const void* bias,
                         const int32_t* slots, int64_t n_slots, void* state, void* y, void* stream);

/* ---- Selective scan, per channel d and state n of N; channel d reads B and C of
 * group d / (D / G):
 *
 *   D_t = dt_t + dt_bias, or log(1 + e^that) with GL_FLAG_SOFTPLUS
 *   h_t = exp(D_t A[d][n]) h_(t-1) + D_t x_t B_t[n],   h_0 given or zero
 *   y_t = (sum_n C_t[n] h_t + skip[d] x_t) (z_t / (1 + e^-z_t), if z is given)
 *
 *   x, dt, z, y and gradients    [B][T][D]      io (tokens less than 2^19 elements apart)
 *   B, C and gradients           [B][T][G][N]   io
 *   A, dA                        [D][N]         par, dense
 *   skip, dt_bias and gradients  [D]            par (NULL = zero)
 *   states                       [n][D][N]      par, dense
 *
 * Numerical preconditions (not checked on the device): finite inputs, D_t >= 0
 * and A <= 0 (every factor is then a contraction; a state that grows is computed
 * as long as its growth over 1024 tokens stays within the type); with
 * GL_FLAG_SOFTPLUS dt_t may be -infinity: the token then passes by.  A value that is
 * not finite reaches its own channel's later tokens only, in a backward also the
 * earlier ones and the sums over channels and tokens that it is part of.
 *
 * Arithmetic: fp32 (fp64 if io is F64) throughout, outputs rounded once.
 * state_out may be state_in itself, and dstate_in dstate_out. */
#define GL_FLAG_SOFTPLUS 32u

typedef struct {
  int64_t B, T, D, N, G;  /* N in 1..256, D a multiple of G */
  int64_t n_seq;
  int32_t io_dtype;
  uint32_t flags;         /* GL_FLAG_SOFTPLUS */
  gl_rows_t sx, sdt, sz, sB, sC, sy;
  gl_rows_t sdy, sdx, sddt, sdz, sdB, sdC;
} gl_ssm_desc_t;

/* Bytes of `saved` (what gl_ssm_fwd leaves for gl_ssm_bwd; opaque) and of the
 * workspaces (the forward's is empty).  Without `saved` the backward runs the forward
 * again inside its own workspace, larger by what `saved` takes.  With it the backward's
 * holds the parts of dB and dC, 2 N par values for every token and block of c channels of
 * a group (B T G ceil(D / G / c) of them, an odd N counted as N + 1), and N + 2 for every
 * sequence and channel.  c is 8, 16 or 32, by the work-groups that there are; while the parts
 * are more than 2^30 bytes it is doubled, but to no more than 32 where N <= 64, 16 where
 * N <= 128, else 8 (half these N in fp64).  So the workspace can be many times the tensors
 * (N = 256: 128 times a bf16 x); a batch may be given in pieces, and a sequence in pieces
 * that hand their states on. */
gl_status_t gl_ssm_saved_size(const gl_ssm_desc_t* desc, size_t* saved_bytes);
gl_status_t gl_ssm_workspace_size(const gl_ssm_desc_t* desc, int have_saved, size_t* fwd_ws_bytes,
                                  size_t* bwd_ws_bytes);
gl_status_t gl_ssm_fwd(const gl_ssm_desc_t* desc, const void* x, const void* dt, const void* A, const void* B,
                       const void* C, const void* skip, const void* z, const void* dt_bias, const void* state_in,
                       const int32_t* cu_seqlens, void* y, void* state_out, void* saved, void* ws, size_t ws_bytes,
                       void* stream);

/* Gradients of L = sum <dy_t, y_t> + <dstate_out, h_T>.  dz is written if z is
 * given; dskip, ddt_bias and dstate_in may be NULL. */
gl_status_t gl_ssm_bwd(const gl_ssm_desc_t* desc, const void* x, const void* dt, const void* A, const void* B,
                       const void* C, const void* skip, const void* z, const void* dt_bias, const void* state_in,
                       const int32_t* cu_seqlens, const void* dy, const void* dstate_out, const void* saved,
                       void* dx, void* ddt, void* dA, void* dB, void* dC, void* dskip, void* dz, void* ddt_bias,
                       void* dstate_in, void* ws, size_t ws_bytes, void* stream);

/* One token of B sequences, x, dt, z, y [B][D], B, C [B][G][N] (strides b and g),
 * against a pool of n_slots states updated in place; slots, T and n_seq as in
 * gl_conv_step.  Dense rows (all-zero strides) are of less than 2^19 channels. */
gl_status_t gl_ssm_step(const gl_ssm_desc_t* desc, const void* x, const void* dt, const void* A, const void* B,
                        const void* C, const void* skip, const void* z, const void* dt_bias, const int32_t* slots,
                        int64_t n_slots, void* state, void* y, void* stream);

/* ---- Between two blocks: what a block gives is normed (if wx is given), scaled and
 * added to the residual, and the sum is normed for the next block.  Per row of d:
 *
 *   u = wx * x / rms(x)  (wx NULL: u = x),   r_out = r + scale * u,
 *   n = w * r_out / rms(r_out),              rms(v) = sqrt(mean(v^2) + eps)
 *
 * (in both norms; the squares are summed in fp32, fp64 if io is F64 or rows are of fewer
 * than 8, and have to stay within it: elements up to 1e17 in fp32).
 *
 *   x, n, dn, dx            [B][T][d]  io
 *   r, r_out, dr_out, dr    [B][T][d]  res: the io dtype, or F32 with BF16 io
 *   w, wx, scale            [d]        io (scale NULL = ones)
 *   dw, dwx, dscale         [d]        par (sums over the rows in a fixed order)
 * n is made of r_out before that is rounded.  r_out may be r itself.
 * The backward reads x and r again (no saved tensor); dr_out NULL = zero; dw, dwx
 * and dscale may be NULL. */
typedef struct {
  int64_t B, T, d;  /* d in 1..16384 */
  int32_t io_dtype, res_dtype;
  uint32_t flags, reserved;  /* 0 */
  double eps;
  gl_rows_t sx, sr, sn, sro;
  gl_rows_t sdn, sdro, sdx, sdr;
} gl_addnorm_desc_t;

gl_status_t gl_addnorm_fwd(const gl_addnorm_desc_t* desc, const void* x, const void* r, const void* w, const void* wx,
                           const void* scale, void* n, void* r_out, void* stream);
gl_status_t gl_addnorm_workspace_size(const gl_addnorm_desc_t* desc, size_t* bwd_ws_bytes);
gl_status_t gl_addnorm_bwd(const gl_addnorm_desc_t* desc, const void* x, const void* r, const void* w, const void* wx,
                           const void* scale, const void* dn, const void* dr_out, void* dx, void* dr, void* dw,
                           void* dwx, void* dscale, void* ws, size_t ws_bytes, void* stream);

/* ---- After a block's heads: every row of d is normed and gated,
 *
 *   y = w * x / rms(x) * silu(z),    or with GL_FLAG_GATE_FIRST
 *   y = w * v / rms(v),  v = x * silu(z);        silu(z) = z / (1 + e^-z), z NULL: 1
 *
 *   x, z, y and gradients   [B][T][G][d]   io
 *   w                       [d], or [G][d] with GL_FLAG_GROUP_WEIGHTS   io (NULL = ones)
 *   dw                      as w           par (NULL = not wanted) */
#define GL_FLAG_GATE_FIRST 64u
#define GL_FLAG_GROUP_WEIGHTS 128u

typedef struct {
  int64_t B, T, G, d;  /* d in 1..16384 */
  int32_t io_dtype;
  uint32_t flags;
  double eps;
  gl_rows_t sx, sz, sy;
  gl_rows_t sdy, sdx, sdz;
} gl_gatenorm_desc_t;

gl_status_t gl_gatenorm_fwd(const gl_gatenorm_desc_t* desc, const void* x, const void* z, const void* w, void* y,
                            void* stream);
gl_status_t gl_gatenorm_workspace_size(const gl_gatenorm_desc_t* desc, size_t* bwd_ws_bytes);
gl_status_t gl_gatenorm_bwd(const gl_gatenorm_desc_t* desc, const void* x, const void* z, const void* w,
                            const void* dy, void* dx, void* dz, void* dw, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GL_SSM_H */
