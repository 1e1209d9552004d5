// gl_ssm.cpp -- host side of include/gl_ssm.h: argument checks, workspace layout and
// launches.  Every check runs before the first launch; nothing here allocates
// device memory.
#include "gl_ssm.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "ssm.hpp"

namespace {

gl_status_t fail(gl_status_t st, const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  gls::set_last_error(text);
  return st;
}

gl_status_t hip_status(hipError_t e, const char* where) {
  if (e == hipErrorInvalidConfiguration) return fail(GL_ERROR_NOT_SUPPORTED, "%s: sizes above the launch limits", where);
  return e == hipSuccess ? GL_SUCCESS : fail(GL_ERROR_HIP, "%s: %s", where, hipGetErrorString(e));
}

constexpr size_t kAlign = 256;
size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
size_t elem_of(int io) { return io == GL_DTYPE_F64 ? 8 : io == GL_DTYPE_F32 ? 4 : 2; }
size_t par_of(int io) { return io == GL_DTYPE_F64 ? 8 : 4; }

// Pointers that a call reads or writes (`need`: not NULL) or may (else).
gl_status_t check_ptrs(bool need, std::initializer_list<const void*> ps, size_t align) {
  for (const void* p : ps) {
    if (!p && need) return fail(GL_ERROR_INVALID_VALUE, "NULL input or output pointer");
    if (reinterpret_cast<uintptr_t>(p) % align)
      return fail(GL_ERROR_MISALIGNED, "pointer %p not %zu-byte aligned", p, align);
  }
  return GL_SUCCESS;
}

gl_status_t check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return GL_SUCCESS;
  if (!ws) return fail(GL_ERROR_INVALID_VALUE, "workspace is NULL (%zu bytes needed)", need);
  if (reinterpret_cast<uintptr_t>(ws) & 15) return fail(GL_ERROR_MISALIGNED, "workspace not 16-byte aligned");
  if (have < need) return fail(GL_ERROR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", have, need);
  return GL_SUCCESS;
}

gl_status_t check_io(int io) {
  return io < GL_DTYPE_F64 || io > GL_DTYPE_BF16 ? fail(GL_ERROR_INVALID_VALUE, "unknown io_dtype %d", io) : GL_SUCCESS;
}
gl_status_t check_strides(std::initializer_list<gl_rows_t> ss) {
  for (const gl_rows_t& s : ss)
    if (s.b < 0 || s.t < 0 || s.g < 0) return fail(GL_ERROR_INVALID_VALUE, "negative stride");
  return GL_SUCCESS;
}
gl_status_t check_seqs(int64_t n_seq, int64_t B, int64_t T) {
  if (n_seq < 0) return fail(GL_ERROR_INVALID_VALUE, "negative n_seq");
  if (n_seq > 0 && B != 1) return fail(GL_ERROR_INVALID_VALUE, "packed sequences need B = 1");
  if (n_seq > 0 && T > 0x7fffffffLL) return fail(GL_ERROR_NOT_SUPPORTED, "packed T above 2^31-1");
  return GL_SUCCESS;
}
gl_status_t check_cu(int64_t n_seq, const int32_t* cu) {
  if (n_seq > 0 && !cu) return fail(GL_ERROR_INVALID_VALUE, "n_seq > 0 needs cu_seqlens");
  if (n_seq == 0 && cu) return fail(GL_ERROR_INVALID_VALUE, "cu_seqlens needs n_seq > 0");
  if (reinterpret_cast<uintptr_t>(cu) & 3) return fail(GL_ERROR_MISALIGNED, "cu_seqlens not 4-byte aligned");
  return GL_SUCCESS;
}
gl_status_t check_slots(int64_t B, const int32_t* slots, int64_t n_slots, const void* state, size_t align) {
  if (n_slots < 0) return fail(GL_ERROR_INVALID_VALUE, "n_slots is negative");
  if (!slots && n_slots < B)
    return fail(GL_ERROR_INVALID_VALUE, "%lld states for %lld rows", (long long)n_slots, (long long)B);
  if (reinterpret_cast<uintptr_t>(slots) & 3) return fail(GL_ERROR_MISALIGNED, "slots not 4-byte aligned");
  return check_ptrs(n_slots > 0, {state}, align);
}
// Products of sizes that index threads, work-groups or bytes stay far inside 64 and 31 bits.
gl_status_t check_sizes(std::initializer_list<int64_t> ns, double most) {
  double n = 1;
  for (int64_t v : ns) n *= std::max<double>(1.0, static_cast<double>(v));
  return n > most ? fail(GL_ERROR_NOT_SUPPORTED, "sizes above the launch limits") : GL_SUCCESS;
}

gls::Rows rows(const gl_rows_t& s, int64_t T, int64_t G, int64_t d) {
  if (s.b == 0 && s.t == 0 && s.g == 0) return {T * G * d, G * d, d};
  return {s.b, s.t, s.g};
}

constexpr int64_t kMaxTokenStride = int64_t(1) << 19;

struct Cut {  // runs of a workspace
  char* at;
  void* take(size_t bytes) {
    void* p = at;
    at += round_up(bytes);
    return p;
  }
};

#define TRY(call)                                \
  do {                                           \
    const gl_status_t st_ = (call);              \
    if (st_ != GL_SUCCESS) return st_;           \
  } while (0)

// ------------------------------------------------------------ convolution
// (A step is one token of each row, whatever T its descriptor holds.)
gl_status_t check_conv(const gl_conv_desc_t* d, bool step = false) {
  if (!d) return fail(GL_ERROR_INVALID_VALUE, "desc is NULL");
  if (d->B < 0 || d->T < 0 || d->D < 0) return fail(GL_ERROR_INVALID_VALUE, "negative B, T or D");
  if (d->K < 1) return fail(GL_ERROR_INVALID_VALUE, "K must be >= 1");
  TRY(check_io(d->io_dtype));
  if (d->flags & ~GL_FLAG_SILU) return fail(GL_ERROR_INVALID_VALUE, "unknown flags");
  TRY(check_seqs(d->n_seq, d->B, d->T));
  TRY(check_strides({d->sx, d->sy, d->sdy, d->sdx}));
  if (d->K > 8) return fail(GL_ERROR_NOT_SUPPORTED, "K above 8");
  if (d->D > (1 << 24)) return fail(GL_ERROR_NOT_SUPPORTED, "D above 2^24");
  const int64_t n = d->n_seq ? d->n_seq : d->B;
  TRY(check_sizes({d->B, step ? 1 : d->T, d->D}, 5e11));
  return check_sizes({n, d->D, 8}, 2e11);
}

gls::ConvArgs conv_args(const gl_conv_desc_t* d) {
  gls::ConvArgs a;
  a.n_seq = d->n_seq;
  a.N = d->n_seq ? d->n_seq : d->B;
  a.B = d->B; a.T = d->T;
  a.D = static_cast<int>(d->D); a.K = static_cast<int>(d->K);
  a.silu = (d->flags & GL_FLAG_SILU) != 0;
  a.sx = rows(d->sx, d->T, 1, d->D);
  a.sy = rows(d->sy, d->T, 1, d->D);
  a.sdy = rows(d->sdy, d->T, 1, d->D);
  a.sdx = rows(d->sdx, d->T, 1, d->D);
  return a;
}

// ------------------------------------------------------------ selective scan
struct SsmPlan {
  size_t par = 4, elem = 2, saved = 0, bc = 0, bwd_ws = 0;  // bwd_ws: with `saved` given
};

gl_status_t check_ssm(const gl_ssm_desc_t* d, bool step = false) {
  if (!d) return fail(GL_ERROR_INVALID_VALUE, "desc is NULL");
  if (d->B < 0 || d->T < 0 || d->D < 0) return fail(GL_ERROR_INVALID_VALUE, "negative B, T or D");
  if (d->N < 1) return fail(GL_ERROR_INVALID_VALUE, "N must be >= 1");
  if (d->G < 1 || d->D % d->G)
    return fail(GL_ERROR_INVALID_VALUE, "D must be a multiple of G >= 1 (%lld, %lld)", (long long)d->D, (long long)d->G);
  TRY(check_io(d->io_dtype));
  if (d->flags & ~GL_FLAG_SOFTPLUS) return fail(GL_ERROR_INVALID_VALUE, "unknown flags");
  TRY(check_seqs(d->n_seq, d->B, d->T));
  TRY(check_strides({d->sx, d->sdt, d->sz, d->sB, d->sC, d->sy, d->sdy, d->sdx, d->sddt, d->sdz, d->sdB, d->sdC}));
  if (d->N > 256) return fail(GL_ERROR_NOT_SUPPORTED, "N above 256");
  if (d->D > (1 << 24)) return fail(GL_ERROR_NOT_SUPPORTED, "D above 2^24");
  // the kernels keep a lane's place in a tile of 1024 tokens as 32 bits
  for (const gl_rows_t& s : {d->sx, d->sdt, d->sz, d->sy, d->sdy, d->sdx, d->sddt, d->sdz})
    if (rows(s, 1, 1, d->D).t >= kMaxTokenStride)
      return fail(GL_ERROR_NOT_SUPPORTED, "a token stride above %lld elements", (long long)kMaxTokenStride - 1);
  const int64_t n = d->n_seq ? d->n_seq : d->B, T = step ? 1 : d->T;
  TRY(check_sizes({n, d->D, 16}, 2e9));  // work-groups, lanes of a step / 256
  TRY(check_sizes({d->B, T, d->G, d->N}, 2e11));
  return check_sizes({d->B, T, d->D, d->N}, 1e15);
}

gls::SsmArgs ssm_args(const gl_ssm_desc_t* d) {
  gls::SsmArgs a;
  a.packed = d->n_seq > 0;
  a.N = a.packed ? d->n_seq : d->B;
  a.B = d->B; a.T = d->T;
  a.D = static_cast<int>(d->D); a.Ns = static_cast<int>(d->N); a.G = static_cast<int>(d->G);
  a.softplus = (d->flags & GL_FLAG_SOFTPLUS) != 0;
  const auto x = [&](const gl_rows_t& s) { return rows(s, d->T, 1, d->D); };
  const auto bc = [&](const gl_rows_t& s) { return rows(s, d->T, d->G, d->N); };
  a.sx = x(d->sx); a.sdt = x(d->sdt); a.sz = x(d->sz); a.sy = x(d->sy);
  a.sdy = x(d->sdy); a.sdx = x(d->sdx); a.sddt = x(d->sddt); a.sdz = x(d->sdz);
  a.sB = bc(d->sB); a.sC = bc(d->sC); a.sdB = bc(d->sdB); a.sdC = bc(d->sdC);
  return a;
}

gl_status_t plan_ssm(const gl_ssm_desc_t* d, SsmPlan* p) {
  TRY(check_ssm(d));
  p->par = par_of(d->io_dtype);
  p->elem = elem_of(d->io_dtype);
  const gls::SsmArgs a = ssm_args(d);
  p->saved = round_up(static_cast<size_t>(gls::chunk_slots(a.packed, a.N, a.T, gls::ssm_ck(d->io_dtype, a))) * a.D *
                      a.Ns * p->par);
  p->bc = round_up(gls::ssm_bc_bytes(d->io_dtype, a));
  p->bwd_ws = p->bc + round_up(static_cast<size_t>(a.N) * (a.Ns + 2) * a.D * p->par);
  return GL_SUCCESS;
}

gl_status_t check_ssm_inputs(const SsmPlan& p, bool tokens, const void* x, const void* dt, const void* A, const void* B,
                             const void* C, const void* skip, const void* z, const void* dt_bias) {
  TRY(check_ptrs(tokens, {x, dt, B, C}, p.elem));
  TRY(check_ptrs(false, {z}, p.elem));
  TRY(check_ptrs(true, {A}, p.par));
  return check_ptrs(false, {skip, dt_bias}, p.par);
}

// ------------------------------------------------------------ norms
gl_status_t check_norm(int64_t B, int64_t T, int64_t G, int64_t d, int io, double eps) {
  if (B < 0 || T < 0 || G < 0) return fail(GL_ERROR_INVALID_VALUE, "negative B, T or G");
  if (d < 1) return fail(GL_ERROR_INVALID_VALUE, "d must be >= 1");
  TRY(check_io(io));
  if (!(eps >= 0) || !std::isfinite(eps)) return fail(GL_ERROR_INVALID_VALUE, "eps must be finite and >= 0");
  if (d > 16384) return fail(GL_ERROR_NOT_SUPPORTED, "d above 16384");
  if (G > 65535) return fail(GL_ERROR_NOT_SUPPORTED, "G above 65535");
  return check_sizes({B, T, G}, 2e9);
}
gl_status_t check_addnorm(const gl_addnorm_desc_t* d) {
  if (!d) return fail(GL_ERROR_INVALID_VALUE, "desc is NULL");
  TRY(check_norm(d->B, d->T, 1, d->d, d->io_dtype, d->eps));
  if (d->res_dtype != d->io_dtype && !(d->res_dtype == GL_DTYPE_F32 && d->io_dtype == GL_DTYPE_BF16))
    return fail(GL_ERROR_INVALID_VALUE, "res_dtype must be io_dtype, or F32 with BF16 io");
  if (d->flags || d->reserved) return fail(GL_ERROR_INVALID_VALUE, "unknown flags");
  return check_strides({d->sx, d->sr, d->sn, d->sro, d->sdn, d->sdro, d->sdx, d->sdr});
}
gl_status_t check_gatenorm(const gl_gatenorm_desc_t* d) {
  if (!d) return fail(GL_ERROR_INVALID_VALUE, "desc is NULL");
  TRY(check_norm(d->B, d->T, d->G, d->d, d->io_dtype, d->eps));
  if (d->flags & ~(GL_FLAG_GATE_FIRST | GL_FLAG_GROUP_WEIGHTS)) return fail(GL_ERROR_INVALID_VALUE, "unknown flags");
  return check_strides({d->sx, d->sz, d->sy, d->sdy, d->sdx, d->sdz});
}
gls::AddNormArgs addnorm_args(const gl_addnorm_desc_t* d) {
  gls::AddNormArgs a;
  a.B = d->B; a.T = d->T; a.d = static_cast<int>(d->d);
  a.res_f32 = d->res_dtype != d->io_dtype;
  a.eps = d->eps;
  const auto x = [&](const gl_rows_t& s) { return rows(s, d->T, 1, d->d); };
  a.sx = x(d->sx); a.sr = x(d->sr); a.sn = x(d->sn); a.sro = x(d->sro);
  a.sdn = x(d->sdn); a.sdro = x(d->sdro); a.sdx = x(d->sdx); a.sdr = x(d->sdr);
  return a;
}
gls::GateNormArgs gatenorm_args(const gl_gatenorm_desc_t* d) {
  gls::GateNormArgs a;
  a.B = d->B; a.T = d->T; a.G = static_cast<int>(d->G); a.d = static_cast<int>(d->d);
  a.first = (d->flags & GL_FLAG_GATE_FIRST) != 0;
  a.group_w = (d->flags & GL_FLAG_GROUP_WEIGHTS) != 0;
  a.eps = d->eps;
  const auto x = [&](const gl_rows_t& s) { return rows(s, d->T, d->G, d->d); };
  a.sx = x(d->sx); a.sz = x(d->sz); a.sy = x(d->sy);
  a.sdy = x(d->sdy); a.sdx = x(d->sdx); a.sdz = x(d->sdz);
  return a;
}

}  // namespace

extern "C" {

gl_status_t gl_conv_fwd(const gl_conv_desc_t* desc, const void* x, const void* w, const void* bias,
                        const void* state_in, const int32_t* cu_seqlens, void* y, void* state_out, void* stream) {
  TRY(check_conv(desc));
  gls::ConvArgs a = conv_args(desc);
  if (a.N * a.D == 0) return GL_SUCCESS;
  TRY(check_cu(desc->n_seq, cu_seqlens));
  const size_t e = elem_of(desc->io_dtype);
  TRY(check_ptrs(a.B * a.T > 0, {x, y}, e));
  TRY(check_ptrs(true, {w}, e));
  TRY(check_ptrs(false, {bias, state_in, state_out}, e));
  a.x = x; a.w = w; a.bias = bias; a.state_in = state_in; a.cu = cu_seqlens; a.y = y;
  a.state_out = a.K > 1 ? state_out : nullptr;
  return hip_status(gls::launch_conv_fwd(desc->io_dtype, a, static_cast<hipStream_t>(stream)), "convolution launch");
}

gl_status_t gl_conv_workspace_size(const gl_conv_desc_t* desc, size_t* bwd_ws_bytes) {
  TRY(check_conv(desc));
  if (!bwd_ws_bytes) return fail(GL_ERROR_INVALID_VALUE, "bwd_ws_bytes is NULL");
  *bwd_ws_bytes = round_up(gls::conv_bwd_ws(desc->io_dtype, conv_args(desc)));
  return GL_SUCCESS;
}

gl_status_t gl_conv_bwd(const gl_conv_desc_t* desc, const void* x, const void* w, const void* bias,
                        const void* state_in, const int32_t* cu_seqlens, const void* dy, const void* dstate_out,
                        void* dx, void* dw, void* dbias, void* dstate_in, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_conv(desc));
  gls::ConvArgs a = conv_args(desc);
  if (a.D == 0) return GL_SUCCESS;
  if (a.N > 0) TRY(check_cu(desc->n_seq, cu_seqlens));
  const size_t e = elem_of(desc->io_dtype), p = par_of(desc->io_dtype);
  TRY(check_ptrs(a.B * a.T > 0, {x, dy, dx}, e));
  TRY(check_ptrs(true, {w}, e));
  TRY(check_ptrs(false, {bias, state_in, dstate_out, dstate_in}, e));
  TRY(check_ptrs(false, {dw, dbias}, p));
  if (dw || dbias) TRY(check_ws(ws, ws_bytes, round_up(gls::conv_bwd_ws(desc->io_dtype, a))));
  a.x = x; a.w = w; a.bias = bias; a.state_in = state_in; a.cu = cu_seqlens; a.dy = dy; a.dstate_out = dstate_out;
  a.dx = dx; a.dw = dw; a.dbias = dbias; a.dstate_in = dstate_in;
  a.part = dw || dbias ? ws : nullptr;
  return hip_status(gls::launch_conv_bwd(desc->io_dtype, a, static_cast<hipStream_t>(stream)),
                    "convolution backward launch");
}

gl_status_t gl_conv_step(const gl_conv_desc_t* desc, const void* x, const void* w, const void* bias,
                         const int32_t* slots, int64_t n_slots, void* state, void* y, void* stream) {
  TRY(check_conv(desc, true));
  if (desc->n_seq) return fail(GL_ERROR_INVALID_VALUE, "a step takes no packed sequences");
  gl_conv_desc_t one = *desc;
  one.T = 1;
  gls::ConvArgs a = conv_args(&one);
  if (a.B * a.D == 0) {
    return n_slots < 0 ? fail(GL_ERROR_INVALID_VALUE, "n_slots is negative") : GL_SUCCESS;
  }
  const size_t e = elem_of(desc->io_dtype);
  TRY(check_slots(a.B, slots, n_slots, a.K > 1 ? state : x, e));
  TRY(check_ptrs(true, {x, w, y}, e));
  TRY(check_ptrs(false, {bias}, e));
  a.x = x; a.w = w; a.bias = bias; a.slots = slots; a.n_slots = n_slots; a.state_out = state; a.y = y;
  return hip_status(gls::launch_conv_step(desc->io_dtype, a, static_cast<hipStream_t>(stream)),
                    "convolution step launch");
}

gl_status_t gl_ssm_saved_size(const gl_ssm_desc_t* desc, size_t* saved_bytes) {
  SsmPlan p;
  TRY(plan_ssm(desc, &p));
  if (!saved_bytes) return fail(GL_ERROR_INVALID_VALUE, "saved_bytes is NULL");
  *saved_bytes = p.saved;
  return GL_SUCCESS;
}

gl_status_t gl_ssm_workspace_size(const gl_ssm_desc_t* desc, int have_saved, size_t* fwd_ws_bytes,
                                  size_t* bwd_ws_bytes) {
  SsmPlan p;
  TRY(plan_ssm(desc, &p));
  if (!fwd_ws_bytes || !bwd_ws_bytes) return fail(GL_ERROR_INVALID_VALUE, "size pointer is NULL");
  *fwd_ws_bytes = 0;
  *bwd_ws_bytes = p.bwd_ws + (have_saved ? 0 : p.saved);
  return GL_SUCCESS;
}

gl_status_t gl_ssm_fwd(const gl_ssm_desc_t* desc, const void* x, const void* dt, const void* A, const void* B,
                       const void* C, const void* skip, const void* z, const void* dt_bias, const void* state_in,
                       const int32_t* cu_seqlens, void* y, void* state_out, void* saved, void* ws, size_t ws_bytes,
                       void* stream) {
  SsmPlan p;
  TRY(plan_ssm(desc, &p));
  gls::SsmArgs a = ssm_args(desc);
  if (a.N * a.D == 0) return GL_SUCCESS;
  const bool tokens = a.B * a.T > 0;
  TRY(check_cu(desc->n_seq, cu_seqlens));
  TRY(check_ssm_inputs(p, tokens, x, dt, A, B, C, skip, z, dt_bias));
  TRY(check_ptrs(tokens, {y}, p.elem));
  TRY(check_ptrs(false, {state_in, state_out}, p.par));
  TRY(check_ptrs(false, {saved}, 16));
  TRY(check_ws(ws, ws_bytes, 0));
  a.x = x; a.dt = dt; a.A = A; a.Bm = B; a.Cm = C; a.skip = skip; a.z = z; a.bias = dt_bias;
  a.state_in = state_in; a.cu = cu_seqlens; a.y = y; a.state_out = state_out; a.ckpt = saved;
  return hip_status(gls::launch_ssm_fwd(desc->io_dtype, a, static_cast<hipStream_t>(stream)), "selective scan launch");
}

gl_status_t gl_ssm_bwd(const gl_ssm_desc_t* desc, const void* x, const void* dt, const void* A, const void* B,
                       const void* C, const void* skip, const void* z, const void* dt_bias, const void* state_in,
                       const int32_t* cu_seqlens, const void* dy, const void* dstate_out, const void* saved,
                       void* dx, void* ddt, void* dA, void* dB, void* dC, void* dskip, void* dz, void* ddt_bias,
                       void* dstate_in, void* ws, size_t ws_bytes, void* stream) {
  SsmPlan p;
  TRY(plan_ssm(desc, &p));
  gls::SsmArgs a = ssm_args(desc);
  if (a.D == 0 && a.B * a.T == 0) return GL_SUCCESS;
  const bool tokens = a.B * a.T > 0;
  if (a.N > 0) TRY(check_cu(desc->n_seq, cu_seqlens));
  if (a.D > 0) TRY(check_ssm_inputs(p, tokens, x, dt, A, B, C, skip, z, dt_bias));
  TRY(check_ptrs(tokens && a.D > 0, {dy, dx, ddt}, p.elem));
  TRY(check_ptrs(tokens, {dB, dC}, p.elem));
  TRY(check_ptrs(tokens && a.D > 0 && z, {dz}, p.elem));
  TRY(check_ptrs(a.D > 0, {dA}, p.par));
  TRY(check_ptrs(false, {dskip, ddt_bias, state_in, dstate_out, dstate_in}, p.par));
  TRY(check_ptrs(false, {saved}, 16));
  TRY(check_ws(ws, ws_bytes, p.bwd_ws + (saved ? 0 : p.saved)));
  a.x = x; a.dt = dt; a.A = A; a.Bm = B; a.Cm = C; a.skip = skip; a.z = z; a.bias = dt_bias;
  a.state_in = state_in; a.cu = cu_seqlens; a.dy = dy; a.dstate_out = dstate_out;
  a.dx = dx; a.ddt = ddt; a.dA = dA; a.dB = dB; a.dC = dC; a.dskip = dskip; a.dz = dz; a.dbias = ddt_bias;
  a.dstate_in = dstate_in;
  Cut w{static_cast<char*>(ws)};
  a.part_bc = w.take(p.bc);
  a.part_par = w.take(static_cast<size_t>(a.N) * (a.Ns + 2) * a.D * p.par);
  a.ckpt = const_cast<void*>(saved);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (!gls::ssm_bwd_fits(desc->io_dtype, a))  // before the forward below is launched
    return hip_status(hipErrorInvalidConfiguration, "selective scan backward launch");
  if (!saved && p.saved) {
    a.ckpt = w.take(p.saved);
    // a.y and a.state_out NULL: the states before the tiles only
    TRY(hip_status(gls::launch_ssm_fwd(desc->io_dtype, a, s), "selective scan states launch"));
  }
  return hip_status(gls::launch_ssm_bwd(desc->io_dtype, a, s), "selective scan backward launch");
}

gl_status_t gl_ssm_step(const gl_ssm_desc_t* desc, const void* x, const void* dt, const void* A, const void* B,
                        const void* C, const void* skip, const void* z, const void* dt_bias, const int32_t* slots,
                        int64_t n_slots, void* state, void* y, void* stream) {
  TRY(check_ssm(desc, true));
  if (desc->n_seq) return fail(GL_ERROR_INVALID_VALUE, "a step takes no packed sequences");
  const SsmPlan p{par_of(desc->io_dtype), elem_of(desc->io_dtype)};
  gl_ssm_desc_t one = *desc;
  one.T = 1;
  gls::SsmArgs a = ssm_args(&one);
  if (a.B * a.D == 0) {
    return n_slots < 0 ? fail(GL_ERROR_INVALID_VALUE, "n_slots is negative") : GL_SUCCESS;
  }
  TRY(check_slots(a.B, slots, n_slots, state, p.par));
  TRY(check_ssm_inputs(p, true, x, dt, A, B, C, skip, z, dt_bias));
  TRY(check_ptrs(true, {y}, p.elem));
  a.x = x; a.dt = dt; a.A = A; a.Bm = B; a.Cm = C; a.skip = skip; a.z = z; a.bias = dt_bias;
  a.slots = slots; a.n_slots = n_slots; a.state_out = state; a.y = y;
  return hip_status(gls::launch_ssm_step(desc->io_dtype, a, static_cast<hipStream_t>(stream)),
                    "selective scan step launch");
}

gl_status_t gl_addnorm_fwd(const gl_addnorm_desc_t* desc, const void* x, const void* r, const void* w, const void* wx,
                           const void* scale, void* n, void* r_out, void* stream) {
  TRY(check_addnorm(desc));
  if (desc->B * desc->T == 0) return GL_SUCCESS;
  gls::AddNormArgs a = addnorm_args(desc);
  const size_t e = elem_of(desc->io_dtype), re = elem_of(desc->res_dtype);
  TRY(check_ptrs(true, {x, w, n}, e));
  TRY(check_ptrs(true, {r, r_out}, re));
  TRY(check_ptrs(false, {wx, scale}, e));
  a.x = x; a.r = r; a.w = w; a.wx = wx; a.scale = scale; a.n = n; a.r_out = r_out;
  return hip_status(gls::launch_addnorm_fwd(desc->io_dtype, a, static_cast<hipStream_t>(stream)),
                    "residual norm launch");
}

static size_t addnorm_ws(const gl_addnorm_desc_t* d) {
  return round_up(3 * static_cast<size_t>(gls::addnorm_parts(addnorm_args(d))) * d->d * par_of(d->io_dtype));
}
gl_status_t gl_addnorm_workspace_size(const gl_addnorm_desc_t* desc, size_t* bwd_ws_bytes) {
  TRY(check_addnorm(desc));
  if (!bwd_ws_bytes) return fail(GL_ERROR_INVALID_VALUE, "bwd_ws_bytes is NULL");
  *bwd_ws_bytes = addnorm_ws(desc);
  return GL_SUCCESS;
}

gl_status_t gl_addnorm_bwd(const gl_addnorm_desc_t* desc, const void* x, const void* r, const void* w, const void* wx,
                           const void* scale, const void* dn, const void* dr_out, void* dx, void* dr, void* dw,
                           void* dwx, void* dscale, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_addnorm(desc));
  gls::AddNormArgs a = addnorm_args(desc);
  const bool any = a.B * a.T > 0;
  const size_t e = elem_of(desc->io_dtype), re = elem_of(desc->res_dtype);
  TRY(check_ptrs(any, {x, w, dn, dx}, e));
  TRY(check_ptrs(any, {r, dr}, re));
  TRY(check_ptrs(false, {wx, scale}, e));
  TRY(check_ptrs(false, {dr_out}, re));
  TRY(check_ptrs(false, {dw, dwx, dscale}, par_of(desc->io_dtype)));
  if (dw || dwx || dscale) TRY(check_ws(ws, ws_bytes, addnorm_ws(desc)));
  a.x = x; a.r = r; a.w = w; a.wx = wx; a.scale = scale; a.dn = dn; a.dro = dr_out; a.dx = dx; a.dr = dr;
  a.dw[0] = dw; a.dw[1] = dwx; a.dw[2] = dscale;
  a.part = ws;
  return hip_status(gls::launch_addnorm_bwd(desc->io_dtype, a, static_cast<hipStream_t>(stream)),
                    "residual norm backward launch");
}

gl_status_t gl_gatenorm_fwd(const gl_gatenorm_desc_t* desc, const void* x, const void* z, const void* w, void* y,
                            void* stream) {
  TRY(check_gatenorm(desc));
  if (desc->B * desc->T * desc->G == 0) return GL_SUCCESS;
  gls::GateNormArgs a = gatenorm_args(desc);
  const size_t e = elem_of(desc->io_dtype);
  TRY(check_ptrs(true, {x, y}, e));
  TRY(check_ptrs(false, {z, w}, e));
  a.x = x; a.z = z; a.w = w; a.y = y;
  return hip_status(gls::launch_gatenorm_fwd(desc->io_dtype, a, static_cast<hipStream_t>(stream)), "gated norm launch");
}

static size_t gatenorm_ws(const gl_gatenorm_desc_t* d) {
  const gls::GateNormArgs a = gatenorm_args(d);
  return round_up(static_cast<size_t>(gls::gatenorm_parts(a)) * (a.group_w ? a.G : 1) * a.d * par_of(d->io_dtype));
}
gl_status_t gl_gatenorm_workspace_size(const gl_gatenorm_desc_t* desc, size_t* bwd_ws_bytes) {
  TRY(check_gatenorm(desc));
  if (!bwd_ws_bytes) return fail(GL_ERROR_INVALID_VALUE, "bwd_ws_bytes is NULL");
  *bwd_ws_bytes = gatenorm_ws(desc);
  return GL_SUCCESS;
}

gl_status_t gl_gatenorm_bwd(const gl_gatenorm_desc_t* desc, const void* x, const void* z, const void* w,
                            const void* dy, void* dx, void* dz, void* dw, void* ws, size_t ws_bytes, void* stream) {
  TRY(check_gatenorm(desc));
  gls::GateNormArgs a = gatenorm_args(desc);
  const bool any = a.B * a.T * a.G > 0;
  const size_t e = elem_of(desc->io_dtype);
  TRY(check_ptrs(any, {x, dy, dx}, e));
  TRY(check_ptrs(any && z, {dz}, e));
  TRY(check_ptrs(false, {z, w}, e));
  TRY(check_ptrs(false, {dw}, par_of(desc->io_dtype)));
  if (!any && !dw) return GL_SUCCESS;
  if (dw) TRY(check_ws(ws, ws_bytes, gatenorm_ws(desc)));
  a.x = x; a.z = z; a.w = w; a.dy = dy; a.dx = dx; a.dz = dz; a.dw = dw;
  a.part = ws;
  return hip_status(gls::launch_gatenorm_bwd(desc->io_dtype, a, static_cast<hipStream_t>(stream)),
                    "gated norm backward launch");
}

}  // extern "C"
