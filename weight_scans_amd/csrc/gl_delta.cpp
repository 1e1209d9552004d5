// gl_delta.cpp -- host side of include/gl_delta.h: argument checks, choice of
// kernels, workspace layout and launches.  Every check runs before the first
// launch; nothing here allocates device memory.
#include "gl_delta.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "delta.hpp"

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
  return e == hipSuccess ? GL_SUCCESS : fail(GL_ERROR_HIP, "%s: %s", where, hipGetErrorString(e));
}

constexpr size_t kAlign = 256;
size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// Pointers that a call reads or writes (`need`: not NULL) or may (else).
gl_status_t check_ptrs(bool need, std::initializer_list<const void*> ps, size_t align = 16) {
  for (const void* p : ps) {
    if (!p && need) return fail(GL_ERROR_INVALID_VALUE, "NULL input or output pointer");
    if (reinterpret_cast<uintptr_t>(p) % align)
      return fail(GL_ERROR_MISALIGNED, "pointer %p not %zu-byte aligned", p, align);
  }
  return GL_SUCCESS;
}

bool zero(const gl_strides_t& s) { return s.b == 0 && s.h == 0 && s.t == 0; }
gls::Str3 dense(const gl_strides_t& s, int64_t H, int64_t T, int64_t d) {
  if (zero(s)) return {H * T * d, T * d, d};
  return {s.b, s.h, s.t};
}
bool negative(const gl_strides_t& s) { return s.b < 0 || s.h < 0 || s.t < 0; }

struct Plan {
  int io = 0;
  size_t comp = 4, gate = 4, elem = 2;  // bytes of a state's, a gate's and an io element
  size_t align = 2;                     // of q, k, v, y and their gradients
  int64_t N = 0, tok = 0;
  bool packed = false;
  bool chunk = false;                   // the chunked matrix-core path
  bool chunk32 = false;                 // its fp32 form
  bool brief = false;                   // so short that a forward which saves nothing goes token by token
  int64_t slots = 0;                    // its chunk slots
  int n_seg = 1;                        // segments per sequence of the bf16 forward
  size_t seg_bytes = 0, m_bytes = 0;    // their first states (last adjoints), their M
  size_t saved = 0, fwd_ws = 0, bwd_ws = 0;  // bwd_ws: with `saved` given
  size_t state_bytes = 0, err_bytes = 0, gate_bytes = 0, y_bytes = 0, last_bytes = 0, z_bytes = 0;
  const char* name = "";
};

gls::DeltaArgs base_args(const gl_delta_desc_t* d, const Plan& p) {
  gls::DeltaArgs a;
  a.N = p.N; a.B = d->B; a.T = d->T;
  a.H = static_cast<int>(d->H); a.Hk = static_cast<int>(d->Hk);
  a.dk = static_cast<int>(d->dk); a.dv = static_cast<int>(d->dv);
  a.gate_io = d->gate_dtype == d->io_dtype;
  a.scale = d->scale;
  a.sq = dense(d->sq, d->Hk, d->T, d->dk);
  a.sk = dense(d->sk, d->Hk, d->T, d->dk);
  a.sv = dense(d->sv, d->H, d->T, d->dv);
  a.sy = dense(d->sy, d->H, d->T, d->dv);
  a.sg = dense(d->sg, d->H, d->T, 1);
  a.sdq = dense(d->sdq, d->Hk, d->T, d->dk);
  a.sdk = dense(d->sdk, d->Hk, d->T, d->dk);
  a.sdv = dense(d->sdv, d->H, d->T, d->dv);
  a.sdy = dense(d->sdy, d->H, d->T, d->dv);
  a.sdg = dense(d->sdg, d->H, d->T, 1);
  return a;
}

// Sequences shorter than this (packed: their mean) go token by token: with one
// launch instead of two where nothing is saved, and in training where so few
// tokens leave the chunks' tiles all but empty.  Token by token against chunks,
// bf16, 8 x 16 heads of 128: forward 16 tokens 15 / 19 us, 32 tokens 24 / 20;
// backward 4 tokens 48 / 27, 8 tokens 74 / 27 (1 x 16 heads: forward 16 tokens 11
// / 14, 32 tokens 16 / 14; backward 4 tokens 20 / 20, 8 tokens 26 / 21).  All of equal
// lengths: the host does not know those of packed sequences, so a long one among many
// of a token or two is walked token by token too (0.3 us each, a chunk of 64 2.3).
constexpr int64_t kChunkFrom = 4, kChunkFwdFrom = 24;

// Segments of the chunked bf16 kernels.  Forward: n of them take two passes of 1 / n of the
// chunks each plus some 2 us a segment to join them, and need n times the
// work-groups, of which one fits a CU.  With / without at 16 heads of 128: 32768
// tokens 543 / 1031 us, 2048 tokens 61 / 74; 4 heads of 64: 32768 tokens 103 / 739,
// 4096 tokens 46 / 101; 32 heads of 128, 4096 tokens, where the rule says no: 162
// with three, 151 without.
int segments_of(const gl_delta_desc_t* d, const Plan& p) {
  const int64_t chunks = std::max<int64_t>(1, d->T / (std::max<int64_t>(p.N, 1) * gls::kDeltaChunk));
  const int64_t heads = std::max<int64_t>(1, p.N * d->H), groups = heads * ((d->dv + 31) / 32);
  if (d->segments > 0)
    return static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>({static_cast<int64_t>(d->segments), chunks, 1024, (1 << 28) / heads})));
  const int64_t n = std::min<int64_t>(
      {256 / groups, static_cast<int64_t>(std::sqrt(1.5 * static_cast<double>(chunks))), chunks / 8});
  return n >= 3 ? static_cast<int>(n) : 1;
}

gl_status_t make_plan(const gl_delta_desc_t* d, Plan* p) {
  if (!d) return fail(GL_ERROR_INVALID_VALUE, "desc is NULL");
  if (d->B < 0 || d->T < 0 || d->H < 0 || d->Hk < 0 || d->n_seq < 0)
    return fail(GL_ERROR_INVALID_VALUE, "negative B, T, H, Hk or n_seq");
  if (d->dk < 1 || d->dv < 1) return fail(GL_ERROR_INVALID_VALUE, "dk and dv must be >= 1");
  if (d->io_dtype < GL_DTYPE_F64 || d->io_dtype > GL_DTYPE_BF16)
    return fail(GL_ERROR_INVALID_VALUE, "unknown io_dtype %d", d->io_dtype);
  if (d->gate_dtype != d->io_dtype && !(d->gate_dtype == GL_DTYPE_F32 && d->io_dtype == GL_DTYPE_BF16))
    return fail(GL_ERROR_INVALID_VALUE, "gate_dtype must be io_dtype, or F32 with BF16 io");
  if (d->flags & ~GL_FLAG_GENERIC) return fail(GL_ERROR_INVALID_VALUE, "unknown flags");
  if (d->segments > (1u << 20)) return fail(GL_ERROR_INVALID_VALUE, "segments above 2^20");
  if (!(std::isfinite(d->scale))) return fail(GL_ERROR_INVALID_VALUE, "scale is not finite");
  if (d->H > 0 && (d->Hk == 0 || d->H % d->Hk))
    return fail(GL_ERROR_INVALID_VALUE, "H must be a multiple of Hk (%lld, %lld)", (long long)d->H, (long long)d->Hk);
  if (d->n_seq > 0 && d->B != 1) return fail(GL_ERROR_INVALID_VALUE, "packed sequences need B = 1");
  for (const gl_strides_t& s : {d->sq, d->sk, d->sv, d->sy, d->sg, d->sdq, d->sdk, d->sdv, d->sdy, d->sdg})
    if (negative(s)) return fail(GL_ERROR_INVALID_VALUE, "negative stride");
  if (d->dk > gls::kGenericMaxD || d->dv > gls::kGenericMaxD)
    return fail(GL_ERROR_NOT_SUPPORTED, "dk/dv above %d", gls::kGenericMaxD);
  p->packed = d->n_seq > 0;
  if (p->packed && d->T > 0x7fffffffLL) return fail(GL_ERROR_NOT_SUPPORTED, "packed T above 2^31-1");
  p->N = p->packed ? d->n_seq : d->B;
  p->tok = d->B * d->T;
  const double n_all = std::max(1.0, double(p->N)) * std::max(1.0, double(d->T)) * std::max(1.0, double(d->H));
  if (double(p->N) * double(d->H) * 8 > 2147483647.0 || n_all * 128 * 128 * 8 > 4e18 ||
      double(std::max(d->H, d->Hk)) > 1e6)
    return fail(GL_ERROR_NOT_SUPPORTED, "sizes above the launch limits");
  p->io = d->io_dtype;
  p->comp = p->io == GL_DTYPE_F64 ? 8 : 4;
  p->gate = d->gate_dtype == GL_DTYPE_F64 ? 8 : d->gate_dtype == GL_DTYPE_F32 ? 4 : 2;
  p->elem = p->io == GL_DTYPE_F64 ? 8 : p->io == GL_DTYPE_F32 ? 4 : 2;
  p->align = p->elem;
  const size_t dd = static_cast<size_t>(d->dk) * d->dv;
  const gls::DeltaArgs a = base_args(d, *p);
  const int64_t shared = p->packed ? p->N : 1;  // sequences that share T tokens
  const bool chunks = !(d->flags & GL_FLAG_GENERIC) && d->T >= kChunkFrom * shared;
  p->brief = d->T < kChunkFwdFrom * shared;
  if (chunks && gls::delta_chunk_ok(p->io, a)) {
    p->chunk = true;
    p->align = 16;
    p->name = d->dk <= 64 ? (d->dv <= 64 ? "delta-mfma-bf16-64x64" : "delta-mfma-bf16-64x128")
                          : (d->dv <= 64 ? "delta-mfma-bf16-128x64" : "delta-mfma-bf16-128x128");
    p->slots = gls::chunk_slots(p->packed, p->N, d->T, gls::kDeltaChunk);
    if (double(p->slots) * double(d->H) > 2147483647.0)
      return fail(GL_ERROR_NOT_SUPPORTED, "chunks above the launch limits");
    const size_t rec = static_cast<size_t>(p->slots) * d->H;
    p->n_seg = segments_of(d, *p);
    const size_t segs = p->n_seg > 1 ? static_cast<size_t>(p->N) * d->H * p->n_seg : 0;
    p->seg_bytes = round_up(segs * dd * 4);
    p->m_bytes = round_up(segs * d->dk * d->dk * 4);
    p->fwd_ws = round_up(rec * gls::kYf * 2);
    p->state_bytes = round_up(rec * gls::delta_row_tiles(a.dv) * (gls::delta_wide(a.dk) / 16) * gls::kPiece * 2);
    p->err_bytes = round_up(rec * 4 * gls::delta_row_tiles(a.dv) * gls::kPiece * 2);
    // what is workspace in a forward that saves nothing
    p->gate_bytes = round_up(rec * gls::kGates * 4) + p->seg_bytes + p->m_bytes;
    p->y_bytes = round_up(rec * gls::delta_row_tiles(a.dv) * 4096);
    p->last_bytes = round_up(static_cast<size_t>(p->N) * d->H * dd * 4);
    p->z_bytes = round_up(rec * gls::delta_row_tiles(a.dv) * 64 * 4);
    p->saved = p->gate_bytes + 2 * round_up(rec * gls::kYf * 2) + p->state_bytes + p->err_bytes + p->y_bytes +
               p->last_bytes;
    p->bwd_ws = p->state_bytes + p->err_bytes + 2 * p->z_bytes + p->seg_bytes;
    return GL_SUCCESS;
  }
  if (chunks && gls::delta_chunk_f32_ok(p->io, a)) {
    p->chunk32 = true;
    p->align = 16;
    p->name = d->dk <= 64 ? "delta-mfma-f32-64" : "delta-mfma-f32-128";
    p->slots = gls::chunk_slots(p->packed, p->N, d->T, gls::kDeltaChunk);
    if (double(p->slots) * double(d->H) > 2147483647.0)
      return fail(GL_ERROR_NOT_SUPPORTED, "chunks above the launch limits");
    const size_t rec = static_cast<size_t>(p->slots) * d->H, tiles = gls::delta_row_tiles(a.dv);
    p->gate_bytes = round_up(rec * gls::kGates * 4);
    p->fwd_ws = 2 * round_up(rec * gls::kY32 * 4);
    p->state_bytes = round_up(rec * tiles * gls::delta_wide(a.dk) * 16 * 4);
    p->y_bytes = p->err_bytes = round_up(rec * tiles * 64 * 16 * 4);
    p->z_bytes = round_up(rec * tiles * 64 * 4);
    p->last_bytes = round_up(static_cast<size_t>(p->N) * d->H * dd * 4);
    p->saved = p->gate_bytes + p->fwd_ws + p->state_bytes + p->err_bytes + p->y_bytes + p->last_bytes;
    p->bwd_ws = p->state_bytes + p->err_bytes + 2 * p->z_bytes;
    return GL_SUCCESS;
  }
  const int ck = gls::serial_ck(p->io);
  p->name = p->io == GL_DTYPE_F64 ? "delta-serial-f64" : p->io == GL_DTYPE_F32 ? "delta-serial-f32" : "delta-serial-bf16";
  p->saved = round_up(static_cast<size_t>(gls::chunk_slots(p->packed, p->N, d->T, ck)) * d->H * dd * p->comp);
  const size_t tiles = (d->dv + gls::kSerialRows - 1) / gls::kSerialRows;
  p->bwd_ws = 2 * round_up(tiles * d->H * p->tok * d->dk * p->comp) + 2 * round_up(tiles * d->H * p->tok * p->comp);
  return GL_SUCCESS;
}

gl_status_t check_cu(const Plan& p, const int32_t* cu) {
  if (p.packed && !cu) return fail(GL_ERROR_INVALID_VALUE, "n_seq > 0 needs cu_seqlens");
  if (!p.packed && cu) return fail(GL_ERROR_INVALID_VALUE, "cu_seqlens needs n_seq > 0");
  if (reinterpret_cast<uintptr_t>(cu) & 3) return fail(GL_ERROR_MISALIGNED, "cu_seqlens not 4-byte aligned");
  return GL_SUCCESS;
}

struct Cut {  // runs of a workspace
  char* at;
  template <typename T>
  void take(T*& p, size_t bytes) {
    p = reinterpret_cast<T*>(at);
    at += round_up(bytes);
  }
};

// Chunked path: arguments with `saved` and the forward's workspace laid out.
gls::ChunkArgs chunk_args(const gls::DeltaArgs& a, const Plan& p, void* saved, void* ws) {
  gls::ChunkArgs c;
  c.a = a;
  c.slots = p.slots;
  const size_t rec = static_cast<size_t>(p.slots) * a.H;
  Cut w{static_cast<char*>(ws)};
  if (ws) {
    w.take(c.yf, rec * gls::kYf * 2);
  }
  c.n_seg = p.n_seg;
  Cut g{static_cast<char*>(saved)};
  Cut& s = saved ? g : w;
  s.take(c.gates, rec * gls::kGates * 4);
  s.take(c.seg_s, p.seg_bytes);
  s.take(c.seg_m, p.m_bytes);
  if (saved) {
    s.take(c.ytf, rec * gls::kYf * 2);
    s.take(c.ptf, rec * gls::kYf * 2);
    s.take(c.sf, p.state_bytes);
    s.take(c.ef, p.err_bytes);
    s.take(c.yb, p.y_bytes);
    s.take(c.st, p.last_bytes);
  }
  return c;
}

// The same in fp32.
gls::ChunkArgs chunk32_args(const gls::DeltaArgs& a, const Plan& p, void* saved, void* ws) {
  gls::ChunkArgs c;
  c.a = a;
  c.slots = p.slots;
  const size_t y = static_cast<size_t>(p.slots) * a.H * gls::kY32 * 4;
  Cut w{static_cast<char*>(ws)};
  if (ws) {
    w.take(c.y32, y);
    w.take(c.p32, y);
  }
  if (saved) {
    Cut s{static_cast<char*>(saved)};
    s.take(c.gates, p.gate_bytes);
    s.take(c.yt32, y);
    s.take(c.pt32, y);
    s.take(c.s32, p.state_bytes);
    s.take(c.e32, p.err_bytes);
    s.take(c.yb, p.y_bytes);
    s.take(c.st, p.last_bytes);
  } else {
    w.take(c.gates, p.gate_bytes);
  }
  return c;
}

gl_status_t chunk_fwd(const gls::ChunkArgs& c, hipStream_t s) {
  const gl_status_t st = hip_status(gls::launch_delta_prep(c, s), "delta chunk preparation launch");
  return st != GL_SUCCESS ? st : hip_status(gls::launch_delta_chunk_fwd(c, s), "delta forward launch");
}

gl_status_t check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return GL_SUCCESS;
  if (!ws) return fail(GL_ERROR_INVALID_VALUE, "workspace is NULL (%zu bytes needed)", need);
  if (misaligned(ws)) return fail(GL_ERROR_MISALIGNED, "workspace not 16-byte aligned");
  if (have < need) return fail(GL_ERROR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", have, need);
  return GL_SUCCESS;
}

}  // namespace

extern "C" {

gl_status_t gl_delta_saved_size(const gl_delta_desc_t* desc, size_t* saved_bytes) {
  Plan p;
  const gl_status_t st = make_plan(desc, &p);
  if (st != GL_SUCCESS) return st;
  if (!saved_bytes) return fail(GL_ERROR_INVALID_VALUE, "saved_bytes is NULL");
  *saved_bytes = p.saved;
  return GL_SUCCESS;
}

gl_status_t gl_delta_workspace_size(const gl_delta_desc_t* desc, int have_saved, size_t* fwd_ws_bytes,
                                    size_t* bwd_ws_bytes) {
  Plan p;
  const gl_status_t st = make_plan(desc, &p);
  if (st != GL_SUCCESS) return st;
  if (!fwd_ws_bytes || !bwd_ws_bytes) return fail(GL_ERROR_INVALID_VALUE, "size pointer is NULL");
  // without `saved` the forward's gate factors are workspace too
  *fwd_ws_bytes = p.fwd_ws + (have_saved ? 0 : p.gate_bytes);
  *bwd_ws_bytes = p.bwd_ws + (have_saved ? 0 : p.saved + p.fwd_ws);
  return GL_SUCCESS;
}

gl_status_t gl_delta_fwd(const gl_delta_desc_t* desc, const void* q, const void* k, const void* v,
                         const void* log_alpha, const void* beta, const void* state_in,
                         const int32_t* cu_seqlens, void* y, void* state_out, void* saved, void* ws,
                         size_t ws_bytes, void* stream) {
  Plan p;
  gl_status_t st = make_plan(desc, &p);
  if (st != GL_SUCCESS) return st;
  if (p.N * desc->H == 0) return GL_SUCCESS;
  if ((st = check_cu(p, cu_seqlens)) != GL_SUCCESS) return st;
  if (p.tok > 0 && (st = check_ptrs(true, {q, k, v, y}, saved ? p.align : p.elem)) != GL_SUCCESS) return st;
  if (p.tok > 0 && (st = check_ptrs(true, {log_alpha, beta}, p.gate)) != GL_SUCCESS) return st;
  if ((st = check_ptrs(false, {state_in, state_out, saved})) != GL_SUCCESS) return st;
  if ((st = check_ws(ws, ws_bytes, p.fwd_ws + (saved ? 0 : p.gate_bytes))) != GL_SUCCESS) return st;
  if (p.tok == 0 && !state_out) return GL_SUCCESS;
  gls::DeltaArgs a = base_args(desc, p);
  a.q = q; a.k = k; a.v = v; a.la = log_alpha; a.be = beta;
  a.state_in = state_in; a.cu = cu_seqlens; a.y = y; a.state_out = state_out; a.ckpt = saved;
  // Chunks, or token by token (without the workspace) where that is allowed and
  // faster, or the only way: alignment and the strides of y are known here only
  if (p.chunk || p.chunk32) {
    const bool rows = p.chunk ? gls::delta_rows_ok(a.sy, a.dv) : gls::delta_rows_f32_ok(a.sy, a.dv);
    const bool fits = rows && !(misaligned(q) || misaligned(k) || misaligned(v) || misaligned(y));
    if (saved && p.tok > 0 && !fits)
      return fail(rows ? GL_ERROR_MISALIGNED : GL_ERROR_NOT_SUPPORTED,
                  "q, k, v, y of a training call: 16-byte aligned, rows apart, strides multiples of 16 bytes");
    if (saved || (fits && !p.brief)) {
      const hipStream_t s = static_cast<hipStream_t>(stream);
      return p.chunk ? chunk_fwd(chunk_args(a, p, saved, ws), s)
                     : hip_status(gls::launch_delta_chunk_f32(chunk32_args(a, p, saved, ws), s), "delta forward launch");
    }
  }
  return hip_status(gls::launch_delta_serial_fwd(p.io, a, static_cast<hipStream_t>(stream)), "delta forward launch");
}

gl_status_t gl_delta_bwd(const gl_delta_desc_t* desc, const void* q, const void* k, const void* v,
                         const void* log_alpha, const void* beta, const void* state_in,
                         const int32_t* cu_seqlens, const void* dy, const void* dstate_out,
                         const void* saved, void* dq, void* dk, void* dv, void* dlog_alpha, void* dbeta,
                         void* dstate_in, void* ws, size_t ws_bytes, void* stream) {
  Plan p;
  gl_status_t st = make_plan(desc, &p);
  if (st != GL_SUCCESS) return st;
  if (desc->H == 0 && desc->Hk > 0 && p.tok > 0) {  // keys that no value head reads
    if ((st = check_ptrs(true, {dq, dk}, p.elem)) != GL_SUCCESS) return st;
    gls::DeltaArgs a = base_args(desc, p);
    a.dq = dq; a.dk_ = dk;
    return hip_status(gls::launch_delta_serial_bwd(p.io, a, static_cast<hipStream_t>(stream)), "delta backward launch");
  }
  if (p.N * desc->H == 0) return GL_SUCCESS;
  if ((st = check_cu(p, cu_seqlens)) != GL_SUCCESS) return st;
  if (p.tok > 0 && (st = check_ptrs(true, {q, k, v, dy, dq, dk, dv}, p.align)) != GL_SUCCESS) return st;
  if (p.tok > 0 && (st = check_ptrs(true, {log_alpha, beta, dlog_alpha, dbeta}, p.gate)) != GL_SUCCESS) return st;
  if ((st = check_ptrs(false, {state_in, dstate_out, saved, dstate_in})) != GL_SUCCESS) return st;
  const size_t need = p.bwd_ws + (saved ? 0 : p.saved + p.fwd_ws);
  if ((st = check_ws(ws, ws_bytes, need)) != GL_SUCCESS) return st;
  if (p.tok == 0 && !dstate_in) return GL_SUCCESS;
  gls::DeltaArgs a = base_args(desc, p);
  a.q = q; a.k = k; a.v = v; a.la = log_alpha; a.be = beta;
  a.state_in = state_in; a.cu = cu_seqlens; a.dy = dy; a.dstate_out = dstate_out;
  a.dq = dq; a.dk_ = dk; a.dv_ = dv; a.dla = dlog_alpha; a.dbe = dbeta; a.dstate_in = dstate_in;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Cut w{static_cast<char*>(ws)};
  if (p.chunk) {
    if (p.tok > 0 && !(gls::delta_rows_ok(a.sdy, a.dv) && gls::delta_rows_ok(a.sdv, a.dv) &&
                       gls::delta_rows_ok(a.sdq, a.dk) && gls::delta_rows_ok(a.sdk, a.dk)))
      return fail(GL_ERROR_NOT_SUPPORTED, "strides of dy, dq, dk, dv: multiples of 8, rows apart");
    uint16_t *lf, *gf;
    float *zf, *bf, *seg_l;
    char *again, *fws;
    w.take(lf, p.state_bytes);
    w.take(gf, p.err_bytes);
    w.take(zf, p.z_bytes);
    w.take(bf, p.z_bytes);
    w.take(seg_l, p.seg_bytes);
    w.take(again, saved ? 0 : p.saved);
    w.take(fws, saved ? 0 : p.fwd_ws);
    gls::ChunkArgs c = chunk_args(a, p, saved ? const_cast<void*>(saved) : again, saved ? nullptr : fws);
    if (!saved && (st = chunk_fwd(c, s)) != GL_SUCCESS) return st;  // a.y and a.state_out NULL: what is saved only
    c.lf = lf;
    c.gf = gf;
    c.zf = zf;
    c.bf = bf;
    c.seg_l = seg_l;
    return hip_status(gls::launch_delta_chunk_bwd(c, s), "delta backward launch");
  }
  if (p.chunk32) {
    if (p.tok > 0 && !(gls::delta_rows_f32_ok(a.sdy, a.dv) && gls::delta_rows_f32_ok(a.sdv, a.dv)))
      return fail(GL_ERROR_NOT_SUPPORTED, "strides of dy, dv: multiples of 4, rows apart");
    float *lf, *gf, *zf, *bf;
    char *again, *fws;
    w.take(lf, p.state_bytes);
    w.take(gf, p.err_bytes);
    w.take(zf, p.z_bytes);
    w.take(bf, p.z_bytes);
    w.take(again, saved ? 0 : p.saved);
    w.take(fws, saved ? 0 : p.fwd_ws);
    gls::ChunkArgs c = chunk32_args(a, p, saved ? const_cast<void*>(saved) : again, saved ? nullptr : fws);
    if (!saved && (st = hip_status(gls::launch_delta_chunk_f32(c, s), "delta forward launch")) != GL_SUCCESS) return st;
    c.l32 = lf;
    c.g32 = gf;
    c.zf = zf;
    c.bf = bf;
    return hip_status(gls::launch_delta_chunk_f32_bwd(c, s), "delta backward launch");
  }
  const size_t tiles = (desc->dv + gls::kSerialRows - 1) / gls::kSerialRows;
  w.take(a.part_dq, tiles * desc->H * p.tok * desc->dk * p.comp);
  w.take(a.part_dk, tiles * desc->H * p.tok * desc->dk * p.comp);
  w.take(a.part_la, tiles * desc->H * p.tok * p.comp);
  w.take(a.part_be, tiles * desc->H * p.tok * p.comp);
  a.ckpt = const_cast<void*>(saved);
  if (!saved && p.saved) {
    w.take(a.ckpt, p.saved);
    st = hip_status(gls::launch_delta_serial_fwd(p.io, a, s), "delta states launch");  // a.y NULL: states only
    if (st != GL_SUCCESS) return st;
  }
  return hip_status(gls::launch_delta_serial_bwd(p.io, a, s), "delta backward launch");
}

gl_status_t gl_delta_step(const gl_delta_desc_t* desc, const void* q, const void* k, const void* v,
                          const void* log_alpha, const void* beta, const int32_t* slots, int64_t n_slots,
                          void* state, void* y, void* stream) {
  Plan p;
  gl_status_t st = make_plan(desc, &p);
  if (st != GL_SUCCESS) return st;
  if (p.packed) return fail(GL_ERROR_INVALID_VALUE, "a step takes no packed sequences");
  if (n_slots < 0) return fail(GL_ERROR_INVALID_VALUE, "n_slots is negative");
  if (desc->B * desc->H == 0) return GL_SUCCESS;
  if (!slots && n_slots < desc->B)
    return fail(GL_ERROR_INVALID_VALUE, "%lld states for %lld rows", (long long)n_slots, (long long)desc->B);
  if ((st = check_ptrs(true, {q, k, v, y}, p.elem)) != GL_SUCCESS) return st;
  if ((st = check_ptrs(true, {log_alpha, beta}, p.gate)) != GL_SUCCESS) return st;
  if ((st = check_ptrs(n_slots > 0, {state})) != GL_SUCCESS) return st;
  if (reinterpret_cast<uintptr_t>(slots) & 3) return fail(GL_ERROR_MISALIGNED, "slots not 4-byte aligned");
  gl_delta_desc_t one = *desc;
  one.T = 1;
  gls::DeltaArgs a = base_args(&one, p);
  a.q = q; a.k = k; a.v = v; a.la = log_alpha; a.be = beta;
  a.slots = slots; a.n_slots = n_slots; a.state_out = state; a.y = y;
  return hip_status(gls::launch_delta_step(p.io, a, static_cast<hipStream_t>(stream)), "delta step launch");
}

const char* gl_delta_path_name(const gl_delta_desc_t* desc) {
  Plan p;
  return make_plan(desc, &p) == GL_SUCCESS ? p.name : nullptr;
}

// ------------------------------------------------------ norms and rotation
static gl_status_t check_qk(const gl_qknorm_desc_t* d) {
  if (!d) return fail(GL_ERROR_INVALID_VALUE, "desc is NULL");
  if (d->B < 0 || d->T < 0 || d->Hq < 0 || d->Hk < 0 || d->n_pos < 0)
    return fail(GL_ERROR_INVALID_VALUE, "negative B, T, Hq, Hk or n_pos");
  if (d->d < 1) return fail(GL_ERROR_INVALID_VALUE, "d must be >= 1");
  if (d->rot < 0 || d->rot > d->d || d->rot % 2) return fail(GL_ERROR_INVALID_VALUE, "rot must be even and in 0..d");
  if (d->rot > 0 && d->n_pos < 1) return fail(GL_ERROR_INVALID_VALUE, "a rotation needs tables of n_pos >= 1 rows");
  if (d->io_dtype < GL_DTYPE_F64 || d->io_dtype > GL_DTYPE_BF16)
    return fail(GL_ERROR_INVALID_VALUE, "unknown io_dtype %d", d->io_dtype);
  if (d->flags & ~GL_FLAG_INTERLEAVED) return fail(GL_ERROR_INVALID_VALUE, "unknown flags");
  if (!(d->eps >= 0) || !std::isfinite(d->eps) || !std::isfinite(d->q_scale) || !std::isfinite(d->k_scale))
    return fail(GL_ERROR_INVALID_VALUE, "eps must be finite and >= 0, the scales finite");
  for (const gl_strides_t& s : {d->sq, d->sk, d->soq, d->sok, d->sdoq, d->sdok, d->sdq, d->sdk})
    if (negative(s)) return fail(GL_ERROR_INVALID_VALUE, "negative stride");
  if (d->d > 256) return fail(GL_ERROR_NOT_SUPPORTED, "d above 256");
  if (double(d->B) * double(d->T) * (double(d->Hq) + double(d->Hk)) * 16 > 2147483647.0 * 256)
    return fail(GL_ERROR_NOT_SUPPORTED, "sizes above the launch limits");
  if (d->Hq > (1 << 20) || d->Hk > (1 << 20)) return fail(GL_ERROR_NOT_SUPPORTED, "more than 2^20 heads");
  return GL_SUCCESS;
}

static gls::QkArgs qk_args(const gl_qknorm_desc_t* d, const void* q, const void* k, const void* wq, const void* wk,
                           const void* cos, const void* sin, const int32_t* pos) {
  gls::QkArgs a{};
  a.x[0] = q; a.x[1] = k;
  a.w[0] = wq; a.w[1] = wk;
  a.Hn[0] = static_cast<int>(d->Hq); a.Hn[1] = static_cast<int>(d->Hk);
  a.scale[0] = d->q_scale; a.scale[1] = d->k_scale;
  a.sx[0] = dense(d->sq, d->Hq, d->T, d->d);
  a.sx[1] = dense(d->sk, d->Hk, d->T, d->d);
  a.so[0] = dense(d->soq, d->Hq, d->T, d->d);
  a.so[1] = dense(d->sok, d->Hk, d->T, d->d);
  a.sdo[0] = dense(d->sdoq, d->Hq, d->T, d->d);
  a.sdo[1] = dense(d->sdok, d->Hk, d->T, d->d);
  a.cos = cos; a.sin = sin; a.pos = pos;
  a.B = d->B; a.T = d->T; a.n_pos = d->n_pos; a.pos0 = d->pos0;
  a.d = static_cast<int>(d->d); a.rot = static_cast<int>(d->rot);
  a.interleaved = (d->flags & GL_FLAG_INTERLEAVED) != 0;
  a.eps = d->eps;
  return a;
}

static size_t qk_elem(const gl_qknorm_desc_t* d) { return d->io_dtype == GL_DTYPE_F64 ? 8 : d->io_dtype == GL_DTYPE_F32 ? 4 : 2; }
static size_t qk_comp(const gl_qknorm_desc_t* d) { return d->io_dtype == GL_DTYPE_F64 ? 8 : 4; }

static gl_status_t check_qk_ptrs(const gl_qknorm_desc_t* d, const void* q, const void* k, const void* wq,
                                 const void* wk, const void* cos, const void* sin, const int32_t* pos) {
  gl_status_t st;
  if (d->Hq && (st = check_ptrs(true, {q}, qk_elem(d))) != GL_SUCCESS) return st;
  if (d->Hk && (st = check_ptrs(true, {k}, qk_elem(d))) != GL_SUCCESS) return st;
  if ((st = check_ptrs(false, {wq, wk}, qk_elem(d))) != GL_SUCCESS) return st;
  if (d->rot && (st = check_ptrs(true, {cos, sin}, qk_comp(d))) != GL_SUCCESS) return st;
  if (reinterpret_cast<uintptr_t>(pos) & 3) return fail(GL_ERROR_MISALIGNED, "pos not 4-byte aligned");
  return GL_SUCCESS;
}

gl_status_t gl_qknorm_rope_fwd(const gl_qknorm_desc_t* desc, const void* q, const void* k, const void* wq,
                               const void* wk, const void* cos, const void* sin, const int32_t* pos, void* out_q,
                               void* out_k, void* stream) {
  gl_status_t st = check_qk(desc);
  if (st != GL_SUCCESS) return st;
  if (desc->B * desc->T * (desc->Hq + desc->Hk) == 0) return GL_SUCCESS;
  if ((st = check_qk_ptrs(desc, q, k, wq, wk, cos, sin, pos)) != GL_SUCCESS) return st;
  if (desc->Hq && (st = check_ptrs(true, {out_q}, qk_elem(desc))) != GL_SUCCESS) return st;
  if (desc->Hk && (st = check_ptrs(true, {out_k}, qk_elem(desc))) != GL_SUCCESS) return st;
  gls::QkArgs a = qk_args(desc, q, k, wq, wk, cos, sin, pos);
  a.out[0] = out_q; a.out[1] = out_k;
  return hip_status(gls::launch_qknorm_fwd(desc->io_dtype, a, static_cast<hipStream_t>(stream)),
                    "query / key norm launch");
}

gl_status_t gl_qknorm_rope_workspace_size(const gl_qknorm_desc_t* desc, size_t* bwd_ws_bytes) {
  const gl_status_t st = check_qk(desc);
  if (st != GL_SUCCESS) return st;
  if (!bwd_ws_bytes) return fail(GL_ERROR_INVALID_VALUE, "bwd_ws_bytes is NULL");
  const gls::QkArgs a = qk_args(desc, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
  *bwd_ws_bytes = round_up(2 * static_cast<size_t>(gls::qknorm_bwd_parts(desc->io_dtype, a)) * desc->d *
                           (desc->io_dtype == GL_DTYPE_F64 ? 8 : 4));
  return GL_SUCCESS;
}

gl_status_t gl_qknorm_rope_bwd(const gl_qknorm_desc_t* desc, const void* q, const void* k, const void* wq,
                               const void* wk, const void* cos, const void* sin, const int32_t* pos,
                               const void* dout_q, const void* dout_k, void* dq, void* dk, void* dwq, void* dwk,
                               void* ws, size_t ws_bytes, void* stream) {
  gl_status_t st = check_qk(desc);
  if (st != GL_SUCCESS) return st;
  const bool any = desc->B * desc->T > 0;
  if (any && (st = check_qk_ptrs(desc, q, k, wq, wk, cos, sin, pos)) != GL_SUCCESS) return st;
  if (any && desc->Hq && (st = check_ptrs(true, {dout_q, dq}, qk_elem(desc))) != GL_SUCCESS) return st;
  if (any && desc->Hk && (st = check_ptrs(true, {dout_k, dk}, qk_elem(desc))) != GL_SUCCESS) return st;
  if ((st = check_ptrs(false, {dwq, dwk}, qk_comp(desc))) != GL_SUCCESS) return st;
  if ((!any || desc->Hq + desc->Hk == 0) && !dwq && !dwk) return GL_SUCCESS;
  size_t need = 0;
  if ((st = gl_qknorm_rope_workspace_size(desc, &need)) != GL_SUCCESS) return st;
  if ((st = check_ws(ws, ws_bytes, need)) != GL_SUCCESS) return st;
  gls::QkArgs a = qk_args(desc, q, k, wq, wk, cos, sin, pos);
  a.dout[0] = dout_q; a.dout[1] = dout_k;
  a.out[0] = dq; a.out[1] = dk;
  a.so[0] = dense(desc->sdq, desc->Hq, desc->T, desc->d);
  a.so[1] = dense(desc->sdk, desc->Hk, desc->T, desc->d);
  a.dw[0] = dwq; a.dw[1] = dwk;
  a.part = ws;
  a.n_part = gls::qknorm_bwd_parts(desc->io_dtype, a);
  return hip_status(gls::launch_qknorm_bwd(desc->io_dtype, a, static_cast<hipStream_t>(stream)),
                    "query / key norm backward launch");
}

}  // extern "C"
