"""The gated delta rule and the query / key norms with the position rotation:
torch tensors into the C ABI of ``include/gl_delta.h`` (no compute here).

    y, state, saved = gl_delta_fwd(q, k, v, log_alpha, beta, state=S0, want_state=True, save=True)
    dq, dk, dv, dlog_alpha, dbeta, dS0 = gl_delta_bwd(q, k, v, log_alpha, beta, dy, saved, ...)
    y1 = gl_delta_step(q1, k1, v1, log_alpha1, beta1, state)        # one token, state in place
    y, state = delta_rule(q, k, v, log_alpha, beta)                  # autograd-aware
    qn, kn = gl_qknorm_rope_fwd(q, k, wq, wk, cos, sin, pos=pos)
    dq, dk, dwq, dwk = gl_qknorm_rope_bwd(q, k, wq, wk, cos, sin, dqn, dkn, pos=pos)
    qn, kn = qknorm_rope(q, k, wq, wk, cos, sin)                     # autograd-aware

Shapes: q, k [B,Hk,T,dk], v [B,H,T,dv] (H a multiple of Hk), log_alpha, beta
[B,H,T], states [B,H,dv,dk] in fp32 (fp64 for fp64 io); with cu_seqlens [n + 1]
(int32, on the device) B is 1 and the states are [n,H,dv,dk].  Tensors of heads
may be views with any strides whose last dimension is contiguous (slices of a
fused projection's [B,T,H,d]); outputs take the order of dimensions of the
input that they belong to.
"""
from __future__ import annotations

import ctypes

from . import GLScanError, _io_code, _ptr, _stream, _torch, gate_dtype  # noqa: F401
from . import lib as _load

DELTA_EXPORTS = (
    "gl_delta_saved_size",
    "gl_delta_workspace_size",
    "gl_delta_fwd",
    "gl_delta_bwd",
    "gl_delta_step",
    "gl_delta_path_name",
    "gl_qknorm_rope_fwd",
    "gl_qknorm_rope_workspace_size",
    "gl_qknorm_rope_bwd",
)

GL_FLAG_INTERLEAVED = 8


class Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("t", ctypes.c_int64)]


class DeltaDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "T", "H", "Hk", "dk", "dv", "n_seq")] + [
        ("io_dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("segments", ctypes.c_uint32), ("scale", ctypes.c_double)] + [
        (n, Strides) for n in ("sq", "sk", "sv", "sy", "sg", "sdq", "sdk", "sdv", "sdy", "sdg")]


class QkDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "T", "Hq", "Hk", "d", "rot", "n_pos", "pos0")] + [
        ("io_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32), ("eps", ctypes.c_double),
        ("q_scale", ctypes.c_double), ("k_scale", ctypes.c_double)] + [
        (n, Strides) for n in ("sq", "sk", "soq", "sok", "sdoq", "sdok", "sdq", "sdk")]


_lib = None


def delta_lib():
    """libglscan.so with the argument types of gl_delta.h set."""
    global _lib
    if _lib is None:
        L = _load()
        P, S, I64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
        pd, pk, ps = ctypes.POINTER(DeltaDesc), ctypes.POINTER(QkDesc), ctypes.POINTER(ctypes.c_size_t)
        L.gl_delta_saved_size.argtypes = [pd, ps]
        L.gl_delta_workspace_size.argtypes = [pd, ctypes.c_int, ps, ps]
        L.gl_delta_fwd.argtypes = [pd] + [P] * 11 + [S, P]
        L.gl_delta_bwd.argtypes = [pd] + [P] * 17 + [S, P]
        L.gl_delta_step.argtypes = [pd] + [P] * 6 + [I64] + [P] * 3
        L.gl_qknorm_rope_fwd.argtypes = [pk] + [P] * 10
        L.gl_qknorm_rope_workspace_size.argtypes = [pk, ps]
        L.gl_qknorm_rope_bwd.argtypes = [pk] + [P] * 14 + [S, P]
        for n in DELTA_EXPORTS:
            getattr(L, n).restype = ctypes.c_int
        L.gl_delta_path_name.argtypes = [pd]
        L.gl_delta_path_name.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(status):
    if status != 0:
        raise GLScanError(status, _load().gl_last_error().decode())


def make_delta_desc(B, T, H, Hk, dk, dv, io_dtype, gate_dtype, *, n_seq=0, flags=0, segments=0,
                    scale=1.0) -> DeltaDesc:
    return DeltaDesc(B, T, H, Hk, dk, dv, n_seq, io_dtype, gate_dtype, flags, segments, scale)


def delta_path_name(desc: DeltaDesc) -> str | None:
    r = delta_lib().gl_delta_path_name(ctypes.byref(desc))
    return r.decode() if r else None


def delta_saved_size(desc: DeltaDesc) -> int:
    n = ctypes.c_size_t()
    _check(delta_lib().gl_delta_saved_size(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def delta_workspace_size(desc: DeltaDesc, have_saved: bool):
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(delta_lib().gl_delta_workspace_size(ctypes.byref(desc), int(have_saved), ctypes.byref(f),
                                               ctypes.byref(b)))
    return f.value, b.value


# ---------------------------------------------------------------- checks
def _on_gpu(tensors):
    device = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must be on a GPU device")
        if device is None:
            device = t.device
        elif t.device != device:
            raise ValueError("all tensors must be on one device")
    return device


def _rows(t, name):
    """Strides of a tensor whose last dimension is a row."""
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return _three(t.stride()[:-1], t.shape[:-1], name)


def _three(st, shape, name):
    st = [s if n > 1 else 0 for s, n in zip(st, shape)]
    if not any(st):
        if any(n > 1 for n in shape):
            raise ValueError(f"{name} is one row broadcast: make it contiguous")
        return Strides(64, 64, 64)  # one row: not used, but zeros would mean dense
    return Strides(*st)


def _empty_like_order(t, shape, dtype):
    """Empty [B,H,T,...] in t's order of heads and tokens."""
    torch = _torch()
    if len(shape) > 2 and t.dim() > 2 and t.shape[1] > 1 and t.shape[2] > 1 and t.stride(1) < t.stride(2):
        B, H, T = shape[:3]
        return torch.empty((B, T, H, *shape[3:]), dtype=dtype, device=t.device).transpose(1, 2)
    return torch.empty(shape, dtype=dtype, device=t.device)


class _On:
    """Makes the tensors' device current for the call."""

    def __init__(self, device):
        self.guard = None
        torch = _torch()
        if device.index is not None and device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(device)

    def __enter__(self):
        if self.guard:
            self.guard.__enter__()

    def __exit__(self, *e):
        if self.guard:
            self.guard.__exit__(*e)


def _delta_desc(q, k, v, log_alpha, beta, scale, state, cu, flags, segments):
    torch = _torch()
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[0] != q.shape[0] or v.shape[2] != q.shape[2]:
        raise ValueError("q, k must be [B,Hk,T,dk] and v [B,H,T,dv]")
    B, Hk, T, dk = q.shape
    H, dv = v.shape[1], v.shape[3]
    if tuple(log_alpha.shape) != (B, H, T) or tuple(beta.shape) != (B, H, T):
        raise ValueError("log_alpha and beta must be [B,H,T]")
    if q.dtype not in (torch.float64, torch.float32, torch.bfloat16):
        raise TypeError("q must be float64, float32 or bfloat16")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must share the io dtype")
    if log_alpha.dtype != beta.dtype or beta.dtype not in (q.dtype, gate_dtype(q.dtype)):
        raise TypeError(f"log_alpha and beta must both be {q.dtype} or {gate_dtype(q.dtype)}")
    _on_gpu((q, k, v, log_alpha, beta, state, cu))
    n = B
    if cu is not None:
        if cu.dtype != torch.int32 or cu.dim() != 1 or cu.numel() < 2 or not cu.is_contiguous():
            raise ValueError("cu_seqlens must be a contiguous int32 tensor of n + 1 >= 2 values")
        if B != 1:
            raise ValueError("packed sequences need B = 1")
        n = cu.numel() - 1
    _check_state(state, (n, H, dv, dk), q.dtype, "state")
    desc = make_delta_desc(B, T, H, Hk, dk, dv, _io_code(q.dtype), _io_code(beta.dtype),
                           n_seq=0 if cu is None else n, flags=flags, segments=segments,
                           scale=dk ** -0.5 if scale is None else scale)
    desc.sq, desc.sk, desc.sv = _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
    if log_alpha.stride() != beta.stride():
        raise ValueError("log_alpha and beta must have the same strides")
    desc.sg = _three(beta.stride(), beta.shape, "beta")
    return desc, n


def _check_state(t, shape, io, name):
    if t is None:
        return
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    if t.dtype != gate_dtype(io):
        raise TypeError(f"{name} must be {gate_dtype(io)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def gl_delta_fwd(q, k, v, log_alpha, beta, *, scale=None, state=None, want_state=False, save=False,
                 cu_seqlens=None, flags=0, segments=0):
    """Gated delta rule over whole sequences.  Returns (y, final state or None,
    saved or None).  scale: of y, 1/sqrt(dk) by default."""
    torch = _torch()
    desc, n = _delta_desc(q, k, v, log_alpha, beta, scale, state, cu_seqlens, flags, segments)
    L = delta_lib()
    B, H, T, dv = v.shape
    y = _empty_like_order(v, (B, H, T, dv), v.dtype)
    desc.sy = _rows(y, "y")
    out = torch.empty((n, H, dv, q.shape[3]), dtype=gate_dtype(q.dtype), device=q.device) if want_state else None
    saved = torch.empty(max(delta_saved_size(desc), 16), dtype=torch.uint8, device=q.device) if save else None
    need, _ = delta_workspace_size(desc, save)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    with _On(q.device):
        _check(L.gl_delta_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                              _ptr(state), _ptr(cu_seqlens), _ptr(y), _ptr(out), _ptr(saved), _ptr(ws), need,
                              _stream(q.device)))
    return y, out, saved


def gl_delta_bwd(q, k, v, log_alpha, beta, dy, saved=None, *, scale=None, state=None, dstate=None,
                 want_dstate=None, cu_seqlens=None, flags=0, segments=0):
    """Gradients for upstream dy [B,H,T,dv] and dstate (of the final state, or
    None).  Returns (dq, dk, dv, dlog_alpha, dbeta, dstate of the first state);
    the last is None unless `state` was given or want_dstate is true."""
    torch = _torch()
    desc, n = _delta_desc(q, k, v, log_alpha, beta, scale, state, cu_seqlens, flags, segments)
    L = delta_lib()
    B, H, T, dvv = v.shape
    if dy.shape != v.shape or dy.dtype != v.dtype:
        raise ValueError("dy must have the shape and dtype of v")
    _on_gpu((q, dy, dstate, saved))
    _check_state(dstate, (n, H, dvv, q.shape[3]), q.dtype, "dstate")
    dq, dk = _empty_like_order(q, q.shape, q.dtype), _empty_like_order(k, k.shape, k.dtype)
    dv = _empty_like_order(v, v.shape, v.dtype)
    dla, db = (torch.empty_strided(beta.shape, beta.stride(), dtype=beta.dtype, device=q.device)
               if _dense(beta) else torch.empty(beta.shape, dtype=beta.dtype, device=q.device) for _ in range(2))
    desc.sdq, desc.sdk, desc.sdv = _rows(dq, "dq"), _rows(dk, "dk"), _rows(dv, "dv")
    desc.sdy, desc.sdg = _rows(dy, "dy"), _three(db.stride(), db.shape, "dbeta")
    if want_dstate is None:
        want_dstate = state is not None
    ds = torch.empty((n, H, dvv, q.shape[3]), dtype=gate_dtype(q.dtype), device=q.device) if want_dstate else None
    _, need = delta_workspace_size(desc, saved is not None)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    with _On(q.device):
        _check(L.gl_delta_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                              _ptr(state), _ptr(cu_seqlens), _ptr(dy), _ptr(dstate), _ptr(saved), _ptr(dq),
                              _ptr(dk), _ptr(dv), _ptr(dla), _ptr(db), _ptr(ds), _ptr(ws), need,
                              _stream(q.device)))
    return dq, dk, dv, dla, db, ds


def _dense(t):
    """Whether t's elements fill its memory once in some order of its dimensions."""
    expect = 1
    for n, s in sorted(((n, s) for n, s in zip(t.shape, t.stride()) if n > 1), key=lambda x: x[1]):
        if s != expect:
            return False
        expect *= n
    return True


def gl_delta_step(q, k, v, log_alpha, beta, state, *, scale=None, slots=None, y=None):
    """One token of each row: q, k [B,Hk,dk], v [B,H,dv], gates [B,H]; `state`
    [n,H,dv,dk] is updated in place, row b's at slots[b] (int32; outside
    0..n-1: nothing to do, y = 0), or at b.  Returns y [B,H,dv]."""
    torch = _torch()
    if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[0] != q.shape[0] or state.dim() != 4:
        raise ValueError("q, k must be [B,Hk,dk], v [B,H,dv] and state [n,H,dv,dk]")
    B, Hk, dk = q.shape
    H, dv = v.shape[1:]
    if tuple(log_alpha.shape) != (B, H) or tuple(beta.shape) != (B, H):
        raise ValueError("log_alpha and beta must be [B,H]")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must share the io dtype")
    if log_alpha.dtype != beta.dtype or beta.dtype not in (q.dtype, gate_dtype(q.dtype)):
        raise TypeError(f"log_alpha and beta must both be {q.dtype} or {gate_dtype(q.dtype)}")
    _check_state(state, (state.shape[0], H, dv, dk), q.dtype, "state")
    if slots is None:
        if state.shape[0] < B:
            raise ValueError(f"{state.shape[0]} states for {B} rows")
    elif slots.dtype != torch.int32 or tuple(slots.shape) != (B,) or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous int32 tensor [B]")
    if y is None:
        y = torch.empty((B, H, dv), dtype=v.dtype, device=v.device)
    elif tuple(y.shape) != (B, H, dv) or y.dtype != v.dtype:
        raise ValueError("y must be [B,H,dv] of v's dtype")
    _on_gpu((q, k, v, log_alpha, beta, state, slots, y))
    if log_alpha.stride() != beta.stride():
        raise ValueError("log_alpha and beta must have the same strides")
    desc = make_delta_desc(B, 1, H, Hk, dk, dv, _io_code(q.dtype), _io_code(beta.dtype),
                           scale=dk ** -0.5 if scale is None else scale)
    desc.sq, desc.sk, desc.sv, desc.sy = _rows(q, "q"), _rows(k, "k"), _rows(v, "v"), _rows(y, "y")
    desc.sg = _three(beta.stride(), beta.shape, "beta")
    with _On(q.device):
        _check(delta_lib().gl_delta_step(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                         _ptr(slots), state.shape[0], _ptr(state), _ptr(y), _stream(q.device)))
    return y


# ---------------------------------------------------------------- norms and rotation
def _qk_desc(q, k, wq, wk, cos, sin, pos, pos0, eps, q_scale, k_scale, interleaved):
    torch = _torch()
    if q.dim() != 4 or k.dim() != 4 or q.shape[0] != k.shape[0] or q.shape[2:] != k.shape[2:]:
        raise ValueError("q must be [B,Hq,T,d] and k [B,Hk,T,d]")
    B, Hq, T, d = q.shape
    if q.dtype not in (torch.float64, torch.float32, torch.bfloat16) or k.dtype != q.dtype:
        raise TypeError("q and k must share float64, float32 or bfloat16")
    for w in (wq, wk):
        if w is not None and (tuple(w.shape) != (d,) or w.dtype != q.dtype or not w.is_contiguous()):
            raise ValueError("wq and wk must be contiguous [d] of q's dtype")
    rot, n_pos = 0, 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None:
        if cos.dim() != 2 or cos.shape != sin.shape or not cos.is_contiguous() or not sin.is_contiguous():
            raise ValueError("cos and sin must be contiguous [n_pos, rot/2]")
        if cos.dtype != gate_dtype(q.dtype) or sin.dtype != cos.dtype:
            raise TypeError(f"cos and sin must be {gate_dtype(q.dtype)}")
        n_pos, rot = cos.shape[0], 2 * cos.shape[1]
    if pos is not None and (pos.dtype != torch.int32 or tuple(pos.shape) != (B, T) or not pos.is_contiguous()):
        raise ValueError("pos must be a contiguous int32 tensor [B,T]")
    _on_gpu((q, k, wq, wk, cos, sin, pos))
    desc = QkDesc(B, T, Hq, k.shape[1], d, rot, n_pos, pos0, _io_code(q.dtype),
                  GL_FLAG_INTERLEAVED if interleaved else 0, eps, q_scale, k_scale)
    desc.sq, desc.sk = _rows(q, "q"), _rows(k, "k")
    return desc


def gl_qknorm_rope_fwd(q, k, wq=None, wk=None, cos=None, sin=None, *, pos=None, pos0=0, eps=1e-6,
                       q_scale=1.0, k_scale=1.0, interleaved=False):
    """Root-mean-square norm of every head's row of q [B,Hq,T,d] and k
    [B,Hk,T,d], weights wq, wk [d], and the rotation by the tables cos, sin
    [n_pos, rot/2] at pos [B,T] (or pos0 + t).  Returns the two results, dense
    [B,H,T,d] (what gl_delta_fwd reads row after row)."""
    torch = _torch()
    desc = _qk_desc(q, k, wq, wk, cos, sin, pos, pos0, eps, q_scale, k_scale, interleaved)
    oq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    ok = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    with _On(q.device):
        _check(delta_lib().gl_qknorm_rope_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(cos),
                                              _ptr(sin), _ptr(pos), _ptr(oq), _ptr(ok), _stream(q.device)))
    return oq, ok


def gl_qknorm_rope_bwd(q, k, wq, wk, cos, sin, dqn, dkn, *, pos=None, pos0=0, eps=1e-6, q_scale=1.0,
                       k_scale=1.0, interleaved=False):
    """Gradients of gl_qknorm_rope_fwd for upstream dqn, dkn: (dq, dk, dwq,
    dwk), dq and dk in their inputs' order of dimensions, dwq and dwk [d] in
    fp32 (fp64), None where there is no weight."""
    torch = _torch()
    desc = _qk_desc(q, k, wq, wk, cos, sin, pos, pos0, eps, q_scale, k_scale, interleaved)
    if dqn.shape != q.shape or dkn.shape != k.shape or dqn.dtype != q.dtype or dkn.dtype != k.dtype:
        raise ValueError("dqn and dkn must have the shapes and dtype of q and k")
    _on_gpu((q, dqn, dkn))
    dq, dk = _empty_like_order(q, q.shape, q.dtype), _empty_like_order(k, k.shape, k.dtype)
    desc.sdoq, desc.sdok, desc.sdq, desc.sdk = (_rows(dqn, "dqn"), _rows(dkn, "dkn"), _rows(dq, "dq"),
                                                _rows(dk, "dk"))
    gd = gate_dtype(q.dtype)
    dwq, dwk = (None if w is None else torch.empty(w.shape, dtype=gd, device=q.device) for w in (wq, wk))
    n = ctypes.c_size_t()
    _check(delta_lib().gl_qknorm_rope_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    ws = torch.empty(max(n.value, 16), dtype=torch.uint8, device=q.device)
    with _On(q.device):
        _check(delta_lib().gl_qknorm_rope_bwd(
            ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(cos), _ptr(sin), _ptr(pos), _ptr(dqn),
            _ptr(dkn), _ptr(dq), _ptr(dk), _ptr(dwq), _ptr(dwk), _ptr(ws), n.value, _stream(q.device)))
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------- autograd
def _make_functions():
    torch = _torch()

    class DeltaRule(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, log_alpha, beta, state, scale, cu_seqlens, want_state):
            y, out, saved = gl_delta_fwd(q, k, v, log_alpha, beta, scale=scale, state=state,
                                         want_state=want_state, save=True, cu_seqlens=cu_seqlens)
            ctx.save_for_backward(q, k, v, log_alpha, beta, state, cu_seqlens, saved)
            ctx.scale = scale
            return y, out

        @staticmethod
        def backward(ctx, dy, dstate):
            q, k, v, log_alpha, beta, state, cu_seqlens, saved = ctx.saved_tensors
            grads = gl_delta_bwd(q, k, v, log_alpha, beta, dy.contiguous(), saved, scale=ctx.scale, state=state,
                                 dstate=None if dstate is None else dstate.contiguous(), cu_seqlens=cu_seqlens)
            return (*grads, None, None, None)

    class QkNormRope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, wq, wk, cos, sin, pos, opts):
            ctx.save_for_backward(q, k, wq, wk, cos, sin, pos)
            ctx.opts = opts
            return gl_qknorm_rope_fwd(q, k, wq, wk, cos, sin, pos=pos, **opts)

        @staticmethod
        def backward(ctx, dqn, dkn):
            q, k, wq, wk, cos, sin, pos = ctx.saved_tensors
            dq, dk, dwq, dwk = gl_qknorm_rope_bwd(q, k, wq, wk, cos, sin, dqn.contiguous(), dkn.contiguous(),
                                                  pos=pos, **ctx.opts)
            dwq, dwk = (None if g is None else g.to(w.dtype) for g, w in ((dwq, wq), (dwk, wk)))
            return dq, dk, dwq, dwk, None, None, None, None

    return DeltaRule, QkNormRope


_fns = None


def _functions():
    global _fns
    if _fns is None:
        _fns = _make_functions()
    return _fns


def delta_rule(q, k, v, log_alpha, beta, *, scale=None, state=None, cu_seqlens=None, want_state=False):
    """Autograd-aware gl_delta_fwd: (y, final state or None)."""
    return _functions()[0].apply(q, k, v, log_alpha, beta, state, scale, cu_seqlens, want_state)


def qknorm_rope(q, k, wq=None, wk=None, cos=None, sin=None, *, pos=None, pos0=0, eps=1e-6, q_scale=1.0,
                k_scale=1.0, interleaved=False):
    """Autograd-aware gl_qknorm_rope_fwd."""
    opts = dict(pos0=pos0, eps=eps, q_scale=q_scale, k_scale=k_scale, interleaved=interleaved)
    return _functions()[1].apply(q, k, wq, wk, cos, sin, pos, opts)
