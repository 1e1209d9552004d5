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

from . import GLScanError, _io_code, _torch, gate_dtype
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


_KINDS = {"gl_delta_fwd": 0, "gl_delta_bwd": 1, "gl_delta_step": 2, "gl_qknorm_rope_fwd": 3, "gl_qknorm_rope_bwd": 4}
_calls: dict = {}


def _run(name, numbers, tensors, plan, pos0=0):
    """Calls `name` of the library on `tensors` on the current stream and returns
    its outputs.  `plan` checks the tensors and returns (descriptor, workspace
    bytes, count, outputs); it runs where no call of the same numbers, shapes,
    strides, types and devices came before: a decoding loop makes thousands of
    one kind, and the checks cost more than the launch."""
    calls = _calls.get((name, numbers))
    if calls is None:
        from . import _fastcall  # needs torch to be imported
        fn = ctypes.cast(getattr(delta_lib(), name), ctypes.c_void_p).value
        calls = _fastcall.Calls(_KINDS[name], fn)
        if len(_calls) >= 256:
            _calls.clear()
        _calls[name, numbers] = calls
    index = tensors[0].get_device()
    if index < 0:
        plan()
        raise ValueError("all tensors must be on a GPU device")
    stream = _torch()._C._cuda_getCurrentRawStream(index)
    out = calls.call(stream, pos0, *tensors)
    if out is None:
        desc, ws, count, outputs = plan()
        calls.record(desc, ctypes.addressof(desc), ws, count, outputs, *tensors)
        out = calls.call(stream, pos0, *tensors)
    if type(out) is not tuple:
        _check(out)
    return out


def _strides_like(t, shape):
    """Strides of an output of `shape` [B,H,T,...] in t's order of heads and tokens."""
    st = [1]
    for n in reversed(shape[1:]):
        st.append(st[-1] * max(n, 1))
    st.reverse()
    if len(shape) > 2 and t.dim() > 2 and t.shape[1] > 1 and t.shape[2] > 1 and t.stride(1) < t.stride(2):
        row = st[2]
        st[1], st[2] = row, row * shape[1]
    return tuple(st)


def _with(desc, name, shape, strides):
    setattr(desc, name, _three(strides[:3], shape[:3], name))


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
    desc.sg = _gate_strides(log_alpha, beta)
    return desc, n


def _moves(t):
    """t's strides in the dimensions that have any: those of one element say nothing."""
    return [s for s, n in zip(t.stride(), t.shape) if n > 1]


def _gate_strides(log_alpha, beta):
    if _moves(log_alpha) != _moves(beta):
        raise ValueError("log_alpha and beta must have the same strides")
    return _three(beta.stride(), beta.shape, "beta")


def _check_state(t, shape, io, name):
    if t is None:
        return
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    if t.dtype != gate_dtype(io):
        raise TypeError(f"{name} must be {gate_dtype(io)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _contiguous(shape, dtype):
    """Output of _run: dense, of shape."""
    st = [1]
    for n in reversed(shape[1:]):
        st.append(st[-1] * max(n, 1))
    return tuple(shape), tuple(reversed(st)), dtype


def _num(x):
    """A scale or eps as the number it is now.  One that is a tensor would be remembered
    by which tensor it is (calls of one kind are found by their numbers)."""
    return x if x is None or type(x) is float else float(x)


def gl_delta_fwd(q, k, v, log_alpha, beta, *, scale=None, state=None, want_state=False, save=False,
                 cu_seqlens=None, flags=0, segments=0):
    """Gated delta rule over whole sequences.  Returns (y, final state or None,
    saved or None).  scale: of y, 1/sqrt(dk) by default."""
    scale = _num(scale)

    def plan():
        desc, n = _delta_desc(q, k, v, log_alpha, beta, scale, state, cu_seqlens, flags, segments)
        shape, strides = tuple(v.shape), _strides_like(v, v.shape)
        _with(desc, "sy", shape, strides)
        return desc, delta_workspace_size(desc, save)[0], 0, (
            (shape, strides, v.dtype),
            _contiguous((n, v.shape[1], v.shape[3], q.shape[3]), gate_dtype(q.dtype)) if want_state else None,
            _contiguous((max(delta_saved_size(desc), 16),), _torch().uint8) if save else None)
    return _run("gl_delta_fwd", (scale, bool(want_state), bool(save), flags, segments),
                (q, k, v, log_alpha, beta, state, cu_seqlens), plan)


def gl_delta_bwd(q, k, v, log_alpha, beta, dy, saved=None, *, scale=None, state=None, dstate=None,
                 want_dstate=None, cu_seqlens=None, flags=0, segments=0):
    """Gradients for upstream dy [B,H,T,dv] and dstate (of the final state, or
    None).  Returns (dq, dk, dv, dlog_alpha, dbeta, dstate of the first state);
    the last is None unless `state` was given or want_dstate is true."""
    if want_dstate is None:
        want_dstate = state is not None
    scale = _num(scale)

    def plan():
        desc, n = _delta_desc(q, k, v, log_alpha, beta, scale, state, cu_seqlens, flags, segments)
        if dy.shape != v.shape or dy.dtype != v.dtype:
            raise ValueError("dy must have the shape and dtype of v")
        _on_gpu((q, dy, dstate, saved))
        states = _contiguous((n, v.shape[1], v.shape[3], q.shape[3]), gate_dtype(q.dtype))
        _check_state(dstate, states[0], q.dtype, "dstate")
        if saved is not None and (saved.dtype != _torch().uint8 or not saved.is_contiguous()
                                  or saved.numel() < delta_saved_size(desc)):
            raise ValueError("saved must be what gl_delta_fwd returned for these inputs")
        outs = []
        for name, t in (("sdq", q), ("sdk", k), ("sdv", v), ("sdg", log_alpha), ("sdg", beta)):
            st = tuple(t.stride()) if t.dim() == 3 and _dense(t) else _strides_like(t, t.shape)
            outs.append((tuple(t.shape), st, t.dtype))
            _with(desc, name, t.shape, st)
        desc.sdy = _rows(dy, "dy")
        return (desc, delta_workspace_size(desc, saved is not None)[1], 0,
                (*outs, states if want_dstate else None))
    return _run("gl_delta_bwd", (scale, bool(want_dstate), flags, segments),
                (q, k, v, log_alpha, beta, state, cu_seqlens, dy, dstate, saved), plan)


def _dense(t):
    """Whether t's elements fill its memory once in some order of its dimensions."""
    expect = 1
    for n, s in sorted(((n, s) for n, s in zip(t.shape, t.stride()) if n > 1), key=lambda x: x[1]):
        if s != expect:
            return False
        expect *= n
    return t.numel() > 0


def gl_delta_step(q, k, v, log_alpha, beta, state, *, scale=None, slots=None, y=None):
    """One token of each row: q, k [B,Hk,dk], v [B,H,dv], gates [B,H]; `state`
    [n,H,dv,dk] is updated in place, row b's at slots[b] (int32; outside
    0..n-1: nothing to do, y = 0), or at b.  Returns y [B,H,dv]."""
    scale = _num(scale)

    def plan():
        torch = _torch()
        if q.dim() != 3 or k.shape != q.shape or v.dim() != 3 or v.shape[0] != q.shape[0] or state.dim() != 4:
            raise ValueError("q, k must be [B,Hk,dk], v [B,H,dv] and state [n,H,dv,dk]")
        B, Hk, dk = q.shape
        H, dv = v.shape[1:]
        if tuple(log_alpha.shape) != (B, H) or tuple(beta.shape) != (B, H):
            raise ValueError("log_alpha and beta must be [B,H]")
        if q.dtype not in (torch.float64, torch.float32, torch.bfloat16):
            raise TypeError("q must be float64, float32 or bfloat16")
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
        if y is not None and (tuple(y.shape) != (B, H, dv) or y.dtype != v.dtype):
            raise ValueError("y must be [B,H,dv] of v's dtype")
        _on_gpu((q, k, v, log_alpha, beta, state, slots, y))
        desc = make_delta_desc(B, 1, H, Hk, dk, dv, _io_code(q.dtype), _io_code(beta.dtype),
                               scale=dk ** -0.5 if scale is None else scale)
        desc.sq, desc.sk, desc.sv = _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
        desc.sy = _three((H * dv, dv), (B, H), "y") if y is None else _rows(y, "y")
        desc.sg = _gate_strides(log_alpha, beta)
        return desc, 0, state.shape[0], (_contiguous((B, H, dv), v.dtype) if y is None else None,)
    out = _run("gl_delta_step", scale, (q, k, v, log_alpha, beta, slots, state, y), plan)[0]
    return out if y is None else y


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
    eps, q_scale, k_scale = _num(eps), _num(q_scale), _num(k_scale)

    def plan():
        desc = _qk_desc(q, k, wq, wk, cos, sin, pos, pos0, eps, q_scale, k_scale, interleaved)
        return desc, 0, 0, (_contiguous(q.shape, q.dtype), _contiguous(k.shape, q.dtype))
    return _run("gl_qknorm_rope_fwd", (eps, q_scale, k_scale, bool(interleaved)), (q, k, wq, wk, cos, sin, pos), plan,
                pos0)


def gl_qknorm_rope_bwd(q, k, wq, wk, cos, sin, dqn, dkn, *, pos=None, pos0=0, eps=1e-6, q_scale=1.0,
                       k_scale=1.0, interleaved=False):
    """Gradients of gl_qknorm_rope_fwd for upstream dqn, dkn: (dq, dk, dwq,
    dwk), dq and dk in their inputs' order of dimensions, dwq and dwk [d] in
    fp32 (fp64), None where there is no weight."""
    eps, q_scale, k_scale = _num(eps), _num(q_scale), _num(k_scale)

    def plan():
        desc = _qk_desc(q, k, wq, wk, cos, sin, pos, pos0, eps, q_scale, k_scale, interleaved)
        if dqn.shape != q.shape or dkn.shape != k.shape or dqn.dtype != q.dtype or dkn.dtype != k.dtype:
            raise ValueError("dqn and dkn must have the shapes and dtype of q and k")
        _on_gpu((q, dqn, dkn))
        sq, sk = _strides_like(q, q.shape), _strides_like(k, k.shape)
        desc.sdoq, desc.sdok = _rows(dqn, "dqn"), _rows(dkn, "dkn")
        _with(desc, "sdq", q.shape, sq)
        _with(desc, "sdk", k.shape, sk)
        n = ctypes.c_size_t()
        _check(delta_lib().gl_qknorm_rope_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
        dw = gate_dtype(q.dtype)
        return desc, max(n.value, 16), 0, (
            (tuple(q.shape), sq, q.dtype), (tuple(k.shape), sk, q.dtype),
            None if wq is None else _contiguous(wq.shape, dw), None if wk is None else _contiguous(wk.shape, dw))
    return _run("gl_qknorm_rope_bwd", (eps, q_scale, k_scale, bool(interleaved)),
                (q, k, wq, wk, cos, sin, pos, dqn, dkn), plan, pos0)


# ---------------------------------------------------------------- autograd
def _aligned(t):
    """t if it begins on 16 bytes, else a dense copy (contiguous() would return a
    dense slice of a longer tensor as it is)."""
    return t if t.data_ptr() % 16 == 0 else t.clone(memory_format=_torch().contiguous_format)


def _whole(t):
    """t as it is if it is dense in some order of its heads and tokens and begins on
    16 bytes, else a dense copy."""
    return _aligned(t if _dense(t) and t.stride(-1) == 1 else t.contiguous())


def _make_functions():
    torch = _torch()
    # the kernels leave no graph behind: gradients of gradients are refused, not lost
    once = torch.autograd.function.once_differentiable

    class DeltaRule(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, log_alpha, beta, state, scale, cu_seqlens, want_state):
            y, out, saved = gl_delta_fwd(q, k, v, log_alpha, beta, scale=scale, state=state,
                                         want_state=want_state, save=True, cu_seqlens=cu_seqlens)
            ctx.save_for_backward(q, k, v, log_alpha, beta, state, cu_seqlens, saved)
            ctx.scale = scale
            return y, out

        @staticmethod
        @once
        def backward(ctx, dy, dstate):
            q, k, v, log_alpha, beta, state, cu_seqlens, saved = ctx.saved_tensors
            dstate = None if dstate is None else _aligned(dstate.contiguous())
            grads = gl_delta_bwd(q, k, v, log_alpha, beta, _whole(dy), saved, scale=ctx.scale, state=state,
                                 dstate=dstate, cu_seqlens=cu_seqlens)
            return (*grads, None, None, None)

    class QkNormRope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, wq, wk, cos, sin, pos, opts):
            ctx.save_for_backward(q, k, wq, wk, cos, sin, pos)
            ctx.opts = opts
            return gl_qknorm_rope_fwd(q, k, wq, wk, cos, sin, pos=pos, **opts)

        @staticmethod
        @once
        def backward(ctx, dqn, dkn):
            q, k, wq, wk, cos, sin, pos = ctx.saved_tensors
            dq, dk, dwq, dwk = gl_qknorm_rope_bwd(q, k, wq, wk, cos, sin, _whole(dqn), _whole(dkn), pos=pos,
                                                  **ctx.opts)
            dwq, dwk = (None if g is None else g.to(w.dtype) for g, w in ((dwq, wq), (dwk, wk)))
            return dq, dk, dwq, dwk, None, None, None, None

    return DeltaRule, QkNormRope


_fns = None


def _functions():
    global _fns
    if _fns is None:
        _fns = _make_functions()
    return _fns


def _no_duals(inputs):
    """Refuses dual tensors: they want a forward-mode derivative, which there is not."""
    forward_ad = _torch().autograd.forward_ad
    if forward_ad._current_level >= 0 and any(
            t is not None and forward_ad.unpack_dual(t).tangent is not None for t in inputs):
        raise NotImplementedError("the delta rule has no forward-mode derivative")


def _no_gradient(error, names, *values):
    """Refuses what wants a gradient that the functions do not form."""
    torch = _torch()
    if torch.is_grad_enabled():
        for x in values:
            if torch.is_tensor(x) and x.requires_grad:
                raise error(f"no gradient is formed for {names}: detach it")


def delta_rule(q, k, v, log_alpha, beta, *, scale=None, state=None, cu_seqlens=None, want_state=False):
    """Autograd-aware gl_delta_fwd: (y, final state or None).  Nothing is kept
    for a backward where no gradient is wanted.  Gates of different strides are
    copied into one order, a state that is broadcast or does not begin on 16 bytes
    into one that is and does, and so are q, k, v that do not in training."""
    _no_gradient(TypeError, "scale", scale)
    if log_alpha.shape == beta.shape and (log_alpha.stride() != beta.stride() or 0 in beta.stride()):
        order = _moves(log_alpha)
        if order != _moves(beta) or not any(order):  # one order for both; one number for all written out
            log_alpha, beta = log_alpha.contiguous(), beta.contiguous()
    if state is not None:
        state = _aligned(state.contiguous())
    inputs = (q, k, v, log_alpha, beta, state)
    _no_duals(inputs)
    if not (_torch().is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs)):
        return gl_delta_fwd(q, k, v, log_alpha, beta, scale=scale, state=state, want_state=want_state,
                            cu_seqlens=cu_seqlens)[:2]
    # slices that begin between two 16-byte units: training wants them aligned
    q, k, v = (_aligned(t) for t in (q, k, v))
    return _functions()[0].apply(q, k, v, log_alpha, beta, state, _num(scale), cu_seqlens, want_state)


def qknorm_rope(q, k, wq=None, wk=None, cos=None, sin=None, *, pos=None, pos0=0, eps=1e-6, q_scale=1.0,
                k_scale=1.0, interleaved=False):
    """Autograd-aware gl_qknorm_rope_fwd."""
    _no_gradient(TypeError, "the scales and eps", q_scale, k_scale, eps)
    _no_gradient(ValueError, "cos and sin", cos, sin)
    opts = dict(pos0=int(pos0), eps=_num(eps), q_scale=_num(q_scale), k_scale=_num(k_scale), interleaved=interleaved)
    return _functions()[1].apply(q, k, wq, wk, cos, sin, pos, opts)
