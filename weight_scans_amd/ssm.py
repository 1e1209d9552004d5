"""The selective state space scan, the short causal convolution before it and the
norms before and after a block: torch tensors into the C ABI of
``include/gl_ssm.h`` (no compute here).

    y, state = gl_conv_fwd(x, w, bias, state=S0, want_state=True)
    dx, dw, dbias, dS0 = gl_conv_bwd(x, w, bias, dy, state=S0, ...)
    y1 = gl_conv_step(x1, w, bias, state)                    # one token, state in place
    y, state = causal_conv(x, w, bias)                        # autograd-aware
    y, state, saved = gl_ssm_fwd(x, dt, A, B, C, skip, z, dt_bias, state=S0, save=True)
    dx, ddt, dA, dB, dC, dskip, dz, ddt_bias, dS0 = gl_ssm_bwd(x, dt, ..., dy, saved, ...)
    y1 = gl_ssm_step(x1, dt1, A, B1, C1, skip, z1, dt_bias, state)
    y, state = selective_scan(x, dt, A, B, C, skip, z, dt_bias)   # autograd-aware
    n, r_out = gl_addnorm_fwd(x, r, w, wx, scale)             # r + scale * norm(x), and its norm
    dx, dr, dw, dwx, dscale = gl_addnorm_bwd(x, r, w, wx, scale, dn, dr_out)
    n, r_out = add_norm(x, r, w, wx, scale)                   # autograd-aware
    y = gl_gatenorm_fwd(x, z, w)                              # norm(x) * silu(z)
    dx, dz, dw = gl_gatenorm_bwd(x, z, w, dy)
    y = gated_norm(x, z, w)                                   # autograd-aware

Shapes: rows x, dt, z, y [B,T,D]; B, C [B,T,G,N] (channel d reads group
d / (D / G)) or [B,T,N]; A [D,N], skip, dt_bias [D]; convolution weights [D,K];
states [B,D,N] of the scan and [B,K-1,D] (the last inputs, oldest first) of the
convolution; with cu_seqlens [n + 1] (int32, on the device) B is 1 and there are
n states, and tokens behind the last sequence add nothing: outputs and gradients
are zero there.  A, skip, dt_bias and the scan's states are fp32 (fp64 for fp64 io),
all others of the io dtype; the residual of add_norm is either.  Tensors of rows
may be views with any strides whose last dimension is contiguous (slices of a
fused projection); outputs are dense.
"""
from __future__ import annotations

import ctypes

from . import _io_code, _torch, gate_dtype
from . import lib as _load
from .delta import _check, _contiguous, _no_gradient, _num, _on_gpu, _run

SSM_EXPORTS = (
    "gl_conv_fwd",
    "gl_conv_workspace_size",
    "gl_conv_bwd",
    "gl_conv_step",
    "gl_ssm_saved_size",
    "gl_ssm_workspace_size",
    "gl_ssm_fwd",
    "gl_ssm_bwd",
    "gl_ssm_step",
    "gl_addnorm_fwd",
    "gl_addnorm_workspace_size",
    "gl_addnorm_bwd",
    "gl_gatenorm_fwd",
    "gl_gatenorm_workspace_size",
    "gl_gatenorm_bwd",
)

GL_FLAG_SILU, GL_FLAG_SOFTPLUS = 16, 32
GL_FLAG_GATE_FIRST, GL_FLAG_GROUP_WEIGHTS = 64, 128


class Rows(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("t", ctypes.c_int64), ("g", ctypes.c_int64)]


def _fields(numbers, strides, extra=()):
    return ([(n, ctypes.c_int64) for n in numbers] + [("io_dtype", ctypes.c_int32)] + list(extra) +
            [(n, Rows) for n in strides])


class ConvDesc(ctypes.Structure):
    _fields_ = _fields(("B", "T", "D", "K", "n_seq"), ("sx", "sy", "sdy", "sdx"), [("flags", ctypes.c_uint32)])


class SsmDesc(ctypes.Structure):
    _fields_ = _fields(("B", "T", "D", "N", "G", "n_seq"),
                       ("sx", "sdt", "sz", "sB", "sC", "sy", "sdy", "sdx", "sddt", "sdz", "sdB", "sdC"),
                       [("flags", ctypes.c_uint32)])


class AddNormDesc(ctypes.Structure):
    _fields_ = _fields(("B", "T", "d"), ("sx", "sr", "sn", "sro", "sdn", "sdro", "sdx", "sdr"),
                       [("res_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
                        ("eps", ctypes.c_double)])


class GateNormDesc(ctypes.Structure):
    _fields_ = _fields(("B", "T", "G", "d"), ("sx", "sz", "sy", "sdy", "sdx", "sdz"),
                       [("flags", ctypes.c_uint32), ("eps", ctypes.c_double)])


_lib = None


def ssm_lib():
    """libglscan.so with the argument types of gl_ssm.h set."""
    global _lib
    if _lib is None:
        L = _load()
        P, S, I64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
        pc, pm, pa, pg = (ctypes.POINTER(c) for c in (ConvDesc, SsmDesc, AddNormDesc, GateNormDesc))
        ps = ctypes.POINTER(ctypes.c_size_t)
        L.gl_conv_fwd.argtypes = [pc] + [P] * 8
        L.gl_conv_workspace_size.argtypes = [pc, ps]
        L.gl_conv_bwd.argtypes = [pc] + [P] * 12 + [S, P]
        L.gl_conv_step.argtypes = [pc] + [P] * 4 + [I64] + [P] * 3
        L.gl_ssm_saved_size.argtypes = [pm, ps]
        L.gl_ssm_workspace_size.argtypes = [pm, ctypes.c_int, ps, ps]
        L.gl_ssm_fwd.argtypes = [pm] + [P] * 14 + [S, P]
        L.gl_ssm_bwd.argtypes = [pm] + [P] * 23 + [S, P]
        L.gl_ssm_step.argtypes = [pm] + [P] * 9 + [I64] + [P] * 3
        L.gl_addnorm_fwd.argtypes = [pa] + [P] * 8
        L.gl_addnorm_workspace_size.argtypes = [pa, ps]
        L.gl_addnorm_bwd.argtypes = [pa] + [P] * 13 + [S, P]
        L.gl_gatenorm_fwd.argtypes = [pg] + [P] * 5
        L.gl_gatenorm_workspace_size.argtypes = [pg, ps]
        L.gl_gatenorm_bwd.argtypes = [pg] + [P] * 8 + [S, P]
        for n in SSM_EXPORTS:
            getattr(L, n).restype = ctypes.c_int
        _lib = L
    return _lib


def _size(name, desc):
    n = ctypes.c_size_t()
    _check(getattr(ssm_lib(), name)(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def ssm_workspace_size(desc: SsmDesc, have_saved: bool):
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(ssm_lib().gl_ssm_workspace_size(ctypes.byref(desc), int(have_saved), ctypes.byref(f), ctypes.byref(b)))
    return f.value, b.value


# ---------------------------------------------------------------- checks
def _rows(t, name, lead=2):
    """Strides of [B,T,..] or [B,T,G,..] (lead = 3), of [B,..] and [B,G,..] (one token)
    whose last dimension is a row."""
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    st = [s if n > 1 else 0 for s, n in zip(t.stride()[:-1], t.shape[:-1])]
    if not any(st):
        if any(n > 1 for n in t.shape[:-1]):
            raise ValueError(f"{name} is one row broadcast: make it contiguous")
        return Rows(64, 64, 64)  # one row: not used, but zeros would mean dense
    if lead == 2:
        return Rows(st[0], st[1] if len(st) > 1 else 0, 0)
    return Rows(st[0], st[1], st[2]) if len(st) == 3 else Rows(st[0], 0, st[1])


def _io(x, *others):
    torch = _torch()
    if x.dtype not in (torch.float64, torch.float32, torch.bfloat16):
        raise TypeError("x must be float64, float32 or bfloat16")
    for t in others:
        if t is not None and t.dtype != x.dtype:
            raise TypeError(f"tensors of the io dtype must all be {x.dtype}")
    return _io_code(x.dtype)


def _dense(t, shape, dtype, name):
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _same(t, x, name):
    if t is None:
        return
    if t.shape != x.shape:
        raise ValueError(f"{name} must be {list(x.shape)}")
    if t.dtype != x.dtype:
        raise TypeError(f"{name} must be {x.dtype}")


def _sequences(cu, B):
    """Number of packed sequences (0: none) and of states."""
    if cu is None:
        return 0, B
    torch = _torch()
    if cu.dtype != torch.int32 or cu.dim() != 1 or cu.numel() < 2 or not cu.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous int32 tensor of n + 1 >= 2 values")
    if B != 1:
        raise ValueError("packed sequences need B = 1")
    return cu.numel() - 1, cu.numel() - 1


def _slots(slots, B, state):
    if slots is None:
        if state.shape[0] < B:
            raise ValueError(f"{state.shape[0]} states for {B} rows")
    elif slots.dtype != _torch().int32 or tuple(slots.shape) != (B,) or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous int32 tensor [B]")


def _out(t):
    return _contiguous(tuple(t.shape), t.dtype)


# ---------------------------------------------------------------- convolution
def _conv_desc(x, w, bias, state, cu, silu):
    if x.dim() != 3 or w.dim() != 2 or w.shape[0] != x.shape[2]:
        raise ValueError("x must be [B,T,D] and w [D,K]")
    io = _io(x)
    B, T, D = x.shape
    K = w.shape[1]
    _dense(w, (D, K), x.dtype, "w")
    _dense(bias, (D,), x.dtype, "bias")
    n_seq, n = _sequences(cu, B)
    _dense(state, (n, max(K - 1, 0), D), x.dtype, "state")
    _on_gpu((x, w, bias, state, cu))
    desc = ConvDesc(B, T, D, K, n_seq, io, GL_FLAG_SILU if silu else 0)
    desc.sx = _rows(x, "x")
    return desc, n


def gl_conv_fwd(x, w, bias=None, *, state=None, want_state=False, cu_seqlens=None, silu=True):
    """Causal convolution of x [B,T,D] with w [D,K], its bias and SiLU.  Returns
    (y, the last K - 1 inputs of each sequence [n,K-1,D] or None)."""
    def plan():
        desc, n = _conv_desc(x, w, bias, state, cu_seqlens, silu)
        return desc, 0, 0, (_out(x), _contiguous((n, w.shape[1] - 1, x.shape[2]), x.dtype) if want_state else None)
    return _run("gl_conv_fwd", (bool(want_state), bool(silu)), (x, w, bias, state, cu_seqlens), plan)


def gl_conv_bwd(x, w, bias, dy, *, state=None, dstate=None, want_dstate=None, cu_seqlens=None, silu=True):
    """Gradients for upstream dy [B,T,D] and dstate (of the last inputs, or None).
    Returns (dx, dw, dbias, dstate of the first state): dw [D,K] and dbias [D] in
    fp32 (fp64), dbias None without a bias, the last None unless `state` was given
    or want_dstate is true."""
    if want_dstate is None:
        want_dstate = state is not None

    def plan():
        desc, n = _conv_desc(x, w, bias, state, cu_seqlens, silu)
        _same(dy, x, "dy")
        states = _contiguous((n, w.shape[1] - 1, x.shape[2]), x.dtype)
        _dense(dstate, states[0], x.dtype, "dstate")
        _on_gpu((x, dy, dstate))
        desc.sdy = _rows(dy, "dy")
        par = gate_dtype(x.dtype)
        return desc, max(_size("gl_conv_workspace_size", desc), 16), 0, (
            _out(x), _contiguous(tuple(w.shape), par), None if bias is None else _contiguous(tuple(bias.shape), par),
            states if want_dstate else None)
    return _run("gl_conv_bwd", (bool(want_dstate), bool(silu)), (x, w, bias, state, cu_seqlens, dy, dstate), plan)


def gl_conv_step(x, w, bias, state, *, slots=None, silu=True):
    """One token of each row, x [B,D]: `state` [n,K-1,D] moves on by one input in
    place, row b's at slots[b] (int32; outside 0..n-1: nothing to do, y = 0), or at
    b.  Returns y [B,D]."""
    def plan():
        if x.dim() != 2 or w.dim() != 2 or w.shape[0] != x.shape[1] or state.dim() != 3:
            raise ValueError("x must be [B,D], w [D,K] and state [n,K-1,D]")
        io = _io(x)
        B, D = x.shape
        _dense(w, tuple(w.shape), x.dtype, "w")
        _dense(bias, (D,), x.dtype, "bias")
        _dense(state, (state.shape[0], w.shape[1] - 1, D), x.dtype, "state")
        _slots(slots, B, state)
        _on_gpu((x, w, bias, state, slots))
        desc = ConvDesc(B, 1, D, w.shape[1], 0, io, GL_FLAG_SILU if silu else 0)
        desc.sx = _rows(x, "x")
        return desc, 0, state.shape[0], (_out(x),)
    return _run("gl_conv_step", bool(silu), (x, w, bias, slots, state), plan)[0]


# ---------------------------------------------------------------- selective scan
def _ssm_desc(x, dt, A, B, C, skip, z, dt_bias, softplus, tokens):
    """tokens: 2 leading dimensions [B,T], or 1 [B] (a step)."""
    if x.dim() != tokens + 1:
        raise ValueError("x must be [B,T,D]" if tokens == 2 else "x must be [B,D]")
    io = _io(x, B, C)
    D = x.shape[-1]
    _same(dt, x, "dt")
    _same(z, x, "z")
    if A.dim() != 2 or A.shape[0] != D:
        raise ValueError("A must be [D,N]")
    N, lead = A.shape[1], tuple(x.shape[:-1])
    G = B.shape[-2] if B.dim() == tokens + 2 else 1
    for t, name in ((B, "B"), (C, "C")):
        if tuple(t.shape) not in ((*lead, G, N), (*lead, N) if G == 1 else None) or t.dim() != B.dim():
            raise ValueError(f"{name} must be [..., G, N] (or [..., N]) with x's leading dimensions and A's states")
    par = gate_dtype(x.dtype)
    _dense(A, (D, N), par, "A")
    _dense(skip, (D,), par, "skip")
    _dense(dt_bias, (D,), par, "dt_bias")
    desc = SsmDesc(lead[0], lead[1] if tokens == 2 else 1, D, N, G, 0, io, GL_FLAG_SOFTPLUS if softplus else 0)
    desc.sx, desc.sdt = _rows(x, "x"), _rows(dt, "dt")
    if z is not None:
        desc.sz = _rows(z, "z")
    bc = 3 if B.dim() == tokens + 2 else 2
    desc.sB, desc.sC = _rows(B, "B", bc), _rows(C, "C", bc)
    return desc, par


def _ssm_whole(x, dt, A, B, C, skip, z, dt_bias, state, cu, softplus):
    desc, par = _ssm_desc(x, dt, A, B, C, skip, z, dt_bias, softplus, 2)
    desc.n_seq, n = _sequences(cu, x.shape[0])
    states = _contiguous((n, *A.shape), par)
    _dense(state, states[0], par, "state")
    _on_gpu((x, dt, A, B, C, skip, z, dt_bias, state, cu))
    return desc, par, states


def gl_ssm_fwd(x, dt, A, B, C, skip=None, z=None, dt_bias=None, *, state=None, want_state=False, save=False,
               cu_seqlens=None, softplus=True):
    """Selective scan over whole sequences, gated by silu(z) if z is given.  Returns
    (y, final state [n,D,N] or None, saved or None)."""
    def plan():
        desc, par, states = _ssm_whole(x, dt, A, B, C, skip, z, dt_bias, state, cu_seqlens, softplus)
        return desc, ssm_workspace_size(desc, True)[0], 0, (
            _out(x), states if want_state else None,
            _contiguous((max(_size("gl_ssm_saved_size", desc), 16),), _torch().uint8) if save else None)
    return _run("gl_ssm_fwd", (bool(want_state), bool(save), bool(softplus)),
                (x, dt, A, B, C, skip, z, dt_bias, state, cu_seqlens), plan)


def gl_ssm_bwd(x, dt, A, B, C, skip, z, dt_bias, dy, saved=None, *, state=None, dstate=None, want_dstate=None,
               cu_seqlens=None, softplus=True):
    """Gradients for upstream dy [B,T,D] and dstate (of the final state, or None).
    Returns (dx, ddt, dA, dB, dC, dskip, dz, ddt_bias, dstate of the first state);
    those of absent inputs are None, the last unless `state` was given or
    want_dstate is true."""
    if want_dstate is None:
        want_dstate = state is not None

    def plan():
        desc, par, states = _ssm_whole(x, dt, A, B, C, skip, z, dt_bias, state, cu_seqlens, softplus)
        _same(dy, x, "dy")
        _dense(dstate, states[0], par, "dstate")
        _on_gpu((x, dy, dstate, saved))
        desc.sdy = _rows(dy, "dy")
        if saved is not None and (saved.dtype != _torch().uint8 or not saved.is_contiguous()
                                  or saved.numel() < _size("gl_ssm_saved_size", desc)):
            raise ValueError("saved must be what gl_ssm_fwd returned for these inputs")
        return desc, max(ssm_workspace_size(desc, saved is not None)[1], 16), 0, (
            _out(x), _out(x), _out(A), _out(B), _out(C), None if skip is None else _out(skip),
            None if z is None else _out(z), None if dt_bias is None else _out(dt_bias), states if want_dstate else None)
    return _run("gl_ssm_bwd", (bool(want_dstate), bool(softplus)),
                (x, dt, A, B, C, skip, z, dt_bias, state, cu_seqlens, dy, dstate, saved), plan)


def gl_ssm_step(x, dt, A, B, C, skip, z, dt_bias, state, *, slots=None, softplus=True):
    """One token of each row: x, dt, z [B,D], B, C [B,G,N] (or [B,N]); `state`
    [n,D,N] is updated in place, row b's at slots[b] (int32; outside 0..n-1: nothing
    to do, y = 0), or at b.  Returns y [B,D]."""
    def plan():
        desc, par = _ssm_desc(x, dt, A, B, C, skip, z, dt_bias, softplus, 1)
        if state.dim() != 3:
            raise ValueError("state must be [n,D,N]")
        _dense(state, (state.shape[0], *A.shape), par, "state")
        _slots(slots, x.shape[0], state)
        _on_gpu((x, dt, A, B, C, skip, z, dt_bias, state, slots))
        return desc, 0, state.shape[0], (_out(x),)
    return _run("gl_ssm_step", bool(softplus), (x, dt, A, B, C, skip, z, dt_bias, slots, state), plan)[0]


# ---------------------------------------------------------------- norms
def _addnorm_desc(x, r, w, wx, scale, eps):
    if x.dim() != 3 or r.shape != x.shape:
        raise ValueError("x and r must be [B,T,d]")
    io = _io(x)
    if r.dtype not in (x.dtype, gate_dtype(x.dtype)):
        raise TypeError(f"r must be {x.dtype} or {gate_dtype(x.dtype)}")
    B, T, d = x.shape
    for t, name in ((w, "w"), (wx, "wx"), (scale, "scale")):
        _dense(t, (d,), x.dtype, name)
    _on_gpu((x, r, w, wx, scale))
    desc = AddNormDesc(B, T, d, io, _io_code(r.dtype), 0, 0, eps)
    desc.sx, desc.sr = _rows(x, "x"), _rows(r, "r")
    return desc


def gl_addnorm_fwd(x, r, w, wx=None, scale=None, *, eps=1e-6):
    """r_out = r + scale * u with u = x, or x's root-mean-square norm times wx, and n =
    w times the norm of r_out.  x, r [B,T,d] (r of x's dtype, or fp32 with bf16),
    w, wx, scale [d].  Returns (n, r_out)."""
    eps = _num(eps)

    def plan():
        return _addnorm_desc(x, r, w, wx, scale, eps), 0, 0, (_out(x), _out(r))
    return _run("gl_addnorm_fwd", eps, (x, r, w, wx, scale), plan)


def gl_addnorm_bwd(x, r, w, wx, scale, dn, dr_out=None, *, eps=1e-6):
    """Gradients of gl_addnorm_fwd: (dx, dr, dw, dwx, dscale), the last three [d] in
    fp32 (fp64), None where there is no wx or scale.  dr_out None: zero."""
    eps = _num(eps)

    def plan():
        desc = _addnorm_desc(x, r, w, wx, scale, eps)
        _same(dn, x, "dn")
        _same(dr_out, r, "dr_out")
        _on_gpu((x, dn, dr_out))
        desc.sdn = _rows(dn, "dn")
        if dr_out is not None:
            desc.sdro = _rows(dr_out, "dr_out")
        dw = _contiguous(tuple(w.shape), gate_dtype(x.dtype))
        return desc, max(_size("gl_addnorm_workspace_size", desc), 16), 0, (
            _out(x), _out(r), dw, None if wx is None else dw, None if scale is None else dw)
    return _run("gl_addnorm_bwd", eps, (x, r, w, wx, scale, dn, dr_out), plan)


def _gatenorm_desc(x, z, w, eps, gate_first):
    if x.dim() not in (3, 4):
        raise ValueError("x must be [B,T,d] or [B,T,G,d]")
    io = _io(x)
    _same(z, x, "z")
    d, G = x.shape[-1], x.shape[2] if x.dim() == 4 else 1
    groups = w is not None and w.dim() == 2
    _dense(w, (G, d) if groups else (d,), x.dtype, "w")
    _on_gpu((x, z, w))
    desc = GateNormDesc(x.shape[0], x.shape[1], G, d, io, (GL_FLAG_GATE_FIRST if gate_first else 0) |
                        (GL_FLAG_GROUP_WEIGHTS if groups else 0), eps)
    desc.sx = _rows(x, "x", x.dim() - 1)
    if z is not None:
        desc.sz = _rows(z, "z", x.dim() - 1)
    return desc


def gl_gatenorm_fwd(x, z=None, w=None, *, eps=1e-6, gate_first=False):
    """Root-mean-square norm of every row of x [B,T,d] or [B,T,G,d], times w [d] or
    [G,d] and silu(z); gate_first: of x silu(z).  Returns y, dense."""
    eps = _num(eps)

    def plan():
        return _gatenorm_desc(x, z, w, eps, gate_first), 0, 0, (_out(x),)
    return _run("gl_gatenorm_fwd", (eps, bool(gate_first)), (x, z, w), plan)[0]


def gl_gatenorm_bwd(x, z, w, dy, *, eps=1e-6, gate_first=False):
    """Gradients of gl_gatenorm_fwd: (dx, dz, dw), dw in fp32 (fp64), None where there
    is no z or w."""
    eps = _num(eps)

    def plan():
        desc = _gatenorm_desc(x, z, w, eps, gate_first)
        _same(dy, x, "dy")
        _on_gpu((x, dy))
        desc.sdy = _rows(dy, "dy", x.dim() - 1)
        return desc, max(_size("gl_gatenorm_workspace_size", desc), 16), 0, (
            _out(x), None if z is None else _out(x),
            None if w is None else _contiguous(tuple(w.shape), gate_dtype(x.dtype)))
    return _run("gl_gatenorm_bwd", (eps, bool(gate_first)), (x, z, w, dy), plan)


# ---------------------------------------------------------------- autograd
def _row_tensor(t):
    """t, or a dense copy where its last dimension is not contiguous, it is broadcast or
    its tokens lie too far apart for the scan."""
    if t is None:
        return t
    moves = [s for s, n in zip(t.stride()[:-1], t.shape) if n > 1]
    if (t.stride(-1) == 1 or t.shape[-1] <= 1) and 0 not in moves and (t.dim() < 3 or t.stride(1) < 1 << 19):
        return t
    return t.contiguous()


def _make_functions():
    torch = _torch()
    # the kernels leave no graph behind: gradients of gradients are refused, not lost
    once = torch.autograd.function.once_differentiable

    class CausalConv(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, bias, state, cu_seqlens, want_state, silu):
            ctx.save_for_backward(x, w, bias, state, cu_seqlens)
            ctx.silu = silu
            return gl_conv_fwd(x, w, bias, state=state, want_state=want_state, cu_seqlens=cu_seqlens, silu=silu)

        @staticmethod
        @once
        def backward(ctx, dy, dstate):
            x, w, bias, state, cu_seqlens = ctx.saved_tensors
            dx, dw, dbias, ds = gl_conv_bwd(x, w, bias, _row_tensor(dy), state=state,
                                            dstate=None if dstate is None else dstate.contiguous(),
                                            cu_seqlens=cu_seqlens, silu=ctx.silu)
            return dx, dw.to(w.dtype), None if dbias is None else dbias.to(bias.dtype), ds, None, None, None

    class SelectiveScan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, dt, A, B, C, skip, z, dt_bias, state, cu_seqlens, want_state, softplus):
            y, out, saved = gl_ssm_fwd(x, dt, A, B, C, skip, z, dt_bias, state=state, want_state=want_state, save=True,
                                       cu_seqlens=cu_seqlens, softplus=softplus)
            ctx.save_for_backward(x, dt, A, B, C, skip, z, dt_bias, state, cu_seqlens, saved)
            ctx.softplus = softplus
            return y, out

        @staticmethod
        @once
        def backward(ctx, dy, dstate):
            *args, state, cu_seqlens, saved = ctx.saved_tensors
            grads = gl_ssm_bwd(*args, _row_tensor(dy), saved, state=state,
                               dstate=None if dstate is None else dstate.contiguous(), cu_seqlens=cu_seqlens,
                               softplus=ctx.softplus)
            return (*grads, None, None, None)

    class AddNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, r, w, wx, scale, eps):
            ctx.save_for_backward(x, r, w, wx, scale)
            ctx.eps = eps
            return gl_addnorm_fwd(x, r, w, wx, scale, eps=eps)

        @staticmethod
        @once
        def backward(ctx, dn, dr):
            x, r, w, wx, scale = ctx.saved_tensors
            dx, dres, *dws = gl_addnorm_bwd(x, r, w, wx, scale, _row_tensor(dn), _row_tensor(dr), eps=ctx.eps)
            return dx, dres, *(None if g is None else g.to(w.dtype) for g in dws), None

    class GatedNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, z, w, eps, gate_first):
            ctx.save_for_backward(x, z, w)
            ctx.opts = dict(eps=eps, gate_first=gate_first)
            return gl_gatenorm_fwd(x, z, w, **ctx.opts)

        @staticmethod
        @once
        def backward(ctx, dy):
            x, z, w = ctx.saved_tensors
            dx, dz, dw = gl_gatenorm_bwd(x, z, w, _row_tensor(dy), **ctx.opts)
            return dx, dz, None if dw is None else dw.to(w.dtype), None, None

    return CausalConv, SelectiveScan, AddNorm, GatedNorm


_fns = None


def _functions():
    global _fns
    if _fns is None:
        _fns = _make_functions()
    return _fns


def _no_duals(what, inputs):
    """Refuses dual tensors: they want a forward-mode derivative, which there is not."""
    forward_ad = _torch().autograd.forward_ad
    if forward_ad._current_level >= 0 and any(
            t is not None and forward_ad.unpack_dual(t).tangent is not None for t in inputs):
        raise NotImplementedError(f"{what} has no forward-mode derivative")


def _wants_gradient(inputs):
    return _torch().is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs)


def causal_conv(x, w, bias=None, *, state=None, cu_seqlens=None, want_state=False, silu=True):
    """Autograd-aware gl_conv_fwd: (y, last inputs or None).  Inputs whose rows are
    broadcast or not contiguous are copied."""
    x = _row_tensor(x)
    w, bias, state = (None if t is None else t.contiguous() for t in (w, bias, state))
    inputs = (x, w, bias, state)
    _no_duals("the causal convolution", inputs)
    if not _wants_gradient(inputs):
        return gl_conv_fwd(*inputs[:3], state=state, want_state=want_state, cu_seqlens=cu_seqlens, silu=silu)
    return _functions()[0].apply(*inputs, cu_seqlens, bool(want_state), bool(silu))


def selective_scan(x, dt, A, B, C, skip=None, z=None, dt_bias=None, *, state=None, cu_seqlens=None,
                   want_state=False, softplus=True):
    """Autograd-aware gl_ssm_fwd: (y, final state or None).  Nothing is kept for a
    backward where no gradient is wanted.  Inputs whose rows are broadcast or not
    contiguous are copied."""
    x, dt, B, C, z = (_row_tensor(t) for t in (x, dt, B, C, z))
    A, skip, dt_bias, state = (None if t is None else t.contiguous() for t in (A, skip, dt_bias, state))
    inputs = (x, dt, A, B, C, skip, z, dt_bias, state)
    _no_duals("the selective scan", inputs)
    if not _wants_gradient(inputs):
        return gl_ssm_fwd(*inputs[:8], state=state, want_state=want_state, cu_seqlens=cu_seqlens, softplus=softplus)[:2]
    return _functions()[1].apply(*inputs, cu_seqlens, bool(want_state), bool(softplus))


def add_norm(x, r, w, wx=None, scale=None, *, eps=1e-6):
    """Autograd-aware gl_addnorm_fwd: (n, r_out).  Inputs whose rows are broadcast or
    not contiguous are copied."""
    _no_gradient(TypeError, "eps", eps)
    x, r = _row_tensor(x), _row_tensor(r)
    w, wx, scale = (None if t is None else t.contiguous() for t in (w, wx, scale))
    _no_duals("the residual norm", (x, r, w, wx, scale))
    return _functions()[2].apply(x, r, w, wx, scale, _num(eps))


def gated_norm(x, z=None, w=None, *, eps=1e-6, gate_first=False):
    """Autograd-aware gl_gatenorm_fwd.  Inputs whose rows are broadcast or not
    contiguous are copied."""
    _no_gradient(TypeError, "eps", eps)
    x, z = _row_tensor(x), _row_tensor(z)
    w = None if w is None else w.contiguous()
    _no_duals("the gated norm", (x, z, w))
    return _functions()[3].apply(x, z, w, _num(eps), bool(gate_first))
