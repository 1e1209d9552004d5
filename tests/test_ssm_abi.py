"""C-ABI checks of include/gl_ssm.h that need no GPU: header, binding and library
agree, and bad arguments are refused before anything is launched (the pointers
passed here are never dereferenced)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import weight_scans_amd as ws
from weight_scans_amd import AddNormDesc, ConvDesc, GateNormDesc, Rows, SsmDesc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gl_ssm.h")
BF16, F32, F64 = ws.GL_DTYPE_BF16, ws.GL_DTYPE_F32, ws.GL_DTYPE_F64
FAKE = 0x10000  # 16-byte aligned, never dereferenced
INVALID, UNSUPPORTED, MISALIGNED, SMALL = 1, 2, 3, 4
KINDS = {
    "conv": (ConvDesc, dict(B=2, T=30, D=64, K=4, io_dtype=BF16)),
    "ssm": (SsmDesc, dict(B=2, T=30, D=64, N=16, G=2, io_dtype=BF16)),
    "addnorm": (AddNormDesc, dict(B=2, T=30, d=64, io_dtype=BF16, res_dtype=F32, eps=1e-6)),
    "gatenorm": (GateNormDesc, dict(B=2, T=30, G=2, d=64, io_dtype=BF16, eps=1e-6)),
}


def desc(kind, **kw):
    cls, base = KINDS[kind]
    d = cls(**(base | {k: v for k, v in kw.items() if not k.startswith("s")}))
    for k, v in kw.items():
        if k.startswith("s"):
            setattr(d, k, Rows(*v))
    return d


def call(name, d, pointers, wsp=FAKE, nb=1 << 50):
    """name of the library on d and these addresses, with those that take one also a
    workspace and its size."""
    f = getattr(ws.ssm_lib(), name)
    args = [ctypes.byref(d), *pointers]
    if ctypes.c_size_t in f.argtypes:
        args += [wsp, nb]
    return f(*args, None)


# every pointer of a call: its name, whether it must be there, its alignment (e: an
# element's, p: a parameter's, 4, 16)
CONV_IN = [("x", 1, "e"), ("w", 1, "e"), ("bias", 0, "e")]
SSM_IN = [("x", 1, "e"), ("dt", 1, "e"), ("A", 1, "p"), ("B", 1, "e"), ("C", 1, "e"), ("skip", 0, "p"), ("z", 0, "e"),
          ("dt_bias", 0, "p")]
CALLS = {
    "gl_conv_fwd": CONV_IN + [("state_in", 0, "e"), ("cu", None, 4), ("y", 1, "e"), ("state_out", 0, "e")],
    "gl_conv_bwd": CONV_IN + [("state_in", 0, "e"), ("cu", None, 4), ("dy", 1, "e"), ("dstate_out", 0, "e"), ("dx", 1, "e"),
                              ("dw", 0, "p"), ("dbias", 0, "p"), ("dstate_in", 0, "e")],
    "gl_conv_step": CONV_IN + [("slots", 0, 4), ("n_slots", None, None), ("state", 1, "e"), ("y", 1, "e")],
    "gl_ssm_fwd": SSM_IN + [("state_in", 0, "p"), ("cu", None, 4), ("y", 1, "e"), ("state_out", 0, "p"), ("saved", 0, 16)],
    "gl_ssm_bwd": SSM_IN + [("state_in", 0, "p"), ("cu", None, 4), ("dy", 1, "e"), ("dstate_out", 0, "p"), ("saved", 0, 16),
                            ("dx", 1, "e"), ("ddt", 1, "e"), ("dA", 1, "p"), ("dB", 1, "e"), ("dC", 1, "e"),
                            ("dskip", 0, "p"), ("dz", 1, "e"), ("ddt_bias", 0, "p"), ("dstate_in", 0, "p")],
    "gl_ssm_step": SSM_IN + [("slots", 0, 4), ("n_slots", None, None), ("state", 1, "p"), ("y", 1, "e")],
    "gl_addnorm_fwd": [("x", 1, "e"), ("r", 1, "r"), ("w", 1, "e"), ("wx", 0, "e"), ("scale", 0, "e"), ("n", 1, "e"),
                       ("r_out", 1, "r")],
    "gl_addnorm_bwd": [("x", 1, "e"), ("r", 1, "r"), ("w", 1, "e"), ("wx", 0, "e"), ("scale", 0, "e"), ("dn", 1, "e"),
                       ("dr_out", 0, "r"), ("dx", 1, "e"), ("dr", 1, "r"), ("dw", 0, "p"), ("dwx", 0, "p"),
                       ("dscale", 0, "p")],
    "gl_gatenorm_fwd": [("x", 1, "e"), ("z", 0, "e"), ("w", 0, "e"), ("y", 1, "e")],
    "gl_gatenorm_bwd": [("x", 1, "e"), ("z", 0, "e"), ("w", 0, "e"), ("dy", 1, "e"), ("dx", 1, "e"), ("dz", 1, "e"),
                        ("dw", 0, "p")],
}


def kind_of(name):
    return name.split("_")[1]


def pointers(name, **edit):
    """All pointers of a call, with those of `edit` in place of the usual ones."""
    usual = {"cu": None, "n_slots": 8}
    return [edit.get(n, usual.get(n, FAKE)) for n, *_ in CALLS[name]]


def declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(gl_\w+)\s*\(", text)))


def test_header_binding_and_library_agree():
    assert sorted(ws.SSM_EXPORTS) == declared_functions()
    for name in declared_functions():
        assert hasattr(ws.lib(), name), name
    assert set(CALLS) == {n for n in ws.SSM_EXPORTS if not n.endswith("_size")}


def test_descriptors_have_the_layout_of_the_header(tmp_path):
    """Sizes and offsets as the C compiler sees them, and the values of the flags."""
    classes = (("gl_conv_desc_t", ConvDesc), ("gl_ssm_desc_t", SsmDesc), ("gl_addnorm_desc_t", AddNormDesc),
               ("gl_gatenorm_desc_t", GateNormDesc), ("gl_rows_t", Rows))
    flags = ("GL_FLAG_SILU", "GL_FLAG_SOFTPLUS", "GL_FLAG_GATE_FIRST", "GL_FLAG_GROUP_WEIGHTS")
    lines, want = [], []
    for c_name, cls in classes:
        lines.append(f'printf("%zu\\n", sizeof({c_name}));')
        lines += [f'printf("%zu\\n", offsetof({c_name}, {f[0]}));' for f in cls._fields_]
        want += [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_]
    lines += [f'printf("%u\\n", {f});' for f in flags]
    want += [getattr(ws, f) for f in flags]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "gl_ssm.h"\nint main(void) {\n' + "\n".join(lines) +
                   "\nreturn 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    assert [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()] == want


BAD = {
    "conv": [(dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(D=-1), INVALID), (dict(K=0), INVALID),
             (dict(n_seq=-1), INVALID), (dict(n_seq=3), INVALID), (dict(io_dtype=3), INVALID), (dict(io_dtype=-1), INVALID),
             (dict(flags=1), INVALID), (dict(flags=32), INVALID), (dict(sx=(1, -8, 0)), INVALID),
             (dict(sdx=(-1, 0, 0)), INVALID), (dict(K=9), UNSUPPORTED), (dict(D=(1 << 24) + 1), UNSUPPORTED),
             (dict(B=1, n_seq=1, T=1 << 31), UNSUPPORTED), (dict(B=1 << 40), UNSUPPORTED)],
    "ssm": [(dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(D=-2), INVALID), (dict(N=0), INVALID), (dict(G=0), INVALID),
            (dict(G=3), INVALID), (dict(n_seq=-1), INVALID), (dict(n_seq=3), INVALID), (dict(io_dtype=3), INVALID),
            (dict(flags=16), INVALID), (dict(sB=(1, 1, -1)), INVALID), (dict(sddt=(0, -2, 0)), INVALID),
            (dict(N=257), UNSUPPORTED), (dict(D=1 << 25), UNSUPPORTED), (dict(B=1, n_seq=1, T=1 << 31), UNSUPPORTED),
            (dict(B=1 << 40), UNSUPPORTED), (dict(sz=(64, 1 << 19, 0)), UNSUPPORTED),
            (dict(sdy=(64, 1 << 40, 0)), UNSUPPORTED), (dict(D=1 << 19), UNSUPPORTED)],
    "addnorm": [(dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(d=0), INVALID), (dict(io_dtype=3), INVALID),
                (dict(res_dtype=F64), INVALID), (dict(io_dtype=F32, res_dtype=BF16), INVALID),
                (dict(io_dtype=F64, res_dtype=F32), INVALID), (dict(flags=1), INVALID), (dict(reserved=1), INVALID),
                (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
                (dict(sro=(0, -1, 0)), INVALID), (dict(d=16385), UNSUPPORTED), (dict(B=1 << 40), UNSUPPORTED)],
    "gatenorm": [(dict(B=-1), INVALID), (dict(G=-1), INVALID), (dict(d=0), INVALID), (dict(io_dtype=-1), INVALID),
                 (dict(flags=1), INVALID), (dict(flags=256), INVALID), (dict(eps=-1.0), INVALID),
                 (dict(sdz=(0, 0, -1)), INVALID), (dict(d=16385), UNSUPPORTED), (dict(G=65536), UNSUPPORTED),
                 (dict(T=1 << 40), UNSUPPORTED)],
}


@pytest.mark.parametrize("kind,kw,code", [(k, kw, code) for k, cases in BAD.items() for kw, code in cases])
def test_descriptors_refused(kind, kw, code):
    d, n, m = desc(kind, **kw), ctypes.c_size_t(), ctypes.c_size_t()
    for name in CALLS:
        if kind_of(name) == kind:
            assert call(name, d, pointers(name)) == code, name
    L = ws.ssm_lib()
    if kind == "ssm":
        assert L.gl_ssm_saved_size(ctypes.byref(d), ctypes.byref(n)) == code
        assert L.gl_ssm_workspace_size(ctypes.byref(d), 1, ctypes.byref(n), ctypes.byref(m)) == code
    else:
        assert getattr(L, f"gl_{kind}_workspace_size")(ctypes.byref(d), ctypes.byref(n)) == code
    assert ws.lib().gl_last_error()


def test_null_arguments():
    L, n = ws.ssm_lib(), ctypes.c_size_t()
    assert L.gl_ssm_saved_size(None, ctypes.byref(n)) == INVALID
    assert L.gl_ssm_workspace_size(None, 0, ctypes.byref(n), ctypes.byref(n)) == INVALID
    assert L.gl_ssm_saved_size(ctypes.byref(desc("ssm")), None) == INVALID
    assert L.gl_ssm_workspace_size(ctypes.byref(desc("ssm")), 0, None, ctypes.byref(n)) == INVALID
    for kind in ("conv", "addnorm", "gatenorm"):
        f = getattr(L, f"gl_{kind}_workspace_size")
        assert f(None, ctypes.byref(n)) == INVALID and f(ctypes.byref(desc(kind)), None) == INVALID


@pytest.mark.parametrize("io", [BF16, F32, F64])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_pointers_refused(name, io):
    kind = kind_of(name)
    kw = dict(io_dtype=io) | (dict(res_dtype=F32 if io == BF16 else io) if kind == "addnorm" else {})
    d = desc(kind, **kw)
    size = {"e": {BF16: 2, F32: 4, F64: 8}[io], "p": 8 if io == F64 else 4, "r": 8 if io == F64 else 4, 4: 4, 16: 16}
    for n, need, align in CALLS[name]:
        if n == "n_slots":
            continue
        if need:
            assert call(name, d, pointers(name, **{n: None})) == INVALID, n
        if n != "cu":
            assert call(name, d, pointers(name, **{n: FAKE + size[align] // 2})) == MISALIGNED, n
    assert b"aligned" in ws.lib().gl_last_error()


def test_sequence_tables_refused():
    for name in ("gl_conv_fwd", "gl_conv_bwd", "gl_ssm_fwd", "gl_ssm_bwd"):
        kind = kind_of(name)
        assert call(name, desc(kind), pointers(name, cu=FAKE)) == INVALID               # a table without n_seq
        assert call(name, desc(kind, B=1, n_seq=2), pointers(name)) == INVALID           # n_seq without a table
        assert call(name, desc(kind, B=1, n_seq=2), pointers(name, cu=FAKE + 2)) == MISALIGNED
    for name in ("gl_conv_step", "gl_ssm_step"):
        assert call(name, desc(kind_of(name), B=1, n_seq=2), pointers(name)) == INVALID


def test_steps_refused():
    for name in ("gl_conv_step", "gl_ssm_step"):
        d = desc(kind_of(name))
        assert call(name, d, pointers(name, n_slots=-1)) == INVALID
        assert call(name, d, pointers(name, n_slots=1, slots=None)) == INVALID  # two rows, one state


def test_workspaces_refused():
    L, n, m = ws.ssm_lib(), ctypes.c_size_t(), ctypes.c_size_t()
    for name in ("gl_conv_bwd", "gl_addnorm_bwd", "gl_gatenorm_bwd"):
        kind = kind_of(name)
        getattr(L, f"gl_{kind}_workspace_size")(ctypes.byref(desc(kind)), ctypes.byref(n))
        assert n.value > 0
        assert call(name, desc(kind), pointers(name), nb=n.value - 1) == SMALL
        assert call(name, desc(kind), pointers(name), wsp=None) == INVALID
        assert call(name, desc(kind), pointers(name), wsp=FAKE + 8) == MISALIGNED
    d = desc("ssm")
    sizes = {}
    for have in (0, 1):
        assert L.gl_ssm_workspace_size(ctypes.byref(d), have, ctypes.byref(m), ctypes.byref(n)) == 0
        sizes[have] = n.value
        edit = {} if have else {"saved": None}
        assert call("gl_ssm_bwd", d, pointers("gl_ssm_bwd", **edit), nb=n.value - 1) == SMALL
        assert call("gl_ssm_bwd", d, pointers("gl_ssm_bwd", **edit), wsp=None) == INVALID
        assert call("gl_ssm_bwd", d, pointers("gl_ssm_bwd", **edit), wsp=FAKE + 8) == MISALIGNED
    L.gl_ssm_saved_size(ctypes.byref(d), ctypes.byref(n))
    assert n.value > 0 and sizes[0] >= sizes[1] + n.value


def test_nothing_to_do_needs_nothing():
    for name, kw in (("gl_conv_fwd", dict(B=0)), ("gl_conv_step", dict(B=0)), ("gl_ssm_fwd", dict(B=0)),
                     ("gl_ssm_step", dict(B=0)), ("gl_conv_fwd", dict(D=0)), ("gl_conv_bwd", dict(D=0)),
                     ("gl_ssm_fwd", dict(D=0)), ("gl_ssm_bwd", dict(B=0, D=0)), ("gl_addnorm_fwd", dict(T=0)),
                     ("gl_gatenorm_fwd", dict(G=0)), ("gl_gatenorm_bwd", dict(B=0))):
        none = [0 if n == "n_slots" else None for n, *_ in CALLS[name]]
        assert call(name, desc(kind_of(name), **kw), none, wsp=None if "ssm_bwd" not in name else FAKE) == 0, name


def test_binding_refuses_on_the_cpu():
    """Shapes, types and devices, before anything is launched."""
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    A, bc = torch.zeros(8, 3), torch.zeros(2, 5, 3)
    for f, error in (
            (lambda: ws.gl_conv_fwd(x, w), ValueError),                                    # on the CPU
            (lambda: ws.gl_conv_fwd(x[0], w), ValueError),
            (lambda: ws.gl_conv_fwd(x.half(), w.half()), TypeError),
            (lambda: ws.gl_conv_fwd(x, w.double()), TypeError),
            (lambda: ws.gl_conv_fwd(x, w.T.contiguous().T), ValueError),
            (lambda: ws.gl_conv_fwd(x, w, state=torch.zeros(2, 4, 8)), ValueError),
            (lambda: ws.gl_conv_fwd(x, w, cu_seqlens=torch.zeros(3, dtype=torch.int32)), ValueError),  # B = 2
            (lambda: ws.gl_conv_fwd(x[:1], w, cu_seqlens=torch.zeros(3)), ValueError),
            (lambda: ws.gl_conv_step(x[:, 0], w, None, torch.zeros(1, 3, 8)), ValueError),
            (lambda: ws.gl_conv_step(x[:, 0], w, None, torch.zeros(2, 3, 8), slots=torch.zeros(2)), ValueError),
            (lambda: ws.gl_ssm_fwd(x, x, A, bc, bc), ValueError),                          # on the CPU
            (lambda: ws.gl_ssm_fwd(x, x[:, :4], A, bc, bc), ValueError),
            (lambda: ws.gl_ssm_fwd(x, x, A.bfloat16(), bc, bc), TypeError),
            (lambda: ws.gl_ssm_fwd(x, x, A, bc[:, :4], bc), ValueError),
            (lambda: ws.gl_ssm_fwd(x, x, A, bc, bc.double()), TypeError),
            (lambda: ws.gl_ssm_fwd(x, x, A, bc, bc, torch.zeros(7)), ValueError),
            (lambda: ws.gl_ssm_fwd(x, x, A, bc, bc, state=torch.zeros(2, 8, 4)), ValueError),
            (lambda: ws.gl_ssm_step(x, x, A, bc, bc, None, None, None, torch.zeros(2, 8, 3)), ValueError),
            (lambda: ws.gl_ssm_bwd(x, x, A, bc, bc, None, None, None, x[:, :2]), ValueError),
            (lambda: ws.gl_addnorm_fwd(x, x, torch.zeros(8)), ValueError),                 # on the CPU
            (lambda: ws.gl_addnorm_fwd(x, x.bfloat16(), torch.zeros(8)), TypeError),
            (lambda: ws.gl_addnorm_fwd(x, x, torch.zeros(9)), ValueError),
            (lambda: ws.gl_gatenorm_fwd(x, x[:, :2]), ValueError),
            (lambda: ws.gl_gatenorm_fwd(x, None, torch.zeros(2, 8)), ValueError),
            (lambda: ws.gl_gatenorm_fwd(x[0]), ValueError)):
        with pytest.raises(error):
            f()


def test_unknown_gradients_refused():
    x = torch.zeros(2, 5, 8)
    eps = torch.tensor(1e-6, requires_grad=True)
    with pytest.raises(TypeError, match="eps"):
        ws.add_norm(x, x, torch.ones(8), eps=eps)
    with pytest.raises(TypeError, match="eps"):
        ws.gated_norm(x, eps=eps)


@pytest.mark.parametrize("T", [0, 7, 1 << 40])
def test_convolution_step_does_not_use_the_tokens_of_its_descriptor(T):
    """A step takes the descriptor of any number of tokens: sizes are checked as for one."""
    none = [0 if n == "n_slots" else None for n, *_ in CALLS["gl_conv_step"]]
    assert call("gl_conv_step", desc("conv", B=0, T=T), none) == 0


@pytest.mark.parametrize("T", [0, 7, 1 << 40])
def test_scan_step_does_not_use_the_tokens_of_its_descriptor(T):
    """Likewise of the scan's step, whose sizes were checked as those of T tokens."""
    none = [0 if n == "n_slots" else None for n, *_ in CALLS["gl_ssm_step"]]
    assert call("gl_ssm_step", desc("ssm", B=0, T=T), none) == 0


ROWS_64 = {s: (64, 64, 64) for s in ("sx", "sdt", "sz", "sB", "sC", "sy", "sdy", "sdx", "sddt", "sdz", "sdB", "sdC")}


@pytest.mark.parametrize("name,kw,edit", [
    ("gl_conv_fwd", dict(B=1 << 14, T=1, D=65537, K=8), {}),
    ("gl_conv_step", dict(B=1 << 17, T=1, D=65537), dict(slots=FAKE)),
    # a later launch of the call: gradients of the first states
    ("gl_conv_bwd", dict(B=1 << 14, T=1, D=1 << 16, K=8), {}),
    # work-groups of one channel each, in the forward and in the backward with and without saved states
    ("gl_ssm_fwd", dict(B=512, T=1, D=1 << 15, G=1 << 15, N=1), {}),
    ("gl_ssm_bwd", dict(B=512, T=1, D=1 << 15, G=1 << 15, N=1), {}),
    ("gl_ssm_bwd", dict(B=512, T=1, D=1 << 15, G=1 << 15, N=1), dict(saved=None)),
    # its sums over sequences
    ("gl_ssm_bwd", dict(B=1, T=1, D=1 << 24, G=1, N=256, **ROWS_64), {}),
    ("gl_ssm_bwd", dict(B=1, T=1, D=1 << 24, G=1, N=256, **ROWS_64), dict(saved=None)),
    ("gl_addnorm_fwd", dict(B=1 << 14, T=1 << 15, d=64), {}),
    ("gl_gatenorm_fwd", dict(B=1 << 14, T=1 << 15, G=1, d=64), {}),
    # sums for the weights of very many groups
    ("gl_gatenorm_bwd", dict(B=1, T=1, G=65535, d=16384, flags=ws.GL_FLAG_GROUP_WEIGHTS), {}),
    ("gl_gatenorm_bwd", dict(B=0, T=1, G=65535, d=16384, flags=ws.GL_FLAG_GROUP_WEIGHTS), {}),
])
def test_sizes_above_a_launch_are_refused_before_the_first(name, kw, edit):
    """Not supported, where a launch would have failed behind others that had written."""
    usual = dict(n_slots=1 << 20)
    assert call(name, desc(kind_of(name), **kw), pointers(name, **(usual | edit)), nb=1 << 62) == UNSUPPORTED
    assert b"limits" in ws.lib().gl_last_error()


@pytest.mark.parametrize("io,B,T,D,N,G,channels", [
    (BF16, 4, 4096, 2048, 16, 1, 32), (BF16, 1, 32768, 2048, 16, 1, 8),
    # above 2^30 bytes of parts more channels, as far as there are: 32 to 64 states, 16 to 128, 8 to 256 (fp64: half)
    (BF16, 1, 32769, 2048, 16, 1, 16), (F32, 1, 65537, 2048, 16, 1, 32), (BF16, 1, 131072, 2048, 16, 1, 32),
    (BF16, 8, 8192, 4096, 64, 1, 32), (F32, 2, 16384, 4096, 128, 2, 16), (BF16, 4, 4096, 2048, 256, 1, 8),
    (F64, 2, 16384, 4096, 64, 1, 16), (F32, 1, 40000, 520, 64, 2, 16)])
def test_workspace_of_the_scan_backward(io, B, T, D, N, G, channels):
    """What the header says: the parts of dB and dC, 2 N values a token and block of channels, and those of the
    parameters, N + 2 a channel and sequence, to 256 bytes each."""
    n, m = ctypes.c_size_t(), ctypes.c_size_t()
    d = desc("ssm", B=B, T=T, D=D, N=N, G=G, io_dtype=io)
    assert ws.ssm_lib().gl_ssm_workspace_size(ctypes.byref(d), 1, ctypes.byref(n), ctypes.byref(m)) == 0
    par, up = 8 if io == F64 else 4, lambda x: -(-x // 256) * 256
    blocks = G * -(-(D // G) // channels)
    assert n.value == 0 and m.value == up(2 * N * blocks * B * T * par) + up(B * (N + 2) * D * par)
