"""C-ABI checks of include/gl_delta.h that need no GPU: header, binding and
library agree, descriptors choose their kernels, and bad arguments are refused
before anything is launched (the pointers passed here are never dereferenced)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import weight_scans_amd as ws
from weight_scans_amd.delta import DeltaDesc, QkDesc, Strides

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gl_delta.h")
BF16, F32, F64 = ws.GL_DTYPE_BF16, ws.GL_DTYPE_F32, ws.GL_DTYPE_F64
FAKE = 0x10000  # 16-byte aligned, never dereferenced
INVALID, UNSUPPORTED, MISALIGNED, SMALL = 1, 2, 3, 4


def declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(gl_\w+)\s*\(", text)))


def test_header_binding_and_library_agree():
    assert sorted(ws.DELTA_EXPORTS) == declared_functions()
    for name in declared_functions():
        assert hasattr(ws.lib(), name), name


def test_descriptors_have_the_layout_of_the_header(tmp_path):
    """Sizes and offsets as the C compiler sees them."""
    lines = []
    for c_name, cls in (("gl_delta_desc_t", DeltaDesc), ("gl_qknorm_desc_t", QkDesc), ("gl_strides_t", Strides)):
        lines.append(f'printf("%zu\\n", sizeof({c_name}));')
        lines += [f'printf("%zu\\n", offsetof({c_name}, {f[0]}));' for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "gl_delta.h"\nint main(void) {\n' +
                   "\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for cls in (DeltaDesc, QkDesc, Strides):
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f[0]).offset for f in cls._fields_]
    assert got == want


# ------------------------------------------------------------ the delta rule
def desc(**kw):
    strides = {k: kw.pop(k) for k in list(kw) if k.startswith("s") and k not in ("scale", "segments")}
    a = dict(B=2, T=100, H=4, Hk=2, dk=64, dv=64, io_dtype=BF16, gate_dtype=BF16)
    a.update(kw)
    d = ws.make_delta_desc(**a)
    for n, s in strides.items():
        setattr(d, n, Strides(*s))
    return d


def status(name, *args):
    return getattr(ws.delta_lib(), name)(*args)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(H=-4), INVALID), (dict(Hk=-2), INVALID),
    (dict(n_seq=-1), INVALID), (dict(dk=0), INVALID), (dict(dv=0), INVALID),
    (dict(Hk=3), INVALID), (dict(Hk=0), INVALID), (dict(H=1, Hk=2), INVALID),
    (dict(io_dtype=3), INVALID), (dict(io_dtype=-1), INVALID), (dict(gate_dtype=F64), INVALID),
    (dict(io_dtype=F32, gate_dtype=BF16), INVALID), (dict(io_dtype=F64, gate_dtype=F32), INVALID),
    (dict(flags=2), INVALID), (dict(flags=8), INVALID), (dict(segments=(1 << 20) + 1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(n_seq=3), INVALID),  # packed sequences need B = 1
    (dict(sq=(1, -8, 8)), INVALID), (dict(sdv=(-1, 0, 0)), INVALID),
    (dict(dk=129), UNSUPPORTED), (dict(dv=200), UNSUPPORTED),
    (dict(B=1, n_seq=1, T=1 << 31), UNSUPPORTED), (dict(B=1 << 40), UNSUPPORTED), (dict(H=1 << 21), UNSUPPORTED),
])
def test_descriptors_refused(kw, code):
    d, n, m = desc(**kw), ctypes.c_size_t(), ctypes.c_size_t()
    assert status("gl_delta_saved_size", ctypes.byref(d), ctypes.byref(n)) == code
    assert status("gl_delta_workspace_size", ctypes.byref(d), 1, ctypes.byref(n), ctypes.byref(m)) == code
    assert fwd(d) == code and bwd(d) == code and step(d) == code
    assert ws.delta_path_name(d) is None
    assert ws.lib().gl_last_error()


def test_null_arguments():
    d, n = desc(), ctypes.c_size_t()
    assert status("gl_delta_saved_size", None, ctypes.byref(n)) == INVALID
    assert status("gl_delta_saved_size", ctypes.byref(d), None) == INVALID
    assert status("gl_delta_workspace_size", ctypes.byref(d), 0, None, ctypes.byref(n)) == INVALID
    assert status("gl_delta_workspace_size", ctypes.byref(d), 0, ctypes.byref(n), None) == INVALID
    assert status("gl_delta_path_name", None) is None


@pytest.mark.parametrize("kw,path", [
    (dict(), "delta-mfma-bf16-64x64"), (dict(gate_dtype=F32), "delta-mfma-bf16-64x64"),
    (dict(dk=8, dv=128), "delta-mfma-bf16-64x128"), (dict(dk=72, dv=8), "delta-mfma-bf16-128x64"),
    (dict(dk=128, dv=128, B=1, n_seq=3), "delta-mfma-bf16-128x128"),
    (dict(T=3), "delta-serial-bf16"), (dict(T=4), "delta-mfma-bf16-64x64"),
    (dict(B=1, n_seq=26), "delta-serial-bf16"),  # 100 tokens of 26 sequences
    (dict(dk=60), "delta-serial-bf16"), (dict(dv=4), "delta-serial-bf16"),
    (dict(flags=ws.GL_FLAG_GENERIC), "delta-serial-bf16"),
    (dict(sq=(0, 64, 64)), "delta-mfma-bf16-64x64"), (dict(sk=(0, 64, 0)), "delta-serial-bf16"),
    (dict(sv=(0, 64, 1 << 23)), "delta-serial-bf16"), (dict(sq=(0, 6400, 68)), "delta-serial-bf16"),
    (dict(io_dtype=F32, gate_dtype=F32), "delta-mfma-f32-64"),
    (dict(io_dtype=F32, gate_dtype=F32, dk=68, dv=20), "delta-mfma-f32-128"),
    (dict(io_dtype=F32, gate_dtype=F32, dk=66), "delta-serial-f32"),
    (dict(io_dtype=F32, gate_dtype=F32, T=2), "delta-serial-f32"),
    (dict(io_dtype=F64, gate_dtype=F64), "delta-serial-f64"),
])
def test_paths(kw, path):
    assert ws.delta_path_name(desc(**kw)) == path


def test_sizes():
    for kw in (dict(), dict(dk=128, dv=128), dict(io_dtype=F32, gate_dtype=F32), dict(io_dtype=F64, gate_dtype=F64),
               dict(flags=ws.GL_FLAG_GENERIC)):
        d = desc(**kw)
        saved = ws.delta_saved_size(d)
        f1, b1 = ws.delta_workspace_size(d, True)
        f0, b0 = ws.delta_workspace_size(d, False)
        assert saved > 0 and f0 >= f1 and b0 >= b1 + saved
    assert ws.delta_saved_size(desc(T=0)) == 0 and ws.delta_saved_size(desc(B=0)) == 0
    # segments: a first state and a transition each
    one, four = (ws.delta_workspace_size(desc(B=1, T=4096, segments=n), False)[0] for n in (1, 4))
    assert four >= one + 4 * 4 * 2 * 64 * 64 * 4
    # never more than one a chunk, and chosen for few heads and many chunks only
    assert (ws.delta_workspace_size(desc(segments=50, T=128), True)
            == ws.delta_workspace_size(desc(segments=2, T=128), True))
    auto = lambda **kw: ws.delta_workspace_size(desc(**kw), True) > ws.delta_workspace_size(desc(segments=1, **kw), True)
    assert auto(B=1, T=1 << 15) and not auto(B=8, H=16, T=4096) and not auto(B=1, T=512)


def ptrs(n, edit=()):
    p = [FAKE] * n
    for i, v in edit:
        p[i] = v
    return [None if x is None else ctypes.c_void_p(x) for x in p]


def fwd(d, edit=(), wsp=FAKE, nb=1 << 40):
    p = ptrs(10, [(6, None)] + list(edit))  # q k v log_alpha beta state_in cu y state_out saved
    return status("gl_delta_fwd", ctypes.byref(d), *p, wsp, nb, None)


def bwd(d, edit=(), wsp=FAKE, nb=1 << 40):
    # q k v log_alpha beta state_in cu dy dstate_out saved dq dk dv dlog_alpha dbeta dstate_in
    p = ptrs(16, [(6, None)] + list(edit))
    return status("gl_delta_bwd", ctypes.byref(d), *p, wsp, nb, None)


def step(d, edit=(), n_slots=8):
    p = ptrs(8, edit)  # q k v log_alpha beta slots | state y
    return status("gl_delta_step", ctypes.byref(d), *p[:6], n_slots, *p[6:], None)


@pytest.mark.parametrize("kw", [dict(), dict(io_dtype=F64, gate_dtype=F64), dict(T=5), dict(T=3),
                                dict(io_dtype=F32, gate_dtype=F32)])
def test_pointers_refused(kw):
    d = desc(**kw)
    chunk = "mfma-bf16" in ws.delta_path_name(d)
    odd = FAKE + 8 if chunk else FAKE + 1  # not a whole row group / not a whole element
    for i in (0, 1, 2, 7):
        assert fwd(d, [(i, None)]) == INVALID, i
        assert fwd(d, [(i, odd)]) == MISALIGNED, i
    for i in (3, 4):
        assert fwd(d, [(i, None)]) == INVALID and fwd(d, [(i, FAKE + 1)]) == MISALIGNED, i
    for i in (5, 8, 9):
        assert fwd(d, [(i, FAKE + 8)]) == MISALIGNED, i
    for i in (0, 1, 2, 7, 10, 11, 12):
        assert bwd(d, [(i, None)]) == INVALID and bwd(d, [(i, odd)]) == MISALIGNED, i
    for i in (3, 4, 13, 14):
        assert bwd(d, [(i, None)]) == INVALID and bwd(d, [(i, FAKE + 1)]) == MISALIGNED, i
    for i in (5, 8, 9, 15):
        assert bwd(d, [(i, FAKE + 8)]) == MISALIGNED, i
    assert b"aligned" in ws.lib().gl_last_error()


def test_workspaces_refused():
    for kw in (dict(), dict(B=1, T=4096, segments=4), dict(io_dtype=F32, gate_dtype=F32)):
        d = desc(**kw)
        need = ws.delta_workspace_size(d, False)
        for call, n in ((lambda **a: fwd(d, [(9, None)], **a), need[0]),
                        (lambda **a: bwd(d, [(9, None)], **a), need[1])):
            assert n > 0
            assert call(nb=n - 1) == SMALL and call(wsp=None, nb=n) == INVALID
            assert call(wsp=FAKE + 4, nb=n) == MISALIGNED


def test_sequence_tables_refused():
    assert fwd(desc(), [(6, FAKE)]) == INVALID               # a table without n_seq
    packed = desc(B=1, n_seq=2)
    assert fwd(packed) == INVALID and bwd(packed) == INVALID  # n_seq without a table
    assert fwd(packed, [(6, FAKE + 2)]) == MISALIGNED
    assert step(packed) == INVALID


def test_strides_of_outputs_refused_on_the_matrix_path():
    assert fwd(desc(sy=(6400, 64, 68))) == UNSUPPORTED
    assert fwd(desc(sy=(0, 0, 32))) == UNSUPPORTED
    for n in ("sdy", "sdv", "sdq", "sdk"):
        assert bwd(desc(**{n: (6400, 64, 60)})) == UNSUPPORTED, n


def test_steps_refused():
    d = desc()
    for i in (0, 1, 2, 3, 4, 6, 7):
        assert step(d, [(i, None)]) == INVALID, i
    for i in (0, 1, 2, 3, 4, 7):
        assert step(d, [(i, FAKE + 1)]) == MISALIGNED, i
    assert step(d, [(6, FAKE + 8)]) == MISALIGNED and step(d, [(5, FAKE + 2)]) == MISALIGNED
    assert step(d, n_slots=-1) == INVALID
    assert step(d, [(5, None)], n_slots=1) == INVALID  # two rows, one state


def test_nothing_to_do_needs_nothing():
    none = [(i, None) for i in range(16)]
    for kw in (dict(B=0), dict(H=0, Hk=0)):
        assert fwd(desc(**kw), none[:10], wsp=None, nb=0) == 0
        assert bwd(desc(**kw), none, wsp=None, nb=0) == 0
        assert step(desc(**kw), none[:8], n_slots=0) == 0
    assert fwd(desc(T=0), none[:10], wsp=None, nb=0) == 0  # no token and no state wanted
    assert bwd(desc(T=0), none, wsp=None, nb=0) == 0


# ------------------------------------------------------ norms and rotation
def qk(**kw):
    d = QkDesc(B=2, T=5, Hq=4, Hk=2, d=64, rot=32, n_pos=16, io_dtype=BF16, eps=1e-6, q_scale=1.0, k_scale=1.0)
    for n, v in kw.items():
        setattr(d, n, Strides(*v) if isinstance(v, tuple) else v)
    return d


def qk_fwd(d, edit=()):
    return status("gl_qknorm_rope_fwd", ctypes.byref(d), *ptrs(9, edit), None)  # q k wq wk cos sin pos | q k


def qk_bwd(d, edit=(), wsp=FAKE, nb=1 << 40):
    # q k wq wk cos sin pos | dout_q dout_k | dq dk dwq dwk
    return status("gl_qknorm_rope_bwd", ctypes.byref(d), *ptrs(13, edit), wsp, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hk=-1), INVALID),
    (dict(d=0), INVALID), (dict(rot=-2), INVALID), (dict(rot=3), INVALID), (dict(rot=66), INVALID),
    (dict(n_pos=0), INVALID), (dict(n_pos=-1), INVALID), (dict(io_dtype=4), INVALID), (dict(flags=1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(q_scale=float("inf")), INVALID),
    (dict(k_scale=float("nan")), INVALID), (dict(sq=(0, -1, 1)), INVALID), (dict(sdok=(0, 0, -8)), INVALID),
    (dict(d=257), UNSUPPORTED), (dict(Hq=(1 << 20) + 1), UNSUPPORTED), (dict(B=1 << 40), UNSUPPORTED),
])
def test_norm_descriptors_refused(kw, code):
    d, n = qk(**kw), ctypes.c_size_t()
    assert qk_fwd(d) == code and qk_bwd(d) == code
    assert status("gl_qknorm_rope_workspace_size", ctypes.byref(d), ctypes.byref(n)) == code


def test_norm_pointers_refused():
    d = qk()
    assert status("gl_qknorm_rope_fwd", None, *ptrs(9), None) == INVALID
    for i in (0, 1, 4, 5, 7, 8):
        assert qk_fwd(d, [(i, None)]) == INVALID, i
    for i in (0, 1, 2, 3, 4, 5, 7, 8):
        assert qk_fwd(d, [(i, FAKE + 1)]) == MISALIGNED, i
    assert qk_fwd(d, [(6, FAKE + 2)]) == MISALIGNED
    for i in (0, 1, 4, 5, 7, 8, 9, 10):
        assert qk_bwd(d, [(i, None)]) == INVALID, i
    for i in (0, 1, 2, 3, 4, 5, 7, 8, 9, 10, 11, 12):
        assert qk_bwd(d, [(i, FAKE + 1)]) == MISALIGNED, i
    n = ctypes.c_size_t()
    assert status("gl_qknorm_rope_workspace_size", ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
    assert qk_bwd(d, nb=n.value - 1) == SMALL and qk_bwd(d, wsp=None) == INVALID
    assert qk_bwd(d, wsp=FAKE + 4) == MISALIGNED
    none = [(i, None) for i in range(13)]
    assert qk_fwd(qk(T=0), none[:9]) == 0 and qk_bwd(qk(B=0), none, wsp=None, nb=0) == 0


# ------------------------------------------------------ the torch binding
def tensors(B=1, H=2, Hk=1, T=20, dk=16, dv=24, dt=torch.float32):
    q, k = torch.zeros(B, Hk, T, dk, dtype=dt), torch.zeros(B, Hk, T, dk, dtype=dt)
    return q, k, torch.zeros(B, H, T, dv, dtype=dt), torch.zeros(B, H, T, dtype=dt), torch.zeros(B, H, T, dtype=dt)


def test_binding_refuses_wrong_tensors():
    q, k, v, a, b = tensors()
    cases = [
        (ValueError, (q[0], k, v, a, b)), (ValueError, (q, k[..., :8], v, a, b)), (ValueError, (q, k, v[:, :, :9], a, b)),
        (ValueError, (q, k, v, a[..., None], b)), (ValueError, (q, k, v, a, b[:, :1])),
        (TypeError, (q.half(), k.half(), v.half(), a, b)), (TypeError, (q, k, v.double(), a, b)),
        (TypeError, (q, k, v, a, b.double())), (TypeError, (q, k, v, a.bfloat16(), b.bfloat16())),
        (ValueError, (q, k, v, a, b)),  # not on a GPU
    ]
    for err, args in cases:
        with pytest.raises(err):
            ws.gl_delta_fwd(*args)
        with pytest.raises(err):
            ws.gl_delta_bwd(*args, v)
        with pytest.raises(err):
            ws.gl_delta_step(*(t[:, :, 0] if t.dim() > 2 else t for t in args), torch.zeros(1, 2, 24, 16))
    for n in ("wq", "wk"):
        with pytest.raises(ValueError):
            ws.gl_qknorm_rope_fwd(q, k, **{n: torch.zeros(17)})
    with pytest.raises(ValueError):
        ws.gl_qknorm_rope_fwd(q, k, cos=torch.zeros(4, 8))
    with pytest.raises(ValueError):
        ws.gl_qknorm_rope_fwd(q, k)  # not on a GPU
    with pytest.raises(TypeError):
        ws.gl_qknorm_rope_fwd(q, k.double())
