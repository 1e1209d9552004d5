"""What calls of include/gl_delta.h read and write on the GPU: states updated in
place, and nothing outside the outputs, `saved` and the workspaces whatever the
sequence table holds."""
import ctypes

import pytest
import torch

import weight_scans_amd as ws
from delta_ref import inputs
from test_gpu_delta import BF16, F32, F64, to_gpu

pytestmark = pytest.mark.gpu

CODE = {F64: ws.GL_DTYPE_F64, F32: ws.GL_DTYPE_F32, BF16: ws.GL_DTYPE_BF16}


def ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def call(name, desc, tensors, workspace):
    status = getattr(ws.delta_lib(), name)(ctypes.byref(desc), *(ptr(t) for t in tensors), ptr(workspace),
                                           workspace.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert status == 0, ws.lib().gl_last_error()


def space(n):
    return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype,T,segments,flags", [
    (BF16, 600, 3, 0), (BF16, 600, 2, 0), (BF16, 130, 1, 0), (BF16, 5, 0, 0), (BF16, 0, 0, 0), (F32, 200, 0, 0),
    (F64, 40, 0, 0), (BF16, 2600, 0, 0), (F32, 100, 0, ws.GL_FLAG_GENERIC)])
@pytest.mark.parametrize("d", [64, 128])
def test_states_updated_in_place(dtype, T, segments, flags, d):
    """state_out = state_in and dstate_in = dstate_out: the bits of calls with states apart."""
    B, H, Hk = 1, 2, 1
    x = inputs(T + d, B, H, Hk, max(T, 1), d, d, dtype)
    g = to_gpu(x, dtype, dtype)
    g = {n: t if "state" in n else t[:, :, :T].contiguous() for n, t in g.items()}
    args = [g[n] for n in ("q", "k", "v", "log_alpha", "beta")]
    kw = dict(state=g["state"], flags=flags, segments=segments)
    desc = ws.make_delta_desc(B, T, H, Hk, d, d, CODE[dtype], CODE[dtype], flags=flags, segments=segments,
                              scale=d ** -0.5)
    for save in (True, False):
        y, end, saved = ws.gl_delta_fwd(*args, want_state=True, save=save, **kw)
        state, y1, saved1 = g["state"].clone(), torch.empty_like(y), space(ws.delta_saved_size(desc)) if save else None
        call("gl_delta_fwd", desc, [*args, state, None, y1, state, saved1], space(ws.delta_workspace_size(desc, save)[0]))
        assert torch.equal(y, y1) and torch.equal(end, state)
        want = ws.gl_delta_bwd(*args, g["dy"], saved, dstate=g["dstate"], **kw)
        got, dstate = [torch.empty_like(t) for t in args], g["dstate"].clone()
        call("gl_delta_bwd", desc, [*args, g["state"], None, g["dy"], dstate, saved1, *got, dstate],
             space(ws.delta_workspace_size(desc, save)[1]))
        for a, b in zip(want, [*got, dstate]):
            assert torch.equal(a, b)


GUARD = 1 << 16


class Guarded:
    """Memory of n bytes between two runs of a known byte."""

    def __init__(self, n):
        self.n = max(n, 16)
        self.all = torch.full((self.n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.inside = self.all[GUARD : GUARD + self.n]

    def like(self, t):
        return self.inside[: t.numel() * t.element_size()].view(t.dtype).view(t.shape)

    def whole(self):
        return bool((self.all[:GUARD] == 0xA5).all()) and bool((self.all[GUARD + self.n :] == 0xA5).all())


@pytest.mark.parametrize("table", [[0, 30, 30, 100], [-5, 1 << 30, 40, 90], [0, 90, 10, 100], [100, 100, 0, 0],
                                   [50, 20, 70, 30], [-(1 << 31), (1 << 31) - 1, -(1 << 31), (1 << 31) - 1],
                                   [99, 100, 98, 200], [0, 0, 0, 0]])
@pytest.mark.parametrize("dtype,d,segments,flags", [(BF16, 64, 1, 0), (BF16, 128, 2, 0), (BF16, 40, 0, 0), (F32, 64, 0, 0),
                                                    (F32, 100, 0, 0), (F64, 33, 0, 0), (BF16, 64, 0, ws.GL_FLAG_GENERIC)])
def test_any_sequence_table_stays_inside(table, dtype, d, segments, flags):
    """Tables out of range and out of order are clamped (host arithmetic over all kinds of
    tables: every slot and token is one of the call's), so outputs, saved and workspaces
    keep what lies around them."""
    T, H, Hk, n = 100, 2, 1, 3
    x = inputs(d, 1, H, Hk, T, d, d, dtype, n=n)
    g = to_gpu(x, dtype, dtype)
    args = [g[m] for m in ("q", "k", "v", "log_alpha", "beta")]
    cu = torch.tensor(table, dtype=torch.int32, device="cuda")
    desc = ws.make_delta_desc(1, T, H, Hk, d, d, CODE[dtype], CODE[dtype], n_seq=n, flags=flags, segments=segments,
                              scale=d ** -0.5)
    room = lambda t: Guarded(t.numel() * t.element_size())  # noqa: E731
    for save in (True, False):
        y, end = room(g["v"]), room(g["state"])
        saved = Guarded(ws.delta_saved_size(desc)) if save else None
        fws, bws = (Guarded(b) for b in ws.delta_workspace_size(desc, save))
        call("gl_delta_fwd", desc, [*args, g["state"], cu, y.like(g["v"]), end.like(g["state"]),
                                    saved.inside if save else None], fws.inside)
        outs = [room(t) for t in args] + [room(g["dstate"])]
        call("gl_delta_bwd", desc, [*args, g["state"], cu, g["dy"], g["dstate"], saved.inside if save else None,
                                    *(o.like(t) for o, t in zip(outs, [*args, g["dstate"]]))], bws.inside)
        torch.cuda.synchronize()
        for m in [y, end, fws, bws, *outs] + ([saved] if save else []):
            assert m.whole()
