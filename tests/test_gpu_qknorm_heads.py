"""Query / key norms on the GPU where one of the two has no heads, or no token is
there: values and gradients of the other, weight gradients of zero."""
import pytest
import torch

import weight_scans_amd as ws
from delta_ref import qknorm, rel
from test_gpu_qknorm import BF16, DW_TOL, F32, F64, TOL

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("Hq,Hk", [(5, 0), (0, 2)])
@pytest.mark.parametrize("d,rot", [(64, 32), (50, 20), (7, 2)])
def test_one_without_heads(Hq, Hk, d, rot, dtype):
    torch.manual_seed(d)
    B, T = 2, 37
    make = lambda *s: torch.randn(s, device="cuda", dtype=F64).to(dtype)  # noqa: E731
    q, k, dq, dk = make(B, Hq, T, d), make(B, Hk, T, d), make(B, Hq, T, d), make(B, Hk, T, d)
    wq, wk = make(d), make(d)
    gd = F64 if dtype == F64 else F32
    cos, sin = torch.randn(2, T, rot // 2, device="cuda", dtype=gd)
    oq, ok = ws.gl_qknorm_rope_fwd(q, k, wq, wk, cos, sin)
    gq, gk, gwq, gwk = ws.gl_qknorm_rope_bwd(q, k, wq, wk, cos, sin, dq, dk)
    assert oq.shape == q.shape and ok.shape == k.shape and gq.shape == q.shape and gk.shape == k.shape
    c = lambda t: t.detach().double().cpu()  # noqa: E731
    x, w, o, up, gx, gw, none = (q, wq, oq, dq, gq, gwq, gwk) if Hq else (k, wk, ok, dk, gk, gwk, gwq)
    xx, ww = c(x).requires_grad_(True), c(w).requires_grad_(True)
    y = qknorm(xx, ww, c(cos), c(sin), torch.arange(T)[None].expand(B, T), 1e-6, 1.0)
    rx, rw = torch.autograd.grad((y * c(up)).sum(), [xx, ww])
    assert rel(o, y) <= TOL[dtype] and rel(gx, rx) <= TOL[dtype] and rel(gw, rw) <= DW_TOL[dtype]
    assert (none == 0).all()


@pytest.mark.parametrize("B,T,Hq,Hk", [(0, 5, 2, 1), (2, 0, 2, 1), (2, 5, 0, 0)])
def test_without_rows_the_weights_get_zero(B, T, Hq, Hk):
    q, k = torch.randn(B, Hq, T, 64, device="cuda"), torch.randn(B, Hk, T, 64, device="cuda")
    w = torch.randn(64, device="cuda")
    gq, gk, gwq, gwk = ws.gl_qknorm_rope_bwd(q, k, w, w, None, None, q, k)
    assert gq.shape == q.shape and gk.shape == k.shape and (gwq == 0).all() and (gwk == 0).all()
