"""The norms around a block on rows of 8 to 63 elements, the narrowest that are computed
in fp32, against their definitions in 64 bits and those ones' gradients.

Tolerances (2-norm): those of wider rows for values drawn alike.  Where one element is M times the
others, v = M e_k + small ones, the gradient dv = r (g - hat mean(g hat)) all but cancels in that
element (hat_k^2 / d is 1 but for 1 / M^2): it is off by a few roundings of r g_k, as much as the other
elements' own values are (r g_j), so that dv as a whole keeps the bound of wider rows.  What multiplies that
element's dv by something M times as large as its other factors is off by M times that, of
a sum whose other terms have no such factor: the gate's gradient where the gate comes first (dz = dv x
silu'(z)) and the block norm's weight (dwx = sum dr hat(x)).  They get M times the bound."""
import pytest
import torch

import ssm_ref as ref
import weight_scans_amd as ws
from ssm_ref import BF16, F32, F64, rel
from test_gpu_blocknorm import add_case, check, gate_case, rows
from test_gpu_conv import SUM_TOL, TOL, dev

pytestmark = pytest.mark.gpu

SIZES = [8, 9, 15, 16, 33, 40, 63]
M = 30.0


@pytest.mark.parametrize("dtype,res", [(F64, F64), (F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("d", SIZES)
@pytest.mark.parametrize("post", [False, True])
def test_add_norm(d, post, dtype, res):
    add_case(d, 2, 19, d, dtype, res, post=post)
    add_case(d + 100, 3, 70, d, dtype, res, post=post, dro=False)


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("d", SIZES)
def test_gated_norm(d, first, dtype):
    gate_case(d, 2, 17, 3, d, dtype, first)
    gate_case(d + 100, 1, 45, 2, d, dtype, first, group=True)


def peaked(seed, dtype, *shape):
    """Rows of which one element, another one in each, is M times the size of the others."""
    x = rows(seed, dtype, *shape)
    at = torch.arange(x[..., 0].numel()).view(*shape[:-1], 1) % shape[-1]
    return x.scatter(-1, at, M * (1 - 2.0 * (at % 2)).to(F64))


@pytest.mark.parametrize("dtype,res", [(F64, F64), (F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("d", [8, 9, 16, 40])
@pytest.mark.parametrize("post", [False, True])
def test_add_norm_of_one_large_element(d, post, dtype, res):
    B, T = 2, 23
    x, r, dn, dr = peaked(1, dtype, B, T, d), peaked(2, res, B, T, d), rows(3, dtype, B, T, d), rows(4, res, B, T, d)
    w, wx, sc = (rows(5 + i, dtype, d) for i in range(3))
    wx = wx if post else None
    leaves = {n: t.requires_grad_(True) for n, t in (("x", x), ("r", r), ("w", w), ("wx", wx), ("scale", sc)) if t is not None}
    n, ro = ref.add_norm(x, r, w, wx, sc, 1e-6)
    want = dict(zip(leaves, torch.autograd.grad((n * dn).sum() + (ro * dr).sum(), list(leaves.values()))))
    at = lambda t, k: dev(None if t is None else t.detach(), k)  # noqa: E731
    args = (at(x, dtype), at(r, res), at(w, dtype), at(wx, dtype), at(sc, dtype))
    ng, rg = ws.gl_addnorm_fwd(*args)
    got = ws.gl_addnorm_bwd(*args, at(dn, dtype), at(dr, res))
    torch.cuda.synchronize()
    errs = {"n": (rel(ng, n), TOL[dtype]), "r": (rel(rg, ro), TOL[res])}
    for name, t in zip(("x", "r", "w", "wx", "scale"), got):
        if name in want:
            errs["d" + name] = (rel(t, want[name]), TOL[t.dtype] if name in ("x", "r") else SUM_TOL[dtype] * (
                M if name == "wx" else 1))
    check(errs)


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("d", [8, 9, 16, 40])
def test_gated_norm_of_one_large_element(d, first, dtype):
    B, T, G = 2, 11, 2
    x, z, dy, w = peaked(1, dtype, B, T, G, d), rows(2, dtype, B, T, G, d), rows(3, dtype, B, T, G, d), rows(4, dtype, d)
    leaves = [t.requires_grad_(True) for t in (x, z, w)]
    y = ref.gated_norm(*leaves, 1e-6, first)
    want = torch.autograd.grad((y * dy).sum(), leaves)
    args = [dev(t.detach(), dtype) for t in leaves]
    yg = ws.gl_gatenorm_fwd(*args, gate_first=first)
    got = ws.gl_gatenorm_bwd(*args, dev(dy, dtype), gate_first=first)
    torch.cuda.synchronize()
    errs = {"y": (rel(yg, y), TOL[dtype])}
    # bf16: the rounding, and beside it the fp32 bound times M
    dz = TOL[dtype] if not first else M * TOL[dtype] if dtype != BF16 else TOL[BF16] + M * TOL[F32]
    for name, t, u, bound in zip(("x", "z", "w"), got, want, (TOL[dtype], dz, SUM_TOL[dtype])):
        errs["d" + name] = (rel(t, u), bound)
    check(errs)
