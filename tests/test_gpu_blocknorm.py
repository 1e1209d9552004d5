"""The norms around a block on the GPU against their definitions in 64 bits and
those ones' gradients.

Tolerances (2-norm): what is rounded to bf16 once 4e-3 (each value is off by at most half a
step, 2^-8 = 3.91e-3 of it, and so the norm of all); fp32 1e-6 for rows (a few
roundings of 6e-8; sums over a row are off by less), 2e-6 for the weights' sums; fp64
1e-12."""
import pytest
import torch

import ssm_ref as ref
import weight_scans_amd as ws
from ssm_ref import BF16, F32, F64, par, rel
from test_gpu_conv import SUM_TOL, TOL, dev

pytestmark = pytest.mark.gpu


def check(errs):
    print({n: f"{e:.1e}" for n, (e, _) in errs.items()}, flush=True)
    for n, (e, bound) in errs.items():
        assert e <= bound, (n, e, bound)


def rows(seed, dtype, *shape, big=1.0):
    g = torch.Generator().manual_seed(seed)
    return (big * torch.randn(shape, generator=g, dtype=F64)).to(dtype).double()


def add_case(seed, B, T, d, dtype, res=None, post=True, scale=True, strided=False, dro=True, eps=1e-6):
    res = res or dtype
    x, r, dn, dr = rows(seed, dtype, B, T, d), rows(seed + 1, res, B, T, d, big=2), rows(seed + 2, dtype, B, T, d), rows(
        seed + 3, res, B, T, d)
    w, wx, sc = (rows(seed + 4 + i, dtype, d) for i in range(3))
    wx, sc = wx if post else None, sc if scale else None
    leaves = {n: t.requires_grad_(True) for n, t in (("x", x), ("r", r), ("w", w), ("wx", wx), ("scale", sc)) if t is not None}
    n, ro = ref.add_norm(x, r, w, wx, sc, eps)
    loss = (n * dn).sum() + ((ro * dr).sum() if dro else 0)
    want = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    at = lambda t, k, s=False: dev(None if t is None else t.detach(), k, s)  # noqa: E731
    args = (at(x, dtype, strided), at(r, res, strided), at(w, dtype), at(wx, dtype), at(sc, dtype))
    ng, rg = ws.gl_addnorm_fwd(*args, eps=eps)
    got = ws.gl_addnorm_bwd(*args, at(dn, dtype, strided), at(dr, res, strided) if dro else None, eps=eps)
    torch.cuda.synchronize()
    errs = {"n": (rel(ng, n), TOL[dtype]), "r": (rel(rg, ro), TOL[res])}
    for name, t in zip(("x", "r", "w", "wx", "scale"), got):
        if name not in want:
            assert t is None
            continue
        assert t.dtype == (res if name == "r" else dtype if name == "x" else par(dtype))
        errs["d" + name] = (rel(t, want[name]), SUM_TOL[dtype] if name not in ("x", "r") else TOL[t.dtype])
    check(errs)


@pytest.mark.parametrize("dtype,res", [(F64, F64), (F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("d", [1, 7, 64, 128, 136, 500, 512, 1000, 2048, 4104])
@pytest.mark.parametrize("post", [False, True])
def test_add_norm_sizes(d, post, dtype, res):
    add_case(d, 2, 19, d, dtype, res, post=post)


@pytest.mark.parametrize("dtype,d", [(F32, 8192), (BF16, 8200), (BF16, 16384), (F32, 16383), (F64, 16384)])
def test_add_norm_wide(d, dtype):
    add_case(d, 1, 3, d, dtype)


@pytest.mark.parametrize("dtype,res", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("kw", [dict(scale=False), dict(scale=False, post=False), dict(dro=False), dict(strided=True),
                                dict(strided="odd"), dict(eps=0.5)])
def test_add_norm_without_and_strided(kw, dtype, res):
    add_case(3, 3, 37, 264, dtype, res, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_add_norm_many_rows(dtype):
    """More rows than parts of the sums."""
    add_case(5, 3, 1400, 96, dtype)
    add_case(6, 1, 2100, 640, dtype)


def gate_case(seed, B, T, G, d, dtype, first=False, group=False, z=True, w=True, strided=False, order="btgd", eps=1e-6):
    x, dy = rows(seed, dtype, B, T, G, d), rows(seed + 1, dtype, B, T, G, d)
    zz = rows(seed + 2, dtype, B, T, G, d) if z else None
    ww = rows(seed + 3, dtype, *((G, d) if group else (d,))) if w else None
    leaves = {n: t.requires_grad_(True) for n, t in (("x", x), ("z", zz), ("w", ww)) if t is not None}
    y = ref.gated_norm(x, zz, ww, eps, first)
    want = dict(zip(leaves, torch.autograd.grad((y * dy).sum(), list(leaves.values()))))

    def at(t, s=False):
        t = dev(None if t is None else t.detach(), dtype, s)
        return t.transpose(1, 2).contiguous().transpose(1, 2) if s is False and t is not None and t.dim() == 4 and order == "bgtd" else t
    args = (at(x, strided), at(zz, strided), at(ww))
    yg = ws.gl_gatenorm_fwd(*args, eps=eps, gate_first=first)
    got = ws.gl_gatenorm_bwd(*args, at(dy, strided), eps=eps, gate_first=first)
    torch.cuda.synchronize()
    errs = {"y": (rel(yg, y), TOL[dtype])}
    for name, t in zip(("x", "z", "w"), got):
        if name not in want:
            assert t is None
            continue
        errs["d" + name] = (rel(t, want[name]), SUM_TOL[dtype] if name == "w" else TOL[dtype])
    check(errs)


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("G,d", [(1, 1), (3, 7), (2, 64), (4, 128), (2, 200), (1, 513), (2, 1000), (1, 2048), (1, 5000)])
def test_gated_norm_sizes(G, d, first, dtype):
    gate_case(G + d, 2, 17, G, d, dtype, first)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("kw", [dict(group=True), dict(z=False), dict(w=False), dict(z=False, w=False), dict(strided=True),
                                dict(strided="odd"), dict(order="bgtd", group=True), dict(order="bgtd"), dict(eps=0.5)])
def test_gated_norm_without_and_strided(kw, first, dtype):
    gate_case(7, 2, 40, 3, 72, dtype, first, **kw)


@pytest.mark.parametrize("group", [False, True])
def test_gated_norm_many_rows(group):
    gate_case(9, 2, 1100, 8, 64, F32, group=group)
    gate_case(10, 1, 1300, 2, 600, BF16, group=group)


def test_zero_rows_and_rows_of_zeros():
    x = torch.zeros(1, 4, 32, device="cuda")
    w = torch.ones(32, device="cuda")
    n, r = ws.gl_addnorm_fwd(x, x, w, w)
    assert not n.any() and not r.any()
    got = ws.gl_addnorm_bwd(x, x, w, w, None, torch.ones_like(x))
    assert all(t.isfinite().all() for t in got if t is not None)
    assert ws.gl_gatenorm_fwd(x, x, w).isfinite().all()
    for shape in ((0, 3, 32), (2, 0, 32)):
        e = torch.zeros(shape, device="cuda")
        assert ws.gl_addnorm_fwd(e, e, w)[0].shape == shape
        assert not ws.gl_addnorm_bwd(e, e, w, None, None, e)[2].any()
        assert not ws.gl_gatenorm_bwd(e, e, w, e)[2].any()


def test_large_gates():
    """Gates so negative that e^-z overflows, and as large."""
    z = torch.tensor([-200.0, -100.0, -30.0, 0.0, 30.0, 200.0], device="cuda").expand(1, 5, 6).contiguous()
    x = torch.randn(1, 5, 6, device="cuda")
    y = ws.gl_gatenorm_fwd(x, z)
    want = ref.gated_norm(x.double().cpu(), z.double().cpu(), None, 1e-6, False)
    assert rel(y, want) <= 1e-6 and y.isfinite().all()
    dx, dz, _ = ws.gl_gatenorm_bwd(x, z, None, torch.ones_like(x))
    assert dx.isfinite().all() and dz.isfinite().all()


def test_autograd_and_differences():
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=F64).cuda().requires_grad_(True)  # noqa: E731
    assert torch.autograd.gradcheck(lambda *a: ws.add_norm(*a), (rnd(2, 3, 5), rnd(2, 3, 5), rnd(5), rnd(5), rnd(5)),
                                    eps=1e-6, atol=1e-7)
    for first in (False, True):
        assert torch.autograd.gradcheck(lambda *a: ws.gated_norm(*a, gate_first=first),
                                        (rnd(2, 3, 2, 5), rnd(2, 3, 2, 5), rnd(2, 5)), eps=1e-6, atol=1e-7)
