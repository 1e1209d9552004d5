"""Query / key norms with the rotation on the GPU against the definition in 64
bits and its autograd gradients.

Tolerances (2-norm): fp64 1e-12; fp32 1e-6 for rows (a few roundings of 6e-8),
4e-6 for the weights' sums; bf16 rows 2.5e-3 (one rounding, 1.7e-3 rms); the
weights' fp32 sums of bf16 runs as fp32's."""
import pytest
import torch

import weight_scans_amd as ws
from delta_ref import qknorm, rel

pytestmark = pytest.mark.gpu

F64, F32, BF16 = torch.float64, torch.float32, torch.bfloat16
TOL = {F64: 1e-12, F32: 1e-6, BF16: 2.5e-3}
DW_TOL = {F64: 1e-12, F32: 4e-6, BF16: 4e-6}


def case(seed, B, T, Hq, Hk, d, rot, dtype, interleaved=False, order="bthd", weights=True, pos="table", eps=1e-6,
         edit=None):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=F64).to(dtype).double()  # noqa: E731
    q, k, dq, dk = rnd(B, Hq, T, d), rnd(B, Hk, T, d), rnd(B, Hq, T, d), rnd(B, Hk, T, d)
    wq, wk = ((1 + 0.1 * rnd(d)).to(dtype).double() for _ in range(2)) if weights else (None, None)
    if edit:
        edit(q, k)
        q, k = q.to(dtype).double(), k.to(dtype).double()  # what the GPU receives
    gd = F64 if dtype == F64 else F32
    n_pos = T + 37
    ang = torch.arange(n_pos, dtype=F64)[:, None] * 100.0 ** (-torch.arange(rot // 2, dtype=F64) / max(1, rot // 2))
    cos, sin = (ang.cos().to(gd).double(), ang.sin().to(gd).double()) if rot else (None, None)
    p = torch.randint(-2, n_pos + 2, (B, T), generator=g) if pos == "table" else (7 + torch.arange(T)).expand(B, T)
    leaves = [t for t in (q, k, wq, wk) if t is not None]
    for t in leaves:
        t.requires_grad_(True)
    yq = qknorm(q, wq, cos, sin, p, eps, 0.7, interleaved)
    yk = qknorm(k, wk, cos, sin, p, eps, d ** -0.5, interleaved)
    want = torch.autograd.grad((yq * dq).sum() + (yk * dk).sum(), leaves)
    if not weights:
        want = (*want, None, None)

    def dev(t, kind=dtype):
        return None if t is None else t.detach().to(kind).cuda()
    if order == "bthd":  # slices of one buffer, as a fused projection writes it
        buf = torch.full((B, T, (Hq + Hk + 1) * d), torch.nan, dtype=dtype, device="cuda")
        gq = buf[..., : Hq * d].view(B, T, Hq, d).transpose(1, 2)
        gk = buf[..., Hq * d : (Hq + Hk) * d].view(B, T, Hk, d).transpose(1, 2)
        gq.copy_(dev(q))
        gk.copy_(dev(k))
    else:
        gq, gk = dev(q), dev(k)
    args = (gq, gk, dev(wq), dev(wk), dev(cos, gd), dev(sin, gd))
    opts = dict(eps=eps, q_scale=0.7, k_scale=d ** -0.5, interleaved=interleaved)
    opts |= {"pos": p.to(torch.int32).cuda()} if pos == "table" else {"pos0": 7}
    oq, ok = ws.gl_qknorm_rope_fwd(*args, **opts)
    got = ws.gl_qknorm_rope_bwd(*args, dev(dq), dev(dk), **opts)
    torch.cuda.synchronize()
    errs = {"q": (rel(oq, yq), TOL[dtype]), "k": (rel(ok, yk), TOL[dtype])}
    for n, a, b in zip(("dq", "dk", "dwq", "dwk"), got, want):
        if b is None:
            assert a is None
        else:
            errs[n] = (rel(a, b), (DW_TOL if "w" in n else TOL)[dtype])
    print({n: f"{e:.1e}" for n, (e, _) in errs.items()}, flush=True)
    for n, (e, tol) in errs.items():
        assert e <= tol, (n, e)
    return oq, ok, got


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 64), (64, 32), (128, 64), (80, 32), (256, 256), (16, 16),
                                   (48, 0), (96, 96)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_sizes(d, rot, dtype, interleaved):
    case(d + rot, 2, 33, 6, 2, d, rot, dtype, interleaved)


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("d,rot", [(1, 0), (2, 2), (5, 4), (72, 20), (100, 100), (130, 66), (255, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_odd_sizes(d, rot, dtype, interleaved):
    case(d * 3 + rot, 2, 9, 3, 1, d, rot, dtype, interleaved, order="bhtd")


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("d,rot", [(32, 30), (34, 16), (66, 0), (126, 62), (194, 194), (250, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_even_sizes(d, rot, dtype, interleaved):
    case(d + 7 * rot, 3, 21, 4, 3, d, rot, dtype, interleaved, order="bthd")


def test_rows_that_are_not_aligned():
    """Slices of a wider row: strides that 16 bytes do not divide."""
    for dtype in (F32, BF16):
        wide = torch.randn(2, 20, 3, 64 + 1, device="cuda").to(dtype)[..., :64].transpose(1, 2)
        oq, ok = ws.gl_qknorm_rope_fwd(wide, wide, q_scale=0.5)
        want = qknorm(wide.double().cpu(), None, None, None, None, 1e-6, 0.5)
        assert rel(oq, want) <= TOL[dtype] and rel(ok, 2 * want) <= TOL[dtype]
        dq, dk, _, _ = ws.gl_qknorm_rope_bwd(wide, wide, None, None, None, None, oq, ok, q_scale=0.5)
        x = wide.double().cpu().requires_grad_(True)
        z = qknorm(x, None, None, None, None, 1e-6, 0.5)
        ref = torch.autograd.grad((z * oq.double().cpu()).sum(), x)[0]
        # the gradient of half the squared norm nearly cancels (|out| hardly depends on |x|): against |dz| / |x|
        scale = 0.5 * oq.double().cpu().norm() / x.detach().norm() * 64 ** 0.5
        assert float((dq.double().cpu() - ref).norm()) <= 4 * TOL[dtype] * float(scale)
        assert torch.isfinite(dk.double()).all()


@pytest.mark.parametrize("B,T", [(1, 1), (64, 1), (1, 777), (3, 300)])
@pytest.mark.parametrize("Hq,Hk", [(16, 8), (1, 1), (5, 0), (0, 2)])
def test_tokens_and_heads(B, T, Hq, Hk):
    case(B * T, B, T, max(Hq, 1), max(Hk, 1), 128, 128, BF16)
    if Hq == 0 or Hk == 0:
        q = torch.randn(B, Hq, T, 64, device="cuda", dtype=BF16)
        k = torch.randn(B, Hk, T, 64, device="cuda", dtype=BF16)
        oq, ok = ws.gl_qknorm_rope_fwd(q, k)
        x, o = (q, oq) if Hq else (k, ok)
        assert rel(o, qknorm(x.double().cpu(), None, None, None, None, 1e-6, 1.0)) <= TOL[BF16]


def test_without_weights_and_with_a_running_position():
    for dtype in (F64, F32, BF16):
        case(1, 2, 40, 4, 2, 64, 64, dtype, weights=False, pos="run")
        case(2, 2, 40, 4, 2, 20, 8, dtype, weights=False, pos="run", order="bhtd")


def test_zero_rows_and_large_values():
    """A row of zeros (eps alone under the root) and rows near the type's ends."""
    def edit(q, k):
        q[0, 0, 0] = 0
        k[0, 0, 1] = 0
        q[0, 1, 2] *= 1e15
        k[0, 0, 3] *= 1e-3
    for dtype in (F32, BF16):
        case(3, 1, 8, 2, 2, 64, 64, dtype, edit=edit)
        case(4, 1, 8, 2, 2, 30, 10, dtype, edit=edit, order="bhtd")


def test_gradient_against_differences():
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=F64).cuda()  # noqa: E731
    q, k, wq, wk, dq, dk = rnd(1, 2, 3, 32), rnd(1, 1, 3, 32), rnd(32), rnd(32), rnd(1, 2, 3, 32), rnd(1, 1, 3, 32)
    cos, sin = rnd(3, 8), rnd(3, 8)
    got = ws.gl_qknorm_rope_bwd(q, k, wq, wk, cos, sin, dq, dk)
    for i in range(4):
        at = [q, k, wq, wk]
        d = rnd(*at[i].shape)

        def loss(h):
            z = list(at)
            z[i] = at[i] + h * d
            a, b = ws.gl_qknorm_rope_fwd(*z, cos, sin)
            return float((a * dq).sum() + (b * dk).sum())
        num, ana = (loss(1e-5) - loss(-1e-5)) / 2e-5, float((got[i] * d).sum())
        assert abs(num - ana) <= 1e-7 * max(1.0, abs(ana)), i


def test_autograd_repeats_bitwise():
    g = torch.Generator(device="cuda").manual_seed(6)
    x = [torch.randn(s, generator=g, device="cuda").to(BF16).requires_grad_(True)
         for s in ((2, 4, 500, 64), (2, 2, 500, 64), (64,), (64,))]
    ang = torch.randn((500, 32), generator=g, device="cuda")
    runs = []
    for _ in range(2):
        a, b = ws.qknorm_rope(*x, ang.cos(), ang.sin(), k_scale=0.125)
        runs.append([a, b, *torch.autograd.grad(a.float().sum() + b.float().square().sum(), x)])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d,rot", [(92, 46), (84, 84), (64, 64), (128, 64), (20, 8), (7, 2)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_slices_of_a_fused_row_at_any_element(d, rot, dtype):
    """q and k inside one wider row, k's part at an offset that no 16 bytes divide."""
    torch.manual_seed(d)
    rows = torch.randn(2, 13, 1 + 3 * d + 2 * d, device="cuda").to(dtype)
    q = rows[..., 1 : 1 + 3 * d].unflatten(-1, (3, d)).transpose(1, 2)
    k = rows[..., 1 + 3 * d :].unflatten(-1, (2, d)).transpose(1, 2)
    wide = torch.randn(2, d + 1, device="cuda").to(dtype)
    wq, wk = wide[0, 1:], wide[1, 1:]
    cos, sin = torch.randn(2, 16 * (rot // 2) + 1, device="cuda")[:, 1:].unflatten(-1, (16, rot // 2))
    oq, ok = ws.gl_qknorm_rope_fwd(q, k, wq, wk, cos, sin)
    dq = torch.randn(2, 3, 13, d + 1, device="cuda").to(dtype)[..., 1:]
    dk = torch.randn(2, 2, 13, d + 1, device="cuda").to(dtype)[..., 1:]
    got = ws.gl_qknorm_rope_bwd(q, k, wq, wk, cos, sin, dq, dk)
    pos = torch.arange(13)[None].expand(2, 13)
    c = lambda t: t.detach().double().cpu()  # noqa: E731
    for x, w, o, up, gx, gw in ((q, wq, oq, dq, got[0], got[2]), (k, wk, ok, dk, got[1], got[3])):
        xx, ww = c(x).requires_grad_(True), c(w).requires_grad_(True)
        y = qknorm(xx, ww, c(cos), c(sin), pos, 1e-6, 1.0)
        rx, rw = torch.autograd.grad((y * c(up)).sum(), [xx, ww])
        assert rel(o, y) <= TOL[dtype]
        assert rel(gx, rx) <= TOL[dtype] and rel(gw, rw) <= DW_TOL[dtype]
