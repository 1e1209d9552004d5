"""The autograd forms of the gated delta rule and of the norms on the GPU: what
they cannot differentiate they refuse, and gradients arrive from any place."""
import ctypes

import pytest
import torch
from torch.autograd import forward_ad

import weight_scans_amd as ws
from delta_ref import delta, inputs, rel
from test_gpu_delta import BF16, F32, F64, STATE_TOL, TOL, to_gpu

pytestmark = pytest.mark.gpu

NAMES = ["q", "k", "v", "log_alpha", "beta", "state"]


def leaves(seed, dtype, T=80, B=1, H=2, Hk=2, d=64):
    x = inputs(seed, B, H, Hk, T, d, d, dtype)
    return x, {n: t.requires_grad_(True) for n, t in to_gpu(x, dtype, dtype).items()}


def rule(p, **kw):
    return ws.delta_rule(*[p[n] for n in NAMES[:5]], state=p["state"], **kw)


def test_forward_mode_is_refused():
    """There is no forward-mode derivative: a dual tensor is not taken for a constant."""
    _, p = leaves(1, F32)
    p = {n: t.detach() for n, t in p.items()}
    for n in NAMES:
        with forward_ad.dual_level():
            duals = {**p, n: forward_ad.make_dual(p[n], torch.ones_like(p[n]))}
            with pytest.raises(RuntimeError):
                rule(duals)
    with forward_ad.dual_level():
        assert torch.equal(rule(p)[0], rule(p)[0])  # no dual among them
        with pytest.raises(RuntimeError):
            ws.qknorm_rope(forward_ad.make_dual(p["q"], torch.ones_like(p["q"])), p["k"])


def test_second_derivatives_are_refused():
    """Gradients of gradients would lose what runs through the rule or the norms."""
    _, p = leaves(2, F32)
    y, end = rule(p, want_state=True)
    dq, = torch.autograd.grad(y.square().sum() + end.square().sum(), p["q"], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (dq.square().sum() + p["q"].square().sum()).backward()
    qn, kn = ws.qknorm_rope(p["q"], p["k"])
    dq, = torch.autograd.grad(qn.pow(3).sum() + kn.pow(3).sum(), p["q"], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (dq.square().sum() + p["q"].square().sum()).backward()


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("T", [3, 80])
def test_gradients_that_begin_anywhere(dtype, T):
    """Upstream gradients that are slices of a longer vector: of y, of the final state, of both norms."""
    x, p = leaves(3, dtype, T)
    for n in NAMES:
        x[n].requires_grad_(True)
    wy, wend = delta(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], 0.125, x["state"])
    up, ups = x["dy"], x["dstate"]
    want = torch.autograd.grad((wy * up).sum() + (wend * ups).sum(), [x[n] for n in NAMES])
    y, end = rule(p, want_state=True)
    side = torch.zeros(3, device="cuda")
    a = (torch.cat([side.to(y.dtype), y.flatten()]) * torch.cat([side.to(y.dtype), up.to(y.dtype).cuda().flatten()])).sum()
    b = (torch.cat([side.to(end.dtype), end.flatten()])
         * torch.cat([side.to(end.dtype), ups.to(end.dtype).cuda().flatten()])).sum()
    torch.autograd.backward([a, b])
    for n, w in zip(NAMES, want):
        assert rel(p[n].grad, w) <= (2 * STATE_TOL[dtype] if n == "state" else TOL[dtype]), n
    qn, kn = ws.qknorm_rope(p["q"], p["k"])
    ref = torch.autograd.grad(qn, p["q"], x["dy"].to(dtype).cuda())[0]
    qn, kn = ws.qknorm_rope(p["q"], p["k"])
    both = torch.cat([side[:1].to(dtype), qn.flatten(), kn.flatten()])
    w = torch.cat([side[:1].to(dtype), x["dy"].to(dtype).cuda().flatten(), torch.zeros_like(kn).flatten()])
    assert rel(torch.autograd.grad((both * w).sum(), p["q"])[0], ref.double().cpu()) <= TOL[dtype]
