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


def test_gates_of_other_strides():
    """Strides of dimensions of one element say nothing; gates in different orders are
    brought into one for the autograd form."""
    x = inputs(4, 1, 4, 2, 70, 64, 64, BF16, F32)
    g = to_gpu(x, BF16, F32)
    both = torch.cat([g["log_alpha"], g["beta"]], 1)
    log_alpha, beta = both[:, :4], g["beta"]
    assert log_alpha.stride() != beta.stride()
    q, k, v = g["q"], g["k"], g["v"]
    y0, s0, _ = ws.gl_delta_fwd(q, k, v, g["log_alpha"], g["beta"], want_state=True)
    y1, s1, saved = ws.gl_delta_fwd(q, k, v, log_alpha, beta, want_state=True, save=True)
    assert rel(y1, y0.double().cpu()) <= TOL[BF16] and rel(s1, s0.double().cpu()) <= STATE_TOL[BF16]
    one = ws.gl_delta_bwd(q, k, v, g["log_alpha"], g["beta"], g["dy"])
    for a, b in zip(ws.gl_delta_bwd(q, k, v, log_alpha, beta, g["dy"], saved)[:5], one[:5]):
        assert torch.equal(a, b)
    pools = [torch.zeros((1, 4, 64, 64), device="cuda") for _ in range(2)]
    tok = lambda *t: [z[:, :, 0] for z in t]  # noqa: E731
    ya = ws.gl_delta_step(*tok(q, k, v, g["log_alpha"], g["beta"]), pools[0])
    one = torch.cat([g["log_alpha"][:, :, 0], g["beta"][:, :, 0]], 1)
    yb = ws.gl_delta_step(*tok(q, k, v), one[:, :4], one[:, 4:].contiguous(), pools[1])
    assert torch.equal(ya, yb) and torch.equal(*pools)
    with pytest.raises(ValueError):  # heads 70 and 1 elements apart: strides that matter
        ws.gl_delta_step(*tok(q, k, v), both[:, :4, 0], g["beta"][:, :, 0].contiguous(), pools[1])


@pytest.mark.parametrize("B", [1, 2])
def test_gates_of_other_orders_in_autograd(B):
    x = inputs(5, B, 4, 2, 70, 64, 64, BF16, F32)
    for n in ("log_alpha", "beta"):
        x[n].requires_grad_(True)
    y, _ = delta(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], 0.125)
    want = torch.autograd.grad((y * x["dy"]).sum(), [x["log_alpha"], x["beta"]])
    g = to_gpu(x, BF16, F32)
    la = g["log_alpha"].clone().requires_grad_(True)
    be = g["beta"].transpose(1, 2).contiguous().requires_grad_(True)  # [B,T,H]
    got, _ = ws.delta_rule(g["q"], g["k"], g["v"], la, be.transpose(1, 2))
    (got.float() * g["dy"].float()).sum().backward()
    assert rel(got, y) <= TOL[BF16]
    assert rel(la.grad, want[0]) <= TOL[BF16] and rel(be.grad.transpose(1, 2), want[1]) <= TOL[BF16]
    with torch.no_grad():
        again, _ = ws.delta_rule(g["q"], g["k"], g["v"], la, be.transpose(1, 2))
    assert rel(again, y) <= TOL[BF16]


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
def test_key_heads_without_value_heads(dtype):
    """No value head reads the keys: their gradients are zero, not left as they were."""
    B, Hk, T, d = 2, 3, 70, 16
    q = torch.ones((B, Hk, T, d), dtype=dtype, device="cuda")
    none = torch.ones((B, 0, T, d), dtype=dtype, device="cuda")
    gates = torch.ones((B, 0, T), dtype=dtype, device="cuda")
    code = {F64: ws.GL_DTYPE_F64, F32: ws.GL_DTYPE_F32, BF16: ws.GL_DTYPE_BF16}[dtype]
    desc = ws.make_delta_desc(B, T, 0, Hk, d, d, code, code)
    wide = [torch.full((B, T, Hk, d + 8), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    for n in ("sdq", "sdk"):
        s = wide[0].stride()
        setattr(desc, n, ws.delta.Strides(s[0], s[2], s[1]))
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    args = [ptr(q), ptr(q)] + [None] * 8 + [ptr(w) for w in wide] + [None] * 4
    status = ws.delta_lib().gl_delta_bwd(ctypes.byref(desc), *args, None, 0,
                                         ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert status == 0
    for w in wide:
        assert (w[..., :d] == 0).all() and (w[..., d:] == 7).all()
    dq, dk = ws.gl_delta_bwd(q, q, none, gates, gates, none)[:2]
    assert (dq == 0).all() and (dk == 0).all()


def test_numbers_held_in_tensors():
    """A scale that is a tensor is read at each call, not remembered by which tensor it is."""
    _, p = leaves(6, F32)
    p = {n: t.detach() for n, t in p.items()}
    scale = torch.tensor(0.5)
    for s in (0.5, 0.25, 2.0):
        scale.fill_(s)
        assert torch.equal(rule(p, scale=scale)[0], rule(p, scale=s)[0])
        one = [p[n][:, :, 0] for n in NAMES[:5]]
        assert torch.equal(ws.gl_delta_step(*one, p["state"].clone(), scale=scale),
                           ws.gl_delta_step(*one, p["state"].clone(), scale=s))
        for a, b in zip(ws.gl_qknorm_rope_fwd(p["q"], p["k"], q_scale=scale, k_scale=scale, eps=scale),
                        ws.gl_qknorm_rope_fwd(p["q"], p["k"], q_scale=s, k_scale=s, eps=s)):
            assert torch.equal(a, b)


def test_what_takes_no_gradient_is_refused():
    """No gradient is formed for the scales and the tables: one that wants it is not left without."""
    _, p = leaves(7, F32)
    scale = torch.tensor(0.5, requires_grad=True)
    table = torch.rand(100, 8, device="cuda", requires_grad=True)
    with pytest.raises(TypeError):
        rule(p, scale=scale)
    with pytest.raises(TypeError):
        ws.qknorm_rope(p["q"], p["k"], q_scale=scale)
    for tables in ((table, table.detach()), (table.detach(), table)):
        with pytest.raises(ValueError):
            ws.qknorm_rope(p["q"], p["k"], None, None, *tables)
        with torch.no_grad():
            ws.qknorm_rope(p["q"], p["k"], None, None, *tables)


@pytest.mark.parametrize("dtype,d", [(F64, 7), (F32, 7), (BF16, 64)])
@pytest.mark.parametrize("T", [2, 70])
def test_states_and_gates_that_are_broadcast_or_begin_anywhere(dtype, d, T):
    """A first state shared by the batch, one out of a pool whose entries are no 16 bytes
    long, gates that are one number for all: as their copies, gradients included."""
    x, p = leaves(8, dtype, T, B=2, d=d)
    p = {n: t.detach() for n, t in p.items()}
    st = p["state"].dtype
    first = p["state"][:1].clone().requires_grad_(True)
    pool = torch.cat([torch.zeros(1, 2, d, d, dtype=st, device="cuda"), p["state"]]).flatten()
    pool = torch.cat([torch.zeros(1, dtype=st, device="cuda"), pool]).requires_grad_(True)
    gate = torch.tensor(-0.25, dtype=p["beta"].dtype, device="cuda", requires_grad=True)
    wide = gate.expand(2, 2, T)
    cases = [(first, first.expand(2, -1, -1, -1), p["log_alpha"], p["beta"]),
             (pool, pool[1:].view(3, 2, d, d)[1:], p["log_alpha"], p["beta"]),
             (gate, p["state"], wide, -wide), (gate, p["state"], wide, p["beta"])]
    for leaf, state, log_alpha, beta in cases:
        copies = [t.clone(memory_format=torch.contiguous_format) for t in (state, log_alpha, beta)]
        both = []
        for s, a, b in ((state, log_alpha, beta), copies):
            with torch.no_grad():
                quiet = ws.delta_rule(p["q"], p["k"], p["v"], a, b, state=s, want_state=True)
            y, end = ws.delta_rule(p["q"], p["k"], p["v"], a, b, state=s, want_state=True)
            g, = torch.autograd.grad([y, end], leaf, [p["dy"], p["dstate"]], retain_graph=True)
            both.append([*quiet, y, end, g])
        for a, b in zip(*both):
            assert torch.equal(a, b)
