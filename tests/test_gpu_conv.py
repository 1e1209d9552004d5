"""The short causal convolution on the GPU against its definition in 64 bits and
that one's gradients.

Tolerances (2-norm): what is rounded to bf16 once 4e-3 (each value is off by at most half a
step, 2^-8 = 3.91e-3 of it, and so the norm of all, beside some 1e-6 of fp32); fp32 1e-6 (some ten roundings of 6e-8, the exponential of
the gate among them), sums for the weights 2e-6 (their terms' errors do not grow);
fp64 1e-12.  The inputs are values of their type, so that the oracle has the same."""
import pytest
import torch

import ssm_ref as ref
import weight_scans_amd as ws
from ssm_ref import BF16, F32, F64, par, rel

pytestmark = pytest.mark.gpu

TOL = {F64: 1e-12, F32: 1e-6, BF16: 4e-3}
SUM_TOL = {F64: 1e-12, F32: 2e-6, BF16: 2e-6}


def inputs(seed, B, T, D, K, dtype, lens=None, state=True, bias=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=F64).to(dtype).double()  # noqa: E731
    n = B if lens is None else len(lens)
    return {"x": rnd(B, T, D), "w": rnd(D, K) * 0.5, "bias": rnd(D) * 0.25 if bias else None,
            "state": rnd(n, K - 1, D) if state else None, "dy": rnd(B, T, D), "dstate": rnd(n, K - 1, D)}


def dev(t, dtype, strided=False):
    if t is None:
        return None
    t = t.to(dtype).cuda()
    if not strided:
        return t
    buf = torch.full((*t.shape[:-1], 2 * t.shape[-1] + 3), torch.nan, dtype=dtype, device="cuda")
    out = buf[..., 1 : 1 + t.shape[-1]] if strided == "odd" else buf[..., : t.shape[-1]]
    return out.copy_(t)


def cu(lens):
    if lens is None:
        return None
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")


def case(seed, B, T, D, K, dtype, lens=None, state=True, bias=True, silu=True, strided=False, dstate=True):
    x = inputs(seed, B, T, D, K, dtype, lens, state, bias)
    leaves = {n: x[n].requires_grad_(True) for n in ("x", "w", "bias", "state") if x[n] is not None}
    y, end = ref.conv(x["x"], x["w"], x["bias"], x["state"], lens, silu)
    loss = (y * x["dy"]).sum() + ((end * x["dstate"]).sum() if dstate else 0)
    want = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)))
    g = {n: dev(None if t is None else t.detach(), dtype, strided if n in ("x", "dy") else False) for n, t in x.items()}
    yg, eg = ws.gl_conv_fwd(g["x"], g["w"], g["bias"], state=g["state"], want_state=True, cu_seqlens=cu(lens), silu=silu)
    got = ws.gl_conv_bwd(g["x"], g["w"], g["bias"], g["dy"], state=g["state"], dstate=g["dstate"] if dstate else None,
                         cu_seqlens=cu(lens), silu=silu)
    torch.cuda.synchronize()
    assert torch.equal(eg.cpu(), end.detach().to(dtype))  # they are inputs
    errs = {"y": (rel(yg, y), TOL[dtype])}
    for n, t in zip(("x", "w", "bias", "state"), got):
        if n not in want:
            assert t is None
            continue
        assert t.dtype == (par(dtype) if n in ("w", "bias") else dtype)
        w = torch.zeros_like(t, dtype=F64, device="cpu") if want[n] is None else want[n]
        errs["d" + n] = (rel(t, w), (SUM_TOL if n in ("w", "bias") else TOL)[dtype])
    print({n: f"{e:.1e}" for n, (e, _) in errs.items()}, flush=True)
    for n, (e, tol) in errs.items():
        assert e <= tol, (n, e)


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("D,T", [(64, 100), (40, 33), (7, 50), (300, 3), (1, 1), (8, 2)])
def test_sizes(D, T, K, dtype):
    case(D + T + K, 2, T, D, K, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kw", [dict(bias=False), dict(silu=False), dict(state=False), dict(state=False, dstate=False),
                                dict(strided=True), dict(strided="odd"), dict(bias=False, silu=False, strided="odd")])
def test_without_and_strided(kw, dtype):
    case(5, 3, 70, 48, 4, dtype, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K", [2, 4, 7])
@pytest.mark.parametrize("lens", [[5, 0, 1, 40, 2, 16, 0], [0, 0, 3], [1] * 9, [130], [0, 64, 64, 0], [2, 3, 1, 1, 4]])
def test_packed(lens, K, dtype):
    case(len(lens) + K, 1, sum(lens), 24, K, dtype, lens=lens)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_runs_of_many_tokens(dtype):
    """Enough channels and tokens for runs of several tokens a thread, and several parts of the sums."""
    case(9, 2, 1500, 320, 4, dtype)
    case(10, 1, 3000, 257, 3, dtype, lens=[1000, 1, 0, 1700, 299])


def test_no_tokens_no_rows():
    for B, T in ((2, 0), (0, 5)):
        x = torch.randn(B, T, 16, device="cuda")
        w, state = torch.randn(16, 4, device="cuda"), torch.randn(B, 3, 16, device="cuda")
        y, end = ws.gl_conv_fwd(x, w, state=state, want_state=True)
        assert y.shape == x.shape and torch.equal(end, state)
        dstate = torch.randn_like(state)
        dx, dw, dbias, ds = ws.gl_conv_bwd(x, w, None, x, state=state, dstate=dstate)
        assert dx.shape == x.shape and dbias is None and not dw.any() and torch.equal(ds, dstate)


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("K", [1, 2, 4, 6])
@pytest.mark.parametrize("D", [64, 13])
def test_step(D, K, dtype):
    """Tokens one by one against a pool: outputs of whole passes (same sums in the same
    order, to a rounding), rows with nothing to do, states of others untouched."""
    x = inputs(D + K, 4, 6, D, K, dtype)
    g = {n: dev(None if t is None else t, dtype) for n, t in x.items()}
    pool = torch.randn(7, K - 1, D, device="cuda").to(dtype)
    slots = torch.tensor([5, -1, 0, 7], dtype=torch.int32, device="cuda")
    pool[5], pool[0] = g["state"][0], g["state"][2]
    before = pool.clone()
    y, end = ws.gl_conv_fwd(g["x"], g["w"], g["bias"], state=g["state"], want_state=True)
    for t in range(6):
        yt = ws.gl_conv_step(g["x"][:, t], g["w"], g["bias"], pool, slots=slots)
        for b in (0, 2):
            assert rel(yt[b], y[b, t]) <= TOL[dtype]
        assert not yt[1].any() and not yt[3].any()
    torch.cuda.synchronize()
    assert torch.equal(pool[5], end[0]) and torch.equal(pool[0], end[2])
    for k in (1, 2, 3, 4, 6):
        assert torch.equal(pool[k], before[k])
    one = g["state"].clone()  # without slots
    ws.gl_conv_step(g["x"][:, 0], g["w"], g["bias"], one)
    assert K == 1 or torch.equal(one[:, -1], g["x"][:, 0])


def test_autograd_and_differences():
    """The wrapper's gradients against differences of the forward, in 64 bits."""
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=F64).cuda().requires_grad_(True)  # noqa: E731
    args = (rnd(2, 5, 3), rnd(3, 3), rnd(3), rnd(2, 2, 3))
    f = lambda x, w, b, s: ws.causal_conv(x, w, b, state=s, want_state=True)  # noqa: E731
    assert torch.autograd.gradcheck(f, args, eps=1e-6, atol=1e-7)


def test_not_finite_stays_in_its_channel_and_window():
    x = torch.randn(1, 40, 16, device="cuda")
    w = torch.randn(16, 5, device="cuda")
    clean = ws.gl_conv_fwd(x, w)[0]
    x[0, 20, 3] = torch.inf
    y = ws.gl_conv_fwd(x, w)[0]
    hit = torch.zeros(1, 40, 16, dtype=torch.bool, device="cuda")
    hit[0, 20:25, 3] = True
    assert torch.equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("lens", [[70, 0, 20], [90, 0], [0, 0], [2, 1]])
@pytest.mark.parametrize("D,K,behind", [(40, 4, 1), (7, 3, 300), (64, 8, 40), (16, 1, 5)])
def test_tokens_behind_the_last_sequence(D, K, behind, lens, dtype):
    """They hold NaN: their outputs and gradients are zero, the others as without them."""
    T = sum(lens)
    g = {n: dev(t, dtype) for n, t in inputs(D + T, 1, T, D, K, dtype, lens).items()}
    p = {n: torch.cat([t, torch.full((1, behind, D), torch.nan, dtype=dtype, device="cuda")], 1) if n in ("x", "dy") else t
         for n, t in g.items()}
    run = lambda a: (*ws.gl_conv_fwd(a["x"], a["w"], a["bias"], state=a["state"], want_state=True,  # noqa: E731
                                     cu_seqlens=cu(lens)),
                     *ws.gl_conv_bwd(a["x"], a["w"], a["bias"], a["dy"], state=a["state"], dstate=a["dstate"],
                                     cu_seqlens=cu(lens)))
    # both are within the tolerance of the definition
    for n, want, got in zip(("y", "end", "x", "w", "bias", "state"), run(g), run(p)):
        if n in ("y", "x"):
            assert not got[:, T:].any(), n
            got = got[:, :T]
        assert rel(got, want) <= 2 * (SUM_TOL if n in ("w", "bias") else TOL)[dtype], n
