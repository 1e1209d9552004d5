"""The selective scan on the GPU against its definition in 64 bits, token by token,
and that one's gradients.

Tolerances (2-norm): what is rounded to bf16 once 4e-3 (each value is off by at most half a
step, 2^-8 = 3.91e-3 of it, and so the norm of all).  fp32: a decay e^(D A) is off by
its argument's rounding and its own, (|D A| + 2) 6e-8, and a state carries what
came in k tokens ago through k of them: with a memory of L = 1 / |D A| tokens the
errors of L decays of about 1.3e-7 add up, by their squares, to 1.3e-7 sqrt(L),
2.3e-6 for L = 300 (the inputs' is at most that, as no sequence is longer but
test_few_channels', whose memory is as long in the first of their 16 states or more at
most); with the sums' own roundings 4e-6, and twice that for gradients, which
carry a state and an adjoint.  fp64 1e-12.  The inputs are values of their type."""
import pytest
import torch

import ssm_ref as ref
import weight_scans_amd as ws
from ssm_ref import BF16, F32, F64, par, rel
from test_gpu_conv import cu, dev

pytestmark = pytest.mark.gpu

TOL = {F64: 1e-12, F32: 4e-6}
NAMES = ("x", "dt", "A", "B", "C", "skip", "z", "dt_bias", "state")


def tol(name, dtype, grad):
    if dtype == BF16 and name in ("y", "x", "dt", "B", "C", "z"):
        return 4e-3
    return TOL[par(dtype)] * (2 if grad else 1)


def inputs(seed, B, T, D, N, G, dtype, lens=None, state=True, gate=True, skip=True, bias=True, softplus=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=F64)  # noqa: E731
    io = lambda t: t.to(dtype).double()  # noqa: E731
    pr = lambda t: t.to(par(dtype)).double()  # noqa: E731
    n = B if lens is None else len(lens)
    step = torch.exp(torch.rand(D, generator=g, dtype=F64) * 4.6 - 5.8)  # 0.003 .. 0.3
    dt = 0.5 * rnd(B, T, D) if softplus else step * torch.exp(0.5 * rnd(B, T, D))
    return {"x": io(rnd(B, T, D)), "dt": io(dt), "A": pr(-torch.exp(torch.arange(1, N + 1).double().log() + 0.1 * rnd(D, N))),
            "B": io(rnd(B, T, G, N)), "C": io(rnd(B, T, G, N)), "skip": pr(1 + 0.1 * rnd(D)) if skip else None,
            "z": io(rnd(B, T, D)) if gate else None,
            "dt_bias": pr(step + torch.log(-torch.expm1(-step)) if softplus else 0.01 * torch.rand(D, generator=g, dtype=F64))
            if bias else None,
            "state": pr(0.3 * rnd(n, D, N)) if state else None, "dy": io(rnd(B, T, D)), "dstate": pr(0.3 * rnd(n, D, N))}


def to_gpu(x, dtype, strided=False):
    out = {}
    for n, t in x.items():
        kind = par(dtype) if n in ("A", "skip", "dt_bias", "state", "dstate") else dtype
        out[n] = dev(None if t is None else t.detach(), kind, strided if n in ("x", "dt", "z", "B", "C", "dy") else False)
    return out


def check(errs):
    print({n: f"{e:.1e}" for n, (e, _) in errs.items()}, flush=True)
    for n, (e, bound) in errs.items():
        assert e <= bound, (n, e, bound)


def case(seed, B, T, D, N, G, dtype, lens=None, strided=False, softplus=True, dstate=True, saved=True, **kw):
    x = inputs(seed, B, T, D, N, G, dtype, lens, softplus=softplus, **kw)
    leaves = {n: x[n].requires_grad_(True) for n in NAMES if x[n] is not None}
    y, end = ref.scan(*(x[n] for n in NAMES), lens, softplus)
    loss = (y * x["dy"]).sum() + ((end * x["dstate"]).sum() if dstate else 0)
    want = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)))
    g = to_gpu(x, dtype, strided)
    args = [g[n] for n in NAMES[:8]]
    kw = dict(cu_seqlens=cu(lens), softplus=softplus, state=g["state"])
    yg, eg, keep = ws.gl_ssm_fwd(*args, want_state=True, save=saved, **kw)
    got = ws.gl_ssm_bwd(*args, g["dy"], keep, dstate=g["dstate"] if dstate else None, **kw)
    torch.cuda.synchronize()
    errs = {"y": (rel(yg, y), tol("y", dtype, False)), "end": (rel(eg, end), tol("end", dtype, False))}
    for n, t in zip(NAMES, got):
        if n not in want:
            assert t is None, n
            continue
        w = torch.zeros(t.shape, dtype=F64) if want[n] is None else want[n]
        errs["d" + n] = (rel(t, w), tol(n, dtype, True))
    check(errs)
    return g, args, kw, (yg, eg), got


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("N", [16, 1, 3, 8, 24, 64])
@pytest.mark.parametrize("D,T,B", [(64, 70, 2), (40, 33, 1), (5, 300, 2), (33, 1, 3), (96, 17, 1)])
def test_sizes(D, T, B, N, dtype):
    case(D + T + N, B, T, D, N, 1, dtype)


@pytest.mark.parametrize("dtype,N", [(F32, 65), (BF16, 128), (F32, 200), (F32, 256), (BF16, 256), (F64, 33), (F64, 100),
                                     (F64, 256)])
def test_many_states(N, dtype):
    """The kernels of fewer channels a work-group."""
    case(N, 1, 40, 20, N, 1, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("G", [2, 3])
@pytest.mark.parametrize("kw", [dict(), dict(gate=False), dict(skip=False, bias=False), dict(softplus=False),
                                dict(softplus=False, bias=False), dict(state=False), dict(state=False, dstate=False),
                                dict(strided=True), dict(strided="odd"), dict(saved=False)])
def test_groups_and_without(G, kw, dtype):
    case(G, 2, 90, 36 * G, 8, G, dtype, **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens", [[5, 0, 1, 40, 2, 16, 0], [0, 0, 3], [1] * 7, [300], [0, 256, 17, 0], [128, 128, 1]])
def test_packed(lens, dtype):
    case(len(lens), 1, sum(lens), 40, 16, 1, dtype, lens=lens)


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("D,T", [(40, 90), (12, 300), (64, 17)])
def test_tokens_that_pass_by(D, T, dtype):
    """Steps of softplus(-inf) or of the type's lowest value are 0: the state stays, dt's gradient is 0; also for
    all tokens of a row."""
    x = inputs(D, 3, T, D, 8, 1, dtype)
    low = torch.finfo(dtype).min
    x["dt"][0, : T // 2], x["dt"][1] = -torch.inf, low
    x["dt"][2, 1::2] = low
    leaves = {n: x[n].requires_grad_(True) for n in NAMES}
    y, end = ref.scan(*(x[n] for n in NAMES), None, True)
    want = torch.autograd.grad((y * x["dy"]).sum() + (end * x["dstate"]).sum(), list(leaves.values()))
    g = to_gpu(x, dtype)
    args = [g[n] for n in NAMES[:8]]
    yg, eg, saved = ws.gl_ssm_fwd(*args, state=g["state"], want_state=True, save=True)
    got = ws.gl_ssm_bwd(*args, g["dy"], saved, state=g["state"], dstate=g["dstate"])
    assert torch.equal(eg[1], g["state"][1])
    assert not got[1][0, : T // 2].any() and not got[1][1].any() and not got[1][2, 1::2].any()
    errs = {"y": (rel(yg, y), tol("y", dtype, False)), "end": (rel(eg, end), tol("end", dtype, False))}
    check(errs | {"d" + n: (rel(t, w), tol(n, dtype, True)) for n, t, w in zip(NAMES, got, want)})


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("lens", [[70, 0, 20], [90, 0], [0, 0]])
@pytest.mark.parametrize("D,G,behind", [(40, 2, 1), (12, 1, 300), (130, 1, 40)])
def test_tokens_behind_the_last_sequence(D, G, behind, lens, dtype):
    """They hold NaN: their outputs and gradients are zero, the others as without them."""
    T, N = sum(lens), 5
    g = to_gpu(inputs(D + T, 1, T, D, N, G, dtype, lens), dtype)
    pad = lambda n, t: t if n not in ("x", "dt", "B", "C", "z", "dy") else torch.cat(  # noqa: E731
        [t, torch.full((1, behind, *t.shape[2:]), torch.nan, dtype=dtype, device="cuda")], 1)
    p = {n: pad(n, t) for n, t in g.items()}
    kw = dict(cu_seqlens=cu(lens), state=g["state"])
    run = lambda a, save: (lambda f: (*f[:2], *ws.gl_ssm_bwd(  # noqa: E731
        *(a[n] for n in NAMES[:8]), a["dy"], f[2], dstate=a["dstate"], **kw)))(
            ws.gl_ssm_fwd(*(a[n] for n in NAMES[:8]), want_state=True, save=save, **kw))
    for save in (True, False):
        # both are within the tolerance of the definition
        for n, want, got in zip(("y", "end", *(NAMES)), run(g, save), run(p, save)):
            if n in ("x", "dt", "B", "C", "z", "y"):
                assert not got[:, T:].any(), n
                got = got[:, :T]
            assert rel(got, want) <= 2 * tol(n, dtype, True), n


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("N", [16, 100, 200])
@pytest.mark.parametrize("lens", [[200], [1100], [700, 0, 401], [1030, 3]])
def test_few_channels(lens, N, dtype):
    """Eight channels a work-group, slots of few and of many tokens, several tiles a sequence."""
    case(len(lens) + N, 1, sum(lens), 12, N, 1, dtype, lens=lens)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,D", [(4, 2048), (8, 4096), (1, 64)])
def test_channels_a_work_group(B, D, dtype):
    """Sizes at which the forward gives its work-groups 32, 64 and 16 channels, over several tiles: a sample of the
    channels against the definition."""
    T, N = 280, 4
    x = inputs(B + D, B, T, D, N, 1, dtype)
    pick = torch.arange(0, D, max(1, D // 16))
    g = to_gpu(x, dtype)
    args = [g[n] for n in NAMES[:8]]
    y, end, saved = ws.gl_ssm_fwd(*args, state=g["state"], want_state=True, save=True)
    got = ws.gl_ssm_bwd(*args, g["dy"], saved, state=g["state"], dstate=g["dstate"])
    torch.cuda.synchronize()
    cut = lambda n, t: t if t is None or n in ("B", "C") else t[pick] if n in ("A", "skip", "dt_bias") else (  # noqa: E731
        t[:, pick] if "state" in n else t[..., pick])
    s = {n: cut(n, t) for n, t in x.items()}
    leaves = {n: s[n].requires_grad_(True) for n in NAMES if n not in ("B", "C")}
    yr, er = ref.scan(*(s[n] for n in NAMES), None, True)
    want = torch.autograd.grad((yr * s["dy"]).sum() + (er * s["dstate"]).sum(), list(leaves.values()))
    errs = {"y": (rel(cut("y", y.cpu()), yr), tol("y", dtype, False)),
            "end": (rel(cut("state", end.cpu()), er), tol("end", dtype, False))}
    for (n, _), w in zip(leaves.items(), want):
        errs["d" + n] = (rel(cut(n, got[NAMES.index(n)].cpu()), w), tol(n, dtype, True))
    check(errs)


def test_a_long_sequence_against_its_parts():
    """Cut in two with the state handed over, forward and back: what a whole pass gives."""
    g = to_gpu(inputs(4, 1, 3000, 48, 16, 1, F32), F32)
    args = [g[n] for n in NAMES[:8]]
    y, end, saved = ws.gl_ssm_fwd(*args, state=g["state"], want_state=True, save=True)
    whole = ws.gl_ssm_bwd(*args, g["dy"], saved, state=g["state"], dstate=g["dstate"])
    part = lambda lo, hi: [t if t is None or t.dim() < 3 else t[:, lo:hi] for t in args]  # noqa: E731
    y0, mid, s0 = ws.gl_ssm_fwd(*part(0, 1111), state=g["state"], want_state=True, save=True)
    y1, last, s1 = ws.gl_ssm_fwd(*part(1111, 3000), state=mid, want_state=True, save=True)
    b1 = ws.gl_ssm_bwd(*part(1111, 3000), g["dy"][:, 1111:], s1, state=mid, dstate=g["dstate"])
    b0 = ws.gl_ssm_bwd(*part(0, 1111), g["dy"][:, :1111], s0, state=g["state"], dstate=b1[8])
    errs = {"y": (rel(torch.cat([y0, y1], 1), y), 8e-6), "end": (rel(last, end), 8e-6), "dstate": (rel(b0[8], whole[8]), 1.6e-5)}
    for i, n in enumerate(NAMES[:8]):
        both = b0[i] + b1[i] if n in ("A", "skip", "dt_bias") else torch.cat([b0[i], b1[i]], 1)
        errs["d" + n] = (rel(both, whole[i]), 1.6e-5)
    check(errs)


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("N,G", [(16, 1), (5, 2), (1, 1), (64, 2), (130, 1)])
def test_step(N, G, dtype):
    """Tokens one by one against a pool: whole passes, rows with nothing to do, other states untouched."""
    D, T = 24, 5
    x = inputs(N + G, 4, T, D, N, G, dtype)
    g = to_gpu(x, dtype)
    y, end = ref.scan(*(x[n] for n in NAMES), None, True)
    pool = torch.randn(7, D, N, device="cuda").to(par(dtype))
    slots = torch.tensor([5, -1, 0, 7], dtype=torch.int32, device="cuda")
    pool[5], pool[0] = g["state"][0], g["state"][2]
    before = pool.clone()
    tok = lambda n, t: g[n][:, t] if n in ("x", "dt", "B", "C", "z") else g[n]  # noqa: E731
    for t in range(T):
        yt = ws.gl_ssm_step(*(tok(n, t) for n in NAMES[:8]), pool, slots=slots)
        for b in (0, 2):
            assert rel(yt[b], y[b, t]) <= tol("y", dtype, False)
        assert not yt[1].any() and not yt[3].any()
    torch.cuda.synchronize()
    assert rel(pool[5], end[0]) <= tol("end", dtype, False) and rel(pool[0], end[2]) <= tol("end", dtype, False)
    for k in (1, 2, 3, 4, 6):
        assert torch.equal(pool[k], before[k])
    one = g["state"].clone()  # without slots, and with a pool of no state
    assert rel(ws.gl_ssm_step(*(tok(n, 0) for n in NAMES[:8]), one), y[:, 0]) <= tol("y", dtype, False)
    none = ws.gl_ssm_step(*(tok(n, 0) for n in NAMES[:8]), one[:0], slots=slots)
    assert not none.any()


def test_flat_groups_dimension():
    """B and C without their dimension of groups."""
    g = to_gpu(inputs(8, 2, 20, 16, 8, 1, F32), F32)
    args = [g[n] for n in NAMES[:8]]
    flat = [t[:, :, 0] if n in ("B", "C") else t for n, t in zip(NAMES, args)]
    a, b = ws.gl_ssm_fwd(*args)[0], ws.gl_ssm_fwd(*flat)[0]
    assert torch.equal(a, b)
    da, db = ws.gl_ssm_bwd(*args, g["dy"]), ws.gl_ssm_bwd(*flat, g["dy"])
    assert db[3].shape == flat[3].shape and torch.equal(da[3][:, :, 0], db[3])
    one = lambda args: [t[:, 0] if n in ("x", "dt", "B", "C", "z") else t for n, t in zip(NAMES, args)]  # noqa: E731
    assert torch.equal(ws.gl_ssm_step(*one(args), g["state"].clone()), ws.gl_ssm_step(*one(flat), g["state"].clone()))


def test_no_tokens_no_rows():
    for B, T in ((2, 0), (0, 5)):
        g = to_gpu(inputs(1, B, T, 16, 4, 1, F32), F32)
        args = [g[n] for n in NAMES[:8]]
        y, end, saved = ws.gl_ssm_fwd(*args, state=g["state"], want_state=True, save=True)
        assert y.shape == g["x"].shape and torch.equal(end, g["state"])
        got = ws.gl_ssm_bwd(*args, g["dy"], saved, state=g["state"], dstate=g["dstate"])
        torch.cuda.synchronize()
        assert torch.equal(got[8], g["dstate"])
        assert not any(got[i].any() for i in (2, 5, 7))


def test_extreme_steps():
    """Steps that forget everything at once (decays that underflow), and steps of nearly none."""
    x = inputs(6, 1, 200, 32, 8, 1, F32)
    x["dt"][:, 50] = 300.0
    x["dt"][:, 60:70] = -80.0
    x["dt"][:, 120] = 30.0
    y, end = ref.scan(*(x[n] for n in NAMES), None, True)
    g = to_gpu(x, F32)
    yg, eg, _ = ws.gl_ssm_fwd(*(g[n] for n in NAMES[:8]), state=g["state"], want_state=True)
    check({"y": (rel(yg, y), 4e-6), "end": (rel(eg, end), 4e-6)})


def test_not_finite_stays_in_its_channel_and_later():
    g = to_gpu(inputs(7, 1, 600, 40, 16, 1, F32), F32)
    args = {n: g[n] for n in NAMES[:8]}
    clean = ws.gl_ssm_fwd(*args.values())[0]
    g["x"][0, 300, 5] = torch.nan
    y = ws.gl_ssm_fwd(*args.values())[0]
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[0, 300:, 5] = True
    assert torch.equal(y[~hit], clean[~hit]) and y[0, 300:, 5].isnan().all()


def test_autograd_and_differences():
    """The wrapper's gradients against differences of the forward, in 64 bits."""
    x = inputs(2, 2, 6, 4, 2, 2, F64)
    args = [x[n].cuda().requires_grad_(True) for n in NAMES]
    f = lambda *a: ws.selective_scan(*a[:8], state=a[8], want_state=True)  # noqa: E731
    assert torch.autograd.gradcheck(f, args, eps=1e-6, atol=1e-6)


def test_results_do_not_depend_on_the_run():
    """Sums in a fixed order: the bits of a second call."""
    g = to_gpu(inputs(3, 2, 700, 96, 16, 1, BF16), BF16)
    args = [g[n] for n in NAMES[:8]]
    _, _, saved = ws.gl_ssm_fwd(*args, save=True)
    a, b = (ws.gl_ssm_bwd(*args, g["dy"], saved) for _ in range(2))
    assert all(torch.equal(s, t) for s, t in zip(a, b) if s is not None)


@pytest.mark.parametrize("T,channels", [(32896, 16), (65600, 32)])
def test_more_channels_where_the_parts_are_large(T, channels):
    """Sequences whose parts of dB and dC would take more than 2^30 bytes at eight channels a work-group: 16 and 32
    instead, with what the same tokens give in pieces of eight channels each (fp32; bounds as above)."""
    D, N, piece = 512, 64, 16448
    size = lambda t: ws.ssm_workspace_size(ws.SsmDesc(1, t, D, N, 1, 0, 1, ws.GL_FLAG_SOFTPLUS), True)[1]  # noqa: E731
    par = 4 * (N + 2) * D
    assert size(piece) == 2 * N * (D // 8) * piece * 4 + par
    assert size(T) == 2 * N * (D // channels) * T * 4 + par
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    A = -torch.arange(1, N + 1, device="cuda") * torch.exp(0.1 * rnd(D, N))
    bias = torch.rand(D, generator=g, device="cuda") * 3 - 4  # steps of some 0.02 .. 0.3
    args = [rnd(1, T, D), 0.5 * rnd(1, T, D), A, rnd(1, T, 1, N), rnd(1, T, 1, N), 1 + 0.1 * rnd(D), rnd(1, T, D), bias]
    dy, state, dstate = rnd(1, T, D), 0.3 * rnd(1, D, N), 0.3 * rnd(1, D, N)
    y, end, saved = ws.gl_ssm_fwd(*args, state=state, want_state=True, save=True)
    whole = ws.gl_ssm_bwd(*args, dy, saved, state=state, dstate=dstate)
    cuts = [*range(0, T, piece), T]
    part = lambda lo, hi: [t if t.dim() < 3 else t[:, lo:hi] for t in args]  # noqa: E731
    st, ys, keep = state, [], []
    for lo, hi in zip(cuts, cuts[1:]):
        yp, nxt, s = ws.gl_ssm_fwd(*part(lo, hi), state=st, want_state=True, save=True)
        ys.append(yp)
        keep.append((lo, hi, st, s))
        st = nxt
    adj, parts = dstate, []
    for lo, hi, first, s in reversed(keep):
        parts.insert(0, ws.gl_ssm_bwd(*part(lo, hi), dy[:, lo:hi], s, state=first, dstate=adj))
        adj = parts[0][8]
    errs = {"y": (rel(torch.cat(ys, 1), y), 8e-6), "end": (rel(st, end), 8e-6), "dstate": (rel(adj, whole[8]), 1.6e-5)}
    for i, n in enumerate(NAMES[:8]):
        both = sum(p[i].double() for p in parts) if n in ("A", "skip", "dt_bias") else torch.cat([p[i] for p in parts], 1)
        errs["d" + n] = (rel(both, whole[i]), 1.6e-5)
    check(errs)
