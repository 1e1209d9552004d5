"""What calls of include/gl_ssm.h read and write on the GPU: nothing outside the
outputs, `saved` and the workspaces whatever the sequence table holds, states
updated in place; calls on other streams and in captured graphs; what the autograd
wrappers refuse."""
import ctypes

import pytest
import torch

import ssm_ref as ref
import weight_scans_amd as ws
from ssm_ref import BF16, F32, F64, rel
from test_gpu_delta_memory import CODE, Guarded, ptr, space
from test_gpu_ssm import NAMES, inputs, to_gpu

pytestmark = pytest.mark.gpu

TABLES = [[0, 30, 30, 100], [-5, 1 << 30, 40, 90], [0, 90, 10, 100], [100, 100, 0, 0], [50, 20, 70, 30],
          [-(1 << 31), (1 << 31) - 1, -(1 << 31), (1 << 31) - 1], [99, 100, 98, 200], [0, 0, 0, 0]]


def call(name, desc, tensors, workspace=None):
    args = [ptr(t) for t in tensors]
    if ctypes.c_size_t in getattr(ws.ssm_lib(), name).argtypes:
        args += [ptr(workspace), 0 if workspace is None else workspace.numel()]
    status = getattr(ws.ssm_lib(), name)(ctypes.byref(desc), *args,
                                         ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert status == 0, ws.lib().gl_last_error()


class Outputs:
    """Outputs like these tensors, each between guard bytes."""

    def __init__(self, tensors):
        self.of = [None if t is None else Guarded(t.numel() * t.element_size()) for t in tensors]
        self.t = [None if t is None else g.like(t) for g, t in zip(self.of, tensors)]

    def whole(self):
        torch.cuda.synchronize()
        return all(g is None or g.whole() for g in self.of)


@pytest.mark.parametrize("table", TABLES)
@pytest.mark.parametrize("dtype,D,N", [(BF16, 40, 16), (F32, 64, 5), (F64, 20, 3)])
def test_scan_stays_inside_for_any_table(table, dtype, D, N):
    T = 100
    g = to_gpu(inputs(D, 1, T, D, N, 1, dtype, lens=[T, 0, 0]), dtype)
    args = [g[n] for n in NAMES[:8]]
    desc = ws.SsmDesc(1, T, D, N, 1, 3, CODE[dtype], ws.GL_FLAG_SOFTPLUS)
    size = ctypes.c_size_t()
    ws.ssm_lib().gl_ssm_saved_size(ctypes.byref(desc), ctypes.byref(size))
    saved, work = Guarded(size.value), Guarded(ws.ssm_workspace_size(desc, True)[1])
    cu = torch.tensor(table, dtype=torch.int32, device="cuda")
    fwd = Outputs([g["x"], g["state"]])
    call("gl_ssm_fwd", desc, [*args, g["state"], cu, *fwd.t, saved.inside])
    bwd = Outputs([g["x"], g["x"], g["A"], g["B"], g["C"], g["skip"], g["z"], g["dt_bias"], g["state"]])
    call("gl_ssm_bwd", desc, [*args, g["state"], cu, g["dy"], g["dstate"], saved.inside, *bwd.t], work.inside)
    assert fwd.whole() and bwd.whole() and saved.whole() and work.whole()
    again = Guarded(ws.ssm_workspace_size(desc, False)[1])
    call("gl_ssm_bwd", desc, [*args, g["state"], cu, g["dy"], g["dstate"], None, *bwd.t], again.inside)
    assert bwd.whole() and again.whole()


@pytest.mark.parametrize("table", TABLES)
@pytest.mark.parametrize("dtype,D,K", [(BF16, 40, 4), (BF16, 33, 7), (F32, 64, 2), (F64, 6, 3)])
def test_convolution_stays_inside_for_any_table(table, dtype, D, K):
    T = 100
    x, dy, w, bias = (torch.randn(s, device="cuda").to(dtype) for s in ((1, T, D), (1, T, D), (D, K), (D,)))
    state, dstate = (torch.randn(3, K - 1, D, device="cuda").to(dtype) for _ in range(2))
    desc = ws.ConvDesc(1, T, D, K, 3, CODE[dtype], ws.GL_FLAG_SILU)
    size = ctypes.c_size_t()
    ws.ssm_lib().gl_conv_workspace_size(ctypes.byref(desc), ctypes.byref(size))
    work = Guarded(size.value)
    cu = torch.tensor(table, dtype=torch.int32, device="cuda")
    fwd = Outputs([x, state])
    call("gl_conv_fwd", desc, [x, w, bias, state, cu, *fwd.t])
    par = w.double() if dtype == F64 else w.float()
    bwd = Outputs([x, par, par[:, 0].contiguous(), state])
    call("gl_conv_bwd", desc, [x, w, bias, state, cu, dy, dstate, *bwd.t], work.inside)
    assert fwd.whole() and bwd.whole() and work.whole()


@pytest.mark.parametrize("d,dtype", [(7, BF16), (100, F32), (264, BF16), (2048, BF16), (4100, F32)])
def test_norms_stay_inside(d, dtype):
    x, r, dn, dr = (torch.randn(2, 9, d, device="cuda").to(dtype) for _ in range(4))
    w = torch.randn(d, device="cuda").to(dtype)
    desc = ws.AddNormDesc(2, 9, d, CODE[dtype], CODE[dtype], 0, 0, 1e-6)
    size = ctypes.c_size_t()
    ws.ssm_lib().gl_addnorm_workspace_size(ctypes.byref(desc), ctypes.byref(size))
    work, out, back = Guarded(size.value), Outputs([x, r]), Outputs([x, r, w.float(), w.float(), w.float()])
    call("gl_addnorm_fwd", desc, [x, r, w, w, w, *out.t])
    call("gl_addnorm_bwd", desc, [x, r, w, w, w, dn, dr, *back.t], work.inside)
    assert out.whole() and back.whole() and work.whole()
    desc = ws.GateNormDesc(2, 3, 3, d, CODE[dtype], ws.GL_FLAG_GROUP_WEIGHTS, 1e-6)
    ws.ssm_lib().gl_gatenorm_workspace_size(ctypes.byref(desc), ctypes.byref(size))
    gw = torch.randn(3, d, device="cuda").to(dtype)
    work, out, back = Guarded(size.value), Outputs([x]), Outputs([x, x, gw.float()])
    call("gl_gatenorm_fwd", desc, [x, r, gw, *out.t])
    call("gl_gatenorm_bwd", desc, [x, r, gw, dn, *back.t], work.inside)
    assert out.whole() and back.whole() and work.whole()


@pytest.mark.parametrize("dtype,T,D", [(BF16, 600, 64), (F32, 70, 24), (F64, 40, 8), (BF16, 0, 16)])
def test_states_updated_in_place(dtype, T, D):
    """state_out = state_in, dstate_in = dstate_out and r_out = r: the bits of calls with them apart."""
    B, N = 2, 16
    g = to_gpu(inputs(T + D, B, T, D, N, 1, dtype), dtype)
    args = [g[n] for n in NAMES[:8]]
    y, end, saved = ws.gl_ssm_fwd(*args, state=g["state"], want_state=True, save=True)
    want = ws.gl_ssm_bwd(*args, g["dy"], saved, state=g["state"], dstate=g["dstate"])
    desc = ws.SsmDesc(B, T, D, N, 1, 0, CODE[dtype], ws.GL_FLAG_SOFTPLUS)
    state, y1, s1 = g["state"].clone(), torch.empty_like(y), torch.empty_like(saved)
    call("gl_ssm_fwd", desc, [*args, state, None, y1, state, s1])
    assert torch.equal(y, y1) and torch.equal(end, state)
    got, dstate = [torch.empty_like(t) for t in want[:8]], g["dstate"].clone()
    call("gl_ssm_bwd", desc, [*args, g["state"], None, g["dy"], dstate, s1, *got, dstate],
         space(ws.ssm_workspace_size(desc, True)[1]))
    for a, b in zip(want, [*got, dstate]):
        assert torch.equal(a, b)
    x, r, w = torch.randn(1, 5, 48, device="cuda"), torch.randn(1, 5, 48, device="cuda"), torch.randn(48, device="cuda")
    n, ro = ws.gl_addnorm_fwd(x, r, w)
    n1, r1 = torch.empty_like(n), r.clone()
    call("gl_addnorm_fwd", ws.AddNormDesc(1, 5, 48, CODE[F32], CODE[F32], 0, 0, 1e-6), [x, r1, w, None, None, n1, r1])
    assert torch.equal(n, n1) and torch.equal(ro, r1)


def block(x, r, w, conv_w, A, bc, skip, bias, nw):
    """A block as a model runs it: norm, convolution, scan, gated norm."""
    n, r = ws.add_norm(x, r, w)
    u, _ = ws.causal_conv(n, conv_w)
    N = A.shape[1]
    y, _ = ws.selective_scan(u, n, A, bc[..., :N], bc[..., N:], skip, None, bias)
    return ws.gated_norm(y, n, nw), r


def block_inputs(seed, dtype=BF16, B=2, T=130, D=64, N=16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return [rnd(B, T, D).to(dtype), rnd(B, T, D).to(dtype), rnd(D).to(dtype), rnd(D, 4).to(dtype), -rnd(D, N).exp(),
            rnd(B, T, 2 * N).to(dtype), rnd(D), rnd(D) - 3, rnd(D).to(dtype)]


def test_the_block_together():
    """All operators in a row against their definitions in 64 bits, values and gradients (fp32; some four
    operators of up to 8e-6 one after another, whose errors the next ones pass on about as they are: 5e-5)."""
    args = [t.requires_grad_(True) for t in block_inputs(1, F32)]
    y, r = block(*args)
    dy, dr = torch.randn_like(y), torch.randn_like(r)
    got = torch.autograd.grad((y * dy).sum() + (r * dr).sum(), args)
    c = [t.detach().double().cpu().requires_grad_(True) for t in args]
    x, r0, w, cw, A, bc, skip, bias, nw = c
    n, rr = ref.add_norm(x, r0, w, None, None, 1e-6)
    u, _ = ref.conv(n, cw, None, None, None, True)
    N = A.shape[1]
    s, _ = ref.scan(u, n, A, bc[:, :, None, :N], bc[:, :, None, N:], skip, None, bias, None, None, True)
    yr = ref.gated_norm(s, n, nw, 1e-6, False)
    want = torch.autograd.grad((yr * dy.double().cpu()).sum() + (rr * dr.double().cpu()).sum(), c)
    assert rel(y, yr) <= 5e-5 and rel(r, rr) <= 1e-6
    for a, b in zip(got, want):
        assert rel(a, b) <= 5e-5


def test_other_streams():
    """Two streams at once: the bits of calls one after another."""
    a, b = block_inputs(2), block_inputs(3)
    want = [block(*a), block(*b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(5):
        for i, (s, x) in enumerate(zip(streams, (a, b))):
            with torch.cuda.stream(s):
                got[i] = block(*x)
        torch.cuda.synchronize()
        for u, v in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(u, v))


def grads(args):
    leaves = [t.detach().requires_grad_(True) for t in args]
    y, r = block(*leaves)
    return torch.autograd.grad((y.float() * 0.5).sum() + (r.float() * 0.25).sum(), leaves)


def test_captured_graphs():
    """Forward and backward of the block in two graphs that share a memory pool, replayed between eager
    work: every replay has the eager call's bits."""
    xs = [block_inputs(4), block_inputs(5)]
    want = [(block(*x), grads(x)) for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x in xs:
            grads(x)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs, pool = [], [], torch.cuda.graph_pool_handle()
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            outs.append((block(*x), grads(x)))
        graphs.append(graph)
    for i in (0, 1, 1, 0, 0, 1):
        graphs[i].replay()
        torch.cuda.synchronize()
        for a, b in zip((*want[i][0], *want[i][1]), (*outs[i][0], *outs[i][1])):
            assert torch.equal(a, b)
        grads(xs[1 - i])  # eager work between the replays
        torch.cuda.synchronize()


def test_steps_in_a_captured_graph():
    """A decoding step (convolution and scan against their pools) captured and replayed: the pools move on as
    with eager calls."""
    B, D, N, K = 5, 64, 16, 4
    x, dt, z = (torch.randn(B, D, device="cuda").to(BF16) for _ in range(3))
    Bm, Cm = (torch.randn(B, N, device="cuda").to(BF16) for _ in range(2))
    w, A, bias = torch.randn(D, K, device="cuda").to(BF16), -torch.rand(D, N, device="cuda"), torch.randn(D, device="cuda") - 3
    slots = torch.tensor([3, 0, 6, -1, 2], dtype=torch.int32, device="cuda")
    conv, scan = torch.randn(7, K - 1, D, device="cuda").to(BF16), torch.randn(7, D, N, device="cuda")

    def step(conv, scan):
        u = ws.gl_conv_step(x, w, None, conv, slots=slots)
        return ws.gl_ssm_step(u, dt, A, Bm, Cm, None, z, bias, scan, slots=slots)
    c0, s0 = conv.clone(), scan.clone()
    ys = [step(c0, s0) for _ in range(4)]
    c1, s1 = conv.clone(), scan.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(c1, s1)
    c1.copy_(conv), s1.copy_(scan)
    for want in ys:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert torch.equal(c0, c1) and torch.equal(s0, s1)


def test_second_derivatives_and_duals_are_refused():
    args = [t.requires_grad_(True) for t in block_inputs(6, F32, 1, 6, 8, 2)]
    y, _ = block(*args)
    first = torch.autograd.grad(y.sum(), args, create_graph=True, allow_unused=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(first[0].sum(), args)
    x = torch.randn(1, 4, 8, device="cuda")
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        for f in (lambda: ws.causal_conv(dual, torch.ones(8, 2, device="cuda")),
                  lambda: ws.selective_scan(dual, x, -torch.ones(8, 2, device="cuda"), x[..., :2], x[..., 2:4]),
                  lambda: ws.add_norm(dual, x, torch.ones(8, device="cuda")), lambda: ws.gated_norm(dual, x)):
            with pytest.raises(NotImplementedError):
                f()


def test_broadcast_and_transposed_inputs_are_copied():
    """Expanded rows and gradients, rows whose columns lie apart, and tokens far apart."""
    x = torch.randn(8, 2, 30, device="cuda").permute(1, 2, 0).requires_grad_(True)  # columns apart
    dt = torch.randn(1, 1, 8, device="cuda").expand(2, 30, 8)
    bc = torch.randn(2, 30, 3, device="cuda")
    A = -torch.rand(1, 3, device="cuda").expand(8, 3)
    y, _ = ws.selective_scan(x, dt, A, bc, bc)
    (g,) = torch.autograd.grad(y.sum(), [x])  # an expanded upstream gradient
    y1, _, saved = ws.gl_ssm_fwd(x.detach().contiguous(), dt.contiguous(), A.contiguous(), bc, bc, save=True)
    want = ws.gl_ssm_bwd(x.detach().contiguous(), dt.contiguous(), A.contiguous(), bc, bc, None, None, None,
                         torch.ones_like(y1), saved)[0]
    assert torch.equal(y, y1) and torch.equal(g, want)
    far = torch.randn(30, 1 << 19, device="cuda")[:, :8].unsqueeze(0)  # tokens 2^19 apart
    with pytest.raises(ws.GLScanError):
        ws.gl_ssm_fwd(far, far, A.contiguous(), bc[:1], bc[:1])
    assert torch.equal(ws.selective_scan(far, far, A, bc[:1], bc[:1])[0],
                       ws.gl_ssm_fwd(*(t.contiguous() for t in (far, far, A, bc[:1], bc[:1])))[0])


def test_offsets_past_32_bits():
    """A batch whose later rows lie beyond 2^32 bytes: the bits of the same rows alone."""
    T, D, N = 600, 64, 4
    rows = 1 << 31  # elements between the batches, 4 GiB in bf16
    buf = torch.zeros(rows + T * D, dtype=BF16, device="cuda")
    x = buf.as_strided((2, T, D), (rows, D, 1))
    x.copy_(torch.randn(2, T, D, device="cuda"))
    A, bc, w = -torch.rand(D, N, device="cuda"), torch.randn(2, T, N, device="cuda").to(BF16), torch.randn(D, 4, device="cuda").to(BF16)
    y = ws.gl_ssm_fwd(x, x, A, bc, bc)[0]
    c = ws.gl_conv_fwd(x, w)[0]
    n = ws.gl_gatenorm_fwd(x, x)
    r = ws.gl_addnorm_fwd(x, x, w[:, 0].contiguous())[0]
    one = x[1:].clone()
    assert torch.equal(y[1:], ws.gl_ssm_fwd(one, one, A, bc[1:], bc[1:])[0])
    assert torch.equal(c[1:], ws.gl_conv_fwd(one, w)[0])
    assert torch.equal(n[1:], ws.gl_gatenorm_fwd(one, one))
    assert torch.equal(r[1:], ws.gl_addnorm_fwd(one, one, w[:, 0].contiguous())[0])


@pytest.mark.parametrize("T", [0, 7, 4096])
@pytest.mark.parametrize("dtype,D,K", [(BF16, 64, 4), (F32, 13, 2), (F64, 6, 6)])
def test_convolution_step_with_the_descriptor_of_a_prompt(T, dtype, D, K):
    """Dense rows of a step are D apart whatever T the descriptor holds: the bits of T = 1, the rest untouched."""
    B = 5
    x, w, bias, state = (torch.randn(s, device="cuda").to(dtype) for s in ((B, D), (D, K), (D,), (B, K - 1, D)))
    want, ends = torch.empty_like(x), state.clone()

    def step(T, st, y):
        desc = ws.ConvDesc(B, T, D, K, 0, CODE[dtype], ws.GL_FLAG_SILU)
        status = ws.ssm_lib().gl_conv_step(ctypes.byref(desc), ptr(x), ptr(w), ptr(bias), None, B, ptr(st), ptr(y),
                                           ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert status == 0, ws.lib().gl_last_error()
    step(1, ends, want)
    out = Outputs([x, state])
    out.t[1].copy_(state)
    step(T, out.t[1], out.t[0])
    assert out.whole() and torch.equal(out.t[0], want) and torch.equal(out.t[1], ends)


@pytest.mark.parametrize("T", [0, 7, 4096, 1 << 40])
@pytest.mark.parametrize("dtype,D,N", [(BF16, 64, 16), (F32, 14, 5)])
def test_scan_step_with_the_descriptor_of_a_prompt(T, dtype, D, N):
    """Likewise the scan's step, with dense B and C of two groups."""
    B = 5
    g = to_gpu(inputs(D, B, 1, D, N, 2, dtype), dtype)
    args = [t[:, 0].contiguous() if n in ("x", "dt", "B", "C", "z") else t for n, t in g.items() if n in NAMES[:8]]
    want, ends = torch.empty_like(args[0]), g["state"].clone()

    def step(T, st, y):
        desc = ws.SsmDesc(B, T, D, N, 2, 0, CODE[dtype], ws.GL_FLAG_SOFTPLUS)
        status = ws.ssm_lib().gl_ssm_step(ctypes.byref(desc), *(ptr(t) for t in args), None, B, ptr(st), ptr(y),
                                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert status == 0, ws.lib().gl_last_error()
    step(1, ends, want)
    out = Outputs([want, ends])
    out.t[1].copy_(g["state"])
    step(T, out.t[1], out.t[0])
    assert out.whole() and torch.equal(out.t[0], want) and torch.equal(out.t[1], ends)
