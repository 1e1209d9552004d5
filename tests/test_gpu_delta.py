"""The gated delta rule on the GPU against the token-by-token definition in 64
bits and its autograd gradients.

Tolerances (2-norm of the error over that of the reference), from the
arithmetic: fp64 1e-10.  fp32: 1e-5 (some 1e3 roundings of 6e-8 in quadrature,
and room).  bf16 outputs: 5e-3 (the final rounding is 1.7e-3 rms; the
matrix-core path rounds up to three operands of the last products, 1.7e-3 each,
in quadrature 3.4e-3).  States of bf16 runs: 1e-5 (operands of 16 bits,
2.8e-6 rms each, some four of them).  Gate gradients in fp32 of bf16 runs: as
bf16 outputs."""
import pytest
import torch

import weight_scans_amd as ws
from delta_ref import delta, inputs, rel

pytestmark = pytest.mark.gpu

TOL = {torch.float64: 1e-10, torch.float32: 1e-5, torch.bfloat16: 5e-3}
STATE_TOL = {torch.float64: 1e-10, torch.float32: 1e-5, torch.bfloat16: 1e-5}
F64, F32, BF16 = torch.float64, torch.float32, torch.bfloat16


def to_gpu(x, dtype, gate, order="bhtd"):
    st = F64 if dtype == F64 else F32
    kind = {"log_alpha": gate, "beta": gate, "state": st, "dstate": st}
    out = {}
    for n, t in x.items():
        t = t.detach().to(kind.get(n, dtype)).cuda()
        if order == "bthd" and n in ("q", "k", "v", "dy", "log_alpha", "beta"):
            t = t.transpose(1, 2).contiguous().transpose(1, 2)
        out[n] = t
    return out


def cu_of(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")


def run_case(seed, B, H, Hk, T, dk, dv, dtype, gate=None, lens=None, order="bhtd", flags=0, with_state=True,
             decay="mix", scale=None, edit=None, saved=True, segments=0):
    gate = gate or dtype
    x = inputs(seed, B, H, Hk, T, dk, dv, dtype, gate, None if lens is None else len(lens), decay)
    if edit:
        edit(x)
    names = ["q", "k", "v", "log_alpha", "beta"] + (["state"] if with_state else [])
    for n in names:
        x[n].requires_grad_(True)
    sc = dk ** -0.5 if scale is None else scale
    y, end = delta(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], sc, x["state"] if with_state else None, lens)
    loss = (y * x["dy"]).sum() + ((end * x["dstate"]).sum() if with_state else 0)
    want = torch.autograd.grad(loss, [x[n] for n in names], allow_unused=True)
    g = to_gpu(x, dtype, gate, order)
    cu = None if lens is None else cu_of(lens)
    st, dst = (g["state"], g["dstate"]) if with_state else (None, None)
    gy, gend, sv = ws.gl_delta_fwd(g["q"], g["k"], g["v"], g["log_alpha"], g["beta"], scale=scale, state=st,
                                   want_state=True, save=saved, cu_seqlens=cu, flags=flags, segments=segments)
    got = ws.gl_delta_bwd(g["q"], g["k"], g["v"], g["log_alpha"], g["beta"], g["dy"], sv, scale=scale, state=st,
                          dstate=dst, cu_seqlens=cu, flags=flags, segments=segments)
    torch.cuda.synchronize()
    errs = {"y": (rel(gy, y), TOL[dtype]), "state": (rel(gend, end), STATE_TOL[dtype])}
    for n, a, b in zip(names, got, want):
        b = torch.zeros_like(x[n]) if b is None else b
        assert torch.isfinite(a.double()).all(), n
        errs["d" + n] = (rel(a, b), STATE_TOL[dtype] if n == "state" else TOL[dtype])
    print({n: f"{e:.1e}" for n, (e, _) in errs.items()}, flush=True)
    for n, (e, tol) in errs.items():
        assert e <= tol, (n, e, tol)
    return g, gy, gend, got


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 129, 300])
@pytest.mark.parametrize("dtype", [F64, F32, BF16])
def test_lengths(T, dtype):
    run_case(T, 2, 4, 2, T, 64, 64, dtype)


@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 20), (16, 128), (40, 24), (64, 128), (72, 96), (100, 128), (128, 17),
                                   (128, 64), (128, 128)])
@pytest.mark.parametrize("dtype", [F64, F32, BF16])
def test_head_sizes(dk, dv, dtype):
    run_case(dk * 131 + dv, 1, 3, 1, 70, dk, dv, dtype)


@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 2), (5, 5), (8, 1)])
@pytest.mark.parametrize("order", ["bhtd", "bthd"])
def test_shared_heads_and_orders(H, Hk, order):
    for dtype in (F32, BF16):
        run_case(H, 2, H, Hk, 100, 64, 64, dtype, order=order)


@pytest.mark.parametrize("lens", [[5], [0, 1, 0], [64, 64], [1, 63, 65, 0, 130, 2], [0, 0, 200, 1], [3] * 20])
@pytest.mark.parametrize("dtype,d", [(F32, 64), (BF16, 64), (BF16, 128), (BF16, 24)])
def test_packed(lens, dtype, d):
    run_case(len(lens), 1, 4, 2, sum(lens), d, d, dtype, lens=lens, order="bthd")


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
def test_without_states_and_without_saved(dtype):
    run_case(5, 2, 2, 2, 150, 64, 64, dtype, with_state=False)
    run_case(6, 2, 2, 1, 150, 128, 64, dtype, saved=False)


def test_fp32_gates_of_bf16():
    run_case(7, 2, 4, 4, 200, 64, 64, BF16, gate=F32)
    run_case(8, 1, 2, 2, 200, 128, 128, BF16, gate=F32, decay="near1")


def test_generic_flag_is_the_serial_path():
    d = ws.make_delta_desc(1, 100, 2, 2, 64, 64, ws.GL_DTYPE_BF16, ws.GL_DTYPE_BF16, flags=ws.GL_FLAG_GENERIC)
    assert ws.delta_path_name(d) == "delta-serial-bf16"
    run_case(9, 1, 2, 2, 100, 64, 64, BF16, flags=ws.GL_FLAG_GENERIC)


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
def test_forgetting_and_idle_tokens(dtype, d):
    """log_alpha = -inf (forget before the write), 0 (keep all), tokens that write
    nothing (beta = 0) and overwrite exactly (beta = 1)."""
    def edit(x):
        x["log_alpha"][0, 0, 3] = x["log_alpha"][0, 0, 70] = x["log_alpha"][0, 1, 0] = -torch.inf
        x["log_alpha"][0, 1, 40:100] = 0.0
        x["beta"][0, 0, 10:90] = 0.0
        x["beta"][0, 1, ::2] = 1.0
        x["log_alpha"][1, 0, 20:40] = -torch.inf
        x["log_alpha"][1, 1, :] = -60.0
        x["beta"][1, 1, :] = 0.0
    # the reference's exp(-inf) * S has gradient 0 * inf at log_alpha = -inf only
    # through exp itself, which torch gives as 0
    run_case(d, 2, 2, 2, 140, d, d, dtype, edit=edit)


def test_broadcast_keys_and_strided_gates():
    """q and k expanded over the batch (stride 0), gates as slices of a wider row."""
    x = inputs(3, 2, 4, 2, 90, 64, 64, BF16, F32)
    x["q"], x["k"] = (x[n][:1].expand(2, -1, -1, -1) for n in "qk")
    y, end = delta(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], 0.125)
    g = to_gpu(x, BF16, F32)
    q, k = (g[n][:1].contiguous().expand(2, -1, -1, -1) for n in "qk")
    wide = torch.zeros((2, 90, 8), device="cuda")
    wide[..., :4] = g["log_alpha"].transpose(1, 2)
    wide2 = torch.ones((2, 90, 8), device="cuda")
    wide2[..., :4] = g["beta"].transpose(1, 2)
    gy, gend, _ = ws.gl_delta_fwd(q, k, g["v"], wide[..., :4].transpose(1, 2), wide2[..., :4].transpose(1, 2),
                                  want_state=True)
    assert rel(gy, y) <= TOL[BF16] and rel(gend, end) <= STATE_TOL[BF16]


def test_gradient_against_differences():
    """fp64: central differences of the GPU's own forward along random directions
    (step 1e-5: truncation 1e-10, rounding 1e-16 / 1e-5)."""
    x = inputs(11, 1, 2, 1, 21, 10, 7, F64)
    g = to_gpu(x, F64, F64)
    names = ["q", "k", "v", "log_alpha", "beta", "state"]

    def loss(z):
        y, end, _ = ws.gl_delta_fwd(z["q"], z["k"], z["v"], z["log_alpha"], z["beta"], state=z["state"],
                                    want_state=True)
        return float((y * g["dy"]).sum() + (end * g["dstate"]).sum())
    got = ws.gl_delta_bwd(g["q"], g["k"], g["v"], g["log_alpha"], g["beta"], g["dy"], state=g["state"],
                          dstate=g["dstate"])
    gen = torch.Generator().manual_seed(1)
    for i, n in enumerate(names):
        d = torch.randn(g[n].shape, generator=gen, dtype=F64).cuda()
        h = 1e-5
        num = (loss({**g, n: g[n] + h * d}) - loss({**g, n: g[n] - h * d})) / (2 * h)
        ana = float((got[i] * d).sum())
        assert abs(num - ana) <= 1e-7 * max(1.0, abs(ana)), (n, num, ana)


@pytest.mark.parametrize("dtype", [F64, F32, BF16])
@pytest.mark.parametrize("dk,dv,H,Hk", [(128, 128, 4, 2), (64, 64, 3, 3), (128, 64, 2, 1), (20, 33, 2, 2),
                                        (7, 5, 1, 1), (96, 80, 6, 3)])
def test_step(dtype, dk, dv, H, Hk):
    """Tokens one at a time reproduce the whole-sequence definition; states in a
    pool, other slots untouched, a row without a slot idle."""
    B, T, n = 3, 4, 6
    x = inputs(dk + dv, B, H, Hk, T, dk, dv, dtype, n=n)
    slots = [4, 0, 3]
    y, end = delta(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], dk ** -0.5, x["state"][slots])
    g = to_gpu(x, dtype, dtype)
    pool = g["state"].clone()
    sl = torch.tensor(slots + [-1, n], dtype=torch.int32, device="cuda")
    pad = lambda t: torch.cat([t, t[:2]])  # noqa: E731
    for t in range(T):
        yt = ws.gl_delta_step(pad(g["q"][:, :, t]), pad(g["k"][:, :, t]), pad(g["v"][:, :, t]),
                              pad(g["log_alpha"][:, :, t]), pad(g["beta"][:, :, t]), pool, slots=sl)
        assert rel(yt[:3], y[:, :, t]) <= TOL[dtype]
        assert (yt[3:] == 0).all()
    assert rel(pool[slots], end) <= STATE_TOL[dtype]
    assert torch.equal(pool[[1, 2, 5]], g["state"][[1, 2, 5]])


def test_prefill_then_steps():
    x = inputs(21, 2, 4, 2, 70, 128, 128, BF16)
    g = to_gpu(x, BF16, BF16, "bthd")
    names = ["q", "k", "v", "log_alpha", "beta"]
    y, end, _ = ws.gl_delta_fwd(*[g[n] for n in names], want_state=True)
    _, mid, _ = ws.gl_delta_fwd(*[g[n][:, :, :66] for n in names], want_state=True)
    outs = [ws.gl_delta_step(*[g[n][:, :, t] for n in names], mid) for t in range(66, 70)]
    assert rel(torch.stack(outs, 2), y[:, :, 66:].double().cpu()) <= TOL[BF16]
    assert rel(mid, end.double().cpu()) <= 2 * STATE_TOL[BF16]


def test_autograd_and_streams():
    """delta_rule through autograd on another stream than the tensors' own, twice:
    the same bits."""
    x = inputs(31, 2, 4, 2, 130, 64, 64, BF16)
    names = ["q", "k", "v", "log_alpha", "beta", "state"]
    for n in names:
        x[n].requires_grad_(True)
    y, end = delta(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], 0.125, x["state"])
    want = torch.autograd.grad((y * x["dy"]).sum() + end.square().sum(), [x[n] for n in names])
    g = to_gpu(x, BF16, BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    runs = []
    with torch.cuda.stream(side):
        for _ in range(2):
            leaves = [g[n].detach().clone().requires_grad_(True) for n in names]
            yy, ee = ws.delta_rule(*leaves[:5], state=leaves[5], want_state=True)
            ((yy.float() * g["dy"].float()).sum() + ee.square().sum()).backward()
            runs.append([yy.detach(), ee.detach()] + [p.grad for p in leaves])
    side.synchronize()
    for a, b in zip(*runs):
        assert torch.equal(a, b)
    assert rel(runs[0][0], y) <= TOL[BF16] and rel(runs[0][1], end) <= STATE_TOL[BF16]
    for n, a, b in zip(names, runs[0][2:], want):
        assert rel(a, b) <= (2 * STATE_TOL[BF16] if n == "state" else TOL[BF16]), n


def test_graph_replays():
    """A captured step and prefill replay to the eager bits, with eager work between."""
    x = inputs(41, 2, 2, 2, 100, 64, 64, BF16)
    g = to_gpu(x, BF16, BF16)
    names = ["q", "k", "v", "log_alpha", "beta"]
    eager_y, eager_end, _ = ws.gl_delta_fwd(*[g[n] for n in names], state=g["state"], want_state=True)
    one = [g[n][:, :, 0].contiguous() for n in names]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pool = g["state"].clone()
    with torch.cuda.stream(side):
        ws.gl_delta_fwd(*[g[n] for n in names], state=g["state"], want_state=True)
        ws.gl_delta_step(*one, pool)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    pool.copy_(g["state"])
    with torch.cuda.graph(graph):
        y, end, _ = ws.gl_delta_fwd(*[g[n] for n in names], state=g["state"], want_state=True)
        y1 = ws.gl_delta_step(*one, pool)
    check = g["state"].clone()
    for _ in range(3):
        graph.replay()
        want1 = ws.gl_delta_step(*one, check)
        torch.cuda.synchronize()
        assert torch.equal(y, eager_y) and torch.equal(end, eager_end)
        assert torch.equal(y1, want1) and torch.equal(pool, check)


def test_bad_sequence_table_stays_inside():
    """Starts out of range and out of order are clamped: nothing outside the
    tensors is written (the guard rows around them keep their values)."""
    x = inputs(51, 1, 2, 2, 100, 64, 64, BF16, n=3)
    g = to_gpu(x, BF16, BF16)
    cu = torch.tensor([-5, 1 << 30, 40, 90], dtype=torch.int32, device="cuda")
    y, end, _ = ws.gl_delta_fwd(g["q"], g["k"], g["v"], g["log_alpha"], g["beta"], state=g["state"],
                                want_state=True, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert y.shape == g["v"].shape and end.shape == g["state"].shape


def test_empty():
    x = inputs(61, 2, 2, 2, 1, 64, 64, BF16)
    g = to_gpu(x, BF16, BF16)
    none = [g[n][:, :, :0] for n in ("q", "k", "v", "log_alpha", "beta")]
    y, end, saved = ws.gl_delta_fwd(*none, state=g["state"], want_state=True, save=True)
    assert y.numel() == 0 and torch.equal(end, g["state"])
    grads = ws.gl_delta_bwd(*none, g["dy"][:, :, :0], saved, state=g["state"], dstate=g["dstate"])
    assert torch.equal(grads[5], g["dstate"])
    _, end, _ = ws.gl_delta_fwd(*none, want_state=True)
    assert (end == 0).all()


@pytest.mark.parametrize("dk,dv,T,lens", [
    (64, 64, 64, None), (64, 64, 65, None), (64, 64, 1, None), (20, 36, 200, None), (128, 128, 257, None),
    (96, 80, 130, None), (4, 4, 70, None), (64, 64, 264, [1, 63, 0, 65, 130, 5]), (128, 44, 200, [0, 200])])
@pytest.mark.parametrize("order", ["bhtd", "bthd"])
def test_fp32_chunks(dk, dv, T, lens, order):
    """fp32 on the matrix cores; here a forward that saves nothing."""
    d = ws.make_delta_desc(1, T, 4, 2, dk, dv, ws.GL_DTYPE_F32, ws.GL_DTYPE_F32)
    assert ws.delta_path_name(d).startswith("delta-mfma-f32" if T >= 4 else "delta-serial-f32")
    run_case(dk + T, 1 if lens else 2, 4, 2, T, dk, dv, F32, lens=lens, order=order, saved=False)


def test_fp32_chunks_forgetting():
    def edit(x):
        x["log_alpha"][0, 0, 3] = x["log_alpha"][0, 0, 70] = x["log_alpha"][0, 1, 0] = -torch.inf
        x["log_alpha"][0, 1, 40:100] = 0.0
        x["beta"][0, 0, 10:90] = 0.0
        x["beta"][0, 1, ::2] = 1.0
        x["log_alpha"][1, 0, 20:40] = -torch.inf
        x["log_alpha"][1, 1, :] = -60.0
    run_case(5, 2, 2, 2, 140, 64, 64, F32, edit=edit, saved=False)


@pytest.mark.parametrize("T", [70, 5])
def test_bf16_unaligned_views_take_the_serial_kernel(T):
    x = inputs(4, 1, 2, 2, T, 64, 64, BF16, BF16)
    y, end = delta(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], 0.125, x["state"])
    g = to_gpu(x, BF16, BF16)
    wide = lambda t: torch.nn.functional.pad(t, (4, 4))[..., 4:-4]  # noqa: E731
    args = wide(g["q"]), wide(g["k"]), wide(g["v"]), g["log_alpha"], g["beta"]
    got, gend, _ = ws.gl_delta_fwd(*args, state=g["state"], want_state=True)
    assert rel(got, y) <= TOL[BF16] and rel(gend, end) <= STATE_TOL[BF16]
    with pytest.raises(ws.GLScanError):
        ws.gl_delta_fwd(*args, state=g["state"], save=True)


def test_fp32_unaligned_views_take_the_serial_kernel():
    """Slices of a wider row that start at 4 bytes: same results, token by token."""
    x = inputs(4, 1, 2, 2, 70, 64, 64, F32, F32)
    y, _ = delta(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], 0.125, x["state"])
    g = to_gpu(x, F32, F32)
    wide = lambda t: torch.nn.functional.pad(t, (1, 3))[..., 1:-3]
    got, _, _ = ws.gl_delta_fwd(wide(g["q"]), wide(g["k"]), g["v"], g["log_alpha"], g["beta"], state=g["state"])
    assert rel(got, y) <= TOL[F32]


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (24, 72), (128, 40), (72, 128)])
@pytest.mark.parametrize("segments,T,lens", [(2, 129, None), (3, 400, None), (5, 64 * 5, None), (7, 64 * 11 + 1, None),
                                             (4, 700, [1, 0, 500, 64, 135]), (100, 300, None)])
def test_segments(dk, dv, segments, T, lens):
    """The chunks of a sequence cut into segments that run at once."""
    run_case(dk + T, 1, 2, 1, T, dk, dv, BF16, lens=lens, order="bthd", segments=segments, decay="near1")


def test_segments_chosen_for_few_heads_and_long_sequences():
    """One head of 2,600 tokens is cut by itself; results as for one segment."""
    g, y, end, _ = run_case(11, 1, 1, 1, 2600, 64, 64, BF16, saved=False)
    one, end1, _ = ws.gl_delta_fwd(g["q"], g["k"], g["v"], g["log_alpha"], g["beta"], state=g["state"],
                                   want_state=True, segments=1)
    assert rel(y, one.double().cpu()) <= TOL[BF16] and rel(end, end1.double().cpu()) <= STATE_TOL[BF16]
    again = ws.gl_delta_fwd(g["q"], g["k"], g["v"], g["log_alpha"], g["beta"], state=g["state"], want_state=True)
    assert torch.equal(again[0], y) and torch.equal(again[1], end)


@pytest.mark.parametrize("dk,dv,T,lens", [
    (64, 64, 64, None), (64, 64, 65, None), (20, 36, 200, None), (128, 128, 257, None), (96, 80, 130, None),
    (4, 4, 70, None), (64, 64, 264, [1, 63, 0, 65, 130, 5]), (128, 44, 200, [0, 200]), (128, 128, 700, None)])
@pytest.mark.parametrize("H,Hk,decay", [(4, 2, "mix"), (3, 3, "near1"), (3, 1, "base")])
def test_fp32_training_chunks(dk, dv, T, lens, H, Hk, decay):
    run_case(dk + T + H, 1 if lens else 2, H, Hk, T, dk, dv, F32, lens=lens, order="bthd", decay=decay)


@pytest.mark.parametrize("dtype", [F32, F64])
def test_serial_training(dtype):
    run_case(9, 1, 4, 2, 100, 64, 72, dtype, flags=ws.GL_FLAG_GENERIC)
    run_case(10, 1, 2, 2, 100, 128, 30, dtype, lens=[0, 17, 70, 13])


def test_fp32_long_sequence_gradients():
    """The decay's gradient is a sum over what follows: no error may grow along it."""
    run_case(12, 1, 1, 1, 3000, 16, 16, F32, decay="near1")
    run_case(13, 1, 1, 1, 3000, 16, 16, BF16, gate=F32, decay="near1")


@pytest.mark.parametrize("T,lens", [(3, None), (4, None), (15, None), (16, None), (40, [3, 1, 0, 2, 34]),
                                    (12, [3, 3, 3, 3]), (11, [3, 3, 3, 2])])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_around_the_shortest_chunked_sequences(T, lens, dtype):
    for saved in (True, False):
        run_case(T, 1 if lens else 3, 4, 2, T, 64, 64, dtype, lens=lens, saved=saved)


@pytest.mark.parametrize("segments", [2, 3, 6])
def test_segments_without_saved(segments):
    run_case(70 + segments, 2, 2, 2, 64 * 9 + 7, 64, 64, BF16, gate=F32, saved=False, segments=segments)
    run_case(80 + segments, 1, 3, 1, 64 * 9 + 7, 128, 96, BF16, with_state=False, segments=segments, decay="base")


def test_calls_of_one_kind_then_others():
    """Checked calls are remembered by shapes, strides, types and devices: a call
    that differs in any of them is checked anew, and refused or right."""
    x = inputs(50, 3, 4, 2, 1, 64, 64, BF16)
    g = to_gpu(x, BF16, BF16)
    one = {n: g[n][:, :, 0].contiguous() for n in ("q", "k", "v", "log_alpha", "beta")}
    names = list(one)
    step = lambda state, **kw: ws.gl_delta_step(*[kw.get(n, one[n]) for n in names], state)  # noqa: E731
    first = g["state"].clone()
    y = step(first)
    for _ in range(2):
        again = g["state"].clone()
        assert torch.equal(step(again), y) and torch.equal(again, first)
    strided = torch.nn.functional.pad(one["v"], (0, 64))[..., :64]
    again = g["state"].clone()
    assert torch.equal(step(again, v=strided), y) and torch.equal(again, first)
    for bad, err in ((dict(v=one["v"].cpu()), ValueError), (dict(v=one["v"].float()), TypeError),
                     (dict(k=one["k"][..., :32]), ValueError), (dict(log_alpha=one["log_alpha"][:2]), ValueError),
                     (dict(q=one["q"].cpu()), ValueError), (dict(beta=one["beta"].double()), TypeError)):
        with pytest.raises(err):
            step(g["state"].clone(), **bad)
    with pytest.raises(ValueError):
        step(g["state"][:2].clone())
    assert torch.equal(step(g["state"].clone()), y)
    # running positions are no new kind of call
    q = g["q"]
    cos, sin = torch.rand(2, 40, 32, device="cuda")
    for p in range(3):
        a = ws.gl_qknorm_rope_fwd(q, q, cos=cos, sin=sin, pos0=p)[0]
        pos = torch.full((3, 1), p, dtype=torch.int32, device="cuda")
        assert torch.equal(a, ws.gl_qknorm_rope_fwd(q, q, cos=cos, sin=sin, pos=pos)[0])


def test_autograd_of_unaligned_slices():
    x = inputs(61, 1, 2, 2, 80, 64, 64, BF16, BF16)
    names = ["q", "k", "v", "log_alpha", "beta"]
    for n in names:
        x[n].requires_grad_(True)
    y, _ = delta(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], 0.125)
    want = torch.autograd.grad((y * x["dy"]).sum(), [x[n] for n in names])
    g = to_gpu(x, BF16, BF16)
    leaves = [torch.nn.functional.pad(g[n], (4, 4)) if n in "qkv" else g[n].clone() for n in names]
    for p in leaves:
        p.requires_grad_(True)
    got, _ = ws.delta_rule(*[p[..., 4:-4] if p.dim() == 4 else p for p in leaves])
    (got.float() * g["dy"].float()).sum().backward()
    assert rel(got, y) <= TOL[BF16]
    for n, p, w in zip(names, leaves, want):
        assert rel(p.grad[..., 4:-4] if p.dim() == 4 else p.grad, w) <= TOL[BF16], n
