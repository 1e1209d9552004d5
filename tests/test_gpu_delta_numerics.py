"""The gated delta rule on the GPU where its numbers are hard: gates that are not
numbers, strong forgetting, sequences of very unequal lengths, long ones.  The
oracle is the token-by-token definition in 64 bits."""
import pytest
import torch

import weight_scans_amd as ws
from delta_ref import delta, inputs, rel
from test_gpu_delta import BF16, F32, F64, STATE_TOL, TOL, run_case, to_gpu

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ not a number
@pytest.mark.parametrize("dtype,gate,T,segments", [(BF16, BF16, 140, 0), (BF16, F32, 140, 0), (F32, F32, 140, 0),
                                                   (F64, F64, 140, 0), (BF16, BF16, 3, 0), (BF16, BF16, 700, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_decay_that_is_no_number(dtype, gate, T, segments, d):
    """It reaches its own token, every later one and the state; other heads and the
    chunks of 64 before it keep their values; its gradient is no number."""
    bad = T // 2
    x = inputs(d + T, 1, 2, 2, T, d, d, dtype, gate)
    want, end = delta(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], d ** -0.5, x["state"])
    x["log_alpha"][0, 0, bad] = torch.nan
    g = to_gpu(x, dtype, gate)
    args = [g[n] for n in ("q", "k", "v", "log_alpha", "beta")]
    for save in (True, False):
        y, state, saved = ws.gl_delta_fwd(*args, state=g["state"], want_state=True, save=save, segments=segments)
        assert torch.isnan(y[0, 0, bad:]).all() and torch.isnan(state[0, 0]).all()
        sure = bad // 64 * 64
        if sure:
            assert rel(y[0, 0, :sure], want[0, 0, :sure]) <= TOL[dtype]
        assert rel(y[0, 1], want[0, 1]) <= TOL[dtype] and rel(state[0, 1], end[0, 1]) <= STATE_TOL[dtype]
        grads = ws.gl_delta_bwd(*args, g["dy"], saved, state=g["state"], dstate=g["dstate"], segments=segments)
        assert torch.isnan(grads[3][0, 0, bad])
        assert all(torch.isfinite(t[0, 1].double()).all() for t in grads)


# ------------------------------------------------------------ strong forgetting
# dlog_alpha per head (2-norm), its gates in fp32.  Where a token keeps less than 2^-5.5 the
# gradient is a sum of what crosses the token, of factors rounded once each (bf16: 1.7e-3 rms, up
# to three of them in quadrature 3e-3, and room for terms that cancel: 1e-2; fp32: products of 64
# tokens and 128 rows, 1e-5).  Where it keeps more, it is a running difference of terms that the
# factor does not scale: 3e-6 (fp32 2e-7) of them a token, in quadrature over 500 (64) tokens,
# and 45 times that (1 / 0.022): 3e-3 (7e-5).
DECAY_TOL = {BF16: 1e-2, F32: 1e-4, F64: 1e-10}


def decay_gradient(x, dtype, gate, lens=None, segments=0, H=2):
    names = ["q", "k", "v", "log_alpha", "beta", "state"]
    for n in names:
        x[n].requires_grad_(True)
    d = x["q"].shape[-1]
    y, end = delta(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], d ** -0.5, x["state"], lens)
    want = torch.autograd.grad((y * x["dy"]).sum() + (end * x["dstate"]).sum(), x["log_alpha"])[0]
    g = to_gpu(x, dtype, gate)
    cu = None if lens is None else torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32).cuda()
    args = [g[n] for n in names[:5]]
    _, _, saved = ws.gl_delta_fwd(*args, state=g["state"], save=True, cu_seqlens=cu, segments=segments)
    got = ws.gl_delta_bwd(*args, g["dy"], saved, state=g["state"], dstate=g["dstate"], cu_seqlens=cu,
                          segments=segments)[3]
    return got.double().cpu(), want


@pytest.mark.parametrize("decay", [-1.0, -3.0, -3.3, -5.0, -8.0, -15.0, -40.0])
@pytest.mark.parametrize("dtype,dk,dv,H,Hk", [(BF16, 64, 64, 2, 2), (BF16, 128, 128, 2, 1), (BF16, 128, 40, 3, 1),
                                              (BF16, 24, 128, 2, 2), (F32, 64, 64, 2, 2), (F32, 128, 100, 4, 2),
                                              (F64, 64, 64, 2, 2)])
def test_decay_gradient_of_uniform_decays(decay, dtype, dk, dv, H, Hk):
    gate = F64 if dtype == F64 else F32
    x = inputs(int(-10 * decay) + dk, 1, H, Hk, 330, dk, dv, dtype, gate)
    x["log_alpha"] = (decay * (1 + 0.02 * torch.randn(x["log_alpha"].shape, dtype=F64))).to(gate).double()
    got, want = decay_gradient(x, dtype, gate)
    for h in range(H):
        e = rel(got[0, h], want[0, h])
        print(f"head {h}: {e:.1e}", flush=True)
        assert e <= DECAY_TOL[dtype], (h, e)


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128), (F64, 64)])
@pytest.mark.parametrize("segments,lens", [(0, None), (3, None), (0, [1, 200, 0, 65, 134])])
def test_decay_gradient_of_single_strong_tokens(dtype, d, segments, lens):
    """Among tokens that keep nearly all, those that keep little, judged by themselves."""
    gate = F64 if dtype == F64 else F32
    x = inputs(d + segments, 1, 2, 2, 400, d, d, dtype, gate, n=None if lens is None else len(lens), decay="near1")
    for first, v in ((3, -4.0), (5, -9.0), (8, -20.0)):
        x["log_alpha"][:, :, first::17] = v
    got, want = decay_gradient(x, dtype, gate, lens, segments)
    for h in range(2):
        for first in (3, 5, 8):
            e = rel(got[0, h, first::17], want[0, h, first::17])
            print(f"head {h} tokens {first}::17: {e:.1e}", flush=True)
            assert e <= DECAY_TOL[dtype], (h, first, e)
        assert rel(got[0, h], want[0, h]) <= DECAY_TOL[dtype]


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 64), (F64, 64)])
@pytest.mark.parametrize("boundary", [100, 256])
def test_decay_gradient_before_a_boundary(dtype, d, boundary):
    """A token that forgets everything ends a text; the text behind it has gradients a
    thousand times as large, of which nothing may be left in the one before."""
    gate = F64 if dtype == F64 else F32
    x = inputs(d, 1, 2, 2, 500, d, d, dtype, gate, decay="near1")
    x["log_alpha"][:, :, boundary] = -torch.inf
    x["dy"][:, :, boundary:] *= 1024
    x["dstate"] *= 1024
    got, want = decay_gradient(x, dtype, gate)
    assert (got[:, :, boundary] == 0).all()
    for h in range(2):
        e = rel(got[0, h, :boundary], want[0, h, :boundary])
        print(f"head {h}: {e:.1e}", flush=True)
        assert e <= DECAY_TOL[dtype], (h, e)


# ------------------------------------------------------------ one rounding
@pytest.mark.parametrize("dk,dv,T,decay", [(64, 64, 200, "mix"), (128, 128, 200, "near1"), (64, 128, 130, "base"),
                                           (128, 40, 330, "near1")])
def test_value_gradients_are_rounded_once(dk, dv, T, decay):
    """dv = beta G leaves the reverse recurrence's fp32: 1.7e-3 rms of its rounding, in
    quadrature with some 1e-5 of the recurrence; 2e-3 with room."""
    x = inputs(dk + dv + T, 1, 4, 2, T, dk, dv, BF16, decay=decay)
    names = ["q", "k", "v", "log_alpha", "beta"]
    for n in names:
        x[n].requires_grad_(True)
    y, _ = delta(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], dk ** -0.5)
    want = torch.autograd.grad((y * x["dy"]).sum(), x["v"])[0]
    g = to_gpu(x, BF16, BF16)
    args = [g[n] for n in names]
    for segments in (1, 2):
        _, _, saved = ws.gl_delta_fwd(*args, save=True, segments=segments)
        got = ws.gl_delta_bwd(*args, g["dy"], saved, segments=segments)[2]
        for h in range(4):
            assert rel(got[0, h], want[0, h]) <= 2e-3, (segments, h)


# ------------------------------------------------------------ lengths
@pytest.mark.parametrize("lens", [[700] + [1] * 30, [1] * 30 + [700], [2, 900, 0] + [1] * 230, [65] + [3] * 200])
@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 64)])
def test_packed_of_very_unequal_lengths(lens, dtype, d):
    for saved in (True, False):
        run_case(len(lens), 1, 2, 1, sum(lens), d, d, dtype, lens=lens, order="bthd", saved=saved)


@pytest.mark.parametrize("dk,dv,segments", [(64, 64, 1), (128, 128, 0)])
def test_long_sequences(dk, dv, segments):
    run_case(dk, 1, 2, 1, 4100, dk, dv, BF16, gate=F32, decay="near1", segments=segments)
