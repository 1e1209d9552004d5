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
