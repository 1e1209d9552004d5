"""The selective state space scan with its short causal convolution, and the norms
before and after a block with its gate and residual scale, as cases that can be
timed and compared.

`run` takes a prepared state through ONE pass of an operator: in its plain form
(elementary torch operations in 32 bits, rounded once at the end) where `own` is
false, through the public calls of weight_scans_amd where it is true.  `exact`
gives the same outputs from the operators' definitions in 64 bits.

Causal convolution, per channel d of x [B,T,D], K taps, x before a sequence's
first token from its state (its last K - 1 inputs) or zero:

    p_t = bias + sum_j w[d,j] x_(t-K+1+j),     y_t = silu(p_t)

Selective scan, per channel d and state n (B, C shared by D / G channels):

    D_t = softplus(dt_t + bias),   h_t = exp(D_t A[d,n]) h_(t-1) + D_t x_t B_t[n]
    y_t = (sum_n C_t[n] h_t + skip[d] x_t) silu(z_t)

Residual norm, per row:   u = wx * x / rms(x) (or x),  r' = r + s * u,
                          n = w * r' / rms(r')
Gated norm, per row:      y = w * x / rms(x) * silu(z),  or of v = x silu(z):  w * v / rms(v)

with rms(x) = sqrt(mean(x^2) + eps).
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ the cases
def _conv(name, op, B, T, D, K, dtype, seqs=0, state=False, bias=True, silu=True):
    return {"name": name, "op": op, "B": B, "T": T, "D": D, "K": K, "dtype": dtype, "seqs": seqs,
            "state": state, "bias": bias, "silu": silu}


def _scan(name, op, B, T, D, N, G, dtype, seqs=0, state=False, gate=True):
    return {"name": name, "op": op, "B": B, "T": T, "D": D, "N": N, "G": G, "dtype": dtype,
            "seqs": seqs, "state": state, "gate": gate}


def _norm(name, op, B, T, d, dtype, res="io", post=False, scale=True):
    return {"name": name, "op": op, "B": B, "T": T, "d": d, "dtype": dtype, "res": res, "post": post,
            "scale": scale}


def _gate(name, op, B, T, G, d, dtype, first=False, shared=True):
    return {"name": name, "op": op, "B": B, "T": T, "G": G, "d": d, "dtype": dtype, "first": first,
            "shared": shared}


def listed():
    return [
        # a full serving batch's next token: the windows of a pool move on by one input
        _conv("conv_step", "conv_step", 256, 1, 2048, 4, "bf16"),
        # prompts packed one after another in fp32, an odd number of channels, three taps
        _conv("conv_packed", "conv_fwd", 1, 3001, 1001, 3, "f32", 7, True),
        # training, forward and backward, ahead of a layer of 2048 channels
        _conv("conv_train", "conv_train", 4, 4096, 2048, 4, "bf16"),
        # a full serving batch's next token out of a pool of states in another order
        _scan("scan_step", "scan_step", 256, 1, 2048, 16, 1, "bf16"),
        # a few short prompts, one of no token and one of one among them, that continue
        # from cached states: little to share out over the chip
        _scan("scan_packed", "scan_fwd", 1, 777, 2048, 16, 1, "bf16", 5, True),
        # one long document
        _scan("scan_long", "scan_fwd", 1, 32768, 2048, 16, 1, "bf16", 0, True),
        # training at the width of the larger scans' workload
        _scan("scan_train", "scan_train", 4, 4096, 2048, 16, 1, "bf16"),
        # training in fp32 on odd sizes: groups of channels, first states, no gate
        _scan("scan_odd", "scan_train", 3, 1021, 520, 24, 2, "f32", 0, True, False),
        # between two blocks of one decoding step: all latency
        _norm("norm_decode", "norm_fwd", 64, 1, 2048, "bf16"),
        # between two blocks in training: the residual in fp32, norms on both sides
        _norm("norm_train", "norm_train", 4, 4096, 2048, "bf16", "f32", True),
        # after the heads of a layer in training: every head's row normed, then gated
        _gate("gate_train", "gate_train", 4, 4096, 16, 128, "bf16"),
        # rows of an odd length in fp32, gated before the norm, weights of each group
        _gate("gate_odd", "gate_train", 3, 1021, 2, 997, "f32", True, False),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_step", "conv_fwd", "conv_train", "scan_step", "scan_fwd", "scan_fwd", "scan_train",
                     "scan_train", "norm_fwd", "norm_train", "gate_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.endswith("step"):
        B, T, seqs = _logint(rng, 1, 256), 1, 0
    else:
        seqs = rng.randrange(2, 12) if rng.random() < 0.3 else 0
        B = 1 if seqs else _logint(rng, 1, 8)
        T = _logint(rng, 1, 4096 if op.endswith("train") else 32768)
    if op.startswith("norm"):
        B, T = _logint(rng, 1, 8), _logint(rng, 1, 4096)
        return {"op": op, "B": B, "T": T, "d": _width(rng, B * T, 32, 4096, 4 * 4096 * 2048), "dtype": dtype,
                "res": rng.choice(["io", "f32"]), "post": rng.random() < 0.5, "scale": rng.random() < 0.7}
    if op.startswith("gate"):
        B, T, G = _logint(rng, 1, 8), _logint(rng, 1, 4096), rng.choice([1, 2, 8, 16])
        return {"op": op, "B": B, "T": T, "G": G, "d": _width(rng, B * T * G, 16, 2048, 4 * 4096 * 2048),
                "dtype": dtype, "first": rng.random() < 0.5, "shared": rng.random() < 0.5}
    if op.startswith("conv"):
        return {"op": op, "B": B, "T": T, "D": _width(rng, B * T, 64, 6144, 4 * 4096 * 2048), "K": rng.choice([2, 3, 4, 4]),
                "dtype": dtype, "seqs": seqs, "state": rng.random() < 0.6, "bias": rng.random() < 0.7,
                "silu": rng.random() < 0.8}
    N = rng.choice([16, 16, 16, 8, 64, rng.randrange(1, 65)])
    G = rng.choice([1, 1, 2, 4])
    most = (1 if dtype == "bf16" else 0.25) * (2 if op == "scan_train" else 4) * 4096 * 2048 * 16
    D = _width(rng, B * T * N * G, 64 // G, 4096 // G, most) * G
    return {"op": op, "B": B, "T": T, "D": D, "N": N, "G": G, "dtype": dtype, "seqs": seqs,
            "state": rng.random() < 0.6, "gate": rng.random() < 0.7}


def _width(rng, rows, lo, hi, most):
    """Columns of a row, half the time a multiple of 64, no more than `most` elements in all."""
    hi = max(lo, min(hi, int(most / rows)))
    w = _logint(rng, lo, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.5 and hi >= 64 else w


def _size(case):
    return {"bf16": 2, "f32": 4}[case["dtype"]]


def _sets(case):
    return case["seqs"] or case["B"]


def work(case):
    e, op, tok = _size(case), case["op"], case["B"] * case["T"]
    if op.startswith("norm"):
        n, r = tok * case["d"], 4 if case["res"] == "f32" else e
        if op == "norm_fwd":
            return {"bytes": n * (2 * e + 2 * r), "flops": 8 * n}
        # forward: x, r -> n, r'; backward: x, r, dn, dr' -> dx, dr
        return {"bytes": n * (5 * e + 5 * r), "flops": 30 * n}
    if op.startswith("gate"):
        n = tok * case["G"] * case["d"]
        return {"bytes": n * 8 * e, "flops": 30 * n}
    if op.startswith("conv"):
        n, K = tok * case["D"], case["K"]
        st = _sets(case) * case["D"] * (K - 1) * e
        if op == "conv_step":
            return {"bytes": 2 * n * e + 2 * st, "flops": n * (2 * K + 5)}
        if op == "conv_fwd":
            return {"bytes": 2 * n * e + (2 if case["state"] else 1) * st, "flops": n * (2 * K + 5)}
        # forward: x -> y; backward: x, dy -> dx
        return {"bytes": 5 * n * e + (4 * st if case["state"] else 0), "flops": n * (8 * K + 18)}
    D, N, G = case["D"], case["N"], case["G"]
    row, bc, z = tok * D * e, 2 * tok * G * N * e, 1 if case["gate"] else 0
    st = _sets(case) * D * N * 4
    # an exponential, two products and two sums of products an element and token
    if op == "scan_step":
        return {"bytes": (3 + z) * row + bc + 2 * st, "flops": tok * D * (7 * N + 10)}
    if op == "scan_fwd":
        return {"bytes": (3 + z) * row + bc + (2 if case["state"] else 1) * st, "flops": tok * D * (7 * N + 10)}
    states = 4 * st if case["state"] else 0
    # forward: x, dt, z -> y; backward: x, dt, z, dy -> dx, ddt, dz
    return {"bytes": (8 + 3 * z) * row + 3 * bc + states, "flops": tok * D * (24 * N + 30)}


# ------------------------------------------------------------------ the inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lengths(case, seed):
    """Lengths of the packed sequences: uneven shares of T, one empty, one of one token."""
    n, T = case["seqs"], case["T"]
    r = np.random.RandomState(seed % (1 << 31))
    w = np.exp(r.uniform(0, 2, n))
    cuts = np.floor(np.cumsum(w) / w.sum() * T).astype(np.int64)
    cuts[-1] = T
    lens = np.diff(np.concatenate([[0], cuts]))
    if n > 2 and T > 2:
        i, j = r.choice(n, 2, replace=False)
        k = (set(range(n)) - {int(i), int(j)}).pop()
        lens[k] += lens[i] + lens[j] - 1
        lens[i], lens[j] = 0, 1
    if lens.min() < 0:
        lens[:] = 0
        lens[-1] = T
    return [int(x) for x in lens]


def _slots(case, g, s):
    n = case["B"] + case["B"] // 4  # the pool has a few more states than the batch takes
    s["slots"] = torch.randperm(n, generator=g, device="cuda")[: case["B"]].to(torch.int32)
    return n


def prepare(case, seed):
    g, t = _gen(seed), _TYPES[case["dtype"]]
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = {"case": case}
    s["state"] = s["cu"] = s["lens"] = s["dstate"] = None
    if case.get("seqs"):
        s["lens"] = _lengths(case, seed)
        s["cu"] = torch.tensor([0] + list(np.cumsum(s["lens"])), dtype=torch.int32, device="cuda")
    kind = case["op"].split("_")[0]
    {"conv": _prepare_conv, "scan": _prepare_scan, "norm": _prepare_norm, "gate": _prepare_gate}[kind](case, g, t, s, rand)
    return s


def _prepare_conv(case, g, t, s, rand):
    B, T, D, K = case["B"], case["T"], case["D"], case["K"]
    # a slice of a fused projection's output: the gate's columns stand behind it
    s["x"] = rand(B, T, 2 * D).to(t)[..., :D]
    s["w"] = (rand(D, K) * K ** -0.5).to(t)
    s["bias"] = (0.1 * rand(D)).to(t) if case["bias"] else None
    if case["op"] == "conv_step":
        s["x"] = s["x"][:, 0]
        s["state"] = rand(_slots(case, g, s), K - 1, D).to(t)
    elif case["state"]:
        s["state"] = rand(_sets(case), K - 1, D).to(t)
    if case["op"] == "conv_train":
        s["dy"] = rand(B, T, D).to(t)
        if case["state"]:
            s["dstate"] = rand(_sets(case), K - 1, D).to(t)


def _prepare_scan(case, g, t, s, rand):
    B, T, D, N, G = case["B"], case["T"], case["D"], case["N"], case["G"]
    x = rand(B, T, D)
    s["x"] = (x * torch.sigmoid(x)).to(t)
    s["dt"] = (0.5 * rand(B, T, D)).to(t)
    # steps between 0.001 and 0.1, and decays -1 .. -N that training has moved
    step = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -torch.exp(torch.arange(1, N + 1, device="cuda").float().log() + 0.1 * rand(D, N))
    bc = rand(B, T, 2 * G * N).to(t)  # one projection's output
    s["B"] = bc[..., : G * N].view(B, T, G, N)
    s["C"] = bc[..., G * N :].view(B, T, G, N)
    s["skip"] = 1 + 0.1 * rand(D)
    s["z"] = rand(B, T, 2 * D).to(t)[..., D:] if case["gate"] else None
    if case["op"] == "scan_step":
        s["state"] = 0.3 * rand(_slots(case, g, s), D, N)
        for n in ("x", "dt", "B", "C", "z"):
            s[n] = None if s[n] is None else s[n][:, 0]
    elif case["state"]:
        s["state"] = 0.3 * rand(_sets(case), D, N)
    if case["op"] == "scan_train":
        s["dy"] = rand(B, T, D).to(t)
        if case["state"]:
            s["dstate"] = 0.3 * rand(_sets(case), D, N)


def _prepare_norm(case, g, t, s, rand):
    shape = (case["B"], case["T"], case["d"])
    r = torch.float32 if case["res"] == "f32" else t
    s["x"], s["r"] = rand(*shape).to(t), (2 * rand(*shape)).to(r)
    s["w"] = (1 + 0.1 * rand(case["d"])).to(t)
    s["wx"] = (1 + 0.1 * rand(case["d"])).to(t) if case["post"] else None
    s["scale"] = (0.5 + 0.1 * rand(case["d"])).to(t) if case["scale"] else None
    if case["op"] == "norm_train":
        s["dn"], s["dr_out"] = rand(*shape).to(t), rand(*shape).to(r)


def _prepare_gate(case, g, t, s, rand):
    B, T, G, d = case["B"], case["T"], case["G"], case["d"]
    s["x"] = rand(B, T, G, d).to(t)
    s["z"] = rand(B, T, 2 * G * d).to(t)[..., G * d :].view(B, T, G, d)
    s["w"] = (1 + 0.1 * rand(*((d,) if case["shared"] else (G, d)))).to(t)
    s["dy"] = rand(B, T, G, d).to(t)


# ------------------------------------------------------------------ one pass
def run(s):
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


def _own_conv_step(s):
    import weight_scans_amd as ws
    y = ws.gl_conv_step(s["x"], s["w"], s["bias"], s["state"], slots=s["slots"], silu=s["case"]["silu"])
    return {"y": y, "state": s["state"]}


def _own_conv_fwd(s):
    import weight_scans_amd as ws
    y, state = ws.gl_conv_fwd(s["x"], s["w"], s["bias"], state=s["state"], want_state=True, cu_seqlens=s["cu"],
                              silu=s["case"]["silu"])
    return {"y": y, "state": state}


def _own_conv_train(s):
    import weight_scans_amd as ws
    with_state = s["state"] is not None
    y, state = ws.gl_conv_fwd(s["x"], s["w"], s["bias"], state=s["state"], want_state=with_state, cu_seqlens=s["cu"],
                              silu=s["case"]["silu"])
    dx, dw, dbias, dstate = ws.gl_conv_bwd(s["x"], s["w"], s["bias"], s["dy"], state=s["state"], dstate=s["dstate"],
                                           cu_seqlens=s["cu"], silu=s["case"]["silu"])
    out = {"y": y, "dx": dx, "dw": dw, "dbias": dbias}
    return out | ({"state": state, "dstate_in": dstate} if with_state else {})


def _scan_args(s):
    return s["x"], s["dt"], s["A"], s["B"], s["C"], s["skip"], s["z"], s["dt_bias"]


def _own_scan_step(s):
    import weight_scans_amd as ws
    y = ws.gl_ssm_step(*_scan_args(s), s["state"], slots=s["slots"])
    return {"y": y, "state": s["state"]}


def _own_scan_fwd(s):
    import weight_scans_amd as ws
    y, state, _ = ws.gl_ssm_fwd(*_scan_args(s), state=s["state"], want_state=True, cu_seqlens=s["cu"])
    return {"y": y, "state": state}


def _own_scan_train(s):
    import weight_scans_amd as ws
    with_state = s["state"] is not None
    y, state, saved = ws.gl_ssm_fwd(*_scan_args(s), state=s["state"], want_state=with_state, save=True,
                                    cu_seqlens=s["cu"])
    dx, ddt, dA, dB, dC, dskip, dz, dbias, dstate = ws.gl_ssm_bwd(
        *_scan_args(s), s["dy"], saved, state=s["state"], dstate=s["dstate"], cu_seqlens=s["cu"])
    out = {"y": y, "dx": dx, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dskip": dskip, "dz": dz, "dbias": dbias}
    return out | ({"state": state, "dstate_in": dstate} if with_state else {})


def _own_norm_fwd(s):
    import weight_scans_amd as ws
    n, r = ws.gl_addnorm_fwd(s["x"], s["r"], s["w"], s["wx"], s["scale"], eps=EPS)
    return {"n": n, "r": r}


def _own_norm_train(s):
    import weight_scans_amd as ws
    dx, dr, dw, dwx, dscale = ws.gl_addnorm_bwd(s["x"], s["r"], s["w"], s["wx"], s["scale"], s["dn"], s["dr_out"],
                                                eps=EPS)
    return _own_norm_fwd(s) | {"dx": dx, "dr": dr, "dw": dw, "dwx": dwx, "dscale": dscale}


def _own_gate_train(s):
    import weight_scans_amd as ws
    y = ws.gl_gatenorm_fwd(s["x"], s["z"], s["w"], eps=EPS, gate_first=s["case"]["first"])
    dx, dz, dw = ws.gl_gatenorm_bwd(s["x"], s["z"], s["w"], s["dy"], eps=EPS, gate_first=s["case"]["first"])
    return {"y": y, "dx": dx, "dz": dz, "dw": dw}


# ------------------------------------------------------------------ the plain form: the convolution
def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _bounds(s):
    """(sequence, its tokens) in the batch's layout: rows of B, or runs of the packed axis."""
    if s["lens"] is None:
        return [(slice(None), slice(None), slice(0, s["case"]["T"]))]
    cu = np.concatenate([[0], np.cumsum(s["lens"])])
    return [(slice(n, n + 1), slice(None), slice(int(cu[n]), int(cu[n + 1]))) for n in range(len(s["lens"]))]


def _window(s, sets, run):
    """x of these tokens behind the K - 1 inputs before them, fp32."""
    case = s["case"]
    x = s["x"][:, run].float()
    if s["state"] is not None:
        return torch.cat([s["state"][sets].float(), x], 1)
    return torch.cat([torch.zeros((x.shape[0], case["K"] - 1, case["D"]), device="cuda"), x], 1)


def _taps(s, full, T):
    w = s["w"].float()
    p = sum(full[:, j : j + T] * w[:, j] for j in range(s["case"]["K"]))
    return p if s["bias"] is None else p + s["bias"].float()


def _plain_conv_fwd(s, want=True):
    K, t = s["case"]["K"], s["x"].dtype
    ys, ends = [], []
    for sets, rows, run in _bounds(s):
        full = _window(s, sets, run)
        p = _taps(s, full, run.stop - run.start)
        ys.append(p * _sigmoid(p) if s["case"]["silu"] else p)
        ends.append(full[:, full.shape[1] - (K - 1) :])
    out = {"y": torch.cat(ys, 1).to(t)}
    return out | ({"state": torch.cat(ends).to(t)} if want else {})


def _plain_conv_step(s):
    at, t = s["slots"].long(), s["x"].dtype
    full = torch.cat([s["state"][at].float(), s["x"].float()[:, None]], 1)
    p = _taps(s, full, 1)[:, 0]
    s["state"][at] = full[:, 1:].to(t)
    return {"y": (p * _sigmoid(p) if s["case"]["silu"] else p).to(t), "state": s["state"]}


def _plain_conv_train(s):
    case, t = s["case"], s["x"].dtype
    K, D, with_state = case["K"], case["D"], s["state"] is not None
    w = s["w"].float()
    dw, dbias = torch.zeros((D, K), device="cuda"), torch.zeros(D, device="cuda")
    dxs, firsts = [], []
    for sets, rows, run in _bounds(s):
        T = run.stop - run.start
        full = _window(s, sets, run)
        p, dp = _taps(s, full, T), s["dy"][:, run].float()
        if case["silu"]:
            g = _sigmoid(p)
            dp = dp * g * (1 + p * (1 - g))
        dfull = torch.zeros_like(full)
        if s["dstate"] is not None:
            dfull[:, full.shape[1] - (K - 1) :] += s["dstate"][sets].float()
        for j in range(K):
            dfull[:, j : j + T] += dp * w[:, j]
            dw[:, j] += (dp * full[:, j : j + T]).sum(1).sum(0)
        dbias += dp.sum(1).sum(0)
        dxs.append(dfull[:, K - 1 :])
        firsts.append(dfull[:, : K - 1])
    out = _plain_conv_fwd(s, with_state) | {"dx": torch.cat(dxs, 1).to(t), "dw": dw,
                                            "dbias": None if s["bias"] is None else dbias}
    return out | ({"dstate_in": torch.cat(firsts).to(t)} if with_state else {})


# ------------------------------------------------------------------ the plain form: the selective scan
def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _spread(x, D):
    """[.., G, N] -> [.., D, N] fp32"""
    return x.float().repeat_interleave(D // x.shape[-2], -2)


def _plain_scan_step(s):
    at, D, t = s["slots"].long(), s["case"]["D"], s["x"].dtype
    x = s["x"].float()
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(dt[..., None] * s["A"]) * s["state"][at] + (dt * x)[..., None] * _spread(s["B"], D)
    y = (h * _spread(s["C"], D)).sum(-1) + s["skip"] * x
    if s["z"] is not None:
        y = y * s["z"].float() * _sigmoid(s["z"].float())
    s["state"][at] = h
    return {"y": y.to(t), "state": s["state"]}


SPAN = 1024  # tokens whose states the plain form holds at once


def _first(s, sets, N):
    case = s["case"]
    if s["state"] is not None:
        return s["state"][sets]
    return torch.zeros((N, case["D"], case["N"]), device="cuda")


def _span(s, run, dt, h):
    """States after each token of `run` [B,span,D,N], and their decays."""
    D = s["case"]["D"]
    a = torch.exp(dt[..., None] * s["A"])
    hs = (dt * s["x"][:, run].float())[..., None] * _spread(s["B"][:, run], D)
    for t in range(hs.shape[1]):
        h = torch.addcmul(hs[:, t], a[:, t], h, out=hs[:, t])
    return hs, a


def _plain_scan(s, keep=False):
    case, D = s["case"], s["case"]["D"]
    ys, ends, firsts = [], [], []
    for sets, rows, run in _bounds(s):
        h = _first(s, sets, s["x"].shape[0])
        for lo in range(run.start, run.stop, SPAN):
            part = slice(lo, min(lo + SPAN, run.stop))
            if keep:
                firsts.append((sets, part, h, part.stop == run.stop))
            dt = _softplus(s["dt"][:, part].float() + s["dt_bias"])
            hs, _ = _span(s, part, dt, h)
            h = hs[:, -1].clone()
            y = (hs * _spread(s["C"][:, part], D)).sum(-1) + s["skip"] * s["x"][:, part].float()
            ys.append(y)
        ends.append(h)
    return torch.cat(ys, 1), torch.cat(ends), firsts


def _gated(s, y):
    if s["z"] is not None:
        y = y * s["z"].float() * _sigmoid(s["z"].float())
    return y.to(s["x"].dtype)


def _plain_scan_fwd(s):
    y, end, _ = _plain_scan(s)
    return {"y": _gated(s, y), "state": end}


def _plain_scan_train(s):
    case, t = s["case"], s["x"].dtype
    D, N, G = case["D"], case["N"], case["G"]
    with_state = s["state"] is not None
    y, end, spans = _plain_scan(s, True)
    dy, x, raw = s["dy"].float(), s["x"].float(), s["dt"].float() + s["dt_bias"]
    out = {"y": _gated(s, y), "dz": None}
    if s["z"] is not None:
        z = s["z"].float()
        g = _sigmoid(z)
        out["dz"] = (dy * y * g * (1 + z * (1 - g))).to(t)
        dy = dy * z * g
    dx, ddt = torch.empty_like(x), torch.empty_like(x)
    dB, dC = (torch.empty(s["B"].shape, device="cuda") for _ in range(2))
    dA = torch.zeros((D, N), device="cuda")
    first = torch.zeros((_sets(case), D, N), device="cuda")
    shared = lambda v: v.view(*v.shape[:2], G, D // G, N).sum(3)  # noqa: E731
    lam = None
    for sets, part, h0, last in reversed(spans):
        if last:  # what reaches the state after the last token of the sequence
            lam = s["dstate"][sets].clone() if s["dstate"] is not None else torch.zeros_like(h0)
        dt, xs, dys = _softplus(raw[:, part]), x[:, part], dy[:, part]
        hs, a = _span(s, part, dt, h0)
        Bs = _spread(s["B"][:, part], D)
        gs = dys[..., None] * _spread(s["C"][:, part], D)
        for i in range(gs.shape[1] - 1, -1, -1):
            gs[:, i] += lam
            lam = a[:, i] * gs[:, i]
        first[sets] = lam
        dC[:, part] = shared(hs * dys[..., None])
        dB[:, part] = shared(gs * (dt * xs)[..., None])
        du = (gs * Bs).sum(-1)
        before = torch.cat([h0[:, None], hs[:, :-1]], 1)
        gq = gs * a * before
        dA += (gq * dt[..., None]).sum(1).sum(0)
        ddt[:, part] = (xs * du + (gq * s["A"]).sum(-1)) * _sigmoid(raw[:, part])
        dx[:, part] = dt * du + s["skip"] * dys
    if s["lens"] is not None and s["dstate"] is not None:  # sequences of no token pass it through
        for n, length in enumerate(s["lens"]):
            if length == 0:
                first[n] = s["dstate"][n]
    out |= {"dx": dx.to(t), "ddt": ddt.to(t), "dA": dA, "dB": dB.to(t), "dC": dC.to(t),
            "dskip": (dy * x).sum(1).sum(0), "dbias": ddt.sum(1).sum(0)}
    return out | ({"state": end, "dstate_in": first} if with_state else {})


# ------------------------------------------------------------------ the plain form: the norms
def _rrms(x):
    return (x.square().mean(-1, keepdim=True) + EPS).rsqrt()


def _plain_norm_fwd(s):
    x, r = s["x"].float(), s["r"].float()
    u = x if s["wx"] is None else s["wx"].float() * (x * _rrms(x))
    r = r + (u if s["scale"] is None else s["scale"].float() * u)
    return {"n": (s["w"].float() * (r * _rrms(r))).to(s["x"].dtype), "r": r.to(s["r"].dtype)}


def _rows(x):
    """Sum over the rows, in steps: a long sum of 32 bits keeps its last places so."""
    return x.sum(1).sum(0)


def _plain_norm_train(s):
    x, r, t = s["x"].float(), s["r"].float(), s["x"].dtype
    rx = _rrms(x) if s["wx"] is not None else None
    u = x if rx is None else s["wx"].float() * (x * rx)
    sc = None if s["scale"] is None else s["scale"].float()
    r = r + (u if sc is None else sc * u)
    rr = _rrms(r)
    hat, dn = r * rr, s["dn"].float()
    g = s["w"].float() * dn
    dr = s["dr_out"].float() + rr * (g - hat * (g * hat).mean(-1, keepdim=True))
    du = dr if sc is None else sc * dr
    out = _plain_norm_fwd(s) | {"dr": dr.to(s["r"].dtype), "dw": _rows(dn * hat), "dwx": None,
                                "dscale": None if sc is None else _rows(dr * u), "dx": du.to(t)}
    if rx is not None:
        xh, g = x * rx, s["wx"].float() * du
        out["dwx"] = _rows(du * xh)
        out["dx"] = (rx * (g - xh * (g * xh).mean(-1, keepdim=True))).to(t)
    return out


def _plain_gate_train(s):
    x, z, w, dy, t = s["x"].float(), s["z"].float(), s["w"].float(), s["dy"].float(), s["x"].dtype
    sig = _sigmoid(z)
    gate, slope = z * sig, sig * (1 + z * (1 - sig))
    v = x * gate if s["case"]["first"] else x
    rv = _rrms(v)
    hat = v * rv
    if s["case"]["first"]:
        y, dg = w * hat, dy
    else:
        y, dg = w * hat * gate, dy * gate
    dw = _rows(dg * hat)
    g = w * dg
    dv = rv * (g - hat * (g * hat).mean(-1, keepdim=True))
    dx, dz = (dv * gate, dv * x * slope) if s["case"]["first"] else (dv, dy * w * hat * slope)
    return {"y": y.to(t), "dx": dx.to(t), "dz": dz.to(t), "dw": dw.sum(0) if s["case"]["shared"] else dw}


_OWN = {"conv_step": _own_conv_step, "conv_fwd": _own_conv_fwd, "conv_train": _own_conv_train,
        "scan_step": _own_scan_step, "scan_fwd": _own_scan_fwd, "scan_train": _own_scan_train,
        "norm_fwd": _own_norm_fwd, "norm_train": _own_norm_train, "gate_train": _own_gate_train}
_PLAIN = {"conv_step": _plain_conv_step, "conv_fwd": _plain_conv_fwd,
          "conv_train": _plain_conv_train,
          "scan_step": _plain_scan_step, "scan_fwd": _plain_scan_fwd, "scan_train": _plain_scan_train,
          "norm_fwd": _plain_norm_fwd, "norm_train": _plain_norm_train, "gate_train": _plain_gate_train}


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f = {n: (x.double() if torch.is_tensor(x) and x.is_floating_point() else x) for n, x in s.items()}
    kind = case["op"].split("_")[0]
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm, "gate": _exact_gate}[kind](case, f)


def _silu64(p):
    return p / (1 + torch.exp(-p))


def _dsilu64(p):
    e = torch.exp(-p)
    return (1 + e + p * e) / (1 + e).square()


def _exact_conv(case, f):
    K, T = case["K"], case["T"]
    if case["op"] == "conv_step":
        at = f["slots"].long()
        pool = f["state"].clone()
        p = (pool[at] * f["w"].T[: K - 1]).sum(1) + f["x"] * f["w"][:, K - 1]
        p = p if f["bias"] is None else p + f["bias"]
        pool[at] = torch.stack([*pool[at].unbind(1)[1:], f["x"]], 1)
        return {"y": _silu64(p) if case["silu"] else p, "state": pool}
    train, with_state = case["op"] == "conv_train", f["state"] is not None
    lens = f["lens"] or [T]
    y, dx = torch.zeros_like(f["x"]), torch.zeros_like(f["x"])
    dw, dbias = torch.zeros_like(f["w"]), torch.zeros_like(f["w"][:, 0])
    ends, firsts, lo = [], [], 0
    for n, length in enumerate(lens):
        # one tap after another: what token t sees of the input `back` tokens before it
        seen, run = [], slice(lo, lo + length)
        st = (f["state"][n : n + 1] if case["seqs"] else f["state"]) if with_state else None
        x = f["x"][:, run]
        rows = x.shape[0]
        if st is None:
            st = torch.zeros((rows, K - 1, case["D"]), dtype=torch.float64, device="cuda")
        t = torch.arange(length, device="cuda")
        for j in range(K):
            back = K - 1 - j
            src = t - back
            v = torch.empty_like(x)
            v[:, src >= 0] = x[:, src[src >= 0]]
            v[:, src < 0] = st[:, src[src < 0] + K - 1]
            seen.append(v)
        p = sum(v * f["w"][:, j] for j, v in enumerate(seen))
        p = p if f["bias"] is None else p + f["bias"]
        y[:, run] = _silu64(p) if case["silu"] else p
        both = torch.cat([st, x], 1)
        ends.append(both[:, length:])
        if train:
            dp = f["dy"][:, run] * (_dsilu64(p) if case["silu"] else 1)
            dbias += dp.sum((0, 1))
            dst = torch.zeros_like(st)
            for j, v in enumerate(seen):
                dw[:, j] += (dp * v).sum((0, 1))
                src = t - (K - 1 - j)
                dx[:, lo + src[src >= 0]] += (dp * f["w"][:, j])[:, src >= 0]
                dst.index_add_(1, src[src < 0] + K - 1, (dp * f["w"][:, j])[:, src < 0])
            if f["dstate"] is not None:
                de = f["dstate"][n : n + 1] if case["seqs"] else f["dstate"]
                for i in range(K - 1):  # the i-th input kept is number length + i of both
                    if length + i < K - 1:
                        dst[:, length + i] += de[:, i]
                    else:
                        dx[:, lo + length + i - (K - 1)] += de[:, i]
            firsts.append(dst)
        lo += length
    out = {"y": y}
    if train:
        out |= {"dx": dx, "dw": dw, "dbias": None if f["bias"] is None else dbias}
    if not train or with_state:
        out["state"] = torch.cat(ends)
    if train and with_state:
        out["dstate_in"] = torch.cat(firsts)
    return out


def _compose(a, b, reverse=False):
    """s_t = a_t s_(t-1) + b_t from s = 0, along dim 0, by doubling (reverse: from the end)."""
    if reverse:
        return _compose(a.flip(0), b.flip(0)).flip(0)
    a, b, step = a.clone(), b.clone(), 1
    while step < a.shape[0]:
        b[step:] += a[step:] * b[:-step].clone()
        a[step:] *= a[:-step].clone()
        step *= 2
    return b


def _exact_scan(case, f):
    D, N, G = case["D"], case["N"], case["G"]
    wide = torch.arange(D, device="cuda") // (D // G)
    delta = torch.logaddexp(f["dt"] + f["dt_bias"], torch.zeros((), dtype=torch.float64, device="cuda"))
    if case["op"] == "scan_step":
        at = f["slots"].long()
        pool = f["state"].clone()
        h = pool[at] * (delta[..., None] * f["A"]).exp() + (delta * f["x"])[..., None] * f["B"][:, wide]
        y = (f["C"][:, wide] * h).sum(-1) + f["skip"] * f["x"]
        pool[at] = h
        return {"y": y if f["z"] is None else y * _silu64(f["z"]), "state": pool}
    train, with_state = case["op"] == "scan_train", f["state"] is not None
    zero = lambda x: torch.zeros_like(x)  # noqa: E731
    out = {"y": zero(f["x"])}
    end = torch.zeros((_sets(case), D, N), dtype=torch.float64, device="cuda")
    if train:
        out |= {"dz": None if f["z"] is None else zero(f["x"]), "dx": zero(f["x"]), "ddt": zero(f["x"]),
                "dA": zero(f["A"]), "dB": zero(f["B"]), "dC": zero(f["C"]), "dskip": zero(f["skip"]),
                "dbias": zero(f["skip"])}
        first = zero(end)
    seqs = [(b, b, 0, case["T"]) for b in range(case["B"])]
    if case["seqs"]:
        cu = np.concatenate([[0], np.cumsum(f["lens"])])
        seqs = [(n, 0, int(cu[n]), int(cu[n + 1])) for n in range(case["seqs"])]
    most = max(1, (1 << 28) // max(1, max(hi - lo for _, _, lo, hi in seqs) * N))  # channels at a time
    for n, b, lo, hi in seqs:
        for c in range(0, D, most):
            ch, run = slice(c, min(D, c + most)), (b, slice(lo, hi))
            h0 = f["state"][n, ch] if with_state else torch.zeros_like(f["A"][ch])
            last = f["dstate"][n, ch] if f["dstate"] is not None else torch.zeros_like(h0)
            if hi == lo:
                end[n, ch] = h0
                if train:
                    first[n, ch] = last
                continue
            d, x, w = delta[run][:, ch], f["x"][run][:, ch], wide[ch]
            Bn, Cn = f["B"][run][:, w], f["C"][run][:, w]
            a = (d[..., None] * f["A"][ch]).exp()
            bx = (d * x)[..., None] * Bn
            bx[0] += a[0] * h0
            h = _compose(a, bx)
            end[n, ch] = h[-1]
            y = (h * Cn).sum(-1) + f["skip"][ch] * x
            gate = 1 if f["z"] is None else _silu64(f["z"][run][:, ch])
            out["y"][b, lo:hi, ch] = y * gate
            if not train:
                continue
            dy = f["dy"][run][:, ch]
            if f["z"] is not None:
                out["dz"][b, lo:hi, ch] = dy * y * _dsilu64(f["z"][run][:, ch])
            dy = dy * gate
            g = dy[..., None] * Cn
            g[-1] += last
            g = _compose(torch.cat([torch.zeros_like(a[:1]), a[1:].flip(0)]), g.flip(0)).flip(0)
            first[n, ch] = a[0] * g[0]
            out["dB"][b, lo:hi].index_add_(1, w, g * (d * x)[..., None])
            out["dC"][b, lo:hi].index_add_(1, w, h * dy[..., None])
            du = (g * Bn).sum(-1)
            kept = g * (h - (d * x)[..., None] * Bn)  # g a_t h_(t-1)
            out["dA"][ch] += (kept * d[..., None]).sum(0)
            ddt = (du * x + (kept * f["A"][ch]).sum(-1)) * (1 - torch.exp(-d))  # sigmoid = 1 - e^-softplus
            out["ddt"][b, lo:hi, ch] = ddt
            out["dx"][b, lo:hi, ch] = du * d + f["skip"][ch] * dy
            out["dskip"][ch] += (dy * x).sum(0)
            out["dbias"][ch] += ddt.sum(0)
    if not train or with_state:
        out["state"] = end
    if train and with_state:
        out["dstate_in"] = first
    return out


def _hat64(x):
    return x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()


def _through64(g, x):
    """Gradient of x for the gradient g of _hat64(x)."""
    ms = x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS
    return g / ms.sqrt() - x * ((g * x).sum(-1, keepdim=True) / x.shape[-1]) / ms.pow(1.5)


def _exact_norm(case, f):
    x, one = f["x"], torch.ones(case["d"], dtype=torch.float64, device="cuda")
    sc = one if f["scale"] is None else f["scale"]
    u = x if f["wx"] is None else f["wx"] * _hat64(x)
    r = f["r"] + sc * u
    out = {"n": f["w"] * _hat64(r), "r": r}
    if case["op"] == "norm_fwd":
        return out
    dr = f["dr_out"] + _through64(f["w"] * f["dn"], r)
    out |= {"dr": dr, "dw": (f["dn"] * _hat64(r)).sum((0, 1)), "dwx": None, "dx": sc * dr,
            "dscale": None if f["scale"] is None else (dr * u).sum((0, 1))}
    if f["wx"] is not None:
        out["dwx"] = (sc * dr * _hat64(x)).sum((0, 1))
        out["dx"] = _through64(f["wx"] * sc * dr, x)
    return out


def _exact_gate(case, f):
    x, z, w, dy = f["x"], f["z"], f["w"], f["dy"]
    gate, slope = _silu64(z), _dsilu64(z)
    if case["first"]:
        v = x * gate
        y, dw = w * _hat64(v), dy * _hat64(v)
        dv = _through64(w * dy, v)
        dx, dz = dv * gate, dv * x * slope
    else:
        y, dw = w * _hat64(x) * gate, dy * gate * _hat64(x)
        dx, dz = _through64(w * dy * gate, x), dy * w * _hat64(x) * slope
    return {"y": y, "dx": dx, "dz": dz, "dw": dw.sum((0, 1, 2) if case["shared"] else (0, 1))}
