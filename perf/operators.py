"""The gated delta rule (chunked and recurrent) and the norms of queries and keys
with the position rotation, as cases that can be timed and compared.

`run` takes a prepared state through ONE pass of an operator: in its plain form
(elementary torch operations in 32 bits, rounded once at the end) where `own` is
false, through the public calls of weight_scans_amd where it is true.  `exact`
gives the same outputs from the operators' definitions, token by token, in 64
bits.

Gated delta rule, per sequence and value head (S is dv x dk, S_0 given or zero):

    e_t = v_t - a_t S_{t-1} k_t,           a_t = exp(log_alpha_t)
    S_t = a_t S_{t-1} + beta_t e_t k_t^T,  y_t = scale S_t q_t

Norm and rotation, per token and head (weight w, pairs (i, i + rot/2) or
(2i, 2i + 1) of the first rot columns turned by the position's angles):

    y = s Rot_pos(w * x / sqrt(mean(x^2) + eps))
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

C = 64  # tokens a chunk of the plain form
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def _delta(name, op, B, H, Hk, T, dk, dv, dtype, layout="bhtd", seqs=0, state=False, decay="base"):
    return {"name": name, "op": op, "B": B, "H": H, "Hk": Hk, "T": T, "dk": dk, "dv": dv,
            "dtype": dtype, "layout": layout, "seqs": seqs, "state": state, "decay": decay}


def _qk(name, op, B, T, Hq, Hk, d, rot, dtype, layout="bthd", pairs="half"):
    return {"name": name, "op": op, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "d": d, "rot": rot,
            "dtype": dtype, "layout": layout, "pairs": pairs}


def listed():
    return [
        # one user's next token: 16 states of 64 KB, a call that is all latency
        _delta("step_one", "step", 1, 16, 16, 1, 128, 128, "bf16"),
        # a full serving batch out of a pool of states in another order
        _delta("step_many", "step", 256, 16, 8, 1, 128, 128, "bf16"),
        # a prefill of a few short prompts packed one after another (one of no token and one of
        # one among them) that continue from cached states
        _delta("prefill_packed", "fwd", 1, 16, 8, 777, 128, 128, "bf16", "bthd", 5, True),
        # one long document: few heads, 512 chunks, abrupt forgetting
        _delta("prefill_long", "fwd", 1, 16, 16, 32768, 128, 128, "bf16", "bhtd", 0, True, "mix"),
        # fp32 throughout
        _delta("prefill_f32", "fwd", 4, 8, 8, 1024, 64, 64, "f32", "bhtd", 0, True),
        # heads of other sizes, three keys' heads for six values' heads, an odd length
        _delta("prefill_odd", "fwd", 2, 6, 3, 1023, 96, 80, "bf16", "bthd", 0, True, "near1"),
        # training, forward and backward, at the two layer shapes of the scans' workloads
        _delta("train_64", "train", 8, 16, 16, 4096, 64, 64, "bf16"),
        _delta("train_128", "train", 4, 16, 16, 4096, 128, 128, "bf16", "bthd", 0, False, "near1"),
        # training on packed sequences with shared key heads and gradients of the first states
        _delta("train_packed", "train", 1, 8, 4, 3001, 64, 64, "bf16", "bthd", 7, True),
        # the norms and the rotation of one decoding step
        _qk("qk_decode", "qk_fwd", 64, 1, 16, 8, 128, 128, "bf16"),
        # the norms and the rotation, forward and backward, of a training step
        _qk("qk_train", "qk_train", 4, 4096, 16, 8, 128, 128, "bf16"),
        # fp32, part of an odd head turned, neighbouring pairs, an odd length
        _qk("qk_odd", "qk_train", 3, 1021, 6, 2, 80, 32, "f32", "bhtd", "next"),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "fwd", "fwd", "train", "train", "qk_fwd", "qk_train"])
    if op.startswith("qk"):
        d = rng.choice([64, 128, 128, rng.randrange(32, 130, 2)])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4])
        while True:
            B, T = _logint(rng, 1, 64), _logint(rng, 1, 8192)
            if B * T * (Hq + Hk) * d <= 4 * 4096 * 24 * 128:
                break
        return {"op": op, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "d": d,
                "rot": rng.choice([d, d, d // 4 * 2]),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "layout": rng.choice(["bthd", "bhtd"]),
                "pairs": rng.choice(["half", "half", "next"])}
    Hk = rng.choice([1, 2, 4, 8, 16])
    H = Hk * rng.choice([1, 1, 2, 3])
    dk = rng.choice([64, 128, 128, rng.randrange(16, 129, 8)])
    dv = rng.choice([dk, dk, 64, 128, rng.randrange(16, 129, 8)])
    dtype, seqs, T = "bf16", 0, 1
    if op == "step":
        B = _logint(rng, 1, 256)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if B * H * dk * dv > 256 * 16 * 128 * 128:
            B = 64
    else:
        if rng.random() < 0.2:
            dtype = "f32"
        most = 4 * 8 * 1024 * 64 * 64 if dtype == "f32" else 4 * 16 * 4096 * 128 * 128
        while True:
            B, T = _logint(rng, 1, 8), _logint(rng, 1, 32768)
            if B * T * H * dk * dv <= most and (op == "fwd" or T <= 8192):
                break
        if rng.random() < 0.3:
            B, seqs = 1, rng.randrange(2, 12)
    return {"op": op, "B": B, "H": H, "Hk": Hk, "T": T, "dk": dk, "dv": dv, "dtype": dtype,
            "layout": rng.choice(["bthd", "bhtd"]), "seqs": seqs, "state": bool(rng.random() < 0.6),
            "decay": rng.choice(["base", "near1", "mix"])}


def _size(case):
    return {"bf16": 2, "f32": 4}[case["dtype"]]


def _sets(case):
    return case["seqs"] or case["B"]


def work(case):
    e = _size(case)
    if case["op"].startswith("qk"):
        n = case["B"] * case["T"] * (case["Hq"] + case["Hk"]) * case["d"]
        table = case["B"] * case["T"] * case["rot"] * 4 + case["B"] * case["T"] * 4
        if case["op"] == "qk_fwd":
            return {"bytes": 2 * n * e + table, "flops": 8 * n}
        return {"bytes": 5 * n * e + table, "flops": 24 * n}
    H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
    tok = case["B"] * case["T"]
    q, v, s = tok * Hk * dk * e, tok * H * dv * e, H * dk * dv * 4
    gates = 2 * tok * H * e
    if case["op"] == "step":
        return {"bytes": 2 * q + 2 * v + gates + 2 * case["B"] * s, "flops": 6 * tok * H * dk * dv}
    states = (2 if case["state"] else 1) * _sets(case) * s
    if case["op"] == "fwd":
        return {"bytes": 2 * q + 2 * v + gates + states, "flops": 6 * tok * H * dk * dv}
    states = (2 * _sets(case) * s) if case["state"] else 0
    return {"bytes": 4 * q + 4 * v + 2 * gates + states, "flops": 22 * tok * H * dk * dv}


# ------------------------------------------------------------------ the inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lengths(case, seed):
    """Lengths of the packed sequences: log-uniform shares of T, one empty, one of one token."""
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


def _heads(case, g, T, H, d, dtype, unit):
    """[B, H, T, d]: rows of unit length, as after a norm, or of N(0, 1).  "bthd": a view of
    [B, T, H, d], as a projection writes it."""
    B = case["B"]
    x = torch.randn((B, T, H, d) if case["layout"] == "bthd" else (B, H, T, d), generator=g, device="cuda")
    if unit:
        x = x / x.square().sum(-1, keepdim=True).sqrt()
    x = x.to(dtype)
    return x.transpose(1, 2) if case["layout"] == "bthd" else x


def _gate(case, g, dtype):
    """log_alpha and beta [B, H, T]."""
    B, H, T = case["B"], case["H"], case["T"]
    z = torch.randn((B, H, T), generator=g, device="cuda")
    if case["decay"] == "base":
        z = 3 + z
    elif case["decay"] == "near1":
        z = 5 + math.sqrt(0.5) * z
    else:
        coin = torch.rand((B, H, T), generator=g, device="cuda") < 0.5
        z = torch.where(coin, 6 + math.sqrt(0.5) * z, z)
    beta = torch.rand((B, H, T), generator=g, device="cuda")
    return (-torch.log1p(torch.exp(-z))).to(dtype), beta.to(dtype)


def prepare(case, seed):
    g, t = _gen(seed), _TYPES[case["dtype"]]
    if case["op"].startswith("qk"):
        return _prepare_qk(case, g, t)
    H, Hk, dk, dv, T, B = case["H"], case["Hk"], case["dk"], case["dv"], case["T"], case["B"]
    s = {"case": case, "scale": dk ** -0.5}
    s["q"] = _heads(case, g, T, Hk, dk, t, True)
    s["k"] = _heads(case, g, T, Hk, dk, t, True)
    s["v"] = _heads(case, g, T, H, dv, t, False)
    s["log_alpha"], s["beta"] = _gate(case, g, t)
    s["state"] = s["cu"] = s["lens"] = None
    if case["op"] == "step":
        n = B + B // 4  # the pool has a few more states than the batch takes
        s["state"] = 0.3 * torch.randn((n, H, dv, dk), generator=g, device="cuda")
        s["slots"] = torch.randperm(n, generator=g, device="cuda")[:B].to(torch.int32)
        for x in ("q", "k", "v", "log_alpha", "beta"):
            s[x] = s[x][:, :, 0].contiguous()
        return s
    if case["seqs"]:
        s["lens"] = _lengths(case, seed)
        s["cu"] = torch.tensor([0] + list(np.cumsum(s["lens"])), dtype=torch.int32, device="cuda")
    if case["state"]:
        s["state"] = 0.3 * torch.randn((_sets(case), H, dv, dk), generator=g, device="cuda")
    if case["op"] == "train":
        s["dy"] = _heads(case, g, T, H, dv, t, False)
        if case["state"]:
            s["dstate"] = 0.3 * torch.randn((_sets(case), H, dv, dk), generator=g, device="cuda")
    return s


def _prepare_qk(case, g, t):
    B, T, Hq, Hk, d, rot = case["B"], case["T"], case["Hq"], case["Hk"], case["d"], case["rot"]
    if case["layout"] == "bthd":  # slices of a fused projection's output (values behind them)
        buf = torch.randn((B, T, (Hq + 2 * Hk) * d), generator=g, device="cuda").to(t)
        q = buf[..., : Hq * d].view(B, T, Hq, d).transpose(1, 2)
        k = buf[..., Hq * d : (Hq + Hk) * d].view(B, T, Hk, d).transpose(1, 2)
    else:
        q = torch.randn((B, Hq, T, d), generator=g, device="cuda").to(t)
        k = torch.randn((B, Hk, T, d), generator=g, device="cuda").to(t)
    n = max(T, 4096) + 64
    angle = torch.arange(n, device="cuda", dtype=torch.float64)[:, None]
    angle = angle * 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) / max(1, rot // 2))
    s = {"case": case, "q": q, "k": k, "cos": angle.cos().float(), "sin": angle.sin().float(),
         "q_scale": d ** -0.5, "k_scale": d ** -0.5}
    s["wq"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(t)
    s["wk"] = (1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(t)
    first = torch.randint(0, n - T + 1, (B, 1), generator=g, device="cuda")
    s["pos"] = (first + torch.arange(T, device="cuda")).to(torch.int32)
    if case["op"] == "qk_train":
        s["dqn"] = torch.randn((B, Hq, T, d), generator=g, device="cuda").to(t)
        s["dkn"] = torch.randn((B, Hk, T, d), generator=g, device="cuda").to(t)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _OWN[op](s)
    return _PLAIN[op](s)


def _own_step(s):
    import weight_scans_amd as ws
    y = ws.gl_delta_step(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["state"],
                         scale=s["scale"], slots=s["slots"])
    return {"y": y, "state": s["state"]}


def _own_fwd(s):
    import weight_scans_amd as ws
    y, state, _ = ws.gl_delta_fwd(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], scale=s["scale"],
                                  state=s["state"], want_state=True, cu_seqlens=s["cu"])
    return {"y": y, "state": state}


def _own_train(s):
    import weight_scans_amd as ws
    with_state = s["state"] is not None
    y, state, saved = ws.gl_delta_fwd(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], scale=s["scale"],
                                      state=s["state"], want_state=with_state, save=True, cu_seqlens=s["cu"])
    dq, dk, dv, dla, db, ds = ws.gl_delta_bwd(
        s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["dy"], saved, scale=s["scale"],
        state=s["state"], dstate=s.get("dstate"), cu_seqlens=s["cu"])
    out = {"y": y, "dq": dq, "dk": dk, "dv": dv, "dlog_alpha": dla, "dbeta": db}
    if with_state:
        out |= {"state": state, "dstate_in": ds}
    return out


def _own_qk_fwd(s):
    import weight_scans_amd as ws
    qn, kn = ws.gl_qknorm_rope_fwd(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], pos=s["pos"], eps=EPS,
                                   q_scale=s["q_scale"], k_scale=s["k_scale"],
                                   interleaved=s["case"]["pairs"] == "next")
    return {"q": qn, "k": kn}


def _own_qk_train(s):
    import weight_scans_amd as ws
    out = _own_qk_fwd(s)
    dq, dk, dwq, dwk = ws.gl_qknorm_rope_bwd(
        s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["dqn"], s["dkn"], pos=s["pos"], eps=EPS,
        q_scale=s["q_scale"], k_scale=s["k_scale"], interleaved=s["case"]["pairs"] == "next")
    return out | {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


# ------------------------------------------------------------------ the plain form: the gated delta rule
def _plain_step(s):
    case = s["case"]
    r = case["H"] // case["Hk"]
    q, k = (s[n].float().repeat_interleave(r, 1) for n in ("q", "k"))
    at = s["slots"].long()
    S = s["state"][at] * s["log_alpha"].float().exp()[..., None, None]
    e = s["v"].float() - (S * k[:, :, None]).sum(-1)
    S = S + (s["beta"].float()[..., None] * e)[..., None] * k[:, :, None]
    y = (S * q[:, :, None]).sum(-1) * s["scale"]
    s["state"][at] = S
    return {"y": y.to(s["v"].dtype), "state": s["state"]}


class _Ragged:
    """Sequences side by side, padded to a whole number of chunks, and back."""

    def __init__(self, s):
        T = s["case"]["T"]
        self.lens = s["lens"]
        longest = T if self.lens is None else max(max(self.lens), 1)
        self.NC = -(-longest // C)
        L = self.NC * C
        self.T, self.L = T, L
        if self.lens is not None:
            cu = s["cu"].long()
            t = torch.arange(L, device="cuda")
            self.there = t[None] < (cu[1:] - cu[:-1])[:, None]
            self.at = torch.where(self.there, cu[:-1, None] + t[None], 0)

    def out(self, x):
        """[B, H, T, ...] -> fp32 [N, H, NC, C, ...], zero where no token is."""
        x = x.float()
        if self.lens is None:
            pad = torch.zeros((*x.shape[:2], self.L - self.T, *x.shape[3:]), device=x.device)
            x = torch.cat([x, pad], 2)
        else:
            x = x[0].transpose(0, 1)[self.at]  # [N, L, H, ...]
            x = x * self.there.view(*self.there.shape, *[1] * (x.dim() - 2))
            x = x.transpose(1, 2)
        return x.reshape(*x.shape[:2], self.NC, C, *x.shape[3:]).contiguous()

    def back(self, x):
        """[N, H, NC, C, ...] -> [B, H, T, ...]"""
        x = x.reshape(*x.shape[:2], self.L, *x.shape[4:])
        if self.lens is None:
            return x[:, :, : self.T]
        return x.transpose(1, 2)[self.there].transpose(0, 1)[None]


def _mT(x):
    return x.transpose(-1, -2).contiguous()


def _chunks(s):
    """What the chunks are in themselves: I + A with A strictly lower triangular has the
    inverse (I - A)(I + A^2)(I + A^4) ... (I + A^32), A^64 being zero."""
    case = s["case"]
    r = case["H"] // case["Hk"]
    g = _Ragged(s)
    q, k, v = g.out(s["q"]).repeat_interleave(r, 1) * s["scale"], g.out(s["k"]).repeat_interleave(r, 1), g.out(s["v"])
    la, be = g.out(s["log_alpha"]), g.out(s["beta"])
    l = la.cumsum(-1)
    low = torch.ones((C, C), dtype=torch.bool, device="cuda").tril()
    D = torch.where(low, l[..., :, None] - l[..., None, :], -torch.inf).exp()
    kT = _mT(k)
    L = (D * (k @ kT)).tril(-1)
    P = D * (q @ kT)
    A = be[..., None] * L
    eye = torch.eye(C, device="cuda")
    A2 = A @ A
    A4 = A2 @ A2
    A8 = A4 @ A4
    A16 = A8 @ A8
    A32 = A16 @ A16
    inv = (eye - A) @ (eye + A2) @ (eye + A4) @ (eye + A8) @ (eye + A16) @ (eye + A32)
    gam, last = l.exp()[..., None], l[..., -1:]
    rest = (last - l).exp()[..., None]
    return g, q, k, v, be, l, L, P, inv, gam, rest, last.exp()[..., None]


def _plain_states(s, ch):
    g, q, k, v, be, l, L, P, inv, gam, rest, whole = ch
    U0, W = inv @ (be[..., None] * v), inv @ (be[..., None] * gam * k)
    N, H = k.shape[:2]
    dv, dk = s["case"]["dv"], s["case"]["dk"]
    S = s["state"] if s["state"] is not None else torch.zeros((N, H, dv, dk), device="cuda")
    # (NC is the number of chunks of the longest sequence: the recurrence itself)
    states, Us = [], []
    kr = rest * k
    for c in range(g.NC):
        states.append(S)
        U = U0[:, :, c] - W[:, :, c] @ _mT(S)
        S = whole[:, :, c] * S + _mT(U) @ kr[:, :, c]
        Us.append(U)
    return torch.stack(states, 2), torch.stack(Us, 2), S


def _plain_out(s, ch, states, U):
    g, q, P, gam = ch[0], ch[1], ch[7], ch[9]
    return g.back((gam * q) @ _mT(states) + P @ U).to(s["v"].dtype)


def _plain_fwd(s):
    ch = _chunks(s)
    states, U, S = _plain_states(s, ch)
    return {"y": _plain_out(s, ch, states, U), "state": S}


def _plain_train(s):
    case, t = s["case"], s["v"].dtype
    ch = _chunks(s)
    states, U, S_T = _plain_states(s, ch)
    g, q, k, v, be, l, L, P, inv, gam, rest, whole = ch
    y = _plain_out(s, ch, states, U)
    do = g.out(s["dy"])
    PTdo, invT = _mT(P) @ do, _mT(inv)
    gq, gk, kr = gam * q, gam * k, rest * k
    lam = s["dstate"] if case["state"] else torch.zeros_like(S_T)
    lams, Gs = [None] * g.NC, [None] * g.NC
    for c in range(g.NC - 1, -1, -1):
        lams[c] = lam
        dU = PTdo[:, :, c] + kr[:, :, c] @ _mT(lam)
        Gs[c] = invT[:, :, c] @ dU
        F = be[:, :, c, :, None] * Gs[c]
        lam = whole[:, :, c] * lam + _mT(do[:, :, c]) @ gq[:, :, c] - _mT(F) @ gk[:, :, c]
    Lam, G = torch.stack(lams, 2), torch.stack(Gs, 2)
    F = be[..., None] * G
    E = v - gk @ _mT(states) - L @ U
    low = torch.ones((C, C), dtype=torch.bool, device="cuda").tril()
    D = torch.where(low, l[..., :, None] - l[..., None, :], -torch.inf).exp()
    dP = D * (do @ _mT(U))
    dL = (D * (F @ _mT(U))).tril(-1)
    dq = gam * (do @ states) + dP @ k
    dk = _mT(dP) @ q + rest * (U @ Lam) - gam * (F @ states) - dL @ k - _mT(dL) @ k
    db = (G * E).sum(-1)
    # dL/dlog(alpha_t) = <dL/dS_t-1, S_t-1>, carried back from the chunk's end
    z = (q * dq).sum(-1) - (v * F).sum(-1)
    nxt = torch.cat([states[:, :, 1:], S_T[:, :, None]], 2)
    z = z.flip(-1).cumsum(-1).flip(-1) + (Lam * nxt).sum((-1, -2))[..., None]
    r = case["H"] // case["Hk"]
    shared = lambda x: x.view(x.shape[0], -1, r, *x.shape[2:]).sum(2)  # noqa: E731
    out = {"y": y, "dq": g.back(shared(dq) * s["scale"]).to(t), "dk": g.back(shared(dk)).to(t),
           "dv": g.back(F).to(t), "dlog_alpha": g.back(z).to(t), "dbeta": g.back(db).to(t)}
    if case["state"]:
        out |= {"state": S_T, "dstate_in": lam}
    return out


# ------------------------------------------------------------------ the plain form: norms and rotation
def _turn(x, cos, sin, rot, pairs, back=False):
    if back:
        sin = -sin
    a, b = (x[..., : rot // 2], x[..., rot // 2 : rot]) if pairs == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    u, w = a * cos - b * sin, b * cos + a * sin
    u = torch.cat([u, w], -1) if pairs == "half" else torch.stack([u, w], -1).flatten(-2)
    return torch.cat([u, x[..., rot:]], -1)


def _table(s):
    at = s["pos"].long()
    return s["cos"][at][:, None], s["sin"][at][:, None]


def _plain_qk_one(s, x, w, scale):
    x = x.float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    y = _turn(x * r * w.float() * scale, *_table(s), s["case"]["rot"], s["case"]["pairs"])
    return y.to(w.dtype)


def _plain_qk_fwd(s):
    return {"q": _plain_qk_one(s, s["q"], s["wq"], s["q_scale"]), "k": _plain_qk_one(s, s["k"], s["wk"], s["k_scale"])}


def _plain_qk_grad(s, x, w, scale, dy):
    x = x.float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = x * r
    dz = _turn(dy.float(), *_table(s), s["case"]["rot"], s["case"]["pairs"], True) * scale
    dw = (dz * n).sum(2).sum((0, 1))  # in steps: a long sum of 32 bits keeps its last places so
    dn = dz * w.float()
    return (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(w.dtype), dw


def _plain_qk_train(s):
    out = _plain_qk_fwd(s)
    dq, dwq = _plain_qk_grad(s, s["q"], s["wq"], s["q_scale"], s["dqn"])
    dk, dwk = _plain_qk_grad(s, s["k"], s["wk"], s["k_scale"], s["dkn"])
    return out | {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


_OWN = {"step": _own_step, "fwd": _own_fwd, "train": _own_train, "qk_fwd": _own_qk_fwd, "qk_train": _own_qk_train}
_PLAIN = {"step": _plain_step, "fwd": _plain_fwd, "train": _plain_train, "qk_fwd": _plain_qk_fwd,
          "qk_train": _plain_qk_train}


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f = {n: (x.double() if torch.is_tensor(x) and x.is_floating_point() else x) for n, x in s.items()}
    if case["op"].startswith("qk"):
        return _exact_qk(case, f)
    r = case["H"] // case["Hk"]
    if case["op"] == "step":
        pool = f["state"].clone()
        at = s["slots"].long()
        q, k = f["q"].repeat_interleave(r, 1), f["k"].repeat_interleave(r, 1)
        y, S = _token(pool[at], q, k, f["v"], f["log_alpha"].exp(), f["beta"])[:2]
        pool[at] = S
        return {"y": y * s["scale"], "state": pool}
    bounds = [(0, case["T"])]
    if case["seqs"]:
        cu = [0] + list(np.cumsum(s["lens"]))
        bounds = list(zip(cu[:-1], cu[1:]))
    q, k = f["q"].repeat_interleave(r, 1), f["k"].repeat_interleave(r, 1)
    a = f["log_alpha"].exp()
    train = case["op"] == "train"
    y = torch.zeros(f["v"].shape, dtype=torch.float64, device="cuda")
    out = {"y": y}
    if train:
        out |= {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(y),
                "dlog_alpha": torch.zeros_like(a), "dbeta": torch.zeros_like(a)}
    ends, firsts = [], []
    for n, (lo, hi) in enumerate(bounds):
        rows = slice(n, n + 1) if case["seqs"] else slice(None)
        N, H, dv, dk = (1 if case["seqs"] else case["B"]), case["H"], case["dv"], case["dk"]
        S = f["state"][rows] if case["state"] else torch.zeros((N, H, dv, dk), dtype=torch.float64, device="cuda")
        before = []
        for t in range(lo, hi):
            if train:
                before.append(S)
            yt, S, _ = _token(S, q[:, :, t], k[:, :, t], f["v"][:, :, t], a[:, :, t], f["beta"][:, :, t])
            y[:, :, t] = yt * s["scale"]
        ends.append(S)
        if train:
            lam = f["dstate"][rows] if case["state"] else torch.zeros_like(S)
            for t in range(hi - 1, lo - 1, -1):
                lam = _token_back(out, t, lam, before.pop(), q, k, f["v"], a, f["beta"], f["dy"], s["scale"])
            firsts.append(lam)
    if train:
        for n in ("dq", "dk"):
            x = out[n]
            out[n] = x.view(x.shape[0], -1, r, *x.shape[2:]).sum(2)
    if case["op"] == "fwd" or case["state"]:
        out["state"] = torch.cat(ends)
    if train and case["state"]:
        out["dstate_in"] = torch.cat(firsts)
    return out


def _token(S, q, k, v, a, b):
    S = a[..., None, None] * S
    e = v - (S @ k[..., None])[..., 0]
    S = S + (b[..., None] * e)[..., None] * k[..., None, :]
    return (S @ q[..., None])[..., 0], S, e


def _token_back(out, t, lam, S0, q, k, v, a, b, dy, scale):
    """One token of the adjoint: lam = dL/dS_t (later reads only) -> dL/dS_t-1."""
    qt, kt, vt, at, bt = q[:, :, t], k[:, :, t], v[:, :, t], a[:, :, t], b[:, :, t]
    _, S1, e = _token(S0, qt, kt, vt, at, bt)
    g = dy[:, :, t] * scale
    lam = lam + g[..., None] * qt[..., None, :]
    du = (lam @ kt[..., None])[..., 0]
    fe = bt[..., None] * du
    u = bt[..., None] * e
    into = lam - fe[..., None] * kt[..., None, :]
    out["dq"][:, :, t] = (g[..., None, :] @ S1)[..., 0, :]
    out["dk"][:, :, t] = (u[..., None, :] @ lam)[..., 0, :] - at[..., None] * (fe[..., None, :] @ S0)[..., 0, :]
    out["dv"][:, :, t] = fe
    out["dbeta"][:, :, t] = (du * e).sum(-1)
    out["dlog_alpha"][:, :, t] = at * (into * S0).sum((-1, -2))
    return at[..., None, None] * into


def _exact_qk(case, f):
    d, rot, half = case["d"], case["rot"], case["rot"] // 2
    first = torch.arange(half, device="cuda") * (1 if case["pairs"] == "half" else 2)
    second = first + (half if case["pairs"] == "half" else 1)
    at = f["pos"].long()
    cos, sin = f["cos"][at][:, None], f["sin"][at][:, None]
    out = {}
    for n in ("q", "k"):
        x, w, sc = f[n], f["w" + n], f[n + "_scale"]
        rms = (x.square().sum(-1, keepdim=True) / d + EPS).sqrt()
        z = sc * w * x / rms
        y = z.clone()
        y[..., first] = cos * z[..., first] - sin * z[..., second]
        y[..., second] = sin * z[..., first] + cos * z[..., second]
        out[n] = y
        if case["op"] == "qk_train":
            dy = f["d%sn" % n]
            dz = dy.clone()
            dz[..., first] = cos * dy[..., first] + sin * dy[..., second]
            dz[..., second] = cos * dy[..., second] - sin * dy[..., first]
            out["dw" + n] = (sc * dz * x / rms).sum((0, 1, 2))
            h = sc * w * dz
            out["d" + n] = h / rms - x * (h * x).sum(-1, keepdim=True) / (d * rms ** 3)
    return out
