"""Plain 64-bit forms of the gated delta rule and of the query / key norms with
rotation, for the tests: token by token from the definitions, differentiable by
torch autograd, on the CPU."""
import torch


def delta(q, k, v, log_alpha, beta, scale, state=None, lens=None):
    """fp64 tensors [B,Hk,T,dk], [B,H,T,dv], [B,H,T] -> (y, final states).
    lens: lengths of packed sequences (B = 1)."""
    B, H, T, dv = v.shape
    r = H // q.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    dk = q.shape[-1]
    n = B if lens is None else len(lens)
    if state is None:
        state = torch.zeros((n, H, dv, dk), dtype=torch.float64)
    bounds, at = [], 0
    for x in ([T] if lens is None else lens):
        bounds.append((at, at + x))
        at += x
    ys, ends = [], []
    for i, (lo, hi) in enumerate(bounds):
        S = state if lens is None else state[i : i + 1]
        for t in range(lo, hi):
            S = log_alpha[:, :, t].exp()[..., None, None] * S
            e = v[:, :, t] - (S * k[:, :, t, None]).sum(-1)
            S = S + (beta[:, :, t, None] * e)[..., None] * k[:, :, t, None]
            ys.append(scale * (S * q[:, :, t, None]).sum(-1))
        ends.append(S)
    y = torch.stack(ys, 2) if ys else v * 0
    return y, torch.cat(ends)


def qknorm(x, w, cos, sin, pos, eps, scale, interleaved=False):
    """x [B,H,T,d], w [d] or None, cos / sin [n, rot/2] or None, pos [B,T]."""
    y = scale * x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        y = y * w
    if cos is None or cos.shape[1] == 0:
        return y
    half = cos.shape[1]
    p = pos.clamp(0, cos.shape[0] - 1)
    c, s = cos[p][:, None], sin[p][:, None]
    turned, rest = y[..., : 2 * half], y[..., 2 * half :]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else turned.chunk(2, -1)
    a, b = a * c - b * s, a * s + b * c
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, rest], -1)


def rel(got, want):
    """2-norm of the difference over that of the reference."""
    got, want = got.detach().double().cpu(), want.detach()
    n = want.norm()
    return float((got - want).norm() / n) if n > 0 else float(got.norm())


def unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt()


def inputs(seed, B, H, Hk, T, dk, dv, dtype, gate=None, n=None, decay="mix"):
    """Rounded inputs as fp64 tensors (exact upcasts): dict of q, k, v,
    log_alpha, beta, dy, state, dstate."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    gate = gate or dtype
    z = rnd(B, H, T)
    if decay == "mix":
        z = torch.where(torch.rand((B, H, T), generator=g) < 0.5, 6 + 0.7 * z, z)
    elif decay == "near1":
        z = 5 + 0.7 * z
    x = {"q": unit(rnd(B, Hk, T, dk)), "k": unit(rnd(B, Hk, T, dk)), "v": rnd(B, H, T, dv), "dy": rnd(B, H, T, dv)}
    x = {a: b.to(dtype).double() for a, b in x.items()}
    x["log_alpha"] = torch.nn.functional.logsigmoid(z).to(gate).double()
    x["beta"] = torch.rand((B, H, T), generator=g, dtype=torch.float64).to(gate).double()
    n = B if n is None else n
    st = torch.float64 if dtype == torch.float64 else torch.float32
    x["state"], x["dstate"] = (0.3 * rnd(n, H, dv, dk)).to(st).double(), (0.3 * rnd(n, H, dv, dk)).to(st).double()
    return x
