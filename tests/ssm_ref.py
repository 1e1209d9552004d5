"""The definitions of include/gl_ssm.h token by token and row by row, in 64 bits on
the CPU, differentiable; and what the tests of them share."""
import torch

F64, F32, BF16 = torch.float64, torch.float32, torch.bfloat16


def rel(got, want):
    """Relative 2-norm of the difference (0 where both are empty or zero)."""
    got, want = got.detach().double().cpu(), want.detach().double().cpu()
    assert got.shape == want.shape, (got.shape, want.shape)
    if not want.numel():
        return 0.0
    n = float(want.norm())
    d = float((got - want).norm())
    return d / n if n else d


def par(dtype):
    return F64 if dtype == F64 else F32


def silu(x):
    return x / (1 + torch.exp(-x))


def bounds(T, lens):
    """(state, batch rows, first token, last) of every sequence."""
    if lens is None:
        return [(slice(None), slice(None), 0, T)]
    out, lo = [], 0
    for n, length in enumerate(lens):
        out.append((slice(n, n + 1), slice(0, 1), lo, lo + length))
        lo += length
    return out


def conv(x, w, bias, state, lens, act):
    """(y, last inputs); x [B,T,D], w [D,K], state [n,K-1,D] or None."""
    K, ys, ends = w.shape[1], [], []
    for n, b, lo, hi in bounds(x.shape[1], lens):
        rows = x[b]
        st = state[n] if state is not None else torch.zeros(rows.shape[0], K - 1, x.shape[2], dtype=x.dtype)
        full = torch.cat([st, rows[:, lo:hi]], 1)
        p = sum((full[:, j : j + hi - lo] * w[:, j] for j in range(K)), torch.zeros_like(rows[:, lo:hi]))
        p = p if bias is None else p + bias
        ys.append(silu(p) if act else p)
        ends.append(full[:, full.shape[1] - (K - 1) :])
    return torch.cat(ys, 1), torch.cat(ends)


def scan(x, dt, A, B, C, skip, z, dt_bias, state, lens, softplus):
    """(y, final states); B, C [B,T,G,N], state [n,D,N] or None."""
    D, wide = x.shape[2], torch.arange(x.shape[2]) // (x.shape[2] // B.shape[2])
    d = dt if dt_bias is None else dt + dt_bias
    d = torch.logaddexp(d, torch.zeros((), dtype=d.dtype)) if softplus else d
    ys, ends = [], []
    for n, b, lo, hi in bounds(x.shape[1], lens):
        rows = x[b].shape[0]
        h = state[n] if state is not None else torch.zeros(rows, D, A.shape[1], dtype=x.dtype)
        for t in range(lo, hi):
            dd = d[b][:, t, :, None]
            h = (dd * A).exp() * h + dd * x[b][:, t, :, None] * B[b][:, t][:, wide]
            ys.append((n, b, t, (h * C[b][:, t][:, wide]).sum(-1)))
        ends.append(h)
    y = torch.stack([v for *_, v in ys], 1) if ys else torch.zeros_like(x)
    if skip is not None:
        y = y + skip * x
    return (y if z is None else y * silu(z)), torch.cat(ends)


def hat(x, eps):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt()


def add_norm(x, r, w, wx, scale, eps):
    u = x if wx is None else wx * hat(x, eps)
    r = r + (u if scale is None else scale * u)
    return w * hat(r, eps), r


def gated_norm(x, z, w, eps, first):
    g = 1 if z is None else silu(z)
    y = hat(x * g, eps) if first else hat(x, eps) * g
    return y if w is None else y * w
