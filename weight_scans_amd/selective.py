"""A layer of the selective state space scan, and a small command that trains and
serves one.

The layer shows the operators of ``ssm.py`` together as a model uses them:

    add_norm:        the residual takes the block before, and is normed for this one
    projection    -> x and the gate z (views of one [B,T,...] tensor)
    causal_conv:     x over its last few tokens, SiLU
    projections   -> steps dt, B and C (views of one tensor)
    selective_scan:  y and the state after the last token (training, prefill)
    gated_norm:      y's norm, gated by z (or the scan gates it: gate="scan")
    gl_conv_step, gl_ssm_step on pools of states (decoding, any rows of the batch)

    python -m weight_scans_amd.selective [--steps N] [--tokens N]

learns to repeat the token that stood some tokens before (the scan has to carry it),
then prefills prompts of different lengths packed one after another and decodes from
their states, and checks the decoded outputs against whole passes.
"""
from __future__ import annotations

import argparse
import math

import torch

from .ssm import add_norm, causal_conv, gated_norm, gl_conv_step, gl_ssm_step, selective_scan


class Selective(torch.nn.Module):
    """x [B,T,width] -> y [B,T,width] with `inner` channels of `states` states each, a
    convolution of `taps` tokens, and steps from `rank` columns.  gate: "norm" (the
    gated norm, over groups of inner / groups channels) or "scan" (the scan's own)."""

    def __init__(self, width, inner=None, states=16, taps=4, rank=None, groups=1, gate="norm", device="cuda",
                 dtype=torch.bfloat16):
        super().__init__()
        if gate not in ("norm", "scan"):
            raise ValueError('gate must be "norm" or "scan"')
        self.inner, self.states, self.groups, self.gate = inner or 2 * width, states, groups, gate
        self.rank = rank or max(1, width // 16)
        make = dict(device=device, dtype=dtype, bias=False)
        par = torch.float64 if dtype == torch.float64 else torch.float32
        self.xz = torch.nn.Linear(width, 2 * self.inner, **make)
        self.dbc = torch.nn.Linear(self.inner, self.rank + 2 * states, **make)
        self.dt = torch.nn.Linear(self.rank, self.inner, **make)
        self.out = torch.nn.Linear(self.inner, width, **make)
        self.taps = torch.nn.Parameter(torch.randn(self.inner, taps, device=device).mul(taps ** -0.5).to(dtype))
        self.taps_bias = torch.nn.Parameter(torch.zeros(self.inner, device=device, dtype=dtype))
        # decays -1 .. -states, steps between 0.001 and 0.1
        self.log_a = torch.nn.Parameter(torch.arange(1, states + 1, device=device, dtype=par).log().repeat(self.inner, 1))
        step = torch.exp(torch.rand(self.inner, device=device, dtype=par) * math.log(100.0) + math.log(1e-3))
        self.dt_bias = torch.nn.Parameter(step + torch.log(-torch.expm1(-step)))
        self.skip = torch.nn.Parameter(torch.ones(self.inner, device=device, dtype=par))
        self.norm = torch.nn.Parameter(torch.ones(groups, self.inner // groups, device=device, dtype=dtype))

    def pools(self, n):
        """Zero states of n sequences: the convolution's last inputs and the scan's."""
        at = dict(device=self.taps.device)
        return (torch.zeros(n, self.taps.shape[1] - 1, self.inner, dtype=self.taps.dtype, **at),
                torch.zeros(n, self.inner, self.states, dtype=self.skip.dtype, **at))

    def _scan_inputs(self, x):
        """dt [..,inner], A, B and C [..,states] (views) of the convolved x."""
        d, b, c = self.dbc(x).split([self.rank, self.states, self.states], -1)
        return self.dt(d), -self.log_a.exp(), b, c

    def _close(self, y, z):
        if self.gate == "norm":
            split = lambda t: t.unflatten(-1, (self.groups, -1))  # noqa: E731
            y = gated_norm(split(y), split(z), self.norm).flatten(-2)
        return self.out(y)

    def forward(self, x, states=None, cu_seqlens=None, want_state=False):
        """The layer over whole sequences (training, prefill); packed prompts: B = 1 and
        cu_seqlens.  Returns (y, the states after the last tokens: a pair, or None)."""
        x, z = self.xz(x).split(self.inner, -1)
        conv, scan = states or (None, None)
        x, conv = causal_conv(x, self.taps, self.taps_bias, state=conv, cu_seqlens=cu_seqlens, want_state=want_state)
        y, scan = selective_scan(x, *self._scan_inputs(x), self.skip, z if self.gate == "scan" else None, self.dt_bias,
                                 state=scan, cu_seqlens=cu_seqlens, want_state=want_state)
        return self._close(y, z), (conv, scan) if want_state else None

    @torch.no_grad()
    def step(self, x, pools, slots=None):
        """One token of each row, x [B,width]: updates the pools in place, row b's at
        slots[b] (or at b)."""
        x, z = self.xz(x).split(self.inner, -1)
        x = gl_conv_step(x, self.taps, self.taps_bias, pools[0], slots=slots)
        dt, a, b, c = self._scan_inputs(x)
        y = gl_ssm_step(x, dt, a, b, c, self.skip, z if self.gate == "scan" else None, self.dt_bias, pools[1], slots=slots)
        return self._close(y[:, None], z[:, None])[:, 0]


class SelectiveModel(torch.nn.Module):
    """Embedding, blocks on a residual path in fp32 (fp64), logits over the tokens."""

    def __init__(self, tokens, width, layers=2, **layer):
        super().__init__()
        at = dict(device=layer.get("device", "cuda"), dtype=layer.get("dtype", torch.bfloat16))
        self.residual = torch.float64 if at["dtype"] == torch.float64 else torch.float32
        self.embed = torch.nn.Embedding(tokens, width, **at)
        self.layers = torch.nn.ModuleList(Selective(width, **layer) for _ in range(layers))
        self.norms = torch.nn.ParameterList(torch.ones(width, **at) for _ in range(layers + 1))
        self.scales = torch.nn.ParameterList(torch.ones(width, **at) for _ in range(layers))
        self.head = torch.nn.Linear(width, tokens, bias=False, **at)

    def pools(self, n):
        return [layer.pools(n) for layer in self.layers]

    def _through(self, ids, block):
        """Logits: block(i, normed input) is the i-th layer."""
        x = self.embed(ids)
        r = torch.zeros(x.shape, dtype=self.residual, device=x.device)
        n, r = add_norm(x, r, self.norms[0])
        for i, scale in enumerate(self.scales):
            n, r = add_norm(block(i, n), r, self.norms[i + 1], None, scale)
        return self.head(n)

    def forward(self, ids, states=None, cu_seqlens=None, want_state=False):
        ends = []

        def block(i, n):
            y, end = self.layers[i](n, None if states is None else states[i], cu_seqlens, want_state)
            ends.append(end)
            return y
        return self._through(ids, block), ends

    @torch.no_grad()
    def step(self, ids, pools, slots=None):
        return self._through(ids[:, None], lambda i, n: self.layers[i].step(n[:, 0], pools[i], slots)[:, None])[:, 0]


def train(model, steps, vocab, batch=32, length=64, back=8, lr=3e-3, seed=0, say=print):
    """Mean loss of the answers at the first and the last steps; the answer at a token
    is the one that stood `back` tokens before it."""
    rng = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=lr, weight_decay=0.0)
    losses = []
    for i in range(steps):
        ids = torch.randint(0, vocab, (batch, length), generator=rng).cuda()
        logits, _ = model(ids)
        loss = torch.nn.functional.cross_entropy(logits[:, back:].flatten(0, 1).float(), ids[:, :-back].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if i % 50 == 0 or i == steps - 1:
            say(f"step {i}: loss {losses[-1].item():.3f}")
    n = max(1, min(5, steps // 2))
    return torch.stack(losses[:n]).mean().item(), torch.stack(losses[-n:]).mean().item()


@torch.no_grad()
def serve(model, lens, tokens, vocab, seed=0):
    """Prefills prompts of `lens` tokens packed one after another into pools of states,
    decodes `tokens` more of each (given ones, so that a whole pass over the same ids
    has the same answers), and returns both: logits [n,tokens,vocab]."""
    rng = torch.Generator().manual_seed(seed)
    ids = [torch.randint(0, vocab, (n + tokens,), generator=rng).cuda() for n in lens]
    prompts = torch.cat([s[:n] for s, n in zip(ids, lens)])[None]
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")
    _, pools = model(prompts, cu_seqlens=cu, want_state=True)
    slots = torch.arange(len(lens), dtype=torch.int32, device="cuda").flip(0).contiguous()  # any order of rows
    rows = slots.tolist()
    out = []
    for t in range(tokens):
        out.append(model.step(torch.stack([ids[r][lens[r] + t] for r in rows]), pools, slots))
    want = torch.stack([model(ids[r][None])[0][0, lens[r] :] for r in rows])
    return torch.stack(out, 1), want


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=300)
    p.add_argument("--tokens", type=int, default=32, help="decoded tokens a prompt")
    args = p.parse_args(argv)
    torch.manual_seed(0)
    vocab = 32
    model = SelectiveModel(vocab, 128, states=16)
    first, last = train(model, args.steps, vocab)
    print(f"answers: loss {first:.3f} -> {last:.3f}")
    got, want = serve(model, [37, 0, 130, 64], args.tokens, vocab)
    diff = float((got.float() - want.float()).norm() / want.float().norm())
    print(f"decoded against whole passes: relative difference {diff:.4f}")
    return first, last, diff


if __name__ == "__main__":
    main()
