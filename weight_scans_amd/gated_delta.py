"""A layer of gated delta-rule heads, and a small command that trains and serves one.

The layer shows the operators of ``delta.py`` together as a model uses them:

    projection -> q, k, v (views of one [B,T,...] tensor) and the gates
    qknorm_rope: rows of q and k to unit length, weights, rotation by position
    delta_rule:  y and the state after the last token (training, prefill)
    gl_delta_step on a pool of states (decoding, any rows of the batch)

    python -m weight_scans_amd.gated_delta [--steps N] [--tokens N]

learns to answer a key with the value that it was given earlier in the sequence
(which takes the fast weight: the pairs are new in every sequence), then
prefills prompts of different lengths packed one after another and decodes from
their states, and checks the decoded outputs against whole passes.
"""
from __future__ import annotations

import argparse

import torch

from .delta import delta_rule, gl_delta_step, gl_qknorm_rope_fwd, qknorm_rope

KEYS = 16  # of the command's task; its tokens are a key, or a key with a value


class GatedDelta(torch.nn.Module):
    """x [B,T,width] -> y [B,T,width].  `heads` value heads of `dv` columns read
    `key_heads` query / key heads of `dk` (heads a multiple of key_heads); the
    first `rot` columns of q and k are turned by position (0: none)."""

    def __init__(self, width, heads, dk=64, dv=64, key_heads=None, rot=0, max_pos=4096, base=10000.0,
                 device="cuda", dtype=torch.bfloat16):
        super().__init__()
        self.heads, self.key_heads, self.dk, self.dv = heads, key_heads or heads, dk, dv
        self.split = [self.key_heads * dk, self.key_heads * dk, heads * dv]
        make = dict(device=device, dtype=dtype, bias=False)
        self.qkv = torch.nn.Linear(width, sum(self.split), **make)
        self.gates = torch.nn.Linear(width, 2 * heads, device=device, dtype=dtype)
        self.out = torch.nn.Linear(heads * dv, width, **make)
        self.wq = torch.nn.Parameter(torch.ones(dk, device=device, dtype=dtype))
        self.wk = torch.nn.Parameter(torch.ones(dk, device=device, dtype=dtype))
        with torch.no_grad():  # gates start at slow forgetting, half writes
            self.gates.bias.copy_(torch.cat([torch.full((heads,), 4.0), torch.zeros(heads)]))
        table = torch.float64 if dtype == torch.float64 else torch.float32
        cos = sin = None
        if rot:
            freq = base ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
            angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
            cos, sin = angle.cos().to(device, table), angle.sin().to(device, table)
        self.register_buffer("cos", cos, persistent=False)
        self.register_buffer("sin", sin, persistent=False)

    def _project(self, x):
        """q, k [B,Hk,T,dk], v [B,H,T,dv] (views), log_alpha, beta [B,H,T]."""
        q, k, v = (t.unflatten(-1, (-1, d)).transpose(1, 2)
                   for t, d in zip(self.qkv(x).split(self.split, -1), (self.dk, self.dk, self.dv)))
        a, b = self.gates(x).transpose(1, 2).split(self.heads, 1)
        return q, k, v, torch.nn.functional.logsigmoid(a), torch.sigmoid(b)

    def _norm_opts(self):
        # rows of unit length (before their weights)
        return dict(q_scale=self.dk ** -0.5, k_scale=self.dk ** -0.5)

    def forward(self, x, state=None, pos=None, pos0=0, cu_seqlens=None, want_state=False):
        """The layer over whole sequences (training, prefill).  pos [B,T] int32, or
        the tokens stand at pos0, pos0 + 1, ...; packed prompts: B = 1 and
        cu_seqlens.  Returns (y, states after the last tokens or None)."""
        q, k, v, log_alpha, beta = self._project(x)
        q, k = qknorm_rope(q, k, self.wq, self.wk, self.cos, self.sin, pos=pos, pos0=pos0, **self._norm_opts())
        y, state = delta_rule(q, k, v, log_alpha, beta, scale=1.0, state=state, cu_seqlens=cu_seqlens,
                              want_state=want_state)
        return self.out(y.transpose(1, 2).flatten(-2)), state

    @torch.no_grad()
    def step(self, x, states, pos, slots=None):
        """One token of each row, x [B,width] at positions pos [B] (int32): updates
        `states` [n,H,dv,dk] in place, row b's at slots[b] (or at b)."""
        q, k, v, log_alpha, beta = self._project(x[:, None])
        q, k = gl_qknorm_rope_fwd(q, k, self.wq, self.wk, self.cos, self.sin, pos=pos[:, None].contiguous(),
                                  **self._norm_opts())
        y = gl_delta_step(*(t[:, :, 0] for t in (q, k, v, log_alpha, beta)), states, scale=1.0, slots=slots)
        return self.out(y.flatten(-2))


class Recall(torch.nn.Module):
    """Embedding, two layers with a residual path, logits over the tokens."""

    def __init__(self, tokens, width, **layer):
        super().__init__()
        device, dtype = layer.get("device", "cuda"), layer.get("dtype", torch.bfloat16)
        self.embed = torch.nn.Embedding(tokens, width, device=device, dtype=dtype)
        self.layers = torch.nn.ModuleList(GatedDelta(width, **layer) for _ in range(2))
        self.norms = torch.nn.ModuleList(torch.nn.RMSNorm(width, device=device, dtype=dtype) for _ in range(3))
        self.head = torch.nn.Linear(width, tokens, bias=False, device=device, dtype=dtype)

    def forward(self, ids, states=None, pos=None, cu_seqlens=None, want_state=False):
        x, ends = self.embed(ids), []
        for i, layer in enumerate(self.layers):
            y, end = layer(self.norms[i](x), None if states is None else states[i], pos=pos, cu_seqlens=cu_seqlens,
                           want_state=want_state)
            x, ends = x + y, ends + [end]
        return self.head(self.norms[2](x)), ends

    @torch.no_grad()
    def step(self, ids, states, pos, slots=None):
        x = self.embed(ids)
        for i, layer in enumerate(self.layers):
            x = x + layer.step(self.norms[i](x), states[i], pos, slots)
        return self.head(self.norms[2](x))


def recall_batch(rng, batch, pairs, keys):
    """Sequences of `pairs` tokens that each stand for one of `keys` keys with one of
    `keys` values, new in every sequence, then the keys alone in another order;
    ids [B,2 pairs] and the values asked for [B,pairs]."""
    k = torch.stack([torch.randperm(keys, generator=rng)[:pairs] for _ in range(batch)])
    v = torch.randint(0, keys, (batch, pairs), generator=rng)
    order = torch.stack([torch.randperm(pairs, generator=rng) for _ in range(batch)])
    return torch.cat([keys + keys * k + v, k.gather(1, order)], 1), v.gather(1, order)


def train(model, steps, batch=64, pairs=12, keys=KEYS, lr=3e-3, seed=0, say=print):
    """Mean loss of the answers at the first and the last steps."""
    rng = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=lr, weight_decay=0.0)
    losses = []
    for i in range(steps):
        ids, answers = (t.cuda() for t in recall_batch(rng, batch, pairs, keys))
        logits, _ = model(ids)
        loss = torch.nn.functional.cross_entropy(logits[:, pairs:].flatten(0, 1).float(), answers.flatten())
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
    """Prefills prompts of `lens` tokens packed one after another into a pool of
    states, decodes `tokens` more of each (given ones, so that a whole pass over
    the same ids has the same answers), and returns both: logits [n,tokens,vocab]."""
    rng = torch.Generator().manual_seed(seed)
    ids = [torch.randint(0, vocab, (n + tokens,), generator=rng).cuda() for n in lens]
    prompts = torch.cat([s[:n] for s, n in zip(ids, lens)])[None]
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(n) for n in lens]).to("cuda", torch.int32)[None]
    _, states = model(prompts, pos=pos, cu_seqlens=cu, want_state=True)
    slots = torch.arange(len(lens), dtype=torch.int32, device="cuda").flip(0).contiguous()  # any order of rows
    rows = slots.tolist()
    at = torch.tensor([lens[r] for r in rows], dtype=torch.int32, device="cuda")
    out = []
    for t in range(tokens):
        x = torch.stack([ids[r][lens[r] + t] for r in rows])
        out.append(model.step(x, states, at + t, slots))
    got = torch.stack(out, 1)
    want = torch.stack([model(ids[r][None])[0][0, lens[r] :] for r in rows])
    return got, want


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=300)
    p.add_argument("--tokens", type=int, default=32, help="decoded tokens a prompt")
    args = p.parse_args(argv)
    torch.manual_seed(0)
    vocab = KEYS + KEYS * KEYS
    model = Recall(vocab, 256, heads=4, key_heads=2, dk=64, dv=64, rot=32)
    first, last = train(model, args.steps)
    print(f"answers: loss {first:.3f} -> {last:.3f}")
    got, want = serve(model, [37, 0, 130, 64], args.tokens, vocab)
    diff = float((got.float() - want.float()).norm() / want.float().norm())
    print(f"decoded against whole passes: relative difference {diff:.4f}")
    return first, last, diff


if __name__ == "__main__":
    main()
