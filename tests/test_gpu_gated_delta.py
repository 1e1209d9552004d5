"""The layer that runs the norms, the delta rule and its steps together: values
and parameter gradients against the same layer written out in 64 bits on the
CPU, decoding against whole passes, and the command."""
import pytest
import torch

from delta_ref import delta, qknorm, rel
from weight_scans_amd import gated_delta

pytestmark = pytest.mark.gpu


def plain(layer, params, x, state):
    """GatedDelta.forward in fp64 from the definitions."""
    B, T, _ = x.shape
    heads = lambda t, d: t.unflatten(-1, (-1, d)).transpose(1, 2)  # noqa: E731
    q, k, v = (x @ params["qkv.weight"].T).split(layer.split, -1)
    a, b = (x @ params["gates.weight"].T + params["gates.bias"]).transpose(1, 2).split(layer.heads, 1)
    pos = torch.arange(T)[None].expand(B, T)
    cos, sin = (t.double().cpu() for t in (layer.cos, layer.sin))
    q = qknorm(heads(q, layer.dk), params["wq"], cos, sin, pos, 1e-6, layer.dk ** -0.5)
    k = qknorm(heads(k, layer.dk), params["wk"], cos, sin, pos, 1e-6, layer.dk ** -0.5)
    y, end = delta(q, k, heads(v, layer.dv), torch.nn.functional.logsigmoid(a), torch.sigmoid(b), 1.0, state)
    return y.transpose(1, 2).flatten(-2) @ params["out.weight"].T, end


@pytest.mark.parametrize("dtype,tol", [
    (torch.float64, 1e-9),   # as the operators, 1e-10, and the library's products
    (torch.float32, 5e-5)])  # 1e-5 of the operators, a few of them in a row
@pytest.mark.parametrize("T", [5, 90])
def test_layer_values_and_gradients(dtype, tol, T):
    torch.manual_seed(T)
    layer = gated_delta.GatedDelta(48, 4, dk=32, dv=24, key_heads=2, rot=16, dtype=dtype)
    x = torch.randn(2, T, 48, dtype=dtype, device="cuda", requires_grad=True)
    state = (0.3 * torch.randn(2, 4, 24, 32, dtype=dtype, device="cuda")).requires_grad_(True)
    dy = torch.randn(2, T, 48, dtype=dtype, device="cuda")
    names, leaves = zip(*layer.named_parameters())
    y, end = layer(x, state, want_state=True)
    got = torch.autograd.grad((y * dy).sum() + end.square().sum(), [x, state, *leaves])
    cx, cs, *cp = (t.detach().double().cpu().requires_grad_(True) for t in (x, state, *leaves))
    wy, wend = plain(layer, dict(zip(names, cp)), cx, cs)
    want = torch.autograd.grad((wy * dy.double().cpu()).sum() + wend.square().sum(), [cx, cs, *cp])
    assert rel(y, wy) <= tol and rel(end, wend) <= tol
    for n, a, b in zip(("x", "state") + names, got, want):
        assert rel(a, b) <= tol, n


def test_decoding_continues_packed_prompts():
    """fp32 throughout, where steps and whole passes differ by roundings of 6e-8 only."""
    torch.manual_seed(1)
    model = gated_delta.Recall(32, 64, heads=4, key_heads=2, dk=32, dv=32, rot=32, dtype=torch.float32)
    got, want = gated_delta.serve(model, [3, 0, 70, 1], 6, 32)
    assert rel(got, want.double().cpu()) <= 1e-4


def test_command_learns_to_recall():
    first, last, diff = gated_delta.main(["--steps", "120", "--tokens", "4"])
    assert last < 0.7 * first
    assert diff <= 3e-2  # two layers in bf16, some four roundings of 2e-3 each and the logits'
