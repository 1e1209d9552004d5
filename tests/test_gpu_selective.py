"""The layer that runs the convolution, the selective scan, the norms and their steps
together: values and parameter gradients against the same layer written out in 64
bits on the CPU, decoding against whole passes, and the command."""
import pytest
import torch

import ssm_ref as ref
from ssm_ref import rel
from weight_scans_amd import selective

pytestmark = pytest.mark.gpu


def plain(layer, p, x, conv, scan):
    """Selective.forward in fp64 from the definitions."""
    x, z = (x @ p["xz.weight"].T).split(layer.inner, -1)
    x, conv = ref.conv(x, p["taps"], p["taps_bias"], conv, None, True)
    d, b, c = (x @ p["dbc.weight"].T).split([layer.rank, layer.states, layer.states], -1)
    y, scan = ref.scan(x, d @ p["dt.weight"].T, -p["log_a"].exp(), b[:, :, None], c[:, :, None], p["skip"],
                       z if layer.gate == "scan" else None, p["dt_bias"], scan, None, True)
    if layer.gate == "norm":
        split = lambda t: t.unflatten(-1, (layer.groups, -1))  # noqa: E731
        y = ref.gated_norm(split(y), split(z), p["norm"], 1e-6, False).flatten(-2)
    return y @ p["out.weight"].T, conv, scan


@pytest.mark.parametrize("dtype,tol", [
    (torch.float64, 1e-9),   # as the operators, 1e-12, and the library's products
    (torch.float32, 5e-5)])  # 1e-5 of the operators, a few of them in a row
@pytest.mark.parametrize("T,gate,groups", [(5, "norm", 1), (90, "norm", 3), (40, "scan", 1)])
def test_layer_values_and_gradients(dtype, tol, T, gate, groups):
    torch.manual_seed(T)
    layer = selective.Selective(32, inner=48, states=8, rank=4, groups=groups, gate=gate, dtype=dtype)
    x = torch.randn(2, T, 32, dtype=dtype, device="cuda", requires_grad=True)
    conv, scan = layer.pools(2)
    conv, scan = (torch.randn_like(t).mul(0.3).requires_grad_(True) for t in (conv, scan))
    dy = torch.randn(2, T, 32, dtype=dtype, device="cuda")
    names, leaves = zip(*((n, t) for n, t in layer.named_parameters() if gate == "norm" or n != "norm"))
    y, ends = layer(x, (conv, scan), want_state=True)
    got = torch.autograd.grad((y * dy).sum() + ends[0].square().sum() + ends[1].square().sum(), [x, conv, scan, *leaves])
    cx, cc, cs, *cp = (t.detach().double().cpu().requires_grad_(True) for t in (x, conv, scan, *leaves))
    wy, wc, wsn = plain(layer, dict(zip(names, cp)), cx, cc, cs)
    want = torch.autograd.grad((wy * dy.double().cpu()).sum() + wc.square().sum() + wsn.square().sum(), [cx, cc, cs, *cp])
    assert rel(y, wy) <= tol and rel(ends[0], wc) <= tol and rel(ends[1], wsn) <= tol
    for n, a, b in zip(("x", "conv", "scan") + names, got, want):
        assert rel(a, b) <= tol, n


@pytest.mark.parametrize("gate", ["norm", "scan"])
def test_decoding_continues_packed_prompts(gate):
    """fp32 throughout, where steps and whole passes differ by roundings of 6e-8 only."""
    torch.manual_seed(1)
    model = selective.SelectiveModel(32, 64, states=16, gate=gate, dtype=torch.float32)
    got, want = selective.serve(model, [3, 0, 70, 1, 300], 6, 32)
    assert rel(got, want.double().cpu()) <= 1e-4


def test_command_runs():
    first, last, diff = selective.main(["--steps", "12", "--tokens", "4"])
    assert first == first and last == last  # numbers
    assert diff <= 3e-2  # two layers in bf16, some four roundings of 2e-3 each and the logits'


@pytest.mark.parametrize("dtype,tol", [
    (torch.float64, 1e-9),   # as the layer's
    (torch.float32, 1e-4)])  # two layers of 5e-5
@pytest.mark.parametrize("gate", ["norm", "scan"])
def test_gradients_of_the_model(gate, dtype, tol):
    """What training steps on: the loss of the answers and its gradient of every parameter, against the model
    written out in 64 bits."""
    torch.manual_seed(3)
    back, vocab = 4, 11
    model = selective.SelectiveModel(vocab, 24, layers=2, inner=40, states=6, rank=3, gate=gate, dtype=dtype)
    with torch.no_grad():  # weights of ones hide what multiplies them
        for t in (*model.norms, *model.scales):
            t.add_(0.3 * torch.randn_like(t))
    ids = torch.randint(0, vocab, (3, 30)).cuda()
    names, leaves = zip(*((n, t) for n, t in model.named_parameters() if gate == "norm" or not n.endswith(".norm")))
    entropy = lambda x, i: torch.nn.functional.cross_entropy(x[:, back:].flatten(0, 1), i[:, :-back].flatten())  # noqa: E731
    loss = entropy(model(ids)[0], ids)
    got = torch.autograd.grad(loss, leaves)

    c = [t.detach().double().cpu().requires_grad_(True) for t in leaves]
    p = dict(zip(names, c))
    x = p["embed.weight"][ids.cpu()]
    n, r = ref.add_norm(x, torch.zeros_like(x), p["norms.0"], None, None, 1e-6)
    for i, layer in enumerate(model.layers):
        own = {k.removeprefix(f"layers.{i}."): t for k, t in p.items() if k.startswith(f"layers.{i}.")}
        n, r = ref.add_norm(plain(layer, own, n, None, None)[0], r, p[f"norms.{i + 1}"], None, p[f"scales.{i}"], 1e-6)
    wanted = entropy(n @ p["head.weight"].T, ids.cpu())
    assert abs(float(loss.detach()) - float(wanted.detach())) <= tol * float(wanted.detach())
    for k, a, b in zip(names, got, torch.autograd.grad(wanted, c)):
        assert float(b.norm()) > 0 and rel(a, b) <= tol, k
