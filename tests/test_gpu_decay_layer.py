"""The layer of examples/decay_layer.py: linear attention and layer norm run together, forward, backward and
decoding, against the layer's formulas in 64 bits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "decay_layer.py")
U = 2.0 ** -8      # of bf16


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decay_layer", _path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(layer, p, x, lengths):
    """The layer in 64 bits from parameters p and x, token by token."""
    def norm(x, w, b):
        c = x - x.mean(-1, keepdim=True)
        return c * torch.rsqrt(c.square().mean(-1, keepdim=True) + 1e-5) * w + b

    a = norm(x, p["norm_in.0"], p["norm_in.1"])
    H, G = layer.heads, layer.heads // layer.qk_heads
    q, k = ((a @ p[w]).view(len(x), H // G, 128).repeat_interleave(G, 1) for w in ("wq", "wk"))
    v = (a @ p["wv"]).view(len(x), H, 128)
    gamma = torch.exp(layer.log_decay.double()).view(H, 1, 1)
    out, t = [], 0
    for n in lengths:
        S = torch.zeros(H, 128, 128, dtype=torch.float64, device=x.device)
        for _ in range(n):
            S = gamma * S + v[t][:, :, None] * k[t][:, None, :]
            out.append(128 ** -0.5 * (S @ q[t][:, :, None])[:, :, 0])
            t += 1
    o = norm(torch.stack(out), p["norm_out.0"], p["norm_out.1"])
    return x + o.reshape(len(x), -1) @ p["wo"]


def distance(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


def test_forward_and_gradients(example):
    # Errors in the mean square: a bf16 rounding is at most u / sqrt(3) = 0.58 u of its value, on the way to y or to a
    # gradient there are at most 16 (the layer's tensors forwards and backwards, the attention's operands), and a
    # product or norm passes its operands' relative errors on, at most doubled by the two norms: 2 sqrt(16) 0.58 u.
    limit = 2 * 16 ** 0.5 * 0.58 * U
    lengths = [70, 1, 130]
    layer = example.DecayLayer(256, 4, groups=2)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(sum(lengths), 256, generator=gen, device="cuda").bfloat16().requires_grad_()
    dy = torch.randn(x.shape, generator=gen, device="cuda").bfloat16()
    cu = torch.tensor([0, 70, 71, 201], device="cuda")
    y, _ = layer(x, cu)
    y.backward(dy)
    assert layer.status() == 0
    p = {n: w.detach().double().requires_grad_() for n, w in layer.named_parameters()}
    x64 = x.detach().double().requires_grad_()
    ref = reference(layer, p, x64, lengths)
    ref.backward(dy.double())
    assert distance(y, ref.detach()) < limit
    assert distance(x.grad, x64.grad) < limit
    for n, w in layer.named_parameters():
        assert distance(w.grad, p[n].grad) < limit, n


def test_prompts_continued_token_by_token(example):
    # The same tokens in one pass and one by one. Both round q, k, v, o and the norms to bf16 at the same places and
    # differ in the attention (its operands, three roundings) and in what follows from it (five): each side is off by
    # at most sqrt(8) 0.58 u, doubled by the norm.
    limit = 2 * 2 ** 0.5 * 8 ** 0.5 * 0.58 * U
    layer = example.DecayLayer(256, 4)
    gen = torch.Generator(device="cuda").manual_seed(4)
    n, T = 3, 40
    x = torch.randn(n, T, 256, generator=gen, device="cuda").bfloat16()
    cu = torch.arange(n + 1, device="cuda") * T
    with torch.no_grad():
        y, state = layer(x.reshape(n * T, 256), cu)
        cut = T - 9
        head, s = layer(x[:, :cut].reshape(n * cut, 256), torch.arange(n + 1, device="cuda") * cut)
    assert distance(head.view(n, cut, 256), y.view(n, T, 256)[:, :cut].double()) < limit
    for t in range(cut, T):
        out = layer.step(x[:, t].contiguous(), s)
        assert distance(out, y.view(n, T, 256)[:, t].double()) < limit
    assert distance(s, state.double()) < limit


def test_training_and_generating(example):
    layer, teacher = example.DecayLayer(256, 4, groups=2, seed=0), example.DecayLayer(256, 4, groups=2, seed=7)
    losses = example.train(layer, teacher, [100, 1, 31], 12)
    assert losses[-1] < 0.95 * losses[0]
    cu = torch.tensor([0, 5, 12], device="cuda")
    x = torch.randn(12, 256, device="cuda").bfloat16()
    y, more, state = example.generate(layer, x, cu, 4)
    assert y.shape == (12, 256) and more.shape == (2, 4, 256) and state.shape == (2, 4, 128, 128)
    assert torch.isfinite(more.float()).all()
