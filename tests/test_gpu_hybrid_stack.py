"""The stack of examples/hybrid_stack.py: the gated recurrence, the norm of queries and keys with rotation, the linear
attention and the layer norm run together, forward, backward and decoding, against the formulas in 64 bits.

Tolerances. What bf16 tensors between the operators cost is computed: the formulas in 64 bits once more, with every
tensor that the stack holds in bf16 rounded to it there, forwards and backwards (`Rounded`). Its distance from the
formulas without any rounding is what such roundings do to each result; the stack's roundings are as many, at the same
places, of values that differ by the roundings before, so its distance is the same in the mean square. Twice that
is allowed, which leaves as much again for the mixers' own arithmetic (the attention's operands in two bf16 parts, 16 bits,
and fp32)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "hybrid_stack.py")
LENGTHS = [70, 1, 130]


class Rounded(torch.autograd.Function):
    """To bf16 and on in 64 bits, the gradient too."""

    @staticmethod
    def forward(ctx, x):
        return x.bfloat16().double()

    @staticmethod
    def backward(ctx, dx):
        return dx.bfloat16().double()


def exactly(x):
    return x


rounded = Rounded.apply


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_stack", _path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def norm(x, w, b):
    c = x - x.mean(-1, keepdim=True)
    return c * torch.rsqrt(c.square().mean(-1, keepdim=True) + 1e-5) * w + b


def recurrent(p, x, lengths, held):
    z, g, i = held(held(norm(x, p["norm.0"], p["norm.1"])) @ p["w"]).chunk(3, 1)
    log_a = -torch.exp(p["A_log"]) * torch.sigmoid(g)
    a, b = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a)) * torch.sigmoid(i) * z
    out, states, t = [], [], 0
    for n in lengths:
        h = torch.zeros_like(p["A_log"])
        for _ in range(n):
            h = a[t] * h + b[t]
            out.append(h)
            t += 1
        states.append(h)
    return held(x + held(held(torch.stack(out)) @ p["wo"])), torch.stack(states)


def attention(layer, p, x, lengths, held):
    H, Hqk = layer.heads, layer.qk_heads
    heads = held(held(norm(x, p["norm.0"], p["norm.1"])) @ p["w"]).unflatten(1, (-1, 128))
    q, k, v = heads.split([Hqk, Hqk, H], 1)
    at = torch.cat([torch.arange(n) for n in lengths]).to(x.device).double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), at[:, None] * layer.inv_freq.double())[:, None]

    def turned(s, w):
        s = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + 1e-6) * w
        s = torch.complex(s[..., :64], s[..., 64:]) * turn
        return held(torch.cat([s.real, s.imag], -1)).repeat_interleave(H // Hqk, 1)

    q, k = turned(q, p["q_weight"]), turned(k, p["k_weight"])
    gamma = torch.exp(layer.log_decay.double()).view(H, 1, 1)
    out, states, t = [], [], 0
    for n in lengths:
        S = torch.zeros(H, 128, 128, dtype=torch.float64, device=x.device)
        for _ in range(n):
            S = gamma * S + v[t][:, :, None] * k[t][:, None, :]
            out.append(128 ** -0.5 * (S @ q[t][:, :, None])[:, :, 0])
            t += 1
        states.append(S)
    o = held(norm(held(torch.stack(out)), p["norm_out.0"], p["norm_out.1"]))
    return held(x + held(o.reshape(len(x), -1) @ p["wo"])), torch.stack(states)


def reference(stack, x, lengths, held, dy=None):
    """{name: value} of the outputs, the states and, where dy is given, every gradient."""
    p = {n: w.detach().double().requires_grad_() for n, w in stack.named_parameters()}
    y = x64 = x.detach().double().requires_grad_()
    out = {}
    for n, layer in enumerate(stack.layers):
        of = {k[len(f"layers.{n}."):]: v for k, v in p.items() if k.startswith(f"layers.{n}.")}
        y, out[f"state {n}"] = recurrent(of, y, lengths, held) if n % 2 == 0 else attention(layer, of, y, lengths, held)
    out["y"] = y
    if dy is not None:
        y.backward(dy.double())
        out.update({"d " + n: w.grad for n, w in p.items()}, **{"d x": x64.grad})
    return {n: v.detach() for n, v in out.items()}


def distance(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


def test_forward_and_gradients(example):
    stack = example.HybridStack(256, 4, groups=2)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(sum(LENGTHS), 256, generator=gen, device="cuda").bfloat16().requires_grad_()
    dy = torch.randn(x.shape, generator=gen, device="cuda").bfloat16()
    cu = torch.tensor([0] + LENGTHS, device="cuda").cumsum(0)
    y, states = stack(x, cu)
    y.backward(dy)
    assert stack.status() == 0 and len(states) == 2
    got = {"y": y.detach(), "d x": x.grad, **{f"state {n}": s for n, s in enumerate(states)},
           **{"d " + n: w.grad for n, w in stack.named_parameters()}}
    exact, held = (reference(stack, x, LENGTHS, h, dy) for h in (exactly, rounded))
    assert set(got) == set(exact)
    for n in exact:
        assert distance(got[n], exact[n]) < 2 * distance(held[n], exact[n]), n


def test_prompts_continued_token_by_token(example):
    # Both ways are within twice the roundings' distance of the formulas, so within four times of each other.
    stack = example.HybridStack(256, 4)
    gen = torch.Generator(device="cuda").manual_seed(4)
    n, T = 3, 40
    x = torch.randn(n, T, 256, generator=gen, device="cuda").bfloat16()
    exact, held = (reference(stack, x.reshape(n * T, 256), [T] * n, h) for h in (exactly, rounded))
    limit = {k: 4 * distance(held[k], exact[k]) for k in exact}
    with torch.no_grad():
        y, states = stack(x.reshape(n * T, 256), torch.arange(n + 1, device="cuda") * T)
        cut = T - 9
        head, s = stack(x[:, :cut].reshape(n * cut, 256), torch.arange(n + 1, device="cuda") * cut)
    out = [head.view(n, cut, 256)]
    for t in range(cut, T):
        out.append(stack.step(x[:, t].contiguous(), torch.full((n,), t, device="cuda"), s)[:, None])
    assert distance(torch.cat(out, 1).view(n * T, 256), y.double()) < limit["y"]
    for k, (a, b) in enumerate(zip(s, states)):
        assert distance(a, b.double()) < limit[f"state {k}"]


def test_training_and_generating(example):
    stack, teacher = example.HybridStack(256, 4, groups=2, seed=0), example.HybridStack(256, 4, groups=2, seed=7)
    losses = example.train(stack, teacher, [100, 1, 31], 3)
    assert all(torch.isfinite(torch.tensor(losses)))
    cu = torch.tensor([0, 5, 12], device="cuda")
    x = torch.randn(12, 256, device="cuda").bfloat16()
    y, more, states = example.generate(stack, x, cu, 4)
    assert y.shape == (12, 256) and more.shape == (2, 4, 256) and states[0].shape == (2, 256) and states[1].shape == (2, 4, 128, 128)
    assert torch.isfinite(more.float()).all()


def test_a_step_captured_and_replayed(example):
    """Decoding as a serving loop runs it: one graph of all layers, replayed token after token."""
    stack = example.HybridStack(256, 4, pairs=2)
    gen = torch.Generator(device="cuda").manual_seed(5)
    with torch.no_grad():
        _, states = stack(torch.randn(20, 256, generator=gen, device="cuda").bfloat16(), torch.tensor([0, 12, 20], device="cuda"))
    again = [s.clone() for s in states]
    tokens = torch.randn(5, 2, 256, generator=gen, device="cuda").bfloat16()
    x, positions = tokens[0].clone(), torch.tensor([12, 8], device="cuda")
    start = [s.clone() for s in states]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        stack.step(x, positions, states)           # the libraries' first calls, outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = stack.step(x, positions, states)
    for s, b in zip(states, start):
        s.copy_(b)
    for t in range(5):
        x.copy_(tokens[t])
        graph.replay()
        want = stack.step(tokens[t], torch.tensor([12 + t, 8 + t], device="cuda"), again)
        assert torch.equal(y, want)
        positions += 1
    assert all(torch.equal(a, b) for a, b in zip(states, again))
