"""A residual layer of a language model on the library's linear attention and layer norm, in training and in
serving:

    a = layernorm(x);  q, k, v = a Wq, a Wk, a Wv;  o = linear attention(q, k, v), a fixed decay for each head
    y = x + layernorm(o, over each head's 128 values) Wo

``python examples/decay_layer.py`` trains the layer on packed sequences towards another one's outputs, then runs a
batch of prompts and continues it token by token.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from kimi_delta_attention_15_gb300 import ops  # noqa: E402

DIM = 128


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        y, mean, rstd = ops.layernorm_fwd(x, weight, bias)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        g = ops.layernorm_bwd(x, dy.contiguous(), weight, mean, rstd)
        return g["dx"], g["dweight"], g["dbias"]


class LinearAttention(torch.autograd.Function):
    """o and the final states; the decays are constants of the model. A malformed cu_seqlens is found on the device:
    ops.device_status of the workspace in `check` tells, where a program wants to wait for it."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, h0, cu_seqlens, check):
        o, hT, workspace = ops.linattn_fwd(q, k, v, log_decay, h0=h0, cu_seqlens=cu_seqlens)
        check.append(workspace)
        ctx.save_for_backward(q, k, v, log_decay, h0, cu_seqlens)
        ctx.set_materialize_grads(False)
        return o, hT

    @staticmethod
    def backward(ctx, do, dhT):
        q, k, v, log_decay, h0, cu_seqlens = ctx.saved_tensors
        do = torch.zeros_like(v) if do is None else do.contiguous()
        dhT = None if dhT is None else dhT.contiguous()
        g = ops.linattn_bwd(q, k, v, log_decay, do, h0=h0, cu_seqlens=cu_seqlens, dhT=dhT, want_dh0=h0 is not None)
        return g["dq"], g["dk"], g["dv"], None, g["dh0"], None, None


class DecayLayer(torch.nn.Module):
    def __init__(self, width, heads, groups=1, device="cuda", seed=0):
        super().__init__()
        gen = torch.Generator(device=device).manual_seed(seed)

        def matrix(rows, columns):
            w = torch.randn(rows, columns, generator=gen, device=device) / rows ** 0.5
            return torch.nn.Parameter(w.bfloat16())

        self.heads, self.qk_heads = heads, heads // groups
        self.wq, self.wk = matrix(width, self.qk_heads * DIM), matrix(width, self.qk_heads * DIM)
        self.wv, self.wo = matrix(width, heads * DIM), matrix(heads * DIM, width)
        self.norm_in = torch.nn.ParameterList([torch.ones(width, device=device), torch.zeros(width, device=device)])
        self.norm_out = torch.nn.ParameterList([torch.ones(DIM, device=device), torch.zeros(DIM, device=device)])
        # slopes from 2^-(8/heads) down to 2^-8: memories from one token to some hundred
        h = torch.arange(heads, device=device, dtype=torch.float32)
        self.register_buffer("log_decay", -torch.exp2(-8.0 * (h + 1.0) / heads))
        self.check = []

    def project(self, x):
        a = LayerNorm.apply(x, *self.norm_in)
        return ((a @ self.wq).view(-1, self.qk_heads, DIM), (a @ self.wk).view(-1, self.qk_heads, DIM),
                (a @ self.wv).view(-1, self.heads, DIM))

    def close(self, x, o):
        return x + LayerNorm.apply(o, *self.norm_out).view(o.shape[0], -1) @ self.wo

    def forward(self, x, cu_seqlens, state=None):
        """Packed tokens x [T, width]; the outputs and the states [N, heads, 128, 128] after each sequence."""
        self.check.clear()
        o, state = LinearAttention.apply(*self.project(x), self.log_decay, state, cu_seqlens, self.check)
        return self.close(x, o), state

    @torch.no_grad()
    def step(self, x, state):
        """The next token x [N, width] of every sequence; the states are updated in place."""
        return self.close(x, ops.linattn_decode(*self.project(x), self.log_decay, state))

    def status(self):
        return ops.device_status(self.check[0])


def train(layer, teacher, lengths, steps, lr=2e-3, seed=1):
    """A few steps towards the teacher's outputs on packed sequences of these lengths; the losses."""
    dev = layer.log_decay.device
    gen = torch.Generator(device=dev).manual_seed(seed)
    cu = torch.tensor([0] + lengths, device=dev).cumsum(0)
    width = layer.wq.shape[0]
    losses = []
    for _ in range(steps):
        x = torch.randn(sum(lengths), width, generator=gen, device=dev).bfloat16()
        with torch.no_grad():
            target, _ = teacher(x, cu)
        y, _ = layer(x, cu)
        loss = (y.float() - target.float()).square().mean()
        layer.zero_grad()
        loss.backward()
        with torch.no_grad():
            for p in layer.parameters():        # the sign's step, as the first one of Adam
                p -= lr * p.grad.sign()
        losses.append(loss.item())
    if layer.status() != 0:
        raise ops.KdaError(f"device status {layer.status()}")
    return losses


def generate(layer, x, cu_seqlens, tokens):
    """The prompts (of one token at least) in one pass, then `tokens` more for each sequence, every output the next input."""
    with torch.no_grad():
        y, state = layer(x, cu_seqlens)
    last, out = y[cu_seqlens[1:] - 1], []
    for _ in range(tokens):
        last = layer.step(last, state)
        out.append(last)
    return y, torch.stack(out, 1), state


def main():
    if not torch.cuda.is_available():
        raise SystemExit("this example needs a GPU")
    layer, teacher = DecayLayer(512, 8, groups=2, seed=0), DecayLayer(512, 8, groups=2, seed=7)
    losses = train(layer, teacher, [700, 129, 1, 218], 30)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    cu = torch.tensor([0, 100, 357, 365], device="cuda")
    x = torch.randn(365, 512, device="cuda").bfloat16()
    y, more, state = generate(layer, x, cu, 16)
    print(f"prompts {tuple(y.shape)}, continued {tuple(more.shape)}, states {tuple(state.shape)}")


if __name__ == "__main__":
    main()
