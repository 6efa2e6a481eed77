"""A stack that alternates a recurrent layer with a linear attention layer, in training and in serving, on packed
sequences of any lengths:

    a = layernorm(x);  z, g, i = a W;  x = x + recurrence(z, g, i) Wo                      a state of `width` channels
    a = layernorm(x);  q, k, v = a W;  q, k = their norm and rotation by the positions;
                       x = x + layernorm(linear attention(q, k, v), over each head) Wo     a state of 128 x 128 a head

``python examples/hybrid_stack.py`` trains the stack towards another one's outputs, then runs a batch of prompts and
continues it token by token.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from decay_layer import DIM, LayerNorm, LinearAttention  # noqa: E402
from kimi_delta_attention_15_gb300 import ops  # noqa: E402


class Recurrence(torch.autograd.Function):
    """y and the final states from the columns p = [z, g_raw, i_raw] of one projection; the gradient of p comes as columns
    of one buffer too. A malformed cu_seqlens is found on the device: ops.device_status of the workspaces in `check`."""

    @staticmethod
    def forward(ctx, p, A_log, h0, cu_seqlens, check):
        z, g, i = p.chunk(3, 1)
        y, hT, kept, workspace = ops.recurrence_fwd(z, g, i, A_log, h0=h0, cu_seqlens=cu_seqlens, want_kept=True)
        check.append(workspace)
        ctx.save_for_backward(p, A_log, h0, cu_seqlens, kept)
        ctx.set_materialize_grads(False)
        return y, hT

    @staticmethod
    def backward(ctx, dy, dhT):
        p, A_log, h0, cu_seqlens, kept = ctx.saved_tensors
        z, g, i = p.chunk(3, 1)
        dy = torch.zeros(z.shape, dtype=p.dtype, device=p.device) if dy is None else dy
        dp = torch.empty_like(p)
        grads = dict(zip(("dx", "dg_raw", "di_raw"), dp.chunk(3, 1)))
        grads.update(dA_log=torch.empty_like(A_log), dh0=torch.empty_like(h0) if h0 is not None else None)
        ops.recurrence_bwd(z, g, i, A_log, dy.contiguous(), kept, h0=h0, cu_seqlens=cu_seqlens,
                           dhT=None if dhT is None else dhT.contiguous(), grads=grads)
        return dp, grads["dA_log"], grads["dh0"], None, None


class QkNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, inv_freq)
        return ops.qknorm_fwd(q, k, q_weight, k_weight, positions, inv_freq)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, *rest = ctx.saved_tensors
        g = ops.qknorm_bwd(q, k, dq.contiguous(), dk.contiguous(), *rest)
        return g["dq"], g["dk"], g["dq_weight"], g["dk_weight"], None, None


def matrix(gen, rows, columns, device):
    return torch.nn.Parameter((torch.randn(rows, columns, generator=gen, device=device) / rows ** 0.5).bfloat16())


def norm_of(width, device):
    return torch.nn.ParameterList([torch.ones(width, device=device), torch.zeros(width, device=device)])


class RecurrentLayer(torch.nn.Module):
    def __init__(self, width, device, gen):
        super().__init__()
        self.norm, self.w, self.wo = norm_of(width, device), matrix(gen, width, 3 * width, device), matrix(gen, width, width, device)
        # decays of an open gate between 0.9^8 and 0.999^8 a token
        rate = -8.0 * torch.log(0.9 + 0.099 * torch.rand(width, generator=gen, device=device))
        self.A_log = torch.nn.Parameter(torch.log(rate))

    def forward(self, x, positions, cu_seqlens, state, check):
        y, state = Recurrence.apply(LayerNorm.apply(x, *self.norm) @ self.w, self.A_log, state, cu_seqlens, check)
        return x + y @ self.wo, state

    def step(self, x, positions, state):
        z, g, i = (LayerNorm.apply(x, *self.norm) @ self.w).chunk(3, 1)
        return x + ops.recurrence_decode(z, g, i, self.A_log, state) @ self.wo


class AttentionLayer(torch.nn.Module):
    def __init__(self, width, heads, groups, device, gen):
        super().__init__()
        self.heads, self.qk_heads = heads, heads // groups
        self.norm, self.norm_out = norm_of(width, device), norm_of(DIM, device)
        self.w = matrix(gen, width, (2 * self.qk_heads + heads) * DIM, device)
        self.wo = matrix(gen, heads * DIM, width, device)
        self.q_weight, self.k_weight = (torch.nn.Parameter(torch.ones(DIM, device=device)) for _ in range(2))
        h = torch.arange(heads, device=device, dtype=torch.float32)
        self.register_buffer("log_decay", -torch.exp2(-8.0 * (h + 1.0) / heads))
        self.register_buffer("inv_freq", 10000.0 ** (-torch.arange(0, DIM, 2, device=device) / DIM))

    def project(self, x, positions):
        heads = (LayerNorm.apply(x, *self.norm) @ self.w).unflatten(1, (-1, DIM))
        q, k, v = heads.split([self.qk_heads, self.qk_heads, self.heads], 1)
        q, k = QkNorm.apply(q, k, self.q_weight, self.k_weight, positions, self.inv_freq)
        return q, k, v.contiguous()

    def close(self, x, o):
        return x + LayerNorm.apply(o, *self.norm_out).view(o.shape[0], -1) @ self.wo

    def forward(self, x, positions, cu_seqlens, state, check):
        o, state = LinearAttention.apply(*self.project(x, positions), self.log_decay, state, cu_seqlens, check)
        return self.close(x, o), state

    def step(self, x, positions, state):
        return self.close(x, ops.linattn_decode(*self.project(x, positions), self.log_decay, state))


class HybridStack(torch.nn.Module):
    def __init__(self, width, heads, groups=1, pairs=1, device="cuda", seed=0):
        super().__init__()
        gen = torch.Generator(device=device).manual_seed(seed)
        self.layers = torch.nn.ModuleList()
        for _ in range(pairs):
            self.layers += [RecurrentLayer(width, device, gen), AttentionLayer(width, heads, groups, device, gen)]
        self.check = []

    def forward(self, x, cu_seqlens, states=None):
        """Packed tokens x [T, width]; the outputs and each layer's states after each sequence."""
        self.check.clear()
        at = torch.arange(x.shape[0], device=x.device)
        positions = at - cu_seqlens[torch.searchsorted(cu_seqlens, at, right=True) - 1]
        after = []
        for n, layer in enumerate(self.layers):
            x, s = layer(x, positions, cu_seqlens, None if states is None else states[n], self.check)
            after.append(s)
        return x, after

    @torch.no_grad()
    def step(self, x, positions, states):
        """The next token x [N, width], at positions [N], of every sequence; the states are updated in place."""
        for layer, state in zip(self.layers, states):
            x = layer.step(x, positions, state)
        return x

    def status(self):
        """0, or the first error that a layer's call of the last forward pass found on the device."""
        return next((s for s in map(ops.device_status, self.check) if s), 0)


def train(stack, teacher, lengths, steps, lr=2e-3, seed=1):
    """A few steps towards the teacher's outputs on packed sequences of these lengths; the losses."""
    dev = stack.layers[0].A_log.device
    gen = torch.Generator(device=dev).manual_seed(seed)
    cu = torch.tensor([0] + lengths, device=dev).cumsum(0)
    losses = []
    for _ in range(steps):
        x = torch.randn(sum(lengths), stack.layers[0].w.shape[0], generator=gen, device=dev).bfloat16()
        with torch.no_grad():
            target, _ = teacher(x, cu)
        y, _ = stack(x, cu)
        loss = (y.float() - target.float()).square().mean()
        stack.zero_grad()
        loss.backward()
        with torch.no_grad():
            for p in stack.parameters():        # the sign's step, as the first one of Adam
                p -= lr * p.grad.sign()
        losses.append(loss.item())
    if stack.status() != 0:
        raise ops.KdaError(stack.status(), "hybrid_stack")
    return losses


def generate(stack, x, cu_seqlens, tokens):
    """The prompts (of one token at least) in one pass, then `tokens` more for each sequence, every output the next input."""
    with torch.no_grad():
        y, states = stack(x, cu_seqlens)
    last, out, positions = y[cu_seqlens[1:] - 1], [], cu_seqlens[1:] - cu_seqlens[:-1]
    for n in range(tokens):
        last = stack.step(last, positions + n, states)
        out.append(last)
    return y, torch.stack(out, 1), states


def main():
    if not torch.cuda.is_available():
        raise SystemExit("this example needs a GPU")
    stack, teacher = HybridStack(512, 8, groups=2, pairs=2, seed=0), HybridStack(512, 8, groups=2, pairs=2, seed=7)
    losses = train(stack, teacher, [700, 129, 1, 218], 30)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    cu = torch.tensor([0, 100, 357, 365], device="cuda")
    x = torch.randn(365, 512, device="cuda").bfloat16()
    y, more, states = generate(stack, x, cu, 16)
    print(f"prompts {tuple(y.shape)}, continued {tuple(more.shape)}, {len(states)} layers' states")


if __name__ == "__main__":
    main()
