"""The linear attention and its gradient in 64 bits as masked products over whole sequences, for sizes at which the
recurrence of linattn_oracle.py takes too long. On the device that the inputs are on, one head at a time.

    W_ij = gamma^{i-j} for j <= i, else 0
    o = scale ((W . Q K^T) V + gamma^{i+1} S0 q_i),  hT = gamma^T S0 + sum_j gamma^{T-1-j} v_j k_j^T
    dq = scale ((W . dO V^T) K + gamma^{i+1} S0^T do_i)
    dk = scale (W . dO V^T)^T Q + gamma^{T-1-j} dhT^T v_j,  dv = scale (W . Q K^T)^T dO + gamma^{T-1-j} dhT k_j
    dh0 = gamma^T dhT + scale sum_i gamma^{i+1} do_i q_i^T
"""
import torch

D = 128


def slow_decays(H):
    """Memories from some tens to ten thousand tokens, another one for each head, one without any decay."""
    g = -torch.logspace(-1.7, -4.0, H)
    g[H // 2] = 0.0
    return g


def reference(d, scale=D ** -0.5, backward=True):
    H, G, lens = d["H"], d["G"], d["lens"]
    dev = d["q"].device
    T, N = sum(lens), len(lens)
    out = {x: torch.zeros(T, H, D, dtype=torch.float64, device=dev) for x in ("o", "dq", "dk", "dv")}
    out.update({x: torch.zeros(N, H, D, D, dtype=torch.float64, device=dev) for x in ("hT", "dh0")})
    zero = torch.zeros(D, D, dtype=torch.float64, device=dev)
    for n, first in enumerate(sum(lens[:n]) for n in range(N)):
        L, at = lens[n], slice(first, first + lens[n])
        i = torch.arange(L, dtype=torch.float64, device=dev)
        for h in range(H):
            q, k = d["q"][at, h // G].double(), d["k"][at, h // G].double()
            v, do = d["v"][at, h].double(), d["do"][at, h].double()
            S0 = d["h0"][n, h].double() if d["h0"] is not None else zero
            R0 = d["dhT"][n, h].double() if d["dhT"] is not None else zero
            g = d["log_decay"][h].double()

            def power(x):
                return torch.where(x == 0, torch.ones_like(x), torch.exp(g * x))

            apart = i[:, None] - i[None, :]
            W = torch.where(apart >= 0, power(apart.clamp(min=0)), torch.zeros((), dtype=torch.float64, device=dev))
            after, left = power(i + 1)[:, None], power(L - 1 - i)[:, None]
            whole = power(torch.full((), float(L), dtype=torch.float64, device=dev))
            A = W * (q @ k.T)
            out["o"][at, h] = scale * (A @ v + after * (q @ S0.T))
            out["hT"][n, h] = whole * S0 + v.T @ (left * k)
            if backward:
                B = W * (do @ v.T)
                out["dq"][at, h] = scale * (B @ k + after * (do @ S0))
                out["dk"][at, h] = scale * (B.T @ q) + left * (v @ R0)
                out["dv"][at, h] = scale * (A.T @ do) + left * (k @ R0.T)
                out["dh0"][n, h] = whole * R0 + scale * (do.T @ (after * q))
    for x in ("dq", "dk"):
        out[x] = out[x].view(T, H // G, G, D).sum(2)
    return out if backward else {x: out[x] for x in ("o", "hT")}
