"""64-bit definitions of the linear attention with a decay for each head and of the layer
norm, for the tests: the recurrence token by token, its derivative by the reverse recurrence,
and the norm's derivative from its formula. CPU tensors in, float64 CPU tensors out."""
import torch

D = 128


def make(lens, H, G=1, seed=0, h0=False, dhT=False, log_decay=None):
    """Inputs: q, k, v, do ~ N(0,1) in bf16, states 0.1 N(0,1), slopes from 0 to about -0.9."""
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)

    def bf(*s):
        return torch.randn(*s, generator=g).to(torch.bfloat16)

    d = dict(lens=tuple(lens), H=H, G=G, q=bf(T, H // G, D), k=bf(T, H // G, D), v=bf(T, H, D), do=bf(T, H, D),
             cu_seqlens=torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int64))
    if log_decay is None:
        log_decay = -torch.exp2(-8.0 * torch.arange(H) / max(H, 1)) * 0.9
        log_decay[-1] = 0.0
    d["log_decay"] = torch.as_tensor(log_decay, dtype=torch.float32).expand(H).contiguous()
    d["h0"] = 0.1 * torch.randn(N, H, D, D, generator=g) if h0 else None
    d["dhT"] = 0.1 * torch.randn(N, H, D, D, generator=g) if dhT else None
    return d


def _heads(x, G):
    return x.double().repeat_interleave(G, dim=1)


def _start(x, N, H):
    return x.double().clone() if x is not None else torch.zeros(N, H, D, D, dtype=torch.float64)


def forward(d, scale=D ** -0.5):
    H, G, N = d["H"], d["G"], len(d["lens"])
    q, k, v = _heads(d["q"], G), _heads(d["k"], G), d["v"].double()
    gamma = torch.exp(d["log_decay"].double())[:, None, None]
    S, o = _start(d["h0"], N, H), torch.zeros_like(v)
    for n in range(N):
        s = S[n]
        for t in range(int(d["cu_seqlens"][n]), int(d["cu_seqlens"][n + 1])):
            s = gamma * s + v[t][:, :, None] * k[t][:, None, :]
            o[t] = scale * (s @ q[t][:, :, None])[:, :, 0]
        S[n] = s
    return dict(o=o, hT=S)


def loss(d, scale=D ** -0.5):
    f = forward(d, scale)
    out = (f["o"] * d["do"].double()).sum()
    return out + (f["hT"] * d["dhT"].double()).sum() if d["dhT"] is not None else out


def backward(d, scale=D ** -0.5):
    H, G, N = d["H"], d["G"], len(d["lens"])
    q, k, v, do = _heads(d["q"], G), _heads(d["k"], G), d["v"].double(), d["do"].double()
    gamma = torch.exp(d["log_decay"].double())[:, None, None]
    S, R = _start(d["h0"], N, H), _start(d["dhT"], N, H)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for n in range(N):
        t0, t1 = int(d["cu_seqlens"][n]), int(d["cu_seqlens"][n + 1])
        s = S[n]
        for t in range(t0, t1):
            s = gamma * s + v[t][:, :, None] * k[t][:, None, :]
            dq[t] = scale * (s.transpose(1, 2) @ do[t][:, :, None])[:, :, 0]
        r = R[n]
        for t in reversed(range(t0, t1)):
            r = r + scale * do[t][:, :, None] * q[t][:, None, :]
            dv[t] = (r @ k[t][:, :, None])[:, :, 0]
            dk[t] = (r.transpose(1, 2) @ v[t][:, :, None])[:, :, 0]
            r = gamma * r
        R[n] = r
    T = q.shape[0]
    return dict(dq=dq.view(T, H // G, G, D).sum(2), dk=dk.view(T, H // G, G, D).sum(2), dv=dv, dh0=R)


def norm_forward(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + eps)
    y = xc * rstd[:, None]
    y = y * (w.double() if w is not None else 1.0) + (b.double() if b is not None else 0.0)
    return dict(y=y, mean=mean, rstd=rstd)


def norm_backward(x, dy, w, mean, rstd):
    """From the given statistics, as the operator takes them."""
    x, dy, mean, rstd = x.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    h = (x - mean) * rstd
    a = dy * (w.double() if w is not None else 1.0)
    dx = rstd * (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True))
    return dict(dx=dx, dweight=(dy * h).sum(0), dbias=dy.sum(0))
