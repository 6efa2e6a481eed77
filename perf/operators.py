"""Cases of the linear attention with a decay for each head and of the layer norm.

Operators (K = V = 128 and the layouts of ``include/kda.h``: tokens [T, H, 128] bf16, states
[N, H, V, K] fp32 value-first, packed sequences through int64 offsets, q and k with H / G heads):

  linattn_fwd     S_t = exp(log_decay[h]) S_{t-1} + v_t k_t^T,  o_t = scale S_t q_t; the final states
  linattn_bwd     gradients of sum_t <o_t, do_t> + <S_T, dhT> with respect to q, k, v and the initial state
  linattn_decode  one token for each request, the state updated in place
  layernorm_fwd   y = (x - mean) rstd weight + bias over rows; mean and rstd
  layernorm_bwd   gradients with respect to x, weight and bias

``run`` computes them in elementary torch operations in 32 bits where ``own`` is false, and calls the
framework where it is true. ``exact`` is the recurrence, token by token, in 64 bits.
"""
import math

import torch

own = False

DIM = 128
SCALE = 1.0 / math.sqrt(DIM)
CHUNK = 64      # of the plain form
EPS = 1e-5


def listed():
    return [
        # a short packed batch of three sequences: latency, lengths around the chunk sizes
        {"name": "fwd_packed_17_33_65_H4", "op": "linattn_fwd", "lens": "17,33,65", "B": 1, "H": 4, "G": 1, "states": True},
        # one ordinary prompt: fewer (sequence, head) pairs than the card has multiprocessors
        {"name": "fwd_T4096_H32", "op": "linattn_fwd", "lens": "4096", "B": 1, "H": 32, "G": 1, "states": False},
        # a packed training batch of six ragged sequences, with a state carried in and out
        {"name": "fwd_packed6_H96", "op": "linattn_fwd", "lens": "1300,547,2048,963,271,3063", "B": 1, "H": 96, "G": 1,
         "states": True},
        # the backward pass of the short packed batch
        {"name": "bwd_packed_17_33_65_H4", "op": "linattn_bwd", "lens": "17,33,65", "B": 1, "H": 4, "G": 1, "states": True},
        # the backward pass with four value heads to a query/key head: dq, dk are sums over the group
        {"name": "bwd_T4096_H32_G4", "op": "linattn_bwd", "lens": "4096", "B": 1, "H": 32, "G": 4, "states": False},
        # the largest training step
        {"name": "bwd_T8192_H96", "op": "linattn_bwd", "lens": "8192", "B": 1, "H": 96, "G": 1, "states": False},
        # decoding a few requests of a small model: latency
        {"name": "decode_4req_H4", "op": "linattn_decode", "requests": 4, "H": 4, "G": 1},
        # decoding a full serving batch
        {"name": "decode_256req_H96", "op": "linattn_decode", "requests": 256, "H": 96, "G": 1},
        # the norm of a few tokens
        {"name": "norm_fwd_115x512", "op": "layernorm_fwd", "rows": 115, "width": 512, "dtype": "bfloat16"},
        # the norm of a training batch over a model width of 96 heads
        {"name": "norm_fwd_8192x12288", "op": "layernorm_fwd", "rows": 8192, "width": 12288, "dtype": "bfloat16"},
        # the backward pass of a norm over each head's 128 values
        {"name": "norm_bwd_131072x128", "op": "layernorm_bwd", "rows": 131072, "width": 128, "dtype": "bfloat16"},
        # the backward pass of a norm on a 32-bit residual stream, an odd number of rows
        {"name": "norm_bwd_4099x4096_fp32", "op": "layernorm_bwd", "rows": 4099, "width": 4096, "dtype": "float32"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["linattn_fwd", "linattn_fwd", "linattn_bwd", "linattn_bwd", "linattn_decode", "layernorm_fwd",
                     "layernorm_bwd"])
    if op in ("linattn_fwd", "linattn_bwd"):
        G = rng.choice([1, 1, 2, 4])
        H = G * _spread(rng, 1, 96 // G)
        most = min(16384, 786432 // H)          # tokens: no more than the largest listed case has
        T = _spread(rng, 1, most)
        kind = rng.choice(["one", "batch", "packed"])
        B, lens = 1, [T]
        if kind == "batch":
            B = rng.randint(1, 4)
            lens = [max(1, T // B)]
        elif kind == "packed":
            n = rng.randint(2, 8)
            cuts = sorted(rng.randint(0, T) for _ in range(n - 1))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [T])]      # empty sequences among them
        return {"op": op, "lens": ",".join(map(str, lens)), "B": B, "H": H, "G": G, "states": rng.random() < 0.5}
    if op == "linattn_decode":
        G = rng.choice([1, 1, 2, 4])
        H = G * _spread(rng, 1, 96 // G)
        return {"op": op, "requests": _spread(rng, 1, 256), "H": H, "G": G}
    width = rng.choice([DIM * _spread(rng, 1, 96), _spread(rng, 32, 12288)])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    most = 8192 * 12288 // width // (2 if dtype == "float32" else 1)
    return {"op": op, "rows": _spread(rng, 1, min(most, 262144)), "width": width, "dtype": dtype}


def _lens(case):
    return [int(x) for x in case["lens"].split(",")] * (case["B"] if "," not in case["lens"] else 1)


def _log_decay(H, device):
    """Fixed slopes from 2^-(8/H) down to 2^-8, the first head without any decay."""
    g = -torch.exp2(-8.0 * (torch.arange(H, device=device, dtype=torch.float32) + 1.0) / H)
    g[0] = 0.0
    return g


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32) * std).to(dtype)

    op = case["op"]
    s = {"case": case}
    if op == "linattn_decode":
        n, H, Hqk = case["requests"], case["H"], case["H"] // case["G"]
        s.update(q=normal(n, Hqk, DIM), k=normal(n, Hqk, DIM), v=normal(n, H, DIM), log_decay=_log_decay(H, dev),
                 state=normal(n, H, DIM, DIM, dtype=torch.float32))
    elif op in ("linattn_fwd", "linattn_bwd"):
        lens, H, Hqk = _lens(case), case["H"], case["H"] // case["G"]
        T, N = sum(lens), len(lens)
        s.update(q=normal(T, Hqk, DIM), k=normal(T, Hqk, DIM), v=normal(T, H, DIM), log_decay=_log_decay(H, dev), lens=lens,
                 cu=None, h0=None, dhT=None)
        if "," in case["lens"]:
            s["cu"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int64, device=dev)
        if case["states"]:
            s["h0"] = normal(N, H, DIM, DIM, dtype=torch.float32, std=0.1)
        if op == "linattn_bwd":
            s["do"] = normal(T, H, DIM)
            if case["states"]:
                s["dhT"] = normal(N, H, DIM, DIM, dtype=torch.float32, std=0.1)
    else:
        rows, width, dtype = case["rows"], case["width"], getattr(torch, case["dtype"])
        # rows of different size and offset, as a residual stream has them
        level = torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device=dev))
        x = torch.randn(rows, width, generator=gen, device=dev)
        s["x"] = (level * (x + 0.3)).to(dtype)
        s["weight"] = 1.0 + normal(width, dtype=torch.float32, std=0.1)
        s["bias"] = normal(width, dtype=torch.float32, std=0.1)
        if op == "layernorm_bwd":
            s["dy"] = normal(rows, width, dtype=dtype)
            f = s["x"].double()                 # what the forward pass left for the backward pass
            s["mean"] = f.mean(1).float()
            s["rstd"] = torch.rsqrt((f - f.mean(1, keepdim=True)).square().mean(1) + EPS).float()
            del f
    return s


# ------------------------------------------------------------------ the framework's operators
def _framework(s):
    from kimi_delta_attention_15_gb300 import ops
    op = s["case"]["op"]
    if op == "linattn_fwd":
        B = s["case"]["B"]
        o, hT, s["workspace"] = ops.linattn_fwd(s["q"], s["k"], s["v"], s["log_decay"], h0=s["h0"], cu_seqlens=s["cu"], B=B,
                                                scale=SCALE, workspace=s.get("workspace"))
        return {"o": o, "hT": hT}
    if op == "linattn_bwd":
        if "workspace" not in s:
            B = s["case"]["B"]
            H, G, N, T = s["case"]["H"], s["case"]["G"], len(s["lens"]), s["q"].shape[0]
            s["workspace"] = ops.linattn_alloc_workspace(ops.linattn_shape(T // B, H, N, B, scale=SCALE, groups=G),
                                                         s["q"].device, backward=True)
        return ops.linattn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"], s["workspace"], h0=s["h0"],
                               cu_seqlens=s["cu"], dhT=s["dhT"], B=s["case"]["B"], scale=SCALE)
    if op == "linattn_decode":
        o = ops.linattn_decode(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=SCALE)
        return {"o": o, "state": s["state"]}
    if op == "layernorm_fwd":
        y, mean, rstd = ops.layernorm_fwd(s["x"], s["weight"], s["bias"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    return ops.layernorm_bwd(s["x"], s["dy"], s["weight"], s["mean"], s["rstd"])


# ------------------------------------------------------------------------- the plain forms
def _decayed(q, k, v, g, s0, first, n):
    """The chunked sum over padded sequences: out_i = exp(g (i + first)) s0 q_i + sum_{j <= i} exp(g (i - j)) (q_i . k_j) v_j,
    and the state exp(g (n - 1 + first)) s0 + sum_j exp(g (n - j - 1)) v_j k_j^T after the last of a sequence's n tokens
    (without the exponent's first step where `first` is 0). q, k, v [N, H, L, 128] (rows past n zero), s0 [N, H, 128, 128]."""
    N, H, L, _ = q.shape
    c = L // CHUNK
    q, k, v = (x.reshape(N, H, c, CHUNK, DIM) for x in (q, k, v))
    g = g.view(1, H, 1, 1, 1)
    i = torch.arange(CHUNK, device=q.device, dtype=torch.float32)
    apart = i[:, None] - i[None, :]
    weight = torch.where(apart >= 0, torch.exp(g * apart.clamp(min=0)), torch.zeros((), device=q.device))
    out = ((q @ k.transpose(-1, -2)) * weight) @ v
    grown = v.transpose(-1, -2) @ (k * torch.exp(g * (CHUNK - 1 - i)[:, None]))      # what each chunk adds to the state
    m = torch.arange(c, device=q.device, dtype=torch.float32)
    between = m[:, None] - 1 - m[None, :]                                            # whole chunks from one to another
    carry = torch.where(between >= 0, torch.exp(g.view(H, 1, 1) * CHUNK * between.clamp(min=0)), torch.zeros((), device=q.device))
    state = (carry @ grown.reshape(N, H, c, DIM * DIM)).reshape(N, H, c, DIM, DIM)
    within = torch.exp(g * (i + 1)[:, None])
    out = out + within * (q @ state.transpose(-1, -2))
    t = (m[:, None] * CHUNK + i[None, :] + first).view(1, 1, c, CHUNK, 1)
    out = out + torch.exp(g * t) * (q @ s0[:, :, None].transpose(-1, -2))
    left = n.view(N, 1, 1) - 1 - torch.arange(L, device=q.device).view(1, 1, L)
    w = torch.where(left >= 0, torch.exp(g.view(1, H, 1) * left.clamp(min=0)), torch.zeros((), device=q.device))
    last = v.reshape(N, H, L, DIM).transpose(-1, -2) @ (k.reshape(N, H, L, DIM) * w[..., None])
    return out.reshape(N, H, L, DIM), last


def _plain_linattn(s, backward):
    lens, H, G = s["lens"], s["case"]["H"], s["case"]["G"]
    N, T, dev = len(lens), s["q"].shape[0], s["q"].device
    L = max(CHUNK, -(-max(lens) // CHUNK) * CHUNK)
    cu = s["cu"] if s["cu"] is not None else torch.arange(N + 1, device=dev) * lens[0]
    n = cu[1:] - cu[:-1]
    at = torch.arange(L, device=dev)
    valid = at[None, :] < n[:, None]
    forth = (cu[:-1, None] + at).clamp(max=max(T - 1, 0))
    back = (cu[1:, None] - 1 - at).clamp(min=0)
    g = s["log_decay"]
    zero = torch.zeros(N, H, DIM, DIM, device=dev)
    h0 = s["h0"] if s["h0"] is not None else zero

    def rows(x, index):
        x = x.float()
        if x.shape[1] != H:
            x = x.repeat_interleave(G, dim=1)
        return torch.where(valid[:, :, None, None], x[index], torch.zeros((), device=dev)).transpose(1, 2)

    def flat(x, index):
        out = torch.empty(T, H, DIM, device=dev)
        out[index[valid]] = x.transpose(1, 2)[valid]
        return out

    q, k, v = (rows(s[x], forth) for x in ("q", "k", "v"))
    whole = torch.exp(g.view(1, H, 1, 1) * n.view(N, 1, 1, 1).float())
    if not backward:
        o, last = _decayed(q, k, v, g, h0, 1, n)
        return {"o": (SCALE * flat(o, forth)).bfloat16(), "hT": whole * h0 + last}
    do = rows(s["do"], forth)
    dq = SCALE * flat(_decayed(do, v, k, g, h0.transpose(-1, -2), 1, n)[0], forth)
    q, k, v, do = (rows(s[x], back) for x in ("q", "k", "v", "do"))
    dhT = s["dhT"] if s["dhT"] is not None else zero
    dk = flat(_decayed(v, do, SCALE * q, g, dhT.transpose(-1, -2), 0, n)[0], back)
    dv, last = _decayed(k, q, SCALE * do, g, dhT, 0, n)
    if G > 1:
        dq, dk = (x.view(T, H // G, G, DIM).sum(2) for x in (dq, dk))
    return {"dq": dq.bfloat16(), "dk": dk.bfloat16(), "dv": flat(dv, back).bfloat16(),
            "dh0": whole * dhT + torch.exp(g).view(1, H, 1, 1) * last}


def _plain(s):
    op = s["case"]["op"]
    if op in ("linattn_fwd", "linattn_bwd"):
        return _plain_linattn(s, op == "linattn_bwd")
    if op == "linattn_decode":
        G = s["case"]["G"]
        q, k = (s[x].float().repeat_interleave(G, dim=1) for x in ("q", "k"))
        state = s["state"]
        state.mul_(torch.exp(s["log_decay"]).view(1, -1, 1, 1)).add_(s["v"].float()[..., :, None] * k[..., None, :])
        return {"o": (SCALE * (state @ q[..., None])[..., 0]).bfloat16(), "state": state}
    x, w = s["x"].float(), s["weight"]
    if op == "layernorm_fwd":
        mean = x.mean(1, keepdim=True)
        rstd = torch.rsqrt((x - mean).square().mean(1, keepdim=True) + EPS)
        y = (x - mean) * rstd * w + s["bias"]
        return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    dy, mean, rstd = s["dy"].float(), s["mean"][:, None], s["rstd"][:, None]
    h = (x - mean) * rstd
    a = dy * w
    dx = rstd * (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * h).sum(0), "dbias": dy.sum(0)}


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------------- the work
def work(case):
    op = case["op"]
    if op == "linattn_decode":
        n, H, Hqk = case["requests"], case["H"], case["H"] // case["G"]
        return {"bytes": n * (H * (2 * DIM * DIM * 4 + 2 * DIM * 2) + Hqk * 2 * DIM * 2) + 4 * H, "flops": n * H * 5 * DIM * DIM}
    if op in ("linattn_fwd", "linattn_bwd"):
        lens, H, Hqk = _lens(case), case["H"], case["H"] // case["G"]
        T, states = sum(lens), len(lens) * H * DIM * DIM * 4
        if op == "linattn_fwd":
            return {"bytes": T * (2 * Hqk + 2 * H) * DIM * 2 + states * (2 if case["states"] else 1) + 4 * H,
                    "flops": T * H * 4 * DIM * DIM}
        return {"bytes": T * (4 * Hqk + 3 * H) * DIM * 2 + states * (3 if case["states"] else 1) + 4 * H,
                "flops": T * H * 10 * DIM * DIM}
    size = case["rows"] * case["width"]
    e = 2 if case["dtype"] == "bfloat16" else 4
    if op == "layernorm_fwd":
        return {"bytes": 2 * size * e + 8 * case["width"] + 8 * case["rows"], "flops": 8 * size}
    return {"bytes": 3 * size * e + 12 * case["width"] + 8 * case["rows"], "flops": 14 * size}


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """From the definitions: the recurrence over single tokens, and the norm's derivative written out for its statistics."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "linattn_decode":
        heads = torch.arange(case["H"], device="cuda") // case["G"]
        S = s.pop("state").double() * torch.exp(s["log_decay"].double())[None, :, None, None]
        S += torch.einsum("nhv,nhk->nhvk", s["v"].double(), s["k"].double()[:, heads])
        return {"o": SCALE * torch.einsum("nhvk,nhk->nhv", S, s["q"].double()[:, heads]), "state": S}
    if op in ("linattn_fwd", "linattn_bwd"):
        return _recurrence(s, op == "linattn_bwd")
    x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
    d = x.shape[1]
    var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
    sigma = torch.sqrt(var + EPS)
    if op == "layernorm_fwd":
        return {"y": torch.addcmul(b, (x - mean) / sigma, w), "mean": mean[:, 0], "rstd": 1 / sigma[:, 0]}
    dy = s["dy"].double()
    xc = x - mean
    dweight, dbias = torch.einsum("rc,rc->c", dy, xc / sigma), dy.sum(0)
    gw = dy * w                                             # y = xc / sigma: through xc, then through sigma
    dsigma = -(gw * xc).sum(1, keepdim=True) / sigma ** 2
    dxc = gw / sigma + dsigma * xc / (sigma * d)
    return {"dx": dxc - dxc.sum(1, keepdim=True) / d, "dweight": dweight, "dbias": dbias}


def _recurrence(s, backward):
    lens, H, G = s["lens"], s["case"]["H"], s["case"]["G"]
    N, T = len(lens), s["q"].shape[0]
    if max(lens) * N * H > 4 * 786432:
        return None
    heads = torch.arange(H, device="cuda") // G
    gamma = torch.exp(s["log_decay"].double()).view(1, H, 1, 1)
    start = [sum(lens[:n]) for n in range(N)]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    do = s["do"].double() if backward else None
    by_length = sorted(range(N), key=lambda n: -lens[n])
    first = torch.tensor([start[n] for n in by_length], device="cuda")
    order = torch.tensor(by_length, device="cuda")

    def state(x):
        return x.double()[order] if x is not None else torch.zeros(N, H, DIM, DIM, dtype=torch.float64, device="cuda")

    def outer_into(S, a, b):            # S += a b^T
        S.view(-1, DIM, DIM).baddbmm_(a.reshape(-1, DIM, 1), b.reshape(-1, 1, DIM))

    def times(S, a):
        return torch.bmm(S.view(-1, DIM, DIM), a.reshape(-1, DIM, 1)).view(-1, H, DIM)

    S, steps = state(s["h0"]), max(lens)
    active = [sum(1 for x in lens if x > t) for t in range(steps)]
    out = torch.empty(T, H, DIM, dtype=torch.float64, device="cuda")
    for t in range(steps):
        a = active[t]
        row, St = first[:a] + t, S[:a]
        St.mul_(gamma)
        outer_into(St, v[row], k[row][:, heads])
        out[row] = times(St.transpose(-1, -2).contiguous(), do[row]) if backward else times(St, q[row][:, heads])
    if not backward:
        hT = torch.empty_like(S)
        hT[order] = S
        return {"o": SCALE * out, "hT": hT}
    dq = (SCALE * out).view(T, H // G, G, DIM).sum(2)
    R = state(s["dhT"])
    dk, dv = torch.empty_like(out), torch.empty_like(out)
    for t in reversed(range(steps)):
        a = active[t]
        row, Rt = first[:a] + t, R[:a]
        outer_into(Rt, SCALE * do[row], q[row][:, heads])       # the adjoint of the state after token t
        dv[row] = times(Rt, k[row][:, heads])
        dk[row] = times(Rt.transpose(-1, -2).contiguous(), v[row])
        Rt.mul_(gamma)
    dh0 = torch.empty_like(R)
    dh0[order] = R
    return {"dq": dq, "dk": dk.view(T, H // G, G, DIM).sum(2), "dv": dv, "dh0": dh0}
