"""Cases of the gated recurrence over channels and of the norm of queries and keys with the position rotation.

Operators (tokens [T, D] or [T, H, head], bf16 or fp32; packed sequences through int64 offsets; parameters and states fp32):

  recurrence_fwd     u_t = exp(A_log) sigmoid(g_raw_t), a_t = exp(-u_t)
                     h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_raw_t) x_t for each channel; y_t = h_t and the final states
  recurrence_bwd     gradients of sum_t <y_t, dy_t> + <hT, dhT> with respect to x, g_raw, i_raw, A_log and the initial state
  recurrence_decode  one token for each request, the state updated in place
  qknorm_fwd         each head of q and k divided by its root mean square, times a weight, its first columns rotated by the
                     angles position * inv_freq
  qknorm_bwd         gradients with respect to q, k and both weights

``run`` computes them in elementary torch operations in 32 bits where ``own`` is false, and calls the framework where it
is true. ``exact`` follows the definitions in 64 bits, token by token, and by complex numbers and their derivatives.
"""
import math

import torch

own = False

DIM = 128
BLOCK = 64      # the forward pass of the recurrence keeps the state before every 64th token for the backward pass
EPS = 1e-6
MOST = 8192 * 12288


def listed():
    return [
        # a short packed batch of three sequences over a width of 4 x 128: latency, lengths around the block sizes
        {"name": "rec_fwd_packed_17_33_65_D512", "op": "recurrence_fwd", "lens": "17,33,65", "B": 1, "D": 512, "fused": False,
         "states": True, "dtype": "bfloat16"},
        # a packed batch of six ragged prompts at a width of 32 x 128, its three inputs the columns of one projection,
        # states carried in and out
        {"name": "rec_fwd_packed6_D4096", "op": "recurrence_fwd", "lens": "1300,547,2048,963,271,3063", "B": 1, "D": 4096,
         "fused": True, "states": True, "dtype": "bfloat16"},
        # the largest training step, at a width of 96 x 128
        {"name": "rec_fwd_T8192_D12288", "op": "recurrence_fwd", "lens": "8192", "B": 1, "D": 12288, "fused": False,
         "states": False, "dtype": "bfloat16"},
        # the backward pass of the short packed batch
        {"name": "rec_bwd_packed_17_33_65_D512", "op": "recurrence_bwd", "lens": "17,33,65", "B": 1, "D": 512, "fused": False,
         "states": True, "dtype": "bfloat16"},
        # the backward pass over one very long sequence of few channels in 32 bits, an odd number of tokens
        {"name": "rec_bwd_T65537_D256_fp32", "op": "recurrence_bwd", "lens": "65537", "B": 1, "D": 256, "fused": False,
         "states": False, "dtype": "float32"},
        # the backward pass of the largest training step, gradients into the columns of one buffer
        {"name": "rec_bwd_T8192_D12288", "op": "recurrence_bwd", "lens": "8192", "B": 1, "D": 12288, "fused": True,
         "states": False, "dtype": "bfloat16"},
        # decoding a few requests of a small model: latency
        {"name": "rec_decode_4req_D512", "op": "recurrence_decode", "requests": 4, "D": 512, "dtype": "bfloat16"},
        # decoding a full serving batch
        {"name": "rec_decode_256req_D12288", "op": "recurrence_decode", "requests": 256, "D": 12288, "dtype": "bfloat16"},
        # queries and keys of one token for each of 64 requests, far positions, four query heads to a key head
        {"name": "qk_fwd_64req_H32_G4", "op": "qknorm_fwd", "T": 64, "H": 32, "G": 4, "head": DIM, "rotary": DIM,
         "interleaved": False, "fused": True, "dtype": "bfloat16"},
        # the queries and keys of the largest training step, read out of one projection of queries, keys and values
        {"name": "qk_fwd_T8192_H96", "op": "qknorm_fwd", "T": 8192, "H": 96, "G": 1, "head": DIM, "rotary": DIM,
         "interleaved": False, "fused": True, "dtype": "bfloat16"},
        # the backward pass in 32 bits at an odd number of tokens, half of each head rotated, neighbours paired
        {"name": "qk_bwd_T4099_H32_G4_half_fp32", "op": "qknorm_bwd", "T": 4099, "H": 32, "G": 4, "head": DIM, "rotary": 64,
         "interleaved": True, "fused": False, "dtype": "float32"},
        # the backward pass of the largest training step, gradients into the columns of one buffer
        {"name": "qk_bwd_T8192_H96", "op": "qknorm_bwd", "T": 8192, "H": 96, "G": 1, "head": DIM, "rotary": DIM,
         "interleaved": False, "fused": True, "dtype": "bfloat16"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["recurrence_fwd", "recurrence_fwd", "recurrence_bwd", "recurrence_bwd", "recurrence_decode", "qknorm_fwd",
                     "qknorm_bwd"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    fused = rng.random() < 0.5
    most = MOST // (2 if dtype == "float32" else 1)
    if op == "recurrence_decode":
        D = rng.choice([DIM * _spread(rng, 1, 96), _spread(rng, 8, 12288)])
        return {"op": op, "requests": _spread(rng, 1, 256), "D": D, "dtype": dtype}
    if op in ("recurrence_fwd", "recurrence_bwd"):
        D = rng.choice([DIM * _spread(rng, 1, 96), DIM * _spread(rng, 1, 96), _spread(rng, 8, 12288)])
        T = _spread(rng, 1, min(65537, most // D))
        kind = rng.choice(["one", "batch", "packed"])
        B, lens = 1, [T]
        if kind == "batch":
            B = rng.randint(1, 4)
            lens = [max(1, T // B)]
        elif kind == "packed":
            n = rng.randint(2, 40)
            cuts = sorted(rng.randint(0, T) for _ in range(n - 1))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [T])]      # empty sequences among them
        return {"op": op, "lens": ",".join(map(str, lens)), "B": B, "D": D, "fused": fused, "states": rng.random() < 0.5,
                "dtype": dtype}
    head = rng.choice([DIM, DIM, 64, 256, 8 * rng.randint(2, 32)])
    rotary = rng.choice([head, head, head // 16 * 8, 0])
    G = rng.choice([1, 2, 4, 8])
    H = G * _spread(rng, 1, 96 // G)
    T = _spread(rng, 1, min(32768, 2 * most // ((H + H // G) * head)))
    return {"op": op, "T": T, "H": H, "G": G, "head": head, "rotary": rotary, "interleaved": rng.random() < 0.5, "fused": fused,
            "dtype": dtype}


def _lens(case):
    return [int(x) for x in case["lens"].split(",")] * (case["B"] if "," not in case["lens"] else 1)


def _columns(fused, *parts):
    """The tensors as they are, or as columns of one buffer of rows."""
    if not fused:
        return parts
    rows = parts[0].shape[0]
    whole = torch.cat([p.reshape(rows, -1) for p in parts], 1)
    return tuple(c.view(p.shape) if p.dim() == 2 else c.unflatten(1, p.shape[1:])
                 for c, p in zip(whole.split([p[0].numel() if rows else 0 for p in parts], 1), parts))


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dtype = getattr(torch, case["dtype"])

    def normal(*shape, dtype=dtype, std=1.0, mean=0.0):
        return (mean + std * torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)).to(dtype)

    op = case["op"]
    s = {"case": case}
    if op.startswith("recurrence"):
        D = case["D"]
        # decays of an open gate from 0.9^8 to 0.999^8 a token, as such layers start with
        s["A_log"] = torch.log(-8.0 * torch.log(0.9 + 0.099 * torch.rand(D, generator=gen, device=dev)))
        if op == "recurrence_decode":
            n = case["requests"]
            s.update(x=normal(n, D), g_raw=normal(n, D), i_raw=normal(n, D), state=normal(n, D, dtype=torch.float32))
            return s
        lens = _lens(case)
        T, N = sum(lens), len(lens)
        s["x"], s["g_raw"], s["i_raw"] = _columns(case["fused"], normal(T, D), normal(T, D), normal(T, D))
        s.update(lens=lens, cu=None, h0=None, dhT=None)
        if "," in case["lens"]:
            s["cu"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int64, device=dev)
        if case["states"]:
            s["h0"] = normal(N, D, dtype=torch.float32)
        if op == "recurrence_bwd":
            s["dy"] = normal(T, D)
            if case["states"]:
                s["dhT"] = normal(N, D, dtype=torch.float32)
            # what the forward pass left: the state before every 64th token
            s["kept"] = torch.zeros(-(-T // BLOCK), D, device=dev)
            h = _plain_scan(s)
            s["kept"][1:] = h[BLOCK - 1:T - 1:BLOCK]
            if case["fused"]:
                s["grads"] = dict(zip(("dx", "dg_raw", "di_raw"), torch.empty(T, 3 * D, device=dev, dtype=dtype).split(D, 1)))
                s["grads"].update(dA_log=torch.empty(D, device=dev),
                                  dh0=torch.empty(N, D, device=dev))
        return s
    T, H, Hk, head, rotary = case["T"], case["H"], case["H"] // case["G"], case["head"], case["rotary"]
    # heads of different size, as projections give them
    q, k = (normal(T, n, head) * torch.exp(normal(1, n, 1, std=0.5)) for n in (H, Hk))
    s["q"], s["k"], _ = _columns(case["fused"], q, k, normal(T, Hk, head))
    s["q_weight"], s["k_weight"] = (normal(head, dtype=torch.float32, std=0.1, mean=1.0) for _ in range(2))
    # positions of packed prompts, or of requests that are anywhere in a long context
    s["positions"] = torch.randint(0, 1 << 20, (T,), generator=gen, device=dev) if T <= 256 else \
        torch.arange(T, device=dev) % max(1, T // 3)
    s["inv_freq"] = 10000.0 ** (-torch.arange(0, rotary, 2, device=dev, dtype=torch.float32) / max(1, rotary))
    if op == "qknorm_bwd":
        s["dq_out"], s["dk_out"] = normal(T, H, head), normal(T, Hk, head)
        if case["fused"]:
            flat = torch.empty(T, (H + 2 * Hk) * head, device=dev, dtype=dtype)
            s["grads"] = {"dq": flat[:, :H * head].unflatten(1, (H, head)),
                          "dk": flat[:, H * head:(H + Hk) * head].unflatten(1, (Hk, head)),
                          "dq_weight": torch.empty(head, device=dev), "dk_weight": torch.empty(head, device=dev)}
    return s


# ------------------------------------------------------------------ the framework's operators
def _framework(s):
    from kimi_delta_attention_15_gb300 import ops
    op = s["case"]["op"]
    if op == "recurrence_fwd":
        y, hT, _, s["workspace"] = ops.recurrence_fwd(s["x"], s["g_raw"], s["i_raw"], s["A_log"], h0=s["h0"],
                                                      cu_seqlens=s["cu"], B=s["case"]["B"], workspace=s.get("workspace"))
        return {"y": y, "hT": hT}
    if op == "recurrence_bwd":
        if "workspace" not in s:
            s["workspace"] = ops.recurrence_alloc_workspace(ops.recurrence_shape(
                s["x"].shape[0] // s["case"]["B"], s["case"]["D"], len(s["lens"]), s["case"]["B"]), s["x"].device, backward=True)
        return ops.recurrence_bwd(s["x"], s["g_raw"], s["i_raw"], s["A_log"], s["dy"], s["kept"], s["workspace"], h0=s["h0"],
                                  cu_seqlens=s["cu"], dhT=s["dhT"], B=s["case"]["B"], grads=s.get("grads"))
    if op == "recurrence_decode":
        y = ops.recurrence_decode(s["x"], s["g_raw"], s["i_raw"], s["A_log"], s["state"])
        return {"y": y, "state": s["state"]}
    rotation = dict(eps=EPS, interleaved=s["case"]["interleaved"])
    if op == "qknorm_fwd":
        q, k = ops.qknorm_fwd(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"], **rotation)
        return {"q": q, "k": k}
    return ops.qknorm_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"],
                          grads=s.get("grads"), **rotation)


# ------------------------------------------------------------------------- the plain forms
def _gates(x, g_raw, i_raw, A_log):
    u = torch.exp(A_log) * torch.sigmoid(g_raw.float())
    em = -torch.expm1(-u)                       # 1 - a
    return u, em, torch.sqrt(em * (2.0 - em)), torch.sigmoid(i_raw.float()) * x.float()


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the first dimension, from zero: within pieces of about sqrt(T) tokens, all pieces
    at once, then from piece to piece."""
    T, D = a.shape
    L = max(1, math.isqrt(T))
    C = -(-T // L)
    pad = C * L - T
    if pad:
        a = torch.cat([a, torch.ones(pad, D, device=a.device)])
        b = torch.cat([b, torch.zeros(pad, D, device=a.device)])
    a, h = a.view(C, L, D).clone(), b.view(C, L, D).clone()
    for t in range(1, L):
        h[:, t] += a[:, t] * h[:, t - 1]
        a[:, t] *= a[:, t - 1]
    for c in range(1, C):
        h[c] += a[c] * h[c - 1, -1]
    return h.view(C * L, D)[:T]


def _bounds(s):
    """First and last tokens of the sequences that have tokens, and which sequences these are."""
    cu = s["cu"] if s["cu"] is not None else torch.arange(len(s["lens"]) + 1, device=s["x"].device) * s["lens"][0]
    some = torch.tensor([n for n, length in enumerate(s["lens"]) if length], dtype=torch.int64, device=cu.device)
    return cu[:-1][some], cu[1:][some] - 1, some


def _plain_scan(s):
    u, em, m, ix = _gates(s["x"], s["g_raw"], s["i_raw"], s["A_log"])
    a, b = 1.0 - em, m * ix
    first, _, some = _bounds(s)
    if s["h0"] is not None:
        b[first] += a[first] * s["h0"][some]
    a[first] = 0.0
    return _scan(a, b)


def _plain_recurrence(s, backward):
    N, D, dev = len(s["lens"]), s["case"]["D"], s["x"].device
    zero = torch.zeros(N, D, device=dev)
    h0 = s["h0"] if s["h0"] is not None else zero
    h = _plain_scan(s)
    first, last, some = _bounds(s)
    if not backward:
        hT = h0.clone()
        hT[some] = h[last]
        return {"y": h.to(s["x"].dtype), "hT": hT}
    u, em, m, ix = _gates(s["x"], s["g_raw"], s["i_raw"], s["A_log"])
    a = 1.0 - em
    before = torch.cat([zero[:1], h[:-1]])
    before[first] = h0[some]
    dhT = s["dhT"] if s["dhT"] is not None else zero
    dy = s["dy"].float()
    dy[last] += dhT[some]
    after = torch.cat([a[1:], zero[:1]])
    after[last] = 0.0
    G = _scan(after.flip(0), dy.flip(0)).flip(0)
    i = torch.sigmoid(s["i_raw"].float())
    dix = G * m
    ratio = torch.where(m > 0, u / m, torch.zeros((), device=dev))
    duu = G * (ix * a * a * ratio - u * a * before)
    dh0 = dhT.clone()
    dh0[some] = a[first] * G[first]
    to = s["x"].dtype
    return {"dx": (dix * i).to(to), "dg_raw": (duu * torch.sigmoid(-s["g_raw"].float())).to(to),
            "di_raw": (dix * ix * torch.sigmoid(-s["i_raw"].float())).to(to), "dA_log": duu.sum(0), "dh0": dh0}


def _rotated(x, cos, sin, interleaved):
    """The first columns of each head in pairs, each turned by its angle; [T, H, head] by [T, pairs]."""
    pairs = cos.shape[1]
    front, rest = x[..., :2 * pairs], x[..., 2 * pairs:]
    a, b = (front[..., 0::2], front[..., 1::2]) if interleaved else (front[..., :pairs], front[..., pairs:])
    cos, sin = cos[:, None], sin[:, None]
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1), rest], -1)


def _plain_qknorm(s, backward):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    interleaved = s["case"]["interleaved"]
    out = {}
    for name in ("q", "k"):
        x, w = s[name].float(), s[name + "_weight"]
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        if not backward:
            out[name] = _rotated(x * r * w, cos, sin, interleaved).to(s[name].dtype)
            continue
        g = _rotated(s["d" + name + "_out"].float(), cos, -sin, interleaved)
        xh = x * r
        gw = g * w
        out["d" + name] = (r * (gw - xh * (gw * xh).mean(-1, keepdim=True))).to(s[name].dtype)
        out["d" + name + "_weight"] = (g * xh).sum((0, 1))
    return out


def _plain(s):
    op = s["case"]["op"]
    if op in ("recurrence_fwd", "recurrence_bwd"):
        return _plain_recurrence(s, op == "recurrence_bwd")
    if op == "recurrence_decode":
        u, em, m, ix = _gates(s["x"], s["g_raw"], s["i_raw"], s["A_log"])
        state = s["state"]
        state.mul_(1.0 - em).add_(m * ix)
        return {"y": state.to(s["x"].dtype), "state": state}
    return _plain_qknorm(s, op == "qknorm_bwd")


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------------- the work
def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == "bfloat16" else 4
    if op == "recurrence_decode":
        n = case["requests"] * case["D"]
        return {"bytes": n * (4 * e + 8) + 4 * case["D"], "flops": 20 * n}
    if op in ("recurrence_fwd", "recurrence_bwd"):
        lens, D = _lens(case), case["D"]
        n, states = sum(lens) * D, len(lens) * D * 4
        if op == "recurrence_fwd":
            return {"bytes": n * 4 * e + states * (2 if case["states"] else 1) + 4 * D, "flops": 20 * n}
        kept = -(-sum(lens) // BLOCK) * D * 4
        return {"bytes": n * 7 * e + kept + states * (3 if case["states"] else 1) + 8 * D, "flops": 45 * n}
    T, H, Hk, head, rotary = case["T"], case["H"], case["H"] // case["G"], case["head"], case["rotary"]
    n = T * (H + Hk) * head
    small = 8 * T + 2 * rotary
    if op == "qknorm_fwd":
        return {"bytes": 2 * n * e + small + 8 * head, "flops": 7 * n}
    return {"bytes": 3 * n * e + small + 16 * head, "flops": 16 * n}


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("qknorm"):
        return _exact_qknorm(s, op == "qknorm_bwd")
    lam = torch.exp(s["A_log"].double())
    if op == "recurrence_decode":
        log_a = -lam / (1 + torch.exp(-s["g_raw"].double()))
        state = torch.exp(log_a) * s["state"].double() + \
            torch.sqrt(-torch.expm1(2 * log_a)) * s["x"].double() / (1 + torch.exp(-s["i_raw"].double()))
        return {"y": state, "state": state}
    return _exact_recurrence(s, lam, op == "recurrence_bwd")


def _exact_recurrence(s, lam, backward):
    """Token by token, every sequence's own loop taken together, longest first."""
    lens, D = s["lens"], s["case"]["D"]
    N, T = len(lens), sum(lens)
    by_length = sorted(range(N), key=lambda n: -lens[n])
    order = torch.tensor(by_length, device="cuda")
    first = torch.tensor([sum(lens[:n]) for n in by_length], device="cuda")
    steps = max(lens)
    active = [0] * steps
    for length in lens:
        if length:
            active[length - 1] += 1
    for t in reversed(range(steps - 1)):
        active[t] += active[t + 1]

    def state(x):
        return x.double()[order] if x is not None else torch.zeros(N, D, dtype=torch.float64, device="cuda")

    log_a = -lam / (1 + torch.exp(-s["g_raw"].double()))
    a, r = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a))
    gate = 1 / (1 + torch.exp(-s["i_raw"].double()))
    x = s["x"].double()
    add = r * gate * x
    S = state(s["h0"])
    out = torch.empty(T, D, dtype=torch.float64, device="cuda")     # the states after, or before where backward
    for t in range(steps):
        n = active[t]
        row, St = first[:n] + t, S[:n]
        if backward:
            out[row] = St
        St.mul_(a[row]).add_(add[row])
        if not backward:
            out[row] = St
    if not backward:
        hT = torch.empty_like(S)
        hT[order] = S
        return {"y": out, "hT": hT}
    del add
    R = state(s["dhT"])
    dy = s["dy"].double()
    adj = torch.empty_like(out)                                     # the adjoint of the state after each token
    for t in reversed(range(steps)):
        n = active[t]
        row, Rt = first[:n] + t, R[:n]
        Rt.add_(dy[row])
        adj[row] = Rt
        Rt.mul_(a[row])
    del dy
    dh0 = torch.empty_like(R)
    dh0[order] = R
    # through log a: a itself, and r with dr / dlog a = -a^2 / r
    # where a gate is closed so far that r is 0 in 64 bits, that term's limit with the gate's own slope is 0
    dlog = adj * a * out - torch.where(r > 0, adj * gate * x * a * a / r, torch.zeros((), dtype=torch.float64, device="cuda"))
    dg = dlog * log_a / (1 + torch.exp(s["g_raw"].double()))        # dlog a / dg_raw = log a (1 - sigmoid)
    return {"dx": adj * r * gate, "dg_raw": dg, "di_raw": adj * r * x * gate * (1 - gate), "dA_log": (dlog * log_a).sum(0),
            "dh0": dh0}


def _exact_qknorm(s, backward):
    """The pairs as complex numbers times exp(i angle); gradients by the chain rule of torch in 64 bits."""
    case = s["case"]
    R, T = case["rotary"], case["T"]
    turn = torch.polar(torch.ones(T, 1, R // 2, dtype=torch.float64, device="cuda"),
                       (s["positions"].double()[:, None] * s["inv_freq"].double())[:, None])
    out = {}
    for name in ("q", "k"):
        x = s[name].detach().double().requires_grad_(backward)
        w = s[name + "_weight"].double().requires_grad_(backward)
        with torch.set_grad_enabled(backward):
            z = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
            f = z[..., :R]
            f = f.unflatten(-1, (R // 2, 2)) if case["interleaved"] else f.unflatten(-1, (2, R // 2)).transpose(-1, -2)
            f = torch.complex(f[..., 0], f[..., 1]) * turn
            f = torch.stack([f.real, f.imag], -1)
            f = f if case["interleaved"] else f.transpose(-1, -2)
            y = torch.cat([f.flatten(-2), z[..., R:]], -1)
        if not backward:
            out[name] = y
        else:
            out["d" + name], out["d" + name + "_weight"] = torch.autograd.grad(y, (x, w), s["d" + name + "_out"].double())
    return out
