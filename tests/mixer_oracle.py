"""The gated recurrence over channels and the norm of queries and keys with the position rotation in 64 bits, on
the CPU, from their formulas, with a running bound of what arithmetic in 32 bits may be off by.

The bounds. E = 2^-24, half a step of fp32. A gate sigmoid(z) comes from an exponential of a rounded product (relative error
at most 2 |z| E), two roundings and a reciprocal: within (4 |z| + 8) E. u = exp(A_log) sigmoid(g) so is within kappa =
(4 |g| + 4 |A_log| + 4 |i| + 64) E of its value, with room for a sum of up to 32 of them; 1 - a of it at most as much (its
derivative times u over itself is at most 1) plus the two bits that 1 - exp(-u) may lose above u = 1/4, m half of that, the
product m i x the sum. A step of the recurrence adds these to what came before and rounds, at most 4 E of the states
it reads and writes:
    bound_t = a bound_{t-1} + kappa (em |h_{t-1}| + |b_t|) + 4 E (|h_{t-1}| + |h_t|) + tiny_t
tiny: a sigmoid below fp32's range (2^-126) counts as 0 or as 2^-126, so that m is off by sqrt(2 exp(A_log) 2^-126) there.
A state that is put together from a piece's own sum and a decay exp(-sum u) times what came before it has the errors of the
steps that it stands for, in another order. The adjoint G has the same recurrence backwards."""
import torch

E = 2.0 ** -24
HALF = {torch.float32: E, torch.bfloat16: 2.0 ** -8}      # the outputs' own rounding


def sequences(lens):
    t = 0
    for n, length in enumerate(lens):
        yield n, t, t + length
        t += length


def recurrence(x, g, i, A_log, lens, h0=None, dy=None, dhT=None):
    """Outputs (and gradients where dy is given) as {name: (value, bound)}, in 64 bits."""
    x, g, i, A = (v.double().cpu() for v in (x, g, i, A_log))
    T, D = x.shape
    N = len(lens)
    h0 = torch.zeros(N, D, dtype=torch.float64) if h0 is None else h0.double().cpu()
    lam = torch.exp(A)
    s, si = torch.sigmoid(g), torch.sigmoid(i)
    cs, ci = torch.sigmoid(-g), torch.sigmoid(-i)      # 1 - s would lose everything where a gate is open
    u = lam * s
    em = -torch.expm1(-u)
    a = torch.exp(-u)
    m = torch.sqrt(-torch.expm1(-2 * u))
    b = m * si * x
    kappa = (4 * g.abs() + 4 * i.abs() + 4 * A.abs() + 64) * E
    tiny = 2.0 ** -62 * (1 + lam) * (1 + x.abs())
    h, before = torch.empty_like(x), torch.empty_like(x)
    eh, ebefore = torch.empty_like(x), torch.empty_like(x)
    hT, eT = h0.clone(), torch.zeros_like(h0)
    for n, first, last in sequences(lens):
        S, e = h0[n], torch.zeros(D, dtype=torch.float64)
        for t in range(first, last):
            before[t], ebefore[t] = S, e
            new = a[t] * S + b[t]
            e = a[t] * e + kappa[t] * (em[t] * S.abs() + b[t].abs()) + 4 * E * (S.abs() + new.abs()) + tiny[t]
            S = new
            h[t], eh[t] = S, e
        hT[n], eT[n] = S, e
    out = {"y": (h, eh), "hT": (hT, eT)}
    if dy is None:
        return out
    dy = dy.double().cpu()
    dhT = torch.zeros(N, D, dtype=torch.float64) if dhT is None else dhT.double().cpu()
    G, eG = torch.empty_like(x), torch.empty_like(x)
    dh0, e0 = dhT.clone(), torch.zeros_like(dhT)
    for n, first, last in sequences(lens):
        R, e = dhT[n], torch.zeros(D, dtype=torch.float64)
        for t in reversed(range(first, last)):
            new = R + dy[t]
            e = e + 2 * E * (R.abs() + new.abs())
            G[t], eG[t] = new, e
            R = a[t] * new
            e = a[t] * e + kappa[t] * em[t] * new.abs() + 4 * E * (new.abs() + R.abs())
        dh0[n], e0[n] = R, e
    ratio = torch.where(m > 0, u / m, torch.zeros_like(m))
    p, q = si * x * a * a * ratio, u * a * before
    duu = G * (p - q)
    # a^2 within 2 kappa em / a of its value: as an addition, since kappa em <= kappa
    eduu = eG * (p - q).abs() + G.abs() * (4 * kappa * (p.abs() + q.abs() + (si * x * ratio).abs() * em + u * em * before.abs()) +
                                           u * a * ebefore + tiny)
    dx, di = G * m * si, G * m * x * si * ci
    out.update(dx=(dx, eG * (m * si).abs() + 3 * kappa * dx.abs() + tiny * G.abs()),
               di_raw=(di, eG * (m * x * si * ci).abs() + 4 * kappa * di.abs() + tiny * G.abs()),
               dg_raw=(duu * cs, (eduu + 2 * kappa * duu.abs()) * cs),
               dA_log=(duu.sum(0), eduu.sum(0) + (T + 64) * E * duu.abs().sum(0)),
               dh0=(dh0, e0))
    return out


def check(name, got, ref):
    """got against (value, bound) within the bound and half a step of its type."""
    value, bound = ref
    got = got.detach().cpu()
    assert torch.isfinite(got).all(), name
    lim = bound + HALF[got.dtype] * (value.abs() + bound) + 1e-37
    off = ((got.double().reshape(value.shape) - value).abs() / lim).max().item() if value.numel() else 0.0
    assert off <= 1.0, (name, off)
    return off


# 1 / (2 pi) in 320 binary places
TURN = 0x28be60db9391054a7f09d5f47d4d377036d8a5664f10e4107f9458eaf7aef1586dc91b8e909374b8


def angles(positions, inv_freq):
    """position * inv_freq modulo 2 pi, in whole numbers up to the last step; [T, pairs]."""
    f = [float(v).as_integer_ratio() for v in inv_freq.cpu().tolist()]
    rows = []
    for p in positions.cpu().tolist():
        row = []
        for num, den in f:
            turns = (p * num * TURN // den) % (1 << 320)
            if turns >> 319:
                turns -= 1 << 320
            row.append(turns / (1 << 320) * 6.283185307179586)
        rows.append(row)
    return torch.tensor(rows, dtype=torch.float64).reshape(len(rows), len(f))


def turned(z, theta, interleaved):
    R = 2 * theta.shape[1]
    c, s = torch.cos(theta)[:, None], torch.sin(theta)[:, None]
    y = z.clone()
    ia = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    ib = ia + (1 if interleaved else R // 2)
    y[..., ia] = z[..., ia] * c - z[..., ib] * s
    y[..., ib] = z[..., ib] * c + z[..., ia] * s
    return y


def partner(x, R, interleaved):
    """Each rotated column's other one, itself elsewhere."""
    y = x.clone()
    ia = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    ib = ia + (1 if interleaved else R // 2)
    y[..., ia], y[..., ib] = x[..., ib], x[..., ia]
    return y


def qknorm(x, w, theta, interleaved, eps, dy=None):
    """One side, {name: (value, bound)}. A row's sum of squares has at most 8 + 5 dependent roundings, its root and reciprocal four:
    z is within 16 E; a sine or cosine within 8 E (the angle's own rounding, pi E, and two steps), so a rotated column within
    32 E of its two sides' magnitudes. The gradient has the two means besides, of magnitudes."""
    x = x.double().cpu()
    head, R = x.shape[-1], 2 * theta.shape[1]
    w = torch.ones(head, dtype=torch.float64) if w is None else w.double().cpu()
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    z = x * r * w
    if dy is None:
        size = z.abs() + (partner(z, R, interleaved).abs() if R else 0.0)
        return {"y": (turned(z, theta, interleaved), 32 * E * size)}
    dy = dy.double().cpu()
    g = turned(dy, -theta, interleaved)
    size = dy.abs() + (partner(dy, R, interleaved).abs() if R else 0.0)
    xh = x * r
    dx = r * (g * w - xh * (g * w * xh).mean(-1, keepdim=True))
    edx = 64 * E * r * (size * w.abs() + xh.abs() * (size * w.abs() * xh.abs()).mean(-1, keepdim=True))
    rows = x.shape[0] * x.shape[1]
    return {"dx": (dx, edx), "dw": ((g * xh).sum((0, 1)), (rows + 96) * E * (size * xh.abs()).sum((0, 1)))}
