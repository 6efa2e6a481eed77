"""Layer norm on the GPU against its formula in 64 bits.

Tolerances, from the number formats: a statistic is a sum of at most a few hundred dependent fp32
roundings (the rest runs in parallel lanes), taken as 256 units of e = 2^-24 of the sum of
magnitudes at worst and far fewer in the mean. y: e times 64 times (1 + |mean| / sigma), the second
term from the mean's own rounding; bf16 (8 significant bits) adds u = 2^-8 of the value. dweight, dbias: rows + 64
roundings of the sum of magnitudes, true of any order of summation."""
import pytest
import torch

import linattn_oracle as O
from kimi_delta_attention_15_gb300 import ops

pytestmark = pytest.mark.gpu
E, U = 2.0 ** -24, 2.0 ** -8
EPS = 1e-5


def make(rows, width, dtype, seed=0, offset=0.3):
    g = torch.Generator().manual_seed(seed + rows + width)
    level = torch.exp(0.5 * torch.randn(rows, 1, generator=g))
    x = (level * (torch.randn(rows, width, generator=g) + offset)).to(dtype)
    dy = torch.randn(rows, width, generator=g).to(dtype)
    w = 1.0 + 0.1 * torch.randn(width, generator=g)
    b = 0.1 * torch.randn(width, generator=g)
    return x, dy, w, b


def check_forward(x, w, b, eps=EPS):
    y, mean, rstd = ops.layernorm_fwd(x.cuda(), None if w is None else w.cuda(), None if b is None else b.cuda(), eps=eps)
    torch.cuda.synchronize()
    flat = x.reshape(-1, x.shape[-1])
    ref = O.norm_forward(flat, w, b, eps)
    mu, rs = ref["mean"].abs()[:, None], ref["rstd"][:, None]
    size = flat.double().abs().mean(1)
    assert ((mean.double().cpu() - ref["mean"]).abs() <= 64 * E * size).all()
    assert ((rstd.double().cpu() - ref["rstd"]).abs() <= 64 * E * (1 + mu * rs)[:, 0] * ref["rstd"]).all()
    got = y.double().cpu().reshape(flat.shape)
    h = ((flat.double() - ref["mean"][:, None]) * rs).abs()
    lim = 64 * E * (1 + mu * rs) * (1 + h) * (w.double().abs() if w is not None else 1.0) + 4 * E * ref["y"].abs() + \
        4 * E * (b.double().abs() if b is not None else 0.0)
    if x.dtype == torch.bfloat16:
        lim = lim * (1 + U) + U * ref["y"].abs()
    assert ((got - ref["y"]).abs() <= lim).all(), ((got - ref["y"]).abs() / lim).max()
    assert y.dtype == x.dtype and y.shape == x.shape
    return y, mean, rstd


def check_backward(x, dy, w, mean, rstd):
    g = ops.layernorm_bwd(x.cuda(), dy.cuda(), None if w is None else w.cuda(), mean, rstd)
    torch.cuda.synchronize()
    flat, fdy = x.reshape(-1, x.shape[-1]), dy.reshape(-1, x.shape[-1])
    ref = O.norm_backward(flat, fdy, w, mean.cpu(), rstd.cpu())
    rs = rstd.double().cpu()[:, None]
    h = (flat.double() - mean.double().cpu()[:, None]) * rs
    a = fdy.double() * (w.double() if w is not None else 1.0)
    # three terms, the two means sums of magnitudes
    size = rs * (a.abs() + a.abs().mean(1, keepdim=True) + h.abs() * (a * h).abs().mean(1, keepdim=True))
    lim = 64 * E * size
    if x.dtype == torch.bfloat16:
        lim = lim * (1 + U) + U * ref["dx"].abs()
    got = g["dx"].double().cpu().reshape(flat.shape)
    assert ((got - ref["dx"]).abs() <= lim).all(), ((got - ref["dx"]).abs() / lim).max()
    n = flat.shape[0] + 64
    assert ((g["dweight"].double().cpu() - ref["dweight"]).abs() <= n * E * (fdy.double() * h).abs().sum(0)).all()
    assert ((g["dbias"].double().cpu() - ref["dbias"]).abs() <= n * E * fdy.double().abs().sum(0)).all()
    return g


SIZES = [(1, 1), (3, 2), (1, 128), (5, 7), (33, 128), (1000, 128), (257, 256), (64, 512), (7, 1000), (19, 1024), (9, 1536),
         (5, 2048), (33, 4096), (6, 4104), (5, 5000), (3, 8192), (4, 12288), (2, 16384), (2, 16392), (2, 20001), (700, 33),
         (2000, 64), (3, 40960)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,width", SIZES)
def test_forward_and_backward(rows, width, dtype):
    x, dy, w, b = make(rows, width, dtype)
    _, mean, rstd = check_forward(x, w, b)
    check_backward(x, dy, w, mean, rstd)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", [128, 1000, 4097])
def test_without_weight_and_bias(width, dtype):
    x, dy, w, b = make(40, width, dtype, seed=1)
    _, mean, rstd = check_forward(x, None, None)
    check_backward(x, dy, None, mean, rstd)
    check_forward(x, w, None)
    check_forward(x, None, b)


def test_higher_dimensions():
    x, dy, w, b = make(6 * 5, 128, torch.bfloat16, seed=2)
    x, dy = x.view(6, 5, 128), dy.view(6, 5, 128)
    y, mean, rstd = check_forward(x, w, b)
    g = check_backward(x, dy, w, mean, rstd)
    assert g["dx"].shape == x.shape and mean.shape == (30,)


@pytest.mark.parametrize("offset", [100.0, -1000.0])
def test_a_mean_far_from_zero(offset):
    x, dy, w, b = make(20, 777, torch.float32, seed=3, offset=offset)
    _, mean, rstd = check_forward(x, w, b)
    check_backward(x, dy, w, mean, rstd)


def test_constant_rows():
    """No variance at all: rstd = 1 / sqrt(eps), y = bias."""
    x = torch.full((4, 256), 3.0)
    b = torch.randn(256, generator=torch.Generator().manual_seed(4))
    y, _, rstd = ops.layernorm_fwd(x.cuda(), torch.ones(256).cuda(), b.cuda(), eps=EPS)
    assert torch.allclose(y.cpu(), b.expand(4, 256), atol=1e-6)
    assert torch.allclose(rstd.cpu().double(), torch.full((4,), EPS, dtype=torch.float64).rsqrt(), rtol=1e-6)


def test_no_rows():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = ops.layernorm_fwd(x)
    assert y.shape == (0, 64)
    g = ops.layernorm_bwd(x, x, None, mean, rstd)
    assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()


def test_non_finite_rows_stay_alone():
    x, dy, w, b = make(9, 512, torch.float32, seed=5)
    x[4, 7], x[6, 0] = float("nan"), float("inf")
    y, mean, rstd = ops.layernorm_fwd(x.cuda(), w.cuda(), b.cuda())
    g = ops.layernorm_bwd(x.cuda(), dy.cuda(), w.cuda(), mean, rstd)
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.isfinite(y[keep]).all() and torch.isfinite(g["dx"][keep]).all()
    assert torch.isnan(y[4]).all() and torch.isnan(y[6]).all()


ODD = [(40, 1), (40, 3), (50, 5), (41, 9), (64, 17), (33, 65), (70, 131), (300, 201), (20, 333), (25, 501), (17, 607), (19, 1001),
       (9, 2049), (13, 4097), (12, 7777), (11, 9733), (10, 12289), (9, 16383)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,width", ODD)
def test_rows_that_start_anywhere(rows, width, dtype):
    """Widths that are no multiple of 16 bytes: rows share 16-byte units with their neighbours, of which nothing may
    leak in (rows of NaN and infinity change no other row's outputs) and nothing may be overwritten."""
    x, dy, w, b = make(rows, width, dtype, seed=width)
    _, mean, rstd = check_forward(x, w, b)
    check_backward(x, dy, w, mean, rstd)
    x, dy, w, b = x.cuda(), dy.cuda(), w.cuda(), b.cuda()
    y, mean, rstd = ops.layernorm_fwd(x, w, b)
    g = ops.layernorm_bwd(x, dy, w, mean, rstd)
    bad, dbad = x.clone(), dy.clone()
    bad[1], bad[rows // 2], bad[-1] = float("nan"), float("inf"), float("nan")
    dbad[1], dbad[rows // 2], dbad[-1] = float("inf"), float("nan"), float("nan")
    keep = [r for r in range(rows) if r not in (1, rows // 2, rows - 1)]
    pad = 64
    room = [torch.full((rows * width + 2 * pad,), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    out = [t[pad:-pad].view(rows, width) for t in room]
    y2, mean2, rstd2 = ops.layernorm_fwd(bad, w, b, y=out[0])
    ops.layernorm_bwd(bad, dbad, w, mean2, rstd2, grads=dict(dx=out[1]))
    assert torch.equal(y2[keep], y[keep]) and torch.equal(out[1][keep], g["dx"][keep])
    assert torch.equal(mean2[keep], mean[keep]) and torch.equal(rstd2[keep], rstd[keep])
    for t in room:
        assert (t[:pad] == 7).all() and (t[-pad:] == 7).all()


def test_gradients_not_wanted_and_guards():
    x, dy, w, b = (t.cuda() for t in make(50, 1000, torch.bfloat16, seed=6))
    _, mean, rstd = ops.layernorm_fwd(x, w, b)
    full = ops.layernorm_bwd(x, dy, w, mean, rstd)
    some = ops.layernorm_bwd(x, dy, w, mean, rstd, want_dweight=False)
    assert some["dweight"] is None and torch.equal(some["dx"], full["dx"]) and torch.equal(some["dbias"], full["dbias"])
    none = ops.layernorm_bwd(x, dy, w, mean, rstd, want_dweight=False, want_dbias=False)
    assert none["dbias"] is None and torch.equal(none["dx"], full["dx"])
    big = torch.full((66, 1000), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.layernorm_fwd(x, w, b, y=big[8:58])
    assert (big[:8] == 7).all() and (big[58:] == 7).all() and not (big[8:58] == 7).all()


@pytest.mark.parametrize("rows,width", [(3000, 128), (700, 4096), (400, 1001)])
def test_repeated_calls_agree_bit_for_bit(rows, width):
    x, dy, w, b = (t.cuda() for t in make(rows, width, torch.bfloat16, seed=7))
    outs = []
    for _ in range(2):
        y, mean, rstd = ops.layernorm_fwd(x, w, b)
        outs.append((y, mean, rstd, *ops.layernorm_bwd(x, dy, w, mean, rstd).values()))
    for a, c in zip(*outs):
        assert torch.equal(a, c)


def test_gradient_against_differences():
    """<dx, step> against the central difference of the 64-bit loss (fp32 input: errors of 64 e)."""
    x, dy, w, b = make(12, 300, torch.float32, seed=9)
    _, mean, rstd = ops.layernorm_fwd(x.cuda(), w.cuda(), b.cuda(), eps=EPS)
    g = ops.layernorm_bwd(x.cuda(), dy.cuda(), w.cuda(), mean, rstd)
    gen = torch.Generator().manual_seed(10)
    loss = lambda x, w, b: (O.norm_forward(x, w, b, EPS)["y"] * dy.double()).sum()
    e = 1e-5
    for i, name in enumerate(("dx", "dweight", "dbias")):
        args = [x.double(), w.double(), b.double()]
        step = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + e * step, args[i] - e * step
        want = ((loss(*up) - loss(*down)) / (2 * e)).item()
        got = (g[name].double().cpu() * step).sum().item()
        tol = 64 * E * g[name].double().norm().item() * step.norm().item() + 1e-6 * abs(want)
        assert abs(want - got) <= tol, (name, want, got, tol)
