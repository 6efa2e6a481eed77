"""The 64-bit definitions the GPU tests compare with, against central differences (CPU)."""
import pytest
import torch

import linattn_oracle as O


@pytest.mark.parametrize("lens,H,G", [((5,), 2, 1), ((3, 0, 4), 4, 2), ((1,), 1, 1)])
def test_linattn_gradient_equals_central_differences(lens, H, G):
    d = O.make(lens, H, G, seed=3, h0=True, dhT=True)
    d = {k: (v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v) for k, v in d.items()}
    grads = O.backward(d)
    gen = torch.Generator().manual_seed(4)
    for name in ("q", "k", "v", "h0"):
        step = torch.randn(d[name].shape, generator=gen, dtype=torch.float64)
        e = 1e-5      # the loss is quadratic in q, k and linear in v, h0 up to products: error e^2
        up, down = O.loss(dict(d, **{name: d[name] + e * step})), O.loss(dict(d, **{name: d[name] - e * step}))
        want, got = (up - down) / (2 * e), (grads["d" + name] * step).sum()
        assert abs(want - got) <= 1e-7 * max(1.0, abs(float(got))), name


def test_linattn_recurrence_equals_the_masked_product():
    d = O.make((9,), 2, 1, seed=5)
    q, k, v = (d[x].double().transpose(0, 1) for x in ("q", "k", "v"))
    i = torch.arange(9, dtype=torch.float64)
    w = torch.exp(d["log_decay"].double().view(2, 1, 1) * (i[:, None] - i[None, :])) * (i[:, None] >= i[None, :])
    o = O.D ** -0.5 * ((q @ k.transpose(1, 2)) * w) @ v
    assert torch.allclose(O.forward(d)["o"], o.transpose(0, 1), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("width", [1, 2, 7, 64])
def test_norm_gradient_equals_central_differences(width):
    gen = torch.Generator().manual_seed(width)
    x, dy = (torch.randn(3, width, generator=gen, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(width, generator=gen, dtype=torch.float64) for _ in range(2))
    f = O.norm_forward(x, w, b, 1e-2)
    g = O.norm_backward(x, dy, w, f["mean"], f["rstd"])
    loss = lambda x, w, b: (O.norm_forward(x, w, b, 1e-2)["y"] * dy).sum()
    e = 1e-5
    for i, name in enumerate(("dx", "dweight", "dbias")):
        args = [x, w, b]
        step = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + e * step, args[i] - e * step
        want, got = (loss(*up) - loss(*down)) / (2 * e), (g[name] * step).sum()
        # third derivatives of 1 / sqrt(var + 0.01) reach 1e3 here: e^2 * 1e3
        assert abs(want - got) <= 1e-6 * max(1.0, abs(float(got))), name
