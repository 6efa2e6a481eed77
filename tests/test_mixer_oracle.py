"""The 64-bit oracle of the gated recurrence and of the norm with rotation: gradients against central differences
and against torch's own derivatives, angles against 64 bits, states through cuts."""
import pytest
import torch

import mixer_oracle as O

F64 = torch.float64


def case(lens, D, seed=0):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=F64)
    return dict(x=r(T, D), g=r(T, D), i=r(T, D), A_log=r(D), h0=r(N, D)), r(T, D), r(N, D)


def loss(c, lens, dy, dhT):
    o = O.recurrence(lens=lens, **c)
    return (o["y"][0] * dy).sum() + (o["hT"][0] * dhT).sum()


@pytest.mark.parametrize("lens", [[1], [5], [3, 0, 4]])
def test_recurrence_gradients_by_differences(lens):
    c, dy, dhT = case(lens, 3)
    o = O.recurrence(lens=lens, dy=dy, dhT=dhT, **c)
    for name, out in (("x", "dx"), ("g", "dg_raw"), ("i", "di_raw"), ("A_log", "dA_log"), ("h0", "dh0")):
        for at in range(c[name].numel()):
            d = torch.zeros_like(c[name]).view(-1)
            d[at] = 1e-5
            d = d.view(c[name].shape)
            up, down = (loss({**c, name: c[name] + s * d}, lens, dy, dhT) for s in (1, -1))
            # the difference is off by the third derivative times 1e-10 and by rounding, 1e-16 over 1e-5
            assert abs((up - down).item() / 2e-5 - o[out][0].view(-1)[at].item()) < 1e-8, (name, at)


def test_recurrence_by_its_formula():
    c, _, _ = case([2], 1, seed=1)
    a = torch.exp(-torch.exp(c["A_log"]) * torch.sigmoid(c["g"]))
    b = torch.sqrt(1 - a * a) * torch.sigmoid(c["i"]) * c["x"]
    y = O.recurrence(lens=[2], **c)["y"][0]
    assert torch.allclose(y[0], a[0] * c["h0"][0] + b[0], atol=1e-14)
    assert torch.allclose(y[1], a[1] * (a[0] * c["h0"][0] + b[0]) + b[1], atol=1e-14)


def test_recurrence_cut_in_two():
    c, _, _ = case([20], 4, seed=2)
    whole = O.recurrence(lens=[20], **c)
    cut = lambda p, h0: O.recurrence(c["x"][p], c["g"][p], c["i"][p], c["A_log"], [c["x"][p].shape[0]], h0)
    first = cut(slice(0, 7), c["h0"])
    second = cut(slice(7, 20), first["hT"][0])
    assert torch.allclose(second["y"][0], whole["y"][0][7:], atol=1e-14)
    assert torch.allclose(second["hT"][0], whole["hT"][0], atol=1e-14)


def test_an_oracle_with_a_mistake_is_told():
    """Half the bound of a wrong recurrence: a planted mistake of one part in a thousand shows."""
    c, _, _ = case([40], 4, seed=3)
    o = O.recurrence(lens=[40], **c)
    wrong = dict(c, A_log=c["A_log"] + 1e-3)
    with pytest.raises(AssertionError):
        O.check("y", O.recurrence(lens=[40], **wrong)["y"][0].float(), o["y"])
    O.check("y", o["y"][0].float(), o["y"])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("head,rotary", [(8, 8), (16, 8), (24, 0)])
def test_qknorm_gradients(head, rotary, interleaved):
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(3, 2, head, generator=gen, dtype=F64, requires_grad=True)
    w = torch.randn(head, generator=gen, dtype=F64, requires_grad=True)
    dy = torch.randn(3, 2, head, generator=gen, dtype=F64)
    theta = torch.randn(3, rotary // 2, generator=gen, dtype=F64)
    z = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    y = O.turned(z, theta, interleaved)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert torch.allclose(O.qknorm(x.detach(), w.detach(), theta, interleaved, 1e-6)["y"][0], y.detach(), atol=1e-14)
    g = O.qknorm(x.detach(), w.detach(), theta, interleaved, 1e-6, dy)
    assert torch.allclose(g["dx"][0], dx, atol=1e-13) and torch.allclose(g["dw"][0], dw, atol=1e-13)


def test_angles():
    p = torch.tensor([0, 1, -1, 12345, 1 << 20])
    f = torch.tensor([1.0, 0.1, 1e-4])
    a = O.angles(p, f)
    want = p.double()[:, None] * f.double()
    assert ((torch.cos(a) - torch.cos(want)).abs() < 1e-9).all() and ((torch.sin(a) - torch.sin(want)).abs() < 1e-9).all()


def test_a_rotation_by_pairs():
    z = torch.arange(8, dtype=F64).view(1, 1, 8)
    quarter = torch.full((1, 2), torch.pi / 2, dtype=F64)
    assert torch.allclose(O.turned(z, quarter, False)[0, 0], torch.tensor([-2., -3, 0, 1, 4, 5, 6, 7], dtype=F64), atol=1e-14)
    assert torch.allclose(O.turned(z, quarter, True)[0, 0], torch.tensor([-1., 0, -3, 2, 4, 5, 6, 7], dtype=F64), atol=1e-14)
