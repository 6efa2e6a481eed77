"""Layer norm on the GPU with more rows than its blocks take at once: second and later rows of a block or warp, buffers of rows
used again, sums of dweight and dbias over several rows of a thread. Sizes go several rounds through every form (rows by
warps, rows by blocks with one to eight units a thread, a block for each row), aligned and not, and end inside a
round. Limits are those of test_gpu_layernorm.py, with the 64-bit formula evaluated on the GPU."""
import pytest
import torch

import linattn_oracle as O
from kimi_delta_attention_15_gb300 import ops

pytestmark = pytest.mark.gpu
E, U = 2.0 ** -24, 2.0 ** -8
EPS = 1e-5

SIZES = [(700001, 7), (160003, 33), (60005, 128), (40003, 131), (30007, 256), (20003, 501), (15001, 512), (19001, 777), (18403, 1024),
         (10007, 2048), (5001, 4096), (3207, 4097), (1607, 8191), (1613, 12288), (1603, 12289), (1003, 16384), (401, 20001)]


def make(rows, width, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + width)
    level = torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    x = (level * (torch.randn(rows, width, generator=g, device="cuda") + 0.3)).to(dtype)
    dy = torch.randn(rows, width, generator=g, device="cuda").to(dtype)
    w = 1.0 + 0.1 * torch.randn(width, generator=g, device="cuda")
    return x, dy, w, 0.1 * torch.randn(width, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,width", SIZES)
def test_every_row_against_the_formula(rows, width, dtype):
    x, dy, w, b = make(rows, width, dtype)
    y, mean, rstd = ops.layernorm_fwd(x, w, b, eps=EPS)
    ref = O.norm_forward(x, w, b, EPS)
    mu, rs = ref["mean"].abs()[:, None], ref["rstd"][:, None]
    assert ((mean.double() - ref["mean"]).abs() <= 64 * E * x.double().abs().mean(1)).all()
    assert ((rstd.double() - ref["rstd"]).abs() <= 64 * E * (1 + mu * rs)[:, 0] * ref["rstd"]).all()
    h = ((x.double() - ref["mean"][:, None]) * rs).abs()
    lim = 64 * E * (1 + mu * rs) * (1 + h) * w.double().abs() + 4 * E * ref["y"].abs() + 4 * E * b.double().abs()
    if dtype == torch.bfloat16:
        lim = lim * (1 + U) + U * ref["y"].abs()
    assert ((y.double() - ref["y"]).abs() <= lim).all()
    del ref, h, lim, y
    g = ops.layernorm_bwd(x, dy, w, mean, rstd)
    ref = O.norm_backward(x, dy, w, mean, rstd)
    rs = rstd.double()[:, None]
    h = (x.double() - mean.double()[:, None]) * rs
    n = rows + 64
    assert ((g["dweight"].double() - ref["dweight"]).abs() <= n * E * (dy.double() * h).abs().sum(0)).all()
    assert ((g["dbias"].double() - ref["dbias"]).abs() <= n * E * dy.double().abs().sum(0)).all()
    a = dy.double() * w.double()
    lim = 64 * E * rs * (a.abs() + a.abs().mean(1, keepdim=True) + h.abs() * (a * h).abs().mean(1, keepdim=True))
    if dtype == torch.bfloat16:
        lim = lim * (1 + U) + U * ref["dx"].abs()
    assert ((g["dx"].double() - ref["dx"]).abs() <= lim).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,width", SIZES)
def test_sums_over_rows_take_each_row_once(rows, width, dtype):
    """Small whole numbers, half ones after the given statistics: every product and sum is exact in fp32 in any order, so a
    row left out or taken twice shows."""
    g = torch.Generator(device="cuda").manual_seed(rows - width)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").float()
    x, dy = whole(rows, width).to(dtype), whole(rows, width).to(dtype)
    mean, rstd = whole(rows).clamp(-1, 1), torch.exp2(whole(rows).clamp(-1, 1))
    got = ops.layernorm_bwd(x, dy, None, mean, rstd)
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    assert torch.equal(got["dweight"].double(), (dy.double() * h).sum(0))
    assert torch.equal(got["dbias"].double(), dy.double().sum(0))


def test_forward_and_backward_in_a_graph():
    """The backward's sum over blocks is launched while the kernel before it still runs: captured and replayed too."""
    x, dy, w, b = make(5001, 1024, torch.bfloat16)
    y, mean, rstd = ops.layernorm_fwd(x, w, b)
    ws = torch.empty(ops.load().kda_layernorm_workspace_size(5001, 1024), dtype=torch.uint8, device="cuda")
    g = ops.layernorm_bwd(x, dy, w, mean, rstd, workspace=ws)
    outs = dict(y=y, mean=mean, rstd=rstd, **g)
    eager = {k: t.clone() for k, t in outs.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.layernorm_fwd(x, w, b, y=y, mean=mean, rstd=rstd)
        ops.layernorm_bwd(x, dy, w, mean, rstd, grads=g, workspace=ws)
    for _ in range(3):
        for t in outs.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k, t in outs.items():
            assert torch.equal(t, eager[k]), k
