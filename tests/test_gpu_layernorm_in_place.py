"""Layer norm with its outputs in the place of its inputs, in every form and where rows share 16-byte units."""
import pytest
import torch

from kimi_delta_attention_15_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,width", [(50, 1), (4001, 7), (40003, 131), (60005, 128), (2003, 501), (19001, 777), (5001, 4096), (3207, 4097),
                                        (1003, 16384), (301, 16385), (401, 20001), (70, 40960)])
def test_in_place_equals_out_of_place(rows, width, dtype):
    g = torch.Generator(device="cuda").manual_seed(width)
    x, dy = (torch.randn(rows, width, generator=g, device="cuda").to(dtype) for _ in range(2))
    w, b = (torch.randn(width, generator=g, device="cuda") for _ in range(2))
    y, mean, rstd = ops.layernorm_fwd(x, w, b)
    want = ops.layernorm_bwd(x, dy, w, mean, rstd)
    own = x.clone()
    _, mean2, rstd2 = ops.layernorm_fwd(own, w, b, y=own)
    assert torch.equal(own, y) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
    for take in ("dy", "x"):
        ins = dict(x=x.clone(), dy=dy.clone())
        sums = dict(dweight=torch.empty(width, device="cuda"), dbias=torch.empty(width, device="cuda"))
        got = ops.layernorm_bwd(ins["x"], ins["dy"], w, mean, rstd, grads=dict(dx=ins[take], **sums))
        for k in want:
            assert torch.equal(got[k], want[k]), (take, k)
