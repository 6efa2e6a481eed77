"""Layer norm called by several host threads at once."""
import threading

import pytest
import torch

from kimi_delta_attention_15_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,widths", [(torch.bfloat16, (8192, 5000, 1536)), (torch.float32, (4096, 2500, 600))])
def test_threads_with_rows_of_different_lengths(dtype, widths):
    """Widths that run the same kernel with shared memory of different sizes: no call changes what another may use."""
    errors = []

    def work(width):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                x = torch.randn(4, width, device="cuda").to(dtype)
                y, mean, rstd = ops.layernorm_fwd(x)
                g = ops.layernorm_bwd(x, x, None, mean, rstd)
                dx = g["dx"].clone()
                out = [torch.empty_like(t) for t in (y, mean, rstd)]
                for _ in range(2000):
                    ops.layernorm_fwd(x, y=out[0], mean=out[1], rstd=out[2])
                    ops.layernorm_bwd(x, x, None, mean, rstd, grads=g)
            stream.synchronize()
            assert torch.equal(out[0], y) and torch.equal(out[1], mean) and torch.equal(g["dx"], dx)
        except Exception as e:      # noqa: BLE001 (shown by the test's own thread)
            errors.append(f"width {width}: {e}")

    threads = [threading.Thread(target=work, args=(w,)) for w in widths]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
