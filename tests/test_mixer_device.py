"""Calls of the gated recurrence and of the norm of queries and keys on tensors of a device that is not the current one
(CPU: two devices are pretended, the library is a stub; see test_binding_device)."""
import pytest

from kimi_delta_attention_15_gb300 import ops
from test_binding_device import BF, F32, U8, Gpus, OnGpu, Stream


def every_call(dev, **kw):
    import torch
    bf, f = (lambda *s: OnGpu(dev, BF, *s)), (lambda *s: OnGpu(dev, F32, *s))
    ws = OnGpu(dev, U8, 4096)
    x, A, state, kept = bf(8, 16), f(16), f(1, 16), f(1, 16)
    q, k, w = bf(8, 4, 64), bf(8, 2, 64), f(64)
    rotation = (OnGpu(dev, torch.int64, 8), f(32))
    return [
        ("kda_recurrence_fwd", lambda: ops.recurrence_fwd(x, x, x, A, workspace=ws, y=x, hT=state, **kw)),
        ("kda_recurrence_fwd", lambda: ops.recurrence_fwd(x=x, g_raw=x, i_raw=x, A_log=A, workspace=ws, y=x, hT=state, **kw)),
        ("kda_recurrence_bwd", lambda: ops.recurrence_bwd(x, x, x, A, x, kept, ws, grads=dict(dx=x, dg_raw=x, di_raw=x), **kw)),
        ("kda_recurrence_decode", lambda: ops.recurrence_decode(x, x, x, A, f(8, 16), y=x, **kw)),
        ("kda_qknorm_fwd", lambda: ops.qknorm_fwd(q, k, w, w, *rotation, q_out=q, k_out=k, **kw)),
        ("kda_qknorm_fwd", lambda: ops.qknorm_fwd(q=q, q_out=q, **kw)),
        ("kda_qknorm_bwd", lambda: ops.qknorm_bwd(q, k, q, k, w, w, *rotation, workspace=ws, grads=dict(dq=q, dk=k), **kw)),
    ]


@pytest.mark.parametrize("current", [0, 1])
@pytest.mark.parametrize("dev", [0, 1])
def test_calls_run_on_their_tensors_device(monkeypatch, current, dev):
    gpus = Gpus(monkeypatch, current)
    for name, call in every_call(dev):
        gpus.calls.clear()
        call()
        assert gpus.calls == [(name, dev, 100 + dev)], name
        assert gpus.current == current


def test_a_stream_of_the_tensors_device(monkeypatch):
    gpus = Gpus(monkeypatch, 0)
    for name, call in every_call(1, stream=Stream(1)):
        gpus.calls.clear()
        call()
        assert gpus.calls == [(name, 1, 501)], name


def test_a_stream_or_a_tensor_of_another_device_is_refused(monkeypatch):
    gpus = Gpus(monkeypatch, 0)
    for name, call in every_call(1, stream=Stream(0)):
        with pytest.raises(ValueError, match="^stream: on cuda:0; the tensors are on cuda:1"):
            call()
    x, A = OnGpu(1, BF, 8, 16), OnGpu(1, F32, 16)
    for call in (lambda: ops.recurrence_fwd(x, OnGpu(0, BF, 8, 16), x, A), lambda: ops.recurrence_fwd(x, x, x, OnGpu(0, F32, 16)),
                 lambda: ops.recurrence_decode(x, x, x, A, OnGpu(0, F32, 8, 16)),
                 lambda: ops.qknorm_fwd(OnGpu(1, BF, 8, 4, 64), OnGpu(0, BF, 8, 2, 64)),
                 lambda: ops.qknorm_fwd(OnGpu(1, BF, 8, 4, 64), None, OnGpu(0, F32, 64))):
        with pytest.raises(ValueError, match="one CUDA device"):
            call()
    assert not gpus.calls
