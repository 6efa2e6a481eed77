"""Calls on tensors of a device that is not the current one (CPU: two devices are pretended, the library is a stub that
records which device is current and which stream it is given)."""
import contextlib
import math

import pytest
import torch

from kimi_delta_attention_15_gb300 import ops

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


class OnGpu:
    def __init__(self, index, dtype, *shape):
        self.index, self.dtype, self.shape, self.device = index, dtype, shape, torch.device("cuda", index)

    def numel(self):
        return math.prod(self.shape)

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 1 << 20


class Stream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 500 + index


class Gpus:
    """The current device, and the library's calls as (name, device current then, stream)."""

    def __init__(self, monkeypatch, current):
        self.current, self.calls, self.stream_now = current, [], None
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.current, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", self.raw, raising=False)
        monkeypatch.setattr(torch.cuda, "current_stream", self.of)
        monkeypatch.setattr(torch.cuda, "device", self.device)
        monkeypatch.setattr(torch.cuda, "stream", self.stream)
        monkeypatch.setattr(ops, "_lib", self)
        monkeypatch.setattr(ops, "load", lambda *a: self)

    def raw(self, dev):
        return self.stream_now.cuda_stream if self.stream_now else 100 + dev

    def of(self, device=None):
        s = Stream(self.current)
        s.cuda_stream = 100 + self.current
        return s

    @contextlib.contextmanager
    def device(self, index):
        before, self.current = self.current, index
        yield
        self.current = before

    @contextlib.contextmanager
    def stream(self, s):
        before, self.stream_now = self.stream_now, s
        with self.device(s.device_index):
            yield
        self.stream_now = before

    def __getattr__(self, name):
        def call(*args):
            stream = args[-1]
            self.calls.append((name, self.current, getattr(stream, "value", stream)))
            return 0
        return call


def every_call(dev, **kw):
    bf = lambda *s: OnGpu(dev, BF, *s)
    f = lambda *s: OnGpu(dev, F32, *s)
    ws = OnGpu(dev, U8, 4096)
    tok, head, state = bf(8, 2, 128), f(2), f(1, 2, 128, 128)
    kda = (tok, tok, tok, tok, bf(8, 2), head, f(2, 128))
    x, row = bf(4, 16), f(4)
    one, st = bf(1, 2, 128), f(1, 2, 128, 128)
    return [
        ("kda_fwd", lambda: ops.fwd(*kda, workspace=ws, o=tok, hT=state, **kw)),
        ("kda_fwd_static_scratch", lambda: ops.fwd_static_scratch(*kda, o=tok, hT=state, **kw)),
        ("kda_bwd", lambda: ops.bwd(*kda, tok, ws, grads=dict(dq=tok, dk=tok, dv=tok, dg_raw=tok, dbeta_raw=bf(8, 2), dA_log=head,
                                                              ddt_bias=f(2, 128), dh0=None), **kw)),
        ("kda_decode", lambda: ops.decode(one, one, one, one, bf(1, 2), head, f(2, 128), st, o=one, **kw)),
        ("kda_linattn_fwd", lambda: ops.linattn_fwd(tok, tok, tok, head, workspace=ws, o=tok, hT=state, **kw)),
        ("kda_linattn_fwd", lambda: ops.linattn_fwd(q=tok, k=tok, v=tok, log_decay=head, workspace=ws, o=tok, hT=state, **kw)),
        ("kda_linattn_bwd", lambda: ops.linattn_bwd(tok, tok, tok, head, tok, ws, grads=dict(dq=tok, dk=tok, dv=tok), **kw)),
        ("kda_linattn_decode", lambda: ops.linattn_decode(one, one, one, head, st, o=one, **kw)),
        ("kda_layernorm_fwd", lambda: ops.layernorm_fwd(x, y=x, mean=row, rstd=row, **kw)),
        ("kda_layernorm_bwd", lambda: ops.layernorm_bwd(x, x, None, row, row, workspace=ws, grads=dict(dx=x), **kw)),
        ("kda_get_device_status", lambda: ops.device_status(ws, **kw)),
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
        assert gpus.current == 0


def test_a_stream_of_another_device_is_refused(monkeypatch):
    gpus = Gpus(monkeypatch, 0)
    for name, call in every_call(1, stream=Stream(0)):
        with pytest.raises(ValueError, match="^stream: on cuda:0; the tensors are on cuda:1"):
            call()
    assert not gpus.calls
