"""Refusals of the linear attention and layer norm entry points (CPU): the C ABI's status
codes before any CUDA call, and the binding's checks of sizes, dtypes and layout."""
import ctypes

import pytest
import torch

import linattn_oracle as O
from kimi_delta_attention_15_gb300 import build, ops

DEVICE_MSG = "one CUDA device"


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ops.load()


def _fwd(lib, shape, ptr=16, ws_bytes=1 << 40, cu=None, ws=1024, bad=None):
    p = [ctypes.c_void_p(ptr) for _ in range(7)]        # q k v log_decay h0 o hT
    if bad is not None:
        p[bad] = ctypes.c_void_p(ptr + 8)
    return lib.kda_linattn_fwd(ctypes.byref(shape), *p[:5], cu, *p[5:], ctypes.c_void_p(ws), ws_bytes, None)


def _bwd(lib, shape, ptr=16, ws_bytes=1 << 40, cu=None, ws=1024, bad=None):
    p = [ctypes.c_void_p(ptr) for _ in range(11)]       # q k v log_decay h0 | do dhT dq dk dv dh0
    if bad is not None:
        p[bad] = ctypes.c_void_p(ptr + 8)
    return lib.kda_linattn_bwd(ctypes.byref(shape), *p[:5], cu, *p[5:], ctypes.c_void_p(ws), ws_bytes, None)


@pytest.mark.parametrize("call,n", [(_fwd, 7), (_bwd, 11)])
def test_linattn_status_codes(lib, call, n):
    s = ops.linattn_shape(64, 2, 1)
    assert call(lib, s, ptr=0) == 1                      # NULL
    for i in range(n):
        assert call(lib, s, bad=i) == 2                  # each pointer 16-byte aligned
    assert call(lib, s, ws_bytes=16) == 5
    assert call(lib, s, ws=0) == 5
    assert call(lib, s, ws=1032) == 2
    assert call(lib, s, cu=ctypes.c_void_p(20)) == 2     # offsets 8-byte aligned
    u = ops.linattn_shape(64, 2, 1)
    u.K = 64
    assert call(lib, u) == 4
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(lib, ops.linattn_shape(64, 2, 1, scale=scale)) == 4
    assert call(lib, ops.linattn_shape(64, 0, 1)) == 3
    assert call(lib, ops.linattn_shape(-1, 2, 1)) == 3
    assert call(lib, ops.linattn_shape(64, 2, 3)) == 3              # three sequences need offsets
    assert call(lib, ops.linattn_shape(64, 2, 2, B=2), cu=ctypes.c_void_p(16)) == 3     # packed has B = 1
    assert call(lib, ops.linattn_shape(64, 6, 1, groups=4)) == 3
    assert call(lib, ops.linattn_shape(64, 6, 1, groups=-1)) == 3
    assert call(lib, ops.linattn_shape(1 << 30, 2, 1)) == 3         # B T H at most 2^31 - 1
    null = ctypes.POINTER(ops.LinattnShape)()
    assert lib.kda_linattn_workspace_size(null, 0) == 0
    assert lib.kda_linattn_fwd(null, *[None] * 9, 0, None) == 1


def test_linattn_workspace_size(lib):
    f, b = (ops.linattn_workspace_size(ops.linattn_shape(1000, 8, 1), x) for x in (False, True))
    assert 0 < f <= b
    g = ops.linattn_workspace_size(ops.linattn_shape(1000, 8, 1, groups=4), True)
    assert g >= b + 2 * 1000 * 8 * 128 * 4               # the value heads' fp32 shares of dq and dk
    assert ops.linattn_workspace_size(ops.linattn_shape(1000, 8, 1, groups=3)) == 0


def test_workspace_of_many_sequences(lib):
    """Only segments of sequences of several keep states (64 KB each): with n segments' length of tokens between n and
    2 n of them, whatever the number of sequences."""
    few, many = (ops.linattn_workspace_size(ops.linattn_shape(100000, 4, n), True) for n in (10, 65535))
    assert many <= 2 * few + 65535 * 64


def test_linattn_decode_status_codes(lib):
    def call(n=2, H=3, groups=1, scale=0.1, ptr=16, bad=None):
        p = [ctypes.c_void_p(ptr) for _ in range(6)]
        if bad is not None:
            p[bad] = ctypes.c_void_p(ptr + 8)
        return lib.kda_linattn_decode(n, H, groups, scale, *p, None)
    assert call(n=-1) == 3 and call(H=0) == 3 and call(groups=2) == 3 and call(groups=-1) == 3
    assert call(n=1 << 30, H=8) == 3
    assert call(scale=float("nan")) == 4 and call(scale=0.0) == 4
    assert call(ptr=0) == 1
    for i in range(6):
        assert call(bad=i) == 2
    assert call(n=0, ptr=0) == 0


def test_layernorm_status_codes(lib):
    def fwd(rows=4, width=8, dtype=0, eps=1e-5, ptr=16, bad=None):
        p = [ctypes.c_void_p(ptr) for _ in range(6)]
        if bad is not None:
            p[bad] = ctypes.c_void_p(ptr + 8)
        return lib.kda_layernorm_fwd(rows, width, dtype, eps, *p, None)

    def bwd(rows=4, width=8, dtype=0, ptr=16, bad=None, ws=1024, ws_bytes=1 << 30):
        p = [ctypes.c_void_p(ptr) for _ in range(8)]
        if bad is not None:
            p[bad] = ctypes.c_void_p(ptr + 8)
        return lib.kda_layernorm_bwd(rows, width, dtype, *p, ctypes.c_void_p(ws), ws_bytes, None)

    for f, n in ((fwd, 6), (bwd, 8)):
        assert f(rows=-1) == 3 and f(width=0) == 3 and f(width=(1 << 20) + 1) == 3 and f(rows=1 << 60, width=1 << 20) == 3
        assert f(dtype=2) == 4 and f(dtype=-1) == 4
        assert f(ptr=0) == 1
        for i in range(n):
            assert f(bad=i) == 2
    for eps in (0.0, -1e-5, float("nan"), float("inf")):
        assert fwd(eps=eps) == 4
    assert fwd(rows=0, ptr=0) == 0
    assert bwd(ws=0) == 5 and bwd(ws_bytes=16) == 5 and bwd(ws=1032) == 2
    assert lib.kda_layernorm_workspace_size(4, 0) == 0


def test_binding_passes_valid_calls_up_to_the_device_check():
    for lens, H, G in (((70,), 4, 1), ((17, 0, 65), 8, 4), ((0,), 2, 1)):
        d = O.make(lens, H, G, h0=True, dhT=True)
        cu = d["cu_seqlens"] if len(lens) > 1 else None
        with pytest.raises(ValueError, match=DEVICE_MSG):
            ops.linattn_fwd(d["q"], d["k"], d["v"], d["log_decay"], h0=d["h0"], cu_seqlens=cu)
        with pytest.raises(ValueError, match=DEVICE_MSG):
            ops.linattn_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["do"], h0=d["h0"], cu_seqlens=cu, dhT=d["dhT"])
    with pytest.raises(ValueError, match=DEVICE_MSG):
        x = torch.zeros(3, 5, 33)
        ops.layernorm_fwd(x, torch.ones(33), torch.zeros(33))


def test_binding_refuses_mistakes():
    d = O.make((40, 30), 4, 2, h0=True)
    call = lambda **kw: ops.linattn_fwd(*[{**d, **kw}[x] for x in ("q", "k", "v", "log_decay")], h0={**d, **kw}["h0"],
                                        cu_seqlens=d["cu_seqlens"], workspace=kw.get("workspace"))
    with pytest.raises(ValueError, match="^k:"):
        call(k=d["k"][:, :1].contiguous())
    with pytest.raises(ValueError, match="^log_decay:"):
        call(log_decay=d["log_decay"][:3])
    with pytest.raises(ValueError, match="^log_decay: dtype"):
        call(log_decay=d["log_decay"].double())
    with pytest.raises(ValueError, match="^h0:"):
        call(h0=d["h0"][:1])
    with pytest.raises(ValueError, match="must be contiguous"):
        call(v=d["v"].transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(ValueError, match="multiple of query/key heads"):
        call(q=d["q"].repeat(1, 3, 1)[:, :3].contiguous())
    with pytest.raises(ValueError, match="^workspace: dtype"):
        call(workspace=torch.zeros(64))
    with pytest.raises(ValueError, match="^state:"):
        ops.linattn_decode(d["q"], d["k"], d["v"], d["log_decay"], torch.zeros(3, 4, 128, 128))
    x = torch.zeros(4, 6)
    with pytest.raises(ValueError, match="^x: dtype"):
        ops.layernorm_fwd(x.half())
    with pytest.raises(ValueError, match="no row"):
        ops.layernorm_fwd(torch.zeros(4, 0))
    with pytest.raises(ValueError, match="^weight:"):
        ops.layernorm_fwd(x, torch.ones(5))
    with pytest.raises(ValueError, match="^weight: dtype"):
        ops.layernorm_fwd(x, torch.ones(6).bfloat16())
    with pytest.raises(ValueError, match="^dy: dtype"):
        ops.layernorm_bwd(x, x.bfloat16(), None, torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError, match="^mean:"):
        ops.layernorm_bwd(x, x, None, torch.zeros(3), torch.zeros(4))
