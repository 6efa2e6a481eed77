"""The gated recurrence over channels on the GPU against the recurrence in 64 bits; tolerances are the running bounds of
mixer_oracle."""
import pytest
import torch

import mixer_oracle as O
from kimi_delta_attention_15_gb300 import ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(lens, D, dtype=BF, states=True, fused=False, seed=0, shift=0.0, A=None, spread=1.0):
    """Inputs on the CPU; `fused`: token tensors as columns of one buffer on the GPU."""
    gen = torch.Generator().manual_seed(seed + 1000 * D + sum(lens))
    T, N = sum(lens), len(lens)
    r = lambda *s: torch.randn(*s, generator=gen)
    c = dict(x=r(T, D), g=spread * r(T, D) + shift, i=r(T, D), dy=r(T, D))
    c = {k: v.to(dtype) for k, v in c.items()}
    c["A_log"] = torch.log(-8 * torch.log(0.9 + 0.099 * torch.rand(D, generator=gen))) if A is None else torch.full((D,), float(A))
    c["h0"], c["dhT"] = (r(N, D), r(N, D)) if states else (None, None)
    c.update(lens=lens, fused=fused)
    return c


def columns(fused, *parts):
    parts = [p.cuda() for p in parts]
    if not fused:
        return parts
    whole = torch.cat(parts, 1)
    return whole.split(parts[0].shape[1], 1)


def offsets(lens):
    return torch.tensor([0] + lens).cumsum(0).cuda()


def dev(t):
    return None if t is None else t.cuda()


def run(c, packed=True, B=1, **kw):
    x, g, i = columns(c["fused"], c["x"], c["g"], c["i"])
    cu = offsets(c["lens"]) if packed else None
    args = (x, g, i, c["A_log"].cuda())
    y, hT, kept, ws = ops.recurrence_fwd(*args, h0=dev(c["h0"]), cu_seqlens=cu, B=B, want_kept=True, **kw)
    assert ops.device_status(ws) == 0
    grads = None
    T, D = c["x"].shape
    if c["fused"]:
        dx, dg, di = torch.empty(T, 3 * D, dtype=x.dtype, device="cuda").split(D, 1)
        grads = dict(dx=dx, dg_raw=dg, di_raw=di, dA_log=torch.empty(D, device="cuda"), dh0=torch.empty(len(c["lens"]), D, device="cuda"))
    ws2 = ops.recurrence_alloc_workspace(ops.recurrence_shape(T if packed else T // B, D, len(c["lens"]), 1 if packed else B, x.dtype),
                                         "cuda", backward=True)
    out = ops.recurrence_bwd(*args, c["dy"].cuda(), kept, ws2, h0=dev(c["h0"]), cu_seqlens=cu, dhT=dev(c["dhT"]), B=B, grads=grads)
    assert ops.device_status(ws2) == 0
    return dict(out, y=y, hT=hT, kept=kept)


def verify(c, got):
    ref = O.recurrence(c["x"], c["g"], c["i"], c["A_log"], c["lens"], c["h0"], c["dy"], c["dhT"])
    for name in ("y", "hT", "dx", "dg_raw", "di_raw", "dA_log", "dh0"):
        O.check(name, got[name], ref[name])
    T = sum(c["lens"])
    if T:
        rows = torch.arange(0, T, ops.RECURRENCE_BLOCK)[1:] - 1
        h, e = ref["y"]
        zero = torch.zeros(1, h.shape[1], dtype=torch.float64)
        O.check("kept", got["kept"], (torch.cat([zero, h[rows]]), torch.cat([zero, e[rows]])))


LENS = [[1], [2], [7], [8], [9], [15], [16], [17], [63], [64], [65], [127], [128], [129], [300], [17, 33, 65], [0, 5, 0, 0, 130, 0],
        [64, 64, 64], [1] * 70, [16, 112, 1, 128, 127], [0, 0, 3]]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_lengths(lens, dtype):
    c = make(lens, 72, dtype)
    verify(c, run(c))


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [1, 2, 3, 7, 8, 31, 63, 64, 65, 100, 128, 200, 516, 1000])
def test_widths(D, dtype, fused):
    c = make([70, 1, 130], D, dtype, fused=fused)
    verify(c, run(c))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_without_states(dtype):
    c = make([5, 0, 100, 61], 40, dtype, states=False)
    verify(c, run(c))


@pytest.mark.parametrize("B,T", [(1, 100), (3, 50), (4, 128), (5, 1), (2, 0)])
def test_batches(B, T):
    c = make([T] * B, 48)
    verify(c, run(c, packed=False, B=B))
    if T:       # the same as [B, T, D], and as columns of a buffer of that shape
        x, g, i = (torch.cat([c[k].cuda()] * 2, 1).view(B, T, 96)[..., :48] for k in ("x", "g", "i"))
        y, hT, _, _ = ops.recurrence_fwd(x, g, i, c["A_log"].cuda(), h0=dev(c["h0"]))
        want = run(c, packed=False, B=B)
        assert y.shape == (B, T, 48) and torch.equal(y.view(B * T, 48), want["y"]) and torch.equal(hT, want["hT"])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,D", [([5000], 64), ([3001], 24), ([1000, 0, 2222, 5, 700], 130), ([4097], 8)])
def test_long_sequences_of_few_channels(lens, D, dtype):
    c = make(lens, D, dtype, fused=True)
    verify(c, run(c))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,D", [([1024], 520), ([700, 0, 333, 1, 66], 1024), ([3000, 40], 1540), ([2000], 2500), ([64] * 17, 1001)])
def test_clusters_of_many_blocks(lens, D, dtype):
    c = make(lens, D, dtype)
    verify(c, run(c))


def test_many_channels():
    c = make([150, 37], 6000)
    verify(c, run(c))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_sequences(dtype):
    gen = torch.Generator().manual_seed(9)
    lens = torch.randint(0, 4, (1500,), generator=gen).tolist()
    c = make(lens, 16, dtype)
    verify(c, run(c))


@pytest.mark.parametrize("shift,A", [(-9.0, 0.0), (-14.0, -1.0), (0.0, -12.0)])
def test_memories_of_many_thousand_tokens(shift, A):
    """1 - a of 1e-4 to 1e-6: a rounded a alone would be off by as much as 1e-2 of the state."""
    c = make([6000], 8, F32, shift=shift, A=A, spread=0.1)
    verify(c, run(c))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,D", [([40], 8), ([70, 130], 72), ([5000, 3], 24), ([200, 1900, 1000], 136), ([300], 2000)])
def test_states_that_decay_by_many_orders(lens, D, dtype):
    """A state of 1e14 and its gradient are down at 1 after some thirty tokens, and exact there: a run's decay less 1 on
    the state before it, added to that state, would leave an absolute error of 1e-7 of it."""
    c = make(lens, D, dtype, A=0.7, spread=0.2)
    c["h0"], c["dhT"] = 1e14 * c["h0"], 1e14 * c["dhT"]
    verify(c, run(c))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("A,shift", [(2.0, 4.0), (2.0, 0.0), (0.0, 4.0)])
def test_strong_decays(A, shift, dtype):
    for lens, D in (([2500, 64, 1436], 136), ([4000], 128), ([9000, 17], 9)):
        c = make(lens, D, dtype, shift=shift, A=A, spread=5.0, fused=True)
        verify(c, run(c))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("A", [-20.0, 3.0, 9.0])
def test_wide_gates(A, dtype):
    c = make([100, 90], 32, dtype, A=A, spread=20.0)
    verify(c, run(c))


@pytest.mark.parametrize("gate", [1e4, -1e4, 100.0, -100.0, 3e38, -3e38])
def test_saturated_gates(gate):
    """Open all the way, a = exp(-exp(A_log)); closed all the way, the state stays and nothing is written."""
    D = 16
    for k in ("g", "i"):
        c = make([70], D, F32, A=-1.0)
        c[k] = torch.full_like(c[k], gate)
        got = run(c)
        if abs(gate) < 1e30:
            c[k] = torch.full_like(c[k], max(-90.0, min(90.0, gate)))      # the same gate to 1e-39
            verify(c, got)
        else:
            assert all(torch.isfinite(got[n]).all() for n in ("y", "hT", "dx", "dg_raw", "di_raw", "dA_log", "dh0"))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_token_stays_in_its_sequence_and_channel(value):
    lens = [100, 150, 60]
    c = make(lens, 64, F32)
    clean = run(c)
    for name in ("x", "g", "i", "dy"):
        bad = dict(c, **{name: c[name].clone()})
        bad[name][120, 5] = value
        got = run(bad)
        for out in ("y", "dx", "dg_raw", "di_raw"):
            same = got[out] == clean[out]
            same[100:250, 5] = True
            assert same.all(), (name, out)
        for out in ("hT", "dh0"):
            same = got[out] == clean[out]
            same[1, 5] = True
            assert same.all(), (name, out)
        same = got["dA_log"] == clean["dA_log"]
        same[5] = True
        assert same.all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,D", [(1, 1), (3, 7), (4, 512), (33, 100), (2, 2056), (257, 64)])
def test_decode(n, D, dtype):
    c = make([1] * n, D, dtype)
    for fused in (False, True):
        x, g, i = columns(fused, c["x"], c["g"], c["i"])
        state = c["h0"].cuda()
        y = ops.recurrence_decode(x, g, i, c["A_log"].cuda(), state)
        ref = O.recurrence(c["x"], c["g"], c["i"], c["A_log"], c["lens"], c["h0"])
        O.check("y", y, ref["y"])
        O.check("state", state, ref["hT"])
    state, x = c["h0"].cuda(), c["x"].cuda()
    assert torch.equal(ops.recurrence_decode(x, c["g"].cuda(), c["i"].cuda(), c["A_log"].cuda(), state, y=x), y)
    assert ops.recurrence_decode(x[:0], x[:0], x[:0], c["A_log"].cuda(), state[:0]).shape == (0, D)


def test_prompts_cut_and_continued_token_by_token():
    lens, D = [90, 33], 24
    c = make(lens, D, F32)
    ref = O.recurrence(c["x"], c["g"], c["i"], c["A_log"], lens, c["h0"])
    cut = [60, 1]
    rows = lambda a, b: torch.cat([torch.arange(a[0], b[0]), 90 + torch.arange(a[1], b[1])])
    part = lambda r: [c[k][r].cuda() for k in ("x", "g", "i")]
    A = c["A_log"].cuda()
    r = rows([0, 0], cut)
    y, state, _, _ = ops.recurrence_fwd(*part(r), A, h0=c["h0"].cuda(), cu_seqlens=offsets(cut))
    O.check("y", y, tuple(v[r] for v in ref["y"]))
    for s in range(29):
        r = torch.tensor([60 + s, 90 + 1 + s])
        y = ops.recurrence_decode(*part(r), A, state)
        O.check("y", y, tuple(v[r] for v in ref["y"]))


def test_outputs_in_place():
    c = make([70, 130], 72, F32)
    want = run(c)
    cu, A = offsets(c["lens"]), c["A_log"].cuda()
    for at in range(3):
        args = [c[k].cuda() for k in ("x", "g", "i")]
        y, hT, _, _ = ops.recurrence_fwd(*args, A, h0=c["h0"].cuda(), cu_seqlens=cu, y=args[at])
        assert y is args[at] and torch.equal(y, want["y"]) and torch.equal(hT, want["hT"])
    x, g, i, dy = (c[k].cuda() for k in ("x", "g", "i", "dy"))
    for places in ((x, g, i), (dy, x, g), (i, dy, x)):
        x, g, i, dy = (t.copy_(c[k]) for t, k in ((x, "x"), (g, "g"), (i, "i"), (dy, "dy")))
        grads = dict(dx=places[0], dg_raw=places[1], di_raw=places[2], dA_log=torch.empty_like(A), dh0=None)
        ops.recurrence_bwd(x, g, i, A, dy, want["kept"], h0=c["h0"].cuda(), cu_seqlens=cu, dhT=c["dhT"].cuda(), grads=grads)
        for n in ("dx", "dg_raw", "di_raw", "dA_log"):
            assert torch.equal(grads[n], want[n]), n


def test_in_place_over_a_long_sequence():
    c = make([5000], 24, F32)
    want = run(c)
    x, g, i, dy = (c[k].cuda() for k in ("x", "g", "i", "dy"))
    A, h0 = c["A_log"].cuda(), c["h0"].cuda()
    grads = dict(dx=dy, dg_raw=x, di_raw=g, dA_log=torch.empty_like(A), dh0=None)
    ops.recurrence_bwd(x, g, i, A, dy, want["kept"], h0=h0, dhT=c["dhT"].cuda(), grads=grads)
    assert torch.equal(dy, want["dx"]) and torch.equal(x, want["dg_raw"]) and torch.equal(g, want["di_raw"])
    g = c["g"].cuda()
    y, _, _, _ = ops.recurrence_fwd(c["x"].cuda(), g, i, A, h0=h0, y=g)
    assert torch.equal(y, want["y"])


def test_a_state_is_refused_in_the_place_of_another():
    c = make([5], 8)
    x, h = c["x"].cuda(), c["h0"].cuda()
    with pytest.raises(ops.KdaError, match="UNSUPPORTED"):
        ops.recurrence_fwd(x, x, x, c["A_log"].cuda(), h0=h, hT=h)


def test_rows_and_columns_around_the_outputs_stay():
    c = make([40, 25], 24, F32)
    x, g, i = (c[k].cuda() for k in ("x", "g", "i"))
    buf = torch.full((80, 40), 7.0, device="cuda")
    ops.recurrence_fwd(x, g, i, c["A_log"].cuda(), cu_seqlens=offsets(c["lens"]), y=buf[:65, 8:32])
    inside = torch.zeros(80, 40, dtype=torch.bool)
    inside[:65, 8:32] = True
    assert (buf.cpu()[~inside] == 7.0).all() and (buf.cpu()[inside] != 7.0).all()


@pytest.mark.parametrize("lens,D", [([700, 1, 300], 200), ([6000], 24)])
def test_the_same_bits_every_time(lens, D):
    c = make(lens, D)
    a, b = run(c), run(c)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_malformed_offsets_are_reported():
    c = make([100], 16)
    args = [c[k].cuda() for k in ("x", "g", "i")] + [c["A_log"].cuda()]
    kept = torch.zeros(2, 16, device="cuda")
    for cu in ([0, 40, 30, 100], [0, 40, 120, 100], [1, 40, 50, 100], [0, 10, 20, 99], [0, -5, 20, 100], [0, 1 << 40, -(1 << 50), 100],
               [100, 0, 0, 0], [7, 7, 7, 7]):
        bad = torch.tensor(cu, device="cuda")
        y, hT, k, ws = ops.recurrence_fwd(*args, cu_seqlens=bad, want_kept=True)
        assert ops.device_status(ws) == 6
        ws = ops.recurrence_alloc_workspace(ops.recurrence_shape(100, 16, 3), "cuda", True)
        ops.recurrence_bwd(*args, c["dy"].cuda(), kept, ws, cu_seqlens=bad)
        assert ops.device_status(ws) == 6
        _, _, _, ws = ops.recurrence_fwd(*args, cu_seqlens=torch.tensor([0, 30, 40, 100], device="cuda"), workspace=ws)
        assert ops.device_status(ws) == 0


@pytest.mark.parametrize("lens,D", [([17, 33, 65], 64), ([5000], 24)])
def test_captured_and_replayed(lens, D):
    c = make(lens, D)
    want = run(c)
    x, g, i, dy = (c[k].cuda() for k in ("x", "g", "i", "dy"))
    A, h0, dhT, cu = c["A_log"].cuda(), c["h0"].cuda(), c["dhT"].cuda(), offsets(lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, hT, kept, _ = ops.recurrence_fwd(x, g, i, A, h0=h0, cu_seqlens=cu, want_kept=True)
        grads = ops.recurrence_bwd(x, g, i, A, dy, kept, h0=h0, cu_seqlens=cu, dhT=dhT)
    for _ in range(2):
        for t in (y, hT, kept, *grads.values()):
            t.fill_(float("nan"))
        graph.replay()
        got = dict(grads, y=y, hT=hT, kept=kept)
        assert all(torch.equal(got[k], want[k]) for k in want)
    x.zero_()
    graph.replay()
    y0, _, _, _ = ops.recurrence_fwd(x, g, i, A, h0=h0, cu_seqlens=cu)
    assert torch.equal(y, y0)


def test_on_other_streams_at_once():
    cases = [make([6000], 24, seed=s) for s in range(3)]
    want = [run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    args = [[c[k].cuda() for k in ("x", "g", "i", "A_log", "dy", "h0", "dhT")] for c in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = []
        for s, (x, g, i, A, dy, h0, dhT) in zip(streams, args):
            y, hT, kept, _ = ops.recurrence_fwd(x, g, i, A, h0=h0, want_kept=True, stream=s)
            got.append(dict(ops.recurrence_bwd(x, g, i, A, dy, kept, h0=h0, dhT=dhT, stream=s), y=y, hT=hT, kept=kept))
    torch.cuda.synchronize()
    assert all(torch.equal(a[k], b[k]) for a, b in zip(want, got) for k in a)


def test_offsets_beyond_32_bits():
    """Token tensors of 2.2 G elements: short sequences at both ends are those of a small call."""
    T, D = 137000, 16384
    lens = [100, T - 250, 150]
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, g, i, dy = (torch.empty(T, D, dtype=BF, device="cuda").normal_(generator=gen) for _ in range(4))
    A, h0 = torch.full((D,), -1.0, device="cuda"), torch.randn(3, D, generator=gen, device="cuda")
    y, hT, kept, _ = ops.recurrence_fwd(x, g, i, A, h0=h0, cu_seqlens=offsets(lens), want_kept=True)
    grads = ops.recurrence_bwd(x, g, i, A, dy, kept, h0=h0, cu_seqlens=offsets(lens))
    for n, r in ((0, slice(0, 100)), (2, slice(T - 150, T))):
        for cols in (slice(0, 8), slice(D - 8, D)):
            ref = O.recurrence(x[r, cols], g[r, cols], i[r, cols], A[cols], [r.stop - r.start], h0[n:n + 1, cols], dy[r, cols])
            O.check("y", y[r, cols], ref["y"])
            O.check("hT", hT[n:n + 1, cols], ref["hT"])
            for name in ("dx", "dg_raw", "di_raw"):
                O.check(name, grads[name][r, cols], ref[name])
