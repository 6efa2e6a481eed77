"""The norm of queries and keys with the position rotation on the GPU against its formulas in 64 bits; tolerances
are the bounds of mixer_oracle."""
import pytest
import torch

import mixer_oracle as O
from kimi_delta_attention_15_gb300 import ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def make(T, Hq, Hk, head, rotary, dtype=BF, seed=0, far=1 << 20, weights=True):
    gen = torch.Generator().manual_seed(seed + T + 100 * head + rotary)
    r = lambda *s: torch.randn(*s, generator=gen)
    c = dict(q=r(T, Hq, head), k=r(T, Hk, head), dq_out=r(T, Hq, head), dk_out=r(T, Hk, head))
    c = {n: (v * torch.exp(r(1, v.shape[1], 1))).to(dtype) for n, v in c.items()}
    c["q_weight"], c["k_weight"] = (1 + 0.2 * r(head), 1 + 0.2 * r(head)) if weights else (None, None)
    c["positions"] = torch.randint(0, far, (T,), generator=gen)
    c["inv_freq"] = 10000.0 ** (-torch.arange(0, rotary, 2) / max(1, rotary))
    return c


def inputs(c, fused):
    """q, k on the GPU, as they are or as columns of a projection of queries, keys and values."""
    if not fused:
        return c["q"].cuda(), c["k"].cuda()
    T, Hq, head = c["q"].shape
    Hk = c["k"].shape[1]
    whole = torch.cat([c["q"].reshape(T, -1), c["k"].reshape(T, -1), torch.zeros(T, 2 * Hk * head, dtype=c["q"].dtype)], 1).cuda()
    return whole[:, :Hq * head].unflatten(1, (Hq, head)), whole[:, Hq * head:(Hq + Hk) * head].unflatten(1, (Hk, head))


def dev(t):
    return None if t is None else t.cuda()


def run(c, interleaved=False, fused=False):
    q, k = inputs(c, fused)
    rest = (dev(c["q_weight"]), dev(c["k_weight"]), c["positions"].cuda(), c["inv_freq"].cuda())
    yq, yk = ops.qknorm_fwd(q, k, *rest, eps=EPS, interleaved=interleaved)
    grads = None
    if fused:
        buf = torch.cat([q.flatten(1), k.flatten(1)], 1)
        grads = dict(dq=buf[:, :q[0].numel()].unflatten(1, q.shape[1:]), dk=buf[:, q[0].numel():].unflatten(1, k.shape[1:]),
                     dq_weight=torch.empty(q.shape[-1], device="cuda"), dk_weight=torch.empty(q.shape[-1], device="cuda"))
    g = ops.qknorm_bwd(q, k, c["dq_out"].cuda(), c["dk_out"].cuda(), *rest, eps=EPS, interleaved=interleaved, grads=grads)
    return dict(g, q=yq, k=yk)


def verify(c, got, interleaved):
    theta = O.angles(c["positions"], c["inv_freq"])
    for n in ("q", "k"):
        if c[n].shape[1] == 0:
            continue
        O.check(n, got[n], O.qknorm(c[n], c[n + "_weight"], theta, interleaved, EPS)["y"])
        ref = O.qknorm(c[n], c[n + "_weight"], theta, interleaved, EPS, c["d" + n + "_out"])
        O.check("d" + n, got["d" + n], ref["dx"])
        O.check("d" + n + "_weight", got["d" + n + "_weight"], ref["dw"])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 4, 1), (3, 5, 2), (64, 32, 8), (130, 7, 7), (1, 96, 96), (33, 2, 3)])
def test_tokens_and_heads(T, Hq, Hk, dtype, interleaved):
    c = make(T, Hq, Hk, 128, 128, dtype)
    verify(c, run(c, interleaved), interleaved)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("head,rotary", [(8, 8), (8, 0), (16, 16), (16, 8), (24, 24), (40, 16), (64, 64), (80, 80), (96, 32), (120, 104),
                                         (128, 64), (128, 0), (136, 136), (192, 192), (256, 256), (256, 64), (248, 248)])
def test_head_sizes(head, rotary, dtype, interleaved, fused):
    c = make(9, 5, 2, head, rotary, dtype)
    verify(c, run(c, interleaved, fused), interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_many_tokens(interleaved):
    c = make(6500, 3, 1, 64, 64)
    verify(c, run(c, interleaved), interleaved)


@pytest.mark.parametrize("T,Hq,Hk,head,dtype", [(2600, 24, 8, 64, BF), (2433, 9, 3, 128, F32), (5000, 12, 12, 72, BF)])
def test_tokens_left_after_whole_rounds(T, Hq, Hk, head, dtype):
    """More tokens than warps: the last ones are shared by several."""
    c = make(T, Hq, Hk, head, head, dtype)
    verify(c, run(c, True), True)


@pytest.mark.parametrize("far", [1 << 31, 1 << 40])
def test_far_positions(far):
    """Angles of many turns. A fraction of a turn is off by 2^-64 of its position, 2^-24 of a turn at 2^40: four of the eight
    steps that the bound allows a sine are left for it."""
    c = make(40, 2, 1, 128, 128, F32, far=far)
    c["positions"][::2] -= far
    verify(c, run(c), False)


def test_frequencies_of_any_size():
    c = make(30, 2, 1, 64, 64, F32, far=1 << 16)
    gen = torch.Generator().manual_seed(3)
    c["inv_freq"] = torch.exp2(40 * torch.rand(32, generator=gen) - 30) * torch.where(torch.rand(32, generator=gen) < 0.5, -1.0, 1.0)
    c["inv_freq"][:4] = torch.tensor([0.0, 1e-42, 2.0 ** -100, 2.0 ** 23 + 1])
    verify(c, run(c), False)


def test_without_weights_and_keys():
    c = make(20, 3, 2, 128, 128, weights=False)
    got = run(c)
    verify(c, got, False)
    q, dq = c["q"].cuda(), c["dq_out"].cuda()
    rest = dict(positions=c["positions"].cuda(), inv_freq=c["inv_freq"].cuda())
    yq, yk = ops.qknorm_fwd(q, **rest)
    assert yk is None and torch.equal(yq, got["q"])
    g = ops.qknorm_bwd(q, None, dq, None, **rest)
    assert torch.equal(g["dq"], got["dq"]) and g["dk"] is None and g["dk_weight"] is None
    # the weight's sum is split over other warps where there are no keys: another order
    O.check("dq_weight", g["dq_weight"], O.qknorm(c["q"], None, O.angles(c["positions"], c["inv_freq"]), False, EPS, c["dq_out"])["dw"])
    g = ops.qknorm_bwd(q, None, dq, None, **rest, want_dweight=False)
    assert torch.equal(g["dq"], got["dq"]) and g["dq_weight"] is None
    g = ops.qknorm_bwd(q, None, dq, None, **rest, grads=dict(dq=torch.empty_like(q)))
    assert torch.equal(g["dq"], got["dq"])


def test_norm_alone():
    c = make(20, 3, 2, 96, 0)
    verify(c, run(c), False)
    y, _ = ops.qknorm_fwd(c["q"].cuda(), c["k"].cuda(), c["q_weight"].cuda(), c["k_weight"].cuda())
    assert torch.equal(y, run(c)["q"])


def test_zero_and_huge_rows():
    """A row of zeros stays zero; rows of 1e15 and 1e-15 are as others (the square of the latter is lost beside eps)."""
    c = make(4, 2, 1, 64, 64, F32)
    c["q"][0] = 0
    c["q"][1] *= 1e15
    c["q"][2] *= 1e-15
    got = run(c)
    assert (got["q"][0] == 0).all()
    verify(c, got, False)


def test_a_bad_head_stays_by_itself():
    c = make(6, 4, 2, 64, 64, F32)
    clean = run(c)
    c["q"][2, 1, 7] = float("nan")
    c["dk_out"][3, 0, 2] = float("inf")
    got = run(c)
    for n, at in (("q", (2, 1)), ("dq", (2, 1)), ("k", None), ("dk", (3, 0))):
        same = got[n] == clean[n]
        if at:
            same[at] = True
        assert same.all(), n


def test_no_tokens():
    q = torch.empty(0, 3, 64, dtype=BF, device="cuda")
    assert ops.qknorm_fwd(q, q)[0].shape == (0, 3, 64)
    g = ops.qknorm_bwd(q, q, q, q)
    assert (g["dq_weight"] == 0).all() and (g["dk_weight"] == 0).all()


def test_batches():
    c = make(12, 3, 2, 64, 64)
    want = run(c)
    q, k = (c[n].cuda().view(3, 4, *c[n].shape[1:]) for n in ("q", "k"))
    rest = (c["q_weight"].cuda(), c["k_weight"].cuda(), c["positions"].cuda().view(3, 4), c["inv_freq"].cuda())
    yq, yk = ops.qknorm_fwd(q, k, *rest)
    assert yq.shape == q.shape and torch.equal(yq.flatten(0, 1), want["q"]) and torch.equal(yk.flatten(0, 1), want["k"])


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(interleaved):
    c = make(50, 4, 2, 128, 64)
    want = run(c, interleaved)
    q, k = inputs(c, True)
    rest = (c["q_weight"].cuda(), c["k_weight"].cuda(), c["positions"].cuda(), c["inv_freq"].cuda())
    ops.qknorm_fwd(q, k, *rest, interleaved=interleaved, q_out=q, k_out=k)
    assert torch.equal(q, want["q"]) and torch.equal(k, want["k"])
    for over in ("x", "dy"):
        q, k, dq, dk = (c[n].cuda() for n in ("q", "k", "dq_out", "dk_out"))
        grads = dict(dq=q if over == "x" else dq, dk=k if over == "x" else dk)
        ops.qknorm_bwd(q, k, dq, dk, *rest, interleaved=interleaved, grads=grads)
        assert torch.equal(grads["dq"], want["dq"]) and torch.equal(grads["dk"], want["dk"])


def test_around_the_outputs_stays():
    c = make(10, 2, 1, 64, 64, F32)
    buf = torch.full((12, 3 * 64 + 16), 7.0, device="cuda")
    ops.qknorm_fwd(c["q"].cuda(), c["k"].cuda(), positions=c["positions"].cuda(), inv_freq=c["inv_freq"].cuda(),
                   q_out=buf[:10, 8:136].unflatten(1, (2, 64)), k_out=buf[:10, 136:200].unflatten(1, (1, 64)))
    inside = torch.zeros(12, 208, dtype=torch.bool)
    inside[:10, 8:200] = True
    assert (buf.cpu()[~inside] == 7.0).all() and (buf.cpu()[inside] != 7.0).all()


def test_the_same_bits_and_captured():
    c = make(700, 6, 2, 128, 128)
    want = run(c)
    again = run(c)
    assert all(torch.equal(want[n], again[n]) for n in want)
    q, k, dq, dk = (c[n].cuda() for n in ("q", "k", "dq_out", "dk_out"))
    rest = (c["q_weight"].cuda(), c["k_weight"].cuda(), c["positions"].cuda(), c["inv_freq"].cuda())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yq, yk = ops.qknorm_fwd(q, k, *rest)
        g = ops.qknorm_bwd(q, k, dq, dk, *rest)
    for _ in range(2):
        for t in (yq, yk, *g.values()):
            t.fill_(float("nan"))
        graph.replay()
        got = dict(g, q=yq, k=yk)
        assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("T,Hq,Hk,head,rotary,interleaved,dtype", [
    (387, 18, 9, 240, 240, True, F32), (198, 72, 9, 200, 0, False, F32), (387, 18, 9, 192, 192, True, F32), (900, 72, 9, 128, 128, False, F32),
    (900, 72, 9, 256, 256, False, F32), (900, 72, 9, 128, 128, False, BF), (3000, 27, 9, 72, 72, True, BF)])
def test_rows_stay_until_they_are_read(T, Hq, Hk, head, rotary, interleaved, dtype):
    """Several blocks of rows to a warp, which arrive in the places of those before them, many times over."""
    c = make(T, Hq, Hk, head, rotary, dtype, seed=5)
    want = run(c, interleaved)
    verify(c, want, interleaved)
    for _ in range(60):
        got = run(c, interleaved)
        assert all(torch.equal(got[n], want[n]) for n in want)


def test_on_other_streams_at_once():
    cases = [make(900, 6, 2, 128, 128, seed=s) for s in range(3)]
    want = [run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    args = [[c[n].cuda() for n in ("q", "k", "dq_out", "dk_out", "q_weight", "k_weight", "positions", "inv_freq")] for c in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, (q, k, dq, dk, *rest) in zip(streams, args):
            yq, yk = ops.qknorm_fwd(q, k, *rest, stream=s)
            got.append(dict(ops.qknorm_bwd(q, k, dq, dk, *rest, stream=s), q=yq, k=yk))
    torch.cuda.synchronize()
    assert all(torch.equal(a[n], b[n]) for a, b in zip(want, got) for n in a)


def test_offsets_beyond_32_bits():
    T, H, head = 140000, 128, 128
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, dq = (torch.empty(T, H, head, dtype=BF, device="cuda").normal_(generator=gen) for _ in range(2))
    p, f = torch.arange(T, device="cuda"), 10000.0 ** (-torch.arange(0, 128, 2, device="cuda") / 128)
    y, _ = ops.qknorm_fwd(q, positions=p, inv_freq=f)
    g = ops.qknorm_bwd(q, None, dq, None, positions=p, inv_freq=f, want_dweight=False)
    r = slice(T - 3, T)
    theta = O.angles(p[r], f)
    O.check("y", y[r], O.qknorm(q[r], None, theta, False, EPS)["y"])
    O.check("dq", g["dq"][r], O.qknorm(q[r], None, theta, False, EPS, dq[r])["dx"])
