"""Linear attention with a decay for each head on the GPU, against the 64-bit recurrence.

Tolerances, from the number formats. A bf16 value (8 significant bits) is rounded by at most
u = 2^-8 of itself, by 0.43 u in the mean square over its mantissas. A bf16 output carries its
own rounding and those of the two operands that are rounded once (the scores inside a chunk, the
state between chunks), which act on disjoint parts of the sum: sqrt(2) 0.43 u = 0.6 u normwise; u
leaves a factor 1.6 for samples of a few hundred values. Elementwise the error is a sum of many
independent roundings, sigma about 0.6 u of the size of its terms, plus u of the value: 8 u. The size of
the terms is taken as the rms of the token's 128 values (tokens and heads differ), or of the whole
tensor's for a token whose terms happen to cancel.
The fp32 states are sums of fp32-accurate products: 1e-5 is 168 roundings of 2^-24. A value
below fp32's smallest normal number may be flushed to zero."""
import pytest
import torch

import linattn_oracle as O
from kimi_delta_attention_15_gb300 import ops

pytestmark = pytest.mark.gpu
U = 2.0 ** -8
TINY = 2.0 ** -126


def check(name, x, ref):
    fp32 = x.dtype == torch.float32
    x, ref = x.double().cpu(), ref.double().cpu().reshape(x.shape)
    if not ref.numel():
        return
    assert torch.isfinite(x).all(), name
    norm = ref.norm()
    if ref.abs().max() <= TINY:
        assert (x.abs() <= 2 * TINY).all(), name
        return
    rel = ((x - ref).norm() / norm).item()
    size = torch.maximum(ref.abs(), ref.square().mean(-1, keepdim=True).sqrt())
    worst = ((x - ref).abs() / size.clamp(min=(norm / ref.numel() ** 0.5).item())).max().item()
    assert rel <= (1e-5 if fp32 else U), f"{name}: rel {rel:.3e}"
    assert worst <= (2e-4 if fp32 else 8 * U), f"{name}: elementwise {worst:.3e}"


def dev(d):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def run(d, packed=None, scale=ops.SCALE, backward=True):
    c = dev(d)
    cu = c["cu_seqlens"] if (len(d["lens"]) > 1 if packed is None else packed) else None
    args = (c["q"], c["k"], c["v"], c["log_decay"])
    o, hT, ws = ops.linattn_fwd(*args, h0=c["h0"], cu_seqlens=cu, scale=scale)
    assert ops.device_status(ws) == 0
    out = dict(o=o, hT=hT)
    if backward:
        shape = ops._linattn_shape_of(c["q"], c["v"], cu, 1, scale)
        ws = ops.linattn_alloc_workspace(shape, "cuda", backward=True)
        out.update(ops.linattn_bwd(*args, c["do"], ws, h0=c["h0"], cu_seqlens=cu, dhT=c["dhT"], scale=scale))
        assert ops.device_status(ws) == 0
    torch.cuda.synchronize()
    return out


def check_all(d, out, scale=ops.SCALE):
    ref = O.forward(d, scale)
    if "dq" in out:
        ref.update(O.backward(d, scale))
    for k, x in out.items():
        check(k, x, ref[k])


# one token, the chunk length (128) and its neighbours, several chunks
@pytest.mark.parametrize("T", [1, 2, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700])
def test_lengths(T):
    d = O.make((T,), 3, seed=T, h0=T % 2 == 0, dhT=T % 3 == 0)
    check_all(d, run(d))


@pytest.mark.parametrize("lens", [(17, 33, 65), (0, 128, 0, 1, 300), (1,) * 9, (0, 0, 5), (129, 127)])
@pytest.mark.parametrize("states", [False, True])
def test_packed(lens, states):
    d = O.make(lens, 4, seed=sum(lens), h0=states, dhT=states)
    check_all(d, run(d))


@pytest.mark.parametrize("H,G", [(4, 2), (6, 3), (8, 8), (5, 1)])
def test_grouped_heads(H, G):
    d = O.make((150, 90), H, G, seed=H, h0=True, dhT=True)
    check_all(d, run(d))


@pytest.mark.parametrize("value", [0.0, -1e-4, -0.05, -1.0, -20.0, -200.0, float("-inf")])
def test_decays(value):
    """From no decay at all to one that keeps nothing of the token before."""
    d = O.make((300,), 2, seed=7, h0=True, dhT=True, log_decay=value)
    check_all(d, run(d))


@pytest.mark.parametrize("lens,H,G", [((1,), 2, 1), ((2,), 16, 4), ((1, 0, 1), 9, 1), ((6,), 2, 2), ((100,), 1, 1), ((60, 68), 3, 1)])
def test_short_calls_round_their_outputs_only(lens, H, G):
    """Within a chunk that starts from zero, short calls carry no rounding but the outputs' own: 0.43 u in the mean
    square, give or take 0.026 u (6%) for the 128 values of a row at least, three times that for a limit."""
    d = O.make(lens, H, G, seed=23 + len(lens))
    out, ref = run(d), {**O.forward(d), **O.backward(d)}
    for k in ("o", "dq", "dk", "dv"):
        x, r = out[k].double().cpu(), ref[k].double()
        assert ((x - r.reshape(x.shape)).norm() / r.norm()).item() <= 0.51 * U, k


@pytest.mark.parametrize("lens,H,G", [((1,), 1, 1), ((0, 1, 3), 2, 1), ((40, 130), 3, 1), ((300, 1, 211), 2, 2), ((512,), 1, 1)])
def test_short_calls_with_states_round_their_outputs_only(lens, H, G):
    """The same for every chunk of a call of up to 512 tokens, with states carried in."""
    d = O.make(lens, H, G, seed=33 + len(lens), h0=True, dhT=True)
    out, ref = run(d), {**O.forward(d), **O.backward(d)}
    check_all(d, out)
    for k in ("o", "dq", "dk", "dv"):
        x, r = out[k].double().cpu(), ref[k].double()
        assert ((x - r.reshape(x.shape)).norm() / r.norm()).item() <= 0.51 * U, k


@pytest.mark.parametrize("scale", [1.0, 0.01])
def test_scale(scale):
    d = O.make((200,), 2, seed=8, h0=True, dhT=True)
    check_all(d, run(d, scale=scale), scale)


def test_batch_of_fixed_length_equals_packed():
    d = O.make((90,) * 3, 4, seed=9, h0=True, dhT=True)
    c = dev(d)
    four = {k: c[k].view(3, 90, -1, 128) for k in ("q", "k", "v", "do")}
    o, hT, _ = ops.linattn_fwd(four["q"], four["k"], four["v"], c["log_decay"], h0=c["h0"])
    g = ops.linattn_bwd(four["q"], four["k"], four["v"], c["log_decay"], four["do"], h0=c["h0"], dhT=c["dhT"])
    check_all(d, dict(o=o, hT=hT, **g))


def test_no_tokens_at_all():
    d = O.make((0, 0), 2, seed=10, h0=True, dhT=True)
    out = run(d)
    assert torch.equal(out["hT"].cpu(), d["h0"]) and torch.equal(out["dh0"].cpu(), d["dhT"])
    d = O.make((0,), 2, seed=10)
    out = run(d, packed=False)
    assert (out["hT"] == 0).all() and (out["dh0"] == 0).all()


def test_a_long_sequence_on_few_heads():
    """Few (sequence, head) pairs and many chunks: the split over the sequence, if any, is exact."""
    d = O.make((5000,), 2, seed=11, h0=True, dhT=True)
    check_all(d, run(d))
    d = O.make((3000, 1, 700, 0, 1299), 1, seed=12, h0=True, dhT=True)
    check_all(d, run(d))


@pytest.mark.parametrize("n,H,G", [(60, 8, 2), (3, 120, 1)])
def test_more_units_than_multiprocessors(n, H, G):
    """Each persistent block goes through several (sequence, head) pairs of one or two chunks, some empty."""
    gen = torch.Generator().manual_seed(n)
    lens = tuple(int(x) for x in torch.randint(0, 260, (n,), generator=gen))
    d = O.make(lens, H, G, seed=n, h0=True, dhT=True)
    check_all(d, run(d))
    d = O.make(lens, H, G, seed=n)
    check_all(d, run(d))


def test_outputs_not_wanted():
    d = dev(O.make((130,), 2, seed=13))
    args = (d["q"], d["k"], d["v"], d["log_decay"])
    o, hT, _ = ops.linattn_fwd(*args, want_hT=False)
    assert hT is None
    g = ops.linattn_bwd(*args, d["do"], want_dh0=False)
    assert g["dh0"] is None
    full = ops.linattn_bwd(*args, d["do"])
    o2, _, _ = ops.linattn_fwd(*args)
    check("o", o, o2.double().cpu())
    for k in ("dq", "dk", "dv"):
        check(k, g[k], full[k].double().cpu())


def test_repeated_calls_agree_bit_for_bit_and_on_another_stream():
    d = O.make((400, 77), 4, 2, seed=14, h0=True, dhT=True)
    a = run(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = run(d)
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_workspace_may_hold_anything():
    """Nothing is read from the workspace that the call itself has not written."""
    d = dev(O.make((513, 20), 4, 2, seed=15, h0=True, dhT=True))
    args = (d["q"], d["k"], d["v"], d["log_decay"])
    shape = ops._linattn_shape_of(d["q"], d["v"], d["cu_seqlens"], 1, ops.SCALE)
    outs = []
    for fill in (0, 255):
        ws = torch.full((ops.linattn_workspace_size(shape, True),), fill, dtype=torch.uint8, device="cuda")
        o, hT, _ = ops.linattn_fwd(*args, h0=d["h0"], cu_seqlens=d["cu_seqlens"], workspace=ws)
        ws.fill_(fill)
        g = ops.linattn_bwd(*args, d["do"], ws, h0=d["h0"], cu_seqlens=d["cu_seqlens"], dhT=d["dhT"])
        assert ops.device_status(ws) == 0
        outs.append(dict(o=o, hT=hT, **g))
    for k in outs[0]:
        assert torch.equal(outs[0][k], outs[1][k]), k


def test_nothing_is_written_outside_the_tensors():
    """Outputs as views between guard rows; the rows of a neighbour hold infinities, which must not leak in."""
    d = dev(O.make((100,), 2, seed=16))
    T, H = 100, 2
    big = {k: torch.full((T + 256, H, 128), float("inf"), dtype=torch.bfloat16, device="cuda") for k in ("q", "k", "v", "do")}
    for k, x in big.items():
        x[128:128 + T] = d[k]
    ins = {k: x[128:128 + T] for k, x in big.items()}
    out = {k: torch.full((T + 256, H, 128), 7.0, dtype=torch.bfloat16, device="cuda") for k in ("o", "dq", "dk", "dv")}
    mid = {k: x[128:128 + T] for k, x in out.items()}
    ops.linattn_fwd(ins["q"], ins["k"], ins["v"], d["log_decay"], o=mid["o"])
    g = dict(dq=mid["dq"], dk=mid["dk"], dv=mid["dv"], dh0=None)
    ops.linattn_bwd(ins["q"], ins["k"], ins["v"], d["log_decay"], ins["do"], grads=g)
    torch.cuda.synchronize()
    host = {k: (v.cpu() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    ref = {**O.forward(host), **O.backward(host)}
    for k, x in out.items():
        assert (x[:128] == 7.0).all() and (x[128 + T:] == 7.0).all(), k
        check(k, mid[k], ref[k])


def test_non_finite_tokens_stay_in_their_sequence_and_head():
    d = O.make((140, 60, 200), 3, seed=17)
    clean = run(d)
    for name in ("q", "k", "v", "do"):
        d[name][150, 1, 5] = float("nan")           # the second sequence, head 1
    out = run(d)
    for k in ("o", "dq", "dk", "dv"):
        for head in range(3):
            for a, b in ((0, 140), (140, 200), (200, 400)):
                if (a, head) != (140, 1):
                    assert torch.equal(out[k][a:b, head], clean[k][a:b, head]), (k, head, a)


@pytest.mark.parametrize("bad", [[0, 40, 30, 100], [0, 50, 100, 99], [1, 50, 70, 100], [0, -5, 70, 100], [0, 1 << 40, 70, 100]])
def test_malformed_offsets_set_the_device_status(bad):
    d = dev(O.make((50, 20, 30), 2, seed=18))
    cu = torch.tensor(bad, dtype=torch.int64, device="cuda")
    o = torch.full_like(d["v"], 7.0)
    hT = torch.full((3, 2, 128, 128), 7.0, device="cuda")
    args = (d["q"], d["k"], d["v"], d["log_decay"])
    _, _, ws = ops.linattn_fwd(*args, cu_seqlens=cu, o=o, hT=hT)
    assert ops.device_status(ws) == 6
    assert (o == 7.0).all() and (hT == 7.0).all()
    g = {k: torch.full_like(d["v"], 7.0) for k in ("dq", "dk", "dv")}
    g["dh0"] = hT
    ws = ops.linattn_alloc_workspace(ops.linattn_shape(100, 2, 3), "cuda", backward=True)
    ops.linattn_bwd(*args, d["do"], ws, cu_seqlens=cu, grads=g)
    assert ops.device_status(ws) == 6
    for x in g.values():
        assert (x == 7.0).all()
    good = O.make((50, 20, 30), 2, seed=18)         # the next call is not affected
    check_all(good, run(good))


@pytest.mark.parametrize("N,H,lens", [(160, 1, (100,)), (3, 1, (4000,)), (1100, 1, (1500,))])
def test_malformed_offsets_of_many_or_long_sequences(N, H, lens):
    """The same where a kernel of its own lists the sequences: many of them, or long ones that are split."""
    T = N - 1 + lens[0]
    x = torch.ones(T, H, 128, dtype=torch.bfloat16, device="cuda")
    log_decay = torch.full((H,), -0.1, device="cuda")
    cu = torch.tensor(list(range(N)) + [T], dtype=torch.int64)
    for at, value in ((0, 1), (N // 2, T + 1), (N, T - 1)):
        bad = cu.clone()
        bad[at] = value
        o, hT = torch.full_like(x, 7.0), torch.full((N, H, 128, 128), 7.0, device="cuda")
        _, _, ws = ops.linattn_fwd(x, x, x, log_decay, cu_seqlens=bad.cuda(), o=o, hT=hT)
        assert ops.device_status(ws) == 6
        assert (o == 7.0).all() and (hT == 7.0).all()


def test_many_short_sequences_beside_long_ones():
    """More sequences than the listing kernel takes at a time; the long ones are split, among the others."""
    lens = [2, 0, 1] * 380
    lens[5], lens[700], lens[-1] = 1900, 2300, 1500
    d = O.make(tuple(lens), 1, seed=21, h0=True, dhT=True)
    check_all(d, run(d))


def test_calls_given_a_stream():
    """`stream`: the call's own tensors belong to it too, so that their memory is not handed out while it runs."""
    d = O.make((300, 45), 4, 2, seed=22, h0=True, dhT=True)
    a, c, side = run(d), dev(d), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args = (c["q"], c["k"], c["v"], c["log_decay"])
    for _ in range(20):
        b = ops.linattn_bwd(*args, c["do"], h0=c["h0"], cu_seqlens=c["cu_seqlens"], dhT=c["dhT"], stream=side)
        o, hT, ws = ops.linattn_fwd(*args, h0=c["h0"], cu_seqlens=c["cu_seqlens"], stream=side)
        torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")      # what the current stream allocates meanwhile
    side.synchronize()
    for k, x in dict(o=o, hT=hT, **b).items():
        assert torch.equal(x, a[k]), k


def test_gradient_against_differences_of_the_loss():
    """<gradient, step> against the central difference of the 64-bit loss along the step: bf16 gradients
    carry at most u each, and n independent errors add up to that times |grad| |step| / sqrt(n)
    in the inner product; five of these are allowed."""
    d = O.make((180,), 2, 2, seed=19, h0=True, dhT=True)
    out = run(d)
    gen = torch.Generator().manual_seed(20)
    for name in ("q", "k", "v", "h0"):
        step = torch.randn(d[name].shape, generator=gen, dtype=torch.float64)
        e = 1e-4
        up, down = (O.loss(dict(d, **{name: d[name].double() + s * step})) for s in (e, -e))
        g = out["d" + name].double().cpu()
        want, got = ((up - down) / (2 * e)).item(), (g * step).sum().item()
        tol = 5 * U * g.norm().item() * step.norm().item() / g.numel() ** 0.5
        assert abs(want - got) <= tol, (name, want, got, tol)


@pytest.mark.parametrize("n_req,H,G", [(1, 1, 1), (37, 4, 1), (5, 6, 3), (64, 8, 4)])
def test_decode_one_step(n_req, H, G):
    d = O.make((1,) * n_req, H, G, seed=n_req, h0=True)
    c = dev(d)
    state = c["h0"].clone()
    o = ops.linattn_decode(c["q"], c["k"], c["v"], c["log_decay"], state)
    torch.cuda.synchronize()
    ref = O.forward(d)
    check("o", o, ref["o"])
    # one fused multiply-add, the exponential (2 units) and the product: 4 roundings of the two terms
    terms = (torch.exp(d["log_decay"].double())[None, :, None, None] * d["h0"].double()).abs() + \
        (d["v"].double()[:, :, :, None] * d["k"].double().repeat_interleave(G, 1)[:, :, None, :]).abs()
    assert ((state.double().cpu() - ref["hT"]).abs() <= 4 * 2.0 ** -24 * terms + 1e-37).all()


def test_prompt_then_tokens_equals_the_whole_prompt():
    T, first, H = 160, 131, 4
    d = O.make((T,), H, 2, seed=21)
    c = dev(d)
    o, state, _ = ops.linattn_fwd(c["q"][:first].contiguous(), c["k"][:first].contiguous(), c["v"][:first].contiguous(),
                                  c["log_decay"])
    outs = [o]
    for t in range(first, T):
        outs.append(ops.linattn_decode(c["q"][t:t + 1].clone(), c["k"][t:t + 1].clone(), c["v"][t:t + 1].clone(),
                                       c["log_decay"], state))
    torch.cuda.synchronize()
    check_all(d, dict(o=torch.cat(outs), hT=state))


def test_decode_in_a_graph():
    d = dev(O.make((1,) * 8, 4, seed=22, h0=True))
    args = (d["q"], d["k"], d["v"], d["log_decay"])
    o = torch.empty_like(d["v"])
    eager = d["h0"].clone()
    for _ in range(3):
        ops.linattn_decode(*args, eager, o=o)
    want = o.clone()
    state = d["h0"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.linattn_decode(*args, state, o=o)
    state.copy_(d["h0"])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(state, eager) and torch.equal(o, want)


def test_forward_and_backward_in_a_graph():
    c = dev(O.make((300, 45), 4, 2, seed=23, h0=True, dhT=True))
    args = (c["q"], c["k"], c["v"], c["log_decay"])
    shape = ops._linattn_shape_of(c["q"], c["v"], c["cu_seqlens"], 1, ops.SCALE)
    ws = ops.linattn_alloc_workspace(shape, "cuda", backward=True)
    o, hT = torch.empty_like(c["v"]), torch.empty_like(c["h0"])
    g = dict(dq=torch.empty_like(c["q"]), dk=torch.empty_like(c["k"]), dv=torch.empty_like(c["v"]), dh0=torch.empty_like(hT))

    def step():
        ops.linattn_fwd(*args, h0=c["h0"], cu_seqlens=c["cu_seqlens"], workspace=ws, o=o, hT=hT)
        ops.linattn_bwd(*args, c["do"], ws, h0=c["h0"], cu_seqlens=c["cu_seqlens"], dhT=c["dhT"], grads=g)

    step()
    torch.cuda.synchronize()
    outs = dict(o=o, hT=hT, **g)
    eager = {k: v.clone() for k, v in outs.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in outs.values():
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert ops.device_status(ws) == 0
    for k, x in outs.items():
        assert torch.equal(x, eager[k]), k
