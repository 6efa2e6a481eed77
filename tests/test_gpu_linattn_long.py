"""Linear attention on the GPU where one block goes through many chunks, units or segments: against masked products
in 64 bits, with decays that still tell after thousands of tokens. Tolerances are those of test_gpu_linattn.py."""
import pytest
import torch

import linattn_oracle as O
import linattn_products as P
from kimi_delta_attention_15_gb300 import ops
from test_gpu_linattn import check, dev, run

pytestmark = pytest.mark.gpu


def against_products(lens, H, G=1, seed=1, backward=True, states=True):
    d = O.make(lens, H, G, seed=seed, h0=states, dhT=states, log_decay=P.slow_decays(H))
    out = run(d, backward=backward)
    ref = P.reference(dev(d), backward=backward)
    for k, x in out.items():
        check(k, x, ref[k])
    return d, out


# Split calls of more units than multiprocessors. In the pass over the segments' own states a sequence's last segment
# (reversed: its first) has no chunks, nor has a whole sequence; empty sequences have none in the main pass. In each of these
# a block takes such a unit before one with chunks, of another head or direction.
@pytest.mark.parametrize("lens,H,backward", [((3600,), 17, True), ((1983, 0, 1466, 211), 17, True), ((8870,), 23, True),
                                             ((512, 0, 821, 1, 1, 419, 725), 21, False), ((214, 1059, 0, 0, 0, 0, 1), 11, False),
                                             ((1, 0, 0, 1224, 0, 80, 80), 4, True), ((0, 129, 1) * 400, 1, True)])
def test_units_without_chunks_before_units_with(lens, H, backward):
    d, out = against_products(lens, H, backward=backward)
    for _ in range(3):
        again = run(d, backward=backward)
        for k, x in out.items():
            assert torch.equal(x, again[k]), k


@pytest.mark.parametrize("lens,H,G", [((1, 100, 2600, 40, 2, 512, 300, 1), 4, 2), ((1500, 3, 700, 1, 1, 129), 24, 1), ((4000,), 2, 1)])
@pytest.mark.parametrize("states", [False, True])
def test_the_first_rows_of_every_sequence_round_their_outputs_only(lens, H, G, states):
    """The bound that test_gpu_linattn.py derives for short calls holds for the first 512 rows of each sequence (for dk and
    dv the last 512, where their sums start), whatever else is in the call: short sequences among long ones too."""
    d = O.make(lens, H, G, seed=31, h0=states, dhT=states)
    out, ref = run(d), P.reference(dev(d))
    for n, length in enumerate(lens):
        first = sum(lens[:n])
        most = min(length, 512)
        for k in ("o", "dq", "dk", "dv"):
            at = slice(first, first + most) if k in ("o", "dq") else slice(first + length - most, first + length)
            x, r = out[k][at].double(), ref[k][at]
            assert ((x - r).norm() / r.norm()).item() <= 0.51 * 2.0 ** -8, (k, n)


# fixed and packed lengths that are split into segments, the last one short, shared heads among them; with decays under which a
# wrong weight of a segment's state shows
@pytest.mark.parametrize("lens,H,G", [((2950,), 4, 1), ((3000,), 8, 4), ((2100, 0, 900, 131), 6, 3), ((4099, 1), 8, 8), ((1, 1700, 260), 5, 1)])
@pytest.mark.parametrize("states", [False, True])
def test_split_sequences(lens, H, G, states):
    against_products(lens, H, G, seed=len(lens) + H, states=states)


# no segments: units of up to 24 chunks, and blocks that go through several of them
@pytest.mark.parametrize("lens,H,G", [((3001,), 152, 1), ((1000,), 120, 4), ((1000, 900, 1), 100, 2), ((1000, 900, 1, 300), 60, 1)])
def test_long_units_one_after_another(lens, H, G):
    against_products(lens, H, G, seed=H)


@pytest.mark.parametrize("B,T,H,G", [(3, 1500, 4, 1), (2, 2500, 8, 4), (3, 700, 64, 2)])
def test_batches_of_long_sequences(B, T, H, G):
    d = O.make((T,) * B, H, G, seed=B, h0=True, dhT=True, log_decay=P.slow_decays(H))
    c = dev(d)
    four = {k: c[k].view(B, T, -1, 128) for k in ("q", "k", "v", "do")}
    o, hT, _ = ops.linattn_fwd(four["q"], four["k"], four["v"], c["log_decay"], h0=c["h0"])
    g = ops.linattn_bwd(four["q"], four["k"], four["v"], c["log_decay"], four["do"], h0=c["h0"], dhT=c["dhT"])
    ref = P.reference(c)
    for k, x in dict(o=o, hT=hT, **g).items():
        check(k, x, ref[k])


@pytest.mark.parametrize("lens", [(3000,), (1900, 0, 700)])
def test_split_calls_in_a_graph(lens):
    """Three dependent launches a call (four when packed), shared heads: captured and replayed."""
    d = O.make(lens, 8, 4, seed=6, h0=True, dhT=True, log_decay=P.slow_decays(8))
    c, ref = dev(d), P.reference(dev(d))
    cu = c["cu_seqlens"] if len(lens) > 1 else None
    args = (c["q"], c["k"], c["v"], c["log_decay"])
    ws = ops.linattn_alloc_workspace(ops._linattn_shape_of(c["q"], c["v"], cu, 1, ops.SCALE), "cuda", backward=True)
    o, hT = torch.empty_like(c["v"]), torch.empty_like(c["h0"])
    g = dict(dq=torch.empty_like(c["q"]), dk=torch.empty_like(c["k"]), dv=torch.empty_like(c["v"]), dh0=torch.empty_like(hT))

    def step():
        ops.linattn_fwd(*args, h0=c["h0"], cu_seqlens=cu, workspace=ws, o=o, hT=hT)
        ops.linattn_bwd(*args, c["do"], ws, h0=c["h0"], cu_seqlens=cu, dhT=c["dhT"], grads=g)

    step()
    torch.cuda.synchronize()
    outs = dict(o=o, hT=hT, **g)
    eager = {k: x.clone() for k, x in outs.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for x in outs.values():
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert ops.device_status(ws) == 0
        for k, x in outs.items():
            assert torch.equal(x, eager[k]), k
    for k, x in outs.items():
        check(k, x, ref[k])


@pytest.mark.parametrize("lens,H", [((700,), 4), ((3000,), 8), ((512, 0, 821, 1, 1, 419, 725), 21), ((2500, 130, 2500, 257), 20), ((60, 5), 2)])
def test_final_states_in_the_place_of_the_initial_ones(lens, H):
    """Segments of one sequence run at the same time: the last writes the state while the first may not have read it yet."""
    d = dev(O.make(lens, H, seed=H, h0=True, log_decay=P.slow_decays(H)))
    cu = d["cu_seqlens"] if len(lens) > 1 else None
    args = (d["q"], d["k"], d["v"], d["log_decay"])
    o, hT, _ = ops.linattn_fwd(*args, h0=d["h0"], cu_seqlens=cu)
    for _ in range(5):
        state = d["h0"].clone()
        o2, same, ws = ops.linattn_fwd(*args, h0=state, hT=state, cu_seqlens=cu)
        assert same is state and ops.device_status(ws) == 0
        assert torch.equal(o2, o) and torch.equal(state, hT)
