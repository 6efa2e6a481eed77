"""Linear attention on the GPU where one block goes through many chunks, units or segments: against masked products
in 64 bits, with decays that still tell after thousands of tokens. Tolerances are those of test_gpu_linattn.py."""
import pytest
import torch

import linattn_oracle as O
import linattn_products as P
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
