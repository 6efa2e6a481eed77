"""The masked products of linattn_products.py against the recurrence of linattn_oracle.py (CPU, 64 bits)."""
import pytest
import torch

import linattn_oracle as O
import linattn_products as P


@pytest.mark.parametrize("lens,H,G,decay", [((40,), 2, 1, None), ((7, 0, 33, 1), 4, 2, None), ((9, 5), 3, 3, -0.01),
                                            ((20,), 1, 1, float("-inf"))])
def test_products_equal_the_recurrence(lens, H, G, decay):
    d = O.make(lens, H, G, seed=3, h0=True, dhT=True, log_decay=decay)
    got, want = P.reference(d), {**O.forward(d), **O.backward(d)}
    for k, x in want.items():
        assert torch.allclose(got[k].view(x.shape), x, rtol=1e-11, atol=1e-11), k
    assert set(P.reference(d, backward=False)) == {"o", "hT"}


def test_slow_decays_differ():
    g = P.slow_decays(17)
    assert len(set(g.tolist())) == 17 and (g <= 0).all() and g.min() > -0.021 and (g == 0).sum() == 1
