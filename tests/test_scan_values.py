"""The gated recurrence where its values leave the ordinary: normalisers up to the largest with
logits below where their gates saturate, slopes of gates that forget, infinite inputs and states."""
import numpy as np
import pytest

from oracle import ops_oracle as oo

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

from test_scan import BF16, F16, F32, check, host, inputs, near  # noqa: E402

# one block a tile, and rows split over a cluster (more than two steps of a block, few tiles)
FORMS = [(3, 90, 96), (1, 700, 64)]


@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("tau", [1000.0, 1420.0, 2048.0, 2.0 ** 20])
@pytest.mark.parametrize("B,L,D", FORMS)
def test_large_normalisers(B, L, D, tau, dtype, tied):
    """Logits around -tau / 2, where the gate leaves its expansion, far below it, the type's lowest
    value and -inf, each in a few rows between ordinary ones."""
    x, z, M, h0, dh, dlast = inputs(B, L, D, dtype, state=True, seed=int(tau) % 97 + L)
    g = torch.Generator().manual_seed(1)
    low = torch.finfo(dtype).min
    for k, v in enumerate((-tau / 2, -tau, -1e4, -2 * tau, low, float("-inf"))):
        at = torch.rand(B, L, generator=g) < 0.02
        at[:, 5 + 7 * k] = True
        z[at] = ((0.8 + 0.4 * torch.rand(int(at.sum()), D, generator=g)) * max(v, low / 2) if v > low else
                 torch.full((int(at.sum()), D), v)).to(dtype)
    check(x, z, M, h0, dh, dlast, tau=tau, tied=tied)


@pytest.mark.parametrize("tau", [16.0, 2048.0, 2.0 ** 20])
def test_minus_infinity_empties_at_every_normaliser(tau):
    """Prompt and step agree, and nothing of before a logit of -inf is left."""
    from scale_gated_linear_b200 import gated_scan, gated_scan_step
    for B, L, D in FORMS:
        x, z, _, h0, _, _ = (None if t is None else t.cuda() for t in inputs(B, L, D, F32, state=True, seed=8))
        z[:, L // 2] = float("-inf")
        h, last = gated_scan(x, z, initial_state=h0, gate_normalizer=tau)
        assert torch.equal(h[:, L // 2], x[:, L // 2])
        state = h0.clone()
        gated_scan_step(x[:, L // 2], z[:, L // 2], state, gate_normalizer=tau)
        assert torch.equal(state, x[:, L // 2])
