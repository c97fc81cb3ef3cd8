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


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("tau", [0.25, 1.0, 3.0])
@pytest.mark.parametrize("L,at", [(1, 0), (700, 400)])
def test_slopes_of_gates_that_forget(L, at, tau, dtype):
    """dz = g (h0 - x) a (1 - sigmoid(z)) / tau of one valid row, relative to itself, down to a of
    1e-35. With U = 2^-24 the argument of e^-|z| is off by 2 U |z| (product and constant), that of
    a = e^-(S / tau) by 6 U S / tau (S: 3 U, two products, the constant), each exponential by 4 U,
    1 + e by U, each reciprocal by 2 U and the products, g and h0 - x by U each: 24 U besides."""
    from scale_gated_linear_b200 import gated_scan_backward, gated_scan_forward
    D, U = 64, 2.0 ** -24
    g = torch.Generator().manual_seed(3)
    sign = torch.where(torch.rand(1, L, D, generator=g) < 0.5, -1.0, 1.0)
    x, dh = torch.full((1, L, D), 0.5).to(dtype), (sign * (1 + torch.rand(1, L, D, generator=g))).to(dtype)
    z = torch.linspace(-30 if tau >= 1 else -18, -1, D).expand(1, L, D).to(dtype).contiguous()
    h0, M = 1 + torch.rand(1, D, generator=g), torch.zeros(1, L, dtype=torch.uint8)
    M[:, at] = 1
    for tied in (False, True):
        _, _, saved = gated_scan_forward(x.cuda(), z.cuda(), mask=M.cuda(), initial_state=h0.cuda(), gate_normalizer=tau, tied=tied)
        dz = host(gated_scan_backward(dh.cuda(), None, saved)[1])
        want = oo.scan_backward(host(dh), None, host(x), host(z), tau, tied, M.numpy(), host(h0))[1]
        s = oo.softplus_neg(host(z)[0, at]) / tau
        err = U * (2 * np.abs(host(z)[0, at]) + 6 * s + 24) * np.abs(want[0, at])
        near(torch.from_numpy(dz[0, at]), want[0, at], err, dtype)
        assert not dz[0, M[0].numpy() == 0].any()
