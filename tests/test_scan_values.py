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


def same_values(got, want, dtype, err=1e-5):
    """The same infinities and NaN, and finite values within half a step and err of the largest."""
    got, half = host(got), 0.0 if dtype == F32 else torch.finfo(dtype).eps / 2
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isposinf(got), np.isposinf(want)) and np.array_equal(np.isneginf(got), np.isneginf(want))
    f = np.isfinite(want)
    if f.any():
        scale = np.abs(want[f]).max()
        assert (np.abs(got[f] - want[f]) <= half * np.abs(want[f]) + err * scale).all()


@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("tau", [1.0, 16.0])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("mask", [None, "random"])
@pytest.mark.parametrize("B,L,D", FORMS + [(2, 130, 33), (1, 16, 2), (1, 1, 1)])
def test_infinite_inputs_and_states(B, L, D, mask, dtype, tau, tied):
    """a h + u of an infinite h is infinite: such a state stays what it is over gates and padded rows, until an
    infinity of the other sign or a gate of zero makes it NaN. The other channels keep their bits."""
    from scale_gated_linear_b200 import gated_scan, gated_scan_backward, gated_scan_forward
    x, z, M, h0, dh, dlast = inputs(B, L, D, dtype, bias=1.0, mask=mask, state=True, seed=L)
    if M is not None:
        M[:, L // 3] = 1
    clean = [None if t is None else t.cuda() for t in (x, z, M, h0, dh, dlast)]
    kw = dict(tied=tied, gate_normalizer=tau)
    inf = float("inf")
    x, z, h0, dh, dlast = (t.clone() for t in (x, z, h0, dh, dlast))
    x[0, L // 3, 0] = inf
    h0[-1, D // 2] = -inf
    dh[0, L // 3, D - 1] = -inf
    dlast[-1, D // 3] = inf
    if D > 8 and L > 8:
        x[0, L // 3, 5], x[0, L // 2, 5] = inf, -inf        # NaN from the second on, where it is valid
        x[0, L // 3, 6], z[0, L // 2, 6] = -inf, -inf       # a gate of zero: 0 * inf
        x[0, L // 3, 7] = float("nan")
    cu = [None if t is None else t.cuda() for t in (x, z, M, h0, dh, dlast)]

    def both(x, z, M, h0, dh, dlast):
        h, last, saved = gated_scan_forward(x, z, mask=M, initial_state=h0, **kw)
        h2, last2 = gated_scan(x, z, mask=M, initial_state=h0, **kw)
        for a, b in ((h, h2), (last, last2)):
            assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
        return (h, last, *gated_scan_backward(dh, dlast, saved))

    got, before = both(*cu), both(*clean)
    m = None if M is None else M.numpy()
    with np.errstate(invalid="ignore"):
        args = (host(x), host(z), tau, tied, m, host(h0))
        want = (*oo.scan(*args)[:2], *oo.scan_backward(host(dh), host(dlast), *args)[:3])
    for k, (a, w) in enumerate(zip(got, want)):
        same_values(a, w, F32 if k in (1, 4) else dtype)
    touched = torch.zeros(B, D, dtype=torch.bool)
    touched[0, [0, D - 1]] = True
    touched[-1, [D // 2, D // 3]] = True
    if D > 8 and L > 8:
        touched[0, 5:8] = True
    for a, b in zip(got, before):
        keep = ~touched if a.dim() == 2 else ~touched[:, None].expand(B, L, D)
        assert torch.equal(a.cpu()[keep], b.cpu()[keep])


def test_infinite_states_in_place():
    """The state taken on in its own buffer, as the C entry allows, with an infinity in it."""
    import ctypes
    from scale_gated_linear_b200 import _lib, gated_scan_backward, gated_scan_forward
    lib = _lib.load()
    for B, L, D in FORMS:
        x, z, _, h0, dh, dlast = (None if t is None else t.cuda() for t in inputs(B, L, D, F32, state=True, seed=2))
        h0[0, 3], dlast[0, 5] = float("inf"), float("-inf")
        cfg = _lib.ScanConfig(0, 2, D, 0, 16.0)
        rows = lambda t: _lib.Rows(t.data_ptr(), L * D, D)
        want, wlast, saved = gated_scan_forward(x, z, initial_state=h0)
        h, state, kept = torch.empty_like(x), h0.clone(), torch.empty_like(saved.states)
        st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        _lib.check(lib.msgla_scan_forward(cfg, B, L, rows(x), rows(z), None, state.data_ptr(), rows(h), state.data_ptr(),
                                          kept.data_ptr(), st))
        assert torch.equal(h, want) and torch.equal(state, wlast) and torch.equal(kept, saved.states)
        assert state[0, 3] == float("inf") and torch.isinf(state).sum() == 1
        dx, dz, grad = torch.empty_like(x), torch.empty_like(x), dlast.clone()
        _lib.check(lib.msgla_scan_backward(cfg, B, L, rows(x), rows(z), None, kept.data_ptr(), rows(dh), grad.data_ptr(),
                                           rows(dx), rows(dz), grad.data_ptr(), st))
        torch.cuda.synchronize()
        for a, b in zip((dx, dz, grad), gated_scan_backward(dh, dlast, saved)):
            assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
        assert grad[0, 5] == float("-inf") and torch.isinf(grad).sum() == 1 and not torch.isnan(grad).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tau", [1.0, 16.0])
def test_step_of_infinite_states(tau, dtype):
    from scale_gated_linear_b200 import gated_scan_step
    B, D = 3, 40
    x, z, _, h0, _, _ = inputs(B, 1, D, dtype, state=True, seed=5)
    inf = float("inf")
    h0[0, 0], h0[1, 1], h0[2, 2], h0[0, 3], x[0, 0, 4], x[1, 0, 1] = inf, -inf, inf, inf, -inf, inf
    z[0, 0, 3] = -inf
    M = torch.tensor([1, 1, 0], dtype=torch.uint8)
    for tied in (False, True):
        state = h0.cuda()
        h = gated_scan_step(x[:, 0].cuda(), z[:, 0].cuda(), state, mask=M.cuda(), gate_normalizer=tau, tied=tied)
        with np.errstate(invalid="ignore"):
            want, last, _ = oo.scan(host(x), host(z), tau, tied, M.numpy()[:, None], host(h0))
        same_values(h, want[:, 0], dtype)
        same_values(state, last, F32)


@pytest.mark.parametrize("B,L,D", FORMS)
def test_infinite_values_without_output_gradients(B, L, D):
    """No gradient of h, an infinite state and an infinite gradient of the last one."""
    from scale_gated_linear_b200 import gated_scan_backward, gated_scan_forward
    x, z, _, h0, _, dlast = inputs(B, L, D, F32, bias=1.0, state=True, seed=6)
    h0[0, 2], dlast[0, 4] = float("inf"), float("-inf")
    for tied in (False, True):
        saved = gated_scan_forward(x.cuda(), z.cuda(), initial_state=h0.cuda(), tied=tied)[2]
        got = gated_scan_backward(None, dlast.cuda(), saved)
        with np.errstate(invalid="ignore"):
            want = oo.scan_backward(None, host(dlast), host(x), host(z), 16.0, tied, None, host(h0))[:3]
        for a, w in zip(got, want):
            same_values(a, w, F32)


@pytest.mark.parametrize("tau", [1.0, 16.0])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,L,D", FORMS + [(1, 1, 2)])
def test_nan_logits(B, L, D, dtype, tau):
    """A NaN among the logits makes its channel NaN from its token on, an infinite state's too, and what comes before
    it in the gradients; the step agrees."""
    from scale_gated_linear_b200 import gated_scan_backward, gated_scan_forward, gated_scan_step
    x, z, _, h0, dh, dlast = inputs(B, L, D, dtype, bias=1.0, state=True, seed=7)
    z[0, L // 2, :2], h0[0, 1], dlast[0, 1] = float("nan"), float("inf"), float("-inf")
    h, last, saved = gated_scan_forward(x.cuda(), z.cuda(), initial_state=h0.cuda(), gate_normalizer=tau)
    got = (h, last, *gated_scan_backward(dh.cuda(), dlast.cuda(), saved))
    with np.errstate(invalid="ignore"):
        args = (host(x), host(z), tau, False, None, host(h0))
        want = (*oo.scan(*args)[:2], *oo.scan_backward(host(dh), host(dlast), *args)[:3])
    for k, (a, w) in enumerate(zip(got, want)):
        same_values(a, w, F32 if k in (1, 4) else dtype)
    state = h0.cuda()
    gated_scan_step(x[:, L // 2].cuda(), z[:, L // 2].cuda(), state, gate_normalizer=tau)
    assert torch.isnan(state[0, :2]).all() and not torch.isnan(state[1:]).any()
