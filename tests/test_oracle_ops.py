"""Pins of the fp64 oracle of the gated recurrence and of group normalisation: closed
forms and central differences, no GPU."""
import numpy as np
import pytest

from oracle import ops_oracle as oo


def differences(f, a, step=1e-6):
    """Central differences of the scalar f in every element of a."""
    d = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + step
        hi = f()
        a[i] = keep - step
        lo = f()
        a[i] = keep
        d[i] = (hi - lo) / (2 * step)
    return d


def test_constant_gate_is_a_geometric_sum():
    L, z, tau = 50, 0.7, 4.0
    a = (1 / (1 + np.exp(-z))) ** (1 / tau)
    h, last, _ = oo.scan(np.ones((1, L, 1)), np.full((1, L, 1), z), tau)
    want = (1 - a ** np.arange(1, L + 1)) / (1 - a)
    assert np.allclose(h[0, :, 0], want, rtol=1e-13) and last[0, 0] == h[0, -1, 0]
    tied, _, _ = oo.scan(np.ones((1, L, 1)), np.full((1, L, 1), z), tau, tied=True)
    assert np.allclose(tied[0, :, 0], want * (1 - a), rtol=1e-12)


def test_gate_limits():
    z = np.array([[[np.inf], [-np.inf], [np.inf]]])
    x = np.array([[[2.0], [3.0], [5.0]]])
    h, last, _ = oo.scan(x, z, 16.0, h0=np.array([[1.0]]))
    assert h[0, :, 0].tolist() == [3.0, 3.0, 8.0]
    h, _, _ = oo.scan(x, z, 16.0, tied=True, h0=np.array([[1.0]]))
    assert h[0, :, 0].tolist() == [1.0, 3.0, 3.0]


def test_padding_is_skipped():
    rng = np.random.default_rng(0)
    x, z, m = rng.normal(size=(1, 9, 3)), rng.normal(size=(1, 9, 3)), np.array([[0, 1, 1, 0, 0, 1, 0, 1, 0]])
    x[:, m[0] == 0] = np.nan
    h, last, _ = oo.scan(x, z, 2.0, mask=m, h0=np.ones((1, 3)))
    short, slast, _ = oo.scan(x[:, m[0] == 1], z[:, m[0] == 1], 2.0, h0=np.ones((1, 3)))
    assert np.array_equal(h[:, m[0] == 1], short) and np.array_equal(last, slast) and not h[:, m[0] == 0].any()


@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("tau", [1.0, 16.0])
def test_scan_gradients_are_differences(tied, tau):
    rng = np.random.default_rng(1)
    B, L, D = 2, 6, 3
    x, z, h0 = rng.normal(size=(B, L, D)), rng.normal(size=(B, L, D)) * 2, rng.normal(size=(B, D))
    m = rng.random((B, L)) < 0.7
    dh, dlast = rng.normal(size=(B, L, D)), rng.normal(size=(B, D))

    def loss():
        h, last, _ = oo.scan(x, z, tau, tied, m, h0)
        return (h * dh).sum() + (last * dlast).sum()

    dx, dz, dh0, _ = oo.scan_backward(dh, dlast, x, z, tau, tied, m, h0)
    for got, a in ((dx, x), (dz, z), (dh0, h0)):
        assert np.allclose(got, differences(loss, a), atol=1e-8)


def test_norm_statistics():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(2, 40, 12)) * 3 + 5
    y = oo.group_norm(x, 3, eps=1e-12).reshape(2, 40, 3, 4)
    assert np.allclose(y.mean((1, 3)), 0, atol=1e-12) and np.allclose((y ** 2).mean((1, 3)), 1)
    r = oo.group_norm(x, 3, eps=1e-12, center=False).reshape(2, 40, 3, 4)
    assert np.allclose((r ** 2).mean((1, 3)), 1)
    m = np.zeros((2, 40), int)
    m[0, 5:9] = 1
    part = oo.group_norm(x, 3, mask=m)
    assert np.array_equal(part[0, 5:9], oo.group_norm(x[:1, 5:9], 3)[0]) and not part[1].any() and not part[0, :5].any()


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
def test_norm_gradients_are_differences(center, gated, act):
    rng = np.random.default_rng(3)
    x, w, b = rng.normal(size=(2, 4, 6)) + 0.5, rng.normal(size=6), rng.normal(size=6)
    gate = rng.normal(size=(2, 4, 6)) if gated else None
    m, dy = np.array([[1, 0, 1, 1], [1, 1, 1, 0]]), rng.normal(size=(2, 4, 6))
    kw = dict(gate=gate, mask=m, act=act, eps=1e-3, center=center)
    _, (dx, dw, db, dg) = oo.group_norm(x, 2, w, b, dy=dy, **kw)
    for got, a in ((dx, x), (dw, w), (db, b)) + (((dg, gate),) if gated else ()):
        assert np.allclose(got, differences(lambda: (oo.group_norm(x, 2, w, b, **kw) * dy).sum(), a), atol=1e-7)
