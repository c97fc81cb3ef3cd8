"""Group normalisation over sequences at the borders of its forms: samples held in the shared memory of
a cluster up to the most that it holds, and larger ones in two passes, with 16-byte vectors."""
import numpy as np
import pytest

from oracle import ops_oracle as oo

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

from test_group_norm import BF16, F16, F32, check, host, near  # noqa: E402

# norm_error counts 192 roundings, for at most 96 additions in a row in one thread. A thread of the held
# form adds up to 400 values (1600 rows of a block by 32 at once, 8 channels): 400 + 96 < 3 * 192.
HELD = 3


def compare(x, G, w, b, gate, mask, act, center, dy, eps, factor, dtype):
    """Forward and backward on the GPU against the oracle; x [N, S, C]."""
    from scale_gated_linear_b200 import group_norm_backward, group_norm_forward
    cu = lambda t: None if t is None else t.cuda()
    y, saved = group_norm_forward(x.cuda(), G, cu(w), cu(b), gate=cu(gate), mask=cu(mask), activation=act, eps=eps, center=center)
    dx, dw, db, dg = group_norm_backward(dy.cuda(), saved)
    args = dict(gate=host(gate), mask=None if mask is None else mask.numpy(), act=act, eps=eps, center=center, dy=host(dy))
    wy, (wx, ww, wb, wg) = oo.group_norm(host(x), G, host(w), host(b), **args)
    ey, (ex, ew, eb, eg) = oo.norm_error(host(x), G, host(w), host(b), **args)
    near(y, wy, factor * ey, dtype)
    near(dx, wx, factor * ex, dtype)
    near(dw, ww, factor * ew, F32)
    near(db, wb, factor * eb, F32)
    if gate is not None:
        near(dg, wg, factor * eg, dtype)


@pytest.mark.parametrize("dtype,C", [(BF16, 8), (F16, 8), (F32, 4)])
@pytest.mark.parametrize("S", [12635, 101072, 101073, 102400, 102401])
def test_long_samples_of_one_vector(S, dtype, C):
    """One vector a row: the valid marks of the rows take a sixteenth of the rows' own bytes, and samples
    from about 10^5 rows on no longer fit a cluster."""
    g = torch.Generator().manual_seed(S)
    x, dy = (torch.randn(1, S, C, generator=g) * 2 + 0.5).to(dtype), torch.randn(1, S, C, generator=g).to(dtype)
    w, b = 1 + 0.3 * torch.randn(C, generator=g), 0.3 * torch.randn(C, generator=g)
    mask = (torch.rand(1, S, generator=g) < 0.9).to(torch.uint8) if S == 102400 else None
    compare(x, 1, w, b, None, mask, "silu", True, dy, 1e-5, HELD, dtype)


@pytest.mark.parametrize("N,S,C,G,dtype,gated,center", [
    (1, 12000, 64, 1, BF16, False, True),   # about 190 KB a block forward, two passes backward
    (1, 6200, 64, 4, BF16, False, True),    # the same backward
    (1, 4100, 64, 2, F16, True, False),     # with a gate
    (2, 6300, 32, 1, F32, False, False), (1, 3000, 32, 4, F32, True, True)])
def test_held_near_the_limit(N, S, C, G, dtype, gated, center):
    g = torch.Generator().manual_seed(S)
    r = lambda *s: torch.randn(*s, generator=g)
    x, dy, gate = (r(N, S, C) * 2 + 0.5).to(dtype), r(N, S, C).to(dtype), r(N, S, C).to(dtype) if gated else None
    mask = (torch.rand(N, S, generator=g) < 0.8).to(torch.uint8)
    compare(x, G, 1 + 0.3 * r(C), 0.3 * r(C), gate, mask, "silu", center, dy, 1e-5, HELD, dtype)


# A group of more than 256 vectors, a tile of more than 1.6 MB, and groups that tile borders cut
@pytest.mark.parametrize("mask", [None, "random", "empty"])
@pytest.mark.parametrize("N,S,C,G,dtype", [(2, 300, 4096, 1, BF16), (3, 300, 2048, 1, F32), (2, 14000, 64, 1, BF16),
                                           (1, 7001, 64, 2, F32), (2, 65, 6600, 3, F16)])
def test_two_passes(N, S, C, G, dtype, mask):
    for gated, center in ((True, False), (False, True)):
        check(N, S, C, G, dtype, act="silu", gated=gated, mask=mask, center=center, seed=S, eps=1e-3)


@pytest.mark.parametrize("N,S,C,G,dtype", [(2, 300, 4096, 1, BF16), (1, 14000, 64, 1, BF16), (1, 7001, 64, 2, F32), (2, 1030, 32, 1, F32)])
def test_forms_agree(N, S, C, G, dtype):
    """The same rows from an odd start, which are taken one element at a time: within both forms' bounds."""
    from scale_gated_linear_b200 import group_norm
    g = torch.Generator().manual_seed(S)
    x = (torch.randn(N, S, C, generator=g) + 3).to(dtype)
    odd = torch.empty(x.numel() + 1, dtype=dtype, device="cuda")[1:].view(x.shape).copy_(x)
    a, b = group_norm(x.cuda(), G, activation="silu"), group_norm(odd, G, activation="silu")
    ey = oo.norm_error(host(x), G, act="silu")
    near(a, host(b), 2 * HELD * ey + (0 if dtype == F32 else 2.0 ** -8) * np.abs(host(b)), dtype)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("N,S,C,G", [(2, 4096, 64, 1), (1, 16384, 8, 1), (1, 1000, 256, 8), (2, 14000, 64, 1), (2, 300, 2048, 1)])
def test_constant_samples(N, S, C, G, center):
    """No variance: y = bias to the bit, though 300.1 does not add up exactly. A mean that is off by a few of
    its own steps would give (x - mean)^2 far above this eps. Not centred: one to within 600 roundings."""
    from scale_gated_linear_b200 import group_norm
    b = torch.randn(C, device="cuda")
    y = group_norm(torch.full((N, S, C), 300.1, device="cuda"), G, None, b, eps=1e-12, center=center)
    if center:
        assert torch.equal(y, b.expand(N, S, C))
    else:
        assert (y - b - 1).abs().max() <= 600 * 2.0 ** -24 * (1 + 2 * b.abs().max())


@pytest.mark.parametrize("N,S,C,G", [(2, 4096, 64, 1), (1, 16384, 8, 1), (1, 1000, 256, 8), (2, 14000, 64, 1), (2, 300, 2048, 1)])
def test_far_mean(N, S, C, G):
    """A mean of 300 standard deviations in samples of many rows. The mean may be rounded by U |mean| some 24
    times (blocks of rows are joined by their means, in fewer than 20 steps), beside the sums' roundings of
    values of order one."""
    from scale_gated_linear_b200 import group_norm
    g = torch.Generator().manual_seed(C)
    x = torch.randn(N, S, C, generator=g) + 300
    want = oo.group_norm(host(x), G)
    err = 2.0 ** -24 * (24 * 301 + 3 * 192 * (1 + np.abs(want)))
    near(group_norm(x.cuda(), G), want, err, F32)


def test_workspace_of_many_short_samples():
    """A forward keeps two numbers a group and tile, a backward two a channel beside them: below the tensors' own bytes
    forward, twice the f32 bytes of a row a sample backward."""
    import ctypes
    from scale_gated_linear_b200 import _lib
    lib, n = _lib.load(), ctypes.c_size_t()
    N, S, C = 1000000, 2, 64
    for G in (1, 4):
        cfg = _lib.NormConfig(0, 0, C, G, 0, 1, 1e-5)
        assert lib.msgla_group_norm_workspace_size(cfg, N, S, 0, ctypes.byref(n)) == 0 and n.value <= N * (8 * (G + 4) + 4) + 1024
        assert lib.msgla_group_norm_workspace_size(cfg, N, S, 1, ctypes.byref(n)) == 0 and n.value <= N * (8 * (G + 4) + 4 + 8 * C) + 1024


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape,G", [((6, 96), 3), ((3, 9000), 2), ((2, 40, 64), 4), ((1, 2000, 40), 5), ((2, 300, 4096), 2), ((2, 21, 33), 3)])
def test_values_that_are_not_finite(shape, G, dtype, center):
    """A NaN makes its group NaN, in y and in the gradients; an infinity too where the mean is taken off, and else
    leaves x / inf: the weight-less finite values at the bias. Other groups keep their bits."""
    from scale_gated_linear_b200 import group_norm, group_norm_backward, group_norm_forward
    g = torch.Generator().manual_seed(1)
    x, dy = torch.randn(*shape, generator=g).to(dtype).cuda(), torch.randn(*shape, generator=g).to(dtype).cuda()
    cg = shape[-1] // G
    b = torch.randn(shape[-1], generator=g).cuda()
    clean = group_norm(x, G, None, b, center=center)
    hit = torch.zeros(shape, dtype=torch.bool, device="cuda")
    hit[-1, ..., cg:2 * cg] = True
    at = (-1, cg + 1) if len(shape) == 2 else (-1, shape[1] // 2, cg + 1)
    for bad in (float("nan"), float("inf")):
        x2 = x.clone()
        x2[at] = bad
        y, saved = group_norm_forward(x2, G, None, b, center=center)
        assert torch.equal(y[~hit], clean[~hit])
        if bad != bad or center:
            assert torch.isnan(y[hit]).all()
            dx, _, db, _ = group_norm_backward(dy, saved)
            assert torch.isnan(dx[hit]).all() and not torch.isnan(dx[~hit]).any()
        else:
            want = b.to(dtype).expand(shape).clone()
            want[at] = bad - bad
            assert torch.equal(y[hit].nan_to_num(7.0), want[hit].nan_to_num(7.0))
