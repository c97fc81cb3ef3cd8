"""GPU parity of the gated recurrence (forward, gradients, single tokens) against the fp64
oracle, at sizes, masks, strides and gate values where it can go wrong. A result may be off
by half a step of its type plus the bound that oracle.ops_oracle.scan_error derives for the
32-bit arithmetic on the same inputs."""
import numpy as np
import pytest

from oracle import ops_oracle as oo

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(got, ref, err, dtype):
    """|got - ref| within half a step of dtype and the f32 bound (and half the smallest f16 step)."""
    got, half = host(got), 0.0 if dtype == F32 else torch.finfo(dtype).eps / 2
    tol = half * np.abs(ref) + err * (1 + half) + 2.0 ** -25 * (dtype == F16) + 1e-37
    assert np.isfinite(got).all()
    worst = (np.abs(got - ref) - tol).max() if got.size else 0.0
    assert worst <= 0, f"off by {np.abs(got - ref).max():.3e}, {worst:.3e} more than allowed"


def inputs(B, L, D, dtype, bias=0.0, mask=None, state=False, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    M = None
    if mask == "random":
        M = (torch.rand(B, L, generator=g) < 0.7).to(torch.uint8)
    elif mask == "empty":  # one sequence with nothing in it, one with its last token alone
        M = torch.ones(B, L, dtype=torch.uint8)
        M[0] = 0
        M[-1, :-1] = 0
    elif mask in ("left", "right"):
        pos, pad = torch.arange(L)[None], torch.randint(0, L + 1, (B, 1), generator=g)
        M = (pos >= pad if mask == "left" else pos < L - pad).to(torch.uint8)
    x, z, dh = r(B, L, D).to(dtype), (r(B, L, D) * spread + bias).to(dtype), r(B, L, D).to(dtype)
    h0, dlast = (r(B, D), r(B, D)) if state else (None, None)
    return x, z, M, h0, dh, dlast


def check(x, z, M, h0, dh, dlast, tau=16.0, tied=False, view=lambda t: t.cuda()):
    """Forward and backward through the explicit pair, against the oracle."""
    from scale_gated_linear_b200 import gated_scan, gated_scan_backward, gated_scan_forward
    cu = lambda t: None if t is None else t.cuda()
    poison = lambda t: t if M is None else torch.where(M.bool()[..., None], t, torch.full_like(t, float("nan")))
    dtype = x.dtype
    gx, gz, gdh, gm, gh0 = view(poison(x)), view(poison(z)), view(poison(dh)), cu(M), cu(h0)
    h, last, saved = gated_scan_forward(gx, gz, mask=gm, initial_state=gh0, gate_normalizer=tau, tied=tied)
    dx, dz, dh0 = gated_scan_backward(gdh, cu(dlast), saved)
    h2, last2 = gated_scan(gx, gz, mask=gm, initial_state=gh0, gate_normalizer=tau, tied=tied)
    assert torch.equal(h, h2) and torch.equal(last, last2)
    a = [host(t) for t in (x, z)]
    m, s0, d, dl = (None if M is None else M.numpy()), host(h0), host(dh), host(dlast)
    want, wlast, _ = oo.scan(*a, tau, tied, m, s0)
    wx, wz, w0, _ = oo.scan_backward(d, dl, *a, tau, tied, m, s0)
    e, ex, ez, e0 = oo.scan_error(*a, tau, tied, m, s0, d, dl)
    near(h, want, e[:, 1:] if m is None else e[:, 1:] * (m[..., None] != 0), dtype)
    near(last, wlast, e[:, -1], F32)
    near(dx, wx, ex, dtype)
    near(dz, wz, ez, dtype)
    assert (dh0 is None) == (h0 is None)
    if h0 is not None:
        near(dh0, w0, e0, F32)


@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("B,L,D", [(1, 1, 1), (2, 3, 7), (1, 16, 64), (3, 63, 66), (2, 64, 65), (2, 65, 130), (1, 128, 2),
                                   (2, 129, 40), (1, 257, 96), (5, 200, 333)])
def test_sizes(B, L, D, dtype, tied):
    check(*inputs(B, L, D, dtype, bias=1.0, state=True, seed=L + D), tied=tied)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,L,D,tau", [(1, 1500, 64, 16.0), (1, 2111, 34, 1.0), (2, 1025, 128, 16.0), (1, 4096, 32, 8.0)])
def test_long_sequences(B, L, D, tau, dtype):
    """More rows than one block holds, alone and with few channels (rows split over blocks)."""
    check(*inputs(B, L, D, dtype, bias=3.0, state=True, seed=L), tau=tau, tied=True)


@pytest.mark.parametrize("B,D,L", [(40, 256, 40), (300, 64, 5), (2, 4096, 70), (33, 512, 130)])
def test_many_channels(B, D, L):
    """More channel tiles than the GPU runs at once."""
    check(*inputs(B, L, D, BF16, seed=D))


@pytest.mark.parametrize("mask", ["left", "right", "random", "empty"])
@pytest.mark.parametrize("B,L,D,dtype", [(4, 150, 66, BF16), (3, 301, 33, F32), (2, 64, 128, F16), (2, 1, 8, BF16)])
def test_padding(B, L, D, dtype, mask):
    """NaN in every padded row of x, gate and dh: none of it may be read."""
    for state in (False, True):
        check(*inputs(B, L, D, dtype, mask=mask, state=state, seed=L), tied=state)


@pytest.mark.parametrize("tau", [0.25, 1.0, 3.7, 16.0, 1000.0])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gate_values(tau, dtype):
    """Logits from -60 to 60: gates that forget at once, and gates within 1e-20 of one."""
    x, z, M, h0, dh, dlast = inputs(2, 140, 64, dtype, state=True, seed=3)
    z = (torch.linspace(-60, 60, 140 * 64).view(140, 64)[torch.randperm(140, generator=torch.Generator().manual_seed(1))]
         .expand(2, 140, 64).to(dtype).contiguous())
    for tied in (False, True):
        check(x, z, M, h0, dh, dlast, tau=tau, tied=tied)


def test_infinite_logits():
    """-inf empties the state before its token, +inf keeps it whole."""
    x, z, M, h0, dh, dlast = inputs(2, 90, 32, F32, state=True, seed=4)
    z[:, 10] = float("-inf")
    z[:, 50] = float("-inf")
    z[:, 20:30] = float("inf")
    from scale_gated_linear_b200 import gated_scan
    for tied, tau in ((False, 16.0), (True, 16.0), (False, 1.0), (True, 1.0)):
        kw = dict(tied=tied, gate_normalizer=tau)
        h, _ = gated_scan(x.cuda(), z.cuda(), initial_state=h0.cuda(), **kw)
        parts = [gated_scan(x[:, a:b].cuda(), z[:, a:b].cuda(), **kw)[0] for a, b in ((10, 50), (50, 90))]
        want = oo.scan(host(x), host(z), tau, tied, None, host(h0))[0]
        near(h, want, 1e-5 * (1 + np.abs(want)), F32)
        for got, part in ((h[:, 10:50], parts[0]), (h[:, 50:], parts[1])):  # nothing of before is left
            near(got, host(part), 1e-5 * (1 + np.abs(host(part))), F32)


def test_gates_near_one_keep_their_digits():
    """Equal logits of 10: a = 1 - 2.837e-6 at every token. a rounded to f32 is 1 - 48 * 2^-24
    (2.861e-6), and the state after 6000 tokens would be off by 0.8 %. Allowed is what the
    roundings of the state itself can add up to: two a token, each at most U |h_t|, where h grows
    in a line to its last value, so 2 U * 6000 / 2 = 6000 U = 3.6e-4 of it, and 1e-5 for c."""
    from scale_gated_linear_b200 import gated_scan
    L, D = 6000, 64
    z = torch.full((1, L, D), 10.0, dtype=BF16)
    h, last = gated_scan(torch.ones(1, L, D, dtype=BF16).cuda(), z.cuda(), tied=True)
    c = -np.expm1(-oo.softplus_neg(10.0) / 16)
    assert np.allclose(host(last), -np.expm1(L * np.log1p(-c)), rtol=L * 2.0 ** -24 + 1e-5, atol=0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("view", ["fused", "odd_rows", "odd_start", "time_major", "every_other_row"])
def test_strides(view, dtype):
    B, L, D = 3, 77, 34

    def lay(t):
        if view == "fused":
            p = torch.full((B, L, 2 * D), 99.0, dtype=dtype)
            p[..., D:] = t
            return p.cuda()[..., D:]
        if view == "odd_rows":
            p = torch.full((B, L, D + 1), 99.0, dtype=dtype)
            p[..., :D] = t
            return p.cuda()[..., :D]
        if view == "odd_start":
            p = torch.full((B * L * D + 1,), 99.0, dtype=dtype)
            p[1:] = t.reshape(-1)
            return p.cuda()[1:].view(B, L, D)
        if view == "time_major":
            return t.transpose(0, 1).contiguous().cuda().transpose(0, 1)
        p = torch.full((B, 2 * L, D), 99.0, dtype=dtype)
        p[:, ::2] = t
        return p.cuda()[:, ::2]

    check(*inputs(B, L, D, dtype, state=True, mask="random", seed=5), view=lay, tied=True)


def test_expanded_inputs():
    """Rows and sequences with stride 0, and the gradient of what was expanded."""
    from scale_gated_linear_b200 import gated_scan
    g = torch.Generator().manual_seed(6)
    z1, x = torch.randn(1, 1, 32, generator=g), torch.randn(3, 70, 32, generator=g)
    zg, xg = z1.cuda().requires_grad_(), x.cuda().requires_grad_()
    h, last = gated_scan(xg, zg.expand(3, 70, 32))
    h.sum().backward()
    z = np.broadcast_to(host(z1), x.shape)
    ones = np.ones(x.shape)
    wx, wz, _, _ = oo.scan_backward(ones, None, host(x), z)
    e, ex, ez, _ = oo.scan_error(host(x), z, 16.0, False, None, None, ones)
    near(h, oo.scan(host(x), z)[0], e[:, 1:], F32)
    near(xg.grad, wx, ex, F32)
    n = 210 * 2.0 ** -24
    near(zg.grad, wz.sum((0, 1), keepdims=True), ez.sum((0, 1), keepdims=True) + n * np.abs(wz).sum((0, 1), keepdims=True), F32)


def test_autograd_matches_the_explicit_pair_and_differences():
    from scale_gated_linear_b200 import gated_scan, gated_scan_backward, gated_scan_forward
    x, z, M, h0, dh, dlast = (None if t is None else t.cuda() for t in inputs(2, 100, 24, F32, state=True, mask="left", seed=7))
    leaves = [t.clone().requires_grad_() for t in (x, z, h0)]
    h, last = gated_scan(leaves[0], leaves[1], initial_state=leaves[2], mask=M, tied=True)
    got = torch.autograd.grad((h, last), leaves, (dh, dlast))
    _, _, saved = gated_scan_forward(x, z, mask=M, initial_state=h0, tied=True)
    for a, b in zip(got, gated_scan_backward(dh, dlast, saved)):
        assert torch.equal(a, b)
    # a directional difference in 64 bits of the oracle, at the kernel's gradient
    g = np.random.default_rng(8)
    way = [g.normal(size=t.shape) for t in (x, z, h0)]
    args = [host(t) for t in (x, z, h0)]
    def loss(s):
        hh, ll, _ = oo.scan(args[0] + s * way[0], args[1] + s * way[1], 16.0, True, host(M), args[2] + s * way[2])
        return (hh * host(dh)).sum() + (ll * host(dlast)).sum()
    want = (loss(1e-5) - loss(-1e-5)) / 2e-5
    have = sum((host(a) * b).sum() for a, b in zip(got, way))
    assert abs(have - want) <= 1e-4 * sum(np.abs(host(a) * b).sum() for a, b in zip(got, way))


def test_one_output_alone_has_gradients():
    from scale_gated_linear_b200 import gated_scan
    x, z, _, h0, dh, dlast = (None if t is None else t.cuda() for t in inputs(2, 70, 16, F32, state=True, seed=9))
    xa, za, xb, zb = (t.clone().requires_grad_() for t in (x, z, x, z))
    (gated_scan(xa, za)[0] * dh).sum().backward()
    (gated_scan(xb, zb)[1] * dlast).sum().backward()
    wx, wz, _, _ = oo.scan_backward(host(dh), None, host(x), host(z))
    vx, vz, _, _ = oo.scan_backward(None, host(dlast), host(x), host(z))
    _, ex, ez, _ = oo.scan_error(host(x), host(z), 16.0, False, None, None, host(dh))
    _, fx, fz, _ = oo.scan_error(host(x), host(z), 16.0, False, None, None, None, host(dlast))
    for got, want, err in ((xa, wx, ex), (za, wz, ez), (xb, vx, fx), (zb, vz, fz)):
        near(got.grad, want, err, F32)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("B,D", [(1, 1), (1, 64), (3, 333), (257, 128), (5, 4096)])
def test_step(B, D, dtype):
    from scale_gated_linear_b200 import gated_scan_step
    x, z, _, h0, _, _ = inputs(B, 1, D, dtype, bias=1.0, state=True, seed=B)
    for tied in (False, True):
        for M in (None, torch.arange(B) % 3 != 1):
            gx, gz = x[:, 0].clone(), z[:, 0].clone()
            if M is not None:
                gx[~M], gz[~M] = float("nan"), float("nan")
            state = h0.cuda()
            h = gated_scan_step(gx.cuda(), gz.cuda(), state, mask=None if M is None else M.cuda(), tied=tied)
            m = None if M is None else M.numpy()[:, None]
            want, last, _ = oo.scan(host(x), host(z), 16.0, tied, m, host(h0))
            e = oo.scan_error(host(x), host(z), 16.0, tied, m, host(h0))
            near(h, want[:, 0], e[:, 1] * (1 if m is None else m), dtype)
            near(state, last, e[:, 1], F32)
            if M is not None:
                assert torch.equal(state.cpu()[~M], h0[~M])


def test_prefill_in_parts_and_steps_go_on():
    """A prompt in one call, in uneven parts, and token by token end in the same state."""
    from scale_gated_linear_b200 import gated_scan, gated_scan_step
    x, z, _, h0, _, _ = (None if t is None else t.cuda() for t in inputs(3, 300, 66, BF16, bias=2.0, state=True, seed=11))
    h, last = gated_scan(x, z, initial_state=h0, tied=True)
    state, outs = h0, []
    for a, b in ((0, 1), (1, 130), (130, 130), (130, 260)):
        o, state = gated_scan(x[:, a:b], z[:, a:b], initial_state=state, tied=True)
        outs.append(o)
    for t in range(260, 300):
        outs.append(gated_scan_step(x[:, t], z[:, t], state, tied=True)[:, None])
    e = oo.scan_error(host(x), host(z), 16.0, True, None, host(h0))
    want, wlast, _ = oo.scan(host(x), host(z), 16.0, True, None, host(h0))
    for got in (h, torch.cat(outs, 1)):
        near(got, want, 2 * e[:, 1:], BF16)
    near(last, wlast, e[:, -1], F32)
    near(state, wlast, 2 * e[:, -1], F32)


def test_gradients_of_nothing_are_zero():
    from scale_gated_linear_b200 import gated_scan_backward, gated_scan_forward
    x, z, _, h0, _, _ = (None if t is None else t.cuda() for t in inputs(2, 70, 40, BF16, state=True, seed=19))
    for g in gated_scan_backward(None, None, gated_scan_forward(x, z, initial_state=h0)[2]):
        assert not g.any()


@pytest.mark.parametrize("D,L", [(64, 5000), (1024, 2500), (4096, 600), (4160, 600)])
def test_forms_agree(D, L):
    """Rows split over clusters of several sizes, and one block a tile: parts of a sequence that
    take other forms give what the whole gives. A state forgets in about 16 / softplus(-2) = 126
    rows, each with two roundings of U, mostly of either sign: 1e-5 of the largest value (the
    worst sum of one sign would be 2 * 126 U = 1.5e-5)."""
    from scale_gated_linear_b200 import gated_scan, gated_scan_backward, gated_scan_forward
    x, z, _, _, dh, _ = (None if t is None else t.cuda() for t in inputs(1, L, D, F32, bias=2.0, seed=D))
    h, last, saved = gated_scan_forward(x, z, tied=True)
    dx, dz, _ = gated_scan_backward(dh, None, saved)
    cut = 200
    state, hs = gated_scan(x[:, :cut], z[:, :cut], tied=True)[1], []
    tail = gated_scan(x[:, cut:], z[:, cut:], initial_state=state, tied=True)
    for c in range(0, D, 64):  # tile by tile
        part = slice(c, min(c + 64, D))
        if c % 1024 == 0:
            a, _, s = gated_scan_forward(x[..., part], z[..., part], tied=True)
            b, g, _ = gated_scan_backward(dh[..., part], None, s)
            hs.append((h[..., part] - a).abs().max() <= 1e-5 * a.abs().max())
            hs.append((dx[..., part] - b).abs().max() <= 1e-5 * b.abs().max())
            hs.append((dz[..., part] - g).abs().max() <= 1e-5 * g.abs().max())
    assert all(hs)
    assert (tail[0] - h[:, cut:]).abs().max() <= 1e-5 * h.abs().max() and (tail[1] - last).abs().max() <= 1e-5 * last.abs().max()


def test_empty_calls():
    from scale_gated_linear_b200 import gated_scan, gated_scan_backward, gated_scan_forward, gated_scan_step
    e = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")
    h0 = torch.randn(2, 8, device="cuda")
    h, last = gated_scan(e(2, 0, 8), e(2, 0, 8), initial_state=h0)
    assert h.shape == (2, 0, 8) and torch.equal(last, h0)
    assert not gated_scan(e(2, 0, 8), e(2, 0, 8))[1].any()
    _, _, saved = gated_scan_forward(e(2, 0, 8), e(2, 0, 8), initial_state=h0)
    dx, dz, d0 = gated_scan_backward(None, h0, saved)
    assert dx.shape == dz.shape == (2, 0, 8) and torch.equal(d0, h0)
    h, last = gated_scan(e(0, 5, 8), e(0, 5, 8))
    assert h.shape == (0, 5, 8) and last.shape == (0, 8)
    assert gated_scan_step(e(0, 8), e(0, 8), torch.empty(0, 8, device="cuda")).shape == (0, 8)


def test_outputs_stay_inside_their_view():
    """h into the middle of a larger buffer: what lies around it stays as it was."""
    from scale_gated_linear_b200 import gated_scan, gated_scan_step
    x, z, _, h0, _, _ = inputs(2, 71, 37, BF16, state=True, seed=12)
    buf = torch.full((2, 80, 50), 7.0, dtype=BF16, device="cuda")
    out = buf[:, 5:76, 6:43]
    want, _ = gated_scan(x.cuda(), z.cuda())
    got, _ = gated_scan(x.cuda(), z.cuda(), out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, want)
    out.fill_(7.0)
    assert (buf == 7.0).all()
    buf = torch.full((2, 50), 7.0, dtype=BF16, device="cuda")
    gated_scan_step(x[:, 0].cuda(), z[:, 0].cuda(), h0.cuda(), out=buf[:, 6:43])
    buf[:, 6:43] = 7.0
    assert (buf == 7.0).all()


def test_same_inputs_give_the_same_bits():
    from scale_gated_linear_b200 import gated_scan_backward, gated_scan_forward
    x, z, M, h0, dh, dlast = (None if t is None else t.cuda() for t in inputs(4, 1100, 128, BF16, state=True, mask="random", seed=13))
    first = None
    for _ in range(3):
        h, last, saved = gated_scan_forward(x, z, mask=M, initial_state=h0)
        got = (h, last, *gated_scan_backward(dh, dlast, saved))
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, got))
        first = got


def test_streams():
    """Two calls at once on streams of their own, and a stream given by argument."""
    from scale_gated_linear_b200 import gated_scan
    x, z, _, _, _, _ = (None if t is None else t.cuda() for t in inputs(2, 3000, 256, BF16, seed=14))
    want, wlast = gated_scan(x, z)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                got.append(gated_scan(x, z))
        got.append(gated_scan(x, z, stream=s1))
    torch.cuda.synchronize()
    assert all(torch.equal(h, want) and torch.equal(last, wlast) for h, last in got)


def test_captured_and_replayed():
    from scale_gated_linear_b200 import gated_scan_backward, gated_scan_forward
    x, z, M, h0, dh, dlast = (None if t is None else t.cuda() for t in inputs(2, 700, 96, BF16, state=True, mask="left", seed=15))
    gated_scan_forward(x, z)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, last, saved = gated_scan_forward(x, z, mask=M, initial_state=h0)
        grads = gated_scan_backward(dh, dlast, saved)
    for seed in (16, 17):
        nx, nz, nM, nh0, ndh, ndl = inputs(2, 700, 96, BF16, state=True, mask="left", seed=seed)
        for a, b in zip((x, z, M, h0, dh, dlast), (nx, nz, nM, nh0, ndh, ndl)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        eh, elast, esaved = gated_scan_forward(x, z, mask=M, initial_state=h0)
        for a, b in zip((h, last, *grads), (eh, elast, *gated_scan_backward(dh, dlast, esaved))):
            assert torch.equal(a, b)


def test_capture_with_autograd():
    """A captured forward and backward works on leaves of its own, and is refused while an
    eager graph of the same leaf lives."""
    from scale_gated_linear_b200 import MSGLAError, gated_scan
    x, z, _, _, dh, _ = (None if t is None else t.cuda() for t in inputs(1, 130, 32, F32, seed=18))
    x, z = x.requires_grad_(), z.requires_grad_()
    eager = torch.autograd.grad(gated_scan(x, z)[0], (x, z), dh)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(gated_scan(x, z)[0], (x, z), dh)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, got))
    living = gated_scan(x, z)
    torch.cuda.synchronize()
    with pytest.raises(MSGLAError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            gated_scan(x, z)
    del living
    torch.cuda.synchronize()


def test_refusals():
    from scale_gated_linear_b200 import MSGLAError, gated_scan, gated_scan_backward, gated_scan_forward, gated_scan_step
    x = torch.zeros(2, 9, 16, dtype=BF16, device="cuda")
    s = torch.zeros(2, 16, device="cuda")
    bad = [
        lambda: gated_scan(x.cpu(), x.cpu()), lambda: gated_scan(x.double(), x.double()),
        lambda: gated_scan(x[0], x[0]), lambda: gated_scan(x, x.float()), lambda: gated_scan(x, x[:, :8]),
        lambda: gated_scan(x, x.transpose(1, 2).contiguous().transpose(1, 2)),
        lambda: gated_scan(x, x, mask=torch.ones(2, 8, dtype=torch.uint8, device="cuda")),
        lambda: gated_scan(x, x, mask=torch.ones(2, 9, device="cuda")),
        lambda: gated_scan(x, x, mask=torch.ones(2, 9, dtype=torch.uint8)),
        lambda: gated_scan(x, x, initial_state=s.bfloat16()), lambda: gated_scan(x, x, initial_state=s[:1]),
        lambda: gated_scan(x, x, gate_normalizer=0.0), lambda: gated_scan(x, x, gate_normalizer=float("nan")),
        lambda: gated_scan(x, x, gate_normalizer=float("inf")), lambda: gated_scan(x, x, out=x),
        lambda: gated_scan(x, x.clone(), out=torch.zeros(1, 9, 16, dtype=BF16, device="cuda").expand(2, 9, 16)),
        lambda: gated_scan(x[..., :0], x[..., :0]),
        lambda: gated_scan(x.float().requires_grad_(), x.float(), out=x.float()),
        lambda: gated_scan(x.float().requires_grad_(), x.float(), stream=torch.cuda.Stream()),
        lambda: gated_scan_backward(x.float(), None, gated_scan_forward(x, x)[2]),
        lambda: gated_scan_backward(x, s[:1], gated_scan_forward(x, x)[2]),
        lambda: gated_scan_step(x[:, 0], x[:, 0], s.bfloat16()), lambda: gated_scan_step(x[:, 0], x[:, 0], s.t().contiguous().t()),
        lambda: gated_scan_step(x[:, 0], x[:, 0], s.clone().requires_grad_()), lambda: gated_scan_step(x, x, s),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(MSGLAError):
            f()
            pytest.fail(f"call {k} was taken")
