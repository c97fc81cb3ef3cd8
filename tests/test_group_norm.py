"""GPU parity of group normalisation (activation, output gate, gradients) against the fp64
oracle, and of the recurrence and the normalisation run together. A result may be off by
half a step of its type plus the bound that oracle.ops_oracle.norm_error derives."""
import numpy as np
import pytest

from oracle import ops_oracle as oo

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def near(got, ref, err, dtype):
    got, half = host(got), 0.0 if dtype == F32 else torch.finfo(dtype).eps / 2
    tol = half * np.abs(ref) + err * (1 + half) + 2.0 ** -25 * (dtype == F16) + 1e-37
    assert np.isfinite(got).all()
    worst = (np.abs(got - ref) - tol).max() if got.size else 0.0
    assert worst <= 0, f"off by {np.abs(got - ref).max():.3e}, {worst:.3e} more than allowed"


def make_mask(kind, N, S, g):
    if kind is None:
        return None
    if kind == "empty":
        M = torch.ones(N, S, dtype=torch.uint8)
        M[0] = 0
        M[-1, 1:] = 0
        return M
    return (torch.rand(N, S, generator=g) < 0.7).to(torch.uint8)


def check(N, S, C, G, dtype=BF16, act="none", gated=False, mask=None, center=True, affine=True, eps=1e-5, seed=0,
          view=lambda t: t.cuda(), mean=0.5, std=2.0):
    """[N, S, C] ([N, C] when S is None), forward and backward, against the oracle."""
    from scale_gated_linear_b200 import group_norm, group_norm_backward, group_norm_forward
    g = torch.Generator().manual_seed(seed)
    shape = (N, C) if S is None else (N, S, C)
    r = lambda *s: torch.randn(*s, generator=g)
    x, dy = (r(*shape) * std + mean).to(dtype), r(*shape).to(dtype)
    gate = r(*shape).to(dtype) if gated else None
    w, b = (1 + 0.3 * r(C), 0.3 * r(C)) if affine else (None, None)
    M = make_mask(mask, N, S or 1, g)
    cu = lambda t: None if t is None else t.cuda()

    def lay(t):
        if t is None:
            return None
        if M is not None:
            t = torch.where(M.view(shape[:-1]).bool()[..., None], t, torch.full_like(t, float("nan")))
        return view(t)

    kw = dict(gate=lay(gate), mask=None if M is None else M.view(shape[:-1]).cuda(), activation=act, eps=eps, center=center)
    gx, gw, gb = lay(x), cu(w), cu(b)
    y, saved = group_norm_forward(gx, G, gw, gb, **kw)
    dx, dw, db, dg = group_norm_backward(lay(dy), saved)
    assert torch.equal(y, group_norm(gx, G, gw, gb, **kw))
    full = (N, S or 1, C)
    h = lambda t: None if t is None else host(t).reshape(full)
    args = dict(gate=h(gate), mask=None if M is None else M.numpy(), act=act, eps=eps, center=center, dy=h(dy))
    wy, (wx, ww, wb, wg) = oo.group_norm(h(x), G, host(w), host(b), **args)
    ey, (ex, ew, eb, eg) = oo.norm_error(h(x), G, host(w), host(b), **args)
    near(y.reshape(full), wy, ey, dtype)
    near(dx.reshape(full), wx, ex, dtype)
    if gated:
        near(dg.reshape(full), wg, eg, dtype)
    assert (dw is None) == (db is None) == (not affine)
    if affine:
        near(dw, ww, ew, F32)
        near(db, wb, eb, F32)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("N,C,G", [(1, 8, 1), (5, 64, 4), (37, 130, 13), (3, 2048, 4), (300, 96, 3), (2, 1000, 1), (9, 33, 1),
                                   (4, 4096, 2), (2, 6000, 1), (7, 512, 32), (2, 24, 24), (700, 520, 2), (3, 8192, 1), (2, 9000, 1), (5, 5001, 3), (2, 5001, 1)])
def test_rows(N, C, G, dtype, center):
    """Every row by itself: narrow and wide groups, odd widths, groups of one channel."""
    check(N, None, C, G, dtype, act="silu", gated=True, center=center, seed=C)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,S,C,G", [(1, 2, 32, 4), (2, 3, 7, 7), (3, 100, 64, 2), (1, 1000, 40, 5), (2, 65, 130, 13),
                                     (1, 257, 512, 16), (4, 33, 1024, 1), (2, 700, 8, 1), (1, 5, 4100, 4), (9, 16, 96, 3)])
def test_sequences(N, S, C, G, dtype):
    check(N, S, C, G, dtype, act="silu", seed=S + C, eps=1e-3)


@pytest.mark.parametrize("act", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("S", [None, 50])
def test_activations(act, gated, S):
    check(6, S, 96, 4, BF16, act=act, gated=gated)
    check(6, S, 90, 2, F32, act=act, gated=gated, center=False, affine=False)


@pytest.mark.parametrize("mask", ["random", "empty"])
@pytest.mark.parametrize("N,S,C,G,dtype", [(11, None, 96, 3, BF16), (4, 60, 64, 4, F16), (3, 301, 36, 3, F32), (3, 40, 520, 1, BF16)])
def test_padding(N, S, C, G, dtype, mask):
    """NaN in every padded row of x, gate and dy: none of it may be read."""
    for gated in (False, True):
        check(N, S, C, G, dtype, act="sigmoid", gated=gated, mask=mask, seed=3, eps=1e-3)


@pytest.mark.parametrize("S", [None, 64])
def test_far_mean(S):
    """A mean of 300 standard deviations: squares summed without taking it off would lose the variance."""
    check(4, S, 256, 4, F32, mean=300.0, std=1.0, seed=4)


@pytest.mark.parametrize("S", [None, 30])
def test_constant_rows(S):
    """No variance at all: xhat = 0 and y = bias (multiples of 2.5 add up and divide exactly)."""
    from scale_gated_linear_b200 import group_norm
    shape = (3, 32) if S is None else (3, S, 32)
    b = torch.randn(32, device="cuda")
    y = group_norm(torch.full(shape, 2.5, device="cuda"), 4, None, b)
    assert torch.equal(y, b.expand(shape))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("view", ["fused", "odd_rows", "odd_start", "time_major"])
@pytest.mark.parametrize("S", [None, 21])
def test_strides(view, S, dtype):
    C = 48

    def lay(t):
        if view == "fused":
            p = torch.full((*t.shape[:-1], 2 * C), 99.0, dtype=dtype)
            p[..., C:] = t
            return p.cuda()[..., C:]
        if view == "odd_rows":
            p = torch.full((*t.shape[:-1], C + 1), 99.0, dtype=dtype)
            p[..., :C] = t
            return p.cuda()[..., :C]
        if view == "odd_start":
            p = torch.full((t.numel() + 1,), 99.0, dtype=dtype)
            p[1:] = t.reshape(-1)
            return p.cuda()[1:].view(t.shape)
        return t.transpose(0, 1).contiguous().cuda().transpose(0, 1) if S else t.cuda()[:, :]

    check(5, S, C, 3, dtype, act="silu", gated=True, mask="random", view=lay, seed=5, eps=1e-3)


def test_autograd_matches_the_explicit_pair():
    from scale_gated_linear_b200 import group_norm, group_norm_backward, group_norm_forward
    g = torch.Generator().manual_seed(6)
    x, gate, dy = (torch.randn(3, 20, 64, generator=g).cuda() for _ in range(3))
    w, b = torch.randn(64, generator=g).cuda(), torch.randn(64, generator=g).cuda()
    leaves = [t.clone().requires_grad_() for t in (x, w, b, gate)]
    y = group_norm(leaves[0], 4, leaves[1], leaves[2], gate=leaves[3], activation="silu")
    got = torch.autograd.grad(y, leaves, dy)
    y2, saved = group_norm_forward(x, 4, w, b, gate=gate, activation="silu")
    assert torch.equal(y, y2)
    for a, c in zip(got, group_norm_backward(dy, saved)):
        assert torch.equal(a, c)
    # weight alone, and an expanded output gradient
    wl = w.clone().requires_grad_()
    group_norm(x, 4, wl).sum().backward()
    _, (_, ww, _, _) = oo.group_norm(host(x), 4, host(w), dy=np.ones(x.shape))
    _, (_, ew, _, _) = oo.norm_error(host(x), 4, host(w), dy=np.ones(x.shape))
    near(wl.grad, ww, ew, F32)


def test_empty_calls():
    from scale_gated_linear_b200 import group_norm, group_norm_backward, group_norm_forward
    w = torch.ones(8, device="cuda")
    for shape in ((0, 8), (0, 4, 8), (3, 0, 8)):
        x = torch.empty(shape, dtype=BF16, device="cuda")
        assert group_norm(x, 2, w, w).shape == shape
        y, saved = group_norm_forward(x, 2, w, w)
        dx, dw, db, dg = group_norm_backward(y, saved)
        assert dx.shape == shape and not dw.any() and not db.any() and dg is None


def test_outputs_stay_inside_their_view():
    from scale_gated_linear_b200 import group_norm
    for S in (None, 19):
        shape = (6, 37) if S is None else (6, S, 37)
        x = torch.randn(shape, device="cuda").to(BF16)
        buf = torch.full((*shape[:-1], 50), 7.0, dtype=BF16, device="cuda")
        out = buf[..., 6:43]
        assert torch.equal(group_norm(x, 1, out=out), group_norm(x, 1))
        out.fill_(7.0)
        assert (buf == 7.0).all()


def test_same_inputs_give_the_same_bits_on_streams_and_in_graphs():
    from scale_gated_linear_b200 import group_norm_backward, group_norm_forward
    g = torch.Generator().manual_seed(7)
    for shape, G in (((3000, 256), 4), ((2, 1500, 96), 6)):
        x, dy = torch.randn(shape, generator=g).cuda().to(BF16), torch.randn(shape, generator=g).cuda().to(BF16)
        w, b = torch.randn(shape[-1], generator=g).cuda(), torch.randn(shape[-1], generator=g).cuda()

        def both(stream=None):
            y, saved = group_norm_forward(x, G, w, b, activation="silu", stream=stream)
            return (y, *group_norm_backward(dy, saved, stream=stream)[:3])

        want = both()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = [both(s) for _ in range(3) for s in streams]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(both())
        with torch.cuda.graph(graph2 := torch.cuda.CUDAGraph()):  # two graphs, replayed at once
            got.append(both())
        for _ in range(3):
            with torch.cuda.stream(streams[0]):
                graph.replay()
            with torch.cuda.stream(streams[1]):
                graph2.replay()
        torch.cuda.synchronize()
        for t in got:
            assert all(torch.equal(a, c) for a, c in zip(t, want))


def test_refusals():
    from scale_gated_linear_b200 import MSGLAError, group_norm, group_norm_backward, group_norm_forward
    x = torch.zeros(4, 9, 16, dtype=BF16, device="cuda")
    w = torch.zeros(16, device="cuda")
    bad = [
        lambda: group_norm(x.cpu(), 4), lambda: group_norm(x.double(), 4), lambda: group_norm(x, 3), lambda: group_norm(x, 0),
        lambda: group_norm(x, -4), lambda: group_norm(x[None], 4), lambda: group_norm(x[0, 0], 4),
        lambda: group_norm(x, 4, w.bfloat16()), lambda: group_norm(x, 4, w[:8]), lambda: group_norm(x, 4, None, w.cpu()),
        lambda: group_norm(x, 4, activation="tanh"), lambda: group_norm(x, 4, eps=0.0), lambda: group_norm(x, 4, eps=float("inf")),
        lambda: group_norm(x, 4, gate=x[:, :3]), lambda: group_norm(x, 4, gate=x.float()), lambda: group_norm(x, 4, out=x),
        lambda: group_norm(x, 4, mask=torch.ones(4, 8, dtype=torch.bool, device="cuda")),
        lambda: group_norm(x, 4, mask=torch.ones(4, 9, dtype=torch.int32, device="cuda")),
        lambda: group_norm(x.transpose(1, 2).contiguous().transpose(1, 2), 4),
        lambda: group_norm_backward(x.float(), group_norm_forward(x, 4)[1]),
        lambda: group_norm_backward(x[:2], group_norm_forward(x, 4)[1]),
        lambda: group_norm(x.float().requires_grad_(), 4, out=x.float()),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(MSGLAError):
            f()
            pytest.fail(f"call {k} was taken")


def mixer(x, p, heads, mask=None, state=None, norm=True):
    """One mixer: a fused projection, the recurrence, the heads' normalisation under a gate."""
    from scale_gated_linear_b200 import gated_scan, group_norm
    B, L, d = x.shape
    u, z, g = (x @ p["W"].t()).chunk(3, -1)
    h, last = gated_scan(u, z, mask=mask, initial_state=state, tied=True)
    D = u.shape[-1]
    y = group_norm(h.reshape(B * L, D), heads, p["w"], p["b"], gate=g.reshape(B * L, D), activation="silu")
    return y.view(B, L, D), last


def test_together_training_gradients():
    """Projection, recurrence and gated head norm on a padded batch: gradients of every
    weight against a directional difference in 64 bits."""
    rng = np.random.default_rng(20)
    B, L, d, D, heads = 3, 90, 24, 48, 4
    P = {"W": rng.normal(size=(3 * D, d)) / np.sqrt(d), "w": 1 + 0.1 * rng.normal(size=D), "b": 0.1 * rng.normal(size=D)}
    X, dY = rng.normal(size=(B, L, d)), rng.normal(size=(B, L, D))
    M = np.ones((B, L), np.uint8)
    M[0, :40] = 0
    M[1] = 0
    P = {k: v.astype(np.float32).astype(np.float64) for k, v in P.items()}
    X = X.astype(np.float32).astype(np.float64)
    p = {k: torch.tensor(v, dtype=F32, device="cuda", requires_grad=True) for k, v in P.items()}
    x = torch.tensor(X, dtype=F32, device="cuda", requires_grad=True)
    y, _ = mixer(x, p, heads, torch.tensor(M, device="cuda"))
    dy = torch.tensor(dY, dtype=F32, device="cuda")
    got = torch.autograd.grad(y, [x, p["W"], p["w"], p["b"]], dy)

    def loss(Xs, Ws, ws, bs):
        u, z, g = np.split(Xs @ Ws.T, 3, -1)
        h, _, _ = oo.scan(u, z, 16.0, True, M)
        yy = oo.group_norm(h.reshape(B * L, 1, D), heads, ws, bs, gate=g.reshape(B * L, 1, D), act="silu")
        return (yy.reshape(B, L, D) * host(dy)).sum()

    args = [X, P["W"], P["w"], P["b"]]
    for k in range(4):
        way = rng.normal(size=args[k].shape)
        step = 1e-6
        hi, lo = ([a + (step * s) * way if i == k else a for i, a in enumerate(args)] for s in (1, -1))
        want = (loss(*hi) - loss(*lo)) / (2 * step)
        have, size = (host(got[k]) * way).sum(), np.abs(host(got[k]) * way).sum()
        assert abs(have - want) <= 1e-4 * size


def test_together_serving():
    """Prompt, then tokens one by one through the step and the head norm: the outputs of the
    whole sequence in one call, within twice a step of bf16 (both sides round h and y)."""
    from scale_gated_linear_b200 import gated_scan_step, group_norm
    g = torch.Generator().manual_seed(21)
    B, L, d, D, heads = 2, 60, 32, 64, 4
    p = {"W": (torch.randn(3 * D, d, generator=g) / d ** 0.5).cuda().to(BF16), "w": torch.ones(D).cuda(), "b": torch.zeros(D).cuda()}
    x = torch.randn(B, L, d, generator=g).cuda().to(BF16)
    with torch.no_grad():
        proj = x @ p["W"].t()
        u, z, gate = proj.chunk(3, -1)
        from scale_gated_linear_b200 import gated_scan
        h, _ = gated_scan(u, z, tied=True)
        whole = group_norm(h.reshape(-1, D), heads, p["w"], p["b"], gate=gate.reshape(-1, D), activation="silu").view(B, L, D)
        _, state = gated_scan(u[:, :40], z[:, :40], tied=True)
        for t in range(40, L):
            ht = gated_scan_step(u[:, t], z[:, t], state, tied=True)
            y = group_norm(ht, heads, p["w"], p["b"], gate=gate[:, t], activation="silu")
            ref = host(whole[:, t])
            assert (np.abs(host(y) - ref) <= 2 * 2.0 ** -7 * (np.abs(ref) + np.abs(ref).max() * 2.0 ** -3)).all()
