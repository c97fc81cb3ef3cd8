"""Calls of the operators next to the layer that are easily left out: another device's sizes, errors of
an earlier call, forward-mode derivatives, captured steps, version counters, arguments of other types."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]
pytestmark = gpu

from scale_gated_linear_b200 import (MSGLAError, _lib, gated_scan, gated_scan_backward, gated_scan_forward,  # noqa: E402
                                     gated_scan_step, group_norm, group_norm_backward, group_norm_forward)

BF16, F32 = torch.bfloat16, torch.float32


def randn(*shape, dtype=F32, seed=0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def test_workspace_sizes_are_of_the_named_device():
    """A size for a device that does not exist is refused: it would be that of the current one."""
    lib, n = _lib.load(), ctypes.c_size_t()
    for gradients in (0, 1):
        for S in (1, 4, 5000):
            good = _lib.NormConfig(0, 0, 64, 4, 0, 1, 1e-5)
            assert lib.msgla_group_norm_workspace_size(good, 8, S, gradients, ctypes.byref(n)) == 0
            bad = _lib.NormConfig(torch.cuda.device_count(), 0, 64, 4, 0, 1, 1e-5)
            assert lib.msgla_group_norm_workspace_size(bad, 8, S, gradients, ctypes.byref(n)) < 0


def test_a_failed_call_leaves_no_error_behind():
    """A call for a device that does not exist fails; the good calls after it do not report its error."""
    lib = _lib.load()
    x, z, s = randn(2, 64), randn(2, 64, seed=1), randn(2, 64, seed=2)
    good = [lambda: gated_scan_step(x, z, s), lambda: group_norm(x, 4), lambda: group_norm(x[None], 4),
            lambda: group_norm_backward(x, group_norm_forward(x, 4)[1]),
            lambda: group_norm_backward(x[None], group_norm_forward(x[None], 4)[1]), lambda: gated_scan(x[None], z[None])]
    for f in good:
        f()
    rows = lambda t: _lib.Rows(t.data_ptr(), 64, 0)
    for f in good:
        bad = _lib.ScanConfig(torch.cuda.device_count(), 2, 64, 0, 16.0)
        out = torch.empty_like(x)
        assert lib.msgla_scan_step(bad, 2, rows(x), rows(z), None, s.data_ptr(), rows(out), None) < 0
        f()
    torch.cuda.synchronize()


def test_forward_mode_is_refused():
    """A dual tensor's tangent would be dropped, and a derivative of zero reported."""
    import torch.autograd.forward_ad as fwd
    x, z, s, w = randn(2, 5, 16), randn(2, 5, 16, seed=1), randn(2, 16), torch.ones(16, device="cuda")
    with fwd.dual_level():
        dual = lambda t: fwd.make_dual(t, torch.ones_like(t))
        calls = [lambda: gated_scan(dual(x), z), lambda: gated_scan(x, dual(z)), lambda: gated_scan(x, z, initial_state=dual(s)),
                 lambda: gated_scan_step(dual(x[:, 0]), z[:, 0], s), lambda: gated_scan_step(x[:, 0], dual(z[:, 0]), s),
                 lambda: gated_scan_step(x[:, 0], z[:, 0], dual(s)), lambda: group_norm(dual(x), 4),
                 lambda: group_norm(x, 4, dual(w)), lambda: group_norm(x, 4, w, dual(w)), lambda: group_norm(x, 4, gate=dual(x))]
        for k, f in enumerate(calls):
            for grad in (True, False):
                with torch.set_grad_enabled(grad), pytest.raises(MSGLAError):
                    f()
                    pytest.fail(f"call {k} was taken")
        gated_scan(x, z, initial_state=s)  # without tangents inside a dual level
        group_norm(x, 4, w, gate=x)
        gated_scan_step(x[:, 0], z[:, 0], s.clone())


def test_numbers_given_as_tensors_are_read_anew():
    """gate_normalizer, tied, eps and center as tensors that change between calls."""
    x, z = randn(2, 40, 16), randn(2, 40, 16, seed=1)
    tau, tied = torch.tensor(16.0), torch.tensor(False)
    first = gated_scan(x, z, gate_normalizer=tau, tied=tied)[0]
    assert torch.equal(first, gated_scan(x, z)[0])
    tau.fill_(2.0)
    tied.fill_(True)
    assert torch.equal(gated_scan(x, z, gate_normalizer=tau, tied=tied)[0], gated_scan(x, z, gate_normalizer=2.0, tied=True)[0])
    s, t = randn(2, 16), randn(2, 16)
    gated_scan_step(x[:, 0], z[:, 0], s, gate_normalizer=tau)
    gated_scan_step(x[:, 0], z[:, 0], t, gate_normalizer=2.0)
    assert torch.equal(s, t)
    eps, center = torch.tensor(0.5), torch.tensor(True)
    group_norm(x, 2, eps=eps, center=center)
    eps.fill_(2.0)
    center.fill_(False)
    assert torch.equal(group_norm(x, 2, eps=eps, center=center), group_norm(x, 2, eps=2.0, center=False))


def test_numbers_that_are_none():
    x = randn(2, 5, 16)
    for f in (lambda: gated_scan(x, x, gate_normalizer="16s"), lambda: gated_scan(x, x, gate_normalizer=None),
              lambda: gated_scan(x, x, gate_normalizer=[16.0]), lambda: gated_scan_step(x[:, 0], x[:, 0], x[:, 1].clone(), gate_normalizer=None),
              lambda: group_norm(x, 4, eps=None), lambda: group_norm(x, 4, eps="x"), lambda: group_norm(x, 4, activation=["silu"]),
              lambda: group_norm(x, 4.0), lambda: group_norm(x, None)):
        with pytest.raises(MSGLAError):
            f()


def test_updates_in_place_are_seen_by_autograd():
    """A state (or an output buffer) that a living graph has saved: its backward reports the change,
    as after torch's own in-place operations, in place of a wrong gradient."""
    x, z, state = randn(2, 16), randn(2, 16, seed=1), randn(2, 16, seed=2)
    w = torch.ones(16, device="cuda", requires_grad=True)
    seq = randn(2, 3, 16)

    def changed(t, call):
        y = (t * w).sum()
        with torch.no_grad():
            call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()

    changed(state, lambda: gated_scan_step(x, z, state))
    h = torch.zeros_like(x)
    changed(h, lambda: gated_scan_step(x, z, state, out=h))
    hs = torch.zeros_like(seq)
    changed(hs, lambda: gated_scan(seq, seq, out=hs))
    changed(hs, lambda: group_norm(seq, 4, out=hs))
    changed(hs, lambda: gated_scan_forward(seq, seq, out=hs))
    changed(hs, lambda: group_norm_forward(seq, 4, out=hs))
    with torch.inference_mode():  # tensors without a version counter
        s = state.clone()
        gated_scan_step(x, z, s, out=torch.empty_like(x))
    gated_scan_step(x, z, s)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_captured_steps(dtype):
    """Tokens through the step and a head norm in one replayed graph: what the eager calls give."""
    B, D, heads = 5, 96, 4
    xs, zs, gs = (randn(6, B, D, dtype=dtype, seed=k) for k in range(3))
    w = randn(D)
    x, z, g, mask = xs[0].clone(), zs[0].clone(), gs[0].clone(), torch.ones(B, dtype=torch.uint8, device="cuda")
    state = randn(B, D, seed=9)

    def token(x, z, g, state, mask):
        return group_norm(gated_scan_step(x, z, state, mask=mask, tied=True), heads, w, gate=g, activation="silu")

    with torch.no_grad():
        token(x, z, g, state.clone(), mask)
        torch.cuda.synchronize()
        kept = state.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = token(x, z, g, state, mask)
        want = kept.clone()
        for k in range(6):
            for a, b in ((x, xs[k]), (z, zs[k]), (g, gs[k])):
                a.copy_(b)
            mask.copy_((torch.arange(B) % 3 != k % 3).to(torch.uint8))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, token(xs[k], zs[k], gs[k], want, mask)) and torch.equal(state, want)


def test_saved_states_have_the_librarys_size():
    lib, n = _lib.load(), ctypes.c_size_t()
    for code, dtype in ((0, BF16), (1, torch.float16), (2, F32)):
        for L in (1, 7, 8, 9, 16, 17, 100):
            x = randn(2, L, 24, dtype=dtype)
            states = gated_scan_forward(x, x)[2].states
            assert lib.msgla_scan_saved_size(_lib.ScanConfig(0, code, 24, 0, 16.0), 2, L, ctypes.byref(n)) == 0
            assert states.numel() * 4 == n.value


def test_a_captured_call_refuses_a_leaf_whose_node_is_held():
    """A wrapper that keeps a leaf's gradient node: torch does not tell the node's stream. The explicit
    pair is what such a program captures."""
    w, x = torch.ones(16, device="cuda", requires_grad=True), randn(4, 16)
    held = torch.autograd.graph.get_gradient_edge(w).node
    group_norm(x, 4, w)
    torch.cuda.synchronize()
    with pytest.raises(MSGLAError, match="explicit"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            group_norm(x, 4, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, saved = group_norm_forward(x, 4, w.detach())
        grads = group_norm_backward(x, saved)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, group_norm(x, 4, w.detach())) and grads[1].shape == w.shape
    del held


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 37), (F32, 64), (F32, 33)])
@pytest.mark.parametrize("order", ["batch", "time"])
def test_outputs_beside_other_rows(dtype, D, order):
    """Rows of one tensor: h beside x and the gate, dx and dz as halves of the joint gradient, y beside its gate."""
    B, L = 3, 70
    joint = lambda n: (torch.zeros(B, L, n * D, dtype=dtype, device="cuda") if order == "batch" else
                       torch.zeros(L, B, n * D, dtype=dtype, device="cuda").transpose(0, 1))
    x, z, dh = (randn(B, L, D, dtype=dtype, seed=k) for k in range(3))
    p = joint(3)
    p[..., :D], p[..., D:2 * D] = x, z
    want, last, saved = gated_scan_forward(x, z)
    gated_scan(p[..., :D], p[..., D:2 * D], out=p[..., 2 * D:])
    assert torch.equal(p[..., 2 * D:], want) and torch.equal(p[..., :D], x) and torch.equal(p[..., D:2 * D], z)
    group_norm(p[..., :D], 1, gate=p[..., D:2 * D], out=p[..., 2 * D:])
    assert torch.equal(p[..., 2 * D:], group_norm(x, 1, gate=z)) and torch.equal(p[..., D:2 * D], z)
    state = last.clone()
    gated_scan_step(p[:, 5, :D], p[:, 5, D:2 * D], state, out=p[:, 5, 2 * D:])
    assert torch.equal(p[:, 5, 2 * D:], gated_scan_step(x[:, 5], z[:, 5], last.clone()))
    g = joint(2)
    rows = lambda t: _lib.Rows(t.data_ptr(), t.stride(0), t.stride(1))
    cfg = _lib.ScanConfig(0, {BF16: 0, F32: 2}[dtype], D, 0, 16.0)
    _lib.check(_lib.load().msgla_scan_backward(cfg, B, L, rows(x), rows(z), None, saved.states.data_ptr(), rows(dh), None,
                                               rows(g[..., :D]), rows(g[..., D:]), None,
                                               ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)))
    dx, dz, _ = gated_scan_backward(dh, None, saved)
    assert torch.equal(g[..., :D], dx) and torch.equal(g[..., D:], dz)
    with pytest.raises(MSGLAError):  # shifted by less than a row's width
        gated_scan(p[..., :D], p[..., D:2 * D], out=p[..., D + 1:2 * D + 1])
