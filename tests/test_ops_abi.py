"""Refusals of the C entry points of the recurrence and of group normalisation, made before
the device is touched: no GPU needed (the pointers are never read)."""
import ctypes

import pytest

from scale_gated_linear_b200 import _lib

P = 1 << 30  # a plausible, aligned device address


def rows(at, sb=64, sl=8):
    return _lib.Rows(at, sb, sl)


def scan_cfg(**kw):
    c = _lib.ScanConfig(0, 0, 8, 0, 16.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def norm_cfg(**kw):
    c = _lib.NormConfig(0, 0, 8, 2, 0, 1, 1e-5)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


SCAN_BAD = [dict(dtype=3), dict(dtype=-1), dict(D=0), dict(D=(1 << 24) + 1), dict(tied=2), dict(gate_normalizer=0.0),
            dict(gate_normalizer=-1.0), dict(gate_normalizer=float("nan")), dict(gate_normalizer=float("inf")),
            dict(gate_normalizer=1e-40)]


@pytest.mark.parametrize("kw", SCAN_BAD)
def test_scan_rejects_bad_config(kw):
    lib, n = _lib.load(), ctypes.c_size_t()
    assert lib.msgla_scan_saved_size(scan_cfg(**kw), 1, 1, ctypes.byref(n)) == -1
    assert lib.msgla_scan_forward(scan_cfg(**kw), 0, 0, None, None, None, None, None, None, None, None) == -1
    assert lib.msgla_scan_step(scan_cfg(**kw), 0, None, None, None, None, None, None) == -1
    assert lib.msgla_last_error().decode()


def test_scan_sizes():
    lib, n = _lib.load(), ctypes.c_size_t()
    for dtype, rows in ((0, 16), (1, 16), (2, 8)):
        for L, want in ((0, 0), (1, 1), (rows, 1), (rows + 1, 2), (1 << 20, (1 << 20) // rows)):
            assert lib.msgla_scan_saved_size(scan_cfg(dtype=dtype), 3, L, ctypes.byref(n)) == 0 and n.value == 3 * want * 8 * 4
    for B, L in ((-1, 1), (65536, 1), (1, -1), (1, (1 << 30) + 1)):
        assert lib.msgla_scan_saved_size(scan_cfg(), B, L, ctypes.byref(n)) == -1
    assert lib.msgla_scan_saved_size(scan_cfg(), 1, 1, None) == -1
    assert lib.msgla_scan_saved_size(None, 1, 1, ctypes.byref(n)) == -1


def scan_call(B=2, L=8, x=None, z=None, M=None, h0=None, h=None, last=P + (4 << 20), saved=None, cfg=None):
    return _lib.load().msgla_scan_forward(cfg or scan_cfg(), B, L, x or rows(P), z or rows(P + (1 << 20)), M, h0,
                                          h or rows(P + (2 << 20)), last, saved, None)


@pytest.mark.parametrize("kw", [
    dict(x=rows(0)), dict(z=rows(0)), dict(h=rows(0)), dict(last=None), dict(x=rows(P + 1)), dict(last=P + (4 << 20) + 2),
    dict(x=rows(P, -64)), dict(x=rows(P, 64, -8)), dict(x=rows(P, 1 << 46)), dict(z=rows(P + 4096, 1 << 45, 1 << 45), B=60000),
    dict(h=rows(P + (2 << 20), 64, 0)), dict(h=rows(P + (2 << 20), 64, 7)), dict(h=rows(P + (2 << 20), 0, 8)),
    dict(h=rows(P + (2 << 20), 63, 8)), dict(h=rows(P)), dict(h=rows(P + 254)), dict(h=rows(P + (1 << 20))),
    dict(last=P), dict(h0=P + (4 << 20) + 4), dict(saved=P), dict(saved=P + (4 << 20)), dict(M=P + (2 << 20) + 3),
    dict(saved=P + (3 << 20) + 2),
])
def test_scan_rejects_bad_buffers(kw):
    assert scan_call(**kw) == -1
    assert _lib.load().msgla_last_error().decode()


def test_scan_backward_and_step_reject():
    lib, c = _lib.load(), scan_cfg()
    x, z, d, dx, dz = (rows(P + (k << 20)) for k in range(5))
    last = P + (8 << 20)
    ok = [c, 2, 8, x, z, None, P + (6 << 20), d, None, dx, dz, last, None]
    for at, bad in ((3, rows(0)), (4, None), (6, None), (9, None), (10, rows(0)), (10, dx), (9, x), (9, d), (11, P + (6 << 20)),
                    (11, P + (3 << 20)), (11, last + 2), (8, P + 2), (7, rows(P + (2 << 20) + 1)), (5, P + (3 << 20)),
                    (8, last + 4)):
        a = list(ok)
        a[at] = bad
        assert lib.msgla_scan_backward(*a) == -1, (at, bad)
    ok = [c, 2, x, z, None, P + (5 << 20), d, None]
    for at, bad in ((2, None), (3, rows(0)), (5, None), (5, P), (6, None), (6, x), (6, rows(P + (2 << 20), 0)),
                    (6, rows(P + (2 << 20), 7)), (5, P + (5 << 20) + 1), (4, P + (5 << 20) + 5), (1, -1), (1, 65536)):
        a = list(ok)
        a[at] = bad
        assert lib.msgla_scan_step(*a) == -1, (at, bad)


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(C=0), dict(C=(1 << 24) + 1), dict(groups=0), dict(groups=3), dict(activation=3),
                                dict(activation=-1), dict(center=2), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan"))])
def test_norm_rejects_bad_config(kw):
    lib, n = _lib.load(), ctypes.c_size_t()
    assert lib.msgla_group_norm_workspace_size(norm_cfg(**kw), 1, 1, 0, ctypes.byref(n)) == -1
    assert lib.msgla_group_norm_forward(norm_cfg(**kw), 0, 0, None, None, None, None, None, None, None, None, 0, None) == -1
    assert lib.msgla_group_norm_backward(norm_cfg(**kw), 0, 0, *[None] * 12, 0, None) == -1


@pytest.mark.parametrize("N,S", [(-1, 1), (1, -1), (1 << 31, 1), (1 << 30, 2), (1 << 16, 1 << 15), (1 << 30, 1)])
def test_norm_rejects_bad_sizes(N, S):
    lib, n = _lib.load(), ctypes.c_size_t()
    assert lib.msgla_group_norm_workspace_size(norm_cfg(), N, S, 1, ctypes.byref(n)) == -1


def test_norm_rejects_bad_buffers():
    lib, c = _lib.load(), norm_cfg()
    n = ctypes.c_size_t()
    x, g, y, dy, dg = (rows(P + (k << 20)) for k in range(5))
    w, st, ws, big = P + (6 << 20), P + (7 << 20), P + (16 << 20), 1 << 22
    ok = [c, 2, 8, x, g, w, None, None, y, st, ws, big, None]
    for at, bad in ((3, None), (3, rows(0)), (4, rows(0)), (8, None), (8, x), (8, rows(P + (2 << 20), 64, 7)), (5, w + 2), (9, w),
                    (9, P + 2), (9, P), (7, P + (2 << 20)), (3, rows(P + 1))):
        a = list(ok)
        a[at] = bad
        assert lib.msgla_group_norm_forward(*a) == -1, (at, bad)
    ok = [c, 2, 8, x, g, w, None, None, st, dy, y, dg, P + (8 << 20), P + (9 << 20), ws, big, None]
    for at, bad in ((8, None), (9, None), (10, None), (11, None), (4, None), (10, x), (11, y), (12, w), (13, P + (8 << 20)), (12, st),
                    (12, P + 2), (10, dy)):
        a = list(ok)
        a[at] = bad
        assert lib.msgla_group_norm_backward(*a) == -1, (at, bad)
    for backward in (0, 1):  # a workspace that is missing, short or misaligned
        assert lib.msgla_group_norm_workspace_size(c, 2, 8, backward, ctypes.byref(n)) == 0
        if n.value:
            for bad, size in ((None, big), (ws, n.value - 1), (ws + 8, big)):
                a = [c, 2, 8, x, g, w, None, None, y, st, bad, size, None] if not backward else \
                    [c, 2, 8, x, g, w, None, None, st, dy, y, dg, None, None, bad, size, None]
                f = lib.msgla_group_norm_backward if backward else lib.msgla_group_norm_forward
                assert f(*a) == -6
