"""Which buffers of one call may lie where: rows side by side are taken, everything else that meets an output
is refused before the device is touched. No GPU needed (the pointers are never read: without one the
calls that are taken end at the device)."""
import ctypes

import pytest

from scale_gated_linear_b200 import _lib

P = 1 << 30


def refused(at_h, sb, sl, B=3, L=5, D=8, x=P, x_strides=None):
    """Whether h at `at_h` elements past x, of 2 bytes each, is refused. The device does not exist, so that a call that
    is taken never gets to a launch."""
    cfg = _lib.ScanConfig(4096, 0, D, 0, 16.0)
    rows = lambda at, st: _lib.Rows(at, *st)
    st = _lib.load().msgla_scan_forward(cfg, B, L, rows(x, x_strides or (sb, sl)), rows(P + (1 << 24), (L * D, D)), None, None,
                                        rows(x + 2 * at_h, (sb, sl)), P + (1 << 26), None, None)
    assert st < 0
    return st == -1


@pytest.mark.parametrize("at_h,sb,sl,kw,want", [
    (8, 80, 16, {}, False), (-8, 80, 16, {}, False),     # halves of [B, L, 2 D], either way round
    (8, 16, 48, {}, False), (8, 120, 24, {}, False),     # [L, B, 2 D], thirds
    (7, 80, 16, {}, True), (9, 80, 16, {}, True),        # a row's end inside the other, or in the next slot
    (0, 80, 16, {}, True), (16, 80, 16, {}, True),       # the same rows, rows of the next slot
    (8, 79, 16, {}, True), (8, 80, 15, {}, True),        # slots too narrow
    (8, 80, 16, {"x_strides": (160, 32)}, True),         # other strides
    (40, 80, 8, {}, False), (41, 80, 8, {}, True),       # whole sequences side by side in [B, 2, L, D]
    (39, 80, 8, {}, True), (24, 16, 48, {"B": 1}, False), (8, 16, 0, {"L": 1}, False), (8, 15, 0, {"L": 1}, True),
])
def test_rows_beside_rows(at_h, sb, sl, kw, want):
    assert refused(at_h, sb, sl, **kw) is want


def test_two_gradients_side_by_side():
    lib, cfg = _lib.load(), _lib.ScanConfig(4096, 0, 8, 0, 16.0)
    for dz, want in ((P + 16, False), (P + 14, True), (P, True), (P + 18, True)):
        st = lib.msgla_scan_backward(cfg, 2, 4, _lib.Rows(P + (1 << 20), 32, 8), _lib.Rows(P + (2 << 20), 32, 8), None, P + (3 << 20), None,
                                     None, _lib.Rows(P, 64, 16), _lib.Rows(dz, 64, 16), None, None)
        assert st < 0 and (st == -1) is want
    # a state buffer is no rows: beside them in span or not at all
    st = lib.msgla_scan_step(cfg, 2, _lib.Rows(P, 64, 0), _lib.Rows(P + (2 << 20), 8, 0), None, P + 16, _lib.Rows(P + (4 << 20), 8, 0), None)
    assert st == -1
