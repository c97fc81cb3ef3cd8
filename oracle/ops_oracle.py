"""Plain fp64 CPU oracle of the gated recurrence and of group normalisation.

TEST INFRASTRUCTURE, numpy alone, no code shared with the product. The recurrence is
written token by token, its gradients as the adjoint recurrence token by token; each
function's gradients are pinned by central differences in tests/test_oracle_ops.py.

``scan_error`` and ``norm_error`` bound what 32-bit arithmetic may add to the exact
values; a result stored in fewer bits is off by half a step of its type besides.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # unit roundoff of f32


def softplus_neg(z):
    """log(1 + e^-z) = -log(sigmoid(z)), exact to 64 bits for every z (0 at +inf, inf at -inf)."""
    z = np.asarray(z, dtype=np.float64)
    with np.errstate(over="ignore"):
        return np.where(z > 0, np.log1p(np.exp(-np.abs(z))), -np.minimum(z, 0) + np.log1p(np.exp(-np.abs(z))))


def scan(x, z, tau=16.0, tied=False, mask=None, h0=None):
    """h [B, L, D], the state after the last row and the states before every row
    [B, L + 1, D] for x, z [B, L, D]. Padded rows are never read."""
    B, L, D = x.shape
    states = np.zeros((B, L + 1, D))
    if h0 is not None:
        states[:, 0] = h0
    out = np.zeros((B, L, D))
    for b in range(B):
        for t in range(L):
            states[b, t + 1] = states[b, t]
            if mask is not None and not mask[b, t]:
                continue
            s = softplus_neg(z[b, t]) / tau
            a, c = np.exp(-s), -np.expm1(-s)
            states[b, t + 1] = a * states[b, t] + (c * x[b, t] if tied else x[b, t])
            out[b, t] = states[b, t + 1]
    return out, states[:, L].copy(), states


def scan_backward(dh, dlast, x, z, tau=16.0, tied=False, mask=None, h0=None):
    """Gradients (dx, dz, dh0) of sum(dh * h) + sum(dlast * last), and g_t = dL/dh_t."""
    B, L, D = x.shape
    _, _, states = scan(x, z, tau, tied, mask, h0)
    dx, dz, g_all = np.zeros((B, L, D)), np.zeros((B, L, D)), np.zeros((B, L, D))
    dh0 = np.zeros((B, D))
    for b in range(B):
        carry = np.zeros(D) if dlast is None else np.array(dlast[b], dtype=np.float64)
        for t in range(L - 1, -1, -1):
            if mask is not None and not mask[b, t]:
                continue
            s = softplus_neg(z[b, t]) / tau
            a, c = np.exp(-s), -np.expm1(-s)
            g = carry + (0 if dh is None else dh[b, t])
            g_all[b, t] = g
            dx[b, t] = c * g if tied else g
            with np.errstate(over="ignore"):
                down = 1 / (1 + np.exp(z[b, t]))
            dz[b, t] = g * (states[b, t] - (x[b, t] if tied else 0)) * a * down / tau
            carry = a * g
        dh0[b] = carry
    return dx, dz, dh0, g_all


def _error_recurrence(a, c, v, prev, u, start=0.0):
    """|error| of v_t = a_t v_{t-1} + u_t along axis 0 in f32: every row hands its error on
    through a_t and adds the roundings of its product and sum, and the error of c_t
    (8 U of c_t: two interpolations and four roundings) times what it multiplies."""
    e = np.zeros_like(v)
    last = np.full_like(v[0], start)
    for t in range(v.shape[0]):
        last = a[t] * last + U * (np.abs(prev[t]) + np.abs(v[t]) + 8 * c[t] * np.abs(prev[t]) + 9 * np.abs(u[t]))
        e[t] = last
    return e


def scan_error(x, z, tau, tied, mask, h0, dh=None, dlast=None):
    """Bounds of the f32 error of (states [B, L + 1, D], dx, dz, dh0). The factor 8 covers the
    order of the sums: rows are joined in blocks (local results, products of the decays), where
    every value passes through up to three products and sums where the token-by-token form has one."""
    B, L, D = x.shape
    _, _, states = scan(x, z, tau, tied, mask, h0)
    keep = np.ones((B, L), bool) if mask is None else np.asarray(mask) != 0
    z_, x_ = np.where(keep[..., None], z, 0), np.where(keep[..., None], x, 0)
    s = softplus_neg(z_) / tau
    a, c = np.where(keep[..., None], np.exp(-s), 1.0), np.where(keep[..., None], -np.expm1(-s), 0.0)
    u = np.where(keep[..., None], c * x_ if tied else x_, 0)
    # sums of magnitudes: nothing cancels in the blocks' partial results
    mag = np.abs(states[:, 0]).copy()
    mags = np.zeros((B, L + 1, D))
    mags[:, 0] = mag
    for t in range(L):
        mags[:, t + 1] = a[:, t] * mags[:, t] + np.abs(u[:, t])
    e = np.zeros((B, L + 1, D))
    for b in range(B):
        e[b, 1:] = _error_recurrence(a[b], c[b], mags[b, 1:], mags[b, :-1], u[b])
    if dh is None and dlast is None:
        return 8 * e
    dx, dz, dh0, g = scan_backward(dh, dlast, x, z, tau, tied, mask, h0)
    d = np.zeros((B, L, D)) if dh is None else np.where(keep[..., None], dh, 0)
    gm = np.zeros((B, L + 1, D))  # magnitudes handed down: gm[t] = a_t (|dh_t| + gm[t + 1])
    gm[:, L] = 0 if dlast is None else np.abs(dlast)
    for t in range(L - 1, -1, -1):
        gm[:, t] = a[:, t] * (np.abs(d[:, t]) + gm[:, t + 1])
    eg = np.zeros((B, L + 1, D))
    for t in range(L - 1, -1, -1):
        gt = np.abs(d[:, t]) + gm[:, t + 1]
        eg[:, t] = a[:, t] * eg[:, t + 1] + U * (2 * gt + 8 * c[:, t] * gt)
    gt = np.abs(d) + gm[:, 1:]
    with np.errstate(over="ignore"):
        down = 1 / (1 + np.exp(z_)) / tau
    xm = np.abs(x_) if tied else 0
    edx = eg[:, 1:] * (c if tied else 1) + 9 * U * gt * (c if tied else 1)
    edz = ((eg[:, 1:] + 2 * U * gt) * (mags[:, :-1] + xm) + gt * (e[:, :-1] + U * (mags[:, :-1] + xm))) * (a + 2 * U) * down
    edz += (12 * U * (a + U) + 2 * U) * gt * (mags[:, :-1] + xm) * down
    keep3 = keep[..., None]
    return 8 * e, 8 * np.where(keep3, edx, 0), 8 * np.where(keep3, edz, 0), 8 * eg[:, 0]


def _act(kind, v):
    if kind == "none":
        return v, np.ones_like(v)
    s = 1 / (1 + np.exp(-v))
    return (s, s * (1 - s)) if kind == "sigmoid" else (v * s, s * (1 + v * (1 - s)))


def group_norm(x, groups, w=None, b=None, gate=None, mask=None, act="none", eps=1e-5, center=True, dy=None):
    """y for x [N, S, C], and with dy also (dx, dw, db, dgate)."""
    N, S, C = x.shape
    cg = C // groups
    w = np.ones(C) if w is None else w
    b = np.zeros(C) if b is None else b
    y, dx, dg = np.zeros(x.shape), np.zeros(x.shape), np.zeros(x.shape)
    dw, db = np.zeros(C), np.zeros(C)
    for n in range(N):
        rows = np.arange(S) if mask is None else np.flatnonzero(mask[n])
        if len(rows) == 0:
            continue
        for g in range(groups):
            ch = slice(g * cg, (g + 1) * cg)
            v = x[n, rows, ch]
            mean = v.mean() if center else 0.0
            rstd = 1 / np.sqrt(((v - mean) ** 2).mean() + eps)
            xhat = (v - mean) * rstd
            v = xhat * w[ch] + b[ch]
            gt = None if gate is None else gate[n, rows, ch]
            f, df = _act(act, v if gt is None else gt)
            y[n, rows, ch] = f if gt is None else v * f
            if dy is None:
                continue
            d = dy[n, rows, ch]
            dv = d * (df if gt is None else f)
            if gt is not None:
                dg[n, rows, ch] = d * v * df
            dw[ch] += (dv * xhat).sum(0)
            db[ch] += dv.sum(0)
            dxh = dv * w[ch]
            dx[n, rows, ch] = rstd * (dxh - (dxh.mean() if center else 0.0) - xhat * (dxh * xhat).mean())
    return y if dy is None else (y, (dx, dw, db, None if gate is None else dg))


def norm_error(x, groups, w=None, b=None, gate=None, mask=None, act="none", eps=1e-5, center=True, dy=None):
    """Bounds of the f32 error of y, and with dy of (dx, dw, db, dgate). K counts roundings: a
    sum takes at most 96 additions in a row in one thread and fewer than 32 joins after
    it, a value passes fewer than 64 other roundings (sigmoid's 8, products, differences). The
    squares of samples held in shared memory take up to 200 additions in a row, of which the
    root of the variance hands on half; their mean is corrected by a second sum."""
    K = 192 * U
    N, S, C = x.shape
    cg = C // groups
    w = np.ones(C) if w is None else w
    b = np.zeros(C) if b is None else b
    ey, edx, edg = np.zeros(x.shape), np.zeros(x.shape), np.zeros(x.shape)
    edw, edb = np.zeros(C), np.zeros(C)
    for n in range(N):
        rows = np.arange(S) if mask is None else np.flatnonzero(mask[n])
        if len(rows) == 0:
            continue
        for g in range(groups):
            ch = slice(g * cg, (g + 1) * cg)
            v = x[n, rows, ch]
            mean = v.mean() if center else 0.0
            rstd = 1 / np.sqrt(((v - mean) ** 2).mean() + eps)
            xhat = (v - mean) * rstd
            exh = K * (np.abs(v) * rstd + np.abs(mean) * rstd + np.abs(xhat) * (1 + np.abs(v).mean() * rstd))
            v = xhat * w[ch] + b[ch]
            ev = exh * np.abs(w[ch]) + K * (np.abs(v) + np.abs(b[ch]))
            gt = None if gate is None else gate[n, rows, ch]
            f, df = _act(act, v if gt is None else gt)
            slope = 1.2  # largest |act'|; |act''| stays below 1
            ey[n, rows, ch] = (slope * ev + K * (np.abs(f) + np.abs(v))) if gt is None else ev * np.abs(f) + np.abs(v) * K * (np.abs(f) + 1)
            if dy is None:
                continue
            d = np.abs(dy[n, rows, ch])
            dv = d * np.abs(df if gt is None else f)
            edv = d * ((ev + K * (1 + np.abs(v))) if gt is None else K * (np.abs(f) + 1))
            if gt is not None:
                edg[n, rows, ch] = d * (ev * np.abs(df) + np.abs(v) * K * (1 + np.abs(gt)))
            edw[ch] += (edv * np.abs(xhat) + dv * exh + K * dv * np.abs(xhat)).sum(0)
            edb[ch] += (edv + K * dv).sum(0)
            dxh, edxh = dv * np.abs(w[ch]), edv * np.abs(w[ch])
            m2, em2 = (dxh * np.abs(xhat)).mean(), (edxh * np.abs(xhat) + dxh * exh + K * dxh * np.abs(xhat)).mean()
            edx[n, rows, ch] = rstd * (edxh + edxh.mean() + K * (dxh + dxh.mean()) + exh * m2 + np.abs(xhat) * (em2 + K * m2)
                                       + K * (1 + np.abs(v).mean() * rstd) * (dxh + dxh.mean() + np.abs(xhat) * m2))
    return ey if dy is None else (ey, (edx, edw, edb, None if gate is None else edg))
