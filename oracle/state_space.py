"""fp64 oracle of a state-space layer's operators: the selective scan, the short convolution with its
carried window and layer norm, each with its gradients, written token by token from the formulas.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``: only the test suite imports it; the library
never does, and they share no code.

``*_scale`` functions give, for every output, the sum of the absolute values of the terms it is made
of: rounding errors of the fp32 kernels are bounded by a multiple of it.
"""
from __future__ import annotations

import numpy as np


def _f(x):
    return None if x is None else np.asarray(x, np.float64)


def softplus(x):
    return np.logaddexp(x, 0.0)


def sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def scan_core(u, delta, A, B, C, skip, cu, h0):
    """h_t = exp(delta A) h_{t-1} + delta u B_t and y = C h + skip u.  B, C [T, G, n].
    Returns y [T, D], the state before every token [T, D, n] and the final states."""
    T, D = u.shape
    G, n = B.shape[1:]
    grp = np.arange(D) // (D // G)
    y, before, last = np.zeros((T, D)), np.zeros((T, D, n)), np.array(h0)
    for s in range(len(cu) - 1):
        h = np.array(h0[s])
        for t in range(cu[s], cu[s + 1]):
            before[t] = h
            h = np.exp(delta[t][:, None] * A) * h + (delta[t] * u[t])[:, None] * B[t][grp]
            y[t] = (h * C[t][grp]).sum(1) + skip * u[t]
        last[s] = h
    return y, before, last


def scan_core_bwd(u, delta, A, A_factor, B, C, skip, cu, before, dy, dlast):
    """Gradients of scan_core with respect to u, delta, A (times A_factor: of A_log), B, C, skip and h0."""
    T, D = u.shape
    G, n = B.shape[1:]
    grp = np.arange(D) // (D // G)
    g = dict(du=np.zeros((T, D)), ddelta=np.zeros((T, D)), dA_log=np.zeros((D, n)), dB=np.zeros((T, G, n)),
             dC=np.zeros((T, G, n)), dskip=(dy * u).sum(0), dh0=np.array(dlast))
    for s in range(len(cu) - 1):
        dh = np.array(dlast[s])
        for t in reversed(range(cu[s], cu[s + 1])):
            a = np.exp(delta[t][:, None] * A)
            h = a * before[t] + (delta[t] * u[t])[:, None] * B[t][grp]
            dh = dh + dy[t][:, None] * C[t][grp]
            np.add.at(g["dC"][t], grp, dy[t][:, None] * h)
            np.add.at(g["dB"][t], grp, dh * (delta[t] * u[t])[:, None])
            db, e = (dh * B[t][grp]).sum(1), dh * before[t] * a
            g["du"][t] = db * delta[t] + skip * dy[t]
            g["ddelta"][t] = db * u[t] + (e * A_factor).sum(1)
            g["dA_log"] += e * delta[t][:, None] * A_factor
            dh = a * dh
        g["dh0"][s] = dh
    return g


def _scan_terms(u, dt, A_log, B, C, cu, skip, z, dt_bias, h0):
    u, dt, A_log, B, C, skip, z, dt_bias, h0 = map(_f, (u, dt, A_log, B, C, skip, z, dt_bias, h0))
    D, n = A_log.shape
    skip = np.zeros(D) if skip is None else skip
    pre = dt + (0.0 if dt_bias is None else dt_bias)
    h0 = np.zeros((len(cu) - 1, D, n)) if h0 is None else h0
    return u, pre, softplus(pre), -np.exp(A_log), B, C, skip, z, h0


def selective_scan(u, dt, A_log, B, C, cu, skip=None, z=None, dt_bias=None, h0=None, scale=False):
    """(out, final states); with ``scale`` of the absolute values of all terms."""
    u, _, delta, A, B, C, skip, z, h0 = _scan_terms(u, dt, A_log, B, C, cu, skip, z, dt_bias, h0)
    if scale:
        u, B, C, skip, h0 = map(np.abs, (u, B, C, skip, h0))
    y, _, last = scan_core(u, delta, A, B, C, skip, cu, h0)
    gate = 1.0 if z is None else z * sigmoid(z)
    return y * (np.abs(gate) if scale else gate), last


def selective_scan_bwd(u, dt, A_log, B, C, cu, dout, skip=None, z=None, dt_bias=None, h0=None, dlast=None, scale=False):
    """Gradients by name as kda_selective_scan_bwd returns them; with ``scale`` of absolute values."""
    u, pre, delta, A, B, C, skip, z, h0 = _scan_terms(u, dt, A_log, B, C, cu, skip, z, dt_bias, h0)
    dout = _f(dout)
    dlast = np.zeros_like(h0) if dlast is None else _f(dlast)
    A_factor = A
    gate = np.ones_like(u) if z is None else z * sigmoid(z)
    dgate = np.zeros_like(u) if z is None else sigmoid(z) * (1 + z * (1 - sigmoid(z)))
    if scale:
        u, B, C, skip, h0, dout, dlast, A_factor, gate = map(np.abs, (u, B, C, skip, h0, dout, dlast, A_factor, gate))
        dgate = np.abs(dgate) + 0.5   # silu' may vanish: its own rounding does not
    y, before, _ = scan_core(u, delta, A, B, C, skip, cu, h0)
    g = scan_core_bwd(u, delta, A, A_factor, B, C, skip, cu, before, dout * gate, dlast)
    ddt = g["ddelta"] * sigmoid(pre)
    return dict(du=g["du"], ddt=ddt, dA_log=g["dA_log"], dB=g["dB"], dC=g["dC"], dskip=g["dskip"], dz=dout * y * dgate,
                ddt_bias=ddt.sum(0), dinitial_state=g["dh0"])


def _rows(x, h0, cu, s, W):
    """The carried rows and the tokens of sequence s."""
    old = np.zeros((W - 1,) + x.shape[1:]) if h0 is None else h0[s]
    return np.concatenate([old, x[cu[s]:cu[s + 1]]])


def short_conv(x, w, cu, bias=None, h0=None, silu=False, l2norm=False):
    """(y, final windows): x [T, H, d], w [H, d, W], windows [N, W - 1, H, d]."""
    x, w, bias, h0 = map(_f, (x, w, bias, h0))
    W = w.shape[-1]
    y, last = np.zeros_like(x), np.zeros((len(cu) - 1, W - 1) + x.shape[1:])
    for s in range(len(cu) - 1):
        rows = _rows(x, h0, cu, s, W)
        for t in range(cu[s], cu[s + 1]):
            i = t - cu[s]
            p = sum(w[..., j] * rows[i + j] for j in range(W)) + (0.0 if bias is None else bias)
            a = p * sigmoid(p) if silu else p
            y[t] = a / np.sqrt((a * a).sum(-1, keepdims=True) + 1e-12) if l2norm else a
        last[s] = rows[len(rows) - (W - 1):]
    return y, last


def short_conv_bwd(x, w, cu, dy, bias=None, h0=None, dlast=None, silu=False, l2norm=False, scale=False):
    """Gradients by name as kda_short_conv_bwd returns them; with ``scale`` of absolute values."""
    x, w, bias, h0, dy, dlast = map(_f, (x, w, bias, h0, dy, dlast))
    mag = np.abs if scale else (lambda v: v)
    W = w.shape[-1]
    g = dict(dx=np.zeros_like(x), dw=np.zeros_like(w), dbias=np.zeros(x.shape[1:]),
             dinitial_state=np.zeros((len(cu) - 1, W - 1) + x.shape[1:]))
    for s in range(len(cu) - 1):
        rows = _rows(x, h0, cu, s, W)
        drows = np.zeros_like(rows)
        if dlast is not None and W > 1:
            drows[len(rows) - (W - 1):] += mag(dlast[s])
        for t in range(cu[s], cu[s + 1]):
            i = t - cu[s]
            p = sum(w[..., j] * rows[i + j] for j in range(W)) + (0.0 if bias is None else bias)
            sg = sigmoid(p)
            a = p * sg if silu else p
            d = mag(dy[t])
            if l2norm:
                inv = 1 / np.sqrt((a * a).sum(-1, keepdims=True) + 1e-12)
                y = mag(a * inv)
                d = inv * (d + y * (y * d).sum(-1, keepdims=True)) if scale else inv * (d - y * (y * d).sum(-1, keepdims=True))
            if silu:
                d = d * ((np.abs(sg * (1 + p * (1 - sg))) + 0.5) if scale else sg * (1 + p * (1 - sg)))
            for j in range(W):
                drows[i + j] += d * mag(w[..., j])
                g["dw"][..., j] += d * mag(rows[i + j])
            g["dbias"] += d
        g["dinitial_state"][s] = drows[:W - 1]
        g["dx"][cu[s]:cu[s + 1]] = drows[W - 1:]
    return g


def layer_norm(x, w, b=None, eps=1e-5):
    """(y, mean, rstd) of rows x [rows, d]."""
    x, w, b = _f(x), _f(w), _f(b)
    mean = x.mean(-1)
    rstd = 1 / np.sqrt(((x - mean[:, None]) ** 2).mean(-1) + eps)
    return (x - mean[:, None]) * rstd[:, None] * w + (0.0 if b is None else b), mean, rstd


def layer_norm_bwd(x, w, dy, eps=1e-5):
    x, w, dy = _f(x), _f(w), _f(dy)
    _, mean, rstd = layer_norm(x, w, eps=eps)
    xh, g = (x - mean[:, None]) * rstd[:, None], dy * w
    dx = rstd[:, None] * (g - g.mean(-1, keepdims=True) - xh * (g * xh).mean(-1, keepdims=True))
    return dict(dx=dx, dw=(dy * xh).sum(0), dbias=dy.sum(0))
