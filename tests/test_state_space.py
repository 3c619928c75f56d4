"""The state-space operators without a GPU: the oracle's gradients against differences, the workspace
sizes, and every call that has to be refused before anything is enqueued."""
import ctypes

import numpy as np
import pytest
import torch

import __graft_entry__
from oracle import state_space as S

__graft_entry__._builder().build()
import kda_chunkwise_b200 as kda  # noqa: E402

lib = kda.lib
OK, INVALID, UNSUPPORTED = kda.KDA_OK, kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED


def _differences(loss, x, step=1e-5):
    """d loss / d x by central differences (x is changed in place and restored)."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + step
        hi = loss()
        x[i] = keep - step
        lo = loss()
        x[i] = keep
        g[i] = (hi - lo) / (2 * step)
    return g


def _near(a, b, label):
    # central differences: step^2 / 6 of third derivatives of order one, and 1e-16 / step of rounding
    assert np.abs(a - b).max(initial=0.0) <= 1e-7 * (1 + np.abs(b).max(initial=0.0)), label


@pytest.mark.parametrize("gate", [False, True])
def test_scan_oracle_gradients_against_differences(gate):
    r = np.random.default_rng(1)
    cu, D, G, n = [0, 3, 3, 7], 4, 2, 3
    v = dict(u=r.normal(size=(7, D)), dt=r.normal(size=(7, D)), A_log=0.3 * r.normal(size=(D, n)),
             B=r.normal(size=(7, G, n)), C=r.normal(size=(7, G, n)), skip=r.normal(size=D),
             z=r.normal(size=(7, D)) if gate else None, dt_bias=r.normal(size=D), h0=r.normal(size=(3, D, n)))
    dout, dlast = r.normal(size=(7, D)), r.normal(size=(3, D, n))

    def loss():
        out, last = S.selective_scan(cu=cu, **v)
        return (out * dout).sum() + (last * dlast).sum()

    g = S.selective_scan_bwd(cu=cu, dout=dout, dlast=dlast, **v)
    names = dict(u="du", dt="ddt", A_log="dA_log", B="dB", C="dC", skip="dskip", z="dz", dt_bias="ddt_bias",
                 h0="dinitial_state")
    for k, x in v.items():
        if x is not None:
            _near(_differences(loss, x), g[names[k]], k)


@pytest.mark.parametrize("W", [1, 2, 4])
@pytest.mark.parametrize("silu,l2norm", [(False, False), (True, False), (False, True), (True, True)])
def test_conv_oracle_gradients_against_differences(W, silu, l2norm):
    r = np.random.default_rng(2)
    cu, H, d = [0, 1, 1, 6], 2, 3
    v = dict(x=r.normal(size=(6, H, d)), w=r.normal(size=(H, d, W)), bias=r.normal(size=(H, d)),
             h0=r.normal(size=(3, W - 1, H, d)))
    dy, dlast = r.normal(size=(6, H, d)), r.normal(size=(3, W - 1, H, d))

    def loss():
        y, last = S.short_conv(cu=cu, silu=silu, l2norm=l2norm, **v)
        return (y * dy).sum() + (last * dlast).sum()

    g = S.short_conv_bwd(cu=cu, dy=dy, dlast=dlast, silu=silu, l2norm=l2norm, **v)
    for k, name in (("x", "dx"), ("w", "dw"), ("bias", "dbias"), ("h0", "dinitial_state")):
        _near(_differences(loss, v[k]), g[name], k)


def test_norm_oracle_gradients_against_differences():
    r = np.random.default_rng(3)
    x, w, b, dy = r.normal(size=(3, 5)), r.normal(size=5), r.normal(size=5), r.normal(size=(3, 5))
    loss = lambda: (S.layer_norm(x, w, b)[0] * dy).sum()  # noqa: E731
    g = S.layer_norm_bwd(x, w, dy)
    for v, name in ((x, "dx"), (w, "dw"), (b, "dbias")):
        _near(_differences(loss, v), g[name], name)


def test_scan_oracle_closed_forms():
    # delta = log 2 (dt = 0), A = -1: a decay of one half a token; one state, B = C = 1
    T = 5
    one = np.ones((T, 1, 1))
    out, last = S.selective_scan(np.ones((T, 1)), np.zeros((T, 1)), np.zeros((1, 1)), one, one, [0, T])
    assert np.allclose(out[:, 0], 2 * np.log(2) * (1 - 0.5 ** np.arange(1, T + 1)), atol=1e-15)
    assert np.allclose(last[0, 0, 0], out[-1, 0])


# ---- refusals -----------------------------------------------------------------------------------

P = ctypes.c_void_p


def _p(k=0):
    """A pointer that is never followed: aligned, with 16 GiB between any two."""
    return P((k + 1) << 34)


def scan_fwd(**kw):
    a = dict(u=_p(0), dt=_p(1), A_log=_p(2), B=_p(3), C=_p(4), skip=None, z=None, dt_bias=None, cu=_p(5), num_seqs=1, T=8,
             D=8, n=16, G=1, h0=None, hN=None, out=_p(6), dtype=0, ws=_p(7), ws_bytes=1 << 30)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kda_selective_scan_fwd(*a.values(), None)


def scan_step(**kw):
    a = dict(u=_p(0), dt=_p(1), A_log=_p(2), B=_p(3), C=_p(4), skip=None, z=None, dt_bias=None, state=_p(5), out=_p(6),
             dtype=0, N=2, D=8, n=16, G=1)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kda_selective_scan_step(*a.values(), None)


def scan_bwd(**kw):
    a = dict(u=_p(0), dt=_p(1), A_log=_p(2), B=_p(3), C=_p(4), skip=None, z=None, dt_bias=None, cu=_p(5), num_seqs=1, T=8,
             D=8, n=16, G=1, h0=None, dout=_p(6), dhN=None, du=_p(7), ddt=_p(8), dA_log=_p(9), dB=_p(10), dC=_p(11),
             dskip=None, dz=None, ddt_bias=None, dh0=None, dtype=0, ws=_p(12), ws_bytes=1 << 30)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kda_selective_scan_bwd(*a.values(), None)


def conv_fwd(**kw):
    a = dict(x=_p(0), w=_p(1), bias=None, cu=_p(2), num_seqs=1, T=8, H=1, d=64, width=4, silu=1, l2norm=0, h0=None, hN=None,
             y=_p(3), dtype=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kda_short_conv_fwd(*a.values(), None)


def conv_step(**kw):
    a = dict(x=_p(0), w=_p(1), bias=None, state=_p(2), N=2, H=1, d=64, width=4, silu=1, l2norm=0, y=_p(3), dtype=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kda_short_conv_step(*a.values(), None)


def conv_bwd(**kw):
    a = dict(x=_p(0), w=_p(1), bias=None, cu=_p(2), num_seqs=1, T=8, H=1, d=64, width=4, silu=1, l2norm=0, h0=None,
             dy=_p(3), dhN=None, dx=_p(4), dw=_p(5), dbias=None, dh0=None, dtype=0, ws=_p(6), ws_bytes=1 << 30)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kda_short_conv_bwd(*a.values(), None)


def norm_fwd(**kw):
    a = dict(x=_p(0), w=_p(1), b=None, rows=4, d=64, eps=1e-5, y=_p(2), mean=_p(3), rstd=_p(4), dtype=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kda_layer_norm_fwd(*a.values(), None)


def norm_bwd(**kw):
    a = dict(x=_p(0), w=_p(1), mean=_p(2), rstd=_p(3), dy=_p(4), rows=4, d=64, dx=_p(5), dw=_p(6), db=None, dtype=0,
             ws=_p(7), ws_bytes=1 << 30)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kda_layer_norm_bwd(*a.values(), None)


def _off(k, by):
    return P(((k + 1) << 34) + by)


REFUSED = [
    (scan_fwd, dict(n=65), UNSUPPORTED), (scan_fwd, dict(n=0), INVALID), (scan_fwd, dict(D=0), INVALID),
    (scan_fwd, dict(D=9, G=2), INVALID), (scan_fwd, dict(T=-1), INVALID), (scan_fwd, dict(T=1 << 31), INVALID),
    (scan_fwd, dict(num_seqs=-1), INVALID), (scan_fwd, dict(num_seqs=0), INVALID), (scan_fwd, dict(dtype=2), INVALID),
    (scan_fwd, dict(u=None), INVALID), (scan_fwd, dict(cu=None), INVALID), (scan_fwd, dict(out=None), INVALID),
    (scan_fwd, dict(u=_off(0, 1)), INVALID), (scan_fwd, dict(u=_off(0, 2), dtype=1), INVALID), (scan_fwd, dict(h0=_off(8, 2)), INVALID),
    (scan_fwd, dict(ws=_off(7, 8), T=4096), INVALID), (scan_fwd, dict(A_log=_off(2, 2)), INVALID),
    (scan_fwd, dict(out=_off(0, 64)), INVALID), (scan_fwd, dict(h0=_p(8), hN=_off(8, 16)), INVALID),
    (scan_fwd, dict(T=4096, ws_bytes=16), INVALID), (scan_fwd, dict(T=4096, ws=None), INVALID),
    (scan_fwd, dict(T=(1 << 31) - 1), INVALID), (scan_fwd, dict(hN=_p(0)), INVALID), (scan_fwd, dict(out=_p(8), h0=_p(8), hN=_p(8)), INVALID),
    (scan_step, dict(out=_p(5)), INVALID), (conv_fwd, dict(T=(1 << 31) - 1), INVALID), (conv_fwd, dict(hN=_p(3)), INVALID),
    (conv_step, dict(state=_p(3)), INVALID),
    (scan_step, dict(n=65), UNSUPPORTED), (scan_step, dict(N=-1), INVALID), (scan_step, dict(G=3), INVALID),
    (scan_step, dict(state=None), INVALID), (scan_step, dict(dtype=-1), INVALID), (scan_step, dict(out=_p(0)), INVALID),
    (scan_step, dict(state=_off(5, 2)), INVALID), (scan_step, dict(state=_p(3)), INVALID),
    (scan_bwd, dict(n=65), UNSUPPORTED), (scan_bwd, dict(dA_log=None), INVALID), (scan_bwd, dict(num_seqs=0), INVALID),
    (scan_bwd, dict(z=_p(13)), INVALID), (scan_bwd, dict(dout=None), INVALID), (scan_bwd, dict(du=_p(0)), INVALID),
    (scan_bwd, dict(ws_bytes=64), INVALID), (scan_bwd, dict(ws=_off(12, 4)), INVALID), (scan_bwd, dict(dtype=3), INVALID),
    (conv_fwd, dict(width=0), INVALID), (conv_fwd, dict(width=5), INVALID), (conv_fwd, dict(d=96, l2norm=1), UNSUPPORTED),
    (conv_fwd, dict(H=0), INVALID), (conv_fwd, dict(y=_p(0)), INVALID), (conv_fwd, dict(num_seqs=0), INVALID),
    (conv_fwd, dict(x=_off(0, 1)), INVALID), (conv_fwd, dict(h0=_p(5), hN=_off(5, 128)), INVALID),
    (conv_fwd, dict(dtype=7), INVALID),
    (conv_step, dict(state=None), INVALID), (conv_step, dict(width=9), INVALID), (conv_step, dict(y=_p(0)), INVALID),
    (conv_step, dict(state=_p(0)), INVALID), (conv_step, dict(d=100, l2norm=1), UNSUPPORTED), (conv_step, dict(N=-2), INVALID),
    (conv_bwd, dict(dw=None), INVALID), (conv_bwd, dict(dx=_p(3)), INVALID), (conv_bwd, dict(ws_bytes=8), INVALID),
    (conv_bwd, dict(d=32, l2norm=1), UNSUPPORTED), (conv_bwd, dict(dy=None), INVALID), (conv_bwd, dict(num_seqs=0), INVALID),
    (norm_fwd, dict(d=0), INVALID), (norm_fwd, dict(d=16385), UNSUPPORTED), (norm_fwd, dict(eps=-1.0), INVALID),
    (norm_fwd, dict(eps=float("nan")), INVALID), (norm_fwd, dict(y=_p(0)), INVALID), (norm_fwd, dict(rows=-1), INVALID),
    (norm_fwd, dict(w=None), INVALID), (norm_fwd, dict(dtype=2), INVALID),
    (norm_bwd, dict(d=20000), UNSUPPORTED), (norm_bwd, dict(mean=None), INVALID), (norm_bwd, dict(dx=_p(4)), INVALID),
    (norm_bwd, dict(ws=None), INVALID), (norm_bwd, dict(dw=None), INVALID), (norm_bwd, dict(x=_off(0, 1)), INVALID), (norm_bwd, dict(ws=_off(7, 4)), INVALID),
]


@pytest.mark.parametrize("call,kw,status", REFUSED, ids=[f"{c.__name__}-{i}" for i, (c, _, _) in enumerate(REFUSED)])
def test_refused_before_anything_is_enqueued(call, kw, status):
    before = kda.kda_launch_count()
    assert call(**kw) == status
    assert lib.kda_last_error() != b""
    assert kda.kda_launch_count() == before


def test_empty_calls_need_nothing():
    assert scan_fwd(num_seqs=0, T=0, u=None, out=None, A_log=None) == OK
    assert scan_step(N=0, u=None, state=None) == OK
    assert conv_fwd(num_seqs=0, T=0, x=None, y=None) == OK
    assert conv_step(N=0, x=None) == OK
    assert norm_fwd(rows=0, x=None, y=None) == OK


def test_workspace_sizes():
    fwd, bwd = kda.kda_selective_scan_fwd_workspace_size, kda.kda_selective_scan_bwd_workspace_size
    assert fwd(100, 4, 4096, 16) == 0                      # short: not cut
    assert fwd(1 << 20, 512, 4096, 16) == 0                # enough sequences
    assert fwd(1 << 16, 1, 64, 16) > 0                     # one long sequence of few channels is cut
    assert fwd(-1, 1, 64, 16) == 0 and fwd(64, 1, 64, 65) == 0 and fwd(64, 1, 64, 16, 3) == 0
    assert bwd(64, 1, 64, 16) > 0 and bwd(64, 1, 64, 65) == 0 and bwd(64, 1, 65, 16, 2) == 0
    assert bwd(8192, 1, 4096, 16) >= 2 * 4 * (8192 // 64) * 4096 * 16
    assert kda.kda_short_conv_bwd_workspace_size(100, 2, 64, 4) >= 5 * 128 * 4
    assert kda.kda_short_conv_bwd_workspace_size(100, 2, 64, 5) == 0
    assert kda.kda_layer_norm_bwd_workspace_size(100, 64) > 0
    assert kda.kda_layer_norm_bwd_workspace_size(100, 16385) == 0


def test_binding_refuses_what_the_kernels_do_not_take():
    f = torch.zeros
    cu = torch.tensor([0, 4], dtype=torch.int32)
    ok = dict(u=f(4, 8), dt=f(4, 8), A_log=f(8, 16), B=f(4, 1, 16), C=f(4, 1, 16), cu_seqlens=cu)
    with pytest.raises(ValueError, match="CUDA device"):
        kda.kda_selective_scan_fwd(**ok)
    for bad, error in ((dict(u=f(4, 8, dtype=torch.float16)), TypeError), (dict(dt=f(4, 9)), ValueError),
                       (dict(dt=f(4, 8, dtype=torch.bfloat16)), TypeError), (dict(B=f(4, 16)), ValueError),
                       (dict(C=f(16, 1, 4).transpose(0, 2)), ValueError), (dict(cu_seqlens=cu.long()), TypeError),
                       (dict(A_log=f(8, 16, dtype=torch.float64)), TypeError)):
        with pytest.raises(error):
            kda.kda_selective_scan_fwd(**{**ok, **bad})
    with pytest.raises(ValueError, match="state"):
        kda.kda_selective_scan_step(f(2, 8), f(2, 8), f(8, 16), f(2, 1, 16), f(2, 1, 16), f(3, 8, 16))
    with pytest.raises(ValueError, match="initial_state"):
        kda.kda_short_conv_fwd(f(4, 1, 8), f(1, 8, 4), cu, initial_state=f(1, 4, 1, 8))
    with pytest.raises(TypeError):
        kda.kda_layer_norm_fwd(f(4, 8, dtype=torch.float16), f(8))
    with pytest.raises(ValueError):
        kda.kda_layer_norm_fwd(f(4, 8), f(7))


OVERLAPS = [   # outputs over weights, carried states, each other and the workspace
    (scan_fwd, dict(out=_p(2))), (scan_fwd, dict(hN=_p(2))), (scan_fwd, dict(skip=_p(9), out=_p(9))), (scan_fwd, dict(hN=_p(5))),
    (scan_step, dict(state=_p(2))), (scan_step, dict(out=_p(2))),
    (scan_bwd, dict(h0=_p(13), dh0=_p(13))), (scan_bwd, dict(dhN=_p(13), dh0=_p(13))), (scan_bwd, dict(ddt=_p(7))),
    (scan_bwd, dict(dA_log=_p(2))), (scan_bwd, dict(dC=_p(10))), (scan_bwd, dict(ws=_p(0))), (scan_bwd, dict(ws=_p(7))),
    (scan_bwd, dict(dskip=_p(9))), (scan_bwd, dict(dt_bias=_p(13), ddt_bias=_p(13))), (scan_bwd, dict(dh0=_p(6))),
    (conv_fwd, dict(y=_p(1))), (conv_fwd, dict(hN=_p(1))), (conv_step, dict(state=_p(1))),
    (conv_bwd, dict(h0=_p(8), dh0=_p(8))), (conv_bwd, dict(dhN=_p(8), dh0=_p(8))), (conv_bwd, dict(dh0=_p(4))),
    (conv_bwd, dict(dw=_p(1))), (conv_bwd, dict(dbias=_p(5))), (conv_bwd, dict(ws=_p(3))), (conv_bwd, dict(ws=_p(4))),
    (norm_fwd, dict(y=_p(1))), (norm_fwd, dict(mean=_p(4))), (norm_fwd, dict(rstd=_p(2))),
    (norm_bwd, dict(dw=_p(1))), (norm_bwd, dict(db=_p(6))), (norm_bwd, dict(dx=_p(2))), (norm_bwd, dict(ws=_p(0))),
    (norm_bwd, dict(ws=_p(5))),
]


@pytest.mark.parametrize("call,kw", OVERLAPS, ids=[f"{c.__name__}-{i}" for i, (c, _) in enumerate(OVERLAPS)])
def test_overlaps_are_refused(call, kw):
    before = kda.kda_launch_count()
    assert call(**kw) == INVALID
    assert b"overlaps" in lib.kda_last_error()
    assert kda.kda_launch_count() == before


@pytest.mark.parametrize("call", [scan_fwd, scan_step, scan_bwd])
def test_more_channels_than_the_kernels_count_are_refused(call):
    before = kda.kda_launch_count()
    assert call(D=(1 << 24) + 1, n=1) == INVALID
    assert kda.kda_launch_count() == before
    assert kda.kda_selective_scan_bwd_workspace_size(8, 1, (1 << 24) + 1, 1) == 0
