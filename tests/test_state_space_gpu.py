"""GPU parity of the state-space operators against the fp64 oracle (oracle/state_space.py), element by
element, and of a layer made of them.

Tolerances.  H(t) = finfo(t).eps / 2 is the error of one rounding to the storage type t, relative to the
value.  The kernels compute in fp32 (u = 2^-24): every term of a sum carries a relative error that is
bounded by the roundings and approximations on its way, so an output is off by at most that many times
the sum of the terms' absolute values, which the oracle gives (scale).
  scan   a term of a state passes one decay a token: its exponential (2^-22 for the approximation, and
         2^-23 x for the rounded argument x, where x exp(-x) <= 0.37 bounds what is left of the term) and
         one fused product, 2^-23; with a factor of two for both directions of the backward pass that is
         under 2^-20 a token.  softplus, the gate and the sums over states and channels: under 64 u.
  conv   W + 1 products, SiLU and its derivative (2^-20 with the approximate sigmoid); with l2norm the
         norm's relative error is that of p, |p|_abs / |s| times larger.
  norm   sums of at most 64 values a thread and log2(d) levels, 128 u; differences from the mean are off
         by that times |x| + mean |x|.
  sums over tokens (weight gradients) add at most one u a token.
"""
import numpy as np
import pytest
import torch

from oracle import state_space as S

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kda():
    import kda_chunkwise_b200 as m
    return m


def half_step(t):
    return torch.finfo(t).eps / 2


def host(x):
    return None if x is None else x.detach().double().cpu().numpy()


def check(label, got, ref, scale, rel, t=None):
    """|got - ref| <= rel scale + half a step of the storage type."""
    t = t or got.dtype
    got = host(got)
    assert got.shape == ref.shape, label
    bound = rel * scale + half_step(t) * (np.abs(ref) + rel * scale) + 1e-30
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref) / bound, 0)), ref.shape)
        raise AssertionError(f"{label}: {bad.sum()} of {bad.size} off; at {i}: {got[i]} against {ref[i]}, bound {bound[i]}")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def cu_of(lens):
    return [0] + [int(x) for x in np.cumsum(lens)]


def dev_cu(lens):
    return torch.tensor(cu_of(lens), dtype=torch.int32, device="cuda")


def scan_inputs(lens, D, G, n, t, gate=True, skip=True, bias=True, state=True, seed=0, step=0.0):
    g = gen(seed)
    T, N = sum(lens), len(lens)
    r = lambda *s, dt=F32, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(dt)  # noqa: E731
    v = dict(u=r(T, D, dt=t), dt=r(T, D, dt=t), A_log=r(D, n, std=0.5), B=r(T, G, n, dt=t), C=r(T, G, n, dt=t),
             skip=r(D) if skip else None, z=r(T, D, dt=t) if gate else None,
             dt_bias=r(D) + step if bias else None, h0=r(N, D, n) if state else None)
    return v


def oracle_args(v):
    return {k: host(x) for k, x in v.items()}


def call_args(v):
    return (v["u"], v["dt"], v["A_log"], v["B"], v["C"]), dict(skip=v["skip"], z=v["z"], dt_bias=v["dt_bias"],
                                                               initial_state=v["h0"])


def scan_rel(lens):
    return (max(list(lens) + [1]) + 4) * 2.0 ** -20


def check_scan(kda, lens, v, out, last):
    a, cu = oracle_args(v), cu_of(lens)
    ref, ref_last = S.selective_scan(cu=cu, **a)
    sc, sc_last = S.selective_scan(cu=cu, scale=True, **a)
    check("out", out, ref, sc, scan_rel(lens))
    check("final_state", last, ref_last, sc_last, scan_rel(lens))


SHAPES = [  # D, G, n: every number of lanes, states that fill no quad, channels that fill no vector or block
    (1, 1, 1), (7, 1, 3), (40, 1, 4), (128, 1, 5), (130, 2, 8), (33, 3, 11), (64, 1, 16), (40, 4, 16), (100, 1, 16),
    (24, 2, 17), (16, 1, 32), (9, 1, 33), (24, 3, 64), (256, 1, 16), (20, 2, 6), (12, 1, 18), (36, 1, 2),
]
LENS = [[1], [5, 0, 33, 1, 0], [31, 32, 64, 65]]


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,G,n", SHAPES)
@pytest.mark.parametrize("lens", LENS, ids=["one", "short", "tiles"])
def test_scan_forward(kda, D, G, n, lens, t):
    v = scan_inputs(lens, D, G, n, t)
    args, kw = call_args(v)
    out, last = kda.kda_selective_scan_fwd(*args, dev_cu(lens), **kw)
    kda.kda_sync_check()
    assert out.dtype == t and last.dtype == F32
    check_scan(kda, lens, v, out, last)


@pytest.mark.parametrize("gate,skip,bias,state", [(False, False, False, False), (True, False, False, True),
                                                  (False, True, False, False), (False, False, True, True)])
@pytest.mark.parametrize("D,n", [(40, 16), (33, 7)])
def test_scan_forward_optional_arguments(kda, D, n, gate, skip, bias, state):
    lens = [40, 3]
    v = scan_inputs(lens, D, 1, n, BF, gate, skip, bias, state)
    args, kw = call_args(v)
    out, last = kda.kda_selective_scan_fwd(*args, dev_cu(lens), **kw)
    check_scan(kda, lens, v, out, last)
    assert kda.kda_selective_scan_fwd(*args, dev_cu(lens), output_final_state=False, **kw)[1] is None


@pytest.mark.parametrize("lens", [[700, 0, 1, 300], [1000], [256, 512, 257]])
@pytest.mark.parametrize("D,G,n", [(40, 1, 16), (6, 2, 5), (130, 1, 8)])
def test_scan_forward_cut_into_segments(kda, lens, D, G, n):
    assert kda.kda_selective_scan_fwd_workspace_size(sum(lens), len(lens), D, n, G) > 0
    v = scan_inputs(lens, D, G, n, F32)
    args, kw = call_args(v)
    cu = dev_cu(lens)
    out, last = kda.kda_selective_scan_fwd(*args, cu, **kw)
    kda.kda_sync_check()
    check_scan(kda, lens, v, out, last)
    # the final states over the initial ones
    pool = v["h0"].clone()
    out2, last2 = kda.kda_selective_scan_fwd(*args, cu, **{**kw, "initial_state": pool}, final_state=pool)
    assert last2 is pool and torch.equal(last2, last) and torch.equal(out2, out)


@pytest.mark.parametrize("D", [2048, 4096])
def test_scan_forward_more_blocks_than_the_gpu_holds(kda, D):
    """Blocks of long sequences start first; from twice the SMs on, two blocks share one."""
    lens, n = [200, 500, 0, 300], 16
    assert kda.kda_selective_scan_fwd_workspace_size(sum(lens), len(lens), D, n, 2) == 0
    v = scan_inputs(lens, D, 2, n, BF)
    args, kw = call_args(v)
    out, last = kda.kda_selective_scan_fwd(*args, dev_cu(lens), **kw)
    check_scan(kda, lens, v, out, last)


def test_many_short_sequences(kda):
    """Hundreds of sequences of none to five tokens: several to a run, to a tile, to a chunk's rows."""
    r = np.random.default_rng(0)
    lens = [int(x) for x in r.integers(0, 6, size=300)]
    cu = dev_cu(lens)
    for t, D, n in ((BF, 40, 16), (F32, 7, 3)):
        v = scan_inputs(lens, D, 1, n, t)
        args, kw = call_args(v)
        out, last = kda.kda_selective_scan_fwd(*args, cu, **kw)
        check_scan(kda, lens, v, out, last)
        dout = torch.randn(sum(lens), D, generator=gen(1), device="cuda").to(t)
        dlast = torch.randn(len(lens), D, n, generator=gen(2), device="cuda")
        check_scan_grads(lens, v, dout, dlast, kda.kda_selective_scan_bwd(*args, cu, dout, dfinal_state=dlast, **kw))
        x = conv_inputs(lens, 1, D, 4, t, True, True)
        ckw = dict(bias=x["bias"], initial_state=x["h0"], silu=True)
        y, window = kda.kda_short_conv_fwd(x["x"], x["w"], cu, **ckw)
        dy = torch.randn(y.shape, generator=gen(3), device="cuda").to(t)
        dw = torch.randn(window.shape, generator=gen(4), device="cuda").to(t)
        got = kda.kda_short_conv_bwd(x["x"], x["w"], cu, dy, dfinal_state=dw, **ckw)
        ry, rwin, ys, rg, scale = conv_refs(lens, x, True, False, dy, dw)
        check("y", y, ry, ys, 2.0 ** -20)
        assert np.array_equal(host(window), rwin)
        for k in rg:
            check(k, got[k], rg[k], scale[k], 2.0 ** -19 + (sum(lens) * 2.0 ** -24 if k in ("dw", "dbias") else 0.0))


def test_caller_s_workspaces(kda):
    """Workspaces of the caller's, of exactly the size asked for and holding anything, give the same bits; smaller
    ones are refused."""
    lens, D, n = [600, 200], 40, 16
    v = scan_inputs(lens, D, 1, n, BF)
    args, kw = call_args(v)
    cu = dev_cu(lens)
    dout = torch.randn(800, D, generator=gen(1), device="cuda").to(BF)
    x = conv_inputs(lens, 1, 40, 4, BF, True, True)
    rows = x["x"].view(800, 40)
    w = torch.randn(40, generator=gen(2), device="cuda")
    _, mean, rstd = kda.kda_layer_norm_fwd(rows, w)
    calls = [
        (kda.kda_selective_scan_fwd_workspace_size(800, 2, D, n), lambda **s: kda.kda_selective_scan_fwd(*args, cu, **kw, **s)),
        (kda.kda_selective_scan_bwd_workspace_size(800, 2, D, n), lambda **s: kda.kda_selective_scan_bwd(*args, cu, dout, **kw, **s)),
        (kda.kda_short_conv_bwd_workspace_size(800, 1, 40, 4),
         lambda **s: kda.kda_short_conv_bwd(x["x"], x["w"], cu, x["x"], bias=x["bias"], initial_state=x["h0"], **s)),
        (kda.kda_layer_norm_bwd_workspace_size(800, 40), lambda **s: kda.kda_layer_norm_bwd(rows, w, mean, rstd, rows, **s)),
    ]
    values = lambda r: [t for t in (r.values() if isinstance(r, dict) else r) if t is not None]  # noqa: E731
    for size, call in calls:
        assert size > 0
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN in fp32
        for a, b in zip(values(call()), values(call(workspace=ws))):
            assert torch.equal(a, b)
        with pytest.raises(kda.KDAError) as e:
            call(workspace=ws[:size - 16])
        assert e.value.status == kda.KDA_ERR_INVALID_ARG


def test_scan_forward_state_in_place_uncut(kda):
    lens = [33, 0, 70]
    v = scan_inputs(lens, 64, 1, 16, BF)
    args, kw = call_args(v)
    out, last = kda.kda_selective_scan_fwd(*args, dev_cu(lens), **kw)
    pool = v["h0"].clone()
    out2, _ = kda.kda_selective_scan_fwd(*args, dev_cu(lens), **{**kw, "initial_state": pool}, final_state=pool)
    assert torch.equal(pool, last) and torch.equal(out2, out)


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,G,n", SHAPES)
@pytest.mark.parametrize("N", [1, 13])
def test_scan_step(kda, D, G, n, N, t):
    v = scan_inputs([1] * N, D, G, n, t, gate=n != 5, skip=n != 8, bias=n != 3)
    args, kw = call_args(v)
    state = kw.pop("initial_state").clone()
    out = kda.kda_selective_scan_step(*args, state, **kw)
    check_scan(kda, [1] * N, v, out, state)


def test_scan_prompt_then_steps_equals_prompt(kda):
    """A prompt of 9 tokens, then 4 single tokens, against the 13 tokens at once (three sequences)."""
    N, T, P, D, n = 3, 13, 9, 48, 16
    v = scan_inputs([T] * N, D, 1, n, F32)
    args, kw = call_args(v)
    out, last = kda.kda_selective_scan_fwd(*args, dev_cu([T] * N), **kw)
    check_scan(kda, [T] * N, v, out, last)
    rows = lambda x, a, b: None if x is None else x.view((N, T) + x.shape[1:])[:, a:b].flatten(0, 1).contiguous()  # noqa: E731
    weights = dict(skip=v["skip"], dt_bias=v["dt_bias"])
    o, state = kda.kda_selective_scan_fwd(rows(v["u"], 0, P), rows(v["dt"], 0, P), v["A_log"], rows(v["B"], 0, P),
                                          rows(v["C"], 0, P), dev_cu([P] * N), z=rows(v["z"], 0, P),
                                          initial_state=v["h0"], **weights)
    parts = [o.view(N, P, D)]
    for i in range(P, T):
        parts.append(kda.kda_selective_scan_step(rows(v["u"], i, i + 1), rows(v["dt"], i, i + 1), v["A_log"],
                                                 rows(v["B"], i, i + 1), rows(v["C"], i, i + 1), state,
                                                 z=rows(v["z"], i, i + 1), **weights)[:, None])
    check_scan(kda, [T] * N, v, torch.cat(parts, 1).view(N * T, D), state)


def check_scan_grads(lens, v, dout, dlast, g):
    a, cu = oracle_args(v), cu_of(lens)
    extra = dict(dout=host(dout), dlast=host(dlast))
    ref = S.selective_scan_bwd(cu=cu, **extra, **a)
    sc = S.selective_scan_bwd(cu=cu, scale=True, **extra, **a)
    rel = 2 * scan_rel(lens)
    given = dict(dskip="skip", dz="z", ddt_bias="dt_bias", dinitial_state="h0")
    for k in ref:
        if k in given and v[given[k]] is None:
            assert g[k] is None, k
            continue
        check(k, g[k], ref[k], sc[k], rel + (sum(lens) * 2.0 ** -24 if k in ("dA_log", "dskip", "ddt_bias") else 0.0))


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,G,n", SHAPES)
@pytest.mark.parametrize("lens", LENS + [[130, 0, 7]], ids=["one", "short", "tiles", "chunks"])
def test_scan_backward(kda, D, G, n, lens, t):
    v = scan_inputs(lens, D, G, n, t, seed=1)
    args, kw = call_args(v)
    g = gen(2)
    dout = torch.randn(sum(lens), D, generator=g, device="cuda").to(t)
    dlast = torch.randn(len(lens), D, n, generator=g, device="cuda")
    got = kda.kda_selective_scan_bwd(*args, dev_cu(lens), dout, dfinal_state=dlast, **kw)
    kda.kda_sync_check()
    assert got["du"].dtype == got["dB"].dtype == t and got["dA_log"].dtype == F32
    check_scan_grads(lens, v, dout, dlast, got)


@pytest.mark.parametrize("gate,skip,bias,state", [(False, False, False, False), (True, False, False, True),
                                                  (False, True, False, False), (False, False, True, True)])
def test_scan_backward_optional_arguments(kda, gate, skip, bias, state):
    lens, D, n = [70, 3], 36, 16
    v = scan_inputs(lens, D, 1, n, BF, gate, skip, bias, state)
    args, kw = call_args(v)
    dout = torch.randn(sum(lens), D, generator=gen(5), device="cuda").to(BF)
    got = kda.kda_selective_scan_bwd(*args, dev_cu(lens), dout, **kw)
    check_scan_grads(lens, v, dout, None, got)


def test_scan_decays_at_both_ends(kda):
    """Step sizes near zero (a state that stays), and large ones (decays that underflow to zero)."""
    lens, D, n = [60], 32, 16
    for step in (-12.0, 30.0):
        v = scan_inputs(lens, D, 1, n, F32, step=step)
        args, kw = call_args(v)
        out, last = kda.kda_selective_scan_fwd(*args, dev_cu(lens), **kw)
        check_scan(kda, lens, v, out, last)
        dout = torch.randn(60, D, generator=gen(3), device="cuda")
        dlast = torch.randn(1, D, n, generator=gen(4), device="cuda")
        check_scan_grads(lens, v, dout, dlast, kda.kda_selective_scan_bwd(*args, dev_cu(lens), dout, dfinal_state=dlast, **kw))


def test_scan_decay_past_the_largest_float(kda):
    """A = -exp(A_log) past the largest fp32 value: the state is forgotten at once, also in a tile's last rows, which
    stand for no tokens."""
    lens, D, n = [5, 37], 8, 4
    v = scan_inputs(lens, D, 1, n, F32, state=True)
    v["A_log"][:, 0] = 100.0
    args, kw = call_args(v)
    out, last = kda.kda_selective_scan_fwd(*args, dev_cu(lens), **kw)
    assert torch.isfinite(out).all() and torch.isfinite(last).all()
    check_scan(kda, lens, v, out, last)


def test_no_tokens(kda):
    """Batches of empty sequences, and of none: states pass through, weights' gradients are zero."""
    D, n = 12, 8
    for N in (0, 3):
        v = scan_inputs([0] * N, D, 1, n, BF)
        args, kw = call_args(v)
        cu = dev_cu([0] * N)
        out, last = kda.kda_selective_scan_fwd(*args, cu, **kw)
        assert out.shape == (0, D) and torch.equal(last, v["h0"])
        dlast = torch.randn(N, D, n, generator=gen(1), device="cuda")
        g = kda.kda_selective_scan_bwd(*args, cu, out, dfinal_state=dlast, **kw)
        assert torch.equal(g["dinitial_state"], dlast)
        assert not g["dA_log"].any() and not g["dskip"].any() and not g["ddt_bias"].any()
        x = conv_inputs([0] * N, 1, 12, 4, BF, True, True)
        y, window = kda.kda_short_conv_fwd(x["x"], x["w"], cu, bias=x["bias"], initial_state=x["h0"])
        assert y.shape == (0, 1, 12) and torch.equal(window, x["h0"])
        dw = torch.randn(x["h0"].shape, generator=gen(2), device="cuda").to(BF)
        g = kda.kda_short_conv_bwd(x["x"], x["w"], cu, y, bias=x["bias"], initial_state=x["h0"], dfinal_state=dw)
        assert torch.equal(g["dinitial_state"], dw) and not g["dw"].any() and not g["dbias"].any()
    rows, w = torch.empty(0, 40, device="cuda"), torch.ones(40, device="cuda")
    y, mean, rstd = kda.kda_layer_norm_fwd(rows, w)
    g = kda.kda_layer_norm_bwd(rows, w, mean, rstd, rows)
    assert y.shape == (0, 40) and not g["dw"].any() and not g["dbias"].any()
    step = scan_inputs([], D, 1, n, BF)
    args, kw = call_args(step)
    assert kda.kda_selective_scan_step(*args, kw.pop("initial_state"), **kw).shape == (0, D)
    kda.kda_sync_check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scan_sequences_keep_apart(kda, bad):
    """What one sequence holds reaches no other: not its outputs, its state, nor its rows of the gradients."""
    lens, D, n = [40, 37, 50], 40, 16
    v = scan_inputs(lens, D, 1, n, BF)
    args, kw = call_args(v)
    cu, mid = dev_cu(lens), slice(40, 77)
    dout = torch.randn(127, D, generator=gen(6), device="cuda").to(BF)
    out, last = kda.kda_selective_scan_fwd(*args, cu, **kw)
    g = kda.kda_selective_scan_bwd(*args, cu, dout, **kw)
    w = {k: x.clone() if torch.is_tensor(x) else x for k, x in v.items()}
    for k in ("u", "dt", "B", "C", "z"):
        w[k][mid] = bad
    w["h0"][1] = bad
    args2, kw2 = call_args(w)
    dout2 = dout.clone()
    dout2[mid] = bad
    out2, last2 = kda.kda_selective_scan_fwd(*args2, cu, **kw2)
    g2 = kda.kda_selective_scan_bwd(*args2, cu, dout2, **kw2)
    keep = torch.ones(127, dtype=torch.bool, device="cuda")
    keep[mid] = False
    assert torch.equal(out[keep], out2[keep]) and torch.equal(last[[0, 2]], last2[[0, 2]])
    for k in ("du", "ddt", "dB", "dC", "dz"):
        assert torch.equal(g[k][keep], g2[k][keep]), k
    assert torch.equal(g["dinitial_state"][[0, 2]], g2["dinitial_state"][[0, 2]])


# ---- short convolution ---------------------------------------------------------------------------

CONV_SHAPES = [(2, 64, True), (3, 128, True), (1, 8, False), (1, 7, False), (5, 3, False), (1, 1030, False), (1, 1, False)]
CONV_LENS = [[1], [2, 0, 1, 3, 17, 0], [70, 130, 5]]


def conv_inputs(lens, H, d, W, t, bias, state, seed=0):
    g = gen(seed)
    T, N = sum(lens), len(lens)
    r = lambda *s, dt=F32, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(dt)  # noqa: E731
    return dict(x=r(T, H, d, dt=t), w=r(H, d, W, std=0.6), bias=r(H, d, std=0.3) if bias else None,
                h0=r(N, W - 1, H, d, dt=t) if state else None)


def conv_refs(lens, v, silu, l2norm, dy=None, dlast=None):
    a, cu = oracle_args(v), cu_of(lens)
    y, last = S.short_conv(cu=cu, silu=silu, l2norm=l2norm, **a)
    m = {k: None if x is None else np.abs(x) for k, x in a.items()}
    pabs, _ = S.short_conv(cu=cu, **m)     # sum of |terms| of p
    act, _ = S.short_conv(cu=cu, silu=silu, **a)
    # y = s inv: the norm's relative error is |pabs| inv times that of p
    inv = 1 / np.sqrt((act * act).sum(-1, keepdims=True) + 1e-12) if l2norm else np.ones(y.shape[:2] + (1,))
    worse = 1 + (np.sqrt((pabs * pabs).sum(-1, keepdims=True)) * inv if l2norm else 0.0)
    ys = (pabs * inv + np.abs(y)) * worse
    if dy is None:
        return y, last, ys
    extra = dict(dy=host(dy), dlast=host(dlast), silu=silu, l2norm=l2norm)
    g = S.short_conv_bwd(cu=cu, **extra, **a)
    # an error e of p moves the gradient of p by at most (|silu''| <= 0.5, the norm's terms) e times itself
    extra["dy"] = np.abs(host(dy)) * worse * (1 + pabs)
    if l2norm:   # every term of ds is at most inv (|dy| + |y| |y . dy|)
        extra["dy"] = extra["dy"] + 0 * pabs
    scale = S.short_conv_bwd(cu=cu, scale=True, **extra, **a)
    return y, last, ys, g, scale


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H,d,l2norm", CONV_SHAPES)
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("lens", CONV_LENS, ids=["one", "short", "runs"])
def test_conv(kda, H, d, l2norm, W, lens, t):
    silu, bias, state = (W + d) % 2 == 0, W != 2, W != 3 or d % 2 == 0
    v = conv_inputs(lens, H, d, W, t, bias, state, seed=W)
    cu, kw = dev_cu(lens), dict(bias=v["bias"], initial_state=v["h0"], silu=silu, l2norm=l2norm)
    y, last = kda.kda_short_conv_fwd(v["x"], v["w"], cu, **kw)
    g = gen(9)
    dy = torch.randn(v["x"].shape, generator=g, device="cuda").to(t)
    dlast = torch.randn(last.shape, generator=g, device="cuda").to(t)
    got = kda.kda_short_conv_bwd(v["x"], v["w"], cu, dy, dfinal_state=dlast, **kw)
    kda.kda_sync_check()
    ry, rlast, ys, rg, scale = conv_refs(lens, v, silu, l2norm, dy, dlast)
    check("y", y, ry, ys, 2.0 ** -20)
    assert np.array_equal(host(last), rlast)
    for k in ("dx", "dw", "dbias", "dinitial_state"):
        if (k == "dbias" and not bias) or (k == "dinitial_state" and not state):
            assert got[k] is None
        else:
            check(k, got[k], rg[k], scale[k], 2.0 ** -19 + (sum(lens) * 2.0 ** -24 if k in ("dw", "dbias") else 0.0))


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H,d,l2norm", CONV_SHAPES)
@pytest.mark.parametrize("W", [1, 2, 3, 4])
def test_conv_step(kda, H, d, l2norm, W, t):
    N, silu = 5, W != 3
    v = conv_inputs([1] * N, H, d, W, t, W != 2, True, seed=W)
    state = v["h0"].clone()
    y = kda.kda_short_conv_step(v["x"], v["w"], state, bias=v["bias"], silu=silu, l2norm=l2norm)
    ry, rlast, ys = conv_refs([1] * N, v, silu, l2norm)
    check("y", y, ry, ys, 2.0 ** -20)
    assert np.array_equal(host(state), rlast)


def test_conv_state_in_place_and_steps(kda):
    """Prompts in two calls through one pool of windows, then single tokens, against one call: the same bits."""
    N, T, H, d, W = 3, 90, 2, 64, 4
    v = conv_inputs([T] * N, H, d, W, BF, True, True)
    kw = dict(bias=v["bias"], silu=True, l2norm=True)
    y, last = kda.kda_short_conv_fwd(v["x"], v["w"], dev_cu([T] * N), initial_state=v["h0"], **kw)
    x = v["x"].view(N, T, H, d)
    pool, parts = v["h0"].clone(), []
    for a, b in ((0, 2), (2, 80)):
        o, p = kda.kda_short_conv_fwd(x[:, a:b].flatten(0, 1).contiguous(), v["w"], dev_cu([b - a] * N), initial_state=pool,
                                      final_state=pool, **kw)
        assert p is pool
        parts.append(o.view(N, b - a, H, d))
    for i in range(80, T):
        parts.append(kda.kda_short_conv_step(x[:, i].contiguous(), v["w"], pool, **kw)[:, None])
    assert torch.equal(torch.cat(parts, 1).view(N * T, H, d), y) and torch.equal(pool, last)


def test_conv_agrees_with_the_stateless_form(kda):
    lens, H, d = [40, 0, 33], 3, 128
    v = conv_inputs(lens, H, d, 4, BF, False, False)
    y, _ = kda.kda_short_conv_fwd(v["x"], v["w"], dev_cu(lens), l2norm=True)
    old = kda.kda_short_conv(v["x"], v["w"], dev_cu(lens), l2norm=True)
    ry, _, ys = conv_refs(lens, v, False, True)
    check("with window", y, ry, ys, 2.0 ** -20)
    check("stateless", old, ry, ys, 2.0 ** -20)


# ---- layer norm ----------------------------------------------------------------------------------

COLS = [1, 2, 7, 64, 255, 256, 257, 1000, 1024, 1030, 4096, 4099, 8192, 8200, 16383, 16384]


def norm_scale(x, w, dy):
    x, w, dy = host(x), host(w), host(dy)
    _, mean, rstd = S.layer_norm(x, w)
    xs = (np.abs(x) + np.abs(x).mean(-1, keepdims=True)) * rstd[:, None]
    g = np.abs(dy * w)
    dx = rstd[:, None] * (g + g.mean(-1, keepdims=True) + xs * (g * xs).mean(-1, keepdims=True))
    return dict(y=xs * np.abs(w), mean=np.abs(x).mean(-1), rstd=rstd * (1 + (xs * xs).mean(-1)), dx=dx,
                dw=(np.abs(dy) * xs).sum(0), dbias=np.abs(dy).sum(0))


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", COLS)
@pytest.mark.parametrize("rows", [1, 5, 67])
def test_layer_norm(kda, d, rows, t):
    g = gen(d + rows)
    r = lambda *s, dt=F32: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    x, w, b, dy = r(rows, d, dt=t) + 0.5, r(d), r(d) if d % 2 else None, r(rows, d, dt=t)
    y, mean, rstd = kda.kda_layer_norm_fwd(x, w, b, eps=1e-5)
    got = kda.kda_layer_norm_bwd(x, w, mean, rstd, dy, has_bias=b is not None)
    ry, rmean, rrstd = S.layer_norm(host(x), host(w), host(b))
    rg, sc = S.layer_norm_bwd(host(x), host(w), host(dy)), norm_scale(x, w, dy)
    rel = 128 * 2.0 ** -24
    check("y", y, ry, sc["y"] * (1 + (sc["rstd"] / rrstd)[:, None]) + (0 if b is None else np.abs(host(b))), rel)
    check("mean", mean, rmean, sc["mean"], rel)
    check("rstd", rstd, rrstd, sc["rstd"], rel)
    check("dx", got["dx"], rg["dx"], sc["dx"] * (1 + (sc["rstd"] / rrstd)[:, None]), 2 * rel)
    grow = 1 + float((sc["rstd"] / rrstd).max())
    check("dw", got["dw"], rg["dw"], sc["dw"] * grow, 2 * rel + rows * 2.0 ** -24)
    if b is None:
        assert got["dbias"] is None
    else:
        check("dbias", got["dbias"], rg["dbias"], sc["dbias"], 2 * rel + rows * 2.0 ** -24)


def test_layer_norm_many_rows_and_far_mean(kda):
    """More rows than run at once, with a mean a thousand times the spread."""
    rows, d = 5000, 72
    x = torch.randn(rows, d, generator=gen(1), device="cuda") + 1000.0
    w, dy = torch.randn(d, generator=gen(2), device="cuda"), torch.randn(rows, d, generator=gen(3), device="cuda")
    y, mean, rstd = kda.kda_layer_norm_fwd(x, w)
    got = kda.kda_layer_norm_bwd(x, w, mean, rstd, dy, has_bias=False)
    ry = S.layer_norm(host(x), host(w))[0]
    rg, sc = S.layer_norm_bwd(host(x), host(w), host(dy)), norm_scale(x, w, dy)
    # two passes: the spread is taken about the mean, whose error (a few u |x|) enters it squared
    rel = 128 * 2.0 ** -24
    check("y", y, ry, 2 * sc["y"], rel)
    check("dx", got["dx"], rg["dx"], 2 * sc["dx"], 2 * rel)
    check("dw", got["dw"], rg["dw"], 2 * sc["dw"], 2 * rel + rows * 2.0 ** -24)


def test_layer_norm_rows_keep_apart(kda):
    x = torch.randn(9, 300, generator=gen(1), device="cuda").to(BF)
    w = torch.randn(300, generator=gen(2), device="cuda")
    y, mean, rstd = kda.kda_layer_norm_fwd(x, w)
    x2 = x.clone()
    x2[4, 7], x2[5] = float("inf"), float("nan")
    y2 = kda.kda_layer_norm_fwd(x2, w)[0]
    keep = [0, 1, 2, 3, 6, 7, 8]
    assert torch.equal(y[keep], y2[keep])


def test_tensors_off_the_vector_grid(kda):
    """Rows cut out of larger tensors, aligned to their type only: the same bits as dense copies."""
    lens, D, n = [30, 41], 40, 16
    pad = lambda x: torch.cat([x.flatten()[:1], x.flatten()])[1:].view(x.shape)  # noqa: E731  (one element past alignment)
    v = scan_inputs(lens, D, 1, n, BF)
    w = {k: pad(x) for k, x in v.items()}
    assert w["u"].data_ptr() % 16 == 2 and torch.equal(w["u"], v["u"])
    cu = dev_cu(lens)
    (a, kw), (b, kx) = call_args(v), call_args(w)
    dout = torch.randn(71, D, generator=gen(1), device="cuda").to(BF)
    x = conv_inputs(lens, 1, 40, 4, BF, True, True)
    xp = {k: pad(t) for k, t in x.items()}
    ck = lambda c: dict(bias=c["bias"], initial_state=c["h0"], silu=True)  # noqa: E731
    gain = torch.randn(40, generator=gen(2), device="cuda")
    rows, rows_p = x["x"].view(71, 40), xp["x"].view(71, 40)
    _, mean, rstd = kda.kda_layer_norm_fwd(rows, gain)
    st, sp = v["h0"].clone(), pad(v["h0"])
    sk, sx = {**kw}, {**kx}
    sk.pop("initial_state"), sx.pop("initial_state")
    two = lambda c, k: tuple(t[:2].contiguous() if t is not c[2] else t for t in c)  # noqa: E731
    for got, want in (
            (kda.kda_selective_scan_fwd(*b, cu, **kx), kda.kda_selective_scan_fwd(*a, cu, **kw)),
            (kda.kda_selective_scan_bwd(*b, cu, pad(dout), **kx).values(), kda.kda_selective_scan_bwd(*a, cu, dout, **kw).values()),
            (kda.kda_short_conv_fwd(xp["x"], xp["w"], cu, **ck(xp)), kda.kda_short_conv_fwd(x["x"], x["w"], cu, **ck(x))),
            (kda.kda_short_conv_bwd(xp["x"], xp["w"], cu, pad(x["x"]), **ck(xp)).values(),
             kda.kda_short_conv_bwd(x["x"], x["w"], cu, x["x"], **ck(x)).values()),
            ((kda.kda_selective_scan_step(*two(b, 0), sp, skip=kx["skip"], dt_bias=kx["dt_bias"]), sp),
             (kda.kda_selective_scan_step(*two(a, 0), st, skip=kw["skip"], dt_bias=kw["dt_bias"]), st))):
        for g, r in zip(got, want):
            assert torch.equal(g, r)
    # the norm's columns lie on other threads then: sums in another order
    y, ym = kda.kda_layer_norm_fwd(rows_p, pad(gain)), kda.kda_layer_norm_fwd(rows, gain)
    check("y", y[0], host(ym[0]), np.abs(host(ym[0])) + 1, 128 * 2.0 ** -24)
    gp = kda.kda_layer_norm_bwd(rows_p, pad(gain), mean, rstd, pad(dout), has_bias=True)
    gr = kda.kda_layer_norm_bwd(rows, gain, mean, rstd, dout, has_bias=True)
    for k in gr:
        assert (gp[k].float() - gr[k].float()).norm() <= 2.0 ** -7 * gr[k].float().norm(), k


# ---- all of them: determinism, streams, graphs, large offsets, errors ------------------------------


def _all_calls(kda, seed=0):
    """Every entry point once, on the current stream; returns the closures and their outputs' flattener."""
    lens = [300, 0, 90]
    v = scan_inputs(lens, 40, 1, 16, BF, seed=seed)
    args, kw = call_args(v)
    cu = dev_cu(lens)
    dout = torch.randn(390, 40, generator=gen(seed + 1), device="cuda").to(BF)
    c = conv_inputs(lens, 2, 64, 4, BF, True, True, seed=seed)
    ckw = dict(bias=c["bias"], initial_state=c["h0"], silu=True, l2norm=True)
    cdy = torch.randn(c["x"].shape, generator=gen(seed + 2), device="cuda").to(BF)
    w = torch.randn(128, generator=gen(seed + 3), device="cuda")
    step = scan_inputs([1] * 6, 40, 1, 16, BF, seed=seed + 4)
    sargs, skw = call_args(step)
    sstate = skw.pop("initial_state")

    def run(stream=None):
        s = dict(stream=stream)
        state, window = sstate.clone(), c["h0"].clone()
        n, mean, rstd = kda.kda_layer_norm_fwd(c["x"].view(390, 128), w, w, **s)
        outs = [n, mean, rstd, *kda.kda_selective_scan_fwd(*args, cu, **kw, **s),
                *kda.kda_selective_scan_bwd(*args, cu, dout, **kw, **s).values(),
                *kda.kda_short_conv_fwd(c["x"], c["w"], cu, **ckw, **s),
                *kda.kda_short_conv_bwd(c["x"], c["w"], cu, cdy, **ckw, **s).values(),
                *kda.kda_layer_norm_bwd(c["x"].view(390, 128), w, mean, rstd, cdy.view(390, 128), **s).values(),
                kda.kda_selective_scan_step(*sargs, state, **skw, **s), state,
                kda.kda_short_conv_step(c["x"][:3].contiguous(), c["w"], window, bias=c["bias"], silu=True, **s), window]
        return outs

    return run


def test_same_bits_every_time_and_on_another_stream(kda):
    run = _all_calls(kda)
    first = run()
    torch.cuda.synchronize()
    for a, b in zip(first, run()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run()
    side.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    # named by argument: the call's own allocations belong to that stream
    lens = [300, 0, 90]
    v = scan_inputs(lens, 40, 1, 16, BF)
    args, kw = call_args(v)
    cu = dev_cu(lens)
    ref = kda.kda_selective_scan_fwd(*args, cu, **kw)
    torch.cuda.synchronize()
    got = kda.kda_selective_scan_fwd(*args, cu, stream=side, **kw)
    side.synchronize()
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])


def test_captured_and_replayed(kda):
    """Two graphs of all calls, replayed in turn: each has its own workspaces."""
    run = [_all_calls(kda, seed) for seed in (0, 7)]
    want = [r() for r in run]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r in run:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(r())
        graphs.append(g)
    for o in outs:
        for x in o:
            x.zero_()
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        for a, b in zip(w, o):
            assert torch.equal(a, b)


def test_offsets_past_32_bits(kda):
    """Tensors of more than 2^31 elements: the last sequence's rows against a call on those rows alone."""
    D, lens = 32768, [65500, 70]
    T = sum(lens)
    cu, tail = dev_cu(lens), slice(lens[0], T)
    x = torch.randn(1024, D, generator=gen(0), device="cuda").to(BF).repeat(65, 1)[:T].contiguous()
    assert x.numel() > 1 << 31
    A_log = torch.zeros(D, 1, device="cuda")
    B = torch.randn(T, 1, 1, generator=gen(1), device="cuda").to(BF)
    args = lambda r, c: (x[r], x[r], A_log, B[r], B[r], c)  # noqa: E731
    alone = slice(lens[0], T)
    one = dev_cu([70])
    out, last = kda.kda_selective_scan_fwd(*args(slice(0, T), cu), z=x)
    ref, ref_last = kda.kda_selective_scan_fwd(*(a.contiguous() for a in args(alone, one)), z=x[alone].contiguous())
    assert torch.equal(out[tail], ref) and torch.equal(last[1], ref_last[0])
    del out
    g = kda.kda_selective_scan_bwd(*args(slice(0, T), cu), x)
    r = kda.kda_selective_scan_bwd(*(a.contiguous() for a in args(alone, one)), x[alone].contiguous())
    for k in ("du", "ddt", "dB", "dC"):
        assert torch.equal(g[k][tail], r[k]), k
    del g, r
    w = torch.randn(1, D, 4, generator=gen(2), device="cuda")
    x3 = x.view(T, 1, D)
    y, _ = kda.kda_short_conv_fwd(x3, w, cu, silu=True)
    ry, _ = kda.kda_short_conv_fwd(x3[alone].contiguous(), w, one, silu=True)
    assert torch.equal(y[tail], ry)
    g = kda.kda_short_conv_bwd(x3, w, cu, x3, silu=True)
    r = kda.kda_short_conv_bwd(x3[alone].contiguous(), w, one, x3[alone].contiguous(), silu=True)
    assert torch.equal(g["dx"][tail], r["dx"])
    del g, r, y
    flat = x.view(-1, 8192)
    w = torch.randn(8192, generator=gen(3), device="cuda")
    y, mean, rstd = kda.kda_layer_norm_fwd(flat, w)
    end = flat[-50:].contiguous()
    ry, rmean, rrstd = kda.kda_layer_norm_fwd(end, w)
    assert torch.equal(y[-50:], ry) and torch.equal(rstd[-50:], rrstd)
    g = kda.kda_layer_norm_bwd(flat, w, mean, rstd, flat)
    r = kda.kda_layer_norm_bwd(end, w, rmean, rrstd, end)
    assert torch.equal(g["dx"][-50:], r["dx"])


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [0, 40, 90, 99], [1, 40, 90, 100], [0, 40, 200, 100], [0, -5, 90, 100]])
def test_malformed_cu_seqlens_are_reported(kda, cu):
    """Reported by kda_sync_check; the kernels clamp what they read, so nothing is touched outside the tensors."""
    v = scan_inputs([100, 0, 0], 40, 1, 16, BF)
    args, kw = call_args(v)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    x = conv_inputs([100, 0, 0], 1, 40, 4, BF, True, True)
    calls = [lambda: kda.kda_selective_scan_fwd(*args, c, **kw),
             lambda: kda.kda_selective_scan_bwd(*args, c, v["u"], **kw),
             lambda: kda.kda_short_conv_fwd(x["x"], x["w"], c, initial_state=x["h0"]),
             lambda: kda.kda_short_conv_bwd(x["x"], x["w"], c, x["x"], initial_state=x["h0"])]
    for call in calls:
        call()
        with pytest.raises(kda.KDAError) as e:
            kda.kda_sync_check()
        assert e.value.status == kda.KDA_ERR_INVALID_ARG
    kda.kda_sync_check()


# ---- a layer made of them --------------------------------------------------------------------------


def _layer(ops, p, x, cu, window=None, state=None):
    """norm -> projections -> convolution -> scan with gate -> projection, added to x."""
    D, n = p["A_log"].shape
    h = ops["norm"](x, p["nw"], p["nb"])
    uz = h @ p["w_in"]
    u, window = ops["conv"](uz[:, :D].reshape(-1, 1, D).contiguous(), p["cw"], cu, p["cb"], window)
    u = u.view(-1, D)
    dbc = u @ p["w_dbc"]
    B, C = (dbc[:, D + i * n:D + (i + 1) * n].reshape(-1, 1, n).contiguous() for i in range(2))
    o, state = ops["scan"](u, dbc[:, :D].contiguous(), p["A_log"], B, C, cu, p["skip"], uz[:, D:].contiguous(), p["dt_bias"], state)
    return x + o @ p["w_out"], window, state


def _plain_ops():
    """The same operators in elementary torch operations of whatever type they are given, token by token."""
    def norm(x, w, b):
        c = x - x.mean(-1, keepdim=True)
        return c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * w + b

    def conv(x, w, cu, bias, window):
        outs, lasts, cu, W = [], [], cu.tolist(), w.shape[-1]
        for s in range(len(cu) - 1):
            old = x.new_zeros(W - 1, *x.shape[1:]) if window is None else window[s]
            rows = torch.cat([old, x[cu[s]:cu[s + 1]]])
            m = cu[s + 1] - cu[s]
            p = sum(w[..., j] * rows[j:j + m] for j in range(W)) + bias
            outs.append(p * torch.sigmoid(p))
            lasts.append(rows[m:])
        return torch.cat(outs), torch.stack(lasts)

    def scan(u, dt, A_log, B, C, cu, skip, z, dt_bias, state):
        cu, outs, lasts = cu.tolist(), [], []
        delta = torch.logaddexp(dt + dt_bias, torch.zeros_like(dt))
        for s in range(len(cu) - 1):
            h = u.new_zeros(A_log.shape) if state is None else state[s]
            for t in range(cu[s], cu[s + 1]):
                h = torch.exp(-torch.exp(A_log) * delta[t, :, None]) * h + (delta[t] * u[t])[:, None] * B[t]
                outs.append(((h * C[t]).sum(-1) + skip * u[t]) * z[t] * torch.sigmoid(z[t]))
            lasts.append(h)
        return torch.stack(outs), torch.stack(lasts)

    return dict(norm=norm, conv=conv, scan=scan)


def _own_ops(kda):
    return dict(norm=lambda x, w, b: kda.layer_norm(x, w, b),
                conv=lambda x, w, cu, b, s: kda.short_conv(x, w, cu, bias=b, initial_state=s, silu=True),
                scan=lambda u, dt, A, B, C, cu, skip, z, bias, h: kda.selective_scan(u, dt, A, B, C, cu, skip=skip, z=z,
                                                                                     dt_bias=bias, initial_state=h))


def _layer_params(M, D, n, seed=0):
    g = gen(seed)
    r = lambda *s, std=1.0: torch.randn(s, generator=g, device="cuda") * std  # noqa: E731
    return dict(nw=1 + r(M, std=0.1), nb=r(M, std=0.1), w_in=r(M, 2 * D, std=M ** -0.5), cw=r(1, D, 4, std=0.5), cb=r(1, D, std=0.1),
                w_dbc=r(D, D + 2 * n, std=D ** -0.5), A_log=r(D, n, std=0.3), skip=r(D), dt_bias=r(D) - 1,
                w_out=r(D, M, std=D ** -0.5))


def test_layer_in_training(kda):
    """Outputs and every gradient of a layer, fp32 kernels against automatic differentiation in 64 bits.

    Two norms: the layer is a composition of Lipschitz maps of order one on O(1) values, so the fp32 errors of
    its parts (at most 2^-20 a token of memory, 40 tokens, see above) and of its three fp32 products (TF32 is off)
    add to less than 2^-13 of the output's norm."""
    assert not torch.backends.cuda.matmul.allow_tf32
    lens, M, D, n = [40, 0, 23], 24, 36, 16
    cu = dev_cu(lens)
    p = _layer_params(M, D, n)
    x = torch.randn(sum(lens), M, generator=gen(3), device="cuda")
    dy = torch.randn(sum(lens), M, generator=gen(4), device="cuda")
    window = torch.randn(3, 3, 1, D, generator=gen(5), device="cuda")
    state = torch.randn(3, D, n, generator=gen(6), device="cuda")
    results = []
    for ops, t in ((_own_ops(kda), torch.float32), (_plain_ops(), torch.float64)):
        leaves = {k: v.to(t).requires_grad_() for k, v in dict(p, x=x, window=window, state=state).items()}
        q = {k: leaves[k] for k in p}
        out, w, s = _layer(ops, q, leaves["x"], cu, leaves["window"], leaves["state"])
        loss = (out * dy.to(t)).sum() + s.sum() + 0.5 * w.sum()
        grads = torch.autograd.grad(loss, list(leaves.values()))
        results.append(dict(zip(leaves, grads), out=out, last_window=w, last_state=s))
    for k, ref in results[1].items():
        got = results[0][k]
        assert got.dtype == torch.float32
        err = (got.double() - ref).norm() / ref.norm()
        assert err <= 2.0 ** -13, (k, float(err))


def test_layer_gradient_against_differences(kda):
    """The directional derivative of the kernels' own fp32 layer against central differences of its outputs:
    a step of 2^-7 leaves third derivatives of order one times 2^-14 / 6, rounding 2^-20 / 2^-7 of the loss's terms."""
    lens, M, D, n = [17, 5], 8, 12, 8
    cu, p = dev_cu(lens), _layer_params(M, D, n, seed=1)
    x = torch.randn(22, M, generator=gen(3), device="cuda")
    dy = torch.randn(22, M, generator=gen(4), device="cuda")
    ops, step = _own_ops(kda), 2.0 ** -7
    for k in ("A_log", "dt_bias", "skip", "cw", "cb", "nw", "nb"):
        way = torch.randn(p[k].shape, generator=gen(8), device="cuda")
        way /= way.norm()
        leaf = p[k].clone().requires_grad_()
        out = _layer(ops, dict(p, **{k: leaf}), x, cu)[0]
        (g,) = torch.autograd.grad((out * dy).sum(), [leaf])
        with torch.no_grad():
            f = [float((_layer(ops, dict(p, **{k: p[k] + s * way}), x, cu)[0].double() * dy).sum()) for s in (step, -step)]
            size = float((out.double() * dy).abs().sum())
        want, got = (f[0] - f[1]) / (2 * step), float((g.double() * way).sum())
        assert abs(want - got) <= size * (2.0 ** -14 + 2.0 ** -13), (k, want, got, size)


def test_layer_in_serving(kda):
    """A prompt in two calls and then single tokens, through pools of windows and states, against the whole
    sequence at once in 64 bits; bf16 activations (each of the six stored values is off by half a step; two norms)."""
    M, D, n, T, P = 24, 40, 16, 20, 15
    p = _layer_params(M, D, n, seed=2)
    N = 2
    x = torch.randn(N, T, M, generator=gen(3), device="cuda").to(BF)
    q = {k: (v if k in ("nw", "nb", "cw", "cb", "A_log", "skip", "dt_bias") else v.to(BF)) for k, v in p.items()}
    ref = _layer(_plain_ops(), {k: v.double() for k, v in q.items()}, x.double().flatten(0, 1), dev_cu([T] * N))
    windows = torch.zeros(N, 3, 1, D, dtype=BF, device="cuda")
    states = torch.zeros(N, D, n, device="cuda")

    def prompt_ops():
        return dict(norm=lambda x, w, b: kda.kda_layer_norm_fwd(x, w, b)[0],
                    conv=lambda x, w, cu, b, s: kda.kda_short_conv_fwd(x, w, cu, bias=b, initial_state=s, final_state=s, silu=True),
                    scan=lambda u, dt, A, B, C, cu, skip, z, bias, h: kda.kda_selective_scan_fwd(
                        u, dt, A, B, C, cu, skip=skip, z=z, dt_bias=bias, initial_state=h, final_state=h))

    def step_ops():
        return dict(norm=lambda x, w, b: kda.kda_layer_norm_fwd(x, w, b)[0],
                    conv=lambda x, w, cu, b, s: (kda.kda_short_conv_step(x, w, s, bias=b, silu=True), s),
                    scan=lambda u, dt, A, B, C, cu, skip, z, bias, h: (kda.kda_selective_scan_step(
                        u, dt, A, B, C, h, skip=skip, z=z, dt_bias=bias), h))

    parts = []
    for a, b in ((0, 6), (6, P)):
        o = _layer(prompt_ops(), q, x[:, a:b].flatten(0, 1).contiguous(), dev_cu([b - a] * N), windows, states)[0]
        parts.append(o.view(N, b - a, M))
    for i in range(P, T):
        parts.append(_layer(step_ops(), q, x[:, i].contiguous(), None, windows, states)[0].view(N, 1, M))
    out = torch.cat(parts, 1).flatten(0, 1)
    for got, want in ((out, ref[0]), (windows, ref[1]), (states, ref[2])):
        err = (got.double() - want).norm() / want.norm()
        # six stored values on the way, each 2^-8 at most, through maps that stretch by less than four
        assert err <= 6 * 4 * 2.0 ** -8, float(err)


def test_autograd_of_one_output_only(kda):
    """A loss on the outputs alone, and on the final state alone."""
    lens, D, n = [20, 9], 16, 8
    v = scan_inputs(lens, D, 1, n, F32)
    cu = dev_cu(lens)
    for which in (0, 1):
        u = v["u"].clone().requires_grad_()
        res = kda.selective_scan(u, v["dt"], v["A_log"], v["B"], v["C"], cu, skip=v["skip"], z=v["z"], initial_state=v["h0"])
        (g,) = torch.autograd.grad(res[which].sum(), [u])
        dout = torch.ones(29, D, device="cuda") if which == 0 else torch.zeros(29, D, device="cuda")
        want = kda.kda_selective_scan_bwd(v["u"], v["dt"], v["A_log"], v["B"], v["C"], cu, dout, skip=v["skip"], z=v["z"],
                                          initial_state=v["h0"], dfinal_state=torch.ones(2, D, n, device="cuda") if which else None)
        assert torch.equal(g, want["du"])


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 4), (F32, 128), (F32, 2), (BF, 512), (F32, 512)])
def test_norm_gradients_of_large_constant_rows(kda, dtype, d):
    """Rows of one value of 2^110 (whose mean is exact) have xhat = 0, however large mean rstd is: what lies past the
    row's end adds nothing.  With w = 1 and dy = +-1 in turn every sum is exact and dx is rstd dy rounded once."""
    x = torch.full((5, d), 2.0 ** 110, device="cuda", dtype=dtype)
    w = torch.ones(d, device="cuda")
    dy = torch.ones(5, d, device="cuda", dtype=dtype)
    dy[:, 1::2] = -1
    y, mean, rstd = kda.kda_layer_norm_fwd(x, w, eps=1e-12)
    assert torch.equal(mean, torch.full_like(mean, 2.0 ** 110)) and not y.any()
    assert float(mean[0]) * float(rstd[0]) > torch.finfo(F32).max
    g = kda.kda_layer_norm_bwd(x, w, mean, rstd, dy)
    assert torch.equal(g["dx"], (rstd[:, None] * dy.float()).to(dtype))
    assert not g["dw"].any() and torch.equal(g["dbias"], dy.float().sum(0))


def test_training_step_captured_and_replayed(kda):
    """Forward and backward of the three operators in one graph, replayed on other inputs: the eager pass's bits."""
    lens, D, n = [40, 0, 23], 36, 16
    cu, T = dev_cu(lens), sum(lens)
    p = _layer_params(D, D, n, seed=9)
    names = ("nw", "nb", "cw", "cb", "A_log", "skip", "dt_bias")
    data = [torch.randn(T, D, generator=gen(s), device="cuda") for s in (11, 12)]
    B, C, dy = (torch.randn(T, *s, generator=gen(13 + i), device="cuda") for i, s in enumerate(((1, n), (1, n), (D,))))

    def fresh():
        return {k: p[k].clone().requires_grad_() for k in names}

    def step(q, x):
        for v in q.values():
            v.grad = None
        h = kda.layer_norm(x, q["nw"], q["nb"])
        u, _ = kda.short_conv(h.view(T, 1, D), q["cw"], cu, bias=q["cb"], silu=True)
        o, last = kda.selective_scan(u.view(T, D), h, q["A_log"], B, C, cu, skip=q["skip"], z=h, dt_bias=q["dt_bias"])
        loss = (o * dy).sum() + last.sum()
        loss.backward()
        return [loss.detach(), *(v.grad for v in q.values())]

    want = [[t.clone() for t in step(fresh(), x)] for x in data]
    q, x = fresh(), data[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(q, x)
    torch.cuda.current_stream().wait_stream(side)
    for v in q.values():
        v.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(q, x)
    for i in (1, 0, 1):
        x.copy_(data[i])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b)


# ---- convolution with unit rows on tensors off the vector grid -------------------------------------


def off_grid(x):
    """The same values one element past the 16-byte grid."""
    return torch.cat([x.flatten()[:1], x.flatten()])[1:].view(x.shape) if x.numel() else x


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H,d", [(1, 64), (3, 64), (1, 128), (3, 128), (20, 64)])
@pytest.mark.parametrize("W", [1, 3, 4])
def test_conv_unit_rows_off_the_vector_grid(kda, H, d, W, t):
    """One tensor at a time (the carried state alone among them), then all: prompts, single tokens and gradients."""
    lens, silu, bias = [70, 0, 130, 5], W != 3, W != 1
    v = conv_inputs(lens, H, d, W, t, bias, True, seed=W)
    dy = torch.randn(v["x"].shape, generator=gen(9), device="cuda").to(t)
    dlast = torch.randn(v["h0"].shape, generator=gen(10), device="cuda").to(t)
    ry, rlast, ys, rg, scale = conv_refs(lens, v, silu, True, dy, dlast)
    one = conv_inputs([1] * 5, H, d, W, t, bias, True, seed=W + 1)
    oy, olast, oys = conv_refs([1] * 5, one, silu, True)
    cu = dev_cu(lens)
    for moved in (("x",), ("out",), ("initial_state",), ("final_state",), ("dy",), ("dfinal_state",),
                  ("x", "out", "initial_state", "final_state", "dy", "dfinal_state")):
        at = lambda name, x: off_grid(x) if name in moved else x  # noqa: E731
        y, last = kda.kda_short_conv_fwd(at("x", v["x"]), v["w"], cu, bias=v["bias"], initial_state=at("initial_state", v["h0"]),
                                         silu=silu, l2norm=True, out=at("out", torch.zeros_like(v["x"])),
                                         final_state=at("final_state", torch.zeros_like(v["h0"])))
        check(f"{moved} y", y, ry, ys, 2.0 ** -20)
        assert np.array_equal(host(last), rlast), moved
        state = at("initial_state", one["h0"].clone())
        y = kda.kda_short_conv_step(at("x", one["x"]), one["w"], state, bias=one["bias"], silu=silu, l2norm=True,
                                    out=at("out", torch.zeros_like(one["x"])))
        check(f"{moved} step", y, oy, oys, 2.0 ** -20)
        assert np.array_equal(host(state), olast), moved
        g = kda.kda_short_conv_bwd(at("x", v["x"]), v["w"], cu, at("dy", dy), bias=v["bias"],
                                   initial_state=at("initial_state", v["h0"]), dfinal_state=at("dfinal_state", dlast), silu=silu,
                                   l2norm=True)
        for k in ("dx", "dw", "dinitial_state") + (("dbias",) if bias else ()):
            check(f"{moved} {k}", g[k], rg[k], scale[k], 2.0 ** -19 + (sum(lens) * 2.0 ** -24 if k in ("dw", "dbias") else 0.0))
    kda.kda_sync_check()


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,n", [(8, 4), (40, 8), (40, 16), (20, 32), (9, 64)])
def test_scan_backward_past_the_largest_float(kda, D, n, t):
    """Decays past the largest fp32 value backwards: a state that is forgotten at once has no gradient, and neither
    that of A_log nor the rows that fill up a chunk's last tokens (whose decay is one) turn it into NaN."""
    lens = [5, 37, 0, 64, 3]
    v = scan_inputs(lens, D, 1, n, t, state=True)
    v["A_log"][:, 0] = 100.0
    v["A_log"][:3] = 88.8
    args, kw = call_args(v)
    dout = torch.randn(sum(lens), D, generator=gen(3), device="cuda").to(t)
    dlast = 4 * torch.randn(len(lens), D, n, generator=gen(4), device="cuda")
    g = kda.kda_selective_scan_bwd(*args, dev_cu(lens), dout, dfinal_state=dlast, **kw)
    for k, x in g.items():
        assert torch.isfinite(x).all(), k
    assert not g["dA_log"][:, 0].any() and not g["dA_log"][:3].any()
    check_scan_grads(lens, v, dout, dlast, g)


@pytest.mark.parametrize("n", [4, 11, 16, 64])
@pytest.mark.parametrize("T", [5, 33, 70])
def test_scan_backward_infinite_last_input(kda, T, n):
    """The gradient of A_log and of the initial state does not depend on the last token's input, also where that is
    infinite and rows that stand for no token follow it."""
    v = scan_inputs([T], 12, 1, n, F32)
    dout = torch.randn(T, 12, generator=gen(3), device="cuda")
    dlast = torch.randn(1, 12, n, generator=gen(4), device="cuda")
    got = []
    for last in (1.0, float("inf")):
        v["u"][-1] = last
        args, kw = call_args(v)
        got.append(kda.kda_selective_scan_bwd(*args, dev_cu([T]), dout, dfinal_state=dlast, **kw))
    for k in ("dA_log", "dinitial_state"):
        assert torch.isfinite(got[0][k]).all() and torch.equal(got[0][k], got[1][k]), k


def test_scan_without_skip_keeps_infinities(kda):
    """No skip means no term: an infinite input or gradient is not multiplied by zero.  All terms are positive, so the
    formulas give plus infinity from the infinite token on (outputs, states) or up to it (gradients)."""
    T, D, n, at, up = 6, 8, 4, 3, float("inf")
    one = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    u, dt, A_log, BC = one(T, D), one(T, D), torch.zeros(D, n, device="cuda"), one(T, 1, n)
    u[at] = up
    out, last = kda.kda_selective_scan_fwd(u, dt, A_log, BC, BC, dev_cu([T]))
    assert torch.isfinite(out[:at]).all() and (out[at:] == up).all() and (last == up).all()
    state, rows = torch.zeros(1, D, n, device="cuda"), []
    for i in range(T):
        rows.append(kda.kda_selective_scan_step(u[i:i + 1], dt[i:i + 1], A_log, BC[i:i + 1], BC[i:i + 1], state))
    rows = torch.cat(rows)
    assert torch.isfinite(rows[:at]).all() and (rows[at:] == up).all() and (state == up).all()
    dout = one(T, D)
    dout[at] = up
    g = kda.kda_selective_scan_bwd(one(T, D), dt, A_log, BC, BC, dev_cu([T]), dout)
    assert (g["du"][:at + 1] == up).all() and torch.isfinite(g["du"][at + 1:]).all()
    # the output enters the gate's gradient: dz = dout y silu'(z)
    g = kda.kda_selective_scan_bwd(u, dt, A_log, BC, BC, dev_cu([T]), one(T, D), z=one(T, D))
    assert torch.isfinite(g["dz"][:at]).all() and (g["dz"][at:] == up).all()


# ---- launch rules --------------------------------------------------------------------------------


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,n", [(8192, 4), (4096, 8), (4096, 16), (2048, 32), (1024, 64), (128, 64)])
def test_scan_forward_where_blocks_could_share_an_sm(kda, D, n, t):
    """More blocks than twice the SMs hold one each, in both types and for every number of lanes: in bf16 two share an
    SM, in fp32 one has it alone.  (The last case: few blocks, where fp32 has half the staging threads too.)"""
    lens = [90, 150, 0, 33, 70, 1]
    v = scan_inputs(lens, D, 1, n, t)
    args, kw = call_args(v)
    out, last = kda.kda_selective_scan_fwd(*args, dev_cu(lens), **kw)
    check_scan(kda, lens, v, out, last)


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
def test_scan_one_long_sequence_among_short_ones(kda, t):
    """The channels of nine sequences nearly fill the GPU, so that nothing is cut, but one sequence has most of the tokens."""
    lens, D, n = [24, 24, 24, 1500, 0, 24, 24, 24, 24], 512, 16
    assert kda.kda_selective_scan_fwd_workspace_size(sum(lens), len(lens), D, n) == 0
    v = scan_inputs(lens, D, 1, n, t)
    args, kw = call_args(v)
    cu = dev_cu(lens)
    out, last = kda.kda_selective_scan_fwd(*args, cu, **kw)
    check_scan(kda, lens, v, out, last)
    dout = torch.randn(sum(lens), D, generator=gen(3), device="cuda").to(t)
    dlast = torch.randn(len(lens), D, n, generator=gen(4), device="cuda")
    check_scan_grads(lens, v, dout, dlast, kda.kda_selective_scan_bwd(*args, cu, dout, dfinal_state=dlast, **kw))


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,n", [(9, 33), (24, 64)])
def test_scan_forward_cut_past_32_states(kda, D, n, t):
    """Both passes over segments, which stage with different numbers of threads in fp32; the final states in place."""
    lens = [700, 0, 1, 300]
    assert kda.kda_selective_scan_fwd_workspace_size(sum(lens), len(lens), D, n) > 0
    v = scan_inputs(lens, D, 1, n, t)
    args, kw = call_args(v)
    pool = v["h0"].clone()
    out, last = kda.kda_selective_scan_fwd(*args, dev_cu(lens), **{**kw, "initial_state": pool}, final_state=pool)
    assert last is pool
    check_scan(kda, lens, v, out, last)
