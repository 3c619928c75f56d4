"""The operators of a state-space mixer layer, as cases to measure: the selective scan over packed
prompts, its training step and its single-token step; the short causal convolution with its carried
window, in training and for single tokens; layer norm with its backward pass.

``run(state)`` computes one pass, in elementary torch operations or, where ``own`` is true, through
the kernels of kda_chunkwise_b200.  ``exact`` gives the same values in 64 bits, token by token.

Formulas (one sequence; d a channel, m a state index, g(d) = d // (D / G) its group):
  scan   delta = softplus(dt + dt_bias),  A = -exp(A_log)
         h_t[d, m] = exp(delta_t[d] A[d, m]) h_{t-1}[d, m] + delta_t[d] u_t[d] B_t[g(d), m]
         out_t[d] = silu(z_t[d]) (sum_m C_t[g(d), m] h_t[d, m] + skip[d] u_t[d])
  conv   p_t[c] = bias[c] + sum_{j < W} w[c, j] x_{t-(W-1)+j}[c],  s = silu(p),
         y = s, or s / sqrt(|s|^2 + 1e-12) over each head's channels;
         the carried state is the last W - 1 inputs
  norm   y = (x - mean) rstd w + b over the last dimension, rstd = 1 / sqrt(var + eps)
"""
import math
import random

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # one long prompt, one layer: the framework's prefill size (8192 tokens, 32 x 128 channels)
        dict(name="prompt_8192", kind="prompt", dtype="bf16", T=8192, seqs=1, D=4096, n=16, G=1, gate=True, state=False),
        # a serving batch of prompts of ragged lengths, continuing from cached states
        dict(name="prompt_packed", kind="prompt", dtype="bf16", T=5003, seqs=9, D=2048, n=16, G=2, gate=True, state=True),
        # one user's next token: the latency of the call
        dict(name="step_one", kind="step", dtype="bf16", N=1, D=4096, n=16, G=1, gate=True),
        # a full decode batch: the state streams through once
        dict(name="step_batch", kind="step", dtype="bf16", N=256, D=4096, n=16, G=1, gate=True),
        # a small training batch of ragged documents in fp32, a channel count that no vector divides
        dict(name="train_packed", kind="train", dtype="f32", T=2051, seqs=5, D=1030, n=16, G=1, gate=True, state=True),
        # one training sequence of the framework's prefill size
        dict(name="train_8192", kind="train", dtype="bf16", T=8192, seqs=1, D=4096, n=16, G=1, gate=True, state=False),
        # q or k of a KDA layer in training: convolution, SiLU, unit rows per head
        dict(name="conv_train_8192", kind="conv_train", dtype="bf16", T=8192, seqs=4, H=32, d=128, W=4, l2norm=True, bias=False, state=False),
        # ragged documents in fp32, odd channel count, carried windows
        dict(name="conv_train_packed", kind="conv_train", dtype="f32", T=1999, seqs=6, H=1, d=1030, W=3, l2norm=False, bias=True, state=True),
        # one user's next token
        dict(name="conv_step_one", kind="conv_step", dtype="bf16", N=1, H=32, d=128, W=4, l2norm=False, bias=True),
        # a full decode batch of k rows
        dict(name="conv_step_batch", kind="conv_step", dtype="bf16", N=256, H=32, d=128, W=4, l2norm=True, bias=False),
        # the norm before a layer, forward and backward, over the tokens of one training sequence
        dict(name="norm_8192", kind="norm", dtype="bf16", rows=8192, d=4096, bias=True),
        # a few rows of an odd width in fp32
        dict(name="norm_odd", kind="norm", dtype="f32", rows=67, d=1003, bias=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prompt", "step", "train", "conv_train", "conv_step", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    groups = rng.choice([1, 1, 2, 4])
    n = rng.choice([4, 8, 11, 16, 16, 16, 32, 64])
    if kind in ("prompt", "train"):
        T = _log_uniform(rng, 1, 16384)
        most = min(8192, (1 << 28 if dtype == "f32" else 1 << 29) // (T * n))
        D = groups * max(1, _log_uniform(rng, 16, max(17, most)) // groups)
        return dict(kind=kind, dtype=dtype, T=T, seqs=_log_uniform(rng, 1, 40), D=D, n=n, G=groups,
                    gate=rng.random() < 0.7, state=rng.random() < 0.5)
    if kind == "step":
        N = _log_uniform(rng, 1, 512)
        D = groups * max(1, _log_uniform(rng, 16, max(17, min(8192, (1 << 24) // (N * n)))) // groups)
        return dict(kind=kind, dtype=dtype, N=N, D=D, n=n, G=groups, gate=rng.random() < 0.7)
    if kind == "norm":
        rows = _log_uniform(rng, 1, 16384)
        d = _log_uniform(rng, 8, max(9, min(16384, (1 << 24 if dtype == "f32" else 1 << 25) // rows)))
        return dict(kind=kind, dtype=dtype, rows=rows, d=d, bias=rng.random() < 0.7)
    l2norm = rng.random() < 0.5
    if l2norm:
        H, d = rng.randint(1, 32), rng.choice([64, 128])
    else:
        H, d = 1, _log_uniform(rng, 8, 4096)
    case = dict(kind=kind, dtype=dtype, H=H, d=d, W=rng.choice([1, 2, 3, 4, 4]), l2norm=l2norm, bias=rng.random() < 0.5)
    if kind == "conv_step":
        return dict(case, N=_log_uniform(rng, 1, 256))
    T = _log_uniform(rng, 1, 16384)
    T = min(T, max(1, (1 << 24 if dtype == "f32" else 1 << 25) // (H * d)))
    return dict(case, T=T, seqs=_log_uniform(rng, 1, 40), state=rng.random() < 0.5)


def _lengths(case):
    """Ragged lengths that add up to T (empty sequences among them where there are more than 3)."""
    T, n = case["T"], case["seqs"]
    r = random.Random(T * 1009 + n)
    cuts = sorted(r.randint(0, T) for _ in range(n - 1))
    if n > 3:
        cuts[1] = cuts[0]
    ends = [0] + cuts + [T]
    return [b - a for a, b in zip(ends, ends[1:])]


def prepare(case, seed):
    """What a program holds before the call: a layer's weights and the activations."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape, std=1.0, dtype=t):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    f32 = torch.float32
    s = dict(kind=case["kind"])
    if "T" in case:
        lens = _lengths(case)
        s["longest"] = max(lens)
        cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0)
        s["cu"] = cu.to(torch.int32).to(dev)
    if case["kind"] in ("prompt", "train", "step"):
        rows = case.get("T", case.get("N"))
        D, n, G = case["D"], case["n"], case["G"]
        s["u"] = normal(rows, D)
        s["dt"] = normal(rows, D, std=0.7)
        s["B"], s["C"] = normal(rows, G, n), normal(rows, G, n)
        s["z"] = normal(rows, D) if case["gate"] else None
        # step sizes spread over 0.001 .. 0.1, decays of 1 .. n per unit step
        step = torch.exp(uniform(D) * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["A_log"] = torch.log(torch.arange(1, n + 1, device=dev, dtype=f32)).expand(D, n) + normal(D, n, std=0.1, dtype=f32)
        s["A_log"] = s["A_log"].contiguous()
        s["skip"] = 1.0 + normal(D, std=0.1, dtype=f32)
        seqs = case.get("seqs", case.get("N"))
        s["h0"] = normal(seqs, D, n, dtype=f32) if case.get("state", True) else None
        if case["kind"] == "train":
            s["dout"] = normal(rows, D)
            s["dlast"] = normal(seqs, D, n, dtype=f32) if case["state"] else None
    elif case["kind"] == "norm":
        s["x"] = normal(case["rows"], case["d"]) + normal(1, case["d"], std=0.5)
        s["w"] = 1.0 + normal(case["d"], std=0.2, dtype=f32)
        s["b"] = normal(case["d"], std=0.2, dtype=f32) if case["bias"] else None
        s["dy"] = normal(case["rows"], case["d"])
    else:
        rows, H, d, W = case.get("T", case.get("N")), case["H"], case["d"], case["W"]
        seqs = case.get("seqs", case.get("N"))
        s["x"] = normal(rows, H, d)
        s["w"] = normal(H, d, W, std=W ** -0.5, dtype=f32)
        s["b"] = normal(H, d, std=0.2, dtype=f32) if case["bias"] else None
        s["l2norm"] = case["l2norm"]
        s["h0"] = normal(seqs, W - 1, H, d) if case.get("state", True) else None
        if case["kind"] == "conv_train":
            s["dy"] = normal(rows, H, d)
            s["dlast"] = normal(seqs, W - 1, H, d) if case["state"] else None
    return s


def run(s):
    if own:
        return _own(s)
    return {"prompt": _scan, "train": _scan_train, "step": _scan_step, "conv_train": _conv_train,
            "conv_step": _conv_step, "norm": _norm}[s["kind"]](s)


def _own(s):
    import kda_chunkwise_b200 as kda
    kind = s["kind"]
    if kind in ("prompt", "train"):
        kw = dict(skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"], initial_state=s["h0"])
        args = (s["u"], s["dt"], s["A_log"], s["B"], s["C"], s["cu"])
        out, last = kda.kda_selective_scan_fwd(*args, **kw)
        if kind == "prompt":
            return out, last
        return out, last, kda.kda_selective_scan_bwd(*args, s["dout"], dfinal_state=s["dlast"], **kw)
    if kind == "step":
        out = kda.kda_selective_scan_step(s["u"], s["dt"], s["A_log"], s["B"], s["C"], s["h0"], skip=s["skip"],
                                          z=s["z"], dt_bias=s["dt_bias"])
        return out, s["h0"]
    if kind == "norm":
        y, mean, rstd = kda.kda_layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS)
        return y, kda.kda_layer_norm_bwd(s["x"], s["w"], mean, rstd, s["dy"], has_bias=s["b"] is not None)
    kw = dict(bias=s["b"], silu=True, l2norm=s["l2norm"])
    if kind == "conv_step":
        return kda.kda_short_conv_step(s["x"], s["w"], s["h0"], **kw), s["h0"]
    y, last = kda.kda_short_conv_fwd(s["x"], s["w"], s["cu"], initial_state=s["h0"], **kw)
    return y, last, kda.kda_short_conv_bwd(s["x"], s["w"], s["cu"], s["dy"], initial_state=s["h0"],
                                           dfinal_state=s["dlast"], **kw)


# ---- plain forms: elementary torch operations in 32 bits ----------------------------------------


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _heads(x, D):
    """[rows, G, n] -> [rows, D, n]: the group of each channel."""
    return x.float().repeat_interleave(D // x.shape[1], dim=1)


def _ends(cu):
    """Which sequences have tokens, and the first and last token of each."""
    a, b = cu[:-1].long(), cu[1:].long()
    some = b > a
    return some, a, b - 1


def _scan_terms(s):
    """delta [T, D]; the decays a and inputs b of h_t = a_t h_{t-1} + b_t, [T, D, n]."""
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    a = torch.exp(delta[:, :, None] * -torch.exp(s["A_log"]))
    b = (delta * s["u"].float())[:, :, None] * _heads(s["B"], delta.shape[1])
    return delta, a, b


def _linear_recurrence(a, b, longest):
    """All h_t = a_t h_{t-1} + b_t by doubling the span that each entry covers; overwrites both."""
    k = 1
    while k < longest:
        b[k:] += a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _scan_states(s, a, b):
    """h at every token, and the state after every sequence; overwrites a and b."""
    some, first, last = _ends(s["cu"])
    at = first[some]
    h0 = s["h0"] if s["h0"] is not None else a.new_zeros((some.numel(),) + a.shape[1:])
    b[at] += a[at] * h0[some]
    a[at] = 0.0
    h = _linear_recurrence(a, b, s["longest"])
    return h, torch.where(some[:, None, None], h[last.clamp(min=0)], h0)


def _scan_out(s, h):
    y = (h * _heads(s["C"], h.shape[1])).sum(-1) + s["skip"] * s["u"].float()
    gate = 1.0 if s["z"] is None else s["z"].float() * torch.sigmoid(s["z"].float())
    return y, y * gate


def _scan(s):
    _, a, b = _scan_terms(s)
    h, last = _scan_states(s, a, b)
    return _scan_out(s, h)[1].to(s["u"].dtype), last


def _scan_train(s):
    t = s["u"].dtype
    D, (G, n) = s["u"].shape[1], s["B"].shape[1:]
    delta, a, b = _scan_terms(s)
    h, last = _scan_states(s, a, b)
    y, out = _scan_out(s, h)
    u, dout = s["u"].float(), s["dout"].float()
    dz = None
    dy = dout
    if s["z"] is not None:
        sig = torch.sigmoid(s["z"].float())
        dz = dout * y * sig * (1 + s["z"].float() * (1 - sig))
        dy = dout * s["z"].float() * sig
    # the gradient of h_t: C_t dy_t + a_{t+1} dh_{t+1} within a sequence, run backwards in time
    A = -torch.exp(s["A_log"])
    a = torch.exp(delta[:, :, None] * A)
    some, first, final = _ends(s["cu"])
    at, end = first[some], final[some]
    dh = dy[:, :, None] * _heads(s["C"], D)
    if s["dlast"] is not None:
        dh[end] += s["dlast"][some]
    after = torch.cat([a[1:], torch.zeros_like(a[:1])])
    after[end] = 0.0
    dh = _linear_recurrence(after.flip(0), dh.flip(0), s["longest"]).flip(0)
    del after
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[at] = 0.0 if s["h0"] is None else s["h0"][some]
    da = dh * before * a  # the gradient of delta A
    del before
    db = (dh * _heads(s["B"], D)).sum(-1)  # of delta u
    dpre = (db * u + (da * A).sum(-1)) * torch.sigmoid(s["dt"].float() + s["dt_bias"])
    by_group = lambda x: x.reshape(-1, G, D // G, n).sum(2)  # noqa: E731
    dh0 = None
    if s["h0"] is not None:
        dlast = s["dlast"] if s["dlast"] is not None else torch.zeros_like(s["h0"])
        dh0 = torch.where(some[:, None, None], (a * dh)[first.clamp(max=a.shape[0] - 1)], dlast)
    grads = dict(du=(db * delta + dy * s["skip"]).to(t), ddt=dpre.to(t),
                 dA_log=(da * delta[:, :, None]).sum(0) * A,
                 dB=by_group(dh * (delta * u)[:, :, None]).to(t), dC=by_group(h * dy[:, :, None]).to(t),
                 dskip=(dy * u).sum(0), dz=None if dz is None else dz.to(t), ddt_bias=dpre.sum(0),
                 dinitial_state=dh0)
    return out.to(t), last, grads


def _scan_step(s):
    _, a, b = _scan_terms(s)
    s["h0"].copy_(a * s["h0"] + b)
    return _scan_out(s, s["h0"])[1].to(s["u"].dtype), s["h0"]


def _window(s):
    """The W inputs that each token's convolution reads, [T, W, H, d], and where they come from: rows
    of [x; carried states; zero]."""
    x, W, cu = s["x"], s["w"].shape[2], s["cu"].long()
    T, seqs = x.shape[0], cu.numel() - 1
    token = torch.arange(T, device=x.device)
    seq = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    src = token[:, None] + torch.arange(W, device=x.device) - (W - 1)
    early = src - cu[seq][:, None]  # below zero: from the carried state
    old = T + seq[:, None] * (W - 1) + (W - 1) + early
    if s["h0"] is None:
        old = torch.full_like(old, T + seqs * (W - 1))
    src = torch.where(early >= 0, src, old)
    return _rows(s)[src], src


def _rows(s):
    x = s["x"].float()
    old = x.new_zeros((s["cu"].numel() - 1) * (s["w"].shape[2] - 1), *x.shape[1:]) if s["h0"] is None else s["h0"].float().flatten(0, 1)
    return torch.cat([x, old, torch.zeros_like(x[:1])])


def _final_rows(s):
    """The rows of [x; carried states; zero] that the state after each sequence holds, [seqs, W - 1]."""
    W, cu = s["w"].shape[2], s["cu"].long()
    T, seqs = s["x"].shape[0], cu.numel() - 1
    back = torch.arange(W - 1, device=cu.device) - (W - 1)
    pos = (cu[1:] - cu[:-1])[:, None] + back
    old = T + torch.arange(seqs, device=cu.device)[:, None] * (W - 1) + (W - 1) + pos
    if s["h0"] is None:
        old = torch.full_like(old, T + seqs * (W - 1))
    return torch.where(pos >= 0, cu[1:, None] + back, old)


def _conv_out(s, win):
    """The convolution's values, their SiLU and the output."""
    p = (win * s["w"].permute(2, 0, 1)).sum(1)
    if s["b"] is not None:
        p = p + s["b"]
    act = p * torch.sigmoid(p)
    inv = torch.rsqrt((act * act).sum(-1, keepdim=True) + 1e-12)
    return p, act, inv, act * inv if s["l2norm"] else act


def _conv_train(s):
    x, w, t = s["x"], s["w"], s["x"].dtype
    win, src = _window(s)
    p, act, inv, y = _conv_out(s, win)
    rows = _final_rows(s)
    last = _rows(s)[rows].to(t)
    dact = s["dy"].float()
    if s["l2norm"]:
        dact = (dact - y * (y * dact).sum(-1, keepdim=True)) * inv
    sig = torch.sigmoid(p)
    dp = dact * sig * (1 + p * (1 - sig))
    into = torch.zeros_like(_rows(s))
    into.index_add_(0, src.flatten(), (dp[:, None] * w.permute(2, 0, 1)).flatten(0, 1))
    if s["dlast"] is not None:
        into.index_add_(0, rows.flatten(), s["dlast"].float().flatten(0, 1))
    T = x.shape[0]
    grads = dict(dx=into[:T].to(t), dw=(dp[:, None] * win).sum(0).permute(1, 2, 0).contiguous(),
                 dbias=None if s["b"] is None else dp.sum(0),
                 dinitial_state=None if s["h0"] is None else into[T:-1].reshape(s["h0"].shape).to(t))
    return y.to(t), last, grads


def _conv_step(s):
    win = torch.cat([s["h0"], s["x"][:, None]], 1)
    y = _conv_out(s, win.float())[3]
    s["h0"].copy_(win[:, 1:])
    return y.to(s["x"].dtype), s["h0"]


def _norm(s):
    x, t, w = s["x"].float(), s["x"].dtype, s["w"]
    mean = x.mean(-1, keepdim=True)
    rstd = torch.rsqrt(((x - mean) ** 2).mean(-1, keepdim=True) + EPS)
    xhat = (x - mean) * rstd
    y = xhat * w if s["b"] is None else xhat * w + s["b"]
    dy = s["dy"].float()
    g = dy * w
    dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    return y.to(t), dict(dx=dx.to(t), dw=(dy * xhat).sum(0), dbias=None if s["b"] is None else dy.sum(0))


# ---- the definition in 64 bits, token by token --------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    v = {k: x.double() if torch.is_tensor(x) and x.is_floating_point() else x for k, x in s.items()}
    kind = case["kind"]
    if kind in ("prompt", "train"):
        return _exact_scan(case, v, kind == "train")
    if kind == "step":
        h, y = _exact_step(v, v["h0"], 0, slice(None))[:2]
        return y, h
    if kind == "norm":
        return _exact_norm(v)
    return _exact_conv(case, v)


def _exact_step(v, h, i, rows):
    """State and output after the given rows from state h (one row of each sequence)."""
    pre = v["dt"][rows] + v["dt_bias"]
    delta = torch.logaddexp(pre, torch.zeros_like(pre))
    D, G = pre.shape[-1], v["B"].shape[1]
    chan = torch.arange(D, device=pre.device) // (D // G)
    B, C = v["B"][rows][..., chan, :], v["C"][rows][..., chan, :]
    decay = torch.exp(-torch.exp(v["A_log"]) * delta[..., None])
    new = decay * h + (delta * v["u"][rows])[..., None] * B
    y = torch.einsum("...dm,...dm->...d", new, C) + v["skip"] * v["u"][rows]
    gate = 1.0 if v["z"] is None else v["z"][rows] / (1 + torch.exp(-v["z"][rows]))
    return new, y * gate, y, delta, decay, B, C


def _exact_scan(case, v, train):
    T, D, n, G = case["T"], case["D"], case["n"], case["G"]
    if T * D * n > 1 << 30:
        return None
    bounds = v["cu"].tolist()
    out = torch.zeros_like(v["u"])
    lasts, saved = [], []
    for q in range(case["seqs"]):
        h = v["u"].new_zeros(D, n) if v["h0"] is None else v["h0"][q]
        for i in range(bounds[q], bounds[q + 1]):
            if train:
                saved.append(h)
            h, out[i] = _exact_step(v, h, i, i)[:2]
        lasts.append(h)
    last = torch.stack(lasts)
    if not train:
        return out, last
    A = -torch.exp(v["A_log"])
    g = {k: torch.zeros_like(v[m]) for k, m in (("du", "u"), ("ddt", "dt"), ("dA_log", "A_log"), ("dB", "B"), ("dC", "C"),
                                                ("dskip", "skip"), ("ddt_bias", "dt_bias"))}
    g["dz"] = None if v["z"] is None else torch.zeros_like(v["z"])
    g["dinitial_state"] = None if v["h0"] is None else torch.zeros_like(v["h0"])
    for q in range(case["seqs"]):
        dh = torch.zeros_like(lasts[q]) if v["dlast"] is None else v["dlast"][q].clone()
        for i in reversed(range(bounds[q], bounds[q + 1])):
            h = saved[i]
            new, _, y, delta, decay, B, C = _exact_step(v, h, i, i)
            u, do = v["u"][i], v["dout"][i]
            if v["z"] is not None:
                sig = 1 / (1 + torch.exp(-v["z"][i]))
                g["dz"][i] = do * y * (sig + v["z"][i] * sig * (1 - sig))
                do = do * v["z"][i] * sig
            dh = dh + do[:, None] * C
            g["dC"][i] = (do[:, None] * new).view(G, -1, n).sum(1)
            g["dB"][i] = (dh * (delta * u)[:, None]).view(G, -1, n).sum(1)
            dbx, ddecay = torch.einsum("dm,dm->d", dh, B), dh * h * decay
            g["du"][i] = dbx * delta + do * v["skip"]
            g["dskip"] += do * u
            dpre = (dbx * u + torch.einsum("dm,dm->d", ddecay, A)) / (1 + torch.exp(-(v["dt"][i] + v["dt_bias"])))
            g["ddt"][i] = dpre
            g["ddt_bias"] += dpre
            g["dA_log"] += ddecay * delta[:, None] * A
            dh = dh * decay
        if v["h0"] is not None:
            g["dinitial_state"][q] = dh
    return out, last, g


def _exact_conv(case, v):
    """Token by token over time for all sequences' own rows; gradients by automatic differentiation."""
    W, train = case["W"], case["kind"] == "conv_train"
    x, w = v["x"].requires_grad_(), v["w"].requires_grad_()
    bias = None if v["b"] is None else v["b"].requires_grad_()
    seqs = case.get("seqs", case.get("N"))
    h0 = v["h0"] if v["h0"] is not None else x.new_zeros(seqs, W - 1, *x.shape[1:])
    h0.requires_grad_()
    bounds = v["cu"].tolist() if train else list(range(seqs + 1))
    outs, lasts = [], []
    for q in range(seqs) if train else [None]:
        if train:
            rows = torch.cat([h0[q], x[bounds[q]:bounds[q + 1]]])
            m = bounds[q + 1] - bounds[q]
            taps = [rows[j:j + m] for j in range(W)]
            lasts.append(rows[m:m + W - 1])
        else:
            rows = torch.cat([h0, x[:, None]], 1)
            taps = [rows[:, j] for j in range(W)]
            lasts.append(rows[:, 1:])
        p = w[..., 0] * taps[0]
        for j in range(1, W):
            p = p + w[..., j] * taps[j]
        if bias is not None:
            p = p + bias
        y = p / (1 + torch.exp(-p))
        if case["l2norm"]:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) + 1e-12)
        outs.append(y)
    if not train:
        return outs[0].detach(), lasts[0].detach()
    y, last = torch.cat(outs), torch.stack(lasts)
    loss = (y * v["dy"]).sum()
    if v["dlast"] is not None:
        loss = loss + (last * v["dlast"]).sum()
    leaves = [x, w] + ([bias] if bias is not None else []) + [h0]
    got = dict(zip([id(a) for a in leaves], torch.autograd.grad(loss, leaves, allow_unused=True)))
    dh0 = got[id(h0)] if got[id(h0)] is not None else torch.zeros_like(h0)
    return y.detach(), last.detach(), dict(dx=got[id(x)], dw=got[id(w)], dbias=None if bias is None else got[id(bias)],
                                           dinitial_state=None if v["h0"] is None else dh0)


def _exact_norm(v):
    x, w = v["x"].requires_grad_(), v["w"].requires_grad_()
    b = torch.zeros_like(w) if v["b"] is None else v["b"]
    b.requires_grad_()
    c = x - x.sum(-1, keepdim=True) / x.shape[-1]
    y = c / torch.sqrt((c * c).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w + b
    dx, dw, db = torch.autograd.grad((y * v["dy"]).sum(), [x, w, b])
    return y.detach(), dict(dx=dx, dw=dw, dbias=None if v["b"] is None else db)


# ---- what one pass cannot do without ------------------------------------------------------------


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    kind = case["kind"]
    if kind in ("prompt", "train", "step"):
        rows, D, n, G = case.get("T", case.get("N")), case["D"], case["n"], case["G"]
        seqs = case.get("seqs", case.get("N"))
        gate = 1 if case["gate"] else 0
        weights = 4 * D * (n + 2)
        state = 4 * seqs * D * n
        if kind == "train":  # u, dt, z, dout in; out, du, ddt, dz out; B, C and their gradients
            acts = es * rows * ((6 + 2 * gate) * D + 4 * G * n)
            states = state * (4 if case["state"] else 1)
            return dict(bytes=acts + states + 2 * weights, flops=24.0 * rows * D * n)
        acts = es * rows * ((3 + gate) * D + 2 * G * n)
        states = state * (2 if case.get("state", True) else 1)
        return dict(bytes=acts + states + weights, flops=7.0 * rows * D * n)
    if kind == "norm":
        return dict(bytes=4 * es * case["rows"] * case["d"] + 16 * case["d"], flops=20.0 * case["rows"] * case["d"])
    rows, C, W = case.get("T", case.get("N")), case["H"] * case["d"], case["W"]
    seqs = case.get("seqs", case.get("N"))
    state = es * seqs * (W - 1) * C
    if kind == "conv_step":
        return dict(bytes=2 * es * rows * C + 2 * state + 4 * C * (W + 1), flops=(2.0 * W + 8) * rows * C)
    return dict(bytes=4 * es * rows * C + state * (4 if case["state"] else 1) + 8 * C * (W + 1),
                flops=(6.0 * W + 24) * rows * C)
