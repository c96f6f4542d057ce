"""The operators around the recurrence, and a second recurrence: what is run, on which inputs, and their plain forms.

Four operators, as the layers of a recurrent model use them:

  norm  norm_fwd / norm_bwd: RMS or layer norm of rows (of heads or of a hidden vector), and its gradients
  conv  conv_fwd / conv_bwd / conv_step: the short causal convolution over packed sequences, with the tail that a
        following call or single tokens continue from, and its gradients
  scan  scan_fwd / scan_bwd: the selective state space recurrence over packed sequences, and its gradients
  step  scan_step: the same recurrence for single tokens, on states in place

Formulas.  norm: y = (x - m) / sqrt(var + eps) w + b (layer), y = x / sqrt(mean(x^2) + eps) w (rms).
conv: p_t = bias + sum_j w[:, j] x_{t - (W - 1) + j}, y = p sigmoid(p) or p; rows before a sequence come from its tail
[W - 1 rows, oldest first], and the tail after it holds its last W - 1 rows.
scan, per channel c and state n, with v = dt + dt_bias and delta = ln(1 + e^v):
    h_t = e^{delta_t A[c, n]} h_{t-1} + delta_t x_t B_t[g, n],   y_t = (sum_n C_t[g, n] h_t + D[c] x_t) z_t sigmoid(z_t)
where g = c / (channels / groups).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the output norm of one token's 96 heads: what a lone decode step waits for
        dict(name="norm_token", op="norm", rows=96, d=128, kind="rms", dtype="bf16", bias=False, train=False),
        # the same norm over the heads of a training batch of 8K tokens, forward and backward
        dict(name="norm_heads_train", op="norm", rows=786432, d=128, kind="rms", dtype="bf16", bias=False, train=True),
        # layer norm of hidden vectors in 32 bits, an odd number of rows
        dict(name="norm_layer_train", op="norm", rows=4099, d=5120, kind="layer", dtype="f32", bias=True, train=True),
        # packed prompts of very different lengths through the convolution of q, k and v of 96 heads of 128
        dict(name="conv_prompt", op="conv", N=16, L=2048, C=36864, W=4, act=True, bias=False, tail=True, dtype="bf16",
             mode="fwd", pick=1),
        # a training batch of a layer of 8K channels
        dict(name="conv_train", op="conv", N=8, L=2048, C=8192, W=4, act=True, bias=True, tail=False, dtype="bf16",
             mode="train", pick=2),
        # one token for each of 256 requests
        dict(name="conv_step", op="conv", N=256, L=1, C=36864, W=4, act=True, bias=False, tail=True, dtype="bf16",
             mode="step", pick=3),
        # one long prompt: few channels for the card, a long sequential axis
        dict(name="scan_prompt", op="scan", N=1, L=16384, D=4096, G=1, S=16, z=True, h0=False, dtype="bf16", train=False,
             pick=4),
        # a ragged batch of prompts that continue from stored states
        dict(name="scan_batch", op="scan", N=32, L=4096, D=2048, G=1, S=16, z=True, h0=True, dtype="bf16", train=False,
             pick=5),
        # a training batch
        dict(name="scan_train", op="scan", N=8, L=2048, D=4096, G=1, S=16, z=True, h0=False, dtype="bf16", train=True,
             pick=6),
        # in 32 bits, two groups of an odd width, ragged, states of 32, no gate
        dict(name="scan_train_f32", op="scan", N=5, L=701, D=1002, G=2, S=32, z=False, h0=True, dtype="f32", train=True,
             pick=7),
        # one token of one request: latency
        dict(name="step_one", op="step", R=1, D=4096, G=1, S=16, z=True, dtype="bf16"),
        # one token for each of 256 requests: the step that a server repeats
        dict(name="step_batch", op="step", R=256, D=8192, G=1, S=16, z=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "conv", "conv", "scan", "scan", "scan", "step"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "norm":
        d = rng.choice((64, 128, _log(rng, 1, 16384), 8 * _log(rng, 1, 2048)))
        kind = rng.choice(("rms", "layer"))
        return dict(op=op, rows=_log(rng, 1, min(500000, 40000000 // d)), d=d, kind=kind, dtype=dtype,
                    bias=rng.random() < 0.5, train=rng.random() < 0.6)
    if op == "conv":
        mode = rng.choice(("fwd", "train", "step"))
        C = rng.choice((_log(rng, 1, 20000), 8 * _log(rng, 1, 4608)))
        N = _log(rng, 1, 256) if mode == "step" else _log(rng, 1, 40)
        L = 1 if mode == "step" else _log(rng, 1, max(1, min(40000, 400000 // N, 100000000 // (C * N))))
        return dict(op=op, N=N, L=L, C=C, W=rng.choice((1, 2, 3, 4, 4)), act=rng.random() < 0.7, bias=rng.random() < 0.5,
                    tail=mode == "step" or rng.random() < 0.5, dtype=dtype, mode=mode, pick=rng.randrange(1 << 20))
    S, G = rng.choice((8, 16, 16, 16, 32, 64)), rng.choice((1, 1, 1, 2, 3, 8))
    D = G * max(1, rng.choice((_log(rng, 16, 5000), 64 * _log(rng, 1, 64))) // G)
    if op == "step":
        return dict(op=op, R=_log(rng, 1, max(1, min(256, 30000000 // (D * S)))), D=D, G=G, S=S, z=rng.random() < 0.7, dtype=dtype)
    train = rng.random() < 0.5
    N = _log(rng, 1, 24)
    L = _log(rng, 1, max(1, min(2000 if train else 8000, 500000000 // (D * S * N))))
    return dict(op=op, N=N, L=L, D=D, G=G, S=S, z=rng.random() < 0.7, h0=rng.random() < 0.5, dtype=dtype, train=train,
                pick=rng.randrange(1 << 20))


def _lengths(case):
    """Lengths of the packed sequences: the first the case's own, the others spread below it, some of them empty.  A
    batch without stored states or tails is of one length."""
    n, L = case["N"], case["L"]
    if case.get("mode") == "step" or not (case.get("tail") or case.get("h0")):
        return [L] * n
    r = random.Random(case["pick"])
    return [L] + [r.choice((r.randint(0, L), r.randint(0, L), r.randint(0, L), r.randint(0, min(L, 5)))) for _ in range(n - 1)]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    f32, dtype, op = torch.float32, DTYPES[case["dtype"]], case["op"]

    def randn(*shape, scale=1.0, to=f32):
        return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(to)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    s = dict(case)
    if op == "norm":
        rows, d = case["rows"], case["d"]
        s.update(x=(randn(rows, d) * torch.exp(0.5 * randn(rows, 1)) + 0.3 * randn(d)).to(dtype), weight=1 + 0.2 * randn(d),
                 b=0.2 * randn(d) if case["bias"] else None)
        if case["train"]:
            s["dy"] = randn(rows, d, to=dtype)
        return s
    if op == "conv":
        lens, C, W = _lengths(case), case["C"], case["W"]
        T = sum(lens)
        s.update(w=randn(C, W, scale=0.5), b=0.2 * randn(C) if case["bias"] else None, lens=lens,
                 tail_in=randn(case["N"], W - 1, C, to=dtype) if case["tail"] else None)
        s["x"] = randn(T, C, to=dtype)
        s["cu"] = _prefix(lens)
        # the tokens whose window reaches before their sequence, and where the rows of the tail after it come from
        starts = [sum(lens[:i]) for i in range(len(lens))]
        s["early"] = [_indices([(at + i, n, i + W - 1 - k) for n, (at, m) in enumerate(zip(starts, lens)) for i in range(min(k, m))], 3)
                      for k in range(W)]
        rows = [(n, j, starts[n], m - (W - 1) + j) for n, m in enumerate(lens) for j in range(W - 1)]
        s["late"] = _indices([(n, j, at + i) for n, j, at, i in rows if i >= 0], 3)
        s["kept"] = _indices([(n, j, i + W - 1) for n, j, _, i in rows if i < 0], 3)
        s["more"] = _indices([(m - 1 - i,) for m in lens for i in range(m)], 1)[0]  # tokens of its sequence after each
        if case["mode"] == "train":
            s.update(dy=randn(T, C, to=dtype), dtail_out=randn(case["N"], W - 1, C) if case["tail"] else None)
        return s
    D, G, S = case["D"], case["G"], case["S"]
    rows = case["R"] if op == "step" else sum(_lengths(case))
    # deltas of 0.001 to 0.1 where dt is zero, rates from 1 to S as such layers start from, moved by training
    target = torch.exp(rand(D) * math.log(100.0) + math.log(0.001))
    s.update(x=randn(rows, D, to=dtype), dt=randn(rows, D, scale=0.5, to=dtype), B=randn(rows, G, S, to=dtype),
             C=randn(rows, G, S, to=dtype), A=-torch.exp(torch.log(torch.arange(1, S + 1, device="cuda", dtype=f32)) + 0.1 * randn(D, S)),
             Dskip=1 + 0.1 * randn(D), dt_bias=torch.log(torch.expm1(target)), zz=randn(rows, D, to=dtype) if case["z"] else None)
    if op == "step":
        s["state"] = randn(rows, D, S, scale=0.3)
        return s
    lens = _lengths(case)
    s.update(lens=lens, cu=_prefix(lens), state0=randn(case["N"], D, S, scale=0.3) if case["h0"] else None)
    if case["train"]:
        s.update(dy=randn(rows, D, to=dtype), dfinal=randn(case["N"], D, S, scale=0.3) if case["h0"] else None)
    return s


def _indices(rows, width):
    """Columns of a list of index tuples, on the GPU."""
    return torch.tensor(rows, dtype=torch.long).view(-1, width).t().contiguous().cuda()


def _prefix(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ plain forms
def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _norm_plain(s):
    x, w = s["x"].float(), s["weight"]
    d = x.shape[1]
    c = x - x.sum(1, keepdim=True) / d if s["kind"] == "layer" else x
    r = 1 / torch.sqrt((c * c).sum(1, keepdim=True) / d + EPS)
    xh = c * r
    y = xh * w
    if s["b"] is not None:
        y = y + s["b"]
    if not s["train"]:
        return y.to(s["x"].dtype)
    dy = s["dy"].float()
    u = dy * w
    dx = u - xh * ((u * xh).sum(1, keepdim=True) / d)
    if s["kind"] == "layer":
        dx = dx - u.sum(1, keepdim=True) / d
    out = dict(y=y.to(s["x"].dtype), dx=(dx * r).to(s["x"].dtype), dweight=(dy * xh).sum(0))
    if s["b"] is not None:
        out["dbias"] = dy.sum(0)
    return out


def _conv_plain(s):
    x, w, W, dtype = s["x"].float(), s["w"], s["W"], s["x"].dtype
    tail = s["tail_in"].float() if s["tail_in"] is not None else x.new_zeros(s["N"], W - 1, x.shape[1])

    def row(k):  # the row k tokens back
        back = torch.roll(x, k, 0) if k else x
        if k:
            at, n, j = s["early"][k]
            back[at] = tail[n, j]
        return back

    p = x * w[:, W - 1]
    for k in range(1, W):
        p += row(k) * w[:, W - 1 - k]
    if s["b"] is not None:
        p += s["b"]
    y = (p * _sigmoid(p) if s["act"] else p).to(dtype)
    (ln, lj, lt), (kn, kj, kt) = s["late"], s["kept"]
    new_tail = torch.empty_like(tail)
    new_tail[ln, lj] = x[lt]
    new_tail[kn, kj] = tail[kn, kt]
    new_tail = new_tail.to(dtype)
    if s["mode"] != "train":
        return y, new_tail
    dp = s["dy"].float()
    if s["act"]:
        g = _sigmoid(p)
        dp = dp * (g * (1 + p * (1 - g)))
    del p
    dw = torch.stack([(dp * row(W - 1 - c)).sum(0) for c in range(W)], dim=1)
    dx = dp * w[:, W - 1]
    dtail = torch.zeros_like(tail)
    for k in range(1, W):
        dx += torch.roll(dp, -k, 0).masked_fill_((s["more"] < k)[:, None], 0) * w[:, W - 1 - k]
        at, n, j = s["early"][k]
        dtail.index_put_((n, j), dp[at] * w[:, W - 1 - k], accumulate=True)
    if s["dtail_out"] is not None:
        dx.index_put_((lt,), s["dtail_out"][ln, lj], accumulate=True)
        dtail.index_put_((kn, kt), s["dtail_out"][kn, kj], accumulate=True)
    out = dict(y=y, tail=new_tail, dx=dx.to(dtype), dw=dw)
    if s["b"] is not None:
        out["dbias"] = dp.sum(0)
    if s["tail_in"] is not None:
        out["dtail"] = dtail
    return out


def _conv_step_plain(s):
    x, w, tail = s["x"].float(), s["w"], s["tail_in"].float()
    rows = torch.cat((tail, x[:, None]), dim=1)
    p = (rows * w.t()).sum(1)
    if s["b"] is not None:
        p = p + s["b"]
    s["tail_in"].copy_(rows[:, 1:])
    return (p * _sigmoid(p) if s["act"] else p).to(s["x"].dtype), s["tail_in"]


def _delta(s):
    v = s["dt"].float() + s["dt_bias"]
    return torch.where(v > 20, v, torch.log1p(torch.exp(v.clamp(max=20))))


def _spread(t, D):
    """[.., G, S] to [.., D, S]: a group's row for each of its channels."""
    return t.float().repeat_interleave(D // t.shape[-2], dim=-2)


def _scan_plain(s):
    x, dtype, N, D, G, S = s["x"].float(), s["x"].dtype, s["N"], s["D"], s["G"], s["S"]
    T, L, A = x.shape[0], max(s["lens"]), s["A"]
    start = s["cu"][:-1].long()
    length = s["cu"][1:].long() - start
    delta = _delta(s)
    gate = s["zz"].float() if s["zz"] is not None else None
    h = s["state0"].clone() if s["state0"] is not None else x.new_zeros(N, D, S)
    y = x.new_empty(T + 1, D)  # the last row takes what lies past a sequence's end
    piece = max(1, min(L, (1 << 28) // (N * D * S)))
    starts = []

    def inputs(i0):
        i = torch.arange(i0, min(i0 + piece, L), device=x.device)[:, None]
        live = i < length
        at = torch.where(live, start + i, T)
        src = at.clamp(max=T - 1)
        d = torch.where(live[..., None], delta[src], 0)  # past a sequence's end: decay 1, nothing added
        return live, at, src, d, x[src], _spread(s["B"][src], D), _spread(s["C"][src], D)

    def states(h, d, xs, B):
        a = torch.exp(d[..., None] * A)
        H = (d * xs)[..., None] * B
        for j in range(H.shape[0]):
            h = torch.addcmul(H[j], a[j], h, out=H[j])
        return a, H

    for i0 in range(0, L, piece):
        starts.append(h)
        live, at, src, d, xs, B, C = inputs(i0)
        a, H = states(h, d, xs, B)
        h = H[-1].clone()
        y[at] = (H * C).sum(-1)
        del a, H
    y = y[:T] + s["Dskip"] * x
    out = (y * (gate * _sigmoid(gate)) if gate is not None else y).to(dtype)
    if not s["train"]:
        return out, h
    dy = s["dy"].float()
    res = dict(y=out, final_state=h)
    if gate is not None:
        g = _sigmoid(gate)
        res["dz"] = (dy * y * (g * (1 + gate * (1 - g)))).to(dtype)
        dy = dy * (gate * g)
    dx, dd, dB, dC = x.new_empty(T + 1, D), x.new_empty(T + 1, D), x.new_empty(T + 1, G, S), x.new_empty(T + 1, G, S)
    dA = torch.zeros_like(A)
    carry = s["dfinal"].clone() if s["dfinal"] is not None else torch.zeros_like(h)
    for i0 in reversed(range(0, L, piece)):
        live, at, src, d, xs, B, C = inputs(i0)
        h0 = starts.pop()
        a, H = states(h0, d, xs, B)
        dys = torch.where(live[..., None], dy[src], 0)
        g = C.mul_(dys[..., None])  # gradients of the states, last to first
        g[-1] += carry
        for j in reversed(range(g.shape[0] - 1)):
            torch.addcmul(g[j], a[j + 1], g[j + 1], out=g[j])
        carry = a[0] * g[0]
        dC[at] = (H * dys[..., None]).view(*dys.shape[:2], G, D // G, S).sum(-2)
        dB[at] = (g * (d * xs)[..., None]).view(*dys.shape[:2], G, D // G, S).sum(-2)
        gB = B.mul_(g).sum(-1)
        H[1:] = H[:-1].clone()
        H[0] = h0
        q = H.mul_(a).mul_(g)  # g a h_{t-1}
        dA += (q * d[..., None]).sum((0, 1))
        dx[at] = d * gB + s["Dskip"] * dys
        dd[at] = xs * gB + q.mul_(A).sum(-1)
        del a, H, g, q, B, C
    v = s["dt"].float() + s["dt_bias"]
    dd = dd[:T] * _sigmoid(v)
    res.update(dx=dx[:T].to(dtype), ddt=dd.to(dtype), dA=dA, dB=dB[:T].to(dtype), dC=dC[:T].to(dtype), dD=(dy * x).sum(0), ddt_bias=dd.sum(0))
    if s["state0"] is not None:
        res["dstate"] = carry
    return res


def _step_plain(s):
    x, D = s["x"].float(), s["D"]
    delta = _delta(s)
    h = torch.exp(delta[..., None] * s["A"]) * s["state"] + (delta * x)[..., None] * _spread(s["B"], D)
    y = (h * _spread(s["C"], D)).sum(-1) + s["Dskip"] * x
    if s["zz"] is not None:
        z = s["zz"].float()
        y = y * (z * _sigmoid(z))
    s["state"].copy_(h)
    return y.to(s["x"].dtype), s["state"]


def run(s):
    op = s["op"]
    if not own:
        if op == "conv" and s["mode"] == "step":
            return _conv_step_plain(s)
        return {"norm": _norm_plain, "conv": _conv_plain, "scan": _scan_plain, "step": _step_plain}[op](s)
    import kda_gated_delta_02_gb300 as kda
    if op == "norm":
        kind = kda.NORM_LAYER if s["kind"] == "layer" else kda.NORM_RMS
        y = kda.norm_fwd(s["x"], s["weight"], s["b"], eps=EPS, kind=kind)
        if not s["train"]:
            return y
        dx, dw, db = kda.norm_bwd(s["x"], s["dy"], s["weight"], eps=EPS, kind=kind, want_dbias=s["b"] is not None)
        out = dict(y=y, dx=dx, dweight=dw)
        if db is not None:
            out["dbias"] = db
        return out
    if op == "conv":
        act = kda.CONV_SILU if s["act"] else kda.CONV_NONE
        if s["mode"] == "step":
            return kda.conv_step(s["x"], s["w"], s["tail_in"], bias=s["b"], conv_act=act), s["tail_in"]
        y, tail = kda.conv_fwd(s["x"], s["w"], s["cu"], bias=s["b"], tail=s["tail_in"], conv_act=act)
        if s["mode"] != "train":
            return y, tail
        dx, dw, db, dtail = kda.conv_bwd(s["x"], s["w"], s["cu"], s["dy"], bias=s["b"], tail=s["tail_in"],
                                         dtail_out=s["dtail_out"], conv_act=act)
        out = dict(y=y, tail=tail, dx=dx, dw=dw)
        if db is not None:
            out["dbias"] = db
        if dtail is not None:
            out["dtail"] = dtail
        return out
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    more = dict(D=s["Dskip"], z=s["zz"], dt_bias=s["dt_bias"])
    if op == "step":
        return kda.scan_step(*args, s["state"], **more), s["state"]
    more["initial_state"] = s["state0"]
    if not s["train"]:
        return kda.scan_fwd(*args, s["cu"], **more)
    y, final, saved = kda.scan_fwd(*args, s["cu"], save=True, **more)
    dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dstate = kda.scan_bwd(*args, s["cu"], s["dy"], saved, dfinal_state=s["dfinal"], **more)
    out = dict(y=y, final_state=final)
    if dz is not None:
        out["dz"] = dz
    out.update(dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=dD, ddt_bias=ddt_bias)
    if dstate is not None:
        out["dstate"] = dstate
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e, op = 2 if case["dtype"] == "bf16" else 4, case["op"]
    if op == "norm":
        n, d = case["rows"] * case["d"], case["d"]
        vec = 4 * d * (1 + case["bias"])
        if not case["train"]:
            return {"bytes": 2 * e * n + vec, "flops": 5 * n}
        return {"bytes": 4 * e * n + 2 * vec, "flops": 15 * n}
    if op == "conv":
        C, W = case["C"], case["W"]
        n, tails = sum(_lengths(case)) * C, case["N"] * (W - 1) * C
        vec = 4 * C * (W + case["bias"])
        moved = e * tails * (1 + case["tail"])
        flops = n * (2 * W + 5 * case["act"])
        if case["mode"] != "train":
            return {"bytes": 2 * e * n + vec + moved, "flops": flops}
        return {"bytes": 4 * e * n + 2 * vec + moved + (8 * tails if case["tail"] else 0), "flops": 3 * flops}
    D, G, S = case["D"], case["G"], case["S"]
    rows = case["R"] if op == "step" else sum(_lengths(case))
    n = rows * D
    par = 4 * D * (S + 2)
    read = e * (n * (2 + case["z"]) + 2 * rows * G * S)
    if op == "step":
        return {"bytes": read + e * n + par + 8 * n * S, "flops": n * (6 * S + 20)}
    states = 4 * case["N"] * D * S
    fwd = {"bytes": read + e * n + par + states * (1 + case["h0"]), "flops": n * (6 * S + 20)}
    if not case["train"]:
        return fwd
    return {"bytes": fwd["bytes"] + read + e * n + par + (2 * states if case["h0"] else 0), "flops": n * (24 * S + 60)}


# ------------------------------------------------------------------ in 64 bits, from the definition
def _leaf(t):
    return None if t is None else t.double().requires_grad_()


def _exact_norm(s):
    x, w, b = _leaf(s["x"]), _leaf(s["weight"]), _leaf(s["b"])
    if s["kind"] == "layer":
        c = x - x.mean(1, keepdim=True)
        y = c / (c.square().mean(1, keepdim=True) + EPS).sqrt() * w
    else:
        y = x / (x.square().mean(1, keepdim=True) + EPS).sqrt() * w
    if b is not None:
        y = y + b
    if not s["train"]:
        return y.detach()
    leaves = [x, w] + ([b] if b is not None else [])
    grads = torch.autograd.grad(y, leaves, s["dy"].double())
    return dict(zip(["y", "dx", "dweight", "dbias"], [y.detach(), *grads]))


def _exact_conv(s):
    """Blocks of channels; a sequence's rows behind its tail, and windows of them."""
    C, W, N, parts = s["C"], s["W"], s["N"], []
    step = max(1, 60000000 // max(1, s["x"].shape[0] + N * W))
    for c in range(0, C, step):
        k = slice(c, c + step)
        cut = lambda t: None if t is None else _leaf(t[..., k])
        x, tail, w, b = cut(s["x"]), cut(s["tail_in"]), _leaf(s["w"][k]), cut(s["b"])
        ys, tails = [], []
        for n, rows in enumerate(x.split(s["lens"])):
            before = tail[n] if tail is not None else rows.new_zeros(W - 1, rows.shape[1])
            e = torch.cat((before, rows))
            p = sum(e[j:j + rows.shape[0]] * w[:, j] for j in range(W))
            if b is not None:
                p = p + b
            ys.append(torch.nn.functional.silu(p) if s["act"] else p)
            tails.append(e[rows.shape[0]:])
        y, t = torch.cat(ys), torch.stack(tails)
        part = dict(y=y.detach(), tail=t.detach())
        if s["mode"] == "train":
            names, leaves = ["dx", "dw"], [x, w]
            if b is not None:
                names, leaves = names + ["dbias"], leaves + [b]
            if tail is not None:
                names, leaves = names + ["dtail"], leaves + [tail]
            outs, douts = [y], [s["dy"][:, k].double()]
            if s["dtail_out"] is not None:
                outs, douts = outs + [t], douts + [s["dtail_out"][..., k].double()]
            g = torch.autograd.grad(outs, leaves, douts, allow_unused=True)
            part.update(zip(names, [torch.zeros_like(l) if v is None else v for v, l in zip(g, leaves)]))
        parts.append(part)
    out = {n: torch.cat([p[n] for p in parts], dim=0 if n in ("dw", "dbias") else -1) for n in parts[0]}
    return out if s["mode"] == "train" else (out["y"], out["tail"])


def _exact_cell(h, v, x, A, B, C, D, z):
    """One token: the new state and the output."""
    delta = torch.nn.functional.softplus(v, threshold=700.0)
    h = torch.exp(delta.unsqueeze(-1) * A) * h + (delta * x).unsqueeze(-1) * B
    y = torch.einsum("...ds,...ds->...d", h, C) + D * x
    return h, y if z is None else y * torch.nn.functional.silu(z)


def _exact_scan(s):
    """Blocks of one group's channels, all sequences side by side, token by token."""
    N, D, G, S, lens = s["N"], s["D"], s["G"], s["S"], s["lens"]
    T, L, train, per = s["x"].shape[0], max(lens), s["train"], D // G
    dev = s["x"].device
    at = torch.zeros(L, N, dtype=torch.long, device=dev)
    live = torch.zeros(L, N, 1, dtype=torch.bool, device=dev)
    first = 0
    for n, m in enumerate(lens):
        at[:m, n] = torch.arange(first, first + m, device=dev)
        live[:m, n] = True
        first += m
    f64 = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=dev)
    out = dict(y=f64(T, D), final_state=f64(N, D, S))
    if train:
        out.update(dz=f64(T, D), dx=f64(T, D), ddt=f64(T, D), dA=f64(D, S), dB=f64(T, G, S), dC=f64(T, G, S), dD=f64(D),
                   ddt_bias=f64(D), dstate=f64(N, D, S))
    room = 250000000 if train else 2000000000
    block = max(1, min(per, room // max(1, L * N * S)))
    for g in range(G):
        for c in range(g * per, (g + 1) * per, block):
            k = slice(c, min(c + block, (g + 1) * per))
            x, dt, A, D_, bias = _leaf(s["x"][:, k]), _leaf(s["dt"][:, k]), _leaf(s["A"][k]), _leaf(s["Dskip"][k]), _leaf(s["dt_bias"][k])
            B, C = _leaf(s["B"][:, g]), _leaf(s["C"][:, g])
            z = None if s["zz"] is None else _leaf(s["zz"][:, k])
            h0 = _leaf(s["state0"][:, k]) if s["state0"] is not None else f64(N, x.shape[1], S).requires_grad_()
            with torch.set_grad_enabled(train):
                h, ys = h0, []
                v = dt + bias
                vs, xs, Bs, Cs = (t[at].unbind(0) for t in (v, x, B.unsqueeze(1), C.unsqueeze(1)))
                zs = [None] * L if z is None else z[at].unbind(0)
                for i in range(L):
                    new, y = _exact_cell(h, vs[i], xs[i], A, Bs[i], Cs[i], D_, zs[i])
                    h = torch.where(live[i].unsqueeze(-1), new, h)
                    ys.append(y)
                y = torch.stack(ys)[live[..., 0]]
            order = at[live[..., 0]]
            out["y"][order, k] = y.detach()
            out["final_state"][:, k] = h.detach()
            if not train:
                continue
            outs, douts = [y], [s["dy"][order][:, k].double()]
            if s["dfinal"] is not None:
                outs, douts = outs + [h], douts + [s["dfinal"][:, k].double()]
            leaves = [x, dt, A, B, C, D_, bias, h0] + ([z] if z is not None else [])
            gr = torch.autograd.grad(outs, leaves, douts)
            out["dx"][:, k], out["ddt"][:, k], out["dA"][k], out["dD"][k], out["ddt_bias"][k], out["dstate"][:, k] = (
                gr[0], gr[1], gr[2], gr[5], gr[6], gr[7])
            out["dB"][:, g] += gr[3]
            out["dC"][:, g] += gr[4]
            if z is not None:
                out["dz"][:, k] = gr[8]
            del ys, y, h, outs, gr
    if not train:
        return out["y"], out["final_state"]
    if s["zz"] is None:
        del out["dz"]
    if s["state0"] is None:
        del out["dstate"]
    return out


def exact(case, seed):
    op = case["op"]
    if op == "scan" and case["L"] * case["N"] * case["D"] * case["S"] * (4 if case["train"] else 1) > 6e9:
        return None
    s = prepare(case, seed)
    if op == "norm":
        return _exact_norm(s)
    if op == "conv":
        if case["mode"] != "step":
            return _exact_conv(s)
        s["lens"] = [1] * case["N"]
        return _exact_conv(s)
    if op == "scan":
        return _exact_scan(s)
    per, f64 = case["D"] // case["G"], lambda t: None if t is None else t.double()
    B, C = (f64(s[n]).unsqueeze(2).expand(-1, -1, per, -1).flatten(1, 2) for n in ("B", "C"))
    h, y = _exact_cell(f64(s["state"]), f64(s["dt"]) + f64(s["dt_bias"]), f64(s["x"]), f64(s["A"]), B, C, f64(s["Dskip"]), f64(s["zz"]))
    return y, h
