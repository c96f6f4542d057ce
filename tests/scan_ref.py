"""The selective scan and its gradients from their formulas, in 64 bits or (to see what fp32 itself costs) in 32, and a
comparison by norms that sees every part of an output.

How far fp32 may be off.  With u = 2^-24: a token's decay e^{delta A} is off by about 2 u at random (its exponent, below 1
here, its 2^x, the product with the state and the state's rounding), and a state remembers m tokens, so it is off by
2 u sqrt(m) in the root mean square.  m is below 2,000 in the inputs made here (steps of 0.002 and more, rates of a half and
more): 90 u = 5e-6.  A step is off by about |v| + 4 roundings of its softplus, 10 u, in every token by another amount, so it
counts once, not once a token.  Outputs are sums of S such states: no further off, relatively.  FORWARD = 1e-5 is twice
that, BACKWARD = 2e-5 four times: a gradient is a product of a state and of what comes back, each off by that much.  Gates
and sums over tokens or channels add tens of u."""
import numpy as np
import torch

FORWARD, BACKWARD = 1e-5, 2e-5
TOKENS = ("y", "dx", "ddt", "dz", "dB", "dC")  # outputs of a row a token
BOUND = dict.fromkeys(("y", "final_state"), FORWARD)


def inputs(lens, D, G, S, dtype, device="cuda", seed=0):
    """Those of a layer: steps of 0.002 to 0.2 where dt is zero, rates around e."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed + 31 * D + 7 * G + S)
    T, N = sum(lens), len(lens)
    r = lambda *s: torch.randn(s, generator=gen, device=device)
    step = torch.exp(torch.rand(D, generator=gen, device=device) * np.log(100) + np.log(0.002))
    rows = {k: r(T, D).to(dtype) for k in ("x", "z", "dy")}
    return dict(rows, dt=(0.5 * r(T, D)).to(dtype), A=-torch.exp(0.5 * r(D, S) + 1), B=r(T, G, S).to(dtype), C=r(T, G, S).to(dtype),
                D=r(D), dt_bias=torch.log(torch.expm1(step)), h0=r(N, D, S), dfinal=r(N, D, S))


def channels(s, pick):
    """The inputs of some channels alone (of one group)."""
    rows = ("x", "dt", "z", "dy", "h0", "dfinal")
    return {k: v[:, pick] if k in rows else v[pick] if k in ("A", "D", "dt_bias") else v for k, v in s.items()}


def scan(s, lens, ft=np.float64):
    """{output: value}, all of them, by the recurrence and its reverse, in arithmetic of type ft."""
    s = {k: None if v is None else v.detach().cpu().double().numpy().astype(ft) for k, v in s.items()}
    x, A, B, C, dy, one = s["x"], s["A"], s["B"], s["C"], s["dy"], ft(1)
    T, n = x.shape
    G, S = B.shape[1:]
    N, per = len(lens), n // G
    zero = lambda *shape: np.zeros(shape, ft)
    skip = zero(n) if s["D"] is None else s["D"]
    v = s["dt"] if s["dt_bias"] is None else s["dt"] + s["dt_bias"]
    delta, slope = np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v))), one / (one + np.exp(-v))
    gate, dgate = np.ones_like(x), zero(T, n)
    if s["z"] is not None:
        q = one / (one + np.exp(-s["z"]))
        gate, dgate = s["z"] * q, q * (one + s["z"] * (one - q))
    e = dy * gate
    out = dict(y=zero(T, n), final_state=zero(N, n, S), dx=zero(T, n), ddt=zero(T, n), dz=zero(T, n), dB=zero(T, G, S), dC=zero(T, G, S),
               dA=zero(n, S), dstate=zero(N, n, S))
    pre, at = zero(T, n), 0
    for q, L in enumerate(lens):
        h = zero(n, S) if s["h0"] is None else s["h0"][q]
        states = [h]
        for t in range(at, at + L):
            a = np.exp(delta[t][:, None] * A)
            h = a * h + (delta[t] * x[t])[:, None] * np.repeat(B[t], per, axis=0)
            pre[t] = (h * np.repeat(C[t], per, axis=0)).sum(1)
            states.append(h)
        out["final_state"][q] = h
        l = zero(n, S) if s["dfinal"] is None else s["dfinal"][q]
        dA = zero(n, S)
        for t in reversed(range(at, at + L)):
            a, h = np.exp(delta[t][:, None] * A), states[t - at]
            l = l + np.repeat(C[t], per, axis=0) * e[t][:, None]
            ah = l * (a * h)
            lb = (l * np.repeat(B[t], per, axis=0)).sum(1)
            out["dx"][t] = delta[t] * lb + skip * e[t]
            out["ddt"][t] = (x[t] * lb + (ah * A).sum(1)) * slope[t]
            out["dB"][t] = (l * (delta[t] * x[t])[:, None]).reshape(G, per, S).sum(1)
            out["dC"][t] = (states[t - at + 1] * e[t][:, None]).reshape(G, per, S).sum(1)
            dA += delta[t][:, None] * ah
            l = a * l
        out["dA"] += dA
        out["dstate"][q] = l
        at += L
    pre += skip * x
    out.update(y=pre * gate, dz=dy * pre * dgate, dD=(e * x).sum(0), ddt_bias=out["ddt"].sum(0))
    return out


def parts(name, shape, lens):
    """Parts of an output that are compared one by one: up to 32 tokens of one sequence; the states of a sequence; the
    rates of a channel; sums over the tokens whole."""
    if name in TOKENS:
        at = 0
        for L in lens:
            yield from (slice(i, min(i + 32, at + L)) for i in range(at, at + L, 32))
            at += L
    elif name == "dA":
        yield from range(shape[0])
    elif name in ("final_state", "dstate"):
        yield from range(len(lens))
    else:
        yield slice(None)


def off(name, got, want, lens):
    """The largest relative error, in the 2-norm, of a part."""
    got = got.detach().cpu().double().numpy() if isinstance(got, torch.Tensor) else np.asarray(got, np.float64)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    worst = 0.0
    for p in parts(name, want.shape, lens):
        d, size = np.linalg.norm(got[p] - want[p]), np.linalg.norm(want[p])
        worst = max(worst, 0.0 if d == 0 else d / size if size > 0 else np.inf)
        if not np.isfinite(d):
            return np.inf
    return worst


def check(name, got, want, lens):
    """got (a tensor) within fp32's error of want by norms, and a rounding to its own type."""
    bound = BOUND.get(name, BACKWARD) + (torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0)
    worst = off(name, got, want, lens)
    assert worst <= bound, (name, worst, bound)
