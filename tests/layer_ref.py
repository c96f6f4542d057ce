"""Norm, short convolution and selective scan in 64 bits, from their formulas, and how far fp32 arithmetic may be off.

Every function takes torch tensors (any device, any float type) and returns {name: (value, magnitude)} in 64 bits on the
CPU: the magnitude is the same sum with every term's absolute value, so that an fp32 evaluation of n operations in a row is
within n * u * magnitude (u = 2^-24 a rounding; the exponentials are good to 2^-21, counted as eight)."""
import numpy as np
import torch

U = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-x))


def check(got, want, ops, name=""):
    """got (a tensor) within a rounding to its type and `ops` fp32 roundings of want = (value, magnitude)."""
    value, mag = want
    got64, half = f64(got), torch.finfo(got.dtype).eps / 2
    assert got64.shape == value.shape, (name, got64.shape, value.shape)
    bound = half * np.abs(value) + ops * U * mag * (1 + half) + 1e-37
    off = np.abs(got64 - value)
    bad = ~(off <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(np.nanmax(off / bound)), np.argwhere(bad)[:3].tolist(),
                           got64[bad][:3].tolist(), value[bad][:3].tolist())


def norm(x, dy, weight, bias, eps, layer):
    x, dy, w, b = f64(x), f64(dy), f64(weight), f64(bias)
    d = x.shape[1]
    w = np.ones(d) if w is None else w
    b = np.zeros(d) if b is None else b
    m = x.mean(1, keepdims=True) if layer else 0.0
    r = 1 / np.sqrt(((x - m) ** 2).mean(1, keepdims=True) + eps)
    n = (x - m) * r
    # a mean is off by roundings of mean|x|, which r carries into n
    far = (np.abs(x) + (np.abs(x).mean(1, keepdims=True) if layer else 0.0)) * r
    kappa = 1 + far.max(1, keepdims=True)
    out = dict(y=(n * w + b, far * np.abs(w) * kappa + np.abs(b)))
    if dy is not None:
        u = dy * w
        c, s = (u * n).mean(1, keepdims=True), u.mean(1, keepdims=True) if layer else 0.0
        mag = np.abs(u) + far * (np.abs(u) * far).mean(1, keepdims=True) + (np.abs(u).mean(1, keepdims=True) if layer else 0.0)
        out["dx"] = (r * (u - n * c - s), r * mag * kappa)
        out["dweight"] = ((dy * n).sum(0), (np.abs(dy) * far * kappa).sum(0))
        out["dbias"] = (dy.sum(0), np.abs(dy).sum(0))
    return out


def conv(x, w, lens, bias=None, tail=None, act=True, dy=None, dtail_out=None):
    x, w, bias, tail, dy, dto = (f64(t) for t in (x, w, bias, tail, dy, dtail_out))
    C, W = w.shape
    N = len(lens)
    z = lambda *s: np.zeros(s)
    y, ym, new = z(*x.shape), z(*x.shape), z(N, W - 1, C)
    dx, dxm, dw, dwm = z(*x.shape), z(*x.shape), z(C, W), z(C, W)
    db, dbm, dt, dtm = z(C), z(C), z(N, W - 1, C), z(N, W - 1, C)
    at = 0
    for n, L in enumerate(lens):
        ext = np.concatenate((tail[n] if tail is not None else z(W - 1, C), x[at:at + L]))
        new[n] = ext[L:]
        p, pm = z(L, C), z(L, C)
        for j in range(W):
            p += ext[j:j + L] * w[:, j]
            pm += np.abs(ext[j:j + L] * w[:, j])
        if bias is not None:
            p += bias
            pm += np.abs(bias)
        s = sigmoid(p)
        y[at:at + L], ym[at:at + L] = (p * s, 1.1 * pm) if act else (p, pm)
        if dy is not None:
            g = dy[at:at + L]
            q = g * (s * (1 + p * (1 - s))) if act else g
            # the gate's derivative moves by at most half of what p is off by
            qm = np.abs(g) * (1.1 + 0.5 * pm) if act else np.abs(g)
            de, dem = np.zeros_like(ext), np.zeros_like(ext)
            for j in range(W):
                de[j:j + L] += q * w[:, j]
                dem[j:j + L] += qm * np.abs(w[:, j])
                dw[:, j] += (q * ext[j:j + L]).sum(0)
                dwm[:, j] += (qm * np.abs(ext[j:j + L])).sum(0)
            db += q.sum(0)
            dbm += qm.sum(0)
            if dto is not None:
                de[L:] += dto[n]
                dem[L:] += np.abs(dto[n])
            dt[n], dtm[n] = de[:W - 1], dem[:W - 1]
            dx[at:at + L], dxm[at:at + L] = de[W - 1:], dem[W - 1:]
        at += L
    return dict(y=(y, ym), tail=(new, 0 * new), dx=(dx, dxm), dw=(dw, dwm), dbias=(db, dbm), dtail=(dt, dtm))


def softplus(v):
    return np.logaddexp(0.0, v)


def scan(x, dt, A, B, C, lens, D=None, z=None, dt_bias=None, h0=None, softplus_dt=True, dy=None, dfinal=None):
    x, dt, A, B, C, D, z, bias, h0, dy, df = (f64(t) for t in (x, dt, A, B, C, D, z, dt_bias, h0, dy, dfinal))
    T, n = x.shape
    G, S = B.shape[1:]
    N, per = len(lens), n // G
    D = np.zeros(n) if D is None else D
    v = dt + (bias if bias is not None else 0.0)
    delta = softplus(v) if softplus_dt else v
    sg = sigmoid(v) if softplus_dt else np.ones_like(v)
    Bx, Cx = (np.repeat(t, per, axis=1) for t in (B, C))
    gate = z * sigmoid(z) if z is not None else np.ones_like(x)
    dgate = sigmoid(z) * (1 + z * (1 - sigmoid(z))) if z is not None else np.zeros_like(x)
    zero = lambda *s: (np.zeros(s), np.zeros(s))
    y, fin = zero(T, n), zero(N, n, S)
    dx, dd, dz, dB, dC = zero(T, n), zero(T, n), zero(T, n), zero(T, G, S), zero(T, G, S)
    dA, dD, dbias, dh0 = zero(n, S), zero(n), zero(n), zero(N, n, S)
    at = 0
    for q, L in enumerate(lens):
        h = h0[q] if h0 is not None else np.zeros((n, S))
        hm = np.abs(h)
        H, HM = [h], [hm]
        for t in range(at, at + L):
            a = np.exp(delta[t][:, None] * A)
            # an exponent's own rounding moves a by |exponent| roundings
            am = a * (1 + np.abs(delta[t][:, None] * A))
            b = (delta[t] * x[t])[:, None] * Bx[t]
            h, hm = a * h + b, am * np.abs(h) + a * hm + np.abs(b)
            H.append(h)
            HM.append(hm)
            pre, prem = (h * Cx[t]).sum(1) + D * x[t], (hm * np.abs(Cx[t])).sum(1) + np.abs(D * x[t])
            y[0][t], y[1][t] = pre * gate[t], prem * np.abs(gate[t])
            if dy is not None:
                dz[0][t], dz[1][t] = dy[t] * pre * dgate[t], np.abs(dy[t]) * prem * (1.1 + np.abs(dgate[t]))
        fin[0][q], fin[1][q] = h, hm
        if dy is not None:
            l = df[q] if df is not None else np.zeros((n, S))
            lm = np.abs(l)
            for t in reversed(range(at, at + L)):
                e = dy[t] * gate[t]
                a = np.exp(delta[t][:, None] * A)
                am = a * (1 + np.abs(delta[t][:, None] * A))
                hp, hpm = H[t - at], HM[t - at]
                l, lm = l + Cx[t] * e[:, None], lm + np.abs(Cx[t] * e[:, None])
                # a h_{t-1} is formed as a product, or as h_t less what was added: off by roundings of h_t
                ah, ahm = a * hp, am * np.abs(hp) + a * hpm + HM[t - at + 1]
                s1, s1m = (l * Bx[t]).sum(1), (lm * np.abs(Bx[t])).sum(1)
                s2, s2m = (l * A * ah).sum(1), (lm * np.abs(A) * ahm).sum(1)
                dx[0][t], dx[1][t] = delta[t] * s1 + D * e, delta[t] * s1m + np.abs(D * e)
                dd[0][t], dd[1][t] = (x[t] * s1 + s2) * sg[t], (np.abs(x[t]) * s1m + s2m) * sg[t]
                gB, gBm = l * (delta[t] * x[t])[:, None], lm * np.abs(delta[t] * x[t])[:, None]
                gC, gCm = H[t - at + 1] * e[:, None], HM[t - at + 1] * np.abs(e)[:, None]
                for out, val, mag in ((dB, gB, gBm), (dC, gC, gCm)):
                    out[0][t], out[1][t] = val.reshape(G, per, S).sum(1), mag.reshape(G, per, S).sum(1)
                dA[0][...] += delta[t][:, None] * l * ah
                dA[1][...] += delta[t][:, None] * lm * ahm
                dD[0][...] += e * x[t]
                dD[1][...] += np.abs(e * x[t])
                dbias[0][...] += dd[0][t]
                dbias[1][...] += dd[1][t]
                l, lm = a * l, am * np.abs(l) + a * lm
            dh0[0][q], dh0[1][q] = l, lm
        at += L
    return dict(y=y, final_state=fin, dx=dx, ddt=dd, dz=dz, dB=dB, dC=dC, dA=dA, dD=dD, ddt_bias=dbias, dstate=dh0)
