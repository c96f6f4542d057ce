"""Plain references of the paged 4-bit cache operators, in 64 bits on the CPU.

The format and the operators are written out again from their definitions in
include/kda.h (numpy, per token and head); nothing is shared with the library.
"""
import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)])
E4M3[127] = np.nan
NAN_BYTE = 0x7F


def nearest(x, grid):
    """Index of the nearest of the ascending grid to x >= 0; ties to the even index; the largest holds."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    a, b = x - grid[lo], grid[hi] - x
    return np.where((a > b) | ((a == b) & (hi % 2 == 0)), hi, lo)


def quantise(x):
    """(codes [..., d], scale bytes [..., d / 16]) of finite rows x [..., d] (float32): max / 6 and x / scale in fp32."""
    g = np.asarray(x, dtype=np.float32).reshape(*x.shape[:-1], -1, 16)
    six = (np.abs(g).max(-1) / np.float32(6)).astype(np.float64)
    s = nearest(six, E4M3[:127])
    val = E4M3[s].astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(val > 0, g / val, np.float32(0))
    c = nearest(np.abs(y).astype(np.float64), E2M1) + 8 * (y < 0)
    return c.reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


def held(x, head_scale=None):
    """What rows x [T, H, d] come back as (float64)."""
    hs = np.ones(x.shape[1], dtype=np.float32) if head_scale is None else np.asarray(head_scale, dtype=np.float32)
    c, s = quantise(np.asarray(x, dtype=np.float32) / hs[:, None])
    return (value(c, s).astype(np.float32) * hs[:, None]).astype(np.float64)


def value(codes, scales):
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return v * np.repeat(E4M3[scales & 127], 16, axis=-1)


def block_bytes(d):
    return 16 * 9 * d // 8


def decode(cache, d):
    """Keys and values [pages, H, page_size, d] (float64) of cache bytes [pages, H, page_bytes]."""
    P, H, _ = cache.shape
    blk = cache.reshape(P, H, -1, block_bytes(d))
    nb = blk.shape[2]
    a, b = 16 * d // 2, 16 * d // 16
    kc = blk[..., :a].reshape(P, H, nb, 16, d // 2)
    ks = blk[..., a:a + b].reshape(P, H, nb, 16, d // 16)
    vc = blk[..., a + b:2 * a + b].reshape(P, H, nb, d // 16, 16, 8)
    vs = blk[..., 2 * a + b:].reshape(P, H, nb, d // 16, 16)
    vc = np.swapaxes(vc, 3, 4).reshape(P, H, nb, 16, d // 2)
    vs = np.swapaxes(vs, 3, 4)
    out = []
    for c, s in ((kc, ks), (vc, vs)):
        nib = np.stack((c & 15, c >> 4), axis=-1).reshape(*c.shape[:-1], d)
        out.append(value(nib, s).reshape(P, H, nb * 16, d))
    return out


def attention(q, keys, values, table, seq_len, cu, page, scale, window=0):
    """o [T, Hq, d], lse [T, Hq], and per row the sums of p |v| and of |v| [T, Hq, d] and the largest sum of |q||k| [T, Hq],
    float64.

    keys, values [pages, H, page, d] as decode() gives them."""
    T, Hq, d = q.shape
    H = keys.shape[1]
    G = Hq // H
    o, A, V1 = np.zeros((T, Hq, d)), np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    lse, top = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for r in range(len(seq_len)):
        n, L = int(cu[r + 1] - cu[r]), int(seq_len[r])
        pages = table[r, :-(-L // page)]
        for h in range(H):
            K = keys[pages, h].reshape(-1, d)[:L]
            V = values[pages, h].reshape(-1, d)[:L]
            for i in range(n):
                pos = L - n + i
                lo = max(0, pos - window + 1) if window else 0
                if pos < 0 or lo > pos:
                    continue
                k, v = K[lo:pos + 1], V[lo:pos + 1]
                for x in range(G):
                    row = q[cu[r] + i, h * G + x]
                    s = k @ row * scale
                    m = s.max()
                    p = np.exp(s - m)
                    z = p.sum()
                    at = (cu[r] + i, h * G + x)
                    o[at] = (p / z) @ v
                    A[at] = (p / z) @ np.abs(v)
                    V1[at] = np.abs(v).sum(0)
                    lse[at] = m + math.log(z) if z == z else np.nan
                    top[at] = (np.abs(k) @ np.abs(row)).max() * abs(scale)
    return o, lse, A, V1, top


def attention_bounds(o, lse, A, V1, top, bf16):
    """How far the kernel's o and lse may be from the exact ones, per element.

    A score is an fp32 sum of exact products of d <= 128 terms (and of the two
    f16 parts of a 32-bit query, 22 bits): off by at most 2^-17 of sum |q||k|,
    usually far less; a weight then is off by twice that relative to the
    others, by 2^-20 through exponent arithmetic (arguments below 2^4 matter)
    and, for bf16 calls, by its rounding to f16 (2^-11); the accumulation adds
    2^-17.  A weight is held times 2^7 or more, so f16's smallest step is 2^-31
    of the largest weight and every key may be off by half of that.  The output is rounded to bf16 (2^-8) or fp32."""
    d_score = top * 2.0 ** -17
    rel = 2 * d_score + 2.0 ** -17 + 2.0 ** -20 + (2.0 ** -11 if bf16 else 0.0)
    bound_o = 2 * rel[..., None] * A + 2.0 ** -32 * V1 + (2.0 ** -8 if bf16 else 2.0 ** -23) * np.abs(o) + 1e-30
    bound_lse = d_score + 2.0 ** -19 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))
    return bound_o, bound_lse


def plan(context, new, held_pages, table, free, count, page, T):
    """The page plan of a step, request by request: dict of arrays and the status bits (1: lengths, 32: pages)."""
    R, B = table.shape
    table, status = table.copy(), 0
    cu, seq, out_count = [0], [], []
    slots, pos = np.full(T, -1, dtype=np.int64), np.full(T, -1, dtype=np.int64)
    base, used = 0, 0
    for r in range(R):
        rows = max(int(new[r]), 0)
        cu.append(cu[-1] + rows)
        c, h = int(context[r]), int(held_pages[r])
        ok = new[r] >= 0 and c >= 0 and 0 <= h <= B and c + rows <= B * page and cu[-1] <= T
        if not ok:
            status |= 1
        need = max(0, -(-(c + rows) // page) - h) if ok else 0
        if need and base + need > count:
            ok, status = False, status | 32
        if ok and need:
            for i in range(need):
                table[r, h + i] = free[count - 1 - (base + i)]
            used = base + need
        base += need
        seq.append(c + rows if ok else c)
        out_count.append(h + need if ok else h)
        if ok:
            for i in range(rows):
                p = c + i
                slots[cu[r] + i] = table[r, p // page] * page + p % page
                pos[cu[r] + i] = p
    return dict(cu_seqlens=cu, seq_len=seq, slot_map=slots, positions=pos, page_count=out_count,
                free_count=[count - used], table=table), status
