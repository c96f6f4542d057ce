"""kda_norm_fwd / kda_norm_bwd on the GPU against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

import kda_gated_delta_02_gb300 as kda
import layer_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
KINDS = {"rms": kda.NORM_RMS, "layer": kda.NORM_LAYER}


def _rand(gen, *s, dtype=torch.float32):
    return torch.randn(s, generator=gen, device="cuda").to(dtype)


def _inputs(rows, d, dtype, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1000 * d + rows)
    x = (_rand(gen, rows, d) * (0.2 + 3 * torch.rand(rows, 1, generator=gen, device="cuda")) + _rand(gen, d)).to(dtype)
    return x, _rand(gen, rows, d, dtype=dtype), 1 + 0.3 * _rand(gen, d), 0.3 * _rand(gen, d)


# roundings in a row: up to 32 channels a thread and 9 joins of threads, twice, and a dozen operations around them
OPS = 2 * (32 + 9) + 16


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [1, 3, 8, 31, 32, 64, 65, 100, 128, 130, 256, 500, 512, 513, 1000, 1024, 1032, 2048, 2056, 4096, 5001,
                               5120, 8192, 8200, 12000, 16383, 16384])
def test_norm(d, dtype):
    rows = 1 if d == 1 else 37 if d < 600 else 5
    x, dy, w, b = _inputs(rows, d, DTYPES[dtype])
    for name, kind in KINDS.items():
        want = ref.norm(x, dy, w, b, 1e-5, name == "layer")
        ref.check(kda.norm_fwd(x, w, b, eps=1e-5, kind=kind), want["y"], OPS, f"{name} y")
        dx, dw, db = kda.norm_bwd(x, dy, w, eps=1e-5, kind=kind, want_dbias=True)
        ref.check(dx, want["dx"], 2 * OPS, f"{name} dx")
        ref.check(dw, want["dweight"], OPS + rows, f"{name} dw")
        ref.check(db, want["dbias"], OPS + rows, f"{name} db")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 127, 128, 640])
def test_many_rows(d, dtype):
    """More rows than blocks walk at once, of a number that no block divides."""
    x, dy, w, b = _inputs(152 * 8 * 32 + 13, d, DTYPES[dtype])
    want = ref.norm(x, dy, w, None, 1e-6, False)
    ref.check(kda.norm_fwd(x, w), want["y"], OPS)
    dx, dw, db = kda.norm_bwd(x, dy, w)
    assert db is None
    ref.check(dx, want["dx"], 2 * OPS)
    ref.check(dw, want["dweight"], OPS + x.shape[0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (3, 5), (8, 24)])
def test_rows_apart(dtype, offset, pad):
    """Rows inside wider ones, on and off 16-byte boundaries, in and out; nothing around them is written."""
    rows, d = 19, 128
    x0, dy0, w, b = _inputs(rows, d, DTYPES[dtype])
    wide = lambda: torch.full((rows, d + offset + pad), 7.0, dtype=DTYPES[dtype], device="cuda")
    bufs = [wide() for _ in range(4)]
    x, dy, y, dx = (t[:, offset:offset + d] for t in bufs)
    x.copy_(x0)
    dy.copy_(dy0)
    kda.norm_fwd(x, w, b, kind=kda.NORM_LAYER, out=y)
    kda.norm_bwd(x, dy, w, kind=kda.NORM_LAYER, dx=dx)
    want = ref.norm(x0, dy0, w, b, 1e-6, True)
    ref.check(y, want["y"], OPS)
    ref.check(dx, want["dx"], 2 * OPS)
    for t in bufs[2:]:
        assert (t[:, :offset] == 7).all() and (t[:, offset + d:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place_shapes_and_empty(dtype):
    x, dy, w, b = _inputs(24, 64, DTYPES[dtype])
    y = kda.norm_fwd(x, w, b)
    assert torch.equal(kda.norm_fwd(x.view(2, 3, 4, 64), w, b).view(24, 64), y)
    z = x.clone()
    assert kda.norm_fwd(z, w, b, out=z) is z and torch.equal(z, y)
    dx, dw, db = kda.norm_bwd(x, dy, w, want_dbias=True)
    for over in ("x", "dy"):
        c = {"x": x.clone(), "dy": dy.clone()}
        got = kda.norm_bwd(c["x"], c["dy"], w, dx=c[over], want_dbias=True)
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)
    got = kda.norm_bwd(x, dy, w, want_dweight=False)
    assert torch.equal(got[0], dx) and got[1] is None and got[2] is None
    e = x[:0]
    assert kda.norm_fwd(e, w, b).shape == (0, 64)
    dx, dw, db = kda.norm_bwd(e, e, w, want_dbias=True)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    assert torch.equal(kda.norm_fwd(x), kda.norm_fwd(x, torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")))


@pytest.mark.parametrize("d", [8, 64, 200, 1024, 6000])
def test_values_that_are_not_finite_stay_in_their_row(d):
    x, dy, w, b = _inputs(9, d, torch.float32)
    for kind in KINDS.values():
        good, gx = kda.norm_fwd(x, w, b, kind=kind), kda.norm_bwd(x, dy, w, kind=kind)[0]
        for bad in (float("inf"), float("-inf"), float("nan")):
            xb = x.clone()
            xb[4, d // 2] = bad
            y, dx = kda.norm_fwd(xb, w, b, kind=kind), kda.norm_bwd(xb, dy, w, kind=kind)[0]
            keep = torch.arange(9, device="cuda") != 4
            assert torch.equal(y[keep], good[keep]) and torch.equal(dx[keep], gx[keep])
            assert y[4, d // 2].isnan()
    zero = torch.zeros(3, d, device="cuda")
    for kind in KINDS.values():  # rows without spread: eps alone
        assert torch.equal(kda.norm_fwd(zero, w, b, kind=kind), b.expand(3, d))


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_channel(dtype):
    """Layer norm of a single channel: the bias, whatever the row, and no gradient of it."""
    x, dy, w, b = _inputs(700, 1, DTYPES[dtype])
    assert torch.equal(kda.norm_fwd(x, w, b, kind=kda.NORM_LAYER), b.to(x.dtype).expand(700, 1))
    dx, dw, _ = kda.norm_bwd(x, dy, w, kind=kda.NORM_LAYER)
    assert not dx.any() and not dw.any()


def test_large_mean_costs_no_digits():
    """The variance is taken of differences: a mean a thousand times the spread leaves n right to a thousand roundings."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    x = 1000 + _rand(gen, 7, 1024)
    ref.check(kda.norm_fwd(x, kind=kda.NORM_LAYER), ref.norm(x, None, None, None, 1e-6, True)["y"], OPS)
    n = ref.norm(x, None, None, None, 1e-6, True)["y"][0]
    assert np.abs(ref.f64(kda.norm_fwd(x, kind=kda.NORM_LAYER)) - n).max() < 4 * 1000 * 2.0 ** -24 * 16


def test_same_bits_again_and_captured():
    x, dy, w, b = _inputs(5000, 128, torch.bfloat16)
    first = (kda.norm_fwd(x, w, b), *kda.norm_bwd(x, dy, w, want_dbias=True))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        again = (kda.norm_fwd(x, w, b), *kda.norm_bwd(x, dy, w, want_dbias=True))
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(first, again))


@pytest.mark.parametrize("kind", KINDS)
def test_gradients_against_differences(kind):
    """(f(p + e v) - f(p - e v)) / 2e of f = sum(y g) in 64 bits over fp32 outputs: e = 2^-7 leaves e^2 of the third
    derivative and 2^-24 / e of each output."""
    x, dy, w, b = _inputs(6, 96, torch.float32)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    dx, dw, db = kda.norm_bwd(x, dy, w, kind=KINDS[kind], want_dbias=True)
    f = lambda x, w, b: (kda.norm_fwd(x, w, b, eps=1e-6, kind=KINDS[kind]).double() * dy.double()).sum()
    e = 2.0 ** -7
    for which, grad in enumerate((dx, dw, db)):
        p = [x, w, b]
        v = _rand(gen, *p[which].shape)
        up, down = list(p), list(p)
        up[which], down[which] = p[which] + e * v, p[which] - e * v
        diff = float((f(*up) - f(*down)) / (2 * e))
        want, size = float((grad.double() * v.double()).sum()), float((grad.double().abs() * v.double().abs()).sum())
        assert abs(diff - want) < (8 * e * e + 64 * 2.0 ** -24 / e) * size, (which, diff, want, size)
