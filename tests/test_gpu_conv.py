"""kda_conv_fwd / kda_conv_bwd / kda_conv_step on the GPU against the formulas in 64 bits."""
import pytest
import torch

import kda_gated_delta_02_gb300 as kda
import layer_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LENS = {"one": [1], "none": [0, 0], "short": [2, 0, 1, 3, 0, 5], "mixed": [0, 5, 1, 70, 2, 0], "long": [300, 7, 0, 129, 1, 260]}
OPS = 24  # four products and a bias, the gate's exponential (eight), its sum, quotient and product; backward twice over


def _cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def _inputs(lens, C, W, dtype, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 97 * C + W)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    T, N = sum(lens), len(lens)
    return dict(x=r(T, C).to(dtype), w=0.6 * r(C, W), bias=0.3 * r(C), tail=r(N, W - 1, C).to(dtype), dy=r(T, C).to(dtype),
                dto=r(N, W - 1, C), cu=_cu(lens))


def _check_all(s, lens, act, bias, tail, name):
    b, t = s["bias"] if bias else None, s["tail"] if tail else None
    want = ref.conv(s["x"], s["w"], lens, b, t, act, s["dy"], s["dto"])
    kind = kda.CONV_SILU if act else kda.CONV_NONE
    y, new = kda.conv_fwd(s["x"], s["w"], s["cu"], bias=b, tail=t, conv_act=kind)
    ref.check(y, want["y"], OPS, name + " y")
    assert torch.equal(new.double().cpu(), torch.from_numpy(want["tail"][0])), name
    dx, dw, db, dt = kda.conv_bwd(s["x"], s["w"], s["cu"], s["dy"], bias=b, tail=t, dtail_out=s["dto"], conv_act=kind)
    ref.check(dx, want["dx"], 2 * OPS, name + " dx")
    ref.check(dw, want["dw"], 2 * OPS + sum(lens), name + " dw")
    assert (db is None) == (not bias) and (dt is None) == (not tail)
    if bias:
        ref.check(db, want["dbias"], 2 * OPS + sum(lens), name + " dbias")
    if tail:
        ref.check(dt, want["dtail"], 2 * OPS, name + " dtail")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("W", [1, 2, 3, 4])
def test_conv(W, lens, dtype):
    for C in (1, 5, 8, 136) if lens != "long" else (24, 1031):
        s = _inputs(LENS[lens], C, W, DTYPES[dtype])
        for act, bias, tail in ((True, True, True), (False, False, True), (True, False, False)):
            _check_all(s, LENS[lens], act, bias, tail, f"C={C} act={act} bias={bias} tail={tail}")


@pytest.mark.parametrize("W", [2, 4])
def test_many_sequences(W):
    """More sequences than a round of the search for a token's own, runs of empty ones, and long ones over many runs."""
    lens = [(7 * i) % 5 if i % 3 else 0 for i in range(1100)] + [700, 0, 0, 1]
    s = _inputs(lens, 16, W, torch.bfloat16)
    _check_all(s, lens, True, True, True, "")


def test_dy_in_32_bits_beside_bf16():
    lens = LENS["mixed"]
    s = _inputs(lens, 40, 4, torch.bfloat16)
    dy = torch.randn(s["dy"].shape, device="cuda")
    want = ref.conv(s["x"], s["w"], lens, None, None, True, dy)
    dx, dw, _, _ = kda.conv_bwd(s["x"], s["w"], s["cu"], dy)
    ref.check(dx, want["dx"], 2 * OPS)
    ref.check(dw, want["dw"], 2 * OPS + sum(lens))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,pad", [(0, 16), (1, 2), (8, 0)])
def test_rows_apart(dtype, offset, pad):
    """Inputs and outputs inside wider rows; rows past the last sequence and channels around stay as they were."""
    lens, C, W = [3, 0, 37, 2], 48, 4
    s = _inputs(lens, C, W, DTYPES[dtype])
    N, T, P = len(lens), sum(lens), sum(lens) + 6
    buf = lambda *lead: torch.full((*lead, C + offset + pad), 7.0, dtype=DTYPES[dtype], device="cuda")
    bufs = [buf(P), buf(P), buf(P), buf(P), buf(N, W - 1), buf(N, W - 1)]
    x, dy, y, dx, tail, new = (t[..., offset:offset + C] for t in bufs)
    x[:T], dy[:T], tail[...] = s["x"], s["dy"], s["tail"]
    want = ref.conv(s["x"], s["w"], lens, None, s["tail"], True, s["dy"])
    kda.conv_fwd(x, s["w"], s["cu"], tail=tail, out=y, tail_out=new)
    _, dw, _, dt = kda.conv_bwd(x, s["w"], s["cu"], dy, tail=tail, dx=dx)
    ref.check(y[:T], want["y"], OPS)
    ref.check(dx[:T], want["dx"], 2 * OPS)
    ref.check(dw, want["dw"], 2 * OPS + T)
    ref.check(dt, want["dtail"], 2 * OPS)
    assert torch.equal(new.double().cpu(), torch.from_numpy(want["tail"][0]))
    for t in (bufs[2], bufs[3], bufs[5]):
        assert (t[..., :offset] == 7).all() and (t[..., offset + C:] == 7).all()
    assert (bufs[2][T:] == 7).all() and (bufs[3][T:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C,W", [(5, 4), (264, 4), (64, 1), (96, 2), (1000, 3)])
def test_parts_and_single_tokens_continue(dtype, C, W):
    """A prompt whole, in two parts, and token by token: the same bits, and the same tail."""
    lens = [9, 4, 21]
    s = _inputs(lens, C, W, DTYPES[dtype])
    y, new = kda.conv_fwd(s["x"], s["w"], s["cu"], bias=s["bias"], tail=s["tail"])
    rows = s["x"].split(lens)
    first, tail = kda.conv_fwd(torch.cat([r[:2] for r in rows]), s["w"], _cu([2, 2, 2]), bias=s["bias"], tail=s["tail"])
    rest, tail = kda.conv_fwd(torch.cat([r[2:] for r in rows]), s["w"], _cu([n - 2 for n in lens]), bias=s["bias"], tail=tail)
    parts = [torch.cat((a, b)) for a, b in zip(first.split([2, 2, 2]), rest.split([n - 2 for n in lens]))]
    assert torch.equal(torch.cat(parts), y) and torch.equal(tail, new)
    tail = s["tail"].clone()
    for i in range(4):
        got = kda.conv_step(torch.stack([r[i] for r in rows]), s["w"], tail, bias=s["bias"])
        assert torch.equal(got, torch.stack([p[i] for p in parts]))
    assert torch.equal(tail[1], new[1])


def test_values_that_are_not_finite_stay_where_they_are_seen():
    lens, C = [20, 30], 16
    s = _inputs(lens, C, 4, torch.float32)
    y = kda.conv_fwd(s["x"], s["w"], s["cu"], conv_act=kda.CONV_NONE)[0]
    x = s["x"].clone()
    x[18, 3] = float("nan")
    got = kda.conv_fwd(x, s["w"], s["cu"], conv_act=kda.CONV_NONE)[0]
    seen = torch.zeros_like(y, dtype=torch.bool)
    seen[18:20, 3] = True  # the sequence ends: the next one does not see it
    assert got[seen].isnan().all() and torch.equal(got[~seen], y[~seen])
    big = torch.full((4, 8), 3e38, device="cuda")
    w = torch.ones(8, 1, device="cuda")
    assert torch.equal(kda.conv_fwd(big, w, _cu([4]))[0], big) and not kda.conv_fwd(-big, w, _cu([4]))[0].any()


def test_bad_sequences_are_reported_and_skipped():
    x, w = torch.randn(50, 8, device="cuda"), torch.randn(8, 4, device="cuda")
    for cu in ([0, 30, 20, 50], [0, 10, 60], [-3, 10, 50], [5, 2, 50]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
        kda.conv_fwd(x, w, cut, status=status)
        assert status.item() == kda.STATUS_BAD_SEQLENS, cu
        status.zero_()
        kda.conv_bwd(x, w, cut, x, status=status)
        assert status.item() == kda.STATUS_BAD_SEQLENS, cu


def test_same_bits_again_and_captured():
    lens = [400, 3, 1000, 77]
    s = _inputs(lens, 520, 4, torch.bfloat16)
    call = lambda: (*kda.conv_fwd(s["x"], s["w"], s["cu"], bias=s["bias"], tail=s["tail"]),
                    *kda.conv_bwd(s["x"], s["w"], s["cu"], s["dy"], bias=s["bias"], tail=s["tail"], dtail_out=s["dto"]))
    first = call()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        again = call()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_gradients_against_differences():
    """Central differences of f = sum(y g) + sum(tail h), e = 2^-7: e^2 of the third derivative, 2^-24 / e of each output."""
    lens = [11, 2, 0, 30]
    s = _inputs(lens, 12, 4, torch.float32)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    grads = kda.conv_bwd(s["x"], s["w"], s["cu"], s["dy"], bias=s["bias"], tail=s["tail"], dtail_out=s["dto"])

    def f(x, w, bias, tail):
        y, new = kda.conv_fwd(x, w, s["cu"], bias=bias, tail=tail)
        return (y.double() * s["dy"].double()).sum() + (new.double() * s["dto"].double()).sum()

    p, e = [s["x"], s["w"], s["bias"], s["tail"]], 2.0 ** -7
    for which, grad in enumerate(grads):
        v = torch.randn(p[which].shape, generator=gen, device="cuda")
        up, down = list(p), list(p)
        up[which], down[which] = p[which] + e * v, p[which] - e * v
        diff, want = float((f(*up) - f(*down)) / (2 * e)), float((grad.double() * v.double()).sum())
        size = float((grad.double().abs() * v.double().abs()).sum())
        assert abs(diff - want) < (8 * e * e + 64 * 2.0 ** -24 / e) * size, (which, diff, want, size)
