"""kda_scan_fwd / kda_scan_bwd / kda_scan_step on the GPU against the formulas in 64 bits."""
import math

import pytest
import torch

import kda_gated_delta_02_gb300 as kda
import layer_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate")


def _cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def _inputs(rows, D, G, S, dtype, N=1, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 31 * D + 7 * G + S)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    step = torch.exp(torch.rand(D, generator=gen, device="cuda") * math.log(100) + math.log(0.002))
    return dict(x=r(rows, D).to(dtype), dt=(0.5 * r(rows, D)).to(dtype), A=-torch.exp(r(D, S) * 0.5 + 1), B=r(rows, G, S).to(dtype),
                C=r(rows, G, S).to(dtype), D=r(D), z=r(rows, D).to(dtype), dt_bias=torch.log(torch.expm1(step)),
                h0=r(N, D, S), dy=r(rows, D).to(dtype), dfinal=r(N, D, S))


def _args(s):
    return s["x"], s["dt"], s["A"], s["B"], s["C"]


def _ops(lens, S):
    """Roundings in a row: three a token along a sequence (product, addition, the exponential's eight are in a's
    magnitude once each), the sum over S states, the gates and softplus."""
    return 12 * max([*lens, 1]) + S + 64


def _check_all(s, lens, D, S, options, name, per):
    z, h0, bias, skip, soft = options
    kw = dict(D=s["D"] if skip else None, z=s["z"] if z else None, dt_bias=s["dt_bias"] if bias else None)
    init, dfin = (s["h0"], s["dfinal"]) if h0 else (None, None)
    dt = s["dt"] if soft else (s["dt"].float().abs() * 0.1).to(s["dt"].dtype)
    want = ref.scan(s["x"], dt, s["A"], s["B"], s["C"], lens, h0=init, softplus_dt=soft, dy=s["dy"], dfinal=dfin, **kw)
    args, cu, ops = (s["x"], dt, s["A"], s["B"], s["C"]), _cu(lens), _ops(lens, S)
    y, fin = kda.scan_fwd(*args, cu, initial_state=init, dt_softplus=soft, **kw)
    ref.check(y, want["y"], ops, name + " y")
    ref.check(fin, want["final_state"], ops, name + " final")
    y2, fin2, saved = kda.scan_fwd(*args, cu, initial_state=init, dt_softplus=soft, save=True, **kw)
    assert torch.equal(y, y2) and torch.equal(fin, fin2)
    grads = kda.scan_bwd(*args, cu, s["dy"], saved, initial_state=init, dfinal_state=dfin, dt_softplus=soft, **kw)
    T = sum(lens)
    more = dict(dB=per, dC=per, dA=T, dD=T, ddt_bias=T)
    for g, key in zip(grads, GRADS):
        have = dict(dD=skip, dz=z, ddt_bias=bias, dstate=h0).get(key, True)
        assert (g is None) == (not have), key
        if have:
            ref.check(g, want[key], 2 * ops + more.get(key, 0), f"{name} {key}")


OPTIONS = {"all": (True, True, True, True, True), "bare": (False, False, False, False, True), "delta": (True, True, False, False, False)}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("options", OPTIONS)
@pytest.mark.parametrize("S", [8, 16, 32, 64])
def test_scan(S, options, dtype):
    for lens, D, G in (([1], 1, 1), ([0, 3, 0, 17, 1, 8, 0], 5, 1), ([33, 2], 64, 2), ([9, 16, 24], 130, 1), ([20], 129, 3),
                       ([7, 31], 256, 8)):
        s = _inputs(sum(lens), D, G, S, DTYPES[dtype], len(lens))
        _check_all(s, lens, D, S, OPTIONS[options], f"lens={lens} D={D} G={G}", D // G)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("S,D,G", [(16, 48, 1), (64, 40, 2), (8, 33, 1), (32, 16, 1)])
def test_segments(S, D, G, dtype):
    """Sequences that are cut into segments, forward and back, among short and empty ones."""
    lens = [700, 0, 5, 400, 130]
    lib = kda.load_library()
    T = sum(lens)
    assert lib.kda_scan_workspace_size(len(lens), T, D, G, S) > 0
    s = _inputs(T, D, G, S, DTYPES[dtype], len(lens))
    for options in (OPTIONS["all"], OPTIONS["bare"]):
        _check_all(s, lens, D, S, options, f"{options}", D // G)


def test_uneven_sequences_are_cut():
    """Enough channels for the GPU, one sequence far longer than the mean: it alone is cut, the outputs are the same."""
    D, S, lens = 4096, 16, [3, 1, 0, 40] * 8 + [4100] + [2] * 31
    T, N = sum(lens), len(lens)
    assert kda.load_library().kda_scan_workspace_size(N, T, D, 1, S) > 0
    s = _inputs(T, D, 1, S, torch.bfloat16, N)
    kw = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    y, fin, saved = kda.scan_fwd(*_args(s), _cu(lens), initial_state=s["h0"], save=True, **kw)
    grads = kda.scan_bwd(*_args(s), _cu(lens), s["dy"], saved, initial_state=s["h0"], dfinal_state=s["dfinal"], **kw)
    pick = torch.tensor([0, 77, 1000, 4095], device="cuda")
    cut = {k: (v[:, pick] if k in ("x", "dt", "z", "h0", "dy", "dfinal") else v[pick] if k in ("A", "D", "dt_bias") else v).contiguous()
           for k, v in s.items()}
    want = ref.scan(*_args(cut), lens, D=cut["D"], z=cut["z"], dt_bias=cut["dt_bias"], h0=cut["h0"], dy=cut["dy"], dfinal=cut["dfinal"])
    ops = _ops(lens, S)
    ref.check(y[:, pick], want["y"], ops, "y")
    ref.check(fin[:, pick], want["final_state"], ops, "final")
    for g, key in zip(grads, GRADS):
        if key in ("dx", "ddt", "dz", "dstate"):
            ref.check(g[:, pick], want[key], 2 * ops, key)
        elif key not in ("dB", "dC"):
            ref.check(g[pick], want[key], 2 * ops + T, key)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,pad", [(0, 16), (1, 2), (8, 8)])
def test_rows_apart(dtype, offset, pad):
    """Rows inside wider ones; rows past the last sequence are left as they were."""
    lens, D, G, S = [18, 0, 5], 72, 3, 16
    T = sum(lens)
    P = T + 5
    s = _inputs(P, D, G, S, DTYPES[dtype], len(lens))
    wide = {}
    for k in ("x", "dt", "z", "dy", "B", "C"):
        w = s[k][0].numel()
        buf = torch.full((P, w + offset + pad), 7.0, dtype=s[k].dtype, device="cuda")
        v = buf[:, offset:offset + w]
        wide[k] = v if s[k].dim() == 2 else v.unflatten(1, (G, S))
        wide[k][...] = s[k]
    out = torch.full((P, D + offset + pad), 7.0, dtype=s["x"].dtype, device="cuda")
    kw = dict(D=s["D"], z=wide["z"], dt_bias=s["dt_bias"])
    args = (wide["x"], wide["dt"], s["A"], wide["B"], wide["C"])
    _, fin, saved = kda.scan_fwd(*args, _cu(lens), save=True, out=out[:, offset:offset + D], **kw)
    grads = kda.scan_bwd(*args, _cu(lens), wide["dy"], saved, **kw)
    want = ref.scan(*(t[:T] if t is not s["A"] else t for t in _args(s)), lens, D=s["D"], z=s["z"][:T], dt_bias=s["dt_bias"], dy=s["dy"][:T])
    ops = _ops(lens, S)
    ref.check(out[:T, offset:offset + D], want["y"], ops)
    ref.check(fin, want["final_state"], ops)
    for g, key in zip(grads, GRADS):
        if g is not None:
            ref.check(g[:T] if key in ("dx", "ddt", "dz", "dB", "dC") else g, want[key], 2 * ops + D // G + T, key)
    assert (out[:T, :offset] == 7).all() and (out[:T, offset + D:] == 7).all() and (out[T:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,G,S", [(1, 1, 8), (40, 2, 16), (257, 1, 16), (96, 3, 32), (24, 8, 64), (4096, 1, 16)])
def test_step(D, G, S, dtype):
    """Single tokens against the formulas, and as a continuation of a prompt."""
    for R in (1, 2, 7, 33):
        s = _inputs(R, D, G, S, DTYPES[dtype], R)
        for z, bias, skip, soft in ((True, True, True, True), (False, False, False, True), (True, False, True, False)):
            dt = s["dt"] if soft else (s["dt"].float().abs() * 0.1).to(s["dt"].dtype)
            kw = dict(D=s["D"] if skip else None, z=s["z"] if z else None, dt_bias=s["dt_bias"] if bias else None)
            want = ref.scan(s["x"], dt, s["A"], s["B"], s["C"], [1] * R, h0=s["h0"], softplus_dt=soft, **kw)
            state = s["h0"].clone()
            y = kda.scan_step(s["x"], dt, s["A"], s["B"], s["C"], state, dt_softplus=soft, **kw)
            ref.check(y, want["y"], _ops([1], S), f"R={R}")
            ref.check(state, want["final_state"], _ops([1], S), f"R={R}")


def test_prompt_then_tokens():
    """norm, convolution and scan of a layer: a prompt and then single tokens give what the whole sequence gives."""
    lens, more, D, S = [37, 5, 64], 6, 160, 16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    full = [n + more for n in lens]
    T = sum(full)
    s = _inputs(T, D, 1, S, torch.float32, len(lens))
    hidden, nw, cw, cb = r(T, D), 1 + 0.1 * r(D), 0.5 * r(D, 4), 0.1 * r(D)
    kw = dict(D=s["D"], dt_bias=s["dt_bias"])
    u, tail = kda.conv_fwd(kda.norm_fwd(hidden, nw), cw, _cu(full), bias=cb)
    y, fin = kda.scan_fwd(u, s["dt"], s["A"], s["B"], s["C"], _cu(full), z=s["z"], **kw)
    starts = [sum(full[:i]) for i in range(len(full))]
    prompt = torch.cat([torch.arange(a, a + n) for a, n in zip(starts, lens)]).cuda()
    pu, ptail = kda.conv_fwd(kda.norm_fwd(hidden[prompt], nw), cw, _cu(lens), bias=cb)
    py, state = kda.scan_fwd(pu, s["dt"][prompt], s["A"], s["B"][prompt], s["C"][prompt], _cu(lens), z=s["z"][prompt], **kw)
    assert torch.equal(py, y[prompt])
    for i in range(more):
        at = torch.tensor([a + n + i for a, n in zip(starts, lens)], device="cuda")
        su = kda.conv_step(kda.norm_fwd(hidden[at], nw), cw, ptail, bias=cb)
        assert torch.equal(su, u[at])
        sy = kda.scan_step(su, s["dt"][at], s["A"], s["B"][at], s["C"][at], state, z=s["z"][at], **kw)
        # the same operations but for the order of the sum over states
        assert (sy - y[at]).abs().max() < 64 * 2.0 ** -24 * y.abs().max() * S
    assert torch.equal(ptail, tail) and (state - fin).abs().max() < 64 * 2.0 ** -24 * fin.abs().max()


def test_values_that_are_not_finite_stay_in_their_channel():
    lens, D, S = [30, 20], 70, 16
    s = _inputs(50, D, 1, S, torch.float32, 2)
    y, fin = kda.scan_fwd(*_args(s), _cu(lens), z=s["z"])
    x = s["x"].clone()
    x[11, 9] = float("nan")
    got, gfin = kda.scan_fwd(x, *_args(s)[1:], _cu(lens), z=s["z"])
    seen = torch.zeros_like(y, dtype=torch.bool)
    seen[11:30, 9] = True
    assert got[seen].isnan().all() and torch.equal(got[~seen], y[~seen])
    assert gfin[0, 9].isnan().all() and torch.equal(gfin[1], fin[1])
    # steps of infinity forget the state; steps past the exponential's range do not overflow
    dt = torch.full_like(s["dt"], 3e4)
    y, fin = kda.scan_fwd(s["x"], dt, *_args(s)[2:], _cu(lens))
    assert torch.isfinite(y).all() and torch.isfinite(fin).all()


def test_bad_sequences_are_reported_and_skipped():
    s = _inputs(600, 8, 1, 16, torch.float32, 3)
    for cu in ([0, 300, 200, 600], [0, 100, 601, 601], [-3, 100, 200, 600]):
        cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        y, fin, saved = kda.scan_fwd(*_args(s), cut, save=True, status=status)
        assert status.item() == kda.STATUS_BAD_SEQLENS, cu
        status.zero_()
        kda.scan_bwd(*_args(s), cut, s["dy"], saved, status=status)
        assert status.item() == kda.STATUS_BAD_SEQLENS, cu


@pytest.mark.parametrize("dtype", DTYPES)
def test_first_tokens_have_no_gradient_of_the_rates(dtype):
    """Sequences of one token from zero states: no decay was applied, so dA is zero to the bit."""
    s = _inputs(9, 40, 1, 16, DTYPES[dtype], 9)
    cu = _cu([1] * 9)
    saved = kda.scan_fwd(*_args(s), cu, z=s["z"], save=True)[2]
    grads = kda.scan_bwd(*_args(s), cu, s["dy"], saved, z=s["z"], dfinal_state=s["dfinal"])
    assert not grads[2].any() and grads[0].any() and grads[3].any()


def test_no_tokens():
    """Empty sequences alone: states pass through, gradients too; sums are zero."""
    s = _inputs(0, 24, 1, 16, torch.bfloat16, 2)
    cu = _cu([0, 0])
    y, fin, saved = kda.scan_fwd(*_args(s), cu, initial_state=s["h0"], D=s["D"], dt_bias=s["dt_bias"], save=True)
    assert y.shape == (0, 24) and torch.equal(fin, s["h0"])
    grads = kda.scan_bwd(*_args(s), cu, s["dy"], saved, initial_state=s["h0"], dfinal_state=s["dfinal"], D=s["D"], dt_bias=s["dt_bias"])
    assert torch.equal(grads[8], s["dfinal"]) and not any(grads[i].any() for i in (2, 5, 7))


@pytest.mark.parametrize("n", [1, 8, 13, 700])
def test_rates_of_infinity_forget(n):
    """A = -inf: a state is what the last token put there, to the end of a tile that the sequence does not fill."""
    s = _inputs(n, 16, 1, 16, torch.float32)
    s["A"][3, 5] = float("-inf")
    y, fin = kda.scan_fwd(*_args(s), _cu([n]), initial_state=s["h0"])
    v = s["dt"][-1, 3].double()
    want = torch.nn.functional.softplus(v) * s["x"][-1, 3].double() * s["B"][-1, 0, 5].double()
    assert torch.isfinite(y).all() and torch.isfinite(fin).all() and abs(fin[0, 3, 5].double() - want) <= 16 * ref.U * abs(want)
    state = s["h0"].clone()
    kda.scan_step(s["x"][-1:], s["dt"][-1:], s["A"], s["B"][-1:], s["C"][-1:], state)
    assert abs(state[0, 3, 5].double() - want) <= 16 * ref.U * abs(want)


@pytest.mark.parametrize("lens,D", [([300, 3, 500, 77], 64), ([100] * 40, 1024)])
def test_same_bits_again_and_captured(lens, D):
    s = _inputs(sum(lens), D, 1, 16, torch.bfloat16, len(lens))
    kw = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], initial_state=s["h0"])
    cu = _cu(lens)

    def call():
        y, fin, saved = kda.scan_fwd(*_args(s), cu, save=True, **kw)
        return (y, fin, *kda.scan_bwd(*_args(s), cu, s["dy"], saved, dfinal_state=s["dfinal"], **kw))

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
    """Central differences of f = sum(y g) + sum(final h): e^2 of the third derivative, 2^-24 / e of each output."""
    lens, D, G, S = [40, 0, 13], 20, 2, 16
    s = _inputs(sum(lens), D, G, S, torch.float32, len(lens))
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0")
    cu = _cu(lens)

    def fwd(p, **kw):
        return kda.scan_fwd(p["x"], p["dt"], p["A"], p["B"], p["C"], cu, D=p["D"], z=p["z"], dt_bias=p["dt_bias"],
                            initial_state=p["h0"], **kw)

    def f(p):
        y, fin = fwd(p)
        return (y.double() * s["dy"].double()).sum() + (fin.double() * s["dfinal"].double()).sum()

    saved = fwd(s, save=True)[2]
    grads = kda.scan_bwd(*_args(s), cu, s["dy"], saved, D=s["D"], z=s["z"], dt_bias=s["dt_bias"], initial_state=s["h0"],
                         dfinal_state=s["dfinal"])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    e = 2.0 ** -8
    for name, grad in zip(names, grads):
        v = torch.randn(s[name].shape, generator=gen, device="cuda")
        diff = float((f({**s, name: s[name] + e * v}) - f({**s, name: s[name] - e * v})) / (2 * e))
        want, size = float((grad.double() * v.double()).sum()), float((grad.double().abs() * v.double().abs()).sum())
        assert abs(diff - want) < (32 * e * e + 256 * 2.0 ** -24 / e) * size, (name, diff, want, size)
