"""Calls of the norm, convolution and scan that their documentation allows beside the usual ones: sequences that begin
behind the first row, more sequences than a grid's second axis holds, single tokens inside wider rows, captured, on another
stream and past 32-bit offsets, and several threads on one stream."""
import threading

import pytest
import torch

import kda_gated_delta_02_gb300 as kda
import layer_ref
import scan_ref as ref

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
DTYPES = {"bf16": BF, "f32": F32}
GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, device="cuda")


def _cu(lens, first=0):
    return torch.tensor([first + sum(lens[:i]) for i in range(len(lens) + 1)], dtype=I32, device="cuda")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[20, 0, 3, 40], [700, 0, 5, 400, 130]])
@pytest.mark.parametrize("before,behind", [(5, 0), (3, 9), (130, 2)])
def test_rows_before_the_first_sequence(before, behind, lens, dtype):
    """cu_seqlens that starts past 0: rows before it belong to no sequence, as those behind the last; NaN there is not seen."""
    D, G, S, T, N = 40, 2, 16, sum(lens), len(lens)
    s = ref.inputs(lens, D, G, S, DTYPES[dtype])
    want, cu, cut = ref.scan(s, lens), _cu(lens, before), slice(before, before + T)

    def wide(t):
        w = torch.full((before + T + behind, *t.shape[1:]), float("nan"), dtype=t.dtype, device="cuda")
        w[cut] = t
        return w

    def kept(t):
        return bool((t[:before] == 7).all() and (t[before + T:] == 7).all())

    w = {k: wide(v) if k in ("x", "dt", "z", "dy", "B", "C") else v for k, v in s.items()}
    out = torch.full_like(w["x"], 7)
    args, more = (w["x"], w["dt"], w["A"], w["B"], w["C"], cu), dict(D=w["D"], z=w["z"], dt_bias=w["dt_bias"], initial_state=w["h0"])
    status = torch.zeros(1, dtype=I32, device="cuda")
    _, fin, saved = kda.scan_fwd(*args, save=True, out=out, status=status, **more)
    grads = kda.scan_bwd(*args, w["dy"], saved, dfinal_state=w["dfinal"], status=status, **more)
    assert kept(out)
    for name, got in zip(("y", "final_state", *GRADS), (out, fin, *grads)):
        ref.check(name, got[cut] if name in ref.TOKENS else got, want[name], lens)
    # the convolution, the same way
    r, W = _gen(3), 4
    cw, cb, tail, dto = 0.5 * r(D, W), r(D), r(N, W - 1, D).to(DTYPES[dtype]), r(N, W - 1, D)
    y, dx = torch.full_like(w["x"], 7), torch.full_like(w["x"], 7)
    _, new = kda.conv_fwd(w["x"], cw, cu, bias=cb, tail=tail, out=y, status=status)
    _, dw, db, dt = kda.conv_bwd(w["x"], cw, cu, w["dy"], bias=cb, tail=tail, dtail_out=dto, dx=dx, status=status)
    want = layer_ref.conv(s["x"], cw, lens, cb, tail, True, s["dy"], dto)
    assert kept(y) and kept(dx) and status.item() == 0
    ops = 24  # four products and a bias, the gate; backward twice over
    for name, got, n in (("y", y[cut], ops), ("dx", dx[cut], 2 * ops), ("dw", dw, 2 * ops + T), ("dbias", db, 2 * ops + T), ("dtail", dt, 2 * ops)):
        layer_ref.check(got, want[name], n, name)
    assert torch.equal(new.double().cpu(), torch.from_numpy(want["tail"][0]))


def test_more_sequences_than_a_grids_second_axis():
    """70,000 sequences of one token, and a long one behind them: each is its own single token."""
    n, last, D, S = 70000, 300, 8, 8
    r, lens = _gen(5), [1] * 70000 + [300]
    T, N, cu = n + last, n + 1, torch.arange(n + 2, dtype=I32, device="cuda")
    cu[-1] = T
    x, dt, B, C, A, tail = r(T, D), r(T, D), r(T, 1, S), r(T, 1, S), -torch.exp(r(D, S)), r(N, 3, D)
    h0, w = r(N, D, S), r(D, 4)
    y, fin, saved = kda.scan_fwd(x, dt, A, B, C, cu, initial_state=h0, save=True)
    state, ctail = h0[:n].clone(), tail[:n].clone()
    sy = kda.scan_step(x[:n], dt[:n], A, B[:n], C[:n], state)
    near = lambda p, q: (p - q).norm() <= ref.FORWARD * q.norm()  # (the sum over states in another order)
    assert near(y[:n], sy) and near(fin[:n], state)
    cy, new = kda.conv_fwd(x, w, cu, tail=tail)
    assert torch.equal(cy[:n], kda.conv_step(x[:n], w, ctail)) and torch.equal(new[:n], ctail)
    end, args = _cu([last]), tuple(t[n:].clone() for t in (x, dt))
    want = kda.scan_fwd(*args, A, B[n:].clone(), C[n:].clone(), end, initial_state=h0[n:].clone(), save=True)
    assert near(y[n:], want[0]) and near(fin[n:], want[1])
    got = kda.scan_bwd(x, dt, A, B, C, cu, x, saved, initial_state=h0)
    few = kda.scan_bwd(*args, A, B[n:].clone(), C[n:].clone(), end, args[0], want[2], initial_state=h0[n:].clone())
    for i in (0, 1, 3, 4, 8):
        assert (got[i][n:] - few[i]).norm() <= ref.BACKWARD * few[i].norm(), i
    for p, q in zip(kda.conv_bwd(x, w, cu, x, tail=tail)[::3], kda.conv_bwd(x[n:].clone(), w, end, x[n:].clone(), tail=tail[n:].clone())[::3]):
        assert torch.equal(p[n:], q)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,pad", [(0, 16), (1, 2), (8, 8)])
def test_single_tokens_inside_wider_rows(dtype, offset, pad):
    """Rows of a fused projection, a tail that is part of a wider one: the same bits as with rows of their own, and nothing
    beside them is written."""
    R, D, G, S, W, t = 7, 72, 3, 16, 4, DTYPES[dtype]
    r = _gen(7)

    def wide(v, axis):
        v = v.to(t)
        buf = torch.full((*v.shape[:axis], v[(0,) * axis].numel() + offset + pad), 7.0, dtype=t, device="cuda")
        view = buf[..., offset:buf.shape[-1] - pad].unflatten(-1, v.shape[axis:])
        view.copy_(v)
        return buf, view, v

    x, dt, z = (wide(r(R, D), 1) for _ in range(3))
    B, C = (wide(r(R, G, S), 1) for _ in range(2))
    out, y = wide(r(R, D), 1), wide(r(R, D), 1)
    tail, A, h, skip, bias, w = wide(r(R, W - 1, D), 2), -torch.exp(r(D, S)), r(R, D, S), r(D), r(D), r(D, W)
    states = [h.clone(), h.clone()]
    kda.scan_step(x[1], dt[1], A, B[1], C[1], states[0], D=skip, z=z[1], dt_bias=bias, out=out[1])
    kda.conv_step(x[1], w, tail[1], bias=bias, out=y[1])
    want = kda.scan_step(x[2], dt[2], A, B[2], C[2], states[1], D=skip, z=z[2], dt_bias=bias)
    assert torch.equal(out[1], want) and torch.equal(*states)
    own = tail[2].clone()
    assert torch.equal(y[1], kda.conv_step(x[2], w, own, bias=bias)) and torch.equal(tail[1], own)
    for buf, _, _ in (out, y, tail):
        assert (buf[..., :offset] == 7).all() and (buf[..., buf.shape[-1] - pad:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_single_tokens_captured_and_on_a_stream(dtype):
    """Replays of a captured step move the state and the tail on as eager steps do; so do steps on a stream of their own."""
    R, D, S, t = 33, 130, 16, DTYPES[dtype]
    r = _gen(8)
    x, dt, B, C, A, w = r(R, D).to(t), r(R, D).to(t), r(R, 1, S).to(t), r(R, 1, S).to(t), -torch.exp(r(D, S)), r(D, 4)
    h0, t0 = r(R, D, S), r(R, 3, D).to(t)

    def step(state, tail, **kw):
        u = kda.conv_step(x, w, tail, **kw)
        return u, kda.scan_step(u, dt, A, B, C, state, **kw)

    own = (h0.clone(), t0.clone())
    want = [tuple(v.clone() for v in (*step(*own), *own)) for _ in range(3)]
    state, tail = h0.clone(), t0.clone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        outs = step(state, tail)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((*outs, state, tail), want[i])), i
    state, tail = h0.clone(), t0.clone()
    torch.cuda.synchronize()
    for i in range(3):
        outs = step(state, tail, stream=side)
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((*outs, state, tail), want[i])), i


def test_single_tokens_past_32_bit_offsets():
    """Tails and states of more than 2^31 elements: the last requests equal those of a call on them alone."""
    r, last = _gen(9), 20
    R, C = 32768, 32768
    x, tail, w = r(64, C).to(BF).repeat(R // 64, 1), r(64, 3, C).to(BF).repeat(R // 64, 1, 1), r(C, 4)
    assert tail.numel() > 1 << 31
    few = tail[-last:].clone()
    y = kda.conv_step(x, w, tail)
    assert torch.equal(y[-last:], kda.conv_step(x[-last:].clone(), w, few)) and torch.equal(tail[-last:], few)
    del x, tail, y
    R, D, S = 4096, 40000, 16
    x, dt, B, C = r(R, D).to(BF), r(R, D).to(BF), r(R, 1, S).to(BF), r(R, 1, S).to(BF)
    state, A = r(R, D, S), -torch.exp(r(D, S))
    assert state.numel() > 1 << 31
    few = state[-last:].clone()
    y = kda.scan_step(x, dt, A, B, C, state)
    own = kda.scan_step(*(t[-last:].clone() for t in (x, dt)), A, *(t[-last:].clone() for t in (B, C)), few)
    assert torch.equal(y[-last:], own) and torch.equal(state[-last:], few)


def test_threads_on_one_stream():
    """Four threads, each with inputs of its own, on the same stream: every call's workspace is its own until it is done."""
    lens, D, S = [500, 3, 200], 96, 16
    N, T, cu, work = len(lens), sum(lens), _cu(lens), []
    for i in range(4):
        s, r = ref.inputs(lens, D, 1, S, BF, seed=i), _gen(20 + i)
        w, nw = r(D, 4), r(D)

        def call(s=s, w=w, nw=nw):
            more = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], initial_state=s["h0"])
            args = (s["x"], s["dt"], s["A"], s["B"], s["C"], cu)
            y, fin, saved = kda.scan_fwd(*args, save=True, **more)
            return (y, fin, *kda.scan_bwd(*args, s["dy"], saved, dfinal_state=s["dfinal"], **more), *kda.conv_bwd(s["x"], w, cu, s["dy"])[:2],
                    *kda.norm_bwd(s["x"], s["dy"], nw)[:2])

        work.append((call, [t.clone() for t in call()]))
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        call, want = work[i]
        for k in range(40):
            got = call()
            torch.cuda.current_stream().synchronize()
            if not all(torch.equal(p, q) for p, q in zip(got, want)):
                wrong.append((i, k))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:5]
