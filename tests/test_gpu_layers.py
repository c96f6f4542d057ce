"""Norm, convolution and the recurrences as layers use them together: a KDA layer's prompt, its next token and its training
step; guard bands, streams and two calls at once for the new entry points."""
import numpy as np
import pytest
import torch

import kda_gated_delta_02_gb300 as kda
import layer_ref as ref

pytestmark = pytest.mark.gpu
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, device="cuda")


def _cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=I32, device="cuda")


def _err(got, want):
    return float(np.abs(ref.f64(got) - want).max() / np.abs(want).max())


def _unit(x):
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6)


@pytest.mark.parametrize("lens", [[5, 70], [1, 3, 0, 130]])
def test_kda_layer_prompt_then_token(oracle, lens):
    """Projections -> conv_fwd -> chunk_fwd -> norm_fwd, and decode_verify_replay from the state and tail that these
    leave, against the whole sequences through the oracle.  Bars as the prefill's and the verify's own (bf16 operands)."""
    H, d, R = 2, 128, len(lens)
    r, C = _gen(1), 3 * 2 * 128
    full = [n + 1 for n in lens]
    qkv, g, b = r(sum(full), C).to(BF), r(sum(full), H * d).to(BF), r(sum(full), H).to(BF)
    w, nw = 0.5 * r(C, 4), 1 + 0.1 * r(d)
    starts = [sum(full[:i]) for i in range(R)]
    prompt = torch.cat([torch.arange(a, a + n) for a, n in zip(starts, lens)]).cuda()
    status = torch.zeros(1, dtype=I32, device="cuda")
    # q, k and v as parts of one projection: each its own call, with the tails in one buffer
    cu, tail, parts = _cu(lens), torch.empty(R, 3, C, dtype=BF, device="cuda"), []
    for i in range(3):
        cut = slice(i * H * d, (i + 1) * H * d)
        y, t = kda.conv_fwd(qkv[prompt][:, cut], w[cut], cu, tail_out=tail[:, :, cut], status=status)
        assert t.data_ptr() == tail[:, :, cut].data_ptr()
        parts.append(y.view(-1, H, d))
    q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(BF) for t in parts[:2])
    o, S = kda.chunk_fwd(q, k, parts[2], -torch.nn.functional.softplus(g[prompt].float()).view(-1, H, d),
                         torch.sigmoid(b[prompt].float()), cu, status=status)
    y = kda.norm_fwd(o, nw)
    state, last = S.to(BF), torch.tensor([a + n for a, n in zip(starts, lens)], device="cuda")
    none = lambda n: torch.zeros(R, 0, n, dtype=BF, device="cuda")
    y1 = kda.decode_verify_replay(state, tail, w, none(C), none(H * d), none(H), torch.zeros(R, dtype=I32, device="cuda"),
                                  qkv[last].view(R, 1, C), g[last].view(R, 1, -1), b[last].view(R, 1, H), nw, status=status)
    assert status.item() == 0
    u = ref.conv(qkv, w, full)["y"][0].reshape(-1, 3, H, d)
    og, _ = oracle.prefill(_unit(u[:, 0]), _unit(u[:, 1]), u[:, 2].copy(), -ref.softplus(ref.f64(g)).reshape(-1, H, d),
                           ref.sigmoid(ref.f64(b)), np.array([*starts, sum(full)], dtype=np.int32))
    want = og / np.sqrt((og * og).mean(-1, keepdims=True) + 1e-6) * ref.f64(nw)
    assert _err(y, want[prompt.cpu().numpy()]) <= 3e-2
    assert _err(y1[:, 0], want[last.cpu().numpy()]) <= 3e-2
    assert torch.equal(tail, kda.conv_fwd(qkv, w, _cu(full))[1])


def test_kda_layer_training_step(oracle):
    """norm -> conv -> recurrence -> norm and the way back, with the types that the calls hand one another (chunk_bwd's
    gradients are fp32, conv_bwd takes them beside bf16 rows), against the oracle's reverse mode between the formulas."""
    lens, H, d = [70, 9], 2, 128
    r, C, T = _gen(2), 3 * 2 * 128, 79
    cu = _cu(lens)
    x, xw, w, ow = r(T, C).to(BF), 1 + 0.1 * r(C), 0.5 * r(C, 4), 1 + 0.1 * r(d)
    g, beta, dy = -torch.nn.functional.softplus(r(T, H, d)), torch.sigmoid(r(T, H)), r(T, H, d).to(BF)
    n = kda.norm_fwd(x, xw)
    u, _ = kda.conv_fwd(n, w, cu)
    q, k, v = (t.contiguous().view(T, H, d) for t in u.split(H * d, dim=1))
    q, k = q * d ** -0.5, k * d ** -0.5
    o, _, saved = kda.chunk_fwd_train(q, k, v, g, beta, cu)
    kda.norm_fwd(o, ow)
    do, dow, _ = kda.norm_bwd(o, dy, ow)
    dq, dk, dv, _, _, _ = kda.chunk_bwd_saved(q, k, v, g, beta, cu, do, saved)
    du = torch.cat([t.reshape(T, H * d) for t in (dq * d ** -0.5, dk * d ** -0.5, dv)], dim=1)
    assert du.dtype == F32
    dn, dw, _, _ = kda.conv_bwd(n, w, cu, du)
    dx, dxw, _ = kda.norm_bwd(x, dn, xw)
    # the same chain in 64 bits from the start
    rn = ref.norm(x, None, xw, None, 1e-6, False)["y"][0]
    ru = ref.conv(torch.from_numpy(rn), w, lens)["y"][0].reshape(T, 3, H, d)
    sc = d ** -0.5
    args = [np.ascontiguousarray(t) for t in (ru[:, 0] * sc, ru[:, 1] * sc, ru[:, 2])] + [ref.f64(g), ref.f64(beta), cu.cpu().numpy()]
    ro, _ = oracle.prefill(*args)
    back = ref.norm(torch.from_numpy(ro.reshape(-1, d)), dy.reshape(-1, d), ow, None, 1e-6, False)
    grads = oracle.backward(*args, back["dx"][0].reshape(T, H, d))
    rdu = np.concatenate([t.reshape(T, H * d) for t in (grads[0] * sc, grads[1] * sc, grads[2])], axis=1)
    conv = ref.conv(torch.from_numpy(rn), w, lens, dy=torch.from_numpy(rdu))
    last = ref.norm(x, torch.from_numpy(conv["dx"][0]), xw, None, 1e-6, False)
    for name, got, want in (("dx", dx, last["dx"][0]), ("dxw", dxw, last["dweight"][0]), ("dw", dw, conv["dw"][0]), ("dow", dow, back["dweight"][0])):
        assert _err(got, want) <= 5e-2, (name, _err(got, want))


# ------------------------------------------------------------------ every entry point's outputs
def _calls(dtype, D=72, G=3, S=16):
    """name -> (call, {output: shape and type})."""
    lens = [20, 0, 3, 40]
    N, T = len(lens), sum(lens)
    r, cu = _gen(7), _cu(lens)
    t = lambda *s: r(*s).to(dtype)
    x, dt, z, dy, B, C = t(T, D), t(T, D), t(T, D), t(T, D), t(T, G, S), t(T, G, S)
    A, skip, bias, w, cb = -torch.exp(r(D, S)), r(D), r(D), r(D, 4), r(D)
    tail, h0, dto, dh = t(N, 3, D), r(N, D, S), r(N, 3, D), r(N, D, S)
    scan = dict(D=skip, z=z, dt_bias=bias, initial_state=h0)
    _, _, saved = kda.scan_fwd(x, dt, A, B, C, cu, save=True, **scan)

    def step(state=None, out=None, **kw):
        state.copy_(r0)
        return kda.scan_step(x[:N], dt[:N], A, B[:N], C[:N], state, D=skip, z=z[:N], dt_bias=bias, out=out, **kw), state

    def conv_step(tail=None, out=None, **kw):
        tail.copy_(t0)
        return kda.conv_step(x[:N], w, tail, bias=cb, out=out, **kw), tail

    r0, t0 = r(N, D, S), t(N, 3, D)
    rows = ((T, D), dtype)
    return {
        "norm_fwd": (lambda **kw: (kda.norm_fwd(x, skip, cb, kind=kda.NORM_LAYER, **kw),), dict(out=rows)),
        "norm_bwd": (lambda **kw: kda.norm_bwd(x, dy, skip, want_dbias=True, **kw), dict(dx=rows)),
        "conv_fwd": (lambda **kw: kda.conv_fwd(x, w, cu, bias=cb, tail=tail, **kw), dict(out=rows, tail_out=((N, 3, D), dtype))),
        "conv_bwd": (lambda **kw: kda.conv_bwd(x, w, cu, dy, bias=cb, tail=tail, dtail_out=dto, **kw), dict(dx=rows)),
        "conv_step": (conv_step, dict(tail=((N, 3, D), dtype), out=((N, D), dtype))),
        "scan_fwd": (lambda **kw: kda.scan_fwd(x, dt, A, B, C, cu, save=True, **scan, **kw),
                     dict(out=rows, final_state=((N, D, S), F32), saved=((saved.numel(),), F32))),
        "scan_bwd": (lambda **kw: kda.scan_bwd(x, dt, A, B, C, cu, dy, saved, dfinal_state=dh, **scan, **kw), dict()),
        "scan_step": (step, dict(state=((N, D, S), F32), out=((N, D), dtype))),
    }


def _need(outs, dtype):
    return {k: torch.empty(s, dtype=d, device="cuda") for k, (s, d) in outs.items()}


@pytest.mark.parametrize("dtype", [BF, F32])
def test_guard_bands(dtype):
    """Outputs in the middle of larger buffers, whose bands stay as they were; workspaces that large calls share."""
    for name, (call, outs) in _calls(dtype).items():
        want = call(**(_need(outs, dtype) if name.endswith("step") else {}))
        want = [w.clone() for w in want if w is not None]
        full, views = {}, {}
        for k, (shape, d) in outs.items():
            n = int(np.prod(shape))
            full[k] = torch.full((n + 8192,), 7.0, dtype=d, device="cuda")
            views[k] = full[k][4096:4096 + n].view(shape)
        # (slots of `saved` that no state belongs to are not written)
        got = [w for w in call(**views) if w is not None]
        for i, (p, q) in enumerate(zip(got, want)):
            if "saved" in outs and i == 2:
                continue
            assert torch.equal(p, q), (name, i)
        for k, f in full.items():
            assert (f[:4096] == 7).all() and (f[-4096:] == 7).all(), (name, k)


@pytest.mark.parametrize("width", [40, 41])
def test_outputs_beside_inputs_in_one_buffer(width):
    """Inputs and outputs as neighbouring columns of the same rows (width: on and off 16-byte boundaries)."""
    lens, n = [50, 7], 57
    cu, r = _cu(lens), _gen(11)
    rows = r(n, 6 * width).to(BF)
    col = lambda i: rows[:, i * width:(i + 1) * width]
    x, w, nw = col(0).clone(), r(width, 4), r(width)
    want_norm, want_conv = kda.norm_fwd(x, nw), kda.conv_fwd(x, w, cu)[0]
    dt, B, C, A = r(n, width).to(BF), r(n, 1, 16).to(BF), r(n, 1, 16).to(BF), -torch.exp(r(width, 16))
    want_scan = kda.scan_fwd(x, dt, A, B, C, cu, z=x)[0]
    want_dx = kda.conv_bwd(x, w, cu, x)[0]
    kda.norm_fwd(col(0), nw, out=col(1))
    kda.conv_fwd(col(0), w, cu, out=col(2))
    kda.scan_fwd(col(0), dt, A, B, C, cu, z=col(0), out=col(3))
    kda.conv_bwd(col(0), w, cu, col(0), dx=col(4))
    for i, want in enumerate((x, want_norm, want_conv, want_scan, want_dx)):
        assert torch.equal(col(i), want), i
    for bad in (lambda: kda.conv_fwd(col(0), w, cu, out=rows[:, width - 8:2 * width - 8]),
                lambda: kda.scan_fwd(col(0), dt, A, B, C, cu, out=rows[:, 8:width + 8]),
                lambda: kda.norm_fwd(col(0), nw, out=rows[:, 1:width + 1])):
        with pytest.raises(kda.KDAError, match="invalid argument"):
            bad()


def test_offsets_past_32_bits():
    """Rows, saved states and partial sums whose places pass 2^31 elements: the last rows equal those of calls on them alone."""
    r = _gen(13)
    # norm: 17M rows of 128
    x = r(1 << 14, 128).to(BF).repeat(1040, 1)
    assert x.numel() > 1 << 31
    w = r(128)
    y = kda.norm_fwd(x, w)
    assert torch.equal(y[-(1 << 14):], y[:1 << 14]) and torch.equal(y[-5:], kda.norm_fwd(x[-5:].clone(), w))
    dx = kda.norm_bwd(x, x, w)[0]
    assert torch.equal(dx[-(1 << 14):], dx[:1 << 14])
    del x, y, dx
    # convolution: 70,000 tokens of 32,768 channels in two sequences, the second the last 100
    T, C = 70000, 32768
    x, w, cu = r(1000, C).to(BF).repeat(70, 1), 0.5 * r(C, 4), _cu([T - 100, 100])
    assert x.numel() > 1 << 31
    y, tail = kda.conv_fwd(x, w, cu)
    few = kda.conv_fwd(x[-100:].clone(), w, _cu([100]))
    assert torch.equal(y[-100:], few[0]) and torch.equal(tail[1:], few[1])
    dx = kda.conv_bwd(x, w, cu, x)[0]
    assert torch.equal(dx[-100:], kda.conv_bwd(x[-100:].clone(), w, _cu([100]), x[-100:].clone())[0])
    del x, y, dx
    # scan: states of 4,096 channels saved 33,000 times
    T, D, S, last = 264000, 4096, 16, 100
    x, dt = (r(1000, D).to(BF).repeat(264, 1) for _ in range(2))
    B, C = (r(T, 1, S).to(BF) for _ in range(2))
    A, bias, cu = -torch.exp(r(D, S)), -3 + r(D), _cu([T - last, last])
    y, fin, saved = kda.scan_fwd(x, dt, A, B, C, cu, dt_bias=bias, save=True)
    assert saved.numel() > 1 << 31
    end = [t[-last:].clone() for t in (x, dt, B, C)]
    want = kda.scan_fwd(end[0], end[1], A, end[2], end[3], _cu([last]), dt_bias=bias, save=True)
    # (one is cut into segments, the other is not: the same states but for roundings)
    near = lambda p, q: (p.double() - q.double()).norm() <= 2.0 ** -8 * q.double().norm()
    assert near(y[-last:], want[0]) and near(fin[1], want[1][0])
    got = kda.scan_bwd(x, dt, A, B, C, cu, x, saved, dt_bias=bias)
    few = kda.scan_bwd(end[0], end[1], A, end[2], end[3], _cu([last]), end[0], want[2], dt_bias=bias)
    for i in (0, 1, 3, 4):
        assert near(got[i][-last:], few[i]), i


def test_streams_and_two_calls_at_once():
    """Calls on a stream of their own while the current one is busy; two of them side by side; the same bits."""
    calls = _calls(BF)
    want = {n: [w.clone() for w in c(**(_need(o, BF) if n.endswith("step") else {})) if w is not None] for n, (c, o) in calls.items()}
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(3):
        busy = (busy @ busy).clamp(-1, 1)
    got = []
    for side in sides:
        # (inputs are complete; the steps restore theirs on the current stream, so they stay out of this)
        got.append({n: c(stream=side) for n, (c, o) in calls.items() if not n.endswith("step")})
    torch.cuda.synchronize()
    for res in got:
        for n, outs in res.items():
            for i, (p, q) in enumerate(zip([w for w in outs if w is not None], want[n])):
                assert (n == "scan_fwd" and i == 2) or torch.equal(p, q), (n, i)


def test_graphs_on_one_workspace():
    """Two captured graphs on the same workspaces, replayed in turn on one stream."""
    lens, D, S = [900, 3, 700], 64, 16
    N, T = len(lens), sum(lens)
    lib, r, cu = kda.load_library(), _gen(9), _cu(lens)
    ws = torch.empty(max(lib.kda_scan_workspace_size(N, T, D, 1, S), lib.kda_scan_bwd_workspace_size(N, T, D, 1, S)), dtype=torch.uint8,
                     device="cuda")
    assert lib.kda_scan_workspace_size(N, T, D, 1, S) > 0
    sets = []
    for _ in range(2):
        x, dt, dy, B, C = (r(T, *s).to(BF) for s in ((D,), (D,), (D,), (1, S), (1, S)))
        sets.append((x, dt, -torch.exp(r(D, S)), B, C, dy))

    def call(x, dt, A, B, C, dy):
        y, fin, saved = kda.scan_fwd(x, dt, A, B, C, cu, save=True, workspace=ws)
        return (y, fin, *[g for g in kda.scan_bwd(x, dt, A, B, C, cu, dy, saved, workspace=ws) if g is not None])

    want = [[t.clone() for t in call(*s)] for s in sets]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            outs.append(call(*s))
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(p, q) for p, q in zip(o, w))


def test_timing_families():
    """Every launch is counted under its family."""
    calls = _calls(BF)
    kda.kernel_timing_start()
    for n, (c, o) in calls.items():
        c(**(_need(o, BF) if n.endswith("step") else {}))
    t = kda.kernel_timing_stop()
    assert t["kda_norm"]["launches"] == 2 and t["kda_conv"]["launches"] == 3 and t["kda_scan"]["launches"] == 2
    assert t["kda_scan_bwd"]["launches"] == 1 and t["kda_sums"]["launches"] == 4 and "kda_scan_segment" not in t
