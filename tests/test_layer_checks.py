"""Refusals of the norm, convolution and scan calls (binding and C ABI, no GPU)."""
import ctypes
import weakref

import pytest
import torch

import kda_gated_delta_02_gb300 as kda

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Fake:
    """A tensor's dtype, shape and layout with a CUDA device, for the checks that come before any pointer is used."""

    def __init__(self, *shape, dtype=F32, device=0, t=None):
        self.t, self.index = torch.empty(shape, dtype=dtype) if t is None else t, device

    def __getattr__(self, name):
        return getattr(self.t, name)

    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index

    def view(self, *s):
        return Fake(t=self.t.view(*s), device=self.index)

    def as_strided(self, *s):
        return Fake(t=self.t.as_strided(*s), device=self.index)

    def __getitem__(self, k):
        return Fake(t=self.t[k], device=self.index)


@pytest.fixture(autouse=True)
def no_cuda(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(kda, "_raw_stream", lambda device: 0)

    real = torch.empty_like
    monkeypatch.setattr(torch, "empty_like", lambda t: Fake(*t.shape, dtype=t.dtype) if isinstance(t, Fake) else real(t))
    monkeypatch.setattr(kda._Device, "new", lambda self, *s, dtype=F32: Fake(*s, dtype=dtype))
    monkeypatch.setattr(kda._Device, "out", lambda self, t, like: Fake(*like.shape, dtype=like.dtype) if t is None else t)

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: 0

            def called(*a):
                raise AssertionError(f"{name} was called")
            return called

    monkeypatch.setattr(kda, "load_library", Lib)


def _conv(**kw):
    a = dict(x=Fake(7, 12, dtype=BF), conv_w=Fake(12, 4), cu_seqlens=Fake(3, dtype=I32), bias=Fake(12), tail=Fake(2, 3, 12, dtype=BF))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad,msg", [
    (dict(x=Fake(7, 12, dtype=torch.float16)), "unsupported input dtype"),
    (dict(x=Fake(7, 3, 4, dtype=BF)), "x must be"),
    (dict(conv_w=Fake(12)), "conv_w"),
    (dict(conv_w=Fake(11, 4)), "conv_w must have shape"),
    (dict(conv_w=Fake(12, 4, dtype=BF)), "conv_w must be"),
    (dict(conv_w=Fake(t=torch.empty(4, 12).t())), "conv_w must be contiguous"),
    (dict(cu_seqlens=Fake(3, dtype=torch.int64)), "cu_seqlens must be"),
    (dict(cu_seqlens=Fake(1, dtype=I32)), "cu_seqlens must be int32"),
    (dict(bias=Fake(11)), "bias must have shape"),
    (dict(tail=Fake(2, 3, 12)), "tail must be"),
    (dict(tail=Fake(2, 2, 12, dtype=BF)), "tail must have shape"),
    (dict(tail=Fake(t=torch.empty(2, 5, 12, dtype=BF)[:, :3])), "the same way apart"),
    (dict(x=Fake(t=torch.empty(12, 7, dtype=BF).t())), "rows must be contiguous"),
    (dict(x=Fake(t=torch.empty(1, 12, dtype=BF).expand(7, 12))), "must not overlap"),
    (dict(bias=Fake(12, device=1)), "must be on cuda:0"),
    (dict(x=torch.empty(7, 12, dtype=BF)), "CUDA tensors"),
    (dict(out=Fake(7, 12)), "out must be"),
    (dict(tail_out=Fake(2, 3, 11, dtype=BF)), "tail_out must have shape"),
])
def test_conv_fwd_rejects(bad, msg):
    with pytest.raises(kda.KDAError, match=msg):
        kda.conv_fwd(**_conv(**bad))


def test_conv_bwd_and_step_reject():
    dy = Fake(7, 12, dtype=BF)
    for bad, msg in ((dict(dy=Fake(7, 12, dtype=torch.float16)), "dy must be"), (dict(dy=Fake(6, 12, dtype=BF)), "dy must have shape"),
                     (dict(dtail_out=Fake(2, 3, 12, dtype=BF)), "dtail_out must be"), (dict(dx=Fake(7, 12)), "dx must be")):
        with pytest.raises(kda.KDAError, match=msg):
            kda.conv_bwd(**{**_conv(dy=dy), **bad})
    with pytest.raises(kda.KDAError, match="dy must be"):  # bf16 beside 32-bit activations
        kda.conv_bwd(**_conv(x=Fake(7, 12), tail=Fake(2, 3, 12), dy=dy))
    with pytest.raises(kda.KDAError, match="tail must have shape"):
        kda.conv_step(Fake(7, 12, dtype=BF), Fake(12, 4), Fake(6, 3, 12, dtype=BF))


def test_norm_rejects():
    x = Fake(7, 12, dtype=BF)
    for bad, msg in ((dict(x=Fake(7, 12, dtype=torch.float64)), "unsupported input dtype"), (dict(weight=Fake(11)), "weight must have shape"),
                     (dict(weight=Fake(12, dtype=BF)), "weight must be"), (dict(bias=Fake(1, 12)), "bias must have shape"),
                     (dict(out=Fake(7, 12)), "out must be"), (dict(out=Fake(6, 12, dtype=BF)), "out must have shape"),
                     (dict(x=Fake(t=torch.empty(2, 7, 24, dtype=BF)[..., :12])), "contiguous, or rows"),
                     (dict(x=Fake(7, 0, dtype=BF)), "x must be"), (dict(weight=Fake(12, device=1)), "must be on cuda:0")):
        with pytest.raises(kda.KDAError, match=msg):
            kda.norm_fwd(**{**dict(x=x), **bad})
    with pytest.raises(kda.KDAError, match="dy must be"):
        kda.norm_bwd(x, Fake(7, 12))
    with pytest.raises(kda.KDAError, match="dx must have shape"):
        kda.norm_bwd(x, x, dx=Fake(7, 11, dtype=BF))


def test_another_device_becomes_the_current_one(monkeypatch):
    """Tensors on a device that is not the current one: the call goes there, with that device's current stream."""
    monkeypatch.setattr(torch.cuda, "device", lambda index: ("device", index))
    monkeypatch.setattr(kda, "_raw_stream", lambda device: 0x100 + device)
    there, here = kda._Device(Fake(3, device=1), None), kda._Device(Fake(3), None)
    assert there.guard == ("device", 1) and there.stream == 0x101 and here.guard is kda._here and here.stream == 0x100

    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0x77

    monkeypatch.setattr(torch.cuda, "stream", lambda s: ("stream", s))
    assert kda._Device(Fake(3, device=1), Stream).guard == ("stream", Stream) and kda._Device(Fake(3, device=1), Stream).stream == 0x77
    with pytest.raises(kda.KDAError, match="stream is on cuda:1"):
        kda._Device(Fake(3), Stream)


def _scan(**kw):
    a = dict(x=Fake(9, 24), dt=Fake(9, 24), A=Fake(24, 16), B=Fake(9, 2, 16), C=Fake(9, 2, 16), cu_seqlens=Fake(3, dtype=I32))
    a.update(kw)
    return a


@pytest.mark.parametrize("bad,msg", [
    (dict(x=Fake(9, 24, dtype=BF)), "dt must be"), (dict(dt=Fake(9, 23)), "dt must have shape"), (dict(A=Fake(24, 15)), "A must have shape"),
    (dict(B=Fake(9, 32)), "must be"), (dict(C=Fake(9, 1, 16)), "C must have shape"), (dict(z=Fake(9, 24, dtype=BF)), "z must be"),
    (dict(D=Fake(23)), "D must have shape"), (dict(dt_bias=Fake(24, dtype=BF)), "dt_bias must be"),
    (dict(initial_state=Fake(2, 24, 15)), "initial_state must have shape"), (dict(final_state=Fake(3, 24, 16)), "final_state must have shape"),
    (dict(cu_seqlens=Fake(3)), "cu_seqlens must be"), (dict(B=Fake(t=torch.empty(9, 2, 32)[..., ::2])), "rows must be contiguous"),
    (dict(z=Fake(9, 24, device=1)), "must be on cuda:0"), (dict(out=Fake(9, 23)), "out must have shape"),
])
def test_scan_fwd_rejects(bad, msg):
    with pytest.raises(kda.KDAError, match=msg):
        kda.scan_fwd(**_scan(**bad))


def test_scan_bwd_and_step_reject(monkeypatch):
    class Lib:
        def __getattr__(self, name):
            return lambda *a: 4000 if name == "kda_scan_saved_size" else 0

    monkeypatch.setattr(kda, "load_library", Lib)
    a = _scan(dy=Fake(9, 24))
    with pytest.raises(kda.KDAError, match="saved must hold 1000"):
        kda.scan_bwd(**a, saved=Fake(999))
    with pytest.raises(kda.KDAError, match="saved must hold 1000"):
        kda.scan_fwd(**_scan(), save=True, saved=Fake(999))
    with pytest.raises(kda.KDAError, match="dy must have shape"):
        kda.scan_bwd(**{**a, "dy": Fake(9, 23)}, saved=Fake(1000))
    with pytest.raises(kda.KDAError, match="dfinal_state must have shape"):
        kda.scan_bwd(**a, saved=Fake(1000), dfinal_state=Fake(1, 24, 16))
    with pytest.raises(kda.KDAError, match="state must have shape"):
        kda.scan_step(a["x"], a["dt"], a["A"], a["B"], a["C"], Fake(8, 24, 16))


# ------------------------------------------------------------------ C ABI
@pytest.fixture
def lib(monkeypatch):
    monkeypatch.undo()
    return kda.load_library()


class Room:
    """Host memory cut into 16-byte aligned pieces: the calls below are refused before they use any."""

    def __init__(self):
        self.buf = ctypes.create_string_buffer(1 << 20)
        self.at = (ctypes.addressof(self.buf) + 63) & ~63

    def __call__(self, n):
        p, self.at = self.at, self.at + (n + 63) // 64 * 64
        return p


def test_norm_abi_refuses_before_any_launch(lib):
    r = Room()
    x, y, w, b, dy, dx, ws = (r(8192) for _ in range(7))
    need = lib.kda_norm_bwd_workspace_size(6, 40, 1)
    ws = r(need)

    def fwd(x=x, w=w, b=b, rows=6, d=40, xs=40, ys=40, kind=0, y=y, dt=1):
        return lib.kda_norm_fwd(x, w, b, rows, d, xs, ys, 1e-6, kind, y, dt, None)

    assert fwd(rows=-1) == -1 and fwd(d=0) == -1 and fwd(kind=2) == -1 and fwd(dt=2) == -1 and fwd(x=None) == -1 and fwd(y=None) == -1
    assert fwd(d=16385, xs=16385, ys=16385) == -2 and fwd(xs=39) == -1 and fwd(ys=39) == -1 and fwd(rows=0, x=None, y=None) == 0
    assert fwd(x=x + 2) == -3 and fwd(w=w + 4) == -3
    assert fwd(y=x + 4 * 40) == -1 and fwd(y=x, ys=41) == -1 and fwd(y=w) == -1  # over an input, but not row for row

    def bwd(dy=dy, dx=dx, dw=w, db=b, ws=ws, wb=need, weight=None, xs=40):
        return lib.kda_norm_bwd(x, dy, weight, 6, 40, xs, 40, 40, 1e-6, 0, dx, dw, db, 1, ws, wb, None)

    assert bwd(dy=None) == -1 and bwd(dx=None) == -1 and bwd(wb=need - 1) == -4 and bwd(ws=None) == -4 and bwd(dw=w + 4) == -3
    assert bwd(dx=dy + 4) == -1 and bwd(dw=b) == -1 and bwd(dw=dx) == -1 and bwd(ws=x) == -1 and bwd(weight=w) == -1 and bwd(xs=39) == -1


def test_conv_abi_refuses_before_any_launch(lib):
    r = Room()
    x, y, tail, out, cu, w, b, dy, dx, dw, db, dt, dto = (r(4096) for _ in range(13))
    need = lib.kda_conv_bwd_workspace_size(20, 24, 4)
    ws = r(need)

    def fwd(x=x, cu=cu, w=w, tail=tail, N=3, T=20, C=24, W=4, xs=24, ts=24, ys=24, os=24, act=1, y=y, out=out, dt=1):
        return lib.kda_conv_fwd(x, cu, w, b, tail, N, T, C, W, xs, ts, ys, os, act, y, out, dt, None, None)

    assert fwd(N=0) == -1 and fwd(T=-1) == -1 and fwd(C=0) == -1 and fwd(W=0) == -1 and fwd(W=5) == -1 and fwd(act=2) == -1 and fwd(dt=3) == -1
    assert fwd(x=None) == -1 and fwd(cu=None) == -1 and fwd(w=None) == -1 and fwd(y=None) == -1 and fwd(T=2 ** 30 + 1) == -2
    assert fwd(xs=23) == -1 and fwd(ts=23) == -1 and fwd(ys=23) == -1 and fwd(os=23) == -1
    assert fwd(x=x + 2) == -3 and fwd(w=w + 4) == -3 and fwd(cu=cu + 4) == -3
    assert fwd(y=x) == -1 and fwd(out=tail) == -1 and fwd(out=y) == -1 and fwd(y=x + 4 * 23, xs=48, ys=48) == -1

    def bwd(dy=dy, dx=dx, dw=dw, db=db, dt=dt, dto=dto, ddt=1, ws=ws, wb=need, dtype=1):
        return lib.kda_conv_bwd(x, cu, w, b, tail, dy, dto, 3, 20, 24, 4, 24, 24, 24, 24, 1, dx, dw, db, dt, dtype, ddt, ws, wb, None, None)

    assert bwd(dy=None) == -1 and bwd(dx=None) == -1 and bwd(ddt=0) == -1 and bwd(wb=need - 1) == -4 and bwd(ws=None) == -4
    assert bwd(dx=dy) == -1 and bwd(dx=x) == -1 and bwd(dt=dto) == -1 and bwd(dw=db) == -1 and bwd(dw=w) == -1 and bwd(dt=dt + 4) == -3

    def step(x=x, tail=tail, y=y, R=3, C=24, W=4):
        return lib.kda_conv_step(x, w, b, tail, R, C, W, 24, 24, 24, 1, y, 1, None)

    assert step(R=0) == -1 and step(tail=None) == -1 and step(y=x) == -1 and step(tail=x) == -1 and step(W=5) == -1


def test_scan_abi_refuses_before_any_launch(lib):
    r = Room()
    T, D, G, S, N = 600, 8, 2, 16, 2
    rows, bc, st = T * D * 4, T * G * S * 4, N * D * S * 4
    x, dt, z, y, dy, dx, ddt, dz = (r(rows) for _ in range(8))
    B, C, dB, dC = (r(bc) for _ in range(4))
    A, skip, bias, cu, h0, h1, dA, dskip, dbias, dh0, dh1 = (r(st) for _ in range(11))
    saved_bytes, need, need_bwd = (lib.kda_scan_saved_size(N, T, D, S), lib.kda_scan_workspace_size(N, T, D, G, S),
                                   lib.kda_scan_bwd_workspace_size(N, T, D, G, S))
    assert saved_bytes == (T // 8 + N) * D * S * 4 and 0 < need < need_bwd
    saved = r(saved_bytes)
    ws = (ctypes.create_string_buffer(need_bwd + 64))
    w = (ctypes.addressof(ws) + 63) & ~63

    def fwd(x=x, dt=dt, A=A, B=B, C=C, z=z, cu=cu, N=N, T=T, D=D, G=G, S=S, xs=8, bs=32, h0=h0, h1=h1, y=y, saved=saved, t=1, w=w, wb=need):
        return lib.kda_scan_fwd(x, dt, A, B, C, skip, z, bias, cu, N, T, D, G, S, xs, 8, bs, 32, 8, 8, h0, h1, 1, y, saved, t, w, wb,
                                None, None)

    assert fwd(N=0) == -1 and fwd(T=-1) == -1 and fwd(G=3) == -1 and fwd(G=0) == -1 and fwd(t=2) == -1 and fwd(T=2 ** 30 + 1) == -2
    assert fwd(S=24) == -2 and fwd(S=128) == -2 and fwd(x=None) == -1 and fwd(A=None) == -1 and fwd(cu=None) == -1 and fwd(y=None) == -1
    assert fwd(xs=7) == -1 and fwd(bs=31) == -1 and fwd(x=x + 1) == -3 and fwd(A=A + 4) == -3 and fwd(h0=h0 + 8) == -3
    assert fwd(wb=need - 1) == -4 and fwd(w=None) == -4
    assert fwd(y=x) == -1 and fwd(h1=h0) == -1 and fwd(saved=h0) == -1 and fwd(h1=A) == -1 and fwd(w=x) == -1 and fwd(y=z) == -1

    def bwd(dy=dy, saved=saved, dx=dx, ddt=ddt, dA=dA, dB=dB, dC=dC, dz=dz, z=z, dh0=dh0, w=w, wb=need_bwd):
        return lib.kda_scan_bwd(x, dt, A, B, C, skip, z, bias, cu, dy, dh1, saved, N, T, D, G, S, 8, 8, 32, 32, 8, 8, 1, dx, ddt, dA, dB,
                                dC, dskip, dz, dbias, dh0, 1, w, wb, None, None)

    assert bwd(dy=None) == -1 and bwd(saved=None) == -1 and bwd(dA=None) == -1 and bwd(dB=None) == -1 and bwd(dz=None) == -1
    assert bwd(wb=need_bwd - 1) == -4 and bwd(w=None) == -4 and bwd(dx=dx + 4) == -3
    assert bwd(dx=dy) == -1 and bwd(dx=ddt) == -1 and bwd(dB=dC) == -1 and bwd(dh0=dh1) == -1 and bwd(dA=A) == -1 and bwd(dx=x) == -1

    def step(x=x, state=h0, y=y, R=3, G=G, S=S):
        return lib.kda_scan_step(x, dt, A, B, C, skip, z, bias, state, R, D, G, S, 8, 8, 32, 32, 8, 8, 1, y, 1, None)

    assert step(R=0) == -1 and step(S=4) == -2 and step(G=3) == -1 and step(state=None) == -1 and step(state=h0 + 4) == -3
    assert step(y=x) == -1 and step(state=A) == -1 and step(y=h0) == -1


def test_workspaces_and_sizes(lib):
    """Whole sequences need no workspace; few or uneven long ones do.  Nothing for shapes that are refused."""
    assert lib.kda_scan_workspace_size(8, 255, 64, 1, 16) == 0
    assert lib.kda_scan_workspace_size(1, 20000, 64, 1, 16) > 0
    assert lib.kda_scan_workspace_size(2, 1000, 64, 1, 12) == 0 and lib.kda_scan_bwd_workspace_size(2, 1000, 64, 3, 16) == 0
    assert lib.kda_conv_bwd_workspace_size(1000, 64, 5) == 0 and lib.kda_norm_bwd_workspace_size(10, 16385, 0) == 0
    # a partial row of W + 1 columns per run of 8 to 128 tokens
    n = lib.kda_conv_bwd_workspace_size(4096, 8192, 4)
    assert 4096 // 128 * 5 * 8192 * 4 <= n <= 4096 // 8 * 5 * 8192 * 4
    # a unit's sums (16-byte rows) and a partial row of B and C per tile of 128 channels (16 states) and token
    N, T, D = 600, 511, 130
    up = lambda x: (x + 255) // 256 * 256
    assert lib.kda_scan_bwd_workspace_size(N, T, D, 1, 16) == up(N * ((D * 18 + 3) // 4 * 4) * 4) + up(2 * T * 32 * 4)


# ------------------------------------------------------------------ memory that a call makes for itself
def test_workspaces_live_until_the_library_call_has_returned(monkeypatch):
    """A workspace that the binding makes is held until the launches that use it are enqueued."""
    made, alive, size = [], {}, 1 << 14

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: size

            def called(*a):
                alive[name] = [m() is not None for m in made]
                return 0
            return called

    lib, real = Lib(), torch.empty

    def empty(*shape, **kw):  # (the workspace is all that these calls make so: their outputs are the fixture's fakes)
        if kw.get("dtype") is not torch.uint8:
            return real(*shape, **kw)
        t = Fake(t=real(*shape, dtype=torch.uint8))
        made.append(weakref.ref(t))
        return t

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(kda, "load_library", lambda: lib)
    x, dy, saved = Fake(7, 12, dtype=BF), Fake(7, 12, dtype=BF), Fake(size // 4)
    scan = _scan()
    calls = {"kda_norm_bwd": lambda: kda.norm_bwd(x, dy), "kda_conv_bwd": lambda: kda.conv_bwd(**_conv(dy=dy)),
             "kda_scan_fwd": lambda: kda.scan_fwd(**scan), "kda_scan_bwd": lambda: kda.scan_bwd(**scan, dy=scan["x"], saved=saved)}
    for name, call in calls.items():
        del made[:]
        call()
        assert alive[name] == [True], name
        assert [r() for r in made] == [None], name  # and no longer than the call


def test_sizes_past_31_bits_are_refused():
    """The C ABI's sizes are 32-bit integers: larger ones are refused, not cut off."""
    far = lambda *s, dtype=F32: Fake(t=torch.empty(s, dtype=dtype, device="meta"))
    n = 2 ** 32 + 8
    cu, w = Fake(3, dtype=I32), Fake(1, 4)
    calls = [lambda: kda.norm_fwd(far(1, n)), lambda: kda.norm_bwd(far(1, n), far(1, n)),
             lambda: kda.conv_fwd(far(n, 1), w, cu), lambda: kda.conv_fwd(Fake(8, 1), w, far(n, dtype=I32)),
             lambda: kda.conv_bwd(far(n, 1), w, cu, far(n, 1)), lambda: kda.conv_fwd(far(2, n), far(n, 1), cu),
             lambda: kda.conv_fwd(Fake(2, 1), far(1, n), cu), lambda: kda.conv_step(far(n, 1), w, far(n, 3, 1))]
    for rows, D, S, G in ((n, 1, 8, 1), (2, n, 8, 1), (2, 1, n, 1), (2, 1, 8, n)):
        x, A, B = far(rows, D), far(D, S), far(rows, G, S)
        calls += [lambda a=(x, x, A, B, B): kda.scan_fwd(*a, cu), lambda a=(x, x, A, B, B): kda.scan_bwd(*a, cu, a[0], Fake(9)),
                  lambda a=(x, x, A, B, B), s=far(rows, D, S): kda.scan_step(*a, s)]
    x, A, B = Fake(2, 1), Fake(1, 8), Fake(2, 1, 8)
    calls += [lambda: kda.scan_fwd(x, x, A, B, B, far(n, dtype=I32))]
    for i, call in enumerate(calls):
        with pytest.raises(kda.KDAError, match="below 2\\^31"):
            call()
            pytest.fail(str(i))
