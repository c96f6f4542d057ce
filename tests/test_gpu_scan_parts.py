"""The scan's variants and cuts on the GPU, held to what fp32 itself costs (scan_ref's norms, part by part): sequences cut
into segments both ways, 8 and 16 states to a thread, and the bias of the hardware's 2^x."""
import numpy as np
import pytest
import torch

import kda_gated_delta_02_gb300 as kda
import scan_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate")
BARE = dict.fromkeys(("D", "z", "dt_bias", "h0", "dfinal"))


def _cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def _forward(s, cu, **kw):
    return kda.scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], cu, D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                        initial_state=s["h0"], **kw)


def _both(s, lens):
    """{output: value} of both calls."""
    cu = _cu(lens)
    y, fin, saved = _forward(s, cu, save=True)
    plain = _forward(s, cu)
    assert torch.equal(plain[0], y) and torch.equal(plain[1], fin)
    grads = kda.scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], cu, s["dy"], saved, D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                         initial_state=s["h0"], dfinal_state=s["dfinal"])
    return dict(zip(("y", "final_state", *GRADS), (y, fin, *grads)))


def _check(got, want, lens):
    for name, g in got.items():
        if g is not None:
            ref.check(name, g, want[name], lens)


def _is_cut(lens, D, G, S):
    """Whether the forward and the backward cut sequences: segments' states take workspace beside that of whole ones."""
    lib, N, T = kda.load_library(), len(lens), sum(lens)
    up = lambda n: (n + 255) // 256 * 256
    tile = 2048 // S  # channels of a block of the backward
    whole = up(N * ((D * S + 2 * D + 3) // 4 * 4) * 4) + up((D // G + tile - 1) // tile * T * G * 2 * S * 4)
    return lib.kda_scan_workspace_size(N, T, D, G, S) > 0, lib.kda_scan_bwd_workspace_size(N, T, D, G, S) > whole


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("S,D,G", [(8, 33, 1), (16, 48, 1), (32, 16, 1), (64, 40, 2)])
def test_cut_sequences(S, D, G, dtype):
    lens = [700, 0, 5, 400, 130]
    assert _is_cut(lens, D, G, S) == (True, True)
    s = ref.inputs(lens, D, G, S, DTYPES[dtype])
    _check(_both(s, lens), ref.scan(s, lens), lens)
    bare = {**s, **BARE}
    _check(_both(bare, lens), ref.scan(bare, lens), lens)


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_long_sequence(dtype):
    lens = [9000]
    assert _is_cut(lens, 24, 3, 16) == (True, True)
    s = ref.inputs(lens, 24, 3, 16, DTYPES[dtype])
    _check(_both(s, lens), ref.scan(s, lens), lens)


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_of_many_sequences_is_cut(dtype):
    """Channels for all SMs, so that the walk keeps 16 states a thread, and one sequence past four times the mean."""
    D, S, lens = 4096, 16, [3, 1, 0, 40] * 8 + [4100] + [2] * 31
    assert _is_cut(lens, D, 1, S) == (True, True)
    s = ref.inputs(lens, D, 1, S, DTYPES[dtype])
    got, pick = _both(s, lens), torch.tensor([0, 77, 1000, 4095], device="cuda")
    want = ref.scan(ref.channels(s, pick), lens)
    for name in ("y", "final_state", "dx", "ddt", "dz", "dstate"):
        ref.check(name, got[name][:, pick], want[name], lens)
    for name in ("dA", "dD", "ddt_bias"):
        ref.check(name, got[name][pick], want[name], lens)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("S,D,G", [(16, 2056, 1), (16, 2064, 2), (32, 1040, 2), (64, 528, 2), (64, 520, 1)])
def test_sixteen_states_a_thread(S, D, G, dtype):
    """Blocks enough for the walk of 16 states a thread: a channel in one thread, in two and in four lanes, in groups whose
    last tile is not full."""
    lens = [1 + (5 * i) % 13 if i % 7 else 0 for i in range(40)]
    tiles = (D // G + 2048 // S - 1) // (2048 // S)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert _is_cut(lens, D, G, S)[0] is False and len(lens) * G * tiles >= 4 * sms
    s = ref.inputs(lens, D, G, S, DTYPES[dtype])
    _check(_both(s, lens), ref.scan(s, lens), lens)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("S,D,G", [(8, 130, 1), (16, 72, 3), (32, 129, 3), (64, 48, 2)])
def test_whole_sequences(S, D, G, dtype):
    lens = [20, 0, 1, 17, 8, 40]
    assert _is_cut(lens, D, G, S) == (False, False)
    s = ref.inputs(lens, D, G, S, DTYPES[dtype])
    _check(_both(s, lens), ref.scan(s, lens), lens)


def test_gradients_of_cut_sequences_against_differences():
    """f = sum(y g) + sum(final h) along v, of the gradient's own signs, so that (f(p + e v) - f(p - e v)) / 2e is the sum of
    |gradient| |v|: e^2 of the third derivative and 2^-24 / e of each output, as for whole sequences."""
    lens, D, G, S = [700, 0, 5, 400, 130], 20, 2, 16
    assert _is_cut(lens, D, G, S) == (True, True)
    s = ref.inputs(lens, D, G, S, torch.float32)
    cu, got = _cu(lens), _both(s, lens)

    def f(p):
        y, fin = _forward(p, cu)
        return float((y.double() * s["dy"].double()).sum() + (fin.double() * s["dfinal"].double()).sum())

    gen, e = torch.Generator(device="cuda"), 2.0 ** -8
    gen.manual_seed(6)
    for name, grad in zip(("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0"), GRADS):
        v = torch.randn(s[name].shape, generator=gen, device="cuda").abs() * got[grad].sign()
        diff = (f({**s, name: s[name] + e * v}) - f({**s, name: s[name] - e * v})) / (2 * e)
        want = float((got[grad].double() * v.double()).sum())
        assert abs(diff - want) < (32 * e * e + 256 * 2.0 ** -24 / e) * want, (name, diff, want)


@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("lens", [[1], [2], [3, 8], [40, 1, 5], [300, 0, 200]])
def test_rates_of_states_that_forget(lens, S):
    """Decays down to e^-19 a token: what is left of a state beside what is added keeps its relative precision in dA, element
    by element.  All terms are positive, so that every one is within its own roundings: 8.5 for each unit of an exponent up to
    19.5, 60 each for the state and what comes back, 40 for products and sums, in all below 512."""
    D, G = 34, 2
    s, r = ref.inputs(lens, D, G, S, torch.float32), lambda *n: 0.5 + torch.rand(n, device="cuda")
    torch.manual_seed(S)
    s = {k: r(*v.shape) for k, v in s.items()}
    s.update(D=None, z=None, dt_bias=None, dt=1.5 * s["dt"] - 1.75, A=-torch.linspace(0.5, 20, S, device="cuda").repeat(D, 1))
    got, want = _both(s, lens), ref.scan(s, lens)
    off = np.abs(got["dA"].double().cpu().numpy() - want["dA"]) / want["dA"]
    assert off.max() <= 512 * 2.0 ** -24, off.max() * 2 ** 24
    for name in ("dB", "dC", "dx", "ddt"):
        ref.check(name, got[name], want[name], lens)


# ------------------------------------------------------------------ the hardware's 2^x
def _decays(tokens, back):
    """A state of 1 that only decays, by 2^-7 to 2^-3 powers of two a token or so: the mean over the states of what a token's
    factor is off by, in 2^-24."""
    D, S = 4096, 16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    r = lambda *s: torch.rand(s, generator=gen, device="cuda")
    A = -torch.exp2(-3 - 4 * r(D, S))
    dt = (0.5 + 0.5 * r(1, D)).expand(tokens, D).contiguous()
    zero, bc, one = torch.zeros(tokens, D, device="cuda"), torch.zeros(tokens, 1, S, device="cuda"), torch.ones(1, D, S, device="cuda")
    if back == "step":
        end = one.clone()
        for t in range(tokens):
            kda.scan_step(zero[:1], dt[:1], A, bc[:1], bc[:1], end, dt_softplus=False)
    else:
        args = (zero, dt, A, bc, bc, _cu([tokens]))
        _, end, saved = kda.scan_fwd(*args, initial_state=one, dt_softplus=False, save=True)
        if back == "back":
            end = kda.scan_bwd(*args, zero, saved, initial_state=one, dfinal_state=one, dt_softplus=False)[8]
    want = np.exp(tokens * dt[0].double().cpu().numpy()[:, None] * A.double().cpu().numpy())
    return float((end[0].double().cpu().numpy() / want - 1).mean() / tokens * 2 ** 24)


@pytest.mark.parametrize("back,tokens", [("walk", 255), ("back", 95), ("step", 200)])
def test_decays_are_not_low_on_average(back, tokens):
    """ex2.approx is low by 0.28 to 0.44 of 2^-24 for arguments of 2^-7 to 2^-3 (measured, octave by octave), 0.37 on
    average; the addend of a quarter leaves 0.12.  Roundings of the state are as often up as down, and the mean over 65,536
    states is good to 0.01: what is left is below the quarter, which it would not be without the addend."""
    assert abs(_decays(tokens, back)) < 0.25
